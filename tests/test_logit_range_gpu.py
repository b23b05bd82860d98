"""pda_decode where every logit of a row is far below zero: the maximum is found all the same."""
import pytest
import torch

import shared_ref as S
from test_int8_query_rows_gpu import decode
from test_shared_gpu import check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("kind,dim", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("int8_tensor", 128),
                                      ("e4m3_tensor", 128)])
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** 100, 2.0 ** 115])
def test_rows_of_logits_below_zero(kind, dim, size):
    w = S.make([(0, [(300, 2), (9, 1)])], kind=kind, dim=dim, dev=DEV, seed=dim)
    w.q = (w.q.float().abs() * -size).to(torch.bfloat16)
    k = w.cache[0]
    if k.dtype is torch.uint8:
        k.bitwise_and_(0x7f)  # E4M3 codes without their sign
    else:
        k.abs_()
    w.values[0] = w.values[0].abs()
    out, lse = decode(w, w.dim ** -0.5)
    o, ob, l, lb = S.attention(w)
    assert float(l.max()) < -0.01 * size
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")
