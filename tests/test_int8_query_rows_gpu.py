"""int8 caches meet an f16 query: rows of ordinary size keep their bits beside rows and heads
of any other size."""
import pytest
import torch

import shared_ref as S
from paged_split_kv_03_gb300 import binding as B
from test_shared_gpu import check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def decode(w, scale):
    dec = B.Decoder(w.params, device=DEV)
    t = S.device_tables(w)
    out = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(w.q.shape[:2], device=DEV)
    B.pda_decode(dec.plan, w.q, *w.cache, t.page_table, t.kv_indptr, t.kv_len, t.qo_indptr, max(w.rows),
                 None, scale, *w.scale, out, lse, dec.scratch)
    assert dec.status() == 0
    return out, lse


@pytest.mark.parametrize("size", [2.0 ** 11, 2.0 ** 13, 2.0 ** 15, 2.0 ** 17, 2.0 ** 100, 2.0 ** -9, 2.0 ** -100])
@pytest.mark.parametrize("kind,dim,hkv,group,rows", [
    ("int8_tensor", 128, 2, 4, 1), ("int8_token", 128, 2, 8, 8), ("int8_tensor", 256, 1, 8, 3),
    ("int8_token", 256, 2, 16, 2), ("int8_tensor", 128, 1, 5, 7), ("int8_tensor", 64, 2, 4, 2)])
def test_one_row_or_head_of_another_size(kind, dim, hkv, group, rows, size):
    """With the bounds of each row's own elements: bf16 elements from 2^-14 on are exact in f16,
    those below it off by 2^-25, and a row that leaves the type's range loses 2^-25 of its
    largest element; the sums of D products are fp32."""
    reqs = [(300, rows), (max(9, rows), rows), (77, 1)]
    w = S.make([(0, reqs)], kind=kind, dim=dim, hkv=hkv, group=group, dev=DEV, seed=dim)
    q = w.q.float()
    q[0, 0] *= size                     # one head of a row
    q[rows:2 * rows, hkv * group - 1] *= size   # one head of a request
    q[-1] *= size                       # a whole row
    w.q = q.to(torch.bfloat16)
    out, lse = decode(w, w.dim ** -0.5)
    o, ob, l, lb = S.attention(w)
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")
