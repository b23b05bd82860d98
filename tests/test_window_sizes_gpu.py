"""Sliding windows up to the largest int32: one that reaches past a request's tokens hides
nothing, bit for bit."""
import pytest
import torch

from paged_split_kv_03_gb300 import binding as B
from paged_split_kv_03_gb300.synth import SCALE_TENSOR, make_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_dtype,dim", [("bf16", 128), ("e4m3", 256), ("bf16", 64)])
def test_window_past_the_context(kv_dtype, dim):
    kw = {} if kv_dtype == "bf16" else dict(scale_mode=SCALE_TENSOR)
    wl = make_workload(name="window", batch=4, rows=[1, 3, 2, 4], kv_lens=[700, 300, 65, 1500],
                       num_qo_heads=8, num_kv_heads=2, head_dim=dim, page_size=16, kv_dtype=kv_dtype,
                       windows=[9, 9, 9, 9], seed=1, device=torch.device("cuda", 0), **kw)
    dec = B.Decoder(B.params_for(wl), device="cuda")
    got = []
    for w in ([0] * 4, [2 ** 31 - 1, 2 ** 31 - 2, 66, 2 ** 31 - 1500], [701, 2 ** 30, 2 ** 31 - 1, 1501]):
        wl.window.copy_(torch.tensor(w, dtype=torch.int32))
        out = torch.zeros(wl.total_rows, 8, dim, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(wl.total_rows, 8, device="cuda")
        dec.run(wl, out, lse)
        got.append((out, lse))
    assert dec.status() == 0 and bool(torch.isfinite(got[0][1]).all())
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
