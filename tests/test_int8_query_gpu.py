"""int8 caches meet an f16 query: bf16 queries beyond f16's range keep their power of two."""
import pytest
import torch

from gpu_helpers import oracle_ref, run_decode
from paged_split_kv_03_gb300.synth import SCALE_TENSOR, SCALE_TOKEN_HEAD, make_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** 15, 1.0, 2.0 ** -9, 2.0 ** -100])
@pytest.mark.parametrize("mode,dim,rows", [(SCALE_TENSOR, 128, 1), (SCALE_TOKEN_HEAD, 256, 5),
                                           (SCALE_TOKEN_HEAD, 128, 8), (SCALE_TENSOR, 64, 2)])
def test_queries_of_any_size(mode, dim, rows, size):
    wl = make_workload(name="int8q", batch=3, rows=[rows] * 3, kv_lens=[300, 9, 77], num_qo_heads=8,
                       num_kv_heads=2, head_dim=dim, page_size=16, kv_dtype="int8", scale_mode=mode,
                       seed=2, device=torch.device("cuda", 0))
    wl.q = (wl.q.float() * size).to(torch.bfloat16)
    wl.sm_scale = dim ** -0.5 / size
    out, lse, status, _ = run_decode(wl)
    ref_o, ref_l = oracle_ref(wl)
    assert status == 0
    # weights rounded to f16 or bf16 (2^-8) and the output to bf16, of values below 5
    assert abs(out.numpy() - ref_o).max() <= 5 * 2 * 2.0 ** -8
    assert abs(lse.numpy() - ref_l).max() <= 1e-3
