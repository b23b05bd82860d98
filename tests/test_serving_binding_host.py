"""What the binding refuses before the library sees a pointer: tensors of another
device, caches and scales of another type or too small for the plan, scratches that
are too small. On the CPU: the tensors only say that they are on a CUDA device, and
every call here is refused."""
import ctypes

import pytest
import torch

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B
from paged_split_kv_03_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load_library()


class On:
    """A CPU tensor that says it is on CUDA device ``dev``."""

    def __init__(self, t, dev=0):
        self.t, self.dev = t, dev

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


def refused(code, call, *args):
    """The call raises PdaError of that code, or ValueError where code is None."""
    with pytest.raises(ValueError if code is None else B.PdaError) as e:
        call(*args)
    if code is not None:
        assert e.value.code == code, e.value


HEADS, PAGE, PAGES, ROWS = 2, 16, 4, 3


def expand_args(kind):
    plan = B.pda_plan(ref.mla_plan(HEADS, kind=kind, page=PAGE, pages=PAGES, num_sms=152))[0]
    width = 640 if kind == "records" else 576
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    shape = dict(e4m3=(1,), e4m3_token=(PAGES, PAGE, 1), records=(PAGES, PAGE, 1, 4)).get(kind)
    w = torch.zeros(HEADS, 128, 512, dtype=torch.bfloat16)
    kv = torch.zeros(ROWS, HEADS, 128, dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    return plan, dict(k_pages=torch.zeros(PAGES, PAGE, 1, width, dtype=dt), page_table=torch.zeros(
        4, dtype=torch.int32), kv_indptr=ints, tok_indptr=ints, k_scale=None if shape is None else
        torch.zeros(shape), w_uk=w, w_uv=w, latent=torch.zeros(ROWS, 576, dtype=torch.bfloat16), k=kv,
        v=kv, split_scratch=torch.zeros(256, dtype=torch.uint8))


def expand(code, kind, **change):
    plan, a = expand_args(kind)
    a = {k: v if v is None or isinstance(v, On) else On(v) for k, v in {**a, **change}.items()}
    refused(code, B.pda_mla_expand, plan, *a.values())


def test_caches_of_other_types_and_sizes():
    small = (PAGES - 1, PAGE, 1)
    expand(None, "bf16", k_pages=torch.zeros(*small, 576, dtype=torch.bfloat16))
    expand(None, "bf16", k_pages=torch.zeros(PAGES, PAGE, 1, 576, dtype=torch.uint8))
    expand(None, "bf16", k_pages=torch.zeros(PAGES, PAGE, 1, 576, dtype=torch.float16))
    expand(None, "bf16", k_pages=torch.zeros(PAGES, PAGE, 1, 576, dtype=torch.float32))
    for kind in ("e4m3", "records"):
        expand(None, kind, k_pages=torch.zeros(PAGES, PAGE, 1, 640, dtype=torch.bfloat16))
        expand(None, kind, k_pages=torch.zeros(*small, 640, dtype=torch.uint8))
    expand(None, "records", k_pages=torch.zeros(PAGES, PAGE, 1, 576, dtype=torch.uint8))
    # a view that starts too late in its memory
    expand(None, "bf16", k_pages=torch.zeros(PAGES, PAGE, 1, 576, dtype=torch.bfloat16)[1:])


def test_scales_of_other_types_and_sizes():
    for kind, few in (("e4m3", (0,)), ("e4m3_token", (PAGES - 1, PAGE, 1)),
                      ("records", (PAGES, PAGE, 1))):
        expand(None, kind, k_scale=torch.zeros(few))
        expand(None, kind, k_scale=torch.zeros(PAGES, PAGE, 1, 4, dtype=torch.float16))
    expand(None, "records", k_scale=torch.zeros(PAGES, PAGE, 1, 8)[..., ::2])


@pytest.mark.parametrize("name", ["k_pages", "page_table", "kv_indptr", "tok_indptr", "k_scale", "w_uk",
                                  "w_uv", "latent", "k", "v", "split_scratch"])
def test_expand_takes_tensors_of_the_plans_device_alone(name):
    _, a = expand_args("records")
    expand(B.PDA_ERR_INVALID, "records", **{name: On(a[name], dev=1)})
    expand(None, "records", **{name: On(a[name], dev=-1)})


def test_append_checks_both_caches():
    p = B.PdaParams(num_qo_heads=2, num_kv_heads=2, head_dim=128, page_size=PAGE, max_batch=1,
                    max_q_len=1, max_kv_len=64, num_pages=PAGES, kv_stride_page=PAGE * 256,
                    kv_stride_token=256, kv_stride_head=128, num_sms=152, kv_dtype=B.PDA_INT8,
                    scale_mode=B.PDA_SCALE_TOKEN_HEAD)
    plan = B.pda_plan(p)[0]
    new = torch.zeros(ROWS, 2, 128, dtype=torch.bfloat16)
    good = dict(k_new=new, v_new=new, slot_map=torch.zeros(ROWS, dtype=torch.int64), num_rows=None,
                k_pages=torch.zeros(PAGES, PAGE, 2, 128, dtype=torch.int8),
                v_pages=torch.zeros(PAGES, PAGE, 2, 128, dtype=torch.uint8),
                k_scale=torch.zeros(PAGES, PAGE, 2), v_scale=torch.zeros(PAGES, PAGE, 2),
                split_scratch=torch.zeros(256, dtype=torch.uint8))
    short, half = torch.zeros(PAGES, PAGE, 127, 2), torch.zeros(PAGES, PAGE)
    for change, code in ((dict(v_pages=good["v_pages"][1:]), None), (dict(k_pages=good["k_pages"][1:]), None),
                         (dict(v_pages=short.to(torch.bfloat16)), None), (dict(v_scale=half), None),
                         (dict(k_pages=good["k_pages"].view(torch.float8_e4m3fn)), None),
                         (dict(v_scale=On(good["v_scale"], dev=2)), B.PDA_ERR_INVALID),
                         (dict(slot_map=On(good["slot_map"], dev=1)), B.PDA_ERR_INVALID),
                         (dict(num_rows=On(torch.zeros(1, dtype=torch.int32), dev=1)), B.PDA_ERR_INVALID)):
        a = {k: v if v is None or isinstance(v, On) else On(v) for k, v in {**good, **change}.items()}
        refused(code, B.pda_append_slots, plan, *a.values())


def test_prefill_scratch_has_to_hold_the_plans_partials():
    plan = B.pda_plan(ref.mla_plan(HEADS, num_sms=152))[0]
    pre, nbytes, _ = B.pda_prefill_plan(plan, ROWS, 2000)
    assert pre.splits > 1 and nbytes > 256
    kv = On(torch.zeros(2000, HEADS, 128, dtype=torch.bfloat16))
    ptr = On(torch.zeros(2, dtype=torch.int32))
    args = (On(torch.zeros(ROWS, HEADS, 192, dtype=torch.bfloat16)), kv, kv,
            On(torch.zeros(2000, 64, dtype=torch.bfloat16)), ptr, ptr, None, True, 0.1,
            On(torch.zeros(ROWS, HEADS, 128, dtype=torch.bfloat16)), None)
    scratch = torch.zeros(nbytes, dtype=torch.uint8)
    refused(B.PDA_ERR_SCRATCH, B.pda_mla_prefill, pre, *args, On(scratch[256:]))
    refused(B.PDA_ERR_SCRATCH, B.pda_mla_prefill, pre, *args, On(scratch.new_zeros(256)))
    refused(B.PDA_ERR_INVALID, B.pda_mla_prefill, pre, *args, On(scratch, dev=1))


def test_rows_of_the_latent_calls_end_where_the_header_says(lib):
    """8388480 rows pass the checks up to the missing output, one more is refused first."""
    plan, okp = B.pda_plan(ref.mla_plan(HEADS, num_sms=152))[0], 0x10000
    for rows, code in ((8388480, B.PDA_ERR_NULL), (8388481, B.PDA_ERR_INVALID)):
        assert lib.pda_mla_project(ctypes.byref(plan), okp, okp, 131072, None, rows, None, okp,
                                   None) == code
        assert lib.pda_mla_absorb(ctypes.byref(plan), okp, 384, 192, okp, 131072, 1.0, None, rows, None,
                                  okp, None) == code
        assert lib.pda_mla_expand(ctypes.byref(plan), okp, okp, okp, okp, None, okp, okp, 131072, okp, okp,
                                  None, 512, 256, rows, okp, None) == code
