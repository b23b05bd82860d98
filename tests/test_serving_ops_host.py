"""Refusals of the calls around decode on the CPU: every host check returns its
code before anything is launched (pointers here are numbers, never read)."""
import ctypes

import pytest

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B
from paged_split_kv_03_gb300 import build as build_mod

OKP, ODD = 0x10000, 0x10002


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def plan_of(**kw):
    return B.pda_plan(ref.mla_plan(16, num_sms=152, **kw))[0]


def gqa_plan(head_dim=128, **kw):
    p = B.PdaParams(num_qo_heads=4, num_kv_heads=2, head_dim=head_dim, page_size=16, max_batch=3,
                    max_q_len=1, max_kv_len=100, num_pages=8, kv_stride_page=16 * 2 * head_dim,
                    kv_stride_token=2 * head_dim, kv_stride_head=head_dim, num_sms=152)
    for k, v in kw.items():
        setattr(p, k, v)
    return B.pda_plan(p)[0]


def bad_plan():
    p = plan_of()
    p.magic = 1
    return p


TABLES = dict(cached_len=OKP, new_len=OKP + 64, request=None, block_table=OKP + 128, table_stride=8,
              free_pages=OKP, free_count=OKP, free_left=OKP + 4, kv_len=OKP + 256, kv_indptr=OKP,
              page_table=OKP, qo_indptr=OKP, tok_indptr=OKP, slot_map=OKP, positions=OKP,
              table_rows=3, table_cols=8, page_table_cap=24, rows_cap=24)


@pytest.mark.parametrize("change,code", [
    (dict(cached_len=None), B.PDA_ERR_NULL), (dict(new_len=None), B.PDA_ERR_NULL),
    (dict(block_table=None), B.PDA_ERR_NULL), (dict(free_left=None), B.PDA_ERR_NULL),
    (dict(kv_len=None), B.PDA_ERR_NULL), (dict(page_table=None), B.PDA_ERR_NULL),
    (dict(qo_indptr=None), B.PDA_ERR_NULL), (dict(free_pages=None), B.PDA_ERR_NULL),
    (dict(table_rows=2), B.PDA_ERR_INVALID), (dict(table_rows=0), B.PDA_ERR_INVALID),
    (dict(table_stride=7), B.PDA_ERR_INVALID), (dict(table_cols=-1), B.PDA_ERR_INVALID),
    (dict(page_table_cap=-1), B.PDA_ERR_INVALID), (dict(rows_cap=-1), B.PDA_ERR_INVALID),
    (dict(free_left=OKP), B.PDA_ERR_INVALID), (dict(kv_len=OKP), B.PDA_ERR_INVALID),
    (dict(kv_len=OKP + 64), B.PDA_ERR_INVALID),
    (dict(positions=ODD), B.PDA_ERR_ALIGNMENT), (dict(slot_map=OKP + 4), B.PDA_ERR_ALIGNMENT),
    (dict(tok_indptr=ODD), B.PDA_ERR_ALIGNMENT)])
def test_tables_refusals(lib, change, code):
    t = B.PdaTables(**{**TABLES, **change})
    plan = gqa_plan()
    assert lib.pda_build_tables(ctypes.byref(plan), ctypes.byref(t), OKP, None) == code


def test_tables_refusals_of_plan_and_scratch(lib):
    t, plan = B.PdaTables(**TABLES), gqa_plan()
    call = lib.pda_build_tables
    assert call(None, ctypes.byref(t), OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(plan), None, OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(plan), ctypes.byref(t), None, None) == B.PDA_ERR_SCRATCH
    assert call(ctypes.byref(plan), ctypes.byref(t), OKP + 128, None) == B.PDA_ERR_SCRATCH
    assert call(ctypes.byref(bad_plan()), ctypes.byref(t), OKP, None) == B.PDA_ERR_PLAN
    big = gqa_plan(max_batch=65537)
    t.table_rows = 70000
    assert call(ctypes.byref(big), ctypes.byref(t), OKP, None) == B.PDA_ERR_INVALID


APPEND = dict(k=OKP, ks=256, v=OKP, vs=256, slots=OKP, rows=5, num=OKP, kp=OKP, vp=OKP, ksc=None,
              vsc=None, scratch=OKP)


def append(lib, plan, **kw):
    a = {**APPEND, **kw}
    return lib.pda_append_slots(ctypes.byref(plan), a["k"], a["ks"], a["v"], a["vs"], a["slots"],
                                a["rows"], a["num"], a["kp"], a["vp"], a["ksc"], a["vsc"],
                                a["scratch"], None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), B.PDA_ERR_INVALID), (dict(k=None), B.PDA_ERR_NULL), (dict(v=None), B.PDA_ERR_NULL),
    (dict(slots=None), B.PDA_ERR_NULL), (dict(kp=None), B.PDA_ERR_NULL), (dict(vp=None), B.PDA_ERR_NULL),
    (dict(scratch=None), B.PDA_ERR_SCRATCH), (dict(scratch=OKP + 8), B.PDA_ERR_SCRATCH),
    (dict(ks=255), B.PDA_ERR_INVALID), (dict(vs=248), B.PDA_ERR_INVALID),
    (dict(ks=260), B.PDA_ERR_ALIGNMENT), (dict(vs=257), B.PDA_ERR_ALIGNMENT),
    (dict(k=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(vp=OKP + 8), B.PDA_ERR_ALIGNMENT),
    (dict(slots=OKP + 4), B.PDA_ERR_ALIGNMENT), (dict(num=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(rows=0, k=None, slots=None), B.PDA_OK)])
def test_append_refusals(lib, change, code):
    assert append(lib, gqa_plan(), **change) == code


def test_append_refusals_of_scales_and_latents(lib):
    e4 = gqa_plan(kv_dtype=B.PDA_E4M3, scale_mode=B.PDA_SCALE_TOKEN_HEAD)
    assert append(lib, e4) == B.PDA_ERR_NULL
    assert append(lib, e4, ksc=OKP) == B.PDA_ERR_NULL
    assert append(lib, e4, ksc=OKP, vsc=ODD) == B.PDA_ERR_ALIGNMENT
    rec = plan_of(kind="records")
    lat = dict(v=None, vp=None, vs=0)
    assert append(lib, rec, ks=576, **lat) == B.PDA_ERR_NULL
    assert append(lib, rec, ks=576, ksc=OKP + 4, **lat) == B.PDA_ERR_ALIGNMENT
    assert append(lib, rec, ks=568, ksc=OKP, **lat) == B.PDA_ERR_INVALID
    assert append(lib, bad_plan(), ks=576, **lat) == B.PDA_ERR_PLAN


def absorb(lib, plan, **kw):
    a = {**dict(q=OKP, sr=16 * 192, sh=192, w=OKP, wh=131072, qs=1.0, out=OKP, rows=3, num=None,
                scratch=OKP), **kw}
    return lib.pda_mla_absorb(ctypes.byref(plan), a["q"], a["sr"], a["sh"], a["w"], a["wh"], a["qs"],
                              a["out"], a["rows"], a["num"], a["scratch"], None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), B.PDA_ERR_NULL), (dict(w=None), B.PDA_ERR_NULL), (dict(out=None), B.PDA_ERR_NULL),
    (dict(rows=-1), B.PDA_ERR_INVALID), (dict(wh=65528), B.PDA_ERR_INVALID),
    (dict(wh=65540), B.PDA_ERR_ALIGNMENT), (dict(sh=184), B.PDA_ERR_INVALID),
    (dict(sr=16 * 192 + 4), B.PDA_ERR_ALIGNMENT), (dict(sh=196), B.PDA_ERR_ALIGNMENT),
    (dict(q=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(w=OKP + 8), B.PDA_ERR_ALIGNMENT),
    (dict(out=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(num=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(scratch=None), B.PDA_ERR_SCRATCH), (dict(rows=0, q=None, out=None), B.PDA_OK)])
def test_absorb_refusals(lib, change, code):
    assert absorb(lib, plan_of(), **change) == code


def test_mla_refusals_of_plans(lib):
    e4 = plan_of(kind="e4m3")
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert absorb(lib, e4, qs=s) == B.PDA_ERR_INVALID
    assert absorb(lib, bad_plan()) == B.PDA_ERR_PLAN
    assert absorb(lib, gqa_plan()) == B.PDA_ERR_UNSUPPORTED
    two = ref.mla_plan(16, num_sms=152)
    two.num_kv_heads, two.kv_stride_token, two.kv_stride_page = 2, 1152, 64 * 1152
    assert absorb(lib, B.pda_plan(two)[0]) == B.PDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,code", [
    (dict(o=None), B.PDA_ERR_NULL), (dict(w=None), B.PDA_ERR_NULL), (dict(out=None), B.PDA_ERR_NULL),
    (dict(rows=-1), B.PDA_ERR_INVALID), (dict(wh=100), B.PDA_ERR_INVALID),
    (dict(o=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(scratch=OKP + 16), B.PDA_ERR_SCRATCH),
    (dict(rows=0, o=None), B.PDA_OK)])
def test_project_refusals(lib, change, code):
    a = {**dict(o=OKP, w=OKP, wh=131072, out=OKP, rows=3, num=None, scratch=OKP), **change}
    plan = plan_of()
    assert lib.pda_mla_project(ctypes.byref(plan), a["o"], a["w"], a["wh"], a["out"], a["rows"],
                               a["num"], a["scratch"], None) == code


@pytest.mark.parametrize("change,code", [
    (dict(pages=None), B.PDA_ERR_NULL), (dict(table=None), B.PDA_ERR_NULL),
    (dict(tok=None), B.PDA_ERR_NULL), (dict(wuv=None), B.PDA_ERR_NULL), (dict(lat=None), B.PDA_ERR_NULL),
    (dict(v=None), B.PDA_ERR_NULL), (dict(scale=None), B.PDA_ERR_NULL),
    (dict(scale=OKP + 4), B.PDA_ERR_ALIGNMENT), (dict(pages=OKP + 8), B.PDA_ERR_ALIGNMENT),
    (dict(tok=ODD), B.PDA_ERR_ALIGNMENT), (dict(st=16 * 256 + 2), B.PDA_ERR_ALIGNMENT),
    (dict(sh=120), B.PDA_ERR_INVALID), (dict(tokens=-1), B.PDA_ERR_INVALID),
    (dict(scratch=None), B.PDA_ERR_SCRATCH), (dict(tokens=0, lat=None), B.PDA_OK)])
def test_expand_refusals(lib, change, code):
    a = {**dict(pages=OKP, table=OKP, ptr=OKP, tok=OKP, scale=OKP, wuk=OKP, wuv=OKP, wh=131072,
                lat=OKP, k=OKP, v=OKP, st=16 * 256, sh=256, tokens=9, scratch=OKP), **change}
    plan = plan_of(kind="records")
    assert lib.pda_mla_expand(ctypes.byref(plan), a["pages"], a["table"], a["ptr"], a["tok"],
                              a["scale"], a["wuk"], a["wuv"], a["wh"], a["lat"], a["k"], a["v"],
                              a["st"], a["sh"], a["tokens"], a["scratch"], None) == code


def test_prefill_plan_chunks(lib):
    """Few (head, tile) items: the keys are cut into chunks of whole tiles, at least two of
    them, that fill the SMs about once; many items are not cut."""
    pre, nbytes, _ = B.pda_prefill_plan(plan_of(max_kv=8192), 64, 8192)
    assert pre.tiles == 1 and pre.splits == 8 and pre.chunk_tokens == 1024  # 16 heads, 152 SMs: 9 -> 8
    cells = pre.splits * 64 * 16
    assert nbytes == 256 + cells * 4 + cells * 512
    pre, nbytes, _ = B.pda_prefill_plan(plan_of(max_kv=8192), 4096, 8192)
    assert pre.tiles == 16 and pre.splits == 1 and nbytes == 256
    pre, _, _ = B.pda_prefill_plan(plan_of(max_kv=380), 1, 600)
    assert pre.splits == 1 and pre.chunk_tokens == 384
    pre, _, _ = B.pda_prefill_plan(plan_of(max_kv=1100, batch=3), 3, 3300)
    assert pre.tiles == 3 and pre.splits == 3 and pre.chunk_tokens == 384


def test_prefill_plan(lib):
    pre, nbytes, rc = B.pda_prefill_plan(plan_of(batch=4), 100, 900)
    assert rc == 0 and pre.magic == B.PDA_PREFILL_MAGIC
    assert pre.struct_bytes == ctypes.sizeof(B.PdaPrefillPlan)
    assert nbytes == pre.scratch_bytes >= 256 and nbytes % 256 == 0
    assert (pre.num_qo_heads, pre.batch, pre.rows, pre.tokens) == (16, 4, 100, 900)
    many = plan_of(batch=8193)
    for args, code in (((plan_of(), 0, 5), B.PDA_ERR_INVALID), ((many, 9000, 9000), B.PDA_ERR_INVALID),
                       ((plan_of(), 2 ** 31 - 1, 5), B.PDA_ERR_INVALID),
                       ((plan_of(), 5, 2 ** 31 - 1), B.PDA_ERR_INVALID), ((plan_of(), 5, 0), B.PDA_ERR_INVALID),
                       ((gqa_plan(), 5, 5), B.PDA_ERR_UNSUPPORTED), ((bad_plan(), 5, 5), B.PDA_ERR_PLAN)):
        assert B.pda_prefill_plan(*args, check=False)[2] == code
    assert lib.pda_prefill_plan(None, 5, 5, ctypes.byref(pre), None) == B.PDA_ERR_NULL
    plan = plan_of()
    assert lib.pda_prefill_plan(ctypes.byref(plan), 5, 5, None, None) == B.PDA_ERR_NULL


@pytest.mark.parametrize("change,code", [
    (dict(q=None), B.PDA_ERR_NULL), (dict(k=None), B.PDA_ERR_NULL), (dict(v=None), B.PDA_ERR_NULL),
    (dict(rope=None), B.PDA_ERR_NULL), (dict(qo=None), B.PDA_ERR_NULL), (dict(out=None), B.PDA_ERR_NULL),
    (dict(scratch=None), B.PDA_ERR_SCRATCH), (dict(scratch=OKP + 4), B.PDA_ERR_SCRATCH),
    (dict(win=OKP, causal=0), B.PDA_ERR_UNSUPPORTED), (dict(qr=100), B.PDA_ERR_INVALID),
    (dict(kh=64), B.PDA_ERR_INVALID), (dict(rs=56), B.PDA_ERR_INVALID),
    (dict(qh=196), B.PDA_ERR_ALIGNMENT), (dict(kt=4100), B.PDA_ERR_ALIGNMENT),
    (dict(rs=577), B.PDA_ERR_ALIGNMENT), (dict(rope=OKP + 2), B.PDA_ERR_ALIGNMENT),
    (dict(lse=ODD), B.PDA_ERR_ALIGNMENT), (dict(win=ODD), B.PDA_ERR_ALIGNMENT)])
def test_prefill_refusals(lib, change, code):
    a = {**dict(q=OKP, qr=16 * 192, qh=192, k=OKP, v=OKP, kt=16 * 256, kh=256, rope=OKP, rs=576, qo=OKP,
                tok=OKP, win=None, causal=1, out=OKP, lse=None, scratch=OKP), **change}
    pre = B.pda_prefill_plan(plan_of(), 10, 10)[0]
    assert lib.pda_mla_prefill(ctypes.byref(pre), a["q"], a["qr"], a["qh"], a["k"], a["v"], a["kt"],
                               a["kh"], a["rope"], a["rs"], a["qo"], a["tok"], a["win"], a["causal"],
                               0.1, a["out"], a["lse"], a["scratch"], None) == code
    pre.struct_bytes += 8
    assert lib.pda_mla_prefill(ctypes.byref(pre), *[OKP, 16 * 192, 192, OKP, OKP, 4096, 256, OKP, 576, OKP,
                               OKP, None, 1, 0.1, OKP, None, OKP, None]) == B.PDA_ERR_PLAN


def test_no_spills_in_the_new_kernels(lib):
    """Registers decide the softmax loop's pace: at most four spilled bytes (of the prefill's
    item bookkeeping), none elsewhere."""
    found = {}
    for name, (regs, stack, st, ld) in build_mod.ptxas_reports().items():
        for k in ("prefill", "product", "expand", "gather_latent", "append_slots", "build_tables"):
            if k in name and "prefill_join" not in name:
                found.setdefault(k, []).append((st, ld))
    assert len(found) == 6, sorted(found)
    for k, v in found.items():
        assert max(v) <= ((4, 16) if k == "prefill" else (0, 0)), (k, v)
