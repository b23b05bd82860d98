"""Refusals of decode behind shared prefixes on the CPU: every host check returns its code
before anything is launched (pointers here are numbers, never read), and the binding
refuses tensors that the library cannot see through."""
import ctypes

import pytest
import torch

import pages_ref as ref
from paged_split_kv_03_gb300 import binding as B
from paged_split_kv_03_gb300 import build as build_mod
from test_pages_host import ODD, OKP, bad_plan, ints, on

NEXT = 0x20000


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def plan_of(kind="bf16", **kw):
    return B.pda_plan(ref.plan_params(kind, **{**dict(num_sms=152, batch=4, max_kv=4096), **kw}))[0]


def shared_of(kind="bf16", groups=2, own=0, **kw):
    return B.pda_shared_plan(plan_of(kind, **kw), groups, own)[0]


def code_of(plan, groups=1, own=0):
    return B.pda_shared_plan(plan, groups, own, check=False)[2]


def test_plan_refusals(lib):
    sp, n, p = B.PdaSharedPlan(), ctypes.c_size_t(0), plan_of()
    call = lib.pda_shared_plan
    assert call(None, 1, 0, ctypes.byref(sp), ctypes.byref(n)) == B.PDA_ERR_NULL
    assert call(ctypes.byref(p), 1, 0, None, ctypes.byref(n)) == B.PDA_ERR_NULL
    assert call(ctypes.byref(p), 1, 0, ctypes.byref(sp), None) == B.PDA_OK  # (bytes: in the plan)
    assert code_of(bad_plan()) == B.PDA_ERR_PLAN
    for groups in (0, -1, 1025):
        assert code_of(p, groups) == B.PDA_ERR_INVALID
    assert code_of(p, 1024) == B.PDA_OK
    assert code_of(p, 1, -1) == B.PDA_ERR_INVALID
    # (fewer requests than groups: some are empty)
    assert code_of(p, 9) == B.PDA_OK


@pytest.mark.parametrize("kind,kw", [("latent", {}), ("records", {}), ("bf16", dict(dim=512)),
                                     ("bf16", dict(page=4)), ("bf16", dict(page=1))])
def test_caches_that_are_not_built(lib, kind, kw):
    assert code_of(plan_of(kind, **kw)) == B.PDA_ERR_UNSUPPORTED


def test_axis_of_the_work(lib):
    """Tiles of all items, eight each, and 24 an item have to stay in 31 bits."""
    big = dict(heads=8, dim=256, max_q=8, hq=128, batch=4096)  # 4096 blocks of 128 rows a head
    assert code_of(plan_of(max_kv=16384, **big)) == B.PDA_OK
    assert code_of(plan_of(max_kv=1 << 20, **big)) == B.PDA_ERR_INVALID


def test_plan_says_what_it_needs(lib):
    p = plan_of(max_q=2, hq=8, heads=2, dim=128)
    few, n_few, _ = B.pda_shared_plan(p, 2, 100)
    many, n_many, _ = B.pda_shared_plan(p, 2)
    assert few.own.max_kv_len == 100 and many.own.max_kv_len == 4096 and few.max_kv_len == 4096
    assert few.scratch_bytes == n_few and few.own.scratch_bytes == n_few and few.groups == 2
    # two row tiles of 128 x 128 fp32 for each SM, 16 (kv head, row) cells of the batch and more;
    # stage 1's parts of every own token only where own tokens are many
    assert n_few >= 4 * (152 * 256 * 129 + 4 * 2 * 8 * 129)
    assert n_many > n_few
    for k in ("first_offset", "main_lse_offset", "main_o_offset", "area_lse_offset", "area_o_offset"):
        assert getattr(few, k) % 256 == 0 and 0 < getattr(few, k) < n_few
    assert B.pda_shared_plan(p, 2, 1 << 30)[0].own.max_kv_len == 4096


TABLES = dict(page_table=OKP, kv_indptr=OKP, kv_len=OKP, qo_indptr=OKP, window=None, group_indptr=OKP,
              prefix=NEXT, own_indptr=NEXT + 64, own_len=NEXT + 128)
WRONG = [(dict([(k, None)]), B.PDA_ERR_NULL) for k in TABLES if k != "window"]
WRONG += [(dict([(k, ODD)]), B.PDA_ERR_ALIGNMENT) for k in TABLES]
WRONG += [(dict(own_len=OKP), B.PDA_ERR_INVALID), (dict(own_indptr=OKP), B.PDA_ERR_INVALID)]


def decode(lib, sp, tables=None, **kw):
    a = {**dict(q=OKP, k=OKP, v=OKP, max_q=1, ks=None, vs=None, out=OKP, lse=OKP, scratch=OKP), **kw}
    t = B.PdaSharedTables(**(tables or TABLES))
    return lib.pda_decode_shared(ctypes.byref(sp), a["q"], a["k"], a["v"], ctypes.byref(t), a["max_q"], 1.0,
                                 a["ks"], a["vs"], a["out"], a["lse"], a["scratch"], None)


@pytest.mark.parametrize("change,code", WRONG)
def test_table_refusals(lib, change, code):
    sp, tables = shared_of(), {**TABLES, **change}
    t = B.PdaSharedTables(**tables)
    assert lib.pda_share_tables(ctypes.byref(sp), ctypes.byref(t), OKP, None) == code
    assert decode(lib, sp, tables) == code


def test_refusals_of_plan_and_scratch(lib):
    sp, t = shared_of(), B.PdaSharedTables(**TABLES)
    call = lib.pda_share_tables
    assert call(None, ctypes.byref(t), OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(sp), None, OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(sp), ctypes.byref(t), None, None) == B.PDA_ERR_SCRATCH
    assert call(ctypes.byref(sp), ctypes.byref(t), OKP + 128, None) == B.PDA_ERR_SCRATCH
    assert decode(lib, sp, scratch=None) == B.PDA_ERR_SCRATCH
    assert decode(lib, sp, scratch=OKP + 16) == B.PDA_ERR_SCRATCH
    for change in (dict(magic=1), dict(struct_bytes=8)):
        bad = shared_of()
        for k, v in change.items():
            setattr(bad, k, v)
        assert call(ctypes.byref(bad), ctypes.byref(t), OKP, None) == B.PDA_ERR_PLAN
        assert decode(lib, bad) == B.PDA_ERR_PLAN
    bad = shared_of()
    bad.own.magic = 1
    assert decode(lib, bad) == B.PDA_ERR_PLAN


@pytest.mark.parametrize("change,code", [
    (dict(q=None), B.PDA_ERR_NULL), (dict(k=None), B.PDA_ERR_NULL), (dict(v=None), B.PDA_ERR_NULL),
    (dict(out=None), B.PDA_ERR_NULL), (dict(max_q=0), B.PDA_ERR_INVALID), (dict(max_q=2), B.PDA_ERR_INVALID),
    (dict(q=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(k=OKP + 8), B.PDA_ERR_ALIGNMENT),
    (dict(out=OKP + 8), B.PDA_ERR_ALIGNMENT)])
def test_decode_refusals(lib, change, code):
    assert decode(lib, shared_of(), **change) == code


def test_decode_refusals_of_scales(lib):
    sp = shared_of("e4m3_token")
    assert decode(lib, sp) == B.PDA_ERR_NULL
    assert decode(lib, sp, ks=OKP) == B.PDA_ERR_NULL


def test_one_group_needs_no_bounds(lib):
    """(What is left to refuse without a device is the device.)"""
    sp, tables = shared_of(groups=1), {**TABLES, "group_indptr": None}
    t = B.PdaSharedTables(**tables)
    if not torch.cuda.is_available():
        assert lib.pda_share_tables(ctypes.byref(sp), ctypes.byref(t), OKP, None) == B.PDA_ERR_INVALID
        assert decode(lib, sp, tables) == B.PDA_ERR_INVALID


def test_binding_refuses(lib):
    sp = shared_of(groups=2, pages=8, max_q=2, hq=4)
    scratch = on(torch.zeros(sp.scratch_bytes, dtype=torch.uint8))
    tables = dict(page_table=ints(9), kv_indptr=ints(5), kv_len=ints(4), qo_indptr=ints(5), window=None,
                  group_indptr=ints(3), prefix=on(torch.zeros(2, 2, dtype=torch.int32)), own_indptr=ints(4),
                  own_len=ints(4))
    wrong = (("kv_indptr", ints(4)), ("kv_len", ints(5)), ("qo_indptr", ints(4)), ("window", ints(3)),
             ("group_indptr", ints(2)), ("prefix", ints(4)), ("own_len", ints(4).long()),
             ("own_indptr", torch.zeros(4, dtype=torch.int32)),
             ("page_table", on(torch.zeros(18, dtype=torch.int32)[::2])))
    q = on(torch.zeros(3, 4, 128, dtype=torch.bfloat16))
    cache = on(torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16))
    step = dict(q=q, k_pages=cache, v_pages=cache, max_q_len=2, sm_scale=1.0, k_scale=None, v_scale=None,
                out=q, lse=on(torch.zeros(3, 4)))
    for k, v in wrong:
        with pytest.raises(ValueError):
            B.pda_share_tables(sp, **{**tables, k: v}, scratch=scratch)
        with pytest.raises(ValueError):
            B.pda_decode_shared(sp, **step, **{**tables, k: v}, scratch=scratch)
    for k, v in (("q", q[:, :3]), ("q", q.float()), ("out", on(torch.zeros(2, 4, 128, dtype=torch.bfloat16))),
                 ("lse", on(torch.zeros(3, 3))), ("v_pages", cache.float()),
                 ("k_pages", on(torch.zeros(7, 16, 2, 128, dtype=torch.bfloat16)))):
        with pytest.raises(ValueError):
            B.pda_decode_shared(sp, **{**step, k: v}, **tables, scratch=scratch)
    small = on(torch.zeros(sp.scratch_bytes - 1, dtype=torch.uint8))
    with pytest.raises(B.PdaError):
        B.pda_share_tables(sp, **tables, scratch=small)
    with pytest.raises(B.PdaError):
        B.pda_decode_shared(sp, **step, **tables, scratch=small)


def test_spills(lib):
    """Bytes spilled (stores + loads) by builds of the new kernels that are accepted now: the
    prefix kernel compiles to 128 registers for roles that run with 64 to 216, the most with
    int8 codes and scales per token; the own tokens' kernel spills next to nothing."""
    found = {k: [] for k in ("shared_prefix", "own_join", "shared_join", "share_tables")}
    for name, (regs, stack, st, ld) in build_mod.ptxas_reports().items():
        for k in found:
            if k in name:
                found[k].append(st + ld)
    assert [len(found[k]) for k in found] == [15, 15, 3, 1], found
    assert max(found["shared_join"] + found["share_tables"]) <= 8, found
    assert max(found["own_join"]) <= 24, found
    assert max(found["shared_prefix"]) <= 320, found
