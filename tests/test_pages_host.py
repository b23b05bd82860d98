"""Refusals of the calls over shared pages on the CPU: every host check returns its code
before anything is launched (pointers here are numbers, never read), and the binding
refuses tensors that the library cannot see through."""
import ctypes

import pytest
import torch

import pages_ref as ref
from paged_split_kv_03_gb300 import binding as B
from paged_split_kv_03_gb300 import build as build_mod

OKP, ODD = 0x10000, 0x10002


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def plan_of(kind="bf16", **kw):
    return B.pda_plan(ref.plan_params(kind, num_sms=152, **kw))[0]


def bad_plan():
    p = plan_of()
    p.magic = 1
    return p


FORKS = dict(parent=OKP, child=OKP + 64, shared_len=OKP + 128, block_table=OKP, table_stride=8,
             free_pages=OKP, free_count=OKP, free_left=OKP + 4, child_len=OKP + 192, copy_src=OKP,
             copy_dst=OKP, copy_tokens=OKP, table_rows=4, table_cols=8, forks=3)


@pytest.mark.parametrize("change,code", [
    (dict(parent=None), B.PDA_ERR_NULL), (dict(child=None), B.PDA_ERR_NULL),
    (dict(shared_len=None), B.PDA_ERR_NULL), (dict(block_table=None), B.PDA_ERR_NULL),
    (dict(free_pages=None), B.PDA_ERR_NULL), (dict(free_count=None), B.PDA_ERR_NULL),
    (dict(free_left=None), B.PDA_ERR_NULL), (dict(child_len=None), B.PDA_ERR_NULL),
    (dict(copy_src=None), B.PDA_ERR_NULL), (dict(copy_dst=None), B.PDA_ERR_NULL),
    (dict(copy_tokens=None), B.PDA_ERR_NULL), (dict(forks=-1), B.PDA_ERR_INVALID),
    (dict(forks=65537), B.PDA_ERR_INVALID), (dict(table_rows=-1), B.PDA_ERR_INVALID),
    (dict(table_cols=-1), B.PDA_ERR_INVALID), (dict(table_stride=7), B.PDA_ERR_INVALID),
    (dict(free_left=OKP), B.PDA_ERR_INVALID), (dict(child_len=OKP + 128), B.PDA_ERR_INVALID),
    (dict(parent=ODD), B.PDA_ERR_ALIGNMENT), (dict(copy_tokens=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(free_left=ODD), B.PDA_ERR_ALIGNMENT)])
def test_fork_refusals(lib, change, code):
    f, plan = B.PdaForks(**{**FORKS, **change}), plan_of()
    assert lib.pda_fork_tables(ctypes.byref(plan), ctypes.byref(f), OKP, None) == code


def test_fork_refusals_of_plan_and_scratch(lib):
    f, plan = B.PdaForks(**FORKS), plan_of()
    call = lib.pda_fork_tables
    assert call(None, ctypes.byref(f), OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(plan), None, OKP, None) == B.PDA_ERR_NULL
    assert call(ctypes.byref(bad_plan()), ctypes.byref(f), OKP, None) == B.PDA_ERR_PLAN
    assert call(ctypes.byref(plan), ctypes.byref(f), None, None) == B.PDA_ERR_SCRATCH
    assert call(ctypes.byref(plan), ctypes.byref(f), OKP + 16, None) == B.PDA_ERR_SCRATCH


def copy(lib, plan, **kw):
    a = {**dict(k=OKP, v=OKP, ks=None, vs=None, src=OKP, dst=OKP, tok=OKP, n=3, num=OKP, scratch=OKP),
         **kw}
    return lib.pda_copy_pages(ctypes.byref(plan), a["k"], a["v"], a["ks"], a["vs"], a["src"], a["dst"],
                              a["tok"], a["n"], a["num"], a["scratch"], None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), B.PDA_ERR_NULL), (dict(v=None), B.PDA_ERR_NULL), (dict(src=None), B.PDA_ERR_NULL),
    (dict(dst=None), B.PDA_ERR_NULL), (dict(n=-1), B.PDA_ERR_INVALID),
    (dict(scratch=None), B.PDA_ERR_SCRATCH), (dict(scratch=OKP + 8), B.PDA_ERR_SCRATCH),
    (dict(k=OKP + 8), B.PDA_ERR_ALIGNMENT), (dict(v=OKP + 4), B.PDA_ERR_ALIGNMENT),
    (dict(src=ODD), B.PDA_ERR_ALIGNMENT), (dict(tok=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(num=ODD), B.PDA_ERR_ALIGNMENT), (dict(n=0, src=None, dst=None), B.PDA_OK)])
def test_copy_refusals(lib, change, code):
    assert copy(lib, plan_of(), **change) == code


def test_copy_refusals_of_scales_latents_and_plans(lib):
    tok = plan_of("e4m3_token")
    assert copy(lib, tok) == B.PDA_ERR_NULL
    assert copy(lib, tok, ks=OKP) == B.PDA_ERR_NULL
    assert copy(lib, tok, ks=OKP, vs=ODD) == B.PDA_ERR_ALIGNMENT
    assert copy(lib, plan_of("records"), v=None) == B.PDA_ERR_NULL  # its scales
    assert copy(lib, plan_of("latent"), v=None, n=0) == B.PDA_OK
    assert copy(lib, plan_of("e4m3_tensor"), n=0) == B.PDA_OK      # one scale: nothing to copy
    assert copy(lib, bad_plan()) == B.PDA_ERR_PLAN


PAGES = dict(lengths=OKP, request=None, block_table=OKP, table_stride=8, free_pages=OKP,
             free_left=OKP, new_table=OKP, copy_src=OKP, copy_dst=OKP, num_copies=OKP, requests=3,
             table_rows=3, table_cols=8, max_copies=4)


@pytest.mark.parametrize("call", ["pda_free_pages", "pda_compact_pages"])
@pytest.mark.parametrize("change,code", [
    (dict(lengths=None), B.PDA_ERR_NULL), (dict(block_table=None), B.PDA_ERR_NULL),
    (dict(free_pages=None), B.PDA_ERR_NULL), (dict(free_left=None), B.PDA_ERR_NULL),
    (dict(requests=-1), B.PDA_ERR_INVALID), (dict(requests=4), B.PDA_ERR_INVALID),
    (dict(table_rows=-1), B.PDA_ERR_INVALID), (dict(table_cols=-1), B.PDA_ERR_INVALID),
    (dict(table_stride=7), B.PDA_ERR_INVALID), (dict(lengths=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(request=ODD), B.PDA_ERR_ALIGNMENT), (dict(free_left=ODD), B.PDA_ERR_ALIGNMENT)])
def test_free_and_compact_refusals(lib, call, change, code):
    p, plan = B.PdaPages(**{**PAGES, **change}), plan_of()
    assert getattr(lib, call)(ctypes.byref(plan), ctypes.byref(p), OKP, None) == code


@pytest.mark.parametrize("change,code", [
    (dict(new_table=None), B.PDA_ERR_NULL), (dict(copy_src=None), B.PDA_ERR_NULL),
    (dict(copy_dst=None), B.PDA_ERR_NULL), (dict(num_copies=None), B.PDA_ERR_NULL),
    (dict(max_copies=-1), B.PDA_ERR_INVALID), (dict(new_table=ODD), B.PDA_ERR_ALIGNMENT),
    (dict(copy_dst=ODD), B.PDA_ERR_ALIGNMENT)])
def test_compact_refusals(lib, change, code):
    p, plan = B.PdaPages(**{**PAGES, **change}), plan_of()
    assert lib.pda_compact_pages(ctypes.byref(plan), ctypes.byref(p), OKP, None) == code


def test_free_refusals_of_plan_and_scratch(lib):
    p, plan = B.PdaPages(**PAGES), plan_of()
    for call in (lib.pda_free_pages, lib.pda_compact_pages):
        assert call(None, ctypes.byref(p), OKP, None) == B.PDA_ERR_NULL
        assert call(ctypes.byref(plan), None, OKP, None) == B.PDA_ERR_NULL
        assert call(ctypes.byref(bad_plan()), ctypes.byref(p), OKP, None) == B.PDA_ERR_PLAN
        assert call(ctypes.byref(plan), ctypes.byref(p), None, None) == B.PDA_ERR_SCRATCH
        assert call(ctypes.byref(plan), ctypes.byref(p), OKP + 64, None) == B.PDA_ERR_SCRATCH


def test_page_scratch(lib):
    n = ctypes.c_size_t()
    for pages in (1, 32, 33, 100000):
        plan = plan_of(pages=pages)
        assert lib.pda_pages_scratch(ctypes.byref(plan), ctypes.byref(n)) == 0
        assert n.value % 256 == 0 and n.value >= 256 + 2 * 4 * -(-pages // 32)
        assert B.pda_pages_scratch(plan) == n.value
    plan = plan_of()
    assert lib.pda_pages_scratch(ctypes.byref(plan), None) == B.PDA_ERR_NULL
    assert lib.pda_pages_scratch(None, ctypes.byref(n)) == B.PDA_ERR_NULL
    plan = bad_plan()
    assert lib.pda_pages_scratch(ctypes.byref(plan), ctypes.byref(n)) == B.PDA_ERR_PLAN


class Cuda(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(Cuda)


def ints(n, v=0):
    return on(torch.full((n,), v, dtype=torch.int32))


def test_binding_refuses(lib):
    plan = plan_of(pages=8)
    table, scratch = on(torch.zeros(4, 6, dtype=torch.int32)), on(torch.zeros(4096, dtype=torch.uint8))
    fork = dict(parent=ints(3), child=ints(3), shared_len=ints(3), block_table=table,
                free_pages=ints(5), free_count=ints(1), free_left=ints(1), child_len=ints(3),
                copy_src=ints(3), copy_dst=ints(3), copy_tokens=ints(3), split_scratch=scratch)
    for k, v in (("child", ints(2)), ("parent", ints(3).long()), ("free_left", ints(2)),
                 ("block_table", table.t()), ("copy_src", torch.zeros(3, dtype=torch.int32)),
                 ("copy_dst", on(torch.zeros(6, dtype=torch.int32)[::2]))):
        with pytest.raises(ValueError):
            B.pda_fork_tables(plan, **{**fork, k: v})
    held = dict(lengths=ints(3), request=None, block_table=table, free_pages=ints(8),
                free_left=ints(1), page_scratch=scratch)
    for k, v in (("free_pages", ints(7)), ("request", ints(2)), ("lengths", ints(3).float())):
        with pytest.raises(ValueError):
            B.pda_free_pages(plan, **{**held, k: v})
    with pytest.raises(B.PdaError):
        B.pda_free_pages(plan, **{**held, "page_scratch": on(torch.zeros(256, dtype=torch.uint8))})
    more = dict(new_table=table, copy_src=ints(4), copy_dst=ints(4), num_copies=ints(1))
    for k, v in (("new_table", on(torch.zeros(4, 7, dtype=torch.int32))), ("copy_dst", ints(3)),
                 ("num_copies", ints(2))):
        with pytest.raises(ValueError):
            B.pda_compact_pages(plan, **held, **{**more, k: v})
    cache = on(torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16))
    small = on(torch.zeros(7, 16, 2, 128, dtype=torch.bfloat16))
    cp = dict(k_pages=cache, v_pages=cache, k_scale=None, v_scale=None, copy_src=ints(3),
              copy_dst=ints(3), copy_tokens=None, num_copies=None, split_scratch=scratch)
    for k, v in (("v_pages", small), ("copy_dst", ints(2)), ("copy_tokens", ints(4)),
                 ("num_copies", ints(0)), ("k_pages", cache.float())):
        with pytest.raises(ValueError):
            B.pda_copy_pages(plan, **{**cp, k: v})


def test_no_spills(lib):
    found = {}
    for name, (regs, stack, st, ld) in build_mod.ptxas_reports().items():
        for k in ("fork_tables", "copy_pages", "mark_pages", "list_pages", "renumber", "pages_once", "mark_shared"):
            if k in name:
                found[k] = (stack, st, ld)
    assert len(found) == 7 and set(found.values()) == {(0, 0, 0)}, found
