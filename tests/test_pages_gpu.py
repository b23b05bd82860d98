"""GPU parity of the calls over shared pages with plain implementations: forks, free lists
and moves (equal, every entry), and copies of pages in every cache format (every byte)."""
from __future__ import annotations

import random

import pytest
import torch

import pages_ref as ref
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
MARK = -9


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def strided(block, extra):
    """A block table on the device, its rows ``extra`` entries further apart than its columns."""
    t = ints(block).reshape(len(block), -1)
    wide = torch.full((t.shape[0], t.shape[1] + extra), MARK, dtype=torch.int32, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


# ------------------------------------------------------------------- forks

FORKS = {
    "one_token": dict(lens=[1], children=[(0, 1)]),
    "nothing_shared": dict(lens=[40], children=[(0, 0), (0, 0)], free=0),
    "ends": dict(lens=[64], children=[(0, n) for n in (1, 15, 16, 17, 31, 32, 33, 63, 64)]),
    "page_of_one": dict(lens=[9, 5], children=[(0, 9), (1, 3), (0, 1)], page=1),
    "page_256": dict(lens=[700, 256], children=[(0, 700), (1, 256), (1, 255)], page=256),
    "list_runs_out": dict(lens=[50, 33], children=[(0, 50), (1, 33), (0, 48), (1, 1), (0, 3)], free=2),
    "list_exact": dict(lens=[50, 33], children=[(0, 50), (1, 33), (0, 48), (1, 1)], free=3),
    "list_empty": dict(lens=[50], children=[(0, 50), (0, 48)], free=0),
    "negative": dict(lens=[50], children=[(0, 50), (0, -1), (0, 20)]),
    "above_max_kv": dict(lens=[90], children=[(0, 90), (0, 101), (0, 90)], max_kv=100),
    "above_columns": dict(lens=[40], children=[(0, 40), (0, 49), (0, 8)], cols=3),
    "int32_length": dict(lens=[40], children=[(0, 2 ** 31 - 1), (0, 8)], max_kv=2 ** 31 - 1),
    "rows_out_of_range": dict(lens=[40, 40], children=[(0, 40), (-1, 8), (99, 9), (1, 40)]),
    "many_of_one": dict(lens=[1000], children=[(0, 990)] * 70),
    "more_than_ctas": dict(lens=[60, 200, 31], children=[(i % 3, i % 29) for i in range(700)]),
    "long": dict(lens=[40000], children=[(0, 40000), (0, 39990), (0, 160)]),
}


def fork_case(lens, children, page=16, free=None, max_kv=1 << 20, cols=None, seed=0, poison=()):
    r = random.Random(seed)
    cols = cols if cols is not None else max(ref.ceil(n, page) for n in lens) + 2
    need = sum(n > 0 and n % page > 0 for _, n in children)
    free = need + 2 if free is None else free
    pages = sum(ref.ceil(n, page) for n in lens) + max(free, need) + 3
    ids = list(range(pages))
    r.shuffle(ids)
    rows = list(range(len(lens) + len(children) + 1))
    r.shuffle(rows)
    block = [[-7] * cols for _ in rows]
    for p, n in enumerate(lens):
        for j in range(min(cols, ref.ceil(n, page))):
            block[rows[p]][j] = ids.pop()
    for p, j, v in poison:
        block[rows[p]][j] = v
    parent = [rows[p] if 0 <= p < len(lens) else p for p, _ in children]
    return dict(parent=parent, child=rows[len(lens):len(lens) + len(children)],
                lens=[n for _, n in children], block=block, free_pages=ids[:max(free, 1)],
                free_count=free, page=page, max_kv=max_kv, pages=pages)


def run_fork(c, extra=0):
    dec = B.Decoder(ref.plan_params(page=c["page"], pages=c["pages"], max_kv=c["max_kv"]), device=DEV)
    n = len(c["lens"])
    wide, table = strided(c["block"], extra)
    out = {k: ints([MARK] * n) for k in ("child_len", "copy_src", "copy_dst", "copy_tokens")}
    out["free_left"] = ints([MARK])
    args = [ints(c["parent"]), ints(c["child"]), ints(c["lens"]), table, ints(c["free_pages"]),
            ints([c["free_count"]]), out["free_left"], out["child_len"], out["copy_src"],
            out["copy_dst"], out["copy_tokens"], dec.scratch]
    for _ in range(2):  # the same inputs again: the same outputs
        B.pda_fork_tables(dec.plan, *args)
    want, status = ref.fork(c["parent"], c["child"], c["lens"], [list(r) for r in c["block"]],
                            c["free_pages"], c["free_count"], page=c["page"], max_kv=c["max_kv"],
                            num_pages=c["pages"])
    assert dec.status() == status
    for k, t in out.items():
        assert t.tolist() == want[k], k
    assert table.tolist() == want["block_table"]
    if extra:
        assert bool((wide[:, -extra:] == MARK).all())
    return status


@pytest.mark.parametrize("name", sorted(FORKS))
def test_fork(name):
    run_fork(fork_case(**FORKS[name]), extra=3 if len(name) % 2 else 0)


def test_fork_of_pages_out_of_range():
    c = fork_case([100, 50], [(0, 100), (0, 37), (1, 50), (1, 32)], poison=[(0, 2, -5), (1, 3, 10 ** 6)])
    assert run_fork(c) & B.PDA_STATUS_PAGE_OOB
    c = fork_case([50], [(0, 50)])
    c["free_pages"] = [10 ** 6] * len(c["free_pages"])
    assert run_fork(c) == B.PDA_STATUS_PAGE_OOB


def test_fork_of_itself_and_of_nothing():
    c = fork_case([50, 20], [(0, 50), (1, 20)])
    c["child"][1] = c["parent"][1]
    assert run_fork(c) == B.PDA_STATUS_TABLE_INVALID
    c = fork_case([50], [])
    run_fork(c)


# ------------------------------------------------------- free and compacted

def held_case(lens, *, page=16, shared=0.0, spare=6, rows=0, seed=0, poison=(), request=True,
              max_kv=1 << 20, cols=None):
    r = random.Random(seed)
    need = [ref.ceil(max(n, 0), page) for n in lens]
    cols = cols if cols is not None else max(need + [1]) + 1
    pages = sum(need) + spare
    ids = list(range(pages))
    r.shuffle(ids)
    table_rows = len(lens) + rows
    order = list(range(table_rows))
    if request:
        r.shuffle(order)
    block = [[r.randrange(pages) for _ in range(cols)] for _ in range(table_rows)]  # stale entries
    first = None
    for b, n in enumerate(need):
        row = [ids.pop() for _ in range(n)]
        if first and shared:
            k = min(int(shared * len(first)), n)
            row[:k] = first[:k]
        first = first or row
        block[order[b]][:min(n, cols)] = row[:cols]
    for b, j, v in poison:
        block[order[b]][j] = v
    return dict(lens=lens, request=order[:len(lens)] if request else None, block=block, page=page,
                pages=pages, max_kv=max_kv)


HELD = {
    "one_token": dict(lens=[1]),
    "no_requests": dict(lens=[], rows=2),
    "no_lengths": dict(lens=[0, 0, 0]),
    "one_page_in_all": dict(lens=[16], spare=0),
    "everything_held": dict(lens=[160, 33, 16], spare=0),
    "page_borders": dict(lens=[15, 16, 17, 31, 32, 33]),
    "word_borders": dict(lens=[16] * 31, spare=1),
    "word_borders_over": dict(lens=[16] * 32, spare=1),
    "shared": dict(lens=[400, 300, 350, 17, 400], shared=0.8, spare=40),
    "all_shared": dict(lens=[333] * 40, shared=1.0, spare=200),
    "page_of_one": dict(lens=[50, 9, 0, 3], page=1, spare=77),
    "rows_as_they_are": dict(lens=[40, 80, 3], request=False, rows=2),
    "many_words": dict(lens=[3000, 9000, 160, 5000], spare=30000),
    "many_requests": dict(lens=[(37 * i) % 90 for i in range(1500)], shared=0.3, spare=500),
    "long_rows": dict(lens=[80000, 70001], shared=0.5, spare=3000),
    "negative": dict(lens=[40, -1, 30]),
    "above_max_kv": dict(lens=[40, 120, 30], max_kv=100),
    "above_columns": dict(lens=[40, 100, 30], cols=4),
    "out_of_range": dict(lens=[100, 40], poison=[(0, 2, -1), (1, 1, 10 ** 7), (0, 4, -2 ** 31)]),
}


def run_held(c, most=None, in_place=False, extra=0, pool=None, plan=None):
    plan = plan or B.pda_plan(ref.plan_params(page=c["page"], pages=c["pages"], max_kv=c["max_kv"]))[0]
    pool = pool or B.Pages(plan)
    pool.reset_status()
    wide, table = strided(c["block"], extra)
    free, left = ints([MARK] * (c["pages"] + 2)), ints([MARK])
    req = None if c["request"] is None else ints(c["request"])
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    want, status = ref.compact(c["lens"], c["request"], c["block"], page=c["page"],
                               max_kv=c["max_kv"], num_pages=c["pages"], most=most or 0)
    got = dict(free_pages=free, free_left=left)
    if most is None:
        for _ in range(2):
            B.pda_free_pages(plan, lens, req, table, free, left, pool.scratch)
        assert table.tolist() == c["block"]
    else:
        wide2 = wide if in_place else torch.full_like(wide, MARK)
        new = wide2[:, :table.shape[1]]
        got.update(copy_src=ints([MARK] * (most + 1)), copy_dst=ints([MARK] * (most + 1)),
                   num_copies=ints([MARK]))
        for _ in range(1 if in_place else 2):
            B.pda_compact_pages(plan, lens, req, table, new, free, left, got["copy_src"][:most],
                                got["copy_dst"][:most], got["num_copies"], pool.scratch)
        # entries that do not count stay as they were
        full = [list(r) for r in (c["block"] if in_place else [[MARK] * len(r) for r in c["block"]])]
        for b, n in enumerate(c["lens"]):
            row = c["request"][b] if c["request"] else b
            k = min(len(full[row]), ref.ceil(max(n, 0), c["page"]))
            full[row][:k] = want["new_table"][row][:k]
        assert new.tolist() == full
        if extra:
            assert bool((wide2[:, -extra:] == MARK).all())
    assert pool.status() == status
    for k, t in got.items():
        t = t.tolist()
        assert t == want[k] + [MARK] * (len(t) - len(want[k])), k
    # nothing is left in the scratch for the next call
    assert not bool(pool.scratch[256:256 + 4 * ref.ceil(c["pages"], 32)].any())
    return want


@pytest.mark.parametrize("name", sorted(HELD))
def test_free(name):
    run_held(held_case(**HELD[name]), extra=len(name) % 3)


@pytest.mark.parametrize("most", [0, 1, 5, 1 << 14])
@pytest.mark.parametrize("name", sorted(HELD))
def test_compact(name, most):
    run_held(held_case(**HELD[name]), most=most, in_place=most == 5, extra=len(name) % 2)


@pytest.mark.parametrize("name", sorted(HELD))
@pytest.mark.parametrize("pages", [131073, 400000, 524289])
def test_many_pages(name, pages):
    """The same behind more pages than one CTA lists, and than a CTA marks in shared memory."""
    c = held_case(**{**HELD[name], "spare": pages + len(name)})
    run_held(c, extra=1)
    run_held(c, most=40, in_place=len(name) % 2 == 0)


@pytest.mark.parametrize("n,cols", [(512, 32), (513, 3), (512, 33), (16, 1024), (1, 16385), (1030, 70)])
def test_about_what_one_cta_takes(n, cols):
    r = random.Random(n)
    c = held_case([r.randint(0, 16 * cols) for _ in range(n)], cols=cols, shared=0.7, spare=9)
    run_held(c)
    run_held(c, most=20)


def test_rows_named_twice():
    c = held_case([100, 60], spare=30)
    c["request"], c["lens"] = c["request"] + c["request"][:1], [100, 60, 70]
    run_held(c)
    run_held(c, most=100)
    run_held(c, most=100, in_place=True)


def test_one_scratch_for_both_calls_in_turn():
    a, b = held_case([400, 90, 300], spare=50, seed=1), held_case([64, 700], spare=20, seed=2)
    for c in (a, b):
        c["pages"] = 200
    plan = B.pda_plan(ref.plan_params(page=16, pages=200))[0]
    pool = B.Pages(plan)
    for c, most in ((a, None), (b, 7), (a, 100), (b, None), (a, 0), (a, None)):
        run_held(c, most=most, pool=pool, plan=plan)


# ------------------------------------------------------------------ copies

FORMATS = ["bf16", "e4m3_tensor", "e4m3_token", "int8_token", "records", "latent", "latent_e4m3"]


@pytest.mark.parametrize("tokens", [False, True])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "gaps"])
@pytest.mark.parametrize("kind", FORMATS)
def test_copy(kind, layout, tokens):
    latent = kind in ("records", "latent", "latent_e4m3")
    hnd, gap = layout == "hnd", 16 if layout == "gaps" else 0
    heads, dim, page, pages = (1, 576, 32, 12) if latent else (3, 128, 16, 12)
    g = torch.Generator().manual_seed(len(kind) + len(layout))
    dec = B.Decoder(ref.plan_params(kind, heads=heads, dim=dim, page=page, pages=pages, hnd=hnd, gap=gap),
                    device=DEV)
    src, dst = [3, -1, 7, 0, 5, 11, 40, 2], [1, 4, 9, -1, 6, 10, 8, -3]
    toks = [5, 3, page, 2, 0, page + 9, 4, 1] if tokens else None
    sides, wide = [], []
    for _ in range(1 if latent else 2):
        c, s = ref.filled(g, pages, page, heads, kind, dim, hnd)
        full = torch.full((*c.shape[:-1], c.shape[-1] + gap), 3, dtype=c.dtype)
        full[..., :c.shape[-1]] = c
        wide.append(full.to(DEV))
        sides.append((full, None if s is None else s, None if s is None else s.to(DEV)))
    k, v = wide[0], wide[1] if len(wide) > 1 else None
    one = torch.ones(1, device=DEV) if kind in ("e4m3_tensor", "latent_e4m3") else None
    ks = sides[0][2] if sides[0][2] is not None else one
    vs = None if v is None else sides[1][2] if sides[1][2] is not None else one
    B.pda_copy_pages(dec.plan, k, v, ks, vs, ints(src), ints(dst), None if toks is None else ints(toks),
                     None, dec.scratch)
    assert dec.status() == B.PDA_STATUS_PAGE_OOB  # pages 40 and -3
    for t, (full, s, sd) in zip(wide, sides):
        want = ref.copy(full, src, dst, toks, page, 1 if hnd else 0)
        # the channels of a gap are not the cache's
        w = want.shape[-1] - gap
        assert torch.equal(t.cpu()[..., :w].contiguous().view(torch.uint8),
                           want[..., :w].contiguous().view(torch.uint8))
        if gap:
            assert torch.equal(t.cpu()[..., w:], full[..., w:])
        if s is not None:
            assert torch.equal(sd.cpu(), ref.copy(s, src, dst, toks, page, 0))


@pytest.mark.parametrize("live", [0, 1, 3, 9, -2])
def test_copy_takes_num_copies(live):
    g = torch.Generator().manual_seed(5)
    dec = B.Decoder(ref.plan_params(pages=10), device=DEV)
    c, _ = ref.filled(g, 10, 16, 2, "bf16", 128)
    k, v = c.to(DEV), (c * 2).to(DEV)
    src, dst = [1, 2, 3, 4, 5], [6, 7, 8, 9, 0]
    B.pda_copy_pages(dec.plan, k, v, None, None, ints(src), ints(dst), None, ints([live]), dec.scratch)
    n = max(0, min(live, 5))
    assert torch.equal(k.cpu(), ref.copy(c, src[:n], dst[:n], None, 16, 0))
    assert torch.equal(v.cpu(), ref.copy(c * 2, src[:n], dst[:n], None, 16, 0))
    assert dec.status() == 0


@pytest.mark.parametrize("page,heads,dim", [(1, 1, 64), (8, 1, 64), (128, 8, 256), (256, 2, 512)])
def test_copy_page_sizes(page, heads, dim):
    g = torch.Generator().manual_seed(page)
    dec = B.Decoder(ref.plan_params(heads=heads, dim=dim, page=page, pages=9), device=DEV)
    c, _ = ref.filled(g, 9, page, heads, "bf16", dim)
    k, v = c.to(DEV), c.flip(0).to(DEV)
    src, dst, toks = [8, 2, 4], [0, 1, 3], [page, page // 2 + 1, 1]
    B.pda_copy_pages(dec.plan, k, v, None, None, ints(src), ints(dst), ints(toks), None, dec.scratch)
    assert torch.equal(k.cpu(), ref.copy(c, src, dst, toks, page, 0))
    assert torch.equal(v.cpu(), ref.copy(c.flip(0), src, dst, toks, page, 0))


def test_copy_far_offsets():
    """Pages whose byte offsets pass 32 bits."""
    page, heads, dim, pages = 256, 8, 128, 9000  # 512 KB a page
    dec = B.Decoder(ref.plan_params(heads=heads, dim=dim, page=page, pages=pages), device=DEV)
    k = torch.zeros(pages, page, heads, dim, dtype=torch.bfloat16, device=DEV)
    src, dst = [8999, 3, 8500], [1, 8998, 8497]
    for s in src:
        k[s] = torch.randn(page, heads, dim, device=DEV).to(torch.bfloat16)
    B.pda_copy_pages(dec.plan, k, k, None, None, ints(src), ints(dst), None, None, dec.scratch)
    for s, d in zip(src, dst):
        assert torch.equal(k[s], k[d]) and bool(k[d].any())
    assert int(k.flatten(1).any(1).sum()) == 6 and dec.status() == 0
