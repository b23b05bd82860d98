"""GPU parity of decode behind shared prefixes: the prefixes that requests share (equal, every
entry) and the attention over them and the requests' own tokens against 64 bits, element
by element, for every cache format, odd lengths, windows and groups."""
from __future__ import annotations

import math
import random

import pytest
import torch

import shared_ref as S
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def check(got, want, bound, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    fine = torch.isfinite(want)
    err, lim = (got - want).abs()[fine], bound[fine]
    worst = (err - lim).argmax()
    assert bool((err <= lim).all()), \
        f"{what}: error {err[worst]:.3e}, bound {lim[worst]:.3e}, value {want[fine][worst]:.3e}"


def parity(w, sm_scale=None, shared=None):
    """Both ways of the own tokens: planned for any number of them (stage 1, then the join), and
    for no more than there are (one kernel, where they are few)."""
    dec = B.Decoder(w.params, device=DEV)
    (prefix, ptr, own), status = S.share(w)
    o, ob, l, lb = S.attention(w, sm_scale)
    for sh in [shared] if shared else [B.Shared(dec.plan, len(w.gp) - 1, n) for n in (0, max(own + [1]))]:
        t = S.device_tables(w)
        out, lse = S.run(w, sh, t, sm_scale=sm_scale)
        torch.cuda.synchronize()
        assert t.prefix.reshape(-1).tolist() == prefix
        assert t.own_indptr.tolist() == ptr and t.own_len.tolist() == own
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")
        assert sh.status() == status
    return sh, t


def reqs(n, own=37, rows=1, seed=0):
    r = random.Random(seed)
    return [(max(r.randint(1, own), k), k) for k in (r.randint(1, rows) for _ in range(n))]


KINDS = ["bf16", "e4m3_tensor", "e4m3_token", "int8_tensor", "int8_token"]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_formats(kind, dim):
    # 17 pages of 16: two tiles and 16 keys; 5 requests x 2 rows x 4 heads
    parity(S.make([(17, reqs(5, rows=2))], kind=kind, dim=dim, dev=DEV, seed=dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["e4m3_tensor", "e4m3_token"])
def test_e4m3_query(kind, dim):
    parity(S.make([(40, reqs(3, rows=3))], kind=kind, dim=dim, q8=True, hnd=True, dev=DEV, seed=dim))


@pytest.mark.parametrize("kind", ["bf16", "e4m3_token"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_page_sizes(dim, page, kind):
    # prefixes of 1 page, of less than a tile and a bit more than some tiles
    for pages in (1, max(1, 100 // page), 600 // page + 1):
        parity(S.make([(pages, reqs(4, own=70))], kind=kind, dim=dim, page=page, hnd=page % 64 == 0,
                      dev=DEV, seed=pages))


@pytest.mark.parametrize("kind", ["bf16", "int8_token"])
@pytest.mark.parametrize("dim,hkv,group,requests,rows", [
    (128, 1, 1, 1, 1), (128, 1, 1, 3, 1), (128, 1, 16, 8, 1), (128, 2, 16, 16, 1), (128, 1, 5, 60, 1),
    (128, 2, 24, 12, 8), (128, 8, 8, 33, 1), (64, 4, 3, 50, 4), (64, 1, 8, 32, 1), (256, 2, 8, 17, 2),
    (256, 1, 6, 30, 5), (256, 8, 1, 130, 1)])
def test_rows_and_heads(dim, hkv, group, requests, rows, kind):
    """Packed rows below, at and above one and two tiles."""
    parity(S.make([(19, reqs(requests, own=20, rows=rows))], kind=kind, dim=dim, hkv=hkv, group=group,
                  dev=DEV, seed=requests))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_long_prefix(kind, dim):
    """Many segments of an item over the CTAs, and CTAs that start inside one."""
    parity(S.make([(1301, reqs(9, own=300, rows=2))], kind=kind, dim=dim, hkv=2, group=4, dev=DEV))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_many_items(kind, dim):
    """Several segments a CTA: items of two row tiles, of one, of a few tiles and of many."""
    groups = [(17, reqs(30)), (3, reqs(5)), (40, reqs(9, rows=2)), (1, reqs(1)), (90, reqs(26))]
    parity(S.make(groups, kind=kind, dim=dim, page=128, hkv=8, group=3, hnd=True, dev=DEV, spare=1))


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("bf16", 64), ("e4m3_token", 256)])
def test_groups(kind, dim):
    groups = [(9, reqs(3)), (0, reqs(2)), (30, reqs(1)), (3, []), (1, reqs(7, rows=3)), (100, reqs(40)),
              (2, reqs(2, own=400))]
    parity(S.make(groups, kind=kind, dim=dim, dev=DEV, seed=3))


@pytest.mark.parametrize("dim", [128, 256])
def test_more_groups_than_lanes(dim):
    r = random.Random(5)
    groups = [(r.randint(0, 30), reqs(r.randint(0, 4), seed=i)) for i in range(75)]
    parity(S.make(groups, dim=dim, hkv=2, group=2, dev=DEV))


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 128), ("bf16", 256), ("int8_token", 256),
                                      ("e4m3_tensor", 64)])
def test_windows(kind, dim):
    rs = reqs(8, own=40, rows=4, seed=2)
    windows = [0, 1, 5, 64, 200, 333, 10 ** 6, 2 ** 31 - 1]
    parity(S.make([(30, rs)], kind=kind, dim=dim, windows=windows, dev=DEV))
    # every row's window begins behind some of the prefix, or behind all of it
    parity(S.make([(30, rs)], kind=kind, dim=dim, windows=[100 + 7 * i for i in range(8)], dev=DEV))
    parity(S.make([(30, rs)], kind=kind, dim=dim, windows=[1] * 8, dev=DEV))


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 128), ("e4m3_tensor", 256)])
@pytest.mark.parametrize("scale", [0.3, 0.0, -0.1])
def test_scales_of_the_logits(kind, dim, scale):
    """Peaked weights; equal ones; a negative scale."""
    parity(S.make([(25, reqs(6))], kind=kind, dim=dim, dev=DEV), sm_scale=scale)


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 64)])
def test_gaps_between_heads(kind, dim):
    parity(S.make([(20, reqs(5))], kind=kind, dim=dim, gap=16, dev=DEV))


@pytest.mark.parametrize("kind,dim", [("e4m3_token", 128), ("int8_tensor", 128), ("e4m3_tensor", 256)])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100, 2.0 ** 15, 2.0 ** -9])
def test_queries_far_from_one(kind, dim, size):
    """bf16 queries whose rows leave f16's range; every other row is an ordinary one."""
    w = S.make([(20, reqs(6))], kind=kind, dim=dim, dev=DEV)
    big = w.q.float()
    big[::2] *= size
    w.q = big.to(torch.bfloat16)
    w.q_scale = 1.0
    # the logits stay in reach: those of the scaled rows are, the others go to zero or are huge
    parity(w, sm_scale=w.dim ** -0.5 / size if size > 1 else w.dim ** -0.5)


def test_page_ids_decide():
    """Requests whose tables part early, a page out of range, one request, and none in common."""
    w = S.make([(12, reqs(4, own=50))], dev=DEV, spare=40)
    w.tables[2][7] = next(i for i in range(w.pages) if i not in w.page_table)
    for val, c in zip(w.values, w.cache):  # what stands there is another page's
        x = torch.randn(c.shape[1:]).to(torch.bfloat16)
        c[w.tables[2][7]] = x.to(DEV)
        val[w.tables[2][7]] = x.double()
    w.page_table = [x for t in w.tables for x in t]
    _, t = parity(w)
    assert t.prefix.tolist() == [[0, 7 * 16]]
    w = S.make([(0, reqs(4, own=50))], dev=DEV)
    _, t = parity(w)
    assert t.prefix.tolist() == [[0, 0]]
    w = S.make([(0, [(700, 3)])], dev=DEV)
    _, t = parity(w)
    assert t.prefix.tolist() == [[0, 697 // 16 * 16]] and int(t.own_len) == 700 - 697 // 16 * 16


def test_shares_of_tables_out_of_range():
    w = S.make([(12, reqs(3, own=50)), (4, reqs(2))], dev=DEV)
    for b in range(3):
        w.page_table[w.kv_indptr[b] + 5] = w.pages
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 2), S.device_tables(w)
    B.pda_share_tables(sh.plan, *S.args(t), sh.scratch)
    (prefix, ptr, own), status = S.share(w)
    assert t.prefix.reshape(-1).tolist() == prefix and prefix[:2] == [0, 80]
    assert t.own_indptr.tolist() == ptr and t.own_len.tolist() == own and sh.status() == status


def test_requests_without_rows_and_invalid_ones():
    """They take no part in the prefix; the invalid ones' rows are left as they were."""
    rs = [(40, 1), (30, 2), (50, 1), (20, 0), (33, 1)]
    w = S.make([(10, rs)], dev=DEV)
    w.kv_len[1] = 1                   # fewer tokens than rows
    w.params.max_kv_len = 205
    w.kv_len[2] = 206                 # above the plan
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 1), S.device_tables(w)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    (prefix, ptr, own), status = S.share(w)
    assert t.prefix.reshape(-1).tolist() == prefix and prefix[1] == 160
    assert t.own_indptr.tolist() == ptr and t.own_len.tolist() == own
    assert own[1:4] == [-1, -1, 0]
    assert status == B.PDA_STATUS_KV_LEN_LT_ROWS | B.PDA_STATUS_KV_LEN_GT_MAX and sh.status() == status
    o, ob, l, lb = S.attention(w)
    o[3], l[3] = math.nan, math.nan   # request 2's row
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")


def test_more_own_tokens_than_planned():
    w = S.make([(10, [(40, 1), (90, 1), (64, 1)])], dev=DEV)
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 1, 64), S.device_tables(w)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    assert sh.status() == B.PDA_STATUS_KV_LEN_GT_MAX
    o, ob, l, lb = S.attention(w)
    o[1], l[1] = math.nan, math.nan
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")


def test_groups_out_of_range():
    w = S.make([(4, reqs(2)), (5, reqs(3))], dev=DEV)
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 2), S.device_tables(w)
    t.group_indptr = S.ints([0, 2, 9], DEV)
    B.pda_share_tables(sh.plan, *S.args(t), sh.scratch)
    assert sh.status() == B.PDA_STATUS_TABLE_INVALID
    assert t.prefix[1].tolist() == [-9, -9] and t.own_len[2:].tolist() == [-9] * 3
    assert t.prefix[0].tolist() == [0, 64]


@pytest.mark.parametrize("max_kv", [1000, 4000])  # own tokens by one kernel; by pda_decode's
@pytest.mark.parametrize("page", [8, 16, 64])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 128), ("bf16", 256), ("int8_tensor", 64),
                                      ("e4m3_tensor", 256)])
def test_windows_leave_pages_behind(kind, dim, page, max_kv):
    """Pages in front of every row's window may hold anything, as after they were freed."""
    rs = [(70, 1), (33, 2), (200, 1), (90, 3)]
    w = S.make([(600 // page, rs), (200 // page, rs)], kind=kind, dim=dim, page=page, dev=DEV,
               windows=[100, 333, 230, 95, 40, 35, 52, 150])
    w.params.max_kv_len = max_kv
    seen = set()
    for b, n in enumerate(w.kv_len):
        low = max(0, n - w.rows[b] - w.windows[b] + 1)
        seen.update(w.tables[b][low // page:])
    gone = [i for i in range(w.pages) if i not in seen]
    assert len(gone) > 300 // page
    for c, s in zip(w.cache, w.scale):
        c[gone] = -128 if c.dtype is torch.int8 else 0x7f if c.dtype is torch.uint8 else math.nan
        if s is not None and s.dim() > 1:
            s[gone] = math.nan
    parity(w)


@pytest.mark.parametrize("own", [300, 0])
@pytest.mark.parametrize("bounds", [[0, 2, 4], [1, 3, 6], [0, 2, 9], [0, 3, 2], [-1, 3, 6], [5, 6, 6]])
def test_requests_of_no_group(bounds, own):
    """What the last step left in the tables is not decoded for them."""
    w = S.make([(9, reqs(3)), (12, reqs(3))], dev=DEV)
    w.params.max_kv_len = 4000
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 2, own), S.device_tables(w)
    S.run(w, sh, t)
    torch.cuda.synchronize()
    assert sh.status() == 0
    t.group_indptr = S.ints(bounds, DEV)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    assert sh.status() == B.PDA_STATUS_TABLE_INVALID
    o, ob, l, lb = S.attention(w)
    valid = [a >= 0 and b >= a and b <= 6 for a, b in zip(bounds, bounds[1:])]
    for b in range(6):
        if not any(ok and x <= b < y for ok, x, y in zip(valid, bounds, bounds[1:])):
            o[b], l[b] = math.nan, math.nan
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")


def test_prefixes_that_are_not_of_the_tables():
    """A prefix longer than any request may be is not read."""
    w = S.make([(9, reqs(3)), (12, reqs(3))], dev=DEV)
    w.params.max_kv_len = 4000
    dec = B.Decoder(w.params, device=DEV)
    for own in (100, 0):
        sh, t = B.Shared(dec.plan, 2, own), S.device_tables(w)
        S.run(w, sh, t)
        t.prefix[1] = S.ints([0, 2 ** 31 - 1], DEV)
        out, lse = S.run(w, sh, t, share=False)
        torch.cuda.synchronize()
        assert sh.status() == B.PDA_STATUS_TABLE_INVALID
        o, ob, l, lb = S.attention(w)
        o[3:], l[3:] = math.nan, math.nan
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")


def test_no_lse_and_fewer_rows_than_planned():
    w = S.make([(20, reqs(5, rows=2))], dev=DEV)
    w.params.max_q_len, w.params.max_batch, w.params.batch = 8, 16, 5
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 1), S.device_tables(w)
    out, _ = S.run(w, sh, t, lse=False)
    o, ob, _, _ = S.attention(w)
    check(out, o, ob, "out")
    assert sh.status() == 0


def test_same_as_decode_of_everything():
    """Within both bounds of pda_decode on the whole contexts."""
    w = S.make([(60, reqs(12, own=200, rows=4))], dev=DEV, hkv=2, group=8)
    sh, t = parity(w)
    dec = B.Decoder(w.params, device=DEV)
    out = torch.empty(w.q.shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(w.q.shape[:2], device=DEV)
    B.pda_decode(dec.plan, w.q, *w.cache, t.page_table, t.kv_indptr, t.kv_len, t.qo_indptr, max(w.rows),
                 None, w.dim ** -0.5, None, None, out, lse, dec.scratch)
    o, ob, l, lb = S.attention(w)
    check(out, o, ob, "out of pda_decode")
    check(lse, l, lb, "lse of pda_decode")


def test_calls_repeat_bit_for_bit():
    w = S.make([(200, reqs(20, own=300, rows=2)), (7, reqs(3))], dev=DEV, kind="e4m3_token")
    sh, t = parity(w)
    a = S.run(w, sh, t)
    b = S.run(w, sh, t, share=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dim", [128, 256])
def test_far_pages(dim):
    """Pages whose offsets pass 32 bits, in a cache of 9.4 GB a side."""
    page, hkv = 256, 8
    pages = (9 << 30) // (page * hkv * dim * 2)
    w = S.make([(3, reqs(4, own=500))], dim=dim, page=page, hkv=hkv, group=2, dev="cpu", seed=1)
    w.dev = DEV
    w.q = w.q.to(DEV)
    n = w.pages
    far = {i: pages - 1 - 3 * i for i in range(n)}
    big = []
    for c in w.cache:
        x = torch.empty(pages, *c.shape[1:], dtype=c.dtype, device=DEV)
        for i, at in far.items():
            x[at] = c[i].to(DEV)
        big.append(x)
    w.cache, w.params.num_pages = big, pages
    near = w.page_table
    w.page_table = [far[i] for i in near]
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 1), S.device_tables(w)
    out, lse = S.run(w, sh, t)
    assert t.prefix.tolist() == [[0, 3 * page]] and sh.status() == 0
    o, ob, l, lb = S.attention(w)
    check(out, o, ob, "out")
    check(lse, l, lb, "lse")


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 128), ("bf16", 256), ("int8_tensor", 64)])
def test_waits_that_run_out(kind, dim):
    """Loads withheld: the call ends with its status, and the next one is a normal one."""
    w = S.make([(30, reqs(5))], kind=kind, dim=dim, dev=DEV)
    w.params.wait_limit_us, w.params.inject = 2000, B.PDA_INJECT_WITHHOLD_KV
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 1), S.device_tables(w)
    S.run(w, sh, t)
    torch.cuda.synchronize()
    assert sh.status() & B.PDA_STATUS_WAIT_TIMEOUT
    sh.reset_status()
    w.params.wait_limit_us = w.params.inject = 0
    plan = B.pda_shared_plan(B.pda_plan(w.params)[0], 1)[0]
    sh.plan = plan
    parity(w, shared=sh)
