"""Where decode behind shared prefixes ends what it reads: lists that part while other warps
compare them, requests of no group, bounds of groups that fall, pages behind every window, and
rows that are not their group's."""
from __future__ import annotations

import math
import random
import types

import pytest
import torch

import pages_ref as ref
import shared_ref as S
from paged_split_kv_03_gb300 import binding as B
from test_shared_gpu import check, parity, reqs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("groups", [1, 7])
def test_lists_that_part_while_others_compare(groups):
    """Every request parts from the first one in a stretch of its own, so that the shared length
    falls all the while; each call finds the same."""
    cols, n = 2600, 36 * groups
    r = random.Random(groups)
    page = list(range(cols))
    lists, starts = [], []
    for b in range(n):
        mine = list(page)
        if b % 36:
            at = r.randrange(900, cols)
            mine[at] = 4000 + b
            starts.append(at)
        lists.append(mine)
    table = sum(lists, [])
    ptr, lens, qo = [cols * k for k in range(n + 1)], [16 * cols] * n, list(range(n + 1))
    bounds = [36 * g for g in range(groups + 1)]
    p = ref.plan_params("bf16", heads=1, dim=64, pages=5000, batch=n, max_kv=16 * cols)
    dec = B.Decoder(p, device=DEV)
    sh = B.Shared(dec.plan, groups, 0)
    t = types.SimpleNamespace(page_table=ints(table), kv_indptr=ints(ptr), kv_len=ints(lens), qo_indptr=ints(qo),
                              window=None, group_indptr=ints(bounds), prefix=ints([[-9, -9]] * groups),
                              own_indptr=ints([-9] * n), own_len=ints([-9] * n))
    want = [[0, 16 * min(starts[35 * g:35 * g + 35])] for g in range(groups)]
    for _ in range(50):
        t.prefix.fill_(-9)
        B.pda_share_tables(sh.plan, *S.args(t), sh.scratch)
        assert t.prefix.tolist() == want
    assert sh.status() == 0


@pytest.mark.parametrize("own", [300, 0])  # own tokens by one kernel; by pda_decode's stage 1
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("bf16", 64), ("e4m3_token", 256)])
@pytest.mark.parametrize("bounds", [[0, 2, 4], [1, 3, 6], [0, 3, 2], [-1, 3, 6], [5, 6, 6], [7, 9, 8]])
def test_places_of_requests_of_no_group_are_not_looked_up(bounds, kind, dim, own):
    """No step has written their lengths and places: what stands there leads to page ids out of
    range (and would be seen in the status), and is left as it is."""
    w = S.make([(9, reqs(3)), (12, reqs(3))], kind=kind, dim=dim, dev=DEV)
    w.params.max_kv_len = 4000
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 2, own), S.device_tables(w)
    t.page_table = ints(w.page_table + [w.pages + 7] * 40)
    t.group_indptr = ints(bounds)
    t.own_indptr.fill_(len(w.page_table))
    t.own_len.fill_(30)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    o, ob, l, lb = S.attention(w)
    valid = [(x, y) for x, y in zip(bounds, bounds[1:]) if 0 <= x <= y <= 6]
    for b in range(6):
        if not any(x <= b < y for x, y in valid):
            o[b], l[b] = math.nan, math.nan
            assert int(t.own_len[b]) == 30 and int(t.own_indptr[b]) == len(w.page_table)
    if valid:
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")
    else:
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    assert sh.status() == B.PDA_STATUS_TABLE_INVALID


@pytest.mark.parametrize("own", [300, 0])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("bounds", [
    [0, 5, 3, 6], [0, 3, 2, 6], [0, 6, 0, 6], [4, 6, 0, 4], [3, 3, 0, 6], [0, 3, 2, 3, 6], [0, 2, 9, 2, 6],
    [0] * 20 + [3, 2] + [3] * 20 + [6], [0] * 70 + [5, 4, 5] + [5] * 70 + [6], [1] * 40 + [0] * 40 + [6]])
def test_groups_that_would_list_the_same_requests(bounds, dim, own):
    """Of two groups with a request in common the later one is not decoded, and its requests'
    places are left alone."""
    w = S.make([(9, reqs(3)), (12, reqs(3))], dim=dim, dev=DEV)
    w.params.max_kv_len = 4000
    dec = B.Decoder(w.params, device=DEV)
    groups = len(bounds) - 1
    sh, t = B.Shared(dec.plan, groups, own), S.device_tables(w)
    t.group_indptr, t.prefix = ints(bounds), ints([[-9, -9]] * groups)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    assert sh.status() == B.PDA_STATUS_TABLE_INVALID
    o, ob, l, lb = S.attention(w)
    valid = [0 <= x <= y <= 6 and x >= max(bounds[:g + 1]) for g, (x, y) in enumerate(zip(bounds, bounds[1:]))]
    listed = [b for b in range(6)
              if any(ok and x <= b < y for ok, x, y in zip(valid, bounds, bounds[1:]))]
    assert [row[1] == -9 for row in t.prefix.tolist()] == [not ok for ok in valid]
    assert [b for b in range(6) if int(t.own_len[b]) != -9] == listed
    for b in set(range(6)) - set(listed):
        o[b], l[b] = math.nan, math.nan
    if listed:
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")
    else:
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("max_kv", [1000, 4000])  # own tokens by one kernel; by pda_decode's
@pytest.mark.parametrize("left", [1e-39, 1e-45, math.inf, -1.0, 0.0])
@pytest.mark.parametrize("kind,dim", [("e4m3_token", 64), ("e4m3_token", 128), ("int8_token", 128),
                                      ("e4m3_token", 256)])
def test_scales_of_pages_behind_every_window(kind, dim, left, max_kv):
    """What is left in the scales of pages that no row sees counts for nothing."""
    page = 16
    rs = [(70, 1), (33, 2), (200, 1), (90, 3)]
    w = S.make([(40, rs), (13, rs)], kind=kind, dim=dim, page=page, dev=DEV,
               windows=[100, 333, 230, 95, 40, 35, 52, 150])
    w.params.max_kv_len = max_kv
    seen = set()
    for b, n in enumerate(w.kv_len):
        low = max(0, n - w.rows[b] - w.windows[b] + 1)
        seen.update(w.tables[b][low // page:])
    gone = [i for i in range(w.pages) if i not in seen]
    assert len(gone) > 18
    for s in w.scale:
        s[gone] = left
    parity(w)


@pytest.mark.parametrize("own", [300, 0])
@pytest.mark.parametrize("dim", [128, 256])
def test_rows_outside_their_group(dim, own):
    """A request of fewer than no rows takes those of the one in front out of the group's: they
    are left alone, and not decoded without the prefix."""
    w = S.make([(9, [(30, 3), (20, 1)]), (4, [(30, 1)])], dim=dim, dev=DEV)
    w.qo, w.rows = [0, 3, 1, 1], [3, -2, 0]
    w.params.max_kv_len = 4000
    dec = B.Decoder(w.params, device=DEV)
    sh, t = B.Shared(dec.plan, 2, own), S.device_tables(w)
    t.qo_indptr = ints(w.qo)
    out, lse = S.run(w, sh, t)
    torch.cuda.synchronize()
    assert t.prefix.tolist()[0] == [0, (174 - 3) // 16 * 16]  # the one valid request's whole pages
    assert sh.status() == B.PDA_STATUS_ROWS_GT_MAX
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
