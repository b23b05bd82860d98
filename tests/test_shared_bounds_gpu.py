"""Where decode behind shared prefixes ends what it reads: lists that part while other warps
compare them."""
from __future__ import annotations

import random
import types

import pytest
import torch

import pages_ref as ref
import shared_ref as S
from paged_split_kv_03_gb300 import binding as B

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
