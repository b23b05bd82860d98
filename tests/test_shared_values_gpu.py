"""GPU outputs of decode behind shared prefixes over marked values, within a bound that every page
or tile of V out of place breaks (test_shared_values_host.py)."""
from __future__ import annotations

import pytest
import torch

import shared_ref as S
import values_ref as V
from paged_split_kv_03_gb300 import binding as B
from test_shared_gpu import KINDS, check, reqs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def both_ways(w):
    V.mark(w)
    dec = B.Decoder(w.params, device=DEV)
    (prefix, _, own), status = S.share(w)
    assert status == 0
    ends = [prefix[2 * g + 1] for g in range(len(w.gp) - 1) for _ in range(w.gp[g], w.gp[g + 1])]
    assert max(own) <= 1024 < max(w.kv_len) and max(w.rows) * w.group <= 64
    for most in (max(own), 0):
        sh, t = B.Shared(dec.plan, len(w.gp) - 1, most), S.device_tables(w)
        out, lse = S.run(w, sh, t)
        o, ob, l, lb = V.attention(w, ends, stage1=most == 0)
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")
        assert sh.status() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_every_page_of_a_prefix(kind, dim):
    both_ways(S.make([(300, reqs(5, own=200, rows=2))], kind=kind, dim=dim, dev=DEV, seed=dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", ["e4m3_tensor", "e4m3_token"])
def test_e4m3_query(kind, dim):
    both_ways(S.make([(150, reqs(3, own=90, rows=3))], kind=kind, dim=dim, q8=True, hnd=True, dev=DEV, seed=dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS)
def test_every_page_of_many_items(kind, dim):
    """Several segments a CTA, two row tiles and one, and few of a tile's keys."""
    groups = [(17, reqs(30)), (3, reqs(5)), (40, reqs(9, rows=2)), (1, reqs(1)), (31, reqs(26))]
    both_ways(S.make(groups, kind=kind, dim=dim, page=128, hkv=8, group=3, hnd=True, dev=DEV, spare=1))


@pytest.mark.parametrize("page", [8, 64, 256])
def test_page_sizes(page):
    for kind, dim in (("bf16", 128), ("e4m3_token", 256)):
        both_ways(S.make([(3000 // page, reqs(4, own=70))], kind=kind, dim=dim, page=page, dev=DEV, seed=page))
