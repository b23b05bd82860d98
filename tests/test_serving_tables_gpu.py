"""Block tables at the ends of their types: token offsets that pass int32."""
from __future__ import annotations

import pytest
import torch

from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


@pytest.mark.parametrize("grow,first", [(96, 3), (97, 2)])
def test_token_offsets_past_int32(grow, first):
    """Every request is within max_kv_len, the columns and the capacities; their tokens together
    reach 2^31 - 1 (a request that ends there fits) or pass it: from that request on all are
    listed as empty, and PDA_STATUS_TABLE_FULL is set."""
    page, big = 256, 1 << 30
    cached, new = [big, big - 300, 200, 1000], [1, 2, grow, 1]
    assert sum(cached[:3]) + sum(new[:3]) == (1 << 31) - 1 + (grow - 96)
    have = [-(-c // page) for c in cached]
    want = [-(-(c + n) // page) for c, n in zip(cached, new)]
    cols, cap, free, pages = max(want) + 1, sum(want) + 5, 6, 1000
    p = B.PdaParams(num_qo_heads=1, num_kv_heads=1, head_dim=128, page_size=page, max_batch=4,
                    max_q_len=1, max_kv_len=big + 1, num_pages=pages, kv_stride_page=page * 128,
                    kv_stride_token=128, kv_stride_head=128)
    dec = B.Decoder(p, device=DEV)
    block = torch.randint(0, pages, (4, cols), dtype=torch.int32, device=DEV)
    before = block.clone()
    free_pages = ints([900 + i for i in range(free)])
    kv_len, left = ints([-9] * 4), ints([-9])
    kv_ptr, qo_ptr, tok_ptr = (ints([-9] * 5) for _ in range(3))
    table = torch.full((cap,), -9, dtype=torch.int32, device=DEV)
    slots, pos = ints([-9] * 110, torch.int64), ints([-9] * 110)
    B.pda_build_tables(dec.plan, ints(cached), ints(new), None, block, free_pages, ints([free]), left,
                       kv_len, kv_ptr, table, qo_ptr, tok_ptr, slots, pos, dec.scratch)
    torch.cuda.synchronize()
    assert dec.status() == B.PDA_STATUS_TABLE_FULL
    lens = [c + n if b < first else 0 for b, (c, n) in enumerate(zip(cached, new))]
    npg = [w if b < first else 0 for b, w in enumerate(want)]
    rows = [n if b < first else 0 for b, n in enumerate(new)]

    def indptr(v):
        return [sum(v[:k]) for k in range(5)]

    assert kv_len.tolist() == lens
    assert kv_ptr.tolist() == indptr(npg)
    assert qo_ptr.tolist() == indptr(rows)
    assert tok_ptr.tolist() == indptr(lens)
    taken = 0
    for b in range(4):
        grown = want[b] - have[b] if b < first else 0
        ids = [900 + free - 1 - taken - k for k in range(grown)]
        taken += grown
        row = before[b].clone()
        if grown:
            row[have[b]:want[b]] = ints(ids)
        assert torch.equal(block[b], row), b
        at = indptr(npg)[b]
        assert torch.equal(table[at:at + npg[b]], row[:npg[b]]), b
        for i in range(rows[b]):
            t = cached[b] + i
            assert slots[indptr(rows)[b] + i].item() == row[t // page].item() * page + t % page
            assert pos[indptr(rows)[b] + i].item() == t
    assert left.item() == free - taken
    assert bool((table[sum(npg):] == -9).all()) and bool((pos[sum(rows):] == -9).all())


@pytest.mark.parametrize("cols,cap", [(3, 8), (3, 0), (0, 8), (0, 0)])
def test_arrays_without_entries(cols, cap):
    """A free list, block table or page table of no entries (torch gives such tensors no
    address): requests that need no page are listed, the others refused."""
    p = B.PdaParams(num_qo_heads=1, num_kv_heads=1, head_dim=128, page_size=16, max_batch=3,
                    max_q_len=1, max_kv_len=100, num_pages=10, kv_stride_page=16 * 128,
                    kv_stride_token=128, kv_stride_head=128)
    dec = B.Decoder(p, device=DEV)
    block = torch.full((3, cols), 7, dtype=torch.int32, device=DEV)
    kv_len, left = ints([-9] * 3), ints([-9])
    kv_ptr, qo_ptr, tok_ptr = (ints([-9] * 4) for _ in range(3))
    table = torch.full((cap,), -9, dtype=torch.int32, device=DEV)
    slots, pos = ints([], torch.int64), ints([])
    B.pda_build_tables(dec.plan, ints([16, 0, 0]), ints([0, 0, 5]), None, block, ints([]), ints([0]),
                       left, kv_len, kv_ptr, table, qo_ptr, tok_ptr, slots, pos, dec.scratch)
    torch.cuda.synchronize()
    # request 0 holds a page, request 1 nothing, request 2 wants a page that there is not
    status = (B.PDA_STATUS_NO_PAGES if cols else B.PDA_STATUS_TABLE_INVALID) | \
        (B.PDA_STATUS_TABLE_FULL if cols and not cap else 0)
    assert dec.status() == status
    first = [16, 0, 0] if cols and cap else [0, 0, 0]
    assert kv_len.tolist() == first and tok_ptr.tolist() == [0] + [first[0]] * 3
    assert kv_ptr.tolist() == [0] + [1 if first[0] else 0] * 3
    assert qo_ptr.tolist() == [0] * 4 and left.item() == 0
    assert table.tolist() == ([7] + [-9] * 7 if first[0] else [-9] * cap)
