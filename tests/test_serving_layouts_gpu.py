"""The calls around decode on the layouts that the plan allows beside the dense ones: caches
that are views of larger memory or raw addresses, typed or as bytes, tokens and pages padded."""
from __future__ import annotations

import pytest
import torch

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
PAGE, PAGES, HEADS, TOKENS = 16, 6, 2, 50


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def forms(cache):
    """The same memory as its plan's type, as bytes of either sign, and as an address."""
    return [cache, cache.view(torch.uint8), cache.view(torch.int8), cache.data_ptr()]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_caches_as_views_bytes_and_addresses(kind):
    """A layer's cache inside a pool of layers, given in each form: the same rows go in and
    come out, the layers beside it stay as they were."""
    g = torch.Generator().manual_seed(3)
    dec = B.Decoder(ref.mla_plan(HEADS, kind=kind, page=PAGE, pages=PAGES), device=DEV)
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    pool = torch.zeros(3, PAGES, PAGE, 1, 576, dtype=torch.uint8, device=DEV).to(dt)
    scale = None if kind == "bf16" else torch.tensor([0.02], device=DEV)
    x = torch.randn(TOKENS, 1, 576, generator=g).to(torch.bfloat16).to(DEV)
    slots = torch.randperm(PAGE * PAGES, generator=g)[:TOKENS].to(DEV)
    table, ptr, tok = ints(*range(PAGES)), ints(0, PAGES), ints(0, PAGE * PAGES)
    w = (torch.randn(HEADS, 256, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16).to(DEV)
    seen = []
    for cache in forms(pool[1]):
        pool.view(torch.uint8).fill_(0)
        B.pda_append_slots(dec.plan, x, None, slots, None, cache, None, scale, None, dec.scratch)
        latent = torch.full((PAGE * PAGES, 576), 7.0, dtype=torch.bfloat16, device=DEV)
        kv = torch.empty(PAGE * PAGES, HEADS, 256, dtype=torch.bfloat16, device=DEV)
        B.pda_mla_expand(dec.plan, cache, table, ptr, tok, scale, w[:, :128], w[:, 128:], latent,
                         kv[..., :128], kv[..., 128:], dec.scratch)
        torch.cuda.synchronize()
        assert dec.status() == 0
        assert int(torch.count_nonzero(pool.view(torch.uint8)[0::2])) == 0
        seen.append((pool.view(torch.uint8).cpu().clone(), latent.cpu(), kv.cpu()))
    if kind == "bf16":
        assert torch.equal(seen[0][1][slots.cpu()], x[:, 0].cpu())
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def test_expand_tokens_behind_their_pages():
    """A request with more tokens than its entries of the page table hold: the rest reads as
    zeros, not as the next request's pages, and says so."""
    g = torch.Generator().manual_seed(4)
    dec = B.Decoder(ref.mla_plan(HEADS, page=PAGE, pages=PAGES, batch=3), device=DEV)
    cache = torch.randn(PAGES, PAGE, 1, 576, generator=g).to(torch.bfloat16)
    table = [4, 1, 3, 0, 2]
    tok = [0, 2 * PAGE + 5, 3 * PAGE + 5, 3 * PAGE + 25]  # requests of 2, 1 and 2 pages
    latent = torch.full((tok[3], 576), 7.0, dtype=torch.bfloat16, device=DEV)
    kv = torch.full((tok[3], HEADS, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    w = torch.randn(HEADS, 256, 512, generator=g).to(torch.bfloat16).to(DEV)
    B.pda_mla_expand(dec.plan, cache.to(DEV), ints(*table), ints(0, 2, 3, 5), ints(*tok), None,
                     w[:, :128], w[:, 128:], latent, kv[..., :128], kv[..., 128:], dec.scratch)
    torch.cuda.synchronize()
    assert dec.status() == B.PDA_STATUS_PAGE_OOB
    want = torch.cat([cache[4, :, 0], cache[1, :, 0], torch.zeros(5, 576, dtype=torch.bfloat16),
                      cache[3, :, 0], cache[0, :, 0], cache[2, :4, 0]])
    assert torch.equal(latent.cpu(), want)
    assert bool((kv[2 * PAGE:2 * PAGE + 5] == 0).all())
    assert not bool((kv == 7).all(-1).any())  # every row was written


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_token", "records"])
def test_latent_cache_with_padded_tokens_and_pages(kind):
    """Tokens and pages further apart than their data: what lies between is neither read nor
    written, and the rows are those of the dense cache."""
    g = torch.Generator().manual_seed(5)
    width = 640 if kind == "records" else 576
    x = torch.randn(TOKENS, 1, 576, generator=g).to(torch.bfloat16).to(DEV)
    slots = torch.randperm(PAGE * PAGES, generator=g)[:TOKENS].to(DEV)
    w = (torch.randn(HEADS, 256, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16).to(DEV)
    table, ptr, tok = ints(*reversed(range(PAGES))), ints(0, PAGES), ints(0, PAGE * PAGES)
    seen = []
    for tpad, ppad in ((0, 0), (16, 0), (64, 48)):
        p = ref.mla_plan(HEADS, kind=kind, page=PAGE, pages=PAGES)
        p.kv_stride_token = p.kv_stride_head = width + tpad
        p.kv_stride_page = PAGE * (width + tpad) + ppad
        dec = B.Decoder(p, device=DEV)
        dt = torch.bfloat16 if kind == "bf16" else torch.uint8
        # (0x7F7F is a NaN in bf16, 0x7F one in E4M3)
        whole = torch.full((PAGES * p.kv_stride_page * (2 if kind == "bf16" else 1),), 0x7F,
                           dtype=torch.uint8, device=DEV)
        cache = whole.view(dt).as_strided((PAGES, PAGE, 1, width),
                                          (p.kv_stride_page, width + tpad, width + tpad, 1))
        cache.zero_()
        scale = torch.tensor([0.02], device=DEV) if kind == "e4m3" else \
            torch.ones(PAGES, PAGE, 1, device=DEV) if kind == "e4m3_token" else \
            torch.ones(PAGES, PAGE, 1, 4, device=DEV) if kind == "records" else None
        B.pda_append_slots(dec.plan, x, None, slots, None, cache, None, scale, None, dec.scratch)
        latent = torch.full((PAGE * PAGES, 576), 7.0, dtype=torch.bfloat16, device=DEV)
        kv = torch.empty(PAGE * PAGES, HEADS, 256, dtype=torch.bfloat16, device=DEV)
        B.pda_mla_expand(dec.plan, cache, table, ptr, tok, scale, w[:, :128], w[:, 128:], latent,
                         kv[..., :128], kv[..., 128:], dec.scratch)
        torch.cuda.synchronize()
        assert dec.status() == 0
        between = torch.ones_like(whole, dtype=torch.bool)
        between.view(dt if dt is torch.uint8 else torch.int16).as_strided(cache.shape, cache.stride()).zero_()
        assert bool((whole[between] == 0x7F).all())
        seen.append((cache.contiguous().view(torch.uint8).cpu(), latent.cpu(), kv.cpu(),
                     None if scale is None else scale.cpu()))
    for other in seen[1:]:
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(seen[0], other))


def test_scales_of_other_number_types():
    """Scales as numpy numbers or torch scalars, as pda_decode takes them."""
    import numpy as np
    g = torch.Generator().manual_seed(6)
    dec = B.Decoder(ref.mla_plan(HEADS, kind="e4m3", max_kv=TOKENS), device=DEV)
    pre = B.Prefill(dec.plan, 3, TOKENS)
    w = torch.randn(HEADS, 128, 512, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(3, HEADS, 192, generator=g).to(torch.bfloat16).to(DEV)
    kv = torch.randn(TOKENS, HEADS, 256, generator=g).to(torch.bfloat16).to(DEV)
    rope = torch.randn(TOKENS, 64, generator=g).to(torch.bfloat16).to(DEV)
    seen = []
    for scale in (0.0625, np.float32(0.0625), np.float64(0.0625), torch.tensor(0.0625)):
        q_lat = torch.zeros(3, HEADS, 576, dtype=torch.uint8, device=DEV)
        out = torch.zeros(3, HEADS, 128, dtype=torch.bfloat16, device=DEV)
        B.pda_mla_absorb(dec.plan, q, w, scale, q_lat, None, dec.scratch)
        pre.run(q, kv[..., :128], kv[..., 128:], rope, ints(0, 3), ints(0, TOKENS), scale, out, None)
        seen.append((q_lat.cpu(), out.cpu()))
    assert int(torch.count_nonzero(seen[0][0])) and int(torch.count_nonzero(seen[0][1]))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))
