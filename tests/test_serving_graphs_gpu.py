"""The calls around decode captured into CUDA graphs: replays with other inputs, lengths and
row counts in the same memory give, bit for bit, what eager calls give."""
from __future__ import annotations

import pytest
import torch

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def capture(call):
    """A graph of one call, after an eager one on the capture's stream."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    return g


def same(call, graph, outs, fills, what):
    """The replay writes what the eager call writes, rows left alone included."""
    got = []
    for run in (graph.replay, call):
        for t in outs:
            t.view(torch.uint8).fill_(0x11)
        for fill in fills:
            fill()
        run()
        torch.cuda.synchronize()
        got.append([t.view(torch.uint8).cpu().clone() for t in outs])
    for a, b in zip(*got):
        assert torch.equal(a, b), what
    return got[0]


def rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,heads", [(3, 4), (300, 16), (200, 128)])
def test_products(rows, heads, kind):
    g = torch.Generator().manual_seed(rows)
    dec = B.Decoder(ref.mla_plan(heads, kind=kind), device=DEV)
    w = rand(g, heads, 256, 512, std=512 ** -0.5)
    q, o_lat = rand(g, rows, heads, 192), rand(g, rows, heads, 512)
    n = torch.tensor([rows], dtype=torch.int32, device=DEV)
    q_lat = torch.empty(rows, heads, 576, dtype=torch.bfloat16 if kind == "bf16" else torch.uint8,
                        device=DEV)
    out = torch.empty(rows, heads, 128, dtype=torch.bfloat16, device=DEV)

    def call():
        B.pda_mla_absorb(dec.plan, q, w[:, :128], 0.01, q_lat, n, dec.scratch)
        B.pda_mla_project(dec.plan, o_lat, w[:, 128:], out, n, dec.scratch)

    graph = capture(call)
    for live in (rows, 1, 0, rows // 2 + 1):
        n.fill_(live)
        for t in (q, o_lat, w):
            t.copy_(rand(g, *t.shape, std=0.3))
        got = same(call, graph, (q_lat, out), (), f"{live} rows")
        untouched = [t.reshape(rows, -1)[live:] for t in got]
        assert all(bool((t == 0x11).all()) for t in untouched)
    assert dec.status() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "records"])
def test_append_and_expand(kind):
    """The expansion is two kernels joined by a programmatic launch; behind it, in the same
    graph, the products of the prefill read what both wrote."""
    heads, page, pages, cap, batch = 16, 16, 40, 500, 3
    g = torch.Generator().manual_seed(1)
    dec = B.Decoder(ref.mla_plan(heads, kind=kind, page=page, pages=pages, batch=batch, max_kv=400),
                    device=DEV)
    pre = B.Prefill(dec.plan, 64, cap)
    width, dt = (640, torch.uint8) if kind == "records" else \
        (576, torch.bfloat16 if kind == "bf16" else torch.uint8)
    cache = torch.zeros(pages, page, 1, width, dtype=dt, device=DEV)
    scale = torch.tensor([0.02], device=DEV) if kind == "e4m3" else \
        torch.zeros(pages, page, 1, 4, device=DEV) if kind == "records" else None
    x, w, q = rand(g, cap, 1, 576), rand(g, heads, 256, 512, std=512 ** -0.5), rand(g, 64, heads, 192)
    slots = torch.full((cap,), -1, dtype=torch.int64, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ptr, tok, qo = (torch.zeros(batch + 1, dtype=torch.int32, device=DEV) for _ in range(3))
    latent = torch.empty(cap, 576, dtype=torch.bfloat16, device=DEV)
    kv = torch.empty(cap, heads, 256, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(64, heads, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(64, heads, device=DEV)

    def call():
        B.pda_append_slots(dec.plan, x, None, slots, n, cache, None, scale, None, dec.scratch)
        B.pda_mla_expand(dec.plan, cache, table, ptr, tok, scale, w[:, :128], w[:, 128:], latent,
                         kv[..., :128], kv[..., 128:], dec.scratch)
        pre.run(q, kv[..., :128], kv[..., 128:], latent[:, 512:], qo, tok, 192 ** -0.5, out, lse)

    graph = capture(call)
    for lens, rows in (([300, 17, 100], [30, 17, 1]), ([1, 0, 1], [1, 0, 1]), ([0, 0, 0], [0, 0, 0]),
                       ([16, 383, 64], [3, 60, 1])):
        npg = [-(-k // page) for k in lens]
        ids = torch.randperm(pages, generator=g)[:sum(npg)].int()
        table[:sum(npg)] = ids.to(DEV)
        for t, v in ((ptr, npg), (tok, lens), (qo, rows)):
            t.copy_(torch.tensor([sum(v[:k]) for k in range(batch + 1)], dtype=torch.int32))
        where = [int(ids[sum(npg[:b]) + i // page]) * page + i % page
                 for b in range(batch) for i in range(lens[b])]
        slots[:len(where)] = torch.tensor(where, dtype=torch.int64, device=DEV)
        n.fill_(sum(lens))
        for t in (x, w, q):
            t.copy_(rand(g, *t.shape, std=0.5 if t is not w else 512 ** -0.5))
        clear = [cache.zero_] + ([scale.zero_] if kind == "records" else [])
        got = same(call, graph, (latent, kv, out, lse), clear, f"{lens}")
        assert bool((got[0].reshape(cap, -1)[sum(lens):] == 0x11).all())
        assert bool((got[2].reshape(64, -1)[sum(rows):] == 0x11).all())
        if kind == "bf16" and sum(lens):
            assert torch.equal(got[0].view(torch.bfloat16)[:sum(lens)], x[:sum(lens), 0].cpu())
    assert dec.status() == 0 and pre.status() == 0
