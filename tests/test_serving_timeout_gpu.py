"""The bounded pipeline waits of the latent-attention kernels run out without
a device fault.

As for the decode's stage 1: the host sets a PDA_INJECT_WITHHOLD_* hook, the
loads it names are never issued, and a short wait limit makes their consumers
give up. What was issued has landed by then (milliseconds against
microseconds) and is drained before a CTA leaves. The call returns with
PDA_STATUS_WAIT_TIMEOUT, and the next normal call on the same scratch is
right. Nothing faults, traps or spins without a bound.
"""
from __future__ import annotations


import pytest
import torch

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
LIMIT_US = 2000


def decoders(heads, inject, **kw):
    """(a decoder whose calls withhold loads, a normal one) over one scratch."""
    p = ref.mla_plan(heads, **kw)
    good = B.Decoder(p, device=DEV)
    p.inject, p.wait_limit_us = inject, LIMIT_US
    bad = B.Decoder(p, device=DEV)
    bad.scratch = good.scratch
    return bad, good


def timed_out(dec):
    """Whether the call ended in a timeout and nothing else; the status is cleared."""
    torch.cuda.synchronize()  # every wait was bounded: the kernel returned
    bits = dec.status()
    dec.reset_status()
    return bits == B.PDA_STATUS_WAIT_TIMEOUT


def close(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err - bound).max()):.3e} past its bound"


# one (head, row tile) pair, all of K in flight at once / a few / many with two stages
@pytest.mark.parametrize("rows,heads", [(1, 1), (5, 128), (300, 128)])
def test_project_times_out(rows, heads):
    g = torch.Generator().manual_seed(rows)
    bad, good = decoders(heads, B.PDA_INJECT_WITHHOLD_KV)
    o = torch.randn(rows, heads, 512, generator=g).to(torch.bfloat16)
    w = (torch.randn(heads, 128, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16)
    do, dw = o.to(DEV), w.to(DEV)
    out = torch.full((rows, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    B.pda_mla_project(bad.plan, do, dw, out, None, bad.scratch)
    assert timed_out(bad)
    assert bool((out == 7).all())
    B.pda_mla_project(good.plan, do, dw, out, None, good.scratch)
    torch.cuda.synchronize()
    assert good.status() == 0
    x, mag = ref.product(o, w)
    mag = mag * ref.sum_bound(512)
    close(out, x, mag + ref.BF16_HALF * (x.abs() + mag), "after the timeout")


def absorb_case(kind, rows, heads):
    g = torch.Generator().manual_seed(rows)
    q = torch.randn(rows, heads, 192, generator=g).to(torch.bfloat16)
    w = (torch.randn(heads, 128, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16)
    out = torch.full((rows, heads, 576), 77, device=DEV,
                     dtype=torch.bfloat16 if kind == "bf16" else torch.uint8)
    return q, w, out


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,heads", [(1, 1), (200, 16)])
def test_absorb_times_out(rows, heads, kind):
    bad, good = decoders(heads, B.PDA_INJECT_WITHHOLD_KV, kind=kind)
    q, w, out = absorb_case(kind, rows, heads)
    dq, dw = q.to(DEV), w.to(DEV)
    B.pda_mla_absorb(bad.plan, dq, dw, 0.011, out, None, bad.scratch)
    assert timed_out(bad)
    assert bool((out[..., :512] == 77).all())
    B.pda_mla_absorb(good.plan, dq, dw, 0.011, out, None, good.scratch)
    torch.cuda.synchronize()
    assert good.status() == 0
    x, mag = ref.product(q[..., :128], w.transpose(1, 2))
    mag = mag * ref.sum_bound(128)
    if kind == "bf16":
        close(out[..., :512], x, mag + ref.BF16_HALF * (x.abs() + mag), "after the timeout")
        assert torch.equal(out[..., 512:].cpu(), q[..., 128:])
    else:
        y = (x / 0.011).clamp(-448, 448)
        mag = mag / 0.011 + 2.0 ** -23 * y.abs()
        close(out[..., :512].view(ref.E4M3).float(), y,
              mag + torch.clamp(ref.E4M3_HALF * (y.abs() + mag), min=ref.E4M3_SUB), "after the timeout")


# Neither CTA of a pair loads; only the leader does (its barriers wait for bytes that do not
# come); only the other does (bytes that were not announced).
@pytest.mark.parametrize("hook", ["WITHHOLD_KV", "WITHHOLD_CTA0", "WITHHOLD_CTA1"])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (300, 3), (1100, 128)])
def test_expand_times_out(tokens, heads, hook):
    g = torch.Generator().manual_seed(tokens)
    page = 64
    pages = -(-tokens // page)
    bad, good = decoders(heads, getattr(B, "PDA_INJECT_" + hook), pages=pages)
    cache = torch.randn(pages, page, 1, 576, generator=g).to(torch.bfloat16)
    w = (torch.randn(heads, 256, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16)
    dcache, dw = cache.to(DEV), w.to(DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)
    ptr, tok = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (pages, tokens))
    latent = torch.zeros(tokens, 576, dtype=torch.bfloat16, device=DEV)
    kv = torch.full((tokens, heads, 256), 7.0, dtype=torch.bfloat16, device=DEV)

    def run(dec):
        B.pda_mla_expand(dec.plan, dcache, table, ptr, tok, None, dw[:, :128], dw[:, 128:], latent,
                         kv[..., :128], kv[..., 128:], dec.scratch)

    run(bad)
    assert timed_out(bad)
    assert bool((kv == 7).all())
    run(good)
    torch.cuda.synchronize()
    assert good.status() == 0
    x = cache.reshape(-1, 576)[:tokens]
    assert torch.equal(latent.cpu(), x)
    some = slice(0, tokens, 37)  # every 37th token, all heads
    y, mag = ref.product(x[some, None, :512].expand(-1, heads, 512), w)
    mag = mag * ref.sum_bound(512)
    close(kv[some], y, mag + ref.BF16_HALF * (y.abs() + mag), "after the timeout")


# Keys in one chunk (out and lse stay unwritten) and in several; a last tile that is cleared
# behind the last key, and none. The work counters of the scratch have to survive.
@pytest.mark.parametrize("reqs,heads,chunks", [
    ([(1, 1)], 1, False), ([(300, 300), (5, 128)], 2, False), ([(7, 130)] * 40, 16, False),
    ([(40, 3000)], 2, True), ([(3, 1024), (1, 900)], 4, True)])
def test_prefill_times_out(reqs, heads, chunks):
    g = torch.Generator().manual_seed(heads)
    qo, tok = [0], [0]
    for r, n in reqs:
        qo.append(qo[-1] + r)
        tok.append(tok[-1] + n)
    rows, toks = qo[-1], tok[-1]
    bad, good = decoders(heads, B.PDA_INJECT_WITHHOLD_KV, batch=len(reqs),
                         max_kv=max(n for _, n in reqs))
    pre = [B.Prefill(dec.plan, rows, toks, device=DEV) for dec in (bad, good)]
    pre[1].scratch = pre[0].scratch
    assert (pre[0].plan.splits > 1) == chunks
    q = torch.randn(rows, heads, 192, generator=g).to(torch.bfloat16)
    kv = torch.randn(toks, heads, 256, generator=g).to(torch.bfloat16)
    rope = torch.randn(toks, 64, generator=g).to(torch.bfloat16)
    dq, dkv, drope = q.to(DEV), kv.to(DEV), rope.to(DEV)
    dqo, dtok = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (qo, tok))
    out = torch.full((rows, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows, heads), 7.0, device=DEV)

    def run(p):
        p.run(dq, dkv[..., :128], dkv[..., 128:], drope, dqo, dtok, 192 ** -0.5, out, lse)

    for _ in range(2):
        run(pre[0])
        assert timed_out(pre[0])
        if not chunks:
            assert bool((out == 7).all()) and bool((lse == 7).all())
    for _ in range(2):
        run(pre[1])
        torch.cuda.synchronize()
        assert pre[1].status() == 0
    o, ob, l_, lb = ref.attention(q, kv[..., :128], kv[..., 128:], rope, qo, tok, causal=True,
                                  windows=None, scale=192 ** -0.5)
    close(out, o, ob, "out after the timeout")
    close(lse, l_, lb, "lse after the timeout")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,heads", [(1, 1), (200, 16)])
def test_absorb_writes_nothing_after_a_timeout(rows, heads, kind):
    """The rope channels, which pass through, are left unwritten with the rest."""
    bad, _ = decoders(heads, B.PDA_INJECT_WITHHOLD_KV, kind=kind)
    q, w, out = absorb_case(kind, rows, heads)
    B.pda_mla_absorb(bad.plan, q.to(DEV), w.to(DEV), 0.011, out, None, bad.scratch)
    assert timed_out(bad)
    assert bool((out == 77).all())
