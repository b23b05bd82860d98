"""Values in which the products of weights and V show: each page has one large channel of its
own, so that a page, tile or segment of V that is left out, taken twice or taken from another
place moves an output by far more than a correct kernel may be off; and that bound."""
import math

import torch

import shared_ref as S

LARGEST = {"bf16": 64.0, "e4m3": 448.0, "int8": 127.0}
TILE = 128  # keys


def mark(w):
    """Every token and head of page i: the type's largest value (bf16: 64) in channel i % D."""
    kind = w.kind.split("_")[0]
    cache, scale, value = w.cache[1], w.scale[1], w.values[1]
    code = 0x7e if kind == "e4m3" else LARGEST[kind]
    for i in range(w.pages):
        c = i % w.dim
        cache[i, ..., c] = code
        s = 1.0 if scale is None else scale.double().cpu()[0] if scale.dim() == 1 else scale[i].double().cpu()
        if w.hnd and scale is not None and scale.dim() > 1:
            s = s.T  # (scales stand by token, then head)
        value[i, ..., c] = LARGEST[kind] * s
    return w


def used_pages(w):
    return sorted({p for t in w.tables for p in t})


def parts(w, b):
    """(weights, values, logits, |q||k| and so on of request b), keys of each kv head in order."""
    n, rows = w.kv_len[b], w.rows[b]
    ids = torch.tensor(w.tables[b])
    kv = []
    for val in w.values:
        x = val[ids]
        x = x.transpose(0, 1) if w.hnd else x.permute(2, 0, 1, 3)
        kv.append(x.reshape(w.hkv, -1, w.dim)[:, :n])
    q = w.q.cpu().float().double()[w.qo[b]:w.qo[b + 1]].reshape(rows, w.hkv, w.group, w.dim)
    s = torch.einsum("rhgd,hjd->rhgj", q, kv[0]) * w.dim ** -0.5 * w.q_scale
    see = (torch.arange(n)[None] <= n - rows + torch.arange(rows)[:, None])[:, None, None]
    s = s.masked_fill(~see, -math.inf)
    x = torch.logsumexp(s, -1)
    return torch.exp(s - x[..., None]), kv[1], s, x


def attention(w, ends, stage1):
    """(out, bound, lse, lse bound) in 64 bits; ``ends``: where each request's prefix ends;
    ``stage1``: the own tokens by pda_decode's stage 1, else by the kernel of few own tokens.

    The logits' error d is shared_ref's. Weights are rounded before they meet V: to bf16 (2^-8 of
    each) over bf16 caches, to f16 (2^-11, and 2^-25 of the largest below f16's normal range) over
    8-bit ones; only stage 1 over E4M3 takes its tokens' weights as two E4M3 terms (2^-8, and
    2^-10 of its largest). With a scale per token the largest is that of weight x scale: at
    most the scales' ratio more. Sums of n products are fp32, the output is rounded to bf16."""
    out, bound, lse, lbound = S.attention(w)
    bits8 = w.kind != "bf16"
    ratio = 1.0
    if "token" in w.kind:
        s = w.scale[1][used_pages(w)]
        ratio = float(s.max() / s.min())
    for b, n in enumerate(w.kv_len):
        r0, r1, rows = w.qo[b], w.qo[b + 1], w.rows[b]
        p, v, s, x = parts(w, b)
        lb = lbound[r0:r1].reshape(rows, w.hkv, w.group)
        sums = (n + 200) * 2.0 ** -23
        d = lb - sums - 2.0 ** -21 * x.abs()  # (of shared_ref's lse bound)
        a = torch.einsum("rhgj,hjd->rhgd", p, v.abs())
        o = torch.einsum("rhgj,hjd->rhgd", p, v)
        seen = torch.isfinite(s).double()
        bnd = a * ((2.0 ** -11 if bits8 else 2.0 ** -8) + 2 * d[..., None] + sums) + S.BF16_HALF * o.abs()
        if bits8:
            top = torch.exp(s.amax(-1) - x)[..., None]
            bnd = bnd + 2.0 ** -25 * ratio * top * torch.einsum("rhgj,hjd->rhgd", seen, v.abs())
        if bits8 and stage1:
            e = ends[b]
            own, vo = p[..., e:], v[:, e:].abs()
            bnd = bnd + 2.0 ** -8 * torch.einsum("rhgj,hjd->rhgd", own, vo)
            bnd = bnd + 2.0 ** -10 * ratio * own.amax(-1)[..., None] * torch.einsum("rhgj,hjd->rhgd", seen[..., e:], vo)
        bound[r0:r1] = (bnd * 1.01).reshape(rows, w.hq, w.dim)
    return out, bound, lse, lbound


def mistaken(w, what, at):
    """Outputs with a mistake in the products of weights and V, key ``at`` among those it is made with."""
    out = torch.zeros(w.q.shape, dtype=torch.float64)
    for b, n in enumerate(w.kv_len):
        p, v, _, _ = parts(w, b)
        k0 = at // TILE * TILE
        k1 = min(n, k0 + TILE)
        if what == "tile left out":
            p[..., k0:k1] = 0
        elif what == "tile taken twice":
            p[..., k0:k1] *= 2
        elif what == "V of the next tile":
            v = v.clone()
            m = min(k1 - k0, n - k1)
            v[:, k0:k0 + m] = v[:, k1:k1 + m].clone()
        elif what == "page left out":
            g0 = at // w.page * w.page
            p[..., g0:g0 + w.page] = 0
        elif what == "V of another page":
            v = v.clone()
            g0 = at // w.page * w.page
            v[:, g0:g0 + w.page] = v[:, g0 + w.page:g0 + 2 * w.page].clone()
        else:
            assert what == "nothing"
            p = p * 0
        out[w.qo[b]:w.qo[b + 1]] = torch.einsum("rhgj,hjd->rhgd", p, v).reshape(-1, w.hq, w.dim)
    return out
