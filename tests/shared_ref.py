"""Workloads of requests that share prefixes, and decode attention over them in 64 bits with a
bound of how far a correct kernel may be off, element by element."""
import math
import types

import torch

import pages_ref as ref
from paged_split_kv_03_gb300 import binding as B

E4M3 = torch.float8_e4m3fn
BF16_HALF = 2.0 ** -8


def make(groups, *, kind="bf16", dim=128, page=16, hkv=2, group=4, hnd=False, q8=False, windows=None,
         seed=0, gap=0, spare=3, k_std=1.0, dev="cpu"):
    """``groups``: [(prefix pages, [(own tokens, rows), ...]), ...]. The cache is filled on the
    device; pages that nobody lists hold NaN (codes: 0x7f)."""
    g = torch.Generator().manual_seed(seed)
    ids, tables, kv_len, rows, gp = [], [], [], [], [0]
    n_pages = sum(p + sum(ref.ceil(o, page) for o, _ in rs) for p, rs in groups) + spare
    perm = torch.randperm(n_pages, generator=g).tolist()
    for p, rs in groups:
        pre = [perm.pop() for _ in range(p)]
        for o, r in rs:
            tables.append(pre + [perm.pop() for _ in range(ref.ceil(o, page))])
            kv_len.append(p * page + o)
            rows.append(r)
        gp.append(gp[-1] + len(rs))
    hq = hkv * group
    w = types.SimpleNamespace(kind=kind, dim=dim, page=page, hkv=hkv, hq=hq, group=group, hnd=hnd, q8=q8,
                              tables=tables, kv_len=kv_len, rows=rows, windows=windows, pages=n_pages,
                              gp=gp, dev=dev)
    w.qo = [0]
    for r in rows:
        w.qo.append(w.qo[-1] + max(0, r))
    w.kv_indptr = [0]
    for t in tables:
        w.kv_indptr.append(w.kv_indptr[-1] + len(t))
    w.page_table = [x for t in tables for x in t]
    q = torch.randn(w.qo[-1], hq, dim, generator=g)
    w.q_scale = 1.0
    if q8:
        w.q_scale = 0.01
        w.q = (q / 0.01).clamp(-448, 448).to(E4M3).to(dev)
    else:
        w.q = q.to(torch.bfloat16).to(dev)
    shape = (n_pages, hkv, page) if hnd else (n_pages, page, hkv)
    unused = perm
    w.cache, w.scale, w.values = [], [], []
    for std in (k_std, 1.0):
        x = torch.randn(*shape, dim, generator=g) * std
        x = x.to(torch.bfloat16).float()
        s = None
        if kind == "bf16":
            c, val = x.to(torch.bfloat16), x.to(torch.bfloat16).double()
        else:
            top = 127.0 if "int8" in kind else 448.0
            s = x.abs().amax(-1, keepdim=True) / top if "token" in kind else (x.abs().amax() / top).reshape(1)
            y = (x / s).clamp(-top, top)
            c = y.round().to(torch.int8) if "int8" in kind else y.to(E4M3)
            val = c.double() * s.double()
            c = c if "int8" in kind else c.view(torch.uint8)
            if "token" in kind:
                s = s[..., 0]
                s = (s.transpose(1, 2) if hnd else s).contiguous()
        for u in unused:
            if c.dtype is torch.uint8:
                c[u] = 0x7f
            elif c.dtype is not torch.int8:
                c[u] = math.nan
            if s is not None and s.dim() > 1:
                s[u] = math.nan
        if gap:
            wide = torch.zeros(*c.shape[:-1], dim + gap, dtype=c.dtype)
            wide[..., :dim] = c
            c = wide
        w.cache.append(c.to(dev))
        w.scale.append(None if s is None else s.float().to(dev))
        w.values.append(val)
    w.params = ref.plan_params(kind, heads=hkv, dim=dim, page=page, pages=n_pages, batch=len(kv_len),
                               max_kv=max(kv_len), max_q=max(1, max(rows)), hq=hq, hnd=hnd, q8=q8,
                               gap=gap)
    return w


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def device_tables(w):
    """The step's arrays on the device, and what pda_share_tables writes."""
    d, n = w.dev, len(w.kv_len)
    return types.SimpleNamespace(
        page_table=ints(w.page_table, d), kv_indptr=ints(w.kv_indptr, d), kv_len=ints(w.kv_len, d),
        qo_indptr=ints(w.qo, d), window=None if w.windows is None else ints(w.windows, d),
        group_indptr=None if len(w.gp) == 2 else ints(w.gp, d),
        prefix=torch.full((len(w.gp) - 1, 2), -9, dtype=torch.int32, device=d),
        own_indptr=ints([-9] * n, d), own_len=ints([-9] * n, d))


def args(t):
    return (t.page_table, t.kv_indptr, t.kv_len, t.qo_indptr, t.window, t.group_indptr, t.prefix,
            t.own_indptr, t.own_len)


def run(w, sh, t, *, sm_scale=None, lse=True, max_q=None, share=True, fill=math.nan):
    """One step: (out, lse) of pda_share_tables and pda_decode_shared."""
    if share:
        B.pda_share_tables(sh.plan, *args(t), sh.scratch)
    out = torch.full(w.q.shape, fill, dtype=torch.bfloat16, device=w.dev)
    ls = torch.full(w.q.shape[:2], fill, device=w.dev) if lse else None
    scale = (w.dim ** -0.5 if sm_scale is None else sm_scale) * w.q_scale
    a = args(t)
    B.pda_decode_shared(sh.plan, w.q, w.cache[0], w.cache[1], *a[:4], max_q or max(w.rows), *a[4:], scale,
                        w.scale[0], w.scale[1], out, ls, sh.scratch)
    return out, ls


def attention(w, sm_scale=None):
    """(out, bound, lse, lse bound) in 64 bits.

    With d the largest error of a logit (D products summed in fp32: a step, 2^-23, each; a
    query as two E4M3 terms: 2^-22 of its largest element for each of D; the scales and
    the exponential: 2^-20 of the logit), a weight is off by 2 d relative (its own logit
    and the sum's). Two terms of 4 bits hold a bf16 element's 8; only below 2^-11 of the
    largest, which the first term takes to [224, 448), is the second short of bits: off by
    half of E4M3's smallest step, 2^-10 of 224, 2^-17.8 of the largest. Of the normal
    elements here one in a thousand is that small, so a row has one or two, with 2^-22 for
    each of 64 and more others. It is rounded before it meets v: to bf16 (2^-8), f16 (2^-11) or two E4M3
    terms of it (2^-4 of 2^-4); terms below their normal range are off by half their
    smallest step, 2^-10 of a weight of one, f16's by 2^-25. Sums of L products are fp32,
    their parts joined in fp32 (a step for each), the output rounded to bf16."""
    sm = (w.dim ** -0.5 if sm_scale is None else sm_scale) * w.q_scale
    out = torch.full(w.q.shape, math.nan, dtype=torch.float64)
    lse = out[..., 0].clone()
    bound, lbound = out.clone(), lse.clone()
    q_all = w.q.cpu().float().double()
    for b, n in enumerate(w.kv_len):
        rows = w.rows[b]
        if rows <= 0 or n < rows:
            continue
        ids = torch.tensor(w.tables[b])
        kv = []
        for val in w.values:
            x = val[ids]
            x = x.transpose(0, 1) if w.hnd else x.permute(2, 0, 1, 3)
            kv.append(x.reshape(w.hkv, -1, w.dim)[:, :n])
        k, v = kv
        r0, r1 = w.qo[b], w.qo[b + 1]
        q = q_all[r0:r1].reshape(rows, w.hkv, w.group, w.dim)
        s = torch.einsum("rhgd,hjd->rhgj", q, k) * sm
        mag = torch.einsum("rhgd,hjd->rhgj", q.abs(), k.abs()) * abs(sm)
        top = q.abs().amax(-1)[..., None] * k.abs().sum(-1)[None, :, None] * abs(sm)
        pos = n - rows + torch.arange(rows)[:, None]
        j = torch.arange(n)[None]
        see = j <= pos
        if w.windows is not None and w.windows[b] > 0:
            see = see & (j > pos - w.windows[b])
        see = see[:, None, None]
        s = s.masked_fill(~see, -math.inf)
        x = torch.logsumexp(s, -1)
        p = torch.exp(s - x[..., None])
        o = torch.einsum("rhgj,hjd->rhgd", p, v)
        a = torch.einsum("rhgj,hjd->rhgd", p, v.abs())
        d = ((w.dim * 2.0 ** -23 * mag + 2.0 ** -22 * top).masked_fill(~see, 0).amax(-1)
             + 2.0 ** -20 * s.masked_fill(~see, 0).abs().amax(-1) + 2.0 ** -20)
        weight = BF16_HALF + (2.0 ** -11 if w.kind != "bf16" else 0)
        few = 0.0
        if w.kind != "bf16":  # weights relative to the largest: exp(s - max) = p * exp(x - max)
            one = torch.exp(s.amax(-1) - x)[..., None]
            low = 2.0 ** -10 if "e4m3" in w.kind else 2.0 ** -25
            seen = torch.einsum("rhgj,hjd->rhgd", see.double().expand(s.shape), v.abs())
            few = low * one * seen
        sums = (n + 200) * 2.0 ** -23
        bnd = (a * (weight + 2 * d[..., None] + sums) + few) * 1.01 + BF16_HALF * o.abs()
        out[r0:r1] = o.reshape(rows, w.hq, w.dim)
        bound[r0:r1] = bnd.reshape(rows, w.hq, w.dim)
        lse[r0:r1] = x.reshape(rows, w.hq)
        lbound[r0:r1] = (d + sums + 2.0 ** -21 * x.abs()).reshape(rows, w.hq)
    return out, bound, lse, lbound


def share(w):
    return ref.share(w.page_table, w.kv_indptr, w.kv_len, w.qo, w.windows, w.gp, page=w.page,
                     max_q=w.params.max_q_len, max_kv=w.params.max_kv_len, num_pages=w.pages)
