"""Plain implementations in 64 bits of the calls around decode (block tables,
append by slot map, latent attention's products and prefill), on the CPU."""
from __future__ import annotations

import math

import torch

from paged_split_kv_03_gb300 import binding as B

E4M3 = torch.float8_e4m3fn
BF16_HALF = 2.0 ** -8    # half a step of a rounding, relative to the value
E4M3_HALF = 2.0 ** -4
E4M3_SUB = 2.0 ** -10    # ... below E4M3's normal range, absolute


def mla_plan(heads, *, kind="bf16", page=64, pages=8, batch=1, max_kv=4096, max_q_len=1,
             num_sms=0, device=0):
    """An MLA plan; kind: bf16, e4m3 (per tensor), e4m3_token or records."""
    w = 640 if kind == "records" else 576
    p = B.PdaParams(num_qo_heads=heads, num_kv_heads=1, head_dim=576, head_dim_v=512,
                    page_size=page, max_batch=batch, max_q_len=max_q_len, max_kv_len=max_kv,
                    num_pages=pages, kv_stride_page=page * w, kv_stride_token=w, kv_stride_head=w,
                    device=device, num_sms=num_sms)
    if kind != "bf16":
        p.kv_dtype = B.PDA_E4M3
        p.scale_mode = {"records": B.PDA_SCALE_MLA_BLOCK, "e4m3": B.PDA_SCALE_TENSOR,
                        "e4m3_token": B.PDA_SCALE_TOKEN_HEAD}[kind]
        p.q_dtype = B.PDA_BF16 if kind == "records" else B.PDA_E4M3
    return p


def build_tables(cached, new, request, block_table, free_pages, free_count, page, *, max_kv,
                 page_cap, rows_cap, num_pages):
    """One step's tables by the words of the header, request by request."""
    block = [list(r) for r in block_table]
    cols = len(block[0]) if block else 0
    out = dict(kv_len=[], kv_indptr=[0], page_table=[], qo_indptr=[0], tok_indptr=[0],
               slot_map=[], positions=[])
    status, upto, taken, full = 0, 0, 0, False
    free_count = max(0, free_count)
    for b, (c, n) in enumerate(zip(cached, new)):
        row = request[b] if request is not None else b
        if c < 0 or n < 0 or not 0 <= row < len(block):
            status |= B.PDA_STATUS_TABLE_INVALID
            c = n = 0
            bad = True
        else:
            bad = False
            if c + n > max_kv:
                status |= B.PDA_STATUS_TABLE_INVALID | B.PDA_STATUS_KV_LEN_GT_MAX
                bad = True
            elif -(-(c + n) // page) > cols:
                status |= B.PDA_STATUS_TABLE_INVALID
                bad = True
        if bad:
            c = n = 0
        have, want = -(-c // page), -(-(c + n) // page)
        need = want - have
        upto += need
        granted = need == 0 or upto <= free_count
        if not granted:
            status |= B.PDA_STATUS_NO_PAGES
            n, want = 0, have
        if full or len(out["page_table"]) + want > page_cap or len(out["slot_map"]) + n > rows_cap:
            full = True
            status |= B.PDA_STATUS_TABLE_FULL
            c = n = have = want = 0
            granted = False
        ids = [] if bad else block[row][:have]
        if granted and need:
            start = upto - need
            ids = ids + [free_pages[free_count - 1 - start - k] for k in range(need)]
            block[row][have:want] = ids[have:]
            taken = upto
        ids = ids[:want]
        out["kv_len"].append(c + n)
        out["page_table"] += ids
        for t in range(c, c + n):
            pg = ids[t // page]
            if 0 <= pg < num_pages:
                out["slot_map"].append(pg * page + t % page)
            else:
                out["slot_map"].append(-1)
                status |= B.PDA_STATUS_PAGE_OOB
            out["positions"].append(t)
        out["kv_indptr"].append(len(out["page_table"]))
        out["qo_indptr"].append(len(out["slot_map"]))
        out["tok_indptr"].append(out["tok_indptr"][-1] + c + n)
    out["free_left"] = [free_count - taken]
    out["block_table"] = block
    return out, status


def codes(x, s):
    """E4M3 codes of x / s: one fp32 division, saturating, to nearest even."""
    return (x.float() / s).clamp(-448, 448).to(E4M3)


def records(x):
    """Latents [..., 576] bf16 -> (640-byte records uint8, scales fp32 [..., 4])."""
    b = x[..., :512].float().unflatten(-1, (4, 128))
    s = b.abs().amax(-1)
    s = s / torch.full_like(s, 448.0)
    c = codes(b, torch.where(s > 0, s, torch.ones_like(s))[..., None]).flatten(-2)
    rope = x[..., 512:].contiguous().view(torch.uint8)
    return torch.cat([c.view(torch.uint8), rope], -1), s


def record_values(rec, s):
    nope = rec[..., :512].contiguous().view(E4M3).double().unflatten(-1, (4, 128))
    rope = rec[..., 512:].contiguous().view(torch.bfloat16).double()
    return torch.cat([(nope * s.double()[..., None]).flatten(-2), rope], -1)


def sum_bound(k):
    """Rounding of a sum of k products in fp32, relative to the sum of their
    magnitudes: one step (2^-23, also a truncating adder) for each product."""
    return k * 2.0 ** -23


def product(a, b):
    """(sum_k a b, sum_k |a b|) per head: a [T, H, K], b [H, N, K] -> [T, H, N]."""
    a, b = a.double(), b.double()
    return torch.einsum("thk,hnk->thn", a, b), torch.einsum("thk,hnk->thn", a.abs(), b.abs())


def attention(q, k, v, rope, qo, tok, *, causal, windows, scale):
    """Prefill attention and, element by element, how far a correct kernel may
    be off: (out, out bound, lse, lse bound); rows in no request stay NaN.

    With d the largest error of a logit (192 products summed in fp32, the
    product with the scale and the exponential's 2^-22), a weight is off by
    2 d relative (its own logit and the sum's); the weights are rounded to
    bf16 before they meet v and the sum of products is fp32; then the output
    is rounded."""
    rows, heads = q.shape[:2]
    out = torch.full((rows, heads, 128), math.nan, dtype=torch.float64)
    bound, lse, lbound = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    q, k, v, rope = q.double(), k.double(), v.double(), rope.double()
    for b in range(len(qo) - 1):
        r0, r1, t0, t1 = qo[b], qo[b + 1], tok[b], tok[b + 1]
        n, length = r1 - r0, t1 - t0
        if n == 0:
            continue
        if length == 0:
            out[r0:r1], lse[r0:r1] = 0.0, -math.inf
            bound[r0:r1], lbound[r0:r1] = 0.0, 0.0
            continue
        keys = torch.cat([k[t0:t1], rope[t0:t1, None].expand(length, heads, 64)], -1)
        s = torch.einsum("rhc,jhc->hrj", q[r0:r1], keys) * scale
        mag = torch.einsum("rhc,jhc->hrj", q[r0:r1].abs(), keys.abs()) * abs(scale)
        pos = length - n + torch.arange(n)[:, None]
        j = torch.arange(length)[None]
        see = torch.ones(n, length, dtype=torch.bool)
        if causal:
            see = j <= pos
            if windows is not None and windows[b] > 0:
                see = see & (j > pos - windows[b])
        s = s.masked_fill(~see, -math.inf)
        x = torch.logsumexp(s, -1)
        p = torch.exp(s - x[..., None])
        o = torch.einsum("hrj,jhd->rhd", p, v[t0:t1])
        a = torch.einsum("hrj,jhd->rhd", p, v[t0:t1].abs())
        d = ((sum_bound(192) + 2.0 ** -22) * mag.masked_fill(~see, 0).amax(-1) + 2.0 ** -21).t()
        out[r0:r1], lse[r0:r1] = o, x.t()
        bound[r0:r1] = a * (BF16_HALF + 2 * d + sum_bound(length))[..., None] * 1.01 + BF16_HALF * o.abs()
        lbound[r0:r1] = d + sum_bound(length) + 2.0 ** -22 * x.t().abs()
    return out, bound, lse, lbound
