"""Cases of the serving operators around paged decode: block tables and slot
maps, append through a slot map, and latent (MLA) attention in its absorbed
form (query absorption, output projection) and its expanded form (keys and
values from the cached latents, ragged prefill attention).

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, makes the framework's calls.
"""
import math
import random

import torch

own = False

NOPE, ROPE, QD, LAT, DV = 128, 64, 192, 576, 128  # channels of an MLA head and of its latent
E4M3 = torch.float8_e4m3fn


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a batch: a token a request, a page now and then
        dict(name="tables_decode_bs64", op="tables", batch=64, page=64, cached=4096, new=1,
             tight=False, lens=1),
        # a mixed step of a large batch: prefill chunks beside decode rows, a free list that runs out
        dict(name="tables_mixed_bs512", op="tables", batch=512, page=16, cached=16384, new=513,
             tight=True, lens=2),
        # the latents of a decode step into 640-byte records
        dict(name="append_records_64", op="append", kind="records", rows=64, heads=1, dim=576,
             page=64),
        # a prefill of 8192 rows into an E4M3 cache with a scale per token and head
        dict(name="append_e4m3_8192", op="append", kind="e4m3_token", rows=8192, heads=8, dim=128,
             page=64),
        # one token, all 128 heads on one GPU
        dict(name="absorb_1_h128", op="absorb", rows=1, heads=128, out="bf16"),
        # a large decode batch with two rows a request, E4M3 query
        dict(name="absorb_1024_h128", op="absorb", rows=1024, heads=128, out="e4m3"),
        # a decode batch, 128 heads over 8-way tensor parallelism
        dict(name="project_64_h16", op="project", rows=64, heads=16),
        dict(name="project_1024_h128", op="project", rows=1024, heads=128),
        # a few cached contexts of a tensor-parallel rank, kept as records
        dict(name="expand_records_h16", op="expand", kind="records", batch=3, tokens=701, heads=16,
             page=64, lens=3),
        # a long context on one GPU
        dict(name="expand_bf16_8192_h128", op="expand", kind="bf16", batch=1, tokens=8192,
             heads=128, page=64, lens=4),
        # chunks of a few requests behind cached contexts
        dict(name="prefill_chunks_h16", op="prefill", batch=5, new=257, cached=1900, heads=16,
             causal=True, window=0, lens=5),
        # one long prompt, all heads on one GPU
        dict(name="prefill_4096_h128", op="prefill", batch=1, new=4096, cached=0, heads=128,
             causal=True, window=0, lens=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "absorb", "project", "expand", "prefill"])
    heads = rng.choice([1, 4, 8, 16, 20, 32, 64, 128])
    lens = rng.randrange(1 << 20)
    if op == "tables":
        return dict(op=op, batch=_log(rng, 1, 512), page=rng.choice([1, 16, 32, 64, 128]),
                    cached=_log(rng, 1, 8192), new=rng.choice([1, 2, 8, _log(rng, 9, 513)]),
                    tight=rng.random() < 0.3, lens=lens)
    if op == "append":
        kind = rng.choice(["records", "latent_bf16", "latent_e4m3", "bf16", "e4m3_tensor",
                           "e4m3_token", "int8_token"])
        mla = kind in ("records", "latent_bf16", "latent_e4m3")
        return dict(op=op, kind=kind, rows=_log(rng, 1, 8192),
                    heads=1 if mla else rng.choice([1, 2, 4, 8]),
                    dim=LAT if mla else rng.choice([64, 128]), page=rng.choice([16, 32, 64]))
    if op == "absorb":
        return dict(op=op, rows=_log(rng, 1, 1024), heads=heads, out=rng.choice(["bf16", "e4m3"]))
    if op == "project":
        return dict(op=op, rows=_log(rng, 1, 1024), heads=heads)
    if op == "expand":
        batch = rng.choice([1, 1, 2, 5, 8])
        return dict(op=op, kind=rng.choice(["bf16", "e4m3", "records"]), batch=batch,
                    tokens=_log(rng, 1, 8192 // batch), heads=heads, page=rng.choice([16, 64]),
                    lens=lens)
    batch = rng.choice([1, 1, 2, 5])
    causal = rng.random() < 0.8
    return dict(op=op, batch=batch, new=_log(rng, 1, 2048 // batch), cached=_log(rng, 1, 4096 // batch) - 1,
                heads=min(heads, 64), causal=causal,
                window=_log(rng, 1, 2048) if causal and rng.random() < 0.3 else 0, lens=lens)


def _sizes(case):
    """Ragged (cached, new) lengths of the requests: the first request has the
    case's own, the others down to a quarter of them."""
    r = random.Random(case["lens"])
    n = case["batch"]
    if case["op"] == "expand":
        return [(0, case["tokens"])] + [(0, r.randint(case["tokens"] // 4, case["tokens"]))
                                        for _ in range(n - 1)]
    if case["op"] == "tables":
        return [(r.randint(case["cached"] // 4, case["cached"]),
                 case["new"] if case["new"] <= 8 or r.random() < 0.1 else 1) for _ in range(n)]
    return [(case["cached"], case["new"])] + \
        [(r.randint(case["cached"] // 4, case["cached"]),
          r.randint(max(1, case["new"] // 4), case["new"])) for _ in range(n - 1)]


def _indptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _free(case):
    """Pages on the free list: more than the step takes, or (tight) half of it."""
    need = sum(-(-(c + n) // case["page"]) + -c // case["page"] for c, n in _sizes(case))
    return need // 2 if case["tight"] else need + 7


def _visible(case):
    """Visible (row, key) pairs of the prefill."""
    total = 0
    for c, n in _sizes(case):
        w = case["window"]
        if not case["causal"]:
            total += n * (c + n)
        elif w <= 0:
            total += n * c + n * (n + 1) // 2
        else:
            total += sum(min(w, c + i + 1) for i in range(n))
    return total


def work(case):
    op = case["op"]
    if op == "tables":
        s = _sizes(case)
        pages = sum(-(-(c + n) // case["page"]) for c, n in s)
        rows = sum(n for _, n in s)
        return {"bytes": 3 * 4 * len(s) + 8 * pages + 4 * 4 * (len(s) + 1) + 12 * rows, "flops": 0}
    if op == "append":
        n, d, e = case["rows"] * case["heads"], case["dim"], 2 if "bf16" in case["kind"] else 1
        if case["kind"] == "records":
            return {"bytes": n * (1152 + 640 + 16) + 8 * case["rows"], "flops": 0}
        two = 1 if d == LAT else 2
        scales = 4 if "token" in case["kind"] else 0
        return {"bytes": two * n * (d * (2 + e) + scales) + 8 * case["rows"], "flops": 0}
    h = case["heads"]
    if op in ("absorb", "project"):
        n = case["rows"] * h
        if op == "absorb":
            b = n * (QD * 2 + LAT * (2 if case["out"] == "bf16" else 1))
        else:
            b = n * (512 + DV) * 2
        return {"bytes": b + h * 128 * 512 * 2, "flops": 2 * n * 128 * 512}
    s = _sizes(case)
    if op == "expand":
        t = sum(n for _, n in s)
        per = {"bf16": 1152, "e4m3": 576, "records": 656}[case["kind"]]
        return {"bytes": t * (per + 1152 + h * 512) + h * 256 * 512 * 2, "flops": 2 * t * h * 256 * 512}
    rows, toks = sum(n for _, n in s), sum(c + n for c, n in s)
    return {"bytes": rows * h * (QD + DV) * 2 + rows * h * 4 + toks * (h * 512 + 128),
            "flops": 640 * h * _visible(case)}


# ------------------------------------------------------------------- inputs

def _codes(x, scale):
    return (x / scale).clamp(-448, 448).to(E4M3)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(seed * 1000003 + 17)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    op, st = case["op"], dict(case=case)
    if op == "tables":
        s, p = _sizes(case), case["page"]
        have = [-(-c // p) for c, _ in s]
        cols = max(-(-(c + n) // p) for c, n in s) + 3
        free = _free(case)
        pages = sum(have) + free + 5
        ids = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
        st.update(cached_len=_ints([c for c, _ in s]), new_len=_ints([n for _, n in s]),
                  request=torch.randperm(len(s) + 3, generator=g, device=dev)[:len(s)].int(),
                  free_pages=ids[sum(have):].contiguous(), free_count=_ints([free]), pages=pages,
                  block_table=torch.full((len(s) + 3, cols), -1, dtype=torch.int32, device=dev))
        at = torch.arange(cols, device=dev)[None, :] < _ints(have)[:, None]
        rows = torch.full((len(s), cols), -1, dtype=torch.int32, device=dev)
        rows[at] = ids[:sum(have)]
        st["block_table"][st["request"].long()] = rows
        cap_pages = sum(-(-(c + n) // p) for c, n in s) + 9
        cap_rows = sum(n for _, n in s) + 9
        # what the step writes; entries behind the last request stay as they are
        n1 = len(s) + 1
        st["out"] = dict(kv_len=_ints([-1] * len(s)), kv_indptr=_ints([-1] * n1),
                         page_table=torch.full((cap_pages,), -1, dtype=torch.int32, device=dev),
                         qo_indptr=_ints([-1] * n1), tok_indptr=_ints([-1] * n1),
                         slot_map=torch.full((cap_rows,), -1, dtype=torch.int64, device=dev),
                         positions=torch.full((cap_rows,), -1, dtype=torch.int32, device=dev),
                         free_left=_ints([-1]), block_table=st["block_table"])
        if own:
            st["dec"] = _decoder(dict(heads=1, hkv=1, dim=128, page=p, pages=pages, batch=len(s),
                                      max_kv=max(c + n for c, n in s), kind="bf16"))
        return st
    if op == "append":
        kind, n, h, d, p = case["kind"], case["rows"], case["heads"], case["dim"], case["page"]
        pages = -(-n // p) + 3
        width, dt = {"records": (640, torch.uint8), "latent_bf16": (d, torch.bfloat16),
                     "bf16": (d, torch.bfloat16), "int8_token": (d, torch.int8)}.get(kind, (d, E4M3))
        mla = d == LAT
        st["slot_map"] = torch.randperm(pages * p, generator=g, device=dev)[:n]
        for side in ("k",) if mla else ("k", "v"):
            st[side + "_new"] = randn(n, h, d, std=2.0)
            st[side + "_pages"] = torch.zeros(pages, p, h, width, dtype=torch.uint8 if dt is E4M3 else dt,
                                              device=dev)
            if "token" in kind:
                st[side + "_scale"] = torch.ones(pages, p, h, device=dev)
            elif kind == "records":
                st[side + "_scale"] = torch.ones(pages, p, h, 4, device=dev)
            elif kind in ("e4m3_tensor", "latent_e4m3"):
                st[side + "_scale"] = torch.full((1,), 0.02, device=dev)
        if own:
            st["dec"] = _decoder(dict(heads=h, hkv=h, dim=d, page=p, pages=pages, batch=1, max_kv=n,
                                      kind=kind))
        return st
    h = case["heads"]
    if op in ("absorb", "project"):
        n = case["rows"]
        st["w"] = randn(h, 256, 512, std=512 ** -0.5)  # W_UK (rows 0..127) and W_UV of each head
        if op == "absorb":
            st["q"] = randn(n, h, QD)
            st["q_scale"] = 0.01
            st["out"] = torch.zeros(n, h, LAT, device=dev,
                                    dtype=torch.bfloat16 if case["out"] == "bf16" else E4M3)
        else:
            st["o_lat"] = randn(n, h, 512)
            st["out"] = torch.zeros(n, h, DV, dtype=torch.bfloat16, device=dev)
        if own:
            st["dec"] = _decoder(dict(heads=h, hkv=1, dim=LAT, page=64, pages=1, batch=1, max_kv=64,
                                      kind="latent_e4m3" if case.get("out") == "e4m3" else "latent_bf16"))
        return st
    s = _sizes(case)
    if op == "expand":
        kind, p = case["kind"], case["page"]
        lens = [n for _, n in s]
        t, npg = sum(lens), [-(-n // p) for n in lens]
        pages = sum(npg) + 2
        st.update(tok_indptr=_ints(_indptr(lens)), kv_indptr=_ints(_indptr(npg)),
                  page_table=torch.randperm(pages, generator=g, device=dev)[:sum(npg)].int(),
                  w=randn(h, 256, 512, std=512 ** -0.5), k_scale=None)
        x = randn(pages, p, 1, LAT)
        if kind == "bf16":
            st["k_pages"] = x
        elif kind == "e4m3":
            st["k_scale"] = torch.full((1,), 0.0125, device=dev)
            st["k_pages"] = _codes(x.float(), st["k_scale"]).view(torch.uint8)
        else:
            blocks = x[..., :512].float().reshape(pages, p, 1, 4, 128)
            st["k_scale"] = (blocks.abs().amax(-1) / 448).contiguous()
            rec = torch.empty(pages, p, 1, 640, dtype=torch.uint8, device=dev)
            rec[..., :512] = _codes(blocks, st["k_scale"][..., None]).reshape(pages, p, 1, 512).view(torch.uint8)
            rec[..., 512:] = x[..., 512:].contiguous().view(torch.uint8)
            st["k_pages"] = rec
        st["latent"] = torch.zeros(t, LAT, dtype=torch.bfloat16, device=dev)
        st["kv"] = torch.zeros(t, h, 256, dtype=torch.bfloat16, device=dev)  # k then v of each head
        if own:
            st["dec"] = _decoder(dict(heads=h, hkv=1, dim=LAT, page=p, pages=pages, batch=len(s),
                                      max_kv=max(lens), kind={"bf16": "latent_bf16", "e4m3": "latent_e4m3"}
                                      .get(kind, "records")))
        return st
    rows, toks = sum(n for _, n in s), sum(c + n for c, n in s)
    st.update(q=randn(rows, h, QD), kv=randn(toks, h, 256), latent=randn(toks, LAT),
              qo_indptr=_ints(_indptr([n for _, n in s])),
              tok_indptr=_ints(_indptr([c + n for c, n in s])),
              window=_ints([case["window"]] * len(s)) if case["window"] > 0 else None,
              out=torch.zeros(rows, h, DV, dtype=torch.bfloat16, device=dev),
              lse=torch.zeros(rows, h, device=dev))
    if own:
        from paged_split_kv_03_gb300 import binding as B
        st["dec"] = _decoder(dict(heads=h, hkv=1, dim=LAT, page=64, pages=1, batch=len(s),
                                  max_kv=max(c + n for c, n in s), kind="latent_bf16"))
        st["pre"] = B.Prefill(st["dec"].plan, rows, toks)
    return st


def _decoder(d):
    """The plan and scratch that a serving program keeps."""
    from paged_split_kv_03_gb300 import binding as B
    kind, w = d["kind"], 640 if d["kind"] == "records" else d["dim"]
    p = B.PdaParams(num_qo_heads=d["heads"], num_kv_heads=d["hkv"], head_dim=d["dim"],
                    page_size=d["page"], max_batch=d["batch"], max_q_len=1, max_kv_len=d["max_kv"],
                    num_pages=d["pages"], kv_stride_page=d["page"] * d["hkv"] * w,
                    kv_stride_token=d["hkv"] * w, kv_stride_head=w, device=_dev().index)
    if d["dim"] == LAT:
        p.head_dim_v = 512
    if "bf16" not in kind:
        p.kv_dtype = B.PDA_INT8 if "int8" in kind else B.PDA_E4M3
        p.scale_mode = B.PDA_SCALE_MLA_BLOCK if kind == "records" else \
            B.PDA_SCALE_TOKEN_HEAD if "token" in kind else B.PDA_SCALE_TENSOR
        p.q_dtype = B.PDA_E4M3 if kind == "latent_e4m3" else B.PDA_BF16
    return B.Decoder(p, device=_dev())


# ------------------------------------------------------------------ one pass

def run(st):
    return _OPS[st["case"]["op"]](st)


def _tables(st):
    o, p = st["out"], st["case"]["page"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_build_tables(st["dec"].plan, st["cached_len"], st["new_len"], st["request"],
                           st["block_table"], st["free_pages"], st["free_count"], o["free_left"],
                           o["kv_len"], o["kv_indptr"], o["page_table"], o["qo_indptr"],
                           o["tok_indptr"], o["slot_map"], o["positions"], st["dec"].scratch)
        return o
    cached, new = st["cached_len"].long(), st["new_len"].long()
    have = (cached + p - 1) // p
    want = (cached + new + p - 1) // p
    need = want - have
    upto = need.cumsum(0)
    free = st["free_count"].long()
    granted = (need == 0) | (upto <= free)
    new = torch.where(granted, new, 0)
    pages = torch.where(granted, want, have)
    taken = torch.where(granted & (need > 0), upto, 0).amax()  # a run of the list without holes
    kv_len = cached + new
    zero = torch.zeros(1, dtype=torch.int64, device=cached.device)
    kv_ptr, qo_ptr, tok_ptr = (torch.cat([zero, x.cumsum(0)]) for x in (pages, new, kv_len))
    # the page of entry i: an old one from the block table, or one off the free list's end
    i = torch.arange(o["page_table"].numel(), device=cached.device)
    inside = i < kv_ptr[-1]
    i = torch.minimum(i, kv_ptr[-1] - 1).clamp(min=0)  # behind the last one: the last one again
    b = torch.searchsorted(kv_ptr[1:], i, right=True).clamp(max=cached.numel() - 1)
    j = i - kv_ptr[b]
    grown = (j >= have[b]) & (kv_ptr[-1] > 0)
    row = st["request"].long()[b]
    old = st["block_table"][row, j]
    off = free - 1 - (upto[b] - need[b] + j - have[b])
    fresh = st["free_pages"][torch.where(grown, off, 0)]
    page = torch.where(grown, fresh, old)
    o["page_table"].copy_(torch.where(inside, page, o["page_table"]))
    st["block_table"].index_put_((row, j), page)
    r = torch.arange(o["slot_map"].numel(), device=cached.device)
    b = torch.searchsorted(qo_ptr[1:], r, right=True).clamp(max=cached.numel() - 1)
    t = cached[b] + r - qo_ptr[b]
    inside = r < qo_ptr[-1]
    at = torch.where(inside, kv_ptr[b] + t // p, 0)
    o["slot_map"].copy_(torch.where(inside, o["page_table"][at].long() * p + t % p, o["slot_map"]))
    o["positions"].copy_(torch.where(inside, t, o["positions"]))
    o["kv_len"].copy_(kv_len)
    o["kv_indptr"].copy_(kv_ptr)
    o["qo_indptr"].copy_(qo_ptr)
    o["tok_indptr"].copy_(tok_ptr)
    o["free_left"].copy_(free - taken)
    return o


def _append(st):
    kind = st["case"]["kind"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_append_slots(st["dec"].plan, st["k_new"], st.get("v_new"), st["slot_map"], None,
                           st["k_pages"], st.get("v_pages"), st.get("k_scale"), st.get("v_scale"),
                           st["dec"].scratch)
    else:
        for side in ("k", "v"):
            if side + "_new" not in st:
                continue
            x, pages, slots = st[side + "_new"].float(), st[side + "_pages"], st["slot_map"]
            flat = pages.view(-1, *pages.shape[2:])
            scale = st.get(side + "_scale")
            if kind in ("bf16", "latent_bf16"):
                flat[slots] = st[side + "_new"]
            elif kind in ("e4m3_tensor", "latent_e4m3"):
                flat[slots] = _codes(x, scale).view(torch.uint8)
            elif kind == "records":
                blocks = x[..., :512].unflatten(-1, (4, 128))
                s = blocks.abs().amax(-1)
                s = s / torch.full_like(s, 448.0)
                codes = _codes(blocks, torch.where(s > 0, s, 1.0)[..., None]).flatten(-2)
                scale.view(-1, *scale.shape[2:])[slots] = s
                flat[slots] = torch.cat([codes.view(torch.uint8),
                                         st["k_new"][..., 512:].contiguous().view(torch.uint8)], -1)
            else:
                top = 127.0 if kind == "int8_token" else 448.0
                amax = x.abs().amax(-1)
                s = torch.where(amax > 0, amax / torch.full_like(amax, top), 1.0)
                scale.view(-1, scale.shape[2])[slots] = s
                y = x / s[..., None]
                flat[slots] = y.round().clamp(-127, 127).to(torch.int8) if kind == "int8_token" else \
                    y.clamp(-448, 448).to(E4M3).view(torch.uint8)
    return _caches(st)


def _caches(st):
    """The caches as the values their codes stand for, and the scales written."""
    kind, got = st["case"]["kind"], {}
    for side in ("k", "v"):
        if side + "_pages" not in st:
            continue
        pages = st[side + "_pages"]
        if kind == "records":
            got[side + "_nope"], got[side + "_rope"] = pages[..., :512].view(E4M3), \
                pages[..., 512:].view(torch.bfloat16)
        else:
            got[side] = pages.view(E4M3) if pages.dtype == torch.uint8 else pages
        if "token" in kind or kind == "records":
            got[side + "_scale"] = st[side + "_scale"]
    return got


def _absorb(st):
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_mla_absorb(st["dec"].plan, st["q"], st["w"][:, :128], st["q_scale"], st["out"], None,
                         st["dec"].scratch)
        return st["out"]
    q = st["q"].float()
    lat = torch.matmul(q[..., :NOPE].transpose(0, 1), st["w"][:, :128].float()).transpose(0, 1)
    x = torch.cat([lat, q[..., NOPE:]], -1)
    return x.to(torch.bfloat16) if st["case"]["out"] == "bf16" else _codes(x, st["q_scale"])


def _project(st):
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_mla_project(st["dec"].plan, st["o_lat"], st["w"][:, 128:], st["out"], None,
                          st["dec"].scratch)
        return st["out"]
    o = torch.matmul(st["o_lat"].float().transpose(0, 1), st["w"][:, 128:].float().transpose(1, 2))
    return o.transpose(0, 1).to(torch.bfloat16)


def _latents(st, dtype):
    """The cached latents [tokens, 576] in the order of the requests, dequantised."""
    kind, p = st["case"]["kind"], st["case"]["page"]
    t = torch.arange(st["latent"].shape[0], device=st["latent"].device)
    tok, kv = st["tok_indptr"].long(), st["kv_indptr"].long()
    b = torch.searchsorted(tok[1:], t, right=True)
    i = t - tok[b]
    slot = st["page_table"].long()[kv[b] + i // p] * p + i % p
    x = st["k_pages"].flatten(0, 2)[slot]
    if kind == "bf16":
        return x.to(dtype)
    if kind == "e4m3":
        return x.view(E4M3).to(dtype) * st["k_scale"].to(dtype)
    s = st["k_scale"].flatten(0, 2)[slot].to(dtype)
    nope = x[:, :512].contiguous().view(E4M3).to(dtype).unflatten(1, (4, 128)) * s[..., None]
    return torch.cat([nope.flatten(1), x[:, 512:].contiguous().view(torch.bfloat16).to(dtype)], 1)


def _expand(st):
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_mla_expand(st["dec"].plan, st["k_pages"], st["page_table"], st["kv_indptr"],
                         st["tok_indptr"], st["k_scale"], st["w"][:, :128], st["w"][:, 128:],
                         st["latent"], st["kv"][..., :128], st["kv"][..., 128:], st["dec"].scratch)
        return st["latent"], st["kv"]
    x = _latents(st, torch.float32)
    h = st["case"]["heads"]
    kv = torch.matmul(x[:, :512], st["w"].float().reshape(h * 256, 512).t())
    return x.to(torch.bfloat16), kv.reshape(-1, h, 256).to(torch.bfloat16)


def _prefill(st):
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_mla_prefill(st["pre"].plan, st["q"], st["kv"][..., :128], st["kv"][..., 128:],
                          st["latent"][:, 512:], st["qo_indptr"], st["tok_indptr"], st["window"],
                          st["case"]["causal"], QD ** -0.5, st["out"], st["lse"], st["pre"].scratch)
        return st["out"], st["lse"]
    s = _sizes(st["case"])
    rmax, lmax = max(n for _, n in s), max(c + n for c, n in s)
    dev = st["q"].device
    qo, tok = st["qo_indptr"].long(), st["tok_indptr"].long()
    rows, toks = qo[1:] - qo[:-1], tok[1:] - tok[:-1]
    # requests padded to the longest: [B, rows, H, .] and [B, keys, H, .]
    i, j = torch.arange(rmax, device=dev), torch.arange(lmax, device=dev)
    q = st["q"][(qo[:-1, None] + torch.minimum(i, rows[:, None] - 1))].float()
    at = tok[:-1, None] + torch.minimum(j, toks[:, None] - 1)
    kv, rope = st["kv"][at].float(), st["latent"][at][..., 512:].float()
    k = torch.cat([kv[..., :128], rope[:, :, None].expand(*kv.shape[:3], ROPE)], -1)
    x = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)) * QD ** -0.5
    pos = (toks - rows)[:, None, None] + i[:, None]
    see = (j < toks[:, None, None]) & (i[:, None] < rows[:, None, None])
    if st["case"]["causal"]:
        see = see & (j <= pos)
        if st["window"] is not None:
            see = see & (j > pos - st["window"].long()[:, None, None])
    x = x.masked_fill(~see[:, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., 128:].transpose(1, 2)) / z
    lse = (m + torch.log(z))[..., 0]
    r = torch.arange(st["q"].shape[0], device=dev)
    b = torch.searchsorted(qo[1:], r, right=True)
    return o.transpose(1, 2)[b, r - qo[b]].to(torch.bfloat16), lse.transpose(1, 2)[b, r - qo[b]]


_OPS = dict(tables=_tables, append=_append, absorb=_absorb, project=_project, expand=_expand,
            prefill=_prefill)


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers
    st = prepare(case, seed)
    if op == "append":
        return _exact_append(st)
    if op == "absorb":
        q, w = st["q"].double(), st["w"].double()
        x = torch.cat([torch.einsum("thd,hdc->thc", q[..., :NOPE], w[:, :128]), q[..., NOPE:]], -1)
        return x if case["out"] == "bf16" else (x / st["q_scale"]).clamp(-448, 448)
    if op == "project":
        return torch.einsum("thc,hdc->thd", st["o_lat"].double(), st["w"][:, 128:].double())
    if op == "expand":
        x = _latents(st, torch.float64)
        return x, torch.einsum("tc,hdc->thd", x[:, :512], st["w"].double())
    outs, lses = [], []
    qo, tok = st["qo_indptr"].tolist(), st["tok_indptr"].tolist()
    for b in range(case["batch"]):
        q = st["q"][qo[b]:qo[b + 1]].double()
        kv, rope = st["kv"][tok[b]:tok[b + 1]].double(), st["latent"][tok[b]:tok[b + 1], 512:].double()
        n, length = q.shape[0], kv.shape[0]
        pos = length - n + torch.arange(n, device=q.device)[:, None]
        key = torch.arange(length, device=q.device)[None, :]
        hide = torch.zeros(n, length, dtype=torch.bool, device=q.device)
        if case["causal"]:
            hide |= key > pos
            if case["window"] > 0:
                hide |= key < pos - case["window"] + 1
        per_head = []
        for h in range(case["heads"]):
            s = (q[:, h, :NOPE] @ kv[:, h, :128].t() + q[:, h, NOPE:] @ rope.t()) / math.sqrt(QD)
            s[hide] = -math.inf
            lse = torch.logsumexp(s, 1)
            per_head.append((torch.exp(s - lse[:, None]) @ kv[:, h, 128:], lse))
        outs.append(torch.stack([o for o, _ in per_head], 1))
        lses.append(torch.stack([x for _, x in per_head], 1))
    return torch.cat(outs), torch.cat(lses)


def _exact_append(st):
    """The caches' values before rounding to codes; None for whole numbers."""
    kind, slots, got = st["case"]["kind"], st["slot_map"], {}
    for side in ("k", "v"):
        if side + "_new" not in st:
            continue
        x = st[side + "_new"].double()
        n_slots = st[side + "_pages"].shape[0] * st["case"]["page"]

        def placed(y, fill):
            full = torch.full((n_slots, *y.shape[1:]), fill, dtype=torch.float64, device=y.device)
            full.index_copy_(0, slots, y)
            return full.unflatten(0, (-1, st["case"]["page"]))

        if kind in ("bf16", "latent_bf16"):
            got[side] = placed(x, 0.0)
        elif kind in ("e4m3_tensor", "latent_e4m3"):
            got[side] = placed((x / st[side + "_scale"].double()).clamp(-448, 448), 0.0)
        elif kind == "records":
            b = x[..., :512].reshape(x.shape[0], 1, 4, 128)
            s = b.abs().amax(-1) / 448
            got[side + "_nope"] = placed((b / s[..., None]).reshape(x.shape[0], 1, 512), 0.0)
            got[side + "_rope"] = placed(x[..., 512:], 0.0)
            got[side + "_scale"] = placed(s, 1.0)
        else:
            s = x.abs().amax(-1) / (127 if kind == "int8_token" else 448)
            got[side] = None if kind == "int8_token" else placed(x / s[..., None], 0.0)
            got[side + "_scale"] = placed(s, 1.0)
    return got
