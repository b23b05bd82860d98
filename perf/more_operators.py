"""Cases of the operators over shared pages: forking requests with a copy of the
page they will both write, freeing and compacting the pages of a cache, the
prefixes that the requests of a step share, and decode attention that reads
such a prefix once for all of them.

``run`` computes the plain form with elementary torch operations, or, where
``own`` is true, makes the framework's calls.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # parallel sampling: 16 finished prompts, three more answers of each
        dict(name="fork_48_bf16", op="fork", parents=16, each=3, tokens=2047, page=16, heads=8,
             dim=128, kind="bf16", hnd=False, tight=False, lens=1),
        # a beam step of latent records, the free list too short for all of it
        dict(name="fork_256_records", op="fork", parents=64, each=4, tokens=1000, page=64, heads=1,
             dim=576, kind="records", hnd=False, tight=True, lens=2),
        # the end of a decode step: finished requests are gone from the list
        dict(name="free_bs64", op="free", batch=64, tokens=4096, page=64, shared=0.25, spare=1.0,
             lens=3),
        # many long requests over small pages
        dict(name="free_bs512_page16", op="free", batch=512, tokens=16384, page=16, shared=0.5,
             spare=0.5, lens=4),
        # a few pages a step, beside decode
        dict(name="compact_64_e4m3", op="compact", batch=16, tokens=2048, page=64, heads=8, dim=128,
             kind="e4m3_token", hnd=True, shared=0.25, spare=1.0, most=64, lens=5),
        # the whole cache in one go
        dict(name="compact_all_bf16", op="compact", batch=64, tokens=4096, page=64, heads=8, dim=128,
             kind="bf16", hnd=False, shared=0.25, spare=1.0, most=1 << 20, lens=6),
        # one system prompt for all, a token a request
        dict(name="share_bs64", op="share", batch=64, groups=1, prefix=4096, owned=256, page=64,
             rows=1, window=0, lens=7),
        # many prompts, a few answers of each, verify rows
        dict(name="share_bs512_page16", op="share", batch=512, groups=64, prefix=16384, owned=1024,
             page=16, rows=4, window=2000, lens=8),
        # the smallest decode: four drafts verified behind one short prompt
        dict(name="decode_bs4_d256", op="decode", batch=4, groups=1, prefix=1024, owned=64, page=16,
             rows=4, hq=16, hkv=2, dim=256, kind="bf16", q8=False, hnd=False, window=0, lens=9),
        # a system prompt of 8K tokens for a batch of chats
        dict(name="decode_bs64_d128", op="decode", batch=64, groups=1, prefix=8192, owned=256,
             page=64, rows=1, hq=64, hkv=8, dim=128, kind="bf16", q8=False, hnd=False, window=0,
             lens=10),
        # one long document, a few questions, an E4M3 cache with a scale per token and head
        dict(name="decode_doc_e4m3_d256", op="decode", batch=12, groups=1, prefix=65536, owned=300,
             page=16, rows=2, hq=16, hkv=2, dim=256, kind="e4m3_token", q8=False, hnd=False,
             window=0, lens=11),
        # four long prompts with 32 answers each, E4M3 throughout
        dict(name="decode_groups_e4m3_d128", op="decode", batch=128, groups=4, prefix=32768,
             owned=512, page=64, rows=1, hq=64, hkv=8, dim=128, kind="e4m3_tensor", q8=True,
             hnd=True, window=0, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["fork", "free", "compact", "share", "decode", "decode", "decode"])
    lens = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["bf16", "e4m3_tensor", "e4m3_token", "int8_tensor", "int8_token"])
    if op in ("fork", "compact"):
        kind = rng.choice([kind, "records", "latent_bf16"])
        mla = kind in ("records", "latent_bf16")
        heads, dim = (1, 576) if mla else (rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]))
        if op == "fork":
            return dict(op=op, parents=_log(rng, 1, 64), each=_log(rng, 1, 8),
                        tokens=_log(rng, 1, 4096), page=page, heads=heads, dim=dim, kind=kind,
                        hnd=rng.random() < 0.5 and not mla, tight=rng.random() < 0.3, lens=lens)
        return dict(op=op, batch=_log(rng, 1, 64), tokens=_log(rng, 1, 2048), page=page, heads=heads,
                    dim=dim, kind=kind, hnd=rng.random() < 0.5 and not mla,
                    shared=rng.choice([0.0, 0.3, 0.9]), spare=rng.choice([0.1, 0.5, 1.0]),
                    most=rng.choice([0, 1, 64, 1 << 20]), lens=lens)
    if op == "free":
        return dict(op=op, batch=_log(rng, 1, 512), tokens=_log(rng, 1, 16384), page=max(16, page),
                    shared=rng.choice([0.0, 0.3, 0.9]), spare=rng.choice([0.0, 0.1, 1.0]), lens=lens)
    batch = _log(rng, 1, 512 if op == "share" else 96)
    groups = min(batch, rng.choice([1, 1, 2, 5, _log(rng, 1, 64)]))
    case = dict(op=op, batch=batch, groups=groups, prefix=_log(rng, 1, 16384 // max(1, groups // 4)),
                owned=_log(rng, 8, 700), page=page, rows=rng.choice([1, 1, 2, 5, 8]),
                window=_log(rng, 1, 8192) if rng.random() < 0.2 else 0, lens=lens)
    if op == "decode":
        hkv = rng.choice([1, 2, 4, 8])
        case.update(hq=hkv * rng.choice([1, 2, 3, 4, 6, 8, 16]), hkv=hkv,
                    dim=rng.choice([64, 128, 128, 256]), kind=kind,
                    q8="e4m3" in kind and rng.random() < 0.5, hnd=rng.random() < 0.5)
        while work(case)["flops"] > 1e11:  # no dearer than the largest listed one
            case["batch"] //= 2
            case["groups"] = min(case["groups"], case["batch"])
    return case


# ------------------------------------------------- what the cases stand for

def _ceil(a, b):
    return -(-a // b)


def _forked(case):
    """(tokens of each parent, (parent, shared tokens) of each fork)."""
    r = random.Random(case["lens"])
    have = [case["tokens"]] + [r.randint(max(1, case["tokens"] // 4), case["tokens"])
                               for _ in range(case["parents"] - 1)]
    # most children share all of it, some an earlier part
    return have, [(p, n if r.random() < 0.8 else r.randint(0, n))
                  for p, n in enumerate(have) for _ in range(case["each"])]


def _held(case):
    """[(pages shared with request 0, pages of its own, tokens)] of the live requests."""
    r = random.Random(case["lens"])
    page, out = case["page"], []
    for b in range(case["batch"]):
        n = case["tokens"] if b == 0 else r.randint(max(1, case["tokens"] // 4), case["tokens"])
        pages = _ceil(n, page)
        both = 0 if b == 0 else min(n // page, int(case["shared"] * out[0][1]))
        out.append((both, pages - both, n))
    return out


def _requests(case, seed=0):
    """(pages of each group's prefix, [(group, own tokens, rows)] of the requests)."""
    r = random.Random(case["lens"] + 7919 * seed)
    n, g, page = case["batch"], case["groups"], case["page"]
    cuts = sorted(r.sample(range(1, n), g - 1)) if g > 1 else []
    ptr = [0] + cuts + [n]
    pages = [max(1, case["prefix"] // page)] + \
        [max(1, r.randint(case["prefix"] // 4, case["prefix"]) // page) for _ in range(g - 1)]
    reqs = []
    for i in range(g):
        for _ in range(ptr[i + 1] - ptr[i]):
            rows = case["rows"] if r.random() < 0.7 else r.randint(1, case["rows"])
            reqs.append((i, max(rows, r.randint(max(1, case["owned"] // 4), case["owned"])), rows))
    return pages, reqs


def _bytes_of(case):
    """Bytes of a token's K and V (or latent) with its scales."""
    kind, h, d = case["kind"], case["heads"], case["dim"]
    if kind == "records":
        return 640 + 16
    if kind == "latent_bf16":
        return 1152
    return 2 * h * (d * (2 if kind == "bf16" else 1) + (4 if "token" in kind else 0))


def work(case):
    op = case["op"]
    if op == "fork":
        have, forks = _forked(case)
        page = case["page"]
        part = [n % page for _, n in forks]
        if case["tight"]:
            left = _free_pages(case)
            part = [t for i, t in enumerate(part) if t and sum(x > 0 for x in part[:i + 1]) <= left]
        return {"bytes": sum(8 * (n // page) for _, n in forks) + 28 * len(forks)
                + 2 * sum(part) * _bytes_of(case), "flops": 0}
    if op in ("free", "compact"):
        held, total = _held(case), _pages_in_all(case)
        entries = sum(a + b for a, b, _ in held)
        live = sum(b for _, b, _ in held)
        n = 4 * (entries + total - live) + 8 * len(held)
        if op == "free":
            return {"bytes": n, "flops": 0}
        moved = min(case["most"], _moves(case))
        return {"bytes": n + 4 * entries + 8 * moved + 2 * moved * case["page"] * _bytes_of(case),
                "flops": 0}
    pages, reqs = _requests(case)
    if op == "share":
        return {"bytes": 4 * sum(pages[g] for g, _, _ in reqs) + 20 * len(reqs) + 12 * len(pages),
                "flops": 0}
    d, hq, page = case["dim"], case["hq"], case["page"]
    per = 2 * case["hkv"] * (d * (2 if case["kind"] == "bf16" else 1) + (4 if "token" in case["kind"] else 0))
    rows = sum(r for _, _, r in reqs)
    toks = sum(pages) * page + sum(o for _, o, _ in reqs)
    seen = 0
    for i, (g, o, r) in enumerate(reqs):
        w = case["window"] if i % 2 else 0
        for k in range(r):
            pos = pages[g] * page + o - r + k + 1
            seen += min(pos, w) if w > 0 else pos
    return {"bytes": toks * per + rows * hq * (d * (1 if case["q8"] else 2) + 2 * d + 4),
            "flops": 4 * d * hq * seen}


def _free_pages(case):
    """Length of the free list of a fork: a few more than it takes, or half of it."""
    need = sum(n % case["page"] > 0 for _, n in _forked(case)[1])
    return need // 2 if case["tight"] else need + 5


def _pages_in_all(case):
    live = sum(b for _, b, _ in _held(case))
    return live + int(case["spare"] * live) + 1


def _layout(case):
    """The live pages' ids, in the order in which the requests take them."""
    total, held = _pages_in_all(case), _held(case)
    ids = list(range(total))
    random.Random(case["lens"] + 1).shuffle(ids)
    return ids[:sum(b for _, b, _ in held)]


def _moves(case):
    ids = _layout(case)
    return sum(i >= len(ids) for i in ids)


# ------------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_dev())


def _cache(st, g, pages, page, heads, dim, kind, hnd):
    """Filled caches of both sides in the formats of the plan, [pages, P, H, .] (or H first)."""
    dev = _dev()
    shape = (pages, heads, page) if hnd else (pages, page, heads)

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    for side in ("k",) if dim == 576 else ("k", "v"):
        if kind == "records":
            c = torch.randint(0, 255, (*shape, 640), generator=g, device=dev, dtype=torch.uint8)
            c[..., :512] = randn(*shape, 512).mul_(100).clamp_(-448, 448).to(E4M3).view(torch.uint8)
            c[..., 512:] = randn(*shape, 64).to(torch.bfloat16).view(torch.uint8)
            st[side + "_scale"] = torch.rand(pages, page, heads, 4, generator=g, device=dev) + 0.1
        elif "bf16" in kind:
            c = randn(*shape, dim).to(torch.bfloat16)
        else:
            x = randn(*shape, dim).to(torch.bfloat16).float()
            top = 127.0 if "int8" in kind else 448.0
            if "token" in kind:
                s = x.abs().amax(-1) / top  # [pages, P, H] (or H first); the scales are token first
                st[side + "_scale"] = (s.transpose(1, 2) if hnd else s).contiguous()
                x.div_(s[..., None])
            else:
                s = x.abs().amax() / top
                st[side + "_scale"] = s.reshape(1)
                x.div_(s)
            x.clamp_(-top, top)
            c = x.round_().to(torch.int8) if "int8" in kind else x.to(E4M3).view(torch.uint8)
        st[side + "_pages"] = c


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(seed * 1000003 + 29)
    op, page, st = case["op"], case["page"], dict(case=case)

    def perm(n):
        return torch.randperm(n, generator=g, device=dev).int()

    if op == "fork":
        have, forks = _forked(case)
        npg = [_ceil(n, page) for n in have]
        free, rows = _free_pages(case), len(have) + len(forks)
        ids, cols = perm(sum(npg) + free + 3), max(npg) + 2
        table = torch.full((rows, cols), -1, dtype=torch.int32, device=dev)
        at = torch.arange(cols, device=dev)[None] < _ints(npg)[:, None]
        held = table[:len(have)].clone()
        held[at] = ids[:sum(npg)]
        order = perm(rows).long()  # table rows of the parents, then of the children
        table[order[:len(have)]] = held
        st.update(block_table=table, parent=order[_ints([p for p, _ in forks]).long()].int(),
                  child=order[len(have):].int().contiguous(), shared_len=_ints([n for _, n in forks]),
                  free_pages=ids[sum(npg):sum(npg) + free].contiguous(), free_count=_ints([free]),
                  out=dict(free_left=_ints([-1]), child_len=_ints([-1] * len(forks)),
                           copy_src=_ints([-1] * len(forks)), copy_dst=_ints([-1] * len(forks)),
                           copy_tokens=_ints([-1] * len(forks)), block_table=table))
        _cache(st, g, ids.numel(), page, case["heads"], case["dim"], case["kind"], case["hnd"])
        if own:
            st["dec"] = _decoder(case, ids.numel(), batch=1, max_kv=case["tokens"])
        return st
    if op in ("free", "compact"):
        held, total = _held(case), _pages_in_all(case)
        npg = [a + b for a, b, _ in held]
        cols, rows = max(npg) + 1, len(held) + 2
        # where the pages lie is the case's; which row holds a request is the seed's
        # (nothing moves where pages are only freed: there the ids are the seed's too)
        ids, at, tab = perm(total).tolist() if op == "free" else _layout(case), 0, []
        for a, b, _ in held:
            row = (tab[0][:a] if a else []) + ids[at:at + b]
            at += b
            tab.append(row)
        full = [r + [-1] * (cols - len(r)) for r in tab]
        order = perm(rows)
        table = torch.full((rows, cols), -1, dtype=torch.int32, device=dev)
        table[order[:len(held)].long()] = _ints(full)
        st.update(lengths=_ints([n for _, _, n in held]), request=order[:len(held)].contiguous(),
                  block_table=table, pages=total)
        st["out"] = dict(free_pages=torch.full((total,), -1, dtype=torch.int32, device=dev),
                         free_left=_ints([-1]))
        if op == "compact":
            most = min(case["most"], total)
            st["out"].update(new_table=table.clone(), num_copies=_ints([-1]),
                             copy_src=torch.full((most,), -1, dtype=torch.int32, device=dev),
                             copy_dst=torch.full((most,), -1, dtype=torch.int32, device=dev))
            _cache(st, g, total, page, case["heads"], case["dim"], case["kind"], case["hnd"])
        if own:
            from paged_split_kv_03_gb300 import binding as B
            c = case if op == "compact" else dict(case, heads=1, dim=128, kind="bf16", hnd=False)
            st["dec"] = _decoder(c, total, batch=len(held), max_kv=case["tokens"])
            st["pool"] = B.Pages(st["dec"].plan)
        return st
    # (tables are all lengths: every seed has its own ones, alike to those that `work` counts)
    pages, reqs = _requests(case, seed if op == "share" else 0)
    own_pages = [_ceil(o, page) for _, o, _ in reqs]
    total = sum(pages) + sum(own_pages) + 2
    ids = perm(total)
    cut = [0]
    for n in pages + own_pages:
        cut.append(cut[-1] + n)
    parts = [ids[cut[i]:cut[i + 1]] for i in range(len(cut) - 1)]
    table = torch.cat([torch.cat([parts[q[0]], parts[len(pages) + b]]) for b, q in enumerate(reqs)])
    ptr = [0]
    for b, q in enumerate(reqs):
        ptr.append(ptr[-1] + pages[q[0]] + own_pages[b])
    qo, gp = [0], [0]
    for _, _, r in reqs:
        qo.append(qo[-1] + r)
    for i in range(len(pages)):
        gp.append(gp[-1] + sum(q[0] == i for q in reqs))
    n = len(reqs)
    st.update(page_table=table.contiguous(), kv_indptr=_ints(ptr), qo_indptr=_ints(qo),
              group_indptr=_ints(gp), kv_len=_ints([pages[q[0]] * page + q[1] for q in reqs]),
              window=_ints([case["window"] if b % 2 else 0 for b in range(n)])
              if case["window"] > 0 else None,
              prefix=torch.full((len(pages), 2), -1, dtype=torch.int32, device=dev),
              own_indptr=_ints([-1] * n), own_len=_ints([-1] * n))
    c = dict(case, heads=1, dim=128, kind="bf16", hnd=False) if op == "share" else \
        dict(case, heads=case["hkv"])
    if op == "decode":
        _cache(st, g, total, page, case["hkv"], case["dim"], case["kind"], case["hnd"])
        q = torch.randn(qo[-1], case["hq"], case["dim"], generator=g, device=dev)
        st["q_scale"] = 1.0
        if case["q8"]:
            st["q_scale"] = 0.0125
            st["q"] = (q / 0.0125).clamp(-448, 448).to(E4M3)
        else:
            st["q"] = q.to(torch.bfloat16)
        st["out"] = torch.zeros(q.shape, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(q.shape[:2], device=dev)
    if own:
        from paged_split_kv_03_gb300 import binding as B
        st["dec"] = _decoder(c, total, batch=n, max_q=case["rows"],
                             max_kv=max(pages) * page + case["owned"])
        st["shared"] = B.Shared(st["dec"].plan, len(pages), max(case["owned"], 8))
        if op == "decode":  # the step's tables, once for the layers that use them
            _share(st)
    return st


def _decoder(c, pages, batch, max_kv, max_q=1):
    """The plan and scratch that a serving program keeps."""
    from paged_split_kv_03_gb300 import binding as B
    kind, h, page = c["kind"], c["heads"], c["page"]
    w = 640 if kind == "records" else c["dim"]
    p = B.PdaParams(num_qo_heads=c.get("hq", h), num_kv_heads=h, head_dim=c["dim"], page_size=page,
                    max_batch=batch, max_q_len=max_q, max_kv_len=max(1, max_kv), num_pages=pages,
                    kv_stride_page=page * h * w, kv_stride_token=w if c["hnd"] else h * w,
                    kv_stride_head=page * w if c["hnd"] else w, device=_dev().index)
    if c["dim"] == 576:
        p.head_dim_v = 512
    if "bf16" not in kind:
        p.kv_dtype = B.PDA_INT8 if "int8" in kind else B.PDA_E4M3
        p.scale_mode = B.PDA_SCALE_MLA_BLOCK if kind == "records" else \
            B.PDA_SCALE_TOKEN_HEAD if "token" in kind else B.PDA_SCALE_TENSOR
    p.q_dtype = B.PDA_E4M3 if c.get("q8") else B.PDA_BF16
    return B.Decoder(p, device=_dev())


# ------------------------------------------------------------------ one pass

def run(st):
    return _OPS[st["case"]["op"]](st)


def _fork(st):
    o, p = st["out"], st["case"]["page"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_fork_tables(st["dec"].plan, st["parent"], st["child"], st["shared_len"],
                          st["block_table"], st["free_pages"], st["free_count"], o["free_left"],
                          o["child_len"], o["copy_src"], o["copy_dst"], o["copy_tokens"],
                          st["dec"].scratch)
        B.pda_copy_pages(st["dec"].plan, st["k_pages"], st.get("v_pages"), st.get("k_scale"),
                         st.get("v_scale"), o["copy_src"], o["copy_dst"], o["copy_tokens"], None,
                         st["dec"].scratch)
        return o, _values(st)
    n, free, tab = st["shared_len"].long(), st["free_count"].long(), st["block_table"]
    full, part = n // p, n % p > 0
    upto = part.long().cumsum(0)
    granted = ~part | (upto <= free)
    takes = part & granted
    new = st["free_pages"][torch.where(takes, free - upto, 0)] if st["free_pages"].numel() else \
        torch.full_like(st["parent"], -1)
    j = torch.arange(tab.shape[1], device=n.device)
    theirs = tab[st["parent"].long()]
    mine = tab[st["child"].long()]
    src = theirs.gather(1, full.clamp(max=tab.shape[1] - 1)[:, None])[:, 0]
    mine = torch.where((j < full[:, None]) & granted[:, None], theirs, mine)
    mine = torch.where((j == full[:, None]) & takes[:, None], new[:, None], mine)
    tab[st["child"].long()] = mine
    o["child_len"].copy_(torch.where(granted, n, 0))
    o["copy_src"].copy_(torch.where(takes, src, -1))
    o["copy_dst"].copy_(torch.where(takes, new, -1))
    o["copy_tokens"].copy_(torch.where(takes, n % p, 0))
    o["free_left"].copy_(free - torch.where(takes, upto, 0).amax())
    _copy(st, o["copy_src"], o["copy_dst"], o["copy_tokens"])
    return o, _values(st)


def _copy(st, src, dst, tokens):
    """The first tokens of pages src into pages dst."""
    ok = src >= 0
    src, dst = src[ok].long(), dst[ok].long()
    p, hnd = st["case"]["page"], st["case"]["hnd"]
    keep = None if tokens is None else torch.arange(p, device=src.device) < tokens[ok][:, None]
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        x = st.get(name)
        if x is None or x.dim() == 1:
            continue
        first = x.dim() > 2 and hnd and name.endswith("pages")
        if keep is None:
            x[dst] = x[src]
        else:
            k = keep[:, None, :] if first else keep[:, :, None]
            x[dst] = torch.where(k if x.dim() == 3 else k[..., None], x[src], x[dst])


def _values(st):
    """The caches as the values their codes stand for, and their scales."""
    got, kind = {}, st["case"]["kind"]
    for side in ("k", "v"):
        x = st.get(side + "_pages")
        if x is None:
            continue
        if kind == "records":
            got[side + "_nope"] = x[..., :512].view(E4M3)
            got[side + "_rope"] = x[..., 512:].view(torch.bfloat16)
        else:
            got[side] = x.view(E4M3) if x.dtype == torch.uint8 else x
        if "token" in kind or kind == "records":
            got[side + "_scale"] = st[side + "_scale"]
    return got


def _live(st):
    """Whether a request holds each page."""
    tab = st["block_table"][st["request"].long()].long()
    n = (st["lengths"].long() + st["case"]["page"] - 1) // st["case"]["page"]
    held = torch.arange(tab.shape[1], device=tab.device) < n[:, None]
    live = torch.zeros(st["pages"] + 1, dtype=torch.bool, device=tab.device)
    live[torch.where(held, tab, st["pages"])] = True
    return live[:-1], held


def _list_free(st, live):
    """The pages that nobody holds, the lowest id last."""
    o, n = st["out"], st["pages"]
    free = ~live
    after = free.flip(0).cumsum(0).flip(0) - 1  # free ids above each
    buf = torch.cat([o["free_pages"], o["free_pages"][:1]])
    buf[torch.where(free, after, n)] = torch.arange(n, dtype=torch.int32, device=live.device)
    o["free_pages"].copy_(buf[:n])
    o["free_left"].copy_(free.sum())


def _free(st):
    if own:
        from paged_split_kv_03_gb300 import binding as B
        o = st["out"]
        B.pda_free_pages(st["dec"].plan, st["lengths"], st["request"], st["block_table"],
                         o["free_pages"], o["free_left"], st["pool"].scratch)
        return o
    live, _ = _live(st)
    _list_free(st, live)
    return st["out"]


def _compact(st):
    o = st["out"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_compact_pages(st["dec"].plan, st["lengths"], st["request"], st["block_table"],
                            o["new_table"], o["free_pages"], o["free_left"], o["copy_src"],
                            o["copy_dst"], o["num_copies"], st["pool"].scratch)
        B.pda_copy_pages(st["dec"].plan, st["k_pages"], st.get("v_pages"), st.get("k_scale"),
                         st.get("v_scale"), o["copy_src"], o["copy_dst"], None, o["num_copies"],
                         st["dec"].scratch)
        return o, _values(st)
    n, dev = st["pages"], st["block_table"].device
    live, held = _live(st)
    ids = torch.arange(n, device=dev)
    count = live.sum()
    above = live.flip(0).cumsum(0).flip(0) - 1   # live ids above each live one
    below = (~live).cumsum(0) - 1                # holes below each hole
    most = o["copy_src"].numel()
    moves = (live & (ids >= count)).sum().clamp(max=most)
    moved, filled = live & (above < moves), ~live & (below < moves)
    src = torch.full((n + 1,), -1, dtype=torch.int64, device=dev)
    dst = src.clone()
    src[torch.where(moved, above, n)] = ids
    dst[torch.where(filled, below, n)] = ids
    to = torch.where(moved, dst[torch.where(moved, above, 0)], ids)
    k = torch.arange(most, device=dev) < moves
    o["copy_src"].copy_(torch.where(k, src[:most], o["copy_src"]))
    o["copy_dst"].copy_(torch.where(k, dst[:most], o["copy_dst"]))
    o["num_copies"].copy_(moves)
    rows = st["request"].long()
    tab = st["block_table"][rows].long()
    new = torch.where(held, to[torch.where(held, tab, 0)], o["new_table"][rows].long())
    o["new_table"][rows] = new.int()
    _list_free(st, (live & ~moved) | filled)
    _copy(st, torch.where(k, o["copy_src"], -1), o["copy_dst"], None)
    return o, _values(st)


def _share(st):
    c = st["case"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_share_tables(st["shared"].plan, st["page_table"], st["kv_indptr"], st["kv_len"],
                           st["qo_indptr"], st["window"], st["group_indptr"], st["prefix"],
                           st["own_indptr"], st["own_len"], st["shared"].scratch)
        return st["prefix"], st["own_indptr"], st["own_len"]
    p, n, dev = c["page"], c["batch"], st["kv_len"].device
    length, ptr = st["kv_len"].long(), st["kv_indptr"].long()
    rows = st["qo_indptr"].long().diff()
    group = torch.searchsorted(st["group_indptr"][1:].long(), torch.arange(n, device=dev), right=True)
    most = (length - rows) // p  # whole pages in front of the rows
    j = torch.arange(int(c["prefix"] // p) + c["owned"] // p + 2, device=dev)
    last = st["page_table"].numel() - 1
    mine = st["page_table"][(ptr[:-1, None] + j).clamp(max=last)]
    first = st["group_indptr"].long()[group]
    same = (mine == mine[first]) & (j < most[:, None])
    pages = same.long().cumprod(1).sum(1)
    end = torch.full((c["groups"],), 1 << 40, device=dev).scatter_reduce_(0, group, pages, "amin") * p
    lo = torch.zeros_like(length)
    if st["window"] is not None:
        w = st["window"].long()
        lo = torch.where(w > 0, (length - rows - w + 1).clamp(min=0), 0)
    low = torch.full((c["groups"],), 1 << 40, device=dev).scatter_reduce_(0, group, lo, "amin")
    st["prefix"].copy_(torch.stack([torch.minimum(low // p * p, end), end], 1))
    st["own_indptr"].copy_(ptr[:-1] + end[group] // p)
    st["own_len"].copy_(length - end[group])
    return st["prefix"], st["own_indptr"], st["own_len"]


def _keys(st, b, lens, dtype):
    """Dequantised (k, v) of request b, [Hkv, L, D]."""
    c = st["case"]
    p, n = c["page"], lens[b]
    at = st["starts"][b]
    ids = st["page_table"][at:at + _ceil(n, p)].long()
    got = []
    for side in ("k", "v"):
        x = st[side + "_pages"][ids]
        x = (x.view(E4M3) if x.dtype == torch.uint8 else x).to(dtype)
        x = x.transpose(0, 1) if c["hnd"] else x.permute(2, 0, 1, 3)  # [H, pages, P, D]
        x = x.reshape(c["hkv"], -1, c["dim"])[:, :n]
        s = st.get(side + "_scale")
        if "token" in c["kind"]:
            x = x * s[ids].to(dtype).reshape(-1, c["hkv"]).t()[:, :n, None]
        elif s is not None:
            x = x * s.to(dtype)
        got.append(x)
    return got


def _lens(st):
    """Host copies of what the case says of its requests: lengths, rows' offsets."""
    c = st["case"]
    pages, reqs = _requests(c)
    lens, qo, at = [], [0], [0]
    for g, o, r in reqs:
        lens.append(pages[g] * c["page"] + o)
        qo.append(qo[-1] + r)
        at.append(at[-1] + pages[g] + _ceil(o, c["page"]))
    st["starts"] = at
    return lens, qo


def _decode(st):
    c = st["case"]
    scale = c["dim"] ** -0.5 * st["q_scale"]
    if own:
        from paged_split_kv_03_gb300 import binding as B
        B.pda_decode_shared(st["shared"].plan, st["q"], st["k_pages"], st["v_pages"],
                            st["page_table"], st["kv_indptr"], st["kv_len"], st["qo_indptr"],
                            c["rows"], st["window"], st["group_indptr"], st["prefix"],
                            st["own_indptr"], st["own_len"], scale, st.get("k_scale"),
                            st.get("v_scale"), st["out"], st["lse"], st["shared"].scratch)
        return st["out"], st["lse"]
    lens, qo = _lens(st)
    for b, n in enumerate(lens):
        k, v = _keys(st, b, lens, torch.float32)
        q = st["q"][qo[b]:qo[b + 1]].float()
        rows = q.shape[0]
        q = q.reshape(rows, c["hkv"], -1, c["dim"]).transpose(0, 1)  # [Hkv, R, group, D]
        x = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)) * scale  # [Hkv, R * group, L]
        pos = n - rows + torch.arange(rows, device=k.device)
        j = torch.arange(n, device=k.device)
        see = j <= pos[:, None]
        if st["window"] is not None and b % 2:
            see = see & (j > pos[:, None] - c["window"])
        see = see.repeat_interleave(c["hq"] // c["hkv"], 0)
        x = x.masked_fill(~see, -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        o = torch.matmul(e, v) / z
        st["out"][qo[b]:qo[b + 1]] = o.unflatten(1, (rows, -1)).transpose(0, 1).flatten(1, 2) \
            .to(torch.bfloat16)
        st["lse"][qo[b]:qo[b + 1]] = (m + torch.log(z))[..., 0].unflatten(1, (rows, -1)) \
            .transpose(0, 1).flatten(1, 2)
    return st["out"], st["lse"]


_OPS = dict(fork=_fork, free=_free, compact=_compact, share=_share, decode=_decode)


# -------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["op"] != "decode":
        return None  # whole numbers, and pages that are moved as they are
    st = prepare(case, seed)
    lens, qo = _lens(st)
    group = case["hq"] // case["hkv"]
    out = torch.empty(st["out"].shape, dtype=torch.float64, device=_dev())
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=_dev())
    for b, n in enumerate(lens):
        k, v = _keys(st, b, lens, torch.float64)
        r0, r1 = qo[b], qo[b + 1]
        q = st["q"][r0:r1].double() * st["q_scale"]
        at = n - (r1 - r0) + torch.arange(r1 - r0, device=_dev())[:, None]
        key = torch.arange(n, device=_dev())[None]
        hide = key > at
        if case["window"] > 0 and b % 2:
            hide = hide | (key < at - case["window"] + 1)
        for h in range(case["hq"]):
            s = q[:, h] @ k[h // group].t() / math.sqrt(case["dim"])
            s[hide] = -math.inf
            top = torch.logsumexp(s, 1)
            lse[r0:r1, h] = top
            out[r0:r1, h] = torch.exp(s - top[:, None]) @ v[h // group]
    return out, lse
