"""Plain implementations of the calls over shared pages, from their definitions: forks,
the free list, moves that bring pages together, copies of pages, and the prefixes that
the requests of a group share."""
import torch

from paged_split_kv_03_gb300 import binding as B


def ceil(a, b):
    return -(-a // b)


def plan_params(kind="bf16", *, heads=2, dim=128, page=16, pages=8, batch=1, max_kv=1 << 20, max_q=1,
                hq=None, hnd=False, q8=False, gap=0, **kw):
    """Plan of a cache; ``gap``: channels left unused behind every head's row."""
    if kind in ("records", "latent", "latent_e4m3"):
        dim, heads = 576, 1
    w = (640 if kind == "records" else dim) + gap
    p = B.PdaParams(num_qo_heads=hq or heads, num_kv_heads=heads, head_dim=dim, page_size=page,
                    max_batch=batch, max_q_len=max_q, max_kv_len=max_kv, num_pages=pages,
                    kv_stride_page=page * heads * w, kv_stride_token=w if hnd else heads * w,
                    kv_stride_head=page * w if hnd else w)
    if dim == 576:
        p.head_dim_v = 512
    if kind not in ("bf16", "latent"):
        p.kv_dtype = B.PDA_INT8 if "int8" in kind else B.PDA_E4M3
        p.scale_mode = B.PDA_SCALE_MLA_BLOCK if kind == "records" else \
            B.PDA_SCALE_TOKEN_HEAD if "token" in kind else B.PDA_SCALE_TENSOR
    if q8 or kind == "latent_e4m3":
        p.q_dtype = B.PDA_E4M3
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def fork(parent, child, lens, block, free_pages, free_count, *, page, max_kv, num_pages):
    """(outputs of pda_fork_tables, status bits); ``block`` is changed."""
    rows, cols = len(block), len(block[0]) if block else 0
    out = dict(child_len=[], copy_src=[], copy_dst=[], copy_tokens=[])
    status, taken = 0, 0
    for p, c, n in zip(parent, child, lens):
        bad = not (0 <= p < rows and 0 <= c < rows) or p == c or n < 0 or ceil(max(n, 0), page) > cols
        if n > max_kv:
            bad = True
            status |= B.PDA_STATUS_KV_LEN_GT_MAX
        if bad:
            status |= B.PDA_STATUS_TABLE_INVALID
        ends_inside = not bad and n % page != 0
        taken += ends_inside
        copy = (-1, -1, 0)
        granted = not bad and (not ends_inside or taken <= free_count)
        if not bad and not granted:
            status |= B.PDA_STATUS_NO_PAGES
        if granted:
            for j in range(n // page):
                block[c][j] = block[p][j]
                if not 0 <= block[p][j] < num_pages:
                    status |= B.PDA_STATUS_PAGE_OOB
            if ends_inside:
                new, old = free_pages[free_count - taken], block[p][n // page]
                block[c][n // page] = new
                if 0 <= old < num_pages and 0 <= new < num_pages:
                    copy = (old, new, n % page)
                else:
                    status |= B.PDA_STATUS_PAGE_OOB
        out["child_len"].append(n if granted else 0)
        for k, v in zip(("copy_src", "copy_dst", "copy_tokens"), copy):
            out[k].append(v)
    out["free_left"] = [free_count - min(taken, free_count)]
    out["block_table"] = block
    return out, status


def compact(lengths, request, block, *, page, max_kv, num_pages, most=0):
    """(outputs of pda_compact_pages with at most ``most`` moves, status bits): with none, its
    free list is pda_free_pages'."""
    rows, cols = len(block), len(block[0]) if block else 0
    status, held = 0, []
    for b, n in enumerate(lengths):
        row = request[b] if request else b
        if n < 0 or not 0 <= row < rows:
            status |= B.PDA_STATUS_TABLE_INVALID
            continue
        if n > max_kv:
            status |= B.PDA_STATUS_KV_LEN_GT_MAX | B.PDA_STATUS_TABLE_INVALID
        if ceil(n, page) > cols:
            status |= B.PDA_STATUS_TABLE_INVALID
        held.append((row, min(ceil(n, page), cols)))
    live = set()
    for row, k in held:
        for x in block[row][:k]:
            if 0 <= x < num_pages:
                live.add(x)
            else:
                status |= B.PDA_STATUS_PAGE_OOB
    src, dst = [], []
    high = sorted(live, reverse=True)
    low = [x for x in range(num_pages) if x not in live]
    for s, d in zip(high, low):
        if s < d or len(src) == most:
            break
        src.append(s)
        dst.append(d)
    to = dict(zip(src, dst))
    new = [list(r) for r in block]
    for row, k in held:
        new[row][:k] = [to.get(x, x) for x in block[row][:k]]
    after = (live - set(src)) | set(dst)
    free = [x for x in reversed(range(num_pages)) if x not in after]
    return dict(new_table=new, copy_src=src, copy_dst=dst, num_copies=[len(src)], free_pages=free,
                free_left=[len(free)]), status


def copy(tensor, src, dst, tokens, page, slot_dim):
    """The first tokens of pages ``src`` of a tensor [pages, ...] into pages ``dst``; ``slot_dim``:
    the dimension of a page that counts its tokens."""
    out = tensor.clone()
    for i, (s, d) in enumerate(zip(src, dst)):
        if s == -1 or d == -1 or not (0 <= s < tensor.shape[0] and 0 <= d < tensor.shape[0]):
            continue
        t = page if tokens is None else max(0, min(page, tokens[i]))
        out[d].narrow(slot_dim, 0, t).copy_(tensor[s].narrow(slot_dim, 0, t))
    return out


def share(page_table, kv_indptr, kv_len, qo_indptr, windows, group_indptr, *, page, max_q, max_kv,
          num_pages):
    """(prefix, own_indptr, own_len) of pda_share_tables and its status bits."""
    prefix, status = [], 0
    own_ptr, own_len = [None] * len(kv_len), [None] * len(kv_len)
    for g in range(len(group_indptr) - 1):
        fits = {}
        for b in range(group_indptr[g], group_indptr[g + 1]):
            rows, n = qo_indptr[b + 1] - qo_indptr[b], kv_len[b]
            if rows == 0:
                fits[b] = None
                continue
            bits = (B.PDA_STATUS_ROWS_GT_MAX if rows < 0 or rows > max_q else 0) | \
                (B.PDA_STATUS_KV_LEN_LT_ROWS if n < rows else 0) | \
                (B.PDA_STATUS_KV_LEN_GT_MAX if n > max_kv else 0)
            status |= bits
            fits[b] = not bits
        good = [b for b, ok in fits.items() if ok]
        common, lo = None, None
        for b in good:
            rows, n = qo_indptr[b + 1] - qo_indptr[b], kv_len[b]
            k = 0
            while k < min((n - rows) // page, kv_indptr[b + 1] - kv_indptr[b]):
                x, y = page_table[kv_indptr[b] + k], page_table[kv_indptr[good[0]] + k]
                if x != y or not 0 <= x < num_pages or k >= kv_indptr[good[0] + 1] - kv_indptr[good[0]]:
                    break
                k += 1
            common = k if common is None else min(common, k)
            first = max(0, n - rows - windows[b] + 1) if windows and windows[b] > 0 else 0
            lo = first if lo is None else min(lo, first)
        end = (common or 0) * page
        prefix += [min((lo or 0) // page * page, end), end]
        for b, ok in fits.items():
            own_ptr[b] = kv_indptr[b] + end // page
            own_len[b] = 0 if ok is None else kv_len[b] - end if ok else -1
    return (prefix, own_ptr, own_len), status


def filled(g, pages, page, heads, kind, dim, hnd=False):
    """A cache of random bytes in the plan's format (K, or a latent), and its scales or None."""
    if kind in ("records", "latent", "latent_e4m3"):
        dim, heads = 576, 1
    width = 640 if kind == "records" else dim
    shape = (pages, heads, page, width) if hnd else (pages, page, heads, width)
    if kind in ("bf16", "latent"):
        c = torch.randn(*shape, generator=g).to(torch.bfloat16)
    else:
        c = torch.randint(0, 120, shape, generator=g, dtype=torch.uint8)
        if "int8" in kind:
            c = c.view(torch.int8)
    s = None
    if "token" in kind:
        s = torch.rand(pages, page, heads, generator=g)
    elif kind == "records":
        s = torch.rand(pages, page, heads, 4, generator=g)
    return c, s
