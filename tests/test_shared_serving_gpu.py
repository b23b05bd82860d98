"""The calls over shared pages used together, as a server uses them: forks of a prompt, decode
steps behind what they share, requests that end, the pages freed, moved and decoded from
again, against a host copy of every request's tokens; and the same calls captured into
CUDA graphs, on other streams, and beside one another."""
from __future__ import annotations

import random
import types

import pytest
import torch

import pages_ref as ref
import shared_ref as S
from paged_split_kv_03_gb300 import binding as B
from test_shared_gpu import check, parity, reqs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    """``rows`` requests' table rows over one cache; ``kept`` holds what each has cached."""

    def __init__(self, kind, rows, pages=120, page=16, dim=128, hkv=2, group=4, cols=24, seed=0):
        self.kind, self.page, self.dim, self.hkv, self.group = kind, page, dim, hkv, group
        self.g = torch.Generator().manual_seed(seed)
        self.n, self.pages = rows, pages
        p = ref.plan_params(kind, heads=hkv, dim=dim, page=page, pages=pages, batch=rows,
                            max_kv=page * cols, hq=hkv * group)
        self.dec = B.Decoder(p, device=DEV)
        self.shared, self.held = B.Shared(self.dec.plan, 1, 200), B.Pages(self.dec.plan)
        self.block = torch.full((rows, cols), -7, dtype=torch.int32, device=DEV)
        self.free = ints(list(range(pages - 1, -1, -1)))
        self.count, self.left = ints([pages]), ints([0])
        dt = torch.bfloat16 if kind == "bf16" else torch.uint8
        self.cache = [torch.zeros(pages, page, hkv, dim, dtype=dt, device=DEV) for _ in "kv"]
        self.scale = [torch.zeros(pages, page, hkv, device=DEV) if "token" in kind else None for _ in "kv"]
        self.kept = [[] for _ in range(rows)]  # [(k, v) of a token], in 64 bits

    def grow(self, order, new):
        """One step's tables; the new tokens' K and V are random."""
        n, cap = self.n, sum(new)
        cached = [len(self.kept[r]) for r in order]
        self.kv_len, self.own_len, self.own_indptr = ints([0] * n), ints([0] * n), ints([0] * n)
        self.kv_indptr, self.qo_indptr = ints([0] * (n + 1)), ints([0] * (n + 1))
        self.page_table = ints([-7] * self.block.numel())
        slots = torch.full((cap,), -1, dtype=torch.int64, device=DEV)
        B.pda_build_tables(self.dec.plan, ints(cached), ints(new), ints(order), self.block, self.free, self.count,
                           self.left, self.kv_len, self.kv_indptr, self.page_table, self.qo_indptr, None, slots,
                           None, self.dec.scratch)
        self.count, self.left = self.left, self.count
        x = [torch.randn(cap, self.hkv, self.dim, generator=self.g).to(torch.bfloat16).to(DEV) for _ in "kv"]
        B.pda_append_slots(self.dec.plan, *x, slots, None, *self.cache, *self.scale, self.dec.scratch)
        assert self.dec.status() == 0
        at, got = slots.cpu(), []
        for c, s in zip(self.cache, self.scale):
            val = c if self.kind == "bf16" else c.view(torch.float8_e4m3fn)
            val = val.reshape(-1, self.hkv, self.dim)[at.to(DEV)].double().cpu()
            got.append(val if s is None else val * s.reshape(-1, self.hkv)[at.to(DEV)].double().cpu()[..., None])
        i = 0
        for r, k in zip(order, new):
            for _ in range(k):
                self.kept[r].append((got[0][i], got[1][i]))
                i += 1

    def fork(self, parent, children, shared):
        m = len(children)
        out = [ints([-9] * m) for _ in range(4)]
        B.pda_fork_tables(self.dec.plan, ints([parent] * m), ints(children), ints(shared), self.block, self.free,
                          self.count, self.left, *out, self.dec.scratch)
        B.pda_copy_pages(self.dec.plan, *self.cache, *self.scale, *out[1:], None, self.dec.scratch)
        self.count, self.left = self.left, self.count
        assert out[0].tolist() == shared and self.dec.status() == 0
        for c, k in zip(children, shared):
            self.kept[c] = self.kept[parent][:k]

    def step(self, order, live):
        """The first ``live`` requests of ``order`` decode a token, checked in 64 bits."""
        self.grow(order, [1] * live + [0] * (self.n - live))
        hq = self.hkv * self.group
        q = torch.randn(live, hq, self.dim, generator=self.g).to(torch.bfloat16).to(DEV)
        out, lse = torch.empty_like(q), torch.empty(live, hq, device=DEV)
        prefix = ints([[-9, -9]])
        a = (self.page_table, self.kv_indptr, self.kv_len, self.qo_indptr, None, None, prefix, self.own_indptr,
             self.own_len)
        B.pda_share_tables(self.shared.plan, *a, self.shared.scratch)
        B.pda_decode_shared(self.shared.plan, q, *self.cache, *a[:4], 1, *a[4:], self.dim ** -0.5, *self.scale, out,
                            lse, self.shared.scratch)
        assert self.shared.status() == 0
        # the same tokens in pages of their own
        lens = [len(self.kept[r]) for r in order]
        need = [ref.ceil(k, self.page) for k in lens]
        values = [torch.zeros(sum(need) + 1, self.page, self.hkv, self.dim, dtype=torch.float64) for _ in "kv"]
        tables, at = [], 0
        for r, k in zip(order, need):
            tables.append(list(range(at, at + k)))
            for side in (0, 1):
                if k:
                    rows = torch.stack([t[side] for t in self.kept[r]])
                    values[side][at:at + k].reshape(-1, self.hkv, self.dim)[:len(rows)] = rows
            at += k
        w = types.SimpleNamespace(kind=self.kind, dim=self.dim, page=self.page, hkv=self.hkv, hq=hq,
                                  group=self.group, hnd=False, q=q, q_scale=1.0, tables=tables, kv_len=lens,
                                  rows=[1] * live + [0] * (self.n - live),
                                  qo=[min(k, live) for k in range(self.n + 1)], windows=None, values=values)
        o, ob, l, lb = S.attention(w)
        check(out, o, ob, "out")
        check(lse, l, lb, "lse")
        return prefix.tolist()[0]

    def free_list(self, order, compact=None):
        """The pages that the requests of ``order`` hold, the others' freed (and all moved)."""
        lens, rows = ints([len(self.kept[r]) for r in order]), ints(order)
        pool = ints([-7] * self.pages)
        if compact is None:
            B.pda_free_pages(self.dec.plan, lens, rows, self.block, pool, self.left, self.held.scratch)
        else:
            src, dst, num = ints([-9] * compact), ints([-9] * compact), ints([-9])
            B.pda_compact_pages(self.dec.plan, lens, rows, self.block, self.block, pool, self.left, src, dst, num,
                                self.held.scratch)
            B.pda_copy_pages(self.dec.plan, *self.cache, *self.scale, src, dst, None, num, self.dec.scratch)
        self.count, self.left = self.left, self.count
        self.free = pool
        left = self.count.item()
        block = self.block.cpu()
        live = {int(block[r, j]) for r in order for j in range(ref.ceil(len(self.kept[r]), self.page))}
        assert pool[:left].tolist() == [p for p in range(self.pages - 1, -1, -1) if p not in live]
        assert self.held.status() == 0 and self.dec.status() == 0
        return live


@pytest.mark.parametrize("kind", ["bf16", "e4m3_token"])
def test_a_server(kind):
    s = Server(kind, 6)
    order = list(range(6))
    s.grow(order, [150, 0, 0, 0, 0, 0])
    # four answers share the prompt, one of them an earlier part of it
    s.fork(0, [1, 2, 3, 4], [150, 150, 144, 100])
    for _ in range(3):
        assert s.step(order, 5) == [0, 96]  # whole pages of 100 tokens
    # two end, one starts over behind what is left of the prompt's first page
    s.kept[1], s.kept[4] = [], []
    live = s.free_list([0, 2, 3])
    s.fork(2, [5], [7])
    order = [5, 0, 2, 3, 1, 4]
    assert s.step(order, 4) == [0, 0]  # its page was copied, so none is shared
    assert s.step([0, 2, 3, 5, 1, 4], 3) == [0, 144]
    # without the short one the rest moves to the front, and goes on
    s.kept[5] = []
    live = s.free_list([0, 2, 3], compact=40)
    assert live == set(range(len(live)))
    order = [3, 2, 0, 1, 4, 5]
    for _ in range(20):
        s.step(order, 3)
    assert s.step(order, 1)[1] >= 160  # alone: whole pages in front of its row


def test_a_server_whose_moves_take_several_calls():
    s = Server("bf16", 4, pages=60, seed=1)
    s.grow([0, 1, 2, 3], [100, 33, 64, 200])
    s.fork(3, [1], [180])
    s.kept[0] = []
    for _ in range(8):
        live = s.free_list([1, 2, 3], compact=2)
        s.step([3, 1, 2, 0], 2)
    live = s.free_list([1, 2, 3], compact=2)
    assert live == set(range(len(live)))


# ------------------------------------------------------------------ graphs

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


class Step:
    """A step of up to eight requests in two groups in memory of its own, over one cache."""

    def __init__(self, dec, cache, scale, max_own, groups=2, seed=0):
        self.dec, self.cache, self.scale = dec, cache, scale
        self.sh = B.Shared(dec.plan, groups, max_own)
        self.g = torch.Generator().manual_seed(seed)
        self.table = ints([0] * 1000)
        self.kv_indptr, self.qo = ints([0] * 9), ints([0] * 9)
        self.kv_len, self.window, self.own, self.own_ptr = (ints([0] * 8) for _ in range(4))
        self.bounds, self.prefix = ints([0] * (groups + 1)), ints([[0, 0]] * groups)
        hq, d = dec.plan.num_qo_heads, dec.plan.head_dim
        self.q = torch.zeros(20, hq, d, dtype=torch.bfloat16, device=DEV)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(20, hq, device=DEV)

    def fill(self, prefixes, bounds, own, rows, windows=(0,) * 8):
        """prefixes: shared pages of each group; own tokens and rows of each request (padded)."""
        r = torch.randperm(self.cache[0].shape[0], generator=self.g).tolist()
        table, ptr, lens = [], [0], []
        for i, n in enumerate(prefixes):
            pre = [r.pop() for _ in range(n)]
            for b in range(bounds[i], bounds[i + 1]):
                table += pre + [r.pop() for _ in range(ref.ceil(own[b], 16))] if rows[b] else []
                lens.append(16 * n + own[b] if rows[b] else 0)
                ptr.append(len(table))
        self.table[:len(table)] = ints(table)
        for t, v in ((self.kv_indptr, ptr), (self.kv_len, lens), (self.window, list(windows)),
                     (self.bounds, bounds), (self.qo, [sum(rows[:k]) for k in range(9)])):
            t.copy_(ints(v))
        self.q.copy_(torch.randn(self.q.shape, generator=self.g).to(torch.bfloat16))

    def call(self):
        a = (self.table, self.kv_indptr, self.kv_len, self.qo, self.window, self.bounds, self.prefix, self.own_ptr,
             self.own)
        B.pda_share_tables(self.sh.plan, *a, self.sh.scratch)
        B.pda_decode_shared(self.sh.plan, self.q, *self.cache, *a[:4], 3, *a[4:], 0.09, *self.scale, self.out,
                            self.lse, self.sh.scratch)

    def outs(self):
        return [self.out, self.lse, self.prefix, self.own, self.own_ptr]


def cache_of(kind, dim, hkv=2, pages=400):
    g = torch.Generator().manual_seed(9)
    x = [torch.randn(pages, 16, hkv, dim, generator=g) for _ in "kv"]
    if kind == "bf16":
        return [t.to(torch.bfloat16).to(DEV) for t in x], [None, None]
    return ([(t * 20).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV) for t in x],
            [torch.rand(pages, 16, hkv, generator=g).add(0.1).to(DEV) for _ in "kv"])


FILLS = [([40, 3], [0, 5, 8], [30, 7, 90, 3, 16, 50, 3, 20], [1, 3, 2, 1, 1, 3, 1, 1]),
         ([0, 60], [0, 2, 8], [99, 1, 5, 5, 5, 5, 80, 16], [1, 1, 1, 3, 3, 2, 1, 2]),
         ([7, 7], [0, 4, 8], [3, 17, 64, 80, 0, 0, 0, 0], [3, 3, 1, 2, 0, 0, 0, 0]),   # half the batch empty
         ([0, 0], [0, 0, 8], [0] * 8, [0] * 8),                                          # all of it
         ([100, 0], [0, 8, 8], [9, 8, 7, 6, 5, 4, 3, 1], [1] * 8, [0, 5, 0, 300, 0, 17, 0, 1])]


@pytest.mark.parametrize("max_own", [100, 0])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("e4m3_token", 256)])
def test_steps_in_a_graph(kind, dim, max_own):
    """Replays with other lengths, groups, windows and padded requests in the same memory."""
    cache, scale = cache_of(kind, dim)
    p = ref.plan_params(kind, heads=2, dim=dim, pages=400, batch=8, max_kv=4000, max_q=3, hq=8)
    dec = B.Decoder(p, device=DEV)
    step = Step(dec, cache, scale, max_own)
    step.fill(*FILLS[0])
    graph = capture(step.call)
    for fill in FILLS + FILLS[:1]:
        step.fill(*fill)
        got = same(step.call, graph, step.outs(), (), f"{fill}")
        rows = sum(fill[3])
        assert bool((got[0].reshape(20, -1)[rows:] == 0x11).all())
        assert bool((got[1].reshape(20, -1)[rows:] == 0x11).all())
        assert rows == 0 or bool(torch.isfinite(step.out[:rows].float()).all())
    assert step.sh.status() == 0


def test_two_graphs_share_a_scratch_in_turn():
    cache, scale = cache_of("bf16", 128)
    dec = B.Decoder(ref.plan_params("bf16", heads=2, pages=400, batch=8, max_kv=4000, max_q=3, hq=8), device=DEV)
    steps = [Step(dec, cache, scale, 100, seed=k) for k in range(2)]
    steps[1].sh = steps[0].sh
    want, graphs = [], []
    for s, fill in zip(steps, FILLS):
        s.fill(*fill)
        s.call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.outs()])
        graphs.append(capture(s.call))
    for k in (0, 1, 1, 0, 0, 1):
        for t in steps[k].outs():
            t.zero_()
        graphs[k].replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        rows = int(s.qo[-1])
        assert all(torch.equal(a[:rows], b[:rows]) for a, b in zip(s.outs()[:2], w))
        assert all(torch.equal(a, b) for a, b in zip(s.outs()[2:], w[2:]))


def test_two_steps_at_once():
    """Each with its scratch, on streams of their own, while the current stream is busy."""
    cache, scale = cache_of("e4m3_token", 128)
    dec = B.Decoder(ref.plan_params("e4m3_token", heads=2, pages=400, batch=8, max_kv=4000, max_q=3, hq=8),
                    device=DEV)
    steps = [Step(dec, cache, scale, 100, seed=k) for k in range(2)]
    want = []
    for s, fill in zip(steps, FILLS):
        s.fill(*fill)
        s.call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.outs()])
        for t in s.outs():
            t.zero_()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        busy = busy @ busy * 1e-3
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.call()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        rows = int(s.qo[-1])
        assert all(torch.equal(a[:rows], b[:rows]) for a, b in zip(s.outs()[:2], w))
        assert all(torch.equal(a, b) for a, b in zip(s.outs()[2:], w[2:])) and s.sh.status() == 0


@pytest.mark.parametrize("pages", [300, 140000])  # one kernel; marks in memory
def test_page_calls_in_a_graph(pages):
    """Fork with its copy, free and compact, replayed with other requests and lengths."""
    cols, n, most = 40, 6, 30
    r = random.Random(pages)
    dec = B.Decoder(ref.plan_params("e4m3_token", heads=1, dim=64, pages=pages, batch=n), device=DEV)
    held = B.Pages(dec.plan)
    cache = [torch.zeros(pages, 16, 1, 64, dtype=torch.uint8, device=DEV) for _ in "kv"]
    scale = [torch.zeros(pages, 16, 1, device=DEV) for _ in "kv"]
    block, new = (torch.zeros(n, cols, dtype=torch.int32, device=DEV) for _ in range(2))
    pool, count, left = ints([0] * pages), ints([0]), ints([0])
    parent, child, shared, lens = (ints([0] * k) for k in (2, 2, 2, n))
    forked = [ints([0] * 2) for _ in range(4)]
    out, gone, src, dst, num = ints([0] * pages), ints([0]), ints([0] * most), ints([0] * most), ints([0])

    def call():
        B.pda_fork_tables(dec.plan, parent, child, shared, block, pool, count, left, *forked, dec.scratch)
        B.pda_copy_pages(dec.plan, *cache, *scale, *forked[1:], None, dec.scratch)
        B.pda_free_pages(dec.plan, lens, None, block, out, gone, held.scratch)
        B.pda_compact_pages(dec.plan, lens, None, block, new, out, gone, src, dst, num, held.scratch)
        B.pda_copy_pages(dec.plan, *cache, *scale, src, dst, None, num, dec.scratch)

    graph = None
    for k in range(5):
        ids = r.sample(range(pages), n * cols + 8)
        first = ints(ids[:n * cols]).reshape(n, cols)
        free = ids[n * cols:]
        have = [r.randint(0, 16 * cols) for _ in range(n)] if k else [16 * cols] * n
        if k == 3:
            have = [0] * n
        kids = r.sample(range(1, n), 2)
        data = [torch.randint(0, 127, cache[0].shape, dtype=torch.uint8, device=DEV) for _ in "kv"]

        def reset():
            block.copy_(first)
            for t, v in ((parent, [0, 0]), (child, kids), (shared, [have[0], have[0] // 2]), (lens, have),
                         (count, [8])):
                t.copy_(ints(v))
            pool[:8] = ints(free)
            for c, d in zip(cache, data):
                c.copy_(d)
            for s in scale:
                s.fill_(0.5)

        reset()
        if graph is None:
            graph = capture(call)
        outs = [block, new, left, *forked, out, gone, src, dst, num, *cache, *scale]
        same(call, graph, outs, (reset,), f"round {k}")
    assert dec.status() == 0 and held.status() == 0


# ------------------------------------------------------------ what else may come

@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("int8_token", 256), ("e4m3_tensor", 64)])
def test_many_own_tokens(kind, dim):
    """More than the one kernel of few own tokens takes, beside requests with one."""
    parity(S.make([(9, [(1500, 1), (1, 1), (1025, 2), (700, 1)]), (30, reqs(3))], kind=kind, dim=dim, dev=DEV))


@pytest.mark.parametrize("own", [15, 16, 17, 64, 65, 1023, 1024])
def test_own_lengths(own):
    """About a warp's 16 tokens, its CTA's 64, and the most that one kernel takes."""
    for rows, kind, dim in ((1, "bf16", 128), (3, "e4m3_tensor", 128), (2, "bf16", 256)):
        parity(S.make([(5, [(own, rows), (max(1, own - 1), 1), (own, 1)])], kind=kind, dim=dim, dev=DEV, seed=own))


@pytest.mark.parametrize("same_for", [0, 1, 255, 256, 257, 511, 3000])
def test_long_tables(same_for):
    """Lists that part at the ends of a warp's stretch, in one request of many."""
    cols, n = 3000, 9
    g = torch.Generator().manual_seed(same_for)
    lists = [torch.randperm(4000, generator=g)[:cols].tolist()] * n
    odd = list(lists[0])
    if same_for < cols:
        odd[same_for] = 4000 + 5
    lists[6] = odd
    p = ref.plan_params("bf16", heads=1, dim=64, pages=5000, batch=n, max_kv=16 * cols, max_q=4)
    dec = B.Decoder(p, device=DEV)
    sh = B.Shared(dec.plan, 1, 0)
    lens = [16 * cols - b for b in range(n)]
    rows = [1, 4, 0, 2, 1, 1, 1, 3, 1]
    t = types.SimpleNamespace(
        page_table=ints(sum(lists, [])), kv_indptr=ints([cols * k for k in range(n + 1)]), kv_len=ints(lens),
        qo_indptr=ints([sum(rows[:k]) for k in range(n + 1)]), window=None, group_indptr=None,
        prefix=ints([[-9, -9]]), own_indptr=ints([-9] * n), own_len=ints([-9] * n))
    B.pda_share_tables(sh.plan, *S.args(t), sh.scratch)
    (prefix, ptr, own), status = ref.share(
        sum(lists, []), [cols * k for k in range(n + 1)], lens, [sum(rows[:k]) for k in range(n + 1)], None,
        [0, n], page=16, max_q=4, max_kv=16 * cols, num_pages=5000)
    assert t.prefix.reshape(-1).tolist() == prefix and prefix[1] == 16 * min(same_for, cols - 1)
    assert t.own_indptr.tolist() == ptr and t.own_len.tolist() == own and sh.status() == status == 0


def test_another_device_is_refused():
    """A plan of a device that is not the current one."""
    p = ref.plan_params("bf16", pages=8, batch=2, num_sms=152, device=1)
    plan, _, _ = B.pda_plan(p)
    sp, _, _ = B.pda_shared_plan(plan, 1)
    x = [torch.zeros(4096, dtype=torch.int32, device=DEV) for _ in range(12)]
    at = [t.data_ptr() for t in x]
    import ctypes
    lib = B.load_library()
    t = B.PdaSharedTables(at[0], at[1], at[2], at[3], None, None, at[4], at[5], at[6])
    assert lib.pda_share_tables(ctypes.byref(sp), ctypes.byref(t), at[7], None) == B.PDA_ERR_INVALID
    assert lib.pda_decode_shared(ctypes.byref(sp), at[8], at[9], at[9], ctypes.byref(t), 1, 1.0, None, None, at[10],
                                 None, at[7], None) == B.PDA_ERR_INVALID
    f = B.PdaForks(at[0], at[1], at[2], at[3], 8, at[4], at[5], at[6], at[7], at[8], at[9], at[10], 4, 8, 2)
    assert lib.pda_fork_tables(ctypes.byref(plan), ctypes.byref(f), at[11], None) == B.PDA_ERR_INVALID
    assert lib.pda_copy_pages(ctypes.byref(plan), at[0], at[1], None, None, at[2], at[3], None, 2, None, at[4],
                              None) == B.PDA_ERR_INVALID
