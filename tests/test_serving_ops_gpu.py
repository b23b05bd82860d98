"""GPU parity of the calls around decode against plain implementations in 64
bits: block tables and slot maps (equal), append by slot map (every byte),
the absorbed and the expanded form of latent attention (within the rounding
of their types, element by element), and a serving loop of them together."""
from __future__ import annotations

import math
import random

import pytest
import torch

import serving_ref as ref
from paged_split_kv_03_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def check(got, want, bound, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    fine = torch.isfinite(want)
    err, lim = (got - want).abs()[fine], bound.expand_as(want)[fine]
    if not err.numel():
        return
    worst = (err - lim).argmax()
    assert bool((err <= lim).all()), \
        f"{what}: error {err[worst]:.3e}, bound {lim[worst]:.3e}, value {want[fine][worst]:.3e}"


# ------------------------------------------------------------- block tables

class Tables:
    """Device arrays of one pda_build_tables call."""

    def __init__(self, cached, new, *, page=16, free=None, request=None, extra_rows=0, cols=None,
                 page_cap=None, rows_cap=None, max_kv=1 << 20, seed=0, pages=None, null=()):
        r = random.Random(seed)
        n = len(cached)
        have = [-(-max(c, 0) // page) for c in cached]
        want = [-(-max(c + m, 0) // page) for c, m in zip(cached, new)]
        self.cols = cols if cols is not None else max(want) + 2
        need = sum(max(0, w - h) for w, h in zip(want, have))
        self.free = need + 3 if free is None else free
        self.pages = pages or sum(have) + max(self.free, need) + 4
        ids = list(range(self.pages))
        r.shuffle(ids)
        table_rows = n + extra_rows
        self.request = request
        self.block = [[-7] * self.cols for _ in range(table_rows)]
        for b in range(n):
            row = request[b] if request else b
            if 0 <= row < table_rows:
                for j in range(min(have[b], self.cols)):
                    self.block[row][j] = ids.pop()
        self.free_pages = ids[:max(self.free, 1)]
        self.cached, self.new, self.page, self.max_kv = cached, new, page, max_kv
        self.page_cap = sum(want) + 5 if page_cap is None else page_cap
        self.rows_cap = sum(max(0, m) for m in new) + 5 if rows_cap is None else rows_cap
        p = B.PdaParams(num_qo_heads=1, num_kv_heads=1, head_dim=128, page_size=page, max_batch=n,
                        max_q_len=1, max_kv_len=max_kv, num_pages=self.pages,
                        kv_stride_page=page * 128, kv_stride_token=128, kv_stride_head=128)
        self.dec = B.Decoder(p, device=DEV)
        self.dev = dict(kv_len=ints([-9] * n), kv_indptr=ints([-9] * (n + 1)),
                        page_table=ints([-9] * self.page_cap), qo_indptr=ints([-9] * (n + 1)),
                        tok_indptr=ints([-9] * (n + 1)),
                        slot_map=ints([-9] * self.rows_cap, torch.int64),
                        positions=ints([-9] * self.rows_cap), free_left=ints([-9]),
                        block_table=ints(self.block).reshape(table_rows, self.cols))
        for k in null:
            self.dev[k] = None
        self.inputs = dict(cached_len=ints(cached), new_len=ints(new),
                           request=None if request is None else ints(request),
                           free_pages=ints(self.free_pages), free_count=ints([self.free]))

    def run(self, **kw):
        i, o = self.inputs, self.dev
        return B.pda_build_tables(self.dec.plan, i["cached_len"], i["new_len"], i["request"],
                                  o["block_table"], i["free_pages"], i["free_count"],
                                  o["free_left"], o["kv_len"], o["kv_indptr"], o["page_table"],
                                  o["qo_indptr"], o["tok_indptr"], o["slot_map"], o["positions"],
                                  self.dec.scratch, **kw)

    def compare(self):
        want, status = ref.build_tables(
            self.inputs["cached_len"].tolist(), self.inputs["new_len"].tolist(), self.request,
            self.block, self.free_pages, self.free, self.page, max_kv=self.max_kv,
            page_cap=self.page_cap, rows_cap=self.rows_cap, num_pages=self.pages)
        torch.cuda.synchronize()
        assert self.dec.status() == status
        for name, t in self.dev.items():
            if t is None:
                continue
            got, w = t.cpu().reshape(-1).tolist(), want[name]
            if name == "block_table":
                w = [x for r in w for x in r]
            w = w + [-9] * (len(got) - len(w))  # entries behind the last request stay
            assert got == w, name
        return want, status


TABLES = {
    "one_token": dict(cached=[0], new=[1]),
    "nothing": dict(cached=[0], new=[0], free=0),
    "page_boundaries": dict(cached=[15, 16, 17, 0, 31], new=[1, 1, 1, 16, 2]),
    "page_of_one": dict(cached=[5, 0, 9], new=[3, 4, 0], page=1),
    "big_page": dict(cached=[255, 256, 700], new=[300, 1, 8], page=256),
    "permuted_rows": dict(cached=[40, 3, 0, 65], new=[2, 8, 33, 1], request=[4, 0, 2, 5],
                          extra_rows=2),
    "nine_requests": dict(cached=[7] * 9, new=[20] * 9),
    "prefill_2000": dict(cached=[0, 1000], new=[2000, 1]),
    "free_runs_out": dict(cached=[16, 16, 10, 0, 5], new=[1, 17, 2, 40, 3], free=3),
    "free_exact": dict(cached=[16, 16], new=[1, 17], free=3),
    "free_empty": dict(cached=[16, 4, 0], new=[1, 1, 1], free=0),
    "negative": dict(cached=[4, -1, 6, 3], new=[1, 1, -2, 1]),
    "row_out_of_range": dict(cached=[4, 5, 6], new=[1, 1, 30], request=[0, 9, -1], extra_rows=1),
    "too_many_columns": dict(cached=[30, 30, 30], new=[1, 40, 1], cols=3),
    "above_max_kv": dict(cached=[30, 90, 30], new=[1, 40, 1], max_kv=100),
    "page_cap": dict(cached=[30, 90, 30, 1], new=[1, 40, 1, 1], page_cap=10),
    "rows_cap": dict(cached=[30, 90, 30, 0], new=[5, 40, 1, 0], rows_cap=20),
    "both_caps_and_free": dict(cached=[30, 90, 30, 9], new=[5, 40, 20, 9], rows_cap=30, free=2),
    "int32_lengths": dict(cached=[2 ** 31 - 1, 5], new=[2 ** 31 - 1, 1], cols=8, page_cap=20,
                          rows_cap=20, free=10, pages=40, max_kv=2 ** 31 - 1),
    "no_optional_outputs": dict(cached=[16, 4], new=[1, 9], null=("tok_indptr", "slot_map",
                                                                    "positions")),
}


@pytest.mark.parametrize("name", sorted(TABLES))
def test_tables(name):
    kw = dict(TABLES[name])
    if name == "int32_lengths":
        t = Tables([5, 5], [1, 1], **{k: v for k, v in kw.items() if k not in ("cached", "new")})
        t.inputs["cached_len"].copy_(ints(kw["cached"]))
        t.inputs["new_len"].copy_(ints(kw["new"]))
    else:
        t = Tables(**kw)
    t.run()
    t.compare()
    t.dec.reset_status()
    t.run()  # the same inputs again: the same outputs
    t.compare()


@pytest.mark.parametrize("batch,page,seed", [(255, 16, 1), (256, 64, 2), (257, 16, 3), (700, 32, 4),
                                             (5000, 64, 5)])
def test_tables_large_batches(batch, page, seed):
    r = random.Random(seed)
    cached = [r.choice([0, 1, page - 1, page, r.randint(0, 2000)]) for _ in range(batch)]
    new = [r.choice([0, 1, 1, 1, 8, r.randint(1, 300)]) for _ in range(batch)]
    req = list(range(batch + 3))
    r.shuffle(req)
    need = sum(-(-(c + n) // page) + -c // page for c, n in zip(cached, new))
    for k, free in enumerate((None, need // 2)):
        t = Tables(cached, new, page=page, request=req[:batch], extra_rows=3, free=free,
                   seed=seed + k)
        t.run()
        t.compare()
    t = Tables(cached, new, page=page, request=req[:batch], extra_rows=3, seed=seed,
               page_cap=batch * 8, rows_cap=sum(new) // 2)
    t.run()
    t.compare()


def test_tables_bad_pages_and_graph():
    t = Tables([20, 40], [30, 1])
    t.block[1][2] = t.pages + 3         # holds tokens 32..47: the new row's slot
    t.dev["block_table"][1, 2] = t.pages + 3
    t.run()
    _, status = t.compare()
    assert status == B.PDA_STATUS_PAGE_OOB
    # captured once, replayed with other lengths and another stream's capture
    t = Tables([20, 40, 7], [30, 1, 0], page_cap=60, rows_cap=80, free=20, cols=12)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    t.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        t.run()
    for cached, new in (([20, 40, 7], [30, 1, 0]), ([33, 1, 16], [1, 50, 9]), ([0, 0, 0], [0, 0, 0])):
        t2 = Tables(cached, new, page_cap=60, rows_cap=80, free=20, cols=12, seed=9, pages=t.pages)
        for k in t.dev:
            t.dev[k].copy_(t2.dev[k])
        for k in ("cached_len", "new_len", "free_count"):
            t.inputs[k].copy_(t2.inputs[k])
        t.inputs["free_pages"].fill_(0)
        n = min(len(t.free_pages), len(t2.free_pages))
        t.inputs["free_pages"][:n] = t2.inputs["free_pages"][:n]
        t.block, t.free_pages = t2.block, t.inputs["free_pages"].tolist()
        g.replay()
        t.compare()


# ------------------------------------------------------ append by slot map

APPEND = [(kind, d, h) for kind in ("bf16", "e4m3_tensor", "e4m3_token", "int8_tensor", "int8_token")
          for d, h in ((64, 3), (128, 8), (256, 1), (512, 2)) if d < 512 or "int8" not in kind] + \
    [(k, 576, 1) for k in ("bf16", "e4m3_tensor", "e4m3_token", "records")]


def cache_plan(kind, d, h, page, pages, hnd=False):
    w = 640 if kind == "records" else d
    st = (page * h * w, w, page * w) if hnd else (page * h * w, h * w, w)
    p = B.PdaParams(num_qo_heads=h, num_kv_heads=h, head_dim=d, page_size=page, max_batch=1,
                    max_q_len=1, max_kv_len=page * pages, num_pages=pages, kv_stride_page=st[0],
                    kv_stride_token=st[1], kv_stride_head=st[2])
    if d == 576:
        p.head_dim_v = 512
    if kind != "bf16":
        p.kv_dtype = B.PDA_INT8 if "int8" in kind else B.PDA_E4M3
        p.scale_mode = B.PDA_SCALE_MLA_BLOCK if kind == "records" else \
            B.PDA_SCALE_TOKEN_HEAD if "token" in kind else B.PDA_SCALE_TENSOR
        if d == 576 and kind != "records":
            p.q_dtype = B.PDA_E4M3
    return p


def stored(x, kind, scale):
    """(bytes, scales) of rows x [n, H, D] (bf16) as the cache keeps them."""
    if kind == "bf16":
        return x.contiguous().view(torch.uint8), None
    if kind == "records":
        return ref.records(x)
    s = scale
    if "token" in kind:
        amax = x.float().abs().amax(-1)
        s = torch.where(amax > 0, amax / torch.full_like(amax, 127.0 if "int8" in kind else 448.0),
                        torch.ones_like(amax))
    y = x.float() / (s[..., None] if s.ndim else s)
    if "int8" in kind:
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8), s
    return y.clamp(-448, 448).to(ref.E4M3).view(torch.uint8), s


@pytest.mark.parametrize("hnd", [False, True])
@pytest.mark.parametrize("kind,d,h", APPEND)
def test_append_slots(kind, d, h, hnd):
    page, pages, rows = 16, 9, 61
    dec = B.Decoder(cache_plan(kind, d, h, page, pages, hnd), device=DEV)
    g = torch.Generator().manual_seed(d + h)
    stride = h * d + 24  # rows of a wider tensor
    wide = randn(g, 2, rows, stride, std=2.0)
    wide[:, 0, :d] = 0
    wide[:, 1, 0] = 500.0
    slots = torch.randperm(page * pages, generator=g)[:rows]
    slots[3] = -1
    slots[7] = page * pages          # out of range: skipped, reported
    slots[8] = -2
    live = [i for i in range(rows - 2) if i not in (3, 7, 8)]  # num_rows leaves the last two out
    two = d != 576
    new = [wide[k].to(DEV).as_strided((rows, h, d), (stride, d, 1)) for k in range(2)]
    eb = 2 if kind == "bf16" else 1
    w = 640 if kind == "records" else d * eb
    shape = (pages, h, page, w) if hnd else (pages, page, h, w)
    cache = [torch.full(shape, 0x5A, dtype=torch.uint8, device=DEV) for _ in range(2)]
    sshape = (pages, page, h, 4) if kind == "records" else (pages, page, h)
    per_row = kind == "records" or "token" in kind
    scales = [None, None] if kind == "bf16" else \
        [torch.full(sshape, -1.0, device=DEV) if per_row else torch.tensor([0.03 + k], device=DEV)
         for k in range(2)]
    B.pda_append_slots(dec.plan, new[0], new[1] if two else None, slots.to(DEV), ints([rows - 2]),
                       cache[0], cache[1] if two else None, scales[0], scales[1] if two else None,
                       dec.scratch)
    torch.cuda.synchronize()
    assert dec.status() == B.PDA_STATUS_PAGE_OOB
    for k in range(2 if two else 1):
        x = new[k].cpu()[live]
        got = cache[k].cpu()
        got = (got.transpose(1, 2) if hnd else got).reshape(page * pages, h, w)
        want = torch.full((page * pages, h, w), 0x5A, dtype=torch.uint8)
        data, s = stored(x, kind, None if per_row or scales[k] is None else scales[k].cpu()[0])
        want[slots[live]] = data
        assert torch.equal(got, want), f"side {k}"
        if per_row:
            ws = torch.full((page * pages, *sshape[2:]), -1.0)
            ws[slots[live]] = s
            assert torch.equal(scales[k].cpu().reshape(ws.shape), ws), f"scales {k}"


@pytest.mark.parametrize("rows", [0, 1, 7, 8, 9, 3001])
def test_append_slots_rows(rows):
    """Every count of rows, no bound on the device."""
    dec = B.Decoder(cache_plan("e4m3_token", 128, 2, 64, 64), device=DEV)
    g = torch.Generator().manual_seed(rows)
    k, v = randn(g, rows, 2, 128), randn(g, rows, 2, 128)
    slots = torch.randperm(64 * 64, generator=g)[:rows]
    cache = [torch.zeros(64, 64, 2, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
    sc = [torch.zeros(64, 64, 2, device=DEV) for _ in range(2)]
    B.pda_append_slots(dec.plan, k.to(DEV), v.to(DEV), slots.to(DEV), None, *cache, *sc, dec.scratch)
    assert dec.status() == 0
    for x, c, s in zip((k, v), cache, sc):
        data, ws = stored(x, "e4m3_token", None)
        want, wsc = torch.zeros(4096, 2, 128, dtype=torch.uint8), torch.zeros(4096, 2)
        want[slots], wsc[slots] = data, ws
        assert torch.equal(c.cpu().reshape(4096, 2, 128), want)
        assert torch.equal(s.cpu().reshape(4096, 2), wsc)


@pytest.mark.parametrize("kind", ["e4m3_tensor", "int8_tensor", "e4m3_token", "int8_token"])
def test_append_slots_ties(kind):
    """Quotients at and next to the ties between codes, subnormal codes, zeros of both signs,
    saturation, infinities and NaN, over scales of every size: each code is that of the fp32
    quotient."""
    dec = B.Decoder(cache_plan(kind, 128, 1, 64, 64), device=DEV)
    g = torch.Generator().manual_seed(1)
    rows, n = 64, 64 * 128
    scales = [1.0, 3.0, 0.1, 2.0 ** -20, 7e-39, 1e30, 2.0 ** 126] if "tensor" in kind else [1.0]
    for s in scales:
        # codes' midpoints times the scale, in bf16: some quotients hit the tie exactly
        if "int8" in kind:
            y = torch.randint(-130, 131, (n,), generator=g).float() + 0.5
        else:
            v = torch.arange(256, dtype=torch.uint8).view(ref.E4M3).float()
            v = v[torch.isfinite(v)].unique()
            mid = (v[1:] + v[:-1]) / 2
            y = mid[torch.randint(0, mid.numel(), (n,), generator=g)]
        x = (y.double() * s).float().to(torch.bfloat16)
        x[::7] = torch.randn(x[::7].shape, generator=g).to(torch.bfloat16) * s
        if "tensor" in kind:
            x[5], x[6], x[7], x[8] = math.inf, -math.inf, 0.0, -0.0
            if "int8" not in kind:
                x[9] = math.nan
        x = x.reshape(rows, 1, 128)
        slots = torch.randperm(64 * 64, generator=g)[:rows]
        cache = [torch.zeros(64, 64, 1, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]
        sc = [torch.full((64, 64, 1), -1.0, device=DEV) if "token" in kind else
              torch.tensor([s], device=DEV) for _ in range(2)]
        B.pda_append_slots(dec.plan, x.to(DEV), x.to(DEV), slots.to(DEV), None, *cache, *sc, dec.scratch)
        assert dec.status() == 0
        want = torch.zeros(4096, 1, 128, dtype=torch.uint8)
        want[slots] = stored(x, kind, None if "token" in kind else torch.tensor(s))[0]
        for c in cache:
            got = c.cpu().reshape(4096, 1, 128)
            both_nan = (got & 0x7F == 0x7F) & (want & 0x7F == 0x7F) if "e4m3" in kind else False
            assert bool(((got == want) | both_nan).all()), (kind, s)


# ------------------------------------------------------------ absorbed form

def weights(g, heads, split=False):
    """(w_uk, w_uv) on the device: views of one [H, 256, 512], or two tensors."""
    w = randn(g, heads, 256, 512, std=512 ** -0.5).to(DEV)
    return (w[:, :128].contiguous(), w[:, 128:].contiguous()) if split else (w[:, :128], w[:, 128:])


ROWS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 257, 513]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,heads", [(r, 3) for r in ROWS] + [(1, 1), (1, 128), (65, 16), (300, 20)])
def test_absorb(rows, heads, kind):
    g = torch.Generator().manual_seed(rows * 7 + heads)
    dec = B.Decoder(ref.mla_plan(heads, kind=kind), device=DEV)
    q = torch.full((rows + 2, heads, 200), math.nan, dtype=torch.bfloat16)
    q[:rows, :, :192] = randn(g, rows, heads, 192)
    w_uk, _ = weights(g, heads, split=rows % 2 == 0)
    n = rows + 2                         # two rows behind the last: left as they were
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    out = torch.full((n, heads, 576), 77, dtype=dt, device=DEV)
    scale = 0.011
    B.pda_mla_absorb(dec.plan, q.to(DEV)[..., :192], w_uk, scale, out, ints([rows]), dec.scratch)
    assert dec.status() == 0
    assert bool((out[rows:] == 77).all())
    x, mag = ref.product(q[:rows, :, :128], w_uk.cpu().transpose(1, 2))
    x = torch.cat([x, q[:rows, :, 128:192].double()], -1)
    mag = torch.cat([mag * ref.sum_bound(128), torch.zeros(rows, heads, 64, dtype=torch.float64)], -1)
    if kind == "bf16":
        check(out[:rows], x, mag + ref.BF16_HALF * (x.abs() + mag), "q_lat")
        assert torch.equal(out[:rows, :, 512:].cpu(), q[:rows, :, 128:192])
    else:
        y = (x / scale).clamp(-448, 448)
        mag = mag / scale + 2.0 ** -23 * y.abs()
        check(out[:rows].view(ref.E4M3), y,
              mag + torch.clamp(ref.E4M3_HALF * (y.abs() + mag), min=ref.E4M3_SUB), "q_lat codes")


@pytest.mark.parametrize("rows,heads", [(r, 3) for r in ROWS] + [(1, 1), (1, 128), (65, 16), (300, 20)])
def test_project(rows, heads):
    g = torch.Generator().manual_seed(rows * 5 + heads)
    dec = B.Decoder(ref.mla_plan(heads), device=DEV)
    o = torch.full((rows + 2, heads, 512), math.nan, dtype=torch.bfloat16)
    o[:rows] = randn(g, rows, heads, 512)
    _, w_uv = weights(g, heads, split=rows % 2 == 0)
    out = torch.full((rows + 2, heads, 128), 77.0, dtype=torch.bfloat16, device=DEV)
    B.pda_mla_project(dec.plan, o.to(DEV), w_uv, out, ints([rows]), dec.scratch)
    assert dec.status() == 0
    assert bool((out[rows:] == 77).all())
    x, mag = ref.product(o[:rows], w_uv.cpu())
    mag = mag * ref.sum_bound(512)
    check(out[:rows], x, mag + ref.BF16_HALF * (x.abs() + mag), "out")


def test_absorb_project_bounds_of_rows():
    """num_rows above the rows, zero and negative; rows 0; another stream."""
    g = torch.Generator().manual_seed(3)
    dec = B.Decoder(ref.mla_plan(4), device=DEV)
    q, w = randn(g, 9, 4, 192).to(DEV), randn(g, 4, 256, 512, std=0.05).to(DEV)
    full = torch.zeros(9, 4, 576, dtype=torch.bfloat16, device=DEV)
    B.pda_mla_absorb(dec.plan, q, w[:, :128], 1.0, full, None, dec.scratch)
    for n in (100, 0, -3):
        out = torch.full_like(full, 5.0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        B.pda_mla_absorb(dec.plan, q, w[:, :128], 1.0, out, ints([n]), dec.scratch, stream=s)
        s.synchronize()
        assert torch.equal(out, full) if n == 100 else bool((out == 5).all())
    assert B.pda_mla_absorb(dec.plan, q[:0], w[:, :128], 1.0, full[:0], None, dec.scratch) == 0
    assert dec.status() == 0


# ------------------------------------------------------------ expanded form

def latent_cache(g, kind, pages, page):
    """(pages, k_scale, the values [pages, P, 576] in 64 bits)."""
    x = randn(g, pages, page, 1, 576)
    if kind == "bf16":
        return x, None, x[:, :, 0].double()
    if kind == "records":
        x[0, 0, 0, 128:256] = 0  # a zero block: scale 0
        rec, s = ref.records(x)
        return rec, s, ref.record_values(rec, s)[:, :, 0]
    s = torch.tensor([0.0123]) if kind == "e4m3" else \
        torch.rand(pages, page, 1, generator=g) * 0.02 + 0.001
    c = ref.codes(x, s if kind == "e4m3" else s[..., None])
    return c.view(torch.uint8), s, (c.double() * (s if kind == "e4m3" else s[..., None]).double())[:, :, 0]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e4m3_token", "records"])
@pytest.mark.parametrize("lens,heads,page", [
    ([1], 1, 64), ([0, 5, 0, 0, 130, 1, 0], 3, 16), ([127], 2, 64), ([128, 128], 2, 32),
    ([129, 300], 16, 64), ([700, 1, 33], 20, 8), ([256], 128, 64)])
def test_expand(lens, heads, page, kind):
    g = torch.Generator().manual_seed(sum(lens) + heads)
    npg = [-(-n // page) for n in lens]
    pages = sum(npg) + 2
    total = sum(lens)
    dec = B.Decoder(ref.mla_plan(heads, kind=kind, page=page, pages=pages, batch=len(lens)), device=DEV)
    cache, scale, values = latent_cache(g, kind, pages, page)
    table = torch.randperm(pages, generator=g)[:sum(npg)].int()
    tok, ptr = [0], [0]
    for n, m in zip(lens, npg):
        tok.append(tok[-1] + n)
        ptr.append(ptr[-1] + m)
    cap = total + 3
    latent = torch.full((cap, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    # k and v either interleaved per head or apart
    if heads % 2:
        kv = torch.full((cap, heads, 256), 7.0, dtype=torch.bfloat16, device=DEV)
        k, v = kv[..., :128], kv[..., 128:]
    else:
        k, v = (torch.full((cap, heads, 136), 7.0, dtype=torch.bfloat16, device=DEV)[..., :128]
                for _ in range(2))
    w_uk, w_uv = weights(g, heads, split=heads == 2)
    B.pda_mla_expand(dec.plan, cache.to(DEV), table.to(DEV), ints(ptr), ints(tok),
                     None if scale is None else scale.to(DEV), w_uk, w_uv, latent, k, v, dec.scratch)
    assert dec.status() == 0
    rows = [int(table[ptr[b] + i // page]) * page + i % page
            for b, n in enumerate(lens) for i in range(n)]
    x = values.reshape(-1, 576)[rows]
    check(latent[:total], x, ref.BF16_HALF * 1.001 * x.abs() + 1e-38, "latent")
    lat = latent[:total, None, :512].expand(total, heads, 512).cpu()
    for name, got, w in (("k", k, w_uk), ("v", v, w_uv)):
        y, mag = ref.product(lat, w.cpu())
        mag = mag * ref.sum_bound(512)
        check(got[:total], y, mag + ref.BF16_HALF * (y.abs() + mag), name)
        assert bool((got[total:] == 7).all()), f"{name}: rows behind the last"
    assert bool((latent[total:] == 7).all())


def test_expand_status():
    """A bad page reads as zeros, a request above max_kv_len too; tokens
    smaller than tok_indptr's end writes the first rows alone."""
    g = torch.Generator().manual_seed(5)
    dec = B.Decoder(ref.mla_plan(2, page=16, pages=8, batch=2, max_kv=40), device=DEV)
    cache, _, values = latent_cache(g, "bf16", 8, 16)
    table = [3, 99, 5, 1, 2]
    out = [torch.full((90, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    latent = torch.full((90, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    w_uk, w_uv = weights(g, 2)

    def go(ptr, tok, cap):
        B.pda_mla_expand(dec.plan, cache.to(DEV), ints(table), ints(ptr), ints(tok), None, w_uk, w_uv,
                         latent[:cap], out[0][:cap], out[1][:cap], dec.scratch)
        torch.cuda.synchronize()
        s = dec.status()
        dec.reset_status()
        return s

    assert go([0, 2, 4], [0, 32, 60], 90) == B.PDA_STATUS_PAGE_OOB
    assert torch.equal(latent[:16].cpu().double(), values[3])
    assert bool((latent[16:32] == 0).all()) and bool((out[0][16:32] == 0).all())
    assert torch.equal(latent[32:48].cpu().double(), values[5])
    assert go([0, 3, 5], [0, 41, 60], 90) == B.PDA_STATUS_KV_LEN_GT_MAX
    assert bool((latent[:41] == 0).all()) and bool((out[1][:41] == 0).all())
    latent.fill_(7.0)
    out[0].fill_(7.0)
    assert go([2, 4, 5], [0, 32, 40], 35) == B.PDA_STATUS_TOKENS_GT_CAP
    assert torch.equal(latent[:16].cpu().double(), values[5])
    assert bool((latent[35:] == 7).all()) and bool((out[0][35:] == 7).all())


class Pre:
    """Device arrays of one pda_mla_prefill call; what no request uses is NaN."""

    def __init__(self, reqs, heads, *, causal=True, windows=None, std=1.0, seed=0, rows_cap=None,
                 toks_cap=None, batch=None, max_kv=None, scale=192 ** -0.5):
        g = torch.Generator().manual_seed(seed + 31 * heads + sum(r for r, _ in reqs))
        self.qo, self.tok = [0], [0]
        for r, n in reqs:
            self.qo.append(self.qo[-1] + r)
            self.tok.append(self.tok[-1] + n)
        rows, toks = self.qo[-1], self.tok[-1]
        self.rows_cap, self.toks_cap = rows_cap or rows + 3, toks_cap or toks + 5
        nan = math.nan
        self.q = torch.full((self.rows_cap, heads, 200), nan, dtype=torch.bfloat16)
        self.q[:rows, :, :192] = randn(g, rows, heads, 192, std=std)
        self.kv = torch.full((self.toks_cap, heads, 256), nan, dtype=torch.bfloat16)
        self.kv[:toks] = randn(g, toks, heads, 256)
        self.lat = torch.full((self.toks_cap, 576), nan, dtype=torch.bfloat16)
        self.lat[:toks, 512:] = randn(g, toks, 64)
        self.heads, self.causal, self.windows, self.scale = heads, causal, windows, scale
        self.dec = B.Decoder(ref.mla_plan(heads, batch=len(reqs), max_kv=max_kv or
                                          max(1, max(n for _, n in reqs))), device=DEV)
        self.pre = B.Prefill(self.dec.plan, self.rows_cap, self.toks_cap, device=DEV)
        self.dq, self.dkv, self.dlat = self.q.to(DEV), self.kv.to(DEV), self.lat.to(DEV)
        self.dqo, self.dtok = ints(self.qo), ints(self.tok)
        self.dwin = None if windows is None else ints(windows)
        self.out = torch.full((self.rows_cap, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.rows_cap, heads), 7.0, device=DEV)

    def run(self, lse=True, stream=None):
        self.pre.run(self.dq[..., :192], self.dkv[..., :128], self.dkv[..., 128:],
                     self.dlat[:, 512:], self.dqo, self.dtok, self.scale, self.out,
                     self.lse if lse else None, window=self.dwin, causal=self.causal, stream=stream)

    def compare(self, what="", skip=()):
        torch.cuda.synchronize()
        o, ob, l_, lb = ref.attention(self.q[..., :192], self.kv[..., :128], self.kv[..., 128:],
                                      self.lat[:, 512:], self.qo, self.tok, causal=self.causal,
                                      windows=self.windows, scale=self.scale)
        rest = torch.isnan(o[..., 0]).all(1)
        for b in skip:
            rest[self.qo[b]:self.qo[b + 1]] = True
        assert bool((self.out.cpu()[rest] == 7).all()) and bool((self.lse.cpu()[rest] == 7).all()), \
            f"{what}: rows of no request were written"
        check(self.out.cpu()[~rest], o[~rest], ob[~rest], what + " out")
        check(self.lse.cpu()[~rest], l_[~rest], lb[~rest], what + " lse")


PREFILL = {
    "one_key": ([(1, 1)], 1),
    "two": ([(2, 2)], 3),
    "short_ragged": ([(1, 5), (0, 9), (3, 3), (16, 17), (0, 0), (7, 130)], 2),
    "tile_127": ([(127, 127)], 2),
    "tile_128": ([(128, 128)], 2),
    "tile_129": ([(129, 129)], 2),
    "tile_255": ([(255, 383)], 1),
    "tile_256": ([(256, 256)], 1),
    "tile_257": ([(257, 300)], 1),
    "rows_513": ([(513, 513), (1, 1)], 2),
    "chunk": ([(40, 700), (130, 1000), (300, 301)], 4),
    "decode_like": ([(1, 1500), (2, 900), (1, 1), (8, 64)], 16),
    "one_row_long": ([(1, 5000)], 2),
    "short_items": ([(1 + r % 7, 8 + (r * 37) % 119) for r in range(60)], 40),
    "many": ([(r % 19, r % 19 + r * 3) for r in range(40)], 2),
}


@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill_causal(name):
    reqs, heads = PREFILL[name]
    p = Pre(reqs, heads)
    p.run()
    p.compare(name)
    assert p.pre.status() == 0


@pytest.mark.parametrize("name", ["one_key", "short_ragged", "tile_129", "chunk", "one_row_long"])
def test_prefill_not_causal(name):
    """Every key visible; keys fewer than rows, and none at all, are allowed."""
    reqs, heads = PREFILL[name]
    reqs = reqs + [(5, 2), (140, 0), (3, 128), (200, 1)]
    p = Pre(reqs, heads, causal=False)
    p.run()
    p.compare(name)
    assert p.pre.status() == 0


@pytest.mark.parametrize("w", [1, 2, 63, 64, 65, 127, 128, 129, 300])
def test_prefill_window(w):
    p = Pre([(300, 700), (1, 200), (64, 64), (129, 513)], 2, windows=[w, w, 0, -1])
    p.run()
    p.compare(f"window {w}")
    p = Pre([(700, 700), (260, 2000)], 1, windows=[w, w])
    p.run()
    p.compare(f"window {w} long")


@pytest.mark.parametrize("std,scale", [(8.0, 192 ** -0.5), (30.0, 192 ** -0.5), (1.0, -192 ** -0.5),
                                       (1.0, 0.0), (0.0, 192 ** -0.5)])
def test_prefill_peaked_and_signs(std, scale):
    """Large logits (the running maximum moves far), negative and zero scales."""
    p = Pre([(200, 900), (33, 33)], 2, std=std, scale=scale)
    p.run()
    p.compare(f"std {std} scale {scale}")


def test_prefill_rising_logits():
    """Logits that rise along the keys: the maximum moves in every tile."""
    p = Pre([(150, 1200)], 2)
    ramp = torch.linspace(0, 60, 1205)[:, None, None]
    p.q[:150, :, :192] = 1.0
    p.kv[:1200, :, :128] = (ramp[:1200] * 192 ** 0.5 / 128).to(torch.bfloat16)
    p.dq, p.dkv = p.q.to(DEV), p.kv.to(DEV)
    p.run()
    p.compare("rising")


def test_prefill_no_lse_and_other_requests_poison():
    """Without lse; another request's NaN values reach no one else."""
    p = Pre([(70, 200), (20, 77), (30, 300)], 3)
    p.kv[200:277] = math.nan
    p.lat[200:277] = math.nan
    p.dkv, p.dlat = p.kv.to(DEV), p.lat.to(DEV)
    p.run(lse=False)
    p.lse.copy_(torch.full_like(p.lse, 7.0))
    torch.cuda.synchronize()
    got = p.out.clone()
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), p.out.view(torch.int16))
    o, ob, l_, lb = ref.attention(p.q[..., :192], p.kv[..., :128], p.kv[..., 128:], p.lat[:, 512:],
                                  p.qo, p.tok, causal=True, windows=None, scale=p.scale)
    for r0, r1 in ((0, 70), (90, 120)):
        check(p.out[r0:r1], o[r0:r1], ob[r0:r1], "out")
        check(p.lse[r0:r1], l_[r0:r1], lb[r0:r1], "lse")
    assert bool(torch.isnan(p.out[70:90].float()).all())


def test_prefill_status():
    """A refused request stays unwritten, its bit is set, the others are right."""
    reqs = [(10, 50), (20, 12), (5, 90), (140, 200)]
    p = Pre(reqs, 2, max_kv=250)
    p.run()
    p.compare("fewer keys than rows", skip=[1])
    assert p.pre.status() == B.PDA_STATUS_KV_LEN_LT_ROWS
    p = Pre([(10, 50), (20, 120), (5, 90)], 2, max_kv=100)
    p.run()
    p.compare("above max_kv_len", skip=[1])
    assert p.pre.status() == B.PDA_STATUS_KV_LEN_GT_MAX
    p = Pre([(10, 50), (20, 60), (200, 210)], 2, rows_cap=230, toks_cap=330)
    p.pre = B.Prefill(p.dec.plan, 100, 330, device=DEV)
    p.dq, p.out, p.lse = p.dq[:100], p.out[:100], p.lse[:100]
    p.run()
    torch.cuda.synchronize()
    assert p.pre.status() == B.PDA_STATUS_ROWS_GT_CAP
    assert bool((p.out[30:] == 7).all()) and bool(torch.isfinite(p.out[:30].float()).all())
    p = Pre([(10, 50), (20, 60), (30, 100)], 2, toks_cap=300)
    p.pre = B.Prefill(p.dec.plan, p.rows_cap, 120, device=DEV)
    p.dkv, p.dlat = p.dkv[:120], p.dlat[:120]
    p.run()
    torch.cuda.synchronize()
    assert p.pre.status() == B.PDA_STATUS_TOKENS_GT_CAP
    assert bool((p.out[30:] == 7).all()) and not bool((p.out[:30] == 7).any())
    p.pre.reset_status()
    assert p.pre.status() == 0


def test_prefill_graph_and_streams():
    """Captured once and replayed with other lengths; then two calls at once."""
    shapes = ([(40, 100), (129, 300), (1, 64)], [(0, 0), (250, 512), (3, 3)], [(1, 1), (1, 1), (1, 1)])
    cap = dict(rows_cap=260, toks_cap=540, max_kv=540)
    p = Pre(shapes[0], 3, **cap)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for k, reqs in enumerate(shapes):
        n = Pre(reqs, 3, seed=k, **cap)
        for name in ("dq", "dkv", "dlat", "dqo", "dtok", "out", "lse"):
            getattr(p, name).copy_(getattr(n, name))
        p.q, p.kv, p.lat, p.qo, p.tok = n.q, n.kv, n.lat, n.qo, n.tok
        g.replay()
        p.compare(f"replay {k}")
    a, b = Pre([(300, 900)], 4, seed=5), Pre([(129, 2000), (60, 60)], 2, seed=6)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.run(stream=s1)
        b.run(stream=s2)
    a.compare("stream 1")
    b.compare("stream 2")


def test_prefill_graphs_share_a_scratch():
    """Two graphs over one scratch, with key chunks and without, replayed in turn."""
    a, b = Pre([(30, 3000)], 2, seed=1), Pre([(30, 3000)], 2, seed=2)
    b.pre = a.pre
    assert a.pre.plan.splits > 1
    graphs = []
    for p in (a, b):
        p.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    for _ in range(3):
        a.out.fill_(7.0), b.out.fill_(7.0)
        for g in graphs:
            g.replay()
        a.compare("first")
        b.compare("second")
    assert a.pre.status() == 0


# ------------------------------------------------------- the calls together

def dense_decode(q, lat, w_uk, w_uv, scale):
    """One request's decode rows in 64 bits from its latents: [R, H, 128]."""
    r, length = q.shape[0], lat.shape[0]
    qd, c = q.double(), lat[:, :512]
    k = torch.einsum("tc,hdc->thd", c, w_uk.double())
    v = torch.einsum("tc,hdc->thd", c, w_uv.double())
    s = (torch.einsum("rhd,thd->hrt", qd[..., :128], k) +
         torch.einsum("rhd,td->hrt", qd[..., 128:], lat[:, 512:])) * scale
    pos = length - r + torch.arange(r)[:, None]
    s = s.masked_fill(torch.arange(length)[None] > pos, -math.inf)
    return torch.einsum("hrt,thd->rhd", torch.softmax(s, -1), v)


@pytest.mark.parametrize("kind", ["bf16", "records"])
def test_serving_loop(kind):
    """Prefill, then decode steps: tables -> append -> (expand -> prefill | absorb
    -> decode -> project), the free list handed from step to step, all on the
    device. Compared with dense attention in 64 bits on the cached latents.

    Bound: the expanded form rounds k, v (2^-8 each) and the weights and the
    output; the absorbed form rounds q_lat, the weights, o_lat and the output.
    With logits of standard deviation about 1.3 (keys of unit variance) a
    logit is off by about 2^-8 x sqrt(192) x 192^-1/2 x 2 = 2^-7 at two
    roundings, and outputs stay below 4, so 0.05 holds with room, and the mean
    error below 5e-3; the records' decode adds the two-term E4M3 weights
    (2^-8)."""
    heads, page, pages, batch, cols = 16, 64, 40, 3, 8
    g = torch.Generator().manual_seed(11)
    scale = 192 ** -0.5
    w = randn(g, heads, 256, 512, std=512 ** -0.5).to(DEV)
    w_uk, w_uv = w[:, :128], w[:, 128:]
    max_kv, rows_cap, toks_cap = 450, 420, 1200
    dec = B.Decoder(ref.mla_plan(heads, kind=kind, page=page, pages=pages, batch=batch, max_kv=max_kv,
                                 max_q_len=2), device=DEV)
    pre = B.Prefill(dec.plan, rows_cap, toks_cap, device=DEV)
    width = 640 if kind == "records" else 576
    cache = torch.full((pages, page, 1, width), 0x7F, dtype=torch.uint8, device=DEV) \
        if kind == "records" else torch.full((pages, page, 1, width), math.nan, dtype=torch.bfloat16,
                                             device=DEV)
    scales = torch.full((pages, page, 1, 4), math.nan, device=DEV) if kind == "records" else None
    free = [ints([pages]), ints([0])]
    free_pages = torch.randperm(pages, generator=g).int().to(DEV)
    block = torch.full((batch, cols), -1, dtype=torch.int32, device=DEV)
    i = {k: torch.zeros(n, dtype=torch.int32, device=DEV) for k, n in
         dict(a=batch, b=batch, kv_indptr=batch + 1, qo=batch + 1, tok=batch + 1, pt=batch * cols,
              pos=rows_cap).items()}
    slot = torch.zeros(rows_cap, dtype=torch.int64, device=DEV)
    history = [torch.zeros(0, 576, dtype=torch.float64) for _ in range(batch)]
    for step, new in enumerate(([300, 5, 64], [1, 2, 1], [2, 1, 0], [1, 130, 2])):
        cached, kv_len = (i["a"], i["b"]) if step % 2 == 0 else (i["b"], i["a"])
        rows = sum(new)
        c_new = torch.full((rows_cap, 1, 576), math.nan, dtype=torch.bfloat16)
        c_new[:rows] = randn(g, rows, 1, 576)
        q = torch.full((rows_cap, heads, 192), math.nan, dtype=torch.bfloat16)
        q[:rows] = randn(g, rows, heads, 192)
        q = q.to(DEV)
        B.pda_build_tables(dec.plan, cached, ints(new), None, block, free_pages, free[step % 2],
                           free[1 - step % 2], kv_len, i["kv_indptr"], i["pt"], i["qo"], i["tok"],
                           slot, i["pos"], dec.scratch)
        B.pda_append_slots(dec.plan, c_new.to(DEV), None, slot, i["qo"][batch:], cache, None, scales,
                           None, dec.scratch)
        out = torch.full((rows_cap, heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        if max(new) > 2:
            latent = torch.empty(toks_cap, 576, dtype=torch.bfloat16, device=DEV)
            kv = torch.full((toks_cap, heads, 256), math.nan, dtype=torch.bfloat16, device=DEV)
            lse = torch.empty(rows_cap, heads, device=DEV)
            B.pda_mla_expand(dec.plan, cache, i["pt"], i["kv_indptr"], i["tok"], scales, w_uk, w_uv,
                             latent, kv[..., :128], kv[..., 128:], dec.scratch)
            pre.run(q, kv[..., :128], kv[..., 128:], latent[:, 512:], i["qo"], i["tok"], scale, out, lse)
        else:
            q_lat = torch.zeros(rows_cap, heads, 576, dtype=torch.bfloat16, device=DEV)
            o_lat = torch.zeros(rows_cap, heads, 512, dtype=torch.bfloat16, device=DEV)
            B.pda_mla_absorb(dec.plan, q, w_uk, 1.0, q_lat, i["qo"][batch:], dec.scratch)
            B.pda_decode(dec.plan, q_lat, cache, cache, i["pt"], i["kv_indptr"], kv_len, i["qo"], 2,
                         None, scale, scales, scales, o_lat, None, dec.scratch)
            B.pda_mla_project(dec.plan, o_lat, w_uv, out, i["qo"][batch:], dec.scratch)
        torch.cuda.synchronize()
        assert dec.status() == 0 and pre.status() == 0
        r0 = 0
        for b, n in enumerate(new):
            x = c_new[r0:r0 + n]
            x = ref.record_values(*ref.records(x)) if kind == "records" else x.double()
            history[b] = torch.cat([history[b], x.reshape(n, 576)])
            if n:
                want = dense_decode(q[r0:r0 + n].cpu(), history[b], w_uk.cpu(), w_uv.cpu(), scale)
                err = (out[r0:r0 + n].cpu().double() - want).abs()
                assert err.max() <= 0.05 and err.mean() <= 5e-3, (step, b, err.max(), err.mean())
            r0 += n
        assert bool((out[rows:] == 7).all())
    used = sum(-(-len(h) // page) for h in history)
    assert free[0].item() == pages - used


# ------------------------------------------------- offsets that pass 32 bits

def test_append_and_expand_far_pages():
    """A latent cache of 2^32 elements and more: the last pages are written and read."""
    g = torch.Generator().manual_seed(2)
    page, pages = 64, 120000  # 120000 x 64 x 576 elements = 4.4e9
    dec = B.Decoder(ref.mla_plan(2, page=page, pages=pages), device=DEV)
    cache = torch.zeros(pages, page, 1, 576, dtype=torch.bfloat16, device=DEV)
    x = randn(g, 150, 1, 576)
    slots = torch.tensor([(pages - 1 - i // page) * page + i % page for i in range(150)])
    B.pda_append_slots(dec.plan, x.to(DEV), None, slots.to(DEV), None, cache, None, None, None,
                       dec.scratch)
    latent = torch.zeros(150, 576, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(150, 2, 256, dtype=torch.bfloat16, device=DEV)
    w_uk, w_uv = weights(g, 2)
    B.pda_mla_expand(dec.plan, cache, ints([pages - 1, pages - 2, pages - 3]), ints([0, 3]), ints([0, 150]),
                     None, w_uk, w_uv, latent, kv[..., :128], kv[..., 128:], dec.scratch)
    assert dec.status() == 0
    assert torch.equal(latent.cpu(), x[:, 0])
    assert int(torch.count_nonzero(cache[:100]).item()) == 0
    y, mag = ref.product(x[:, :, :512].expand(150, 2, 512), w_uk.cpu())
    mag = mag * ref.sum_bound(512)
    check(kv[..., :128], y, mag + ref.BF16_HALF * (y.abs() + mag), "k")


def test_expand_and_prefill_far_rows():
    """More than 2^31 elements of k and v: rows and keys at the far end."""
    heads, page, n = 128, 64, 70000  # 70000 x 128 x 256 elements = 2.3e9
    pages = -(-n // page)
    g = torch.Generator(device=DEV).manual_seed(4)
    dec = B.Decoder(ref.mla_plan(heads, page=page, pages=pages, max_kv=n), device=DEV)
    cache = torch.randn(pages, page, 1, 576, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(heads, 256, 512, generator=g, device=DEV) * 512 ** -0.5).to(torch.bfloat16)
    latent = torch.zeros(n, 576, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(n, heads, 256, dtype=torch.bfloat16, device=DEV)
    B.pda_mla_expand(dec.plan, cache, torch.arange(pages, device=DEV).int(), ints([0, pages]),
                     ints([0, n]), None, w[:, :128], w[:, 128:], latent, kv[..., :128], kv[..., 128:],
                     dec.scratch)
    assert dec.status() == 0
    for t in (0, n // 2, n - 1):
        y, mag = ref.product(latent[t:t + 1, None, :512].expand(1, heads, 512).cpu(), w.cpu())
        mag = mag * ref.sum_bound(512)
        check(kv[t:t + 1], y, mag + ref.BF16_HALF * (y.abs() + mag), f"kv of token {t}")
    q = torch.randn(5, heads, 192, generator=g, device=DEV).to(torch.bfloat16)
    pre = B.Prefill(dec.plan, 5, n, device=DEV)
    out = torch.zeros(5, heads, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(5, heads, device=DEV)
    pre.run(q, kv[..., :128], kv[..., 128:], latent[:, 512:], ints([0, 5]), ints([0, n]), 192 ** -0.5,
            out, lse)
    assert pre.status() == 0
    some = [0, 77, 127]
    o, ob, l_, lb = ref.attention(q.cpu()[:, some], kv[:, some, :128].cpu(), kv[:, some, 128:].cpu(),
                                  latent[:, 512:].cpu(), [0, 5], [0, n], causal=True, windows=None,
                                  scale=192 ** -0.5)
    check(out[:, some], o, ob, "out")
    check(lse[:, some], l_, lb, "lse")


def test_prefill_extreme_logits():
    """Logits far below any usual one (all about -3e3), and a scale that is not a number."""
    p = Pre([(3, 200), (140, 400)], 1)
    p.q[:143, :, :192] = -15.0
    p.kv[:600, :, :128] += 15.0
    p.lat[:600, 512:] += 15.0
    p.dq, p.dkv, p.dlat = p.q.to(DEV), p.kv.to(DEV), p.lat.to(DEV)
    p.run()
    p.compare("far below")
    p = Pre([(3, 20)], 1, scale=math.nan)
    p.run()
    torch.cuda.synchronize()
    assert bool(torch.isnan(p.out[:3].float()).all())


def test_calls_refuse_tensors_of_other_shapes():
    g = torch.Generator().manual_seed(0)
    dec = B.Decoder(ref.mla_plan(4), device=DEV)
    w = randn(g, 4, 256, 512).to(DEV)
    out = torch.zeros(3, 4, 576, dtype=torch.bfloat16, device=DEV)
    q = randn(g, 3, 4, 192).to(DEV)
    for bad in (dict(q=q[..., :128]), dict(q=q.float()), dict(q=q.cpu()), dict(w=w[:3, :128]),
                dict(w=w.transpose(1, 2)[:, :128, :128]), dict(out=out[:2]), dict(out=out[..., ::2]),
                dict(num=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(num=torch.zeros(1, dtype=torch.int64, device=DEV))):
        a = {**dict(q=q, w=w[:, :128], out=out, num=None), **bad}
        with pytest.raises(ValueError):
            B.pda_mla_absorb(dec.plan, a["q"], a["w"], 1.0, a["out"], a["num"], dec.scratch)
    with pytest.raises(B.PdaError):
        B.pda_mla_absorb(dec.plan, q, w[:, :128], 1.0, out, None, dec.scratch[8:])
    other = ref.mla_plan(4, num_sms=152, device=1)  # a plan of another device
    plan = B.pda_plan(other)[0]
    with pytest.raises(B.PdaError):
        B.pda_mla_absorb(plan, q, w[:, :128], 1.0, out, None, dec.scratch)
