// pda_tables.cu -- block tables and slot maps of one step, built on the GPU
// from the request lengths, so that a step's pda_decode / pda_append_slots
// arrays need no host round trip and a captured graph can grow its requests.
//
// Mathematics: with have_b = ceil(cached_b / P), want_b = ceil((cached_b +
// new_b) / P) and need_b = want_b - have_b, the pages of request b come off
// the free list at offset E_b = sum_{b' < b} need_b'; it is granted when
// need_b = 0 or E_b + need_b <= free. The prefix counts refused requests too,
// so it is monotone: the granted ones form a run of the list without holes.
// The CSR offsets are exclusive prefix sums of what the listed requests hold.
//
// Bound: latency (a decode step moves tens of kilobytes). So one launch with
// no hand-off between CTAs: every CTA scans all the lengths itself (they stay
// in L2: 12 bytes a request) and then lists only its own requests, a few warps
// to each. A scan of a few hundred requests costs less than the second launch,
// or the device-wide scan with look-back, that would share it. 64 requests of one new
// row 4.1 us, 512 with some of 513 rows 9.6 (the longest request's few warps).

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "pda.h"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroups = 256;                      // CTAs over the requests
constexpr int kMaxBatch = kMaxGroups * kThreads;     // a CTA keeps <= kThreads requests
constexpr int kEntriesPerLane = 4;                   // see the slices rule in the launcher

struct TablesArgs {
  pda_tables t;
  uint32_t* status;
  int batch, page_shift, max_kv_len, num_pages;
};

// What the lengths of request b say, before the free list and the capacities.
struct Lens {
  int64_t row;
  int cached, added, have, want;  // have / want: pages before and after
  uint32_t bad;                   // status bits of an invalid request, else 0
};

__device__ __forceinline__ Lens lens_of(const TablesArgs& a, int b) {
  Lens l;
  const int c = __ldg(a.t.cached_len + b), n = __ldg(a.t.new_len + b);
  const int r = a.t.request ? __ldg(a.t.request + b) : b;
  l.bad = 0u;
  if (c < 0 || n < 0 || r < 0 || r >= a.t.table_rows) l.bad = PDA_STATUS_TABLE_INVALID;
  const int64_t kv = static_cast<int64_t>(c) + n;
  if (!l.bad && kv > a.max_kv_len) l.bad = PDA_STATUS_KV_LEN_GT_MAX | PDA_STATUS_TABLE_INVALID;
  const int64_t round = (1 << a.page_shift) - 1;
  l.have = l.bad ? 0 : static_cast<int>((c + round) >> a.page_shift);
  l.want = l.bad ? 0 : static_cast<int>((kv + round) >> a.page_shift);
  if (l.want > a.t.table_cols) {
    l.bad = PDA_STATUS_TABLE_INVALID;
    l.have = l.want = 0;
  }
  l.cached = l.bad ? 0 : c;
  l.added = l.bad ? 0 : n;
  l.row = r;
  return l;
}

// Exclusive prefix sum of one value per thread; the total goes to *total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the previous scan's readers are done with sh
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh[w];
    all += sh[w];
  }
  *total = all;
  return before + x - v;
}

// A request of this CTA, ready to be listed.
struct Listed {
  int64_t row;        // block_table row
  int32_t page0;      // first entry in page_table
  int32_t row0;       // first new row
  int32_t have;       // entries taken from the block table
  int32_t pages;      // entries listed
  int32_t cached, added;
  int32_t free_top;   // free_pages index of the first new page (the others below it)
};

__global__ void __launch_bounds__(kThreads) build_tables(const __grid_constant__ TablesArgs a) {
  __shared__ int64_t sh[kWarps];
  __shared__ Listed mine[kThreads];
  __shared__ int sh_first;
  const int tid = threadIdx.x;
  const int groups = gridDim.x;
  const int per_cta = (a.batch + groups - 1) / groups;
  const int c0 = blockIdx.x * per_cta, c1 = min(a.batch, c0 + per_cta);
  const bool reporter = blockIdx.x == 0 && blockIdx.y == 0;
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  const int free_count = max(0, __ldg(a.t.free_count));
  if (tid == 0) sh_first = INT_MAX;

  // new pages in front of this thread's requests
  int64_t need = 0, total;
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(a, b);
    need += l.want - l.have;
  }
  const int64_t need0 = block_scan(need, sh, &total);

  // pages, rows and tokens listed in front of them
  uint32_t bits = 0u;
  int64_t pages = 0, rows = 0, toks = 0, upto = need0;
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(a, b);
    const int n = l.want - l.have;
    upto += n;
    const bool granted = n == 0 || upto <= free_count;
    bits |= l.bad | (granted ? 0u : PDA_STATUS_NO_PAGES);
    pages += granted ? l.want : l.have;
    rows += granted ? l.added : 0;
    toks += l.cached + (granted ? l.added : 0);
  }
  const int64_t pages0 = block_scan(pages, sh, &total);
  const int64_t rows0 = block_scan(rows, sh, &total);
  const int64_t toks0 = block_scan(toks, sh, &total);

  // the first request that passes a capacity, if any (the prefixes are
  // monotone, so every later one passes it too)
  auto walk = [&](auto&& each) {
    int64_t u = need0, p = pages0, r = rows0, t = toks0;
    for (int b = b0; b < b1; ++b) {
      const Lens l = lens_of(a, b);
      const int n = l.want - l.have;
      const bool granted = n == 0 || u + n <= free_count;
      Listed e;
      e.row = l.row;
      e.have = l.have;
      e.pages = granted ? l.want : l.have;
      e.cached = l.cached;
      e.added = granted ? l.added : 0;
      e.free_top = static_cast<int32_t>(free_count - 1 - (granted ? u : 0));
      if (!each(b, e, p, r, t, u, granted && n > 0)) return;
      u += n;
      p += e.pages;
      r += e.added;
      t += l.cached + e.added;
    }
  };
  walk([&](int b, const Listed& e, int64_t p, int64_t r, int64_t t, int64_t, bool) {
    if (p + e.pages <= a.t.page_table_cap && r + e.added <= a.t.rows_cap &&
        t + e.cached + e.added <= INT_MAX)
      return true;
    atomicMin(&sh_first, b);
    return false;
  });
  __syncthreads();
  const int first = sh_first;  // requests [first, batch) are listed as empty
  if (reporter) {
    if (first < a.batch) bits |= PDA_STATUS_TABLE_FULL;
    if (bits) atomicOr(a.status, bits);
  }

  // the offsets: each CTA writes those behind its own requests, the first
  // CTA the leading zeros and what is left of the free list
  int64_t taken = 0;
  walk([&](int b, Listed e, int64_t p, int64_t r, int64_t t, int64_t u, bool took) {
    if (b >= first) {
      // capacity reached: this thread's remaining requests end where request
      // `first` would have begun, which only its own thread knows; see below
      return false;
    }
    if (took) taken = u + (e.pages - e.have);
    if (b < c0 || b >= c1) return true;
    e.page0 = static_cast<int32_t>(p);
    e.row0 = static_cast<int32_t>(r);
    mine[b - c0] = e;
    if (blockIdx.y == 0) {
      a.t.kv_len[b] = e.cached + e.added;
      a.t.kv_indptr[b + 1] = static_cast<int32_t>(p + e.pages);
      a.t.qo_indptr[b + 1] = static_cast<int32_t>(r + e.added);
      if (a.t.tok_indptr) a.t.tok_indptr[b + 1] = static_cast<int32_t>(t + e.cached + e.added);
    }
    return true;
  });
  if (reporter) {
    // `taken` rises with b, so the block's largest is the last granted one's
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const int64_t o = __shfl_xor_sync(0xffffffffu, taken, d);
      taken = o > taken ? o : taken;
    }
    __syncthreads();
    if ((tid & 31) == 0) sh[tid >> 5] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) taken = sh[w] > taken ? sh[w] : taken;
      *a.t.free_left = static_cast<int32_t>(free_count - taken);
      a.t.kv_indptr[0] = 0;
      a.t.qo_indptr[0] = 0;
      if (a.t.tok_indptr) a.t.tok_indptr[0] = 0;
    }
  }
  if (first < c1) {
    // empty requests of this CTA: the prefixes in front of request `first`
    __shared__ int64_t at[3];
    walk([&](int b, const Listed&, int64_t p, int64_t r, int64_t t, int64_t, bool) {
      if (b != first) return true;
      at[0] = p;
      at[1] = r;
      at[2] = t;
      return false;
    });
    __syncthreads();
    for (int b = max(c0, first) + tid; b < c1; b += kThreads) {
      Listed e = {};
      mine[b - c0] = e;
      if (blockIdx.y == 0) {
        a.t.kv_len[b] = 0;
        a.t.kv_indptr[b + 1] = static_cast<int32_t>(at[0]);
        a.t.qo_indptr[b + 1] = static_cast<int32_t>(at[1]);
        if (a.t.tok_indptr) a.t.tok_indptr[b + 1] = static_cast<int32_t>(at[2]);
      }
    }
  }
  __syncthreads();

  // list the requests: kWarps / n warps to each of this CTA's n requests
  // (one warp to several when n is larger), times gridDim.y slices
  const int n = c1 - c0;
  if (n <= 0) return;
  const int warp = tid >> 5, lane = tid & 31;
  const int wpr = n < kWarps ? kWarps / n : 1;
  const int step = static_cast<int>(gridDim.y) * wpr * 32;
  const int from = (static_cast<int>(blockIdx.y) * wpr + warp % wpr) * 32 + lane;
  bool oob = false;
  for (int k = warp / wpr; k < n; k += kWarps / wpr) {
    const Listed e = mine[k];
    int32_t* own = a.t.block_table + e.row * a.t.table_stride;
    auto page_of = [&](int j) {
      return j < e.have ? own[j] : __ldg(a.t.free_pages + (e.free_top - (j - e.have)));
    };
#pragma unroll 4
    for (int j = from; j < e.pages; j += step) {
      const int id = page_of(j);
      a.t.page_table[e.page0 + j] = id;
      if (j >= e.have) own[j] = id;
    }
    if (!a.t.slot_map && !a.t.positions) continue;
#pragma unroll 4
    for (int i = from; i < e.added; i += step) {
      const int tok = e.cached + i;
      if (a.t.slot_map) {
        const int id = page_of(tok >> a.page_shift);
        const bool ok = id >= 0 && id < a.num_pages;
        oob |= !ok;
        a.t.slot_map[e.row0 + i] =
            ok ? (static_cast<int64_t>(id) << a.page_shift) + (tok & ((1 << a.page_shift) - 1)) : -1;
      }
      if (a.t.positions) a.t.positions[e.row0 + i] = tok;
    }
  }
  if (oob) atomicOr(a.status, PDA_STATUS_PAGE_OOB);
}

}  // namespace
}  // namespace pda

extern "C" int pda_build_tables(const pda_plan_t* plan, const pda_tables* tables,
                                void* split_scratch, pda_stream_t stream) {
  if (!plan || !tables) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  const pda_tables& t = *tables;
  // (an array of no entries may be NULL)
  if (!t.cached_len || !t.new_len || (!t.block_table && t.table_cols) || !t.free_pages ||
      !t.free_count || !t.free_left || !t.kv_len || !t.kv_indptr ||
      (!t.page_table && t.page_table_cap) || !t.qo_indptr)
    return PDA_ERR_NULL;
  if (!split_scratch || reinterpret_cast<uintptr_t>(split_scratch) % 256) return PDA_ERR_SCRATCH;
  if (t.table_rows < 1 || t.table_cols < 0 || t.table_stride < t.table_cols ||
      t.page_table_cap < 0 || t.rows_cap < 0 || plan->batch > pda::kMaxBatch ||
      t.free_left == t.free_count || t.kv_len == t.cached_len || t.kv_len == t.new_len)
    return PDA_ERR_INVALID;
  if (!t.request && t.table_rows < plan->batch) return PDA_ERR_INVALID;
  auto a4 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
  if (!a4(t.cached_len) || !a4(t.new_len) || !a4(t.request) || !a4(t.block_table) ||
      !a4(t.free_pages) || !a4(t.free_count) || !a4(t.free_left) || !a4(t.kv_len) ||
      !a4(t.kv_indptr) || !a4(t.page_table) || !a4(t.qo_indptr) || !a4(t.tok_indptr) ||
      !a4(t.positions) || reinterpret_cast<uintptr_t>(t.slot_map) % 8)
    return PDA_ERR_ALIGNMENT;
  if (plan->batch == 0) return PDA_OK;
  if (!pda::on_device(plan->device)) return PDA_ERR_INVALID;

  pda::TablesArgs a;
  a.t = t;
  a.status = static_cast<uint32_t*>(split_scratch);
  a.batch = plan->batch;
  a.page_shift = 0;
  while ((1 << a.page_shift) < plan->page_size) ++a.page_shift;
  a.max_kv_len = plan->max_kv_len;
  a.num_pages = plan->num_pages;
  const int groups = plan->batch < pda::kMaxGroups ? plan->batch : pda::kMaxGroups;
  // Slices of a request over CTAs, so that a lane lists about
  // kEntriesPerLane entries when the requests fill the capacities evenly.
  const int per_cta = (plan->batch + groups - 1) / groups;
  const int lanes = 32 * (per_cta < pda::kWarps ? pda::kWarps / per_cta : 1);
  const int64_t rows = t.slot_map || t.positions ? t.rows_cap : 0;  // none are listed without
  const int64_t entries = (t.page_table_cap + rows) / plan->batch;
  int64_t slices = (entries + lanes * pda::kEntriesPerLane - 1) / (lanes * pda::kEntriesPerLane);
  slices = slices < 1 ? 1 : (slices > 32 ? 32 : slices);
  pda::build_tables<<<dim3(groups, static_cast<unsigned>(slices)), pda::kThreads, 0,
                      reinterpret_cast<cudaStream_t>(stream)>>>(a);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  return PDA_OK;
}
