// pda_pages.cu -- the life of a cache's pages beyond growth: forking requests
// that share pages, copying pages, listing the free ones from what the block
// tables still hold, and moving pages together.
//
// Which pages are free follows from the block tables alone (a page is live while a
// listed request holds it, however many do), so a fork counts nothing, no page is
// freed twice or forgotten, and every call gives the same outputs for the same
// inputs, in an order that does not depend on the GPU's schedule.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "pda.h"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------- forks
//
// Mathematics: fork f with n_f shared tokens needs a page of its own when n_f
// ends inside one (both requests would write there): need_f = (n_f mod P > 0),
// taken off the free list at offset sum_{f' < f} need_f', refused forks counted
// too, as pda_build_tables takes its pages.
//
// Bound: latency, as there; so every CTA scans all the forks and lists its own. 48 forks of
// 128 pages with their copies of 8 heads of 128: 5.4 us both calls, 256 of records: 6.4.
constexpr int kMaxGroups = 256;
constexpr int kMaxForks = kMaxGroups * kThreads;  // a CTA keeps <= kThreads forks

struct ForkArgs {
  pda_forks f;
  uint32_t* status;
  int page_shift, max_kv_len, num_pages;
};

struct Fork {
  int parent, child, len;
  uint32_t bad;
};
__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int i) {
  Fork k;
  k.parent = __ldg(a.f.parent + i);
  k.child = __ldg(a.f.child + i);
  k.len = __ldg(a.f.shared_len + i);
  k.bad = 0u;
  const bool rows = k.parent >= 0 && k.parent < a.f.table_rows && k.child >= 0 &&
                    k.child < a.f.table_rows && k.parent != k.child;
  const int64_t pages = (static_cast<int64_t>(k.len) + (1 << a.page_shift) - 1) >> a.page_shift;
  if (!rows || k.len < 0 || pages > a.f.table_cols) k.bad = PDA_STATUS_TABLE_INVALID;
  if (k.len > a.max_kv_len) k.bad |= PDA_STATUS_KV_LEN_GT_MAX | PDA_STATUS_TABLE_INVALID;
  if (k.bad) k.len = 0;
  return k;
}

__global__ void __launch_bounds__(kThreads) fork_tables(const __grid_constant__ ForkArgs a) {
  __shared__ int sums[kWarps];
  __shared__ int upto_s[kThreads];  // pages taken up to and with each of this CTA's forks
  grid_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.f.forks;
  const int per_cta = (n + gridDim.x - 1) / gridDim.x;
  const int c0 = blockIdx.x * per_cta, c1 = min(n, c0 + per_cta);
  const int per = (n + kThreads - 1) / kThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  const int mask = (1 << a.page_shift) - 1;
  const int free_count = max(0, __ldg(a.f.free_count));
  int need = 0;
  uint32_t bits = 0u;
  for (int i = i0; i < i1; ++i) {
    const Fork k = fork_of(a, i);
    bits |= k.bad;
    need += (k.len & mask) != 0;
  }
  int x = need;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int upto = x - need, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += sums[w];
    total += sums[w];
  }
  for (int i = i0; i < i1; ++i) {
    upto += (fork_of(a, i).len & mask) != 0;
    if (i >= c0 && i < c1) upto_s[i - c0] = upto;
  }
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // (the needs are 0 or 1: every page up to the list's end is taken)
    if (total > free_count) bits |= PDA_STATUS_NO_PAGES;
    if (bits) atomicOr(a.status, bits);
    if (tid == 0) *a.f.free_left = free_count - min(total, free_count);
  }
  __syncthreads();

  // kWarps / m warps to each of this CTA's m forks, times gridDim.y slices
  const int m = c1 - c0;
  if (m <= 0) return;
  const int wpf = m < kWarps ? kWarps / m : 1;
  const int step = static_cast<int>(gridDim.y) * wpf * 32;
  const int from = (static_cast<int>(blockIdx.y) * wpf + warp % wpf) * 32 + lane;
  bool oob = false;
  for (int c = warp / wpf; c < m; c += kWarps / wpf) {
    const int i = c0 + c;
    const Fork k = fork_of(a, i);
    const bool part = (k.len & mask) != 0;
    const bool granted = !k.bad && (!part || upto_s[c] <= free_count);
    const int32_t* theirs = a.f.block_table + static_cast<int64_t>(k.parent) * a.f.table_stride;
    int32_t* mine = a.f.block_table + static_cast<int64_t>(k.child) * a.f.table_stride;
    const int full = granted ? k.len >> a.page_shift : 0;
#pragma unroll 4
    for (int j = from; j < full; j += step) {
      const int id = theirs[j];
      oob |= id < 0 || id >= a.num_pages;
      mine[j] = id;
    }
    if (from == 0) {
      int src = -1, dst = -1, tokens = 0;
      if (granted && part) {
        src = theirs[full];
        dst = __ldg(a.f.free_pages + (free_count - upto_s[c]));
        mine[full] = dst;
        tokens = k.len & mask;
        if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
          oob = true;
          src = dst = -1;
          tokens = 0;
        }
      }
      a.f.child_len[i] = granted ? k.len : 0;
      a.f.copy_src[i] = src;
      a.f.copy_dst[i] = dst;
      a.f.copy_tokens[i] = tokens;
    }
  }
  if (oob) atomicOr(a.status, PDA_STATUS_PAGE_OOB);
}

// ------------------------------------------------------------------ copies
//
// Bound: HBM, each byte read and written once. A unit is kPiece bytes of one side
// of one copy; CTAs stride over the units, four 16-byte loads in flight a thread.
// 900 pages of 131 KB, K and V, 472 MB in 72 us, 6.5 TB/s. The launch is under way
// behind a fork's kernel; it waits for that before it reads anything.
constexpr int kPiece = kThreads * 4 * 16;

struct CopyArgs {
  uint8_t* side[2];
  float* scale[2];
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  const int32_t* num_copies;
  uint32_t* status;
  int64_t page_bytes, token_bytes, head_bytes;  // strides
  int copies, sides, page_size, heads, num_pages;
  int row_vecs;      // 16-byte pieces of one (token, head) row
  int layout;        // 0: token, head, channel without gaps; 1: head, token; 2: any strides
  int pieces;        // units of a side of a whole page
  int scale_floats;  // of a token, all heads (0: none)
};

__global__ void __launch_bounds__(kThreads) copy_pages(const __grid_constant__ CopyArgs a) {
  grid_wait();
  // (the lists by plain loads: the kernel in front, beside which this one has started, may have
  // written them, and the read-only path is for memory that nobody writes meanwhile)
  int n = a.copies;
  if (a.num_copies) n = min(n, *a.num_copies);
  const int64_t units = static_cast<int64_t>(max(n, 0)) * a.sides * a.pieces;
  bool oob = false;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = static_cast<int>(u % a.pieces);
    const int64_t r = u / a.pieces;
    const int side = static_cast<int>(r % a.sides), c = static_cast<int>(r / a.sides);
    const int src = a.src[c], dst = a.dst[c];
    if (src == -1 || dst == -1 || src == dst) continue;
    if (src < 0 || dst < 0 || src >= a.num_pages || dst >= a.num_pages) {
      oob = true;
      continue;
    }
    const int tokens = a.tokens ? max(0, min(a.page_size, a.tokens[c])) : a.page_size;
    const uint8_t* from = a.side[side] + src * a.page_bytes;
    uint8_t* to = a.side[side] + dst * a.page_bytes;
    const int run = a.layout == 0 ? tokens * a.heads * a.row_vecs
                                  : a.layout == 1 ? tokens * a.row_vecs : a.row_vecs;
    const int vecs = tokens * a.heads * a.row_vecs;
    uint4 v[4];
    int64_t at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = (piece * 4 + k) * kThreads + static_cast<int>(threadIdx.x);
      at[k] = -1;
      if (i < vecs) {
        const int seg = a.layout == 0 ? 0 : i / run;
        at[k] = static_cast<int64_t>(i - seg * run) * 16;
        if (a.layout == 1) at[k] += seg * a.head_bytes;
        if (a.layout == 2) at[k] += (seg / a.heads) * a.token_bytes + (seg % a.heads) * a.head_bytes;
        v[k] = *reinterpret_cast<const uint4*>(from + at[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k] >= 0) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
    if (piece == 0 && a.scale_floats) {
      const int64_t per = static_cast<int64_t>(a.page_size) * a.scale_floats;
      const float* sf = a.scale[side] + src * per;
      float* st = a.scale[side] + dst * per;
      for (int i = threadIdx.x; i < tokens * a.scale_floats; i += kThreads) st[i] = sf[i];
    }
  }
  if (oob && threadIdx.x == 0) atomicOr(a.status, PDA_STATUS_PAGE_OOB);
}

// ------------------------------------------------------ free and compacted
//
// Mathematics: a bit per page marks the live ones. With F(x) the free ids below
// x and T free in all, free id x stands at place T - 1 - F(x) of the list (the
// lowest id last, taken first), and the id x has x - F(x) live ones below it. With
// N - T = L live ids, a full compaction fills the F(L) holes below L from the
// F(L) live ids from L on; m = min(F(L), max_copies) moves pair the k-th highest
// live id with the k-th lowest hole. Filled holes lie below L, moved ids above, so
// the places after the moves follow from the same counts:
//   x free and not filled:  T - 1 - F(x) + min(m, live ids above x)
//   x moved (k-th highest): T - F(x) + k.
struct PagesArgs {
  pda_pages p;
  uint32_t* status;
  uint32_t* bits;      // live pages, zero between calls
  int32_t* below;      // F at the start of each word (compaction)
  int32_t* head;       // [0] CTAs done, zero between calls; [1] live pages; [2] moves
  int words, words_per_cta, compact;
  int page_shift, max_kv_len, num_pages;
};

// Entries of request r's row (what it lists stays held, invalid or not).
__device__ __forceinline__ int entries_of(const PagesArgs& a, int r, int64_t& row, uint32_t& bad) {
  const int len = __ldg(a.p.lengths + r);
  row = a.p.request ? __ldg(a.p.request + r) : r;
  if (len < 0 || row < 0 || row >= a.p.table_rows) {
    bad |= PDA_STATUS_TABLE_INVALID;
    return 0;
  }
  if (len > a.max_kv_len) bad |= PDA_STATUS_KV_LEN_GT_MAX | PDA_STATUS_TABLE_INVALID;
  const int64_t pages = (static_cast<int64_t>(len) + (1 << a.page_shift) - 1) >> a.page_shift;
  if (pages <= a.p.table_cols) return static_cast<int>(pages);
  bad |= PDA_STATUS_TABLE_INVALID;
  return a.p.table_cols;
}

// Marks kAtOnce ids (-1: none) in `bits`, their loads together and atomics for unset bits only
// (ids that many requests share are set once and read often).
constexpr int kAtOnce = 4;
__device__ __forceinline__ void mark(const PagesArgs& a, uint32_t* bits, const int (&id)[kAtOnce], uint32_t& bad) {
  uint32_t held[kAtOnce];
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    held[k] = 0xffffffffu;
    if (id[k] >= 0 && id[k] < a.num_pages) held[k] = *const_cast<volatile uint32_t*>(bits + (id[k] >> 5));
    else if (id[k] != -1) bad |= PDA_STATUS_PAGE_OOB;
  }
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) {
    const uint32_t bit = 1u << (id[k] & 31);
    if (!(held[k] & bit)) atomicOr(bits + (id[k] >> 5), bit);
  }
}

__global__ void __launch_bounds__(kThreads) mark_pages(const __grid_constant__ PagesArgs a) {
  grid_launch();
  uint32_t bad = 0u;
  for (int r = blockIdx.x; r < a.p.requests; r += gridDim.x) {
    int64_t row;
    const int n = entries_of(a, r, row, bad);
    const int32_t* ids = a.p.block_table + row * a.p.table_stride;
    const int step = static_cast<int>(gridDim.y) * kThreads;
    for (int j0 = blockIdx.y * kThreads + threadIdx.x; j0 < n; j0 += kAtOnce * step) {
      int id[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        id[k] = -1;
        if (j0 + k * step < n) {
          id[k] = __ldg(ids + j0 + k * step);
          if (id[k] == -1) bad |= PDA_STATUS_PAGE_OOB;
        }
      }
      mark(a, a.bits, id, bad);
    }
  }
  if (bad) atomicOr(a.status, bad);
}

__device__ __forceinline__ uint32_t free_word(const PagesArgs& a, const uint32_t* bits, int w) {
  const int left = a.num_pages - (w << 5);
  return ~bits[w] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
}

// Sum over the block of one value per thread. (One-shot code is bound by its instructions'
// way from memory, so it is kept short here and below.)
template <int kT>
__device__ __forceinline__ int block_sum(int v, int* sh) {
  const int lane = threadIdx.x & 31;
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < kT / 32 ? sh[lane] : 0);
}

// Free ids of words [from, to), from a multiple of 4, over the block's threads.
template <int kT>
__device__ __forceinline__ int count_free(const PagesArgs& a, const uint32_t* bits, int from, int to) {
  int n = 0;
  // (whole vectors stay inside the marks, whose memory is a multiple of 256 bytes; the last
  // word's ids past the cache, and words from `to` on, do not count)
#pragma unroll(kT == kThreads ? 4 : 1)
  for (int w = from + 4 * static_cast<int>(threadIdx.x); w < to; w += 4 * kT) {
    const uint4 v = *reinterpret_cast<const uint4*>(bits + w);
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (w + e < to) n += __popc(~x[e]);
  }
  if (threadIdx.x == 0 && to == a.words && from < to) n -= (a.words << 5) - a.num_pages;
  return n;
}

// Lists the free ids of words [w0, w1) (multiples of 4, or the end) and the moves there.
template <int kT>
__device__ __forceinline__ void list_words(const PagesArgs& a, const uint32_t* bits, int32_t* below, int w0, int w1,
                                           bool writes, int* sh, int& live, int& moves) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = block_sum<kT>(count_free<kT>(a, bits, 0, w0), sh);
  const int all = before + block_sum<kT>(count_free<kT>(a, bits, w0, a.words), sh);
  live = a.num_pages - all;
  moves = 0;
  if (a.compact) {
    // holes below the live count
    int holes = count_free<kT>(a, bits, 0, live >> 5);
    if (threadIdx.x == 0 && (live & 31)) holes += __popc(free_word(a, bits, live >> 5) & ((1u << (live & 31)) - 1u));
    moves = min(block_sum<kT>(holes, sh), a.p.max_copies);
  }
  if (writes && threadIdx.x == 0) {
    *a.p.free_left = all;
    if (a.compact) *a.p.num_copies = moves;
  }
  // a warp to 32 words at a time: the words' prefix, then a word a step, a lane an id
  constexpr int kW = kT / 32;
  const int each = max(1, min(32, (w1 - w0 + kW - 1) / kW));  // words of a warp's turn
#pragma unroll 1
  for (int g = w0; g < w1; g += each * kW) {
    const int w = g + warp * each + lane;
    const uint32_t mine = lane < each && w < w1 ? free_word(a, bits, w) : 0u;
    const int count = __popc(mine);
    int x = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    const int of_warp = lane < kW ? sh[lane] : 0;
    const int start = before + x - count + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
    before += __reduce_add_sync(0xffffffffu, of_warp);
    if (a.compact && lane < each && w < w1) below[w] = start;
#pragma unroll 1
    for (int k = 0; k < each; ++k) {
      const int wk = g + warp * each + k;
      if (wk >= w1) break;  // (the same for the whole warp)
      const uint32_t f = __shfl_sync(0xffffffffu, mine, k);
      const int fb = __shfl_sync(0xffffffffu, start, k) + __popc(f & ((1u << lane) - 1u));
      const int id = (wk << 5) + lane;
      if (id >= a.num_pages) continue;
      const bool is_free = f >> lane & 1u;
      const int above = live - (id - fb) - (is_free ? 0 : 1);  // live ids above
      if (is_free) {
        if (fb < moves) a.p.copy_dst[fb] = id;
        else a.p.free_pages[all - 1 - fb + min(moves, above)] = id;
      } else if (above < moves) {
        a.p.copy_src[above] = id;
        a.p.free_pages[all - fb + above] = id;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) list_pages(const __grid_constant__ PagesArgs a) {
  __shared__ int sh[kWarps];
  grid_launch();
  grid_wait();
  const int w0 = blockIdx.x * a.words_per_cta, w1 = min(a.words, w0 + a.words_per_cta);
  int live, moves;
  list_words<kThreads>(a, a.bits, a.below, w0, w1, blockIdx.x == 0, sh, live, moves);
  if (a.compact) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      a.head[1] = live;
      a.head[2] = moves;
    }
    return;
  }
  // the last CTA to get here clears the marks for the next call (compaction: later)
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.head, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  for (int w = threadIdx.x; w < a.words; w += kThreads) a.bits[w] = 0u;
  if (threadIdx.x == 0) a.head[0] = 0;
}

// What page `id` is called after the moves.
__device__ __forceinline__ int renamed(const PagesArgs& a, const uint32_t* bits, const int32_t* below, int live,
                                       int moves, int id) {
  if (moves == 0 || id < live || id >= a.num_pages) return id;
  const int w = id >> 5;
  const uint32_t f = free_word(a, bits, w);
  const int fb = below[w] + __popc(f & ((1u << (id & 31)) - 1u));
  const int k = live - 1 - (id - fb);
  return !(f >> (id & 31) & 1u) && k < moves ? a.p.copy_dst[k] : id;
}

// The tables after the moves.
__global__ void __launch_bounds__(kThreads) renumber(const __grid_constant__ PagesArgs a) {
  grid_wait();
  const int live = a.head[1], moves = a.head[2];
  uint32_t bad = 0u;
  for (int r = blockIdx.x; r < a.p.requests; r += gridDim.x) {
    int64_t row;
    const int n = entries_of(a, r, row, bad);
    const int32_t* ids = a.p.block_table + row * a.p.table_stride;
    int32_t* to = a.p.new_table + row * a.p.table_stride;
    const int step = static_cast<int>(gridDim.y) * kThreads;
    for (int j = blockIdx.y * kThreads + threadIdx.x; j < n; j += step)
      to[j] = renamed(a, a.bits, a.below, live, moves, ids[j]);
  }
  __shared__ int last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.head, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
  }
  __syncthreads();
  if (!last) return;
  for (int w = threadIdx.x; w < a.words; w += kThreads) a.bits[w] = 0u;
  if (threadIdx.x == 0) a.head[0] = 0;
}

// The marks of a CTA in shared memory: what many requests share is set there, where a word
// of marks in memory that every CTA sets at once takes its atomics one by one (512 requests
// of 1024 pages, half of them shared: 15 us).
constexpr int kOnceThreads = 1024;
constexpr int kOnceRequests = 512;               // most requests at a time
constexpr int kOnceEntries = 16 * kOnceThreads;  // entries of the tables that a CTA takes
constexpr int kOnceWords = 4096;                 // most words of marks where one CTA does it all
constexpr int kMarkWords = 16384;                // ... where CTAs mark theirs

struct Rows {
  int row[kOnceRequests], n[kOnceRequests];
};
// Requests first, first + step, ... (`count` of them): their rows and entries. All threads.
__device__ __forceinline__ void rows_of(const PagesArgs& a, Rows& rows, int first, int step, int count, uint32_t& bad) {
  __syncthreads();
  if (threadIdx.x < count) {
    int64_t row;
    rows.n[threadIdx.x] = entries_of(a, first + static_cast<int>(threadIdx.x) * step, row, bad);
    rows.row[threadIdx.x] = static_cast<int>(row);
  }
  __syncthreads();
}
// Their entries, kAtOnce at a time: use(ids, places in the tables); no place: -1.
template <class F>
__device__ __forceinline__ void each_entry(const PagesArgs& a, const Rows& rows, int count, F&& use) {
  const int cols = max(1, a.p.table_cols), rows_on = kOnceThreads / cols, cols_on = kOnceThreads - rows_on * cols;
  int r = threadIdx.x / cols, j = threadIdx.x - r * cols;
#pragma unroll 1
  while (r < count) {
    int id[kAtOnce];
    int64_t at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      at[k] = r < count && j < rows.n[r] ? rows.row[r] * a.p.table_stride + j : -1;
      id[k] = at[k] >= 0 ? a.p.block_table[at[k]] : -1;
      r += rows_on;
      j += cols_on;
      if (j >= cols) {
        j -= cols;
        ++r;
      }
    }
    use(id, at);
  }
}
__device__ __forceinline__ void mark_rows(const PagesArgs& a, const Rows& rows, int count, uint32_t* marks,
                                          uint32_t& bad) {
  each_entry(a, rows, count, [&](const int (&id)[kAtOnce], const int64_t (&at)[kAtOnce]) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (at[k] >= 0 && id[k] == -1) bad |= PDA_STATUS_PAGE_OOB;
    mark(a, marks, id, bad);
  });
}

__global__ void __launch_bounds__(kOnceThreads) mark_shared(const __grid_constant__ PagesArgs a) {
  extern __shared__ __align__(16) uint32_t marks[];  // [words]
  __shared__ Rows rows;
  grid_launch();
  uint32_t bad = 0u;
#pragma unroll 1
  for (int w = threadIdx.x; w < a.words; w += kOnceThreads) marks[w] = 0u;
  const int step = static_cast<int>(gridDim.x);
#pragma unroll 1
  for (int r = blockIdx.x; r < a.p.requests; r += kOnceRequests * step) {
    const int count = min(kOnceRequests, (a.p.requests - r + step - 1) / step);
    rows_of(a, rows, r, step, count, bad);
    mark_rows(a, rows, count, marks, bad);
  }
  __syncthreads();
#pragma unroll 1
  for (int w = threadIdx.x; w < a.words; w += kOnceThreads)
    if (marks[w]) atomicOr(a.bits + w, marks[w]);
  if (bad) atomicOr(a.status, bad);
}

// All of it in one CTA, where the tables and the cache are small: 4096 entries are freed in
// 5.4 us, two launches take 8.9. Bound by latency: what runs once is kept short, since its
// instructions come from memory (the same with its loops unrolled: 9.6 us).
__global__ void __launch_bounds__(kOnceThreads) pages_once(const __grid_constant__ PagesArgs a) {
  extern __shared__ __align__(16) uint32_t marks[];  // [words up to a multiple of 4], then `below`
  __shared__ Rows rows;
  __shared__ int sh[kOnceThreads / 32];
  const int words4 = (a.words + 3) / 4 * 4;
  int32_t* below = reinterpret_cast<int32_t*>(marks + words4);
  uint32_t bad = 0u;
#pragma unroll 1
  for (int w = threadIdx.x; w < words4; w += kOnceThreads) marks[w] = 0u;
  rows_of(a, rows, 0, 1, a.p.requests, bad);
  mark_rows(a, rows, a.p.requests, marks, bad);
  if (bad) atomicOr(a.status, bad);
  __syncthreads();
  int live, moves;
  list_words<kOnceThreads>(a, marks, below, 0, a.words, true, sh, live, moves);
  if (!a.compact) return;
  __syncthreads();  // (the moves' targets and `below` are there)
  each_entry(a, rows, a.p.requests, [&](const int (&id)[kAtOnce], const int64_t (&at)[kAtOnce]) {
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (at[k] >= 0) a.p.new_table[at[k]] = renamed(a, marks, below, live, moves, id[k]);
  });
}

bool a4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

int64_t page_words(const pda_plan_t* plan) { return (static_cast<int64_t>(plan->num_pages) + 31) / 32; }

int page_shift_of(const pda_plan_t* plan) {
  int s = 0;
  while ((1 << s) < plan->page_size) ++s;
  return s;
}

template <class Args>
int launch_next(void (*fn)(Args), dim3 grid, cudaStream_t s, const Args& a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, a) == cudaSuccess) return PDA_OK;
  cudaGetLastError();
  return PDA_ERR_CUDA;
}

int list_call(const pda_plan_t* plan, const pda_pages* pages, void* scratch, pda_stream_t stream,
              bool compact) {
  if (!plan || !pages) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  const pda_pages& p = *pages;
  const bool entries = p.requests > 0 && p.table_cols > 0;
  if ((!p.lengths && p.requests) || (!p.block_table && entries) || !p.free_pages || !p.free_left)
    return PDA_ERR_NULL;
  if (compact && ((!p.new_table && entries) || !p.num_copies ||
                  ((!p.copy_src || !p.copy_dst) && p.max_copies)))
    return PDA_ERR_NULL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return PDA_ERR_SCRATCH;
  if (p.requests < 0 || p.table_cols < 0 || p.table_rows < 0 || p.table_stride < p.table_cols ||
      (compact && p.max_copies < 0) || (!p.request && p.table_rows < p.requests))
    return PDA_ERR_INVALID;
  if (!a4(p.lengths) || !a4(p.request) || !a4(p.block_table) || !a4(p.free_pages) ||
      !a4(p.free_left) ||
      (compact && (!a4(p.new_table) || !a4(p.copy_src) || !a4(p.copy_dst) || !a4(p.num_copies))))
    return PDA_ERR_ALIGNMENT;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  PagesArgs a = {};
  a.p = p;
  char* base = static_cast<char*>(scratch);
  const int64_t words = page_words(plan);
  a.status = reinterpret_cast<uint32_t*>(base);
  a.head = reinterpret_cast<int32_t*>(base) + 16;
  a.bits = reinterpret_cast<uint32_t*>(base + kStatusHeaderBytes);
  a.below = reinterpret_cast<int32_t*>(base + kStatusHeaderBytes + (words * 4 + 255) / 256 * 256);
  a.words = static_cast<int>(words);
  a.compact = compact ? 1 : 0;
  a.page_shift = page_shift_of(plan);
  a.max_kv_len = plan->max_kv_len;
  a.num_pages = plan->num_pages;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (words <= kOnceWords && static_cast<int64_t>(p.requests) * p.table_cols <= kOnceEntries &&
      p.requests <= kOnceRequests) {
    pages_once<<<1, kOnceThreads, static_cast<size_t>((words + 3) / 4 * 4 * 8), s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
  }
  const unsigned gx = static_cast<unsigned>(std::max(1, std::min(p.requests, 4 * plan->num_sms)));
  const unsigned gy = static_cast<unsigned>(
      std::max(1, std::min(64, (p.table_cols + 4 * kThreads - 1) / (4 * kThreads))));
  if (words <= kMarkWords) {
    if (words > 8192 && cudaFuncSetAttribute(reinterpret_cast<const void*>(mark_shared),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMarkWords * 4) != cudaSuccess) {
      cudaGetLastError();
      return PDA_ERR_CUDA;
    }
    const int64_t ctas = (static_cast<int64_t>(p.requests) * p.table_cols + kOnceEntries - 1) / kOnceEntries;
    const unsigned g = static_cast<unsigned>(
        std::max<int64_t>(1, std::min<int64_t>({ctas, p.requests, plan->num_sms})));
    mark_shared<<<g, kOnceThreads, static_cast<size_t>(words * 4), s>>>(a);
  } else {
    mark_pages<<<dim3(gx, gy), kThreads, 0, s>>>(a);
  }
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  // (a CTA's warps list 8 words each, or more)
  const int64_t least = 8 * kWarps;
  const int64_t per = std::max(least, (words + plan->num_sms - 1) / plan->num_sms);
  a.words_per_cta = static_cast<int>(std::min<int64_t>((per + least - 1) / least * least, INT_MAX / 2));
  const unsigned gl = static_cast<unsigned>((words + a.words_per_cta - 1) / a.words_per_cta);
  const int rc = launch_next(list_pages, dim3(gl), s, a);
  if (rc != PDA_OK || !compact) return rc;
  return launch_next(renumber, dim3(gx, gy), s, a);
}

}  // namespace
}  // namespace pda

extern "C" int pda_fork_tables(const pda_plan_t* plan, const pda_forks* forks, void* split_scratch,
                               pda_stream_t stream) {
  using namespace pda;
  if (!plan || !forks) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  const pda_forks& f = *forks;
  if (!f.free_pages || !f.free_count || !f.free_left) return PDA_ERR_NULL;
  if (f.forks > 0 && (!f.parent || !f.child || !f.shared_len || (!f.block_table && f.table_cols) ||
                      !f.child_len || !f.copy_src || !f.copy_dst || !f.copy_tokens))
    return PDA_ERR_NULL;
  if (!split_scratch || reinterpret_cast<uintptr_t>(split_scratch) % 256) return PDA_ERR_SCRATCH;
  if (f.forks < 0 || f.forks > kMaxForks || f.table_rows < 0 || f.table_cols < 0 ||
      f.table_stride < f.table_cols || f.free_left == f.free_count ||
      (f.forks > 0 && f.child_len == f.shared_len))
    return PDA_ERR_INVALID;
  if (!a4(f.parent) || !a4(f.child) || !a4(f.shared_len) || !a4(f.block_table) ||
      !a4(f.free_pages) || !a4(f.free_count) || !a4(f.free_left) || !a4(f.child_len) ||
      !a4(f.copy_src) || !a4(f.copy_dst) || !a4(f.copy_tokens))
    return PDA_ERR_ALIGNMENT;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  ForkArgs a = {};
  a.f = f;
  a.status = static_cast<uint32_t*>(split_scratch);
  a.page_shift = page_shift_of(plan);
  a.max_kv_len = plan->max_kv_len;
  a.num_pages = plan->num_pages;
  const int groups = std::max(1, std::min(f.forks, kMaxGroups));
  const int per_cta = (f.forks + groups - 1) / groups;
  const int lanes = 32 * (per_cta > 0 && per_cta < kWarps ? kWarps / per_cta : 1);
  const int slices = std::max(1, std::min(32, (f.table_cols + 4 * lanes - 1) / (4 * lanes)));
  fork_tables<<<dim3(groups, slices), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

extern "C" int pda_copy_pages(const pda_plan_t* plan, void* k_pages, void* v_pages, float* k_scale,
                              float* v_scale, const int32_t* copy_src, const int32_t* copy_dst,
                              const int32_t* copy_tokens, int32_t copies, const int32_t* num_copies,
                              void* split_scratch, pda_stream_t stream) {
  using namespace pda;
  if (!plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  if (copies < 0) return PDA_ERR_INVALID;
  const bool latent = plan->head_dim == 576;
  const int per_head = plan->scale_mode == PDA_SCALE_MLA_BLOCK    ? 4
                       : plan->scale_mode == PDA_SCALE_TOKEN_HEAD ? 1
                                                                  : 0;
  if (!k_pages || (!latent && !v_pages) || (copies && (!copy_src || !copy_dst))) return PDA_ERR_NULL;
  if (per_head && (!k_scale || (!latent && !v_scale))) return PDA_ERR_NULL;
  if (!split_scratch || reinterpret_cast<uintptr_t>(split_scratch) % 256) return PDA_ERR_SCRATCH;
  auto a16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  if (!a16(k_pages) || (!latent && !a16(v_pages)) || !a4(copy_src) || !a4(copy_dst) ||
      !a4(copy_tokens) || !a4(num_copies) || (per_head && (!a4(k_scale) || (!latent && !a4(v_scale)))))
    return PDA_ERR_ALIGNMENT;
  if (copies == 0) return PDA_OK;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  CopyArgs a = {};
  const int eb = plan->kv_dtype == PDA_BF16 ? 2 : 1;
  a.side[0] = static_cast<uint8_t*>(k_pages);
  a.side[1] = static_cast<uint8_t*>(v_pages);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.src = copy_src;
  a.dst = copy_dst;
  a.tokens = copy_tokens;
  a.num_copies = num_copies;
  a.status = static_cast<uint32_t*>(split_scratch);
  a.page_bytes = plan->kv_stride_page * eb;
  a.token_bytes = plan->kv_stride_token * eb;
  a.head_bytes = plan->kv_stride_head * eb;
  a.copies = copies;
  a.sides = latent ? 1 : 2;
  a.page_size = plan->page_size;
  a.heads = plan->num_kv_heads;
  a.num_pages = plan->num_pages;
  const int row = plan->scale_mode == PDA_SCALE_MLA_BLOCK ? 640 : plan->head_dim * eb;
  a.row_vecs = row / 16;
  a.layout = a.head_bytes == row && a.token_bytes == static_cast<int64_t>(row) * a.heads ? 0
             : a.token_bytes == row                                                      ? 1
                                                                                         : 2;
  const int64_t vecs = static_cast<int64_t>(a.page_size) * a.heads * a.row_vecs;
  if (vecs > INT_MAX - 4 * kThreads) return PDA_ERR_INVALID;
  a.pieces = static_cast<int>((vecs * 16 + kPiece - 1) / kPiece);
  a.scale_floats = per_head * a.heads;
  const int64_t units = static_cast<int64_t>(copies) * a.sides * a.pieces;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, 8LL * plan->num_sms));
  // (behind pda_fork_tables its launch is under way while that kernel runs)
  return launch_next(copy_pages, dim3(grid), reinterpret_cast<cudaStream_t>(stream), a);
}

extern "C" int pda_pages_scratch(const pda_plan_t* plan, size_t* scratch_bytes) {
  if (!plan || !scratch_bytes) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  const int64_t words = pda::page_words(plan);
  *scratch_bytes = static_cast<size_t>(pda::kStatusHeaderBytes + 2 * ((words * 4 + 255) / 256 * 256));
  return PDA_OK;
}

extern "C" int pda_free_pages(const pda_plan_t* plan, const pda_pages* pages, void* page_scratch,
                              pda_stream_t stream) {
  return pda::list_call(plan, pages, page_scratch, stream, false);
}

extern "C" int pda_compact_pages(const pda_plan_t* plan, const pda_pages* pages, void* page_scratch,
                                 pda_stream_t stream) {
  return pda::list_call(plan, pages, page_scratch, stream, true);
}
