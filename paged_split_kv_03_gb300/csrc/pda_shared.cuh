// pda_shared.cuh -- what the kernels of decode behind shared prefixes have in common: their
// arguments, the groups and how the work on their prefixes is cut, and the join of a row's
// parts. Internal to each translation unit but for the arguments and launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "pda.h"
#include "pda_cvt.cuh"
#include "pda_internal.h"

namespace pda {

struct SharedArgs {
  const void* q;
  const int32_t* page_table;
  const int32_t* qo_indptr;
  const int32_t* kv_len;
  const int32_t* window;
  const int32_t* group_indptr;  // NULL: one group of all requests
  const int32_t* prefix;        // [groups][2] tokens
  const int32_t* own_indptr;
  const int32_t* own_len;
  const float* k_scale;
  const float* v_scale;
  float* main_o;    // [kv head][row x group][D] fp32: segments that start their item
  float* main_x;    // ... and their log2 sums
  float* area_o;    // [CTA][rows of an item][D]: the segment a CTA starts inside an item
  float* area_x;
  int* first;       // the cut (per, pay, one), then [groups] where each group's work starts
  uint32_t* status;
  uint64_t wait_limit_ns;
  float sm_scale;
  int batch, groups, hq, hkv, group, page_size, num_pages, max_q_len, max_kv_len;
  int64_t rows_cap;
  int q8;
  int ctas;  // of the prefix kernel
  int one;   // what a tile of a block of at most 128 rows counts
  uint32_t inject;
};

// Whether the requests' own tokens and the join are one kernel (else stage 1, then the
// join). Both start beside the kernel in front of them and end behind the prefix kernel.
bool own_here(const pda_plan_t* own);
int launch_own(const pda_plan_t* own, const SharedArgs& a, const DecodeArgs& o, cudaStream_t s);
int launch_join(const pda_plan_t* own, const SharedArgs& a, const DecodeArgs& o, cudaStream_t s);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMInit = -3.0e38f;  // before any key: finite, so that ex2(-inf - m) = 0
constexpr int kKeys = 128;          // keys of a prefix tile
constexpr int kTile = 128;          // packed rows of a row tile

// A group's rows and its prefix's key tiles.
struct Group {
  int b0, b1, q0, rows, tile0, tiles, low, end;  // tokens [low, end), from tile0's first on
  uint32_t bad;
};
__device__ __forceinline__ Group group_of(const SharedArgs& a, int g) {
  Group r;
  r.b0 = a.group_indptr ? __ldg(a.group_indptr + g) : 0;
  r.b1 = a.group_indptr ? __ldg(a.group_indptr + g + 1) : a.batch;
  r.bad = r.b0 < 0 || r.b1 < r.b0 || r.b1 > a.batch ? PDA_STATUS_TABLE_INVALID : 0u;
  r.q0 = r.rows = r.tile0 = r.tiles = r.low = r.end = 0;
  if (r.bad) return r;
  r.q0 = __ldg(a.qo_indptr + r.b0);
  const int64_t rows = static_cast<int64_t>(__ldg(a.qo_indptr + r.b1)) - r.q0;
  if (r.q0 < 0 || rows < 0 || r.q0 + rows > a.rows_cap) {
    r.bad = PDA_STATUS_ROWS_GT_CAP;
    return r;
  }
  r.rows = static_cast<int>(rows);
  r.low = max(0, __ldg(a.prefix + 2 * g));
  r.end = __ldg(a.prefix + 2 * g + 1);
  if (r.end > a.max_kv_len) r.bad = PDA_STATUS_TABLE_INVALID;  // (not pda_share_tables')
  if (r.bad || r.rows == 0 || r.end <= r.low) return r;
  r.tile0 = r.low / kKeys;
  r.tiles = (r.end - 1) / kKeys + 1 - r.tile0;
  return r;
}

// A group a lane: bad where a bound in front (of a lane in front, or `top`) is above its first
// request, so that no two valid groups list the same one. The highest bound so far to `top`.
__device__ __forceinline__ void no_overlap(Group& r, bool live, int& top) {
  const int lo = live ? r.b0 : INT_MIN;
  if (__any_sync(0xffffffffu, live && (lo < top || r.b1 < lo))) {  // (bounds that never fall: nothing to do)
    int x = lo;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if ((threadIdx.x & 31) >= d) x = max(x, y);
    }
    x = __shfl_up_sync(0xffffffffu, x, 1);
    if (live && lo < ((threadIdx.x & 31) ? max(x, top) : top)) {
      r.bad |= PDA_STATUS_TABLE_INVALID;
      r.rows = r.tiles = 0;
    }
  }
  top = max(top, __reduce_max_sync(0xffffffffu, lo));
}

// How the work is cut. An item is a block of kRows packed rows of a kv head, over the
// prefix's key tiles; group by group, then kv heads, then blocks, the items stand on one
// axis, and CTA c has the stretch [c per, (c + 1) per) of it: the tiles that begin there.
// Where the CTAs have less than two tiles each, a tile counts kFull. Else it counts `one`
// in a last block of one row tile, whose time is that of its loads, and an item is
// longer by `pay` in front of its tiles: a CTA's further segment costs it a query load
// and an epilogue, about three tiles' time (64 requests behind 8192 tokens, 64 / 8 heads
// of 128: CTAs of two segments ended at 34 us, the others at 23). The plan keeps the axis
// below 2^31.
constexpr int kFull = 8, kPay = 3 * kFull;
struct Cut {
  int per = 1, pay = 0, one = kFull;
  __device__ __forceinline__ Cut() {}
  // from the work at kFull a tile, the tiles of single row tiles, and the items
  __device__ __forceinline__ Cut(const SharedArgs& a, int work, int singles, int items) {
    if (work > a.ctas * (2 * kFull - 1)) {
      pay = kPay;
      one = a.one;
    }
    const uint32_t all = work - singles * (kFull - one) + pay * items;
    per = max(kFull, static_cast<int>((all + a.ctas - 1) / static_cast<uint32_t>(a.ctas)));
  }
};
template <int kG>
struct Work {
  int blocks = 0, tiles = 0;
  bool single = false;  // the last block has one row tile, of two
  __device__ __forceinline__ Work() {}
  __device__ __forceinline__ Work(const SharedArgs& a, const Group& r) {
    const int packed = r.rows * a.group;
    tiles = r.tiles;
    if (tiles == 0) return;
    blocks = (packed + kG * kTile - 1) / (kG * kTile);
    single = kG == 2 && packed - (blocks - 1) * (kG * kTile) <= kTile;
  }
  __device__ __forceinline__ int full(const Cut& c) const { return kFull * tiles + c.pay; }
  // of a tile of block b
  __device__ __forceinline__ int weight(const Cut& c, int b) const { return single && b == blocks - 1 ? c.one : kFull; }
  // of a kv head
  __device__ __forceinline__ int head(const Cut& c) const {
    return blocks ? (blocks - 1) * full(c) + weight(c, blocks - 1) * tiles + c.pay : 0;
  }
};
__device__ __forceinline__ int scan32(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Where a row's parts of its group's prefix are.
template <int kG>
struct Parts {
  Group gr;
  Cut cut;
  int g, first = 0;
  // Of group `of` (group_of_request's); a whole warp. What the prefix kernel wrote down (more groups
  // than lanes) is read by `late`, behind that kernel.
  __device__ __forceinline__ Parts(const SharedArgs& a, int of) : g(of) {
    const int lane = threadIdx.x & 31;
    gr = group_of(a, g);
    if (a.groups > 32) return;
    Work<kG> w;
    if (a.groups == 1) {
      if (lane == 0) w = Work<kG>(a, gr);
    } else {
      Group mine = {};
      if (lane < a.groups) mine = group_of(a, lane);
      int top = INT_MIN;
      no_overlap(mine, lane < a.groups, top);
      w = Work<kG>(a, mine);
    }
    const int mine = a.hkv * w.head(Cut()), singles = w.single ? a.hkv * w.tiles : 0, items = a.hkv * w.blocks;
    int upto = mine, upto_s = singles, upto_i = items;
    if (a.groups > 1) {
      upto = scan32(mine, lane);
      upto_s = scan32(singles, lane);
      upto_i = scan32(items, lane);
    }
    const int last = a.groups > 1 ? 31 : 0;
    cut = Cut(a, __shfl_sync(0xffffffffu, upto, last), __shfl_sync(0xffffffffu, upto_s, last),
              __shfl_sync(0xffffffffu, upto_i, last));
    const int before = upto - mine - (upto_s - singles) * (kFull - cut.one) + (upto_i - items) * cut.pay;
    first = __shfl_sync(0xffffffffu, before, g);
  }
  // What keeps its request of rows [q0, q0 + R) from being decoded: rows that the prefix kernel
  // has not seen (a request of fewer than none among the group's) would be without the prefix.
  __device__ __forceinline__ uint32_t bad(int q0, int R) const {
    if (gr.bad) return PDA_STATUS_TABLE_INVALID;
    return gr.tiles && (q0 < gr.q0 || q0 + R > gr.q0 + gr.rows) ? PDA_STATUS_ROWS_GT_MAX : 0u;
  }
  __device__ __forceinline__ void late(const SharedArgs& a) {
    if (a.groups <= 32) return;
    cut.per = a.first[0];
    cut.pay = a.first[1];
    cut.one = a.first[2];
    first = a.first[3 + g];
  }
};
// ... of packed row m and kv head h: how many, and each one's log2 sum and output.
template <int kG, int D>
struct RowParts {
  int segs = 0, c0 = 0, r = 0;
  int64_t head_row = 0;
  __device__ __forceinline__ RowParts() {}
  __device__ __forceinline__ RowParts(const SharedArgs& a, const Parts<kG>& p, int h, int m) {
    constexpr int kRows = kG * kTile;
    const int block = m / kRows;
    r = m % kRows;
    head_row = (h * a.rows_cap + p.gr.q0) * a.group + m;
    if (p.gr.tiles == 0 || m < 0 || m >= p.gr.rows * a.group) return;
    const Work<kG> w(a, p.gr);
    // its first and its last tile
    const uint32_t u = p.first + h * w.head(p.cut) + block * w.full(p.cut) + p.cut.pay;
    const uint32_t per = p.cut.per;
    c0 = u / per;
    segs = (u + (p.gr.tiles - 1) * w.weight(p.cut, block)) / per - c0 + 1;
  }
  __device__ __forceinline__ void part(const SharedArgs& a, int s, const float*& x, const float*& v) const {
    const int64_t at = s == 0 ? head_row : static_cast<int64_t>(c0 + s) * (kG * kTile) + r;
    x = (s == 0 ? a.main_x : a.area_x) + at;
    v = (s == 0 ? a.main_o : a.area_o) + at * D;
  }
};

// The running sum of a row's parts, in kLanes neighbouring lanes.
template <int D, int kLanes>
struct Join {
  static constexpr int kV = D / kLanes;  // channels of a lane
  float top = -INFINITY, sum = 0.f, acc[kV];
  __device__ __forceinline__ Join() {
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.f;
  }
  static __device__ __forceinline__ int first() { return threadIdx.x % kLanes * kV; }
  __device__ __forceinline__ void raise(float to) {
    if (!(to > top)) return;
    const float f = exp2f(top - to);  // -inf: nothing summed yet
    sum *= f;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] *= f;
    top = to;
  }
  // kBatch parts at most at a time, their loads in front of their use
  template <int kBatch, class Place>
  __device__ __forceinline__ void add(int parts, Place&& place) {
#pragma unroll 1
    for (int s0 = 0; s0 < parts; s0 += kBatch) {
      float x[kBatch], v[kBatch][kV];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        x[k] = -INFINITY;
        if (s0 + k < parts) {
          const float *px, *pv;
          place(s0 + k, px, pv);
          x[k] = *px;
          if constexpr (kV == 2) {
            const float2 t = *reinterpret_cast<const float2*>(pv + first());
            v[k][0] = t.x;
            v[k][1] = t.y;
          } else {
#pragma unroll
            for (int e = 0; e < kV; e += 4) {
              const float4 t = *reinterpret_cast<const float4*>(pv + first() + e);
              v[k][e] = t.x;
              v[k][e + 1] = t.y;
              v[k][e + 2] = t.z;
              v[k][e + 3] = t.w;
            }
          }
        }
      }
      float to = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) to = fmaxf(to, x[k]);
      raise(to);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (s0 + k >= parts) break;
        const float w = x[k] == -INFINITY ? 0.f : exp2f(x[k] - top);
        sum += w;
        // a part without a visible key counts for nothing, whatever it holds
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[e] = w != 0.f ? fmaf(w, v[k][e], acc[e]) : acc[e];
      }
    }
  }
  // the row's results; `row`: of out and lse
  __device__ __forceinline__ void write(const DecodeArgs& o, int64_t row) const {
    const float inv = sum > 0.f ? 1.f / sum : sum;  // (NaN stays)
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(o.out) + row * D + first();
    uint32_t w[kV / 2];
#pragma unroll
    for (int e = 0; e < kV; e += 2) w[e / 2] = bf16x2(acc[e] * inv, acc[e + 1] * inv);
    if constexpr (kV == 2) {
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    } else if constexpr (kV == 4) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int e = 0; e < kV / 2; e += 4)
        *reinterpret_cast<uint4*>(dst + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
    }
    if (first() == 0 && o.lse) o.lse[row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * kLn2;
  }
};

// Four 8-bit codes (int8, or E4M3) -> four f16, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi, bool i8) {
  if (i8) {
    // with u = x + 128, the f16 word 0x6400 | u is 1024 + u: subtract 1152
    const uint32_t u = w ^ 0x80808080u;
    uint32_t p, q;
    asm("prmt.b32 %0, %1, %2, 0x5140;" : "=r"(p) : "r"(u), "r"(0x64646464u));
    asm("prmt.b32 %0, %1, %2, 0x7362;" : "=r"(q) : "r"(u), "r"(0x64646464u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(p), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(q), "r"(0x64806480u));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
  }
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace
}  // namespace pda
