// pda_own.cu -- the requests' own tokens behind a shared prefix, and the join with what the
// prefix kernel left of the prefix: one kernel where the own tokens are few, else the join
// alone behind stage 1 of pda_decode.
//
// Mathematics: see pda_shared.cu; the own tokens are ordinary causal (and windowed)
// attention of R rows x the heads of a GQA group, 16 of them a CTA. out = (sum_s 2^(x_s - X)
// o_s + 2^(m - X) O) / (sum_s 2^(x_s - X) + 2^(m - X) l) over the prefix's segments s, with
// (m, l, O) the own tokens' maximum, sum and unnormalised output.
//
// Bound: latency, then HBM. Own contexts are short (a few hundred tokens), and stage 1
// takes 8.7 us for a CTA with 16 or 256 of them, two CTAs an SM: 17 us of 64 requests with 8
// kv heads. So here a warp takes 16 tokens at a time into mma.sync fragments, and a lane
// copies from the cache, two steps ahead, the very bytes of its fragments: nobody waits for
// another lane, and the registers hold O and no keys or values under way (with loads into
// registers instead: 52 us for 50 of 64 requests behind 8192 tokens). Which channel a
// lane's fragment element stands for is free, as long as Q (for S, a sum over channels)
// and O (whose columns are channels) agree, so a lane holds 16 neighbouring bytes of a
// token. Twelve warps an SM (eight or six at head_dim 256) have 100 to 200 KB under way.
// Few rows are shared by a cluster of CTAs, its tokens and then the rows of its join: one
// that joins 16 rows of 76 parts each alone takes 30 us for it, a cluster of four 9.
// Of a CTA's 20 us (64 requests, 8 heads of 128, 64 own tokens and more) its start, page
// lookups and queries are 5, the steps 8, the join of 8 rows of 11 parts 6. Copies of the
// parts through a ring in shared memory (more instructions for the same reads) took 2 us
// longer, K of the next step in registers as long as without, L2 prefetches by the
// prefix kernel as long.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pda.h"
#include "pda_cvt.cuh"
#include "pda_internal.h"
#include "pda_shared.cuh"

namespace pda {
namespace {

constexpr int kMaxWarps = 4;
constexpr int kRows = 16;          // packed rows (query row x head of the group) of a CTA
constexpr int kStep = 16;          // tokens of a warp's step
constexpr int kMaxTiles = 4;       // most row tiles of a request: each reads its tokens again
constexpr int kMaxTokens = 1024;   // most own tokens: four warps share them

constexpr int kStages = 2;         // steps of a warp in shared memory

template <int D, bool k8, bool kTok>
struct Cfg {
  static constexpr int kPieces = D * (k8 ? 1 : 2) / 64;    // 16-byte pieces of a K row a lane has
  static constexpr int kVCh = k8 && D >= 128 ? 16 : 8;     // channels of a lane's piece of a V row
  static constexpr int kSets = D / (8 * kVCh);             // such pieces
  static constexpr int kStride = D + 4;                    // floats of a row of O in shared memory
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kVBytes = kVCh * (k8 ? 1 : 2);      // of a piece of a V row
  // a step's bytes of a warp: K, V, and the scales of four tokens a lane
  static constexpr int kKStage = 32 * 2 * kPieces * 16, kVStage = 32 * kSets * 4 * kVBytes;
  static constexpr int kStage = kKStage + kVStage + (kTok ? 32 * 8 * 4 : 0);
  // a warp's stages, and O in their place behind its last step
  static constexpr int kOBytes = kRows * kStride * 4;
  static constexpr int kRegion = kStages * kStage > kOBytes ? kStages * kStage : kOBytes;
  static constexpr int smem(int warps) { return kQBytes + warps * (kRegion + kRows * 8) + kRows * 4; }
  static constexpr int kWarpsSm = D < 256 ? 12 : k8 ? 8 : 6;  // by their registers or stages
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a b, 16 x 8 x 16.
template <bool kF16>
__device__ __forceinline__ void mma16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A variable's address in CTA `rank` of the cluster, and loads there.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float2 load2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t y, bool high) {
  return __byte_perm(x, y, high ? 0x7632 : 0x5410);
}

// Copies to shared memory, nothing read and zeros written where !ok; the end of a group of
// them; a wait until one group is under way at most.
template <int kBytes>
__device__ __forceinline__ void copy_to(const void* dst, const void* src, bool ok) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(ok ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(src), "n"(kBytes), "r"(ok ? kBytes : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kUnderWay>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kUnderWay) : "memory");
}

template <int D, bool k8, bool kI8, bool kTok>
__global__ void __launch_bounds__(32 * kMaxWarps, D == 256 ? 2 : 3) own_join(const __grid_constant__ SharedArgs a,
                                                     const __grid_constant__ DecodeArgs o) {
  using C = Cfg<D, k8, kTok>;
  constexpr int kG = D <= 128 ? 2 : 1;
  constexpr int eb = k8 ? 1 : 2;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* q_s = smem;  // [16][D] in 16 bits, a row's 16-byte pieces XORed with its low bits
  const int warps = blockDim.x >> 5;
  float* o_s = reinterpret_cast<float*>(smem + C::kQBytes);  // [warp][16][kStride], kRegion bytes apart
  constexpr int kApart = C::kRegion / 4;
  float2* ml_s = reinterpret_cast<float2*>(smem + C::kQBytes + warps * C::kRegion);  // [warp][16]
  float* up_s = reinterpret_cast<float*>(ml_s + warps * kRows);  // a row's power of two
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  uint32_t ctas;  // of the cluster
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int rank = blockIdx.x % ctas, item = blockIdx.x / ctas;
  const int b = item / a.hkv, h = item % a.hkv;
  const int q0 = __ldg(a.qo_indptr + b), R = __ldg(a.qo_indptr + b + 1) - q0;
  const int L = __ldg(a.own_len + b), own = __ldg(a.own_indptr + b);
  const int W = a.window ? __ldg(a.window + b) : 0;
  const int m0 = blockIdx.y * kRows, M = R * a.group;
  // (own_len and own_indptr of a request of no group are not pda_share_tables')
  const int group = group_of_request(a.group_indptr, a.groups, a.batch, b);
  if (group < 0 || R <= 0 || R > o.max_q_len || L < R || L > o.max_kv_len || q0 < 0 || q0 + R > a.rows_cap ||
      m0 >= M) {
    if (tid == 0 && h == 0 && blockIdx.y == 0 && rank == 0) {
      uint32_t bits = 0u;
      if (R < 0 || R > o.max_q_len) bits = PDA_STATUS_ROWS_GT_MAX;
      else if (R > 0 && group < 0) bits = PDA_STATUS_TABLE_INVALID;
      else if (R > 0 && L < R) bits = PDA_STATUS_KV_LEN_LT_ROWS;
      else if (R > 0 && L > o.max_kv_len) bits = PDA_STATUS_KV_LEN_GT_MAX;
      else if (R > 0 && q0 + R > a.rows_cap) bits = PDA_STATUS_ROWS_GT_CAP;
      // (share_tables has said what is wrong where it left a request out)
      if (bits && (L != -1 || group < 0)) atomicOr(a.status, bits);
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }

  // ---- a warp's steps of 16 tokens, kStages - 1 of them under way in front of the one at
  // work; a lane copies what it uses itself, so nothing has to wait for other lanes
  const int low = W > 0 ? max(0, L - R - min(W, L) + 1) : 0;  // the first token that a row sees
  const int from = low / kStep;
  const int steps = (L + kStep - 1) / kStep;
  const int P = a.page_size, shift = 31 - __clz(P);
  const int32_t* pages = a.page_table + own;
  const uint8_t* k_base = static_cast<const uint8_t*>(o.k) + static_cast<int64_t>(h) * o.sh * eb;
  const uint8_t* v_base = static_cast<const uint8_t*>(o.v) + static_cast<int64_t>(h) * o.sh * eb;
  const int n_pages = (L + P - 1) >> shift;
  // the pages of a step's first and last eight tokens
  auto page_at = [&](int t) { return t >> shift < n_pages ? __ldg(pages + (t >> shift)) : -1; };
  const int stride = ctas * warps;
  int s = from + rank * warps + warp, next = s, stage = 0;  // the step at work, the one to copy
  int pg[2] = {page_at(s * kStep), page_at(s * kStep + 8)};  // the pages of `next`
  bool oob = false;
  uint8_t* slots = smem + C::kQBytes + warp * C::kRegion;
  auto copy_step = [&](int to) {
    uint8_t* k_to = slots + to * C::kStage + lane * 16;
    uint8_t* v_to = slots + to * C::kStage + C::kKStage + lane * C::kVBytes;
    float* f_to = reinterpret_cast<float*>(slots + to * C::kStage + C::kKStage + C::kVStage) + lane;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = next * kStep + 8 * e, page = pg[e];
      const bool ok = page >= 0 && page < a.num_pages;
      oob |= !ok && t < L;
      const int64_t at = ok ? (page * o.sp + (t & (P - 1)) * o.st) * eb : 0;
      pg[e] = page_at(t + stride * kStep);
      // K: token g of the half, 16-byte pieces q, q + 4, ... of its row
      const bool k_ok = ok && t + g < L && t + g >= low;
      const uint8_t* k_at = k_base + at + (k_ok ? g * o.st * eb : 0) + q * 16;
#pragma unroll
      for (int i = 0; i < C::kPieces; ++i) copy_to<16>(k_to + (e * C::kPieces + i) * 512, k_at + i * 64, k_ok);
      // V: tokens 2q and 2q + 1 of the half, the g-th piece of each set of channels
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 2 * q + c;
        const bool v_ok = ok && t + row < L && t + row >= low;
        const uint8_t* v_at = v_base + at + (v_ok ? row * o.st * eb : 0) + g * C::kVBytes;
#pragma unroll
        for (int set = 0; set < C::kSets; ++set)
          copy_to<C::kVBytes>(v_to + (set * 4 + 2 * e + c) * (32 * C::kVBytes), v_at + set * 8 * C::kVBytes, v_ok);
        if constexpr (kTok) {
          const int64_t x = v_ok ? (static_cast<int64_t>(page) * P + ((t + row) & (P - 1))) * a.hkv + h : 0;
          copy_to<4>(f_to + (4 * e + 2 * c) * 32, a.k_scale + x, v_ok);
          copy_to<4>(f_to + (4 * e + 2 * c + 1) * 32, a.v_scale + x, v_ok);
        }
      }
    }
    copies_end();
    next += stride;
  };
#pragma unroll 1
  for (int k = 0; k < kStages; ++k) copy_step(k);

  // ---- the queries: eight lanes a row, 16 bits a channel
#pragma unroll 1
  for (int r = tid >> 3; r < kRows; r += blockDim.x >> 3) {
    const int m = m0 + r;
    const bool live = m < M;
    const int64_t at = ((static_cast<int64_t>(q0) + (live ? m / a.group : 0)) * a.hq + h * a.group +
                        (live ? m % a.group : 0)) * D;
    constexpr int kEach = D / 64;  // 16-byte pieces a lane writes
    const int p0 = tid & 7;
    uint4 v[kEach];
    float up = 1.f;
    if (k8 && a.q8) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        uint2 c = make_uint2(0, 0);
        if (live)
          c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.q) + at) + p0 + 8 * k);
        widen4(c.x, v[k].x, v[k].y, false);
        widen4(c.y, v[k].z, v[k].w, false);
      }
    } else {
      uint32_t top = 0u;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        v[k] = make_uint4(0, 0, 0, 0);
        if (live)
          v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at) + p0 + 8 * k);
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] << 16 & 0x7FFF0000u, w[e] & 0x7FFF0000u));
      }
      if constexpr (k8) {
        // f16 operands: a row whose largest element is not in [2^-6, 2^12) without its
        // power of two
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        int ex = static_cast<int>(top >> 23) - 127;
        if (top == 0u || ex == 128 || (ex >= -6 && ex < 12)) ex = 0;
        ex = max(-126, min(126, ex));
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
          uint32_t* w = &v[k].x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = f16x2(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xFFFF0000u) * down);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      *reinterpret_cast<uint4*>(q_s + r * (D * 2) + (((p0 + 8 * k) ^ (r & 7)) << 4)) = v[k];
    if (p0 == 0) up_s[r] = up;
  }
  __syncthreads();

  // ---- a warp's steps of 16 tokens
  float logit = a.sm_scale * kLog2e, v_final = 1.f;
  if (k8 && !kTok) {
    logit *= __ldg(a.k_scale);
    v_final = __ldg(a.v_scale);
  }
  // rows g and g + 8 of the tile: what they see
  int last[2], lo[2];
  float scale[2], m_[2] = {kMInit, kMInit}, l_[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int m = m0 + g + 8 * k;
    last[k] = m < M ? L - R + m / a.group : -1;
    lo[k] = W > 0 ? last[k] - min(W, L) + 1 : 0;  // (L of L tokens is all of them)
    scale[k] = logit * up_s[g + 8 * k];
  }
  float acc[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll 1
  for (; s < steps; s += stride) {
    const int t0 = s * kStep;
    copies_wait<kStages - 1>();
    const uint8_t* mine = slots + stage * C::kStage;
    float ks[2][2], vs[2][2];  // of tokens 2q, 2q + 1 of each half
    if constexpr (kTok) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float* f = reinterpret_cast<const float*>(mine + C::kKStage + C::kVStage) + (4 * e + 2 * c) * 32 + lane;
          ks[e][c] = f[0];
          vs[e][c] = f[32] > 0.f ? f[32] : 1.f;
        }
    }
    // S of 16 rows x 2 x 8 tokens
    float sc[2][4] = {};
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
      uint4 kv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        kv[e] = *reinterpret_cast<const uint4*>(mine + (e * C::kPieces + i) * 512 + lane * 16);
      if constexpr (k8) {
        uint32_t qa[8], qb[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int piece = (2 * (q + 4 * i) + c) ^ g;
          const uint4 x = *reinterpret_cast<const uint4*>(q_s + g * (D * 2) + piece * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(q_s + (g + 8) * (D * 2) + piece * 16);
          qa[4 * c] = x.x, qa[4 * c + 1] = x.y, qa[4 * c + 2] = x.z, qa[4 * c + 3] = x.w;
          qb[4 * c] = y.x, qb[4 * c + 1] = y.y, qb[4 * c + 2] = y.z, qb[4 * c + 3] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w[4] = {kv[e].x, kv[e].y, kv[e].z, kv[e].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x, y;
            widen4(w[c], x, y, kI8);
            mma16<true>(sc[e], qa[2 * c], qb[2 * c], qa[2 * c + 1], qb[2 * c + 1], x, y);
          }
        }
      } else {
        const int piece = (q + 4 * i) ^ g;
        const uint4 x = *reinterpret_cast<const uint4*>(q_s + g * (D * 2) + piece * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(q_s + (g + 8) * (D * 2) + piece * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma16<false>(sc[e], x.x, y.x, x.y, y.y, kv[e].x, kv[e].y);
          mma16<false>(sc[e], x.z, y.z, x.w, y.w, kv[e].z, kv[e].w);
        }
      }
    }
    // logits in log2 units, the rows' maxima, weights
    uint32_t p[2][2];  // [half][row g, g + 8], two tokens each
    float f[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float& x = sc[e][2 * k + c];
          const int t = t0 + 8 * e + 2 * q + c;
          x *= scale[k];
          if constexpr (kTok) x = fmaf(x, ks[e][c], __log2f(vs[e][c]));
          if (t > last[k] || t < lo[k]) x = -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float to = fmaxf(m_[k], mx);
      f[k] = ex2(m_[k] - to);
      m_[k] = to;
      l_[k] *= f[k];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float w0 = ex2(sc[e][2 * k] - to), w1 = ex2(sc[e][2 * k + 1] - to);
        if constexpr (kTok) l_[k] += w0 / vs[e][0] + w1 / vs[e][1];
        else l_[k] += w0 + w1;
        p[e][k] = k8 ? f16x2(w0, w1) : bf16x2(w0, w1);
      }
    }
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        acc[n][0] *= f[0];
        acc[n][1] *= f[0];
        acc[n][2] *= f[1];
        acc[n][3] *= f[1];
      }
    }
    // O: column g of n-tile `set kVCh + j` is channel (set 8 + g) kVCh + j
#pragma unroll
    for (int set = 0; set < C::kSets; ++set) {
      constexpr int kVWords = C::kVBytes / 4;
      uint32_t vv[4][kVWords];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t* src = mine + C::kKStage + (set * 4 + e) * (32 * C::kVBytes) + lane * C::kVBytes;
        if constexpr (kVWords == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          vv[e][0] = x.x, vv[e][1] = x.y, vv[e][2] = x.z, vv[e][3] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          vv[e][0] = x.x, vv[e][1] = x.y;
        }
      }
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        uint32_t x[4][2];  // the word's channels in pairs, of each token
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (k8) {
            widen4(vv[e][w], x[e][0], x[e][1], kI8);
          } else {
            x[e][0] = vv[e][w];
          }
        }
#pragma unroll
        for (int c = 0; c < (k8 ? 2 : 1); ++c)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const int j = w * (k8 ? 4 : 2) + c * 2 + hi;
            mma16<k8>(acc[set * C::kVCh + j], p[0][0], p[0][1], p[1][0], p[1][1], pick(x[0][c], x[1][c], hi),
                      pick(x[2][c], x[3][c], hi));
          }
      }
    }
    __syncwarp();
    copy_step(stage);  // (what it held has been used)
    stage ^= 1;
  }
  copies_wait<0>();
  if (oob) atomicOr(a.status, PDA_STATUS_PAGE_OOB);
  // ---- the warps' parts to shared memory
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    l_[k] += __shfl_xor_sync(0xffffffffu, l_[k], 1);
    l_[k] += __shfl_xor_sync(0xffffffffu, l_[k], 2);
    if (q == 0) ml_s[warp * kRows + g + 8 * k] = make_float2(m_[k], l_[k]);
    float* row = o_s + warp * kApart + (g + 8 * k) * C::kStride;
#pragma unroll
    for (int set = 0; set < C::kSets; ++set)
#pragma unroll
      for (int j = 0; j < C::kVCh; ++j) {
        // columns 2q and 2q + 1
        row[(set * 8 + 2 * q) * C::kVCh + j] = acc[set * C::kVCh + j][2 * k];
        row[(set * 8 + 2 * q + 1) * C::kVCh + j] = acc[set * C::kVCh + j][2 * k + 1];
      }
  }
  // ---- the rows, half a warp each, or a warp where there are warps for it (its halves then
  // take the prefix's parts in turns): the cluster's own parts, then the prefix's
  using J = Join<D, 16>;
  constexpr int kV = J::kV, kBatch = D == 256 ? 80 : 48;
  // `count` parts from other places in shared memory, their loads in front of their use (a
  // load from another CTA takes 200 ns and more)
  // (part c: the first warp's of CTA c, or warp c's of this CTA)
  auto gather = [&](J& join, int count, bool apart, int r, float times) {
    auto at_ml = [&](int c) { return in_cta(ml_s + (apart ? 0 : c * kRows) + r, apart ? c : rank); };
    auto at_o = [&](int c) { return in_cta(o_s + (apart ? 0 : c * kApart) + r * C::kStride, apart ? c : rank); };
    float2 ml[4];
    float v[4][kV];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      ml[c] = make_float2(-INFINITY, 0.f);
      if (c >= count) continue;
      ml[c] = load2(at_ml(c));
      const uint32_t src = at_o(c) + J::first() * 4;
#pragma unroll
      for (int e = 0; e < kV; e += 4) {
        const float4 x = load4(src + e * 4);
        v[c][e] = x.x;
        v[c][e + 1] = x.y;
        v[c][e + 2] = x.z;
        v[c][e + 3] = x.w;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) join.raise(ml[c].x);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c >= count) continue;
      const float f = exp2f(ml[c].x - join.top);
      join.sum = fmaf(f, ml[c].y, join.sum);
#pragma unroll
      for (int e = 0; e < kV; ++e) join.acc[e] = fmaf(f, v[c][e] * times, join.acc[e]);
    }
  };
  Parts<kG> parts(a, group);
  const uint32_t bad = parts.bad(q0, R);
  if (bad && tid == 0 && h == 0 && m0 == 0 && rank == 0) atomicOr(a.status, bad);
  const int live = bad ? 0 : min(kRows, M - m0), hw = lane >> 4;
  __syncthreads();
  if (ctas > 1) {  // one part a CTA, in the first warp's place
#pragma unroll 1
    for (int r = 2 * warp + hw; r < live; r += 2 * warps) {
      J join;
      gather(join, warps, false, r, 1.f);
#pragma unroll
      for (int e = 0; e < kV; ++e) o_s[r * C::kStride + J::first() + e] = join.acc[e];
      // (every lane of the half has read the first warp's maximum: their loads are used)
      __syncwarp(0xffffu << (16 * hw));
      if (J::first() == 0) ml_s[r] = make_float2(join.top, join.sum);
    }
    __syncwarp();
    cluster_sync();
  }
  const int packed = (q0 - parts.gr.q0) * a.group + m0;  // the first row, in the group
  RowParts<kG, D> row(a, parts, h, packed);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the prefix's parts are there
  const bool late = a.groups > 32;
  parts.late(a);
  const int block_end = late ? 0 : kG * kTile - row.r;  // rows behind it (or all) need places of their own
  const bool turns = stride >= live;
  const int r0 = turns ? rank * warps + warp : 2 * (rank * warps + warp) + hw;
#pragma unroll 1
  for (int r = r0; r < live; r += turns ? stride : 2 * stride) {
    J join;
    if (!turns || hw == 0) {
      gather(join, ctas > 1 ? ctas : warps, ctas > 1, r, v_final);
    }
    if (r >= block_end) row = RowParts<kG, D>(a, parts, h, packed + r);
    const int off = r >= block_end ? 0 : r, step = turns ? 2 : 1, at = turns ? hw : 0;
    join.template add<kBatch / kV>((row.segs - at + step - 1) >> (step - 1), [&](int k, const float*& x, const float*& v) {
      row.part(a, k * step + at, x, v);
      x += off;
      v += off * D;
    });
    if (turns) {
      __syncwarp();
      const float top = __shfl_xor_sync(0xffffffffu, join.top, 16), sum = __shfl_xor_sync(0xffffffffu, join.sum, 16);
      const float mine = join.top, to = fmaxf(mine, top);
      const float f0 = mine == -INFINITY ? 0.f : exp2f(mine - to), f1 = top == -INFINITY ? 0.f : exp2f(top - to);
      join.top = to;
      join.sum = join.sum * f0 + sum * f1;
#pragma unroll
      for (int e = 0; e < kV; ++e)
        join.acc[e] = join.acc[e] * f0 + __shfl_xor_sync(0xffffffffu, join.acc[e], 16) * f1;
      if (hw) continue;
    }
    const int i = (m0 + r) / a.group;
    join.write(o, (static_cast<int64_t>(q0) + i) * a.hq + h * a.group + m0 + r - i * a.group);
  }
  __syncwarp();
  if (ctas > 1) cluster_sync();  // the others have read this CTA's parts
}

// ------------------------------------------------------------- the join alone
//
// One warp per (request, row, head): the prefix's segments in order, then stage 1's
// chunks. Bound: reading the parts (L2); where they are is worked out while the kernels
// in front end.
template <int D>
__global__ void __launch_bounds__(256, 3) shared_join(const __grid_constant__ SharedArgs a,
                                                      const __grid_constant__ DecodeArgs o) {
  constexpr int kG = D <= 128 ? 2 : 1;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t per_b = static_cast<int64_t>(o.max_q_len) * a.hq;
  const int b = static_cast<int>(item / per_b);
  const int i = static_cast<int>(item % per_b) / a.hq, head = static_cast<int>(item % a.hq), h = head / a.group;
  bool live = b < a.batch;
  int q0 = 0, R = 0, own = 0;
  if (live) {
    q0 = __ldg(a.qo_indptr + b);
    R = __ldg(a.qo_indptr + b + 1) - q0;
    const int L = __ldg(a.own_len + b), W = a.window ? __ldg(a.window + b) : 0;
    live = i < R && R <= o.max_q_len && L >= R && L <= o.max_kv_len && q0 >= 0 && q0 + R <= a.rows_cap;
    if (live) own = split_range(L, R, W, a.page_size, chunk_for(o, b)).num_splits;
  }
  const int group = live ? group_of_request(a.group_indptr, a.groups, a.batch, b) : 0;
  Parts<kG> parts(a, max(group, 0));
  const uint32_t bad = group < 0 ? PDA_STATUS_TABLE_INVALID : parts.bad(q0, R);
  if (live && bad) {
    if ((threadIdx.x & 31) == 0) atomicOr(a.status, bad);
    live = false;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  parts.late(a);
  const RowParts<kG, D> row(a, parts, h, (q0 + i - parts.gr.q0) * a.group + head % a.group);
  const int64_t own_row = static_cast<int64_t>(q0 + i) * a.hq + head, own_step = o.rows_cap * a.hq;
  Join<D, 32> join;
  join.template add<(D <= 128 ? 8 : 4)>(row.segs + own, [&](int s, const float*& x, const float*& v) {
    if (s < row.segs) return row.part(a, s, x, v);
    const int64_t at = (s - row.segs) * own_step + own_row;
    x = o.part_lse + at;
    v = o.part_o + at * D;
  });
  join.write(o, own_row);
}

using JoinFn = void (*)(SharedArgs, DecodeArgs);
struct Kernel {
  JoinFn fn;
  int (*smem)(int warps);
  int warps_sm;
};
template <int D>
Kernel kernel_for(const pda_plan_t* p) {
  using C16 = Cfg<D, false, false>;
  using C8 = Cfg<D, true, false>;
  using C8T = Cfg<D, true, true>;
  const bool tok = p->scale_mode == PDA_SCALE_TOKEN_HEAD;
  if (p->kv_dtype == PDA_BF16) return {own_join<D, false, false, false>, C16::smem, C16::kWarpsSm};
  if (p->kv_dtype == PDA_INT8)
    return tok ? Kernel{own_join<D, true, true, true>, C8T::smem, C8T::kWarpsSm}
               : Kernel{own_join<D, true, true, false>, C8::smem, C8::kWarpsSm};
  return tok ? Kernel{own_join<D, true, false, true>, C8T::smem, C8T::kWarpsSm}
             : Kernel{own_join<D, true, false, false>, C8::smem, C8::kWarpsSm};
}

int launch(JoinFn fn, dim3 grid, unsigned threads, int smem, unsigned cluster, const SharedArgs& a,
           const DecodeArgs& o, cudaStream_t s) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, fn, a, o) == cudaSuccess) return PDA_OK;
  cudaGetLastError();
  return PDA_ERR_CUDA;
}

}  // namespace

bool own_here(const pda_plan_t* own) {
  return own->max_q_len * own->group <= kMaxTiles * kRows && own->max_kv_len <= kMaxTokens;
}

int launch_own(const pda_plan_t* own, const SharedArgs& a, const DecodeArgs& o, cudaStream_t s) {
  const Kernel k = own->head_dim == 64    ? kernel_for<64>(own)
                   : own->head_dim == 128 ? kernel_for<128>(own)
                                          : kernel_for<256>(own);
  const int tiles = (o.max_q_len * a.group + kRows - 1) / kRows;
  const int64_t items = static_cast<int64_t>(a.batch) * a.hkv * tiles;
  // Few items: clusters of up to four CTAs, while all of them have an SM. Many: as few
  // warps a CTA as end sooner, where four would leave a last wave of few CTAs (a step of
  // 16 tokens takes about 2 us with all SMs at it, a CTA's start and join 6, both from 64
  // requests with 8 kv heads of 128; half of the most tokens taken for all).
  int cluster = 1, warps = kMaxWarps;
  while (cluster < 4 && items * cluster * 2 <= own->num_sms) cluster *= 2;
  if (cluster == 1) {
    const int steps = std::max(1, own->max_kv_len / (2 * kStep));
    double best = 1e30;
    for (int w = kMaxWarps; w >= 1; --w) {
      const int64_t slots = static_cast<int64_t>(std::min(k.warps_sm / w, 227 * 1024 / (k.smem(w) + 1024))) * own->num_sms;
      const double us = static_cast<double>((items + slots - 1) / slots) * ((steps + w - 1) / w * 2.0 + 6.0);
      if (us < best) best = us, warps = w;
    }
  }
  const dim3 grid(static_cast<unsigned>(a.batch * a.hkv * cluster), static_cast<unsigned>(tiles));
  return launch(k.fn, grid, 32u * warps, k.smem(warps), static_cast<unsigned>(cluster), a, o, s);
}

int launch_join(const pda_plan_t* own, const SharedArgs& a, const DecodeArgs& o, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.batch) * o.max_q_len * a.hq;
  const JoinFn fn = own->head_dim == 64 ? shared_join<64> : own->head_dim == 128 ? shared_join<128> : shared_join<256>;
  return launch(fn, dim3(static_cast<unsigned>((warps + 7) / 8)), 256, 0, 1, a, o, s);
}

}  // namespace pda
