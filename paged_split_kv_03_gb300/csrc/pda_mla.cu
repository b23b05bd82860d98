// pda_mla.cu -- the products of latent attention with a head's W_UK and W_UV:
// the query absorbed and the output projected around pda_decode, and the
// cached latents gathered and expanded into keys and values for a prefill.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pda.h"
#include "pda_cvt.cuh"
#include "pda_internal.h"
#include "pda_ptx.cuh"

namespace pda {
namespace {

constexpr int kLat = 512;         // latent channels the products run over
constexpr int kRope = 64;
constexpr int kLatRow = kLat + kRope;
constexpr int kNope = 128;        // channels of a key (without rope) and of a value
constexpr int kQDim = kNope + kRope;

// ------------------------------------------------------ gather of latents
//
// One warp per token: its request by binary search in tok_indptr, its page
// slot, then the row dequantised to bf16. Chunks of 8 channels per lane. Bound:
// latency (five dependent reads); the expansion that follows writes Hq x 512
// bytes a token and its set-up overlaps this kernel.

struct GatherArgs {
  const uint8_t* pages;
  const int32_t* page_table;
  const int32_t* kv_indptr;
  const int32_t* tok_indptr;
  const float* scale;
  __nv_bfloat16* latent;
  uint32_t* status;
  int64_t sp, st;
  int batch, tokens, page_shift, num_pages, max_kv_len;
};

// MODE: 0 bf16, 1 / 2 E4M3 per tensor / per token, 5 records.
template <int MODE>
__global__ void __launch_bounds__(256) gather_latent(const __grid_constant__ GatherArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the expansion may set up
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int total = __ldg(a.tok_indptr + a.batch);
  if (t == 0 && lane == 0 && total > a.tokens) atomicOr(a.status, PDA_STATUS_TOKENS_GT_CAP);
  if (t >= min(total, a.tokens)) return;
  // the last request that starts at or before t and is not empty there
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.tok_indptr + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  const int first = __ldg(a.tok_indptr + lo);
  const int n = __ldg(a.tok_indptr + lo + 1) - first;
  const int i = t - first;
  bool ok = i >= 0 && i < n;
  if (ok && n > a.max_kv_len) {
    if (i == 0 && lane == 0) atomicOr(a.status, PDA_STATUS_KV_LEN_GT_MAX);
    ok = false;
  }
  int page = 0;
  if (ok) {
    // (a token behind its request's pages has none: the next entry is another request's)
    const int p0 = __ldg(a.kv_indptr + lo), p1 = __ldg(a.kv_indptr + lo + 1);
    page = (i >> a.page_shift) < p1 - p0 ? __ldg(a.page_table + p0 + (i >> a.page_shift)) : -1;
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, PDA_STATUS_PAGE_OOB);
      ok = false;
      page = 0;
    }
  }
  const int slot = i & ((1 << a.page_shift) - 1);
  const int64_t off = page * a.sp + slot * a.st;  // elements
  const int64_t sidx = (static_cast<int64_t>(page) << a.page_shift) + slot;
  uint4* dst = reinterpret_cast<uint4*>(a.latent + static_cast<int64_t>(t) * kLatRow);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int c = lane + 32 * k;  // chunk of 8 channels; 64.. are the rope
    if (c >= kLatRow / 8) break;
    uint4 o = make_uint4(0, 0, 0, 0);
    if (ok) {
      if (MODE == 0 || (MODE == 5 && k == 2)) {
        const uint8_t* src = MODE == 0 ? a.pages + (off + c * 8) * 2 : a.pages + off + kLat + lane * 16;
        o = __ldg(reinterpret_cast<const uint4*>(src));
      } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.pages + off + c * 8));
        const float s = MODE == 1 ? __ldg(a.scale)
                        : MODE == 2 ? __ldg(a.scale + sidx) : __ldg(a.scale + sidx * 4 + (c >> 4));
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint16_t code = static_cast<uint16_t>((e < 2 ? w.x : w.y) >> ((e & 1) * 16));
          const float2 f = e4m3x2_to_f2(code);
          // one rounding to bf16: the products' operand type (2^-9 relative)
          out[e] = bf16x2(f.x * s, f.y * s);
        }
        o = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    dst[c] = o;
  }
}

// ------------------------------------------------------- products per head
//
// C_h[t, n] = sum_k A_h[t, k] B_h[n, k], fp32 sums in TMEM, one rounding:
//   absorb   A = q_nope (K = 128), B = W_UK read the other way round: its rows
//            are the K channels, so B is MN-major, as it lies (N = 512)
//   project  A = o_lat (K = 512), B = W_UV (N = 128)
// A CTA has 128 tokens of one head and N columns. Bound: HBM (the weights at
// few rows, A and C at many: 128 x 128 x 512 MACs a row tile and head are 2048
// tensor cycles against 160 KB). Short rows cost nothing but idle MMA lanes,
// as TMA reads no row behind the last. What a CTA has in flight, and how many an
// SM holds, decides (pda_mla_project). The output tile passes through the stages'
// memory so that a warp writes whole 256-byte rows. Measured in graphs of calls: absorb
// of 1024 rows x 128 heads 49 us to bf16 (4.4 TB/s, 151 of the 218 MB written, which a
// plain fill does at 4.0 TB/s), 38 us to E4M3; project 37 us (5.0 TB/s); one row of 128
// heads 6.1 and 4.7 us.

enum { kAbsorb = 0, kProject = 1 };

struct ProductArgs {
  void* out;
  const __nv_bfloat16* q;  // absorb: the rope channels pass through
  int64_t q_row, q_head;
  const int32_t* num_rows;
  uint32_t* status;
  uint64_t wait_limit_ns;
  float inv_scale;         // absorb to E4M3: 1 / q_scale, else 0
  int rows, heads;
  uint32_t inject;         // PDA_INJECT_*, 0 in normal use
};

template <int OP, int N, int STAGES>
struct ProductCfg {
  static constexpr int kK = OP == kAbsorb ? kNope : kLat;
  static constexpr int kBlocks = kK / 64;                        // K blocks of 128 bytes
  static constexpr int kStages = STAGES;
  static constexpr int kABytes = 128 * 128, kBBytes = N * 128, kStage = kABytes + kBBytes;
  static constexpr int kSmem = kStages * kStage + 1024;          // + alignment
  static constexpr int kTotalN = OP == kAbsorb ? kLat : kNope;
  static constexpr int kTmem = N < 32 ? 32 : N;
  static_assert(kStages * kStage >= 128 * N * 2, "the output tile fits the stages");
};

template <int OP, int N, int STAGES, bool E4M3>
__global__ void __launch_bounds__(192)
    product(const __grid_constant__ ProductArgs a, const __grid_constant__ CUtensorMap ta,
            const __grid_constant__ CUtensorMap tb) {
  using C = ProductCfg<OP, N, STAGES>;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  uint8_t* smem = raw + ((1024u - (su32(raw) & 1023u)) & 1023u);
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int rows = a.rows;
  if (a.num_rows) rows = min(rows, __ldg(a.num_rows));
  const int n0 = blockIdx.x * N, h = blockIdx.y, t0 = blockIdx.z * 128;
  if (t0 >= rows) return;
  const bool withhold = (a.inject & PDA_INJECT_WITHHOLD_KV) != 0u;
  auto load = [&](int k) {
    const int s = k % C::kStages;
    uint8_t* st = smem + s * C::kStage;
    bar_expect_tx(full + s, C::kStage);
    tma_load3(su32(st), &ta, k * 64, h, t0, full + s);
    if constexpr (OP == kAbsorb) {  // 64 channels of K x N columns, 64 columns an atom
      for (int c = 0; c < N / 64; ++c)
        tma_load3(su32(st + C::kABytes + c * 8192), &tb, n0 + c * 64, k * 64, h, full + s);
    } else {
      tma_load3(su32(st + C::kABytes), &tb, k * 64, n0, h, full + s);
    }
  };
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      bar_init(full + s, 1);
      bar_init(empty + s, 1);
    }
    bar_init(&done, 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    // the first loads are on their way while TMEM is allocated
    for (int k = 0; k < C::kStages && !withhold; ++k) load(k);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&tmem_slot)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  if (warp == 0) {
    if (lane == 0 && !withhold) {
      int k = C::kStages;
      for (; k < C::kBlocks; ++k) {
        if (!bar_wait(empty + k % C::kStages, ((k / C::kStages) - 1) & 1u, abort_flag, a)) break;
        load(k);
      }
      // Every box issued must have landed before the CTA can exit. Always, not
      // only after an abort seen here: the MMA thread's wait may run out later.
      for (int i = k - C::kStages; i < k; ++i)
        bar_drain(full + i % C::kStages, (i / C::kStages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = idesc(1u, 0, N, OP == kAbsorb ? 1u : 0u);
      bool alive = true;
      for (int k = 0; k < C::kBlocks && alive; ++k) {
        const int s = k % C::kStages;
        alive = bar_wait(full + s, (k / C::kStages) & 1u, abort_flag, a);
        if (!alive) break;
        fence_after();
        const uint32_t st = su32(smem + s * C::kStage);
        const uint64_t ad = sdesc(st, 16, 1024);
        const uint64_t bd = OP == kAbsorb ? sdesc(st + C::kABytes, 8192, 1024)
                                          : sdesc(st + C::kABytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma<false>(tmem, ad + kk * 2, bd + kk * (OP == kAbsorb ? 128 : 2), id, (k | kk) != 0);
        mma_commit(empty + s);
      }
      mma_commit(&done);
      bar_drain(&done, 0);
    }
  } else {
    const int quad = warp & 3;
    // the rope channels pass through: each column block takes its share of the
    // rows, loaded here and written with the tile (a CTA that gives up writes nothing)
    constexpr int kShare = OP == kAbsorb ? 8 * N / kLat : 1;  // rows per group of eight lanes
    uint4 rope[kShare];
    int t[kShare];
    if constexpr (OP == kAbsorb) {
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        t[i] = t0 + quad * 32 + (blockIdx.x * kShare + i) * 4 + (lane >> 3);
        if (t[i] < rows)
          rope[i] = __ldg(reinterpret_cast<const uint4*>(a.q + t[i] * a.q_row + h * a.q_head + kNope) +
                          (lane & 7));
      }
    }
    const bool ok = bar_wait(&done, 0, abort_flag, a);
    if (__all_sync(0xffffffffu, ok) && *abort_flag == 0 && t0 + quad * 32 < rows) {
      fence_after();
      // rows of N values through this warp's share of the stages, 16-byte
      // pieces exchanged by the row's low bits so that neither side conflicts
      constexpr int kRowBytes = N * (E4M3 ? 1 : 2), kPieces = kRowBytes / 16;
      uint8_t* mine = smem + quad * 32 * kRowBytes;
#pragma unroll
      for (int c = 0; c < N; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, v);
        tmem_wait_ld<32>(v);
        uint32_t w[16];
        if constexpr (E4M3) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[4 * e + i]) * a.inv_scale;
            w[e] = e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
        }
#pragma unroll
        for (int p = 0; p < (E4M3 ? 2 : 4); ++p) {
          const int piece = (c * (E4M3 ? 1 : 2)) / 16 + p;
          *reinterpret_cast<uint4*>(mine + lane * kRowBytes + ((piece ^ (lane & 7)) % kPieces) * 16) =
              make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
        }
      }
      __syncwarp();
      for (int i = lane; i < 32 * kPieces; i += 32) {
        const int r = i / kPieces, piece = i % kPieces, t = t0 + quad * 32 + r;
        if (t >= rows) break;
        const uint4 v = *reinterpret_cast<const uint4*>(mine + r * kRowBytes +
                                                        ((piece ^ (r & 7)) % kPieces) * 16);
        const int64_t o = (static_cast<int64_t>(t) * a.heads + h) * (OP == kAbsorb ? kLatRow : kNope) + n0;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + o * (E4M3 ? 1 : 2) + piece * 16) = v;
      }
      if constexpr (OP == kAbsorb) {
#pragma unroll
        for (int i = 0; i < kShare; ++i) {
          if (t[i] >= rows) continue;
          const int64_t o = (static_cast<int64_t>(t[i]) * a.heads + h) * kLatRow + kLat + (lane & 7) * 8;
          if constexpr (E4M3) {
            const uint32_t w[4] = {rope[i].x, rope[i].y, rope[i].z, rope[i].w};
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              c[e] = e4m3x2(__uint_as_float(w[e] << 16) * a.inv_scale,
                            __uint_as_float(w[e] & 0xFFFF0000u) * a.inv_scale);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + o) =
                make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o) = rope[i];
          }
        }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem)
                 : "memory");
}

template <int OP, int N, int STAGES, bool E4M3>
int launch_product(const ProductArgs& a, const CUtensorMap& ta, const CUtensorMap& tb,
                   cudaStream_t s) {
  using C = ProductCfg<OP, N, STAGES>;
  const auto fn = product<OP, N, STAGES, E4M3>;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  fn<<<dim3(C::kTotalN / N, a.heads, (a.rows + 127) / 128), 192, C::kSmem, s>>>(a, ta, tb);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

// ------------------------------------------------------- keys and values
//
// [k | v]_h[t] = [W_UK; W_UV]_h c_t. Bound: the tensor cores (8192 tokens x 128
// heads: 275 GFLOP, 147 us at the measured rate) and writing k and v (537 MB, 134
// us at the 4.0 TB/s that a plain fill reaches) alike; it takes 211 us in a graph of
// calls (220 as calls on changing inputs), 141 without the stores. So the operands must not cost anything on top: a CTA pair
// takes 256 tokens, M = 256 over both SMs, N = 256 (a head's k and v). Each CTA
// keeps its 128 latents (128 KB) in shared memory while half of the head's weights
// (CTA 0 W_UK, CTA 1 W_UV) stream past through a ring of five 16 KB stages: 32
// bytes a cycle from L2 and 2000 cycles from a load to its use. With one CTA and
// all of the weights it was 64 bytes a cycle and 1000 cycles, less than TMA takes.
// A pair takes an equal run of (row tile, head) pairs, head fastest (heads dealt
// out in groups of 4 to 32: 220 to 244 us); two accumulators of 256 columns let a
// head's rows be written while the next one's MMAs run.

struct ExpandArgs {
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int64_t o_row, o_head;
  const int32_t* total;
  uint32_t* status;
  uint64_t wait_limit_ns;
  int tokens, heads;
  uint32_t inject;         // PDA_INJECT_*, 0 in normal use
};

constexpr int kExpStages = 5;
constexpr int kExpA = 8 * 16384, kExpB = 16384;
constexpr int kExpOut = 8 * 2048;  // 32 rows x 64 bytes a warp
constexpr int kExpSmem = kExpA + kExpStages * kExpB + kExpOut + 1024;
constexpr int kExpThreads = 64 + 8 * 32;  // loads, MMAs, eight warps that write

// Every box of a pair has landed when this returns: the leader's part after a
// timeout in either CTA (without one the MMAs have read every box). The leader's
// barriers count both CTAs' bytes; x0 and x1 ring units and t0 and t1 row tiles
// were loaded by CTA 0 and 1, all within a ring (a tile) of what the MMAs gave back.
// A box that only CTA 1 issued is announced first, one that it did not issue is
// taken off. Out of line, so that a CTA's end stays short.
__device__ __noinline__ void drain_pair(uint64_t* full, uint64_t* a_full, uint32_t x0, uint32_t x1,
                                        uint32_t t0, uint32_t t1) {
  auto settle = [](uint64_t* bar, uint32_t k, uint32_t mine, uint32_t other, uint32_t bytes,
                   uint32_t parity) {
    if (k >= mine) bar_expect_tx(bar, bytes);
    else if (k >= other) bar_complete_tx(bar, bytes);
    bar_drain(bar, parity & 1u);
  };
  const uint32_t x = max(x0, x1), t = max(t0, t1);
  for (uint32_t k = x > kExpStages ? x - kExpStages : 0u; k < x; ++k)
    settle(full + k % kExpStages, k, x0, x1, kExpB, k / kExpStages);
  if (t) settle(a_full, t - 1, t0, t1, kExpA, t - 1);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpThreads, 1)
    expand(const __grid_constant__ ExpandArgs a, const __grid_constant__ CUtensorMap ta,
           const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t a_full, a_empty, full[kExpStages], empty[kExpStages], c_full[2], c_free[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ uint32_t issued_units, issued_tiles;  // ring units, row tiles this CTA has loaded
  uint8_t* smem = raw + ((1024u - (su32(raw) & 1023u)) & 1023u);
  uint8_t* ring = smem + kExpA;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    bar_init(&a_full, 1);
    bar_init(&a_empty, 1);
    for (int s = 0; s < kExpStages; ++s) {
      bar_init(full + s, 1);
      bar_init(empty + s, 1);
    }
    for (int c = 0; c < 2; ++c) {
      bar_init(c_full + c, 1);
      bar_init(c_free + c, 16);
    }
    bar_init(&drain, 1);
    abort_word = 0;
    issued_units = issued_tiles = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  cluster_sync();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // this pair's run of (row tile, head) pairs, head fastest
  const int rows = min(a.tokens, __ldg(a.total));
  const int64_t pairs = static_cast<int64_t>((max(rows, 0) + 255) / 256) * a.heads;
  const int64_t me = blockIdx.x / 2, of = gridDim.x / 2;
  const int64_t f0 = pairs * me / of, f1 = pairs * (me + 1) / of;
  // The latents come from the kernel in front of this one. Every thread waits here
  // for it (so does a CTA without work: what follows has to follow both kernels),
  // and no bounded wait below counts its time.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t hooks = PDA_INJECT_WITHHOLD_KV |
                         (rank ? PDA_INJECT_WITHHOLD_CTA1 : PDA_INJECT_WITHHOLD_CTA0);
  if (warp == 0) {
    if (lane == 0) {
      // the leader's barriers count the bytes of both CTAs
      const uint32_t a_bar = on_leader(&a_full);
      bool alive = (a.inject & hooks) == 0u;
      uint32_t x = 0, tiles = 0;
      int tile = -1;
      for (int64_t f = f0; f < f1 && alive; ++f) {
        const int h = static_cast<int>(f % a.heads), t = static_cast<int>(f / a.heads);
        if (t != tile) {
          if (!(alive = bar_wait(&a_empty, (tiles & 1u) ^ 1u, abort_flag, a))) break;
          tile = t;
          ++tiles;
          if (rank == 0) bar_expect_tx(&a_full, 2 * kExpA);
          for (int k = 0; k < 8; ++k)
            tma_load3_pair(su32(smem + k * 16384), &ta, k * 64, 0, t * 256 + rank * 128, a_bar);
        }
        for (int k = 0; k < 8; ++k, ++x) {
          const uint32_t s = x % kExpStages;
          if (!(alive = bar_wait(empty + s, ((x / kExpStages) & 1u) ^ 1u, abort_flag, a))) break;
          if (rank == 0) bar_expect_tx(full + s, 2 * kExpB);
          tma_load3_pair(su32(ring + s * kExpB), rank ? &tv : &tk, k * 64, 0, h, on_leader(full + s));
        }
      }
      issued_units = x;
      issued_tiles = tiles;
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t id = idesc(1u, 0, 256) + ((128u >> 4) << 24);  // M = 256
      const uint64_t ad = sdesc(su32(smem), 16, 1024), bd = sdesc(su32(ring), 16, 1024);
      bool alive = true;
      uint32_t x = 0, tiles = 0, n = 0;
      int tile = -1;
      for (int64_t f = f0; f < f1 && alive; ++f, ++n) {
        const int t = static_cast<int>(f / a.heads);
        if (t != tile) {
          tile = t;
          if (!(alive = bar_wait(&a_full, tiles & 1u, abort_flag, a))) break;
          ++tiles;
        }
        const uint32_t c = n & 1u;
        if (!(alive = bar_wait(c_free + c, ((n >> 1) & 1u) ^ 1u, abort_flag, a))) break;
        for (int k = 0; k < 8; ++k, ++x) {
          const uint32_t s = x % kExpStages;
          if (!(alive = bar_wait(full + s, (x / kExpStages) & 1u, abort_flag, a))) break;
          fence_after();
          const uint64_t ak = ad + k * 1024, bk = bd + s * (kExpB / 16);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma2(tmem + c * 256, ak + kk * 2, bk + kk * 2, id, (k | kk) != 0);
          mma_commit2(empty + s);
        }
        if (!alive) break;
        mma_commit2(c_full + c);
        if (f + 1 == f1 || static_cast<int>((f + 1) / a.heads) != tile) mma_commit2(&a_empty);
      }
      // nothing issued may still run when either CTA releases its TMEM
      mma_commit2(&drain);
    }
    if (lane == 0) bar_drain(&drain, 0);
  } else {
    // a warp writes 32 rows of k (warps 2-5) or of v (6-9)
    const int quad = warp & 3, part = (warp - 2) >> 2;
    uint8_t* mine = ring + kExpStages * kExpB + (warp - 2) * 2048;
    auto place = [&](int r, int piece) {  // no two rows of a quarter warp in one bank
      return reinterpret_cast<uint4*>(mine + r * 64 + ((piece ^ (r >> 1)) & 3) * 16);
    };
    uint32_t n = 0;
    for (int64_t f = f0; f < f1; ++f, ++n) {
      const int h = static_cast<int>(f % a.heads);
      const int64_t t0 = (f / a.heads) * 256 + rank * 128 + quad * 32;  // this warp's rows
      const uint32_t c = n & 1u;
      const bool ok = bar_wait(c_full + c, (n >> 1) & 1u, abort_flag, a);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c * 256 + part * kNope;
      __nv_bfloat16* out = (part ? a.v : a.k) + h * a.o_head + (lane & 3) * 8;
      // 32 columns at a time through shared memory, so that a store writes 64
      // bytes of a row; a row per lane, straight from the registers, wrote 16 (297 us)
#pragma unroll
      for (int col = 0; col < kNope; col += 32) {
        uint32_t v[32];
        tmem_ld32(src + col, v);
        tmem_wait_ld<32>(v);
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = bf16x2(__uint_as_float(v[p * 8 + 2 * e]), __uint_as_float(v[p * 8 + 2 * e + 1]));
          *place(lane, p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          if (t0 + r < rows)
            *reinterpret_cast<uint4*>(out + (t0 + r) * a.o_row + col) = *place(r, lane & 3);
        }
      }
      __syncwarp();
      fence_before();
      if (lane == 0) bar_arrive_at(on_leader(c_free + c));
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) cluster_store(on_cta(&abort_word, rank ^ 1u), 1u);
  __syncwarp();
  cluster_sync();  // the pair's barriers and shared memory are used until here
  // every box issued must have landed before either CTA can exit
  if (*abort_flag) {
    if (tid == 0 && rank == 0)
      drain_pair(full, &a_full, issued_units, cluster_load(on_cta(&issued_units, 1)), issued_tiles,
                 cluster_load(on_cta(&issued_tiles, 1)));
    __syncwarp();
    cluster_sync();
  }
  fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

bool a16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool a4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// The checks that the three entry points share.
int check_mla(const pda_plan_t* plan, int64_t w_stride_head, int rows, const int32_t* num_rows,
              const void* split_scratch) {
  if (!plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  if (!split_scratch || reinterpret_cast<uintptr_t>(split_scratch) % 256) return PDA_ERR_SCRATCH;
  if (plan->head_dim != kLatRow || plan->num_kv_heads != 1) return PDA_ERR_UNSUPPORTED;
  // (row tiles are a grid's z, heads its y)
  if (rows < 0 || rows > 65535 * 128 || plan->num_qo_heads > 65535 || w_stride_head < kNope * kLat)
    return PDA_ERR_INVALID;
  if (w_stride_head % 8 || !a4(num_rows)) return PDA_ERR_ALIGNMENT;
  return PDA_OK;
}

}  // namespace
}  // namespace pda

extern "C" int pda_mla_absorb(const pda_plan_t* plan, const void* q, int64_t q_stride_row,
                              int64_t q_stride_head, const void* w_uk, int64_t w_stride_head,
                              float q_scale, void* q_lat, int32_t rows, const int32_t* num_rows,
                              void* split_scratch, pda_stream_t stream) {
  using namespace pda;
  const int rc = check_mla(plan, w_stride_head, rows, num_rows, split_scratch);
  if (rc != PDA_OK || rows == 0) return rc;
  if (!q || !w_uk || !q_lat) return PDA_ERR_NULL;
  const bool e4m3 = plan->q_dtype == PDA_E4M3;
  // (its reciprocal too has to be a finite number)
  if (e4m3 && !(q_scale > 0.f && q_scale < INFINITY && 1.f / q_scale < INFINITY))
    return PDA_ERR_INVALID;
  if (q_stride_head < kQDim || q_stride_row < kQDim) return PDA_ERR_INVALID;
  if (!a16(q) || !a16(w_uk) || !a16(q_lat) || q_stride_row % 8 || q_stride_head % 8)
    return PDA_ERR_ALIGNMENT;
  ProductArgs p = {};
  p.out = q_lat;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_row = q_stride_row;
  p.q_head = q_stride_head;
  p.num_rows = num_rows;
  p.status = static_cast<uint32_t*>(split_scratch);
  p.wait_limit_ns = static_cast<uint64_t>(plan->wait_limit_us) * 1000ull;
  p.inv_scale = e4m3 ? 1.f / q_scale : 0.f;
  p.rows = rows;
  p.heads = plan->num_qo_heads;
  p.inject = plan->inject;
  CUtensorMap ta, tb;
  if (!make_map3(&ta, q, kNope, p.heads, rows, q_stride_head, q_stride_row, 64, 1, 128) ||
      !make_map3(&tb, w_uk, kLat, kNope, p.heads, kLat, w_stride_head, 64, 64, 1))
    return PDA_ERR_CUDA;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return e4m3 ? launch_product<kAbsorb, 128, 2, true>(p, ta, tb, s)
              : launch_product<kAbsorb, 128, 2, false>(p, ta, tb, s);
}

extern "C" int pda_mla_project(const pda_plan_t* plan, const void* o_lat, const void* w_uv,
                               int64_t w_stride_head, void* out, int32_t rows,
                               const int32_t* num_rows, void* split_scratch, pda_stream_t stream) {
  using namespace pda;
  const int rc = check_mla(plan, w_stride_head, rows, num_rows, split_scratch);
  if (rc != PDA_OK || rows == 0) return rc;
  if (!o_lat || !w_uv || !out) return PDA_ERR_NULL;
  if (!a16(o_lat) || !a16(w_uv) || !a16(out)) return PDA_ERR_ALIGNMENT;
  ProductArgs p = {};
  p.out = out;
  p.num_rows = num_rows;
  p.status = static_cast<uint32_t*>(split_scratch);
  p.wait_limit_ns = static_cast<uint64_t>(plan->wait_limit_us) * 1000ull;
  p.rows = rows;
  p.heads = plan->num_qo_heads;
  p.inject = plan->inject;
  // Few (head, row tile) pairs (half the SMs): four CTAs share a pair's columns,
  // each streams a quarter of the weights, all of K in flight. Up to a pair an
  // SM: one CTA an SM with half of K in flight (four stages against two or three:
  // 5.0 against 6.8 / 5.9 us at one row of 128 heads). More: three CTAs an SM of
  // two stages (1024 rows, 128 heads, 2 / 3 / 4 stages: 36.7 / 38.6 / 43.9 us).
  const int64_t pairs = static_cast<int64_t>(p.heads) * ((rows + 127) / 128);
  const bool few = pairs * 2 <= plan->num_sms;
  CUtensorMap ta, tb;
  if (!make_map3(&ta, o_lat, kLat, p.heads, rows, kLat, static_cast<int64_t>(p.heads) * kLat, 64, 1, 128) ||
      !make_map3(&tb, w_uv, kLat, kNope, p.heads, kLat, w_stride_head, 64, few ? 32 : 128, 1))
    return PDA_ERR_CUDA;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (few) return launch_product<kProject, 32, 8, false>(p, ta, tb, s);
  return pairs <= plan->num_sms ? launch_product<kProject, 128, 4, false>(p, ta, tb, s)
                                : launch_product<kProject, 128, 2, false>(p, ta, tb, s);
}

extern "C" int pda_mla_expand(const pda_plan_t* plan, const void* k_pages,
                              const int32_t* page_table, const int32_t* kv_indptr,
                              const int32_t* tok_indptr, const float* k_scale, const void* w_uk,
                              const void* w_uv, int64_t w_stride_head, void* latent, void* k,
                              void* v, int64_t kv_stride_token, int64_t kv_stride_head,
                              int32_t tokens, void* split_scratch, pda_stream_t stream) {
  using namespace pda;
  const int rc = check_mla(plan, w_stride_head, tokens, nullptr, split_scratch);
  if (rc != PDA_OK || tokens == 0 || plan->batch == 0) return rc;
  if (!k_pages || !page_table || !kv_indptr || !tok_indptr || !w_uk || !w_uv || !latent || !k || !v)
    return PDA_ERR_NULL;
  const bool rec = plan->scale_mode == PDA_SCALE_MLA_BLOCK;
  if (plan->scale_mode != PDA_SCALE_NONE && !k_scale) return PDA_ERR_NULL;
  if (kv_stride_head < kNope || kv_stride_token < kNope) return PDA_ERR_INVALID;
  if (!a16(k_pages) || !a16(w_uk) || !a16(w_uv) || !a16(latent) || !a16(k) || !a16(v) ||
      kv_stride_token % 8 || kv_stride_head % 8 || !a4(page_table) || !a4(kv_indptr) ||
      !a4(tok_indptr) || (rec ? !a16(k_scale) : !a4(k_scale)))
    return PDA_ERR_ALIGNMENT;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  GatherArgs g = {};
  g.pages = static_cast<const uint8_t*>(k_pages);
  g.page_table = page_table;
  g.kv_indptr = kv_indptr;
  g.tok_indptr = tok_indptr;
  g.scale = k_scale;
  g.latent = static_cast<__nv_bfloat16*>(latent);
  g.status = static_cast<uint32_t*>(split_scratch);
  g.sp = plan->kv_stride_page;
  g.st = plan->kv_stride_token;
  g.batch = plan->batch;
  g.tokens = tokens;
  while ((1 << g.page_shift) < plan->page_size) ++g.page_shift;
  g.num_pages = plan->num_pages;
  g.max_kv_len = plan->max_kv_len;
  const unsigned blocks = static_cast<unsigned>((tokens + 7) / 8);
  if (rec) gather_latent<5><<<blocks, 256, 0, s>>>(g);
  else if (plan->kv_dtype == PDA_BF16) gather_latent<0><<<blocks, 256, 0, s>>>(g);
  else if (plan->scale_mode == PDA_SCALE_TENSOR) gather_latent<1><<<blocks, 256, 0, s>>>(g);
  else gather_latent<2><<<blocks, 256, 0, s>>>(g);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  ExpandArgs e = {};
  e.k = static_cast<__nv_bfloat16*>(k);
  e.v = static_cast<__nv_bfloat16*>(v);
  e.o_row = kv_stride_token;
  e.o_head = kv_stride_head;
  e.total = tok_indptr + plan->batch;
  e.status = g.status;
  e.wait_limit_ns = static_cast<uint64_t>(plan->wait_limit_us) * 1000ull;
  e.tokens = tokens;
  e.heads = plan->num_qo_heads;
  e.inject = plan->inject;
  CUtensorMap ta, tk, tv;
  if (!make_map3(&ta, latent, kLat, 1, tokens, kLatRow, kLatRow, 64, 1, 128) ||
      !make_map3(&tk, w_uk, kLat, kNope, e.heads, kLat, w_stride_head, 64, 128, 1) ||
      !make_map3(&tv, w_uv, kLat, kNope, e.heads, kLat, w_stride_head, 64, 128, 1))
    return PDA_ERR_CUDA;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(expand),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kExpSmem) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  const int64_t pairs = static_cast<int64_t>((tokens + 255) / 256) * e.heads;
  const int64_t clusters = plan->num_sms / 2 < 1 ? 1 : plan->num_sms / 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (pairs < clusters ? pairs : clusters)));
  cfg.blockDim = dim3(kExpThreads);
  cfg.dynamicSmemBytes = kExpSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, expand, e, ta, tk, tv) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  return PDA_OK;
}
