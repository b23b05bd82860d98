// pda_prefill.cu -- expanded latent attention of ragged requests (prefill), on
// the 5th-generation tensor cores.
//
// Mathematics: for 256 query rows of one request and head, over tiles of 128
// keys: S = Q K^T with K = [k | k_rope] (192 channels, the rope part shared by
// all heads and read from the latents), an online softmax in log2 units,
// O += P V. The running maximum is lazy: a row moves it only when a logit
// passes it by more than 8, so P <= 2^8, and the sum l of the fp32 weights and
// O are rescaled then; O / l is exact in it. P is rounded to bf16, V's type (2^-9
// relative on average, random), while l sums the unrounded weights.
//
// Bound: the tensor cores (640 flops per row, key and head). A tile of 128 rows
// x 128 keys takes 12 + 8 MMAs, 1280 cycles; its softmax is 16384 exponentials
// plus about four instructions each, hidden behind the other tile's MMAs. So a
// CTA holds two 128-row tiles (96 KB of Q, shared K and V: half the L2 reads of
// one tile), whose S take turns:
//   PV(0, j)  QK(0, j+1)  PV(1, j)  QK(1, j+1)  ...
// S, P (over S, bf16, the MMA's A operand) and O of both fill the 512 TMEM
// columns, so neither P nor O touches shared memory. P is handed over in halves
// of 64 keys, as the way from S to the next S decides the pace.
// Measured, 4096 rows x 128 heads: in graphs of calls over the same inputs 470 us causal
// (1.46 PFLOP/s, 78 % of the measured bf16 burst rate) and 750 to 790 with every key
// visible (1.74 to 1.83, 93 to 98 %); as calls on changing inputs 500 and 854.
//
// Roles: warps 0-3 and 4-7 are the softmax of tile 0 and 1; warp 8 loads (TMA),
// warp 9 issues the MMAs, warp 10 clears V rows behind the last key (0 x NaN),
// warp 11 takes (head, tile, chunk) items off a counter in the scratch; the warps
// pass items on through a ring, so that the loads and MMAs of the next item start
// while this one's rows are written. K and V pass through a ring of 16 KB units:
// three of K (128 keys x 64 channels), two of V (64 keys x 128 channels) a tile.
//
// Few rows: where heads x tiles are at most half the SMs, a tile's keys are cut
// into chunks (pda_prefill_plan), whose normalised partial outputs and log2 sums
// a second kernel joins. 64 rows on 8064 keys, 16 heads: 25 us, 104 uncut.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "pda.h"
#include "pda_cvt.cuh"
#include "pda_internal.h"
#include "pda_ptx.cuh"

namespace pda {
namespace {

constexpr int kNope = 128, kRope = 64, kQDim = kNope + kRope, kDv = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMInit = -3.0e38f;  // before any key: finite, so that ex2(-inf - m) = 0
constexpr float kTh = 8.0f;         // lazy rescale threshold, log2 units

constexpr int kRowsTile = 128;                // rows of one softmax warpgroup
constexpr int kRowsItem = 2 * kRowsTile;      // rows of an item
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kUnit = 16384;                  // bytes of a ring unit
constexpr int kRing = 8;                      // units
constexpr int kUnitsK = 3, kUnitsV = 2, kUnitsTile = kUnitsK + kUnitsV;
constexpr int kQBytes = 2 * 3 * kUnit;        // two tiles of three 64-channel blocks
constexpr int kItems = 3;                     // slots of the item ring
constexpr int kSoftmaxWarps = 8;              // a thread per row
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kCoarse = 256;                  // prefix entries, 32 requests each
constexpr int kMaxBatch = 32 * kCoarse;
constexpr int kLoadWarp = kSoftmaxWarps, kMmaWarp = kLoadWarp + 1, kClearWarp = kLoadWarp + 2;
constexpr int kReaders = kSoftmaxWarps + 3;                  // arrivals that free an item slot
constexpr int kTmemCols = 512;

struct PrefillArgs {
  const int32_t* qo_indptr;
  const int32_t* tok_indptr;
  const int32_t* window;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;    // [splits][rows][heads][128] fp32, normalised
  float* part_lse;  // [splits][rows][heads] fp32, log2 units
  uint32_t* status;
  uint32_t* taken;  // items handed out beyond the first of each CTA; 0 between calls
  uint32_t* done;   // CTAs that have found no more; 0 between calls
  uint64_t wait_limit_ns;
  float sm_scale;
  int heads, batch, max_kv_len, rows, tokens, causal, splits, chunk_tiles;
  uint32_t inject;  // PDA_INJECT_*, 0 in normal use
};

// One request's geometry, and whether it takes part (else its status bits).
struct Request {
  int q0, rows, k0, keys, win;
  uint32_t bad;
};
__device__ __forceinline__ Request request_of(const PrefillArgs& a, int b) {
  Request r;
  r.q0 = __ldg(a.qo_indptr + b);
  r.k0 = __ldg(a.tok_indptr + b);
  const int64_t q1 = __ldg(a.qo_indptr + b + 1), k1 = __ldg(a.tok_indptr + b + 1);
  r.win = a.window ? __ldg(a.window + b) : 0;
  r.bad = 0u;
  if (q1 < r.q0 || r.q0 < 0) r.bad |= PDA_STATUS_ROWS_GT_MAX;
  if (q1 > a.rows) r.bad |= PDA_STATUS_ROWS_GT_CAP;
  if (k1 < r.k0 || r.k0 < 0 || k1 > a.tokens) r.bad |= PDA_STATUS_TOKENS_GT_CAP;
  if (k1 - r.k0 > a.max_kv_len) r.bad |= PDA_STATUS_KV_LEN_GT_MAX;
  if (a.causal && k1 - r.k0 < q1 - r.q0) r.bad |= PDA_STATUS_KV_LEN_LT_ROWS;
  if (q1 == r.q0) r.bad = 0u;  // no rows: nothing to refuse
  r.rows = r.bad ? 0 : static_cast<int>(q1 - r.q0);
  r.keys = r.bad || q1 == r.q0 ? 0 : static_cast<int>(k1 - r.k0);
  return r;
}

// Key tiles [lo, hi) that rows [i, i + n) of a request see (n > 0).
__device__ __forceinline__ void key_tiles(const PrefillArgs& a, const Request& r, int i, int n,
                                          int& lo, int& hi) {
  int first = 0, end = r.keys;
  if (a.causal) {
    const int p = r.keys - r.rows + i;  // position of row i
    end = p + n;
    if (r.win > 0 && p >= r.win) first = p - r.win + 1;
  }
  lo = first / kKeys;
  hi = (end + kKeys - 1) / kKeys;
}

// One item: 256 rows of a request and head, over the key tiles of one chunk.
struct Item {
  int head;       // -1: no more items
  int row0;       // first row in q / out
  int rows;       // 1..256
  int pos;        // position of the first row
  int keys;       // L of the request
  int k0;         // its first token in k / v
  int win;
  int lo0, hi0, lo1, hi1;  // key tiles of both 128-row tiles in this chunk (empty: lo = hi)
  int split;      // chunk, or -1: the only one, out is final
};

struct Shared {
  uint64_t q_full[2], q_empty[2], full[kRing], empty[kRing], s_full[2], p_half[2], p_full[2], o_done[2],
      o_free[2], item_full[kItems], item_empty[kItems], landed[kRing], drain;
  uint32_t tmem;
  int abort_flag;
  Item items[kItems];
  int coarse[kCoarse];
};
constexpr int kSmem = kQBytes + kRing * kUnit + static_cast<int>(sizeof(Shared));
static_assert(kSmem <= 227 * 1024, "shared memory");

// The item ring from a reader's side.
struct ItemReader {
  Shared* sh;
  uint32_t n = 0;
  __device__ explicit ItemReader(Shared* s) : sh(s) {}
  // One thread: the next item, or false after the last one (or an abort).
  __device__ bool next_one(Item& it, const PrefillArgs& a) {
    const uint32_t slot = n % kItems;
    if (!bar_wait(sh->item_full + slot, (n / kItems) & 1u, &sh->abort_flag, a)) return false;
    it = sh->items[slot];
    bar_arrive(sh->item_empty + slot);
    ++n;
    return it.head >= 0;
  }
  // A whole warp (one arrival); warp-uniform.
  __device__ bool next_warp(Item& it, const PrefillArgs& a) {
    const uint32_t slot = n % kItems;
    const bool ok = bar_wait(sh->item_full + slot, (n / kItems) & 1u, &sh->abort_flag, a);
    if (!__all_sync(0xffffffffu, ok)) return false;
    it = sh->items[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(sh->item_empty + slot);
    ++n;
    return it.head >= 0;
  }
};

// ------------------------------------------------------------------- loads
//
// Ring units in the order K_j (3), V_j (2), K_{j+1}, ...: unit x takes the place
// x % 8, which unit x - 8 leaves as soon as the MMAs of row tile 1 have read it.
// V_{j+1} and the first unit of K_{j+2} follow K_j, its other two V_j. Counted
// per unit, a load has 1800 to 3000 cycles at the tensor cores' pace until it is
// needed; counted per tile the later units of K had 1280, less than TMA takes.
__device__ void load_role(const PrefillArgs& a, Shared* sh, uint8_t* q_s, uint8_t* ring,
                          const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tr,
                          const CUtensorMap* tv) {
  volatile int* abort_flag = &sh->abort_flag;
  const uint32_t ring_addr = su32(ring);
  ItemReader reader(sh);
  Item it{};
  uint32_t x = 0, nq0 = 0, nq1 = 0;  // ring unit, Q tiles
  uint32_t parity = 0u;              // uses of each place's `landed` mod 2
  uint32_t tail0 = ~0u - kRing, tail1 = tail0;  // first V units of the last two tiles that use it
  bool alive = (a.inject & PDA_INJECT_WITHHOLD_KV) == 0u;
  auto dst = [&](uint32_t unit) { return ring_addr + unit % kRing * kUnit; };
  auto place = [&](uint32_t unit) {
    return alive = bar_wait(sh->empty + unit % kRing, ((unit / kRing) & 1u) ^ 1u, abort_flag, a);
  };
  auto load_q = [&](int g) {
    if ((g ? it.lo1 >= it.hi1 : it.lo0 >= it.hi0) || !alive) return;
    uint32_t& nq = g ? nq1 : nq0;
    if (!(alive = bar_wait(sh->q_empty + g, (nq & 1u) ^ 1u, abort_flag, a))) return;
    bar_expect_tx(sh->q_full + g, 3 * kUnit);
    for (int c = 0; c < 3; ++c)
      tma_load3(su32(q_s + (g * 3 + c) * kUnit), tq, c * 64, it.head, it.row0 + g * kRowsTile,
                sh->q_full + g);
    ++nq;
  };
  while (alive && reader.next_one(it, a)) {
    const int lo = min(it.lo0, it.lo1), hi = max(it.hi0, it.hi1);
    const int tail = it.keys % kKeys ? it.keys / kKeys : -1;
    load_q(0);
    for (int j = lo; j < hi && alive; ++j) {
      const int tok = it.k0 + j * kKeys;
      for (int c = 0; c < kUnitsK && place(x); ++c, ++x) {
        uint64_t* bar = sh->full + x % kRing;
        bar_expect_tx(bar, kUnit);
        if (c < 2) tma_load3(dst(x), tk, c * 64, it.head, tok, bar);
        else tma_load3(dst(x), tr, 0, 0, tok, bar);
      }
      if (j == lo) load_q(1);
      for (int c = 0; c < kUnitsV && alive && place(x); ++c, ++x) {
        // the last tile's V lands for the clearing warp, which passes it on (a
        // barrier per place: two short items' last tiles may be under way at once)
        const uint32_t slot = x % kRing;
        uint64_t* bar = j == tail ? sh->landed + slot : sh->full + slot;
        bar_expect_tx(bar, kUnit);
        if (j == tail) {
          if (c == 0) tail0 = tail1, tail1 = x;
          parity ^= 1u << slot;
        }
        for (int d = 0; d < 2; ++d)
          tma_load3(dst(x) + d * (kUnit / 2), tv, d * 64, it.head, tok + c * 64, bar);
      }
    }
  }
  // Every box issued must have landed before the CTA can exit: the last unit of
  // each place (what was there before it has been read; two tiles' V at most are
  // among them) and the last Q tiles.
  // Always, not only after an abort seen here: another role's wait may run out
  // later.
  for (uint32_t k = x > kRing ? x - kRing : 0u; k < x; ++k) {
    const uint32_t s = k % kRing;
    if (k - tail0 < kUnitsV || k - tail1 < kUnitsV) bar_drain(sh->landed + s, (parity >> s & 1u) ^ 1u);
    else bar_drain(sh->full + s, (k / kRing) & 1u);
  }
  if (nq0) bar_drain(sh->q_full, (nq0 - 1) & 1u);
  if (nq1) bar_drain(sh->q_full + 1, (nq1 - 1) & 1u);
}

// -------------------------------------------------------------------- MMAs
//
// One thread. Everything it does between MMAs counts: about four MMAs wait in
// the tensor cores' queue, so 256 cycles at a time are hidden and more is lost.
__device__ void mma_role(const PrefillArgs& a, Shared* sh, uint8_t* q_s, uint8_t* ring) {
  volatile int* abort_flag = &sh->abort_flag;
  constexpr uint32_t tmem = 0;  // all columns are ours: they start at 0
  const uint32_t id_s = idesc(1u, 0, kKeys), id_o = idesc(1u, 0, kDv, 1u);
  // descriptors count in 16 bytes
  const uint64_t q_desc = sdesc(su32(q_s), 16, 1024), k_desc = sdesc(su32(ring), 16, 1024),
                 v_desc = sdesc(su32(ring), kUnit / 2, 1024);
  ItemReader reader(sh);
  Item it{};
  uint32_t x = 0;              // first ring unit of tile j
  uint32_t pp = 0u, qp = 0u;   // parities of p_full and of the items, a bit per row tile
  bool alive = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return alive = bar_try(bar, parity & 1u) || bar_wait_slow(bar, parity & 1u, abort_flag, a);
  };
  while (alive && reader.next_one(it, a)) {
    const int lo0 = it.lo0, hi0 = it.hi0, lo1 = it.lo1, hi1 = it.hi1;
    const int lo = min(lo0, lo1), hi = max(hi0, hi1);
    if (lo >= hi) continue;
    // step j: P V of tile j, then Q K of tile j + 1, for both row tiles
    for (int j = lo - 1; j < hi && alive; ++j) {
      const uint32_t x1 = j < lo ? x : x + kUnitsTile;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int from = g ? lo1 : lo0, to = g ? hi1 : hi0;
        const bool do_pv = j >= from && j < to, do_qk = j + 1 >= from && j + 1 < to;
        if (do_pv) {
          if (j == from && !wait(sh->o_free + g, qp >> g)) break;  // the last item's O is read
          if (!wait(sh->p_half + g, pp >> g)) break;
        }
        if (do_pv || (g == 1 && j >= lo)) {
#pragma unroll
          for (int c = 0; c < kUnitsV; ++c) {
            const uint32_t u = x + kUnitsK + c, slot = u % kRing;
            if (do_pv) {
              if (!wait(sh->full + slot, u / kRing)) break;
              if (c == 1) {  // the second half of P's keys
                if (!wait(sh->p_full + g, pp >> g)) break;
                pp ^= 1u << g;
              }
              fence_after();
              const uint64_t vd = v_desc + slot * (kUnit / 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(tmem + 2 * kKeys + g * kDv, tmem + g * kKeys + (c * 4 + kk) * 8, vd + kk * 128,
                       id_o, (c | kk) ? 1u : (j != from ? 1u : 0u));
            }
            if (g == 1) mma_commit(sh->empty + slot);
          }
          if (!alive) break;
          if (do_pv) mma_commit(sh->o_done + g);
        }
        if (do_qk || (g == 1 && j + 1 < hi)) {
          if (do_qk && j + 1 == from) {
            if (!wait(sh->q_full + g, qp >> g)) break;
            qp ^= 1u << g;
          }
#pragma unroll
          for (int c = 0; c < kUnitsK; ++c) {
            const uint32_t u = x1 + c, slot = u % kRing;
            if (do_qk) {
              if (!wait(sh->full + slot, u / kRing)) break;
              if (c == 0) fence_after();
              const uint64_t kd = k_desc + slot * (kUnit / 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma<false>(tmem + g * kKeys, q_desc + (g * 3 + c) * (kUnit / 16) + kk * 2, kd + kk * 2,
                           id_s, (c | kk) != 0);
            }
            if (g == 1) mma_commit(sh->empty + slot);
          }
          if (!alive) break;
          if (do_qk) {
            mma_commit(sh->s_full + g);
            if (j + 2 == to) mma_commit(sh->q_empty + g);
          }
        }
      }
      x = x1;
    }
  }
  // nothing issued may still run when TMEM is released
  mma_commit(&sh->drain);
  bar_drain(&sh->drain, 0);
}

// ------------------------------------------------- V rows behind the last key
__device__ void clear_role(const PrefillArgs& a, Shared* sh, uint8_t* ring) {
  const int lane = threadIdx.x & 31;
  ItemReader reader(sh);
  Item it{};
  uint32_t t = 0, parity = 0u;  // key tiles in front of the item; uses of `landed` mod 2
  while (reader.next_warp(it, a)) {
    const int lo = min(it.lo0, it.lo1), hi = max(it.hi0, it.hi1);
    const int tail = it.keys % kKeys ? it.keys / kKeys : -1;
    if (tail >= lo && tail < hi) {
      const uint32_t x = (t + static_cast<uint32_t>(tail - lo)) * kUnitsTile + kUnitsK;
      for (int c = 0; c < kUnitsV; ++c) {
        const uint32_t slot = (x + c) % kRing;
        const bool ok = bar_wait(sh->landed + slot, parity >> slot & 1u, &sh->abort_flag, a);
        if (!__all_sync(0xffffffffu, ok)) return;
        parity ^= 1u << slot;
      }
      for (int r = it.keys % kKeys; r < kKeys; r += 2) {
        // two rows x 16 pieces of 16 bytes (two 64-channel atoms) a step
        const int row = r + (lane >> 4), piece = lane & 15;
        if (row < kKeys)
          *reinterpret_cast<uint4*>(ring + (x + (row >> 6)) % kRing * kUnit +
                                    (piece >> 3) * (kUnit / 2) + (row & 63) * 128 + (piece & 7) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int c = 0; c < kUnitsV; ++c) bar_arrive(sh->full + (x + c) % kRing);
    }
    t += static_cast<uint32_t>(max(0, hi - lo));
  }
}

// --------------------------------------------------------------- the work list
__device__ void work_role(const PrefillArgs& a, Shared* sh) {
  const int lane = threadIdx.x & 31;
  // tiles in front of every 32 requests, and in all
  int64_t total = 0;
  uint32_t bits = 0u;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int n = 0;
    if (b0 + lane < a.batch) {
      const Request r = request_of(a, b0 + lane);
      bits |= r.bad;
      n = (r.rows + kRowsItem - 1) / kRowsItem;
    }
    if (lane == 0) sh->coarse[b0 >> 5] = static_cast<int>(total);
    total += __reduce_add_sync(0xffffffffu, n);
  }
  __syncwarp();
  if (blockIdx.x == 0) {
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0 && bits) atomicOr(a.status, bits);
  }
  const int64_t items = total * a.heads * a.splits;
  // Heads go in groups, so that their K and V stay in L2; a group's items from the
  // last tiles (the most keys) to the first, chunks of a tile side by side. CTAs
  // take items one by one, as causal tiles differ: in steps of the grid, 4096 x
  // 128 heads took a third longer. A group is worth `rounds` items a CTA: where items
  // differ, enough that its short ones even out the long ones; where they do not, L2 is
  // all that counts. us of a call on inputs that change from call to call, at
  // 1 / 2 / 3 / 4 / 6 / 8 rounds, causal:
  //   4096 rows, 128 heads                535 / 518 / 512 / 522 / 528 / 549
  //   4096 rows, 64 heads                 315 / 271 / 267 / 268 / 268 / 267
  //   8192 rows, 32 heads                 525 / 494 / 483 / 473 / 470 / 470
  //   8 x 256 to 1024 rows, 128 heads     260 / 255 / 245 / 237 / 230 / 227
  //   1024 rows on 5120 keys, 64 heads    147 / 148 / 148 / 149 / 148 / 148
  // and with every key visible:
  //   4096 rows, 128 heads                854 / 878 / 902 / 920 / 948 / 1002
  //   4096 rows, 64 heads                 430 / 441 / 454 / 477 / 477 / 477
  //   2048 rows, 64 heads                 128 / 136 / 136 / 136 / 136 / 136
  // Six would serve many short items better than three and few long ones worse (in a
  // graph over two states, whose addresses stay, six is the better or equal at all of
  // them: 465 against 467 and 250 against 254 us at the first two).
  const int64_t rounds = a.causal ? 3 : 1;
  const int64_t tiles = max(total, static_cast<int64_t>(1));
  const int64_t wish = max(static_cast<int64_t>(1), rounds * gridDim.x / (tiles * a.splits));
  const int64_t groups = max(static_cast<int64_t>(1), a.heads / wish);
  const int64_t group = (a.heads + groups - 1) / groups;
  uint32_t n = 0;
  int64_t x = blockIdx.x;
  auto take = [&]() {
    uint32_t v = 0;
    if (lane == 0) v = atomicAdd(a.taken, 1u);
    x = static_cast<int64_t>(gridDim.x) + __shfl_sync(0xffffffffu, v, 0);
  };
  for (;;) {
    Item it;
    it.head = -1;
    if (x < items) {
      const int split = static_cast<int>(x % a.splits);
      const int64_t y = x / a.splits;
      const int64_t first = y / (group * total) * group;  // the group's first head
      const int64_t wide = min(group, a.heads - first), z = y - first * total;
      const int t = static_cast<int>(total - 1 - z / wide);
      it.head = static_cast<int>(first + z % wide);
      take();
      int c = 0, top = (a.batch + 31) / 32 - 1;
      while (c < top) {
        const int mid = (c + top + 1) >> 1;
        if (sh->coarse[mid] <= t) c = mid;
        else top = mid - 1;
      }
      const int b = 32 * c + lane;
      Request r = {};
      if (b < a.batch) r = request_of(a, b);
      const int mine = (r.rows + kRowsItem - 1) / kRowsItem;
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y2 = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y2;
      }
      const int want = t - sh->coarse[c];
      const int src = __ffs(__ballot_sync(0xffffffffu, upto > want)) - 1;
      const int i = (want - __shfl_sync(0xffffffffu, upto - mine, src)) * kRowsItem;
      r.q0 = __shfl_sync(0xffffffffu, r.q0, src);
      r.rows = __shfl_sync(0xffffffffu, r.rows, src);
      r.k0 = __shfl_sync(0xffffffffu, r.k0, src);
      r.keys = __shfl_sync(0xffffffffu, r.keys, src);
      r.win = __shfl_sync(0xffffffffu, r.win, src);
      it.row0 = r.q0 + i;
      it.rows = min(kRowsItem, r.rows - i);
      it.pos = r.keys - r.rows + i;
      it.keys = r.keys;
      it.k0 = r.k0;
      it.win = a.causal ? r.win : 0;
      int lo, hi;
      key_tiles(a, r, i, it.rows, lo, hi);
      const int chunks = (hi - lo + a.chunk_tiles - 1) / a.chunk_tiles;
      if (split >= max(1, chunks)) continue;  // no such chunk of this tile
      it.split = chunks > 1 ? split : -1;
      const int from = lo + split * a.chunk_tiles, to = min(hi, from + a.chunk_tiles);
      auto part = [&](int g, int& l, int& h) {
        const int rows = min(kRowsTile, it.rows - g * kRowsTile);
        l = h = 0;
        if (rows > 0) key_tiles(a, r, i + g * kRowsTile, rows, l, h);
        l = max(l, from);
        h = min(h, to);
      };
      part(0, it.lo0, it.hi0);
      part(1, it.lo1, it.hi1);
      // an empty tile stands at the other's first key tile
      if (it.lo0 >= it.hi0) it.lo0 = it.hi0 = it.lo1 < it.hi1 ? it.lo1 : from;
      if (it.lo1 >= it.hi1) it.lo1 = it.hi1 = it.lo0;
    }
    const uint32_t slot = n % kItems;
    bool ok = true;
    if (n >= kItems)
      ok = bar_wait(sh->item_empty + slot, ((n / kItems) - 1) & 1u, &sh->abort_flag, a);
    if (!__all_sync(0xffffffffu, ok)) break;
    if (lane == 0) {
      sh->items[slot] = it;
      bar_arrive(sh->item_full + slot);
    }
    __syncwarp();
    ++n;
    if (it.head < 0) break;
  }
  // the last CTA to get here clears the counters for the next call
  if (lane == 0) {
    __threadfence();
    if (atomicInc(a.done, gridDim.x - 1) == gridDim.x - 1) atomicExch(a.taken, 0u);
  }
}

// ------------------------------------------------------------------ softmax
//
// A thread per row, its 128 logits in registers.
__device__ void softmax_role(const PrefillArgs& a, Shared* sh, uint32_t tmem, int warp) {
  volatile int* abort_flag = &sh->abort_flag;
  const int lane = threadIdx.x & 31, quad = warp & 3, g = warp >> 2;
  const int r = quad * 32 + lane;  // row of the tile
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t t_s = tmem + lanes + g * kKeys, t_o = tmem + lanes + 2 * kKeys + g * kDv;
  // logits in log2 units: s * scale, with the sign (or zero) applied to s first
  const float sign = a.sm_scale < 0.f ? -1.f : a.sm_scale == 0.f ? 0.f : 1.f;
  const float scale = sign != 0.f ? fabsf(a.sm_scale) * kLog2e : 1.f;
  ItemReader reader(sh);
  Item it{};
  uint32_t n = 0;  // key tiles seen
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = bar_wait(bar, parity & 1u, abort_flag, a);
    return __all_sync(0xffffffffu, ok);
  };
  while (reader.next_warp(it, a)) {
    const int tile_rows = min(kRowsTile, it.rows - g * kRowsTile);
    const int lo = g ? it.lo1 : it.lo0, hi = g ? it.hi1 : it.hi0;
    if (tile_rows <= 0) continue;
    const int row = g * kRowsTile + r, p = it.pos + row;
    const int last_key = a.causal ? min(p, it.keys - 1) : it.keys - 1;
    const int first_key = it.win > 0 ? p - it.win + 1 : 0;
    // the tile's rows all see the keys [all_lo, all_hi]
    const int all_hi = a.causal ? it.pos + g * kRowsTile : it.keys - 1;
    const int all_lo = it.win > 0 ? it.pos + g * kRowsTile + tile_rows - it.win : 0;
    float m = kMInit, l = 0.f;
    for (int j = lo; j < hi; ++j, ++n) {
      if (!wait(sh->s_full + g, n)) return;
      fence_after();
      const int k0 = j * kKeys;
      if (k0 + kKeys - 1 > all_hi || k0 < all_lo || sign != 1.f) {
        // some row does not see the whole tile: mask S where it stands (masking
        // the registers costs the loop more than the two TMEM trips cost here)
#pragma unroll 1
        for (int c = 0; c < kKeys; c += 32) {
          uint32_t s[32];
          tmem_ld32(t_s + c, s);
          tmem_wait_ld<32>(s);
          const int last = last_key - k0 - c, first = first_key - k0 - c;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = __uint_as_float(s[e]) * sign;
            s[e] = e > last || e < first ? 0xff800000u : __float_as_uint(x);
          }
          tmem_st32(t_s + c, s);
        }
        tmem_wait_st();
      }
      uint32_t s[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) tmem_ld32(t_s + c, s + c);
      tmem_wait_ld<kKeys>(s);
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c]);
#pragma unroll
      for (int e = 4; e < kKeys - 4; e += 8)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mx[c] = max3(mx[c], __uint_as_float(s[e + c]), __uint_as_float(s[e + 4 + c]));
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(s[kKeys - 4 + c]));
      const float ms = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      const bool move = ms > m + kTh;
      if (__any_sync(0xffffffffu, move)) {
        const float f = move ? ex2(m - ms) : 1.f;
        if (move) m = ms;
        l *= f;
        if (j > lo) {  // O holds something: the MMA in front of this one must be done
          if (!wait(sh->o_done + g, n - 1)) return;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < kDv; c += 16) {
            uint32_t o[16];
            tmem_ld16(t_o + c, o);
            tmem_wait_ld<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(t_o + c, o);
          }
        }
      }
      // P over the columns of S, two keys a column
      const uint64_t scale2 = pack2(scale, scale), m2 = pack2(-m, -m);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int k = c * 32 + e * 2;
          float p0, p1;
          unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale2, m2), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
          w[e] = bf16x2(p0, p1);
        }
        tmem_st16(t_s + c * 16, w);
        if (c == 1) {  // the first 64 keys: P V starts on them
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(sh->p_half + g);
        }
      }
      float l0, l1;
      unpack2(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(sh->p_full + g);
    }
    // the rows' outputs: final, or this chunk's partial
    const bool any = lo < hi;
    if (any && !wait(sh->o_done + g, n - 1)) return;
    fence_after();
    const float inv = l > 0.f ? 1.f / l : l;  // no key: 0; NaN stays
    const int64_t at = static_cast<int64_t>(it.row0 + row) * a.heads + it.head;
    const bool live = r < tile_rows;
    const bool final = it.split < 0;
    float* part = a.part_o + static_cast<int64_t>(final ? 0 : it.split) * a.rows * a.heads * kDv;
#pragma unroll 1
    for (int c = 0; c < kDv; c += 32) {
      uint32_t o[32];
      __syncwarp();
      if (any) {
        tmem_ld32(t_o + c, o);
        tmem_wait_ld<32>(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
      // Four lanes exchange 16-byte pieces, so that a store writes 64 bytes of
      // each of eight rows and not 16 of thirty-two (a quarter of the accesses).
      auto put = [&](const uint32_t* w, char* base, int64_t row_bytes) {
        uint32_t v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = w[e];
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          const bool hi = (lane & d) != 0;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (p & d) continue;  // piece p and piece p + d
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t& keep = v[p * 4 + e];
              uint32_t& give = v[(p + d) * 4 + e];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? keep : give, d);
              if (hi) keep = got;
              else give = got;
            }
          }
        }
        // piece k is now this lane's piece (lane & 3) of row 4 (lane / 4) + k
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = quad * 32 + (lane & ~3) + k;
          if (rr < tile_rows)
            *reinterpret_cast<uint4*>(base + rr * row_bytes + (lane & 3) * 16) =
                make_uint4(v[k * 4], v[k * 4 + 1], v[k * 4 + 2], v[k * 4 + 3]);
        }
      };
      const int64_t at0 = static_cast<int64_t>(it.row0 + g * kRowsTile) * a.heads + it.head;
      if (final) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        put(w, reinterpret_cast<char*>(a.out + at0 * kDv + c), static_cast<int64_t>(a.heads) * kDv * 2);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          put(o + h * 16, reinterpret_cast<char*>(part + at0 * kDv + c + h * 16),
              static_cast<int64_t>(a.heads) * kDv * 4);
      }
    }
    __syncwarp();
    if (any) {
      fence_before();
      if (lane == 0) bar_arrive(sh->o_free + g);
    }
    if (live) {
      const float log2_sum = l == 0.f ? -INFINITY : m + __log2f(l);
      if (it.split >= 0)
        a.part_lse[static_cast<int64_t>(it.split) * a.rows * a.heads + at] = log2_sum;
      else if (a.lse)
        a.lse[at] = log2_sum * kLn2;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill(const __grid_constant__ PrefillArgs a, const __grid_constant__ CUtensorMap tq,
            const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tr,
            const __grid_constant__ CUtensorMap tv) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_s = smem;
  uint8_t* ring = smem + kQBytes;
  Shared* sh = reinterpret_cast<Shared*>(smem + kQBytes + kRing * kUnit);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (su32(smem) % 1024u) {  // the swizzled tiles need it
    if (tid == 0) atomicOr(a.status, PDA_STATUS_SMEM_MISALIGNED);
    return;
  }
  if (tid == 0) {
    for (int g = 0; g < 2; ++g) {
      bar_init(sh->q_full + g, 1);
      bar_init(sh->q_empty + g, 1);
      bar_init(sh->s_full + g, 1);
      bar_init(sh->p_half + g, kSoftmaxWarps / 2);
      bar_init(sh->p_full + g, kSoftmaxWarps / 2);
      bar_init(sh->o_done + g, 1);
      bar_init(sh->o_free + g, kSoftmaxWarps / 2);
    }
    for (int u = 0; u < kRing; ++u) {
      bar_init(sh->full + u, 1);
      bar_init(sh->empty + u, 1);
      bar_init(sh->landed + u, 1);
    }
    for (int s = 0; s < kItems; ++s) {
      bar_init(sh->item_full + s, 1);
      bar_init(sh->item_empty + s, kReaders);
    }
    bar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&sh->tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh->tmem;
  // registers: 200 a thread for the softmax, 96 for the others; together less
  // than the 168 x 384 of the launch
  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
  }
  if (warp < kSoftmaxWarps) {
    softmax_role(a, sh, tmem, warp);
  } else if (warp == kLoadWarp) {
    if (lane == 0) load_role(a, sh, q_s, ring, &tq, &tk, &tr, &tv);
  } else if (warp == kMmaWarp) {
    if (elect_one()) mma_role(a, sh, q_s, ring);
  } else if (warp == kClearWarp) {
    clear_role(a, sh, ring);
  } else {
    work_role(a, sh);
  }
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

// ------------------------------------------------------------ join of chunks
//
// One warp per (row, head): four output channels a lane, the chunks' weights
// 2^(lse_s - max) summed in order. Bound: reading the partials (L2).
__global__ void __launch_bounds__(256) prefill_join(const __grid_constant__ PrefillArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t row = item / a.heads;
  // the last request that starts at or before the row
  int b = 0, top = a.batch - 1;
  while (b < top) {
    const int mid = (b + top + 1) >> 1;
    if (__ldg(a.qo_indptr + mid) <= row) b = mid;
    else top = mid - 1;
  }
  const Request r = request_of(a, b);
  const int64_t i = row - r.q0;
  int chunks = 0;
  if (row < a.rows && i >= 0 && i < r.rows) {
    int lo, hi;
    const int i0 = static_cast<int>(i) / kRowsItem * kRowsItem;
    key_tiles(a, r, i0, min(kRowsItem, r.rows - i0), lo, hi);
    chunks = (hi - lo + a.chunk_tiles - 1) / a.chunk_tiles;
  }
  // all of this overlaps the first kernel's tail; its partials are read below
  // (every thread waits, so that what follows this kernel follows both)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (chunks <= 1) return;  // the only chunk wrote the result, or not a row
  const int64_t stride = static_cast<int64_t>(a.rows) * a.heads;
  float m = -INFINITY;
  for (int s = lane; s < chunks; s += 32) m = fmaxf(m, a.part_lse[s * stride + item]);
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < chunks; ++s) {
    const float x = a.part_lse[s * stride + item];
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (s * stride + item) * kDv + lane * 4);
    const float w = x == -INFINITY ? 0.f : exp2f(x - m);
    sum += w;
    if (w != 0.f) {  // a chunk without a visible key counts for nothing
      o[0] = fmaf(w, v.x, o[0]);
      o[1] = fmaf(w, v.y, o[1]);
      o[2] = fmaf(w, v.z, o[2]);
      o[3] = fmaf(w, v.w, o[3]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : sum;
  *reinterpret_cast<uint2*>(a.out + item * kDv + lane * 4) =
      make_uint2(bf16x2(o[0] * inv, o[1] * inv), bf16x2(o[2] * inv, o[3] * inv));
  if (lane == 0 && a.lse) a.lse[item] = sum == 0.f ? -INFINITY : (m + __log2f(sum)) * kLn2;
}

}  // namespace
}  // namespace pda

extern "C" int pda_prefill_plan(const pda_plan_t* plan, int32_t rows, int32_t tokens,
                                pda_prefill_plan_t* out_plan, size_t* scratch_bytes) {
  if (!plan || !out_plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  if (plan->head_dim != pda::kQDim + 384 || plan->num_kv_heads != 1) return PDA_ERR_UNSUPPORTED;
  // (token and row numbers of whole tiles stay int32)
  if (rows < 1 || tokens < 1 || rows > INT_MAX - 512 || tokens > INT_MAX - 512 ||
      plan->batch > pda::kMaxBatch)
    return PDA_ERR_INVALID;
  pda_prefill_plan_t p;
  std::memset(&p, 0, sizeof p);
  p.magic = PDA_PREFILL_MAGIC;
  p.struct_bytes = sizeof p;
  p.num_qo_heads = plan->num_qo_heads;
  p.batch = plan->batch;
  p.max_kv_len = plan->max_kv_len;
  p.num_sms = plan->num_sms;
  p.device = plan->device;
  p.rows = rows;
  p.tokens = tokens;
  // 256-row tiles of all requests: a request's last one may hold one row
  const int64_t tiles = std::min<int64_t>(
      rows, (static_cast<int64_t>(rows) + static_cast<int64_t>(pda::kRowsItem - 1) * plan->batch) /
                pda::kRowsItem);
  p.tiles = static_cast<int32_t>(tiles);
  // Key chunks. With at most half as many items (heads x tiles, by the capacities)
  // as SMs, as many chunks as fit them once, of at least two key tiles (40 rows on
  // up to 700 keys, 4 heads: one chunk 17.7, three of two tiles 13.5, six of one 13.2
  // us). More chunks than SMs cost more than they balance (257 rows on 2157 keys,
  // 16 heads, 96 items: one chunk 39, two 51, three 44 us; 512 rows on 4012 keys, 32
  // items: 2 / 4 / 6 chunks 41 / 30 / 41 us).
  const int64_t items = tiles * plan->num_qo_heads;
  const int64_t max_tiles =
      (std::min<int64_t>(plan->max_kv_len, tokens) + pda::kKeys - 1) / pda::kKeys;
  int64_t splits = std::max<int64_t>(1, plan->num_sms / std::max<int64_t>(1, items));
  splits = std::min<int64_t>(splits, std::max<int64_t>(1, max_tiles / 2));
  const int64_t chunk = (max_tiles + splits - 1) / splits;
  splits = (max_tiles + chunk - 1) / chunk;
  p.splits = static_cast<int32_t>(splits);
  p.chunk_tokens = static_cast<int32_t>(chunk * pda::kKeys);
  p.wait_limit_us = plan->wait_limit_us;
  p.inject = plan->inject;
  p.scratch_bytes = pda::kStatusHeaderBytes;
  if (splits > 1) {
    const int64_t cells = splits * rows * plan->num_qo_heads;
    p.scratch_bytes += (cells * 4 + 255) / 256 * 256 + cells * pda::kDv * 4;
  }
  // (chunk_tokens is an int32: max_kv_len within 127 of 2^31 would pass it)
  if (chunk * pda::kKeys > INT_MAX || items * splits > INT_MAX) return PDA_ERR_INVALID;
  *out_plan = p;
  if (scratch_bytes) *scratch_bytes = static_cast<size_t>(p.scratch_bytes);
  return PDA_OK;
}

extern "C" int pda_mla_prefill(const pda_prefill_plan_t* plan, const void* q, int64_t q_stride_row,
                               int64_t q_stride_head, const void* k, const void* v,
                               int64_t kv_stride_token, int64_t kv_stride_head, const void* k_rope,
                               int64_t k_rope_stride, const int32_t* qo_indptr,
                               const int32_t* tok_indptr, const int32_t* window, int32_t causal,
                               float sm_scale, void* out, float* lse, void* scratch,
                               pda_stream_t stream) {
  using namespace pda;
  if (!plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PREFILL_MAGIC || plan->struct_bytes != sizeof(pda_prefill_plan_t))
    return PDA_ERR_PLAN;
  if (!q || !k || !v || !k_rope || !qo_indptr || !tok_indptr || !out) return PDA_ERR_NULL;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return PDA_ERR_SCRATCH;
  if (window && !causal) return PDA_ERR_UNSUPPORTED;
  if (q_stride_row < kQDim || q_stride_head < kQDim || kv_stride_token < kNope ||
      kv_stride_head < kNope || k_rope_stride < kRope)
    return PDA_ERR_INVALID;
  auto a16 = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
  auto a4 = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 4 == 0; };
  if (!a16(q) || !a16(k) || !a16(v) || !a16(k_rope) || !a16(out) || !a4(lse) || !a4(qo_indptr) ||
      !a4(tok_indptr) || !a4(window) || q_stride_row % 8 || q_stride_head % 8 ||
      kv_stride_token % 8 || kv_stride_head % 8 || k_rope_stride % 8)
    return PDA_ERR_ALIGNMENT;
  if (plan->batch == 0) return PDA_OK;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  PrefillArgs a = {};
  a.qo_indptr = qo_indptr;
  a.tok_indptr = tok_indptr;
  a.window = window;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  char* base = static_cast<char*>(scratch);
  const int64_t cells = static_cast<int64_t>(plan->splits) * plan->rows * plan->num_qo_heads;
  a.status = reinterpret_cast<uint32_t*>(base);
  a.taken = a.status + 16;
  a.done = a.status + 17;
  a.part_lse = reinterpret_cast<float*>(base + kStatusHeaderBytes);
  a.part_o = reinterpret_cast<float*>(base + kStatusHeaderBytes + (cells * 4 + 255) / 256 * 256);
  a.wait_limit_ns = static_cast<uint64_t>(plan->wait_limit_us) * 1000ull;
  a.sm_scale = sm_scale;
  a.heads = plan->num_qo_heads;
  a.batch = plan->batch;
  a.max_kv_len = plan->max_kv_len;
  a.rows = plan->rows;
  a.tokens = plan->tokens;
  a.causal = causal ? 1 : 0;
  a.splits = plan->splits;
  a.chunk_tiles = plan->chunk_tokens / kKeys;
  a.inject = plan->inject;
  CUtensorMap tq, tk, tr, tv;
  if (!make_map3(&tq, q, kQDim, a.heads, a.rows, q_stride_head, q_stride_row, 64, 1, kRowsTile) ||
      !make_map3(&tk, k, kNope, a.heads, a.tokens, kv_stride_head, kv_stride_token, 64, 1, kKeys) ||
      !make_map3(&tr, k_rope, kRope, 1, a.tokens, k_rope_stride, k_rope_stride, 64, 1, kKeys) ||
      !make_map3(&tv, v, kDv, a.heads, a.tokens, kv_stride_head, kv_stride_token, 64, 1, 64))
    return PDA_ERR_CUDA;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(prefill),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  const int64_t items = static_cast<int64_t>(plan->tiles) * a.heads * a.splits;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, plan->num_sms));
  prefill<<<grid, kThreads, kSmem, s>>>(a, tq, tk, tr, tv);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  if (a.splits > 1) {
    const int64_t warps = static_cast<int64_t>(a.rows) * a.heads;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, prefill_join, a) != cudaSuccess) {
      cudaGetLastError();
      return PDA_ERR_CUDA;
    }
  }
  return PDA_OK;
}
