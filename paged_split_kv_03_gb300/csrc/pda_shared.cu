// pda_shared.cu -- decode attention for requests that share a long prefix: the
// prefix's keys and values meet the rows of all of them at once, on the
// 5th-generation tensor cores; each request's own tokens and the join are pda_own.cu's.
//
// Mathematics: with the keys of a row split into those of the prefix, in segments s,
// and its own, in chunks c, each part gives a normalised output o and a log2 sum
// x of its weights; out = sum 2^(x - X) o with X the log2 sum of all of them. A row
// of a group stands at or behind the prefix's end, so it sees all of it but for its
// window. A segment is flash attention: for 128 rows (query rows x heads of a GQA
// group, packed without gaps), over tiles of 128 keys, S = Q K^T, an online softmax
// in log2 units with a lazy maximum (moved when a logit passes it by more than 8, so
// weights stay <= 2^8, within the operands' range), O += P V. P is rounded to the
// operands' 16-bit type, l sums the unrounded weights in fp32.
//
// Types: bf16 caches run bf16 MMAs. E4M3 keys (head_dim 128 and 256) are operands as
// they are: an E4M3 query meets them directly, a bf16 row as the sum of two E4M3 terms
// of it times a power of two that takes its largest element to [224, 448): exact for
// elements from 2^-11 of that on, off by 2^-18 of it at most below. Values, and int8 keys
// and those of head_dim 64, are widened exactly to f16 and meet an f16 P (query). P in
// E4M3 terms would need no widening but four conversions for each pair of weights, 2048
// cycles a tile of 128 x 128 against the 1024 of its MMAs. Scales per tensor meet the
// logits and the output; scales per token and head meet S and P in fp32, the value
// scale as its log2, so that P <= 2^8 whatever the scale.
//
// Bound: the tensor cores from some 100 rows a kv head on, HBM below. Two row tiles
// (head_dim 64 and 128) share each key tile, so that one's softmax runs beside the other's
// MMAs; one row tile of 256 channels, or of few rows, has two S in flight instead. 256 rows
// on 128 keys of 128 channels are 1100 (E4M3 keys: 800) cycles of MMAs each for Q K^T and P V
// and 1024 of exponentials. A longer prefix adds (64 requests, 64 / 8 heads) 1466 TFLOP/s in
// bf16, 1556 in E4M3, 1044 with scales per token, 1179 in int8; 921 at head_dim 64, 852 to
// 1250 at 256; of 16 requests 6.5 TB/s. Around it an item costs its start, 8 us from the launch to the first S (the
// cut 3, the query 1.5 to 5, the first K), and 3 us for its parts. Work is cut over the CTAs
// by key tiles and not by items (see Cut): 16 items of 256 rows keep all SMs busy.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "pda.h"
#include "pda_cvt.cuh"
#include "pda_internal.h"
#include "pda_ptx.cuh"
#include "pda_shared.cuh"

namespace pda {
namespace {

constexpr float kTh = 8.0f;         // lazy rescale threshold, log2 units

constexpr int kUnit = 16384;   // bytes of a ring unit
constexpr int kItems = 3;      // slots of the segment ring
constexpr int kScales = 4;     // slots of the ring of per-token scales, a tile each
constexpr int kCoarse = 32;    // prefix entries, 32 groups each
constexpr int kMaxGroups = 32 * kCoarse;
constexpr int kTmemCols = 512;
constexpr int kO = 2 * kKeys;  // first TMEM column of O; two S in front of it

// One segment: key tiles [t0, t1) of an item.
struct Item {
  int head;    // kv head; -1: no more
  int row0;    // first packed row of the block (of the group: row x group + head)
  int rows;    // packed rows, 1..kRows
  int q0;      // the group's first row in q
  int b0, b1;  // its requests
  int t0, t1;
  int low;     // the first token of the prefix that a row sees, rounded down to a page
  int end;     // the prefix's end, tokens
  int table;   // offset of the prefix's pages in page_table
  int cut;     // the segment does not start its item: its partials go to the CTA's area
};

struct Shared {
  uint64_t q_full[2], q_empty[2], k_full[8], k_empty[8], v_full[8], v_empty[8], raw_full[4], raw_empty[4],
      sc_full[kScales], sc_empty[kScales], s_full[2], p_half[2], p_full[2], o_done[2], o_free[2], odd_done,
      item_full[kItems], item_empty[kItems], drain;
  uint32_t tmem;
  int abort_flag;
  Item items[kItems];
  int coarse[kCoarse];           // work in front of every 32 groups
  int coarse_items[kCoarse];     // items there
  int coarse_singles[kCoarse];   // tiles of single row tiles there
  int coarse_top[kCoarse];       // the highest bound there
  float2 rows[kTile];            // a row's power of two; then its maximum and sum in the odd tiles
};

// ------------------------------------------------------------ configuration
template <int D, bool k8, bool kI8, bool kTok>
struct Cfg {
  static constexpr int kG = D <= 128 ? 2 : 1;  // row tiles of an item
  static constexpr int kRows = kG * kTile;
  static constexpr bool kDirect = k8 && !kI8 && D >= 128;  // E4M3 keys as they are
  static constexpr int kQTerms = kDirect ? 2 : 1;
  // 16 KB units of a K tile (128 keys x 128 bytes) and of a V tile (kVKeys keys x D)
  static constexpr int kUK = kDirect ? D / 128 : D / 64;
  static constexpr int kUV = D / 64;
  static constexpr int kVKeys = 8192 / D;
  static constexpr int kQTile = kQTerms * kUK * kUnit;  // bytes of a row tile's query
  static constexpr int kQBytes = kG * kQTile;
  // rings of K and of V units
  static constexpr int kRK = D == 64 ? 4 : !k8 ? 5 : D == 256 && !kTok ? 4 : 3;
  static constexpr int kRV = D == 64 ? 4 : !k8 ? 5 : kDirect || D == 256 ? 4 : 3;
  // 8-bit caches: codes to widen land in raw slots of kRawKeys keys, as they lie in the cache
  static constexpr int kRawKeys = D <= 128 ? 128 : 64;
  static constexpr int kRawBytes = kRawKeys * D;
  static constexpr int kRawTile = kKeys / kRawKeys;  // slots of a K or V tile
  static constexpr int kRaw = !k8 ? 0 : D == 64 ? 4 : D == 128 && !(kDirect && kTok) ? 3 : 2;
  static constexpr int kScaleBytes = kTok ? (kScales * 3 + 2) * kKeys * 4 : 0;
  static constexpr int kRings = (kRK + kRV) * kUnit;
  static constexpr int kSmem = kQBytes + kRings + kRaw * kRawBytes + kScaleBytes +
                               static_cast<int>(sizeof(Shared));
  static constexpr int kSoft = 4 * kG;              // softmax warps, a thread per row
  static constexpr int kMmaWarp = kSoft, kWorkWarp = kSoft + 1, kProd0 = kSoft + 2;
  // warps that issue loads (see there), and warps that widen codes
  static constexpr int kProds = !k8 ? 6 : kDirect ? 2 : 1;
  static constexpr int kConv0 = kSoft + 4, kConv = !k8 ? 0 : kG == 1 ? 8 : 4;
  static constexpr int kWarps = kSoft + 4 + (k8 ? kConv : 4);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kReaders = kSoft + 1 + kProds + kConv;  // arrivals that free an item
  static_assert(kSmem <= 227 * 1024 && kSmem > 114 * 1024, "one CTA an SM");
  static_assert(kRK <= 8 && kRV <= 8 && kRaw <= 4, "barriers");
  // two row tiles hold V_j and K_{j+1} whole; a K tile is widened from all its raw slots
  static_assert(kG == 1 || (kRK >= kUK && kRV >= kUV), "a tile fits");
  static_assert(!k8 || kRaw >= kRawTile, "a raw tile fits");
};

struct ItemReader {
  Shared* sh;
  uint32_t n = 0;
  __device__ explicit ItemReader(Shared* s) : sh(s) {}
  // One thread: the next segment, or false after the last one (or an abort).
  __device__ bool next_one(Item& it, const SharedArgs& a) {
    const uint32_t slot = n % kItems;
    if (!bar_wait(sh->item_full + slot, (n / kItems) & 1u, &sh->abort_flag, a)) return false;
    it = sh->items[slot];
    bar_arrive(sh->item_empty + slot);
    ++n;
    return it.head >= 0;
  }
  // A whole warp (one arrival); warp-uniform.
  __device__ bool next_warp(Item& it, const SharedArgs& a) {
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

// 4-D tiled TMA load of one box (channel, slot, kv head, page).
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int c, int slot, int head,
                                         int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(slot), "r"(head), "r"(page), "r"(su32(bar))
      : "memory");
}

// The order in which the K and V tiles of a segment of n are needed: with two row tiles
// K0 V0 K1 V1 ..., with two S of one row tile K0 K1 V0 K2 V1 ... . Place i of 2n ->
// (V?, tile).
template <int kG>
__device__ __forceinline__ void tile_order(int i, int n, int& v, int& j) {
  if constexpr (kG == 2) {
    v = i & 1;
    j = i >> 1;
  } else {
    if (i == 2 * n - 1) v = 1, j = n - 1;
    else if (i == 0) v = 0, j = 0;
    else v = (i & 1) ^ 1, j = v ? i / 2 - 1 : (i + 1) / 2;
  }
}

// ------------------------------------------------------------------- loads
//
// Even warps load K, odd ones V, a unit (or raw slot) a warp in turn; one warp loads both
// where both are widened, as they share the raw slots. A unit's boxes (a page's tokens x
// 128 bytes, or a head's codes) are its warp's lanes'. A page behind the prefix, or in
// front of what any row sees, is one past the cache: such a box reads as zeros.
//
// A wait tells a slot's rounds apart by their parity only, so no warp may stand two
// rounds in front of what has been read: with at least as many slots as warps in turn,
// the unit in front of a warp's unit was let in behind the round before the last one.
template <class C, int D, bool k8>
__device__ __forceinline__ void load_role(const SharedArgs& a, Shared* sh, uint8_t* rings, uint8_t* raw,
                                          const CUtensorMap* tk, const CUtensorMap* tv, int pw) {
  constexpr bool kBoth = k8 && !C::kDirect;
  volatile int* abort_flag = &sh->abort_flag;
  const int lane = threadIdx.x & 31;
  const uint32_t turn = kBoth ? 0u : static_cast<uint32_t>(pw >> 1);
  constexpr uint32_t kTurns = kBoth ? 1 : C::kProds / 2;
  static_assert(C::kRK >= kTurns && C::kRV >= kTurns, "slots for all warps in turn");
  ItemReader reader(sh);
  Item it{};
  bool alive = (a.inject & PDA_INJECT_WITHHOLD_KV) == 0u;
  // where this warp's tiles go: a ring, or raw slots
  const int side = kBoth ? 0 : pw & 1;  // 1: V
  const bool to_raw = kBoth || (k8 && side);
  const uint32_t slots = to_raw ? (C::kRaw ? C::kRaw : 1) : side ? C::kRV : C::kRK;
  uint64_t* full = to_raw ? sh->raw_full : side ? sh->v_full : sh->k_full;
  uint64_t* empty = to_raw ? sh->raw_empty : side ? sh->v_empty : sh->k_empty;
  const uint32_t base = su32(to_raw ? raw : rings + (side ? C::kRK * kUnit : 0));
  const uint32_t slot_bytes = to_raw ? C::kRawBytes : kUnit;
  const int units = to_raw ? C::kRawTile : side ? C::kUV : C::kUK;
  const int unit_keys = to_raw ? C::kRawKeys : side ? C::kVKeys : kKeys;
  const int P = a.page_size;
  const int rows = min(P, unit_keys), boxes = unit_keys / rows;  // powers of two
  const int atoms = !k8 && side ? C::kUV : 1;
  const int at = lane % boxes, atom = lane / boxes;
  const uint32_t box = atom * (unit_keys * 128) + at * rows * (to_raw ? D : 128);
  const bool mine = atom < atoms;
  const int per = kBoth ? 2 * units : units;  // this warp's kind of units a key tile
  // unit k of the segment: its tile, its place in it, and K or V
  auto unit_of = [&](uint32_t k, int n, int& v, int& j, int& c) {
    if constexpr (kBoth) {
      tile_order<C::kG>(static_cast<int>(k / units), n, v, j);
    } else {
      v = side;
      j = static_cast<int>(k / units);
    }
    c = static_cast<int>(k % units);
  };
  auto first_key = [&](int j, int c) {
    return (it.t0 + j) * kKeys + (to_raw || side ? c * unit_keys : 0) + at * rows;
  };
  // the page of this lane's box (the lookup of a unit is under way while the one in front
  // of it waits for its place)
  auto page_of = [&](uint32_t k, int n) {
    int v, j, c;
    unit_of(k, n, v, j, c);
    const int key = first_key(j, c);
    if (!mine || key < it.low || key >= it.end) return a.num_pages;
    return __ldg(a.page_table + it.table + key / P);
  };
  uint32_t t = 0, last = 0;  // key tiles in front of the segment; units up to here
  while (alive && reader.next_warp(it, a)) {
    const uint32_t n = it.t1 - it.t0, u0 = t * per, u1 = u0 + n * per;
    uint32_t u = u0 + (turn + kTurns - u0 % kTurns) % kTurns;
    int page = u < u1 ? page_of(u - u0, n) : 0;
    for (; u < u1; u += kTurns) {
      int v, j, c, ahead = 0;
      unit_of(u - u0, n, v, j, c);
      if (u + kTurns < u1) ahead = page_of(u + kTurns - u0, n);
      const uint32_t slot = u % slots;
      int good = 1;
      if (lane == 0) {
        good = bar_wait(empty + slot, ((u / slots) & 1u) ^ 1u, abort_flag, a);
        if (good) bar_expect_tx(full + slot, slot_bytes);
      }
      if (!__shfl_sync(0xffffffffu, good, 0)) {
        alive = false;
        break;
      }
      if (page < 0 || page > a.num_pages) page = a.num_pages;
      const int chan = to_raw ? 0 : k8 ? c * 128 : (side ? atom : c) * 64;
      if (mine)
        tma_page(base + slot * slot_bytes + box, v ? tv : tk, chan, first_key(j, c) % P, it.head, page,
                 full + slot);
      page = ahead;
      last = u + 1;
    }
    t += n;
    if (alive) last = u1;
  }
  // every box issued must have landed before the CTA can exit: the last unit of each slot,
  // whichever warp's it is (after a wait that ran out another warp's may not be coming)
  if (lane == 0)
    for (uint32_t k = last > slots ? last - slots : 0u; k < last; ++k)
      if (alive || k % kTurns == turn) bar_drain(full + k % slots, (k / slots) & 1u);
}

// -------------------------------------------------------------------- MMAs
template <class C, int D, bool k8>
__device__ __forceinline__ void mma_role(const SharedArgs& a, Shared* sh, uint8_t* q_s, uint8_t* rings) {
  volatile int* abort_flag = &sh->abort_flag;
  constexpr uint32_t tmem = 0;  // all columns are ours: they start at 0
  constexpr uint32_t fmt = k8 ? 0u : 1u;
  const uint32_t id_s = idesc(fmt, 0, kKeys), id_o = idesc(fmt, 0, D, 1u);
  const uint64_t q_desc = sdesc(su32(q_s), 16, 1024), k_desc = sdesc(su32(rings), 16, 1024),
                 v_desc = sdesc(su32(rings) + C::kRK * kUnit, C::kVKeys * 128, 1024);
  const int terms = C::kDirect && !a.q8 ? 2 : 1;
  ItemReader reader(sh);
  Item it{};
  uint32_t t = 0;               // key tiles in front of the segment
  uint32_t seq0 = 0, seq1 = 0;  // tiles so far of each softmax warpgroup
  uint32_t qn0 = 0, qn1 = 0;    // queries so far of each row tile
  uint32_t on0 = 0, on1 = 0;    // segments so far of each O
  bool alive = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return alive = bar_try(bar, parity & 1u) || bar_wait_slow(bar, parity & 1u, abort_flag, a);
  };
  // S = Q K^T of row tile g and key tile j (of all the CTA's) into S buffer b
  auto qk = [&](int g, int b, uint32_t j, bool release) {
#pragma unroll
    for (int c = 0; c < C::kUK; ++c) {
      const uint32_t u = j * C::kUK + c, slot = u % C::kRK;
      if (!wait(sh->k_full + slot, u / C::kRK)) return;
      if (c == 0) fence_after();
      const uint64_t kd = k_desc + slot * (kUnit / 16);
      for (int h = 0; h < (C::kDirect ? terms : 1); ++h) {
        const uint64_t qd = q_desc + (g * (C::kQTile / 16) + (h * C::kUK + c) * (kUnit / 16));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma<C::kDirect>(tmem + b * kKeys, qd + kk * 2, kd + kk * 2, id_s, (c | kk | h) != 0);
      }
      if (release) mma_commit(sh->k_empty + slot);
    }
    mma_commit(sh->s_full + b);
  };
  // O_g += P V of key tile j, P over S buffer b
  auto pv = [&](int g, int b, uint32_t j, uint32_t parity, bool first, bool release) {
    if (!wait(sh->p_half + b, parity)) return;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {  // 16 keys a step
      constexpr int kSteps = C::kVKeys / 16;
      const uint32_t u = j * C::kUV + kk / kSteps, slot = u % C::kRV;
      if (kk % kSteps == 0 && !wait(sh->v_full + slot, u / C::kRV)) return;
      if (kk == 4 && !wait(sh->p_full + b, parity)) return;
      if (kk % kSteps == 0 || kk == 4) fence_after();
      mma_ts(tmem + kO + g * D, tmem + b * kKeys + kk * 8,
             v_desc + slot * (kUnit / 16) + (kk % kSteps) * 128, id_o, kk || !first ? 1u : 0u);
      if (release && kk % kSteps == kSteps - 1) mma_commit(sh->v_empty + slot);
    }
    mma_commit(sh->o_done + b);
  };
  while (alive && reader.next_one(it, a)) {
    const int n = it.t1 - it.t0;
    if (C::kG == 2 && it.rows > kTile) {
      // two row tiles take turns
      for (int j = -1; j < n && alive; ++j) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t& seq = g ? seq1 : seq0;
          uint32_t& qn = g ? qn1 : qn0;
          uint32_t& on = g ? on1 : on0;
          if (j >= 0) {
            if (j == 0 && !wait(sh->o_free + g, on++ ^ 1u)) break;  // the last segment's O is read
            pv(g, g, t + j, seq, j == 0, g == 1);
            if (!alive) break;
            ++seq;
          }
          if (j + 1 < n) {
            if (j + 1 == 0 && !wait(sh->q_full + g, qn++)) break;
            qk(g, g, t + j + 1, g == 1);
            if (!alive) break;
            if (j + 2 == n) mma_commit(sh->q_empty + g);
          }
        }
      }
    } else {
      // One row tile, S one key tile ahead of P. With kG = 2 the key tiles take turns
      // between both softmax warpgroups and two O, which the first adds up at the end;
      // with kG = 1 between two S of the one warpgroup.
      auto buf = [&](int j) { return C::kG == 2 ? static_cast<uint32_t>(j & 1) : (seq0 + j) & 1u; };
      const uint32_t s0 = seq0, s1 = seq1;
      const uint32_t b0 = buf(0), b1 = buf(1);
      if (!wait(sh->q_full, qn0++)) break;
      qk(0, b0, t, true);
      if (alive && n > 1) qk(0, b1, t + 1, true);
      if (alive && n <= 2) mma_commit(sh->q_empty);
      for (int j = 0; j < n && alive; ++j) {
        const uint32_t b = j & 1 ? b1 : b0;
        const int g = C::kG == 2 ? j & 1 : 0;
        if (j <= g && !wait(sh->o_free + g, (g ? on1++ : on0++) ^ 1u)) break;
        const uint32_t parity = C::kG == 2 ? (g ? s1 : s0) + (j >> 1) : (s0 + j) >> 1;
        pv(g, b, t + j, parity, j <= g, true);
        if (alive && j + 2 < n) {
          qk(0, b, t + j + 2, true);
          if (j + 3 == n) mma_commit(sh->q_empty);
        }
      }
      if constexpr (C::kG == 2) {
        seq0 += (n + 1) >> 1;
        seq1 += n >> 1;
      } else {
        seq0 += n;
      }
    }
    t += n;
  }
  // nothing issued may still run when TMEM is released
  mma_commit(&sh->drain);
  bar_drain(&sh->drain, 0);
}

// ------------------------------------------------------ codes widened to f16
//
// A raw slot's codes, 16 at a time, into the units of a ring, and the tile's scales per
// token (loaded a tile ahead) into a ring of their own.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, bool i8) {
  uint4 r;
  widen4(lo, r.x, r.y, i8);
  widen4(hi, r.z, r.w, i8);
  return r;
}

template <class C, int D, bool kI8, bool kTok>
__device__ __forceinline__ void widen_role(const SharedArgs& a, Shared* sh, uint8_t* rings,
                                           const uint8_t* raw, float* scales) {
  constexpr int kT = 32 * C::kConv;  // threads
  const int t = threadIdx.x - 32 * C::kConv0, lane = threadIdx.x & 31;
  ItemReader reader(sh);
  Item it{};
  uint32_t xk = 0, xv = 0, y = 0, s = 0;  // units of K and of V, raw slots, tiles of scales
  constexpr uint32_t RR = C::kRaw;
  constexpr int kRowPieces = D / 16;
  const int P = a.page_size;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = bar_wait(bar, parity & 1u, &sh->abort_flag, a);
    return __all_sync(0xffffffffu, ok);
  };
  auto hand_over = [&](uint64_t* bar) {
    fence_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  };
  // 16 codes at `src` to the 32 bytes from 16-byte piece `chunk` on of row r
  auto put = [&](const uint8_t* src, uint8_t* dst, int r, int chunk, int flip) {
    const uint4 w = *reinterpret_cast<const uint4*>(src);
    const uint4 lo = widen8(w.x, w.y, kI8), hi = widen8(w.z, w.w, kI8);
    *reinterpret_cast<uint4*>(dst + sw128(r, (chunk + flip) * 16)) = flip ? hi : lo;
    *reinterpret_cast<uint4*>(dst + sw128(r, (chunk + 1 - flip) * 16)) = flip ? lo : hi;
  };
  const float qk = a.sm_scale * kLog2e;
  // of this thread's key: the scales of the next tile, the page of the one behind it
  float ks = 1.f, vs = 1.f;
  int page = -1;
  auto load_page = [&](int tile) {
    const int key = tile * kKeys + t;
    // (as load_role: pages in front of what any row sees may hold anything)
    page = t < kKeys && key >= it.low && key < it.end ? __ldg(a.page_table + it.table + key / P) : -1;
  };
  auto load_scales = [&](int tile) {
    ks = vs = 1.f;
    if (page >= 0 && page < a.num_pages) {
      const int64_t at = (static_cast<int64_t>(page) * P + (tile * kKeys + t) % P) * a.hkv + it.head;
      ks = __ldg(a.k_scale + at);
      vs = __ldg(a.v_scale + at);
    }
  };
  while (reader.next_warp(it, a)) {
    const int n = it.t1 - it.t0;
    if constexpr (kTok) {
      load_page(it.t0);
      load_scales(it.t0);
      load_page(it.t0 + 1);
    }
    for (int i = 0; i < 2 * n; ++i) {
      int v, j;
      tile_order<C::kG>(i, n, v, j);
      if (!v) {  // the K tiles come in order
        if constexpr (kTok) {
          const uint32_t slot = s % kScales;
          if (!wait(sh->sc_empty + slot, (s / kScales) ^ 1u)) return;
          if (t < kKeys) {
            float* to = scales + slot * 3 * kKeys;
            const float v2 = vs > 0.f ? vs : 1.f;
            to[t] = ks * qk;
            to[kKeys + t] = __log2f(v2);
            to[2 * kKeys + t] = __frcp_rn(v2);
          }
          __syncwarp();
          if (lane == 0) bar_arrive(sh->sc_full + slot);
          ++s;
          load_scales(it.t0 + j + 1);  // (behind the segment: not used)
          load_page(it.t0 + j + 2);
        }
        if constexpr (!C::kDirect) {
          // a unit holds 64 channels of all keys, a raw slot all channels of its keys
          for (int h = 0; h < C::kRawTile; ++h)
            if (!wait(sh->raw_full + (y + h) % RR, (y + h) / RR)) return;
          for (int c = 0; c < C::kUK; ++c, ++xk) {
            const uint32_t slot = xk % C::kRK;
            if (!wait(sh->k_empty + slot, (xk / C::kRK) ^ 1u)) return;
            uint8_t* dst = rings + slot * kUnit;
#pragma unroll
            for (int p = 0; p < 512 / kT; ++p) {
              const int idx = p * kT + t, key = idx >> 2, piece = idx & 3;
              put(raw + (y + key / C::kRawKeys) % RR * C::kRawBytes + key % C::kRawKeys * D + c * 64 + piece * 16,
                  dst, key, piece * 2, 0);
            }
            hand_over(sh->k_full + slot);
          }
          if (lane == 0)
            for (int h = 0; h < C::kRawTile; ++h) bar_arrive(sh->raw_empty + (y + h) % RR);
          y += C::kRawTile;
        }
        continue;
      }
      constexpr int kUnits = C::kRawKeys / C::kVKeys;  // of a raw slot
      for (int h = 0; h < C::kRawTile; ++h, ++y) {
        if (!wait(sh->raw_full + y % RR, y / RR)) return;
        for (int c = 0; c < kUnits; ++c, ++xv) {
          const uint32_t slot = xv % C::kRV;
          if (!wait(sh->v_empty + slot, (xv / C::kRV) ^ 1u)) return;
          const uint8_t* src = raw + y % RR * C::kRawBytes + c * (C::kVKeys * D);
          uint8_t* dst = rings + (C::kRK + slot) * kUnit;
#pragma unroll
          for (int p = 0; p < 512 / kT; ++p) {
            const int idx = p * kT + t, r = idx / kRowPieces, piece = idx % kRowPieces, atom = piece >> 2;
            // (a row's atoms share banks: every other one writes its halves in turn)
            put(src + idx * 16, dst + atom * (C::kVKeys * 128), r, (piece & 3) * 2, atom & 1);
          }
          hand_over(sh->v_full + slot);
        }
        if (lane == 0) bar_arrive(sh->raw_empty + y % RR);
      }
    }
  }
}

// --------------------------------------------------------------- the work list
// The first 32 groups, a group a lane, and where each one's prefix stands in page_table: in
// front of the own pages of its first request that has some (nearly always its first).
template <int kG>
struct Look {
  Group r = {};
  Work<kG> w;
  int table = -1;
  // (`top`: the highest bound in front of the 32)
  __device__ __forceinline__ void at(const SharedArgs& a, int g, int& top) {
    r = {};
    table = -1;
    if (g < a.groups) r = group_of(a, g);
    if (a.groups > 1) no_overlap(r, g < a.groups, top);
    w = Work<kG>(a, r);
    if (!r.bad && r.b1 > r.b0) {
      const int own = __ldg(a.own_len + r.b0), page = __ldg(a.own_indptr + r.b0);
      if (own > 0) table = page;
    }
  }
};

template <int kG>
struct WorkList {
  Look<kG> look;
  int work = 0, items = 0, singles = 0;
  int lane_work = 0, lane_items = 0, lane_singles = 0;  // in front of this lane's group, among the 32
  uint32_t bits = 0u;
  int known = 0;  // the 32 groups that `look` holds
  Cut cut;
  __device__ __forceinline__ void sums(const SharedArgs& a, int lane, int& w32, int& i32, int& s32) {
    const int w = a.hkv * look.w.head(Cut()), i = a.hkv * look.w.blocks;
    const int s = look.w.single ? a.hkv * look.w.tiles : 0;
    int wx = w, ix = i, sx = s, last = 0;
    if (a.groups > 1) {
      wx = scan32(w, lane);
      ix = scan32(i, lane);
      sx = scan32(s, lane);
      last = 31;
    }
    lane_work = wx - w;
    lane_items = ix - i;
    lane_singles = sx - s;
    w32 = __shfl_sync(0xffffffffu, wx, last);
    i32 = __shfl_sync(0xffffffffu, ix, last);
    s32 = __shfl_sync(0xffffffffu, sx, last);
  }
  __device__ __forceinline__ int place(int w, int i, int s) const { return w - s * (kFull - cut.one) + i * cut.pay; }
  __device__ __forceinline__ int coarse(const Shared* sh, int c) const {
    return place(sh->coarse[c], sh->coarse_items[c], sh->coarse_singles[c]);
  }
  __device__ __forceinline__ void prepare(const SharedArgs& a, Shared* sh);
  __device__ __forceinline__ void run(const SharedArgs& a, Shared* sh);
};

// The cut (while the CTA sets up).
template <int kG>
__device__ __forceinline__ void WorkList<kG>::prepare(const SharedArgs& a, Shared* sh) {
  const int lane = threadIdx.x & 31;
  int w32, i32, s32, top = INT_MIN;
#pragma unroll 1
  for (int g0 = 0; g0 < a.groups; g0 += 32) {
    known = g0 >> 5;
    if (lane == 0) sh->coarse_top[known] = top;
    look.at(a, g0 + lane, top);
    bits |= look.r.bad;
    sums(a, lane, w32, i32, s32);
    if (lane == 0) {
      sh->coarse[known] = work;
      sh->coarse_items[known] = items;
      sh->coarse_singles[known] = singles;
    }
    work += w32;
    items += i32;
    singles += s32;
  }
  cut = Cut(a, work, singles, items);
  __syncwarp();
}

// This CTA's segments, in turn.
template <int kG>
__device__ __forceinline__ void WorkList<kG>::run(const SharedArgs& a, Shared* sh) {
  constexpr int kRows = kG * kTile;
  const int lane = threadIdx.x & 31, per = cut.per, pay = cut.pay;
  int w32, i32, s32;
  int pos = blockIdx.x * per;  // (a CTA too many stands at most `per` behind the end)
  const int stop = min(place(work, items, singles), pos + per);
  uint32_t n = 0;
  for (;;) {
    Item it = {};
    it.head = -1;
#pragma unroll 1
    while (pos < stop) {
      int c = 0, top = (a.groups + 31) / 32 - 1;
      while (c < top) {
        const int mid = (c + top + 1) >> 1;
        if (coarse(sh, mid) <= pos) c = mid;
        else top = mid - 1;
      }
      if (c != known) {
        known = c;
        int before = sh->coarse_top[c];
        look.at(a, 32 * c + lane, before);
        sums(a, lane, w32, i32, s32);
      }
      const int start = coarse(sh, c) + place(lane_work, lane_items, lane_singles);
      const int head = look.w.head(cut);
      const int src = __ffs(__ballot_sync(0xffffffffu, start + a.hkv * head > pos)) - 1;
      auto from = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
      const int blocks = from(look.w.blocks), tiles = from(look.w.tiles);
      const int last = from(look.w.weight(cut, look.w.blocks - 1));
      const uint32_t head_len = from(head), full = from(look.w.full(cut));
      uint32_t in = pos - from(start);
      const int h = in / head_len;
      in -= h * head_len;
      const int block = min(static_cast<int>(in / full), blocks - 1);
      in -= block * full;
      const uint32_t w = block == blocks - 1 ? last : kFull;
      // tiles that begin in front of a place of the item
      auto tiles_to = [&](uint32_t x) {
        return x <= static_cast<uint32_t>(pay) ? 0 : min(static_cast<int>((x - pay + w - 1) / w), tiles);
      };
      const uint32_t to = min(w * tiles + pay, in + (stop - pos));
      const int t0 = tiles_to(in), t1 = tiles_to(to);
      pos += to - in;
      if (t0 == t1) continue;
      const int rows = from(look.r.rows), tile0 = from(look.r.tile0);
      it.head = h;
      it.row0 = block * kRows;
      it.rows = min(kRows, rows * a.group - it.row0);
      it.q0 = from(look.r.q0);
      it.b0 = from(look.r.b0);
      it.b1 = from(look.r.b1);
      it.t0 = tile0 + t0;
      it.t1 = tile0 + t1;
      it.low = from(look.r.low);
      it.end = from(look.r.end);
      it.cut = t0 > 0;
      it.table = from(look.table);
#pragma unroll 1
      for (int b = it.b0; it.table < 0 && b < it.b1; b += 32) {
        const uint32_t has =
            __ballot_sync(0xffffffffu, b + lane < it.b1 && __ldg(a.own_len + min(b + lane, it.b1 - 1)) > 0);
        if (has) it.table = __ldg(a.own_indptr + b + __ffs(has) - 1);
      }
      it.table -= it.end / a.page_size;
      break;
    }
    const uint32_t slot = n % kItems;
    bool ok = true;
    if (n >= kItems) ok = bar_wait(sh->item_empty + slot, ((n / kItems) - 1) & 1u, &sh->abort_flag, a);
    if (!__all_sync(0xffffffffu, ok)) break;
    if (lane == 0) {
      sh->items[slot] = it;
      bar_arrive(sh->item_full + slot);
    }
    __syncwarp();
    ++n;
    if (it.head < 0) break;
  }
  // the first CTA says what is wrong with groups, and writes the cut down for the join
  // where the groups are too many for its lanes
  if (blockIdx.x) return;
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (lane == 0) {
    a.first[0] = per;
    a.first[1] = pay;
    a.first[2] = cut.one;
    if (bits) atomicOr(a.status, bits);
  }
  if (a.groups <= 32) return;
#pragma unroll 1
  for (int g0 = 0; g0 < a.groups; g0 += 32) {
    int before = sh->coarse_top[g0 >> 5];
    look.at(a, g0 + lane, before);
    sums(a, lane, w32, i32, s32);
    if (g0 + lane < a.groups) a.first[3 + g0 + lane] = coarse(sh, g0 >> 5) + place(lane_work, lane_items, lane_singles);
  }
}

// ------------------------------------------------------------------ softmax

// The queries of a warp's 32 rows into 128-byte-swizzled units of a row tile, in the
// operands' type; returns the power of two taken out of this lane's row. `at` is its
// element in q, or -1: zeros. Neighbouring lanes take a row's neighbouring 16 bytes. The
// loops are kept short: this runs once a segment, and instructions that are not in the
// SM's cache cost more than their execution (head_dim 256, 16 steps unrolled: 4.5 us).
template <class C, int D, bool k8>
__device__ __forceinline__ float load_query(const SharedArgs& a, uint8_t* q_s, int row0, int64_t at) {
  const int lane = threadIdx.x & 31;
  if constexpr (!k8) {
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // of a row; rows
    const int c = lane % kLanes;
    const uint32_t dst = su32(q_s) + (c >> 3) * kUnit;
#pragma unroll 4
    for (int s = 0; s < 32 / kAtOnce; ++s) {
      const int r = s * kAtOnce + lane / kLanes;
      const int64_t from = __shfl_sync(0xffffffffu, at, r);
      // (no bytes to read: zeros)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + sw128(row0 + r, (c & 7) * 16)),
                   "l"(static_cast<const __nv_bfloat16*>(a.q) + max(from, static_cast<int64_t>(0)) + c * 8),
                   "r"(from >= 0 ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return 1.f;
  } else {
    float up = 1.f;
    auto load = [&](auto&& use, int bytes_shift, auto lanes_c) {
      constexpr int kLanes = decltype(lanes_c)::value;  // of a row
      constexpr int kAtOnce = 32 / kLanes;              // rows
      constexpr int kSteps = 32 / kAtOnce, kBatch = kSteps < 8 ? kSteps : 8;
      const int chunk = lane % kLanes;
#pragma unroll 1
      for (int s0 = 0; s0 < kSteps; s0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int64_t from = __shfl_sync(0xffffffffu, at, (s0 + k) * kAtOnce + lane / kLanes);
          v[k] = make_uint4(0, 0, 0, 0);
          if (from >= 0)
            v[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + (from << bytes_shift)) + chunk);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float u = use(v[k], row0 + (s0 + k) * kAtOnce + lane / kLanes, chunk);
          const float mine = __shfl_sync(0xffffffffu, u, lane % kAtOnce * kLanes);
          if (lane / kAtOnce == s0 + k) up = mine;
        }
      }
    };
    if (a.q8) {
      load([&](uint4 v, int r, int c) {
        if constexpr (C::kDirect) {
          *reinterpret_cast<uint4*>(q_s + (c >> 3) * kUnit + sw128(r, (c & 7) * 16)) = v;
        } else {
          uint8_t* dst = q_s + (c >> 2) * kUnit;
          *reinterpret_cast<uint4*>(dst + sw128(r, (c & 3) * 32)) = widen8(v.x, v.y, false);
          *reinterpret_cast<uint4*>(dst + sw128(r, (c & 3) * 32 + 16)) = widen8(v.z, v.w, false);
        }
        return 1.f;
      }, 0, std::integral_constant<int, D / 16>());
      return up;
    }
    load([&](uint4 q, int r, int c) {
      const uint32_t v[4] = {q.x, q.y, q.z, q.w};
      uint32_t top = 0u;  // largest magnitude's bits, of the row
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(v[e] << 16 & 0x7FFF0000u, v[e] & 0x7FFF0000u));
#pragma unroll
      for (int d = 1; d < D / 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      int ex = static_cast<int>(top >> 23) - 127;
      if constexpr (C::kDirect) {
        // to [224, 448): 1.75 x 2^8 is E4M3's largest
        ex += (top & 0x7FFFFFu) <= 0x600000u ? -8 : -7;
        if (top == 0u || top >= 0x7F800000u) ex = 0;
      } else if (top == 0u || ex == 128 || (ex >= -6 && ex < 12)) {
        ex = 0;  // 2^-6 <= largest < 2^12: as it is; NaN and infinity too
      }
      ex = max(-126, min(126, ex));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      uint32_t w[4], w2[2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = __uint_as_float(v[e] << 16) * down, x1 = __uint_as_float(v[e] & 0xFFFF0000u) * down;
        if constexpr (C::kDirect) {
          const uint32_t c1 = e4m3x2(x0, x1);
          const float2 back = e4m3x2_to_f2(static_cast<uint16_t>(c1));
          const uint32_t c2 = e4m3x2(x0 - back.x, x1 - back.y);
          w[e >> 1] = e & 1 ? w[e >> 1] | c1 << 16 : c1;
          w2[e >> 1] = e & 1 ? w2[e >> 1] | c2 << 16 : c2;
        } else {
          const __half2 p = __floats2half2_rn(x0, x1);
          w[e] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      if constexpr (C::kDirect) {
        uint8_t* dst = q_s + (c >> 4) * kUnit + sw128(r, (c & 15) * 8);
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + C::kUK * kUnit) = make_uint2(w2[0], w2[1]);
      } else {
        *reinterpret_cast<uint4*>(q_s + (c >> 3) * kUnit + sw128(r, (c & 7) * 16)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      return __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    }, 1, std::integral_constant<int, D / 8>());
    return up;
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A thread per row, its 128 logits in registers.
template <class C, int D, bool k8, bool kTok>
__device__ __forceinline__ void softmax_role(const SharedArgs& a, Shared* sh, uint8_t* q_s,
                                             const float* scales, uint32_t tmem, int warp) {
  volatile int* abort_flag = &sh->abort_flag;
  const int lane = threadIdx.x & 31, quad = warp & 3, g = warp >> 2;
  const int r = quad * 32 + lane;  // row of the tile
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t t_o = tmem + lanes + kO + g * D;
  // logits in log2 units: s * scale, with the sign (or zero) applied to s first
  float logit = a.sm_scale * kLog2e, v_final = 1.f;
  if (k8 && !kTok) {
    logit *= __ldg(a.k_scale);
    v_final = __ldg(a.v_scale);
  }
  const float sign = kTok ? 1.f : logit < 0.f ? -1.f : logit == 0.f ? 0.f : 1.f;
  ItemReader reader(sh);
  Item it{};
  uint32_t n = 0, qn = 0, sc = 0, odds = 0;  // key tiles, queries, tiles of scales, odd tiles added
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = bar_wait(bar, parity & 1u, abort_flag, a);
    return __all_sync(0xffffffffu, ok);
  };
  auto buf = [&](uint32_t k) { return C::kG == 2 ? g : static_cast<int>(k & 1u); };
  auto par = [&](uint32_t k) { return C::kG == 2 ? k : k >> 1; };
  while (reader.next_warp(it, a)) {
    // the key tiles in turns with the other warpgroup, or this one's row tile on all
    const bool turns = C::kG == 2 && it.rows <= kTile;
    const int rt = turns ? 0 : g;
    const int tile_rows = min(kTile, it.rows - rt * kTile);
    const int j0 = it.t0 + (turns ? g : 0);  // first key tile of this warpgroup
    if (j0 >= it.t1) {
      if constexpr (kTok) {  // the tiles' scales are let go all the same
        for (int j = it.t0; j < it.t1; ++j, ++sc) {
          if (!wait(sh->sc_full + sc % kScales, sc / kScales)) return;
          if (lane == 0) bar_arrive(sh->sc_empty + sc % kScales);
        }
      }
      continue;
    }
    const int m0 = it.row0 + rt * kTile + r;
    float up = 1.f;
    if (rt == g) {
      int64_t at = -1;
      if (r < tile_rows)
        at = ((static_cast<int64_t>(it.q0) + m0 / a.group) * a.hq + it.head * a.group + m0 % a.group) * D;
      if (!wait(sh->q_empty + g, qn ^ 1u)) return;
      up = load_query<C, D, k8>(a, q_s + g * C::kQTile, quad * 32, at);
      if (turns) sh->rows[r].x = up;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(sh->q_full + g);
      ++qn;
    }
    const float plain = sign != 0.f ? fabsf(logit) : 1.f;
    float scale = kTok ? 1.f : plain * up;
    // first key this row sees
    int first = 0;
    if (a.window && r < tile_rows) {
      const int row = it.q0 + m0 / a.group;
      int b = it.b0, top = it.b1 - 1;
      while (b < top) {
        const int mid = (b + top + 1) >> 1;
        if (__ldg(a.qo_indptr + mid) <= row) b = mid;
        else top = mid - 1;
      }
      const int w = __ldg(a.window + b);
      if (w > 0) first = max(0, __ldg(a.kv_len + b) - (__ldg(a.qo_indptr + b + 1) - row) - w + 1);
    }
    float m = kMInit, l = 0.f;
    for (int j = it.t0; j < it.t1; ++j, ++sc) {
      if (turns && ((j - it.t0) & 1) != g) {
        if constexpr (kTok) {
          if (!wait(sh->sc_full + sc % kScales, sc / kScales)) return;
          if (lane == 0) bar_arrive(sh->sc_empty + sc % kScales);
        }
        continue;
      }
      const int b = buf(n);
      const uint32_t t_s = tmem + lanes + b * kKeys;
      const float* sp = scales + sc % kScales * 3 * kKeys;
      if constexpr (kTok)
        if (!wait(sh->sc_full + sc % kScales, sc / kScales)) return;
      if (!wait(sh->s_full + b, par(n))) return;
      fence_after();
      if (rt != g && j == j0) {  // (the query is there)
        up = sh->rows[r].x;
        if constexpr (!kTok) scale = plain * up;
      }
      const int k0 = j * kKeys;
      const bool hide = __any_sync(0xffffffffu, first > k0) || k0 + kKeys > it.end;
      const float *kp = sp, *lp = sp + kKeys;
      float done = up;
      if (hide || sign != 1.f) {
        // some row does not see the whole tile: mask S where it stands
#pragma unroll 1
        for (int c = 0; c < kKeys; c += 32) {
          uint32_t s[32];
          tmem_ld32(t_s + c, s);
          tmem_wait_ld<32>(s);
          const int last = it.end - 1 - k0 - c, from = first - k0 - c;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x = __uint_as_float(s[e]) * sign;
            if constexpr (kTok) x = fmaf(x * up, kp[c + e], lp[c + e]);
            s[e] = e > last || e < from ? 0xff800000u : __float_as_uint(x);
          }
          tmem_st32(t_s + c, s);
        }
        tmem_wait_st();
        kp = scales + kScales * 3 * kKeys;  // 1, and 0
        lp = kp + kKeys;
        done = 1.f;
      }
      uint32_t s[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) tmem_ld32(t_s + c, s + c);
      tmem_wait_ld<kKeys>(s);
      if constexpr (kTok) {
        const uint64_t up2 = pack2(done, done);
#pragma unroll
        for (int e = 0; e < kKeys; e += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(kp + e);
          const float4 l4 = *reinterpret_cast<const float4*>(lp + e);
          float x0, x1;
          unpack2(fma2(mul2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), up2),
                       pack2(k4.x, k4.y), pack2(l4.x, l4.y)), x0, x1);
          s[e] = __float_as_uint(x0);
          s[e + 1] = __float_as_uint(x1);
          unpack2(fma2(mul2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), up2),
                       pack2(k4.z, k4.w), pack2(l4.z, l4.w)), x0, x1);
          s[e + 2] = __float_as_uint(x0);
          s[e + 3] = __float_as_uint(x1);
        }
      }
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
        if (j > j0) {  // O holds something: the MMA in front of this one must be done
          if (!wait(sh->o_done + buf(n - 1), par(n - 1))) return;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
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
          const uint64_t sk = pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
          float p0, p1;
          unpack2(kTok ? add2(sk, m2) : fma2(sk, scale2, m2), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          if constexpr (kTok) {
            const float2 iv = *reinterpret_cast<const float2*>(sp + 2 * kKeys + k);
            sum[e & 1] = fma2(pack2(p0, p1), pack2(iv.x, iv.y), sum[e & 1]);
          } else {
            sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
          }
          w[e] = k8 ? f16x2(p0, p1) : bf16x2(p0, p1);
        }
        tmem_st16(t_s + c * 16, w);
        if (c == 1) {  // the first 64 keys: P V starts on them
          tmem_wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(sh->p_half + b);
        }
      }
      float l0, l1;
      unpack2(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(sh->p_full + b);
        if constexpr (kTok) bar_arrive(sh->sc_empty + sc % kScales);
      }
      ++n;
    }
    // the rows' partial outputs
    if (!wait(sh->o_done + buf(n - 1), par(n - 1))) return;
    fence_after();
    const bool odd = turns && it.t1 - it.t0 > 1;  // there are odd tiles' O and sums
    if (odd && g == 1) {
      sh->rows[r] = make_float2(m, l);
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh->odd_done);
      continue;
    }
    float f0 = 1.f, f1 = 0.f;
    if (odd) {
      if (!wait(&sh->odd_done, odds++)) return;
      fence_after();
      const float2 other = sh->rows[r];
      const float top = fmaxf(m, other.x);
      f0 = ex2(m - top);
      f1 = ex2(other.x - top);
      l = l * f0 + other.y * f1;
      m = top;
    }
    const float inv = l > 0.f ? v_final / l : l;  // no key: 0; NaN stays
    f0 *= inv;
    f1 *= inv;
    const int64_t at = it.cut ? static_cast<int64_t>(blockIdx.x) * C::kRows + rt * kTile
                              : (it.head * a.rows_cap + it.q0) * a.group + it.row0 + rt * kTile;
    float* part = (it.cut ? a.area_o : a.main_o) + at * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t v[32];
      __syncwarp();
      tmem_ld32(t_o + c, v);
      tmem_wait_ld<32>(v);
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f0);
      if (odd) {
        uint32_t w[32];
        tmem_ld32(t_o + D + c, w);
        tmem_wait_ld<32>(w);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(fmaf(__uint_as_float(w[e]), f1, __uint_as_float(v[e])));
      }
      // Four lanes exchange 16-byte pieces, so that a store writes 64 bytes of
      // each of eight rows and not 16 of thirty-two.
#pragma unroll
      for (int half = 0; half < 32; half += 16) {
#pragma unroll
        for (int d = 1; d <= 2; d <<= 1) {
          const bool hi = (lane & d) != 0;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            if (p & d) continue;  // piece p and piece p + d
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t& keep = v[half + p * 4 + e];
              uint32_t& give = v[half + (p + d) * 4 + e];
              const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? keep : give, d);
              if (hi) keep = got;
              else give = got;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = quad * 32 + (lane & ~3) + k;
          if (rr < tile_rows)
            *reinterpret_cast<uint4*>(part + static_cast<int64_t>(rr) * D + c + half + (lane & 3) * 4) =
                make_uint4(v[half + k * 4], v[half + k * 4 + 1], v[half + k * 4 + 2], v[half + k * 4 + 3]);
        }
      }
    }
    __syncwarp();
    fence_before();
    if (lane == 0) {
      bar_arrive(sh->o_free + g);
      if (odd) bar_arrive(sh->o_free + 1);
    }
    if (r < tile_rows) (it.cut ? a.area_x : a.main_x)[at + r] = l == 0.f ? -INFINITY : m + __log2f(l);
  }
}

template <int D, bool k8, bool kI8, bool kTok>
__global__ void __launch_bounds__(Cfg<D, k8, kI8, kTok>::kThreads, 1)
    shared_prefix(const __grid_constant__ SharedArgs a, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv) {
  using C = Cfg<D, k8, kI8, kTok>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_s = smem;
  uint8_t* rings = smem + C::kQBytes;
  uint8_t* raw = rings + C::kRings;
  float* scales = reinterpret_cast<float*>(raw + C::kRaw * C::kRawBytes);
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kSmem - sizeof(Shared));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (su32(smem) % 1024u) {  // the swizzled tiles need it
    if (tid == 0) atomicOr(a.status, PDA_STATUS_SMEM_MISALIGNED);
    return;
  }
  if (warp == 0) {  // a lane a barrier of each kind
    if (tid < 2) {
      bar_init(sh->q_full + tid, 4);
      bar_init(sh->q_empty + tid, 1);
      bar_init(sh->s_full + tid, 1);
      bar_init(sh->p_half + tid, 4);
      bar_init(sh->p_full + tid, 4);
      bar_init(sh->o_done + tid, 1);
      bar_init(sh->o_free + tid, 4);
    }
    if (tid < C::kRK) {
      bar_init(sh->k_full + tid, k8 && !C::kDirect ? C::kConv : 1);
      bar_init(sh->k_empty + tid, 1);
    }
    if (tid < C::kRV) {
      bar_init(sh->v_full + tid, k8 ? C::kConv : 1);
      bar_init(sh->v_empty + tid, 1);
    }
    if (k8 && tid < C::kRaw) {
      bar_init(sh->raw_full + tid, 1);
      bar_init(sh->raw_empty + tid, k8 ? C::kConv : 1);
    }
    if (kTok && tid < kScales) {
      bar_init(sh->sc_full + tid, kTok ? C::kConv : 1);
      bar_init(sh->sc_empty + tid, C::kSoft);
    }
    if (tid < kItems) {
      bar_init(sh->item_full + tid, 1);
      bar_init(sh->item_empty + tid, C::kReaders);
    }
    if (tid == 0) {
      bar_init(&sh->odd_done, 4);
      bar_init(&sh->drain, 1);
      sh->abort_flag = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (kTok && tid < kKeys) {
    scales[kScales * 3 * kKeys + tid] = 1.f;
    scales[kScales * 3 * kKeys + kKeys + tid] = 0.f;
  }
  WorkList<C::kG> list;
  if (warp == C::kWorkWarp) list.prepare(a, sh);
  if (warp == C::kMmaWarp) {
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
  // the requests' own tokens (stage 1) start where CTAs of this kernel leave room
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // registers a thread: with two row tiles 192 x 256 + 64 x 256 (128 x 512 at the launch),
  // with one 216 x 128 + 104 x 256 (168 x 384), or 96 x 384 with codes to widen (128 x 512)
  if (warp < C::kSoft) {
    if constexpr (C::kG == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  } else {
    if constexpr (C::kG == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else if constexpr (k8) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  }
  if (warp < C::kSoft) {
    softmax_role<C, D, k8, kTok>(a, sh, q_s, scales, tmem, warp);
  } else if (warp == C::kMmaWarp) {
    if (elect_one()) mma_role<C, D, k8>(a, sh, q_s, rings);
  } else if (warp == C::kWorkWarp) {
    list.run(a, sh);
  } else if (k8 && warp >= C::kConv0) {
    if constexpr (k8) widen_role<C, D, kI8, kTok>(a, sh, rings, raw, scales);
  } else if (warp < C::kProd0 + C::kProds) {
    load_role<C, D, k8>(a, sh, rings, raw, &tk, &tv, warp - C::kProd0);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == C::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
}

// ------------------------------------------------------- the prefixes themselves
//
// Mathematics: the whole pages in front of a group's rows whose ids are those of its
// first request: n = min over requests of the equal leading ids, at most (L - R) / P.
//
// Bound: latency. A cluster of CTAs per group; its warps take stretches of the requests'
// lists in turn, the first of all requests first, and leave out those behind what another
// has found to be the end. 64 requests of 80 pages: 4.6 us, 512 of 704 in 64 groups: 7.9
// (a group's lists by one CTA: 17.8).
constexpr int kShareThreads = 256;
constexpr int kShareWarps = kShareThreads / 32;
constexpr int kStretch = 256;  // ids of a stretch

struct TablesArgs {
  pda_shared_tables t;
  int32_t* status;
  int batch, groups, page_size, max_q_len, max_kv_len, num_pages;
};

__global__ void __launch_bounds__(kShareThreads) share_tables(const __grid_constant__ TablesArgs a) {
  __shared__ int sh_pages, sh_low;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ctas, rank;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  rank = cluster_rank();
  const int g = blockIdx.x / ctas;
  if (threadIdx.x == 0) sh_pages = sh_low = INT_MAX;
  cluster_sync();
  const int b0 = a.t.group_indptr ? __ldg(a.t.group_indptr + g) : 0;
  int b1 = a.t.group_indptr ? __ldg(a.t.group_indptr + g + 1) : a.batch;
  uint32_t bits = 0u;
  int top = INT_MIN;  // no bound in front may be above the group's (no_overlap)
  for (int i = lane; i < g; i += 32) top = max(top, __ldg(a.t.group_indptr + i));
  const bool valid = b0 >= 0 && b1 >= b0 && b1 <= a.batch && b0 >= __reduce_max_sync(0xffffffffu, top);
  if (!valid) {
    bits = PDA_STATUS_TABLE_INVALID;
    b1 = b0;
  }
  if ((g == 0 && b0 != 0) || (g == a.groups - 1 && b1 != a.batch)) bits = PDA_STATUS_TABLE_INVALID;
  // a request that takes part: its rows and length, else its status bits
  auto fits = [&](int b, int& rows, int& len) -> bool {
    const int64_t r = static_cast<int64_t>(__ldg(a.t.qo_indptr + b + 1)) - __ldg(a.t.qo_indptr + b);
    len = __ldg(a.t.kv_len + b);
    rows = static_cast<int>(r);
    if (r == 0) return false;
    uint32_t bad = 0u;
    if (r < 0 || r > a.max_q_len) bad |= PDA_STATUS_ROWS_GT_MAX;
    if (len < r) bad |= PDA_STATUS_KV_LEN_LT_ROWS;
    if (len > a.max_kv_len) bad |= PDA_STATUS_KV_LEN_GT_MAX;
    bits |= bad;
    return !bad;
  };
  int lead = -1;  // the first one
  for (int c = b0; c < b1 && lead < 0; c += 32) {
    int rows, len;
    const uint32_t has = __ballot_sync(0xffffffffu, c + lane < b1 && fits(c + lane, rows, len));
    if (has) lead = c + __ffs(has) - 1;
  }
  int* best = &sh_pages;  // the leader's words are the cluster's
  const uint32_t pages_at = on_leader(best), low_at = on_leader(&sh_low);
  auto least = [](uint32_t at, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
  };
  if (lead >= 0) {
    const int32_t* theirs = a.t.page_table + __ldg(a.t.kv_indptr + lead);
    const int most = __ldg(a.t.kv_indptr + lead + 1) - __ldg(a.t.kv_indptr + lead);
    const int n_req = b1 - b0, step = static_cast<int>(ctas) * kShareWarps;
    const int stretches = (max(most, 0) + kStretch - 1) / kStretch;
    // (at least one: it notes the request's first token seen, and its own length)
    const int64_t work = static_cast<int64_t>(n_req) * max(stretches, 1);
    for (int64_t k = static_cast<int64_t>(rank) * kShareWarps + warp; k < work; k += step) {
      const int stretch = static_cast<int>(k / n_req), b = b0 + static_cast<int>(k % n_req);
      const int j0 = stretch * kStretch;
      if (j0) {
        // (one lane's reading, as others lower the word meanwhile: all lanes leave or none)
        const int seen = __shfl_sync(0xffffffffu, static_cast<int>(cluster_load(pages_at)), 0);
        if (j0 >= seen) break;  // as are all behind it
      }
      int rows, len;
      if (!fits(b, rows, len)) continue;
      const int at = __ldg(a.t.kv_indptr + b);
      const int32_t* mine = a.t.page_table + at;
      const int all = max(0, min(min((len - rows) / a.page_size, most), __ldg(a.t.kv_indptr + b + 1) - at));
      const int n = min(all, j0 + kStretch);
      int equal = all;
      bool ok[kStretch / 32];
#pragma unroll
      for (int e = 0; e < kStretch / 32; ++e) {
        const int j = j0 + e * 32 + lane;
        ok[e] = true;
        if (j < n) {
          const int id = __ldg(mine + j);
          ok[e] = id == __ldg(theirs + j) && id >= 0 && id < a.num_pages;
        }
      }
#pragma unroll
      for (int e = kStretch / 32 - 1; e >= 0; --e) {
        const uint32_t differ = __ballot_sync(0xffffffffu, !ok[e]);
        if (differ) equal = j0 + e * 32 + __ffs(differ) - 1;
      }
      if (lane == 0) {
        least(pages_at, equal);
        if (stretch == 0) {
          const int w = a.t.window ? __ldg(a.t.window + b) : 0;
          least(low_at, w > 0 ? static_cast<int>(max(static_cast<int64_t>(0),
                                                     static_cast<int64_t>(len) - rows - w + 1))
                              : 0);
        }
      }
    }
  }
  cluster_sync();
  int pages = lead >= 0 ? static_cast<int>(cluster_load(pages_at)) : 0;
  int low = lead >= 0 ? static_cast<int>(cluster_load(low_at)) : 0;
  cluster_sync();  // (the leader's words are read)
  const int end = pages * a.page_size;
  if (rank == 0) {
    if (threadIdx.x == 0 && valid) {
      a.t.prefix[2 * g] = min(low / a.page_size * a.page_size, end);
      a.t.prefix[2 * g + 1] = end;
    }
    for (int b = b0 + static_cast<int>(threadIdx.x); b < b1; b += kShareThreads) {
      int rows, len;
      const bool ok = fits(b, rows, len);
      a.t.own_indptr[b] = __ldg(a.t.kv_indptr + b) + pages;
      a.t.own_len[b] = rows == 0 ? 0 : ok ? len - end : -1;
    }
    if (bits) atomicOr(a.status, static_cast<int>(bits));
  }
}

// ---------------------------------------------------------------- dispatch
using PrefixFn = void (*)(SharedArgs, CUtensorMap, CUtensorMap);
struct Kernel {
  PrefixFn fn;
  int smem, threads;
  int k_keys, v_keys;  // most tokens of a K box and of a V box
  bool direct;
};
template <int D, bool k8, bool kI8, bool kTok>
Kernel kernel_of() {
  using C = Cfg<D, k8, kI8, kTok>;
  return {shared_prefix<D, k8, kI8, kTok>, C::kSmem, C::kThreads,
          k8 && !C::kDirect ? C::kRawKeys : kKeys, k8 ? C::kRawKeys : C::kVKeys, C::kDirect};
}
template <int D>
Kernel kernel_for(const pda_plan_t& p) {
  const bool tok = p.scale_mode == PDA_SCALE_TOKEN_HEAD;
  if (p.kv_dtype == PDA_BF16) return kernel_of<D, false, false, false>();
  if (p.kv_dtype == PDA_INT8) return tok ? kernel_of<D, true, true, true>() : kernel_of<D, true, true, false>();
  return tok ? kernel_of<D, true, false, true>() : kernel_of<D, true, false, false>();
}
Kernel kernel_for(const pda_plan_t& p) {
  return p.head_dim == 64 ? kernel_for<64>(p) : p.head_dim == 128 ? kernel_for<128>(p) : kernel_for<256>(p);
}

// Tensor map of the cache, (channel, slot, kv head, page): boxes of `rows` tokens x 128
// bytes (swizzled: an operand), or x a head's codes (as they lie).
bool page_map(CUtensorMap* m, const void* base, const pda_plan_t& p, int rows, bool operand) {
  EncodeFn enc = encoder();
  if (!enc) return false;
  const bool wide = p.kv_dtype == PDA_BF16;
  const int64_t eb = wide ? 2 : 1;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.head_dim), static_cast<cuuint64_t>(p.page_size),
                              static_cast<cuuint64_t>(p.num_kv_heads), static_cast<cuuint64_t>(p.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.kv_stride_token * eb),
                                 static_cast<cuuint64_t>(p.kv_stride_head * eb),
                                 static_cast<cuuint64_t>(p.kv_stride_page * eb)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(operand ? 128 / eb : p.head_dim),
                             static_cast<cuuint32_t>(std::min(p.page_size, rows)), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, wide ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             operand ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

bool a4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

int check_plan(const pda_shared_plan_t* sp) {
  if (!sp) return PDA_ERR_NULL;
  if (sp->magic != PDA_SHARED_MAGIC || sp->struct_bytes != sizeof(pda_shared_plan_t) ||
      sp->own.magic != PDA_PLAN_MAGIC)
    return PDA_ERR_PLAN;
  return PDA_OK;
}

int check_tables(const pda_shared_plan_t* sp, const pda_shared_tables* t) {
  if (!t->page_table || !t->kv_indptr || !t->kv_len || !t->qo_indptr || !t->prefix || !t->own_indptr ||
      !t->own_len)
    return PDA_ERR_NULL;
  if (!t->group_indptr && sp->groups != 1) return PDA_ERR_NULL;
  if (t->own_len == t->kv_len || t->own_indptr == t->kv_indptr) return PDA_ERR_INVALID;
  if (!a4(t->page_table) || !a4(t->kv_indptr) || !a4(t->kv_len) || !a4(t->qo_indptr) || !a4(t->window) ||
      !a4(t->group_indptr) || !a4(t->prefix) || !a4(t->own_indptr) || !a4(t->own_len))
    return PDA_ERR_ALIGNMENT;
  return PDA_OK;
}

}  // namespace
}  // namespace pda

extern "C" int pda_shared_plan(const pda_plan_t* plan, int32_t groups, int32_t max_own_len,
                               pda_shared_plan_t* out_plan, size_t* scratch_bytes) {
  using namespace pda;
  if (!plan || !out_plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  if ((plan->head_dim != 64 && plan->head_dim != 128 && plan->head_dim != 256) || plan->page_size < 8)
    return PDA_ERR_UNSUPPORTED;
  if (groups < 1 || groups > kMaxGroups || max_own_len < 0) return PDA_ERR_INVALID;
  if (max_own_len == 0 || max_own_len > plan->max_kv_len) max_own_len = plan->max_kv_len;
  pda_params p;
  std::memset(&p, 0, sizeof p);
  p.num_qo_heads = plan->num_qo_heads;
  p.num_kv_heads = plan->num_kv_heads;
  p.head_dim = plan->head_dim;
  p.page_size = plan->page_size;
  p.q_dtype = plan->q_dtype;
  p.kv_dtype = plan->kv_dtype;
  p.scale_mode = plan->scale_mode;
  p.max_batch = plan->max_batch;
  p.max_q_len = plan->max_q_len;
  p.max_kv_len = max_own_len;
  p.num_pages = plan->num_pages;
  p.kv_stride_page = plan->kv_stride_page;
  p.kv_stride_token = plan->kv_stride_token;
  p.kv_stride_head = plan->kv_stride_head;
  p.device = plan->device;
  p.num_sms = plan->num_sms;
  p.batch = plan->batch;
  p.kernel = plan->kernel;
  p.wait_limit_us = plan->wait_limit_us;
  p.inject = plan->inject;
  pda_shared_plan_t sp;
  std::memset(&sp, 0, sizeof sp);
  const int rc = pda_plan(&p, &sp.own, nullptr);
  if (rc != PDA_OK) return rc;
  sp.magic = PDA_SHARED_MAGIC;
  sp.struct_bytes = sizeof sp;
  sp.groups = groups;
  sp.max_kv_len = plan->max_kv_len;
  const int64_t d = plan->head_dim, rows = d <= 128 ? 2 * kTile : kTile;
  const int64_t cells = sp.own.rows_cap * plan->num_qo_heads;
  // all tiles of all items, what they count and `pay` for each stay in 31 bits
  const int64_t blocks = sp.own.rows_cap * plan->group / rows + groups;
  const int64_t tiles = plan->max_kv_len / kKeys + 2;
  if (sp.own.rows_cap * plan->group > INT_MAX ||
      static_cast<double>(blocks) * plan->num_kv_heads * (kFull * static_cast<double>(tiles) + kPay) > 2.0e9)
    return PDA_ERR_INVALID;
  const int64_t area = static_cast<int64_t>(plan->num_sms) * rows;
  int64_t at = kStatusHeaderBytes;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up256(bytes);
    return here;
  };
  const int64_t parts = own_here(&sp.own) ? 0 : sp.own.max_splits * cells;  // of stage 1
  sp.own.scratch_lse_offset = take(parts * 4);
  sp.own.scratch_o_offset = take(parts * d * 4);
  sp.first_offset = take((3 + static_cast<int64_t>(groups)) * 4);
  sp.main_lse_offset = take(cells * 4);
  sp.main_o_offset = take(cells * d * 4);
  sp.area_lse_offset = take(area * 4);
  sp.area_o_offset = take(area * d * 4);
  sp.own.scratch_bytes = sp.scratch_bytes = at;
  *out_plan = sp;
  if (scratch_bytes) *scratch_bytes = static_cast<size_t>(at);
  return PDA_OK;
}

extern "C" int pda_share_tables(const pda_shared_plan_t* sp, const pda_shared_tables* tables, void* scratch,
                                pda_stream_t stream) {
  using namespace pda;
  int rc = check_plan(sp);
  if (rc != PDA_OK) return rc;
  if (!tables) return PDA_ERR_NULL;
  if ((rc = check_tables(sp, tables)) != PDA_OK) return rc;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return PDA_ERR_SCRATCH;
  if (!on_device(sp->own.device)) return PDA_ERR_INVALID;
  TablesArgs a = {};
  a.t = *tables;
  a.status = static_cast<int32_t*>(scratch);
  a.batch = sp->own.batch;
  a.groups = sp->groups;
  a.page_size = sp->own.page_size;
  a.max_q_len = sp->own.max_q_len;
  a.max_kv_len = sp->max_kv_len;
  a.num_pages = sp->own.num_pages;
  // (eight CTAs a group at most, while they are not more than four an SM)
  unsigned ctas = 8;
  while (ctas > 1 && static_cast<int64_t>(sp->groups) * ctas > 4LL * sp->own.num_sms) ctas /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sp->groups) * ctas);
  cfg.blockDim = dim3(kShareThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, share_tables, a) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  return PDA_OK;
}

extern "C" int pda_decode_shared(const pda_shared_plan_t* sp, const void* q, const void* k_pages,
                                 const void* v_pages, const pda_shared_tables* tables, int32_t max_q_len,
                                 float sm_scale, const float* k_scale, const float* v_scale, void* out,
                                 float* lse, void* scratch, pda_stream_t stream) {
  using namespace pda;
  int rc = check_plan(sp);
  if (rc != PDA_OK) return rc;
  if (!tables) return PDA_ERR_NULL;
  const pda_shared_tables& t = *tables;
  if ((rc = check_tables(sp, tables)) != PDA_OK) return rc;
  if (!scratch || reinterpret_cast<uintptr_t>(scratch) % 256) return PDA_ERR_SCRATCH;
  const pda_plan_t* plan = &sp->own;
  rc = check_decode_args(plan, q, k_pages, v_pages, t.page_table, t.own_indptr, t.own_len, t.qo_indptr,
                         max_q_len, k_scale, v_scale, out, lse);
  if (rc != PDA_OK) return rc;
  if (!on_device(plan->device)) return PDA_ERR_INVALID;
  DecodeArgs o = decode_args(plan, q, k_pages, v_pages, t.page_table, t.own_indptr, t.own_len,
                             t.qo_indptr, max_q_len, t.window, sm_scale, k_scale, v_scale, out, lse, scratch);
  o.final_splits = 0;
  o.group_indptr = t.group_indptr;
  o.groups = sp->groups;
  SharedArgs a = {};
  char* base = static_cast<char*>(scratch);
  a.q = q;
  a.page_table = t.page_table;
  a.qo_indptr = t.qo_indptr;
  a.kv_len = t.kv_len;
  a.window = t.window;
  a.group_indptr = t.group_indptr;
  a.prefix = t.prefix;
  a.own_indptr = t.own_indptr;
  a.own_len = t.own_len;
  a.k_scale = o.k_scale;
  a.v_scale = o.v_scale;
  a.main_x = reinterpret_cast<float*>(base + sp->main_lse_offset);
  a.main_o = reinterpret_cast<float*>(base + sp->main_o_offset);
  a.area_x = reinterpret_cast<float*>(base + sp->area_lse_offset);
  a.area_o = reinterpret_cast<float*>(base + sp->area_o_offset);
  a.first = reinterpret_cast<int*>(base + sp->first_offset);
  a.status = o.status;
  a.wait_limit_ns = o.wait_limit_ns;
  a.sm_scale = sm_scale;
  a.batch = o.batch;
  a.groups = sp->groups;
  a.hq = o.hq;
  a.hkv = o.hkv;
  a.group = o.group;
  a.page_size = o.page_size;
  a.num_pages = o.num_pages;
  a.max_q_len = max_q_len;
  a.max_kv_len = sp->max_kv_len;
  a.rows_cap = o.rows_cap;
  a.q8 = plan->q_dtype == PDA_E4M3;
  a.inject = o.inject;
  a.ctas = plan->num_sms;
  a.one = plan->head_dim == 256 ? kFull : plan->kv_dtype != PDA_BF16 || plan->head_dim == 64 ? 5 : 7;
  const Kernel k = kernel_for(*plan);
  CUtensorMap tk, tv;
  const bool wide = plan->kv_dtype == PDA_BF16;
  if (!page_map(&tk, k_pages, *plan, k.k_keys, wide || k.direct) ||
      !page_map(&tv, v_pages, *plan, k.v_keys, wide))
    return PDA_ERR_CUDA;
  if (cudaFuncSetAttribute(reinterpret_cast<const void*>(k.fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                           k.smem) != cudaSuccess) {
    cudaGetLastError();
    return PDA_ERR_CUDA;
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  k.fn<<<static_cast<unsigned>(a.ctas), k.threads, k.smem, s>>>(a, tk, tv);
  if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
  if (own_here(plan)) return launch_own(plan, a, o, s);
  rc = plan->kernel == PDA_KERNEL_TC ? launch_stage1_tc(plan, o, s, true) : launch_stage1_mma(plan, o, s, true);
  return rc == PDA_OK ? launch_join(plan, a, o, s) : rc;
}
