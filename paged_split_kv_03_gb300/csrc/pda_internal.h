// pda_internal.h -- shared between the planner (host C++) and the CUDA
// translation units. Not part of the public ABI.
#pragma once

#include <stdint.h>

#include <cuda_runtime.h>

#include "pda.h"

#ifdef __CUDACC__
#define PDA_HD __host__ __device__ __forceinline__
#else
#define PDA_HD inline
#endif

namespace pda {

constexpr int kStatusHeaderBytes = 256;  // status word + padding at the start of split_scratch
constexpr int kMaxQLen = 8;              // rows per request ("up to 8 query rows")
constexpr int kMmaRowsPerCta = 64;       // mma.sync path: 4 warps x m16 tiles
constexpr int kTcRowsPerCta = 64;        // tcgen05 path: N of the swapped QK^T MMA

// Arguments of both stage-1 variants and of stage 2 (passed by value).
struct DecodeArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* page_table;
  const int32_t* kv_indptr;
  const int32_t* kv_len;
  const int32_t* qo_indptr;
  const int32_t* window;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  float* part_o;      // [max_splits][rows_cap][Hq][D] fp32, normalised partial output
  float* part_lse;    // [max_splits][rows_cap][Hq] fp32, log2-domain partial LSE
  uint32_t* status;   // sticky device status bits
  float sm_scale;
  int64_t sp, st, sh; // cache strides (elements)
  int batch, hq, hkv, group, head_dim, page_size, num_pages;
  int head_dim_v;  // value channels (MLA: 512 of a 576-channel latent)
  int max_q_len, max_kv_len, max_splits, head_blocks, chunk_pages;
  int tail_from, tail_chunk_pages, head_splits, tail_splits;  // see pda_plan_t
  int64_t merge_item0;  // first (request, row, q head) item the merge grid covers
  int64_t rows_cap;
  int hpc[kMaxQLen + 1];  // q heads per CTA for R rows
  int tma_slot_dim;       // tcgen05 path: tensor-map coordinate holding the slot (1 or 2)
  uint64_t wait_limit_ns; // tcgen05 path: bound of every pipeline wait
  uint32_t inject;        // PDA_INJECT_* test hooks set by the host (0 in normal use)
  int final_splits;       // splits of a request whose results stage 1 writes itself: 1, or 0 where
                          // all are partials, to be joined with those of a shared prefix
  // bounds of the groups of requests that share a prefix, or NULL: stage 1 leaves out
  // requests of no group, whose page_table places and lengths nobody has written
  const int32_t* group_indptr;
  int groups;
};

// The KV range one (request, split) covers. Every kernel derives it from the
// device-resident kv_len / qo_indptr / window, so one plan (and one captured
// graph) serves any lengths up to the plan's maxima.
struct SplitRange {
  int32_t lo;          // first visible key of any row of the request
  int32_t lo_page;     // page holding lo
  int32_t num_pages;   // ceil(L / P)
  int32_t num_splits;  // splits with at least one page of [lo_page, num_pages)
};

PDA_HD SplitRange split_range(int32_t L, int32_t R, int32_t W, int32_t P, int32_t chunk_pages) {
  SplitRange s;
  int32_t p0 = L - R;  // position of the first query row
  s.lo = (W > 0) ? (p0 - W + 1 > 0 ? p0 - W + 1 : 0) : 0;
  s.lo_page = s.lo / P;
  s.num_pages = (L + P - 1) / P;
  int32_t span = s.num_pages - s.lo_page;
  s.num_splits = span > 0 ? (span + chunk_pages - 1) / chunk_pages : 0;
  return s;
}

// KV chunk (pages per split) of request b.
PDA_HD int32_t chunk_for(const DecodeArgs& a, int b) {
  return b >= a.tail_from ? a.tail_chunk_pages : a.chunk_pages;
}

// Stage-1 work item of a CTA: requests [0, tail_from) with head_splits
// splits each come first, then the tail requests with tail_splits; inside
// each part the order is (request, kv head, split, head block), head block
// fastest. False past the last request.
struct WorkItem {
  int b, hkv, split, hb;
};
PDA_HD bool work_item(const DecodeArgs& a, int64_t bid, WorkItem& w) {
  const int64_t head_ctas = (int64_t)a.tail_from * a.hkv * a.head_splits * a.head_blocks;
  int splits = a.head_splits, b0 = 0;
  if (bid >= head_ctas) {
    bid -= head_ctas;
    splits = a.tail_splits;
    b0 = a.tail_from;
  }
  w.hb = static_cast<int>(bid % a.head_blocks);
  bid /= a.head_blocks;
  w.split = static_cast<int>(bid % splits);
  bid /= splits;
  w.hkv = static_cast<int>(bid % a.hkv);
  w.b = b0 + static_cast<int>(bid / a.hkv);
  return w.b < a.batch;
}

// Launchers and resource queries of the two stage-1 variants and stage 2.
int mma_smem_bytes(const pda_plan_t* plan);
int mma_ctas_per_sm(const pda_plan_t* plan);
int launch_stage1_mma(const pda_plan_t* plan, const DecodeArgs& args, cudaStream_t s,
                      bool overlap = false);
bool tc_supported(const pda_plan_t* plan);
int tc_rows_limit(const pda_plan_t* plan);
int tc_variant_rows(const pda_plan_t* plan);
int tc_smem_bytes(const pda_plan_t* plan);
int tc_ctas_per_sm(const pda_plan_t* plan);
// (overlap: beside the kernel in front of it in the stream, whose CTAs let it start and do
// not depend on it; stage 1 ends behind that kernel)
int launch_stage1_tc(const pda_plan_t* plan, const DecodeArgs& args, cudaStream_t s,
                     bool overlap = false);
int launch_stage2(const pda_plan_t* plan, const DecodeArgs& args, cudaStream_t s);

// Host-side checks of pda_decode's arguments (plan, pointers, alignment,
// max_q_len); PDA_OK or the PDA_ERR_* code pda_decode returns for them.
int check_decode_args(const pda_plan_t* plan, const void* q, const void* k_pages,
                      const void* v_pages, const int32_t* page_table, const int32_t* kv_indptr,
                      const int32_t* kv_len, const int32_t* qo_indptr, int32_t max_q_len,
                      const float* k_scale, const float* v_scale, const void* out,
                      const float* lse);

// The arguments of both stages of one pda_decode call (checked before).
DecodeArgs decode_args(const pda_plan_t* plan, const void* q, const void* k_pages,
                       const void* v_pages, const int32_t* page_table, const int32_t* kv_indptr,
                       const int32_t* kv_len, const int32_t* qo_indptr, int32_t max_q_len,
                       const int32_t* window, float sm_scale, const float* k_scale,
                       const float* v_scale, void* out, float* lse, void* split_scratch);

// Whether `device` is the current one.
inline bool on_device(int device) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return dev == device;
}

// Device address of the library's built-in split scratch (the array behind
// pda_decode_static) on the current device, which must be `device`; looked
// up afresh unless `s` is capturing a graph (then the last lookup is used).
int static_scratch(int device, cudaStream_t s, void** out);

#ifdef __CUDACC__
// The group that lists request b: its bounds, indptr[g] and the next, hold the request, are
// requests of the batch, and no bound in front is above them (so no two groups that are decoded
// list the same request); -1: none. NULL: one group of all. A whole warp. (The loads of 128
// groups are under way together: one round trip where a search by halves takes seven.)
__device__ __forceinline__ int group_of_request(const int32_t* indptr, int groups, int batch, int b) {
  if (!indptr) return 0;
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & 31;
  int top = -1;  // the highest bound in front
#pragma unroll 1
  for (int g0 = 0; g0 < groups; g0 += 32 * kAtOnce) {
    int lo[kAtOnce], hi[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int g = g0 + 32 * k + lane;
      lo[k] = hi[k] = -1;
      if (g < groups) {
        lo[k] = __ldg(indptr + g);
        hi[k] = __ldg(indptr + g + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t has = __ballot_sync(0xffffffffu, lo[k] >= 0 && lo[k] <= b && b < hi[k] && hi[k] <= batch);
      // (the first group that holds it decides: its end is a bound above the request)
      const int at = has ? __ffs(has) - 1 : 32;
      top = max(top, __reduce_max_sync(0xffffffffu, lane < at ? lo[k] : -1));
      if (has) return __shfl_sync(0xffffffffu, lo[k], at) >= top ? g0 + 32 * k + at : -1;
    }
  }
  return -1;
}

// The same for stage 1, as a call: its registers are full (inlined, two builds spill), and only
// decodes behind shared prefixes make it.
static __device__ __noinline__ bool no_group_lists(const int32_t* indptr, int groups, int batch, int b) {
  return group_of_request(indptr, groups, batch, b) < 0;
}

// Stage 1's first CTA, on each of its ways out: where the launch overlaps the kernel in
// front of it, what follows stage 1 follows both. (One CTA is enough, and the others make
// room; without such a launch there is nothing to wait for.)
__device__ __forceinline__ void end_behind_previous() {
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

}  // namespace pda
