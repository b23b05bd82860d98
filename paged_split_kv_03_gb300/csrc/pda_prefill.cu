// pda_prefill.cu -- expanded latent attention of ragged requests (prefill).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pda.h"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kNope = 128, kRope = 64, kQDim = kNope + kRope, kDv = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PrefillArgs {
  const __nv_bfloat16* q;
  int64_t q_row, q_head;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t kv_tok, kv_head;
  const __nv_bfloat16* k_rope;
  int64_t rope_tok;
  const int32_t* qo_indptr;
  const int32_t* tok_indptr;
  const int32_t* window;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  float sm_scale;
  int heads, batch, max_kv_len, rows, tokens, causal;
};

// One warp per (row, head): six query channels a lane, an online softmax over
// the visible keys, four value channels a lane.
__global__ void __launch_bounds__(256) prefill(const __grid_constant__ PrefillArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t r = item / a.heads;
  const int h = static_cast<int>(item % a.heads);
  if (r >= a.rows) return;
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.qo_indptr[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo, q0 = a.qo_indptr[b], R = a.qo_indptr[b + 1] - q0;
  const int k0 = a.tok_indptr[b], L = a.tok_indptr[b + 1] - k0;
  const int i = static_cast<int>(r) - q0;
  if (i < 0 || i >= R) return;
  uint32_t bad = 0;
  if (q0 + R > a.rows) bad |= PDA_STATUS_ROWS_GT_CAP;
  if (L < 0 || k0 + L > a.tokens) bad |= PDA_STATUS_TOKENS_GT_CAP;
  if (L > a.max_kv_len) bad |= PDA_STATUS_KV_LEN_GT_MAX;
  if (a.causal && L < R) bad |= PDA_STATUS_KV_LEN_LT_ROWS;
  if (bad) {
    if (lane == 0) atomicOr(a.status, bad);
    return;
  }
  const int p = L - R + i, W = a.window ? a.window[b] : 0;
  const int end = a.causal ? p + 1 : L;
  const int begin = a.causal && W > 0 && p - W + 1 > 0 ? p - W + 1 : 0;
  float q[6], o[4] = {};
  const __nv_bfloat16* qp = a.q + r * a.q_row + h * a.q_head;
  for (int e = 0; e < 6; ++e) q[e] = __bfloat162float(qp[lane + 32 * e]) * a.sm_scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  for (int j = begin; j < end; ++j) {
    const int64_t t = k0 + j;
    const __nv_bfloat16* kp = a.k + t * a.kv_tok + h * a.kv_head;
    const __nv_bfloat16* rp = a.k_rope + t * a.rope_tok;
    float s = 0.f;
    for (int e = 0; e < 4; ++e) s = fmaf(q[e], __bfloat162float(kp[lane + 32 * e]), s);
    for (int e = 0; e < 2; ++e) s = fmaf(q[4 + e], __bfloat162float(rp[lane + 32 * e]), s);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = fmaf(l, f, w);
    const __nv_bfloat16* vp = a.v + t * a.kv_tok + h * a.kv_head;
    for (int e = 0; e < 4; ++e) o[e] = fmaf(o[e], f, w * __bfloat162float(vp[lane + 32 * e]));
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  for (int e = 0; e < 4; ++e) a.out[(r * a.heads + h) * kDv + lane + 32 * e] = __float2bfloat16(o[e] * inv);
  if (a.lse && lane == 0) a.lse[r * a.heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace
}  // namespace pda

extern "C" int pda_prefill_plan(const pda_plan_t* plan, int32_t rows, int32_t tokens,
                                pda_prefill_plan_t* out_plan, size_t* scratch_bytes) {
  if (!plan || !out_plan) return PDA_ERR_NULL;
  if (plan->magic != PDA_PLAN_MAGIC) return PDA_ERR_PLAN;
  if (plan->head_dim != pda::kQDim + 384 || plan->num_kv_heads != 1) return PDA_ERR_UNSUPPORTED;
  if (rows < 1 || tokens < 1) return PDA_ERR_INVALID;
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
  p.splits = 1;
  p.wait_limit_us = plan->wait_limit_us;
  p.scratch_bytes = pda::kStatusHeaderBytes;
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
  PrefillArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_row = q_stride_row;
  a.q_head = q_stride_head;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.kv_tok = kv_stride_token;
  a.kv_head = kv_stride_head;
  a.k_rope = static_cast<const __nv_bfloat16*>(k_rope);
  a.rope_tok = k_rope_stride;
  a.qo_indptr = qo_indptr;
  a.tok_indptr = tok_indptr;
  a.window = window;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.status = static_cast<uint32_t*>(scratch);
  a.sm_scale = sm_scale;
  a.heads = plan->num_qo_heads;
  a.batch = plan->batch;
  a.max_kv_len = plan->max_kv_len;
  a.rows = plan->rows;
  a.tokens = plan->tokens;
  a.causal = causal ? 1 : 0;
  const int64_t blocks = (static_cast<int64_t>(plan->rows) * plan->num_qo_heads + 7) / 8;
  if (blocks > 0x7fffffffLL) return PDA_ERR_INVALID;
  prefill<<<static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}
