// pda_mla.cu -- the products of latent attention with a head's W_UK and W_UV:
// the query absorbed and the output projected around pda_decode, and the
// cached latents gathered and expanded into keys and values for a prefill.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pda.h"
#include "pda_internal.h"

namespace pda {
namespace {

constexpr int kLat = 512;         // latent channels the products run over
constexpr int kRope = 64;
constexpr int kLatRow = kLat + kRope;
constexpr int kNope = 128;        // channels of a key (without rope) and of a value
constexpr int kQDim = kNope + kRope;

__device__ __forceinline__ float bf(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// ------------------------------------------------------ gather of latents
//
// One warp per token: its request by binary search in tok_indptr, its page
// slot, then the row dequantised to bf16. Chunks of 8 channels per lane.
// Bound: HBM / latency; the expansion that follows writes Hq x 512 bytes a token.

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
    page = __ldg(a.page_table + __ldg(a.kv_indptr + lo) + (i >> a.page_shift));
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
          uint32_t h;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(code));
          const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
          // one rounding to bf16: the products' operand type (2^-9 relative)
          const __nv_bfloat162 r = __floats2bfloat162_rn(f.x * s, f.y * s);
          out[e] = *reinterpret_cast<const uint32_t*>(&r);
        }
        o = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
    dst[c] = o;
  }
}

// ------------------------------------------------------- products per head
//
// C_h[t, n] = sum_k A_h[t, k] B_h[n, k]: one CTA per head, 64 tokens and 64
// columns, fp32 sums in registers (4 x 4 per thread), operands widened into
// shared memory 32 channels at a time.

struct ProductArgs {
  const __nv_bfloat16* a;
  int64_t a_row, a_head;
  const __nv_bfloat16* b;     // absorb: W_UK; project: W_UV; expand: W_UK
  const __nv_bfloat16* b2;    // expand: W_UV
  int64_t b_head;
  void* out;                  // absorb, project: out; expand: k
  __nv_bfloat16* out2;        // expand: v
  int64_t o_row, o_head;
  const int32_t* num_rows;
  float q_scale;
  int rows, k, n, e4m3;
};

enum { kAbsorb = 0, kProject = 1, kExpand = 2 };

template <int OP>
__global__ void __launch_bounds__(256) product(const __grid_constant__ ProductArgs p) {
  __shared__ float sa[32][65], sb[32][65];
  int rows = p.rows;
  if (p.num_rows) rows = min(rows, __ldg(p.num_rows));
  const int t0 = blockIdx.x * 64, n0 = blockIdx.y * 64, h = blockIdx.z;
  if (t0 >= rows) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += 32) {
    for (int e = tid; e < 64 * 32; e += 256) {
      const int r = e >> 5, k = k0 + (e & 31);
      sa[e & 31][r] = t0 + r < rows ? bf(p.a + (t0 + r) * p.a_row + h * p.a_head + k) : 0.f;
      const int n = n0 + r;
      const __nv_bfloat16* b = p.b + h * p.b_head;
      float v;
      if (OP == kAbsorb) v = bf(b + static_cast<int64_t>(k) * kLat + n);
      else if (OP == kProject) v = bf(b + static_cast<int64_t>(n) * kLat + k);
      else v = bf((n < kNope ? b : p.b2 + h * p.b_head) + static_cast<int64_t>(n % kNope) * kLat + k);
      sb[e & 31][r] = v;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty * 4 + i;
    if (t >= rows) break;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      const int64_t o = t * p.o_row + h * p.o_head + n;
      if (OP == kExpand && n >= kNope) p.out2[o - kNope] = __float2bfloat16(acc[i][j]);
      else if (OP == kAbsorb && p.e4m3) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(__fdiv_rn(acc[i][j], p.q_scale)));
        static_cast<uint8_t*>(p.out)[o] = static_cast<uint8_t>(c);
      } else static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16(acc[i][j]);
    }
  }
  if (OP == kAbsorb && n0 == 0)  // the rope channels pass through
    for (int e = tid; e < 64 * kRope; e += 256) {
      const int64_t t = t0 + e / kRope;
      if (t >= rows) break;
      const int64_t o = t * p.o_row + h * p.o_head + kLat + e % kRope;
      const __nv_bfloat16 x = p.a[t * p.a_row + h * p.a_head + kNope + e % kRope];
      if (p.e4m3) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(0.f), "f"(__fdiv_rn(__bfloat162float(x), p.q_scale)));
        static_cast<uint8_t*>(p.out)[o] = static_cast<uint8_t>(c);
      } else static_cast<__nv_bfloat16*>(p.out)[o] = x;
    }
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
  if (rows < 0 || w_stride_head < kNope * kLat) return PDA_ERR_INVALID;
  if (w_stride_head % 8 || !a4(num_rows)) return PDA_ERR_ALIGNMENT;
  return PDA_OK;
}

template <int OP>
int launch_product(const pda_plan_t* plan, ProductArgs& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.rows + 63) / 64), static_cast<unsigned>(p.n / 64),
                  static_cast<unsigned>(plan->num_qo_heads));
  product<OP><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
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
  if (e4m3 && !(q_scale > 0.f && q_scale < INFINITY)) return PDA_ERR_INVALID;
  if (q_stride_head < kQDim || q_stride_row < kQDim) return PDA_ERR_INVALID;
  if (!a16(q) || !a16(w_uk) || !a16(q_lat) || q_stride_row % 8 || q_stride_head % 8)
    return PDA_ERR_ALIGNMENT;
  ProductArgs p = {};
  p.a = static_cast<const __nv_bfloat16*>(q);
  p.a_row = q_stride_row;
  p.a_head = q_stride_head;
  p.b = static_cast<const __nv_bfloat16*>(w_uk);
  p.b_head = w_stride_head;
  p.out = q_lat;
  p.o_row = static_cast<int64_t>(plan->num_qo_heads) * kLatRow;
  p.o_head = kLatRow;
  p.num_rows = num_rows;
  p.q_scale = q_scale;
  p.rows = rows;
  p.k = kNope;
  p.n = kLat;
  p.e4m3 = e4m3;
  return launch_product<kAbsorb>(plan, p, reinterpret_cast<cudaStream_t>(stream));
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
  p.a = static_cast<const __nv_bfloat16*>(o_lat);
  p.a_row = static_cast<int64_t>(plan->num_qo_heads) * kLat;
  p.a_head = kLat;
  p.b = static_cast<const __nv_bfloat16*>(w_uv);
  p.b_head = w_stride_head;
  p.out = out;
  p.o_row = static_cast<int64_t>(plan->num_qo_heads) * kNope;
  p.o_head = kNope;
  p.num_rows = num_rows;
  p.rows = rows;
  p.k = kLat;
  p.n = kNope;
  return launch_product<kProject>(plan, p, reinterpret_cast<cudaStream_t>(stream));
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
  ProductArgs p = {};
  p.a = static_cast<const __nv_bfloat16*>(latent);
  p.a_row = kLatRow;
  p.b = static_cast<const __nv_bfloat16*>(w_uk);
  p.b2 = static_cast<const __nv_bfloat16*>(w_uv);
  p.b_head = w_stride_head;
  p.out = k;
  p.out2 = static_cast<__nv_bfloat16*>(v);
  p.o_row = kv_stride_token;
  p.o_head = kv_stride_head;
  p.num_rows = tok_indptr + plan->batch;
  p.rows = tokens;
  p.k = kLat;
  p.n = 2 * kNope;
  return launch_product<kExpand>(plan, p, s);
}
