/*
 * pda.h -- paged split-KV decode attention for GB300 (sm_103a): the C ABI.
 *
 * The operation (per request b with R_b query rows and L_b cached tokens,
 * query row i, query head h, kv head g = h / (Hq / Hkv)):
 *
 *   p_i  = L_b - R_b + i                              row position
 *   V_i  = { j : j <= p_i, and j >= p_i - W_b + 1 if W_b > 0 }
 *   s_j  = sm_scale * (q_i,h . k_j,g)                 j in V_i
 *   out  = sum_j softmax(s)_j * v_j,g                 (bf16)
 *   lse  = ln sum_j exp(s_j)                          (fp32, natural log)
 *
 * with k, v the dequantised cache values (bf16 as stored; E4M3 codes times
 * the per-tensor or per-(token, kv head) scale). Sources, by page and
 * section:
 *  - "perf(attention): run up to 8 query rows per request in the triton
 *    decode kernel" (FreeToken PR #900), "Changes": up to 8 causal query
 *    rows per request (qo_indptr, max_q_len); stage 1 packs query rows x GQA
 *    heads on the M axis and keeps the KV split, each row limited to its own
 *    position and window; stage 2 merges per row; per-row split scratch for
 *    CUDA graphs; a CTA's query heads divide the GQA group.
 *  - same page, "End-to-end A/B": the fp8_per_token_head KV dtype.
 *  - "fp8 support" (FlashMLA PR #54), "Functionality": symmetric per-tensor
 *    FP8 scales.
 *  - "Naive Support for Hopper FP8 Prefill Kernel with Per-Head
 *    Quantization" (FlashInfer PR #869), item 3: QK dequantisation folded
 *    into sm_scale, PV dequantisation folded into the finalize step.
 *  - "[Feature Request] Support q_len > 1 for FP8 decode" (hpc-ops issue
 *    #4): the FP8 decode workload and its byte accounting.
 * Readings taken where the pages are silent: p_i as above (the R new tokens
 * are already in the cache); W counts keys including the row's own, W <= 0
 * means no window; an E4M3 query's scale is folded into sm_scale by the
 * caller; FP8 is OCP E4M3 (e4m3fn).
 *
 * Ownership: every pointer is borrowed. pda_decode allocates nothing, never
 * synchronises, and enqueues work only on `stream`, so it can be captured in
 * a CUDA graph; the same plan and scratch then serve any kv_len, page_table,
 * qo_indptr and window contents within the plan's maxima.
 * Errors: host-side checks return a negative PDA_ERR_* code and launch
 * nothing; the library never aborts and never throws across this ABI.
 * Inputs that only the device can see (a request with kv_len < rows, rows
 * above max_q_len, kv_len above max_kv_len, a page id outside
 * [0, num_pages)) set bits in a status word kept in the scratch header; the
 * affected request's outputs are left unwritten. Kernels never trap.
 */
#ifndef PDA_H_
#define PDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pda_stream_t; /* a cudaStream_t; NULL = legacy default stream */

/* Element types. PDA_INT8 (KV cache only): two's-complement codes whose value
 * is the code times the per-tensor or per-(token, kv head) scale; an int8
 * cache is named beside bf16 and fp8 in "perf(attention): run up to 8 query
 * rows per request in the triton decode kernel", Tested on. */
enum { PDA_BF16 = 0, PDA_E4M3 = 1, PDA_INT8 = 2 };
/* PDA_SCALE_MLA_BLOCK: the mixed-precision MLA latent the FlashMLA page's
 * reviewers accept ("fp8 support", FlashMLA PR #54: nope in 8 bits per token
 * and 128 channels, rope in 16 bits). Each (token, kv head) row of the cache
 * is a 640-byte record: 512 E4M3 nope codes, then the 64 bf16 rope channels;
 * strides are in bytes; k_scale = v_scale = fp32 [num_pages, P, Hkv, 4], the
 * scale of each 128-channel nope block. head_dim 576, head_dim_v 512,
 * kv_dtype PDA_E4M3, q_dtype PDA_BF16. */
enum { PDA_SCALE_NONE = 0, PDA_SCALE_TENSOR = 1, PDA_SCALE_TOKEN_HEAD = 2, PDA_SCALE_MLA_BLOCK = 3 };
enum { PDA_KERNEL_AUTO = 0, PDA_KERNEL_MMA = 1, PDA_KERNEL_TC = 2 };

#define PDA_OK 0
#define PDA_ERR_NULL (-1)        /* a required pointer is NULL */
#define PDA_ERR_INVALID (-2)     /* a size or count is out of range */
#define PDA_ERR_UNSUPPORTED (-3) /* head_dim / page_size / dtype combination not built */
#define PDA_ERR_ALIGNMENT (-4)   /* a base address or stride is not 16-byte aligned */
#define PDA_ERR_SCRATCH (-5)     /* split_scratch NULL or not 256-byte aligned */
#define PDA_ERR_CUDA (-6)        /* a CUDA runtime call failed (launch, device query) */
#define PDA_ERR_PLAN (-7)        /* plan not produced by pda_plan, or from another version */
#define PDA_ERR_TOO_LARGE (-8)   /* plan needs more scratch than pda_decode_static's array */

/* Size of the library's own split-scratch array used by pda_decode_static. */
#define PDA_STATIC_SCRATCH_BYTES (32u << 20)

/* Device status bits (sticky in the scratch header until pda_reset_status). */
#define PDA_STATUS_KV_LEN_LT_ROWS 0x1u  /* kv_len[b] < rows of request b */
#define PDA_STATUS_ROWS_GT_MAX 0x2u     /* rows of request b > max_q_len, or negative */
#define PDA_STATUS_KV_LEN_GT_MAX 0x4u   /* kv_len[b] > plan max_kv_len */
#define PDA_STATUS_PAGE_OOB 0x8u        /* a page id read from page_table outside [0, num_pages) */
#define PDA_STATUS_ROWS_GT_CAP 0x10u    /* qo_indptr[batch] > max_batch * max_q_len */
#define PDA_STATUS_WAIT_TIMEOUT 0x20u   /* a pipeline wait ran past its bound; the CTA gave up */
#define PDA_STATUS_SMEM_MISALIGNED 0x40u /* a stage-1 CTA's shared-memory window was not 1024-byte
                                            aligned; that CTA wrote nothing */
#define PDA_STATUS_TABLE_INVALID 0x80u  /* pda_build_tables: a negative length, or a block-table row or
                                           column out of range */
#define PDA_STATUS_NO_PAGES 0x100u      /* pda_build_tables: the free list ran out */
#define PDA_STATUS_TABLE_FULL 0x200u    /* pda_build_tables: page_table_cap or rows_cap reached */
#define PDA_STATUS_TOKENS_GT_CAP 0x400u /* tok_indptr[batch] > the call's tokens */

/* Everything the planner needs; plain values, no device pointers. */
typedef struct {
  int32_t num_qo_heads;    /* Hq, a multiple of num_kv_heads */
  int32_t num_kv_heads;    /* Hkv >= 1 */
  int32_t head_dim;        /* D: 64, 128, 256 or 512 (512: tcgen05 path, pages >= 8); 576 MLA */
  int32_t page_size;       /* P: power of two in [1, 256] */
  int32_t q_dtype;         /* PDA_BF16, or PDA_E4M3 (then kv_dtype must be PDA_E4M3) */
  int32_t kv_dtype;        /* PDA_BF16, PDA_E4M3 or PDA_INT8 (int8: head_dim <= 256) */
  int32_t scale_mode;      /* PDA_SCALE_NONE for bf16 KV; TENSOR or TOKEN_HEAD for E4M3 / int8;
                              MLA_BLOCK for MLA latent records (E4M3 KV, bf16 Q, 576 / 512) */
  int32_t max_batch;       /* upper bound of `batch` over the plan's lifetime */
  int32_t max_q_len;       /* 1..8: rows per request */
  int32_t max_kv_len;      /* upper bound of kv_len[b] */
  int32_t num_pages;       /* physical pages in k_pages / v_pages */
  int64_t kv_stride_page;  /* cache strides in elements: element (page, slot, kv head, c) */
  int64_t kv_stride_token; /*   lives at page*stride_page + slot*stride_token          */
  int64_t kv_stride_head;  /*   + head*stride_head + c; c is contiguous               */
  int32_t device;          /* CUDA device the plan is for */
  int32_t num_sms;         /* 0: query `device`; > 0: use this SM count (host-only planning) */
  const int32_t* host_kv_len; /* optional host copy of kv_len[batch] for eager planning */
  int32_t batch;           /* requests per call, <= max_batch; 0 = max_batch */
  int32_t chunk_pages;     /* 0: planner chooses the KV chunk per CTA; > 0: forced */
  int32_t kernel;          /* PDA_KERNEL_AUTO, _MMA (mma.sync path) or _TC (tcgen05 path) */
  int32_t head_dim_v;      /* value channels: 0 = head_dim. MLA decode ("fp8 support", FlashMLA
                              PR #54): head_dim 576 (512 latent + 64 rope), head_dim_v 512,
                              one latent cache passed as both k_pages and v_pages, V being its
                              first 512 channels; bf16, or E4M3 with an E4M3 query */
  int32_t wait_limit_us;   /* bound of every pipeline wait (stage 1 on the tcgen05 path, the
                              latent-attention calls), in microseconds; 0 = 2 s. A wait that
                              runs out sets PDA_STATUS_WAIT_TIMEOUT and its CTA gives up: in
                              stage 1 writing nothing; see the latent-attention calls for theirs */
  uint32_t inject;         /* test hooks, 0 in normal use: PDA_INJECT_* */
  /* optional host copies for exact eager planning, used with host_kv_len:
   * qo_indptr[batch + 1] (rows of each request) and window[batch]; NULL = every
   * request has max_q_len rows / no window. The plan stays valid for any
   * device contents within its maxima; these only tune its KV chunk. */
  const int32_t* host_qo_indptr;
  const int32_t* host_window;
} pda_params;

/* Test hooks (pda_params.inject). PDA_INJECT_WITHHOLD_KV: the tcgen05 stage-1 CTAs issue no K/V
 * loads at all, so their consumers' waits run out after wait_limit_us and
 * every CTA returns with PDA_STATUS_WAIT_TIMEOUT set and nothing written.
 * The products of latent attention, pda_mla_expand and pda_mla_prefill issue no
 * loads of their operands either; the other two hooks withhold those of one CTA of each of
 * pda_mla_expand's CTA pairs and touch no other call.
 * They exercise the timeout paths without a device fault. */
#define PDA_INJECT_WITHHOLD_KV 0x1u
#define PDA_INJECT_WITHHOLD_CTA0 0x2u
#define PDA_INJECT_WITHHOLD_CTA1 0x4u
#define PDA_INJECT_ALL 0x7u

/* The plan: plain data, owned by the caller, copied freely. Fields are
 * documented for inspection; pda_decode reads only what pda_plan wrote. */
typedef struct {
  uint32_t magic;          /* PDA_PLAN_MAGIC once planned */
  int32_t num_qo_heads, num_kv_heads, head_dim, page_size;
  int32_t q_dtype, kv_dtype, scale_mode;
  int32_t max_batch, max_q_len, max_kv_len, num_pages, batch;
  int64_t kv_stride_page, kv_stride_token, kv_stride_head;
  int32_t group;           /* Hq / Hkv */
  int32_t kernel;          /* resolved PDA_KERNEL_MMA or PDA_KERNEL_TC */
  int32_t rows_per_cta;    /* cap on query rows x heads packed in one CTA */
  int32_t heads_per_cta[9];/* [R]: q heads per CTA for a request with R rows (divides group) */
  int32_t head_blocks;     /* grid extent over head blocks = group / heads_per_cta[max_q_len] */
  int32_t chunk_pages;     /* KV pages per split (CTA) */
  int32_t max_splits;      /* splits per (request, kv head, head block) */
  int32_t num_sms;
  int64_t grid_ctas;       /* stage-1 CTAs per call */
  int64_t rows_cap;        /* max_batch * max_q_len: rows the scratch holds */
  int64_t scratch_bytes;   /* bytes of split_scratch the caller provides */
  int64_t scratch_lse_offset; /* byte offsets inside split_scratch */
  int64_t scratch_o_offset;
  int32_t stage1_smem_bytes;
  /* Requests [tail_from, batch) use chunks of tail_chunk_pages (and up to
   * tail_splits splits) instead of chunk_pages (head_splits): the planner
   * cuts the requests that would run in a last, partial wave of CTAs into
   * shorter chunks, laid out last in the grid. tail_from = batch: none. */
  int32_t tail_from;
  int32_t tail_chunk_pages;
  int32_t head_splits;
  int32_t tail_splits;
  int32_t head_dim_v;      /* value channels (= head_dim but for MLA) */
  int32_t device;          /* pda_params.device */
  int32_t wait_limit_us;   /* pda_params.wait_limit_us, 0 resolved to 2 s */
  uint32_t inject;         /* pda_params.inject */
  int32_t reserved[7];
} pda_plan_t;

#define PDA_PLAN_MAGIC 0x50444131u /* "PDA1" */

/* Plan one decode shape. Host-only (queries the SM count of params->device
 * unless params->num_sms > 0). Writes *out_plan and, when non-NULL,
 * *split_scratch_bytes (>= 256; the caller allocates that many device bytes,
 * 256-byte aligned, zeroes them once, and passes them to every pda_decode of
 * this plan). Returns PDA_OK or a negative PDA_ERR_* code. */
int pda_plan(const pda_params* params, pda_plan_t* out_plan, size_t* split_scratch_bytes);

/* Paged split-KV decode attention (stage 1: per-chunk partial attention of
 * every (request, kv head, head block, KV chunk); stage 2: per-row
 * log-sum-exp merge of the chunks of every (query row, q head)).
 *   q          [qo_indptr[batch], Hq, D] bf16, or E4M3 codes (q_dtype), rows
 *              of request b at [qo_indptr[b], qo_indptr[b+1]); 16-B aligned
 *   k_pages,   paged cache, bf16, E4M3 codes or int8 codes, strides from the plan;
 *   v_pages    16-B aligned; V is the first head_dim_v channels of each v row (MLA:
 *              pass the latent cache as both)
 *   page_table int32 CSR: pages of request b at [kv_indptr[b], kv_indptr[b+1]),
 *              at least ceil(kv_len[b] / P) of them; only those are read
 *   kv_indptr  int32 [batch + 1];  kv_len int32 [batch]
 *   qo_indptr  int32 [batch + 1], non-decreasing, rows per request <= max_q_len
 *   max_q_len  rows-per-request bound of this call, 1..plan max_q_len
 *   window     int32 [batch] sliding window per request (<= 0: none), or NULL
 *   sm_scale   logit scale (times the query's E4M3 scale when q is E4M3)
 *   k_scale,   NULL (bf16), fp32 [1] (per tensor) or fp32 [num_pages, P, Hkv]
 *              (E4M3 / int8)
 *   v_scale    (per token and kv head), device memory; v_scale per token and head
 *              not below 2^-90 of the largest one that a row sees: the weights are
 *              summed with it, and that of a token with a smaller one may be lost
 *              (a subnormal one: NaN)
 *   out        [qo_indptr[batch], Hq, head_dim_v] bf16
 *   lse        [qo_indptr[batch], Hq] fp32 natural-log LSE, or NULL
 *   split_scratch  plan->scratch_bytes of device memory (see pda_plan)
 * All device pointers; nothing is allocated or synchronised. */
int pda_decode(const pda_plan_t* plan, const void* q, const void* k_pages, const void* v_pages,
               const int32_t* page_table, const int32_t* kv_indptr, const int32_t* kv_len,
               const int32_t* qo_indptr, int32_t max_q_len, const int32_t* window,
               float sm_scale, const float* k_scale, const float* v_scale, void* out,
               float* lse, void* split_scratch, pda_stream_t stream);

/* pda_decode in two halves, for callers that schedule or time them apart.
 * `stages` is a mask: PDA_STAGE_PARTIAL enqueues stage 1 (the partial
 * attention of every KV chunk; requests whose rows have one chunk get their
 * final out / lse here, the others write partials to split_scratch);
 * PDA_STAGE_MERGE enqueues stage 2 (the per-row merge of those partials; no
 * launch when plan->max_splits is 1). Both bits = pda_decode. The merge
 * must follow stage 1 of the same call on the same stream, with the same
 * arguments. Other bits, or none, return PDA_ERR_INVALID. */
#define PDA_STAGE_PARTIAL 1u
#define PDA_STAGE_MERGE 2u
int pda_decode_stages(const pda_plan_t* plan, const void* q, const void* k_pages,
                      const void* v_pages, const int32_t* page_table, const int32_t* kv_indptr,
                      const int32_t* kv_len, const int32_t* qo_indptr, int32_t max_q_len,
                      const int32_t* window, float sm_scale, const float* k_scale,
                      const float* v_scale, void* out, float* lse, void* split_scratch,
                      uint32_t stages, pda_stream_t stream);

/* Quantise-on-append: write the R_b new tokens of every request into the
 * paged cache, the step before decode reads them ("perf(attention): run up
 * to 8 query rows per request in the triton decode kernel", End-to-end A/B:
 * the fp8_per_token_head cache; "fp8 support", Functionality: symmetric
 * per-tensor FP8). Row i < R_b of request b is token L_b - R_b + i; it lands
 * in page page_table[kv_indptr[b] + t / P], slot t % P, kv head h, with the
 * plan's strides. Per kv dtype and scale mode of the plan:
 *   bf16 cache             the bf16 values, copied;
 *   E4M3, per tensor       codes = RNE(sat(x / s)) with s = k_scale[0] (v_scale[0]), read;
 *   E4M3, per token-head   s = amax / 448 over the D values of (token, kv head)
 *                          (1 if amax = 0), written to k_scale / v_scale
 *                          [num_pages, P, Hkv], and codes = RNE(sat(x / s)).
 *   int8, per tensor       codes = RNE(clamp(x / s, +-127)), s read as for E4M3;
 *   int8, per token-head   s = amax / 127 (1 if amax = 0), written as for E4M3;
 *   MLA records            (PDA_SCALE_MLA_BLOCK, head_dim 576) k_new holds the latents:
 *                          per 128-channel block of the first 512, s = amax / 448 to
 *                          k_scale [num_pages, P, Hkv, 4] and codes = RNE(sat(x / s))
 *                          (a zero block: s = 0 and zero codes, so that it adds nothing
 *                          to any sum of the decode) at record bytes [0, 512); the 64
 *                          rope values copied as bf16 to
 *                          bytes [512, 640); v_new, v_pages and v_scale are not used and
 *                          may be NULL; k_new, k_pages and k_scale 16-byte aligned.
 * x / s is one fp32 division; sat clamps to +-448 (E4M3, OCP e4m3fn); RNE
 * ties go to the even code (int8: the even integer).
 *   k_new, v_new  bf16 [qo_indptr[batch], Hkv, D], rows in qo_indptr order
 *   k_pages, v_pages  the cache (written), layout and strides as planned
 *   page_table, kv_indptr, kv_len, qo_indptr  as for pda_decode (kv_len
 *                 counts the new tokens)
 *   k_scale, v_scale  NULL for bf16; fp32 [1] read (per tensor) or fp32
 *                 [num_pages, P, Hkv] written (per token-head)
 *   split_scratch only its status word is used: page ids outside
 *                 [0, num_pages), kv_len < rows and rows > max_q_len set the
 *                 pda_decode status bits and skip that request
 * Returns PDA_OK or a negative code from the host checks (nothing launched).
 * All device pointers; nothing is allocated or synchronised. */
int pda_append_kv(const pda_plan_t* plan, const void* k_new, const void* v_new,
                  const int32_t* page_table, const int32_t* kv_indptr, const int32_t* kv_len,
                  const int32_t* qo_indptr, int32_t max_q_len, void* k_pages, void* v_pages,
                  float* k_scale, float* v_scale, void* split_scratch, pda_stream_t stream);

/* pda_decode without a caller-provided split_scratch (the pages have no
 * counterpart: this serves callers that cannot allocate device memory, such
 * as a plugin whose host framework owns every allocation and hands it only
 * input and output pointers, or code that must not call cudaMalloc under its
 * host's memory budget). The split scratch lives in a fixed
 * PDA_STATIC_SCRATCH_BYTES array of the library's own device memory, which
 * every GPU that loads the library holds until the process exits. Arguments
 * are those of pda_decode minus split_scratch; the host-side checks are
 * pda_decode's and run before anything is enqueued. Returns
 * PDA_ERR_TOO_LARGE when plan->scratch_bytes exceeds the array, and
 * PDA_ERR_INVALID when the current device is not the plan's device (the
 * array is per device). Allocates nothing. All calls share the array and it
 * keeps the last call's contents; each call first clears the status word (an
 * async memset on `stream`). Calls whose GPU work overlaps race on the
 * array: serialise them (one stream). The array's device address is looked
 * up on every call made outside a stream capture; a call made while `stream`
 * is capturing reuses the last lookup on that device, so make the first call
 * on a device before any stream capture. Read or clear the array's status
 * bits with pda_get_status / pda_reset_status and split_scratch = NULL. */
int pda_decode_static(const pda_plan_t* plan, const void* q, const void* k_pages,
                      const void* v_pages, const int32_t* page_table, const int32_t* kv_indptr,
                      const int32_t* kv_len, const int32_t* qo_indptr, int32_t max_q_len,
                      const int32_t* window, float sm_scale, const float* k_scale,
                      const float* v_scale, void* out, float* lse, pda_stream_t stream);

/* ------------------------------------------------- around the decode step
 *
 * Block tables, append for any number of rows, and latent attention (MLA) in
 * its absorbed and its expanded form. The pages have no counterpart of these
 * calls; they make what pda_decode reads and use what it writes. Like
 * pda_decode they allocate nothing, never synchronise and enqueue work only
 * on `stream` (the plan's device must be the current one: PDA_ERR_INVALID),
 * so they can be captured in a CUDA graph; every pointer is borrowed device memory unless it says
 * otherwise. split_scratch: the plan's scratch, of which they use only the
 * status word (pda_mla_prefill: its own scratch). No rows (or tokens): PDA_OK,
 * nothing launched, the row pointers may be NULL. Index arrays hold int32
 * unless stated. Outputs must not overlap inputs. */

/* Arrays of pda_build_tables (device pointers, plain counts). */
typedef struct {
  const int32_t* cached_len; /* [batch] tokens of each request already cached, >= 0 */
  const int32_t* new_len;    /* [batch] tokens this step adds, >= 0 */
  const int32_t* request;    /* [batch] block_table row of each request, all different; NULL = row b */
  int32_t* block_table;      /* [table_rows, table_cols] page ids, rows table_stride apart: entry j of a
                                row holds tokens [jP, jP + P); entries below ceil(cached / P) are read,
                                the grown ones written */
  int64_t table_stride;      /* entries between rows, >= table_cols */
  const int32_t* free_pages; /* free list, taken from its end; at least free_count[0] entries */
  const int32_t* free_count; /* [1] */
  int32_t* free_left;        /* [1] written: free_count minus the pages taken; not free_count itself */
  int32_t* kv_len;           /* [batch] written: cached + new; neither of the two arrays themselves */
  int32_t* kv_indptr;        /* [batch + 1] written: CSR offsets into page_table */
  int32_t* page_table;       /* [page_table_cap] written: pages of every request, in order */
  int32_t* qo_indptr;        /* [batch + 1] written: offsets of the new rows */
  int32_t* tok_indptr;       /* [batch + 1] written: offsets of kv_len (pda_mla_expand); or NULL */
  int64_t* slot_map;         /* [rows_cap] written: page * P + slot of each new row; or NULL */
  int32_t* positions;        /* [rows_cap] written: position of each new row; or NULL */
  int32_t table_rows, table_cols, page_table_cap, rows_cap; /* block_table (page_table) may be NULL
                                where table_cols (page_table_cap) is 0 */
} pda_tables;

/* Block tables and slot maps of one step, from the request lengths. Request
 * b of plan->batch grows from cached_len[b] to kv_len[b] = cached + new
 * tokens; its new pages ceil(kv_len / P) - ceil(cached / P) come off the end
 * of the free list (request by request, in the order of b, the first page
 * from the list's last entry), go into its block_table row, and the request's
 * pages into page_table. Row i of the request is token cached + i.
 * The call reads free_count and writes free_left, so running it again with
 * the same inputs gives the same outputs; the next step passes free_left as
 * free_count (two words used in turn).
 * What a request cannot have, it does not get in part:
 *  - a request whose new pages end past the free list (counted over all the
 *    requests up to it, refused ones too) is left as it was: kv_len = cached,
 *    no rows, no new pages, its old pages listed; PDA_STATUS_NO_PAGES;
 *  - an invalid request (negative length, row or columns out of range,
 *    kv_len above the plan's max_kv_len: PDA_STATUS_KV_LEN_GT_MAX) is listed
 *    with kv_len 0, no rows and no pages; PDA_STATUS_TABLE_INVALID;
 *  - from the first request on whose pages, rows or tokens would pass
 *    page_table_cap, rows_cap or an int32 offset, every request is listed with
 *    kv_len 0, no rows and no pages; PDA_STATUS_TABLE_FULL.
 * Entries of page_table, slot_map and positions behind the last request are
 * left as they were. A page id outside [0, num_pages) is listed as it is; the
 * new rows in it get slot -1, and PDA_STATUS_PAGE_OOB is set. plan->batch may
 * be at most 65536. */
int pda_build_tables(const pda_plan_t* plan, const pda_tables* tables, void* split_scratch,
                     pda_stream_t stream);

/* Append through a slot map: row i of k_new / v_new goes to slot
 * slot_map[i] = page * P + slot of the plan's cache, every kv head of it, in
 * the formats of pda_append_kv, for any number of rows (a prefill). The MLA
 * latents (head_dim 576) are appended too: bf16, E4M3 per tensor or per token
 * (over all 576 channels), or records; their v arguments are not used and may
 * be NULL.
 *   k_new, v_new  bf16 [rows, Hkv, D], rows k_stride / v_stride elements apart
 *                 (multiples of 8, >= Hkv * D)
 *   slot_map      int64 [rows]; -1 = skip the row; other values outside
 *                 [0, num_pages * P) skip it and set PDA_STATUS_PAGE_OOB. Two
 *                 rows of one slot leave a mix of both there.
 *   rows          rows of k_new and slot_map (rows x Hkv below 2^31); num_rows, when not NULL, is one
 *                 device int32: only rows [0, min(rows, *num_rows)) are taken
 *                 (&qo_indptr[batch] in a captured step) */
int pda_append_slots(const pda_plan_t* plan, const void* k_new, int64_t k_stride,
                     const void* v_new, int64_t v_stride, const int64_t* slot_map, int32_t rows,
                     const int32_t* num_rows, void* k_pages, void* v_pages, float* k_scale,
                     float* v_scale, void* split_scratch, pda_stream_t stream);

/* Latent attention. A head's query has 192 channels: 128 without position
 * (nope) and 64 rotated (rope); a token's latent c has 512 channels beside its
 * 64-channel rope key, shared by all heads. With a head's weights W_UK and
 * W_UV [128, 512], its key is [W_UK c, rope] and its value W_UV c:
 *   absorbed: q_lat = [W_UK^T q_nope, q_rope] meets the latent itself
 *             (pda_decode, head_dim 576), and out = W_UV o_lat;
 *   expanded: k = W_UK c and v = W_UV c are made once for a prefill.
 * The plan is an MLA plan (head_dim 576, head_dim_v 512, one kv head);
 * num_qo_heads is the number of heads. Weights are bf16, heads w_stride_head
 * elements apart (a multiple of 8), rows of 512 contiguous: [Hq, 256, 512] with
 * W_UK first is w_uk = w, w_uv = w + 128 * 512, w_stride_head = 256 * 512.
 * Rows, and tokens of pda_mla_expand, are at most 8388480 a call (row tiles of 128
 * in a grid's z): more is PDA_ERR_INVALID.
 * num_rows (device int32 [1], or NULL) bounds the rows as in
 * pda_append_slots; rows past it are left as they were. All sums are fp32,
 * rounded once to the output type. The plan's wait_limit_us bounds every wait
 * of these calls and of a prefill; after PDA_STATUS_WAIT_TIMEOUT none of the
 * call's outputs may be used: the rows of the CTAs that gave up are left as they
 * were (a prefill in key chunks still joins them from what its scratch holds),
 * others are written. The next call on the same scratch is a normal one. */

/* q_lat[t, h, :512] = sum_d q[t, h, d] W_UK[h, d, :] (d < 128), and
 * q_lat[t, h, 512:] = q[t, h, 128:].
 *   q      bf16 [rows, Hq, 192], strides in elements (multiples of 8)
 *   q_lat  [rows, Hq, 576] contiguous, the plan's q_dtype: bf16, or E4M3 codes
 *          RNE(sat(x * (1 / q_scale))) in fp32 (q_scale and its reciprocal
 *          positive and finite; pda_decode's sm_scale takes the scale) */
int pda_mla_absorb(const pda_plan_t* plan, const void* q, int64_t q_stride_row,
                   int64_t q_stride_head, const void* w_uk, int64_t w_stride_head, float q_scale,
                   void* q_lat, int32_t rows, const int32_t* num_rows, void* split_scratch,
                   pda_stream_t stream);

/* out[t, h, d] = sum_c o_lat[t, h, c] W_UV[h, d, c]: o_lat bf16 [rows, Hq, 512]
 * as pda_decode wrote it, out bf16 [rows, Hq, 128], both contiguous. */
int pda_mla_project(const pda_plan_t* plan, const void* o_lat, const void* w_uv,
                    int64_t w_stride_head, void* out, int32_t rows, const int32_t* num_rows,
                    void* split_scratch, pda_stream_t stream);

/* Keys and values of cached tokens, through the page table: token i of
 * request b (i < tok_indptr[b + 1] - tok_indptr[b]) is row tok_indptr[b] + i.
 *   k_pages     the latent cache as planned (bf16, E4M3 or records); k_scale as
 *               for pda_decode (NULL for bf16)
 *   tok_indptr  [batch + 1], non-decreasing, from 0
 *   latent      bf16 [tokens, 576] contiguous, written: the dequantised latents
 *               (their last 64 channels are the rope keys). The products read
 *               these rounded values.
 *   k, v        bf16 [tokens, Hq, 128], written; strides in elements (multiples
 *               of 8) shared by both
 *   tokens      rows of latent, k and v; rows past tok_indptr[batch] are left
 *               as they were
 * A token whose page id is out of range, or that lies behind its request's
 * pages in page_table (PDA_STATUS_PAGE_OOB), or whose request has more than the
 * plan's max_kv_len tokens (PDA_STATUS_KV_LEN_GT_MAX), reads as zeros.
 * tok_indptr[batch] > tokens sets PDA_STATUS_TOKENS_GT_CAP and writes the first
 * `tokens` rows. */
int pda_mla_expand(const pda_plan_t* plan, const void* k_pages, const int32_t* page_table,
                   const int32_t* kv_indptr, const int32_t* tok_indptr, const float* k_scale,
                   const void* w_uk, const void* w_uv, int64_t w_stride_head, void* latent,
                   void* k, void* v, int64_t kv_stride_token, int64_t kv_stride_head,
                   int32_t tokens, void* split_scratch, pda_stream_t stream);

/* The plan of a prefill: plain data, as pda_plan_t. */
typedef struct {
  uint32_t magic;         /* PDA_PREFILL_MAGIC once planned */
  uint32_t struct_bytes;  /* sizeof(pda_prefill_plan_t) as compiled */
  int32_t num_qo_heads, batch, max_kv_len, num_sms, device;
  int32_t rows, tokens;   /* capacities: rows of q, tokens of k / v */
  int32_t tiles;          /* bound on the 256-row tiles of all requests */
  int32_t splits;         /* bound on the key chunks of a tile; 1: not split */
  int32_t chunk_tokens;   /* keys per chunk, a multiple of 128 */
  int32_t wait_limit_us;
  uint32_t inject;        /* pda_params.inject */
  int32_t reserved[2];
  int64_t scratch_bytes;
} pda_prefill_plan_t;

#define PDA_PREFILL_MAGIC 0x50444631u /* "PDF1" */

/* Plan prefills of up to `rows` query rows and `tokens` keys in all, for the
 * heads, batch (at most 8192), max_kv_len and device of `plan` (an MLA plan); both
 * >= 1. Host-only. Whether few rows are cut into key chunks goes by these
 * capacities, not by the lengths on the device: where heads x tiles (256-row
 * tiles of all requests, at most min(rows, rows / 256 + batch)) are at most half
 * the SMs. A program whose steps differ keeps a plan for large ones and one for few
 * rows (64 rows on 8064 keys, 16 heads: 25 us from a plan of 64 rows, 59 from
 * one of 1024, 104 from one of 4096).
 * Writes *out_plan and, when non-NULL, *scratch_bytes (>= 256): device bytes
 * that the caller allocates as for pda_plan (256-byte aligned, zeroed once);
 * pda_get_status reads and pda_reset_status clears its status word. Calls that
 * share a scratch must not overlap: the work counters and the partial outputs
 * are in it. plan->wait_limit_us bounds each wait of a call too; the longest one
 * lasts about as long as three requests' 256-row tiles take (1.7 us for every 128
 * keys each). */
int pda_prefill_plan(const pda_plan_t* plan, int32_t rows, int32_t tokens,
                     pda_prefill_plan_t* out_plan, size_t* scratch_bytes);

/* Expanded latent attention of ragged requests: request b has the query rows
 * [qo_indptr[b], qo_indptr[b + 1]), any number of them, and the keys
 * [tok_indptr[b], tok_indptr[b + 1]); with R rows and L keys, row i sits at
 * p_i = L - R + i and sees, when causal, the keys j <= p_i, and with window[b]
 * = W > 0 also only j >= p_i - W + 1; when not causal (window must be NULL) all
 * L keys. s_j = sm_scale (q_nope . k_j + q_rope . k_rope_j), out = sum_j
 * softmax(s)_j v_j (bf16), lse = ln sum_j exp(s_j) (fp32 or NULL). A row that
 * sees no key (not causal, L = 0) gets out = 0 and lse = -inf.
 *   q       bf16 [rows, Hq, 192], strides in elements (multiples of 8)
 *   k, v    bf16 [tokens, Hq, 128], strides in elements shared by both
 *   k_rope  bf16 [tokens, 64], k_rope_stride elements apart (latent + 512, 576)
 *   out     bf16 [rows, Hq, 128] contiguous; lse fp32 [rows, Hq]
 * Keys and values of a request must be finite for its own rows to be; other
 * requests' and unused rows may hold anything. A request is left unwritten,
 * and its bit set, when its rows are negative (PDA_STATUS_ROWS_GT_MAX), when
 * it is causal with L < R (PDA_STATUS_KV_LEN_LT_ROWS), has L above the plan's
 * max_kv_len (PDA_STATUS_KV_LEN_GT_MAX), or ends past `rows`
 * (PDA_STATUS_ROWS_GT_CAP) or `tokens` (PDA_STATUS_TOKENS_GT_CAP). The weights
 * meet the values in bf16; their sum stays fp32. */
int pda_mla_prefill(const pda_prefill_plan_t* plan, const void* q, int64_t q_stride_row,
                    int64_t q_stride_head, const void* k, const void* v, int64_t kv_stride_token,
                    int64_t kv_stride_head, const void* k_rope, int64_t k_rope_stride,
                    const int32_t* qo_indptr, const int32_t* tok_indptr, const int32_t* window,
                    int32_t causal, float sm_scale, void* out, float* lse, void* scratch,
                    pda_stream_t stream);

/* ------------------------------------------------------- pages that are shared
 *
 * Requests that continue from the same tokens share the pages of them: a fork lists
 * its parent's pages in its own block table row. The pages have no counterpart of
 * these calls. A page is live while a request holds it, however many do, and what
 * requests hold is what their block table rows say; nothing else is counted. The rules
 * of the calls around decode hold: nothing allocated or synchronised, `stream` only,
 * the plan's device current, int32 index arrays on the device, and the same inputs
 * give the same outputs. */

/* Arrays of pda_fork_tables. */
typedef struct {
  const int32_t* parent;     /* [forks] block_table row shared from */
  const int32_t* child;      /* [forks] block_table row written; all different, none of them a parent */
  const int32_t* shared_len; /* [forks] tokens shared, 0 to the parent's length */
  int32_t* block_table;      /* [table_rows, table_cols] as for pda_build_tables; NULL with no columns */
  int64_t table_stride;
  const int32_t* free_pages; /* free list, taken from its end */
  const int32_t* free_count; /* [1] */
  int32_t* free_left;        /* [1] written; not free_count itself */
  int32_t* child_len;        /* [forks] written: shared_len, or 0 (below); not shared_len itself */
  int32_t* copy_src;         /* [forks] written: page to copy, -1: none (pda_copy_pages) */
  int32_t* copy_dst;         /* [forks] written: the child's page for it, or -1 */
  int32_t* copy_tokens;      /* [forks] written: tokens of it that are shared, or 0 */
  int32_t table_rows, table_cols, forks; /* forks: 0 to 65536 */
} pda_forks;

/* Fork requests: child row f lists the first floor(shared_len / P) pages of its
 * parent's row. Where shared_len ends inside a page, which parent and child would
 * both append to, the child gets a page of its own (off the free list's end, forks
 * in order) and the copy lists name what to copy into it, in every layer's cache.
 * A fork whose page lies past the free list (counted over all the forks up to it)
 * is not made: child_len 0, its row left as it was; PDA_STATUS_NO_PAGES. The same
 * for an invalid one (rows out of range or equal, shared_len negative, above the
 * plan's max_kv_len or the columns): PDA_STATUS_TABLE_INVALID (and KV_LEN_GT_MAX).
 * Page ids out of range are listed as they are, but not copied:
 * PDA_STATUS_PAGE_OOB. Entries of a child's row behind shared_len stay as they were. */
int pda_fork_tables(const pda_plan_t* plan, const pda_forks* forks, void* split_scratch,
                    pda_stream_t stream);

/* Copy pages of one cache: K, V and, where the plan's scales are per token, the
 * scales, from page copy_src[i] to copy_dst[i]. No page may be a destination twice,
 * or a source and a destination.
 *   copy_tokens  [copies] tokens of each page to copy (its first ones); NULL = all
 *   copies       entries of the lists; num_copies, when not NULL, is one device
 *                int32: only the first min(copies, *num_copies) are taken
 *   v_pages, v_scale  not used for latents (head_dim 576)
 * An entry with -1 in either list is skipped; another page outside [0, num_pages)
 * too, and sets PDA_STATUS_PAGE_OOB. */
int pda_copy_pages(const pda_plan_t* plan, void* k_pages, void* v_pages, float* k_scale,
                   float* v_scale, const int32_t* copy_src, const int32_t* copy_dst,
                   const int32_t* copy_tokens, int32_t copies, const int32_t* num_copies,
                   void* split_scratch, pda_stream_t stream);

/* Arrays of pda_free_pages and pda_compact_pages. */
typedef struct {
  const int32_t* lengths;    /* [requests] tokens of every request that holds pages, >= 0 */
  const int32_t* request;    /* [requests] block_table row of each, all different; NULL = row b */
  const int32_t* block_table; /* [table_rows, table_cols] page ids; entries below ceil(length / P) count */
  int64_t table_stride;
  int32_t* free_pages;       /* [num_pages] written: the free list, free_left entries */
  int32_t* free_left;        /* [1] written: its length */
  /* pda_compact_pages only: */
  int32_t* new_table;        /* written: the rows after the moves, as far as they count; strided as
                                block_table, which it may be */
  int32_t* copy_src;         /* [max_copies] written: pages to move (pda_copy_pages) */
  int32_t* copy_dst;         /* [max_copies] written: where to */
  int32_t* num_copies;       /* [1] written: how many */
  int32_t requests, table_rows, table_cols, max_copies;
} pda_pages;

/* Bytes of the page_scratch of both calls (256-byte aligned, zeroed once, not
 * shared by calls that overlap); pda_get_status reads and pda_reset_status clears its
 * status word. */
int pda_pages_scratch(const pda_plan_t* plan, size_t* scratch_bytes);

/* The free list from what is held: every page of [0, num_pages) that no listed
 * request holds, from the highest id to the lowest, which pda_build_tables takes
 * first. Requests that are gone, or shorter than they were, are all that a page
 * needs to become free. Every request that holds pages has to be listed, a kept
 * prompt's as well. What an invalid request lists stays held: a length above the
 * columns counts all of them (PDA_STATUS_TABLE_INVALID), above the plan's max_kv_len
 * also PDA_STATUS_KV_LEN_GT_MAX; a negative length or a row out of range lists
 * nothing (PDA_STATUS_TABLE_INVALID). Page ids out of range are passed over
 * (PDA_STATUS_PAGE_OOB). Entries of free_pages behind free_left stay as they were. */
int pda_free_pages(const pda_plan_t* plan, const pda_pages* pages, void* page_scratch,
                   pda_stream_t stream);

/* pda_free_pages, with the live pages moved to the lowest ids: the k-th highest
 * live page goes to the k-th lowest free one, while that lies below it, for at most
 * max_copies pages. The free list and new_table are those after the moves; the
 * caller runs pda_copy_pages (every layer's cache, num_copies) before it uses them.
 * Other tables that name pages (page_table, slot_map) are stale then. */
int pda_compact_pages(const pda_plan_t* plan, const pda_pages* pages, void* page_scratch,
                      pda_stream_t stream);

/* ------------------------------------------------ decode behind shared prefixes
 *
 * pda_decode for requests that continue from the same tokens: the pages that the
 * block tables of a group's requests have in common in front are read once, for the
 * rows of all of them, and only a request's own tokens are read for it alone. The
 * results are pda_decode's. Caches of head_dim 64, 128 and 256 in every kv dtype and
 * scale mode, pages of 8 tokens and more; the latent of MLA (head_dim 576) and
 * head_dim 512 are PDA_ERR_UNSUPPORTED: share its pages, and call pda_decode. */

/* The plan: plain data, as pda_plan_t. */
typedef struct {
  uint32_t magic;         /* PDA_SHARED_MAGIC once planned */
  uint32_t struct_bytes;  /* sizeof(pda_shared_plan_t) as compiled */
  pda_plan_t own;         /* the requests' own tokens: stage 1 of pda_decode */
  int32_t groups;
  int32_t max_kv_len;     /* of the plan given; own.max_kv_len bounds the own tokens */
  int64_t first_offset, main_lse_offset, main_o_offset, area_lse_offset, area_o_offset;
  int64_t scratch_bytes;
  int32_t reserved[4];
} pda_shared_plan_t;

#define PDA_SHARED_MAGIC 0x50445331u /* "PDS1" */

/* Arrays of one step (device pointers). */
typedef struct {
  const int32_t* page_table;   /* the step's tables, as for pda_decode (pda_build_tables) */
  const int32_t* kv_indptr;    /* [batch + 1] */
  const int32_t* kv_len;       /* [batch] */
  const int32_t* qo_indptr;    /* [batch + 1] */
  const int32_t* window;       /* [batch] or NULL */
  const int32_t* group_indptr; /* [groups + 1] the requests of each group, side by side: from 0 to
                                  batch, none below one in front; NULL = one group of all (groups 1) */
  int32_t* prefix;             /* [groups, 2] written: tokens [first, end) of the prefix that the
                                  group's rows see */
  int32_t* own_indptr;         /* [batch] written: a request's own pages in page_table; not kv_indptr */
  int32_t* own_len;            /* [batch] written: its own tokens; not kv_len */
} pda_shared_tables;

/* Plan decodes of the plan's batch in `groups` groups (1 to 1024), with at most
 * max_own_len own tokens a request (0: the plan's max_kv_len; a tight bound plans
 * better chunks). A request that has more is left unwritten by pda_decode_shared
 * (PDA_STATUS_KV_LEN_GT_MAX). Host-only. Writes *out_plan and, when non-NULL,
 * *scratch_bytes, which the caller allocates as for pda_plan (256-byte aligned,
 * zeroed once, not shared by calls that overlap); pda_get_status with &out_plan->own
 * reads and pda_reset_status clears its status word. */
int pda_shared_plan(const pda_plan_t* plan, int32_t groups, int32_t max_own_len,
                    pda_shared_plan_t* out_plan, size_t* scratch_bytes);

/* What the requests of each group share, once a step: with L tokens and R rows of a
 * request, the prefix ends behind the whole pages whose ids all its requests list
 * alike, at most (L - R) / P of them, so that every row stands behind it; `first` is
 * the first token that a row sees (0 without windows), rounded down to a page, at most
 * `end`. Own tokens are the L - end behind it, R of them at least. A request without
 * rows takes no part (own_len 0), nor does an invalid one (own_len -1; L < R, R out
 * of range or L above max_kv_len, with pda_decode's status bits); a page id out of
 * range ends a prefix. A group whose bounds are no requests, or one that starts in front of
 * an earlier bound, is left unwritten, and so are requests of no valid group
 * (PDA_STATUS_TABLE_INVALID). */
int pda_share_tables(const pda_shared_plan_t* plan, const pda_shared_tables* tables, void* scratch,
                     pda_stream_t stream);

/* Decode on the tables that pda_share_tables filled, as pda_decode: q, the caches,
 * scales, out, lse (or NULL), sm_scale and max_q_len are its arguments. An invalid
 * request's rows are left unwritten, with its status bits; so are those of a request
 * with more own tokens than planned, of one in no group or in an invalid one, and of one whose
 * rows are not among its group's (where another's are fewer than none).
 * Keys and values that a row does not see for its window have to be finite where
 * another row of its group sees them; pages that no row of the group sees may hold
 * anything, and so may their scales. After PDA_STATUS_WAIT_TIMEOUT the rows' values mean
 * nothing. */
int pda_decode_shared(const pda_shared_plan_t* plan, const void* q, const void* k_pages,
                      const void* v_pages, const pda_shared_tables* tables, int32_t max_q_len,
                      float sm_scale, const float* k_scale, const float* v_scale, void* out,
                      float* lse, void* scratch, pda_stream_t stream);

/* Copy the device status word of `split_scratch` to *host_bits. Synchronises
 * `stream`. split_scratch = NULL reads the status of pda_decode_static's
 * built-in array on the plan's device (which must be current). */
int pda_get_status(const pda_plan_t* plan, const void* split_scratch, uint32_t* host_bits,
                   pda_stream_t stream);

/* Clear the device status word (an async memset on `stream`); NULL clears
 * that of pda_decode_static's built-in array, as for pda_get_status. */
int pda_reset_status(const pda_plan_t* plan, void* split_scratch, pda_stream_t stream);

/* Static text for a PDA_ERR_* code. */
const char* pda_strerror(int code);

/* Library version (major * 10000 + minor * 100 + patch). */
int pda_version(void);

/* sizeof(pda_params) and sizeof(pda_plan_t) as compiled into the library, so
 * that a binding can check its own struct layout. Returns PDA_OK. */
int pda_struct_sizes(size_t* params_bytes, size_t* plan_bytes);

#ifdef __cplusplus
}
#endif

#endif /* PDA_H_ */
