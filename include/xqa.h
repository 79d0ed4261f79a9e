/*
 * xqa.h — C ABI of the paged E5M2-KV grouped-query decode-attention library
 * (libxqa.so, sm_103a).
 *
 * One decode step: every sequence b contributes one query token with Hq heads;
 * its keys and values live in a paged FP8 E5M2 cache; q head h attends over the
 * ctx_b cached tokens of kv head h / G (G = Hq / Hkv). This is the operation
 * the page "[Kernel][SM70] Pipeline batched E5M2 XQA decode" optimises: one
 * step for many long sequences at once, keys and values stored as E5M2
 * (sections "Purpose" and "Starting bottleneck"). The partial kernel below is built from the phases that page
 * times separately (section "Pending work and gates"): fetching and decoding
 * K, sharing it through shared memory, QK, fetching and decoding V, PV, and
 * the synchronisation between them. The split-KV
 * planner -> forward -> merge structure follows the page "[Kernel][WIP] Follow
 * up FlashNext batch HC fusion and QSA route audit" (section "Test Result").
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are CUDA device pointers (or managed memory)
 *     owned by the caller; the library never frees or retains them.
 *   - The library allocates no memory and reads no environment variables,
 *     never calls abort/exit and never synchronises except in the xqa_read_*
 *     helpers, which say so. Host state it keeps: a per-device "kernel
 *     attributes set" flag, SM count and cluster size that fits, and the cached
 *     cuTensorMapEncodeTiled entry point.
 *     Device state it keeps: the XQA_STATIC_WORKSPACE_BYTES array of
 *     xqa_decode_static_workspace (one per device, shared by every call of
 *     that entry point). Between calls, a caller's workspace keeps the merge
 *     tickets (all zero after every completed call) and the last call's
 *     status words.
 *   - Work is enqueued on `stream` (a cudaStream_t; 0 = legacy default stream)
 *     on the current device. A non-OK return means nothing was enqueued unless
 *     the code is XQA_ERR_LAUNCH.
 *   - Problems only the device can see (a block id outside [0, NB), a context
 *     length outside [0, MBS*BS], a pipeline wait that ran out of time) are
 *     recorded in the status words inside the workspace (read them with
 *     xqa_read_status); the affected (sequence, kv head) output rows are
 *     written as NaN, and no out-of-bounds address is ever read.
 */
#ifndef XQA_H_
#define XQA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum xqa_status {
  XQA_OK = 0,
  XQA_ERR_NULL = 1,        /* a required pointer is NULL */
  XQA_ERR_SHAPE = 2,       /* unsupported or inconsistent dimensions */
  XQA_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
  XQA_ERR_WORKSPACE = 4,   /* workspace smaller than xqa_workspace_size */
  XQA_ERR_LAUNCH = 5,      /* a CUDA call or kernel launch failed */
  XQA_ERR_DEVICE = 6,      /* no usable CUDA device / attribute query failed */
  XQA_ERR_VALUE = 7,       /* a scale that cannot be divided by (not finite, or <= 0) */
  /* written by the device into the workspace status word: */
  XQA_ERR_BAD_BLOCK_ID = 16,    /* block_tables entry outside [0, num_blocks) */
  XQA_ERR_CTX_TOO_LONG = 17,    /* context length < 0 or > MBS * block_size */
  XQA_ERR_DEVICE_TIMEOUT = 18,  /* a pipeline or merge-ticket wait exceeded its time budget */
  XQA_ERR_DRAIN_TIMEOUT = 19,   /* after a timeout, a copy was still in flight when its
                                   CTA exited: the device state is not to be trusted */
  XQA_ERR_BAD_OFFSETS = 20,     /* cu_seqlens descending, negative or past the rows */
  XQA_ERR_NO_PAGES = 21         /* no free page is left (or no room among the free pages) */
} xqa_status_t;

/* KV cache code formats (xqa_shape_t.kv_dtype). */
#define XQA_KV_E5M2 0 /* 1 sign, 5 exponent (bias 15), 2 mantissa bits */
#define XQA_KV_E4M3 1 /* 1 sign, 4 exponent (bias 7), 3 mantissa bits, no inf */
/* 4 bits: E2M1 codes (1 sign, 2 exponent bits of bias 1, 1 mantissa bit: 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6) with one E4M3 scale for every 16 dims of a token. A (page, kv
 * head) slice is XQA_E2M1_SLICE_BYTES contiguous bytes: 16 tokens x 64 code bytes
 * (dim 2i in the low nibble of byte i, dim 2i + 1 in the high one), then 16 tokens x
 * 8 scale bytes. The caches are [NB, Hkv, XQA_E2M1_SLICE_BYTES] (XQA_LAYOUT_HND
 * only), and a value is scale * E4M3(group scale) * E2M1(code). */
#define XQA_KV_E2M1 4
#define XQA_E2M1_SLICE_BYTES 1152

/* 16-bit element types of packed rows. */
#define XQA_F16 0
#define XQA_BF16 1

/* KV cache layouts (xqa_shape_t.kv_layout). */
#define XQA_LAYOUT_HND 0 /* [NB, Hkv, BS, D]: one (page, kv head) slice is contiguous */
#define XQA_LAYOUT_NHD 1 /* [NB, BS, Hkv, D]: token-major pages */

/* Problem dimensions. head_dim must be 128 and block_size 16; Hq must be a
 * multiple of Hkv, and G * q_len <= 16 with G = Hq / Hkv (so G <= 16). */
typedef struct xqa_shape {
  int32_t batch;              /* B: sequences (one query token each), >= 1 */
  int32_t num_q_heads;        /* Hq */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* D = 128 */
  int32_t block_size;         /* BS = 16 tokens per page */
  int32_t max_blocks_per_seq; /* MBS: row length of block_tables */
  int32_t num_blocks;         /* NB: pages in the K (and V) pool */
  float sm_scale;             /* softmax scale; <= 0 selects 1/sqrt(D) */
  int32_t max_ctas;           /* upper bound on split-KV CTAs; 0 = SM count;
                                 values above 1024 are taken as 1024 */
  int32_t min_pages_per_cta;  /* planner lower bound on pages per CTA; 0 = 16
                                 (XQA_KV_E2M1: at most max_blocks_per_seq) */
  int32_t merge_mode;         /* how segments split over several CTAs are merged:
                                 0 = inside the partial kernel (default), by the
                                 last CTA to finish one, or for a segment of
                                 more than 16 pieces (6 when G * q_len > 8) by
                                 its last CTAs to finish, each taking some of
                                 the rows (when max_ctas <= SM count, so that
                                 every CTA is resident at once);
                                 1 = by the separate combine kernel (xqa_combine) */
  int32_t kv_dtype;           /* XQA_KV_E5M2 (0, default), XQA_KV_E4M3 or XQA_KV_E2M1 */
  int32_t kv_layout;          /* XQA_LAYOUT_HND (0, default) or, with the 8-bit
                                 formats, XQA_LAYOUT_NHD */
  int32_t q_len;              /* T: new tokens per sequence; 0 or 1 = single-token
                                 decode. With T > 1, q and out are [B, T, Hq, D],
                                 context_lens count the T new tokens (their K/V
                                 already in the cache) and new token i attends
                                 causally to tokens 0 .. ctx_b - T + i (none if
                                 negative: a zero row). 8-bit formats: values of the
                                 new tokens are to be finite (one that is not reaches
                                 the new tokens before it too) */
} xqa_shape_t;

/* Bytes of device workspace xqa_decode needs for `shape` on the current
 * device (depends on the SM count when max_ctas == 0). Host only. */
xqa_status_t xqa_workspace_size(const xqa_shape_t* shape, size_t* bytes);

/* Number of kernels one xqa_decode call enqueues for `shape` (so a caller can
 * size CUDA graphs or count launches). Host only; *kernels receives 1, 2 or 3. */
xqa_status_t xqa_kernels_per_call(const xqa_shape_t* shape, int32_t* kernels);

/* One decode step of paged GQA attention.
 *
 *   q             device, fp16 [B, Hq, D] ([B, T, Hq, D] with q_len T > 1),
 *                 contiguous, 16-byte aligned
 *   k_cache       device, FP8 codes (shape->kv_dtype) in the shape->kv_layout
 *                 layout: [NB, Hkv, BS, D] (HND: one (page, kv head) slice is
 *                 BS*D = 2048 contiguous bytes) or [NB, BS, Hkv, D] (NHD),
 *                 16-byte aligned; XQA_KV_E2M1: 1152-byte slices (see above)
 *   v_cache       device, same layout as k_cache
 *   block_tables  device, int32 [B, MBS]; entry j of row b is the physical page
 *                 of tokens [16j, 16j+16) of sequence b; entries at or past
 *                 ceil(ctx_b / 16) are never read
 *   context_lens  device, int32 [B]; 0 <= ctx_b <= MBS*BS (0 gives a zero row)
 *   k_scale       per-tensor K scale (the key value is k_scale * FP8(code))
 *   v_scale       per-tensor V scale
 *   out           device, fp16, same shape as q, contiguous, 16-byte aligned
 *   workspace     device, >= xqa_workspace_size bytes, 256-byte aligned; holds
 *                 the plan, the split partials, the merge tickets, the
 *                 status words and each CTA's first pages of the last call
 *                 (a prefetch hint for the next call: any content is safe,
 *                 results never depend on it). Zero-fill it once before its
 *                 first use (e.g.
 *                 cudaMemsetAsync(workspace, 0, bytes)): every call leaves the
 *                 tickets at zero for the next. The tickets and status words
 *                 sit at fixed offsets, so one workspace may serve calls of
 *                 different shapes (sized for the largest). A call that is
 *                 not run to completion, or that reports
 *                 XQA_ERR_DEVICE_TIMEOUT or XQA_ERR_DRAIN_TIMEOUT (or
 *                 xqa_attend_partial with merge_mode 1 not followed by
 *                 xqa_combine) leaves it needing a fresh zero fill
 *
 * out[b, h, :] = sum_t softmax_t(sm_scale * <q[b,h], k_t>) * v_t over the
 * ctx_b tokens of kv head h / G, rounded to fp16 (round to nearest even). A token
 * whose logit is minus infinity (a key with an infinity) has weight 0; a row all of
 * whose logits are is zero, as one of an empty sequence, here and in xqa_prefill and
 * xqa_extend.
 * Kernels enqueued: the split-KV partial kernel, which derives the split plan
 * itself and merges split segments when merge_mode is 0; before it the planner
 * when the batch is too large for the partial kernel to hold the segment table
 * (B * Hkv + 1 > 2048); with merge_mode 1 the log-sum-exp combine after it.
 * The first kernel becomes resident while the previous kernel on the stream
 * still runs and waits for it to complete before reading any input. No host
 * synchronisation; the call may be captured into a CUDA graph. Concurrent
 * calls must not share a workspace. */
xqa_status_t xqa_decode(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens,
                        float k_scale, float v_scale, void* out, const xqa_shape_t* shape,
                        void* workspace, size_t workspace_bytes, void* stream);

/* xqa_decode with the per-tensor scales read from device memory when the
 * kernels run (so a captured CUDA graph picks up new scales on replay):
 * k_scale and v_scale are device pointers to one float each. Results are
 * bitwise equal to xqa_decode called with the same values. */
xqa_status_t xqa_decode_device_scales(const void* q, const uint8_t* k_cache,
                                      const uint8_t* v_cache, const int32_t* block_tables,
                                      const int32_t* context_lens, const float* k_scale,
                                      const float* v_scale, void* out, const xqa_shape_t* shape,
                                      void* workspace, size_t workspace_bytes, void* stream);

/* The three stages of xqa_decode, exposed separately so they can be timed one
 * by one. Called in this order with the same arguments they give exactly the
 * results of xqa_decode. xqa_plan always launches the planner kernel (which
 * publishes the plan in the workspace, see xqa_read_plan); xqa_decode
 * launches it only when the batch needs it (see xqa_kernels_per_call), and
 * xqa_attend_partial must then follow it on the same workspace. With
 * merge_mode 0 the partial kernel merges split segments itself and
 * xqa_combine enqueues nothing. */
xqa_status_t xqa_plan(const int32_t* context_lens, const xqa_shape_t* shape, void* workspace,
                      size_t workspace_bytes, void* stream);
xqa_status_t xqa_attend_partial(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                const int32_t* block_tables, const int32_t* context_lens,
                                float k_scale, float v_scale, void* out,
                                const xqa_shape_t* shape, void* workspace,
                                size_t workspace_bytes, void* stream);
xqa_status_t xqa_combine(const int32_t* context_lens, float v_scale, void* out,
                         const xqa_shape_t* shape, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Exact E5M2 dequantisation (the "E5M2 conversion" phase on its own):
 *   out_fp16_bits[i] = (uint16_t)in[i] << 8        (the fp16 pattern, exact)
 *   out_f32[i]       = (float)fp16(in[i]) * scale  (optional; NULL to skip)
 * in, out_fp16_bits, out_f32: device pointers, n elements each; any
 * alignment. */
xqa_status_t xqa_dequant_e5m2(const uint8_t* in, size_t n, float scale, uint16_t* out_fp16_bits,
                              float* out_f32, void* stream);

/* Exact E4M3 dequantisation with the conversion routes the attention kernel
 * uses for E4M3 caches (every E4M3 value is an fp16 value):
 *   out_fp16_bits[i] = fp16 pattern of E4M3(in[i])      (exact; NaN codes -> NaN)
 *   out_f32[i]       = (float)fp16 * scale              (optional; NULL to skip)
 * Same argument conventions as xqa_dequant_e5m2. */
xqa_status_t xqa_dequant_e4m3(const uint8_t* in, size_t n, float scale, uint16_t* out_fp16_bits,
                              float* out_f32, void* stream);

/* Packed rows of keys and values beside a paged cache (xqa_append, xqa_gather).
 * Row r holds one token's Hkv heads; sequence b owns the rows cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1. Strides are in elements, multiples of 8 (16 bytes); 0
 * selects the contiguous value (Hkv * 128 between rows, 128 between heads), so the
 * rows may be views of a wider tensor. */
typedef struct xqa_rows {
  int32_t batch;              /* B: sequences, >= 1 */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* D = 128 */
  int32_t block_size;         /* BS = 16 tokens per page */
  int32_t max_blocks_per_seq; /* MBS: row length of block_tables */
  int32_t num_blocks;         /* NB: pages in the K (and V) pool */
  int32_t num_rows;           /* rows of k and v (>= 0); rows that belong to no sequence
                                 (behind cu_seqlens[B]) are left alone */
  int32_t kv_dtype;           /* XQA_KV_E5M2, XQA_KV_E4M3 or XQA_KV_E2M1 */
  int32_t kv_layout;          /* XQA_LAYOUT_HND or (8-bit formats) XQA_LAYOUT_NHD */
  int32_t dtype;              /* XQA_F16 or XQA_BF16: type of k and v */
  int64_t k_row_stride, k_head_stride;
  int64_t v_row_stride, v_head_stride;
} xqa_rows_t;

/* Writes new tokens' keys and values into the paged cache.
 *
 *   k, v          device, rows->dtype [num_rows, Hkv, 128] (strided), 16-byte aligned
 *   cu_seqlens    device, int32 [B+1], ascending: sequence b's new rows
 *   block_tables  device, int32 [B, MBS], as for xqa_decode
 *   context_lens  device, int32 [B]: tokens of each sequence, the new ones counted, so
 *                 b's n_b rows go to positions ctx_b - n_b .. ctx_b - 1 (what
 *                 xqa_decode then expects)
 *   k_scale, v_scale  per-tensor scales; k_scale_dev / v_scale_dev, when not NULL,
 *                 point to one device float each, read when the kernel runs
 *   k_cache, v_cache  device, 16-byte aligned; only the new tokens' bytes are written
 *   device_status device int32 or NULL: receives XQA_ERR_CTX_TOO_LONG (a length below
 *                 0, above MBS * 16 or below n_b: none of the sequence's rows is
 *                 written) or XQA_ERR_BAD_BLOCK_ID (the token is not written) if it
 *                 holds XQA_OK; never cleared
 *
 * FP8: code = x / scale in 32 bits, rounded to nearest even, saturated; a NaN stays
 * a NaN code. E2M1, for each group of 16 dims: s = E4M3((max |x| / scale) / 6), code =
 * E2M1(x / (scale * s)), both to nearest even and saturated; a group whose s is 0
 * holds zeros, and one that has a NaN reads back as NaN throughout. Two rows must not
 * name the same cache slot. One kernel, no host synchronisation, no workspace; may be
 * captured into a CUDA graph. A host scale that is not finite or not above 0 is
 * refused (XQA_ERR_VALUE). A device scale is known to the kernel alone and divides as
 * it is, as IEEE division does: by 0, FP8 codes saturate (a NaN where x is 0). */
xqa_status_t xqa_append(const void* k, const void* v, const int32_t* cu_seqlens,
                        const int32_t* block_tables, const int32_t* context_lens, float k_scale,
                        float v_scale, const float* k_scale_dev, const float* v_scale_dev,
                        uint8_t* k_cache, uint8_t* v_cache, const xqa_rows_t* rows,
                        int32_t* device_status, void* stream);

/* Reads cached tokens back as packed rows: the other direction of xqa_append, with
 * the same arguments (k, v written, caches read). Sequence b's n_b rows receive its
 * tokens ctx_b - n_b .. ctx_b - 1 (all of them when n_b = ctx_b), each value scale *
 * code (scale * s * code) in 32 bits, rounded once to rows->dtype. Rows that
 * xqa_append would not write are written as NaN; rows behind the last sequence are
 * left as they are. */
xqa_status_t xqa_gather(const uint8_t* k_cache, const uint8_t* v_cache, const int32_t* cu_seqlens,
                        const int32_t* block_tables, const int32_t* context_lens, float k_scale,
                        float v_scale, const float* k_scale_dev, const float* v_scale_dev,
                        void* k, void* v, const xqa_rows_t* rows, int32_t* device_status,
                        void* stream);

/* Problem dimensions of xqa_prefill. Strides are in elements, multiples of 8 (16
 * bytes); 0 selects the contiguous value (heads * 128 between rows, 128 between
 * heads), so q, k and v may be views of one projection. */
typedef struct xqa_prefill_shape {
  int32_t batch;        /* B: sequences, >= 1 */
  int32_t num_q_heads;  /* Hq, a multiple of Hkv; G = Hq / Hkv <= 128 */
  int32_t num_kv_heads; /* Hkv */
  int32_t head_dim;     /* D = 128 */
  int32_t total_q;      /* rows of q and out (>= 0, total_q * Hq < 2^27) */
  int32_t total_k;      /* rows of k and v (>= 0, <= 2^31 - 512) */
  int32_t dtype;        /* XQA_F16 or XQA_BF16: q, k, v and out */
  int32_t causal;       /* 1: query i of a sequence sees keys 0 .. len_k - len_q + i
                           (the last query sees every key); 0: every key */
  float sm_scale;       /* softmax scale; <= 0 selects 1/sqrt(D) */
  int32_t max_ctas;     /* upper bound on CTAs; 0 = SM count */
  int64_t q_row_stride, q_head_stride;
  int64_t k_row_stride, k_head_stride;
  int64_t v_row_stride, v_head_stride;
  int64_t out_row_stride, out_head_stride;
} xqa_prefill_shape_t;

/* Bytes of device workspace xqa_prefill needs for `shape`. Host only. */
xqa_status_t xqa_prefill_workspace_size(const xqa_prefill_shape_t* shape, size_t* bytes);

/* Attention of whole prompts, packed by sequence.
 *
 *   q             device, shape->dtype [total_q, Hq, 128] (strided), 16-byte aligned
 *   k, v          device, [total_k, Hkv, 128] (strided), 16-byte aligned
 *   cu_seqlens_q  device, int32 [B+1], ascending: sequence b's rows of q and out
 *   cu_seqlens_k  device, int32 [B+1], ascending: its rows of k and v (as many as of q
 *                 for a whole prompt; more when the prompt goes on after cached
 *                 tokens; fewer is allowed)
 *   out           device, [total_q, Hq, 128] (strided), 16-byte aligned
 *   lse           device, fp32 [total_q, Hq] contiguous, or NULL: the natural
 *                 logarithm of the row's sum of exponentials
 *   workspace     device, >= xqa_prefill_workspace_size bytes, 256-byte aligned,
 *                 zero-filled once before its first use; every completed call leaves
 *                 it ready for the next. A decode workspace of at least that size may
 *                 serve both. Concurrent calls must not share one
 *
 * out[i, h] = sum_j softmax_j(sm_scale * <q[i, h], k[j, h / G]>) * v[j, h / G] over the
 * keys that query i sees. A row that sees none is zero, its lse -inf, and so is one whose
 * logits are all minus infinity. Products accumulate in 32 bits, the softmax is in 32
 * bits, its weights are rounded to shape->dtype for the second product, out is rounded
 * once. What a query does not see does not reach its row, infinities and NaN included.
 * Rows of q and out behind cu_seqlens_q[B] are left alone. A sequence whose offsets are
 * bad (XQA_ERR_BAD_OFFSETS, see xqa_read_status) is skipped, and where offsets descend so
 * that sequences overlap, some behind them may be; if only its key offsets are bad, its
 * rows are NaN. One kernel, no host synchronisation; may be captured into a CUDA graph. */
xqa_status_t xqa_prefill(const void* q, const void* k, const void* v, const int32_t* cu_seqlens_q,
                         const int32_t* cu_seqlens_k, void* out, float* lse,
                         const xqa_prefill_shape_t* shape, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Problem dimensions of xqa_extend. Strides are in elements, multiples of 8 (16 bytes); 0
 * selects the contiguous value (Hq * 128 between rows, 128 between heads), so q may be a
 * view of a projection. */
typedef struct xqa_extend_shape {
  int32_t batch;              /* B: sequences, >= 1 */
  int32_t num_q_heads;        /* Hq, a multiple of Hkv; G = Hq / Hkv <= 128 */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* D = 128 */
  int32_t block_size;         /* BS = 16 tokens per page */
  int32_t max_blocks_per_seq; /* MBS: row length of block_tables (<= 2^26) */
  int32_t num_blocks;         /* NB: pages in the K (and V) pool */
  int32_t total_q;            /* rows of q and out (>= 0, total_q * Hq < 2^27) */
  int32_t dtype;              /* XQA_F16 or XQA_BF16: q and out */
  int32_t kv_dtype;           /* XQA_KV_E5M2, XQA_KV_E4M3 or XQA_KV_E2M1 */
  int32_t kv_layout;          /* XQA_LAYOUT_HND or (8-bit formats) XQA_LAYOUT_NHD */
  int32_t causal;             /* 1: query i of a sequence's n sees its tokens 0 ..
                                 ctx - n + i; 0: every one */
  float sm_scale;             /* softmax scale; <= 0 selects 1/sqrt(D) */
  int32_t max_ctas;           /* upper bound on CTAs; 0 = SM count */
  int64_t q_row_stride, q_head_stride;
  int64_t out_row_stride, out_head_stride;
} xqa_extend_shape_t;

/* Bytes of device workspace xqa_extend needs for `shape`. Host only. */
xqa_status_t xqa_extend_workspace_size(const xqa_extend_shape_t* shape, size_t* bytes);

/* Attention of chunks of new tokens over the paged cache: any number of new tokens for
 * each sequence, from one to a whole prompt, their keys and values already in the cache
 * (xqa_append), read there as they lie.
 * Single tokens may stand beside chunks; where all or most sequences have one, xqa_decode
 * (of those sequences' rows of the tables) takes less time for them.
 *
 *   q             device, shape->dtype [total_q, Hq, 128] (strided), 16-byte aligned,
 *                 packed by sequence
 *   k_cache, v_cache  device, as for xqa_decode, 16-byte aligned
 *   block_tables  device, int32 [B, MBS], as for xqa_decode
 *   context_lens  device, int32 [B]: tokens of each sequence, the new ones counted
 *   cu_seqlens    device, int32 [B+1], ascending: sequence b's rows of q and out (none
 *                 for a sequence that has no part in the call)
 *   k_scale, v_scale  per-tensor scales; k_scale_dev / v_scale_dev, when not NULL, point
 *                 to one device float each, read when the kernel runs
 *   out           device, [total_q, Hq, 128] (strided), 16-byte aligned
 *   lse           device, fp32 [total_q, Hq] contiguous, or NULL: the natural logarithm of
 *                 the row's sum of exponentials
 *   workspace     device, >= xqa_extend_workspace_size bytes, 256-byte aligned, zero-filled
 *                 once before its first use; every completed call leaves it ready for the
 *                 next (a call that reports XQA_ERR_DEVICE_TIMEOUT or
 *                 XQA_ERR_DRAIN_TIMEOUT does not). A decode or prompt workspace of at
 *                 least that size may serve too. Concurrent calls must not share one
 *
 * out[i, h] = sum_t softmax_t(sm_scale * k_scale * <q[i, h], K_t>) * v_scale * V_t over
 * the tokens that query i sees. A row that sees none (a context shorter than the new
 * tokens) is zero, its lse -inf, and so is one whose logits are all minus infinity. Codes
 * are taken exactly; products accumulate in 32 bits, the softmax is in 32 bits, its
 * weights are rounded to shape->dtype for the second product, out is rounded once. What a
 * query does not see does not reach its row, infinities and NaN included. Rows behind
 * cu_seqlens[B] are left alone. Results do not depend on what else is in the batch beyond
 * the order of 32-bit sums (where a long sequence is cut into pieces).
 *
 * Errors that only the device sees (xqa_read_status): XQA_ERR_BAD_BLOCK_ID (the rows that
 * see a token of the page are NaN), XQA_ERR_CTX_TOO_LONG (the sequence's rows are NaN),
 * XQA_ERR_BAD_OFFSETS (the sequence is skipped; where offsets descend so that sequences
 * overlap beyond total_q rows, all are), XQA_ERR_VALUE (a device k_scale that is not
 * finite or not above 0: all rows are NaN). A host scale of that kind is refused. Two
 * kernels, no host synchronisation; may be captured into a CUDA graph. */
xqa_status_t xqa_extend(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                        const int32_t* block_tables, const int32_t* context_lens,
                        const int32_t* cu_seqlens, float k_scale, float v_scale,
                        const float* k_scale_dev, const float* v_scale_dev, void* out, float* lse,
                        const xqa_extend_shape_t* shape, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Pages of sequences that grow and end. The pool's free pages are a stack, free_pages[0 ..
 * num_free). */
typedef struct xqa_pages {
  int32_t batch;              /* B: sequences (places for them), 1 .. 16384 */
  int32_t block_size;         /* BS = 16 tokens per page */
  int32_t max_blocks_per_seq; /* MBS: row length of block_tables (< 2^27) */
  int32_t num_blocks;         /* NB: pages in the pool, entries of free_pages (< 2^27) */
  int32_t num_rows;           /* entries of slots and positions (< 2^30): the most new tokens
                                 that a call may assign; not used by xqa_release_pages */
} xqa_pages_t;

/* A step's block tables, offsets, slots and positions from the tokens that each sequence
 * gains.
 *
 *   new_tokens    device, int32 [B]: tokens that sequence b gains, 0 for none
 *   context_lens  device, int32 [B]: its tokens before
 *   block_tables  device, int32 [B, MBS]: entries ceil(c / 16) .. ceil((c + n) / 16) - 1 of
 *                 row b are written, the others left as they are
 *   free_pages    device, int32 [NB]; num_free: device, int32 [1]. Pages are taken from the
 *                 stack's end, sequence after sequence, each one's in the order of its table
 *   new_lens      device, int32 [B]: tokens after the step; may be context_lens
 *   new_free      device, int32 [1]: pages left; may be num_free
 *   cu_seqlens    device, int32 [B+1]: offsets of the new tokens' rows
 *   slots         device, int32 [num_rows], or NULL: page * 16 + position % 16 of each new
 *                 token; -1 in rows behind the last one
 *   positions     device, int32 [num_rows], or NULL: its position in the sequence, or -1
 *   device_status device int32 or NULL: receives the first of these errors if it holds
 *                 XQA_OK. A sequence that meets one gains nothing in this call, the others
 *                 do: XQA_ERR_CTX_TOO_LONG (a negative number or length, or more than MBS *
 *                 16 tokens), XQA_ERR_BAD_OFFSETS (its rows, behind those of every
 *                 sequence before it, would pass num_rows; so would every later one's),
 *                 XQA_ERR_NO_PAGES (the stack has too few pages for it and those before it;
 *                 later ones that need no page are served; a num_free below 0 or above NB
 *                 counts as 0, which new_free then is). XQA_ERR_BAD_BLOCK_ID: a page
 *                 outside [0, NB) in the stack or the table; entries are written as they
 *                 are, slots as -1
 *
 * What the next calls take: block_tables and new_lens as context_lens for all of them,
 * cu_seqlens for xqa_append, xqa_page_bounds and xqa_extend. One kernel, no host
 * synchronisation, no workspace; may be captured into a CUDA graph. */
xqa_status_t xqa_assign_pages(const int32_t* new_tokens, const int32_t* context_lens,
                              int32_t* block_tables, const int32_t* free_pages,
                              const int32_t* num_free, int32_t* new_lens, int32_t* new_free,
                              int32_t* cu_seqlens, int32_t* slots, int32_t* positions,
                              const xqa_pages_t* pages, int32_t* device_status, void* stream);

/* Pages of ended sequences back onto the stack: those of every b with done[b] != 0, in the
 * order of b and of its table, and new_lens[b] = 0 (context_lens[b] where done[b] is 0).
 *
 *   done          device, uint8 [B]
 *   block_tables  device, int32 [B, MBS]; not written: entries past a length are never read
 *   new_lens, new_free  as for xqa_assign_pages; free_pages[num_free ..] is written
 *   device_status as for xqa_assign_pages: XQA_ERR_BAD_BLOCK_ID (an entry outside [0, NB):
 *                 it is left out), XQA_ERR_CTX_TOO_LONG (a length below 0 or above MBS * 16:
 *                 none of the sequence's pages goes back), XQA_ERR_NO_PAGES (more than NB
 *                 pages would be free: those past NB are dropped; or num_free is below 0 or
 *                 above NB: the call releases nothing, free_pages stays, new_lens is
 *                 context_lens and new_free is num_free)
 * A page must not go back twice. One kernel, no host synchronisation, no workspace; may be
 * captured into a CUDA graph. */
xqa_status_t xqa_release_pages(const uint8_t* done, const int32_t* context_lens,
                               const int32_t* block_tables, int32_t* free_pages,
                               const int32_t* num_free, int32_t* new_lens, int32_t* new_free,
                               const xqa_pages_t* pages, int32_t* device_status, void* stream);

/* Bytes of a (page, kv head) slice of the bounds: 128 upper bounds (int8), 128 lower bounds
 * (int8), the exponent e (int8), 15 zeros. For every token t of the page that is in use
 * and every dim d: lower[d] * 2^e <= key[t][d] <= upper[d] * 2^e, the key before k_scale,
 * with 2^(e+6) <= max |key| < 2^(e+7) over the slice (e = 0 where all keys are 0) and the
 * bounds rounded away from the keys to whole numbers. e = -128, bounds 0: a key is not
 * finite. */
#define XQA_BOUNDS_BYTES 272

/* Bounds of the pages that a step's new tokens touched, computed anew from all their tokens.
 *
 *   k_cache, block_tables, context_lens, cu_seqlens  as for xqa_append, after it
 *   bounds        device, uint8 [NB, Hkv, XQA_BOUNDS_BYTES], 16-byte aligned
 *   rows          dimensions as for xqa_append; dtype and strides play no part
 *   device_status device int32 or NULL: as for xqa_append; pages that it would not write
 *                 keep their bounds
 * One kernel, no host synchronisation, no workspace; may be captured into a CUDA graph. */
xqa_status_t xqa_page_bounds(const uint8_t* k_cache, const int32_t* block_tables,
                             const int32_t* context_lens, const int32_t* cu_seqlens,
                             uint8_t* bounds, const xqa_rows_t* rows, int32_t* device_status,
                             void* stream);

/* Problem dimensions of xqa_select. */
typedef struct xqa_select_shape {
  int32_t batch;              /* B: sequences, >= 1 */
  int32_t num_q_heads;        /* Hq, a multiple of Hkv; G = Hq / Hkv <= 16 */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* D = 128 */
  int32_t block_size;         /* BS = 16 tokens per page */
  int32_t max_blocks_per_seq; /* MBS: row length of block_tables (<= 2^24) */
  int32_t num_blocks;         /* NB: pages in the pool */
  int32_t max_pages;          /* K: row length of selected */
  int32_t first_pages;        /* a sequence's first pages that are always taken, >= 0 */
  int32_t last_pages;         /* its last ones, >= 1 (the new token's page among them);
                                 first_pages + last_pages <= max_pages */
  int32_t max_ctas;           /* upper bound on CTAs; 0 = 2 per SM */
} xqa_select_shape_t;

/* Bytes of device workspace xqa_select needs for `shape`. Host only. */
xqa_status_t xqa_select_workspace_size(const xqa_select_shape_t* shape, size_t* bytes);

/* The pages that each sequence's new token is to read, for each kv head: all of them if
 * there are at most K, else the first and last ones and of the others those with the
 * highest scores, the lower page first among equal ones.
 *
 *   q             device, fp16 [B, Hq, 128], contiguous, 16-byte aligned
 *   bounds        device, as xqa_page_bounds writes them, up to date for every page of the
 *                 sequences
 *   block_tables, context_lens  device, as for xqa_decode
 *   selected      device, int32 [B, Hkv, K]: pages (ids of the pool) in the order of the
 *                 sequence, -1 behind the last
 *   selected_lens device, int32 [B, Hkv]: tokens in them; what xqa_decode_selected takes
 *   workspace     device, >= xqa_select_workspace_size bytes, 256-byte aligned, zero-filled
 *                 once before its first use; every completed call leaves it ready for the
 *                 next, of any shape. A workspace of another call of at least that size may
 *                 serve too. Concurrent calls must not share one
 *
 * score(page) = 2^e * sum_d (A_d * upper_d + B_d * lower_d), where A_d (B_d) is the sum of
 * the positive (negative) q8_gd over the G heads, q8 = q / 2^f rounded to nearest even, f
 * the whole number with 2^(f+5) <= max |q| < 2^(f+6) over the group's finite values (others
 * count as 0). The sum is in whole numbers and exact: a choice does not depend on the split
 * of the work or on the batch. Pages whose keys are not finite come before all scores, and
 * so do those whose id is outside [0, NB) (XQA_ERR_BAD_BLOCK_ID, see xqa_read_status):
 * xqa_decode_selected then meets them. A length below 0 or above MBS * 16
 * (XQA_ERR_CTX_TOO_LONG) gives selected_lens -1. One kernel, no host synchronisation; may
 * be captured into a CUDA graph. */
xqa_status_t xqa_select(const void* q, const uint8_t* bounds, const int32_t* block_tables,
                        const int32_t* context_lens, int32_t* selected, int32_t* selected_lens,
                        const xqa_select_shape_t* shape, void* workspace, size_t workspace_bytes,
                        void* stream);

/* xqa_decode over a table of its own for each (sequence, kv head): selected, int32 [B, Hkv,
 * K] with K = shape->max_blocks_per_seq, and selected_lens, int32 [B, Hkv], in place of
 * block_tables and context_lens (all pages but the last of a row are full). One new token
 * for each sequence (q_len 0 or 1); several go as so many sequences. k_scale_dev and
 * v_scale_dev: both NULL, or both pointers to one device float. Everything else is as for
 * xqa_decode, the workspace included. */
xqa_status_t xqa_decode_selected(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                 const int32_t* selected, const int32_t* selected_lens,
                                 float k_scale, float v_scale, const float* k_scale_dev,
                                 const float* v_scale_dev, void* out, const xqa_shape_t* shape,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Self-check of the device-side failure detection: launches one CTA whose
 * threads wait, through the same bounded mbarrier wait the attention kernel
 * uses, on a barrier that nothing ever arrives at. After budget_ns
 * (1 .. 2e9 ns) the wait gives up and the kernel writes XQA_ERR_DEVICE_TIMEOUT
 * to *device_status (a device int32) and returns; the context stays usable.
 * The attention kernel's budget is 1 s. Test use only. */
xqa_status_t xqa_selftest_wait_timeout(int32_t* device_status, uint64_t budget_ns, void* stream);

/* The device-reported status of the last call that used `workspace`:
 * *device_status receives XQA_OK or the first device-reported code in CTA
 * order (each CTA of the partial kernel writes its own status word as it
 * exits). Copies the fixed-size header/ticket/status region (12352 bytes) to
 * the host and synchronises `stream`. Returns XQA_ERR_WORKSPACE if the
 * workspace holds no status (neither zero-filled nor written by a call). */
xqa_status_t xqa_read_status(const void* workspace, int32_t* device_status, void* stream);

/* Copies the planner's output to host memory. Synchronises `stream`.
 *   header[4]          = {CTAs of the last partial launch, CTAs holding work,
 *                         total_pages, num_segments}
 *   seg_start[B*Hkv+1] = exclusive prefix sum of pages per (sequence, kv head)
 *   seg_bad[B*Hkv]     = 1 where the segment's context length is invalid,
 *                        else 0 (may be NULL)
 * The plan is published by the planner kernel when it runs, else by the
 * partial kernel's first CTA.
 *   seg_cost[B*Hkv]    = inclusive prefix sum of the segments' switch costs on
 *                        the cost line the CTAs are cut on: 32 page units per
 *                        non-empty segment, 0 for an empty one (may be NULL) */
xqa_status_t xqa_read_plan(const void* workspace, const xqa_shape_t* shape, int32_t* header,
                           int32_t* seg_start, int32_t* seg_bad, int32_t* seg_cost,
                           void* stream);

/* Size of the device array behind xqa_decode_static_workspace (per device). */
#define XQA_STATIC_WORKSPACE_BYTES ((size_t)8 << 20)

/* xqa_decode for callers that cannot allocate device memory.
 *
 * None of the pages describes this entry point. It exists for callers that
 * are not allowed to call cudaMalloc: a plugin inside a host runtime that owns
 * all device memory through its own pool, a latency-critical path where an
 * allocation (which may synchronise the device) is forbidden, or an operator
 * interface that passes only inputs and outputs and has no workspace hook.
 *
 * Arguments and results are those of xqa_decode, minus the workspace: the
 * split-KV scratch comes from a fixed XQA_STATIC_WORKSPACE_BYTES array in the
 * library's device image, which every device that loads the library holds
 * until the process exits. Nothing is allocated. The array is zero-filled when
 * the library's module loads on a device, and every completed call leaves it
 * ready for the next, so nothing needs clearing.
 *
 *   - Shapes whose xqa_workspace_size exceeds XQA_STATIC_WORKSPACE_BYTES are
 *     rejected with XQA_ERR_WORKSPACE before anything is enqueued (for 152
 *     SMs: B * Hkv up to about 850 segments).
 *   - Every call looks up the array's device address with
 *     cudaGetSymbolAddress, with the caller's device current (a host-side
 *     lookup; nothing is cached, so a device reset that reloads the module
 *     is followed). The first call on a device may load the library's module
 *     there: make it before any stream capture.
 *   - All calls on a device share the one array: calls that may overlap on the
 *     GPU (different streams without ordering, or threads racing on one device)
 *     race on it and corrupt each other. Order them, e.g. on one stream.
 *   - The device status words live in the shared array and are not exposed;
 *     rows affected by a bad block id or context length still come back NaN. */
xqa_status_t xqa_decode_static_workspace(const void* q, const uint8_t* k_cache,
                                         const uint8_t* v_cache, const int32_t* block_tables,
                                         const int32_t* context_lens, float k_scale,
                                         float v_scale, void* out, const xqa_shape_t* shape,
                                         void* stream);

/* Static, NUL-terminated description of a status code. */
const char* xqa_status_string(xqa_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* XQA_H_ */
