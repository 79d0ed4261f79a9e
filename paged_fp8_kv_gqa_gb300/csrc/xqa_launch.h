// xqa_launch.h — host-side launch functions of the libxqa kernels (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace xqa {

struct PartialParams {
  const __half* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  __half* out;
  int32_t* header;     // workspace header (CTAs launched, CTAs with work, pages, segments)
  int32_t* seg_start;  // [nseg + 1]; written here when the plan is derived in the kernel
  int32_t* seg_bad;    // [nseg] bad context-length flags (plan output)
  int32_t* seg_cc;     // [nseg] cost-line prefix (see seg_cost)
  int32_t* tickets;    // [kMaxCtas] merge tickets of split segments, zero between calls
  int32_t* status;     // [kMaxCtas] each CTA's status in this call
  float* partials;     // [(n_max + nseg) * kSlotFloats]
  int32_t* hints;      // [kMaxCtas * kHintPages] first pages of each CTA's range (null: none)
  int batch, num_q_heads, num_kv_heads, group, max_blocks_per_seq, num_blocks;
  int cache_heads;           // kv heads of the cache (num_kv_heads, unless every kv head has
                             // a table of its own: then num_kv_heads is 1)
  int seq_rows, head_rows;   // rows of block_tables from a sequence and from a kv head to the
                             // next: 1 and 0, unless every kv head has its own
  int q_len;                 // new tokens per sequence (q, out: [B, q_len, Hq, D])
  int n_max, min_pages;      // split rule inputs (same values the planner got)
  int fused_merge;           // 1: the last CTA of a split segment merges it
  int merge_helpers;         // CTAs that may share a large segment's final merge (1: the
                             // last alone; more only if every CTA is resident at once)
  int kv_dtype, kv_layout;   // XQA_KV_* code format, XQA_LAYOUT_* cache layout
  double qk_scale_base;      // sm_scale * log2(e); the logit scale is this * k_scale
  float k_scale, v_scale;    // per-tensor scales (used when the pointers are null)
  const float* k_scale_ptr;  // optional device scalars, read when the kernel runs
  const float* v_scale_ptr;
  const uint8_t* k_pool;     // the caches (4-bit: read by plain bulk copies)
  const uint8_t* v_pool;
};

struct CombineParams {
  __half* out;
  const int32_t* header;
  const int32_t* seg_start;
  const int32_t* seg_cc;
  int32_t* tickets;  // read for the bad-piece count, then cleared
  const float* partials;
  int num_q_heads, num_kv_heads, group, q_len;
  float v_scale;
  const float* v_scale_ptr;  // optional device scalar (overrides v_scale)
};

// xqa_append (k, v read, caches written) and xqa_gather (the other way round).
struct RowsParams {
  uint16_t* k;  // [num_rows, Hkv, 128] 16-bit values, strides in elements
  uint16_t* v;
  const int32_t* cu_seqlens;  // [batch + 1]
  const int32_t* block_tables;
  const int32_t* context_lens;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int32_t* status;  // optional: first error of the call
  int batch, num_kv_heads, max_blocks_per_seq, num_blocks, num_rows;
  int kv_dtype, kv_layout, dtype;
  long long k_row_stride, k_head_stride, v_row_stride, v_head_stride;
  float k_scale, v_scale;
  const float* k_scale_ptr;  // optional device scalars (override the values)
  const float* v_scale_ptr;
};

constexpr int kPrefillMaxPieces = 8;

struct PrefillParams {
  const int32_t* cu_q;  // [batch + 1]
  const int32_t* cu_k;
  const uint16_t* v;    // for values that are not finite (read through TMA otherwise)
  uint16_t* out;
  float* lse;         // optional [total_q, Hq]
  int32_t* header;    // workspace header (CTAs launched)
  int32_t* counters;  // [2] units handed out, CTAs done: zero between calls
  int32_t* status;    // [kMaxCtas]
  int batch, num_q_heads, num_kv_heads, group, total_q, total_k, causal;
  int tile_tokens;    // T: tokens of a 128-row tile
  int max_units;      // of offsets that ascend
  int pieces;         // a unit's keys are cut into so many (1: not at all); with more
                      // than 1 there are at least as many CTAs as pieces of all units
  int32_t* tickets;   // pieces written, by unit: zero between calls
  float4* piece_o;    // [units * pieces][2][32 chunks of 4 dims][128 rows]
  float2* piece_ml;   // [units * pieces][2][128]
  float scale_log2;   // sm_scale * log2(e)
  long long v_row_stride, v_head_stride, out_row_stride, out_head_stride;
};

// The least share of the line of work (extend.cu: keys seen, summed over the units) that a
// CTA takes; fewer CTAs work on shorter lines. A unit's start and end count as kExtendUnitKeys
// keys.
constexpr int kExtendMinShare = 384, kExtendUnitKeys = 256;

// A unit of tokens whose keys several CTAs share; pieces < 2: none. (A unit of a bad length or
// scale has no keys to share.)
struct SplitUnit {
  int pieces, q_row, tokens, head;
};

// Length of a key of a one-row-tile unit on chunk attention's line of work, where one of two row
// tiles is 16.
constexpr int kKeyCostOne = 10, kKeyCostOneSlow = 12;

struct ExtendParams {
  const int32_t* cu_q;  // [batch + 1]
  const int32_t* context_lens;
  const int32_t* block_tables;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  uint16_t* out;
  float* lse;         // optional [total_q, Hq]
  int32_t* header;    // workspace header (CTAs launched)
  int32_t* status;    // [kMaxCtas]
  SplitUnit* split;   // [CTAs] the split unit that begins in the CTA's share
  float* piece_o;     // [CTAs][2 units][2 row tiles][128 rows][128]
  float2* piece_ml;   // [CTAs][2][2][128]
  int batch, num_q_heads, num_kv_heads, group, total_q, causal;
  int max_blocks_per_seq, num_blocks, kv_dtype, kv_layout;
  int tile_tokens;    // T: tokens of a 128-row tile
  int key_cost_one;   // of a key of a unit of one row tile (kKeyCostOne or kKeyCostOneSlow)
  double qk_scale_base;      // sm_scale * log2(e); the logit scale is this * k_scale
  float k_scale, v_scale;    // per-tensor scales (used when the pointers are null)
  const float* k_scale_ptr;
  const float* v_scale_ptr;
  long long out_row_stride, out_head_stride;
};

cudaError_t launch_extend(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                          const ExtendParams& p, int dtype, int ctas, cudaStream_t stream);
// xqa_assign_pages and xqa_release_pages.
constexpr int kMaxPagesBatch = 16384;          // sequences: three words each in shared memory

struct PagesParams {
  const int32_t* new_tokens;    // assign
  const uint8_t* done;          // release
  const int32_t* context_lens;
  int32_t* block_tables;        // release: read only
  int32_t* free_pages;          // assign: read only
  const int32_t* num_free;
  int32_t* new_lens;
  int32_t* new_free;
  int32_t* cu_seqlens;
  int32_t* slots;               // optional
  int32_t* positions;           // optional
  int32_t* status;              // optional: first error of the call
  int batch, max_blocks_per_seq, num_blocks, num_rows;
};

// xqa_page_bounds.
struct BoundsParams {
  const uint8_t* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_seqlens;
  uint8_t* bounds;
  int32_t* status;
  int batch, num_kv_heads, max_blocks_per_seq, num_blocks, num_rows, kv_dtype, kv_layout;
};

// xqa_select. CTAs that fit an SM at once (its launch bounds) and pages that a CTA scores at
// a time: 16 for each of its 16 warps.
constexpr int kSelectCtas = 2, kSelectPages = 256;
struct SelectParams {
  const uint16_t* q;  // [B, Hq, 128] fp16
  const uint8_t* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* selected;       // [B * Hkv, max_pages]
  int32_t* selected_lens;  // [B * Hkv]
  int32_t* header;         // workspace header (CTAs launched)
  int32_t* status;         // [kMaxCtas]
  int32_t* tickets;        // [segments of several chunks: <= kMaxCtas / 2] chunks scored: zero
                           // between calls
  uint32_t* keys;          // [B * Hkv, key_stride]
  int key_stride;          // MBS, a multiple of 4
  int batch, num_kv_heads, group, max_blocks_per_seq, num_blocks;
  int max_pages, first_pages, last_pages;
  int chunks, chunk_pages;
};

cudaError_t launch_assign(const PagesParams& p, int cluster, cudaStream_t stream);
cudaError_t launch_release(const PagesParams& p, int cluster, cudaStream_t stream);
cudaError_t launch_bounds(const BoundsParams& p, cudaStream_t stream);
cudaError_t launch_select(const SelectParams& p, int ctas, cudaStream_t stream);
cudaError_t launch_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                           const CUtensorMap& tm_v, const PrefillParams& p, int dtype, int ctas,
                           cudaStream_t stream);
cudaError_t launch_rows(bool append, const RowsParams& p, cudaStream_t stream);
cudaError_t launch_plan(const int32_t* context_lens, int batch, int num_kv_heads,
                        int max_blocks_per_seq, int n_max, int min_pages_per_cta,
                        int32_t* workspace, cudaStream_t stream);
cudaError_t launch_partial(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                           const PartialParams& p, int n_max, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams& p, int num_segments, cudaStream_t stream);
cudaError_t launch_wait_timeout(int32_t* status, unsigned long long budget_ns,
                                cudaStream_t stream);
cudaError_t launch_dequant(int kv_dtype, const uint8_t* in, size_t n, float scale,
                           uint16_t* out16, float* out32, cudaStream_t stream);

}  // namespace xqa
