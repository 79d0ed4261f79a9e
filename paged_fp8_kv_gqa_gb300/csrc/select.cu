// select.cu — the pages worth reading: bounds of each page's keys (xqa_page_bounds) and the
// choice of a few pages for each sequence and kv head from them (xqa_select).
//
// Bounds. For the tokens t of a (page, kv head) and every dim d, in whole steps of one
// power of two for the slice:
//
//   2^e: the largest |k| lies in [2^(e+6), 2^(e+7))      (so it is at most 127 steps)
//   hi_d = ceil(max_t k_td / 2^e),  lo_d = floor(min_t k_td / 2^e)
//
// 128 + 128 + 1 bytes, padded to 272, in place of 2048 codes. No key lies outside them.
//
// Score. With the group's queries in whole steps, q8 = rint(q / 2^f), |q8| <= 64, the
// largest logits that keys within a page's bounds can have, summed over the group, are
//
//   2^f 2^e sum_d (A_d hi_d + B_d lo_d),   A_d = sum_g max(q8_gd, 0), B_d = sum_g min(q8_gd, 0)
//
// (a positive q wants the upper bound, a negative one the lower), so a group costs as much
// as one head. At most 128 x 16 x 64 x 127 < 2^24 in whole numbers: the sum is exact in any
// order, so a choice depends neither on the split of the work nor on the batch, and ties are
// ties. 2^f is common to all pages of a choice and left out.
//
// Their floors are bytes: 2048 + 272 (1152 + 272 in 4 bits) for a slice's bounds, 272 for a
// score, against 4096 for a page's keys and values. Measured: bounds of 49k rows x 4 heads 9.8 us
// (3650 GB/s; by latency: a warp waits for its page ids and then for the codes of two slices at
// a time, in about two rounds of CTAs; loads are its largest stall, with 49 % of the issue
// slots used), of 16 rows 2.7 us; choices of 128 of 1100 pages x 64 12.7 us, of 256 of 8192
// pages x 8 13.9 us (20 MB of bounds, the rest the latencies of scores, ticket, threshold and
// order), of 4 of 5 pages 1.6 us.
#include "xqa_device.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBoundsBytes = XQA_BOUNDS_BYTES;
constexpr int kNotFinite = -128;  // exponent of a slice with an infinity or NaN

__device__ __forceinline__ void raise(int32_t* status, int code) {
  if (status) atomicCAS(status, XQA_OK, code);
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 .. 127
// floor(log2 x) of a normal x > 0
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// Of pairs; a NaN stays one.
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
  const __half2 m = __hmin2_nan(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// ---------------------------------------------------------------------------
// bounds: a warp takes one kv head of the pages that `rows_per` consecutive new rows
// touch. Eight lanes hold the 128 dims of a token, 16 each, so a warp reads four tokens at
// a time and each lane keeps the largest and smallest of four tokens.
// ---------------------------------------------------------------------------
constexpr int kBoundsThreads = 128;

// Codes of 16 neighbouring dims of a token, and their values as 8 half2 (exact: see the formats).
template <int kFmt>
struct Key16 {
  uint4 w;
};
template <>
struct Key16<XQA_KV_E2M1> {
  uint2 w;
  uint32_t s8;
};
template <int kFmt>
__device__ __forceinline__ Key16<kFmt> read_key(const uint8_t* slice, size_t token_stride, int t, int c) {
  Key16<kFmt> k;
  if constexpr (kFmt == XQA_KV_E2M1) {
    k.w = *reinterpret_cast<const uint2*>(slice + t * (kHeadDim / 2) + 8 * c);
    k.s8 = slice[kCodeBytes4 + t * (kHeadDim / kGroup4) + c];
  } else {
    k.w = *reinterpret_cast<const uint4*>(slice + t * token_stride + 16 * c);
  }
  return k;
}
template <int kFmt>
__device__ __forceinline__ void key_values(const Key16<kFmt>& k, uint32_t (&o)[8]) {
  if constexpr (kFmt == XQA_KV_E2M1) {
    const uint32_t sc = e4m3x2_to_f16x2(k.s8 | k.s8 << 8);
    e2m1x8_to_f16x2(k.w.x, o);
    e2m1x8_to_f16x2(k.w.y, o + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = hmul2(o[i], sc);
  } else {
    const uint32_t x[4] = {k.w.x, k.w.y, k.w.z, k.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = KvConv<kFmt>::k_lo(x[i]);
      o[2 * i + 1] = KvConv<kFmt>::k_hi(x[i]);
    }
  }
}

// This lane's codes of a slice: dims 16 (lane & 7) .. of tokens lane / 8, + 4, ... below `fill`.
template <int kFmt>
__device__ __forceinline__ void read_slice(const BoundsParams& p, int page, int head, int fill,
                                           Key16<kFmt> (&k)[4]) {
  const int lane = threadIdx.x & 31;
  const bool nhd = kFmt != XQA_KV_E2M1 && p.kv_layout == XQA_LAYOUT_NHD;
  const size_t stride = nhd ? (size_t)p.num_kv_heads * kHeadDim : kHeadDim;
  const uint8_t* slice =
      p.k_cache + (nhd ? ((size_t)page * kBlockSize * p.num_kv_heads + head) * kHeadDim
                       : ((size_t)page * p.num_kv_heads + head) *
                             (kFmt == XQA_KV_E2M1 ? (size_t)kSliceBytes4 : (size_t)kPageBytes));
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (4 * s + (lane >> 3) < fill) k[s] = read_key<kFmt>(slice, stride, 4 * s + (lane >> 3), lane & 7);
}

template <int kFmt>
__device__ __forceinline__ void bound_slice(const BoundsParams& p, int page, int head, int fill,
                                            const Key16<kFmt> (&codes)[4]) {
  const int lane = threadIdx.x & 31, t0 = lane >> 3;
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) hi[i] = 0xfc00fc00u, lo[i] = 0x7c007c00u;  // -inf, inf
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (4 * s + t0 >= fill) continue;
    uint32_t k[8];
    key_values<kFmt>(codes[s], k);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = hmax2(hi[i], k[i]);
      lo[i] = hmin2(lo[i], k[i]);
    }
  }
  // lanes 8 and 16 apart hold other tokens of the same dims: each keeps one half, then one
  // quarter of the dims (pairs 2 t0, 2 t0 + 1 in the end)
#pragma unroll
  for (int half = 4; half >= 2; half >>= 1) {
    const int off = 4 * half;
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const uint32_t h = __shfl_xor_sync(kAll, up ? hi[i] : hi[i + half], off);
      const uint32_t l = __shfl_xor_sync(kAll, up ? lo[i] : lo[i + half], off);
      hi[i] = hmax2(up ? hi[i + half] : hi[i], h);
      lo[i] = hmin2(up ? lo[i + half] : lo[i], l);
    }
  }
  const int pair = (lane & 16 ? 4 : 0) + (lane & 8 ? 2 : 0);  // of this lane's 16 dims
  // magnitudes order like their patterns, infinities and NaN last
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    top = __vmaxu2(top, __vmaxu2(hi[i] & 0x7fff7fffu, lo[i] & 0x7fff7fffu));
  const uint32_t big = __reduce_max_sync(kAll, max(top & 0xffffu, top >> 16));
  int e = 0;
  if (big >= 0x7c00u) e = kNotFinite;
  else if (big > 0) e = exponent(__half2float(__ushort_as_half((unsigned short)big))) - 6;
  uint32_t up4 = 0, low4 = 0;  // four dims each
  if (e != kNotFinite) {
    const float step = pow2(-e);  // |e| <= 22; the products are exact
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&lo[i]));
      up4 |= ((uint32_t)(__float2int_ru(u.x * step) & 255) | (uint32_t)(__float2int_ru(u.y * step) & 255) << 8)
             << (16 * i);
      low4 |= ((uint32_t)(__float2int_rd(d.x * step) & 255) | (uint32_t)(__float2int_rd(d.y * step) & 255) << 8)
              << (16 * i);
    }
  }
  uint8_t* out = p.bounds + ((size_t)page * p.num_kv_heads + head) * kBoundsBytes;
  const int dim = 16 * (lane & 7) + 2 * pair;
  *reinterpret_cast<uint32_t*>(out + dim) = up4;
  *reinterpret_cast<uint32_t*>(out + kHeadDim + dim) = low4;
  if (lane < 4) *reinterpret_cast<uint32_t*>(out + 2 * kHeadDim + 4 * lane) = lane == 0 ? (uint32_t)(e & 255) : 0u;
}

template <int kFmt>
__global__ void __launch_bounds__(kBoundsThreads, 6) bounds_kernel(const BoundsParams p, int rows_per) {
  // offsets and lengths of a batch that is not large: every step of the search for a row's
  // sequence would be a round trip to memory (49k rows so 12.8 us, not 9.8)
  constexpr int kHeld = 256;
  __shared__ int cu_held[kHeld + 1], ctx_held[kHeld];
  griddep_launch_dependents();
  griddep_wait();
  const bool held = p.batch <= kHeld;
  if (held) {
    for (int i = threadIdx.x; i <= p.batch; i += kBoundsThreads) {
      cu_held[i] = p.cu_seqlens[i];
      if (i < p.batch) ctx_held[i] = p.context_lens[i];
    }
    __syncthreads();
  }
  const int32_t* cu = held ? cu_held : p.cu_seqlens;
  const int32_t* lens = held ? ctx_held : p.context_lens;
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
  const long long r0 = unit / p.num_kv_heads * rows_per;
  const int head = (int)(unit % p.num_kv_heads);
  if (r0 >= p.num_rows) return;
  // a row a lane: is it its page's first new one, and which page is that
  int page = -1, fill = 0;
  const long long r = r0 + lane;
  if (lane < rows_per && r < p.num_rows && r >= cu[0] && r < cu[p.batch]) {
    int lo = 0, hi = p.batch - 1;  // last sequence that begins at or before r
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (cu[m] <= r) lo = m;
      else hi = m - 1;
    }
    const int q0 = cu[lo], q1 = cu[lo + 1], ctx = lens[lo];
    if (r >= q0 && r < q1) {
      if (ctx < 0 || ctx < (long long)q1 - q0 || ctx > (long long)p.max_blocks_per_seq * kBlockSize) {
        raise(p.status, XQA_ERR_CTX_TOO_LONG);
      } else {
        const int pos = ctx - (int)(q1 - r);
        if (r == q0 || pos % kBlockSize == 0) {
          const int j = pos / kBlockSize;
          page = p.block_tables[(size_t)lo * p.max_blocks_per_seq + j];
          fill = min(kBlockSize, ctx - j * kBlockSize);
          if ((uint32_t)page >= (uint32_t)p.num_blocks) {
            raise(p.status, XQA_ERR_BAD_BLOCK_ID);
            page = -1;
          }
        }
      }
    }
  }
  // two slices' codes in flight
  for (uint32_t some = __ballot_sync(kAll, page >= 0); some;) {
    Key16<kFmt> k[2][4];
    int id[2], n[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int src = some ? __ffs(some) - 1 : 0;
      id[e] = some ? __shfl_sync(kAll, page, src) : -1;
      n[e] = __shfl_sync(kAll, fill, src);
      some &= some - 1;  // (0 stays 0)
      if (id[e] >= 0) read_slice<kFmt>(p, id[e], head, n[e], k[e]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (id[e] >= 0) bound_slice<kFmt>(p, id[e], head, n[e], k[e]);
  }
}

// ---------------------------------------------------------------------------
// the choice: a CTA scores a chunk of a segment's pages (segment: sequence and kv head); the
// one that is last to finish a segment's chunks takes its best pages.
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr uint32_t kKeyAlways = 0xffffffffu, kKeyFirst = 0xfffffffeu;  // above every score's

// Orders like the score.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int dp2_lo(uint32_t a, uint32_t b, int c) {  // a: 2 x 16, b: bytes 0, 1
  int d;
  asm("dp2a.lo.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ int dp2_hi(uint32_t a, uint32_t b, int c) {  // bytes 2, 3
  int d;
  asm("dp2a.hi.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

constexpr int kBins = 2048;
constexpr int kKeysInSmem = 8192;  // of a segment of up to 131072 tokens

constexpr int kWarpPages = 16;  // pages of a warp at a time: all their loads in flight at once
constexpr int kQueryParts = kSelectThreads / kHeadDim;

static_assert(kWarpPages * kSelectWarps == kSelectPages, "pages of a CTA at a time");

struct SelectShared {
  alignas(16) uint32_t keys[kKeysInSmem];
  int bins[kBins];
  uint32_t ab[kQueryParts][kHeadDim];  // A (low half), B of some of the heads
  alignas(16) uint32_t pairs[2][kHeadDim / 2];  // A, B of all, of dims 2 i, 2 i + 1
  uint32_t amax[kSelectWarps];
  int count[kSelectWarps][3];
  uint32_t edge[kSelectWarps][2];
  int bin, above, size;  // the bin that holds the key in question; keys above it, in it
  uint32_t some[32], t;  // its keys, where they are few; the key
  int num_some, ties;
  int last;
  int status;
};

// Keys of a segment's pages from .. to - 1 (id: the table's entry of the warp's first page +
// lane; q: element tid + 512 k of the group's queries).
constexpr int kQueryLoads = kMaxCols * kHeadDim / kSelectThreads;
__device__ __forceinline__ void score_pages(const SelectParams& p, int seg, int pages, int from, int to,
                                            int id, const uint32_t (&q)[kQueryLoads],
                                            SelectShared& sh, uint32_t* keys) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 7, at = lane >> 3;
  const int b = seg / p.num_kv_heads, head = seg - b * p.num_kv_heads;
  const int32_t* table = p.block_tables + (size_t)b * p.max_blocks_per_seq;
  // magnitudes order like their patterns; those that are not finite count as 0
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kQueryLoads; ++k) {
    const uint32_t m = q[k] & 0x7fffu;
    if (m < 0x7c00u) top = max(top, m);
  }
  top = __reduce_max_sync(kAll, top);
  if (lane == 0) sh.amax[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) top = max(top, sh.amax[w]);
  const int f = top > 0 ? exponent(__half2float(__ushort_as_half((unsigned short)top))) - 5 : 0;
  const float step = pow2(-f);
  int a = 0, n = 0;  // positive, negative
#pragma unroll
  for (int k = 0; k < kQueryLoads; ++k) {
    if ((q[k] & 0x7c00u) == 0x7c00u) continue;
    const int x = (int)rintf(__half2float(__ushort_as_half((unsigned short)q[k])) * step);
    a += max(x, 0);
    n += min(x, 0);
  }
  sh.ab[tid / kHeadDim][tid % kHeadDim] = (uint32_t)(a & 0xffff) | (uint32_t)n << 16;
  __syncthreads();
  if (tid < kHeadDim / 2) {
    uint32_t v0 = 0, v1 = 0;
#pragma unroll
    for (int r = 0; r < kQueryParts; ++r) {
      v0 = __vadd2(v0, sh.ab[r][2 * tid]);
      v1 = __vadd2(v1, sh.ab[r][2 * tid + 1]);
    }
    sh.pairs[0][tid] = prmt(v0, v1, 0x5410u);
    sh.pairs[1][tid] = prmt(v0, v1, 0x7632u);
  }
  __syncthreads();
  constexpr int kStep = kWarpPages * kSelectWarps;
  for (int j0 = from + kWarpPages * warp; j0 < to; j0 += kStep) {
    const int next = lane < kWarpPages && j0 + kStep + lane < to ? table[j0 + kStep + lane] : 0;
    const bool mine = lane < kWarpPages && j0 + lane < to;
    const bool good = !mine || (uint32_t)id < (uint32_t)p.num_blocks;
    if (!good) record_status(&sh.status, XQA_ERR_BAD_BLOCK_ID);
    const int page0 = mine && good ? id : 0;
    uint4 hi[kWarpPages / 4], lo[kWarpPages / 4];
    int e[kWarpPages / 4];
#pragma unroll
    for (int s = 0; s < kWarpPages / 4; ++s) {
      const int page = __shfl_sync(kAll, page0, 4 * s + at);
      const uint8_t* bd = p.bounds + ((size_t)page * p.num_kv_heads + head) * kBoundsBytes;
      hi[s] = *reinterpret_cast<const uint4*>(bd + 16 * c);
      lo[s] = *reinterpret_cast<const uint4*>(bd + kHeadDim + 16 * c);
      e[s] = (int)(signed char)bd[2 * kHeadDim];
    }
    int sum[kWarpPages / 4];
#pragma unroll
    for (int side = 0; side < 2; ++side) {  // upper bounds with A, lower ones with B
      const uint4 w0 = *reinterpret_cast<const uint4*>(&sh.pairs[side][8 * c]);
      const uint4 w1 = *reinterpret_cast<const uint4*>(&sh.pairs[side][8 * c + 4]);
#pragma unroll
      for (int s = 0; s < kWarpPages / 4; ++s) {
        const uint4 x = side ? lo[s] : hi[s];
        int v = side ? sum[s] : 0;
        v = dp2_lo(w0.x, x.x, v), v = dp2_hi(w0.y, x.x, v);
        v = dp2_lo(w0.z, x.y, v), v = dp2_hi(w0.w, x.y, v);
        v = dp2_lo(w1.x, x.z, v), v = dp2_hi(w1.y, x.z, v);
        v = dp2_lo(w1.z, x.w, v), v = dp2_hi(w1.w, x.w, v);
        sum[s] = v;
      }
    }
    uint32_t key = 0;
#pragma unroll
    for (int s = 0; s < kWarpPages / 4; ++s) {
      int v = sum[s];
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) v += __shfl_xor_sync(kAll, v, off);
      const uint32_t k = e[s] == kNotFinite ? kKeyFirst : key_of((float)v * pow2(max(e[s], -126)));
      const uint32_t got = __shfl_sync(kAll, k, (lane & 3) * 8);  // page 4 s + (lane & 3)
      if (lane >> 2 == s) key = got;
    }
    const int j = j0 + lane;
    if (!good) key = kKeyFirst;  // is met, and reported, by whoever reads it
    if (j < p.first_pages || j >= pages - p.last_pages) key = kKeyAlways;
    if (mine) keys[j] = key;
    id = next;
  }
}

// Keys above t in the low half, equal to it in the high one: of at most 2^15 keys (a lane's of
// 2^24 / 16 / 32).
__device__ __forceinline__ void sum_above(uint32_t& both, uint32_t k, uint32_t t) {
  both += k > t ? 1u : k == t ? 1u << 16 : 0u;
}

// The `take` largest of n keys, the lowest index first among equal ones, as ascending indices.
//
// The take-th largest key t by a histogram over the keys' range, whose bin that holds it is
// the next range: the range shrinks by a factor of 2048 a round, and as it is the keys' own
// (not their leading bits, which scores of one sequence share) its bins fill evenly. Bit by
// bit (32 rounds of counting) the choice of 128 of 1100 pages x 64 took 23.8 us, so 12.7.
template <bool kInSmem>
__device__ __forceinline__ void take_pages(const SelectParams& p, int seg, int n, int take,
                                           const uint32_t* global, SelectShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t* keys = kInSmem ? sh.keys : global;
  // smallest and largest score, and how many pages come before all of them
  uint32_t low = 0xffffffffu, high = 0;
  int always = 0, special = 0;
  for (int i = 4 * tid; i < n; i += 4 * kSelectThreads) {  // (rows of keys are 16-byte aligned)
    const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
    const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (i + x >= n) continue;
      if (w[x] >= kKeyFirst) {
        special += 1;
        always += w[x] == kKeyAlways;
      } else {
        low = min(low, w[x]);
        high = max(high, w[x]);
      }
    }
  }
  special = __reduce_add_sync(kAll, special);
  always = __reduce_add_sync(kAll, always);
  low = __reduce_min_sync(kAll, low);
  high = __reduce_max_sync(kAll, high);
  if (lane == 0) {
    sh.count[warp][0] = special;
    sh.count[warp][1] = always;
    sh.edge[warp][0] = low;
    sh.edge[warp][1] = high;
  }
  __syncthreads();
  special = always = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    special += sh.count[w][0];
    always += sh.count[w][1];
    low = min(low, sh.edge[w][0]);
    high = max(high, sh.edge[w][1]);
  }
  uint32_t t = kKeyFirst;    // the take-th largest key
  int ties = take - always;  // of the keys equal to it, the first so many
  if (special < take) {
    int want = take - special;  // the want-th largest of [low, high]
    for (;;) {
      const int bits = 32 - __clz(high - low);
      const int shift = bits > 11 ? bits - 11 : 0;
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t k = keys[i];
        if (k >= low && k <= high) atomicAdd(&sh.bins[(k - low) >> shift], 1);
      }
      __syncthreads();
      // bins from the top: 4 to a thread, thread 0 the highest; left at zero for the next
      constexpr int kPer = kBins / kSelectThreads;
      int mine[kPer], sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        int& bin = sh.bins[kBins - 1 - (tid * kPer + e)];
        sum += mine[e] = bin;
        bin = 0;
      }
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += x;
      }
      if (lane == 31) sh.count[warp][2] = incl;
      __syncthreads();
      int above = incl - sum;
      for (int w = 0; w < warp; ++w) above += sh.count[w][2];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (above < want && above + mine[e] >= want) {
          sh.bin = kBins - 1 - (tid * kPer + e);
          sh.above = above;
          sh.size = mine[e];
          sh.num_some = 0;
        }
        above += mine[e];
      }
      __syncthreads();
      want -= sh.above;
      const uint32_t start = low + ((uint32_t)sh.bin << shift);
      if (shift == 0) {
        t = start;
        ties = want;
        break;
      }
      high = min(high, start + ((1u << shift) - 1));
      low = start;
      if (sh.size > 32) continue;
      // few are left: a warp ranks them
      for (int i = tid; i < n; i += kSelectThreads) {
        const uint32_t k = keys[i];
        if (k >= low && k <= high) sh.some[atomicAdd(&sh.num_some, 1)] = k;
      }
      __syncthreads();
      if (warp == 0) {
        const bool in = lane < sh.size;
        const uint32_t k = in ? sh.some[lane] : 0u;
        int larger = 0, equal = 0;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint32_t x = __shfl_sync(kAll, k, e);
          larger += e < sh.size && x > k;
          equal += e < sh.size && x == k;
        }
        if (in && larger < want && larger + equal >= want) sh.t = k, sh.ties = want - larger;
      }
      __syncthreads();
      t = sh.t;
      ties = sh.ties;
      break;
    }
  }
  __syncthreads();
  // each warp writes those of a run of keys, behind the ones of the warps before it: their
  // indices first, so that no table entry is waited for on the way
  // (four keys to a lane; keys past n count as none)
  const int run = ((n + kSelectWarps - 1) / kSelectWarps + 127) & ~127;
  const int from = min(n, warp * run), to = min(n, from + run);
  auto four = [&](int i, uint32_t (&k)[4]) {
    const uint4 v = i < to ? *reinterpret_cast<const uint4*>(keys + i) : make_uint4(0, 0, 0, 0);
    k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
  };
  uint32_t both = 0;
  for (int i0 = from; i0 < to; i0 += 128) {
    uint32_t k[4];
    four(i0 + 4 * lane, k);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + 4 * lane + e < to) sum_above(both, k[e], t);
  }
  const int above = __reduce_add_sync(kAll, (int)(both & 0xffff));
  const int equal = __reduce_add_sync(kAll, (int)(both >> 16));
  if (lane == 0) sh.count[warp][0] = above, sh.count[warp][1] = equal;
  __syncthreads();
  int at = 0, eq = 0;
  for (int w = 0; w < warp; ++w) at += sh.count[w][0], eq += sh.count[w][1];
  int32_t* out = p.selected + (size_t)seg * p.max_pages;
  int* list = take <= kBins ? sh.bins : out;
  for (int i0 = from; i0 < to; i0 += 128) {  // at, eq: keys above and equal before i0
    uint32_t k[4];
    four(i0 + 4 * lane, k);
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + 4 * lane + e < to) sum_above(mine, k[e], t);
    uint32_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += x;
    }
    const uint32_t before = incl - mine, all = __shfl_sync(kAll, incl, 31);
    int a = at + (int)(before & 0xffff), q = eq + (int)(before >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i0 + 4 * lane + e >= to) continue;
      if (k[e] > t) list[a++ + min(q, ties)] = i0 + 4 * lane + e;
      else if (k[e] == t && q++ < ties) list[a + q - 1] = i0 + 4 * lane + e;
    }
    at += all & 0xffff;
    eq += all >> 16;
  }
  __syncthreads();
  const int32_t* table = p.block_tables + (size_t)(seg / p.num_kv_heads) * p.max_blocks_per_seq;
  for (int i = tid; i < take; i += kSelectThreads) {
    const int j = list[i];
    if (list == sh.bins) sh.bins[i] = 0;
    out[i] = table[j];
  }
}

// (two CTAs an SM leave 64 registers: 48 bytes a thread are spilled)
__global__ void __launch_bounds__(kSelectThreads, kSelectCtas) select_kernel(const SelectParams p) {
  __shared__ __align__(16) SelectShared sh;
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) sh.status = XQA_OK;
  for (int i = tid; i < kBins; i += kSelectThreads) sh.bins[i] = 0;
  __syncthreads();
  griddep_wait();
  const long long units = (long long)p.batch * p.num_kv_heads * p.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int seg = (int)(u / p.chunks), chunk = (int)(u - (long long)seg * p.chunks);
    const int from = chunk * p.chunk_pages;
    // what the scores need, asked for before the length says whether they are needed (the
    // table's row is as long as it may be)
    const int32_t* table = p.block_tables + (size_t)(seg / p.num_kv_heads) * p.max_blocks_per_seq;
    const int first = from + kWarpPages * (tid >> 5) + lane;
    const int id = lane < kWarpPages && first < p.max_blocks_per_seq ? table[first] : 0;
    uint32_t q[kQueryLoads];
#pragma unroll
    for (int k = 0; k < kQueryLoads; ++k) {
      const int i = tid + k * kSelectThreads;
      q[k] = i < p.group * kHeadDim ? p.q[(size_t)seg * p.group * kHeadDim + i] : 0u;  // [B, Hkv, G, 128]
    }
    const int ctx = p.context_lens[seg / p.num_kv_heads];
    const bool bad = ctx < 0 || ctx > (long long)p.max_blocks_per_seq * kBlockSize;
    const int pages = bad ? 0 : (ctx + kBlockSize - 1) / kBlockSize;
    const int take = min(pages, p.max_pages);
    if (chunk > 0 && (pages <= p.max_pages || from >= pages)) continue;
    int32_t* out = p.selected + (size_t)seg * p.max_pages;
    if (chunk == 0) {  // what does not depend on a score
      for (int i = take + tid; i < p.max_pages; i += kSelectThreads) out[i] = -1;
      if (tid == 0) {
        p.selected_lens[seg] = bad ? -1 : ctx - (pages - take) * kBlockSize;
        if (bad) record_status(&sh.status, XQA_ERR_CTX_TOO_LONG);
      }
    }
    if (pages <= p.max_pages) {  // all of them
      for (int i = tid; i < pages; i += kSelectThreads) {
        const int id = table[i];
        out[i] = id;
        if ((uint32_t)id >= (uint32_t)p.num_blocks) record_status(&sh.status, XQA_ERR_BAD_BLOCK_ID);
      }
      continue;
    }
    // a segment of one chunk keeps its keys here
    const int chunks = (pages + p.chunk_pages - 1) / p.chunk_pages;
    uint32_t* keys = chunks == 1 && pages <= kKeysInSmem ? sh.keys : p.keys + (size_t)seg * p.key_stride;
    score_pages(p, seg, pages, from, min(pages, from + p.chunk_pages), id, q, sh, keys);
    __syncthreads();
    if (tid == 0) {  // (releases what the barrier has put before it)
      const int old = chunks == 1 ? 0 : atom_add_acq_rel_gpu(p.tickets + seg, 1);
      sh.last = old == chunks - 1;
      if (sh.last && chunks > 1) p.tickets[seg] = 0;  // for the next call
    }
    __syncthreads();
    if (sh.last) {
      if (pages > kKeysInSmem) {
        take_pages<false>(p, seg, pages, take, keys, sh);
      } else {
        if (chunks > 1) {  // as many 16-byte loads of a thread in flight as there are
          constexpr int kAtOnce = kKeysInSmem / 4 / kSelectThreads;
          uint4 k[kAtOnce];
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) {
            const int i = 4 * (e * kSelectThreads + tid);
            if (i < pages) k[e] = __ldcg(reinterpret_cast<const uint4*>(keys + i));
          }
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) {
            const int i = 4 * (e * kSelectThreads + tid);
            if (i < pages) *reinterpret_cast<uint4*>(sh.keys + i) = k[e];
          }
        }
        take_pages<true>(p, seg, pages, take, nullptr, sh);
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) {
    p.status[blockIdx.x] = sh.status;
    if (blockIdx.x == 0) p.header[0] = gridDim.x;
  }
}

template <class... Args>
cudaError_t launch(void (*kernel)(Args...), int ctas, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_bounds(const BoundsParams& p, cudaStream_t stream) {
  // a row a warp while they are few (a decode step's are all pages of their own), else a row a
  // lane: of a prompt's rows, those of two or three pages
  const int rows_per = p.num_rows <= 4096 ? 1 : 32;
  const long long units = ((long long)p.num_rows + rows_per - 1) / rows_per * p.num_kv_heads;
  const int ctas = (int)((units + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32));
  switch (p.kv_dtype) {
    case XQA_KV_E2M1: return launch(bounds_kernel<XQA_KV_E2M1>, ctas, kBoundsThreads, stream, p, rows_per);
    case XQA_KV_E4M3: return launch(bounds_kernel<XQA_KV_E4M3>, ctas, kBoundsThreads, stream, p, rows_per);
    default: return launch(bounds_kernel<XQA_KV_E5M2>, ctas, kBoundsThreads, stream, p, rows_per);
  }
}

cudaError_t launch_select(const SelectParams& p, int ctas, cudaStream_t stream) {
  return launch(select_kernel, ctas, kSelectThreads, stream, p);
}

}  // namespace xqa
