// rows.cu — packed rows of keys and values into the paged cache (xqa_append)
// and back (xqa_gather).
//
// Row r of k and v is one token (Hkv heads x 128 dims, fp16 or bf16). Sequence
// b owns the rows cu_seqlens[b] .. cu_seqlens[b+1]-1, which are the last n_b of
// its context_lens[b] tokens: row r sits at position
// context_lens[b] - (cu_seqlens[b+1] - r).
//
//   append, FP8:   code = RNE(x / scale), saturated; NaN stays NaN
//   append, E2M1:  per group of 16 dims s = E4M3(max |x| / scale / 6), then
//                  code = E2M1(x / (scale * s)), ties to even, saturated at 6
//   gather:        x = RNE16(scale * code) or RNE16(scale * (s * code)); the
//                  product s * code is exact in 32 bits
//
// Both move bytes and compute little: 256 B on the 16-bit side of a (row, kv
// head) and 128 B (72 B in 4 bits) on the cache side, for K and V each. Eight
// threads take one (row, kv head): thread p the dims [8p, 8p+8) and [64+8p, 64+8p+8),
// so that every access of the eight is one contiguous run of whole sectors (16 dims
// side by side would write each sector of a packed row in two halves). A 4-bit scale
// group is shared by two neighbouring threads. A thread does K and V of its row
// together: the walk from row to cache slot (a search in cu_seqlens, a length, a table
// entry) is paid once, with four 16-byte loads in flight.
#include <cuda_bf16.h>

#include "xqa_device.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

constexpr int kRowThreads = 128;
constexpr int kLanesPerRow = 8;  // threads of one (row, kv head)

// Quotients by one divisor t, as in IEEE division: q0 = x r with r = RN(1/t),
// then one correction q0 - (q0 t - x) r (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): exact whenever x / t is
// representable, so ties are seen as ties; in this form a zero keeps its sign. A
// divisor that is a power of two needs no correction. Other divisors than those of
// 2^-60 to 2^60 (a scale on the device may be 0, negative or NaN) divide plainly.
struct Divisor {
  float t, r;
  bool exact;  // x r is x / t
  bool slow;   // 1 / t or the correction could leave the normal range
  bool zeros;  // zeros in place of the quotients
};

__device__ __forceinline__ Divisor make_divisor(float t, bool zeros = false) {
  Divisor d;
  d.t = t;
  d.r = zeros ? 0.f : __frcp_rn(t);
  d.exact = zeros || (__float_as_uint(t) & 0x7fffffu) == 0;
  d.slow = !zeros && !(t >= 0x1p-60f && t <= 0x1p60f);
  d.zeros = zeros;
  return d;
}

// The quotients of a thread's 8 neighbouring values; amax: their largest magnitude.
// Quotients past 2^20 (infinities and NaN among them: they saturate in every format)
// go by plain division too.
__device__ __forceinline__ void divide(const uint64_t (&x)[4], float amax, const Divisor& d,
                                       float (&q)[8]) {
  if (!d.slow && amax * d.r < 0x1p20f) {
    const uint64_t r2 = f32x2(d.r, d.r);
    if (d.exact) {
#pragma unroll
      for (int i = 0; i < 4; ++i) split2(mul2(x[i], r2), q[2 * i], q[2 * i + 1]);
    } else {
      const uint64_t t2 = f32x2(d.t, d.t), m2 = f32x2(-d.r, -d.r);
      constexpr uint64_t kSigns = 0x8000000080000000ull;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t q0 = mul2(x[i], r2);
        split2(fma2(fma2(q0, t2, x[i] ^ kSigns), m2, q0), q[2 * i], q[2 * i + 1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      split2(x[i], q[2 * i], q[2 * i + 1]);
      q[2 * i] = d.zeros ? copysignf(0.f, q[2 * i]) : __fdiv_rn(q[2 * i], d.t);
      q[2 * i + 1] = d.zeros ? copysignf(0.f, q[2 * i + 1]) : __fdiv_rn(q[2 * i + 1], d.t);
    }
  }
}

// Two fp32 -> two codes, the first in the low bits.
template <int kFmt>
__device__ __forceinline__ uint32_t cvt_fp8x2(float lo, float hi) {
  unsigned short d;
  if (kFmt == XQA_KV_E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Eight fp32 -> eight E2M1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* x) {
  uint32_t d;
  asm("{\n\t.reg .b8 a, b, c, e;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, e};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return d;
}

// 8 neighbouring values in 32 bits, in pairs; returns the 15-bit pattern of the
// largest magnitude (the patterns order like the magnitudes, infinities and NaN last).
template <int kType>
__device__ __forceinline__ uint32_t unpack8(const uint4& a, uint64_t (&x)[4]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    if (kType == XQA_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[i] = f32x2(f.x, f.y);
    } else {
      x[i] = f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
  }
  return max(top & 0xffffu, top >> 16);
}

template <int kType>
__device__ __forceinline__ float magnitude(uint32_t pattern) {
  return kType == XQA_F16 ? __half2float(__ushort_as_half((unsigned short)pattern))
                          : __uint_as_float(pattern << 16);
}

template <int kType>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (kType == XQA_F16) return pack_half2(lo, hi);
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Where one (row, kv head) lives. `at` indexes 128-value rows of the cache:
// FP8 (any layout): byte offset at * 128; E2M1: slice = at / 16, token = at % 16.
struct RowPlace {
  long long at;
  int state;  // 1: in the cache, 0: not a row of any sequence, -1: bad
};

__device__ __forceinline__ RowPlace find_row(const RowsParams& p, int row, int head) {
  RowPlace r{0, 0};
  // largest b with cu[b] <= row
  int lo = 0, hi = p.batch;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_seqlens[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  if (lo >= p.batch) return r;
  const int beg = p.cu_seqlens[lo], end = p.cu_seqlens[lo + 1];
  if (row < beg || row >= end) return r;
  const int ctx = p.context_lens[lo];
  const long long pos = (long long)ctx - ((long long)end - row);
  // every row of a sequence with a bad length is bad, not only those in front
  // of its first token
  if (ctx < 0 || (long long)ctx > (long long)p.max_blocks_per_seq * kBlockSize ||
      (long long)ctx < (long long)end - beg) {
    r.state = -1;
    if (p.status && head == 0 && (threadIdx.x & (kLanesPerRow - 1)) == 0)
      atomicCAS(p.status, XQA_OK, XQA_ERR_CTX_TOO_LONG);
    return r;
  }
  const int id = p.block_tables[(size_t)lo * p.max_blocks_per_seq + (size_t)(pos / kBlockSize)];
  if (id < 0 || id >= p.num_blocks) {
    r.state = -1;
    if (p.status && head == 0 && (threadIdx.x & (kLanesPerRow - 1)) == 0)
      atomicCAS(p.status, XQA_OK, XQA_ERR_BAD_BLOCK_ID);
    return r;
  }
  const int slot = (int)(pos % kBlockSize);
  r.at = p.kv_layout == XQA_LAYOUT_HND
             ? ((long long)id * p.num_kv_heads + head) * kBlockSize + slot
             : ((long long)id * kBlockSize + slot) * p.num_kv_heads + head;
  r.state = 1;
  return r;
}

// One thread's dims [8 part, 8 part + 8) (a) and 64 on (b) of one row. The threads of
// a row come here together.
template <int kFmt, int kType>
__device__ __forceinline__ void store_codes(uint8_t* cache, long long at, int part, const uint4& a,
                                            const uint4& b, float scale) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t x[4];
    uint32_t top = unpack8<kType>(h ? b : a, x);
    float q[8];
    if (kFmt != XQA_KV_E2M1) {
      divide(x, magnitude<kType>(top), make_divisor(scale), q);
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = cvt_fp8x2<kFmt>(q[4 * i], q[4 * i + 1]) |
               cvt_fp8x2<kFmt>(q[4 * i + 2], q[4 * i + 3]) << 16;
      *reinterpret_cast<uint2*>(cache + at * kHeadDim + 64 * h + 8 * part) = make_uint2(w[0], w[1]);
    } else {
      const unsigned eight = 0xffu << (threadIdx.x & 24);
      top = max(top, __shfl_xor_sync(eight, top, 1));  // the group's other half
      const float amax = magnitude<kType>(top);
      const uint32_t s8 = cvt_fp8x2<XQA_KV_E4M3>(__fdiv_rn(__fdiv_rn(amax, scale), 6.f), 0.f) & 0xffu;
      const uint32_t sh = e4m3x2_to_f16x2(s8);
      const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
      divide(x, amax, make_divisor(s * scale, !(fabsf(s) > 0.f)), q);  // s of 0 or NaN: zeros
      uint8_t* slice = cache + (at / kBlockSize) * kSliceBytes4;
      const int token = (int)(at % kBlockSize);
      *reinterpret_cast<uint32_t*>(slice + token * (kHeadDim / 2) + 32 * h + 4 * part) = cvt_e2m1x8(q);
      // the four scales of this half row in one store
      uint32_t sw = s8 << 8 * (part >> 1);
      sw |= __shfl_xor_sync(eight, sw, 2);
      sw |= __shfl_xor_sync(eight, sw, 4);
      if (part == 0)
        *reinterpret_cast<uint32_t*>(slice + kCodeBytes4 + token * (kHeadDim / kGroup4) + 4 * h) = sw;
    }
  }
}

template <int kFmt, int kType>
__device__ __forceinline__ void load_values(const uint8_t* cache, long long at, int part,
                                            float scale, uint4 (&out)[2]) {
  uint2 c[2];
  uint32_t s8[2] = {0, 0};
  if (kFmt != XQA_KV_E2M1) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      c[h] = *reinterpret_cast<const uint2*>(cache + at * kHeadDim + 64 * h + 8 * part);
  } else {
    const uint8_t* slice = cache + (at / kBlockSize) * kSliceBytes4;
    const int token = (int)(at % kBlockSize);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c[h].x = *reinterpret_cast<const uint32_t*>(slice + token * (kHeadDim / 2) + 32 * h + 4 * part);
      s8[h] = slice[kCodeBytes4 + token * (kHeadDim / kGroup4) + 4 * h + (part >> 1)];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t v[4];  // the codes' values in pairs, fp16 (exact)
    float s = 1.f;
    if (kFmt != XQA_KV_E2M1) {
      using Conv = KvConv<kFmt == XQA_KV_E2M1 ? XQA_KV_E4M3 : kFmt>;
      v[0] = Conv::k_lo(c[h].x);
      v[1] = Conv::k_hi(c[h].x);
      v[2] = Conv::k_lo(c[h].y);
      v[3] = Conv::k_hi(c[h].y);
    } else {
      const uint32_t sh = e4m3x2_to_f16x2(s8[h]);
      s = __low2float(*reinterpret_cast<const __half2*>(&sh));
      e2m1x8_to_f16x2(c[h].x, v);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      uint64_t y = f32x2(f.x, f.y);
      if (kFmt == XQA_KV_E2M1) y = mul2(y, f32x2(s, s));  // exact
      float lo, hi;
      split2(mul2(y, f32x2(scale, scale)), lo, hi);
      o[i] = pack16<kType>(lo, hi);
    }
    out[h] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// kHeads: neighbouring kv heads that a thread takes (append only, see launch_format).
template <int kFmt, int kType, bool kAppend, int kHeads>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsParams p) {
  griddep_launch_dependents();
  const long long u = ((long long)blockIdx.x * kRowThreads + threadIdx.x) / kLanesPerRow;
  const int part = threadIdx.x % kLanesPerRow;
  // Every input may come from the kernels before this one, and some of its sectors may lie
  // in this SM's cache since one of those read them: it may run on the SM after this kernel
  // became resident and before another wrote them. So the loads behind the wait are plain
  // ones: the read-only path promises nothing for bytes that change meanwhile.
  griddep_wait();
  const int per_row = p.num_kv_heads / kHeads;  // a multiple, see launch_format
  if (u >= (long long)p.num_rows * per_row) return;
  const int row = (int)((uint32_t)u / (uint32_t)per_row);
  const int head = ((int)u - row * per_row) * kHeads;
  const uint16_t* kp = p.k + row * p.k_row_stride + head * p.k_head_stride + 8 * part;
  const uint16_t* vp = p.v + row * p.v_row_stride + head * p.v_head_stride + 8 * part;
  const float k_scale = p.k_scale_ptr ? *p.k_scale_ptr : p.k_scale;
  const float v_scale = p.v_scale_ptr ? *p.v_scale_ptr : p.v_scale;
  if constexpr (kAppend) {
    // in flight while the slot is looked up; rows of no sequence are readable too
    uint4 x[kHeads][4];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const uint4* k = reinterpret_cast<const uint4*>(kp + h * p.k_head_stride);
      const uint4* v = reinterpret_cast<const uint4*>(vp + h * p.v_head_stride);
      x[h][0] = k[0], x[h][1] = k[8], x[h][2] = v[0], x[h][3] = v[8];
    }
    const RowPlace r = find_row(p, row, head);
    if (r.state != 1) return;
    const int next = p.kv_layout == XQA_LAYOUT_HND ? kBlockSize : 1;  // the next head's row
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      store_codes<kFmt, kType>(p.k_cache, r.at + h * next, part, x[h][0], x[h][1], k_scale);
      store_codes<kFmt, kType>(p.v_cache, r.at + h * next, part, x[h][2], x[h][3], v_scale);
    }
  } else {
    static_assert(kHeads == 1, "gather");
    const RowPlace r = find_row(p, row, head);
    if (r.state == 0) return;
    uint4 a[2], b[2];
    if (r.state > 0) {
      load_values<kFmt, kType>(p.k_cache, r.at, part, k_scale, a);
      load_values<kFmt, kType>(p.v_cache, r.at, part, v_scale, b);
    } else {
      const uint32_t nan = kType == XQA_F16 ? 0x7fff7fffu : 0x7fc07fc0u;
      a[0] = a[1] = b[0] = b[1] = make_uint4(nan, nan, nan, nan);
    }
    uint4* k = reinterpret_cast<uint4*>(const_cast<uint16_t*>(kp));
    uint4* v = reinterpret_cast<uint4*>(const_cast<uint16_t*>(vp));
    k[0] = a[0];
    k[8] = a[1];
    v[0] = b[0];
    v[8] = b[1];
  }
}

template <int kFmt, int kType, bool kAppend, int kHeads>
cudaError_t launch(cudaLaunchConfig_t cfg, const RowsParams& p) {
  const long long threads = (long long)p.num_rows * (p.num_kv_heads / kHeads) * kLanesPerRow;
  cfg.gridDim = dim3((unsigned)((threads + kRowThreads - 1) / kRowThreads));
  return cudaLaunchKernelEx(&cfg, rows_kernel<kFmt, kType, kAppend, kHeads>, p);
}

// FP8 rows of many tokens are appended two heads to a thread: twice the loads in flight
// for one lookup. 4 heads: 48.6k tokens 28.1 us with one head, 26.0 with two (5750 GB/s),
// 8192 tokens 6.2 and 5.7; fewer leave SMs idle: 4096 tokens 3.7 and 4.5, 256 2.2 and
// 2.6. An odd head would have a thread of its own (3 heads, 16384 tokens: 10.2 and 10.5).
// 4-bit rows and gather hold more registers for each head and lose (append and gather of
// 4-bit rows 50.5 and 53.5 us, gather of 30k FP8 tokens 12.0 and 13.9).
constexpr long long kPairFrom = 1ll << 15;  // (row, kv head) pairs

template <bool kAppend, int kType>
cudaError_t launch_format(int fmt, const cudaLaunchConfig_t& cfg, const RowsParams& p) {
  if constexpr (kAppend) {
    if (fmt != XQA_KV_E2M1 && p.num_kv_heads % 2 == 0 &&
        (long long)p.num_rows * p.num_kv_heads >= kPairFrom)
      return fmt == XQA_KV_E5M2 ? launch<XQA_KV_E5M2, kType, true, 2>(cfg, p)
                                : launch<XQA_KV_E4M3, kType, true, 2>(cfg, p);
  }
  switch (fmt) {
    case XQA_KV_E5M2: return launch<XQA_KV_E5M2, kType, kAppend, 1>(cfg, p);
    case XQA_KV_E4M3: return launch<XQA_KV_E4M3, kType, kAppend, 1>(cfg, p);
    default: return launch<XQA_KV_E2M1, kType, kAppend, 1>(cfg, p);
  }
}

}  // namespace

cudaError_t launch_rows(bool append, const RowsParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (append)
    return p.dtype == XQA_F16 ? launch_format<true, XQA_F16>(p.kv_dtype, cfg, p)
                              : launch_format<true, XQA_BF16>(p.kv_dtype, cfg, p);
  return p.dtype == XQA_F16 ? launch_format<false, XQA_F16>(p.kv_dtype, cfg, p)
                            : launch_format<false, XQA_BF16>(p.kv_dtype, cfg, p);
}

}  // namespace xqa
