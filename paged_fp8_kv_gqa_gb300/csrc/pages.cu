// pages.cu — the pages of growing and ending sequences (xqa_assign_pages, xqa_release_pages).
//
// The pool's free pages are a stack: free_pages[0 .. num_free). A step in which sequence b
// grows by n_b tokens takes ceil((c_b + n_b) / 16) - ceil(c_b / 16) pages for it, sequence
// after sequence, from the stack's end; a sequence that ends puts its pages back, sequence
// after sequence, in the order of its table. So both are prefix sums over the sequences and
// a write for each page and row:
//
//   rows before b   R_b = sum n_a,  pages before b   P_b = sum need_a   (a < b)
//   table[b][first_b + i] = free_pages[num_free - 1 - (P_b + i)],   i < need_b
//   row R_b + i: position c_b + i, slot = page * 16 + position % 16
//
// Sums of whole numbers: any order gives the same tables, nothing is left to the scheduling
// of threads. One cluster of CTAs: each scans all sequences for itself (a few KB from L2,
// where a second kernel or a wait for another CTA's sums would cost more than it), then
// they share the writes. The cluster's barrier stands between the last read of the lengths and
// of the stack's height and the first write, so the new ones may take their place.
//
// Bound by latency: three dependent reads and two block-wide scans. The work itself is 12
// bytes a row and 8 a page. Measured: a step of 16 tokens 3.5 us; 512 sequences of 0-512 new tokens
// 7.5 us; 2 of 16 sequences released 5.2 us, 200 of 512 7.7 us.
#include <cooperative_groups.h>

#include "xqa_device.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

namespace cg = cooperative_groups;

constexpr int kClusterCtas = 16;  // at most; fewer where the device has no place for so many
constexpr int kSmallThreads = 256, kLargeThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void raise(int32_t* status, int code) {
  if (status) atomicCAS(status, XQA_OK, code);
}

// Block-wide exclusive scan of two sums at once; sums: those of all threads. Every warp scans
// the warps' sums for itself.
struct Two {
  long long rows;
  int pages;
};
__device__ __forceinline__ Two warp_scan2(Two v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long r = __shfl_up_sync(kAll, v.rows, off);
    const int p = __shfl_up_sync(kAll, v.pages, off);
    if (lane >= off) v.rows += r, v.pages += p;
  }
  return v;
}
template <int kThreads>
__device__ __forceinline__ Two scan2(Two v, Two* warp_sums, Two& sums) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Two incl = warp_scan2(v);
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const Two w = warp_scan2(lane < kWarps ? warp_sums[lane] : Two{0, 0});
  sums.rows = __shfl_sync(kAll, w.rows, 31);
  sums.pages = __shfl_sync(kAll, w.pages, 31);
  Two before;
  before.rows = __shfl_sync(kAll, w.rows, max(warp - 1, 0));
  before.pages = __shfl_sync(kAll, w.pages, max(warp - 1, 0));
  if (warp == 0) before = Two{0, 0};
  __syncthreads();
  return Two{before.rows + incl.rows - v.rows, before.pages + incl.pages - v.pages};
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kBlockSize - 1) / kBlockSize; }

// Last index i in [0, n) with a[i] <= x (a ascends from a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (a[m] <= x) lo = m;
    else hi = m - 1;
  }
  return lo;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Height of the stack, -1 if the word cannot be one.
__device__ __forceinline__ int stack_height(const PagesParams& p) {
  const int f = *p.num_free;
  if (f >= 0 && f <= p.num_blocks) return f;
  raise(p.status, XQA_ERR_NO_PAGES);
  return -1;
}

template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) assign_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* row0 = smem;                // [batch + 1] first row of each sequence
  int* page0 = row0 + p.batch + 1; // [batch + 1] pages taken before it
  int* old = page0 + p.batch + 1;  // [batch] tokens before the step
  __shared__ Two sums[kThreads / 32];
  __shared__ int height;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  if (tid == 0) height = max(stack_height(p), 0);  // (read behind the first scan)
  Two before{0, 0};
  long long rows = 0;  // served so far
  int taken = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int n = 0, c = 0;
    if (b < p.batch) {
      n = p.new_tokens[b];
      c = p.context_lens[b];
      old[b] = c;
      if (n < 0 || c < 0 || (long long)c + n > (long long)p.max_blocks_per_seq * kBlockSize) {
        raise(p.status, XQA_ERR_CTX_TOO_LONG);
        n = 0;
      }
    }
    const int need = n > 0 ? pages_of(c + n) - pages_of(c) : 0;
    Two all;
    const Two at = scan2<kThreads>(Two{n, need}, sums, all);
    // Refused: rows past the caller's, pages past the stack. Both only begin at some
    // sequence and stay, so the pages of those that are served have no gaps.
    bool refused = false;
    if (n > 0 && before.rows + at.rows + n > p.num_rows) {
      refused = true;
      raise(p.status, XQA_ERR_BAD_OFFSETS);
    } else if (need > 0 && (long long)before.pages + at.pages + need > height) {
      refused = true;
      raise(p.status, XQA_ERR_NO_PAGES);
    }
    const int served = refused ? 0 : n;
    if (__syncthreads_or(refused)) {  // rows and pages of those that are left
      Two left;
      const Two now = scan2<kThreads>(Two{served, refused ? 0 : need}, sums, left);
      if (b < p.batch) {
        row0[b] = (int)(rows + now.rows);
        page0[b] = taken + now.pages;
      }
      rows += left.rows;
      taken += left.pages;
    } else {
      if (b < p.batch) {
        row0[b] = (int)(rows + at.rows);
        page0[b] = taken + at.pages;
      }
      rows += all.rows;
      taken += all.pages;
    }
    before.rows += all.rows;
    before.pages += all.pages;
  }
  if (tid == 0) {
    row0[p.batch] = (int)rows;
    page0[p.batch] = taken;
  }
  if (kCluster) cg::this_cluster().sync();  // every CTA has read what is written below
  else __syncthreads();
  const int free_now = height;
  const int ctas = kCluster ? gridDim.x : 1;
  const int first = blockIdx.x * kThreads + tid, stride = ctas * kThreads;
  for (int b = first; b <= p.batch; b += stride) {
    p.cu_seqlens[b] = row0[b];
    if (b < p.batch) p.new_lens[b] = old[b] + (row0[b + 1] - row0[b]);
    else *p.new_free = free_now - taken;
  }
  for (int i = first; i < taken; i += stride) {
    const int b = last_at_most(page0, p.batch, i);
    const int id = p.free_pages[free_now - 1 - i];
    p.block_tables[(size_t)b * p.max_blocks_per_seq + pages_of(old[b]) + (i - page0[b])] = id;
    if ((uint32_t)id >= (uint32_t)p.num_blocks) raise(p.status, XQA_ERR_BAD_BLOCK_ID);
  }
  if (!p.slots && !p.positions) return;
  // four rows to a thread: one search, four table entries asked for at once, 16-byte writes
  for (int r0 = 4 * first; r0 < p.num_rows; r0 += 4 * stride) {
    int b = r0 < rows ? last_at_most(row0, p.batch, r0) : 0;
    int pos[4], id[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + k;
      pos[k] = id[k] = -1;
      if (r >= rows) continue;
      while (r >= row0[b + 1]) ++b;
      const int c = old[b];
      pos[k] = c + (r - row0[b]);
      const int j = pos[k] / kBlockSize, fresh = j - pages_of(c);  // fresh: its entry is being written
      const int32_t* entry = fresh < 0 ? p.block_tables + (size_t)b * p.max_blocks_per_seq + j
                                       : p.free_pages + (free_now - 1 - (page0[b] + fresh));
      if (p.slots) id[k] = *entry;
    }
    auto write = [&](int32_t* dst, const int (&v)[4]) {
      if (!dst) return;
      if (r0 + 4 <= p.num_rows && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<int4*>(dst + r0) = make_int4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r0 + k < p.num_rows) dst[r0 + k] = v[k];
      }
    };
    write(p.positions, pos);
    if (!p.slots) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (pos[k] < 0) continue;
      if ((uint32_t)id[k] < (uint32_t)p.num_blocks) id[k] = id[k] * kBlockSize + pos[k] % kBlockSize;
      else id[k] = -1, raise(p.status, XQA_ERR_BAD_BLOCK_ID);
    }
    write(p.slots, id);
  }
}

// The entries that go back form one list, sequence after sequence, of which every warp takes
// an equal run: it counts the valid ones, every CTA of the cluster is told, and behind a scan of
// the warps' counts they are written.
constexpr int kPerLane = 8;  // entries of a lane in flight at once
template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) release_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* first = smem;                  // [batch + 1] entries before each sequence's
  int* lens = first + p.batch + 1;    // [batch] new lengths
  constexpr int kWarps = kThreads / 32;
  __shared__ Two sums[kWarps];
  __shared__ int count[kClusterCtas * kWarps];
  __shared__ int height;
  griddep_launch_dependents();
  if (kCluster) cluster_arrive();  // (this CTA runs: its memory is there)
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = kCluster ? gridDim.x : 1;
  const int warp = blockIdx.x * kWarps + (tid >> 5), warps = ctas * kWarps;
  if (tid == 0) height = stack_height(p);
  int entries = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int pages = 0;
    if (b < p.batch) {
      const bool ends = p.done[b] != 0;
      const int c = p.context_lens[b];
      const bool bad = c < 0 || c > (long long)p.max_blocks_per_seq * kBlockSize;
      if (ends && bad) raise(p.status, XQA_ERR_CTX_TOO_LONG);
      pages = ends && !bad ? pages_of(c) : 0;
      lens[b] = ends ? 0 : c;
    }
    Two all;
    const Two at = scan2<kThreads>(Two{0, pages}, sums, all);
    if (b < p.batch) first[b] = entries + at.pages;
    entries += all.pages;
  }
  if (tid == 0) first[p.batch] = entries;
  __syncthreads();
  // (places in the list are unsigned: an end or a step past the last of 2^31 of them wraps otherwise)
  const uint32_t run = (uint32_t)(((long long)entries + 32 * warps - 1) / (32 * warps) * 32);
  const uint32_t from = (uint32_t)min((long long)warp * run, (long long)entries);
  const uint32_t to = min(from + run, (uint32_t)entries);
  // A lane's entries ascend: its sequence is looked for again only where one ends.
  struct At {
    const int32_t* row;  // row[i]: the table's entry of list entry i < next
    uint32_t next;
  };
  auto read = [&](uint32_t i0, At& at, int (&id)[kPerLane]) {  // entries i0 + 32 e + lane; -1 past the run
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const uint32_t i = i0 + 32 * e + lane;
      id[e] = -1;
      if (i >= to) continue;
      if (i >= at.next) {
        const int b = last_at_most(first, p.batch, (int)i);
        at.row = p.block_tables + ((long long)b * p.max_blocks_per_seq - first[b]);
        at.next = first[b + 1];
      }
      id[e] = at.row[i];
    }
  };
  int good = 0, id[kPerLane];
  At place{nullptr, 0};
  for (uint32_t i0 = from; i0 < to; i0 += 32 * kPerLane) {
    read(i0, place, id);
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const bool ok = (uint32_t)id[e] < (uint32_t)p.num_blocks;
      good += ok;
      if (!ok && i0 + 32 * e + lane < to) raise(p.status, XQA_ERR_BAD_BLOCK_ID);
    }
  }
  good = __reduce_add_sync(kAll, good);
  if (kCluster) {
    cluster_wait();
    if (lane < ctas) *cg::this_cluster().map_shared_rank(count + warp, lane) = good;
    cg::this_cluster().sync();  // every count is there, and every CTA has read the lengths
  } else {
    if (lane == 0) count[warp] = good;
    __syncthreads();
  }
  const int free_now = height;
  if (free_now < 0) {  // where the stack ends is not known: nothing goes back, nothing is lost
    for (int b = blockIdx.x * kThreads + tid; b < p.batch; b += ctas * kThreads) p.new_lens[b] = p.context_lens[b];
    if (blockIdx.x == 0 && tid == 0) *p.new_free = *p.num_free;
    return;
  }
  Two all;
  const Two mine = scan2<kThreads>(Two{tid < warps ? count[tid] : 0, 0}, sums, all);
  if (tid < warps) count[tid] = (int)mine.rows;
  __syncthreads();
  if (free_now + all.rows > p.num_blocks && tid == 0) raise(p.status, XQA_ERR_NO_PAGES);
  for (int b = blockIdx.x * kThreads + tid; b < p.batch; b += ctas * kThreads) p.new_lens[b] = lens[b];
  if (blockIdx.x == 0 && tid == 0)
    *p.new_free = (int)min(free_now + all.rows, (long long)p.num_blocks);
  long long at = (long long)free_now + count[warp];
  place.next = 0;
  for (uint32_t i0 = from; i0 < to; i0 += 32 * kPerLane) {
    if (run > 32 * kPerLane) read(i0, place, id);  // (one round's are still there)
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const unsigned some = __ballot_sync(kAll, (uint32_t)id[e] < (uint32_t)p.num_blocks);
      const long long slot = at + __popc(some & ((1u << lane) - 1));
      if ((some >> lane & 1) && slot < p.num_blocks) p.free_pages[slot] = id[e];
      at += __popc(some);
    }
  }
}

cudaLaunchConfig_t config(int ctas, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cfg;
}

}  // namespace

// A small CTA where one round of it takes every sequence and row, a large one where it has few
// rows or pages to write, else a cluster of `cluster` CTAs (1: one alone). When this was chosen a step of 16 tokens took 4.7 us
// in 256 threads, 6.4 in 1024 (a barrier of 32 warps at each turn); 3.5 us now.
cudaError_t launch_assign(const PagesParams& p, int cluster, cudaStream_t stream) {
  const bool small = p.batch <= kSmallThreads && p.num_rows <= 4 * kSmallThreads;
  const bool many = p.num_rows > 4 * kLargeThreads;
  const int ctas = many ? cluster : 1;
  const size_t smem = sizeof(int) * (3 * (size_t)p.batch + 2);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(ctas, small ? kSmallThreads : kLargeThreads, smem, stream, attr);
  if (small) return cudaLaunchKernelEx(&cfg, assign_kernel<kSmallThreads, false>, p);
  return many ? cudaLaunchKernelEx(&cfg, assign_kernel<kLargeThreads, true>, p)
              : cudaLaunchKernelEx(&cfg, assign_kernel<kLargeThreads, false>, p);
}

// (how many pages go back is known to the device alone: the tables' width stands for it)
cudaError_t launch_release(const PagesParams& p, int cluster, cudaStream_t stream) {
  const bool small = p.batch <= kSmallThreads &&
                     (long long)p.batch * p.max_blocks_per_seq <= 32ll * kPerLane * (kSmallThreads / 32);
  const size_t smem = sizeof(int) * (2 * (size_t)p.batch + 1);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(small ? 1 : cluster, small ? kSmallThreads : kLargeThreads,
                                        smem, stream, attr);
  return small ? cudaLaunchKernelEx(&cfg, release_kernel<kSmallThreads, false>, p)
               : cudaLaunchKernelEx(&cfg, release_kernel<kLargeThreads, true>, p);
}

namespace {

// The largest cluster, halving from kClusterCtas, that `fits`.
template <class Fits>
int largest_cluster(Fits fits) {
  int ctas = kClusterCtas;
  while (ctas > 1 && !fits(ctas)) ctas /= 2;
  return ctas;
}

// Whether a cluster of `ctas` CTAs of the kernel with the most shared memory it may ask for has
// a place. (16 are more than every device of an architecture need offer, and a context may be
// limited to some of the SMs.)
bool has_place(void (*kernel)(PagesParams), int ctas, size_t smem) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(ctas, kLargeThreads, smem, nullptr, attr);
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess) return clusters > 0;
  cudaGetLastError();  // (as a size that does not fit may be reported)
  return false;
}

}  // namespace

cudaError_t set_pages_attributes(int* cluster) {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int assign = sizeof(int) * (3 * kMaxPagesBatch + 2), release = sizeof(int) * (2 * kMaxPagesBatch + 1);
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(assign_kernel<kLargeThreads, true>, a, assign)) != cudaSuccess) return e;
  const cudaFuncAttribute any = cudaFuncAttributeNonPortableClusterSizeAllowed;
  if ((e = cudaFuncSetAttribute(assign_kernel<kLargeThreads, true>, any, 1)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(release_kernel<kLargeThreads, true>, any, 1)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(assign_kernel<kLargeThreads, false>, a, assign)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(release_kernel<kLargeThreads, true>, a, release)) != cudaSuccess) return e;
  *cluster = largest_cluster([&](int ctas) {
    return has_place(assign_kernel<kLargeThreads, true>, ctas, assign) &&
           has_place(release_kernel<kLargeThreads, true>, ctas, release);
  });
  return cudaSuccess;
}

}  // namespace xqa
