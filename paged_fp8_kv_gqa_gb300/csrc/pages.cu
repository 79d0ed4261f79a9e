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
// bytes a row and 8 a page.
#include <cooperative_groups.h>

#include "xqa_device.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

namespace cg = cooperative_groups;

constexpr int kPageThreads = 512;
constexpr int kWarps = kPageThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void raise(int32_t* status, int code) {
  if (status) atomicCAS(status, XQA_OK, code);
}

// Block-wide exclusive scan of two sums at once; sums: those of all threads.
struct Two {
  long long rows;
  int pages;
};
__device__ __forceinline__ Two scan2(Two v, Two* warp_sums, Two& sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Two incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long r = __shfl_up_sync(kAll, incl.rows, off);
    const int p = __shfl_up_sync(kAll, incl.pages, off);
    if (lane >= off) incl.rows += r, incl.pages += p;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  Two before{0, 0};
  sums = Two{0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = sums;
    sums.rows += warp_sums[w].rows;
    sums.pages += warp_sums[w].pages;
  }
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

// Height of the stack, 0 if the word cannot be one.
__device__ __forceinline__ int stack_height(const PagesParams& p) {
  const int f = *p.num_free;
  if (f >= 0 && f <= p.num_blocks) return f;
  if (threadIdx.x == 0) raise(p.status, XQA_ERR_NO_PAGES);
  return 0;
}

template <bool kCluster>
__global__ void __launch_bounds__(kPageThreads) assign_kernel(const PagesParams p) {
  extern __shared__ int smem[];
  int* row0 = smem;                // [batch + 1] first row of each sequence
  int* page0 = row0 + p.batch + 1; // [batch + 1] pages taken before it
  int* old = page0 + p.batch + 1;  // [batch] tokens before the step
  __shared__ Two sums[kWarps];
  __shared__ int height;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x;
  if (tid == 0) height = stack_height(p);
  __syncthreads();
  const int free_now = height;
  Two before{0, 0};
  long long rows = 0;  // served so far
  int taken = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kPageThreads) {
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
    const Two at = scan2(Two{n, need}, sums, all);
    // Refused: rows past the caller's, pages past the stack. Both only begin at some
    // sequence and stay, so the pages of those that are served have no gaps.
    bool refused = false;
    if (n > 0 && before.rows + at.rows + n > p.num_rows) {
      refused = true;
      raise(p.status, XQA_ERR_BAD_OFFSETS);
    } else if (need > 0 && (long long)before.pages + at.pages + need > free_now) {
      refused = true;
      raise(p.status, XQA_ERR_NO_PAGES);
    }
    const int served = refused ? 0 : n;
    if (__syncthreads_or(refused)) {  // rows and pages of those that are left
      Two left;
      const Two now = scan2(Two{served, refused ? 0 : need}, sums, left);
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
  const int ctas = kCluster ? gridDim.x : 1;
  const int first = blockIdx.x * kPageThreads + tid, stride = ctas * kPageThreads;
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
  // four rows to a thread: one search, one 16-byte write
  for (int r0 = 4 * first; r0 < p.num_rows; r0 += 4 * stride) {
    int slot[4], pos[4];
    int b = r0 < rows ? last_at_most(row0, p.batch, r0) : 0;
    int page = -1, id = -1;  // the last one looked up
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + k;
      slot[k] = pos[k] = -1;
      if (r >= rows) continue;
      if (r >= row0[b + 1]) {
        do ++b;
        while (r >= row0[b + 1]);
        page = -1;
      }
      pos[k] = old[b] + (r - row0[b]);
      if (!p.slots) continue;
      const int j = pos[k] / kBlockSize;
      if (j != page) {
        page = j;
        const int fresh = j - pages_of(old[b]);  // its table entry is being written
        id = fresh < 0 ? p.block_tables[(size_t)b * p.max_blocks_per_seq + j]
                       : p.free_pages[free_now - 1 - (page0[b] + fresh)];
        if ((uint32_t)id >= (uint32_t)p.num_blocks) {
          raise(p.status, XQA_ERR_BAD_BLOCK_ID);
          id = -1;
        }
      }
      slot[k] = id < 0 ? -1 : id * kBlockSize + pos[k] % kBlockSize;
    }
    auto write = [&](int32_t* dst, const int (&v)[4]) {
      if (!dst) return;
      if (r0 + 4 <= p.num_rows && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<int4*>(dst + r0) = make_int4(v[0], v[1], v[2], v[3]);
      } else {
        for (int k = 0; k < 4; ++k)
          if (r0 + k < p.num_rows) dst[r0 + k] = v[k];
      }
    };
    write(p.slots, slot);
    write(p.positions, pos);
  }
}

// Table entries are taken in pieces of `piece` pages, a warp to a piece: the valid ones are
// counted, every CTA of the cluster is told, and after a scan they are written.
template <bool kCluster>
__global__ void __launch_bounds__(kPageThreads) release_kernel(const PagesParams p, int piece,
                                                               int pieces_per_seq) {
  extern __shared__ int smem[];  // [batch * pieces_per_seq] valid entries, then those before
  __shared__ Two sums[kWarps];
  __shared__ int height;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int ctas = kCluster ? gridDim.x : 1;
  const int warp0 = blockIdx.x * kWarps + (tid >> 5), warps = ctas * kWarps;
  const int items = p.batch * pieces_per_seq;
  if (tid == 0) height = stack_height(p);
  auto range = [&](int item, int& b, int& from, int& to) {  // table entries of a piece
    b = item / pieces_per_seq;
    from = (item - b * pieces_per_seq) * piece;
    to = 0;
    if (!p.done[b]) return;
    const int c = p.context_lens[b];
    if (c < 0 || c > (long long)p.max_blocks_per_seq * kBlockSize) {
      raise(p.status, XQA_ERR_CTX_TOO_LONG);
      return;
    }
    to = min(from + piece, pages_of(c));
  };
  if (kCluster) cg::this_cluster().sync();  // every CTA of the cluster runs: its memory is there
  for (int item = warp0; item < items; item += warps) {
    int b, from, to, count = 0;
    range(item, b, from, to);
    const int32_t* row = p.block_tables + (size_t)b * p.max_blocks_per_seq;
#pragma unroll 4
    for (int j = from + lane; j < to; j += 32) {
      const bool good = (uint32_t)row[j] < (uint32_t)p.num_blocks;
      count += good;
      if (!good) raise(p.status, XQA_ERR_BAD_BLOCK_ID);
    }
    count = __reduce_add_sync(kAll, count);
    if (kCluster) {
      if (lane < ctas) *cg::this_cluster().map_shared_rank(smem + item, lane) = count;
    } else if (lane == 0) {
      smem[item] = count;
    }
  }
  if (kCluster) cg::this_cluster().sync();
  else __syncthreads();
  const int free_now = height;
  long long total = 0;
  for (int i0 = 0; i0 < items; i0 += kPageThreads) {
    const int i = i0 + tid;
    Two all;
    const Two at = scan2(Two{i < items ? smem[i] : 0, 0}, sums, all);
    if (i < items) smem[i] = (int)min(total + at.rows, (long long)p.num_blocks);
    total += all.rows;
  }
  __syncthreads();
  if (free_now + total > p.num_blocks && tid == 0) raise(p.status, XQA_ERR_NO_PAGES);
  for (int item = warp0; item < items; item += warps) {
    int b, from, to;
    range(item, b, from, to);
    const int32_t* row = p.block_tables + (size_t)b * p.max_blocks_per_seq;
    int at = free_now + smem[item];
    for (int j0 = from; j0 < to; j0 += 32) {
      const int id = j0 + lane < to ? row[j0 + lane] : -1;
      const unsigned good = __ballot_sync(kAll, (uint32_t)id < (uint32_t)p.num_blocks);
      const int mine = at + __popc(good & ((1u << lane) - 1));
      if ((good >> lane & 1) && mine < p.num_blocks) p.free_pages[mine] = id;
      at += __popc(good);
    }
  }
  // the lengths: each sequence's only after the last read of it, by any CTA
  if (kCluster) cg::this_cluster().sync();
  else __syncthreads();
  for (int b = blockIdx.x * kPageThreads + tid; b < p.batch; b += ctas * kPageThreads)
    p.new_lens[b] = p.done[b] ? 0 : p.context_lens[b];
  if (blockIdx.x == 0 && tid == 0)
    *p.new_free = (int)min(free_now + total, (long long)p.num_blocks);
}

cudaLaunchConfig_t config(int ctas, size_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPageThreads);
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

constexpr int kClusterCtas = 8;  // the largest portable cluster

}  // namespace

// One CTA where it has a few rounds of rows or entries, else the cluster.
cudaError_t launch_assign(const PagesParams& p, cudaStream_t stream) {
  const int ctas = p.num_rows <= 4 * 4 * kPageThreads ? 1 : kClusterCtas;
  const size_t smem = sizeof(int) * (3 * (size_t)p.batch + 2);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(ctas, smem, stream, attr);
  return ctas > 1 ? cudaLaunchKernelEx(&cfg, assign_kernel<true>, p)
                  : cudaLaunchKernelEx(&cfg, assign_kernel<false>, p);
}

cudaError_t launch_release(const PagesParams& p, cudaStream_t stream) {
  int piece = 512;
  while (((long long)p.max_blocks_per_seq + piece - 1) / piece * p.batch > kMaxReleasePieces) piece *= 2;
  const int per_seq = (p.max_blocks_per_seq + piece - 1) / piece;
  const int items = per_seq * p.batch;
  const int ctas = items <= 4 * kWarps ? 1 : kClusterCtas;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(ctas, sizeof(int) * (size_t)items, stream, attr);
  return ctas > 1 ? cudaLaunchKernelEx(&cfg, release_kernel<true>, p, piece, per_seq)
                  : cudaLaunchKernelEx(&cfg, release_kernel<false>, p, piece, per_seq);
}

cudaError_t set_pages_attributes() {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int assign = sizeof(int) * (3 * kMaxPagesBatch + 2), release = sizeof(int) * kMaxReleasePieces;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(assign_kernel<true>, a, assign)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(assign_kernel<false>, a, assign)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(release_kernel<true>, a, release)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(release_kernel<false>, a, release);
}

}  // namespace xqa
