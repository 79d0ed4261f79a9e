// extend.cu — attention of a chunk of new tokens over the paged cache (xqa_extend).
//
//   out[i, h] = sum_t softmax_t(sm_scale k_scale <q[i, h], K_t>) v_scale V_t,
//   t < ctx, and for causal calls t <= ctx - n + i (i of the sequence's n queries, t its
//   cached tokens, the chunk's own among them); a row that sees nothing, or logits of -inf
//   alone, is zero.
//
// Prompt attention's mathematics (a running maximum and sum over 128-key tiles, products
// on tcgen05, two 128-row tiles worked in turn) on keys and values that are read as they
// lie in the cache: 8 or 4 bits, 16-token pages in any order. Six warps turn each tile's
// codes into the queries' 16-bit type in shared memory; every code's value (times its
// group's scale in a 4-bit cache) is exact there, so the products are those of the cached
// values, and the tensor's scales are applied in 32 bits (to the logits, to out).
//
// Work: a unit is 2 x T consecutive tokens of one sequence and the G heads of one kv head,
// T = floor(128 / G). The units lie on a line, each as long as the keys it sees plus a
// constant, and every CTA takes an equal share of the line: long sequences are cut
// anywhere, at 128-key tiles, without the host knowing a length. A unit cut into pieces
// leaves (O, m, l) of each in 32 bits in the workspace, and a second, small kernel joins
// them with the whole GPU. (Joined by the CTA that wrote a unit's last piece, 32 tokens over
// 131072 took 1340 us, 16 x 32 over 2048 85 us; so 29 and 35 us.)
//
// A unit of at most T tokens fills one row tile only; both chains of product, softmax
// and product then work on it, on every other key tile each, and are joined in the
// epilogue.
//
// Warps: 0-3 and 4-7 softmax of chain 0 and 1 (a thread owns a row), 8-11 epilogue, 12
// tensor core, 13 units and loads, 14-19 codes to 16-bit values. TMEM: S0, S1 (P over
// them), O0, O1: 4 x 128 columns.
//
// Bound by the chain of product, softmax and product where units have two row tiles (4 chunks
// of 1024-2048 tokens up to contexts of 6000-16384, 32/4 heads, E5M2: 642 us, 0.80 of the
// library product's rate for the visible pairs), by one row tile's softmax and the tiles'
// conversion where they have one (16 x 2-32 tokens over 4000-17000, 32/4, E4M3: 72 us, 168 MB,
// 0.34 of the copy rate), by its latencies if it is short (5 tokens over 128: 9.0 us).
//
// Hidden values do not leak: see prompt attention; here rows past the sequence and values
// that are not finite are zeroed as they are converted. A page whose table entry is out of
// range has keys of NaN: the rows that see it are NaN, the others are not touched.
#include <math.h>

#include "xqa_tcgen05.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

constexpr int kKvStages = 3;    // 16-bit K or V tiles
constexpr int kUnitSlots = 3;
constexpr int kExtendThreads = 640;  // whole groups of four warps, as their register split needs
constexpr int kConvertWarps = 6;
constexpr int kTilePages = kTile / kBlockSize;
constexpr float kNoRowMax = -3e38f;     // as in prompt attention
constexpr float kExactMax = 4194304.f;
constexpr float kLazyMax = 8.0f;
constexpr uint32_t kWaitLimit = 2000000000u >> 16;  // about 1 s in units of 2^16 clocks
constexpr int kUnitReaders = 13 + kConvertWarps;  // 8 softmax, 4 epilogue, 1 tensor-core
constexpr int kRawBytes = 4 * kTile * kHeadDim;  // the ring of codes

template <int kFmt>
struct Raw {
  static constexpr int kSlice = kFmt == XQA_KV_E2M1 ? kSliceBytes4 : kPageBytes;
  static constexpr int kBytes = kTilePages * kSlice;  // codes of a tile
  static constexpr int kStages = kRawBytes / kBytes;  // 4, or 7 of 4 bits
};

struct Unit {
  int end;       // 1: no more units
  int bad;       // 1: NaN rows (a bad length or scale)
  int seq;
  int q_row;     // first token's row in q and out
  int tokens;    // 1 .. 2 T
  int head;      // kv head
  int page0;     // first page of the piece within the sequence's table row
  int len_k;     // keys of the piece, from the first of page0
  int vis0;      // keys the first token sees (causal: one more per token)
  int n[2];      // KV tiles row tile 0 / 1 sees
  int split;     // 1: both chains work on row tile 0
  int hidden;    // first key hidden from some token
  int slot;      // place of this piece's (O, m, l); -1: the unit is one piece
};

// A sequence's rows and tokens.
struct Seq {
  int q0, n, ctx;  // ctx: -1 if the length is invalid
};

struct Shared {
  uint64_t raw_full[7], raw_empty[7];
  uint64_t kv_full[kKvStages], kv_empty[kKvStages];
  uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
  uint64_t q_full, q_empty;
  uint64_t s_full[2];
  uint64_t p_full[2][2];
  uint64_t o_full[2], o_free[2];
  uint64_t stat_full[2], stat_free[2];
  uint64_t drain;
  Unit unit[kUnitSlots];
  int not_finite[kUnitSlots];
  int bad_pages[7];              // of the codes' stage, a bit for each page
  int status;
  uint32_t wait_limit;           // of every wait; 0: the CTA is aborted
  uint32_t tmem;
  // the line (block-wide scan)
  long long scan[kExtendThreads / 32][2];
  long long share, extra;        // of a CTA on the line (one more for the first `extra` CTAs)
  long long start_at;            // where the CTA's first sequence begins
  Seq start;
  int start_seq, ctas;           // ctas: that share the line
};

constexpr int kSmemTiles = (2 + kKvStages) * kTileBytes;
constexpr int kSmemStats = 2 * kTile * 2 * 4;
constexpr int kExtendSmem = kSmemTiles + kRawBytes + kSmemStats + 1024;
static_assert(sizeof(Shared) <= 1024, "shared state");
static_assert(kExtendSmem <= 227 * 1024, "shared memory budget");

// ---- the line of work ----
// A sequence of n tokens: np = ceil(n / 2T) units for each kv head; unit i sees base +
// min(step (i + 1), rows) keys at most, and is kKeyCost long for each of them, or key_cost_one if
// it fills one row tile only, and kUnitCost more for its start and end.
constexpr int kKeyCost = 16, kUnitCost = kExtendUnitKeys * kKeyCost;
constexpr int kCutTiles = 8;  // units of fewer tiles are not cut
struct Cost {
  int np;
  long long base;
  int step, rows;
  int last_key;  // cost of a key in the last unit
  __device__ __forceinline__ long long upto(int i) const {  // cost of the units before i < np
    return i * (kUnitCost + kKeyCost * base) + kKeyCost * (step * ((long long)i * (i + 1) / 2));
  }
  __device__ __forceinline__ int key(int i) const { return i == np - 1 ? last_key : kKeyCost; }
  __device__ __forceinline__ long long unit(int i) const {
    return kUnitCost + key(i) * (base + min((long long)step * (i + 1), (long long)rows));
  }
  __device__ __forceinline__ long long head() const { return np == 0 ? 0 : upto(np - 1) + unit(np - 1); }
};

__device__ __forceinline__ Seq read_seq(const ExtendParams& p, int b, int* status) {
  Seq s;
  s.q0 = p.cu_q[b];
  const int q1 = p.cu_q[b + 1];
  s.ctx = p.context_lens[b];
  s.n = 0;
  if (s.q0 >= 0 && q1 >= s.q0 && q1 <= p.total_q) s.n = q1 - s.q0;
  else record_status(status, XQA_ERR_BAD_OFFSETS);
  if (s.ctx < 0 || s.ctx > (long long)p.max_blocks_per_seq * kBlockSize) {
    s.ctx = -1;
    if (s.n > 0) record_status(status, XQA_ERR_CTX_TOO_LONG);
  }
  return s;
}

__device__ __forceinline__ Cost seq_cost(const ExtendParams& p, const Seq& s) {
  Cost c;
  const int per = 2 * p.tile_tokens;
  c.np = (int)(((long long)s.n + per - 1) / per);
  const bool causal = p.causal && s.ctx >= 0;
  c.base = causal ? max(0, s.ctx - s.n) : max(0, s.ctx);
  c.step = causal ? per : 0;
  c.rows = causal ? s.n : 0;
  c.last_key = s.n - (c.np - 1) * per <= p.tile_tokens ? p.key_cost_one : kKeyCost;
  return c;
}

// Quotient of positions of the line (64-bit division is a long chain of instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// Block-wide exclusive scan of a sequence's length on the line, and the sums of it and of the
// rows; every thread calls it.
__device__ __forceinline__ long long scan_all(long long v, int rows, Shared& sh, long long& sum,
                                              long long& sum_rows) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v, all_rows = rows;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(kAll, incl, off);
    if (lane >= off) incl += x;
    all_rows += __shfl_xor_sync(kAll, all_rows, off);
  }
  if (lane == 31) sh.scan[warp][0] = incl, sh.scan[warp][1] = all_rows;
  __syncthreads();
  long long w = lane < kExtendThreads / 32 ? sh.scan[lane][0] : 0;
  long long r = lane < kExtendThreads / 32 ? sh.scan[lane][1] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(kAll, w, off);
    if (lane >= off) w += x;
    r += __shfl_xor_sync(kAll, r, off);
  }
  sum = __shfl_sync(kAll, w, 31);
  sum_rows = r;
  const long long before = __shfl_sync(kAll, w, max(warp - 1, 0));
  __syncthreads();
  return (warp > 0 ? before : 0) + incl - v;
}

struct Ctx {
  const ExtendParams& p;
  Shared& sh;
  uint8_t* tiles;  // Q0, Q1, then the 16-bit ring
  uint8_t* raw;
  float* stats;    // [2][128][2]
  uint32_t tmem;

  __device__ __forceinline__ uint8_t* kv(int stage) const { return tiles + (2 + stage) * kTileBytes; }

  // Warp-uniform wait within the CTA's limit; false ends the role (the CTA is aborted).
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
    volatile uint32_t* limit = &sh.wait_limit;
    const uint32_t t0 = (uint32_t)(clock64() >> 16);
    do {
      if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
    } while (__all_sync(kAll, (uint32_t)(clock64() >> 16) - t0 < *limit));
    *limit = 0;
    return false;
  }
  __device__ __forceinline__ bool get_unit(int i, Unit& u) const {
    const int slot = i % kUnitSlots;
    if (!wait(&sh.unit_full[slot], (i / kUnitSlots) & 1)) return false;
    u = sh.unit[slot];
    return !u.end;
  }
  __device__ __forceinline__ void arrive(uint64_t* bar) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ void free_unit(int i) const { arrive(&sh.unit_empty[i % kUnitSlots]); }
};

// The order in which a unit's tiles pass through the rings: the first `lag` K tiles, then V
// and the K tile `lag` below it in turn (lag: 1, or 2 where the chains take turns).
struct TileOrder {
  int n, lag;
  __device__ __forceinline__ TileOrder(const Unit& u) : n(max(u.n[0], u.n[1])), lag(u.split ? 2 : 1) {}
  // tile of item t (0 .. 2 n - 1), and whether it is V's
  __device__ __forceinline__ int at(int t, bool& is_v) const {
    const int u = t - lag;
    if (u < 0) {
      is_v = false;
      return n - 1 - t;
    }
    const int both = 2 * (n - lag);
    is_v = u >= both || (u & 1) == 0;
    return u >= both ? lag - 1 - (u - both) : n - 1 - (u >> 1) - (is_v ? 0 : lag);
  }
};

// Page ids of a table row, read 32 at a time (four tiles) by a whole warp. Tiles are taken from
// the last to the first, V's one or two behind K's: two groups are in use, the next is on its
// way.
struct PageIds {
  const int32_t* row;
  int pages, group, high, low, next;
  __device__ __forceinline__ int read(int g) const {
    const int i = g * 32 + (threadIdx.x & 31);
    return g >= 0 && i < pages ? row[i] : -1;
  }
  __device__ __forceinline__ void start(const int32_t* r, int n, int tile) {
    row = r;
    pages = n;
    group = tile >> 2;
    high = read(group);
    low = read(group - 1);
    next = read(group - 2);
  }
  // id of page `lane & 7` of a tile; top: V's next tile, the highest still to come
  __device__ __forceinline__ int of(int tile, int top) {
    if (top >> 2 != group) {
      group = top >> 2;
      high = low;
      low = next;
      next = read(group - 2);
    }
    return __shfl_sync(kAll, tile >> 2 == group ? high : low, (tile & 3) * 8 + (threadIdx.x & 7));
  }
};

// Four whole rows of a matrix (a box of one row), one behind the other.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int r0,
                                            int r1, int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(0), "r"(r0), "r"(r1), "r"(r2),
      "r"(r3)
      : "memory");
}

constexpr int kTilesBeforeQ = 3;
static_assert(kTilesBeforeQ < kKvStages + kRawBytes / (kTile * kHeadDim), "room of the rings");
// Codes of a unit's tiles into the ring; item: the ring's number of its first tile.
template <int kFmt>
__device__ __forceinline__ bool load_tiles(const Ctx& c, const Unit& w, const CUtensorMap* tm_q,
                                           const CUtensorMap* tm_k, const CUtensorMap* tm_v, int item,
                                           int& issued, int& q_issued) {
  const ExtendParams& p = c.p;
  Shared& sh = c.sh;
  constexpr int kStages = Raw<kFmt>::kStages, kSlice = Raw<kFmt>::kSlice;
  const int lane = threadIdx.x & 31;
  const TileOrder order(w);
  const int pages = (w.len_k + kBlockSize - 1) / kBlockSize;
  const bool nhd = kFmt != XQA_KV_E2M1 && p.kv_layout == XQA_LAYOUT_NHD;
  PageIds ids;
  ids.start(p.block_tables + (size_t)w.seq * p.max_blocks_per_seq + w.page0, pages, order.n - 1);
  const int q_tiles = w.split ? 1 : 2;
  if (lane < 2 * q_tiles && w.n[lane >> 1] > 0)  // into L2 while the unit before still uses Q's place
    tma_prefetch_4d(tm_q, 64 * (lane & 1), 0, w.head, w.q_row + (lane >> 1) * p.tile_tokens);
  // (few instructions: one warp's, one after the other, are what a tile waits for)
  int jk = order.n - 1, jv = order.n - 1, st = item % kStages;
  uint32_t parity = (item / kStages - 1) & 1;  // (the phase before a ring's first is over)
  for (int t = 0; t < 2 * order.n; ++t) {
    // Q behind the first tiles, which so are on their way while the unit before ends (Q first:
    // 10 to 24 us more a unit). The rings have room for them and more: no tile behind waits
    // for one that waits for Q.
    if (t == min(kTilesBeforeQ, 2 * order.n - 1)) {
      if (q_issued > 0 && !c.wait(&sh.q_empty, (q_issued - 1) & 1)) return false;
      if (lane == 0) {
        const int half = p.group * p.tile_tokens * 128;  // bytes of a half tile
        int row_tiles = 0;
        for (int r = 0; r < q_tiles; ++r) row_tiles += w.n[r] > 0;
        mbar_arrive_expect_tx(&sh.q_full, 2 * half * row_tiles);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (r >= q_tiles || w.n[r] == 0) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_4d(c.tiles + r * kTileBytes + h * kHalfBytes, tm_q, &sh.q_full, 64 * h, 0,
                        w.head, w.q_row + r * p.tile_tokens);
        }
      }
      __syncwarp();
      ++q_issued;
    }
    const bool is_v = jk < 0 || (t >= order.lag && !((t - order.lag) & 1));
    const int j = is_v ? jv : jk;
    const int id = ids.of(j, jv);  // page `lane & 7` of the tile
    jv -= is_v;
    jk -= !is_v;
    const bool want = lane < kTilePages && j * kTilePages + lane < pages;
    const bool good = want && (uint32_t)id < (uint32_t)p.num_blocks;
    const uint32_t none = __ballot_sync(kAll, want && !good);
    uint64_t* full = &sh.raw_full[st];
    uint8_t* dst = c.raw + st * Raw<kFmt>::kBytes + lane * kSlice;
    const CUtensorMap* tm = is_v ? tm_v : tm_k;
    if (nhd) {
      const uint32_t bytes = __popc(__ballot_sync(kAll, good)) * kSlice;
      if (!c.wait(&sh.raw_empty[st], parity)) return false;
      if (lane == 0) {
        sh.bad_pages[st] = none;
        mbar_arrive_expect_tx(full, bytes);
      }
      __syncwarp();
      if (good) tma_load_kv(dst, tm, full, 0, w.head, id * kBlockSize);
    } else {
      // slices are rows of one matrix: four at a time. In place of pages that are not there or
      // not good, the pool's first: their tokens are hidden or replaced
      const int row = good ? id * p.num_kv_heads + w.head : w.head;
      const int r1 = __shfl_down_sync(kAll, row, 1), r2 = __shfl_down_sync(kAll, row, 2);
      const int r3 = __shfl_down_sync(kAll, row, 3);
      if (!c.wait(&sh.raw_empty[st], parity)) return false;
      if (lane == 0) {
        sh.bad_pages[st] = none;
        mbar_arrive_expect_tx(full, kTilePages * kSlice);
      }
      __syncwarp();
      if (lane == 0 || lane == 4) tma_gather4(dst, tm, full, row, r1, r2, r3);
    }
    if (none) record_status(&sh.status, XQA_ERR_BAD_BLOCK_ID);
    issued = item + t + 1;
    if (++st == kStages) st = 0, parity ^= 1;
    __syncwarp();
  }
  return true;
}

// ---- warp 13: the units of this CTA, their queries and codes ----
template <int kFmt>
__device__ __forceinline__ void load_role(const Ctx& c, const CUtensorMap* tm_q,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          bool bad_scale, int& raw_issued, int& q_issued) {
  const ExtendParams& p = c.p;
  Shared& sh = c.sh;
  const int lane = threadIdx.x & 31;
  const int per = 2 * p.tile_tokens;
  const long long share = sh.share, extra = sh.extra;
  const int cta = blockIdx.x;
  const long long lo = cta * share + min((long long)cta, extra);
  const long long hi = lo + share + (cta < extra ? 1 : 0);  // (begin_of(cta + 1))
  auto begin_of = [&](int c) { return c * share + min((long long)c, extra); };
  const float per_share = __frcp_rn((float)share);
  auto owner = [&](long long x) {  // CTA of a position of the line: an estimate, put right
    int c = min((int)((float)x * per_share), sh.ctas - 1);
    while (begin_of(c) > x) --c;
    while (c + 1 < sh.ctas && begin_of(c + 1) <= x) ++c;
    return c;
  };
  int base = -1, b = sh.start_seq, item = 0;  // sequences base .. base + 31, one a lane
  Seq mine{0, 0, 0};
  auto read_chunk = [&]() {
    mine.q0 = mine.n = 0;
    mine.ctx = 0;
    if (base + lane < p.batch) mine = read_seq(p, base + lane, &sh.status);
  };
  SplitUnit split_unit{0, 0, 0, 0};  // the one whose first piece is this CTA's
  long long at = sh.start_at;  // where sequence b begins
  Seq s = sh.start;
  Cost cost = seq_cost(p, s);
  int head = 0, pair = 0;
  long long pos = lo;
  if (lo > at) {  // the unit that holds lo
    const long long one = cost.head();
    if (lo - at >= one) head = (int)quotient(lo - at, one);
    const long long rem = lo - at - head * one;
    int a = 0, z = cost.np - 1;  // the last unit that begins at or before rem
    while (a < z) {
      const int m = (a + z + 1) >> 1;
      if (cost.upto(m) <= rem) a = m;
      else z = m - 1;
    }
    pair = a;
    at += head * one;  // now: where this head begins
  }
  for (int i = 0;; ++i) {
    const int slot = i % kUnitSlots;
    if (i >= kUnitSlots && !c.wait(&sh.unit_empty[slot], (i / kUnitSlots - 1) & 1)) return;
    if (pos >= hi) {
      if (lane == 0) {
        p.split[cta] = split_unit;
        sh.unit[slot].end = 1;
        mbar_arrive(&sh.unit_full[slot]);
      }
      return;
    }
    const long long u0 = at + cost.upto(pair), len = cost.unit(pair);
    const long long x0 = max(lo, u0) - u0, x1 = min(hi, u0 + len) - u0;
    Unit w;
    w.end = 0;
    w.bad = s.ctx < 0 || bad_scale;
    w.seq = b;
    const int tok0 = pair * per;
    w.q_row = s.q0 + tok0;
    w.tokens = min(per, s.n - tok0);
    w.head = head;
    int len_k = w.bad ? 0 : s.ctx;
    int vis0 = p.causal ? len_k - s.n + tok0 + 1 : len_k;
    const int last = p.causal ? min(len_k, vis0 + w.tokens - 1) : len_k;
    const int tiles = last > 0 ? (last - 1) / kTile + 1 : 0;
    w.slot = -1;
    int t0 = 0, t1 = tiles;
    bool some = true;  // there is a tile for this CTA
    if (x0 > 0 || x1 < len) {
      // Tile at which a cut at position x of the unit falls. A short unit is not cut, and no
      // end of less than a quarter of a CTA's share (and of what a unit's start and end cost) is
      // cut off: leaving a piece and joining it costs about as much. Such a cut moves to the
      // unit's end. (Four tiles of two row tiles: 16 short turns 77.4 us, so 74.2.)
      const bool full = cost.key(pair) == kKeyCost;  // (divisors known to the compiler)
      const int cost_one = p.key_cost_one;
      auto in_tiles = [&](long long x) {
        return full                       ? x / (kTile * kKeyCost)
               : cost_one == kKeyCostOne ? x / (kTile * kKeyCostOne)
                                         : x / (kTile * kKeyCostOneSlow);
      };
      const int least = (int)min(full ? 2ll : 4ll, max(1ll, in_tiles(share >> 2)));
      auto tile_of = [&](long long x) {
        const long long y = x - kUnitCost + kTile / 2 * cost.key(pair);
        const int at = (int)min((long long)tiles, in_tiles(max(0ll, y)));
        if (tiles < kCutTiles) return 2 * at < tiles ? 0 : tiles;
        return at < least ? 0 : tiles - at < least ? tiles : at;
      };
      if (x0 > 0) t0 = tile_of(x0);
      if (x1 < len) t1 = tile_of(x1);
      int first = owner(u0), last_cta = owner(u0 + len - 1);
      if (tiles == 0) {
        some = x0 == 0;
      } else {
        some = t1 > t0;
        // cuts at an end leave nothing to the unit's first or last CTAs
        while (first < last_cta && tile_of(begin_of(first + 1) - u0) == 0) ++first;
        while (first < last_cta && tile_of(begin_of(last_cta) - u0) == tiles) --last_cta;
        if (some && first < last_cta) {
          w.slot = 2 * cta + (cta == first);
          if (cta == first) {  // its other pieces are those of the next CTAs
            split_unit.pieces = last_cta - first + 1;
            split_unit.q_row = w.q_row;
            split_unit.tokens = w.tokens;
            split_unit.head = head;
          }
        }
      }
    }
    w.page0 = t0 * kTilePages;
    w.len_k = max(0, min(len_k, t1 * kTile) - t0 * kTile);
    w.vis0 = p.causal ? vis0 - t0 * kTile : w.len_k;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int toks = min(p.tile_tokens, w.tokens - r * p.tile_tokens);
      const int seen = p.causal ? min(w.len_k, w.vis0 + r * p.tile_tokens + toks - 1) : w.len_k;
      w.n[r] = toks > 0 && seen > 0 ? (seen - 1) / kTile + 1 : 0;
    }
    w.split = w.tokens <= p.tile_tokens && w.n[0] >= 2;
    if (w.split) w.n[1] = w.n[0];
    w.hidden = max(0, min(w.vis0, w.len_k));
    if (some && lane == 0) {
      sh.unit[slot] = w;
      sh.not_finite[slot] = 0;
      if (const uint32_t more = max(w.n[0], w.n[1]) >> 16) {  // (an abort stays one)
        const uint32_t limit = *(volatile uint32_t*)&sh.wait_limit;
        if (limit != 0 && limit < (1 + more) * kWaitLimit)
          atomicCAS(&sh.wait_limit, limit, (1 + more) * kWaitLimit);
      }
      mbar_arrive(&sh.unit_full[slot]);
    }
    if (!some) --i;  // the unit's place serves the next one
    else if (max(w.n[0], w.n[1]) > 0) {
      if (!load_tiles<kFmt>(c, w, tm_q, tm_k, tm_v, item, raw_issued, q_issued)) return;
      item += 2 * max(w.n[0], w.n[1]);
    }
    // on to the next unit
    pos = u0 + len;
    if (++pair < cost.np) continue;
    pair = 0;
    at = pos;
    if (++head < p.num_kv_heads || pos >= hi) continue;
    head = 0;
    if (base < 0) {
      base = b & ~31;
      read_chunk();
    }
    for (;;) {  // the next sequence with tokens (there is one: the line goes on)
      const uint32_t some = __ballot_sync(kAll, mine.n > 0 && base + lane > b);
      if (some) {
        b = base + __ffs(some) - 1;
        break;
      }
      base += 32;
      if (base >= p.batch) return;  // cannot be
      b = base - 1;
      read_chunk();
    }
    s.q0 = __shfl_sync(kAll, mine.q0, b - base);
    s.n = __shfl_sync(kAll, mine.n, b - base);
    s.ctx = __shfl_sync(kAll, mine.ctx, b - base);
    cost = seq_cost(p, s);
  }
}

// ---- warp 12: the products ----
// The chains in turn, as in prompt attention: O += P V of a tile, then S of the chain's next
// tile over P.
template <int kType>
__device__ __forceinline__ void tensor_role(const Ctx& c) {
  Shared& sh = c.sh;
  const uint32_t tiles = __shfl_sync(kAll, smem_addr(c.tiles), 0);
  const uint32_t tmem = __shfl_sync(kAll, c.tmem, 0);
  const uint64_t q_desc = desc_k_major(tiles);
  const uint64_t k_desc = desc_k_major(tiles + 2 * kTileBytes);
  const uint64_t v_desc = desc_mn_major(tiles + 2 * kTileBytes);
  int item = 0, units = 0;
  uint32_t ph_p = 0, ph_o = 3;
  // a tile of the ring in turn: its stage, once it is there
  auto stage = [&](int it) { return it % kKvStages; };
  auto arrived = [&](int it) { return c.wait(&sh.kv_full[it % kKvStages], (it / kKvStages) & 1); };
  for (int i = 0;; ++i) {
    Unit w;
    if (!c.get_unit(i, w)) return;
    c.free_unit(i);
    const int n0 = __shfl_sync(kAll, w.n[0], 0), n1 = __shfl_sync(kAll, w.n[1], 0);
    const int split = __shfl_sync(kAll, w.split, 0);
    const int n = max(n0, n1), lag = 1 + split;
    if (n == 0) continue;
    if (!c.wait(&sh.q_full, units & 1)) return;
    ++units;
    auto score = [&](int s, int st) {  // S of chain s
      const uint64_t a = q_desc + (split ? 0 : s) * (kTileBytes >> 4);
      const uint64_t b = k_desc + st * (kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
          tc_mma_ss(tmem + s * kTile, a + off, b + off, instr_desc<kType>(false), k > 0);
        }
        tc_commit(&sh.s_full[s]);
      }
      __syncwarp();
    };
    for (int t = 0; t < lag; ++t, ++item) {  // the first K tiles
      if (!arrived(item)) return;
      tc_fence_after();
#pragma unroll 1
      for (int s = 0; s < 2; ++s)
        if (split ? s == t : (s ? n1 : n0) == n) score(s, stage(item));
      if (elect_one()) tc_commit(&sh.kv_empty[stage(item)]);
      __syncwarp();
    }
    if (n == lag && elect_one()) tc_commit(&sh.q_empty);
    __syncwarp();
    for (int j = n - 1; j >= 0; --j) {
      const int vi = item++;
      const bool next = j >= lag;
      const int ki = next ? item++ : 0;
      if (!arrived(vi)) return;
#pragma unroll 1
      for (int s = 0; s < 2; ++s) {
        const int ns = s ? n1 : n0;
        if (split && ((n - 1 - j) & 1) != s) continue;
        if (j < ns) {
          const bool start = split ? j >= n - 2 : j == ns - 1;
          if (start) {
            if (!c.wait(&sh.o_free[s], ph_o >> s & 1)) return;
            ph_o ^= 1u << s;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // as P's halves are written
            const uint32_t bit = 2 * s + h;
            if (!c.wait(&sh.p_full[s][h], ph_p >> bit & 1)) return;
            ph_p ^= 1u << bit;
            tc_fence_after();
            const uint64_t vb = v_desc + stage(vi) * (kTileBytes >> 4) + h * (4 * 2048 >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma_ts(tmem + 256 + s * kTile, tmem + s * kTile + 32 * h + 8 * k,
                          vb + k * (2048 >> 4), instr_desc<kType>(true), !start || h + k > 0);
            }
            __syncwarp();
          }
          if (j < lag && elect_one()) tc_commit(&sh.o_full[s]);
          __syncwarp();
        }
        // V's place is free behind its last product, while K's is being used
        if ((split || s == 1) && elect_one()) tc_commit(&sh.kv_empty[stage(vi)]);
        __syncwarp();
        if (next && j - lag < ns) {
          if (!arrived(ki)) return;
          tc_fence_after();
          score(s, stage(ki));
        }
      }
      if (next && elect_one()) {
        tc_commit(&sh.kv_empty[stage(ki)]);
        if (j == lag) tc_commit(&sh.q_empty);
      }
      __syncwarp();
    }
  }
}

// ---- warps 14-19: codes to 16-bit values ----
// 16 neighbouring dims of a token, as 8 pairs.
template <int kType>
__device__ __forceinline__ uint32_t half2_as(uint32_t h) {  // exact: at most 6 significant bits
  if (kType == XQA_F16) return h;
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack2<XQA_BF16>(f.x, f.y);
}
template <int kFmt>
struct Codes16 {
  uint4 w;
};
template <>
struct Codes16<XQA_KV_E2M1> {
  uint2 w;
  uint32_t s8;  // the group's scale
};
// Codes of dims 16 group .. 16 group + 15 of a tile's token `row`.
template <int kFmt>
__device__ __forceinline__ Codes16<kFmt> read16(const uint8_t* raw, int row, int group) {
  Codes16<kFmt> c;
  if constexpr (kFmt == XQA_KV_E2M1) {
    const uint8_t* page = raw + (row >> 4) * kSliceBytes4;
    c.w = lds64(page + (row & 15) * (kHeadDim / 2) + 8 * group);
    c.s8 = lds_u8(page + kCodeBytes4 + (row & 15) * (kHeadDim / kGroup4) + group);
  } else {
    c.w = lds128(raw + row * kHeadDim + 16 * group);
  }
  return c;
}
template <int kFmt, int kType>
__device__ __forceinline__ void convert16(const Codes16<kFmt>& c, uint32_t (&o)[8]) {
  if constexpr (kFmt == XQA_KV_E2M1) {
    const uint32_t sc = e4m3x2_to_f16x2(c.s8 | c.s8 << 8);
    e2m1x8_to_f16x2(c.w.x, o);
    e2m1x8_to_f16x2(c.w.y, o + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = half2_as<kType>(hmul2(o[i], sc));
  } else {
    const uint32_t x[4] = {c.w.x, c.w.y, c.w.z, c.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = half2_as<kType>(KvConv<kFmt>::k_lo(x[i]));
      o[2 * i + 1] = half2_as<kType>(KvConv<kFmt>::k_hi(x[i]));
    }
  }
}

// Whether one of 16 values is an infinity or NaN (0: none).
template <int kFmt>
__device__ __forceinline__ uint32_t not_finite16(const Codes16<kFmt>& c) {
  if constexpr (kFmt == XQA_KV_E2M1) {
    return (c.s8 & 0x7fu) == 0x7fu;
  } else {  // a byte's largest exponent, or E4M3's one pattern, is the one that carries
    constexpr uint32_t top = kFmt == XQA_KV_E5M2 ? 0x7c7c7c7cu : 0x7f7f7f7fu;
    constexpr uint32_t one = 0x80808080u - top;
    return (((c.w.x & top) + one) | ((c.w.y & top) + one) | ((c.w.z & top) + one) |
            ((c.w.w & top) + one)) & 0x80808080u;
  }
}

template <int kFmt>
__device__ __forceinline__ void clear16(uint8_t* raw, int row, int group) {
  if constexpr (kFmt == XQA_KV_E2M1) {
    uint8_t* page = raw + (row >> 4) * kSliceBytes4;
    *reinterpret_cast<uint2*>(page + (row & 15) * (kHeadDim / 2) + 8 * group) = make_uint2(0, 0);
    page[kCodeBytes4 + (row & 15) * (kHeadDim / kGroup4) + group] = 0;
  } else {
    *reinterpret_cast<uint4*>(raw + row * kHeadDim + 16 * group) = make_uint4(0, 0, 0, 0);
  }
}

template <int kFmt, int kType>
__device__ __forceinline__ void convert_role(const Ctx& c) {
  Shared& sh = c.sh;
  constexpr int kStages = Raw<kFmt>::kStages;
  const int warp = (threadIdx.x >> 5) - 14, lane = threadIdx.x & 31;
  const uint32_t exp_mask = kType == XQA_F16 ? 0x7c00u : 0x7f80u;
  // Eight lanes take the first 64 dims of one token and the last 64 of its neighbour, the
  // next eight the other halves: whole 128-byte runs are read, and a store's 16-byte
  // chunks, which the swizzle would pair up within one token, fall into different banks.
  const int half = lane >> 2 & 1, group = 4 * half + (lane & 3);
  const int row_in4 = 2 * (lane >> 4) + (half ^ (lane >> 3 & 1));
  int item = 0;
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
    const TileOrder order(u);
    bool found = false;
    for (int t = 0; t < 2 * order.n; ++t, ++item) {
      bool is_v;
      const int j = order.at(t, is_v);
      const int rs = item % kStages, st = item % kKvStages;
      if (!c.wait(&sh.raw_full[rs], (item / kStages) & 1)) return;
      if (item >= kKvStages && !c.wait(&sh.kv_empty[st], (item / kKvStages - 1) & 1)) return;
      uint8_t* raw = c.raw + rs * Raw<kFmt>::kBytes;
      uint8_t* dst = c.kv(st) + half * kHalfBytes;
      const int bad = *(volatile int*)&sh.bad_pages[rs];
      const bool masked = is_v && (j + 1) * kTile > u.hidden;
      // rows row0, row0 + 4 kConvertWarps, ...: a multiple of 8 apart, so that the swizzle is
      // the same for all of a thread's rows
      constexpr int kStep = 4 * kConvertWarps, kTurns = (kTile + kStep - 1) / kStep;
      static_assert(kStep % 8 == 0, "swizzle");
      const int row0 = 4 * warp + row_in4;
      const uint32_t swz0 = ((2 * (group & 3)) ^ (row0 & 7)) * 16, swz1 = swz0 ^ 16;
      auto store = [&](int row, const uint32_t (&o)[8]) {
        *reinterpret_cast<uint4*>(dst + row * 128 + swz0) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + row * 128 + swz1) = make_uint4(o[4], o[5], o[6], o[7]);
      };
      const int past = u.len_k - j * kTile, from = u.hidden - j * kTile;
      uint32_t odd = bad;  // pages that are not there, hidden values that are not finite
      if (masked && !bad) {  // tokens behind the last one become zeros where they lie
#pragma unroll 1
        for (int row = row0; row < kTile; row += kStep) {
          if (row >= past) clear16<kFmt>(raw, row, group);
          else if (row >= from) odd |= not_finite16<kFmt>(read16<kFmt>(raw, row, group));
        }
        odd = __any_sync(kAll, odd);
      }
      if (odd) {
#pragma unroll 1
        for (int row = row0; row < kTile; row += kStep) {
          uint32_t o[8];
          convert16<kFmt, kType>(read16<kFmt>(raw, row, group), o);
          const bool none = bad >> (row >> 4) & 1;
          const bool zero = is_v && (none || row >= past);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (zero) o[k] = 0;
            else if (none) o[k] = 0x7fff7fffu;  // NaN in both types
            else if (masked && row >= from) {
              if ((o[k] & exp_mask) == exp_mask) o[k] &= 0xffff0000u, found = true;
              if ((o[k] & exp_mask << 16) == exp_mask << 16) o[k] &= 0x0000ffffu, found = true;
            }
          }
          store(row, o);
        }
        if (found) *(volatile int*)&sh.not_finite[i % kUnitSlots] = 1;
      } else {
        Codes16<kFmt> w[kTurns];  // every read of the tile before the first use
#pragma unroll
        for (int k = 0; k < kTurns; ++k)
          if (row0 + k * kStep < kTile) w[k] = read16<kFmt>(raw, row0 + k * kStep, group);
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
          if (row0 + k * kStep >= kTile) continue;
          uint32_t o[8];
          convert16<kFmt, kType>(w[k], o);
          store(row0 + k * kStep, o);
        }
      }
      fence_proxy_async_smem();  // before the tensor core reads the tile
      c.arrive(&sh.kv_full[st]);
      c.arrive(&sh.raw_empty[rs]);
    }
    c.free_unit(i);
  }
}

struct RowPos {
  int token;  // within the unit
  int head;   // within the group
  bool valid;
};
__device__ __forceinline__ RowPos row_pos(const ExtendParams& p, const Unit& u, int r, int row) {
  RowPos x;
  const int t = row / p.group;
  x.head = row - t * p.group;
  x.token = r * p.tile_tokens + t;
  x.valid = t < p.tile_tokens && x.token < u.tokens;
  return x;
}
__device__ __forceinline__ int visible(const ExtendParams& p, const Unit& u, const RowPos& r) {
  if (!r.valid) return 0;
  return p.causal ? max(0, min(u.len_k, u.vis0 + r.token)) : u.len_k;
}

// ---- warps 0-7: softmax of chain s; a thread owns a row (as in prompt attention) ----
template <int kType>
__device__ __forceinline__ void softmax_role(const Ctx& c, int s, float sc) {
  const ExtendParams& p = c.p;
  Shared& sh = c.sh;
  const int row = threadIdx.x & 127;
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  const uint32_t s_addr = lane_base + s * kTile, o_addr = lane_base + 256 + s * kTile;
  int ns = 0, nstat = 0;
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
    const int r = u.split ? 0 : s;  // row tile
    const RowPos rp = row_pos(p, u, r, row);
    const int vis = visible(p, u, rp);
    c.free_unit(i);
    const int n = s == 0 ? u.n[0] : u.n[1];
    if (n == 0) continue;
    const bool idle = !__any_sync(kAll, rp.valid);  // no row of this warp is a token's
    // keys that every token of this row tile sees
    const int clear = p.causal ? min(u.len_k, u.vis0 + r * p.tile_tokens) : u.len_k;
    float m = kNoRowMax, m_raw = 0.f, l = 0.f;  // m_raw: m before the scale
    for (int j = u.split ? n - 1 - s : n - 1; j >= 0; j -= 1 + u.split) {
      if (!c.wait(&sh.s_full[s], ns & 1)) return;
      ++ns;
      tc_fence_after();
      if (idle) {  // P is what S left there: rows that nobody reads
        tc_fence_before();
        c.arrive(&sh.p_full[s][0]);
        c.arrive(&sh.p_full[s][1]);
        continue;
      }
      if ((j + 1) * kTile > clear) {  // keys that a row does not see: -inf
        const int lim = vis - j * kTile;
#pragma unroll 1
        for (int q = max(0, __reduce_min_sync(kAll, lim)) >> 5; q < 4; ++q) {
          uint32_t v[32];
          tmem_ld32(s_addr + 32 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * q + k >= lim) v[k] = 0xff800000u;
          tmem_st32(s_addr + 32 * q, v);
        }
        tmem_wait_st();
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t v[32];
        tmem_ld32(s_addr + 32 * q, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(v[k + e])), __uint_as_float(v[k + 4 + e]));
      }
      const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), top = raw * sc;
      const bool moves = top > m + kLazyMax;
      const bool scale_o = moves && m != kNoRowMax;
      const float old = m;
      if (moves) m = top, m_raw = raw;
      uint64_t m2 = f32x2(-m, -m);
      // large maxima are subtracted before the scale (see prompt attention)
      const bool exact = fabsf(m) > kExactMax && m != kNoRowMax && vis > 0;
      if (__any_sync(kAll, scale_o)) {
        const float a = scale_o ? ex2(old - top) : 1.f;
        l *= a;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t o[32];
          tmem_ld32(o_addr + 32 * q, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
          tmem_st32(o_addr + 32 * q, o);
        }
      }
      const bool any_exact = __any_sync(kAll, exact);
      const float minus = exact ? m_raw : 0.f;
      if (exact) m2 = 0;
      const uint64_t sc2 = f32x2(sc, sc);
      uint64_t sum[2] = {0, 0};
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {  // P of 32 keys over S of keys that are read already
        uint32_t v[32], pk[16];
        tmem_ld32(s_addr + 32 * q, v);
        tmem_wait_ld();
        if (any_exact) {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) - minus);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float a, b;
          split2(fma2(f32x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc2, m2), a, b);
          a = ex2(a);
          b = ex2(b);
          sum[k & 1] = add2(sum[k & 1], f32x2(a, b));
          pk[k] = pack2<kType>(a, b);
        }
        tmem_st16(s_addr + 16 * q, pk);
        if (q & 1) {
          tmem_wait_st();
          tc_fence_before();
          c.arrive(&sh.p_full[s][q >> 1]);
        }
      }
      float la, lb;
      split2(add2(sum[0], sum[1]), la, lb);
      l += la + lb;
    }
    if (nstat > 0 && !c.wait(&sh.stat_free[s], (nstat - 1) & 1)) return;
    ++nstat;
    float2* st = reinterpret_cast<float2*>(c.stats) + s * kTile + row;
    *st = make_float2(m, l);
    c.arrive(&sh.stat_full[s]);
  }
}

// Value (before the tensor's scale) of one cached V element if it is not finite, else 0.
template <int kFmt>
__device__ __noinline__ float not_finite_value(const uint8_t* slice, long long token_stride, int slot,
                                               int dim) {
  uint32_t h;
  if constexpr (kFmt == XQA_KV_E2M1) {
    const uint32_t s8 = slice[kCodeBytes4 + slot * (kHeadDim / kGroup4) + dim / kGroup4];
    h = e4m3x2_to_f16x2(s8);
  } else {
    const uint32_t code = slice[slot * token_stride + dim];
    h = KvConv<kFmt>::k_lo(code);
  }
  return (h & 0x7c00u) == 0x7c00u ? __half2float(__ushort_as_half((unsigned short)h)) : 0.f;
}

// ---- warps 8-11: normalise and write, or leave a piece ----
template <int kFmt, int kType>
__device__ __forceinline__ void epilogue_role(const Ctx& c, float v_scale) {
  const ExtendParams& p = c.p;
  Shared& sh = c.sh;
  const int row = threadIdx.x & 127;
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  uint32_t ph = 0;  // a bit for each chain
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
    const bool piece = u.slot >= 0;
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      if (u.split && s == 1) break;
      const RowPos rp = row_pos(p, u, s, row);
      const int n_s = s ? u.n[1] : u.n[0];
      const long long at = (long long)u.q_row + rp.token;
      const int h = u.head * p.group + rp.head;
      uint16_t* out = p.out + at * p.out_row_stride + h * p.out_head_stride;
      const size_t place = (size_t)(u.slot * 2 + s);
      if (n_s == 0) {  // no tokens, or tokens that see nothing
        if (piece) p.piece_ml[place * kTile + row] = make_float2(kNoRowMax, 0.f);
        else if (rp.valid) {
          const uint32_t f = !u.bad ? 0u : kType == XQA_F16 ? 0x7fff7fffu : 0x7fc07fc0u;
#pragma unroll 1
          for (int k = 0; k < kHeadDim / 8; ++k)
            reinterpret_cast<uint4*>(out)[k] = make_uint4(f, f, f, f);
          if (p.lse) p.lse[at * p.num_q_heads + h] = u.bad ? __int_as_float(0x7fc00000) : -INFINITY;
        }
        continue;
      }
      // the chain's (m, l), or both chains' and their weights
      float2 ml;
      float w0 = 1.f, w1 = 0.f;
      if (!c.wait(&sh.stat_full[s], ph >> s & 1)) return;
      ml = reinterpret_cast<const float2*>(c.stats)[s * kTile + row];
      c.arrive(&sh.stat_free[s]);
      if (u.split) {
        if (!c.wait(&sh.stat_full[1], ph >> 1 & 1)) return;
        const float2 b = reinterpret_cast<const float2*>(c.stats)[kTile + row];
        c.arrive(&sh.stat_free[1]);
        const float m = ml.y == 0.f ? b.x : b.y == 0.f ? ml.x : fmaxf(ml.x, b.x);
        // a chain with keys keeps the least weight there is: its infinities and NaN are the row's
        w0 = ml.y != 0.f ? fmaxf(ex2(ml.x - m), 0x1p-149f) : 0.f;
        w1 = b.y != 0.f ? fmaxf(ex2(b.x - m), 0x1p-149f) : 0.f;
        ml = make_float2(m, (ml.y != 0.f ? w0 * ml.y : 0.f) + (b.y != 0.f ? w1 * b.y : 0.f));
        if (!c.wait(&sh.o_full[1], ph >> 1 & 1)) return;
        ph ^= 2u;
      }
      if (!c.wait(&sh.o_full[s], ph >> s & 1)) return;
      ph ^= 1u << s;
      tc_fence_after();
      const bool patch = *(volatile int*)&sh.not_finite[i % kUnitSlots] != 0;
      const int vis = visible(p, u, rp);
      const float rl = ml.y == 0.f ? 0.f : v_scale / ml.y;
      uint16_t* dst[4];  // this lane's 16 bytes of four lanes' rows
      const unsigned long long mine = rp.valid ? reinterpret_cast<unsigned long long>(out) : 0ull;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned long long a = __shfl_sync(kAll, mine, (threadIdx.x & 28) + k);
        dst[k] = a ? reinterpret_cast<uint16_t*>(a) + 8 * (threadIdx.x & 3) : nullptr;
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        __syncwarp();  // rows part ways below
        tmem_ld32(lane_base + 256 + s * kTile + 32 * q, o);
        tmem_wait_ld();
        if (u.split) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t o1[16];
            tmem_ld16(lane_base + 256 + kTile + 32 * q + 16 * e, o1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float a = w0 != 0.f ? w0 * __uint_as_float(o[16 * e + k]) : 0.f;
              const float b = w1 != 0.f ? w1 * __uint_as_float(o1[k]) : 0.f;
              o[16 * e + k] = __float_as_uint(a + b);
            }
          }
        }
        if (q == 3) {  // O is read
          tc_fence_before();
          c.arrive(&sh.o_free[s]);
          if (u.split) c.arrive(&sh.o_free[1]);
        }
        if (patch) {  // infinities and NaN that were zeroed, for rows that see them
          const int32_t* table = p.block_tables + (size_t)u.seq * p.max_blocks_per_seq + u.page0;
#pragma unroll 1
          for (int key = u.hidden; key < vis; ++key) {
            const int id = table[key / kBlockSize];
            if ((uint32_t)id >= (uint32_t)p.num_blocks) continue;
            const bool nhd = kFmt != XQA_KV_E2M1 && p.kv_layout == XQA_LAYOUT_NHD;
            const uint8_t* slice =
                p.v_pool + (nhd ? ((size_t)id * kBlockSize * p.num_kv_heads + u.head) * kHeadDim
                                : ((size_t)id * p.num_kv_heads + u.head) * Raw<kFmt>::kSlice);
            const long long stride = nhd ? (long long)p.num_kv_heads * kHeadDim : kHeadDim;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint(__uint_as_float(o[k]) +
                                     not_finite_value<kFmt>(slice, stride, key % kBlockSize, 32 * q + k));
          }
        }
        if (piece) {  // as it is, a row of 128 values after the other, in runs of 64 bytes
          const int rows = min(p.tile_tokens, u.tokens - s * p.tile_tokens) * p.group;
          float* po = p.piece_o + (place * kTile + (row & ~3)) * kHeadDim + 32 * q + 4 * (row & 3);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = o[16 * e + k];
            trade<1>(w);
            trade<2>(w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((row & ~3) + k < rows)
                *reinterpret_cast<uint4*>(po + k * kHeadDim + 16 * e) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a, b;
            split2(mul2(f32x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), f32x2(rl, rl)),
                   a, b);
            w[k] = pack2<kType>(a, b);
          }
          trade<1>(w);
          trade<2>(w);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k])
              *reinterpret_cast<uint4*>(dst[k] + 32 * q) =
                  make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        }
      }
      if (piece) p.piece_ml[place * kTile + row] = ml;
      else if (p.lse && rp.valid)
        p.lse[at * p.num_q_heads + h] =
            ml.y == 0.f ? -INFINITY : (ml.x + __log2f(ml.y)) * 0.6931471805599453f;
    }
    c.free_unit(i);
  }
}

template <int kFmt, int kType>
__global__ void __launch_bounds__(kExtendThreads, 1)
    extend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const ExtendParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* raw = smem + kSmemTiles;
  float* stats = reinterpret_cast<float*>(raw + kRawBytes);
  Shared& sh = *reinterpret_cast<Shared*>(raw + kRawBytes + kSmemStats);
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0);  // known to be warp-uniform
  const bool aligned = (smem_addr(smem) & 1023u) == 0;  // as the swizzle needs
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Raw<kFmt>::kStages; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kConvertWarps);
    }
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(&sh.kv_full[i], kConvertWarps);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_empty[i], kUnitReaders);
    }
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s][0], 4);
      mbar_init(&sh.p_full[s][1], 4);
      mbar_init(&sh.o_full[s], 1);
      mbar_init(&sh.o_free[s], 4);
      mbar_init(&sh.stat_full[s], 4);
      mbar_init(&sh.stat_free[s], 4);
    }
    mbar_init(&sh.drain, 1);
    sh.wait_limit = kWaitLimit;
    sh.status = aligned ? XQA_OK : XQA_ERR_LAUNCH;
    fence_mbar_init();
  }
  if (warp == 13 && (threadIdx.x & 31) == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // inputs are read, and outputs written, after the kernels before this one
  // the line's length, and the sequence that holds this CTA's first position
  const float ks = p.k_scale_ptr ? *p.k_scale_ptr : p.k_scale;
  const float vs = p.v_scale_ptr ? *p.v_scale_ptr : p.v_scale;
  long long total = 0, rows = 0, mine = 0, excl = 0;
  Seq s{0, 0, 0};
  const bool few = p.batch <= 32;  // every warp scans them for itself
  if (few) {
    const int lane = threadIdx.x & 31;
    if (lane < p.batch) s = read_seq(p, lane, &sh.status);
    mine = seq_cost(p, s).head() * p.num_kv_heads;
    total = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(kAll, total, off);
      if (lane >= off) total += x;
    }
    excl = total - mine;
    total = __shfl_sync(kAll, total, 31);
    rows = ((long long)__reduce_add_sync(kAll, s.n >> 16) << 16) + __reduce_add_sync(kAll, s.n & 0xffff);
  }
  for (int b0 = 0; !few && b0 < p.batch; b0 += kExtendThreads) {
    const int b = b0 + threadIdx.x;
    s = Seq{0, 0, 0};
    if (b < p.batch) s = read_seq(p, b, &sh.status);
    mine = seq_cost(p, s).head() * p.num_kv_heads;
    long long sum, sum_rows;
    excl = total + scan_all(mine, s.n, sh, sum, sum_rows);
    total += sum;
    rows += sum_rows;
  }
  // sequences that overlap (offsets that descend) could have any number of units
  if (rows > p.total_q) total = 0;
  int ctas = 1;
  if (total > 0) ctas = (int)min((long long)gridDim.x, max(1ll, total / (kExtendMinShare * kKeyCost)));
  const long long share = ctas == 1 ? total : quotient(total, ctas), extra = total - share * ctas;
  const long long lo = blockIdx.x * share + min((long long)blockIdx.x, extra);
  const bool works = total > 0 && blockIdx.x < ctas;
  if (p.batch > kExtendThreads && works) {  // once more: a thread keeps one sequence
    long long before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kExtendThreads) {
      const int b = b0 + threadIdx.x;
      s = Seq{0, 0, 0};
      if (b < p.batch) s = read_seq(p, b, &sh.status);
      mine = seq_cost(p, s).head() * p.num_kv_heads;
      long long sum, sum_rows;
      excl = before + scan_all(mine, s.n, sh, sum, sum_rows);
      before += sum;
      if (excl <= lo && lo < excl + mine) sh.start_seq = b, sh.start_at = excl, sh.start = s;
      if (lo < before) break;
    }
  } else if (excl <= lo && lo < excl + mine && (!few || threadIdx.x < 32)) {
    sh.start_seq = threadIdx.x;
    sh.start_at = excl;
    sh.start = s;
  }
  if (threadIdx.x == 0) {
    sh.share = share;
    sh.extra = extra;
    sh.ctas = ctas;
  }
  __syncthreads();
  const float sc = fmaxf((float)(p.qk_scale_base * (double)ks), 0x1p-126f);
  const bool bad_scale = !(ks > 0.f && sc < INFINITY);
  if (bad_scale && works && threadIdx.x == 0) record_status(&sh.status, XQA_ERR_VALUE);
  int raw_issued = 0, q_issued = 0;
  if (aligned && works) {
    const Ctx c{p, sh, smem, raw, stats, sh.tmem};
    __syncwarp();
    // 256 x 136 + 128 x 96 + 256 x 56 are the launch's 640 x 96. (The code is compiled for 96:
    // 20 bytes a thread are spilled, 28 over 4 bits.)
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp == 12) tensor_role<kType>(c);
      else if (warp == 13) load_role<kFmt>(c, &tm_q, &tm_k, &tm_v, bad_scale, raw_issued, q_issued);
      else convert_role<kFmt, kType>(c);
    } else if (warp >= 8) {
      epilogue_role<kFmt, kType>(c, vs);
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
      softmax_role<kType>(c, warp >> 2, sc);
    }
  }
  __syncwarp();
  // Products and their arrivals, and after an abort copies, may be in flight: they end
  // before the CTA's shared memory and TMEM are given up.
  if (aligned && (warp == 12 || warp == 13)) {
    int never = 0;
    bool ok = true;
    if (warp == 12) {
      if (elect_one()) tc_commit(&sh.drain);
      __syncwarp();
      ok = mbar_wait_bounded(&sh.drain, 0, &never);
    } else if (*(volatile uint32_t*)&sh.wait_limit == 0) {
      constexpr int kStages = Raw<kFmt>::kStages;
      for (int k = max(0, raw_issued - kStages); k < raw_issued; ++k)
        ok = mbar_wait_bounded(&sh.raw_full[k % kStages], (k / kStages) & 1, &never) && ok;
      if (q_issued > 0) ok = mbar_wait_bounded(&sh.q_full, (q_issued - 1) & 1, &never) && ok;
    }
    if (!ok) atomicExch(&sh.status, XQA_ERR_DRAIN_TIMEOUT);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(sh.tmem, 512);
  if (threadIdx.x == 0) {
    // no unit to join if the CTA had none or gave up. (Cleared at the start, in front of the
    // roles, the same store cost 10 % of long chunks: 4 chunks 655 us, 719 so.)
    if (!works || !aligned || sh.wait_limit == 0) p.split[blockIdx.x] = SplitUnit{0, 0, 0, 0};
    if (sh.wait_limit == 0) record_status(&sh.status, XQA_ERR_DEVICE_TIMEOUT);
    p.status[blockIdx.x] = sh.status;
    if (blockIdx.x == 0) p.header[0] = gridDim.x;
  }
}

// ---- the join of split units' pieces ----
// A team of 8 lanes has a row, 16 dims a lane. The pieces' (m, l) are read a piece a lane,
// which so weighs its piece for all; then each piece costs sixteen fused products a lane. Up to
// kTeamPieces pieces are one team's work; of more, the block's teams take equal runs, each with
// its own maximum, and join through shared memory. The kernel is a chain of memory round
// trips (the units, (m, l) and O at once, out) and the instructions that are a row's whatever
// its team: teams of 16 lanes in four blocks an SM (64 registers) took 17 us of 4 chunks, so 10.
constexpr int kTeamLanes = 8, kTeamVec = kHeadDim / 4 / kTeamLanes;
constexpr int kJoinThreads = 256, kTeams = kJoinThreads / kTeamLanes, kTeamPieces = 8;
constexpr int kJoinBlocks = 2;  // for each CTA of the kernel before: what an SM holds at once
static_assert(kTeams == 32, "parts of a row: one a lane");

// Weights of parts of a row, one a lane of kLanes (l = 0: a part without keys, whose O was not
// written); m and l become the whole's. A part with keys keeps the least weight there is: its
// infinities and NaN are the row's.
template <int kLanes>
__device__ __forceinline__ float weigh(float& m, float& l) {
  const bool some = l != 0.f;
  float top = some ? m : -INFINITY;
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, off));
  const float w = some ? fmaxf(ex2(m - top), 0x1p-149f) : 0.f;
  float sum = some ? w * l : 0.f;
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  m = top;
  l = sum;
  return w;
}
__device__ __forceinline__ void add(float4& a, float w, const float4& o) {
  a.x = fmaf(w, o.x, a.x);
  a.y = fmaf(w, o.y, a.y);
  a.z = fmaf(w, o.z, a.z);
  a.w = fmaf(w, o.w, a.w);
}

template <int kType>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) join_kernel(const ExtendParams p, int ctas) {
  __shared__ int first[kMaxCtas];      // work items before each split unit
  __shared__ SplitUnit unit[kMaxCtas];
  __shared__ short begin[kMaxCtas];    // the CTA of its first piece
  __shared__ float4 part_o[kTeams][kTeamVec * kTeamLanes];
  __shared__ float2 part_ml[kTeams];
  __shared__ int2 sums[kJoinThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at8 = tid % kTeamLanes, team = tid / kTeamLanes;
  const float vs = p.v_scale_ptr ? *p.v_scale_ptr : p.v_scale;
  // an item: a row a team, or a row of many pieces
  int total = 0, units = 0;
  for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {
    const int c = c0 + tid;
    SplitUnit u{0, 0, 0, 0};
    if (c < ctas) u = p.split[c];
    const int rows = u.pieces > 1 ? u.tokens * p.group : 0;
    const int n = u.pieces <= kTeamPieces ? (rows + kTeams - 1) / kTeams : rows;
    const unsigned some = __ballot_sync(kAll, n > 0);
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += x;
    }
    if (lane == 31) sums[warp] = make_int2(incl, __popc(some));
    __syncthreads();
    int before = total, at = units;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      if (w < warp) before += sums[w].x, at += sums[w].y;
      total += sums[w].x;
      units += sums[w].y;
    }
    if (n > 0) {
      at += __popc(some & ((1u << lane) - 1));
      first[at] = before + incl - n;
      begin[at] = (short)c;
      unit[at] = u;
    }
    __syncthreads();
  }
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int lo = 0, hi = units - 1;  // the last unit that begins at or before the item
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (first[m] <= item) lo = m;
      else hi = m - 1;
    }
    const int cta = begin[lo], pieces = unit[lo].pieces, rows = unit[lo].tokens * p.group;
    const bool many = pieces > kTeamPieces;
    const int at = item - first[lo], r = many ? at : at * kTeams + team;
    const bool valid = r < rows;
    const int t = min(r, rows - 1) / p.group, g = min(r, rows - 1) - t * p.group;
    const int s = t >= p.tile_tokens;
    const int row = (t - s * p.tile_tokens) * p.group + g;
    // piece k is in slot 1 of the first CTA, slot 0 of the others; a CTA has 2 x 2 tiles of rows
    const size_t place0 = (size_t)(4 * cta + s) * kTile + row;
    auto tile = [](int k) { return (4 * k + (k == 0 ? 2 : 0)) * kTile; };
    const int per = many ? (pieces + kTeams - 1) / kTeams : pieces;
    const int k0 = many ? team * per : 0, n = min(pieces - k0, per);  // (n <= 0: none)
    const float* o = p.piece_o + place0 * kHeadDim + 4 * at8;  // dims 4 at8 + 32 x ..
    float4 acc[kTeamVec];
#pragma unroll
    for (int x = 0; x < kTeamVec; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kNoRowMax, l = 0.f;
    // (teams of a warp may have different numbers of rounds: its shuffles are for all)
    for (int c0 = 0; c0 < per; c0 += kTeamLanes) {
      float cm = kNoRowMax, cl = 0.f;
      if (c0 + at8 < n) {
        const float2 ml = __ldcg(p.piece_ml + place0 + tile(k0 + c0 + at8));
        cm = ml.x, cl = ml.y;
      }
      constexpr int kAtOnce = 4;
      static_assert(kTeamLanes % kAtOnce == 0, "lanes of a round");
      float w = 0.f;
      for (int e0 = 0; e0 < min(per - c0, kTeamLanes); e0 += kAtOnce) {
        float4 v[kAtOnce][kTeamVec];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          const bool there = c0 + e0 + e < n;
          const float* x0 = o + (size_t)tile(k0 + c0 + e0 + e) * kHeadDim;
#pragma unroll
          for (int x = 0; x < kTeamVec; ++x)
            v[e][x] = there ? __ldcg(reinterpret_cast<const float4*>(x0 + 4 * kTeamLanes * x))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (e0 == 0) {
          // what these pieces, and the rounds before, weigh in the whole
          const float om = m, ol = l;
          w = weigh<kTeamLanes>(cm, cl);
          m = cm, l = cl;
          if (c0 > 0) {
            m = ol == 0.f ? cm : cl == 0.f ? om : fmaxf(om, cm);
            const float wa = ol != 0.f ? fmaxf(ex2(om - m), 0x1p-149f) : 0.f;
            const float wb = cl != 0.f ? fmaxf(ex2(cm - m), 0x1p-149f) : 0.f;
            l = (ol != 0.f ? wa * ol : 0.f) + (cl != 0.f ? wb * cl : 0.f);
            if (w != 0.f) w = fmaxf(w * wb, 0x1p-149f);
#pragma unroll
            for (int x = 0; x < kTeamVec; ++x) {
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
              if (wa != 0.f) add(a, wa, acc[x]);
              acc[x] = a;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e) {
          const float we = __shfl_sync(kAll, w, e0 + e, kTeamLanes);
          if (we == 0.f) continue;
#pragma unroll
          for (int x = 0; x < kTeamVec; ++x) add(acc[x], we, v[e][x]);
        }
      }
    }
    const long long q = (long long)unit[lo].q_row + t;
    const int h = unit[lo].head * p.group + g;
    uint16_t* out = p.out + q * p.out_row_stride + h * p.out_head_stride;
    auto write = [&](int dim, const float4& a, float rl) {
      *reinterpret_cast<uint2*>(out + dim) =
          make_uint2(pack2<kType>(a.x * rl, a.y * rl), pack2<kType>(a.z * rl, a.w * rl));
    };
    if (many) {
      __syncthreads();  // the item before is read
#pragma unroll
      for (int x = 0; x < kTeamVec; ++x) part_o[team][kTeamLanes * x + at8] = acc[x];
      if (at8 == 0) part_ml[team] = make_float2(m, l);
      __syncthreads();
      if (warp != 0) continue;
      const float2 ml = part_ml[lane];
      m = ml.x, l = ml.y;
      const float w = weigh<kTeams>(m, l);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);  // dims 4 lane ..
#pragma unroll 8
      for (int e = 0; e < kTeams; ++e) {
        const float we = __shfl_sync(kAll, w, e);
        if (we != 0.f) add(a, we, part_o[e][lane]);
      }
      write(4 * lane, a, l == 0.f ? 0.f : vs / l);
    } else if (valid) {
      const float rl = l == 0.f ? 0.f : vs / l;
#pragma unroll
      for (int x = 0; x < kTeamVec; ++x) write(4 * at8 + 4 * kTeamLanes * x, acc[x], rl);
    }
    if (p.lse && valid && (many ? lane : at8) == 0)
      p.lse[q * p.num_q_heads + h] =
          l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
  }
}

template <int kFmt, int kType>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                   const ExtendParams& p, const cudaLaunchConfig_t& cfg) {
  return cudaLaunchKernelEx(&cfg, extend_kernel<kFmt, kType>, tm_q, tm_k, tm_v, p);
}

template <int kFmt, int kType>
cudaError_t set_attribute() {
  return cudaFuncSetAttribute(extend_kernel<kFmt, kType>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kExtendSmem);
}

}  // namespace

cudaError_t launch_extend(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                          const ExtendParams& p, int dtype, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kExtendThreads);
  cfg.dynamicSmemBytes = kExtendSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool f16 = dtype == XQA_F16;
  cudaError_t e;
  switch (p.kv_dtype) {
    case XQA_KV_E5M2:
      e = f16 ? launch<XQA_KV_E5M2, XQA_F16>(tm_q, tm_k, tm_v, p, cfg)
              : launch<XQA_KV_E5M2, XQA_BF16>(tm_q, tm_k, tm_v, p, cfg);
      break;
    case XQA_KV_E4M3:
      e = f16 ? launch<XQA_KV_E4M3, XQA_F16>(tm_q, tm_k, tm_v, p, cfg)
              : launch<XQA_KV_E4M3, XQA_BF16>(tm_q, tm_k, tm_v, p, cfg);
      break;
    default:
      e = f16 ? launch<XQA_KV_E2M1, XQA_F16>(tm_q, tm_k, tm_v, p, cfg)
              : launch<XQA_KV_E2M1, XQA_BF16>(tm_q, tm_k, tm_v, p, cfg);
  }
  // one CTA shares nothing, and so do units of tables that are too short for a cut
  if (e != cudaSuccess || ctas == 1 || p.max_blocks_per_seq <= (kCutTiles - 1) * kTilePages) return e;
  cfg.gridDim = dim3((unsigned)(ctas * kJoinBlocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return f16 ? cudaLaunchKernelEx(&cfg, join_kernel<XQA_F16>, p, ctas)
             : cudaLaunchKernelEx(&cfg, join_kernel<XQA_BF16>, p, ctas);
}

cudaError_t set_extend_attributes() {
  cudaError_t e;
  if ((e = set_attribute<XQA_KV_E5M2, XQA_F16>()) != cudaSuccess) return e;
  if ((e = set_attribute<XQA_KV_E5M2, XQA_BF16>()) != cudaSuccess) return e;
  if ((e = set_attribute<XQA_KV_E4M3, XQA_F16>()) != cudaSuccess) return e;
  if ((e = set_attribute<XQA_KV_E4M3, XQA_BF16>()) != cudaSuccess) return e;
  if ((e = set_attribute<XQA_KV_E2M1, XQA_F16>()) != cudaSuccess) return e;
  return set_attribute<XQA_KV_E2M1, XQA_BF16>();
}

}  // namespace xqa
