// prefill.cu — attention over whole prompts, packed by sequence (xqa_prefill).
//
//   out[i, h] = sum_j softmax_j(sm_scale <q[i, h], k[j, h / G]>) v[j, h / G],
//   j < len_k, and for causal calls j <= len_k - len_q + i (i, j counted within
//   the sequence); a row that sees nothing, or logits of -inf alone, is zero.
//
// One persistent CTA per SM works through units of 2 x 128 rows: the G query
// heads of one kv head for 2 x T consecutive tokens of one sequence, T =
// floor(128 / G), row = token * G + head. So a K or V tile is read once for all
// heads of its group, a short prompt still fills its rows, and the diagonal is
// cut in steps of 2 T tokens. A unit walks the 128-key tiles it can see from the
// last (the diagonal) to the first, with the usual running maximum and sum:
//
//   S = Q K^T             tcgen05, 128 x 128 x 128, fp32 in TMEM
//   P = 2^(S c - m)       softmax warps: TMEM -> registers -> TMEM, 16 bit
//   O = O + P V           tcgen05, P from TMEM, V from shared memory
//
// What bounds it: per 128 x 128 tile the tensor core needs 2 x 512 cycles (8192
// flop per cycle and SM), the exponentials 512 cycles (32 per cycle and SM), so
// the two row tiles of a unit are worked in turn: while one is in the tensor
// core, the other's softmax runs. The running maximum only moves when a logit
// exceeds it by more than 8 (log2), so O is rescaled seldom (P <= 2^8 stays
// exact enough: its rounding is relative); O and the row sum l stay in 32 bits,
// l sums the unrounded P. P is rounded to the inputs' type because a tcgen05
// product has both operands in 16 bits: at most 2^-8 (bf16) or 2^-11 (fp16) of each
// weight, the size of the rounding of out itself.
//
// Measured (32/4 heads): 1 x 16384 tokens bf16 1.39 ms, 1580 TFLOP/s of visible pairs,
// 0.83 of a library product's rate; 16 prompts of 190 to 2048 tokens fp16 164 to 167 us, 0.61:
// a tenth of the tiles is hidden, and a unit of 6 tiles starts and ends its two chains
// of dependent products and softmax anew (about 2 us of its 11).
//
// Warps: 0-3 and 4-7 softmax of row tile 0 and 1 (a thread owns a row), 8-11
// epilogue, 12 tensor core, 13 units and TMA loads, 14-15 the masked V tiles
// (below). TMEM: S0, S1 (P over them), O0, O1: 4 x 128 columns.
//
// Few units and many keys (a prompt of some tokens that goes on after thousands):
// the unit's keys are cut into pieces, one for each CTA, which leave (O, m, l) in 32
// bits in the workspace; the piece that is written last joins them. No CTA waits for
// another.
//
// Hidden values do not leak: a weight of exactly 0 times an infinity or NaN
// would be NaN, so in V tiles that some row of the unit sees in part, rows past
// the sequence are zeroed in shared memory, and values that are not finite are
// zeroed and their rows' sums patched in the epilogue (only for tokens that see
// them). A hidden key only makes its own column of S, which is replaced.
#include <math.h>

#include "xqa_tcgen05.cuh"
#include "xqa_launch.h"

namespace xqa {

namespace {

constexpr int kKvStages = 5;
constexpr int kUnitSlots = 3;
constexpr int kPrefillThreads = 512;
// Running maximum before any visible key: finite, so that 2^(-inf - m) is 0, and
// below the logits of the types' largest values.
constexpr float kNoRowMax = -3e38f;
constexpr float kExactMax = 4194304.f;  // 2^22: half a step of smaller m is at most 1/4
constexpr float kLazyMax = 8.0f;                 // log2 units
constexpr int kMaxPieces = kPrefillMaxPieces;
// Limit of a wait: about 1 s in units of 2^16 clocks. A role may have to wait for a whole
// unit, so a unit of many tiles raises it by as much for every 2^16 of them (0.09 s of work
// at 1.3 us a tile).
constexpr uint32_t kWaitLimit = 2000000000u >> 16;
constexpr int kUnitReaders = 15;  // 8 softmax, 4 epilogue, 1 tensor-core, 2 V warps

// One unit of work, written by the loading warp.
struct Unit {
  int end;       // 1: no more units
  int bad;       // 1: the sequence's key range is invalid: NaN rows
  int q_row;     // first token's row in q and out
  int tokens;    // tokens of the unit (1 .. 2 T)
  int head;      // kv head
  int k_row;     // first key's row in k and v
  int len_k;
  int vis0;      // keys the unit's first token sees (causal: one more per token)
  int n[2];      // KV tiles row tile 0 / 1 sees (0: no tokens, or nothing to see)
  int hidden;    // first key hidden from some token (tiles past it are masked)
  int slot;      // place of this piece's (O, m, l); -1: the unit is one piece
};

struct Shared {
  uint64_t kv_full[kKvStages], kv_empty[kKvStages];
  uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t v_clean[kKvStages];   // the stage's V tile may be used (masked tiles only)
  uint64_t s_full[2];            // S ready
  uint64_t p_full[2][2];         // the first / second 64 keys of P written
  uint64_t o_full[2], o_free[2]; // O complete / read by the epilogue
  uint64_t stat_full[2], stat_free[2];
  uint64_t drain;
  Unit unit[kUnitSlots];
  int not_finite[kUnitSlots];    // the unit's masked V tiles held infinities or NaN
  int status;
  uint32_t wait_limit;           // of every wait; 0: the CTA is aborted
  int joins;                     // this CTA's piece was the last: 1, or -1 if one failed
  uint32_t tmem;
};

constexpr int kSmemTiles = (2 + kKvStages) * kTileBytes;
constexpr int kSmemStats = 2 * kTile * 2 * 4;  // (m, l) of every row
constexpr int kPrefillSmem = kSmemTiles + kSmemStats + 1024;
static_assert(sizeof(Shared) <= 1024, "shared state");
static_assert(kPrefillSmem <= 227 * 1024, "shared memory budget");

// What every warp role works on.
struct Ctx {
  const PrefillParams& p;
  Shared& sh;
  uint8_t* tiles;  // Q0, Q1, then the KV ring
  float* stats;    // [2][128][2]
  uint32_t tmem;

  __device__ __forceinline__ uint8_t* kv(int stage) const { return tiles + (2 + stage) * kTileBytes; }

  // Warp-uniform wait within the CTA's limit; false ends the role (the CTA is aborted).
  // Short: the roles wait in many places and share an instruction cache.
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
  __device__ __forceinline__ bool aborted() const {
    return *(volatile uint32_t*)&sh.wait_limit == 0;
  }
  __device__ __forceinline__ bool get_unit(int i, Unit& u) const {
    const int slot = i % kUnitSlots;
    if (!wait(&sh.unit_full[slot], (i / kUnitSlots) & 1)) return false;
    u = sh.unit[slot];
    return !u.end;
  }
  // One arrival of this warp, after all its lanes are done.
  __device__ __forceinline__ void arrive(uint64_t* bar) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ void free_unit(int i) const { arrive(&sh.unit_empty[i % kUnitSlots]); }
};

// ---- warp 13: the units of this CTA and their TMA loads ----
template <bool kCut>
__device__ __forceinline__ void load_role(const Ctx& c, const CUtensorMap* tm_q,
                                          const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                                          int& kv_issued, int (&q_issued)[2]) {
  const PrefillParams& p = c.p;
  Shared& sh = c.sh;
  const int lane = threadIdx.x & 31;
  const int per_unit = 2 * p.tile_tokens;
  // sequences base .. base + 31, one per lane; units are numbered sequence by
  // sequence, within one from its last tokens (the longest rows) to its first,
  // the kv heads innermost
  int base = -32, total = 0;  // total: units of the chunk
  long long first = 0;        // units before it
  int q0 = 0, len_q = 0, mine = 0, incl = 0;
  int next = blockIdx.x;
  for (int i = 0;; ++i) {
    const int u = kCut ? next / p.pieces : next;
    while (base < p.batch && u >= first + total) {  // the chunk that holds unit u
      first += total;
      base += 32;
      total = 0;
      if (base >= p.batch) break;
      q0 = len_q = mine = 0;
      if (base + lane < p.batch) {
        q0 = p.cu_q[base + lane];
        const int q1 = p.cu_q[base + lane + 1];
        if (q0 >= 0 && q1 >= q0 && q1 <= p.total_q) len_q = q1 - q0;
        else record_status(&sh.status, XQA_ERR_BAD_OFFSETS);
        mine = (int)(((long long)len_q + per_unit - 1) / per_unit) * p.num_kv_heads;
      }
      incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, off);
        if (lane >= off) incl += v;
      }
      total = __shfl_sync(kAll, incl, 31);
    }
    const int slot = i % kUnitSlots;
    if (i >= kUnitSlots && !c.wait(&sh.unit_empty[slot], (i / kUnitSlots - 1) & 1)) return;
    // Offsets that ascend have max_units units at most, and in pieces one a CTA; sequences that
    // overlap may have any number (the call's time would grow with batch times rows).
    const bool over = u >= p.max_units || (kCut && i > 0);
    if (base >= p.batch || over) {  // none left
      if (base < p.batch) record_status(&sh.status, XQA_ERR_BAD_OFFSETS);
      if (lane == 0) {
        sh.unit[slot].end = 1;
        mbar_arrive(&sh.unit_full[slot]);
      }
      return;
    }
    const int at = (int)(u - first);
    const int src = __popc(__ballot_sync(kAll, incl <= at));  // lane of the sequence
    const int s_incl = __shfl_sync(kAll, incl, src), s_mine = __shfl_sync(kAll, mine, src);
    const int s_q0 = __shfl_sync(kAll, q0, src), s_len = __shfl_sync(kAll, len_q, src);
    const int local = at - (s_incl - s_mine);
    const int pairs = s_mine / p.num_kv_heads;
    const int pair = pairs - 1 - local / p.num_kv_heads;
    const int head = local - local / p.num_kv_heads * p.num_kv_heads;
    const int k0 = p.cu_k[base + src], k1 = p.cu_k[base + src + 1];
    Unit w;
    w.end = 0;
    w.bad = (k0 < 0 || k1 < k0 || k1 > p.total_k) ? 1 : 0;
    const int tok0 = pair * per_unit;
    w.q_row = s_q0 + tok0;
    w.tokens = min(per_unit, s_len - tok0);
    w.head = head;
    w.k_row = w.bad ? 0 : k0;
    w.len_k = w.bad ? 0 : k1 - k0;
    // keys seen by the first token; clamped where it is used
    w.vis0 = p.causal ? w.len_k - s_len + tok0 + 1 : w.len_k;
    w.slot = -1;
    if (kCut) {  // the piece's keys, as if they were all
      w.slot = next;
      const int piece = next - u * p.pieces;
      const int last = p.causal ? min(w.len_k, w.vis0 + w.tokens - 1) : w.len_k;
      const int tiles = last > 0 ? (last - 1) / kTile + 1 : 0;
      const int from = tiles * piece / p.pieces * kTile;
      const int to = min(w.len_k, tiles * (piece + 1) / p.pieces * kTile);
      w.k_row += from;
      w.len_k = to - from;
      w.vis0 = p.causal ? w.vis0 - from : w.len_k;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int toks = min(p.tile_tokens, w.tokens - s * p.tile_tokens);
      const int last = p.causal ? min(w.len_k, w.vis0 + s * p.tile_tokens + toks - 1) : w.len_k;
      w.n[s] = toks > 0 && last > 0 ? (last - 1) / kTile + 1 : 0;
    }
    w.hidden = max(0, min(w.vis0, w.len_k));
    if (lane == 0) {
      sh.unit[slot] = w;
      sh.not_finite[slot] = 0;
      if (const uint32_t more = max(w.n[0], w.n[1]) >> 16) {  // (an abort stays one)
        const uint32_t limit = *(volatile uint32_t*)&sh.wait_limit;
        if (limit != 0 && limit < (1 + more) * kWaitLimit)
          atomicCAS(&sh.wait_limit, limit, (1 + more) * kWaitLimit);
      }
      mbar_arrive(&sh.unit_full[slot]);
      if (w.bad) record_status(&sh.status, XQA_ERR_BAD_OFFSETS);
      next = gridDim.x + atomicAdd(p.counters, 1);
    }
    next = __shfl_sync(kAll, next, 0);
    const int n = max(w.n[0], w.n[1]);
    if (n == 0) continue;
    if (lane < 4)  // into L2 while the unit before still uses Q's place
      tma_prefetch_4d(tm_q, 64 * (lane & 1), 0, w.head, w.q_row + (lane >> 1) * p.tile_tokens);
    for (int t = 0; t < 2 * n; ++t) {  // K(n-1), V(n-1), Q, K(n-2), V(n-2), ...
      const int st = kv_issued % kKvStages, j = n - 1 - (t >> 1);
      if (kv_issued >= kKvStages && !c.wait(&sh.kv_empty[st], (kv_issued / kKvStages - 1) & 1))
        return;
      if (lane == 0) {
        const CUtensorMap* tm = (t & 1) ? tm_v : tm_k;
        mbar_arrive_expect_tx(&sh.kv_full[st], kTileBytes);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tma_load_kv(c.kv(st) + h * kHalfBytes, tm, &sh.kv_full[st], 64 * h, w.head,
                      w.k_row + j * kTile);
      }
      ++kv_issued;
      if (t != 1) continue;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (w.n[s] == 0) continue;
        if (q_issued[s] > 0 && !c.wait(&sh.q_empty[s], (q_issued[s] - 1) & 1)) return;
        if (lane == 0) {
          const int box = p.group * p.tile_tokens * 128;  // bytes of a half tile
          mbar_arrive_expect_tx(&sh.q_full[s], 2 * box);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_4d(c.tiles + s * kTileBytes + h * kHalfBytes, tm_q, &sh.q_full[s], 64 * h, 0,
                        w.head, w.q_row + s * p.tile_tokens);
        }
        ++q_issued[s];
      }
    }
  }
}

// ---- warp 12: the products ----
// The row tiles in turn: O += P V of tile j, then S of the next tile (j - 1, or the
// next unit's first), which takes the place of P. The order is fixed, so the row
// tiles settle half a period apart and one's softmax runs under the other's
// products; it runs on across units, so a new unit starts without a gap. At a unit's last
// tile it looks at the next unit only: the ones behind it may be published no earlier than
// the epilogue is done with this one, whose products are not issued yet. A unit without
// tiles there ends the run, and the search for the next with some comes after. Products are
// issued by an elected lane, whose operands stay in uniform registers: under `lane ==
// 0` each cost more to issue than to execute (1 x 16384: 1775 us against 1420). The
// code is kept short: it runs once a tile between the softmax warps' long loops and is
// fetched anew each time (products cut to the keys that a diagonal tile's rows see
// saved less than their code cost: 1 x 16384 1500 us against 1403, ragged prompts
// 205 against 190).
template <int kType>
__device__ __forceinline__ void tensor_role(const Ctx& c) {
  Shared& sh = c.sh;
  const uint32_t tiles = __shfl_sync(kAll, smem_addr(c.tiles), 0);
  const uint32_t tmem = __shfl_sync(kAll, c.tmem, 0);
  const uint64_t q_desc = desc_k_major(tiles);
  const uint64_t k_desc = desc_k_major(tiles + 2 * kTileBytes);  // stage 0 of the ring
  const uint64_t v_desc = desc_mn_major(tiles + 2 * kTileBytes);
  int i = -1;
  // tiles of the current unit (row tile s has n[s]) and of the one after it
  int n[2] = {0, 0}, hidden = 0, n2[2], hidden2 = 0;
  auto next_unit = [&]() {
    Unit w;
    if (!c.get_unit(++i, w)) return false;
    c.free_unit(i);
#pragma unroll
    for (int s = 0; s < 2; ++s) n2[s] = __shfl_sync(kAll, w.n[s], 0);  // uniform
    hidden2 = __shfl_sync(kAll, w.hidden, 0);
    return true;
  };
  bool more = true, begin = true;
  int j = 0;                // tile of the V slot
  int sv = 0, sk = 0;       // ring slots of the V and the K tile in turn
  uint32_t pv = 0, pk = 0;  // their phases
  // phases, a bit for each row tile (P: two) or stage; O is free before its first use
  uint32_t ph_q = 0, ph_p = 0, ph_o = 3, ph_clean = 0;
  for (;;) {
    // V tile j of the current unit (none in a run's first round), then a K tile: j - 1, or
    // the next unit's first
    if (begin) {  // no product is outstanding: past units without tiles
      do {
        if (!next_unit()) return;
      } while (max(n2[0], n2[1]) == 0);
    } else {
      if (!c.wait(&sh.kv_full[sv], pv)) return;
      if ((j + 1) * kTile > hidden) {  // masked: after the V warps are done with it
        if (!c.wait(&sh.v_clean[sv], ph_clean >> sv & 1)) return;
        ph_clean ^= 1u << sv;
      }
      if (j == 0) {
        more = next_unit();
        if (!more && c.aborted()) return;
      }
      sk = sv + 1 == kKvStages ? 0 : sv + 1;
      pk = sk == 0 ? pv ^ 1 : pv;
    }
    const bool cross = j == 0;  // the K tile is the next unit's
    const int nk = cross ? max(n2[0], n2[1]) : 0;
    const bool next = !cross || (more && nk > 0);  // there is one
    if (next && !c.wait(&sh.kv_full[sk], pk)) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t s_tmem = tmem + s * kTile, o_tmem = s_tmem + 256;
      if (!begin && j < n[s]) {
        const bool start = j == n[s] - 1;
        if (start) {
          if (!c.wait(&sh.o_free[s], ph_o >> s & 1)) return;
          ph_o ^= 1u << s;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // as P's halves are written
          const uint32_t bit = 2 * s + h;
          if (!c.wait(&sh.p_full[s][h], ph_p >> bit & 1)) return;
          ph_p ^= 1u << bit;
          tc_fence_after();
          const uint64_t vb = v_desc + sv * (kTileBytes >> 4) + h * (4 * 2048 >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_ts(o_tmem, s_tmem + 32 * h + 8 * k, vb + k * (2048 >> 4),
                        instr_desc<kType>(true), !start || h + k > 0);
          }
          __syncwarp();
        }
        if (cross && elect_one()) tc_commit(&sh.o_full[s]);
        __syncwarp();
      }
      // S: tile j - 1, or the next unit's first; the row tile's first waits for its Q
      if (!(cross ? next && n2[s] == nk : j - 1 < n[s])) continue;
      if (cross || j == n[s]) {
        if (!c.wait(&sh.q_full[s], ph_q >> s & 1)) return;
        ph_q ^= 1u << s;
      }
      tc_fence_after();
      const uint64_t a = q_desc + s * (kTileBytes >> 4), b = k_desc + sk * (kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = ((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4;
          tc_mma_ss(s_tmem, a + off, b + off, instr_desc<kType>(false), k > 0);
        }
        tc_commit(&sh.s_full[s]);
        if (cross ? nk == 1 : j == 1) tc_commit(&sh.q_empty[s]);
      }
      __syncwarp();
    }
    if (elect_one()) {
      if (!begin) tc_commit(&sh.kv_empty[sv]);
      if (next) tc_commit(&sh.kv_empty[sk]);
    }
    __syncwarp();
    if (!next) {
      if (!more) return;
      begin = true;
      continue;
    }
    sv = sk + 1 == kKvStages ? 0 : sk + 1;
    pv = sv == 0 ? pk ^ 1 : pk;
    if (cross) {  // on to the next unit
      n[0] = n2[0], n[1] = n2[1], hidden = hidden2;
      j = nk;
      begin = false;
    }
    --j;
  }
}

// ---- warps 14, 15: V tiles that some row of the unit sees in part ----
template <int kType>
__device__ __forceinline__ void clean_role(const Ctx& c) {
  Shared& sh = c.sh;
  const int t = threadIdx.x & 63;  // 64 threads
  const uint32_t exp_mask = kType == XQA_F16 ? 0x7c00u : 0x7f80u;
  int kv = 0;
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
    const int n = max(u.n[0], u.n[1]);
    bool found = false;
    for (int k = 0; k < 2 * n; ++k, ++kv) {  // every tile: K, V of tile n - 1, then n - 2, ...
      const int st = kv % kKvStages, j = n - 1 - (k >> 1);
      if (!c.wait(&sh.kv_full[st], (kv / kKvStages) & 1)) return;
      if ((k & 1) && (j + 1) * kTile > u.hidden) {
        const int past = min(kTile, u.len_k - j * kTile);  // first row past the sequence
        const int from = max(0, u.hidden - j * kTile);     // first row some token does not see
        uint4* rows = reinterpret_cast<uint4*>(c.kv(st));  // 8 chunks of 16 bytes a row and half
        // the largest magnitude, both halves of a word at once: one test for all
        uint32_t top = 0;
        for (int x = from * 8 + t; x < past * 8; x += 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 w = rows[h * (kHalfBytes / 16) + x];
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                         __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
          }
        }
        if ((top & 0xffffu) >= exp_mask || top >> 16 >= exp_mask) {
          found = true;
          for (int x = from * 8 + t; x < past * 8; x += 64)
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {  // the words of both halves
              uint32_t* w = reinterpret_cast<uint32_t*>(rows + (e >> 2) * (kHalfBytes / 16) + x) + (e & 3);
              uint32_t v = *w;
              if ((v & exp_mask) == exp_mask) v &= 0xffff0000u;
              if ((v & exp_mask << 16) == exp_mask << 16) v &= 0x0000ffffu;
              *w = v;
            }
        }
        for (int x = past * 8 + t; x < kTile * 8; x += 64)
#pragma unroll
          for (int h = 0; h < 2; ++h) rows[h * (kHalfBytes / 16) + x] = make_uint4(0, 0, 0, 0);
        if (found) *(volatile int*)&sh.not_finite[i % kUnitSlots] = 1;
        fence_proxy_async_smem();  // before the tensor core reads the tile
        c.arrive(&sh.v_clean[st]);
      }
      c.arrive(&sh.kv_empty[st]);
    }
    c.free_unit(i);
  }
}

// Row of this thread within its row tile.
struct RowPos {
  int token;  // within the unit
  int head;   // within the group
  bool valid;
};
__device__ __forceinline__ RowPos row_pos(const PrefillParams& p, const Unit& u, int s, int row) {
  RowPos r;
  const int t = row / p.group;
  r.head = row - t * p.group;
  r.token = s * p.tile_tokens + t;
  r.valid = t < p.tile_tokens && r.token < u.tokens;
  return r;
}
__device__ __forceinline__ int visible(const PrefillParams& p, const Unit& u, const RowPos& r) {
  if (!r.valid) return 0;
  return p.causal ? max(0, min(u.len_k, u.vis0 + r.token)) : u.len_k;
}

// ---- warps 0-7: softmax of row tile s; a thread owns a row ----
// Small loops over 32 keys that read S from TMEM again, rather than a row of registers
// and straight code: all roles share the instruction caches, and the roles that run once
// a tile or a unit fetched their code anew (16 ragged prompts 182 us with rows in
// registers and keys masked there, 168 so; 1 x 16384 1405 and 1395; a prompt of 37
// tokens 7.7 and 8.0: its time is these loops' latency).
template <int kType>
__device__ __forceinline__ void softmax_role(const Ctx& c, int s) {
  const PrefillParams& p = c.p;
  Shared& sh = c.sh;
  const int row = threadIdx.x & 127;
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  const uint32_t s_addr = lane_base + s * kTile, o_addr = lane_base + 256 + s * kTile;
  const float sc = p.scale_log2;
  int ns = 0, nstat = 0;  // S tiles, units with work so far
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
    const int vis = visible(p, u, row_pos(p, u, s, row));
    c.free_unit(i);
    const int n = s == 0 ? u.n[0] : u.n[1];
    if (n == 0) continue;
    // keys that every token of this row tile sees
    const int clear = p.causal ? min(u.len_k, u.vis0 + s * p.tile_tokens) : u.len_k;
    float m = kNoRowMax, m_raw = 0.f, l = 0.f;  // m_raw: m before the scale
    for (int j = n - 1; j >= 0; --j) {
      if (!c.wait(&sh.s_full[s], ns & 1)) return;
      tc_fence_after();
      if ((j + 1) * kTile > clear) {  // keys that a row does not see: -inf
        const int lim = vis - j * kTile;
#pragma unroll 1
        for (int q = max(0, __reduce_min_sync(kAll, lim)) >> 5; q < 4; ++q) {
          uint32_t r[32];
          tmem_ld32(s_addr + 32 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * q + k >= lim) r[k] = 0xff800000u;
          tmem_st32(s_addr + 32 * q, r);
        }
        tmem_wait_st();
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // three-operand maxima
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t r[32];
        tmem_ld32(s_addr + 32 * q, r);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(r[k + e])), __uint_as_float(r[k + 4 + e]));
      }
      const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), top = raw * sc;
      const bool moves = top > m + kLazyMax;
      // O holds something: rows whose maximum moves are rescaled (the product that last
      // wrote O was issued before the one that made this S)
      const bool scale_o = moves && m != kNoRowMax;
      const float old = m;
      if (moves) m = top, m_raw = raw;
      uint64_t m2 = f32x2(-m, -m);
      // s * sc - m is rounded once, m before: at the maximum itself up to half a step of
      // m is left, a factor of the whole row that the division by l takes out again, but
      // 2^128 and more once m is large. There the maximum is subtracted first. Each row
      // by its own: its result does not depend on its neighbours, of which those without
      // a token hold anything.
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
        uint32_t r[32], pk[16];
        tmem_ld32(s_addr + 32 * q, r);
        tmem_wait_ld();
        if (any_exact) {
#pragma unroll
          for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) - minus);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float a, b;
          split2(fma2(f32x2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), sc2, m2), a, b);
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
      ++ns;
    }
    if (nstat > 0 && !c.wait(&sh.stat_free[s], (nstat - 1) & 1)) return;
    ++nstat;
    float2* st = reinterpret_cast<float2*>(c.stats) + s * kTile + row;
    *st = make_float2(m, l);
    c.arrive(&sh.stat_full[s]);
  }
}

// ---- warps 8-11: normalise and write ----
// A thread has a row of O. Before a store, four lanes trade their 16-byte units, so that
// the four write 64 contiguous bytes of one row: a store of 32 rows' units kept the next
// unit's first product waiting for O (prompts on prefixes 161 us, 157 so; 1 x 16384 1409
// and 1395). More dims at a time free O earlier, but their code costs more than it saves
// (ragged prompts 182 to 191 us).
template <int kType, bool kCut>
__device__ __forceinline__ void epilogue_role(const Ctx& c) {
  const PrefillParams& p = c.p;
  Shared& sh = c.sh;
  const int row = threadIdx.x & 127;
  const uint32_t lane_base = c.tmem + ((uint32_t)(row & ~31) << 16);
  const uint32_t exp_mask = kType == XQA_F16 ? 0x7c00u : 0x7f80u;
  uint32_t ph = 0;  // a bit for each row tile
  for (int i = 0;; ++i) {
    Unit u;
    if (!c.get_unit(i, u)) return;
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      const RowPos rp = row_pos(p, u, s, row);
      const int n_s = s ? u.n[1] : u.n[0];
      const long long at = (long long)u.q_row + rp.token;
      const int h = u.head * p.group + rp.head;
      uint16_t* out = p.out + at * p.out_row_stride + h * p.out_head_stride;
      if (kCut && n_s == 0) {
        p.piece_ml[(u.slot * 2 + s) * kTile + row] = make_float2(kNoRowMax, 0.f);
        continue;
      }
      if (n_s == 0) {  // no tokens, or tokens that see nothing
        if (rp.valid) {
          const uint32_t f = !u.bad ? 0u : kType == XQA_F16 ? 0x7fff7fffu : 0x7fc07fc0u;
#pragma unroll 1
          for (int k = 0; k < kHeadDim / 8; ++k)
            reinterpret_cast<uint4*>(out)[k] = make_uint4(f, f, f, f);
          if (p.lse) p.lse[at * p.num_q_heads + h] = u.bad ? __int_as_float(0x7fc00000) : -INFINITY;
        }
        continue;
      }
      if (!c.wait(&sh.stat_full[s], ph >> s & 1)) return;
      const float2 ml = reinterpret_cast<const float2*>(c.stats)[s * kTile + row];
      c.arrive(&sh.stat_free[s]);
      if (!c.wait(&sh.o_full[s], ph >> s & 1)) return;
      ph ^= 1u << s;
      tc_fence_after();
      // infinities and NaN of masked V tiles (zeroed there), for rows that see them
      const bool patch = *(volatile int*)&sh.not_finite[i % kUnitSlots] != 0;
      const int vis = visible(p, u, rp);
      const float rl = ml.y == 0.f ? 0.f : 1.f / ml.y;  // a row without a weight: 0
      uint16_t* dst[4];  // this lane's unit of the four lanes' rows
      if (!kCut) {
        const unsigned long long mine = rp.valid ? reinterpret_cast<unsigned long long>(out) : 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned long long a = __shfl_sync(kAll, mine, (threadIdx.x & 28) + k);
          dst[k] = a ? reinterpret_cast<uint16_t*>(a) + 8 * (threadIdx.x & 3) : nullptr;
        }
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        __syncwarp();  // rows part ways below
        tmem_ld32(lane_base + 256 + s * kTile + 32 * q, o);
        tmem_wait_ld();
        if (q == 3) {  // O is read
          tc_fence_before();
          c.arrive(&sh.o_free[s]);
        }
        if (patch) {
#pragma unroll 1
          for (int key = u.hidden; key < vis; ++key) {
            const uint16_t* v = p.v + ((long long)u.k_row + key) * p.v_row_stride +
                                u.head * p.v_head_stride + 32 * q;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t bits = v[k];
              if ((bits & exp_mask) == exp_mask)
                o[k] = __float_as_uint(
                    __uint_as_float(o[k]) +
                    (kType == XQA_F16 ? __half2float(__ushort_as_half((unsigned short)bits))
                                      : __uint_as_float(bits << 16)));
            }
          }
        }
        if (kCut) {  // as it is: [32 chunks of 4 dims][128 rows]
          float4* po = p.piece_o + ((size_t)(u.slot * 2 + s) * 32 + 8 * q) * kTile + row;
          if (rp.valid) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              po[k * kTile] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                          __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
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
      if (kCut) p.piece_ml[(u.slot * 2 + s) * kTile + row] = ml;
      else if (p.lse && rp.valid)
        p.lse[at * p.num_q_heads + h] =
            ml.y == 0.f ? -INFINITY : (ml.x + __log2f(ml.y)) * 0.6931471805599453f;
    }
    c.free_unit(i);
  }
}

// ---- warps 0-7, after the roles: the unit's pieces joined by the last of them. A CTA
// has at most one piece (its unit 0).
template <int kType>
__device__ __forceinline__ void join_pieces(const Ctx& c) {
  const PrefillParams& p = c.p;
  Shared& sh = c.sh;
  // every (O, m, l) of this CTA's piece is written (the epilogue warps arrive)
  asm volatile("bar.sync 1, 384;" ::: "memory");
  const Unit u = sh.unit[0];
  if (u.end) return;  // no piece
  const int unit = u.slot / p.pieces;
  if (threadIdx.x == 0) {
    const bool failed = c.aborted();
    __threadfence();
    const int old = atom_add_acq_rel_gpu(p.tickets + unit, failed ? 1 + kTicketPoison : 1);
    const bool last = (old & kTicketCountMask) == p.pieces - 1;
    sh.joins = !last ? 0 : failed || (old & kTicketPoisonMask) ? -1 : 1;
    if (last) p.tickets[unit] = 0;  // for the next call
  }
  asm volatile("bar.sync 2, 256;" ::: "memory");
  const int joins = sh.joins;
  if (joins == 0) return;
  const size_t first = (size_t)unit * p.pieces * 2;  // its piece k, row tile s: first + 2 k + s
  const bool bad = joins < 0 || u.bad;
  const int rows = u.tokens * p.group;  // <= 256
  // threads of a row: 256 / (rows rounded up to 32, 64, 128 or 256), its dims shared
  // out among them
  const int span = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
  const int r = threadIdx.x & (span - 1), chunks = span / 8;  // chunks of 4 dims for each
  const int c0 = threadIdx.x / span * chunks;
  if (r >= rows) return;
  const int t = r / p.group, g = r - t * p.group, h = u.head * p.group + g;
  const int s = t >= p.tile_tokens ? 1 : 0, row = r - s * p.tile_tokens * p.group;
  const long long at = (long long)u.q_row + t;
  float w[kMaxPieces], top = -INFINITY, sum = 0.f;
  float2 ml[kMaxPieces];
#pragma unroll
  for (int k = 0; k < kMaxPieces; ++k)
    ml[k] = k < p.pieces ? __ldcg(p.piece_ml + (first + 2 * k + s) * kTile + row)
                         : make_float2(kNoRowMax, 0.f);
#pragma unroll
  for (int k = 0; k < kMaxPieces; ++k)
    if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
  // A piece with keys keeps the least weight there is: the infinities and NaN in its O and l
  // (keys of NaN alone leave its maximum at kNoRowMax) are the row's, however small it is.
#pragma unroll
  for (int k = 0; k < kMaxPieces; ++k) {
    w[k] = ml[k].y != 0.f ? fmaxf(ex2(ml[k].x - top), 0x1p-149f) : 0.f;
    if (w[k] != 0.f) sum += w[k] * ml[k].y;
  }
  const float nan = __int_as_float(0x7fc00000);
  const float rl = bad ? nan : sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = p.out + at * p.out_row_stride + h * p.out_head_stride + 4 * c0;
  const float4* po = p.piece_o + ((first + s) * 32 + c0) * kTile + row;
#pragma unroll 1
  for (int q = 0; q < chunks; q += 4) {  // 16 dims, every piece's in flight at once
    float4 v[kMaxPieces][4];
#pragma unroll
    for (int k = 0; k < kMaxPieces; ++k)
      if (w[k] != 0.f)  // (a piece without keys has written none)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = __ldcg(po + ((size_t)k * 64 + q + e) * kTile);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxPieces; ++k)
        if (w[k] != 0.f) {
          a.x += w[k] * v[k][e].x;
          a.y += w[k] * v[k][e].y;
          a.z += w[k] * v[k][e].z;
          a.w += w[k] * v[k][e].w;
        }
      reinterpret_cast<uint2*>(out)[q + e] =
          make_uint2(pack2<kType>(a.x * rl, a.y * rl), pack2<kType>(a.z * rl, a.w * rl));
    }
  }
  if (p.lse && c0 == 0)
    p.lse[at * p.num_q_heads + h] =
        bad ? nan : sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
}

// kCut: units are cut into pieces (p.pieces > 1).
template <int kType, bool kCut>
__global__ void __launch_bounds__(kPrefillThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  float* stats = reinterpret_cast<float*>(smem + kSmemTiles);
  Shared& sh = *reinterpret_cast<Shared*>(smem + kSmemTiles + kSmemStats);
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0);  // known to be warp-uniform
  const bool aligned = (smem_addr(smem) & 1023u) == 0;  // as the swizzle needs
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKvStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 3);  // the tensor-core warp and the V warps
      mbar_init(&sh.v_clean[i], 2);
    }
    for (int i = 0; i < kUnitSlots; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_empty[i], kUnitReaders);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s][0], 4);
      mbar_init(&sh.p_full[s][1], 4);
      mbar_init(&sh.o_full[s], 1);
      mbar_init(&sh.o_free[s], 4);
      mbar_init(&sh.stat_full[s], 4);
      mbar_init(&sh.stat_free[s], 4);
    }
    mbar_init(&sh.drain, 1);
    sh.unit[0].end = 1;  // until there is one
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
  int kv_issued = 0, q_issued[2] = {0, 0};
  if (aligned) {
    const Ctx c{p, sh, smem, stats, sh.tmem};
    __syncwarp();
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      if (warp == 12) tensor_role<kType>(c);
      else if (warp == 13) load_role<kCut>(c, &tm_q, &tm_k, &tm_v, kv_issued, q_issued);
      else clean_role<kType>(c);
    } else if (warp >= 8) {
      if (kCut) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
      epilogue_role<kType, kCut>(c);
      if (kCut) {
        __syncwarp();
        asm volatile("bar.arrive 1, 384;" ::: "memory");
      }
    } else {
      // the join of pieces holds 8 x 16 dims; the sums of the shares, 256 x 192 + 128 x 80
      // and 256 x 144 + 128 x 128, with 128 x 48, stay within the 65,536 of the launch
      if (kCut) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
      else asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
      softmax_role<kType>(c, warp >> 2);
      __syncwarp();
      if (kCut) join_pieces<kType>(c);
    }
  }
  __syncwarp();
  // Products and their arrivals, and after an abort copies, may be in flight:
  // they end before the CTA's shared memory and TMEM are given up.
  if (aligned && (warp == 12 || warp == 13)) {
    int never = 0;
    bool ok = true;
    if (warp == 12) {
      if (elect_one()) tc_commit(&sh.drain);
      __syncwarp();
      ok = mbar_wait_bounded(&sh.drain, 0, &never);
    } else if (*(volatile uint32_t*)&sh.wait_limit == 0) {
      for (int k = max(0, kv_issued - kKvStages); k < kv_issued; ++k)
        ok = mbar_wait_bounded(&sh.kv_full[k % kKvStages], (k / kKvStages) & 1, &never) && ok;
      for (int s = 0; s < 2; ++s)
        if (q_issued[s] > 0)
          ok = mbar_wait_bounded(&sh.q_full[s], (q_issued[s] - 1) & 1, &never) && ok;
    }
    if (!ok) atomicExch(&sh.status, XQA_ERR_DRAIN_TIMEOUT);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(sh.tmem, 512);
  if (threadIdx.x == 0) {
    if (sh.wait_limit == 0) record_status(&sh.status, XQA_ERR_DEVICE_TIMEOUT);
    p.status[blockIdx.x] = sh.status;
    if (blockIdx.x == 0) p.header[0] = gridDim.x;
    // the last CTA leaves the counters at zero for the next call
    __threadfence();
    if (atomicAdd(p.counters + 1, 1) == (int)gridDim.x - 1) {
      p.counters[0] = 0;
      p.counters[1] = 0;
    }
  }
}

}  // namespace

cudaError_t launch_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                           const CUtensorMap& tm_v, const PrefillParams& p, int dtype, int ctas,
                           cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPrefillThreads);
  cfg.dynamicSmemBytes = kPrefillSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool cut = p.pieces > 1;
  if (dtype == XQA_F16)
    return cut ? cudaLaunchKernelEx(&cfg, prefill_kernel<XQA_F16, true>, tm_q, tm_k, tm_v, p)
               : cudaLaunchKernelEx(&cfg, prefill_kernel<XQA_F16, false>, tm_q, tm_k, tm_v, p);
  return cut ? cudaLaunchKernelEx(&cfg, prefill_kernel<XQA_BF16, true>, tm_q, tm_k, tm_v, p)
             : cudaLaunchKernelEx(&cfg, prefill_kernel<XQA_BF16, false>, tm_q, tm_k, tm_v, p);
}

cudaError_t set_prefill_attributes() {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(prefill_kernel<XQA_F16, false>, a, kPrefillSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(prefill_kernel<XQA_F16, true>, a, kPrefillSmem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(prefill_kernel<XQA_BF16, false>, a, kPrefillSmem)) != cudaSuccess) return e;
  return cudaFuncSetAttribute(prefill_kernel<XQA_BF16, true>, a, kPrefillSmem);
}

}  // namespace xqa
