// chunk_work.cuh -- what the kernels for new tokens over the paged cache share: which keys a row sees,
// the plan that cuts the call's (row tile, key tile) units into ranges, a range's way through its row
// tiles, and the arithmetic of queries and weights.
//
// A geometry G says how a kernel goes about it: G::ROWS rows of a row tile, at most G::RANGES ranges,
// G::SWITCH key tiles counted for the start of a row tile, a range per row tile or more while that
// gives each G::MIN_TILES key tiles on average.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "kv8_common.cuh"
#include "share_split.h"
#include "tc_ptx.cuh"

namespace kv8 {
namespace {

using namespace ptx;

// what a call's rows see: all keys before them; with a window; a prefix shared by several sequences apart
constexpr int kPlain = 0, kWindow = 1, kShared = 2;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// ------------------------------------------------------------------ work
// The geometry of chunk.cu: a cluster of four CTAs is a range's.
struct WideGeo {
  static constexpr int ROWS = 256, RANGES = NUM_SMS / 4;
  // A cluster per row tile, or more while that gives each MIN_TILES key tiles on average.  (The ranges
  // differ by up to SWITCH, below, which is counted in front of every row tile, the first of a range
  // among them: 4 tiles fall into ranges of 0 and 4, 16 into 0, 0, 2, 3, 2, 3, 3, 3.)  Device times for
  // 1, 2 and 4, us: one token of 128 heads over 512 keys 30.8, 28.7, 26.7, over 2048 35.4, 32.8, 36.8,
  // over 8192 47.2, 47.0, 41.0; two row tiles of 8 key tiles 32.8, 34.9, 38.7.
  static constexpr int MIN_TILES = 2;
  // What beginning a row tile costs, in key tiles: 19 thousand cycles (the query is loaded and split
  // while the context pair writes its results, and the pipeline fills) against 3.1 thousand a tile.  A
  // prompt of 4096 tokens at 128 heads: 2.40 ms when ranges count 4 for it, 2.17 for 5, 2.04 for 6, 2.06
  // for 7, 2.09 for 8; five sequences without a mask 103, 102, 98, 99, 100 us.
  static constexpr int SWITCH = 6;
};

__device__ __forceinline__ void store_release(unsigned* p, unsigned v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Plan of range k: its first row tile (sequence b, row tile rt, nt key tiles of
// which off come before the range), the unit where the range starts and its units.
struct PlanEntry {
  int32_t b, rt, nt, off;
  int64_t x;
};
template <class G>
struct Plan {
  int64_t n, units, tiles;   // ranges, their units, row tiles
  int64_t part_rows;         // (shared prefixes, all rows by chunk.cu) rows that have parts
  unsigned ready;            // (and in the prefixes' plan) whether the plans are made
  PlanEntry e[G::RANGES];
};

template <int MODE>
struct SeqInfo {
  int64_t q0;  // first row of the query arrays
  int nq, T;
};
template <>
struct SeqInfo<kShared> {
  int64_t q0;
  int nq, T;               // (T counts from the first key, token 64 page0)
  int row, page0, causal;  // row of the block table, first page there
  int part;                // row of its first part (below), or -1
};
template <int MODE>
__device__ __forceinline__ SeqInfo<MODE> seq_info(const ChunkArgs& a, int b, bool tell) {
  if constexpr (MODE == kShared) {
    const int4 u = a.entries[b].u, v = a.entries[b].v;
    return {u.x, u.y, u.z, u.w, v.x, v.y, v.z};
  } else {
    SeqInfo<MODE> s;
    const int64_t q0 = __ldg(&a.q_start[b]), q1 = __ldg(&a.q_start[b + 1]);
    const int64_t T = __ldg(&a.seq_lens[b]), room = (int64_t)a.max_blocks * PAGE;
    const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q;
    if (tell && bad) atomicOr(a.err, ERR_BLOCK_TABLE);
    if (tell && (T < 0 || T > room)) atomicOr(a.err, ERR_SEQ_LEN);
    s.q0 = q0;
    s.nq = bad ? 0 : (int)(q1 - q0);
    s.T = (int)(T < 0 ? 0 : (T > room ? room : T));
    return s;
  }
}
template <class G, int MODE>
__device__ __forceinline__ int row_tiles(const ChunkArgs& a, const SeqInfo<MODE>& s) {
  return (int)(((int64_t)s.nq * a.H + G::ROWS - 1) / G::ROWS);
}
// keys that token i of the sequence sees (with a window: before which its last one ends)
template <int MODE>
__device__ __forceinline__ int limit_of(const ChunkArgs& a, const SeqInfo<MODE>& s, int i) {
  if constexpr (MODE == kPlain) {
    if (!a.causal) return s.T;
  }
  if constexpr (MODE == kShared) {
    if (!s.causal) return s.T;
  }
  const int lim = s.T - s.nq + i + 1;
  return lim < 0 ? 0 : lim;
}
template <class G>
__device__ __forceinline__ int first_token(const ChunkArgs& a, int rt) {
  return (int)((uint32_t)rt * G::ROWS / (uint32_t)a.H);
}
template <class G, int MODE>
__device__ __forceinline__ int last_token(const ChunkArgs& a, const SeqInfo<MODE>& s, int rt) {
  // (Rows have 31 bits.  A division of 32 makes a prompt with a window 3 % faster, and single tokens of 128 heads
  // over 8192 keys 9 % slower, as the kernels are compiled.)
  const int64_t last = MODE == kWindow && G::ROWS == WideGeo::ROWS ? ((uint32_t)rt * G::ROWS + G::ROWS - 1) / (uint32_t)a.H
                                                                   : ((int64_t)rt * G::ROWS + G::ROWS - 1) / a.H;
  return last < s.nq ? (int)last : s.nq - 1;
}
// A window's first key, of a row that sees keys up to lim.
__device__ __forceinline__ int window_from(const ChunkArgs& a, int lim) { return lim > a.window ? lim - a.window : 0; }

// The pages that a row tile reads, in order: all of them from the first; or with a window, the
// first tokens' pages, then those from the first row's window on (its window begins first).
template <int MODE>
struct Pages {
  __device__ __forceinline__ int at(int i) const { return i; }
};
template <>
struct Pages<kWindow> {
  int sinks, skip;  // pages of first tokens; pages between them and the window
  __device__ __forceinline__ int at(int i) const { return i < sinks ? i : i + skip; }
};
// Key tiles of a row tile: those that its last row sees; one where it sees none, so
// that its (empty) rows are written by the same path.
template <class G, int MODE>
__device__ __forceinline__ int key_tiles(const ChunkArgs& a, const SeqInfo<MODE>& s, int rt, Pages<MODE>* pages) {
  const int lim = limit_of(a, s, last_token<G>(a, s, rt));
  if constexpr (MODE == kWindow) {
    const int from = window_from(a, limit_of(a, s, first_token<G>(a, rt))), wp = from / PAGE;
    pages->sinks = ((a.n_sink < from ? a.n_sink : from) + PAGE - 1) / PAGE;
    pages->skip = wp > pages->sinks ? wp - pages->sinks : 0;
    const int n = (lim > 0 ? (lim - 1) / PAGE + 1 : 0) - pages->skip;
    return n > 0 ? (n + 1) / 2 : 1;
  }
  return lim > 0 ? (lim - 1) / TILE + 1 : 1;
}

// What a plan reads first, asked for before anything else it does.
__device__ __forceinline__ void plan_prefetch(const ChunkArgs& a) {
  for (int g = threadIdx.x; g < a.G && g < (int)blockDim.x; g += blockDim.x) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.group_start + g) : "memory");
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.shared_len + g) : "memory");
  }
  for (int b = threadIdx.x; b < a.B && b < 2 * (int)blockDim.x; b += blockDim.x) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q_start + b) : "memory");
    asm volatile("prefetch.global.L1 [%0];" ::"l"(a.seq_lens + b) : "memory");
  }
}

// A plan is one CTA's of PLAN_THREADS threads, whose sums follow one another with a barrier each.
constexpr int PLAN_THREADS = 512, PLAN_WARPS = PLAN_THREADS / 32;
struct PlanScratch {
  int64_t sums[2][PLAN_WARPS];   // of the warps, in turn
  // row tiles, if they are as few: where they begin, their sequence and their place there
  int64_t tile[PLAN_THREADS];
  int2 of[PLAN_THREADS];
};
struct PlanSum {
  PlanScratch& at;
  int turn = 0;
  // inclusive sum over the CTA's threads (of which those from `count` on have nothing to add), and the total
  __device__ __forceinline__ int64_t operator()(int64_t v, int64_t count, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    int64_t* sums = at.sums[turn];
    turn ^= 1;  // (its next use lies behind the next sum's barrier)
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t before = 0, all = 0;
    const int warps = count < PLAN_THREADS ? (int)(count + 31) >> 5 : PLAN_WARPS;
    for (int w = 0; w < warps; ++w) {
      const int64_t u = sums[w];
      before += w < warp ? u : 0;
      all += u;
    }
    *total = all;
    return v + before;
  }
};

// Sequences that share a prefix.  The rows of a group's sequences lie behind one another, so that the
// prefix is one more sequence, whose rows are the group's and which all of them see whole, and the
// others keep the keys behind it; entry g is group g's prefix, entry G + b sequence b.  Either gives
// parts (f32 o, l and M_g of every row), which the join adds up; a sequence that shares nothing
// is as in a call without groups.
//
// The prefix is whole pages that every row of the group sees; a group may take part where its row tiles
// are fewer together than apart by more than the parts cost: SHARE key tiles a row tile (6 for its start, and
// 256 rows of f32 written twice and read twice), and where its sequences have PART_ROWS rows on average
// at most (above, they fill their row tiles, and little is saved).  G is the geometry of what the
// sequences would be computed with otherwise.
constexpr int PART_ROWS = 1024, SHARE = 16;
// Whether the groups that may do, by what the call costs with and without them:
// - in row tiles of 256, WORTH units have to be saved in all (two tokens of 128 heads over 16384 keys save 122
//   and are 11 us slower; four save 244: 55 against 57; 32 over 4000 keys 400: 74 against 87);
// - else in cycles: a unit is NARROW of an SM's, or WIDE of a cluster's; what a call takes besides is START,
//   or START_WIDE and what the join takes longer, JOIN_MORE.  (us, shared and not, by the same call: 64 tokens of 16
//   heads over a prefix of 2000 keys 37 and 35, of 4000 41 and 45, of 8000 48 and 67; 8 over 16384 39 and 31;
//   32 x up to 4 tokens over 3000 keys 41 and 39, over 8000 50 and 62; 32 tokens of 64 heads over 4000 51 and
//   53.  A call without groups saves the plan's weighing and a launch: 30, 40, 62; 26; 33, 56; 46.)
constexpr int WORTH = 300, WIDE_CYCLES = 3100;
template <class G>
constexpr int NARROW = G::ROWS == 16 ? 3200 : 4300;

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int64_t warp_min(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const int64_t u = __shfl_xor_sync(0xffffffffu, v, o);
    v = u < v ? u : v;
  }
  return v;
}

// Whether sequence b's query range ends before it begins.  Ranges of which none does are apart: their row tiles are
// as many as the workspace has room for, at most.
__device__ __forceinline__ bool range_turns(const ChunkArgs& a, int b) {
  return __ldg(&a.q_start[b + 1]) < __ldg(&a.q_start[b]);
}

// Whether the groups' ranges break their order (by a plan's CTA); that and lengths below 0 are told.  And whether the
// queries' do, if asked: `turns`, a thread's own findings and then all of them.
__device__ __forceinline__ bool groups_bad(const ChunkArgs& a, bool tell, bool* turns = nullptr) {
  int bad = 0;
  for (int g = threadIdx.x; g < a.G; g += PLAN_THREADS) {
    const int f = __ldg(&a.group_start[g]), l = __ldg(&a.group_start[g + 1]);
    bad |= f < 0 || l < f || l > a.B;
    if (tell && __ldg(&a.shared_len[g]) < 0) atomicOr(a.err, ERR_SEQ_LEN);
  }
  const bool any = __syncthreads_or(bad || (turns != nullptr && *turns));
  if (turns != nullptr && any) *turns = __syncthreads_or(*turns);
  if (tell && any && threadIdx.x == 0) atomicOr(a.err, ERR_BLOCK_TABLE);
  return any;
}

// (By a plan's CTA.)  The result: the clusters that the prefixes get beside a kernel for few rows,
// `most` at most of the `clusters` there are.  `part_rows`, for a join that asks for it: the rows that have parts.  `turns`: whether query ranges do, and may overlap; nothing is shared then.
template <class G>
__device__ __forceinline__ int make_entries(const ChunkArgs& a, int64_t* part_rows, PlanSum& plan_sum, bool tell, bool* turns,
                                            int most = 0, int clusters = 0) {
  constexpr bool FEW = G::ROWS < WideGeo::ROWS;
  __shared__ unsigned long long sums[2];  // units that the groups save, and those of their prefixes
  if (threadIdx.x < 2) sums[threadIdx.x] = 0ull;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = threadIdx.x; g < a.G; g += PLAN_THREADS) {
    a.entries[g].u = make_int4(0, 0, 0, 0);
    a.entries[g].v = make_int4(0, 0, -1, 0);
  }
  int64_t mine = 0, all = 0;  // (few) the axis's length with nothing shared
  *turns = false;
  for (int b = threadIdx.x; b < a.B; b += PLAN_THREADS) {
    const SeqInfo<kPlain> s = seq_info<kPlain>(a, b, tell);
    a.entries[a.G + b].u = make_int4((int)s.q0, s.nq, s.T, b);
    a.entries[a.G + b].v = make_int4(0, a.causal, -1, 0);
    *turns |= range_turns(a, b);
    if constexpr (FEW) mine += ((int64_t)s.nq * a.H + G::ROWS - 1) / G::ROWS * (((int64_t)s.T + TILE - 1) / TILE + G::SWITCH);
  }
  if (part_rows != nullptr && threadIdx.x == 0) *part_rows = 0;
  if (groups_bad(a, tell, turns) || a.G == 0) return 0;  // (ranges that may overlap: nothing is shared)
  // what each group would share, a warp per group
  for (int g = warp; g < a.G; g += PLAN_WARPS) {
    const int f = __ldg(&a.group_start[g]), l = __ldg(&a.group_start[g + 1]);
    int64_t P = __ldg(&a.shared_len[g]), apart = 0, tokens = 0, members = 0, q0 = INT32_MAX, row = INT32_MAX;
    for (int b = f + lane; b < l; b += 32) {
      const int4 u = a.entries[a.G + b].u;
      // (a range that breaks the order has no query; nothing is shared then)
      if (__ldg(&a.q_start[b + 1]) - __ldg(&a.q_start[b]) != u.y) P = 0;
      if (u.y == 0) continue;
      const int64_t see = a.causal ? (int64_t)u.z - u.y + 1 : u.z;
      P = see < P ? see : P;
      apart += ((int64_t)u.y * a.H + G::ROWS - 1) / G::ROWS;
      tokens += u.y;
      ++members;
      if (row == INT32_MAX) row = b;  // (a sequence without queries need not hold the prefix)
      q0 = u.x < q0 ? u.x : q0;
    }
    P = warp_min(P);
    q0 = warp_min(q0);
    row = warp_min(row);
    apart = warp_sum(apart);
    tokens = warp_sum(tokens);
    members = warp_sum(members);
    P = P > 0 ? P / PAGE : 0;
    const int64_t rows = tokens * a.H, together = (rows + WideGeo::ROWS - 1) / WideGeo::ROWS, tiles = (P + 1) / 2;
    const bool take = members > 1 && P > 0 &&
                      (a.share == KV8_SHARE_ALWAYS ||
                       (rows <= PART_ROWS * members &&
                        together * (tiles + SHARE) * 4 * WIDE_CYCLES < apart * tiles * (FEW ? NARROW<G> : 4 * WIDE_CYCLES)));
    if (take && lane == 0) {
      atomicAdd(&sums[0], (unsigned long long)(apart * tiles));
      atomicAdd(&sums[1], (unsigned long long)(together * (tiles + WideGeo::SWITCH)));
      a.entries[g].u = make_int4((int)q0, (int)tokens, (int)P * PAGE, (int)row);
      a.entries[g].v = make_int4(0, 0, 0, 0);
    }
  }
  if constexpr (FEW) (void)plan_sum(mine, a.B, &all);  // (a barrier)
  else __syncthreads();
  int split = 0;
  {
    const int64_t saved = (int64_t)sums[0], wide = (int64_t)sums[1];
    if (saved == 0) return 0;
    const bool always = a.share == KV8_SHARE_ALWAYS;
    bool take = always || saved - wide > WORTH;
    if constexpr (FEW) {
      int64_t least = INT64_MAX;
      for (int t = 1 + lane; t <= most && t < clusters; t += 32) {
        const int64_t z = split_cost((float)(wide * WIDE_CYCLES), (float)((all - saved) * NARROW<G>), t, NUM_SMS);
        least = z < least ? z : least;
      }
      split = split_taken(warp_min(least), all * NARROW<G> / NUM_SMS + START, always);
      take = split > 0;
    }
    if (!take) {
      for (int g = threadIdx.x; g < a.G; g += PLAN_THREADS) a.entries[g].u.y = 0;
      __syncthreads();
      return 0;
    }
  }
  // the rows of their parts, as far as there is room
  int64_t at = 0;
  for (int g0 = 0; g0 < a.G; g0 += PLAN_THREADS) {
    const int g = g0 + threadIdx.x;
    const int64_t rows = g < a.G ? (int64_t)a.entries[g].u.y * a.H : 0;
    int64_t sum;
    const int64_t from = at + plan_sum(rows, a.G - g0, &sum) - rows;
    if (rows > 0) {
      // (the groups that have room are the first ones: those behind one without begin further on)
      if (from + rows <= a.part_rows) {
        a.entries[g].v.z = (int)from;
        if (part_rows != nullptr)
          atomicMax(reinterpret_cast<unsigned long long*>(part_rows), (unsigned long long)(from + rows));
      } else {
        a.entries[g].u.y = 0;
      }
    }
    at += sum;
  }
  __syncthreads();
  for (int g = warp; g < a.G; g += PLAN_WARPS) {
    const int4 u = a.entries[g].u;
    if (u.y == 0) continue;
    const int f = __ldg(&a.group_start[g]), l = __ldg(&a.group_start[g + 1]), from = a.entries[g].v.z;
    for (int b = f + lane; b < l; b += 32) {
      int4 m = a.entries[a.G + b].u;
      if (m.y == 0) continue;
      const int token = m.x - u.x;
      m.z -= u.z;
      a.entries[a.G + b].u = m;
      a.entries[a.G + b].v = make_int4(u.z / PAGE, a.causal, (int)a.part_rows + from + token * a.H, g);
      if (a.part_seq != nullptr)
        for (int i = 0; i < m.y; ++i) a.part_seq[from / a.H + token + i] = make_int2(g, b);
    }
  }
  __syncthreads();
  return split;
}

// owner[p] of row tile p: its sequence, its place there, the slot of its first part -- slot 2 k is the first
// segment of range k, 2 k + 1 its last -- and the last range that it lies in.
//
// One CTA of PLAN_THREADS threads: row tiles before each of n_seq sequences (base, and
// base_out for who reads the plan), the units of every row tile, their
// total, and the row tile that each range starts in; with `unit`, the units before each row tile, and
// with `owner`, whose it is.  (The sequences are the call's, or entries, from `first` on, and `shift` further on
// for who reads the plan.)  `alone`: a range for every row tile (of which there are `most` at most).
// Query ranges that turn back (and are told) may overlap, and have any number of row tiles.  All of them are computed, but
// none is cut then (`whole`, which a shared call's entries are asked with): a range begins where a row tile does, and
// no row tile has parts, nor an entry in unit or owner, which have room for those of ranges that are apart.
template <int MODE, class G>
__device__ __forceinline__ void make_plan(const ChunkArgs& a, Plan<G>* plan, int64_t* base, int64_t* base_out, int first, int shift,
                                          int n_seq, int most, PlanSum& plan_sum, int64_t* unit, int4* owner,
                                          bool alone = false, bool whole = false) {
  static_assert(G::RANGES <= PLAN_THREADS, "a thread per range");
  PlanScratch& sh = plan_sum.at;
  constexpr int64_t TURN = 1ll << 44;  // (above the row tiles of PLAN_THREADS sequences)
  int64_t pairs = 0;
  for (int b0 = 0; b0 < n_seq; b0 += PLAN_THREADS) {
    const int b = b0 + threadIdx.x;
    int64_t n = b < n_seq ? row_tiles<G>(a, seq_info<MODE>(a, first + b, true)) : 0;
    if (MODE != kShared && b < n_seq && range_turns(a, first + b)) n |= TURN;
    int64_t sum;
    int64_t inc = plan_sum(n, n_seq - b0, &sum);
    if constexpr (MODE != kShared) {
      whole |= sum >= TURN;
      n &= TURN - 1;
      inc &= TURN - 1;
      sum &= TURN - 1;
    }
    if (b < n_seq) {
      base[b] = pairs + inc - n;
      if (base_out != nullptr) base_out[b] = pairs + inc - n;
    }
    pairs += sum;
  }
  if (owner == nullptr && unit == nullptr && !alone) whole = false;  // (nothing that they could exceed)
  if (threadIdx.x == 0) base[n_seq] = pairs;
  __syncthreads();
  // row tile p's sequence (of these) and its place there
  auto find = [&](int64_t p, int* rt) -> int {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (base[mid] <= p) lo = mid; else hi = mid;
    }
    *rt = (int)(p - base[lo]);
    return first + lo;
  };
  int b = 0, rt = 0;
  auto tiles = [&](int64_t p) -> int64_t {
    if (p >= pairs) return 0;
    b = find(p, &rt);
    Pages<MODE> pages;
    return key_tiles<G>(a, seq_info<MODE>(a, b, false), rt, &pages);
  };
  // The ranges are equal on an axis where a row tile is G::SWITCH + nt long, and the border falls on a
  // key tile of it; x counts units (key tiles).
  const bool few = pairs <= PLAN_THREADS;
  int64_t mine = 0, units;
  for (int64_t p = threadIdx.x; p < pairs; p += PLAN_THREADS) mine += tiles(p);
  const int64_t upto = plan_sum(mine, pairs, &units);
  const int64_t total = units + pairs * G::SWITCH;
  int64_t nc = units / G::MIN_TILES > pairs ? units / G::MIN_TILES : pairs;
  nc = nc > most ? most : (nc < 1 ? (units > 0 ? 1 : 0) : nc);
  if (whole) alone = false;
  if (alone) nc = pairs;
  if (threadIdx.x == 0) {
    plan->n = nc;
    plan->units = units;
    plan->tiles = whole ? 0 : pairs;
    if (unit != nullptr && !whole) unit[pairs] = units;
  }
  // Range k begins at k total / nc, so that as many as at nc / total, rounded up, begin before `at`.  (Its products
  // have 32 bits as a rule, and a division of 64 takes five times as long.)
  const bool narrow = total < INT32_MAX / NUM_SMS;
  auto divide = [&](int64_t x, int64_t by) -> int64_t { return narrow ? (int64_t)((uint32_t)x / (uint32_t)by) : x / by; };
  auto ranges_before = [&](int64_t at) -> int { return (int)divide(at * nc + total - 1, total); };
  auto entry = [&](int k, int64_t x, int seq, int place, int64_t n, int64_t S, int64_t before) {
    PlanEntry e;
    e.b = seq + shift;
    e.rt = place;
    e.nt = (int32_t)n;
    e.off = (int32_t)(x - S > G::SWITCH && !whole ? x - S - G::SWITCH : 0);
    e.x = before + e.off;
    plan->e[k] = e;
  };
  if (few) {
    if (threadIdx.x < pairs) {
      sh.tile[threadIdx.x] = upto - mine + threadIdx.x * G::SWITCH;
      sh.of[threadIdx.x] = make_int2(b, rt);
    }
    __syncthreads();
    // a thread per range, which finds its row tile (the last threads, beside the first ones' row tiles)
    const int k = PLAN_THREADS - 1 - (int)threadIdx.x;
    if (k < nc) {
      const int64_t x = alone ? sh.tile[k] : divide(k * total, nc);
      int lo = 0, hi = (int)pairs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.tile[mid] <= x) lo = mid; else hi = mid;
      }
      const int64_t S = sh.tile[lo], end = lo + 1 < pairs ? sh.tile[lo + 1] : total;
      entry(k, x, sh.of[lo].x, sh.of[lo].y, end - S - G::SWITCH, S, S - (int64_t)lo * G::SWITCH);
    }
  }
  int64_t at = 0;
  for (int64_t p0 = 0; p0 < pairs; p0 += PLAN_THREADS) {  // a thread per row tile
    const int64_t p = p0 + threadIdx.x;
    int64_t n = mine, before = upto - mine;  // units before the row tile
    if (!few) {
      int64_t sum;
      n = tiles(p);
      before = at + plan_sum(n, pairs - p0, &sum) - n;
      at += sum;
    }
    if (p >= pairs) continue;
    if (unit != nullptr && !whole) unit[p] = before;
    const int64_t S = before + p * G::SWITCH;
    const int k0 = ranges_before(S), k1 = ranges_before(S + G::SWITCH + n);
    if (owner != nullptr && !whole) {
      // the range that holds its first unit: the last that begins there, or one from before
      const int kh = ranges_before(S + G::SWITCH + 1);
      owner[p] = make_int4(b + shift, rt, 2 * (kh - 1) + (kh > k0 ? 0 : 1), k1 - 1);
    }
    if (!few)
      for (int k = k0; k < k1; ++k) entry(k, divide(k * total, nc), b, rt, n, S, before);
  }
}

// A range's way: one segment (a run of key tiles of one row tile)
// after the other.
template <int MODE, class G>
struct Walk : Pages<MODE> {
  SeqInfo<MODE> s;
  int b, rt, nt, t;   // row tile, its key tiles, first key tile of the segment
  int n;              // key tiles of the segment
  int seg;            // segments before this one
  int64_t left;       // units from this segment on
  __device__ __forceinline__ void start(const ChunkArgs& a, const Plan<G>& plan, int k) {
    const PlanEntry e = plan.e[k];
    b = e.b;
    rt = e.rt;
    nt = e.nt;
    t = e.off;
    left = (k + 1 < plan.n ? plan.e[k + 1].x : plan.units) - e.x;
    seg = 0;
    s = seq_info<MODE>(a, b, false);
    if constexpr (MODE == kWindow) (void)key_tiles<G>(a, s, rt, this);
    n = (int)(left < nt - t ? left : nt - t);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const ChunkArgs& a) {
    left -= n;
    ++seg;
    if (left <= 0) return;
    t = 0;
    if (++rt >= row_tiles<G>(a, s)) {
      rt = 0;
      do {
        s = seq_info<MODE>(a, ++b, false);
      } while (s.nq == 0);
    }
    nt = key_tiles<G>(a, s, rt, this);
    n = (int)(left < nt ? left : nt);
  }
  __device__ __forceinline__ bool whole() const { return t == 0 && n == nt; }
  // whether the row tile's results are final (and not parts that the join adds up)
  __device__ __forceinline__ bool final() const {
    if constexpr (MODE == kShared) {
      if (s.part >= 0) return false;
    }
    return whole();
  }
};

// The block-table entries of 32 of a row tile's pages, one per lane, from page `from` on.
struct PageWindow {
  int64_t from;
  int32_t e;
  // cache slot of the page's first row, or -1 (past the sequence, or an entry out of range)
  template <int MODE, class G>
  __device__ __forceinline__ int64_t slot(const ChunkArgs& a, const Walk<MODE, G>& w, int64_t page, int lane, bool tell) {
    if (page < from || page >= from + 32) {
      from = page;
      e = -1;
      const int64_t at = MODE == kWindow ? w.at((int)page + lane) : page + lane;
      if (at * PAGE < w.s.T) {
        if constexpr (MODE == kShared)
          e = __ldg(&a.block_table[(int64_t)w.s.row * a.max_blocks + w.s.page0 + at]);
        else
          e = __ldg(&a.block_table[(int64_t)w.b * a.max_blocks + at]);
        if (e < 0 || (int64_t)e >= a.n_blocks) {
          if (tell) atomicOr(a.err, ERR_BLOCK_TABLE);
          e = -1;
        }
      }
    }
    const int32_t v = __shfl_sync(0xffffffffu, e, (int)(page - from));
    return v < 0 ? -1 : (int64_t)v * PAGE;
  }
};
// ------------------------------------------------------------------ arithmetic
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 up2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Two e4m3 terms of an f16 pair on its scale: hi = e4m3(x), lo = e4m3(x - hi) (the residual is exact in f16).
__device__ __forceinline__ void split_h2(uint32_t x, uint16_t& hi, uint16_t& lo) {
  const __half2 v = *reinterpret_cast<const __half2*>(&x);
  hi = f16x2_to_e4m3x2(v);
  const uint32_t d = e4m3x2_to_f16x2(hi);
  lo = f16x2_to_e4m3x2(__hsub2(v, *reinterpret_cast<const __half2*>(&d)));
}
__device__ __forceinline__ uint32_t scaled_h2(uint32_t x, __half2 s) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&x), s);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// NaN codes (0x7F, 0xFF) of four bytes set to 0
__device__ __forceinline__ uint32_t no_nan(uint32_t v) {
  return v & ~__vcmpeq4(v & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

__device__ __forceinline__ void sts64(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// ------------------------------------------------------------------ join
// The parts of a row tile's rows (N of them).  With a shared prefix they are those of the row's own keys, then
// those of the prefix.  A warp per row (or per row and SPLIT-th of its channels), a block for 16 rows; or where
// rows have many parts, a block per row, whose WARPS warps take every WARPS-th part each and are added up in order
// (one token of 16 heads over 40000 keys, 152 parts: 25 us, with a warp per row 66).
struct PartsJoin {
  const int64_t* tiles;          // their number
  const int4* owner;
  const float *m, *l, *o;        // [slots][N], and from `whole` on the row tiles that one range held whole
  int64_t whole;
  const int64_t* prefix_base;    // (the prefixes', whose slots lie in front of these)
  const int4* prefix_owner;
  int64_t prefix_slots;
};

constexpr int JOIN_WARPS = 16;

template <int MODE, int N, int SPLIT, int WARPS>
__global__ void __launch_bounds__(JOIN_WARPS * 32, SPLIT == 1 && WARPS == 1 ? 2 : 0)
    parts_join_kernel(const ChunkArgs a, const PartsJoin ps) {
  static_assert(WARPS == 1 || (WARPS == JOIN_WARPS && SPLIT == 1), "a warp per row, or a block");
  constexpr int JOIN_ROWS = JOIN_WARPS / WARPS, BLOCKS = N / JOIN_ROWS * SPLIT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t p = blockIdx.x / BLOCKS;
  const int row = (int)(blockIdx.x % BLOCKS) / SPLIT * JOIN_ROWS + warp / WARPS;
  const int ch = (int)(blockIdx.x % SPLIT) * (DL / SPLIT);
  grid_dependency_wait();  // (every block: what it reads, and that this launch is not over before the kernel is)
  const int64_t tiles = *ps.tiles;
  const int4 of = ps.owner[p];  // (there is room for as many as there are blocks)
  if (p >= tiles) return;
  const int k0 = of.z >> 1, n_own = of.w - k0 + 1;
  const SeqInfo<MODE> s = seq_info<MODE>(a, of.x, false);
  bool shares = false;
  if constexpr (MODE == kShared) shares = s.part >= 0;
  if (n_own == 1 && !shares) return;  // whole
  const int64_t r = (int64_t)of.y * N + row;
  if (r >= (int64_t)s.nq * a.H) return;  // (with a block per row, all of it)
  int n = n_own, prefix_k0 = 0;
  int64_t own_whole = 0, prefix_whole = 0, prefix_row = 0;
  int4 pf = make_int4(0, 0, 0, 0);
  if constexpr (MODE == kShared) {
    if (shares) {
      const int g = a.entries[of.x].v.w;
      const ChunkEntry e = a.entries[g];
      const int64_t in_group = (s.q0 - e.u.x) * a.H + r;
      pf = ps.prefix_owner[ps.prefix_base[g] + in_group / WideGeo::ROWS];
      prefix_k0 = pf.z >> 1;
      n += pf.w - prefix_k0 + 1;
      own_whole = ps.whole + s.part + r;
      prefix_whole = ps.whole + e.v.z + in_group;
      prefix_row = in_group % WideGeo::ROWS - ps.prefix_slots;  // (the prefixes' slots lie in front of these)
    }
  }
  auto slot = [&](int j) -> int64_t {
    if (MODE == kShared && shares) {
      if (j >= n_own) {
        j -= n_own;
        if (n - n_own == 1) return prefix_whole;
        return (int64_t)(j == 0 ? pf.z : 2 * (prefix_k0 + j)) * WideGeo::ROWS + prefix_row;
      }
      if (n_own == 1) return own_whole;
    }
    return (int64_t)(j == 0 ? of.z : 2 * (k0 + j)) * N + row;
  };
  // (the first parts' values are asked for together with the weights of all of them, and the others AT_ONCE at a time)
  constexpr int Q = 4 / SPLIT, AT_ONCE = SPLIT == 1 && WARPS == 1 ? 2 : 4;  // 16-byte units a lane
  const int first = warp % WARPS;
  float4 v[AT_ONCE][Q], acc[Q];
  auto ask = [&](int j0) {
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      if (j0 + i * WARPS >= n) break;
      const float4* o = reinterpret_cast<const float4*>(ps.o + slot(j0 + i * WARPS) * DL + ch) + lane;
#pragma unroll
      for (int c = 0; c < Q; ++c) v[i][c] = o[32 * c];
    }
  };
  float M = -INFINITY, L = 0.f, m0 = -INFINITY, l0 = 0.f;
  if (lane < n) {
    M = m0 = ps.m[slot(lane)];
    l0 = ps.l[slot(lane)];
  }
  ask(first);
  for (int j = lane + 32; j < n; j += 32) M = fmaxf(M, ps.m[slot(j)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int c = 0; c < Q; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int BATCH = WARPS == 1 ? 32 : AT_ONCE * WARPS;  // parts whose weights are at hand, those of each
  constexpr int EACH = BATCH / 32;                          // 32 of them a lane's
  for (int j0 = 0; j0 < n; j0 += BATCH) {
    float wt[EACH];
#pragma unroll
    for (int h = 0; h < EACH; ++h) {
      const int j = j0 + 32 * h + lane;
      wt[h] = 0.f;
      if (j < n) {
        const float m = j == lane ? m0 : ps.m[slot(j)];
        wt[h] = m > -INFINITY ? ex2_approx(m - M) : 1.f;  // (a NaN l stays one)
        L += wt[h] * (j == lane ? l0 : ps.l[slot(j)]);
      }
    }
    for (int i0 = first; i0 < BATCH && j0 + i0 < n; i0 += AT_ONCE * WARPS) {
      if (j0 + i0 > first) ask(j0 + i0);
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int at = i0 + i * WARPS;  // (the same for the warp)
        if (j0 + at >= n) break;
        float w = 0.f;
#pragma unroll
        for (int h = 0; h < EACH; ++h)
          if (at >> 5 == h) w = __shfl_sync(0xffffffffu, wt[h], at & 31);
#pragma unroll
        for (int c = 0; c < Q; ++c) {
          acc[c].x += w * v[i][c].x;
          acc[c].y += w * v[i][c].y;
          acc[c].z += w * v[i][c].z;
          acc[c].w += w * v[i][c].w;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = s.q0 * a.H + r;
  if (first == 0 && ch == 0 && a.lse != nullptr && lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
  if constexpr (WARPS == 1) {
    uint2* out = reinterpret_cast<uint2*>(a.out + at * DL + ch) + lane;
#pragma unroll
    for (int c = 0; c < Q; ++c) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
      const __nv_bfloat162 y = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
      out[32 * c] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
  } else {
    __shared__ float part[WARPS][DL];
#pragma unroll
    for (int c = 0; c < Q; ++c) reinterpret_cast<float4*>(part[warp])[32 * c + lane] = acc[c];
    __syncthreads();
    static_assert(WARPS * 32 == DL, "a thread per channel");
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) x += part[w][threadIdx.x];
    reinterpret_cast<__nv_bfloat16*>(a.out)[at * DL + threadIdx.x] = __float2bfloat16_rn(x * inv);
  }
}

// Its launch for at most `tiles` row tiles, of at most `ranges` ranges: a block per row where row tiles may have
// MANY_PARTS parts each, and with few row tiles more blocks for each.
template <int MODE, int N>
cudaError_t launch_parts_join(const ChunkArgs& a, const PartsJoin& ps, int64_t tiles, int64_t ranges, cudaStream_t s) {
  constexpr int64_t FEW_ROWS_TO_JOIN = 8192, MANY_PARTS = 8;
  const int64_t blocks = tiles * (N / JOIN_WARPS);
  if (ranges >= MANY_PARTS * tiles)
    return launch_after_prep(parts_join_kernel<MODE, N, 1, JOIN_WARPS>, (unsigned)(tiles * N), JOIN_WARPS * 32, 0, s, a, ps);
  if (tiles * N < FEW_ROWS_TO_JOIN)
    return launch_after_prep(parts_join_kernel<MODE, N, 4, 1>, (unsigned)(4 * blocks), JOIN_WARPS * 32, 0, s, a, ps);
  return launch_after_prep(parts_join_kernel<MODE, N, 1, 1>, (unsigned)blocks, JOIN_WARPS * 32, 0, s, a, ps);
}

}  // namespace
}  // namespace kv8
