// chunk.cu -- absorbed MLA attention of a chunk of new tokens per sequence over
// the paged fp8 latent cache, causal inside the chunk:
//   z_t = sm * ( sLc_t <q_lat, dec(Lc_t)> + sRc_t <q_rope, dec(Rc_t)> ),  t < lim
//   out = sum_t softmax(z)_t sLc_t dec(Lc_t),   lse = log sum_t exp(z_t)
// with lim = T - n + i + 1 for token i of the n queries of a sequence of T cached
// tokens (its last n tokens are the chunk itself), or T without the causal mask.
//
// All heads of a sequence read the same keys, so its rows are its (token, head)
// pairs, token after token, whatever the head count; a row tile is 256 of them.
// A work unit is one row tile against one tile of 128 keys: 256 x 128 x 2176 FLOP
// on 75 KB of cache that 36 row tiles read at about the same time, so the tensor
// cores bound it, not memory.
//
// A cluster of four CTAs takes a range of units (of consecutive row tiles, key tiles
// inside).  Two of them compute scores and softmax, two the context; each two form
// a cta_group::2 pair, M = 256, each SM holding 128 of the rows.  One SM's TMEM holds
// O for 128 rows x 512 channels and nothing else, which is why scores and context sit
// on different SMs; the pair halves the shared-memory traffic of B per MMA, which
// is why there are four.
//
// Score pair (cluster ranks 0, 1), per key tile:
//   S_L = Q_lat . Lc, S_R = Q_rope . Rc    kind::f8f6f4, M = 256, N = 128 (each CTA
//         holds one 64-token page of the tile as B), 36 MMAs.  The query is two e4m3
//         terms, hi + residual, on a power-of-two scale per row (a bf16 value is exact in
//         them unless it lies 2^-9 below its row's largest): hi of Lc in TMEM, the rest
//         in shared memory.  S_L is double-buffered in TMEM; S_R is not: its MMAs come last
//         in a tile, when the previous one has long been read.
//   sixteen softmax warps, each 16 rows x 64 tokens of a tile: u = sLc S_L + sRc S_R, per
//         thread p = 2^(c u - M_g + 7), its sum l, and the weights g' = p sLc as f16.  The
//         reference M_g follows the largest weight 2^(c u) sLc of the row, not the largest
//         score, so that the top weights fill the e4m3 range however the row scales differ
//         (a scale under 2^-40 counts as that, so that p stays in range); it is lazy (moves up
//         by more than 2^TAU, down by more than 2^DOWN).  Each page of a tile, so each warp, has
//         its own, which saves the two warps of a row from meeting in every tile (2 %).  g' and
//         M_g go to the row's context CTA by asynchronous remote stores.
// Context pair (ranks 2, 3), per key tile:
//   sixteen warps bring the pages' g' onto one reference, the larger of the two (the other page's
//         by a factor in f16: two roundings of 2^-11, where the terms' own is 2^-9), split it
//         into two e4m3 terms (hi + residual), the A operand, and rescale the rows of O whose
//         reference moved;
//   O += g'_hi V + g'_lo V    M = 256, N = 256 channels (each CTA holds half of them as
//         B, the cache tile read MN-major), 16 MMAs into all 512 TMEM columns.
//   At the end of a row tile the rows are divided by l, rounded to bf16 and written; where
//   the range holds only part of a row tile's keys, the partial (f32 o, l and M_g) goes to the
//   workspace and a second launch joins the parts.
//
// Keys that a row does not see have weight 0; since 0 x NaN is NaN, the context warps also
// clear NaN codes from V tiles that some row of the tile sees only in part (where every row
// sees a NaN, its NaN denominator carries it).
//
// The units of all row tiles are cut into ranges of equal cost, one per cluster, by a one-CTA
// plan kernel from q_start and seq_lens on the device (36 clusters are resident at once: their
// 144 SMs are what a call uses).
//
// What bounds it.  A tile's MMAs take 2304 cycles on a score pair (36 of 64 cycles: 576 channels,
// twice for the query's two terms, at twice the rate of bf16) and 2048 on a context pair.  A tile
// takes about 3100 on normal values with outlying rows: the sixteen warps of either side are a chain
// of waits and arithmetic that long (as traced, which adds a tenth: softmax 380 the wait for S, 840
// reading and scaling it, 470 the largest weight, 380 the reference, 1090 the exponentials and stores;
// context 1000 the split, 2 x 800 the rescale where a reference moved, for a warp's 32 rows three
// tiles of four), at 52 % of the issue slots; the tensor pipe is active 76 % of a score SM's time.
// Ways to overlap two tiles were slower: softmax warps in two groups on alternate tiles wait for the
// one S_R buffer (TMEM is full), and more registers a thread, for two tiles at once, do not fit 19 warps.
//
// Measured, one GB300 (fractions of the bf16 rate of a large matrix product, 1895 TFLOP/s): 2 x 256
// tokens over 65536 keys at 128 heads 6.2 ms, 1500 TFLOP/s, 0.79; a prompt of 4096 tokens 2.04 ms,
// 1150, 0.61 (row tiles begin every 16 key tiles on average); 32 x 4 drafted tokens over up to
// 16384 keys 0.235 ms, 1060, 0.56; one token of 4 heads over 256 keys 22.5 us, of which 4 are the plan,
// 5 the query, 5 the pipeline and 5 the results.
//
// Every wait is bounded (2 s): on a timeout
// the CTA flags the workspace error word, drains its MMAs and copies and meets its cluster
// at the closing barrier.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "kv8_common.cuh"
#include "tc_ptx.cuh"

namespace kv8 {
namespace {

using namespace ptx;

constexpr int ROWS = 256;                    // rows of a row tile: 128 per CTA of a pair
constexpr int CROWS = 128;
constexpr int W_TMA = 0, W_MMA = 1, W_SCALE = 2, W_LANE = 3;
constexpr int N_LANE_WARPS = 16;             // four per TMEM lane quarter, and per scheduler
constexpr int NTHREADS = (W_LANE + N_LANE_WARPS) * 32;
constexpr int MAX_CLUSTERS = NUM_SMS / 4;
// A cluster per row tile, or more while that gives each MIN_TILES key tiles on average.  (The ranges
// differ by up to SWITCH, below, which is counted in front of every row tile, the first of a range
// among them: 4 tiles fall into ranges of 0 and 4, 16 into 0, 0, 2, 3, 2, 3, 3, 3.)  Device times for
// 1, 2 and 4, us: one token of 128 heads over 512 keys 30.8, 28.7, 26.7, over 2048 35.4, 32.8, 36.8,
// over 8192 47.2, 47.0, 41.0; two row tiles of 8 key tiles 32.8, 34.9, 38.7.
constexpr int MIN_TILES = 2;
// What beginning a row tile costs, in key tiles: 19 thousand cycles (the query is loaded and split
// while the context pair writes its results, and the pipeline fills) against 3.1 thousand a tile.  A
// prompt of 4096 tokens at 128 heads: 2.40 ms when ranges count 4 for it, 2.17 for 5, 2.04 for 6, 2.06
// for 7, 2.09 for 8; five sequences without a mask 103, 102, 98, 99, 100 us.
constexpr int SWITCH = 6;
constexpr int BLK = PAGE * 128;              // 8 KB: [64 tokens x 128 bytes]
constexpr int RBLK = PAGE * DR;              // 4 KB: [64 tokens x 64 bytes]
constexpr int KTILE = 4 * BLK + RBLK;        // a score CTA's page of a tile: 36 KB
constexpr int NK = 3;                        // K ring, in tiles; loaded and freed in two halves
constexpr int NSC = 5;                       // row-scale rings, in tiles (see the load warp)
constexpr int VBLK = TILE * 128;             // 16 KB: [128 tokens x 128 channels]
constexpr int VTILE = 2 * VBLK;              // a context CTA's half of the channels
constexpr int NVT = 2;                       // V ring, in tiles
constexpr int SUB = 64;                      // tokens of a softmax warp's share of a tile (a page)
constexpr int OP_ATOM = CROWS * 128;         // 16 KB: [128 rows x 128 tokens], e4m3
constexpr int P_F = CROWS * TILE * 2;        // payload: g' f16 (256 bytes a row), then the two pages' references,
constexpr int P_PAGES = P_F + CROWS * 8;     // then the pages present
constexpr int P_BYTES = P_PAGES + 4;
constexpr int P_STRIDE = 34 * 1024;
constexpr float TAU = 1.0f;
constexpr float P_LOG = 7.0f;                // g' <= 2^(TAU + P_LOG) = 256 <= 448
constexpr float DOWN = 10.0f;
// bounds that keep p and l in range, 2^(P_LOG + TAU + 40 + 50) times a count of keys: the smallest
// log2 of a row scale that sets a reference, and how far below its highest value so far a row's
// reference may come (l and O hold no more than 2^(highest - reference) times what they did there)
constexpr float LG_MIN = -40.0f, DOWN_CAP = 50.0f;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// mbarriers (the same offsets in all four CTAs: commits are multicast).  What passes between CTAs is
// ordered at cluster scope.  Shared memory that one CTA's warps wrote or read, and that another CTA's
// stores overwrite or whose MMAs read it: the warps arrive at their own CTA's barrier, and a warp
// that has nothing else to do waits there and arrives at the other CTA's (the relays).  TMEM alone:
// a relaxed arrival between the fences of tcgen05.  Releases at cluster scope by the sixteen warps
// themselves make drafts 15 % slower where it is the payloads' buffers alone and 45 % with the operands,
// relays of the S buffers and the O halves as well 19 %; this 2 to 4 %.
constexpr int B_KFULL = 0;                   // [2 NK] rank 0: both CTAs' halves of a K half tile loaded
constexpr int B_KEMPTY = B_KFULL + 2 * NK;   // [2 NK] ranks 0, 1: consumed
constexpr int B_SCFULL = B_KEMPTY + 2 * NK;  // [NSC] score: row scales of a tile loaded
constexpr int B_SFULL = B_SCFULL + NSC;      // [2] score: S of a tile in TMEM (commit); its scales prepared, and
                                             // its payload buffer free (the scale warp)
constexpr int B_SEMPTY = B_SFULL + 2;        // [2] rank 0: S read (16 warps x 2 CTAs)
constexpr int B_QREADY = B_SEMPTY + 2;       // score: the row tile's query in place (16 warps; in rank 0 also rank 1's relay)
constexpr int B_PX = B_QREADY + 1;           // [4] score: the four warps of a lane quarter meet
constexpr int B_PFREE = B_PX + 4;            // [2] context: payload buffer read (16 warps); score: the partner's relay of it
constexpr int B_PFULL = B_PFREE + 2;         // [2] context: payload arrived
constexpr int B_VT = B_PFULL + 2;            // [NVT] context: V tile loaded
constexpr int B_VEMPTY = B_VT + NVT;         // [NVT] ranks 2, 3: consumed
constexpr int B_EP = B_VEMPTY + NVT;         // context: a row tile's results have left shared memory
constexpr int B_OP = B_EP + 1;               // [2] context: operand of a tile written (16 warps; in rank 2 also rank 3's
                                             // relay, when its V tile is loaded as well)
constexpr int B_RS = B_OP + 2;               // [2 buffers][2] rank 2: O half ready (16 warps x 2 CTAs)
constexpr int B_ODONE = B_RS + 4;            // [2 buffers][2] ranks 2, 3: a tile's MMAs of an O half done
constexpr int NRF = 4;
constexpr int B_RF = B_ODONE + 4;            // [NRF] context: row factors of a finished row tile arrived
constexpr int B_DRAIN = B_RF + NRF;          // every MMA done
constexpr int NBAR = B_DRAIN + 1;

// shared memory (dynamic, 1024-byte aligned)
constexpr int OFF_FLAGS = 512;               // tmem base, abort flag
constexpr int OFF_FACTS = OFF_FLAGS + 16;    // [8] score: pages present in the tiles of the ring
constexpr int OFF_XL = 1024;                 // score: [128 rows][2 pages] l
constexpr int OFF_XQ = OFF_XL + 1024;        // score: [128 rows][4 parts] query maxima
constexpr int OFF_MG = OFF_XQ + 2048;        // score: [128 rows][2 pages] M_g at a row tile's end
constexpr int OFF_LIM = OFF_MG + 1024;       // score: [128] keys that the rows see
constexpr int OFF_C = OFF_LIM + 512;         // score: [128] the rows' c
constexpr int OFF_WALK = OFF_C + 512;        // score: [16 warps] segments
constexpr int OFF_SC = OFF_WALK + 1024;      // score: [NSC][128][2] row scales
constexpr int OFF_PL = OFF_SC + NSC * 1024;  // score: [NSC] of a tile's 64 token pairs: (sLc, sLc, sRc, sRc), then log2 sLc
constexpr int PL_BYTES = 64 * 16 + 64 * 8;
constexpr int OFF_QL = (OFF_PL + NSC * PL_BYTES + 1023) / 1024 * 1024;  // score: lo of Lc, four atoms
constexpr int OFF_QR = OFF_QL + 4 * OP_ATOM;                      // score: Rc, hi | lo
constexpr int OFF_K = OFF_QR + OP_ATOM;
constexpr int TOTAL_S = OFF_K + NK * KTILE;
constexpr int OFF_RF = 1024;                 // context: [NRF][128] row factors, and the references they go with
constexpr int OFF_P = 5120;                  // context: two payloads
constexpr int OFF_OP = OFF_P + 2 * P_STRIDE; // context: two operands (hi and lo atoms); results on their way out
constexpr int OFF_V = OFF_OP + 4 * OP_ATOM;
constexpr int TOTAL_C = OFF_V + NVT * VTILE;
constexpr int SMEM = TOTAL_S > TOTAL_C ? TOTAL_S : TOTAL_C;
// TMEM columns of a score CTA
constexpr int T_SL = 0, T_SR = 256, T_QH = 384;
static_assert(NSC >= NK + 2 && NSC <= 8 && NVT <= 8 && OFF_FACTS + 32 <= OFF_XL, "rings");
static_assert(NBAR * 8 <= OFF_FLAGS && OFF_RF + NRF * CROWS * 8 <= OFF_P, "shared memory layout");
static_assert(OFF_K % 1024 == 0 && KTILE % 1024 == 0 && OFF_V % 1024 == 0 && P_STRIDE % 1024 == 0, "swizzle atoms");
static_assert(P_BYTES <= P_STRIDE && N_LANE_WARPS * 2048 <= 4 * OP_ATOM, "payload and staging");
static_assert(SMEM <= 232448, "shared memory above the per-CTA limit");

// ------------------------------------------------------------------ work
// Plan of cluster k: its first row tile (sequence b, row tile rt, nt key tiles of
// which off come before the range), the unit where the range starts and its units.
struct PlanEntry {
  int32_t b, rt, nt, off;
  int64_t x;
};
struct Plan {
  int64_t n_clusters, units;
  PlanEntry e[MAX_CLUSTERS];
};

struct SeqInfo {
  int64_t q0;  // first row of the query arrays
  int nq, T;
};
__device__ __forceinline__ SeqInfo seq_info(const ChunkArgs& a, int b, bool tell) {
  SeqInfo s;
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
__device__ __forceinline__ int row_tiles(const ChunkArgs& a, const SeqInfo& s) {
  return (int)(((int64_t)s.nq * a.H + ROWS - 1) / ROWS);
}
// keys that token i of the sequence sees
__device__ __forceinline__ int limit_of(const ChunkArgs& a, const SeqInfo& s, int i) {
  if (!a.causal) return s.T;
  const int lim = s.T - s.nq + i + 1;
  return lim < 0 ? 0 : lim;
}
// key tiles of a row tile: those that its last row sees; one where it sees none, so
// that its (empty) rows are written by the same path
__device__ __forceinline__ int key_tiles(const ChunkArgs& a, const SeqInfo& s, int rt) {
  const int64_t last = ((int64_t)rt * ROWS + ROWS - 1) / a.H;
  const int lim = limit_of(a, s, last < s.nq ? (int)last : s.nq - 1);
  return lim > 0 ? (lim - 1) / TILE + 1 : 1;
}

__device__ __forceinline__ int64_t plan_sum(int64_t v, int64_t* tmp, int64_t* total) {
  // inclusive sum over 1024 threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    tmp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += tmp[warp - 1];
  *total = tmp[31];
  __syncthreads();
  return v;
}

constexpr int PLAN_NEAR = 4096;

// One CTA: row tiles before each sequence (base, in shared memory if they fit), the units of every row tile,
// their total, and the row tile that each cluster's range starts in.
__global__ void __launch_bounds__(1024) plan_kernel(const ChunkArgs a, Plan* plan, int64_t* base, int clusters) {
  grid_dependents_launch();
  __shared__ int64_t tmp[32];
  __shared__ int64_t near[PLAN_NEAR];
  if (a.B < PLAN_NEAR) base = near;
  if (threadIdx.x == 0) *a.err = 0;
  __syncthreads();
  int64_t pairs = 0;
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int64_t n = b < a.B ? row_tiles(a, seq_info(a, b, true)) : 0;
    int64_t sum;
    const int64_t inc = plan_sum(n, tmp, &sum);
    if (b < a.B) base[b] = pairs + inc - n;
    pairs += sum;
  }
  if (threadIdx.x == 0) base[a.B] = pairs;
  __syncthreads();
  int b = 0, rt = 0;
  auto tiles = [&](int64_t p) -> int64_t {
    if (p >= pairs) return 0;
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (base[mid] <= p) lo = mid; else hi = mid;
    }
    b = lo;
    rt = (int)(p - base[lo]);
    return key_tiles(a, seq_info(a, b, false), rt);
  };
  // The ranges are equal on an axis where a row tile is SWITCH + nt long, and the border falls on a
  // key tile of it; x counts units (key tiles).
  int64_t mine = 0, units;
  for (int64_t p = threadIdx.x; p < pairs; p += 1024) mine += tiles(p);
  (void)plan_sum(mine, tmp, &units);
  const int64_t total = units + pairs * SWITCH;
  int64_t nc = units / MIN_TILES > pairs ? units / MIN_TILES : pairs;
  nc = nc > clusters ? clusters : (nc < 1 ? (units > 0 ? 1 : 0) : nc);
  if (threadIdx.x == 0) {
    plan->n_clusters = nc;
    plan->units = units;
  }
  int64_t at = 0;
  for (int64_t p0 = 0; p0 < pairs; p0 += 1024) {
    const int64_t p = p0 + threadIdx.x, n = pairs <= 1024 ? mine : tiles(p);
    int64_t sum;
    const int64_t before = at + plan_sum(n, tmp, &sum) - n;  // units before the row tile
    const int64_t S = before + p * SWITCH, len = n + SWITCH;
    int64_t k = n > 0 ? S * nc / total : nc;
    while (k < nc && k * total / nc < S) ++k;
    for (; k < nc; ++k) {
      const int64_t x = k * total / nc;
      if (x >= S + len) break;
      PlanEntry e;
      e.b = b;
      e.rt = rt;
      e.nt = (int32_t)n;
      e.off = (int32_t)(x - S > SWITCH ? x - S - SWITCH : 0);
      e.x = before + e.off;
      plan->e[k] = e;
    }
    at += sum;
  }
}

// A cluster's way through its range: one segment (a run of key tiles of one row tile)
// after the other.
struct Walk {
  SeqInfo s;
  int b, rt, nt, t;   // row tile, its key tiles, first key tile of the segment
  int n;              // key tiles of the segment
  int seg;            // segments before this one
  int64_t left;       // units from this segment on
  __device__ __forceinline__ void start(const ChunkArgs& a, const Plan& plan, int k) {
    const PlanEntry e = plan.e[k];
    b = e.b;
    rt = e.rt;
    nt = e.nt;
    t = e.off;
    left = (k + 1 < plan.n_clusters ? plan.e[k + 1].x : plan.units) - e.x;
    seg = 0;
    s = seq_info(a, b, false);
    n = (int)(left < nt - t ? left : nt - t);
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const ChunkArgs& a) {
    left -= n;
    ++seg;
    if (left <= 0) return;
    t = 0;
    if (++rt >= row_tiles(a, s)) {
      rt = 0;
      do {
        s = seq_info(a, ++b, false);
      } while (s.nq == 0);
    }
    nt = key_tiles(a, s, rt);
    n = (int)(left < nt ? left : nt);
  }
  __device__ __forceinline__ bool whole() const { return t == 0 && n == nt; }
};

static_assert(sizeof(Walk) * N_LANE_WARPS <= OFF_SC - OFF_WALK, "segments");

// The block-table entries of 32 pages, one per lane, from page `from` on.
struct PageWindow {
  int64_t from;
  int32_t e;
  // cache slot of the page's first row, or -1 (past the sequence, or an entry out of range)
  __device__ __forceinline__ int64_t slot(const ChunkArgs& a, const Walk& w, int64_t page, int lane, bool tell) {
    if (page < from || page >= from + 32) {
      from = page;
      e = -1;
      if ((page + lane) * PAGE < w.s.T) {
        e = __ldg(&a.block_table[(int64_t)w.b * a.max_blocks + page + lane]);
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

// byte offset of 16-byte unit u (0..15) of row r in a payload: unit 4 s + i holds tokens
// 32 s + 8 j + 2 i, + 1 for j = 0 .. 3
__device__ __forceinline__ uint32_t prow(int r, int u) {
  return (uint32_t)(r * 256 + ((u ^ (r & 7)) << 4));
}

struct Workspace {
  Plan* plan;
  float* m;   // [2 MAX_CLUSTERS][256]: slot 2k the first segment of cluster k, 2k + 1 its last
  float* l;
  float* o;   // [..][256][512]
};

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(NTHREADS, 1)
    chunk_kernel(const ChunkArgs a, const Workspace ws, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap smap) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int k = (int)(blockIdx.x >> 2);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + OFF_FLAGS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + OFF_FLAGS + 4);
  uint32_t* facts = reinterpret_cast<uint32_t*>(sm + OFF_FACTS);
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(a.err, ERR_TIMEOUT);
  };
  auto wait = [&](int bar, uint32_t parity) -> bool {
    return mbar_wait_warp(&bars[bar], parity & 1, abort_flag, WAIT_NS);
  };
  auto wait_cluster = [&](int bar, uint32_t parity) -> bool {
    return mbar_wait_cluster_warp(&bars[bar], parity & 1, abort_flag, WAIT_NS);
  };

  // what this CTA's warps have done, told to another CTA (by a whole converged warp)
  auto relay = [&](int bar, uint32_t parity, uint32_t to) -> bool {
    if (!wait(bar, parity)) return false;
    tc_fence_after();
    tc_fence_before();
    if (lane == 0) arrive_cluster(to);
    __syncwarp();
    return true;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) mbar_init(&bars[i], 1);
    const int here = N_LANE_WARPS + (rank == 0 || rank == 2);  // (and the relay of the pair's other CTA)
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_SEMPTY + i], 2 * N_LANE_WARPS);
    mbar_init(&bars[B_QREADY], here);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[B_PX + i], N_LANE_WARPS / 4);
    mbar_init(&bars[B_EP], N_LANE_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_PFREE + i], rank < 2 ? 1 : N_LANE_WARPS);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[B_RS + i], 2 * N_LANE_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_OP + i], here);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_SFULL + i], 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (rank >= 2) {  // what the context CTAs expect first
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&bars[B_PFULL + i], P_BYTES);
      for (int i = 0; i < NRF; ++i) mbar_arrive_expect_tx(&bars[B_RF + i], CROWS * 8);
    }
  }
  if (warp == W_MMA) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the plan
  grid_dependents_launch();  // (the join kernel may come as soon as there is room)
  const bool work = k < ws.plan->n_clusters;
  Walk w;
  if (work) w.start(a, *ws.plan, k);
  else w.left = 0;
  int gt = 0;  // key tiles of the range before this segment

  if (rank < 2) {
    // ================================================================ score CTAs
    const uint32_t kring = smem_u32(sm + OFF_K);
    const uint32_t scr = smem_u32(sm + OFF_SC);
    if (warp == W_TMA) {
      // this CTA's page of every tile, in two halves (Lc 0, 1; then Lc 2, 3 and Rc),
      // and both pages' row scales
      bool ok = true;
      const uint32_t kfull0 = map_to(smem_u32(&bars[B_KFULL]), 0);
      int halves = 0, nsc = 0;
      for (; ok && w.more(); w.next(a)) {
        PageWindow pw;
        pw.from = -64;
        for (int i = 0; ok && i < w.n; ++i) {
          const int g = gt + i, kb = g % NK, sc = g % NSC;
          const int64_t page = 2 * (int64_t)(w.t + i);
          const int64_t s0 = pw.slot(a, w, page, lane, rank == 0);
          const int64_t s1 = pw.slot(a, w, page + 1, lane, rank == 0);
          const int64_t mine = rank == 0 ? s0 : s1;
          const uint32_t pages = (s0 >= 0 ? 1u : 0u) + (s1 >= 0 ? 1u : 0u);
          const uint32_t dst = kring + kb * KTILE;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int bar = 2 * kb + h;
            if (!wait(B_KEMPTY + bar, (uint32_t)(g / NK) ^ 1u)) {
              ok = false;
              break;
            }
            if (rank == 0)
              mbar_arrive_expect_tx_warp(&bars[B_KFULL + bar], pages * (2 * BLK + (h ? RBLK : 0)));
            halves = 2 * g + h + 1;
            if (mine >= 0) {
              tma_load_2d_pair_warp(dst + (2 * h) * BLK, &kmap, 256 * h, (int)mine, kfull0 + bar * 8);
              tma_load_2d_pair_warp(dst + (2 * h + 1) * BLK, &kmap, 256 * h + 128, (int)mine, kfull0 + bar * 8);
              if (h) tma_load_2d_pair_warp(dst + 4 * BLK, &rmap, DL, (int)mine, kfull0 + bar * 8);
            }
          }
          if (!ok) break;
          // the row scales' slots held tile g - 5: the MMAs of tile g - 3, done by now, began
          // their last ones when the softmax warps had read S of tile g - 4, and so were
          // through with tile g - 5
          facts[sc] = (s0 >= 0 ? 1u : 0u) | (s1 >= 0 ? 2u : 0u);
          mbar_arrive_expect_tx_warp(&bars[B_SCFULL + sc], 512u * pages);
          if (s0 >= 0) tma_load_1d_warp(scr + sc * 1024, &smap, (int)(2 * s0), &bars[B_SCFULL + sc]);
          if (s1 >= 0) tma_load_1d_warp(scr + sc * 1024 + 512, &smap, (int)(2 * s1), &bars[B_SCFULL + sc]);
          nsc = g + 1;
        }
        gt += w.n;
      }
      if (!ok) {
        // let what was requested land before the cluster can leave
        if (lane == 0) fail();
        const int zero = 0;
        if (rank == 0)
          for (int i = (halves > 2 * NK ? halves - 2 * NK : 0); i < halves; ++i)
            (void)mbar_wait(&bars[B_KFULL + 2 * ((i >> 1) % NK) + (i & 1)], ((i >> 1) / NK) & 1, &zero, WAIT_NS);
        for (int i = (nsc > NSC ? nsc - NSC : 0); i < nsc; ++i)
          (void)mbar_wait(&bars[B_SCFULL + i % NSC], (i / NSC) & 1, &zero, WAIT_NS);
      }
      __syncwarp();
    } else if (warp == W_SCALE) {
      // the row scales of every tile in the form that the softmax warps use: pairs of tokens,
      // sLc made finite (a scale out of sight may be anything; its weight is 0 then, and in
      // sight the NaN or infinity shows in sRc), and log2 sLc
      bool ok = true;
      for (; ok && w.more(); w.next(a)) {
        // (and meanwhile the next row tile's queries come into L2)
        Walk wn = w;
        wn.next(a);
        if (wn.more()) {
          const int64_t r0 = (int64_t)wn.rt * ROWS + rank * CROWS, rows = (int64_t)wn.s.nq * a.H;
          for (int r = lane; r < CROWS && r0 + r < rows; r += 32) {
            const int64_t tok = wn.s.q0 + (uint32_t)(r0 + r) / (uint32_t)a.H, head = (uint32_t)(r0 + r) % (uint32_t)a.H;
            prefetch_l2(a.q_lat + tok * a.ql_t + head * a.ql_h, DL * 2);
            prefetch_l2(a.q_rope + tok * a.qr_t + head * a.qr_h, DR * 2);
          }
          __syncwarp();
        }
        for (int i = 0; i < w.n; ++i) {
          const int g = gt + i, sc = g % NSC;
          if (!wait(B_SCFULL + sc, (uint32_t)(g / NSC))) {
            ok = false;
            break;
          }
          // (what the softmax warps read there for tile g - 5 is in that tile's payload, and this warp
          // has waited until payload g - 3 was received and read: B_PFREE below)
          float4* pl = reinterpret_cast<float4*>(sm + OFF_PL + sc * PL_BYTES);
          float2* lg = reinterpret_cast<float2*>(pl + 64);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 s = reinterpret_cast<const float4*>(sm + OFF_SC + sc * 1024)[lane + 32 * h];
            const float x = fminf(fmaxf(s.x, 0.f), 3.0e38f), y = fminf(fmaxf(s.z, 0.f), 3.0e38f);
            pl[lane + 32 * h] = make_float4(x, y, fmaf(0.f, s.x, s.y), fmaf(0.f, s.z, s.w));
            lg[lane + 32 * h] = make_float2(fmaxf(lg2_approx(x), LG_MIN), fmaxf(lg2_approx(y), LG_MIN));
          }
          // (the payload buffer of tile g: the context warps have read tile g - 2, and so the softmax
          // warps were through with its S)
          if (g >= 2 && !wait_cluster(B_PFREE + (g & 1), (uint32_t)((g >> 1) - 1))) {
            ok = false;
            break;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_SFULL + (g & 1)]);
        }
        gt += w.n;
      }
      if (!ok && lane == 0) fail();
      __syncwarp();
    } else if (warp == W_MMA) {
      if (rank == 0) {
        const uint32_t id = idesc_f16(ROWS, TILE, false, false);  // e4m3 x e4m3 (format 0)
        const uint64_t kd = smem_desc(kring, 16, 1024, SW128);
        const uint64_t rd = smem_desc(kring + 4 * BLK, 16, 512, SW64);
        const uint64_t ql = smem_desc(smem_u32(sm + OFF_QL), 16, 1024, SW128);
        const uint64_t qr = smem_desc(smem_u32(sm + OFF_QR), 16, 1024, SW128);
        bool ok = true;
        for (; ok && w.more(); w.next(a)) {
          if (!wait_cluster(B_QREADY, (uint32_t)w.seg)) {
            ok = false;
            break;
          }
          for (int i = 0; i < w.n; ++i) {
            const int g = gt + i, kb = g % NK;
            const uint64_t off = (uint64_t)(kb * KTILE >> 4);
            const uint32_t dl = tmem + T_SL + (g & 1) * TILE;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!wait_cluster(B_KFULL + 2 * kb + h, (uint32_t)(g / NK))) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int blk = 0; blk < 2; ++blk) {
                const int c = 2 * h + blk;
                const uint64_t bd = kd + off + (uint64_t)(c * BLK >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_f8_ts_pair_warp(dl, tmem + T_QH + c * 32 + kk * 8, bd + 2 * kk, id, (h | blk | kk) != 0);
                  mma_f8_pair_warp(dl, ql + (uint64_t)(c * OP_ATOM >> 4) + 2 * kk, bd + 2 * kk, id, 1u);
                }
              }
              if (h == 0) mma_commit_pair_warp(&bars[B_KEMPTY + 2 * kb], 3);
            }
            if (!ok) break;
            // S_R (and the other S_L) of the previous tile read
            if (g > 0 && !wait_cluster(B_SEMPTY + ((g - 1) & 1), (uint32_t)((g - 1) >> 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              mma_f8_pair_warp(tmem + T_SR, qr + 2 * kk, rd + off + 2 * kk, id, kk != 0);
              mma_f8_pair_warp(tmem + T_SR, qr + 4 + 2 * kk, rd + off + 2 * kk, id, 1u);
            }
            mma_commit_pair_warp(&bars[B_KEMPTY + 2 * kb + 1], 3);
            mma_commit_pair_warp(&bars[B_SFULL + (g & 1)], 3);
          }
          gt += w.n;
        }
        if (!ok && lane == 0) fail();
        mma_commit_pair_warp(&bars[B_DRAIN], 3);
      } else {
        // rank 1 tells the MMA's issuer of its query
        const uint32_t qready = map_to(smem_u32(&bars[B_QREADY]), 0);
        bool ok = true;
        for (; ok && w.more(); w.next(a)) ok = relay(B_QREADY, (uint32_t)w.seg, qready);
        if (!ok && lane == 0) fail();
      }
      // every MMA of the pair is done and its commits have landed here
      const int zero = 0;
      (void)mbar_wait(&bars[B_DRAIN], 0, &zero, 4 * WAIT_NS);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- query and softmax
      // The four warps of a TMEM lane quarter share its 32 rows: each takes a part of the
      // query's channels for all of them, and one page of every tile for half of them (the two
      // halves meet nowhere and fall out of step, so that one computes while the other waits).
      // A thread holds the rows 8 p + lane / 4, and of the columns the pairs 8 j + 2 (lane %
      // 4), so that a token's scales serve two rows.
      const int q = warp & 3;                 // TMEM lane quarter
      const int part = (warp - W_LANE) >> 2;  // 128 channels of Lc and 16 of Rc
      const int hl = part >> 1, sub = part & 1;  // rows 16 hl .. of the quarter; page of a tile
      const int i4 = lane & 3, r8 = lane >> 2;
      const int row0 = q * 32 + r8;           // the thread's rows: row0 + 8 p
      const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
      float* xl = reinterpret_cast<float*>(sm + OFF_XL);
      uint32_t* xq = reinterpret_cast<uint32_t*>(sm + OFF_XQ);
      float* mgs = reinterpret_cast<float*>(sm + OFF_MG);
      int* lim = reinterpret_cast<int*>(sm + OFF_LIM);
      float* cs = reinterpret_cast<float*>(sm + OFF_C);
      Walk* walk = reinterpret_cast<Walk*>(sm + OFF_WALK) + (warp - W_LANE);  // (it has no registers to spare)
      const int rh = row0 + 16 * hl;          // the thread's rows of a tile: rh, rh + 8
      const int mh = rh + 8 * (i4 & 1);       // the row this lane speaks for there
      uint32_t px = 0;
      auto quarter_sync = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_PX + q]);
        return wait(B_PX + q, px++);
      };
      // The queries of a row tile: two e4m3 terms on the scale that puts a row's largest value
      // in [128, 256); c folds the scale back in, with sm_scale log2 e. Two of the thread's rows
      // at a time, their channels all in flight at once.
      auto load_query = [&](const Walk& x) -> bool {
        const int64_t r0 = (int64_t)x.rt * ROWS + rank * CROWS, rows = (int64_t)x.s.nq * a.H;
        const uint32_t qlo = smem_u32(sm + OFF_QL) + part * OP_ATOM, qrp = smem_u32(sm + OFF_QR);
        if (part == 0) {  // the keys that row q * 32 + lane sees (rows past the last one are copies of it)
          const int tok = (int)((uint32_t)(r0 + q * 32 + lane) / (uint32_t)a.H);
          lim[q * 32 + lane] = limit_of(a, x.s, tok < x.s.nq ? tok : x.s.nq - 1);
        }
#pragma unroll 1
        for (int hl = 0; hl < 2; ++hl) {
          uint4 v[2][5];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int64_t r = r0 + row0 + 16 * hl + 8 * p;
            const uint32_t at = (uint32_t)(r < rows ? r : rows - 1);
            const int64_t tok = x.s.q0 + at / (uint32_t)a.H, head = at % (uint32_t)a.H;
            const uint4* pq = reinterpret_cast<const uint4*>(a.q_lat + tok * a.ql_t + head * a.ql_h + part * 128) + i4;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[p][j] = __ldg(pq + 4 * j);
            v[p][4] = __ldg(reinterpret_cast<const uint4*>(a.q_rope + tok * a.qr_t + head * a.qr_h + part * 16) + (i4 & 1));
          }
          // a row's largest magnitude, as bf16 bits (ordered; 0x7F80 and up is inf or NaN)
          uint32_t top[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t t2 = 0;
#pragma unroll
            for (int j = 0; j < 5; ++j)
              t2 = __vmaxu2(t2, __vmaxu2(__vmaxu2(v[p][j].x & 0x7FFF7FFFu, v[p][j].y & 0x7FFF7FFFu),
                                         __vmaxu2(v[p][j].z & 0x7FFF7FFFu, v[p][j].w & 0x7FFF7FFFu)));
            t2 = __vmaxu2(t2, __shfl_xor_sync(0xffffffffu, t2, 1));
            t2 = __vmaxu2(t2, __shfl_xor_sync(0xffffffffu, t2, 2));
            top[p] = (t2 & 0xFFFFu) > (t2 >> 16) ? (t2 & 0xFFFFu) : (t2 >> 16);
          }
          if (i4 < 2) xq[(row0 + 16 * hl + 8 * i4) * 4 + part] = i4 ? top[1] : top[0];
          if (!quarter_sync()) return false;
          uint32_t hw[16];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int row = row0 + 16 * hl + 8 * p;
            const uint4 m4 = reinterpret_cast<const uint4*>(xq)[row];
            uint32_t mx = m4.x > m4.y ? m4.x : m4.y;
            mx = m4.z > mx ? m4.z : mx;
            mx = m4.w > mx ? m4.w : mx;
            // (a row with a NaN or an infinity is all NaN codes)
            const uint32_t nan = mx >= 0x7F80u ? 0x7F7F7F7Fu : 0u;
            // largest value in [2^e, 2^(e+1)): the scale 2^(7 - e), at most 2^87
            int e = (int)(mx >> 7) - 127;
            e = e < -80 ? -80 : e;
            if (mx == 0 || nan != 0u) e = 7;
            const float sc = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
            if (part == 0 && i4 == 0)
              cs[row] = fmaxf(a.sm_scale * LOG2E * __uint_as_float((uint32_t)(127 - 7 + e) << 23), 1e-37f);
            // (scaled by a power of two a bf16 is exact in f16 wherever it counts: the lo term ends
            // at 2^-10)
            auto terms = [&](uint32_t w0, uint32_t w1, uint32_t& hi, uint32_t& lo) {
              const __half2 a0 = __floats2half2_rn(bf16_lo(w0) * sc, bf16_hi(w0) * sc);
              const __half2 a1 = __floats2half2_rn(bf16_lo(w1) * sc, bf16_hi(w1) * sc);
              uint16_t h0, l0, h1, l1;
              split_h2(*reinterpret_cast<const uint32_t*>(&a0), h0, l0);
              split_h2(*reinterpret_cast<const uint32_t*>(&a1), h1, l1);
              hi = ((uint32_t)h0 | ((uint32_t)h1 << 16)) | nan;
              lo = (uint32_t)l0 | ((uint32_t)l1 << 16);
            };
            uint2 hi, lo;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // channels 32 j + 8 i4 .. + 7 of the part
              terms(v[p][j].x, v[p][j].y, hw[4 * j + 2 * p], lo.x);
              terms(v[p][j].z, v[p][j].w, hw[4 * j + 2 * p + 1], lo.y);
              sts64(qlo + sw128(row, 2 * j + (i4 >> 1)) + (i4 & 1) * 8, lo);
            }
            terms(v[p][4].x, v[p][4].y, hi.x, lo.x);
            terms(v[p][4].z, v[p][4].w, hi.y, lo.y);
            if (i4 < 2) {
              sts64(qrp + sw128(row, part) + i4 * 8, hi);
              sts64(qrp + sw128(row, 4 + part) + i4 * 8, lo);
            }
          }
          __syncwarp();
          tmem_st_16x32(tmem + lane_addr + ((uint32_t)(16 * hl) << 16) + T_QH + part * 32, hw);
        }
        __syncwarp();
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_QREADY]);
        return true;
      };

      bool ok = true, more = w.more();
      if (more) *walk = w;  // (every lane, the same)
      __syncwarp();
      while (ok && more) {
        const Walk& x = *walk;
        ok = load_query(x) && quarter_sync();  // (the sync: cs and lim are read by every part)
        if (!ok) break;
        const int n_tiles = x.n;
        uint64_t c2[2];                       // the rows' c, twice
        float l[2] = {0.f, 0.f};              // this thread's tokens, of its two rows
        float mg = -INFINITY, mhi = -INFINITY;  // row `mh`: its reference, and the highest one so far
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float v = cs[rh + 8 * p];
          c2[p] = pk2(v, v);
        }
        int t0 = x.t * TILE + sub * SUB;
        const int first = lim[q * 32 + 16 * hl];  // the keys that the first of the rows sees
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i, t0 += TILE) {
          const int g = gt + i, buf = g & 1, sc = g % NSC;
          if (!wait(B_SFULL + buf, (uint32_t)(g >> 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float4* s4 = reinterpret_cast<const float4*>(sm + OFF_PL + sc * PL_BYTES) + sub * 32 + i4;
          const float2* g2 = reinterpret_cast<const float2*>(sm + OFF_PL + sc * PL_BYTES + 1024) + sub * 32 + i4;
          const bool here = (facts[sc] >> sub) & 1u;
          uint32_t u[32];    // S_L, then u = sLc S_L + sRc S_R, as pairs of tokens
          {
            const uint32_t tl = tmem + lane_addr + ((uint32_t)(16 * hl) << 16) + T_SL + buf * TILE + sub * SUB;
            const uint32_t tr = tmem + lane_addr + ((uint32_t)(16 * hl) << 16) + T_SR + sub * SUB;
            tmem_ld_16x32(tl, u);
            tmem_ld_16x32(tl + 32, u + 16);
#pragma unroll
            for (int jh = 0; jh < 2; ++jh) {
              uint32_t rr[16];
              tmem_ld_16x32(tr + 32 * jh, rr);
              tmem_wait_ld();
              if (jh == 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster_relaxed(map_to(smem_u32(&bars[B_SEMPTY + buf]), 0));
              }
#pragma unroll
              for (int j4 = 0; j4 < 4; ++j4) {
                const int j = 4 * jh + j4;
                const float4 s = s4[4 * j];
                const uint64_t sl = pk2(s.x, s.y), sr = pk2(s.z, s.w);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  uint32_t* w2 = &u[4 * j + e];
                  const float2 f = up2(fma2(sr, pk2(__uint_as_float(rr[4 * j4 + e]), __uint_as_float(rr[4 * j4 + e + 1])),
                                            mul2(sl, pk2(__uint_as_float(w2[0]), __uint_as_float(w2[1])))));
                  w2[0] = __float_as_uint(f.x);
                  w2[1] = __float_as_uint(f.y);
                }
              }
            }
          }
          auto pair = [&](int p, int j) -> uint64_t {
            return pk2(__uint_as_float(u[4 * j + 2 * p]), __uint_as_float(u[4 * j + 2 * p + 1]));
          };
          if (!here || first - t0 < SUB) {  // some row does not see all of this page
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int n = here ? lim[rh + 8 * p] - t0 - 2 * i4 : 0;
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * j + e >= n) u[4 * j + 2 * p + e] = 0xFF800000u;  // -inf
            }
          }
          // the largest weight of row `mh` over the page: the two rows' over this thread's
          // tokens, then over the four lanes
          float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = g2[4 * j];
            const uint64_t lg = pk2(f.x, f.y);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float2 v = up2(fma2(c2[p], pair(p, j), lg));
              y[p] = max3(y[p], v.x, v.y);
            }
          }
          const bool b0 = i4 & 1;
          float ym = fmaxf(b0 ? y[1] : y[0], __shfl_xor_sync(0xffffffffu, b0 ? y[0] : y[1], 1));
          ym = fmaxf(ym, __shfl_xor_sync(0xffffffffu, ym, 2));
          // its reference there, and the factor of the l added up before
          float mn = mg;
          if (ym > mg + TAU) {
            mn = ym;
          } else if (ym < mg - DOWN && ym >= mhi - DOWN_CAP) {
            mn = ym;
          }
          const float f = mn == mg ? 1.f : (mg > -INFINITY ? ex2_approx(mg - mn) : 0.f);
          mg = mn;
          mhi = fmaxf(mhi, mn);
          if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
            for (int p = 0; p < 2; ++p) l[p] *= __shfl_sync(0xffffffffu, f, (lane & 28) + p);
          }
          const uint32_t to = map_to(smem_u32(sm + OFF_P + buf * P_STRIDE), rank + 2);
          const uint32_t bar = map_to(smem_u32(&bars[B_PFULL + buf]), rank + 2);
          if (i4 < 2) st_async_b32(to + P_F + (sub * CROWS + mh) * 4, __float_as_uint(mn), bar);
          if (warp == W_LANE && lane == 0) st_async_b32(to + P_PAGES, facts[sc], bar);
          // p = 2^(c u - M_g + 7) (nothing in sight so far: u is -inf, and p 0)
          const float mneg = P_LOG - fmaxf(mn, -3.0e38f);
          uint64_t m2[2], ls2[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float mp = __shfl_sync(0xffffffffu, mneg, (lane & 28) + p);
            m2[p] = pk2(mp, mp);
            ls2[p] = pk2(0.f, 0.f);
          }
          const uint32_t dst = to + prow(rh, sub * 8 + i4);
#pragma unroll
          for (int jh = 0; jh < 2; ++jh) {
            uint32_t h[2][4];
#pragma unroll
            for (int j4 = 0; j4 < 4; ++j4) {
              const int j = 4 * jh + j4;
              const float2 s = *reinterpret_cast<const float2*>(s4 + 4 * j);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const float2 z = up2(fma2(c2[p], pair(p, j), m2[p]));
                const uint64_t e = pk2(ex2_approx(z.x), ex2_approx(z.y));
                ls2[p] = add2(ls2[p], e);
                const float2 t2 = up2(mul2(e, pk2(s.x, s.y)));
                const __half2 h2 = __floats2half2_rn(t2.x, t2.y);
                h[p][j4] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            }
            // (unit sub * 8 + 4 jh + i4 of row rh + 8 p: 4 jh turns bit 2 of the swizzled unit)
#pragma unroll
            for (int p = 0; p < 2; ++p)
              st_async_v4((dst ^ (uint32_t)(jh * 64)) + p * 2048, make_uint4(h[p][0], h[p][1], h[p][2], h[p][3]), bar);
          }
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 s = up2(ls2[p]);
            l[p] += s.x + s.y;
          }
        }
        if (!ok) break;
        // ---- the row tile's (or its part's) end: the eight threads of a row add their l
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          l[p] += __shfl_xor_sync(0xffffffffu, l[p], 1);
          l[p] += __shfl_xor_sync(0xffffffffu, l[p], 2);
        }
        if (i4 < 2) {
          xl[mh * 2 + sub] = i4 ? l[1] : l[0];
          mgs[mh * 2 + sub] = mg;
        }
        if (!quarter_sync()) {
          ok = false;
          break;
        }
        if (part == 0) {  // a row per lane
          const int hh = q * 32 + lane;
          // on the scale 2^(7 - the larger reference)
          const float m0 = mgs[hh * 2], m1 = mgs[hh * 2 + 1], mm = fmaxf(m0, m1), M = mm - P_LOG;
          const float L = xl[hh * 2] * (m0 == mm ? 1.f : ex2_approx(m0 - mm)) +
                          xl[hh * 2 + 1] * (m1 == mm ? 1.f : ex2_approx(m1 - mm));
          float f = 1.f;
          if (x.whole()) {
            f = L == 0.f ? 0.f : 1.f / L;  // (a NaN stays one)
            const int64_t r = (int64_t)x.rt * ROWS + rank * CROWS + hh;
            if (a.lse != nullptr && r < (int64_t)x.s.nq * a.H)
              a.lse[x.s.q0 * a.H + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
          } else {
            const int64_t at = (int64_t)(2 * k + (x.seg == 0 ? 0 : 1)) * ROWS + rank * CROWS + hh;
            ws.m[at] = M;
            ws.l[at] = L;
          }
          const int rf = x.seg % NRF;
          const uint32_t to = map_to(smem_u32(sm + OFF_RF + (rf * CROWS + hh) * 8), rank + 2);
          const uint32_t bar = map_to(smem_u32(&bars[B_RF + rf]), rank + 2);
          st_async_b32(to, __float_as_uint(f), bar);
          st_async_b32(to + 4, __float_as_uint(mm), bar);
        }
        gt += n_tiles;
        Walk wn = x;
        wn.next(a);
        more = wn.more();
        __syncwarp();
        *walk = wn;
        __syncwarp();
      }
      if (!ok && lane == 0) fail();
      // the context CTAs' last arrivals at this CTA have landed
      if (ok && gt > 0) {
        const int zero = 0;
        for (int i = gt > 2 ? gt - 2 : 0; i < gt; ++i)
          (void)mbar_wait(&bars[B_PFREE + (i & 1)], (i >> 1) & 1, &zero, WAIT_NS);
      }
      __syncwarp();
    }
  } else {
    // ================================================================ context CTAs
    const uint32_t pbuf = smem_u32(sm + OFF_P);
    const uint32_t vring = smem_u32(sm + OFF_V);
    const int half_of = (int)rank - 2;  // channels 256 h + 128 half_of .. of each O half h
    if (warp == W_TMA) {
      bool ok = true;
      int nv = 0;
      for (; ok && w.more(); w.next(a)) {
        PageWindow pw;
        pw.from = -64;
        for (int i = 0; i < w.n; ++i) {
          const int g = gt + i, vs = g % NVT;
          const int64_t page = 2 * (int64_t)(w.t + i);
          const int64_t s0 = pw.slot(a, w, page, lane, false), s1 = pw.slot(a, w, page + 1, lane, false);
          if (!wait(B_VEMPTY + vs, (uint32_t)(g / NVT) ^ 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx_warp(&bars[B_VT + vs], 2u * BLK * ((s0 >= 0 ? 1u : 0u) + (s1 >= 0 ? 1u : 0u)));
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t dst = vring + vs * VTILE + h * VBLK;
            const int x = 256 * h + 128 * half_of;
            if (s0 >= 0) tma_load_2d_warp(dst, &kmap, x, (int)s0, &bars[B_VT + vs]);
            if (s1 >= 0) tma_load_2d_warp(dst + BLK, &kmap, x, (int)s1, &bars[B_VT + vs]);
          }
          nv = g + 1;
        }
        gt += w.n;
      }
      if (!ok) {
        if (lane == 0) fail();
        const int zero = 0;
        for (int i = (nv > NVT ? nv - NVT : 0); i < nv; ++i)
          (void)mbar_wait(&bars[B_VT + i % NVT], (i / NVT) & 1, &zero, WAIT_NS);
      }
      __syncwarp();
    } else if (warp == W_SCALE) {
      // (no scales here: this warp tells the score CTA which payloads are read, so that its writes of
      // the next ones come after those reads)
      const uint32_t pfree = map_to(smem_u32(&bars[B_PFREE]), rank - 2);
      bool ok = true;
      for (int64_t g = 0; ok && g < w.left; ++g)
        ok = relay(B_PFREE + (int)(g & 1), (uint32_t)(g >> 1), pfree + (int)(g & 1) * 8);
      if (!ok && lane == 0) fail();
      __syncwarp();
    } else if (warp == W_MMA) {
      if (rank == 2) {
        const uint32_t id = idesc_f16(ROWS, 256, false, true);  // A K-major, B = V MN-major
        const uint64_t pd = smem_desc(smem_u32(sm + OFF_OP), 16, 1024, SW128);
        const uint64_t vd = smem_desc(vring, 16, 1024, SW128);
        bool ok = true;
        for (; ok && w.more(); w.next(a)) {
          for (int i = 0; ok && i < w.n; ++i) {
            const int g = gt + i;
            const uint64_t ad = pd + (uint64_t)((g & 1) * 2 * OP_ATOM >> 4);
            if (!wait(B_VT + g % NVT, (uint32_t)(g / NVT)) || !wait_cluster(B_OP + (g & 1), (uint32_t)(g >> 1))) {
              ok = false;
              break;
            }
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!wait_cluster(B_RS + 2 * (g & 1) + h, (uint32_t)(g >> 1))) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t bd = vd + (uint64_t)(((g % NVT) * VTILE + h * VBLK) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                // A: 32 tokens of the hi / lo atom; B: 32 token rows (4 KB)
                mma_f8_pair_warp(tmem + h * 256, ad + 2 * kk, bd + 256 * kk, id, (i > 0 || kk > 0) ? 1u : 0u);
                mma_f8_pair_warp(tmem + h * 256, ad + (OP_ATOM >> 4) + 2 * kk, bd + 256 * kk, id, 1u);
              }
              mma_commit_pair_warp(&bars[B_ODONE + 2 * (g & 1) + h], 0xC);
            }
            if (!ok) break;
            mma_commit_pair_warp(&bars[B_VEMPTY + g % NVT], 0xC);
          }
          gt += w.n;
        }
        if (!ok && lane == 0) fail();
        mma_commit_pair_warp(&bars[B_DRAIN], 0xC);
      } else {
        // rank 3 tells the MMA's issuer of its V tiles and operands
        const uint32_t op = map_to(smem_u32(&bars[B_OP]), 2);
        bool ok = true;
        for (int64_t g = 0; ok && g < w.left; ++g) {
          ok = wait(B_VT + (int)(g % NVT), (uint32_t)(g / NVT));
          ok = ok && relay(B_OP + (int)(g & 1), (uint32_t)(g >> 1), op + (int)(g & 1) * 8);
        }
        if (!ok && lane == 0) fail();
      }
      const int zero = 0;
      (void)mbar_wait(&bars[B_DRAIN], 0, &zero, 4 * WAIT_NS);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- operand, O rescale, results
      const int q = warp & 3;
      const int part = (warp - W_LANE) >> 2;  // 32 tokens of the tile; 64 columns of an O half
      const int hh = q * 32 + lane;
      const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
      const uint32_t rs = map_to(smem_u32(&bars[B_RS]), 2);
      bool ok = true;
      for (; ok && w.more(); w.next(a)) {
        const int lim0 = limit_of(a, w.s, (int)((uint32_t)(w.rt * ROWS) / (uint32_t)a.H));  // the tile's first row sees least
        float ref = -INFINITY, hi = -INFINITY;  // the row's reference in O, and the highest one so far
        for (int i = 0; i < w.n; ++i) {
          const int g = gt + i, pb = g & 1, vs = g % NVT;
          if (!wait_cluster(B_PFULL + pb, (uint32_t)(g >> 1))) {
            ok = false;
            break;
          }
          const uint32_t src = pbuf + pb * P_STRIDE;
          uint32_t pv[4][4];  // [i][j]: tokens 8 j + 2 i, + 1 of the part
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 v = lds128(src + prow(hh, part * 4 + u));
            pv[u][0] = v.x;
            pv[u][1] = v.y;
            pv[u][2] = v.z;
            pv[u][3] = v.w;
          }
          const float m0 = reinterpret_cast<const float*>(sm + OFF_P + pb * P_STRIDE + P_F)[hh];
          const float m1 = reinterpret_cast<const float*>(sm + OFF_P + pb * P_STRIDE + P_F)[CROWS + hh];
          const uint32_t pages = *reinterpret_cast<const uint32_t*>(sm + OFF_P + pb * P_STRIDE + P_PAGES);
          // the payload is read: the next one may be expected, and then come
          __syncwarp();
          if (lane == 0) {
            if (warp == W_LANE) mbar_arrive_expect_tx(&bars[B_PFULL + pb], P_BYTES);
            mbar_arrive(&bars[B_PFREE + pb]);
          }
          // O's reference is the larger of the pages', or above both: the factor of what was added up
          // before, and the one that brings this warp's page onto it
          const float top = fmaxf(m0, m1), own = part < 2 ? m0 : m1, was = ref;
          if (top > ref) {
            ref = top;
          } else if (top < ref - DOWN && top >= hi - DOWN_CAP) {
            ref = top;
          }
          hi = fmaxf(hi, ref);
          const float f = ref == was ? 1.f : (was > -INFINITY ? ex2_approx(was - ref) : 0.f);
          const bool any = __any_sync(0xffffffffu, f != 1.f) && i > 0;
          const __half2 onto = __float2half2_rn(own == ref ? 1.f : ex2_approx(own - ref));
          // the operand buffer was read by the MMAs of tile g - 2 (at a row tile's start they were
          // waited for with its predecessor's results)
          if (i > 1 && !wait(B_ODONE + 2 * pb + 1, (uint32_t)((g >> 1) - 1))) {
            ok = false;
            break;
          }
          const uint32_t opnd = smem_u32(sm + OFF_OP) + pb * 2 * OP_ATOM;
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 16 tokens per 16-byte unit
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {  // tokens 16 j + 4 v .. + 3
              uint16_t h0, l0, h1, l1;
              split_h2(scaled_h2(pv[2 * (v & 1)][2 * j + (v >> 1)], onto), h0, l0);
              split_h2(scaled_h2(pv[2 * (v & 1) + 1][2 * j + (v >> 1)], onto), h1, l1);
              hw[v] = (uint32_t)h0 | ((uint32_t)h1 << 16);
              lw[v] = (uint32_t)l0 | ((uint32_t)l1 << 16);
            }
            const uint32_t off = sw128(hh, part * 2 + j);
            sts128(opnd + off, make_uint4(hw[0], hw[1], hw[2], hw[3]));
            sts128(opnd + OP_ATOM + off, make_uint4(lw[0], lw[1], lw[2], lw[3]));
          }
          if (w.t + i + 1 > lim0 / TILE || pages != 3u) {
            // some row does not see all of this tile: no NaN code may stay in it
            if (!wait(B_VT + vs, (uint32_t)(g / NVT))) {
              ok = false;
              break;
            }
            const uint32_t vb = vring + vs * VTILE + (warp - W_LANE) * 2048 + lane * 16;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 v = lds128(vb + u * 512);
              sts128(vb + u * 512, make_uint4(no_nan(v.x), no_nan(v.y), no_nan(v.z), no_nan(v.w)));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_OP + pb]);
          // rows whose reference moved are rescaled: one half of O after the other, each when the
          // previous tile's MMAs on it are done (the first half while those on the second run)
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (any) {
              if (!wait(B_ODONE + 2 * (pb ^ 1) + h, (uint32_t)((g - 1) >> 1))) {
                ok = false;
                break;
              }
              tc_fence_after();
              __syncwarp();
              const uint32_t col = tmem + lane_addr + h * 256 + part * 64;
#pragma unroll 1
              for (int s = 0; s < 64; s += 32) {
                uint32_t o[32];
                tmem_ld32(col + s, o);
                tmem_wait_ld();
#pragma unroll
                for (int v = 0; v < 32; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * f);
                tmem_st32(col + s, o);
              }
              __syncwarp();
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
            }
            if (lane == 0) arrive_cluster_relaxed(rs + (2 * pb + h) * 8);
          }
          if (!ok) break;
        }
        if (!ok) break;
        const int last = gt + w.n - 1;
        gt += w.n;
        const int rf = w.seg % NRF;
        if (!wait(B_ODONE + 2 * (last & 1) + 1, (uint32_t)(last >> 1)) ||
            !wait_cluster(B_RF + rf, (uint32_t)(w.seg / NRF))) {
          ok = false;
          break;
        }
        tc_fence_after();
        __syncwarp();
        const float2 f2 = reinterpret_cast<const float2*>(sm + OFF_RF + rf * CROWS * 8)[hh];
        const float f = f2.x, up = ref == f2.y ? 1.f : ex2_approx(ref - f2.y);  // (O onto the reference of l)
        // 64 bytes of every row at a time (32 columns of bf16, or 16 of a partial's f32) through
        // shared memory, so that a warp's stores write whole sectors: eight rows each
        const bool whole = w.whole();
        const int64_t r0 = (int64_t)w.rt * ROWS + half_of * CROWS + q * 32;  // the warp's first row
        const int64_t rows = (int64_t)w.s.nq * a.H - r0;
        const int left = (int)(rows < 32 ? rows : 32) - (lane >> 2);         // rows from this lane's first on, by eights
        const uint32_t stage = smem_u32(sm + OFF_OP) + (warp - W_LANE) * 2048;
        const uint32_t put = stage + lane * 64, sw = (lane >> 1) & 3;        // this lane's row, its units turned by sw
        const uint32_t take = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
        const int row_bytes = whole ? DL * 2 : DL * 4;
        uint8_t* dst = (whole ? reinterpret_cast<uint8_t*>(a.out + (w.s.q0 * a.H + r0) * DL)
                              : reinterpret_cast<uint8_t*>(
                                    ws.o + ((int64_t)(2 * k + (w.seg == 0 ? 0 : 1)) * ROWS + half_of * CROWS + q * 32) * DL)) +
                       (lane >> 2) * row_bytes + (lane & 3) * 16;
        auto flush = [&](int byte) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = lds128(take + i * 512);  // (eight rows on, the turn is the same)
            if (8 * i < left) *reinterpret_cast<uint4*>(dst + 8 * i * row_bytes + byte) = v;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int s = 0; s < 128; s += 16) {  // 16 columns at a time
          const int col = (s >> 6) * 256 + part * 64 + (s & 63);
          uint32_t v[16];
          tmem_ld16(tmem + lane_addr + col, v);
          tmem_wait_ld();
          // (a factor of 0: nothing seen, or nothing that counts)
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = f == 0.f ? 0u : __float_as_uint(__uint_as_float(v[j]) * up * f);
          if (whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
              v[j] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            const uint32_t u0 = (s >> 3) & 2;  // the row's first or last two units
            sts128(put + ((u0 ^ sw) << 4), make_uint4(v[0], v[1], v[2], v[3]));
            sts128(put + (((u0 + 1) ^ sw) << 4), make_uint4(v[4], v[5], v[6], v[7]));
            if (s & 16) flush((col - 16) * 2);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              sts128(put + ((u ^ sw) << 4), make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]));
            flush(col * 4);
          }
        }
        tc_fence_before();  // (the loads from O, before the next row tile's MMAs)
        // the factor buffer's next phase, NRF segments on (its bytes come after the payloads of
        // the tiles between, which every warp has to read); and the operand buffers may be
        // written again when every warp's results have left them
        __syncwarp();
        if (lane == 0) {
          if (warp == W_LANE) mbar_arrive_expect_tx(&bars[B_RF + rf], CROWS * 8);
          mbar_arrive(&bars[B_EP]);
        }
        if (!wait(B_EP, (uint32_t)w.seg)) {
          ok = false;
          break;
        }
      }
      if (!ok && lane == 0) fail();
      __syncwarp();
    }
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  tc_fence_before();
  cluster_sync();  // no CTA leaves while another may still write to it
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc_pair(tmem, 512);
}

// Joins the parts of the row tiles that range borders cut: for every cluster k but the
// first, the row tile that it starts in, if cluster k - 1 holds its beginning; a warp per
// row, or per row and SPLIT-th of its channels.  In four parts a single row tile in many
// parts is read by 128 SMs in place of 32 (one token over 8192 keys at 128 heads: 47.0
// against 55.6 us); where most clusters hold a border the blocks that gives cost more
// than that (32 x 4 tokens over up to 16384 keys: 241 against 236 us).
constexpr int JOIN_BLOCKS = ROWS / 8;
constexpr int FEW_ROW_TILES = 8;

template <int SPLIT>
__global__ void __launch_bounds__(256) join_kernel(const ChunkArgs a, const Workspace ws) {
  static_assert(MAX_CLUSTERS <= 64, "two parts a lane");
  const int k = (int)blockIdx.x / (JOIN_BLOCKS * SPLIT) + 1, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x % (JOIN_BLOCKS * SPLIT) / SPLIT * 8 + (threadIdx.x >> 5);
  const int ch = (int)blockIdx.x % SPLIT * (DL / SPLIT);
  // (every block waits, with a row or without: the plan's and the parts' visibility, and that this
  // launch is not over before the chunk kernel is, come with the wait)
  grid_dependency_wait();
  const int64_t nc = ws.plan->n_clusters;
  if (k >= nc) return;
  __shared__ int64_t xs[MAX_CLUSTERS + 1];    // the units where the ranges begin
  if (threadIdx.x <= nc) xs[threadIdx.x] = threadIdx.x < nc ? ws.plan->e[threadIdx.x].x : ws.plan->units;
  const PlanEntry e = ws.plan->e[k];
  __syncthreads();
  const int64_t S = e.x - e.off;              // the row tile's first unit
  const int64_t xp = xs[k - 1];
  const SeqInfo s = seq_info(a, e.b, false);
  const int64_t r = (int64_t)e.rt * ROWS + row;
  // (not whole, nor begun before cluster k - 1)
  const bool mine = e.off != 0 && xp <= S && r < (int64_t)s.nq * a.H;
  auto part = [&](int j) -> int64_t {         // slot of cluster j's part
    return (int64_t)(2 * j + (j == k - 1 && xp < S ? 1 : 0)) * ROWS + row;
  };
  int last = k;
  while (last + 1 < nc && xs[last + 1] < S + e.nt) ++last;
  if (!mine) return;
  // a lane per part: its reference, its sum (a cluster without units has no part); at most
  // MAX_CLUSTERS of them, so two each
  float m[2], wt[2], M = -INFINITY, L = 0.f;
  bool there[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = k - 1 + lane + 32 * h;
    there[h] = j <= last && xs[j] != xs[j + 1];
    m[h] = there[h] ? ws.m[part(j)] : -INFINITY;
    wt[h] = there[h] ? ws.l[part(j)] : 0.f;
    M = fmaxf(M, m[h]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  uint32_t has[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float l = wt[h];
    wt[h] = m[h] > -INFINITY ? ex2_approx(m[h] - M) : 1.f;  // (a NaN l stays one)
    L += wt[h] * l;
    has[h] = __ballot_sync(0xffffffffu, there[h]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  constexpr int N = 4 / SPLIT;  // 16-byte units a lane
  float4 acc[N];
#pragma unroll
  for (int c = 0; c < N; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = min(last - (k - 1) + 1 - 32 * h, 32);
#pragma unroll(SPLIT == 1 ? 4 : 8)
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, wt[h], i);
      const float4* o = reinterpret_cast<const float4*>(ws.o + part(k - 1 + 32 * h + i) * DL + ch) + lane;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float4 v = ((has[h] >> i) & 1u) ? o[32 * c] : make_float4(0.f, 0.f, 0.f, 0.f);
        acc[c].x += w * v.x;
        acc[c].y += w * v.y;
        acc[c].z += w * v.z;
        acc[c].w += w * v.w;
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = s.q0 * a.H + r;
  uint2* out = reinterpret_cast<uint2*>(a.out + at * DL + ch) + lane;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    out[32 * c] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (ch != 0) return;
  if (a.lse != nullptr && lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
}

constexpr int64_t OFF_PLAN = 256, OFF_BASE = 2048;
static_assert(OFF_PLAN + sizeof(Plan) <= OFF_BASE, "plan area");

int64_t most_row_tiles(int B, int H, int64_t total_q) { return total_q * H / ROWS + B; }

// Clusters that a call of these sizes can use, whatever the lengths turn out to be.
int most_clusters(int B, int H, int64_t total_q, int max_blocks) {
  const int64_t keys = ((int64_t)max_blocks * PAGE + TILE - 1) / TILE;
  const int64_t tiles = most_row_tiles(B, H, total_q), units = tiles * (keys > MIN_TILES ? keys : MIN_TILES) / MIN_TILES;
  return (int)(units < 1 ? 1 : (units < MAX_CLUSTERS ? units : MAX_CLUSTERS));
}

int64_t base_bytes(int B) { return ((int64_t)(B + 1) * 8 + 255) / 256 * 256; }

}  // namespace

int64_t chunk_workspace(int B, int H, int64_t total_q, int max_blocks) {
  const int64_t most = most_clusters(B, H, total_q, max_blocks), rows = most > 1 ? 2 * most * ROWS : 0;  // (one cuts no row tile)
  return OFF_BASE + base_bytes(B) + rows * (8 + DL * 4);
}

cudaError_t launch_chunk(ChunkArgs a, void* workspace, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  int fit = 0;  // clusters that the device holds at once
  cudaError_t e = per_device(memo, [](int* v) {
    cudaError_t r = cudaFuncSetAttribute(chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(NUM_SMS, 1, 1);
    cfg.blockDim = dim3(NTHREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    int n = 0;
    r = cudaOccupancyMaxActiveClusters(&n, chunk_kernel, &cfg);
    if (r != cudaSuccess) return r;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    *v = n > MAX_CLUSTERS ? MAX_CLUSTERS : n;
    return cudaSuccess;
  }, &fit);
  if (e != cudaSuccess) return e;
  const int most = most_clusters(a.B, a.H, a.total_q, a.max_blocks);
  const int clusters = most < fit ? most : fit;
  char* p = static_cast<char*>(workspace);
  a.err = reinterpret_cast<unsigned*>(p);
  Workspace ws;
  ws.plan = reinterpret_cast<Plan*>(p + OFF_PLAN);
  int64_t* base = reinterpret_cast<int64_t*>(p + OFF_BASE);
  ws.m = reinterpret_cast<float*>(p + OFF_BASE + base_bytes(a.B));
  ws.l = ws.m + 2 * most * ROWS;
  ws.o = ws.l + 2 * most * ROWS;
  DecodeArgs d{};  // what the cache's tensor maps are made from
  d.codes = a.codes;
  d.scales = a.scales;
  d.block_table = a.block_table;
  d.n_blocks = a.n_blocks;
  CUtensorMap kmap, rmap, smap;
  if ((e = make_cache_map(d, &kmap)) != cudaSuccess || (e = make_rc_map(d, &rmap)) != cudaSuccess ||
      (e = make_scale_map(d, &smap)) != cudaSuccess)
    return e;
  plan_kernel<<<1, 1024, 0, s>>>(a, ws.plan, base, clusters);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after_prep(chunk_kernel, 4 * clusters, NTHREADS, SMEM, s, a, ws, kmap, rmap, smap);
  if (e != cudaSuccess || clusters == 1) return e;
  const unsigned blocks = JOIN_BLOCKS * (clusters - 1);
  if (most_row_tiles(a.B, a.H, a.total_q) < FEW_ROW_TILES)
    return launch_after_prep(join_kernel<4>, 4 * blocks, 256, 0, s, a, ws);
  return launch_after_prep(join_kernel<1>, blocks, 256, 0, s, a, ws);
}

}  // namespace kv8
