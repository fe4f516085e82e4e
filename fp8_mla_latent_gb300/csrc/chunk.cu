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
// With a window (kWindow) a token sees t <= p with t > p - window or t < n_sink.  A row tile's pages are then those
// of the first tokens, and from the one on in which its first row's window begins: the gap between them is
// left out of the order in which pages are walked (chunk_work.cuh, Pages), so that a key tile is any two pages, and
// the plan counts what is walked.  Only row tiles on a window's or the prompt's edge take the masked path.
//
// With shared prefixes (kShared) the plan's sequences are entries: each group's prefix, whose rows are
// those of all its sequences, and each sequence's rest.  Either leaves f32 parts, which a join adds up
// with those that range borders cut (join_parts; one read of 16384 keys for 32 tokens of 128 heads in place of 32).
//
// For 65 to 128 rows a sequence (SOLO) a cluster is two CTAs, one for the scores and one for the context, with
// M = 128 and cta_group::1: half of a pair's rows would be copies.  B is not shared then, so that an MMA reads as
// many bytes for half the rows: shared memory bounds it, about 4800 cycles a tile.  K is a ring of seven Lc blocks.
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
// 16384 keys 0.235 ms, 1060, 0.56; one token of 4 heads over 256 keys 19.0 us, of which 3 are the plan,
// 5 the query, 5 the pipeline and 5 the results.  With a window of 2048 a later chunk of 4096 tokens 2.25 ms,
// 1105 TFLOP/s, 0.57 (a row tile begins every 17 key tiles); 24 x up to 61 tokens of 20 heads, window 1111, 74 us,
// 0.23 (72 row tiles of 11 key tiles: 11 us to a cluster's first weights, 5 for each f32 part's results); clusters of two:
// 32 tokens of 128 heads, window 2048, 46.6 us, 0.20 (7 tiles a cluster, the same starts and ends), 64 with
// a window of 8192 156 us, 0.48.  32 tokens of 128 heads behind a shared prefix of 32768 keys 234 us, 0.65.
//
// Every wait is bounded (2 s): on a timeout
// the CTA flags the workspace error word, drains its MMAs and copies and meets its cluster
// at the closing barrier.
#include <cuda.h>

#include "chunk_work.cuh"

namespace kv8 {
namespace {

constexpr int ROWS = WideGeo::ROWS;           // rows of a row tile: 128 per CTA of a pair
constexpr int CROWS = 128;
constexpr int W_TMA = 0, W_MMA = 1, W_SCALE = 2, W_LANE = 3;
constexpr int N_LANE_WARPS = 16;             // four per TMEM lane quarter, and per scheduler
constexpr int NTHREADS = (W_LANE + N_LANE_WARPS) * 32;
constexpr int MAX_CLUSTERS = WideGeo::RANGES, MIN_TILES = WideGeo::MIN_TILES;
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
constexpr int B_RFULL = B_DRAIN + 1;         // solo score: Rc block loaded
constexpr int B_REMPTY = B_RFULL + 1;        // solo score: consumed
constexpr int B_SFREE = B_REMPTY + 1;        // [NKB] solo score: Lc block consumed
constexpr int B_SFILL = B_KFULL;             // [NKB] solo score: loaded (in place of the halves' barriers)
constexpr int NBAR = B_SFREE + 7;

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
// Solo (one score and one context CTA): K as a ring of Lc blocks [128 tokens x 128 bytes] and an Rc block behind
// it, V as the tile's two halves of 256 channels, each in a place of its own.
constexpr int KBLK = 2 * BLK, NKB = 7;
static_assert(NKB <= 7 && NKB <= 4 * NK, "their barriers");
constexpr int OFF_KR = OFF_K + NKB * KBLK;
constexpr int TOTAL_SOLO_S = OFF_KR + 2 * RBLK, TOTAL_SOLO_C = OFF_V + 4 * VBLK;
constexpr int SMEM_SOLO = TOTAL_SOLO_S > TOTAL_SOLO_C ? TOTAL_SOLO_S : TOTAL_SOLO_C;
static_assert(SMEM_SOLO <= 232448 && OFF_KR % 1024 == 0, "shared memory above the per-CTA limit");
// TMEM columns of a score CTA
constexpr int T_SL = 0, T_SR = 256, T_QH = 384;
static_assert(NSC >= NK + 2 && NSC <= 8 && NVT <= 8 && OFF_FACTS + 32 <= OFF_XL, "rings");
static_assert(NBAR * 8 <= OFF_FLAGS && OFF_RF + NRF * CROWS * 8 <= OFF_P, "shared memory layout");
static_assert(OFF_K % 1024 == 0 && KTILE % 1024 == 0 && OFF_V % 1024 == 0 && P_STRIDE % 1024 == 0, "swizzle atoms");
static_assert(P_BYTES <= P_STRIDE && N_LANE_WARPS * 2048 <= 4 * OP_ATOM, "payload and staging");
static_assert(SMEM <= 232448, "shared memory above the per-CTA limit");

// The cluster of two CTAs is for sequences of 65 to 128 rows, whose row tiles are half of the others'.  (Single tokens
// of 128 heads, us, SWITCH 4, 6 and 8: 32 with a window of 2048 46.0, 46.8, 48.5; 64 with 512 44.0, 43.2, 41.9;
// 64 ragged with 2048 67.4, 66.6, 65.1; 200 ragged with 1000 100.5, 102.6, 104.9.)
struct SoloGeo {
  static constexpr int ROWS = CROWS, RANGES = NUM_SMS / 2, MIN_TILES = 2, SWITCH = 6;
};
template <bool SOLO>
using GeoOf = typename std::conditional<SOLO, SoloGeo, WideGeo>::type;
using Geo = WideGeo;
template <int MODE, bool SOLO = false>
using Way = Walk<MODE, GeoOf<SOLO>>;
static_assert(sizeof(Way<kShared>) * N_LANE_WARPS <= OFF_SC - OFF_WALK && sizeof(Way<kWindow>) <= sizeof(Way<kShared>),
              "segments");

constexpr int PLAN_NEAR = 4096;

// (base: in shared memory if it fits, and for a shared call, whose join reads it, in the workspace as well)
template <int MODE>
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const ChunkArgs a, Plan<Geo>* plan, int64_t* base, int clusters) {
  grid_dependents_launch();
  __shared__ PlanScratch scratch;
  PlanSum sums{scratch};
  __shared__ int64_t near[PLAN_NEAR];
  const int n_seq = MODE == kShared ? a.G + a.B : a.B;
  plan_prefetch(a);
  if (threadIdx.x == 0) *a.err = 0;
  __syncthreads();
  bool turns = false;
  if constexpr (MODE == kShared) (void)make_entries<Geo>(a, &plan->part_rows, sums, true, &turns);
  make_plan<MODE>(a, plan, n_seq < PLAN_NEAR ? near : base, MODE == kShared && n_seq < PLAN_NEAR ? base : nullptr, 0, 0,
                  n_seq, clusters, sums, MODE == kShared ? a.unit : nullptr, nullptr, false, turns);
}
__global__ void __launch_bounds__(PLAN_THREADS) solo_plan_kernel(const ChunkArgs a, Plan<SoloGeo>* plan, int64_t* base,
                                                         int4* owner, int clusters) {
  grid_dependents_launch();
  __shared__ PlanScratch scratch;
  PlanSum sums{scratch};
  __shared__ int64_t near[PLAN_NEAR];
  plan_prefetch(a);
  if (threadIdx.x == 0) *a.err = 0;
  __syncthreads();
  make_plan<kWindow>(a, plan, a.B < PLAN_NEAR ? near : base, nullptr, 0, 0, a.B, clusters, sums, nullptr, owner);
}

// byte offset of 16-byte unit u (0..15) of row r in a payload: unit 4 s + i holds tokens
// 32 s + 8 j + 2 i, + 1 for j = 0 .. 3
__device__ __forceinline__ uint32_t prow(int r, int u) {
  return (uint32_t)(r * 256 + ((u ^ (r & 7)) << 4));
}

template <bool SOLO = false>
struct Workspace {
  static constexpr int ROWS = GeoOf<SOLO>::ROWS;
  Plan<GeoOf<SOLO>>* plan;
  float* m;   // [2 MAX_CLUSTERS][256]: slot 2k the first segment of cluster k, 2k + 1 its last
  float* l;
  float* o;   // [..][256][512]
  int64_t parts;  // (shared prefixes) behind the slots: the parts of row tiles that one cluster held whole
  // where the parts of row `row` of a row tile go, as a row of these arrays
  template <int MODE>
  __device__ __forceinline__ int64_t part_row(const Way<MODE, SOLO>& w, int k, int row) const {
    if constexpr (MODE == kShared) {
      if (w.whole()) return parts + w.s.part + (int64_t)w.rt * ROWS + row;
    }
    return (int64_t)(2 * k + (w.seg == 0 ? 0 : 1)) * ROWS + row;
  }
};

template <int MODE, bool SOLO = false>
__global__ void __cluster_dims__(SOLO ? 2 : 4, 1, 1) __launch_bounds__(NTHREADS, 1)
    chunk_kernel(const ChunkArgs a, const Workspace<SOLO> ws, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap smap) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // score CTAs (the context ones come behind them), rows of a row tile, and the MMAs of a pair or of this CTA
  constexpr int SC = SOLO ? 1 : 2, ROWS = SC * CROWS;
  const uint32_t rank = cluster_rank();
  const int k = (int)(blockIdx.x / (2 * SC));
  auto mma = [](uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t acc) {
    if constexpr (SOLO) mma_f8_warp(d, ad, bd, id, acc);
    else mma_f8_pair_warp(d, ad, bd, id, acc);
  };
  auto mma_ts = [](uint32_t d, uint32_t at, uint64_t bd, uint32_t id, uint32_t acc) {
    if constexpr (SOLO) mma_f8_ts_warp(d, at, bd, id, acc);
    else mma_f8_ts_pair_warp(d, at, bd, id, acc);
  };
  auto commit = [](uint64_t* bar, uint16_t mask) {  // (mask: the pair's CTAs)
    if constexpr (SOLO) mma_commit_warp(bar);
    else mma_commit_pair_warp(bar, mask);
  };
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
    const int here = N_LANE_WARPS + (!SOLO && (rank == 0 || rank == 2));  // (and the relay of the pair's other CTA)
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_SEMPTY + i], SC * N_LANE_WARPS);
    mbar_init(&bars[B_QREADY], here);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[B_PX + i], N_LANE_WARPS / 4);
    mbar_init(&bars[B_EP], N_LANE_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_PFREE + i], rank < SC ? 1 : N_LANE_WARPS);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[B_RS + i], SC * N_LANE_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_OP + i], here);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_SFULL + i], 2);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (rank >= SC) {  // what the context CTAs expect first
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&bars[B_PFULL + i], P_BYTES);
      for (int i = 0; i < NRF; ++i) mbar_arrive_expect_tx(&bars[B_RF + i], CROWS * 8);
    }
  }
  if (warp == W_MMA) {
    if constexpr (SOLO) {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    }
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();  // the plan
  if constexpr (MODE == kShared) {
    // The kernel for few rows runs beside this one: it begins behind the word below, which it reads once and
    // finds set, since this word is everywhere before any of this block's threads lets that kernel come.
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) {
        store_release(&ws.plan->ready, 1u);
        __threadfence();
      }
      __syncthreads();
    }
  }
  grid_dependents_launch();  // (the join kernel may come as soon as there is room)
  const bool work = k < ws.plan->n;
  if constexpr (MODE == kShared) {
    // nothing to do, like the cluster's other CTAs: out of the way of the kernel for few rows, which waits for the SM
    if (!work) {
      __syncthreads();
      tc_fence_before();
      cluster_sync();
      tc_fence_after();
      if (warp == W_MMA) tmem_dealloc_pair(tmem, 512);
      return;
    }
  }
  Way<MODE, SOLO> w;
  if (work) w.start(a, *ws.plan, k);
  else w.left = 0;
  int gt = 0;  // key tiles of the range before this segment

  if (rank < SC) {
    // ================================================================ score CTAs
    const uint32_t kring = smem_u32(sm + OFF_K);
    const uint32_t scr = smem_u32(sm + OFF_SC);
    if (warp == W_TMA) {
      // this CTA's page of every tile, in two halves (Lc 0, 1; then Lc 2, 3 and Rc),
      // and both pages' row scales
      bool ok = true;
      const uint32_t kfull0 = map_to(smem_u32(&bars[B_KFULL]), 0);
      int halves = 0, nsc = 0, tiles = 0;
      for (; ok && w.more(); w.next(a)) {
        PageWindow pw;
        pw.from = -64;
        for (int i = 0; ok && i < w.n; ++i) {
          const int g = gt + i, kb = g % NK, sc = g % NSC;
          const int64_t page = 2 * (int64_t)(w.t + i);
          const int64_t s0 = pw.slot(a, w, page, lane, rank == 0);
          const int64_t s1 = pw.slot(a, w, page + 1, lane, rank == 0);
          const uint32_t pages = (s0 >= 0 ? 1u : 0u) + (s1 >= 0 ? 1u : 0u);
          if constexpr (SOLO) {
            // an Lc block at a time, and the Rc block last
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const int jb = 4 * g + c, slot = jb % NKB;
              if (!wait(B_SFREE + slot, (uint32_t)(jb / NKB) ^ 1u)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx_warp(&bars[B_SFILL + slot], pages * BLK);
              halves = jb + 1;
              const uint32_t dst = kring + slot * KBLK;
              if (s0 >= 0) tma_load_2d_warp(dst, &kmap, 128 * c, (int)s0, &bars[B_SFILL + slot]);
              if (s1 >= 0) tma_load_2d_warp(dst + BLK, &kmap, 128 * c, (int)s1, &bars[B_SFILL + slot]);
            }
            if (!ok || !wait(B_REMPTY, (uint32_t)g ^ 1u)) {
              ok = false;
              break;
            }
            const uint32_t rd = smem_u32(sm + OFF_KR);
            mbar_arrive_expect_tx_warp(&bars[B_RFULL], pages * RBLK);
            tiles = g + 1;
            if (s0 >= 0) tma_load_2d_warp(rd, &rmap, DL, (int)s0, &bars[B_RFULL]);
            if (s1 >= 0) tma_load_2d_warp(rd + RBLK, &rmap, DL, (int)s1, &bars[B_RFULL]);
          } else {
          const int64_t mine = rank == 0 ? s0 : s1;
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
        if constexpr (SOLO) {
          for (int i = (halves > NKB ? halves - NKB : 0); i < halves; ++i)
            (void)mbar_wait(&bars[B_SFILL + i % NKB], (i / NKB) & 1, &zero, WAIT_NS);
          if (tiles > 0) (void)mbar_wait(&bars[B_RFULL], (tiles - 1) & 1, &zero, WAIT_NS);
        } else if (rank == 0)
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
        Way<MODE, SOLO> wn = w;
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
        const uint64_t rd = smem_desc(SOLO ? smem_u32(sm + OFF_KR) : kring + 4 * BLK, 16, 512, SW64);
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
            if constexpr (SOLO) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                const int jb = 4 * g + c, slot = jb % NKB;
                if (!wait(B_SFILL + slot, (uint32_t)(jb / NKB))) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                const uint64_t bd = kd + (uint64_t)(slot * KBLK >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  mma_ts(dl, tmem + T_QH + c * 32 + kk * 8, bd + 2 * kk, id, (c | kk) != 0);
                  mma(dl, ql + (uint64_t)(c * OP_ATOM >> 4) + 2 * kk, bd + 2 * kk, id, 1u);
                }
                commit(&bars[B_SFREE + slot], 0);
              }
            } else {
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
                  mma_ts(dl, tmem + T_QH + c * 32 + kk * 8, bd + 2 * kk, id, (h | blk | kk) != 0);
                  mma(dl, ql + (uint64_t)(c * OP_ATOM >> 4) + 2 * kk, bd + 2 * kk, id, 1u);
                }
              }
              if (h == 0) commit(&bars[B_KEMPTY + 2 * kb], 3);
            }
            }
            if (!ok) break;
            // S_R (and the other S_L) of the previous tile read
            if (g > 0 && !wait_cluster(B_SEMPTY + ((g - 1) & 1), (uint32_t)((g - 1) >> 1))) {
              ok = false;
              break;
            }
            if (SOLO && !wait(B_RFULL, (uint32_t)g)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t rb = SOLO ? rd : rd + off;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              mma(tmem + T_SR, qr + 2 * kk, rb + 2 * kk, id, kk != 0);
              mma(tmem + T_SR, qr + 4 + 2 * kk, rb + 2 * kk, id, 1u);
            }
            commit(SOLO ? &bars[B_REMPTY] : &bars[B_KEMPTY + 2 * kb + 1], 3);
            commit(&bars[B_SFULL + (g & 1)], 3);
          }
          gt += w.n;
        }
        if (!ok && lane == 0) fail();
        commit(&bars[B_DRAIN], 3);
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
      Way<MODE, SOLO>* walk = reinterpret_cast<Way<MODE, SOLO>*>(sm + OFF_WALK) + (warp - W_LANE);  // (it has no registers to spare)
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
      auto load_query = [&](const Way<MODE, SOLO>& x) -> bool {
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
        const Way<MODE, SOLO>& x = *walk;
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
        // (a window: where that of the last of the rows begins)
        const int from = MODE == kWindow ? window_from(a, lim[q * 32 + 16 * hl + 15]) : 0;
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i, t0 += TILE) {
          const int g = gt + i, buf = g & 1, sc = g % NSC;
          if constexpr (MODE == kWindow) t0 = x.at(2 * (x.t + i) + sub) * PAGE;
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
          // some row does not see all of this page
          if (!here || first - t0 < SUB || (MODE == kWindow && t0 < from && a.n_sink - t0 < SUB)) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int n = here ? lim[rh + 8 * p] - t0 - 2 * i4 : 0;
              // (and of the keys before `after`, those from `sinks` on are behind the window)
              const int after = MODE == kWindow ? window_from(a, lim[rh + 8 * p]) - t0 - 2 * i4 : 0;
              const int sinks = MODE == kWindow ? a.n_sink - t0 - 2 * i4 : 0;
#pragma unroll
              for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * j + e >= n || (MODE == kWindow && 8 * j + e < after && 8 * j + e >= sinks))
                    u[4 * j + 2 * p + e] = 0xFF800000u;  // -inf
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
          const uint32_t to = map_to(smem_u32(sm + OFF_P + buf * P_STRIDE), rank + SC);
          const uint32_t bar = map_to(smem_u32(&bars[B_PFULL + buf]), rank + SC);
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
          if (x.final()) {
            f = L == 0.f ? 0.f : 1.f / L;  // (a NaN stays one)
            const int64_t r = (int64_t)x.rt * ROWS + rank * CROWS + hh;
            if (a.lse != nullptr && r < (int64_t)x.s.nq * a.H)
              a.lse[x.s.q0 * a.H + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
          } else {
            const int row = rank * CROWS + hh;
            const int64_t at = ws.part_row(x, k, row);
            if (MODE != kShared || (int64_t)x.rt * ROWS + row < (int64_t)x.s.nq * a.H) {
              ws.m[at] = M;
              ws.l[at] = L;
            }
          }
          const int rf = x.seg % NRF;
          const uint32_t to = map_to(smem_u32(sm + OFF_RF + (rf * CROWS + hh) * 8), rank + SC);
          const uint32_t bar = map_to(smem_u32(&bars[B_RF + rf]), rank + SC);
          st_async_b32(to, __float_as_uint(f), bar);
          st_async_b32(to + 4, __float_as_uint(mm), bar);
        }
        gt += n_tiles;
        Way<MODE, SOLO> wn = x;
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
    const int half_of = (int)rank - SC;  // channels 256 h + 128 half_of .. of each O half h (solo: all of them)
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
          if constexpr (SOLO) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!wait(B_VEMPTY + h, (uint32_t)g ^ 1u)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx_warp(&bars[B_VT + h], 2u * BLK * ((s0 >= 0 ? 1u : 0u) + (s1 >= 0 ? 1u : 0u)));
              nv = 2 * g + h + 1;
#pragma unroll 1
              for (int m = 0; m < 2; ++m) {
                const uint32_t dst = vring + (2 * h + m) * VBLK;
                if (s0 >= 0) tma_load_2d_warp(dst, &kmap, 256 * h + 128 * m, (int)s0, &bars[B_VT + h]);
                if (s1 >= 0) tma_load_2d_warp(dst + BLK, &kmap, 256 * h + 128 * m, (int)s1, &bars[B_VT + h]);
              }
            }
            if (!ok) break;
            continue;
          }
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
        static_assert(NVT == 2, "(solo: halves of tiles)");
        for (int i = (nv > NVT ? nv - NVT : 0); i < nv; ++i)
          (void)mbar_wait(&bars[B_VT + i % NVT], (i / NVT) & 1, &zero, WAIT_NS);
      }
      __syncwarp();
    } else if (warp == W_SCALE) {
      // (no scales here: this warp tells the score CTA which payloads are read, so that its writes of
      // the next ones come after those reads)
      const uint32_t pfree = map_to(smem_u32(&bars[B_PFREE]), rank - SC);
      bool ok = true;
      for (int64_t g = 0; ok && g < w.left; ++g)
        ok = relay(B_PFREE + (int)(g & 1), (uint32_t)(g >> 1), pfree + (int)(g & 1) * 8);
      if (!ok && lane == 0) fail();
      __syncwarp();
    } else if (warp == W_MMA) {
      if (rank == SC) {
        const uint32_t id = idesc_f16(ROWS, 256, false, true);  // A K-major, B = V MN-major
        const uint64_t pd = smem_desc(smem_u32(sm + OFF_OP), 16, 1024, SW128);
        const uint64_t vd = smem_desc(vring, SOLO ? VBLK : 16, 1024, SW128);
        bool ok = true;
        for (; ok && w.more(); w.next(a)) {
          for (int i = 0; ok && i < w.n; ++i) {
            const int g = gt + i;
            const uint64_t ad = pd + (uint64_t)((g & 1) * 2 * OP_ATOM >> 4);
            if ((!SOLO && !wait(B_VT + g % NVT, (uint32_t)(g / NVT))) || !wait_cluster(B_OP + (g & 1), (uint32_t)(g >> 1))) {
              ok = false;
              break;
            }
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if ((SOLO && !wait(B_VT + h, (uint32_t)g)) || !wait_cluster(B_RS + 2 * (g & 1) + h, (uint32_t)(g >> 1))) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t bd = vd + (uint64_t)((SOLO ? 2 * h * VBLK : (g % NVT) * VTILE + h * VBLK) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                // A: 32 tokens of the hi / lo atom; B: 32 token rows (4 KB)
                mma(tmem + h * 256, ad + 2 * kk, bd + 256 * kk, id, (i > 0 || kk > 0) ? 1u : 0u);
                mma(tmem + h * 256, ad + (OP_ATOM >> 4) + 2 * kk, bd + 256 * kk, id, 1u);
              }
              commit(&bars[B_ODONE + 2 * (g & 1) + h], 0xC);
              if constexpr (SOLO) commit(&bars[B_VEMPTY + h], 0);
            }
            if (!ok) break;
            if constexpr (!SOLO) commit(&bars[B_VEMPTY + g % NVT], 0xC);
          }
          gt += w.n;
        }
        if (!ok && lane == 0) fail();
        commit(&bars[B_DRAIN], 0xC);
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
      const uint32_t rs = map_to(smem_u32(&bars[B_RS]), SC);
      bool ok = true;
      for (; ok && w.more(); w.next(a)) {
        const int lim0 = limit_of(a, w.s, first_token<GeoOf<SOLO>>(a, w.rt));  // the tile's first row sees least
        // (a window: that of the tile's last row begins last)
        const int from = MODE == kWindow ? window_from(a, limit_of(a, w.s, last_token<GeoOf<SOLO>>(a, w.s, w.rt))) : 0;
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
          bool part_seen = w.t + i + 1 > lim0 / TILE;
          if constexpr (MODE == kWindow) {
            part_seen = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int t0 = w.at(2 * (w.t + i) + h) * PAGE;
              part_seen |= lim0 - t0 < PAGE || (t0 < from && a.n_sink - t0 < PAGE);
            }
          }
          if (part_seen || pages != 3u) {
            // some row does not see all of this tile: no NaN code may stay in it
            if (!wait(SOLO ? B_VT : B_VT + vs, SOLO ? (uint32_t)g : (uint32_t)(g / NVT)) ||
                (SOLO && !wait(B_VT + 1, (uint32_t)g))) {
              ok = false;
              break;
            }
            constexpr int SHARE_OF_V = (SOLO ? 4 * VBLK : VTILE) / N_LANE_WARPS;
            const uint32_t vb = vring + (SOLO ? 0 : vs * VTILE) + (warp - W_LANE) * SHARE_OF_V + lane * 16;
#pragma unroll
            for (int u = 0; u < SHARE_OF_V / 512; ++u) {
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
        const bool whole = w.final();
        const int64_t r0 = (int64_t)w.rt * ROWS + half_of * CROWS + q * 32;  // the warp's first row
        const int64_t rows = (int64_t)w.s.nq * a.H - r0;
        const int left = (int)(rows < 32 ? rows : 32) - (lane >> 2);         // rows from this lane's first on, by eights
        const uint32_t stage = smem_u32(sm + OFF_OP) + (warp - W_LANE) * 2048;
        const uint32_t put = stage + lane * 64, sw = (lane >> 1) & 3;        // this lane's row, its units turned by sw
        const uint32_t take = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
        const int row_bytes = whole ? DL * 2 : DL * 4;
        uint8_t* dst = (whole ? reinterpret_cast<uint8_t*>(a.out + (w.s.q0 * a.H + r0) * DL)
                              : reinterpret_cast<uint8_t*>(ws.o + ws.part_row(w, k, half_of * CROWS + q * 32) * DL)) +
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
  if (warp == W_MMA) {
    if constexpr (SOLO) tmem_dealloc(tmem, 512);
    else tmem_dealloc_pair(tmem, 512);
  }
}

// Joins the parts of the row tiles that range borders cut: for every cluster k but the
// first, the row tile that it starts in, if cluster k - 1 holds its beginning; a warp per
// row, or per row and SPLIT-th of its channels.  In four parts a single row tile in many
// parts is read by 128 SMs in place of 32 (one token over 8192 keys at 128 heads: 47.0
// against 55.6 us); where most clusters hold a border the blocks that gives cost more
// than that (32 x 4 tokens over up to 16384 keys: 241 against 236 us).
constexpr int JOIN_BLOCKS = ROWS / 8;
constexpr int FEW_ROW_TILES = 8;

// A row of a group with a shared prefix: the parts of the prefix and of the rest, each one whole row
// tile's or those that range borders cut it into, by one warp.
__device__ __forceinline__ void join_parts(const ChunkArgs& a, const Workspace<>& ws, const int64_t* base, int64_t row,
                                           int lane) {
  const int64_t nc = ws.plan->n;
  const int2 of = a.part_seq[row / a.H];
  // where the ranges begin, two a lane (behind the last: never)
  int64_t xs[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) xs[h] = lane + 32 * h < nc ? ws.plan->e[lane + 32 * h].x : INT64_MAX;
  int64_t from[2];   // the parts' row in the slots of cluster 0, or of the whole
  int k0[2], n[2];   // their clusters (n = 0: the row tile is whole), and the first of them's slot
  bool second[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int v = which == 0 ? of.x : a.G + of.y;
    const int part = a.entries[v].v.z;
    const int64_t r = row + (which == 0 ? 0 : a.part_rows) - part;  // row of the entry
    const int64_t p = base[v] + r / ROWS, S = a.unit[p], E = a.unit[p + 1];
    int first = -1, last = -1;  // the last range that begins at S or before, and before E
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      first += __popc(__ballot_sync(0xffffffffu, xs[h] <= S));
      last += __popc(__ballot_sync(0xffffffffu, xs[h] < E));
    }
    const int64_t x0 = __shfl_sync(0xffffffffu, first < 32 ? xs[0] : xs[1], first & 31);
    k0[which] = first;
    second[which] = x0 < S;
    n[which] = last - first + 1;
    from[which] = r % ROWS;
    if (n[which] == 1) from[which] = ws.parts + part + r;
  }
  // a lane per part: its reference, its sum (a cluster without units has no part)
  float m[2][2], wt[2][2], M = -INFINITY, L = 0.f;
  uint32_t has[2][2];
  auto slot = [&](int which, int j) -> int64_t {
    return n[which] == 1 ? from[which] : (int64_t)(2 * (k0[which] + j) + (j == 0 && second[which] ? 1 : 0)) * ROWS + from[which];
  };
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h, k = k0[which] + j;
      const int64_t x0 = __shfl_sync(0xffffffffu, xs[0], k & 31), x1 = __shfl_sync(0xffffffffu, xs[1], k & 31);
      const int64_t y0 = __shfl_sync(0xffffffffu, xs[0], (k + 1) & 31), y1 = __shfl_sync(0xffffffffu, xs[1], (k + 1) & 31);
      const bool there = j < n[which] && (k < 32 ? x0 : x1) != (k + 1 < 32 ? y0 : (k + 1 < 64 ? y1 : INT64_MAX));
      m[which][h] = there ? ws.m[slot(which, j)] : -INFINITY;
      wt[which][h] = there ? ws.l[slot(which, j)] : 0.f;
      has[which][h] = __ballot_sync(0xffffffffu, there);
      M = fmaxf(M, m[which][h]);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float l = wt[which][h], f = m[which][h] > -INFINITY ? ex2_approx(m[which][h] - M) : 1.f;  // (a NaN l stays one)
      L += f * l;
      const int parts = min(n[which] - 32 * h, 32);
#pragma unroll 2
      for (int i = 0; i < parts; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        if (!((has[which][h] >> i) & 1u)) continue;
        const float4* o = reinterpret_cast<const float4*>(ws.o + slot(which, 32 * h + i) * DL) + lane;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 v = o[32 * c];
          acc[c].x += w * v.x;
          acc[c].y += w * v.y;
          acc[c].z += w * v.z;
          acc[c].w += w * v.w;
        }
      }
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int4 u = a.entries[of.x].u;
  const int64_t at = (int64_t)u.x * a.H + row - a.entries[of.x].v.z;
  uint2* out = reinterpret_cast<uint2*>(a.out + at * DL) + lane;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    out[32 * c] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (a.lse != nullptr && lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
}

template <int MODE, int SPLIT>
__global__ void __launch_bounds__(256) join_kernel(const ChunkArgs a, const Workspace<> ws, const int64_t* base, int cut_blocks) {
  static_assert(MAX_CLUSTERS <= 64, "two parts a lane");
  const int k = (int)blockIdx.x / (JOIN_BLOCKS * SPLIT) + 1, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x % (JOIN_BLOCKS * SPLIT) / SPLIT * 8 + (threadIdx.x >> 5);
  const int ch = (int)blockIdx.x % SPLIT * (DL / SPLIT);
  // (every block waits, with a row or without: the plan's and the parts' visibility, and that this
  // launch is not over before the chunk kernel is, come with the wait)
  grid_dependency_wait();
  if constexpr (MODE == kShared) {
    if ((int)blockIdx.x >= cut_blocks) {  // (behind the blocks for the row tiles that were cut)
      const int64_t r = (int64_t)((int)blockIdx.x - cut_blocks) * 8 + (threadIdx.x >> 5);
      if (r < ws.plan->part_rows) join_parts(a, ws, base, r, lane);
      return;
    }
  }
  const int64_t nc = ws.plan->n;
  if (k >= nc) return;
  __shared__ int64_t xs[MAX_CLUSTERS + 1];    // the units where the ranges begin
  if (threadIdx.x <= nc) xs[threadIdx.x] = threadIdx.x < nc ? ws.plan->e[threadIdx.x].x : ws.plan->units;
  const PlanEntry e = ws.plan->e[k];
  __syncthreads();
  const int64_t S = e.x - e.off;              // the row tile's first unit
  const int64_t xp = xs[k - 1];
  const SeqInfo<MODE> s = seq_info<MODE>(a, e.b, false);
  if constexpr (MODE == kShared) {
    if (s.part >= 0) return;
  }
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
static_assert(OFF_PLAN + sizeof(Plan<Geo>) <= OFF_BASE, "plan area");

// What the workspace of a call holds, behind the plan (from sizes alone).
struct Layout {
  int most;         // clusters that a call of these sizes can use, whatever the lengths turn out to be
  int64_t tiles;    // row tiles at most
  int64_t part_rows;
  int64_t entries, unit, part_seq, m, rows, bytes;
};

template <int MODE>
Layout layout_of(int B, int H, int64_t total_q, int max_blocks, int G, int64_t window, int64_t n_sink) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout w;
  int64_t keys = ((int64_t)max_blocks * PAGE + TILE - 1) / TILE;
  w.tiles = total_q * H / ROWS + B;
  if (MODE == kShared) w.tiles += total_q * H / ROWS + G;
  if (MODE == kWindow) {  // (a row tile's tokens lie within ROWS of one another)
    const int64_t seen = window + n_sink + ROWS + 4 * PAGE;
    if (seen / TILE + 1 < keys) keys = seen / TILE + 1;
  }
  const int64_t units = w.tiles * (keys > MIN_TILES ? keys : MIN_TILES) / MIN_TILES;
  w.most = (int)(units < 1 ? 1 : (units < MAX_CLUSTERS ? units : MAX_CLUSTERS));
  w.part_rows = 0;
  if (MODE == kShared && G > 0) {
    const int64_t rows = total_q * H, few = (int64_t)PART_ROWS * B, cap = 1 << 20;
    w.part_rows = rows < few ? rows : few;
    if (w.part_rows > cap) w.part_rows = cap;
  }
  int64_t at = OFF_BASE + up((int64_t)(B + (MODE == kShared ? G : 0) + 1) * 8);
  w.entries = at;
  if (MODE == kShared) at += up((int64_t)(G + B) * (int64_t)sizeof(ChunkEntry));
  w.unit = at;
  if (MODE == kShared) at += up((w.tiles + 1) * 8);
  w.part_seq = at;
  if (MODE == kShared) at += up((w.part_rows / H + 1) * 8);
  w.m = at;
  w.rows = (w.most > 1 ? 2 * (int64_t)w.most * ROWS : 0) + 2 * w.part_rows;  // (one cluster cuts no row tile)
  w.bytes = at + w.rows * (8 + DL * 4);
  return w;
}

// Which kernel a call with a window goes to, by the rows of its sequences on average: up to 64, the one for
// few rows (rows.cu), which reads a tile of keys for 32 rows at once; up to 128, the clusters of two here,
// unless there are few (row tile, key tile) units, over which the other spreads better.  Device times of that
// one, the clusters of two and of four, us, for single tokens of 128 heads: one over 1000 keys 18, 31, 30, over
// 8192 20, 31, 38; 64 over 128 keys 33, 27, 40; 32 over 2048 keys 54, 47, 60; 64 over 8192 keys 262, 156,
// 239.  Of 64 heads: 32 over 2048 keys 35, 44, 56; 64 over 8192 keys 142, 150, 232.
// The average is over all sequences, those without queries among them, and their number is all that the host knows: a
// batch of which most have none may go to row tiles too small for the one that has.  (512 new tokens of 16 heads at
// 8192 keys alone, beside 63 and beside 511 sequences without queries: window 2048 62, 66 and 132 us; 8192 128, 146
// and 377; shared prefixes, in a group that shares nothing, 128, 129 and 382; of 128 heads, window 2048, 301, 301, 336.)
constexpr int FEW_ROWS = 64, FEW_UNITS = 100;
bool few_rows(int B, int H, int64_t total_q, int64_t keys) {
  const int64_t rows = total_q * H;
  return rows <= (int64_t)FEW_ROWS * B || (rows <= (int64_t)CROWS * B && (int64_t)B * (keys / TILE + 1) <= FEW_UNITS);
}
bool solo_rows(int B, int H, int64_t total_q) { return total_q * H <= (int64_t)CROWS * B; }
int64_t window_keys(int max_blocks, int64_t window, int64_t n_sink) {
  const int64_t all = (int64_t)max_blocks * PAGE;
  return window + n_sink < all ? window + n_sink : all;
}

// Clusters of the kernel that the device holds at once.
template <int MODE, bool SOLO = false>
cudaError_t capacity(int* fit) {
  static std::atomic<int> memo[MAX_DEVICES];
  return per_device(memo, [](int* v) {
    constexpr int smem = SOLO ? SMEM_SOLO : SMEM;
    cudaError_t r = cudaFuncSetAttribute(chunk_kernel<MODE, SOLO>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(NUM_SMS, 1, 1);
    cfg.blockDim = dim3(NTHREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    r = cudaOccupancyMaxActiveClusters(&n, chunk_kernel<MODE, SOLO>, &cfg);
    if (r != cudaSuccess) return r;
    if (n < 1) return cudaErrorLaunchOutOfResources;
    *v = n > GeoOf<SOLO>::RANGES ? GeoOf<SOLO>::RANGES : n;
    return cudaSuccess;
  }, fit);
}

template <int MODE>
cudaError_t launch(ChunkArgs a, void* workspace, cudaStream_t s) {
  int fit = 0;
  cudaError_t e = capacity<MODE>(&fit);
  if (e != cudaSuccess) return e;
  const Layout w = layout_of<MODE>(a.B, a.H, a.total_q, a.max_blocks, a.G, a.window, a.n_sink);
  const int clusters = w.most < fit ? w.most : fit;
  char* p = static_cast<char*>(workspace);
  a.err = reinterpret_cast<unsigned*>(p);
  a.entries = reinterpret_cast<ChunkEntry*>(p + w.entries);
  a.unit = reinterpret_cast<int64_t*>(p + w.unit);
  a.part_seq = reinterpret_cast<int2*>(p + w.part_seq);
  a.part_rows = w.part_rows;
  Workspace<> ws;
  ws.plan = reinterpret_cast<Plan<Geo>*>(p + OFF_PLAN);
  int64_t* base = reinterpret_cast<int64_t*>(p + OFF_BASE);
  ws.m = reinterpret_cast<float*>(p + w.m);
  ws.l = ws.m + w.rows;
  ws.o = ws.l + w.rows;
  ws.parts = w.rows - 2 * w.part_rows;
  DecodeArgs d{};  // what the cache's tensor maps are made from
  d.codes = a.codes;
  d.scales = a.scales;
  d.block_table = a.block_table;
  d.n_blocks = a.n_blocks;
  CUtensorMap kmap, rmap, smap;
  if ((e = make_cache_map(d, &kmap)) != cudaSuccess || (e = make_rc_map(d, &rmap)) != cudaSuccess ||
      (e = make_scale_map(d, &smap)) != cudaSuccess)
    return e;
  plan_kernel<MODE><<<1, PLAN_THREADS, 0, s>>>(a, ws.plan, base, clusters);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after_prep(chunk_kernel<MODE>, 4 * clusters, NTHREADS, SMEM, s, a, ws, kmap, rmap, smap);
  const unsigned part_blocks = (unsigned)((w.part_rows + 7) / 8);
  if (e != cudaSuccess || (clusters == 1 && part_blocks == 0)) return e;
  const unsigned blocks = JOIN_BLOCKS * (clusters - 1);
  if (w.tiles < FEW_ROW_TILES)
    return launch_after_prep(join_kernel<MODE, 4>, 4 * blocks + part_blocks, 256, 0, s, a, ws, base, (int)(4 * blocks));
  return launch_after_prep(join_kernel<MODE, 1>, blocks + part_blocks, 256, 0, s, a, ws, base, (int)blocks);
}

// The clusters of two, for a window.
constexpr int64_t OFF_SOLO_BASE = 2560;
static_assert(OFF_PLAN + sizeof(Plan<SoloGeo>) <= OFF_SOLO_BASE, "plan area");

struct SoloLayout {
  int most;
  int64_t tiles, owner, m, rows, bytes;
};
SoloLayout solo_layout(int B, int H, int64_t total_q, int64_t keys) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  SoloLayout w;
  w.tiles = total_q * H / CROWS + B;
  const int64_t units = w.tiles * ((keys + CROWS) / TILE + 4) / SoloGeo::MIN_TILES;
  w.most = (int)(units < 1 ? 1 : (units < SoloGeo::RANGES ? units : SoloGeo::RANGES));
  w.owner = OFF_SOLO_BASE + up((int64_t)(B + 1) * 8);
  w.m = w.owner + up(w.tiles * (int64_t)sizeof(int4));
  w.rows = w.most > 1 ? 2 * (int64_t)w.most * CROWS : 0;  // (one range cuts no row tile)
  w.bytes = w.m + w.rows * (8 + DL * 4);
  return w;
}

cudaError_t launch_solo(ChunkArgs a, const SoloLayout& w, void* workspace, cudaStream_t s) {
  int fit = 0;
  cudaError_t e = capacity<kWindow, true>(&fit);
  if (e != cudaSuccess) return e;
  const int clusters = w.most < fit ? w.most : fit;
  char* p = static_cast<char*>(workspace);
  a.err = reinterpret_cast<unsigned*>(p);
  Workspace<true> ws;
  ws.plan = reinterpret_cast<Plan<SoloGeo>*>(p + OFF_PLAN);
  ws.m = reinterpret_cast<float*>(p + w.m);
  ws.l = ws.m + w.rows;
  ws.o = ws.l + w.rows;
  ws.parts = 0;
  int4* owner = reinterpret_cast<int4*>(p + w.owner);
  DecodeArgs d{};  // what the cache's tensor maps are made from
  d.codes = a.codes;
  d.scales = a.scales;
  d.block_table = a.block_table;
  d.n_blocks = a.n_blocks;
  CUtensorMap kmap, rmap, smap;
  if ((e = make_cache_map(d, &kmap)) != cudaSuccess || (e = make_rc_map(d, &rmap)) != cudaSuccess ||
      (e = make_scale_map(d, &smap)) != cudaSuccess)
    return e;
  solo_plan_kernel<<<1, PLAN_THREADS, 0, s>>>(a, ws.plan, reinterpret_cast<int64_t*>(p + OFF_SOLO_BASE), owner, clusters);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after_prep(chunk_kernel<kWindow, true>, 2 * clusters, NTHREADS, SMEM_SOLO, s, a, ws, kmap, rmap, smap);
  if (e != cudaSuccess || clusters == 1) return e;
  return launch_parts_join<kWindow, CROWS>(a, PartsJoin{&ws.plan->tiles, owner, ws.m, ws.l, ws.o, 0, nullptr, nullptr, 0},
                                           w.tiles, clusters, s);
}

}  // namespace

int64_t chunk_workspace(int B, int H, int64_t total_q, int max_blocks) {
  return layout_of<kPlain>(B, H, total_q, max_blocks, 0, 0, 0).bytes;
}
int64_t window_workspace(int B, int H, int64_t total_q, int max_blocks, int window, int n_sink) {
  if (few_rows(B, H, total_q, window_keys(max_blocks, window, n_sink)))
    return rows_window_workspace(B, H, total_q, max_blocks, window, n_sink);
  if (solo_rows(B, H, total_q)) return solo_layout(B, H, total_q, window_keys(max_blocks, window, n_sink)).bytes;
  return layout_of<kWindow>(B, H, total_q, max_blocks, 0, window, n_sink).bytes;
}
int64_t shared_workspace(int B, int H, int64_t total_q, int max_blocks, int G) {
  if (total_q * H <= (int64_t)FEW_ROWS * B) return rows_shared_workspace(B, H, total_q, max_blocks, G);
  return layout_of<kShared>(B, H, total_q, max_blocks, G, 0, 0).bytes;
}

cudaError_t launch_chunk(const ChunkArgs& a, void* workspace, cudaStream_t s) { return launch<kPlain>(a, workspace, s); }
cudaError_t launch_window(const ChunkArgs& a, void* workspace, cudaStream_t s) {
  const int64_t keys = window_keys(a.max_blocks, a.window, a.n_sink);
  if (few_rows(a.B, a.H, a.total_q, keys)) return launch_rows_window(a, workspace, s);
  if (solo_rows(a.B, a.H, a.total_q)) return launch_solo(a, solo_layout(a.B, a.H, a.total_q, keys), workspace, s);
  return launch<kWindow>(a, workspace, s);
}
cudaError_t launch_shared(const ChunkArgs& a, void* workspace, cudaStream_t s) {
  return a.total_q * a.H <= (int64_t)FEW_ROWS * a.B ? launch_rows_shared(a, workspace, s) : launch<kShared>(a, workspace, s);
}

cudaError_t prefix_capacity(int* clusters) { return capacity<kShared>(clusters); }
cudaError_t launch_prefixes(const ChunkArgs& a, const PrefixParts& p, int clusters, const CUtensorMap& kmap,
                            const CUtensorMap& rmap, const CUtensorMap& smap, cudaStream_t s) {
  Workspace<> ws;
  ws.plan = static_cast<Plan<Geo>*>(p.plan);
  ws.m = p.m;
  ws.l = p.l;
  ws.o = p.o;
  ws.parts = p.whole;
  return launch_after_prep(chunk_kernel<kShared>, 4 * clusters, NTHREADS, SMEM, s, a, ws, kmap, rmap, smap);
}

}  // namespace kv8
