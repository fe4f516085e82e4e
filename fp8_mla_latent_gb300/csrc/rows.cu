// rows.cu -- absorbed MLA attention over the paged fp8 latent cache for sequences of few rows (single
// tokens of a few heads): the same mathematics and precision as chunk.cu,
//   z_t = sm * ( sLc_t <q_lat, dec(Lc_t)> + sRc_t <q_rope, dec(Rc_t)> ),   out = sum_t softmax(z)_t sLc_t dec(Lc_t)
// with the keys as the MMAs' M and a row tile of N = 16 or 32 (token, head) pairs as theirs, on one CTA per SM
// (chunk.cu's 256 rows would be 240 copies for a token of 16 heads, at four SMs a range).
//
// A range of (row tile, key tile) units is one CTA's.  Per key tile of 128 tokens, whose bytes are loaded
// once by TMA and read by both contractions as they are (kind::f8f6f4):
//   S[t][r]  = K_t . Q_r       M = 128, 2 N columns: the query's hi terms, then its lo terms; Lc and Rc apart
//   g'[r][t] = 2^(c u - M_r + 7) sLc_t   as two e4m3 terms; M_r follows the row's largest weight 2^(c u) sLc
//   O[d][r] += sum_t V[t][d] g'[r][t]    four blocks of 128 channels, 2 N columns
// A token is a TMEM lane, so that a row's maximum and sum go over lanes and warps: eight rows are a warp's, reduced
// together (a round halves the values a lane has left, 11 shuffles in place of 40).
//
// N = 16: the keys alternate between two streams, each with eight softmax warps, its own references, sums and
// O (TMEM holds both: 2 x 128 columns, and four buffers of S), which are joined at the row tile's end.  A
// tile's chain -- scores, maximum over its tokens, weights, context -- is longer than the time in which its
// bytes come, so that two of them have to run at once.  N = 32: one stream of sixteen
// warps (shared memory and TMEM hold no second one's weights and O), two buffers of S.
//
// What bounds it.  N = 16: HBM.  A tile takes about 3500 cycles, 75 KB on each of 152 SMs, 6.2 TB/s, 0.92 of the copy rate.
// N = 32: the one chain and the ring of keys, about 4000 cycles.  Around the tiles: plan 2.8 us, first
// query 4 (its load, and the pipeline's), a row tile's end 1.7, join 4.
//
// Measured, one GB300 (device time; fractions of the copy rate, 6775 GB/s, of the bytes in sight): 64 tokens of 16 heads with
// a window of 4096, ragged, 43.3 us, 0.45; of 8192 70.6 us, 0.65; 512 tokens, window 2048, 148 us, 0.63;
// 32 heads, window 8192, 81 us, 0.57; 32 tokens of 16 heads, window 2048, 24.2 us, 0.24; one token, window
// 128, 14.3 us, which is latency.
//
// Warps: 0 loads; 1 issues the scores' MMAs; 2 the context's; 3-18 softmax: stream, eight of the rows, and
// TMEM lane quarter.  Every wait is bounded (2 s); on a timeout the CTA flags the workspace's error word,
// drains its MMAs and copies and leaves.
#include <cuda.h>

#include "chunk_work.cuh"

namespace kv8 {
namespace {

constexpr int NH = 8;                        // rows of a softmax warp
constexpr int KBLK = TILE * 128;             // 16 KB: [128 tokens x 128 bytes]
constexpr int RBLK = TILE * 64;              // 8 KB: [128 tokens x 64 bytes]
constexpr int W_TMA = 0, W_MMA = 1, W_CTX = 2, W_SOFT = 3;
constexpr int N_SOFT = 16;                   // softmax warps: four, one per TMEM lane quarter, for 8 rows of a stream
constexpr int NTHREADS = (W_SOFT + N_SOFT) * 32;
constexpr float TAU = 1.0f, P_LOG = 7.0f, DOWN = 10.0f, LG_MIN = -40.0f, DOWN_CAP = 50.0f;  // (as in chunk.cu)
constexpr uint64_t WAIT_NS = 2000000000ull;

// (us, SWITCH 2, 3 and 5: 64 tokens of 16 heads, ragged windows of 4096 46.3, 43.6, 42.1; 100 with 3000 41.9, 39.4,
// 40.5; 300 with 1000 54.0, 54.4, 56.0; 64 of 32 heads with 8192 57.5, 54.2, 55.2; MIN_TILES 2 changes nothing.)
template <int N>
struct Geo {
  static constexpr int ROWS = N, RANGES = NUM_SMS, SWITCH = 3, MIN_TILES = 1;
};
template <int MODE, int N>
using Way = Walk<MODE, Geo<N>>;

// Per row tile size N: rings, barriers, shared memory and TMEM columns.
template <int N>
struct Cfg {
  static constexpr int NB = 2 * N;                     // columns: hi terms, lo terms
  static constexpr int STREAMS = N_SOFT / 4 / (N / NH);
  static constexpr int SET = N_SOFT / STREAMS;         // a stream's softmax warps
  static constexpr int RL = N == 16 ? 11 : 10, RR = 2;  // rings of Lc blocks and Rc blocks
  static constexpr int NS = 2 * STREAMS;               // S buffers
  static constexpr int NTF = N == 16 ? 4 : 3;          // tiles loaded: barriers, row scales
  static_assert(RL <= 4 * NTF, "tile i's first block has the slot of one of tile i - NTF's, or of a later tile's");
  static constexpr int B_TFULL = 0;                    // [NTF] a tile's Rc block and scales loaded
  static constexpr int B_LFULL = B_TFULL + NTF;        // [RL] an Lc block loaded
  static constexpr int B_LEMPTY = B_LFULL + RL;        // [RL] read by the context's MMAs
  static constexpr int B_REMPTY = B_LEMPTY + RL;       // [RR] read by the scores'
  static constexpr int B_SFULL = B_REMPTY + RR;        // [NS] S of a tile in TMEM
  static constexpr int B_SEMPTY = B_SFULL + NS;        // [NS] read (a stream's warps)
  static constexpr int B_PFULL = B_SEMPTY + NS;        // [2] of even and odd tiles: weights written, O rescaled (a stream's warps)
  static constexpr int B_ODONE = B_PFULL + 2;          // [2] context MMAs done
  static constexpr int B_G = B_ODONE + 2;              // [4] the four warps of a stream's 8 rows meet
  static constexpr int B_QREADY = B_G + 4;             // a row tile's query in place (all softmax warps)
  static constexpr int B_EP = B_QREADY + 1;            // the softmax warps meet
  static constexpr int B_DRAIN = B_EP + 1;             // [2] the issuers' last MMAs
  static constexpr int NBAR = B_DRAIN + 2;
  static constexpr int OFF_FLAGS = 512;                // tmem base, abort flag
  static constexpr int OFF_FACTS = 528;                // [NTF] pages present
  static constexpr int OFF_CS = 640;                   // [2 segments][N] the rows' c
  static constexpr int OFF_LIM = OFF_CS + 8 * N;       // [2][N] the keys that they see
  static constexpr int OFF_REF = OFF_LIM + 8 * N;      // [STREAMS][N] references at a row tile's end
  static constexpr int OFF_LS = OFF_REF + 128;         // [STREAMS][4 warps][N] sums
  static constexpr int OFF_RMAX = OFF_LS + 512;        // [STREAMS][2 buffers][4][N] a tile's largest weights
  static constexpr int OFF_WALK = OFF_RMAX + 1024;     // [16 warps] segments
  static constexpr int OFF_SCR = 4096;                 // [NTF][128][2] row scales
  static constexpr int OFF_Q = OFF_SCR + NTF * TILE * 8;        // [4 blocks][NB x 128 B], [NB x 64 B]
  static constexpr int OFF_P = OFF_Q + 4 * NB * 128 + NB * 64;  // [STREAMS][NB x 128 tokens]
  static constexpr int OFF_L = OFF_P + STREAMS * NB * 128;
  static constexpr int OFF_R = OFF_L + RL * KBLK;
  static constexpr int SMEM = OFF_R + RR * RBLK;
  static constexpr int S_COLS = 2 * NB, T_O = NS * S_COLS, O_COLS = 4 * NB;
  static_assert(N == 16 || N == 32, "two streams, or one");
  static_assert(STREAMS * N * 4 <= 128 && STREAMS * 4 * N * 4 <= 512 && OFF_WALK % 16 == 0, "scratch");
  static_assert(NBAR * 8 <= OFF_FLAGS && OFF_WALK + N_SOFT * 64 <= OFF_SCR, "layout");
  static_assert(OFF_Q % 1024 == 0 && OFF_P % 1024 == 0 && OFF_L % 1024 == 0 && OFF_R % 1024 == 0, "swizzle atoms");
  static_assert(SMEM <= 232448 && T_O + STREAMS * O_COLS <= 512, "shared memory and TMEM");
};
static_assert(sizeof(Way<kShared, 16>) <= 64 && sizeof(Way<kWindow, 16>) <= 64, "segments");

// The reduction over the 32 lanes of each of 8 values: lane l is left with that of value l / 4.
template <bool MAX>
__device__ __forceinline__ float reduce8(const float (&v)[8], int lane) {
  float t[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool up = lane & 16;
    const float send = up ? v[j] : v[j + 4], keep = up ? v[j + 4] : v[j];
    const float recv = __shfl_xor_sync(0xffffffffu, send, 16);
    t[j] = MAX ? fmaxf(keep, recv) : keep + recv;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool up = lane & 8;
    const float send = up ? t[j] : t[j + 2], keep = up ? t[j + 2] : t[j];
    const float recv = __shfl_xor_sync(0xffffffffu, send, 8);
    t[j] = MAX ? fmaxf(keep, recv) : keep + recv;
  }
  {
    const bool up = lane & 4;
    const float send = up ? t[0] : t[1], keep = up ? t[1] : t[0];
    const float recv = __shfl_xor_sync(0xffffffffu, send, 4);
    t[0] = MAX ? fmaxf(keep, recv) : keep + recv;
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    const float recv = __shfl_xor_sync(0xffffffffu, t[0], o);
    t[0] = MAX ? fmaxf(t[0], recv) : t[0] + recv;
  }
  return t[0];
}

// 16-byte unit u (0..3) of row r in a 64-byte-swizzled block
__device__ __forceinline__ uint32_t sw64(int r, int u) {
  return (uint32_t)((r >> 3) * 512 + (r & 7) * 64 + ((u ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <int N>
struct Parts {
  Plan<Geo<N>>* plan;
  float* m;       // [2 RANGES][N]: slot 2k the first segment of range k, 2k + 1 its last; behind them (shared
  float* l;       // prefixes, from `whole` on) the row tiles that one range held whole
  float* o;       // [..][512]
  int64_t whole;
  template <int MODE>
  __device__ __forceinline__ int64_t row(const Way<MODE, N>& w, int k, int r) const {
    if constexpr (MODE == kShared) {
      if (w.whole()) return whole + w.s.part + (int64_t)w.rt * N + r;
    }
    return (int64_t)(2 * k + (w.seg == 0 ? 0 : 1)) * N + r;
  }
};

// kShared: the kernel of the prefixes is launched before this one, which runs beside it on the SMs that the
// plans leave it.  What this one needs of earlier launches are the plans, behind the word `ready`; it waits for
// that kernel when its own work is done, so that the join, which waits for this one, has both's parts.
template <int MODE, int N>
__global__ void __launch_bounds__(NTHREADS, 1)
    rows_kernel(const ChunkArgs a, const Parts<N> ps, unsigned* ready, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap smap) {
  using C = Cfg<N>;
  constexpr int NB = C::NB, STREAMS = C::STREAMS, RL = C::RL, RR = C::RR, NS = C::NS, NTF = C::NTF, S_COLS = C::S_COLS, T_O = C::T_O,
                O_COLS = C::O_COLS;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = (int)blockIdx.x;
  if constexpr (MODE == kShared) {
    // (no wait: the kernel of the prefixes sets it before it lets this one come)
    const bool there = load_acquire(ready) != 0u;
    if (!there && threadIdx.x == 0) atomicOr(a.err, ERR_TIMEOUT);
    if (!__syncthreads_and(there && k < ps.plan->n)) {  // nothing to do
      grid_dependents_launch();
      grid_dependency_wait();
      return;
    }
    grid_dependents_launch();
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_FLAGS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_FLAGS + 4);
  volatile uint32_t* facts = reinterpret_cast<volatile uint32_t*>(sm + C::OFF_FACTS);
  const uint32_t qb = smem_u32(sm + C::OFF_Q), lring = smem_u32(sm + C::OFF_L), rring = smem_u32(sm + C::OFF_R);
  auto fail = [&]() {
    *abort_flag = 1;
    atomicOr(a.err, ERR_TIMEOUT);
  };
  auto wait = [&](int bar, uint32_t parity) -> bool {
    return mbar_wait_warp(&bars[bar], parity & 1, abort_flag, WAIT_NS);
  };
  auto wait_block = [&](int jb) -> bool { return wait(C::B_LFULL + jb % RL, (uint32_t)(jb / RL)); };
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < NS; ++i) mbar_init(&bars[C::B_SEMPTY + i], C::SET);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[C::B_PFULL + i], C::SET);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[C::B_G + i], 4);
    mbar_init(&bars[C::B_QREADY], N_SOFT);
    mbar_init(&bars[C::B_EP], N_SOFT);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == W_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (MODE != kShared) {
    grid_dependency_wait();  // the plan
    grid_dependents_launch();
  }
  Way<MODE, N> w;
  if (k < ps.plan->n) w.start(a, *ps.plan, k);
  else w.left = 0;
  int gt = 0;  // key tiles of the range before this segment

  if (warp == W_TMA) {
    bool ok = true;
    int asked = 0, blocks = 0;  // tiles and Lc blocks whose barriers are armed
    for (; ok && w.more(); w.next(a)) {
      PageWindow pw;
      pw.from = -64;
      for (int i = 0; ok && i < w.n; ++i) {
        const int g = gt + i, tf = g % NTF, rs = g % RR;
        const int64_t page = 2 * (int64_t)(w.t + i);
        const int64_t s0 = pw.slot(a, w, page, lane, true), s1 = pw.slot(a, w, page + 1, lane, true);
        const uint32_t pages = (s0 >= 0 ? 1u : 0u) + (s1 >= 0 ? 1u : 0u);
        uint64_t* tb = &bars[C::B_TFULL + tf];
        if (!wait(C::B_REMPTY + rs, (uint32_t)(g / RR) ^ 1u)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          const int jb = 4 * g + blk, ls = jb % RL;
          if (!wait(C::B_LEMPTY + ls, (uint32_t)(jb / RL) ^ 1u)) {
            ok = false;
            break;
          }
          if (blk == 0) {
            // (tile g - NTF's scales are read: its context's MMAs, which come behind its weights, have freed
            // this block's slot or one before it)
            facts[tf] = (s0 >= 0 ? 1u : 0u) | (s1 >= 0 ? 2u : 0u);
            mbar_arrive_expect_tx_warp(tb, pages * (uint32_t)(2 * PAGE * 4 + PAGE * 64));
            asked = g + 1;
            const uint32_t sd = smem_u32(sm + C::OFF_SCR) + tf * TILE * 8, rd = rring + rs * RBLK;
            if (s0 >= 0) {
              tma_load_1d_warp(sd, &smap, (int)(2 * s0), tb);
              tma_load_2d_warp(rd, &rmap, DL, (int)s0, tb);
            }
            if (s1 >= 0) {
              tma_load_1d_warp(sd + 2 * PAGE * 4, &smap, (int)(2 * s1), tb);
              tma_load_2d_warp(rd + PAGE * 64, &rmap, DL, (int)s1, tb);
            }
          }
          const uint32_t ld = lring + ls * KBLK;
          mbar_arrive_expect_tx_warp(&bars[C::B_LFULL + ls], pages * (uint32_t)(PAGE * 128));
          blocks = jb + 1;
          if (s0 >= 0) tma_load_2d_warp(ld, &kmap, 128 * blk, (int)s0, &bars[C::B_LFULL + ls]);
          if (s1 >= 0) tma_load_2d_warp(ld + PAGE * 128, &kmap, 128 * blk, (int)s1, &bars[C::B_LFULL + ls]);
        }
      }
      gt += w.n;
    }
    if (!ok) {
      // let what was requested land before the CTA can leave
      if (lane == 0) fail();
      const int zero = 0;
      for (int i = blocks > RL ? blocks - RL : 0; i < blocks; ++i)
        (void)mbar_wait(&bars[C::B_LFULL + i % RL], (i / RL) & 1, &zero, WAIT_NS);
      for (int i = asked > NTF ? asked - NTF : 0; i < asked; ++i)
        (void)mbar_wait(&bars[C::B_TFULL + i % NTF], (i / NTF) & 1, &zero, WAIT_NS);
    }
    __syncwarp();
  } else if (warp == W_MMA) {
    const uint32_t id = idesc_f16(128, NB, false, false);  // e4m3 x e4m3 (format 0)
    bool ok = true;
    for (; ok && w.more(); w.next(a)) {
      if (!wait(C::B_QREADY, (uint32_t)w.seg)) {
        ok = false;
        break;
      }
      for (int i = 0; i < w.n; ++i) {
        const int g = gt + i, sb = g % NS;
        if (!wait(C::B_SEMPTY + sb, (uint32_t)(g / NS) ^ 1u)) {
          ok = false;
          break;
        }
        const uint32_t dl = tmem + sb * S_COLS, dr = dl + NB;
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          if (!wait_block(4 * g + blk)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = smem_desc(lring + ((4 * g + blk) % RL) * KBLK, 16, 1024, SW128);
          const uint64_t bd = smem_desc(qb + blk * NB * 128, 16, 1024, SW128);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8_warp(dl, ad + 2 * kk, bd + 2 * kk, id, (blk | kk) != 0);
        }
        if (!ok || !wait(C::B_TFULL + g % NTF, (uint32_t)(g / NTF))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = smem_desc(rring + (g % RR) * RBLK, 16, 512, SW64);
        const uint64_t bd = smem_desc(qb + 4 * NB * 128, 16, 512, SW64);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) mma_f8_warp(dr, ad + 2 * kk, bd + 2 * kk, id, kk != 0);
        mma_commit_warp(&bars[C::B_REMPTY + g % RR]);
        mma_commit_warp(&bars[C::B_SFULL + sb]);
      }
      gt += w.n;
    }
    if (!ok && lane == 0) fail();
    const int zero = 0;
    mma_commit_warp(&bars[C::B_DRAIN]);
    (void)mbar_wait(&bars[C::B_DRAIN], 0, &zero, WAIT_NS);
    __syncwarp();
  } else if (warp == W_CTX) {
    const uint32_t id = idesc_f16(128, NB, true, false);  // A = V, MN-major
    const uint32_t pb = smem_u32(sm + C::OFF_P);
    bool ok = true;
    for (; ok && w.more(); w.next(a)) {
      for (int i = 0; i < w.n; ++i) {
        const int g = gt + i, st = g % STREAMS, pbuf = g & 1;
        // (the blocks have long been there: their waits, for what they order, come before the one that counts)
#pragma unroll 1
        for (int m = 0; ok && m < 4; ++m) ok = wait_block(4 * g + m);
        if (!ok || !wait(C::B_PFULL + pbuf, (uint32_t)(g >> 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int ls = (4 * g + m) % RL;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_warp(tmem + T_O + st * O_COLS + m * NB, smem_desc(lring + ls * KBLK + kk * 4096, KBLK, 1024, SW128),
                        smem_desc(pb + st * NB * 128 + kk * 32, 16, 1024, SW128), id, (i >= STREAMS || kk > 0) ? 1u : 0u);
          mma_commit_warp(&bars[C::B_LEMPTY + ls]);
        }
        mma_commit_warp(&bars[C::B_ODONE + pbuf]);
      }
      gt += w.n;
    }
    if (!ok && lane == 0) fail();
    const int zero = 0;
    mma_commit_warp(&bars[C::B_DRAIN + 1]);
    (void)mbar_wait(&bars[C::B_DRAIN + 1], 0, &zero, WAIT_NS);
    __syncwarp();
  } else {
    // ---------------------------------------------------------- query, softmax, results
    const int sw = warp - W_SOFT;
    const int set = (sw >> 2) / (N / NH), grp = (sw >> 2) % (N / NH), wq = sw & 3;
    const int hb = grp * NH;                     // rows hb .. hb + 7
    const int row = (warp & 3) * 32 + lane;      // token of the tile (TMEM lane); channel of a block of O
    const int half = row >> 6;                   // its page
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    float* cs = reinterpret_cast<float*>(sm + C::OFF_CS);
    int* lim = reinterpret_cast<int*>(sm + C::OFF_LIM);
    float* refs = reinterpret_cast<float*>(sm + C::OFF_REF);
    float* lsum = reinterpret_cast<float*>(sm + C::OFF_LS);
    float* rmax = reinterpret_cast<float*>(sm + C::OFF_RMAX) + set * 8 * N;
    Way<MODE, N>* walk = reinterpret_cast<Way<MODE, N>*>(sm + C::OFF_WALK + sw * 64);
    uint32_t gph = 0, eph = 0;
    auto group_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[C::B_G + (sw >> 2)]);
      return wait(C::B_G + (sw >> 2), gph++);
    };
    auto all_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[C::B_EP]);
      return wait(C::B_EP, eph++);
    };
    // Rows sw, sw + 16 of a row tile's query, by this warp: two e4m3 terms on the scale that puts its largest value
    // in [128, 256), and c, which folds the scale back in, with sm_scale log2 e.  (Rows past the last one
    // are copies of it.)
    auto source = [&](const Way<MODE, N>& x, int hr, const uint16_t*& ql, const uint16_t*& qr) -> int {
      const int64_t r = (int64_t)x.rt * N + hr, rows = (int64_t)x.s.nq * a.H;
      const uint32_t at = (uint32_t)(r < rows ? r : rows - 1);
      const int tok = (int)(at / (uint32_t)a.H), head = (int)(at % (uint32_t)a.H);
      ql = a.q_lat + (x.s.q0 + tok) * a.ql_t + (int64_t)head * a.ql_h;
      qr = a.q_rope + (x.s.q0 + tok) * a.qr_t + (int64_t)head * a.qr_h;
      return tok;
    };
    auto load_row = [&](const Way<MODE, N>& x, int hr) {
      const uint16_t *ql, *qr;
      const int tok = source(x, hr, ql, qr);
      uint4 v[3];
      v[0] = __ldg(reinterpret_cast<const uint4*>(ql) + lane);
      v[1] = __ldg(reinterpret_cast<const uint4*>(ql) + 32 + lane);
      v[2] = lane < 8 ? __ldg(reinterpret_cast<const uint4*>(qr) + lane) : make_uint4(0u, 0u, 0u, 0u);
      // the largest magnitude, as bf16 bits (ordered; 0x7F80 and up is inf or NaN)
      uint32_t t2 = 0;
#pragma unroll
      for (int j = 0; j < 3; ++j)
        t2 = __vmaxu2(t2, __vmaxu2(__vmaxu2(v[j].x & 0x7FFF7FFFu, v[j].y & 0x7FFF7FFFu),
                                   __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t2 = __vmaxu2(t2, __shfl_xor_sync(0xffffffffu, t2, o));
      const uint32_t mx = (t2 & 0xFFFFu) > (t2 >> 16) ? (t2 & 0xFFFFu) : (t2 >> 16);
      const uint32_t nan = mx >= 0x7F80u ? 0x7F7F7F7Fu : 0u;
      int e = (int)(mx >> 7) - 127;
      e = e < -80 ? -80 : e;
      if (mx == 0 || nan != 0u) e = 7;
      const float sc = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      if (lane == 0) {
        const int at = ((x.seg & 1) * N) + hr;
        cs[at] = fmaxf(a.sm_scale * LOG2E * __uint_as_float((uint32_t)(127 - 7 + e) << 23), 1e-37f);
        lim[at] = limit_of(a, x.s, tok);
      }
      auto terms = [&](uint32_t w0, uint32_t w1, uint32_t& hi, uint32_t& lo) {
        const __half2 a0 = __floats2half2_rn(bf16_lo(w0) * sc, bf16_hi(w0) * sc);
        const __half2 a1 = __floats2half2_rn(bf16_lo(w1) * sc, bf16_hi(w1) * sc);
        uint16_t h0, l0, h1, l1;
        split_h2(*reinterpret_cast<const uint32_t*>(&a0), h0, l0);
        split_h2(*reinterpret_cast<const uint32_t*>(&a1), h1, l1);
        hi = ((uint32_t)h0 | ((uint32_t)h1 << 16)) | nan;
        lo = (uint32_t)l0 | ((uint32_t)l1 << 16);
      };
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        uint2 hi, lo;
        terms(v[j].x, v[j].y, hi.x, lo.x);
        terms(v[j].z, v[j].w, hi.y, lo.y);
        if (j < 2) {  // channels 256 j + 8 lane .. + 7: block 2 j + lane / 16, half of its unit lane % 16 / 2
          const uint32_t blk = qb + (2 * j + (lane >> 4)) * NB * 128;
          sts64(blk + sw128(hr, (lane & 15) >> 1) + (lane & 1) * 8, hi);
          sts64(blk + sw128(N + hr, (lane & 15) >> 1) + (lane & 1) * 8, lo);
        } else if (lane < 8) {
          const uint32_t blk = qb + 4 * NB * 128;
          sts64(blk + sw64(hr, lane >> 1) + (lane & 1) * 8, hi);
          sts64(blk + sw64(N + hr, lane >> 1) + (lane & 1) * 8, lo);
        }
      }
    };
    auto load_query = [&](const Way<MODE, N>& x) {
#pragma unroll 1
      for (int hr = sw; hr < N; hr += N_SOFT) load_row(x, hr);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[C::B_QREADY]);
    };
    // byte of weight [r][token `row`] in a K-major [NB x 128] block
    auto p_off = [&](int r) -> uint32_t {
      return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + (((row >> 4) ^ (r & 7)) << 4) + (row & 15));
    };
    const uint32_t to = tmem + lane_addr + T_O + hb;  // O of stream 0, its rows' hi terms

    bool ok = true, more = w.more();
    if (more) {
      *walk = w;  // (every lane, the same)
      __syncwarp();
      load_query(*walk);
    }
    while (ok && more) {
      const Way<MODE, N>& x = *walk;
      const int n_tiles = x.n, sp = (x.seg & 1) * N;
      if (!wait(C::B_QREADY, (uint32_t)x.seg)) {
        ok = false;
        break;
      }
      // per thread its token's share of the rows' sums; per lane row hb + lane % 8's reference, and the highest one so far
      uint64_t c2[NH / 2], lp[NH / 2];
      float mg = -INFINITY, mhi = -INFINITY;
#pragma unroll
      for (int h = 0; h < NH / 2; ++h) {
        c2[h] = pk2(cs[sp + hb + 2 * h], cs[sp + hb + 2 * h + 1]);
        lp[h] = pk2(0.f, 0.f);
      }
      const int lim0 = lim[sp];  // the first row sees least
      const int from = MODE == kWindow ? window_from(a, lim[sp + N - 1]) : 0;  // the last one's window begins last
      {
        // the next row tile's queries, into L2
        Way<MODE, N> wn = x;
        wn.next(a);
        if (wn.more() && lane < N / N_SOFT) {
          const uint16_t *ql, *qr;
          (void)source(wn, sw + N_SOFT * lane, ql, qr);
          prefetch_l2(ql, DL * 2);
          prefetch_l2(qr, DR * 2);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int i = (set + gt) % STREAMS; i < n_tiles; i += STREAMS) {
        const int g = gt + i, sb = g % NS, tf = g % NTF, kk = g / STREAMS;
        if (!wait(C::B_TFULL + tf, (uint32_t)(g / NTF)) || !wait(C::B_SFULL + sb, (uint32_t)(g / NS))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t have = facts[tf];
        bool full = have == 3u;
        int t = 0;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int t0 = x.at(2 * (x.t + i) + p) * PAGE;
          full = full && lim0 - t0 >= PAGE && !(MODE == kWindow && t0 < from && a.n_sink - t0 < PAGE);
          if (half == p) t = t0 + (row & (PAGE - 1));
        }
        const float2 s2 = *reinterpret_cast<const float2*>(sm + C::OFF_SCR + (tf * TILE + row) * 8);
        // (sLc made finite: out of sight it may be anything, in sight the NaN or infinity shows in sRc)
        const float sl = fminf(fmaxf(s2.x, 0.f), 3.0e38f), sr = fmaf(0.f, s2.x, s2.y);
        const float lg = fmaxf(lg2_approx(sl), LG_MIN);
        uint64_t u[NH / 2];  // sLc S_L + sRc S_R, of pairs of rows
        const uint64_t sl2 = pk2(sl, sl), sr2 = pk2(sr, sr), lg2 = pk2(lg, lg);
        {
          uint32_t r0[NH], r1[NH], r2[NH], r3[NH];
          const uint32_t sa = tmem + lane_addr + sb * S_COLS + hb;
          tmem_ld8(sa, r0);
          tmem_ld8(sa + N, r1);
          tmem_ld8(sa + 2 * N, r2);
          tmem_ld8(sa + 3 * N, r3);
          tmem_wait_ld();
          auto two = [](const uint32_t (&r)[NH], int h) {
            return pk2(__uint_as_float(r[2 * h]), __uint_as_float(r[2 * h + 1]));
          };
#pragma unroll
          for (int h = 0; h < NH / 2; ++h)
            u[h] = fma2(sr2, add2(two(r2, h), two(r3, h)), mul2(sl2, add2(two(r0, h), two(r1, h))));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::B_SEMPTY + sb]);
        if (!full) {
          const bool here = (have >> half) & 1u;
          auto sees = [&](int h) {
            const int l = lim[sp + hb + h];
            return here && t < l && (MODE != kWindow || t >= window_from(a, l) || t < a.n_sink);
          };
#pragma unroll
          for (int h = 0; h < NH / 2; ++h) {
            const float2 v = up2(u[h]);
            u[h] = pk2(sees(2 * h) ? v.x : -INFINITY, sees(2 * h + 1) ? v.y : -INFINITY);
          }
        }
        // the rows' largest weights in the tile: over the warp's tokens, then the four warps'
        {
          float y[NH];
#pragma unroll
          for (int h = 0; h < NH / 2; ++h) {
            const float2 v = up2(fma2(c2[h], u[h], lg2));
            y[2 * h] = v.x;
            y[2 * h + 1] = v.y;
          }
          const float ym = reduce8<true>(y, lane);
          if ((lane & 3) == 0) rmax[(kk & 1) * 4 * N + wq * N + hb + (lane >> 2)] = ym;
        }
        if (!group_sync()) {
          ok = false;
          break;
        }
        float f;  // the factor of what row hb + lane % 8 added up before
        bool moved;
        {
          const float* rm = rmax + (kk & 1) * 4 * N + hb + (lane & 7);
          const float ym = fmaxf(fmaxf(rm[0], rm[N]), fmaxf(rm[2 * N], rm[3 * N]));
          float mn = mg;
          if (ym > mg + TAU) {
            mn = ym;
          } else if (ym < mg - DOWN && ym >= mhi - DOWN_CAP) {
            mn = ym;
          }
          f = mn == mg ? 1.f : (mg > -INFINITY ? ex2_approx(mg - mn) : 0.f);
          mg = mn;
          mhi = fmaxf(mhi, mn);
          moved = __any_sync(0xffffffffu, f != 1.f);
        }
        if (moved) {
#pragma unroll
          for (int h = 0; h < NH / 2; ++h)
            lp[h] = mul2(lp[h], pk2(__shfl_sync(0xffffffffu, f, 2 * h), __shfl_sync(0xffffffffu, f, 2 * h + 1)));
        }
        const float mneg = P_LOG - fmaxf(mg, -3.0e38f);  // (nothing in sight so far: u is -inf, and p 0)
        uint32_t phi[2], plo[2];
#pragma unroll
        for (int h = 0; h < NH; h += 4) {
          float z[4];
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int q = (h + j) / 2;
            const float2 e = up2(fma2(c2[q], u[q], pk2(__shfl_sync(0xffffffffu, mneg, h + j),
                                                       __shfl_sync(0xffffffffu, mneg, h + j + 1))));
            const uint64_t p = pk2(ex2_approx(e.x), ex2_approx(e.y));
            lp[q] = add2(lp[q], p);
            const float2 v = up2(mul2(p, sl2));
            z[j] = v.x;
            z[j + 1] = v.y;
          }
          const __half2 x01 = __floats2half2_rn(z[0], z[1]), x23 = __floats2half2_rn(z[2], z[3]);
          uint16_t h01, l01, h23, l23;
          split_h2(*reinterpret_cast<const uint32_t*>(&x01), h01, l01);
          split_h2(*reinterpret_cast<const uint32_t*>(&x23), h23, l23);
          phi[h / 4] = (uint32_t)h01 | ((uint32_t)h23 << 16);
          plo[h / 4] = (uint32_t)l01 | ((uint32_t)l23 << 16);
        }
        // the stream's tile before: its weights are read, and O is at rest
        if (g >= STREAMS && !wait(C::B_ODONE + ((g - STREAMS) & 1), (uint32_t)((g - STREAMS) >> 1))) {
          ok = false;
          break;
        }
        if (moved && i >= STREAMS) {
          tc_fence_after();
          __syncwarp();
          float fh[NH];
#pragma unroll
          for (int h = 0; h < NH; ++h) fh[h] = __shfl_sync(0xffffffffu, f, h);
#pragma unroll 1
          for (int term = 0; term < 2; ++term) {
            uint32_t r[4][8];
#pragma unroll
            for (int m = 0; m < 4; ++m) tmem_ld8(to + set * O_COLS + m * NB + term * N, r[m]);
            tmem_wait_ld();
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
              for (int j = 0; j < 8; ++j) r[m][j] = __float_as_uint(__uint_as_float(r[m][j]) * fh[j]);
              tmem_st8(to + set * O_COLS + m * NB + term * N, r[m]);
            }
          }
          tmem_wait_st();
        }
        if (!full) {
          // some row does not see all of this tile: no NaN code may stay in it
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            if (!wait_block(4 * g + m)) ok = false;
            const uint32_t vb = lring + ((4 * g + m) % RL) * KBLK + (sw % C::SET) * (KBLK / C::SET) + lane * 16;
#pragma unroll
            for (int j = 0; j < KBLK / C::SET / 512; ++j) {
              const uint4 v = lds128(vb + j * 512);
              sts128(vb + j * 512, make_uint4(no_nan(v.x), no_nan(v.y), no_nan(v.z), no_nan(v.w)));
            }
          }
        }
        const uint32_t pb = smem_u32(sm + C::OFF_P) + set * NB * 128;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          sts8(pb + p_off(hb + h), phi[h / 4] >> (8 * (h & 3)));
          sts8(pb + p_off(N + hb + h), plo[h / 4] >> (8 * (h & 3)));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[C::B_PFULL + (g & 1)]);
      }
      if (!ok) break;
      // ---- the row tile's (or its part's) end
      const int last = gt + n_tiles - 1;
      Way<MODE, N> wn = x;
      wn.next(a);
      more = wn.more();
      if (more) {
        // (its last scores are there: nothing reads the query any more)
        if (!wait(C::B_SFULL + last % NS, (uint32_t)(last / NS))) {
          ok = false;
          break;
        }
        load_query(wn);
      }
      bool used[2];  // (a stream each, where there are two)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int l = last - ((last + b) & 1);  // the last even or odd tile
        used[b] = l >= gt;
        if (used[b] && !wait(C::B_ODONE + b, (uint32_t)(l >> 1))) ok = false;
      }
      if (!ok) break;
      {
        float l[NH];
#pragma unroll
        for (int h = 0; h < NH / 2; ++h) {
          const float2 v = up2(lp[h]);
          l[2 * h] = v.x;
          l[2 * h + 1] = v.y;
        }
        const float ls = reduce8<false>(l, lane);
        if ((lane & 3) == 0) lsum[(set * 4 + wq) * N + hb + (lane >> 2)] = ls;
        if (wq == 0 && lane < NH) refs[set * N + hb + lane] = mg;
      }
      if (!all_sync()) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool final = x.final();
      const int rows = (int)((int64_t)x.s.nq * a.H - (int64_t)x.rt * N);  // (from the row tile's first one on)
      const int64_t at0 = final ? x.s.q0 * a.H + (int64_t)x.rt * N : ps.row(x, k, 0);
      // the streams on the larger reference, a row a lane
      float f0, f1;
      {
        const int r = hb + (lane & 7);
        const float* p = lsum + r;
        float M = refs[r], L = (p[0] + p[N]) + (p[2 * N] + p[3 * N]);
        f0 = f1 = 1.f;
        if constexpr (STREAMS == 2) {
          const float m1 = refs[N + r];
          f0 = M >= m1 ? 1.f : ex2_approx(M - m1);
          f1 = m1 >= M ? 1.f : ex2_approx(m1 - M);
          M = fmaxf(M, m1);
          L = L * f0 + ((p[4 * N] + p[5 * N]) + (p[6 * N] + p[7 * N])) * f1;
        }
        M -= P_LOG;
        const float inv = L == 0.f ? 0.f : (final ? 1.f / L : 1.f);  // (a NaN stays one)
        f0 *= inv;
        f1 *= inv;
        if (set == 0 && wq == 0 && lane < NH && r < rows) {
          if (!final) {
            ps.m[at0 + r] = M;
            ps.l[at0 + r] = L;
          } else if (a.lse != nullptr) {
            a.lse[at0 + r] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
          }
        }
      }
#pragma unroll 1
      for (int mm = 0; mm < 4 / STREAMS; ++mm) {
        const int m = 4 / STREAMS * set + mm;  // (two streams' warps take half of the channels each)
        float v[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) v[h] = 0.f;
#pragma unroll
        for (int st = 0; st < STREAMS; ++st) {
          if (STREAMS == 2 && !used[st]) continue;
          uint32_t rh[8], rl[8];
          tmem_ld8(to + st * O_COLS + m * NB, rh);
          tmem_ld8(to + st * O_COLS + m * NB + N, rl);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float f = __shfl_sync(0xffffffffu, st == 0 ? f0 : f1, h);
            // (a factor of 0: nothing seen, or nothing that counts)
            if (f != 0.f) v[h] = fmaf(__uint_as_float(rh[h]) + __uint_as_float(rl[h]), f, v[h]);
          }
        }
        const int64_t at = (at0 + hb) * DL + m * 128 + row;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (hb + h >= rows) continue;
          if (final) reinterpret_cast<__nv_bfloat16*>(a.out)[at + h * DL] = __float2bfloat16_rn(v[h]);
          else ps.o[at + h * DL] = v[h];
        }
      }
      tc_fence_before();
      if (more && !all_sync()) {  // O, the references and the sums may be written again
        ok = false;
        break;
      }
      gt += n_tiles;
      *walk = wn;
      __syncwarp();
    }
    if (!ok && lane == 0) fail();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(tmem, 512);
  if constexpr (MODE == kShared) grid_dependency_wait();
}

constexpr int PLAN_NEAR = 4096;

// (base: in shared memory if it fits)
template <int MODE, int N>
__global__ void __launch_bounds__(PLAN_THREADS) rows_plan_kernel(const ChunkArgs a, Plan<Geo<N>>* plan, int64_t* base, int4* owner,
                                                         int most, bool alone) {
  grid_dependents_launch();
  __shared__ PlanScratch scratch;
  PlanSum sums{scratch};
  __shared__ int64_t near[PLAN_NEAR];
  plan_prefetch(a);
  if (threadIdx.x == 0) *a.err = 0;
  __syncthreads();
  if (MODE == kPlain && a.G > 0) (void)groups_bad(a, true);  // (groups too small to share anything)
  make_plan<MODE>(a, plan, a.B < PLAN_NEAR ? near : base, nullptr, 0, 0, a.B, most, sums, nullptr, owner, alone);
}

// The plans of a call with shared prefixes, each with a copy of the entries of its own, one behind the other:
// block 0 that of the prefixes (whose base the join reads), block 1 that of the sequences.  (The entries are
// worked on in shared memory if they fit.)
constexpr int ENTRIES_NEAR = 1024, SHARED_NEAR = 512;

template <int N>
__global__ void __launch_bounds__(PLAN_THREADS) rows_shared_plan_kernel(const ChunkArgs a, Plan<Geo<N>>* plan, int64_t* base,
                                                                int4* owner, int most, Plan<WideGeo>* prefix_plan,
                                                                int64_t* prefix_base, int4* prefix_owner, int prefix_most,
                                                                int clusters) {
  grid_dependents_launch();
  __shared__ PlanScratch scratch;
  PlanSum sums{scratch};
  __shared__ int64_t near[SHARED_NEAR];
  __shared__ ChunkEntry entries_near[ENTRIES_NEAR];
  const bool own = blockIdx.x == 1;
  const int n = a.G + a.B;
  plan_prefetch(a);
  if (own && threadIdx.x == 0) *a.err = 0;
  __syncthreads();
  ChunkEntry* entries = a.entries + (own ? n : 0);
  ChunkArgs c = a;
  c.entries = n <= ENTRIES_NEAR ? entries_near : entries;
  bool turns;
  const int split = make_entries<Geo<N>>(c, nullptr, sums, own, &turns, prefix_most, clusters);
  if (n <= ENTRIES_NEAR)
    for (int i = threadIdx.x; i < n; i += PLAN_THREADS) entries[i] = entries_near[i];
  if (own) {
    const int left = NUM_SMS - 4 * split;
    make_plan<kShared>(c, plan, a.B < SHARED_NEAR ? near : base, nullptr, a.G, n, a.B, most < left ? most : left, sums, nullptr,
                       owner, false, turns);
  } else {
    if (threadIdx.x == 0) prefix_plan->ready = 0u;
    make_plan<kShared>(c, prefix_plan, a.G < SHARED_NEAR ? near : prefix_base, a.G < SHARED_NEAR ? prefix_base : nullptr, 0, 0,
                       a.G, split, sums, nullptr, prefix_owner);
  }
}

// ------------------------------------------------------------------ host
constexpr int64_t OFF_PLAN = 256, OFF_PREFIX_PLAN = 4096, OFF_BASE = 5376;
static_assert(OFF_PLAN + sizeof(Plan<Geo<16>>) <= OFF_PREFIX_PLAN && OFF_PREFIX_PLAN + sizeof(Plan<WideGeo>) <= OFF_BASE,
              "plan area");

struct Layout {
  int most, prefix_most;         // ranges, and the prefixes' clusters
  int64_t tiles;                 // row tiles at most
  bool alone;                    // a range for each of them
  int64_t part_rows;             // room for rows that have parts
  int64_t owner, entries, prefix_base, prefix_owner, m, prefix_slots, slots, bytes;
  int64_t rows() const { return prefix_slots + slots + 2 * part_rows; }
};
// Short row tiles, if an SM holds one at most, are a range's each: they have no parts, and nothing is launched to
// join them.  Up to 4 key tiles, or 6 where a row tile has less than three SMs.  (us, with ranges of their own and of
// equal length: tokens of 16 heads, window 128: one 14.4 and 15.2, 64 15.0 and 16.4; 256: one 16.5 and 15.9 (of which
// the launch saves the host 1.6), 64 17.0 and 20.1, 140 18.0 and 25.3; 450: one 19.7 and 15.9; 512: 64 20.5 and 21.9.)
constexpr int64_t ALONE_KEYS = 4, ALONE_KEYS_MANY = 6;

template <int N>
int64_t row_tiles_at_most(int B, int H, int64_t total_q) {
  const int64_t by_row = total_q * H / N + B, by_token = total_q * ((H + N - 1) / N);
  return by_row < by_token ? by_row : by_token;
}

// (G < 0: no shared prefixes)
template <int N>
Layout layout_of(int B, int H, int64_t total_q, int64_t keys, int G) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  Layout w{};
  w.tiles = row_tiles_at_most<N>(B, H, total_q);
  const int64_t units = w.tiles * keys;
  w.alone = G < 0 && keys <= (3 * w.tiles > NUM_SMS ? ALONE_KEYS_MANY : ALONE_KEYS) && w.tiles <= NUM_SMS;
  w.most = (int)(w.alone ? w.tiles : (units < 1 ? 1 : (units < NUM_SMS ? units : NUM_SMS)));
  int64_t at = OFF_BASE + up((int64_t)(B + 1) * 8);
  w.owner = at;
  at += up(w.tiles * (int64_t)sizeof(int4));
  if (G >= 0) {
    const int64_t rows = total_q * H, few = (int64_t)PART_ROWS * B, cap = 1 << 20, wide = rows / WideGeo::ROWS + G;
    w.part_rows = rows < few ? rows : few;
    if (w.part_rows > cap) w.part_rows = cap;
    const int64_t u = wide * keys / WideGeo::MIN_TILES;
    w.prefix_most = (int)(u < 1 ? 1 : (u < WideGeo::RANGES ? u : WideGeo::RANGES));
    w.entries = at;
    at += up(2 * (int64_t)(G + B) * (int64_t)sizeof(ChunkEntry));
    w.prefix_base = at;
    at += up((int64_t)(G + 1) * 8);
    w.prefix_owner = at;
    at += up(wide * (int64_t)sizeof(int4));
    w.prefix_slots = 2 * (int64_t)w.prefix_most * WideGeo::ROWS;
  }
  w.m = at;
  w.slots = (w.most > 1 && !w.alone) || G >= 0 ? 2 * (int64_t)w.most * N : 0;  // (one range cuts no row tile)
  w.bytes = at + w.rows() * (8 + DL * 4);
  return w;
}
int64_t all_keys(int max_blocks) { return ((int64_t)max_blocks * PAGE + TILE - 1) / TILE; }
// (a row tile's tokens lie within N of one another, and its window's keys begin and end inside a page)
int64_t window_keys(int max_blocks, int64_t window, int64_t n_sink, int N) {
  const int64_t all = all_keys(max_blocks), pages = (n_sink + PAGE - 1) / PAGE + (window + N - 2 + PAGE - 1) / PAGE + 1;
  return (pages + 1) / 2 < all ? (pages + 1) / 2 : all;
}

// Row tiles of 32: where sequences have more than 16 rows on average.  (us, in row tiles of 16 and of 32: 32
// tokens of 16 heads, window 2048, 24.3 and 26.0, of 20 heads 30.0 and 26.3; 64 with a window of 8192 71 and
// 77, 119 and 79.  Of one token of 128 heads with a window of 1000 17.2 and 18.2, of 8192 21.2 and 20.2.)
bool wide(int B, int H, int64_t total_q) { return total_q * H > 16 * (int64_t)B; }

// Whether a call may have a prefix whose sharing pays, in the plan's terms: what all that its sizes allow for costs apart,
// and with all of it one prefix.  Less than GAIN cycles between them, and the call goes without the plan that weighs and
// the prefixes' launch, which take 5 us.  (64 tokens of 16 heads behind 2000 keys 35 us with them, 30 without; behind
// 4000, shared, 42, and 40; 8 behind 16384 32 and 26; 16 behind 16384, shared, 44, and 39.)
constexpr int64_t GAIN = 12000;
template <int N>
bool pays_to_share(int B, int H, int64_t total_q, int max_blocks) {
  const int64_t keys = all_keys(max_blocks), wide = (total_q * H + WideGeo::ROWS - 1) / WideGeo::ROWS;
  const int64_t apart = row_tiles_at_most<N>(B, H, total_q) * (keys + Geo<N>::SWITCH) * NARROW<Geo<N>> / NUM_SMS + START;
  return apart > wide * (keys + WideGeo::SWITCH) * WIDE_CYCLES / WideGeo::RANGES + START_WIDE + JOIN_MORE + GAIN;
}
bool may_share(int B, int H, int64_t total_q, int max_blocks, int G, int share) {
  if (G < 1 || B < 2 || share == KV8_SHARE_ALWAYS) return G > 0 && B > 1;
  return wide(B, H, total_q) ? pays_to_share<32>(B, H, total_q, max_blocks) : pays_to_share<16>(B, H, total_q, max_blocks);
}

template <int MODE, int N>
cudaError_t launch(ChunkArgs a, const Layout& w, void* workspace, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  int done = 0;
  cudaError_t e = per_device(memo, [](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(rows_kernel<MODE, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<N>::SMEM);
  }, &done);
  if (e != cudaSuccess) return e;
  char* p = static_cast<char*>(workspace);
  a.err = reinterpret_cast<unsigned*>(p);
  float* m = reinterpret_cast<float*>(p + w.m);
  float* l = m + w.rows();
  float* o = l + w.rows();
  Parts<N> ps;
  ps.plan = reinterpret_cast<Plan<Geo<N>>*>(p + OFF_PLAN);
  ps.m = m + w.prefix_slots;
  ps.l = l + w.prefix_slots;
  ps.o = o + w.prefix_slots * DL;
  ps.whole = w.slots;
  int64_t* base = reinterpret_cast<int64_t*>(p + OFF_BASE);
  int64_t* prefix_base = reinterpret_cast<int64_t*>(p + w.prefix_base);
  int4* owner = reinterpret_cast<int4*>(p + w.owner);
  int4* prefix_owner = reinterpret_cast<int4*>(p + w.prefix_owner);
  DecodeArgs d{};  // what the cache's tensor maps are made from
  d.codes = a.codes;
  d.scales = a.scales;
  d.block_table = a.block_table;
  d.n_blocks = a.n_blocks;
  unsigned* ready = nullptr;
  CUtensorMap kmap, rmap, smap;
  if ((e = make_cache_map(d, &kmap)) != cudaSuccess || (e = make_rc_map(d, &rmap)) != cudaSuccess ||
      (e = make_scale_map(d, &smap)) != cudaSuccess)
    return e;
  if constexpr (MODE == kShared) {
    int fit = 0;
    if ((e = prefix_capacity(&fit)) != cudaSuccess) return e;
    const int clusters = w.prefix_most < fit ? w.prefix_most : fit;
    a.entries = reinterpret_cast<ChunkEntry*>(p + w.entries);
    a.part_rows = w.part_rows;
    Plan<WideGeo>* prefix_plan = reinterpret_cast<Plan<WideGeo>*>(p + OFF_PREFIX_PLAN);
    rows_shared_plan_kernel<N><<<2, PLAN_THREADS, 0, s>>>(a, ps.plan, base, owner, w.most, prefix_plan, prefix_base,
                                                           prefix_owner, clusters, fit);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_prefixes(a, PrefixParts{prefix_plan, m, l, o, w.prefix_slots + w.slots}, clusters, kmap, rmap, smap, s);
    if (e != cudaSuccess) return e;
    ready = &prefix_plan->ready;
  } else {
    rows_plan_kernel<MODE, N><<<1, PLAN_THREADS, 0, s>>>(a, ps.plan, base, w.alone ? nullptr : owner, w.most, w.alone);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  e = launch_after_prep(rows_kernel<MODE, N>, w.most, NTHREADS, Cfg<N>::SMEM, s, a, ps, ready, kmap, rmap, smap);
  if (e != cudaSuccess || w.alone || (MODE != kShared && w.most == 1)) return e;
  return launch_parts_join<MODE, N>(a, PartsJoin{&ps.plan->tiles, owner, ps.m, ps.l, ps.o, ps.whole, prefix_base, prefix_owner,
                                                 w.prefix_slots}, w.tiles, w.most, s);
}

}  // namespace

int64_t rows_window_workspace(int B, int H, int64_t total_q, int max_blocks, int window, int n_sink) {
  return wide(B, H, total_q) ? layout_of<32>(B, H, total_q, window_keys(max_blocks, window, n_sink, 32), -1).bytes
                             : layout_of<16>(B, H, total_q, window_keys(max_blocks, window, n_sink, 16), -1).bytes;
}
cudaError_t launch_rows_window(const ChunkArgs& a, void* workspace, cudaStream_t s) {
  if (wide(a.B, a.H, a.total_q))
    return launch<kWindow, 32>(a, layout_of<32>(a.B, a.H, a.total_q, window_keys(a.max_blocks, a.window, a.n_sink, 32), -1),
                               workspace, s);
  return launch<kWindow, 16>(a, layout_of<16>(a.B, a.H, a.total_q, window_keys(a.max_blocks, a.window, a.n_sink, 16), -1),
                             workspace, s);
}

int64_t rows_shared_workspace(int B, int H, int64_t total_q, int max_blocks, int G) {
  const int64_t keys = all_keys(max_blocks);
  const int g = may_share(B, H, total_q, max_blocks, G, KV8_SHARE_ALWAYS) ? G : -1;
  return wide(B, H, total_q) ? layout_of<32>(B, H, total_q, keys, g).bytes : layout_of<16>(B, H, total_q, keys, g).bytes;
}
cudaError_t launch_rows_shared(const ChunkArgs& a, void* workspace, cudaStream_t s) {
  const int64_t keys = all_keys(a.max_blocks);
  const bool w32 = wide(a.B, a.H, a.total_q);
  if (!may_share(a.B, a.H, a.total_q, a.max_blocks, a.G, a.share))
    return w32 ? launch<kPlain, 32>(a, layout_of<32>(a.B, a.H, a.total_q, keys, -1), workspace, s)
               : launch<kPlain, 16>(a, layout_of<16>(a.B, a.H, a.total_q, keys, -1), workspace, s);
  return w32 ? launch<kShared, 32>(a, layout_of<32>(a.B, a.H, a.total_q, keys, a.G), workspace, s)
             : launch<kShared, 16>(a, layout_of<16>(a.B, a.H, a.total_q, keys, a.G), workspace, s);
}

}  // namespace kv8
