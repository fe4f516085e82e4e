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
//   sixteen softmax warps in two groups that take alternate tiles.  A thread owns a row
//         (its TMEM lane) and 64 tokens: u = sLc S_L + sRc S_R, its own running maximum
//         m and denominator l of p = 2^(c u - m), and the weights
//         g'_t = 2^(c u_t + log2 sLc_t - M_g) P_TOP as f16.  The reference M_g follows the
//         largest weight p_t sLc_t of the row, not the largest score, so that the top weights
//         fill the e4m3 range however the row scales differ; it is lazy (moves up by more
//         than 2^TAU, down by more than 2^DOWN) and is handed from tile to tile, and with it
//         from group to group, through shared memory.  g' goes to the row's context CTA by
//         asynchronous remote stores.
// Context pair (ranks 2, 3), per key tile:
//   sixteen warps split g' into two e4m3 terms (hi + residual) in place, as the A operand,
//         and rescale the rows of O whose M_g moved;
//   O += g'_hi V + g'_lo V    M = 256, N = 256 channels (each CTA holds half of them as
//         B, the cache tile read MN-major), 16 MMAs into all 512 TMEM columns.
//   At the end of a row tile the rows are scaled by 2^(M_g - m) / (P_TOP l), rounded to
//   bf16 and written; where the range holds only part of a row tile's keys, the partial
//   (f32 o, m, l) goes to the workspace and a second launch joins the parts.
//
// Keys that a row does not see have weight 0; since 0 x NaN is NaN, the context warps also
// clear NaN codes from V tiles that some row of the tile sees only in part (where every row
// sees a NaN, its NaN denominator carries it).
//
// The units of all row tiles are cut into equal ranges, one per cluster, by a one-CTA plan
// kernel from q_start and seq_lens on the device.  Every wait is bounded (2 s): on a timeout
// the CTA flags the workspace error word, drains its MMAs and copies and meets its cluster
// at the closing barrier.
#include <cuda.h>
#include <cuda_bf16.h>

#include "kv8_common.cuh"
#include "tc_ptx.cuh"

namespace kv8 {
namespace {

using namespace ptx;

constexpr int ROWS = 256;                    // rows of a row tile: 128 per CTA of a pair
constexpr int CROWS = 128;
constexpr int W_TMA = 0, W_MMA = 1, W_LANE = 2;
constexpr int N_LANE_WARPS = 16;             // four per TMEM lane quarter
constexpr int NTHREADS = (W_LANE + N_LANE_WARPS) * 32;
constexpr int MAX_CLUSTERS = NUM_SMS / 4;
constexpr int MIN_TILES = 2;                 // key tiles that are worth a cluster of their own
constexpr int BLK = PAGE * 128;              // 8 KB: [64 tokens x 128 bytes]
constexpr int RBLK = PAGE * DR;              // 4 KB: [64 tokens x 64 bytes]
constexpr int KTILE = 4 * BLK + RBLK;        // a score CTA's page of a tile: 36 KB
constexpr int NK = 3;                        // K ring, in tiles; loaded and freed in two halves
constexpr int NSC = 4;                       // row-scale ring, in tiles (even: a slot is always the same group's)
constexpr int VBLK = TILE * 128;             // 16 KB: [128 tokens x 128 channels]
constexpr int VTILE = 2 * VBLK;              // a context CTA's half of the channels
constexpr int NVT = 4;                       // V ring, in tiles
constexpr int SUB = 64;                      // tokens of a softmax thread's share of a tile
constexpr int OP_ATOM = CROWS * 128;         // 16 KB: [128 rows x 128 tokens], e4m3
constexpr int P_F = CROWS * TILE * 2;        // payload: g' f16 (eight 4 KB chunks), then rescale factors
constexpr int P_BYTES = P_F + CROWS * 4;
constexpr int P_STRIDE = 33 * 1024;
constexpr int CHUNK = 32 * SUB * 2;          // 4 KB: 32 rows x 64 tokens
constexpr float TAU = 1.0f;
constexpr float P_TOP = 128.0f;              // g' <= 2^TAU * P_TOP = 256 <= 448
constexpr float DOWN = 10.0f;
constexpr float DOWN_CAP = 60.0f;
constexpr float K_CAP = 114.0f;              // log2 of the factor that takes p to p / 2^(M_g - m)
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// mbarriers (the same offsets in all four CTAs: commits are multicast)
constexpr int B_KFULL = 0;                   // [2 NK] rank 0: both CTAs' halves of a K half tile loaded
constexpr int B_KEMPTY = B_KFULL + 2 * NK;   // [2 NK] ranks 0, 1: consumed
constexpr int B_SCFULL = B_KEMPTY + 2 * NK;  // [NSC] score: row scales of a tile loaded
constexpr int B_SFULL = B_SCFULL + NSC;      // [2] ranks 0, 1: S of a tile in TMEM
constexpr int B_SEMPTY = B_SFULL + 2;        // [2] rank 0: S read (8 warps x 2 CTAs)
constexpr int B_QREADY = B_SEMPTY + 2;       // rank 0: the row tile's query in place (16 warps x 2)
constexpr int B_PX = B_QREADY + 1;           // [4] score: the four warps of a lane quarter meet
constexpr int B_EX = B_PX + 4;               // [2 groups][4] score: a group's two warps of a quarter
constexpr int B_CH = B_EX + 8;               // [2 groups][4] score: a tile's M_g published
constexpr int B_PFREE = B_CH + 8;            // [2] ranks 0, 1: payload buffer free
constexpr int B_PFULL = B_PFREE + 2;         // [2] context: payload arrived
constexpr int B_VT = B_PFULL + 2;            // [NVT] context: V tile loaded
constexpr int B_VEMPTY = B_VT + NVT;         // [NVT] ranks 2, 3: consumed
constexpr int B_CVT = B_VEMPTY + NVT;        // context: every warp has read the payload
constexpr int B_RS = B_CVT + 1;              // [2] rank 2: operand, V and O half ready (16 warps x 2)
constexpr int B_ODONE = B_RS + 2;            // [2] ranks 2, 3: MMAs of an O half done
constexpr int NRF = 4;
constexpr int B_RF = B_ODONE + 2;            // [NRF] context: row factors of a finished row tile arrived
constexpr int B_DRAIN = B_RF + NRF;          // every MMA done
constexpr int NBAR = B_DRAIN + 1;

// shared memory (dynamic, 1024-byte aligned)
constexpr int OFF_FLAGS = 512;               // tmem base, abort flag
constexpr int OFF_FACTS = OFF_FLAGS + 16;    // [4] pages present in the tiles of the ring
constexpr int OFF_XMAX = 1024;               // score: [2 phases][2 groups][2 halves][128] tile maxima
constexpr int OFF_MG = OFF_XMAX + 4096;      // score: [2][128] M_g after a tile
constexpr int OFF_XL = OFF_MG + 1024;        // score: [4 parts][128] (m, l)
constexpr int OFF_XQ = OFF_XL + 4096;        // score: [4 parts][128] query maxima
constexpr int OFF_SC = OFF_XQ + 2048;        // score: [NSC][128][2] row scales
constexpr int OFF_PL = OFF_SC + NSC * 1024;  // score: [16 warps][3][64] sLc, sRc, log2 sLc
constexpr int OFF_QL = (OFF_PL + 16 * 768 + 1023) / 1024 * 1024;  // score: lo of Lc, four atoms
constexpr int OFF_QR = OFF_QL + 4 * OP_ATOM;                      // score: Rc, hi | lo
constexpr int OFF_K = OFF_QR + OP_ATOM;
constexpr int TOTAL_S = OFF_K + NK * KTILE;
constexpr int OFF_RF = 1024;                 // context: [NRF][128] row factors
constexpr int OFF_P = 4096;                  // context: two payloads / operands
constexpr int OFF_V = OFF_P + 2 * P_STRIDE;
constexpr int TOTAL_C = OFF_V + NVT * VTILE;
constexpr int SMEM = TOTAL_S > TOTAL_C ? TOTAL_S : TOTAL_C;
// TMEM columns of a score CTA
constexpr int T_SL = 0, T_SR = 256, T_QH = 384;
static_assert(NBAR * 8 <= OFF_FLAGS && OFF_RF + NRF * 512 <= OFF_P, "shared memory layout");
static_assert(OFF_K % 1024 == 0 && KTILE % 1024 == 0 && OFF_V % 1024 == 0 && P_STRIDE % 1024 == 0, "swizzle atoms");
static_assert(P_BYTES <= P_STRIDE && 2 * OP_ATOM <= P_STRIDE, "payload and operand share a buffer");
static_assert(SMEM <= 232448, "shared memory above the per-CTA limit");

// ------------------------------------------------------------------ work
// Plan of cluster k: its first row tile (sequence b, row tile rt, nt key tiles of
// which off come before the range), the unit where the range starts and its length.
struct PlanEntry {
  int32_t b, rt, nt, off;
  int64_t x, cnt;
};
struct Plan {
  int64_t n_clusters;
  int64_t pad[3];
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
  return lim > 0 ? (lim + TILE - 1) / TILE : 1;
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

// One CTA: row tiles before each sequence (base), the units of every row tile,
// their total, and the row tile that each cluster's range starts in.
__global__ void __launch_bounds__(1024) plan_kernel(const ChunkArgs a, Plan* plan, int64_t* base, int clusters) {
  grid_dependents_launch();
  __shared__ int64_t tmp[32];
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
  int64_t mine = 0, total;
  for (int64_t p = threadIdx.x; p < pairs; p += 1024) mine += tiles(p);
  (void)plan_sum(mine, tmp, &total);
  int64_t nc = total / MIN_TILES;
  nc = nc > clusters ? clusters : (nc < 1 ? (total > 0 ? 1 : 0) : nc);
  if (threadIdx.x == 0) plan->n_clusters = nc;
  int64_t at = 0;
  for (int64_t p0 = 0; p0 < pairs; p0 += 1024) {
    const int64_t n = tiles(p0 + threadIdx.x);
    int64_t sum;
    const int64_t S = at + plan_sum(n, tmp, &sum) - n;
    int64_t k = n > 0 ? S * nc / total : nc;
    while (k < nc && k * total / nc < S) ++k;
    for (; k < nc; ++k) {
      const int64_t x = k * total / nc;
      if (x >= S + n) break;
      PlanEntry e;
      e.b = b;
      e.rt = rt;
      e.nt = (int32_t)n;
      e.off = (int32_t)(x - S);
      e.x = x;
      e.cnt = (k + 1) * total / nc - x;
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
  __device__ __forceinline__ void start(const ChunkArgs& a, const PlanEntry& e) {
    b = e.b;
    rt = e.rt;
    nt = e.nt;
    t = e.off;
    left = e.cnt;
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
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Two e4m3 terms of four f32 values on their scale: hi = e4m3(x), lo = e4m3(x - hi).
__device__ __forceinline__ void split4(const float* x, uint32_t& hi, uint32_t& lo) {
  const uint16_t h01 = f32x2_to_e4m3x2(x[0], x[1]), h23 = f32x2_to_e4m3x2(x[2], x[3]);
  const uint32_t f01 = e4m3x2_to_f16x2(h01), f23 = e4m3x2_to_f16x2(h23);
  const float2 d01 = __half22float2(*reinterpret_cast<const __half2*>(&f01));
  const float2 d23 = __half22float2(*reinterpret_cast<const __half2*>(&f23));
  const uint16_t l01 = f32x2_to_e4m3x2(x[0] - d01.x, x[1] - d01.y);
  const uint16_t l23 = f32x2_to_e4m3x2(x[2] - d23.x, x[3] - d23.y);
  hi = (uint32_t)h01 | ((uint32_t)h23 << 16);
  lo = (uint32_t)l01 | ((uint32_t)l23 << 16);
}
// The same of an f16 pair (the residual of the hi term is exact in f16).
__device__ __forceinline__ void split_h2(uint32_t x, uint16_t& hi, uint16_t& lo) {
  const __half2 v = *reinterpret_cast<const __half2*>(&x);
  hi = f16x2_to_e4m3x2(v);
  const uint32_t d = e4m3x2_to_f16x2(hi);
  lo = f16x2_to_e4m3x2(__hsub2(v, *reinterpret_cast<const __half2*>(&d)));
}
// NaN codes (0x7F, 0xFF) of four bytes set to 0
__device__ __forceinline__ uint32_t no_nan(uint32_t v) {
  return v & ~__vcmpeq4(v & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// byte offset of 16-byte unit u (0..7) of row r (0..31) in a payload chunk
__device__ __forceinline__ uint32_t prow(int r, int u) {
  return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4));
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

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_SEMPTY + i], 16);
    mbar_init(&bars[B_QREADY], 2 * N_LANE_WARPS);
    for (int i = 0; i < 4; ++i) mbar_init(&bars[B_PX + i], 4);
    for (int i = 0; i < 8; ++i) mbar_init(&bars[B_EX + i], 2);
    mbar_init(&bars[B_CVT], N_LANE_WARPS);
    for (int i = 0; i < 2; ++i) mbar_init(&bars[B_RS + i], 2 * N_LANE_WARPS);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (rank >= 2) {  // what the context CTAs expect first
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&bars[B_PFULL + i], P_BYTES);
      for (int i = 0; i < NRF; ++i) mbar_arrive_expect_tx(&bars[B_RF + i], CROWS * 4);
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
  const bool work = k < ws.plan->n_clusters;
  Walk w;
  if (work) w.start(a, ws.plan->e[k]);
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
          // the row scales' slot held tile g - 4: the MMAs of tile g - 3, done by now, began
          // their last ones when the softmax warps had read S, and the scales, of tile g - 4
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
      }
      // every MMA of the pair is done and its commits have landed here
      const int zero = 0;
      (void)mbar_wait(&bars[B_DRAIN], 0, &zero, 4 * WAIT_NS);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- query and softmax
      const int q = warp & 3;                 // TMEM lane quarter
      const int part = (warp - W_LANE) >> 2;  // quarter of the query's channels
      const int grp = part >> 1, sub = part & 1;  // tiles of this parity; half of the tile's tokens
      const int hh = q * 32 + lane;           // row of this CTA = TMEM lane
      const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
      float* xmax = reinterpret_cast<float*>(sm + OFF_XMAX);
      float* mgs = reinterpret_cast<float*>(sm + OFF_MG);
      float2* xl = reinterpret_cast<float2*>(sm + OFF_XL);
      float* xq = reinterpret_cast<float*>(sm + OFF_XQ);
      float* pl = reinterpret_cast<float*>(sm + OFF_PL) + (warp - W_LANE) * 192;
      const uint32_t qready = map_to(smem_u32(&bars[B_QREADY]), 0);
      const uint32_t sempty = map_to(smem_u32(&bars[B_SEMPTY + grp]), 0);
      const uint32_t ctx_p = map_to(smem_u32(sm + OFF_P), rank + 2) + grp * P_STRIDE;
      const uint32_t ctx_pfull = map_to(smem_u32(&bars[B_PFULL + grp]), rank + 2);
      const uint32_t ctx_rf = map_to(smem_u32(sm + OFF_RF), rank + 2);
      const uint32_t ctx_rfbar = map_to(smem_u32(&bars[B_RF]), rank + 2);
      uint32_t px = 0;
      auto quarter_sync = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_PX + q]);
        return wait(B_PX + q, px++);
      };
      bool ok = true;
      for (; ok && w.more(); w.next(a)) {
        // ---- the query of this row: 128 channels of Lc and 16 of Rc per thread, as two
        // e4m3 terms on the scale that puts the row's largest value in [128, 256)
        const int64_t r = (int64_t)w.rt * ROWS + rank * CROWS + hh;
        const bool real = r < (int64_t)w.s.nq * a.H;
        const int tok = real ? (int)((uint32_t)r / (uint32_t)a.H) : w.s.nq - 1;
        const int head = real ? (int)((uint32_t)r % (uint32_t)a.H) : 0;
        const int lim = limit_of(a, w.s, tok);
        float c;
        {
          const uint4* pq = reinterpret_cast<const uint4*>(a.q_lat + (w.s.q0 + tok) * a.ql_t + head * a.ql_h + part * 128);
          const uint4* pr = reinterpret_cast<const uint4*>(a.q_rope + (w.s.q0 + tok) * a.qr_t + head * a.qr_h + part * 16);
          // the largest magnitude, as bf16 bits (an ordered integer; 0x7F80 and up is inf or NaN)
          uint32_t top = 0;
          const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
          auto most = [&](const uint4& v) {
            top = __vmaxu2(__vmaxu2(top, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu));
            top = __vmaxu2(top, v.w & 0x7FFF7FFFu);
          };
#pragma unroll
          for (int j = 0; j < 16; ++j) most(real ? __ldg(pq + j) : zero4);
#pragma unroll
          for (int j = 0; j < 2; ++j) most(real ? __ldg(pr + j) : zero4);
          top = (top & 0xFFFFu) > (top >> 16) ? (top & 0xFFFFu) : (top >> 16);
          xq[part * CROWS + hh] = __uint_as_float(top);
          if (!quarter_sync()) {
            ok = false;
            break;
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t v = __float_as_uint(xq[p * CROWS + hh]);
            top = v > top ? v : top;
          }
          const bool nan = top >= 0x7F80u;
          // exponent e: max in [2^e, 2^(e+1)); the scale 2^(7 - e), at most 2^87
          int e = (int)(top >> 7) - 127;
          e = e < -80 ? -80 : e;
          if (top == 0 || nan) e = 7;
          const float sc = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
          c = fmaxf(a.sm_scale * LOG2E * __uint_as_float((uint32_t)(127 - 7 + e) << 23), 1e-37f);
          // (a row with a NaN or an infinity is all NaN codes, and c = sm log2 e)
          auto terms = [&](uint32_t w0, uint32_t w1, uint32_t& hi, uint32_t& lo) {
            const float v[4] = {bf16_lo(w0) * sc, bf16_hi(w0) * sc, bf16_lo(w1) * sc, bf16_hi(w1) * sc};
            split4(v, hi, lo);
            if (nan) hi = 0x7F7F7F7Fu;
          };
          const uint32_t qlo = smem_u32(sm + OFF_QL) + part * OP_ATOM, qrp = smem_u32(sm + OFF_QR);
#pragma unroll 1
          for (int hl = 0; hl < 4; ++hl) {  // 32 channels, from cache now
            uint4 x[4];
            uint32_t hw[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = real ? __ldg(pq + 4 * hl + j) : zero4;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t lw[4];
              terms(x[2 * u].x, x[2 * u].y, hw[4 * u], lw[0]);
              terms(x[2 * u].z, x[2 * u].w, hw[4 * u + 1], lw[1]);
              terms(x[2 * u + 1].x, x[2 * u + 1].y, hw[4 * u + 2], lw[2]);
              terms(x[2 * u + 1].z, x[2 * u + 1].w, hw[4 * u + 3], lw[3]);
              sts128(qlo + sw128(hh, 2 * hl + u), make_uint4(lw[0], lw[1], lw[2], lw[3]));
            }
            __syncwarp();
            tmem_st8(tmem + lane_addr + T_QH + part * 32 + 8 * hl, hw);
          }
          const uint4 y0 = real ? __ldg(pr) : zero4, y1 = real ? __ldg(pr + 1) : zero4;
          uint32_t hr[4], lr[4];
          terms(y0.x, y0.y, hr[0], lr[0]);
          terms(y0.z, y0.w, hr[1], lr[1]);
          terms(y1.x, y1.y, hr[2], lr[2]);
          terms(y1.z, y1.w, hr[3], lr[3]);
          sts128(qrp + sw128(hh, part), make_uint4(hr[0], hr[1], hr[2], hr[3]));
          sts128(qrp + sw128(hh, 4 + part), make_uint4(lr[0], lr[1], lr[2], lr[3]));
          __syncwarp();
          tmem_wait_st();
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(qready);
        }
        const uint64_t c2 = pk2(c, c);
        float m = -INFINITY, l = 0.f;   // this thread's tokens
        float mghi = -INFINITY;
        for (int i = 0; i < w.n; ++i) {
          const int g = gt + i;
          if ((g & 1) != grp) continue;
          const int sc = g % NSC;
          if (!wait(B_SCFULL + sc, (uint32_t)(g / NSC))) {
            ok = false;
            break;
          }
          // this half's row scales in planar order, and log2 sLc (this warp's copy)
          const bool here = (facts[sc] >> sub) & 1u;
          {
            const float4 s4 = reinterpret_cast<const float4*>(sm + OFF_SC + sc * 1024)[sub * 32 + lane];
            __syncwarp();
            reinterpret_cast<float2*>(pl)[lane] = make_float2(s4.x, s4.z);
            reinterpret_cast<float2*>(pl + 64)[lane] = make_float2(s4.y, s4.w);
            reinterpret_cast<float2*>(pl + 128)[lane] = make_float2(lg2_approx(s4.x), lg2_approx(s4.z));
            __syncwarp();
          }
          // tokens of this half that the row sees
          const int n = here ? min(max(lim - ((w.t + i) * TILE + sub * SUB), 0), SUB) : 0;
          const bool cut = __any_sync(0xffffffffu, n < SUB);
          if (!wait(B_SFULL + grp, (uint32_t)(g >> 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint64_t u2[SUB / 2];
          float umax = -INFINITY, ymax = -INFINITY;
          const float4* sl4 = reinterpret_cast<const float4*>(pl);
          const float4* sr4 = reinterpret_cast<const float4*>(pl + 64);
          const float4* lg4 = reinterpret_cast<const float4*>(pl + 128);
          const uint32_t tl = tmem + lane_addr + T_SL + grp * TILE + sub * SUB;
          const uint32_t tr = tmem + lane_addr + T_SR + sub * SUB;
#pragma unroll
          for (int j = 0; j < SUB / 8; ++j) {
            uint32_t rl[8], rr[8];
            tmem_ld8(tl + 8 * j, rl);
            tmem_ld8(tr + 8 * j, rr);
            tmem_wait_ld();
            if (j == SUB / 8 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_cluster(sempty);
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {  // tokens 8 j + 4 v ..
              const float4 s4 = sl4[2 * j + v], r4 = sr4[2 * j + v], g4 = lg4[2 * j + v];
              uint64_t ua = fma2(pk2(r4.x, r4.y), pk2(__uint_as_float(rr[4 * v]), __uint_as_float(rr[4 * v + 1])),
                                 mul2(pk2(s4.x, s4.y), pk2(__uint_as_float(rl[4 * v]), __uint_as_float(rl[4 * v + 1]))));
              uint64_t ub = fma2(pk2(r4.z, r4.w), pk2(__uint_as_float(rr[4 * v + 2]), __uint_as_float(rr[4 * v + 3])),
                                 mul2(pk2(s4.z, s4.w), pk2(__uint_as_float(rl[4 * v + 2]), __uint_as_float(rl[4 * v + 3]))));
              if (cut) {
                const int t = 8 * j + 4 * v;
                const float2 fa = up2(ua), fb = up2(ub);
                ua = pk2(t < n ? fa.x : -INFINITY, t + 1 < n ? fa.y : -INFINITY);
                ub = pk2(t + 2 < n ? fb.x : -INFINITY, t + 3 < n ? fb.y : -INFINITY);
              }
              u2[4 * j + 2 * v] = ua;
              u2[4 * j + 2 * v + 1] = ub;
              const float2 fa = up2(ua), fb = up2(ub);
              umax = max3(umax, fa.x, fa.y);
              umax = max3(umax, fb.x, fb.y);
              // (where a token is out of sight u is -inf and y is -inf or NaN, which max drops)
              const float2 ya = up2(fma2(c2, ua, pk2(g4.x, g4.y))), yb = up2(fma2(c2, ub, pk2(g4.z, g4.w)));
              ymax = max3(ymax, ya.x, ya.y);
              ymax = max3(ymax, yb.x, yb.y);
            }
          }
          // M_g after the previous tile (waited for on every tile, also where a row tile
          // begins: the waits then see every phase)
          if (g > 0 && !wait(B_CH + ((g - 1) & 1) * 4 + q, (uint32_t)((g - 1) >> 1))) {
            ok = false;
            break;
          }
          const float mg = i > 0 ? mgs[((g - 1) & 1) * CROWS + hh] : -INFINITY;
          // the tile's largest weight over both halves
          float* xm = xmax + (((g >> 1) & 1) * 2 + grp) * 2 * CROWS + hh;
          xm[sub * CROWS] = ymax;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_EX + grp * 4 + q]);
          if (!wait(B_EX + grp * 4 + q, (uint32_t)(g >> 1))) {
            ok = false;
            break;
          }
          ymax = fmaxf(ymax, xm[(sub ^ 1) * CROWS]);
          mghi = fmaxf(mghi, mg);
          float mgn = mg;
          if (ymax > mg + TAU || (ymax < mg - DOWN && ymax >= mghi - DOWN_CAP && ymax > -INFINITY)) mgn = ymax;
          mghi = fmaxf(mghi, mgn);
          if (sub == 0) {
            mgs[(g & 1) * CROWS + hh] = mgn;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_CH + grp * 4 + q]);
          }
          // this thread's denominator, and the factor from p to g'
          const float mn = fmaxf(m, c * umax);
          l *= m == mn ? 1.f : ex2_approx(m - mn);
          m = mn;
          const float kf = (mn > -INFINITY && mgn > -INFINITY) ? P_TOP * ex2_approx(fminf(mn - mgn, K_CAP)) : 0.f;
          const float mneg = -fmaxf(mn, -3.0e38f);
          const uint64_t m2 = pk2(mneg, mneg), k2 = pk2(kf, kf);
          if (g >= 2 && !wait(B_PFREE + grp, (uint32_t)((g >> 1) - 1))) {
            ok = false;
            break;
          }
          const uint32_t dst = ctx_p + (q * 2 + sub) * CHUNK;
          uint64_t ls2 = pk2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < SUB / 8; ++j) {  // eight tokens, 16 bytes of g'
            uint32_t h[4];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const float4 s4 = sl4[2 * j + v];
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const float2 z = up2(fma2(c2, u2[4 * j + 2 * v + p], m2));
                const uint64_t e = pk2(ex2_approx(z.x), ex2_approx(z.y));
                ls2 = add2(ls2, e);
                float2 x = up2(mul2(mul2(e, k2), p == 0 ? pk2(s4.x, s4.y) : pk2(s4.z, s4.w)));
                if (cut) {
                  const int t = 8 * j + 4 * v + 2 * p;
                  x.x = t < n ? x.x : 0.f;
                  x.y = t + 1 < n ? x.y : 0.f;
                }
                const __half2 h2 = __floats2half2_rn(x.x, x.y);
                h[2 * v + p] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            }
            st_async_v4(dst + prow(lane, j), make_uint4(h[0], h[1], h[2], h[3]), ctx_pfull);
          }
          if (sub == 0) {
            // what the row's O is multiplied by before this tile is added
            const float f = mgn == mg ? 1.f : (mg > -INFINITY ? ex2_approx(mg - mgn) : 0.f);
            st_async_b32(ctx_p + P_F + hh * 4, __float_as_uint(f), ctx_pfull);
          }
          const float2 ls = up2(ls2);
          l += ls.x + ls.y;
        }
        if (!ok) break;
        // ---- the row tile's (or its part's) end: every MMA on this query is done; the
        // four threads of a row join their (m, l)
        const int last = gt + w.n - 1;
        gt += w.n;
        xl[part * CROWS + hh] = make_float2(m, l);
        if (!wait(B_SFULL + (last & 1), (uint32_t)(last >> 1)) || !quarter_sync()) {
          ok = false;
          break;
        }
        if (part == 0) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int p = 0; p < 4; ++p) M = fmaxf(M, xl[p * CROWS + hh].x);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float2 v = xl[p * CROWS + hh];
            L += v.y * (v.x > -INFINITY ? ex2_approx(v.x - M) : 1.f);  // (a NaN l stays one)
          }
          const float mg = mgs[(last & 1) * CROWS + hh];
          float f = mg > -INFINITY ? ex2_approx(mg - M) * (1.f / P_TOP) : 0.f;
          if (L != L) f = L;
          if (w.whole()) {
            f = L > 0.f ? f / L : f;
            if (a.lse != nullptr && real)
              a.lse[(w.s.q0 + tok) * a.H + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
          } else {
            const int64_t at = (int64_t)(2 * k + (w.seg == 0 ? 0 : 1)) * ROWS + rank * CROWS + hh;
            ws.m[at] = M;
            ws.l[at] = L;
          }
          st_async_b32(ctx_rf + (w.seg % NRF) * 512 + hh * 4, __float_as_uint(f), ctx_rfbar + (w.seg % NRF) * 8);
        }
      }
      if (!ok && lane == 0) fail();
      // the context CTAs' last commits to this CTA have landed
      if (ok && gt > 0) {
        const int zero = 0;
        for (int i = gt > 2 ? gt - 2 : 0; i < gt; ++i)
          if ((i & 1) == grp) (void)mbar_wait(&bars[B_PFREE + grp], (i >> 1) & 1, &zero, WAIT_NS);
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
          facts[vs] = (s0 >= 0 ? 1u : 0u) | (s1 >= 0 ? 2u : 0u);
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
    } else if (warp == W_MMA) {
      if (rank == 2) {
        const uint32_t id = idesc_f16(ROWS, 256, false, true);  // A K-major, B = V MN-major
        const uint64_t pd = smem_desc(pbuf, 16, 1024, SW128);
        const uint64_t vd = smem_desc(vring, 16, 1024, SW128);
        bool ok = true;
        for (; ok && w.more(); w.next(a)) {
          for (int i = 0; ok && i < w.n; ++i) {
            const int g = gt + i;
            const uint64_t ad = pd + (uint64_t)((g & 1) * P_STRIDE >> 4);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!wait_cluster(B_RS + h, (uint32_t)g)) {
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
              mma_commit_pair_warp(&bars[B_ODONE + h], 0xC);
            }
            if (!ok) break;
            mma_commit_pair_warp(&bars[B_VEMPTY + g % NVT], 0xC);
            mma_commit_pair_warp(&bars[B_PFREE + (g & 1)], 0x3);
          }
          gt += w.n;
        }
        if (!ok && lane == 0) fail();
        mma_commit_pair_warp(&bars[B_DRAIN], 0xC);
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
        for (int i = 0; i < w.n; ++i) {
          const int g = gt + i, pb = g & 1, vs = g % NVT;
          if (!wait_cluster(B_PFULL + pb, (uint32_t)(g >> 1))) {
            ok = false;
            break;
          }
          const uint32_t src = pbuf + pb * P_STRIDE + (q * 2 + (part >> 1)) * CHUNK;
          uint4 pv[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) pv[u] = lds128(src + prow(lane, 4 * (part & 1) + u));
          const float f = reinterpret_cast<const float*>(sm + OFF_P + pb * P_STRIDE + P_F)[hh];
          const bool any = __any_sync(0xffffffffu, f != 1.f) && i > 0;
          // every warp has read this payload: its buffer may now take the operand, and the
          // next payload (whose bytes come after this tile's MMAs) may be expected
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_CVT]);
          if (!wait(B_CVT, (uint32_t)(g + w.seg))) {
            ok = false;
            break;
          }
          if (warp == W_LANE && lane == 0) mbar_arrive_expect_tx(&bars[B_PFULL + pb], P_BYTES);
          const uint32_t opnd = pbuf + pb * P_STRIDE;
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 16 tokens per 16-byte unit
            const uint32_t x[8] = {pv[2 * j].x, pv[2 * j].y, pv[2 * j].z, pv[2 * j].w,
                                   pv[2 * j + 1].x, pv[2 * j + 1].y, pv[2 * j + 1].z, pv[2 * j + 1].w};
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint16_t h0, l0, h1, l1;
              split_h2(x[2 * v], h0, l0);
              split_h2(x[2 * v + 1], h1, l1);
              hw[v] = (uint32_t)h0 | ((uint32_t)h1 << 16);
              lw[v] = (uint32_t)l0 | ((uint32_t)l1 << 16);
            }
            const uint32_t off = sw128(hh, part * 2 + j);
            sts128(opnd + off, make_uint4(hw[0], hw[1], hw[2], hw[3]));
            sts128(opnd + OP_ATOM + off, make_uint4(lw[0], lw[1], lw[2], lw[3]));
          }
          if (!wait(B_VT + vs, (uint32_t)(g / NVT))) {
            ok = false;
            break;
          }
          if ((w.t + i + 1) * TILE > lim0 || facts[vs] != 3u) {
            // some row does not see all of this tile: no NaN code may stay in it
            const uint32_t vb = vring + vs * VTILE + (warp - W_LANE) * 2048 + lane * 16;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 v = lds128(vb + u * 512);
              sts128(vb + u * 512, make_uint4(no_nan(v.x), no_nan(v.y), no_nan(v.z), no_nan(v.w)));
            }
          }
          fence_proxy_async_smem();
          // each O half: the previous tile's MMAs on it are done (at a row tile's start the
          // results were read after them), then the rows whose reference moved are rescaled
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (i > 0 && !wait(B_ODONE + h, (uint32_t)(g - 1))) {
              ok = false;
              break;
            }
            if (any) {
              tc_fence_after();
              __syncwarp();
              const uint32_t col = tmem + lane_addr + h * 256 + part * 64;
#pragma unroll 1
              for (int c0 = 0; c0 < 64; c0 += 16) {
                uint32_t r[16];
                tmem_ld16(col + c0, r);
                tmem_wait_ld();
#pragma unroll
                for (int v = 0; v < 16; ++v) r[v] = __float_as_uint(__uint_as_float(r[v]) * f);
                tmem_st16(col + c0, r);
              }
              __syncwarp();
              tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(rs + h * 8);
          }
          if (!ok) break;
        }
        if (!ok) break;
        const int last = gt + w.n - 1;
        gt += w.n;
        const int rf = w.seg % NRF;
        if (!wait(B_ODONE, (uint32_t)last) || !wait(B_ODONE + 1, (uint32_t)last) ||
            !wait_cluster(B_RF + rf, (uint32_t)(w.seg / NRF))) {
          ok = false;
          break;
        }
        tc_fence_after();
        __syncwarp();
        const float f = reinterpret_cast<const float*>(sm + OFF_RF + rf * 512)[hh];
        const int64_t r = (int64_t)w.rt * ROWS + half_of * CROWS + hh;
        const bool real = r < (int64_t)w.s.nq * a.H;
        const bool whole = w.whole();
        uint16_t* out = a.out + (w.s.q0 * a.H + r) * DL;
        float* po = ws.o + ((int64_t)(2 * k + (w.seg == 0 ? 0 : 1)) * ROWS + half_of * CROWS + hh) * DL;
#pragma unroll 1
        for (int s = 0; s < 4; ++s) {  // 32 columns at a time
          const int col = (s >> 1) * 256 + part * 64 + (s & 1) * 32;
          uint32_t v[32];
          tmem_ld32(tmem + lane_addr + col, v);
          tmem_wait_ld();
          if (f == 0.f) {  // nothing seen, or nothing that counts
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[j + 2 * e]) * f,
                                                                __uint_as_float(v[j + 2 * e + 1]) * f);
                o[e] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              if (real) *reinterpret_cast<uint4*>(out + col + j) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else if (real) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(po + col + j) =
                  make_float4(__uint_as_float(v[j]) * f, __uint_as_float(v[j + 1]) * f,
                              __uint_as_float(v[j + 2]) * f, __uint_as_float(v[j + 3]) * f);
          }
        }
        // the factor buffer's next use, NRF segments on: its bytes come after this row
        // tile's successor has been accumulated
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_CVT]);
        if (!wait(B_CVT, (uint32_t)(gt + w.seg))) {
          ok = false;
          break;
        }
        if (warp == W_LANE && lane == 0) mbar_arrive_expect_tx(&bars[B_RF + rf], CROWS * 4);
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

// Joins the parts of the row tiles that range borders cut: block (x, k - 1) takes
// eight rows, a warp each, of the row tile that cluster k starts in, if cluster k - 1
// holds its beginning.
__global__ void __launch_bounds__(256) join_kernel(const ChunkArgs a, const Workspace ws) {
  const int k = (int)blockIdx.y + 1, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t nc = ws.plan->n_clusters;
  if (k >= nc) return;
  const PlanEntry e = ws.plan->e[k];
  const int64_t S = e.x - e.off;              // the row tile's first unit
  const int64_t xp = ws.plan->e[k - 1].x;
  if (e.off == 0 || xp > S) return;           // whole, or begun before cluster k - 1
  const SeqInfo s = seq_info(a, e.b, false);
  const int64_t r = (int64_t)e.rt * ROWS + row;
  if (r >= (int64_t)s.nq * a.H) return;
  auto part = [&](int j) -> int64_t {         // slot of cluster j's part
    return (int64_t)(2 * j + (j == k - 1 && xp < S ? 1 : 0)) * ROWS + row;
  };
  int last = k;
  while (last + 1 < nc && ws.plan->e[last + 1].x < S + e.nt) ++last;
  float M = -INFINITY;
  for (int j = k - 1 + lane; j <= last; j += 32) M = fmaxf(M, ws.m[part(j)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f;
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int j = k - 1; j <= last; ++j) {
    const int64_t p = part(j);
    const float m = ws.m[p], l = ws.l[p];
    const float4* o = reinterpret_cast<const float4*>(ws.o + p * DL) + lane;
    const float wt = m > -INFINITY ? ex2_approx(m - M) : 1.f;  // (a NaN l stays one)
    L += wt * l;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 v = o[32 * c];
      acc[c].x += wt * v.x;
      acc[c].y += wt * v.y;
      acc[c].z += wt * v.z;
      acc[c].w += wt * v.w;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = s.q0 * a.H + r;
  uint2* out = reinterpret_cast<uint2*>(a.out + at * DL) + lane;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    out[32 * c] = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (a.lse != nullptr && lane == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
}

constexpr int64_t OFF_PLAN = 256, OFF_BASE = 2048;
static_assert(OFF_PLAN + sizeof(Plan) <= OFF_BASE, "plan area");

// Clusters that a call of these sizes can use, whatever the lengths turn out to be.
int most_clusters(int B, int H, int64_t total_q, int max_blocks) {
  const int64_t row_tiles = total_q * H / ROWS + B, keys = ((int64_t)max_blocks * PAGE + TILE - 1) / TILE;
  const int64_t units = row_tiles * keys / MIN_TILES;
  return (int)(units < 1 ? 1 : (units < MAX_CLUSTERS ? units : MAX_CLUSTERS));
}

int64_t base_bytes(int B) { return ((int64_t)(B + 1) * 8 + 255) / 256 * 256; }

}  // namespace

int64_t chunk_workspace(int B, int H, int64_t total_q, int max_blocks) {
  const int64_t rows = 2ll * most_clusters(B, H, total_q, max_blocks) * ROWS;
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
  join_kernel<<<dim3(ROWS / 8, clusters - 1), 256, 0, s>>>(a, ws);
  return cudaGetLastError();
}

}  // namespace kv8
