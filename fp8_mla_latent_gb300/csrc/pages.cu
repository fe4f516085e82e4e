// pages.cu -- the pages of a paged fp8 latent cache: sequences that grow
// (append), share a prefix (fork), leave (free), a pool that is packed (compact),
// and the page data those steps ask to be moved (copy).  The page tables and the
// reference counts live in device memory and every step runs on the device, so a
// serving loop needs no host round trip between a step and the attention after it.
//
// State (caller's): block_table int32 [B][max_blocks], seq_lens int32 [B] and
// page_refs int32 [n_blocks], the number of held table entries that name a page
// (0 = free).  A sequence holds its first ceil(seq_len / 64) entries.  Free pages
// are taken lowest index first, in the order of the sequences, so every result is
// the same on every run.
//
// The table steps are one launch each of one thread-block cluster, at most
// PG_CTAS CTAs of 1024 threads: a step is a validation that must be complete
// before anything is written (lists, lengths and room: all or nothing; a held entry
// that names no page is met in the walk, and reported), a ranking of the free pages,
// and a walk over table entries; the cluster barrier separates them without a second
// launch, and what they read (a few hundred KB at most) bounds nothing: they are
// launch latency (3 us) and dependent L2 round trips (about 1 us each), so the work
// on them is to have fewer in a row.  A CTA count of one is kept while the entries to
// walk fit one pass of one CTA.  Measured (device time under a profiler): for 2 forks
// of short sequences free 4, fork 9, append 6 us; for 192 forks of up to 4096 tokens
// among 256 sequences free 7, fork 11, append 14 us; compact 10 us for 100 pages, 13 us
// for 6200 in 256 sequences.  (Sequences of thousands of pages were not measured.)
//
// The copy is the only step that moves real data: 2 x 37376 bytes per page and
// layer, an HBM stream.  Bulk copies through a shared-memory ring, issued by one
// thread per CTA, keep about 11 MB of loads in flight over 152 SMs.
#include "kv8_common.cuh"
#include "tc_ptx.cuh"

namespace kv8 {
namespace {

using namespace ptx;

constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_CTAS = 8;        // largest portable cluster
constexpr int PG_ROUNDS = 16;     // pages per lane and pass: 16384 of one CTA
constexpr int ONE_PASS = 8 * PG_THREADS;  // entries one CTA walks before a cluster pays

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// The cluster barrier, from warps made to converge first; it also orders the
// CTAs' global and shared memory accesses.
__device__ __forceinline__ void all_ctas_sync() {
  __syncthreads();
  cluster_sync();
}

__device__ __forceinline__ void flag(unsigned* err, unsigned bit) {
  if (err != nullptr) atomicOr(err, bit);
}

__device__ __forceinline__ int pages_of(int64_t tokens) { return (int)((tokens + PAGE - 1) / PAGE); }

// Inclusive sum over the CTA (every thread); *total gets the CTA's sum.  `tmp`
// holds PG_WARPS + 1 values and may be used again right after.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* tmp, int64_t* total) {
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
  *total = tmp[PG_WARPS - 1];
  __syncthreads();
  return v;
}

// The same of two values; `tmp` holds 2 PG_WARPS.
__device__ __forceinline__ void cta_scan2(int64_t (&v)[2], int64_t* tmp, int64_t (&total)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v[k], o);
      if (lane >= o) v[k] += u;
    }
  if (lane == 31) {
    tmp[warp] = v[0];
    tmp[PG_WARPS + warp] = v[1];
  }
  __syncthreads();
  if (warp < 2) {
    int64_t w = tmp[warp * PG_WARPS + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    tmp[warp * PG_WARPS + lane] = w;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (warp > 0) v[k] += tmp[k * PG_WARPS + warp - 1];
    total[k] = tmp[k * PG_WARPS + PG_WARPS - 1];
  }
  __syncthreads();
}

// One pass over pages [lo, lo + PG_THREADS * PG_ROUNDS) cut at `hi`: lane masks of
// the pages for which `is(refs[p], p)` holds, in index order.  Warp w takes 32 *
// PG_ROUNDS consecutive pages, 32 at a time; every load of the pass is in flight
// at once.  Returns the rank of the warp's first match (over the CTA), the CTA's
// matches in *total and the warp's masks in m.
template <typename F>
__device__ __forceinline__ int64_t rank_pages(const int32_t* refs, int64_t lo, int64_t hi, F is,
                                              uint32_t (&m)[PG_ROUNDS], int64_t* tmp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t p0 = lo + (int64_t)warp * 32 * PG_ROUNDS + lane;
  int32_t r[PG_ROUNDS];
#pragma unroll
  for (int j = 0; j < PG_ROUNDS; ++j) r[j] = p0 + 32 * j < hi ? refs[p0 + 32 * j] : 0;
  int n = 0;
#pragma unroll
  for (int j = 0; j < PG_ROUNDS; ++j) {
    const int64_t p = p0 + 32 * j;
    m[j] = __ballot_sync(0xffffffffu, p < hi && is(r[j], p));
    n += __popc(m[j]);
  }
  const int64_t inc = cta_scan(lane == 0 ? n : 0, tmp, total);
  return __shfl_sync(0xffffffffu, inc, 0) - n;
}

// The pages of a pass in rank order: f(rank, page), on the lane that holds it.
template <typename F>
__device__ __forceinline__ void each_ranked(int64_t rank, int64_t lo, const uint32_t (&m)[PG_ROUNDS], F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < PG_ROUNDS; ++j) {
    if ((m[j] >> lane) & 1u)
      f(rank + __popc(m[j] & below), lo + (int64_t)warp * 32 * PG_ROUNDS + 32 * j + lane);
    rank += __popc(m[j]);
  }
}

constexpr int64_t PASS_PAGES = (int64_t)PG_THREADS * PG_ROUNDS;

// The first `need` free pages: f(rank, page); false, and f not called, if the pool has fewer
// (CTA-wide).  The first pass, mostly the only one, is ranked once for both.
template <typename F>
__device__ __forceinline__ bool take_free(const int32_t* refs, int64_t n_blocks, int64_t need, int64_t* tmp, F f) {
  if (need == 0) return true;
  auto is = [](int32_t r, int64_t) { return r == 0; };
  auto give = [&](int64_t k, int64_t p) {
    if (k < need) f(k, p);
  };
  uint32_t m[PG_ROUNDS];
  int64_t got;
  const int64_t rank = rank_pages(refs, 0, n_blocks, is, m, tmp, &got);
  if (got >= need) {
    each_ranked(rank, 0, m, give);
    return true;
  }
#pragma unroll 1
  for (int64_t lo = PASS_PAGES; lo < n_blocks && got < need; lo += PASS_PAGES) {
    int64_t total;
    (void)rank_pages(refs, lo, n_blocks, is, m, tmp, &total);
    got += total;
  }
  if (got < need) return false;
  got = 0;
#pragma unroll 1
  for (int64_t lo = 0; lo < n_blocks && got < need; lo += PASS_PAGES) {
    int64_t total;
    const int64_t r = rank_pages(refs, lo, n_blocks, is, m, tmp, &total);
    each_ranked(got + r, lo, m, give);
    got += total;
  }
  return true;
}

// The last index i of the ascending a[0..n] with a[i] <= x (a[0] <= x < a[n]).
template <typename T>
__device__ __forceinline__ int last_le(const T* a, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ append
// need_b = ceil((len + new) / 64) - ceil(len / 64) pages for sequence b.  CTA 0
// validates, ranks and writes table, counts, lengths and q_start; then every CTA
// writes a share of dst_slot (token i of sequence b at position len + i).
__global__ void __launch_bounds__(PG_THREADS)
append_kernel(PageTable t, const int32_t* __restrict__ n_new, int32_t* q_start, int64_t* dst_slot,
              int64_t cap, unsigned* err) {
  extern __shared__ int32_t first[];  // CTA 0: [B + 1] pages taken before sequence b, [B] pages it had; then everywhere: q_start
  __shared__ int64_t tmp[2 * PG_WARPS];
  __shared__ unsigned bad;
  const int B = t.B;
  int32_t* had = first + B + 1;
  if (cluster_rank() == 0) {
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    int64_t tokens = 0, pages = 0;
    for (int b0 = 0; b0 < B; b0 += PG_THREADS) {
      const int b = b0 + threadIdx.x;
      int64_t fresh = 0, need = 0;
      if (b < B) {
        const int64_t len = t.seq_lens[b], nn = n_new[b];
        if (len < 0 || nn < 0 || len > (int64_t)t.max_blocks * PAGE) {
          atomicOr(&bad, KV8_PAGES_EINDEX);
        } else if (nn > 0) {
          fresh = nn;
          if (len + nn > (int64_t)t.max_blocks * PAGE) {
            atomicOr(&bad, KV8_PAGES_ENOROOM);
          } else {
            need = pages_of(len + nn) - pages_of(len);
            had[b] = pages_of(len);
            if (len % PAGE != 0) {  // the tokens begin in a page that is this sequence's alone
              const int32_t p = t.block_table[(int64_t)b * t.max_blocks + pages_of(len) - 1];
              if (p < 0 || p >= t.n_blocks || t.page_refs[p] != 1) atomicOr(&bad, KV8_PAGES_EINDEX);
            }
          }
        }
      }
      int64_t inc[2] = {fresh, need}, sum[2];
      cta_scan2(inc, tmp, sum);
      if (b < B) {
        const int64_t at = tokens + inc[0] - fresh, pg = pages + inc[1] - need;
        q_start[b] = (int32_t)(at < INT32_MAX ? at : INT32_MAX);
        first[b] = (int32_t)(pg < INT32_MAX ? pg : INT32_MAX);
      }
      tokens += sum[0];
      pages += sum[1];
    }
    if (threadIdx.x == 0) {
      if (tokens > cap || pages > t.n_blocks) bad |= KV8_PAGES_ENOROOM;
      q_start[B] = (int32_t)(tokens < INT32_MAX ? tokens : INT32_MAX);
      first[B] = (int32_t)(pages < INT32_MAX ? pages : INT32_MAX);
    }
    __syncthreads();
    if (bad == 0 && !take_free(t.page_refs, t.n_blocks, pages, tmp, [&](int64_t k, int64_t p) {
          const int b = last_le(first, B, k);
          t.block_table[(int64_t)b * t.max_blocks + had[b] + (k - first[b])] = (int32_t)p;
          t.page_refs[p] = 1;
        }))
      if (threadIdx.x == 0) bad = KV8_PAGES_ENOROOM;
    __syncthreads();
    if (bad != 0) {
      // nothing is taken, and the call hands out no token
      if (threadIdx.x == 0) flag(err, bad);
      for (int b = threadIdx.x; b <= B; b += PG_THREADS) q_start[b] = 0;
    } else {
      for (int b = threadIdx.x; b < B; b += PG_THREADS) t.seq_lens[b] += n_new[b];
    }
  }
  all_ctas_sync();
  for (int b = threadIdx.x; b <= B; b += PG_THREADS) first[b] = q_start[b];
  __syncthreads();
  const int64_t total = first[B];
  const int64_t stride = (int64_t)cluster_ctas() * PG_THREADS;
  for (int64_t i = (int64_t)cluster_rank() * PG_THREADS + threadIdx.x; i < cap; i += stride) {
    int64_t slot = -1;
    if (i < total) {
      const int b = last_le(first, B, i);
      const int64_t pos = (int64_t)t.seq_lens[b] - n_new[b] + (i - first[b]);
      slot = (int64_t)t.block_table[(int64_t)b * t.max_blocks + pos / PAGE] * PAGE + pos % PAGE;
    }
    dst_slot[i] = slot;
  }
}

// ------------------------------------------------------------------ fork
// dst row := the first entries of src row; whole pages are shared, a last page
// that is only part full is copied to a fresh page (one move), so that a page in
// which tokens are still written belongs to one sequence.  CTA 0 validates and
// takes the fresh pages; then a warp per fork walks its entries, over all CTAs.
__global__ void __launch_bounds__(PG_THREADS)
fork_kernel(PageTable t, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            const int32_t* __restrict__ fork_len, int n, int32_t* moves, int32_t* n_moves, unsigned* err) {
  extern __shared__ unsigned role[];  // CTA 0: [B] 1 = a destination, 2 = a source; then [n + 1] fresh pages before fork i, [n] those pages
  __shared__ int64_t tmp[PG_WARPS + 1];
  __shared__ unsigned bad;
  __shared__ unsigned go;
  const int B = t.B;
  const int lane = threadIdx.x & 31;
  int32_t* first = reinterpret_cast<int32_t*>(role + B);
  if (cluster_rank() == 0) {
    if (threadIdx.x == 0) bad = 0;
    for (int b = threadIdx.x; b < B; b += PG_THREADS) role[b] = 0;
    __syncthreads();
    int64_t pages = 0;
    for (int i0 = 0; i0 < n; i0 += PG_THREADS) {
      const int i = i0 + threadIdx.x;
      int64_t need = 0;
      if (i < n) {
        const int32_t a = src[i], d = dst[i];
        if (a < 0 || a >= B || d < 0 || d >= B || a == d) {
          atomicOr(&bad, KV8_PAGES_EINDEX);
        } else {
          const int64_t len = t.seq_lens[a], take = fork_len != nullptr ? fork_len[i] : len;
          if (len < 0 || len > (int64_t)t.max_blocks * PAGE || take < 0 || take > len || t.seq_lens[d] != 0 ||
              (atomicOr(&role[d], 1u) & 1u) != 0u)
            atomicOr(&bad, KV8_PAGES_EINDEX);
          atomicOr(&role[a], 2u);
          need = take % PAGE != 0;
        }
      }
      int64_t sum;
      const int64_t inc = cta_scan(need, tmp, &sum);
      if (i < n) first[i] = (int32_t)(pages + inc - need);
      pages += sum;
    }
    if (threadIdx.x == 0) first[n] = (int32_t)pages;
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += PG_THREADS)
      if (role[b] == 3u) atomicOr(&bad, KV8_PAGES_EINDEX);
    __syncthreads();
    int32_t* fresh = first + n + 1;
    if (bad == 0 && !take_free(t.page_refs, t.n_blocks, pages, tmp, [&](int64_t k, int64_t p) { fresh[k] = (int32_t)p; }))
      if (threadIdx.x == 0) bad = KV8_PAGES_ENOROOM;
    __syncthreads();
    if (bad == 0) {
      // (a thread per fork: the few lanes that hold the free pages would walk them one by one)
      for (int i = threadIdx.x; i < n; i += PG_THREADS) {
        const int k = first[i];
        if (first[i + 1] == k) continue;
        const int32_t a = src[i], p = fresh[k];
        const int64_t take = fork_len != nullptr ? fork_len[i] : t.seq_lens[a];
        const int64_t col = pages_of(take) - 1;
        moves[2 * k] = t.block_table[(int64_t)a * t.max_blocks + col];
        moves[2 * k + 1] = p;
        t.block_table[(int64_t)dst[i] * t.max_blocks + col] = p;
        t.page_refs[p] = 1;
      }
    }
    if (threadIdx.x == 0) {
      n_moves[0] = bad != 0 ? 0 : (int32_t)pages;
      if (bad != 0) flag(err, bad);
      go = bad == 0;
    }
  }
  all_ctas_sync();  // CTA 0's writes, and `go` there
  uint32_t ok;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(ok) : "r"(map_to(smem_u32(&go), 0)) : "memory");
  if (ok != 0u) {
    const int warps = (int)cluster_ctas() * PG_WARPS;
    for (int i = (int)cluster_rank() * PG_WARPS + (threadIdx.x >> 5); i < n; i += warps) {
      const int64_t take = fork_len != nullptr ? fork_len[i] : t.seq_lens[src[i]];
      const int32_t* from = t.block_table + (int64_t)src[i] * t.max_blocks;
      int32_t* to = t.block_table + (int64_t)dst[i] * t.max_blocks;
      for (int64_t c = lane; c < take / PAGE; c += 32) {
        const int32_t p = from[c];
        to[c] = p;
        if (p >= 0 && p < t.n_blocks) atomicAdd(&t.page_refs[p], 1); else flag(err, KV8_PAGES_EINDEX);
      }
      if (lane == 0) {
        t.seq_lens[dst[i]] = (int32_t)take;
        if (take % PAGE != 0) {
          const int32_t p = from[take / PAGE];
          if (p < 0 || p >= t.n_blocks) flag(err, KV8_PAGES_EINDEX);
        }
      }
    }
  }
  all_ctas_sync();  // CTA 0's shared memory is read above
}

// ------------------------------------------------------------------ free
// Every CTA validates the list and its sequences' lengths by itself; then a warp per
// sequence gives its pages back, over all CTAs.  (A CTA that is behind may read the 0 that
// another one has put in a length's place: that one has found every length good.)
__global__ void __launch_bounds__(PG_THREADS)
free_kernel(PageTable t, const int32_t* __restrict__ seq, int n, unsigned* err) {
  extern __shared__ unsigned role[];  // [B]
  __shared__ unsigned bad;
  const int B = t.B, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) bad = 0;
  for (int b = threadIdx.x; b < B; b += PG_THREADS) role[b] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += PG_THREADS) {
    const int32_t b = seq[i];
    if (b < 0 || b >= B || atomicOr(&role[b], 1u) != 0u) {
      atomicOr(&bad, KV8_PAGES_EINDEX);
    } else {
      const int64_t len = t.seq_lens[b];
      if (len < 0 || len > (int64_t)t.max_blocks * PAGE) atomicOr(&bad, KV8_PAGES_EINDEX);
    }
  }
  __syncthreads();
  if (bad != 0) {
    if (cluster_rank() == 0 && threadIdx.x == 0) flag(err, bad);
    return;
  }
  const int warps = (int)cluster_ctas() * PG_WARPS;
  for (int i = (int)cluster_rank() * PG_WARPS + (threadIdx.x >> 5); i < n; i += warps) {
    const int b = seq[i];
    const int64_t len = t.seq_lens[b];
    int32_t* row = t.block_table + (int64_t)b * t.max_blocks;
    for (int c = lane; c < pages_of(len); c += 32) {
      const int32_t p = row[c];
      row[c] = -1;
      if (p < 0 || p >= t.n_blocks) {
        flag(err, KV8_PAGES_EINDEX);
      } else if (atomicSub(&t.page_refs[p], 1) <= 0) {
        atomicAdd(&t.page_refs[p], 1);  // held by no count: left at what it was
        flag(err, KV8_PAGES_EINDEX);
      }
    }
    __syncwarp();
    if (lane == 0) t.seq_lens[b] = 0;
  }
}

// ------------------------------------------------------------------ compact
// With L live pages, the k-th live page at or above L moves to the k-th free page
// below L: as few moves as can be, no page both source and destination.  Each CTA
// holds its share of the pool as a bitmap of live pages in shared memory, and beside
// it how many pages of the whole pool move before each word's: a table entry finds
// its move by counting bits there (in another CTA's shared memory, mostly), in place
// of a search with a round trip to L2 at each of its steps.
constexpr int64_t MAX_SHARE = KV8_PAGES_MAX_BLOCKS / PG_CTAS;
static_assert(MAX_SHARE >= ONE_PASS && MAX_SHARE % 32 == 0, "the bitmap holds any share");

__global__ void __launch_bounds__(PG_THREADS)
compact_kernel(PageTable t, int32_t* moves, int32_t* n_moves, int32_t* n_live, unsigned* err) {
  __shared__ uint32_t live[MAX_SHARE / 32];
  __shared__ int32_t before[MAX_SHARE / 32];
  __shared__ int64_t tmp[2 * PG_WARPS];
  __shared__ int64_t count[3];  // this CTA's live pages, holes below L, movers from L on
  const int nc = (int)cluster_ctas(), rank = (int)cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t share = ((t.n_blocks + nc - 1) / nc + 31) / 32 * 32;
  const int64_t lo = rank * share < t.n_blocks ? rank * share : t.n_blocks;
  const int64_t hi = lo + share < t.n_blocks ? lo + share : t.n_blocks;
  const int words = (int)((hi - lo + 31) / 32);
  auto count_of = [&](int k, int r) -> int64_t {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to(smem_u32(&count[k]), r)) : "memory");
    return (int64_t)v;
  };
  int64_t n = 0;
#pragma unroll 4
  for (int w = warp; w < words; w += PG_WARPS) {
    const int64_t p = lo + 32 * w + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, p < hi && t.page_refs[p] > 0);
    if (lane == 0) {
      live[w] = m;
      n += __popc(m);
    }
  }
  // a length that cannot be (which entries the sequence holds is not known then) makes the call do
  // nothing: a CTA that meets one says so above its count of live pages
  constexpr int64_t BAD = int64_t(1) << 40;
  for (int b = rank * PG_THREADS + threadIdx.x; b < t.B; b += nc * PG_THREADS) {
    const int64_t len = t.seq_lens[b];
    if (len < 0 || len > (int64_t)t.max_blocks * PAGE) n += BAD;
  }
  int64_t sum;
  (void)cta_scan(n, tmp, &sum);
  if (threadIdx.x == 0) count[0] = sum;
  all_ctas_sync();
  int64_t L = 0;
  for (int r = 0; r < nc; ++r) L += count_of(0, r);
  if (L >= BAD) {
    if (rank == 0 && threadIdx.x == 0) {
      flag(err, KV8_PAGES_EINDEX);
      n_moves[0] = 0;
      if (n_live != nullptr) n_live[0] = (int32_t)t.n_blocks;
    }
    all_ctas_sync();  // this CTA's count is read no more
    return;
  }
  // of word w: the pages below L without an owner, and those from L on that have one
  auto low = [&](int w) -> uint32_t {
    const int64_t d = L - lo - 32 * (int64_t)w;
    return d <= 0 ? 0u : d >= 32 ? 0xffffffffu : (1u << d) - 1u;
  };
  auto holes = [&](int w) -> uint32_t { return ~live[w] & low(w); };  // (L is no more than the pool's pages)
  auto movers = [&](int w) -> uint32_t { return live[w] & ~low(w); };
  const int each = (words + PG_THREADS - 1) / PG_THREADS;  // consecutive words of a thread
  const int w0 = min((int)threadIdx.x * each, words), w1 = min(w0 + each, words);
  int64_t at[2] = {0, 0}, all_of[2], own[2];
  for (int w = w0; w < w1; ++w) {
    at[0] += __popc(holes(w));
    at[1] += __popc(movers(w));
  }
  own[0] = at[0];
  own[1] = at[1];
  cta_scan2(at, tmp, all_of);
  if (threadIdx.x == 0) {
    count[1] = all_of[0];
    count[2] = all_of[1];
  }
  all_ctas_sync();
  int64_t h = at[0] - own[0], v = at[1] - own[1], N = 0;
  for (int r = 0; r < nc; ++r) {
    const int64_t c1 = count_of(1, r), c2 = count_of(2, r);
    if (r < rank) {
      h += c1;
      v += c2;
    }
    N += c2;
  }
  for (int w = w0; w < w1; ++w) {
    before[w] = (int32_t)v;
    for (uint32_t m = holes(w); m != 0; m &= m - 1) moves[2 * h++ + 1] = (int32_t)(lo + 32 * w + __ffs(m) - 1);
    for (uint32_t m = movers(w); m != 0; m &= m - 1) moves[2 * v++] = (int32_t)(lo + 32 * w + __ffs(m) - 1);
  }
  if (rank == 0 && threadIdx.x == 0) {
    n_moves[0] = (int32_t)N;
    if (n_live != nullptr) n_live[0] = (int32_t)L;
  }
  all_ctas_sync();  // the moves, and every word's count
  const int64_t me = (int64_t)rank * PG_THREADS + threadIdx.x, all = (int64_t)nc * PG_THREADS;
  for (int64_t k = me; k < N; k += all) {
    const int32_t s = moves[2 * k], d = moves[2 * k + 1];
    t.page_refs[d] = t.page_refs[s];
    t.page_refs[s] = 0;
  }
  const int64_t entries = (int64_t)t.B * t.max_blocks;
  for (int64_t e = me; e < entries; e += all) {
    const int b = (int)(e / t.max_blocks);
    const int32_t p = t.block_table[e];
    if (e - (int64_t)b * t.max_blocks >= pages_of(t.seq_lens[b])) continue;
    if (p < 0 || p >= t.n_blocks) {
      flag(err, KV8_PAGES_EINDEX);
      continue;
    }
    const int r = (int)(p / share), w = (int)(p - r * share) >> 5;
    uint32_t m;
    int32_t k;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(m) : "r"(map_to(smem_u32(&live[w]), r)) : "memory");
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(k) : "r"(map_to(smem_u32(&before[w]), r)) : "memory");
    const uint32_t bit = 1u << (p & 31);
    if ((m & bit) == 0u) {
      flag(err, KV8_PAGES_EINDEX);
    } else if (p >= L) {
      const int64_t d = L - (p & ~31);  // (below L in this word: they stay)
      if (d > 0) m &= ~((1u << d) - 1u);
      t.block_table[e] = moves[2 * (k + __popc(m & (bit - 1u))) + 1];
    }
  }
  all_ctas_sync();  // this CTA's shared memory is read no more
}

// ------------------------------------------------------------------ copy
// Tasks of a quarter of a page's codes (9216 bytes; the first quarter also takes
// the page's 512 bytes of scales), pair after pair, layer after layer; each CTA
// takes a contiguous range of them.  One thread runs the ring: loads eight tasks
// ahead, a store as soon as its load has landed.  The other warps meanwhile
// mark every destination in a bitmap in shared memory, so that a pair whose source
// another pair overwrites, or whose destination is named twice, is left out
// whatever the order in which CTAs run (the loads are harmless; stores wait for it).
//
// 3500 pages of 4 layers (1.05 GB read and written): 162 us, 6.45 TB/s, 95 % of a plain copy's
// rate on this device.  The thread that issues is what a smaller unit runs into: tasks of
// 6144 bytes took 233 us, and a place in the order found by division at every task 221 us.
// Thirds with the same bytes ahead took 166 us, whole pages 169 us; 16 slots of thirds, 13 ahead,
// 186 us, so more in flight does not help.
constexpr int COPY_THREADS = 256;
constexpr int PARTS = 4;
constexpr int PART_CODES = PAGE * D / PARTS;   // 9216
constexpr int PAGE_SCALES = PAGE * 8;          // 512
constexpr int SLOT = PART_CODES + PAGE_SCALES;
constexpr int COPY_SLOTS = 12;                 // as many as fit beside the bitmaps, 8 at the least
constexpr int COPY_LAG = 4;                    // stores that may still be on their way while loads run ahead
constexpr int COPY_SMEM = 227 * 1024 - 256;
static_assert(PART_CODES % 16 == 0 && PAGE * D % PARTS == 0, "bulk copies move 16-byte units");
static_assert((COPY_SMEM - KV8_PAGES_MAX_BLOCKS / 4) / SLOT >= 8, "the ring beside the largest bitmaps");
constexpr uint64_t COPY_WAIT_NS = 2000000000ull;

__global__ void __launch_bounds__(COPY_THREADS)
copy_kernel(uint8_t* codes, float* scales, int n_layers, int64_t n_slots, const int32_t* __restrict__ moves,
            const int32_t* __restrict__ n_moves, int64_t max_moves, int slots, unsigned* err) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[COPY_SLOTS];
  __shared__ int never;
  const int64_t n_blocks = n_slots / PAGE;
  const int words = (int)((n_blocks + 31) / 32);
  unsigned* named = reinterpret_cast<unsigned*>(ring + slots * SLOT);
  unsigned* twice = named + words;
  int64_t n = max_moves;
  if (n_moves != nullptr) {
    n = *n_moves;
    n = n < 0 ? 0 : (n < max_moves ? n : max_moves);
  }
  const int64_t tasks = n * n_layers * PARTS;
  const int64_t f0 = tasks * blockIdx.x / gridDim.x, f1 = tasks * (blockIdx.x + 1) / gridDim.x;
  if (f0 >= f1) return;
  for (int w = threadIdx.x; w < 2 * words; w += COPY_THREADS) named[w] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) mbar_init(&full[s], 1);
    never = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  auto inside = [&](int32_t p) { return p >= 0 && p < n_blocks; };
  // A place in the order of the tasks, moved on without a division: one for the loads, one
  // for the stores behind them.
  struct Place {
    int64_t pair;
    int layer, part;
    int32_t a, d;   // the pair's pages
  };
  auto name = [&](Place& k) {
    k.a = __ldg(&moves[2 * k.pair]);
    k.d = __ldg(&moves[2 * k.pair + 1]);
  };
  auto next = [&](Place& k) {
    if (++k.part < PARTS) return;
    k.part = 0;
    if (++k.layer < n_layers) return;
    k.layer = 0;
    if (++k.pair < n) name(k);
  };
  Place in;
  in.part = (int)(f0 % PARTS);
  in.layer = (int)(f0 / PARTS % n_layers);
  in.pair = f0 / PARTS / n_layers;
  name(in);
  Place out = in;
  auto load = [&](int s) {
    const uint32_t at = smem_u32(ring + s * SLOT);
    const bool ok = inside(in.a) && inside(in.d) && in.a != in.d;
    const bool first = in.part == 0;
    mbar_arrive_expect_tx(&full[s], ok ? (uint32_t)(PART_CODES + (first ? PAGE_SCALES : 0)) : 0u);
    if (ok) {
      const int64_t row = in.layer * n_slots + (int64_t)in.a * PAGE;
      bulk_load_g2s(at, codes + row * D + in.part * PART_CODES, PART_CODES, &full[s]);
      if (first) bulk_load_g2s(at + PART_CODES, scales + row * 2, PAGE_SCALES, &full[s]);
    }
    next(in);
  };
  const int ahead = slots - COPY_LAG;
  int64_t asked = f0;   // the next task to load, and its slot
  int to = 0;
  if (threadIdx.x == 0) {
    for (; asked < f1 && asked < f0 + ahead; ++asked) load(to++);
  } else {
    for (int64_t i = threadIdx.x - 1; i < n; i += COPY_THREADS - 1) {
      const int32_t a = __ldg(&moves[2 * i]), d = __ldg(&moves[2 * i + 1]);
      if (inside(a) && inside(d) && a != d) {
        const unsigned bit = 1u << (d & 31);
        if (atomicOr(&named[d >> 5], bit) & bit) atomicOr(&twice[d >> 5], bit);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  int s = 0;
  uint32_t phase = 0;
  for (int64_t f = f0; f < f1; ++f) {
    if (asked < f1) {
      // the slot was stored from COPY_LAG tasks ago
      asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(COPY_LAG - 1) : "memory");
      load(to);
      ++asked;
      if (++to == slots) to = 0;
    }
    if (!mbar_wait(&full[s], phase, &never, COPY_WAIT_NS)) {
      flag(err, KV8_PAGES_ETIMEOUT);
      for (int64_t g = f + 1; g < asked; ++g) {  // the loads in flight land first
        if (++s == slots) s = 0, phase ^= 1u;
        (void)mbar_wait(&full[s], phase, &never, COPY_WAIT_NS);
      }
      break;
    }
    bool ok = inside(out.a) && inside(out.d) && out.a != out.d;
    if (!inside(out.a) || !inside(out.d)) flag(err, KV8_PAGES_EINDEX);
    if (ok && (((twice[out.d >> 5] >> (out.d & 31)) & 1u) != 0u || ((named[out.a >> 5] >> (out.a & 31)) & 1u) != 0u)) {
      ok = false;
      flag(err, KV8_PAGES_EINDEX);
    }
    if (ok) {
      const uint32_t at = smem_u32(ring + s * SLOT);
      const int64_t row = out.layer * n_slots + (int64_t)out.d * PAGE;
      bulk_store_s2g(codes + row * D + out.part * PART_CODES, at, PART_CODES);
      if (out.part == 0) bulk_store_s2g(scales + row * 2, at + PART_CODES, PAGE_SCALES);
    }
    next(out);
    bulk_commit();  // one group per task, empty ones too: the count above is in tasks
    if (++s == slots) s = 0, phase ^= 1u;
  }
  bulk_wait_all();
}

// One cluster of `ctas` CTAs.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kernel)(P...), int ctas, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(PG_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A kernel's opt-in to `bytes` of dynamic shared memory on the current device.
template <typename K>
cudaError_t allow_smem(std::atomic<int> (&memo)[MAX_DEVICES], K kernel, int bytes) {
  int done = 0;
  return per_device(memo, [&](int* v) {
    *v = 1;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  }, &done);
}

int ctas_for(int64_t entries) { return entries <= ONE_PASS ? 1 : PG_CTAS; }

}  // namespace

cudaError_t launch_pages_append(const PageTable& t, const int32_t* n_new, int32_t* q_start, int64_t* dst_slot,
                                int64_t cap, unsigned* err, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  const cudaError_t e = allow_smem(memo, append_kernel, (2 * KV8_PAGES_MAX_SEQS + 1) * 4);
  if (e != cudaSuccess) return e;
  return launch_cluster(append_kernel, ctas_for(cap), (size_t)(2 * t.B + 1) * 4, s, t, n_new, q_start, dst_slot, cap, err);
}

cudaError_t launch_pages_fork(const PageTable& t, const int32_t* src, const int32_t* dst, const int32_t* fork_len,
                              int n, int32_t* moves, int32_t* n_moves, unsigned* err, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  const cudaError_t e = allow_smem(memo, fork_kernel, (3 * KV8_PAGES_MAX_SEQS + 1) * 4);
  if (e != cudaSuccess) return e;
  return launch_cluster(fork_kernel, ctas_for((int64_t)n * t.max_blocks), (size_t)(t.B + 2 * n + 1) * 4, s, t, src, dst,
                        fork_len, n, moves, n_moves, err);
}

cudaError_t launch_pages_free(const PageTable& t, const int32_t* seq, int n, unsigned* err, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  const cudaError_t e = allow_smem(memo, free_kernel, KV8_PAGES_MAX_SEQS * 4);
  if (e != cudaSuccess) return e;
  return launch_cluster(free_kernel, ctas_for((int64_t)n * t.max_blocks), (size_t)t.B * 4, s, t, seq, n, err);
}

cudaError_t launch_pages_compact(const PageTable& t, int32_t* moves, int32_t* n_moves, int32_t* n_live, unsigned* err,
                                 cudaStream_t s) {
  const int64_t work = t.n_blocks + (int64_t)t.B * t.max_blocks;
  return launch_cluster(compact_kernel, ctas_for(work), 0, s, t, moves, n_moves, n_live, err);
}

cudaError_t launch_pages_copy(uint8_t* codes, float* scales, int n_layers, int64_t n_slots, const int32_t* moves,
                              const int32_t* n_moves, int64_t max_moves, unsigned* err, cudaStream_t s) {
  static std::atomic<int> memo[MAX_DEVICES];
  const int maps = (int)((n_slots / PAGE + 31) / 32) * 8;
  const cudaError_t e = allow_smem(memo, copy_kernel, COPY_SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tasks = max_moves * n_layers * PARTS;
  int slots = (COPY_SMEM - maps) / SLOT;
  if (slots > COPY_SLOTS) slots = COPY_SLOTS;
  copy_kernel<<<(unsigned)(tasks < NUM_SMS ? tasks : NUM_SMS), COPY_THREADS, (size_t)slots * SLOT + maps, s>>>(
      codes, scales, n_layers, n_slots, moves, n_moves, max_moves, slots, err);
  return cudaGetLastError();
}

}  // namespace kv8
