// chunk.cu -- absorbed MLA attention of a chunk of new tokens per sequence over
// the paged fp8 latent cache, causal inside the chunk:
//   z_t = sm * ( sLc_t <q_lat, dec(Lc_t)> + sRc_t <q_rope, dec(Rc_t)> ),  t < lim
//   out = sum_t softmax(z)_t sLc_t dec(Lc_t)
// with lim = T - n + i + 1 for token i of the n queries of a sequence of T cached
// tokens (its last n tokens are the chunk itself), or T without the causal mask.
//
// One warp per row (a token and a head): a lane holds 16 latent channels and two
// rotary ones, and walks the visible keys with a running maximum and sum.
#include <cuda_bf16.h>

#include "kv8_common.cuh"

namespace kv8 {
namespace {

constexpr int CW = 8;  // rows per CTA
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__global__ void __launch_bounds__(CW * 32) chunk_kernel(const ChunkArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * CW + (threadIdx.x >> 5);
  if (row >= a.total_q * a.H) return;
  const int64_t tok = row / a.H, h = row % a.H;
  // the sequence that holds the token: q_start[b] <= tok < q_start[b + 1]
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= tok) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
  if (tok < q0 || tok >= q1) return;
  if (q0 < 0 || q1 > a.total_q) {
    if (lane == 0) atomicOr(a.err, ERR_BLOCK_TABLE);
    return;
  }
  int64_t T = a.seq_lens[b];
  const int64_t room = (int64_t)a.max_blocks * PAGE;
  if (T < 0 || T > room) {
    if (lane == 0) atomicOr(a.err, ERR_SEQ_LEN);
    T = T < 0 ? 0 : room;
  }
  int64_t lim = a.causal ? T - (q1 - tok) + 1 : T;
  lim = lim < 0 ? 0 : lim;

  const uint16_t* ql = a.q_lat + tok * a.ql_t + h * a.ql_h + lane * 16;
  const uint16_t* qr = a.q_rope + tok * a.qr_t + h * a.qr_h + lane * 2;
  float q[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) q[k] = bf16_f32(ql[k]);
  const float r0 = bf16_f32(qr[0]), r1 = bf16_f32(qr[1]);
  const float c = a.sm_scale * LOG2E;
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  for (int64_t p0 = 0; p0 < lim; p0 += PAGE) {
    const int32_t blk = a.block_table[(int64_t)b * a.max_blocks + p0 / PAGE];
    if (blk < 0 || (int64_t)blk >= a.n_blocks) {
      if (lane == 0) atomicOr(a.err, ERR_BLOCK_TABLE);
      continue;
    }
    const int n = (int)(lim - p0 < PAGE ? lim - p0 : PAGE);
    for (int t = 0; t < n; ++t) {
      const int64_t slot = (int64_t)blk * PAGE + t;
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.codes + slot * D) + lane);
      const uint32_t y = __ldg(reinterpret_cast<const uint16_t*>(a.codes + slot * D + DL) + lane);
      const float sL = __ldg(a.scales + slot * 2), sR = __ldg(a.scales + slot * 2 + 1);
      float v[16], w[4];
      e4m3x4_to_f32(x.x, v);
      e4m3x4_to_f32(x.y, v + 4);
      e4m3x4_to_f32(x.z, v + 8);
      e4m3x4_to_f32(x.w, v + 12);
      e4m3x4_to_f32(y, w);
      float dl = 0.f, dr = w[0] * r0 + w[1] * r1;
#pragma unroll
      for (int k = 0; k < 16; ++k) dl += q[k] * v[k];
      float z = sL * dl + sR * dr;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
      z *= c;
      const float mn = fmaxf(m, z);
      const float al = exp2f(m - mn), p = exp2f(z - mn), pw = p * sL;
      l = l * al + p;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = o[k] * al + pw * v[k];
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
    w[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* out = reinterpret_cast<uint4*>(a.out + row * DL + lane * 16);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (a.lse != nullptr && lane == 0)
    a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

int64_t chunk_workspace(int, int, int64_t, int) { return 256; }

cudaError_t launch_chunk(ChunkArgs a, void* workspace, cudaStream_t s) {
  a.err = static_cast<unsigned*>(workspace);
  const cudaError_t e = cudaMemsetAsync(a.err, 0, sizeof(unsigned), s);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.total_q * a.H;
  chunk_kernel<<<(unsigned)((rows + CW - 1) / CW), CW * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kv8
