// norm.cu -- kv8_norm_quantize_rows: the residual's addition, the RMS norm and the e4m3
// quantizer of rows in one pass.  Per row (f32 throughout):
//   t = x + residual;   y = (t * (1 / sqrt(sum t^2 / width + eps))) * weight
//   scale = max |y| / 448 of the row, or of every `group` channels;  code = e4m3(y * (448 / max |y|))
// with the quantizer's rules of kv8_quantize_rows for zeros, NaN and a subnormal maximum.
//
// A thread keeps its channels in registers, eight (a unit) at a time, E units of them; unit u of the
// row is thread u mod N's, so that a group's units lie in neighbouring lanes.  Rows of up to 32 E units
// are one warp's, longer ones a CTA's.
#include <cuda_bf16.h>

#include "kv8_common.cuh"

namespace kv8 {
namespace {

constexpr int UNIT = 8;       // channels
constexpr int ROW_WARPS = 8;  // rows of a CTA where each is a warp's
constexpr int MAX_THREADS = 1024;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

// A unit at p, of which `left` channels are the row's (VEC: all, at a 16-byte boundary).
template <typename T, bool VEC>
__device__ __forceinline__ void load_unit(const T* p, int left, float (&v)[UNIT]) {
  if constexpr (VEC) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < UNIT / N; ++i) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < N; ++j) v[N * i + j] = to_f32(e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < UNIT; ++j) v[j] = j < left ? to_f32(p[j]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_unit(T* p, int left, const float (&v)[UNIT]) {
  if constexpr (VEC) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < UNIT / N; ++i) {
      uint4 w;
      T* e = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = from_f32<T>(v[N * i + j]);
      reinterpret_cast<uint4*>(p)[i] = w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < UNIT; ++j)
      if (j < left) p[j] = from_f32<T>(v[j]);
  }
}

// Over the row's threads: a warp, or the CTA (through `tmp`, of its own for each call).
template <bool WARP, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if constexpr (!WARP) {
    const int lane = threadIdx.x & 31, n = blockDim.x >> 5;
    if (lane == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < n ? tmp[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, v, o);
      v = MAX ? fmaxf(v, u) : v + u;
    }
  }
  return v;
}

template <typename T, int E, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? ROW_WARPS * 32 : MAX_THREADS) norm_kernel(const NormArgs a) {
  __shared__ float tmp[2][32];
  const int n = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= a.n_rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  float t[E][UNIT];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * n + me) * UNIT;
#pragma unroll
    for (int j = 0; j < UNIT; ++j) t[i][j] = 0.f;
    if (c < a.width) load_unit<T, VEC>(x + c, a.width - c, t[i]);
  }
  if (a.residual != nullptr) {
    const T* r = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* out = a.residual_out == nullptr ? nullptr : static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (i * n + me) * UNIT;
      if (c >= a.width) continue;
      float v[UNIT];
      load_unit<T, VEC>(r + c, a.width - c, v);
#pragma unroll
      for (int j = 0; j < UNIT; ++j) t[i][j] = __fadd_rn(t[i][j], v[j]);
      if (out != nullptr) store_unit<T, VEC>(out + c, a.width - c, t[i]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i)
#pragma unroll
    for (int j = 0; j < UNIT; ++j) ss = fmaf(t[i][j], t[i][j], ss);
  ss = row_reduce<WARP, false>(ss, tmp[0]);
  const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.width), a.eps)));
  T* normed = a.normed == nullptr ? nullptr : static_cast<T*>(a.normed) + row * a.normed_stride;
  float top[E], all = 0.f;  // largest magnitudes, NaN left out
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * n + me) * UNIT;
    top[i] = 0.f;
    if (c < a.width) {
      float w[UNIT];
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(w) = __ldg(reinterpret_cast<const float4*>(a.weight + c));
        *reinterpret_cast<float4*>(w + 4) = __ldg(reinterpret_cast<const float4*>(a.weight + c) + 1);
      } else {
#pragma unroll
        for (int j = 0; j < UNIT; ++j) w[j] = j < a.width - c ? __ldg(a.weight + c + j) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < UNIT; ++j) {
        t[i][j] = __fmul_rn(__fmul_rn(t[i][j], inv), w[j]);
        if (VEC || j < a.width - c) top[i] = fmaxf(top[i], fabsf(t[i][j]));
      }
      if (normed != nullptr) store_unit<T, VEC>(normed + c, a.width - c, t[i]);
    }
    all = fmaxf(all, top[i]);
  }
  float* scales = a.scales + row * a.n_groups;
  if (a.group == 0) {
    all = row_reduce<WARP, true>(all, tmp[1]);
    if (me == 0) scales[0] = __fdiv_rn(all, 448.f);
  } else {
    const int lanes = a.group / UNIT;  // at most 32
#pragma unroll
    for (int i = 0; i < E; ++i) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, top[i], o);
        if (o < lanes) top[i] = fmaxf(top[i], u);
      }
      const int u = i * n + me;
      if ((u & (lanes - 1)) == 0 && u * UNIT < a.width) scales[u / lanes] = __fdiv_rn(top[i], 448.f);
    }
  }
  uint8_t* codes = a.codes + row * a.codes_stride;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * n + me) * UNIT;
    if (c >= a.width) continue;
    const float f = __fdiv_rn(448.f, a.group == 0 ? all : top[i]);
    const bool guard = !isfinite(f);
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < UNIT; j += 2) {
      uint32_t two;
      if (guard) {
        two = (t[i][j] == t[i][j] && signbit(t[i][j]) ? 0x80u : 0u) |
              (t[i][j + 1] == t[i][j + 1] && signbit(t[i][j + 1]) ? 0x8000u : 0u);
      } else {
        float p0 = __fmul_rn(t[i][j], f), p1 = __fmul_rn(t[i][j + 1], f);
        p0 = isnan(p0) ? 0.f : p0;
        p1 = isnan(p1) ? 0.f : p1;
        two = f32x2_to_e4m3x2(p0, p1);
      }
      q[j / 4] |= two << (8 * (j % 4));
    }
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(codes + c) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int j = 0; j < UNIT; ++j)
        if (j < a.width - c) codes[c + j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
    }
  }
}

template <typename T, bool VEC>
cudaError_t launch_as(const NormArgs& a, cudaStream_t s) {
  const int units = (a.width + UNIT - 1) / UNIT;
  const unsigned warps = (unsigned)((a.n_rows + ROW_WARPS - 1) / ROW_WARPS), rows = (unsigned)a.n_rows;
  auto threads = [&](int e) { return ((units + e - 1) / e + 31) / 32 * 32; };
  if (units <= 32) norm_kernel<T, 1, VEC, true><<<warps, ROW_WARPS * 32, 0, s>>>(a);
  else if (units <= 64) norm_kernel<T, 2, VEC, true><<<warps, ROW_WARPS * 32, 0, s>>>(a);
  else if (units <= 1024 && a.n_rows <= NUM_SMS) norm_kernel<T, 1, VEC, false><<<rows, threads(1), 0, s>>>(a);
  else if (units <= 2048) norm_kernel<T, 2, VEC, false><<<rows, threads(2), 0, s>>>(a);
  else norm_kernel<T, 4, VEC, false><<<rows, threads(4), 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const NormArgs& a, cudaStream_t s) {
  // rows that begin at 16-byte boundaries and are whole units
  const int64_t per = 16 / sizeof(T);
  auto even = [&](const void* p, int64_t stride) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride % per == 0 || a.n_rows == 1));
  };
  const bool vec = a.width % UNIT == 0 && even(a.x, a.x_stride) && even(a.residual, a.residual_stride) &&
                   even(a.residual_out, a.residual_out_stride) && even(a.normed, a.normed_stride) &&
                   reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.codes) % UNIT == 0 &&
                   (a.codes_stride % UNIT == 0 || a.n_rows == 1);
  return vec ? launch_as<T, true>(a, s) : launch_as<T, false>(a, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t s) {
  if (dtype == KV8_BF16) return launch_typed<__nv_bfloat16>(a, s);
  if (dtype == KV8_F16) return launch_typed<__half>(a, s);
  return launch_typed<float>(a, s);
}

}  // namespace kv8
