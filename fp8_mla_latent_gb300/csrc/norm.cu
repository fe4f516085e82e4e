// norm.cu -- kv8_norm_quantize_rows: the residual's addition, the RMS norm and the e4m3
// quantizer of rows in one pass.  Per row (f32 throughout):
//   t = x + residual;   y = (t * (1 / sqrt(sum t^2 / width + eps))) * weight
//   scale = max |y| / 448 of the row, or of every `group` channels;  code = e4m3(y * (448 / max |y|))
// with the quantizer's rules of kv8_quantize_rows for zeros, NaN and a subnormal maximum.
//
// A thread keeps its channels in registers, eight (a unit) at a time, up to four units of them; unit u of the
// row is thread u mod N's, so that a group's units lie in neighbouring lanes.  Rows of up to 64 units
// are one warp's, longer ones a CTA's; many long ones go to the kernel with a ring, below.
//
// The kernel right below is for what that one does not take.  It is a chain of loads, a sum, a maximum and
// stores a row: few rows are latency (one of 7168 channels 3.0 us, 64 3.3), short rows the instructions (16384 x 512
// bf16 with a residual 12.0 us, 0.73 of the copy rate; x 128 6.3 us, 0.34).  Rows at odd addresses are read and
// written by the element, 32 neighbours a warp, some 90 instructions for each 32 (16384 x 7169 bf16 with a residual and
// a scale for every 128 channels 390 us, 0.31): such rows with groups, and odd ones that are few, short or over
// 2048 units, are left to it.
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

// the code of a value whose row (or group) has no scale: a signed zero, 0x00 for NaN
__device__ __forceinline__ uint32_t zero_byte(float v) { return v == v && signbit(v) ? 0x80u : 0u; }

// A thread's channels 0 .. 7 of its unit, in a row at p: eight in a row (VEC, at a 16-byte boundary), or
// every 32nd of the 256 that its warp has, so that a warp's accesses lie together;
// `left` channels from the first of them to the row's end.
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
    for (int j = 0; j < UNIT; ++j) v[j] = 32 * j < left ? to_f32(p[32 * j]) : 0.f;
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
      if (32 * j < left) p[32 * j] = from_f32<T>(v[j]);
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

template <typename T, int UNITS, bool VEC, bool WARP>
__global__ void __launch_bounds__(WARP ? ROW_WARPS * 32 : MAX_THREADS) norm_kernel(const NormArgs a) {
  __shared__ float tmp[2][32];
  const int n = WARP ? 32 : blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x, lane = me & 31;
  const int64_t row = WARP ? (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= a.n_rows) return;
  auto at = [&](int i) { return VEC ? (i * n + me) * UNIT : (i * n + me - lane) * UNIT + lane; };
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  // (both rows are asked for before any of the sum is written, which may lie over them)
  float t[UNITS][UNIT];
  const T* r = a.residual == nullptr ? nullptr : static_cast<const T*>(a.residual) + row * a.residual_stride;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = at(i);
#pragma unroll
    for (int j = 0; j < UNIT; ++j) t[i][j] = 0.f;
    if (c >= a.width) continue;
    load_unit<T, VEC>(x + c, a.width - c, t[i]);
    if (r == nullptr) continue;
    float v[UNIT];
    load_unit<T, VEC>(r + c, a.width - c, v);
#pragma unroll
    for (int j = 0; j < UNIT; ++j) t[i][j] = __fadd_rn(t[i][j], v[j]);
  }
  if (a.residual_out != nullptr) {
    T* out = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
      if (at(i) < a.width) store_unit<T, VEC>(out + at(i), a.width - at(i), t[i]);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < UNITS; ++i)
#pragma unroll
    for (int j = 0; j < UNIT; ++j) ss = fmaf(t[i][j], t[i][j], ss);
  ss = row_reduce<WARP, false>(ss, tmp[0]);
  const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.width), a.eps)));
  T* normed = a.normed == nullptr ? nullptr : static_cast<T*>(a.normed) + row * a.normed_stride;
  float all = 0.f;  // largest magnitude, NaN left out
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = at(i);
    if (c >= a.width) continue;
    float w[UNIT];
    if constexpr (VEC) {
      *reinterpret_cast<float4*>(w) = __ldg(reinterpret_cast<const float4*>(a.weight + c));
      *reinterpret_cast<float4*>(w + 4) = __ldg(reinterpret_cast<const float4*>(a.weight + c) + 1);
    } else {
#pragma unroll
      for (int j = 0; j < UNIT; ++j) w[j] = 32 * j < a.width - c ? __ldg(a.weight + c + 32 * j) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < UNIT; ++j) {
      t[i][j] = __fmul_rn(__fmul_rn(t[i][j], inv), w[j]);
      if (!VEC && 32 * j >= a.width - c) t[i][j] = 0.f;  // (nothing times an infinity)
      all = fmaxf(all, fabsf(t[i][j]));
    }
    if (normed != nullptr) store_unit<T, VEC>(normed + c, a.width - c, t[i]);
  }
  float* scales = a.scales + row * a.n_groups;
  if (a.group == 0) {
    all = row_reduce<WARP, true>(all, tmp[1]);
    if (me == 0) scales[0] = __fdiv_rn(all, 448.f);
  }
  uint8_t* codes = a.codes + row * a.codes_stride;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = at(i);
    if (!VEC) {
      float top[UNIT];  // (of the groups that the channels lie in)
#pragma unroll
      for (int j = 0; j < UNIT; ++j) top[j] = a.group == 0 ? all : fabsf(t[i][j]);
      if (a.group != 0) {
        const int span = a.group / 32;  // channels of a thread in a group: 1, 2, 4 or 8
#pragma unroll
        for (int o = 1; o < UNIT; o <<= 1) {
          if (o >= span) break;
#pragma unroll
          for (int j = 0; j < UNIT; j += 2 * o) {
            const float m = fmaxf(top[j], top[j + o]);  // (NaN loses)
#pragma unroll
            for (int k = 0; k < 2 * o; ++k) top[j + k] = m;
          }
        }
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
          if (j & (span - 1)) {
            top[j] = top[j - 1];
            continue;
          }
          top[j] = fmaxf(top[j], 0.f);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
          const int first = c - lane + 32 * j;
          if (lane == 0 && first < a.width) scales[first / a.group] = __fdiv_rn(top[j], 448.f);
        }
      }
      float f = 0.f;
#pragma unroll
      for (int j = 0; j < UNIT; ++j) {
        if (j == 0 || (a.group != 0 && (j & (a.group / 32 - 1)) == 0)) f = __fdiv_rn(448.f, top[j]);
        if (32 * j >= a.width - c) continue;
        uint32_t q;
        if (isfinite(f)) {
          float p = __fmul_rn(t[i][j], f);
          p = isnan(p) ? 0.f : p;
          q = f32x2_to_e4m3x2(p, 0.f) & 0xFFu;
        } else {
          q = zero_byte(t[i][j]);
        }
        codes[c + 32 * j] = (uint8_t)q;
      }
    } else {
      float top = all;
      if (a.group != 0) {
        top = 0.f;
#pragma unroll
        for (int j = 0; j < UNIT; ++j) top = fmaxf(top, fabsf(t[i][j]));
        const int lanes = a.group / UNIT;  // at most 32
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float u = __shfl_xor_sync(0xffffffffu, top, o);
          if (o < lanes) top = fmaxf(top, u);
        }
        if ((lane & (lanes - 1)) == 0 && c < a.width) scales[c / a.group] = __fdiv_rn(top, 448.f);
      }
      if (c >= a.width) continue;
      const float f = __fdiv_rn(448.f, top);
      uint32_t q[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < UNIT; j += 2) {
        uint32_t two;
        if (isfinite(f)) {
          float p0 = __fmul_rn(t[i][j], f), p1 = __fmul_rn(t[i][j + 1], f);
          p0 = isnan(p0) ? 0.f : p0;
          p1 = isnan(p1) ? 0.f : p1;
          two = f32x2_to_e4m3x2(p0, p1);
        } else {
          two = zero_byte(t[i][j]) | (zero_byte(t[i][j + 1]) << 8);
        }
        q[j / 4] |= two << (8 * (j % 4));
      }
      *reinterpret_cast<uint2*>(codes + c) = make_uint2(q[0], q[1]);
    }
  }
}

// Many rows of whole units: a CTA goes over rows gridDim.x apart and keeps the weights in registers.  Each
// thread brings its own channels of the next rows into shared memory by asynchronous copies and reads
// them back itself, so that nothing is waited for together but the row's sums.
//
// HBM bounds it: two CTAs of 16 warps hold one SM's share of the rows in flight (28 KB a CTA at 7168
// channels of two 16-bit inputs; with four rows ahead instead of one it is slower, 131 us against 124).
// With one input the instructions are next: 350 a warp and row of two units a thread, of which two
// thirds do not depend on the units, so 16-bit rows without a residual take four units a thread and three CTAs
// (16384 x 7168 bf16 rows, a scale a row: 90 us with two, 74 with four, and 86 with a scale for every 128 channels; with
// a residual 124 and 127; 4096 f32 rows with a residual 89 and 97).  f32 rows are far from the copy rate, 16384 x
// 7168 without a residual 152 us, 0.57, with one 335, 0.67: a unit is two pieces of 16 bytes there, so that a warp's
// request for one of them takes half of each 32-byte sector, and every sector comes from L2 twice (944 MB of 470).
// Measured, one GB300, 16384 x 7168 bf16 with a residual: 124 us, 6.68 TB/s, 0.99 of the copy rate.
//
// Rows of odd widths (SHIFT) begin anywhere, but if all the row's arrays begin equally far behind a multiple of
// eight elements, `shift` of them, the units are taken from there: whole ones as above, the first and the last
// by the element where they are written.  (What is read with these lies in the 16 bytes of one of the row's own
// elements; it is set to 0.)  A CTA's rows lie a multiple of eight apart, so that it has one shift, and its weights
// stay in registers.  With a scale a group the shift has to be 0 (rows that only end oddly).  16384 x 7169 bf16
// 92 us, 282 by the element (with a residual 163, 0.74 of the copy rate); 16384 x 1501 f16 with a residual and
// normed rows 46, 69 by the element; 517 rows of those 4.9, 5.6.
constexpr int STAGES = 2;

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 of_pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// max(|a|, |b|, c), NaN left out
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two values of a 16-bit type
template <typename T>
__device__ __forceinline__ uint64_t unpack2(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
    return pair_of(f.x, f.y);
  } else {
    return pair_of(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  const float2 f = of_pair(v);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const uint64_t (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = of_pair(v[2 * i]), b = of_pair(v[2 * i + 1]);
      reinterpret_cast<float4*>(p)[i] = make_float4(a.x, a.y, b.x, b.y);
    }
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0]), pack2<T>(v[1]), pack2<T>(v[2]), pack2<T>(v[3]));
  }
}

// the same by the element, for those at c .. c + 7 that lie in [0, width)
template <typename T>
__device__ __forceinline__ void store_some(T* p, int c, int width, const uint64_t (&v)[4]) {
#pragma unroll
  for (int j = 0; j < UNIT; ++j) {
    const float2 f = of_pair(v[j / 2]);
    if (c + j >= 0 && c + j < width) p[j] = from_f32<T>(j & 1 ? f.y : f.x);
  }
}
static_assert(NUM_SMS % UNIT == 0, "a CTA's rows lie a multiple of eight apart");

template <typename T, bool ADD, bool SHIFT, int E, int THREADS>
__global__ void __launch_bounds__(THREADS, E == 2 ? 2 : (THREADS <= 256 ? 3 : 1)) norm_stream_kernel(const NormArgs a) {
  constexpr int Q = UNIT * (int)sizeof(T) / 16;  // 16-byte pieces of a unit
  constexpr int ROWS_IN = ADD ? 2 : 1;
  extern __shared__ __align__(16) uint8_t ring[];                  // [STAGES][ROWS_IN][E][Q][threads] pieces
  __shared__ float4 tmp[4][THREADS / 128];  // (a warp's each; 0 behind the last)
  const int n = blockDim.x, me = threadIdx.x, lane = me & 31;
  for (int i = me; i < 4 * THREADS / 32; i += n) reinterpret_cast<float*>(tmp)[i] = 0.f;
  __syncthreads();
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + me * 16;
  const int shift = SHIFT ? (int)((reinterpret_cast<uintptr_t>(a.x) / sizeof(T) + (uint64_t)blockIdx.x * a.x_stride) % UNIT) : 0;
  auto at = [&](int i) { return (i * n + me) * UNIT - shift; };  // the first channel of a unit
  auto edge = [&](int c) { return SHIFT && (c < 0 || c + UNIT > a.width); };
  const uint32_t stage_bytes = (uint32_t)(ROWS_IN * E * Q * n * 16);
  auto ask = [&](int64_t row, int stage) {
    if (row < a.n_rows) {
#pragma unroll
      for (int w = 0; w < ROWS_IN; ++w) {
        const T* p = w == 0 ? static_cast<const T*>(a.x) + row * a.x_stride
                            : static_cast<const T*>(a.residual) + row * a.residual_stride;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int c = at(i);
          if (c >= a.width) continue;
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            constexpr int PIECE = 16 / (int)sizeof(T);
            if (SHIFT && Q > 1 && (c + (q + 1) * PIECE <= 0 || c + q * PIECE >= a.width)) continue;
            copy_async16(mine + stage * stage_bytes + (uint32_t)(((w * E + i) * Q + q) * n * 16), p + c + q * PIECE);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int64_t row = blockIdx.x;
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) ask(row + (int64_t)k * gridDim.x, k);
  bool odd_weight = false;  // one of this thread's is not finite
  uint64_t wt[E][4];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = at(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) wt[i][j] = 0;
    if (c < a.width) {
      float4 u, v;
      if constexpr (SHIFT) {
        auto w = [&](int j) { return c + j >= 0 && c + j < a.width ? __ldg(a.weight + c + j) : 0.f; };
        u = make_float4(w(0), w(1), w(2), w(3));
        v = make_float4(w(4), w(5), w(6), w(7));
      } else {
        u = __ldg(reinterpret_cast<const float4*>(a.weight + c));
        v = __ldg(reinterpret_cast<const float4*>(a.weight + c) + 1);
      }
      wt[i][0] = pair_of(u.x, u.y);
      wt[i][1] = pair_of(u.z, u.w);
      wt[i][2] = pair_of(v.x, v.y);
      wt[i][3] = pair_of(v.z, v.w);
      odd_weight |= !(u.x * 0.f + u.y * 0.f + u.z * 0.f + u.w * 0.f + v.x * 0.f + v.y * 0.f + v.z * 0.f + v.w * 0.f == 0.f);
    }
  }
  const float per_width = __fdiv_rn(1.f, (float)a.width);
  int stage = 0, turn = 0;
  for (; row < a.n_rows; row += gridDim.x) {
    ask(row + (int64_t)(STAGES - 1) * gridDim.x, stage == 0 ? STAGES - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    uint64_t t[E][4];
    uint64_t ss2 = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = at(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) t[i][j] = 0;
      if (c >= a.width) continue;
#pragma unroll
      for (int w = 0; w < ROWS_IN; ++w) {
        uint64_t v[4];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const uint4 u = lds128(mine + stage * stage_bytes + (uint32_t)(((w * E + i) * Q + q) * n * 16));
          if constexpr (sizeof(T) == 4) {
            v[2 * q] = pair_of(__uint_as_float(u.x), __uint_as_float(u.y));
            v[2 * q + 1] = pair_of(__uint_as_float(u.z), __uint_as_float(u.w));
          } else {
            v[0] = unpack2<T>(u.x);
            v[1] = unpack2<T>(u.y);
            v[2] = unpack2<T>(u.z);
            v[3] = unpack2<T>(u.w);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) t[i][j] = w == 0 ? v[j] : add_pair(t[i][j], v[j]);
      }
      if (edge(c)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = of_pair(t[i][j]);
          const int k = c + 2 * j;
          t[i][j] = pair_of(k >= 0 && k < a.width ? f.x : 0.f, k >= -1 && k + 1 < a.width ? f.y : 0.f);
        }
      }
      if (ADD && a.residual_out != nullptr) {
        T* p = static_cast<T*>(a.residual_out) + row * a.residual_out_stride + c;
        if (edge(c)) store_some<T>(p, c, a.width, t[i]);
        else store_pairs<T>(p, t[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) ss2 = fma_pair(t[i][j], t[i][j], ss2);
    }
    const float2 s2 = of_pair(ss2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // (the row after next writes there again, behind the next one's barrier)
    if (lane == 0) reinterpret_cast<float*>(tmp[turn])[me >> 5] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < THREADS / 128; ++w) {
      const float4 u = tmp[turn][w];
      ss += (u.x + u.y) + (u.z + u.w);
    }
    const float inv = rsqrtf(__fadd_rn(__fmul_rn(ss, per_width), a.eps));
    const uint64_t inv2 = pair_of(inv, inv);
    const bool odd = odd_weight || !(ss + inv < INFINITY);  // (otherwise no y is NaN)
    float top[E], all = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = at(i);
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t[i][j] = mul_pair(mul_pair(t[i][j], inv2), wt[i][j]);
        const float2 f = of_pair(t[i][j]);
        m = max_abs(f.x, f.y, m);
      }
      if (c >= a.width) m = 0.f;  // (nothing times an infinity)
      if (a.normed != nullptr && c < a.width) {
        T* p = static_cast<T*>(a.normed) + row * a.normed_stride + c;
        if (edge(c)) store_some<T>(p, c, a.width, t[i]);
        else store_pairs<T>(p, t[i]);
      }
      top[i] = m;
      all = fmaxf(all, m);
    }
    float* scales = a.scales + row * a.n_groups;
    if (a.group == 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
      if (lane == 0) reinterpret_cast<float*>(tmp[2 + turn])[me >> 5] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < THREADS / 128; ++w) {
        const float4 u = tmp[2 + turn][w];
        all = fmaxf(all, fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)));
      }
      if (me == 0) scales[0] = __fdiv_rn(all, 448.f);
    } else {
      const int lanes = a.group / UNIT;  // 4 .. 32
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (o >= lanes) break;
#pragma unroll
        for (int i = 0; i < E; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      }
      // (the divisions of a lane group's E groups of channels, one by each of its first lanes)
      const int k = lane & (lanes - 1), u = k * n + me - k;
#pragma unroll
      for (int i = 0; i < E; ++i) all = k == i ? top[i] : all;
      if (k < E && u * UNIT < a.width) scales[u / lanes] = __fdiv_rn(all, 448.f);
    }
    const float fr = __fdiv_rn(448.f, all);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = at(i);
      const float f = a.group == 0 ? fr : __shfl_sync(0xffffffffu, fr, (lane & ~(a.group / UNIT - 1)) + i);
      if (c >= a.width) continue;
      uint32_t q[2];
      if (f < INFINITY) {  // (f is not NaN: NaN is left out of the maximum)
        const uint64_t f2 = pair_of(f, f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 u = of_pair(mul_pair(t[i][2 * h], f2)), v = of_pair(mul_pair(t[i][2 * h + 1], f2));
          q[h] = (uint32_t)f32x2_to_e4m3x2(u.x, u.y) | ((uint32_t)f32x2_to_e4m3x2(v.x, v.y) << 16);
        }
        if (odd || f == 0.f) {  // the NaN codes to 0 (what is finite saturates below them)
#pragma unroll
          for (int h = 0; h < 2; ++h) q[h] &= ~__vcmpeq4(q[h] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 u = of_pair(t[i][2 * h]), v = of_pair(t[i][2 * h + 1]);
          q[h] = zero_byte(u.x) | (zero_byte(u.y) << 8) | (zero_byte(v.x) << 16) | (zero_byte(v.y) << 24);
        }
      }
      uint8_t* p = a.codes + row * a.codes_stride + c;
      if (edge(c)) {
#pragma unroll
        for (int j = 0; j < UNIT; ++j)
          if (c + j >= 0 && c + j < a.width) p[j] = (uint8_t)(q[j / 4] >> (8 * (j & 3)));
      } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
      }
    }
    turn ^= 1;
    if (++stage == STAGES) stage = 0;
  }
}

constexpr size_t STREAM_SMEM = 220 * 1024;

template <typename T, bool ADD, bool SHIFT, int E, int THREADS>
cudaError_t launch_stream(const NormArgs& a, int units, cudaStream_t s) {
  const int threads = ((units + E - 1) / E + 31) / 32 * 32;
  const size_t smem = (size_t)STAGES * (ADD ? 2 : 1) * E * UNIT * sizeof(T) * threads;
  static std::atomic<int> memo[THREADS / 32][MAX_DEVICES];
  int per_sm = 0;
  const cudaError_t e = per_device(memo[threads / 32 - 1], [&](int* v) {
    auto kernel = norm_stream_kernel<T, ADD, SHIFT, E, THREADS>;
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)STREAM_SMEM);
    if (r != cudaSuccess) return r;
    int k = 0;
    r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, kernel, threads, smem);
    *v = k < 1 ? 1 : k;
    return r;
  }, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t cap = (int64_t)NUM_SMS * per_sm;
  norm_stream_kernel<T, ADD, SHIFT, E, THREADS><<<(unsigned)(a.n_rows < cap ? a.n_rows : cap), threads, smem, s>>>(a);
  return cudaGetLastError();
}

// Whether rows go to the kernel with a ring: many, of more units than a warp's.
template <typename T>
bool streams(const NormArgs& a, int units) {
  return units > 64 && a.n_rows > NUM_SMS && units <= (sizeof(T) == 2 ? 2048 : 1024);  // (two rows of twice 16384 values of 32 bits do not fit)
}
template <typename T, bool SHIFT>
cudaError_t launch_streams(const NormArgs& a, int units, cudaStream_t s) {
  const bool add = a.residual != nullptr;
  if (units <= 1024) {
    if (add) return launch_stream<T, true, SHIFT, 2, 512>(a, units, s);
    if constexpr (sizeof(T) == 4) return launch_stream<T, false, SHIFT, 2, 512>(a, units, s);
    else return launch_stream<T, false, SHIFT, 4, 256>(a, units, s);
  }
  if constexpr (sizeof(T) == 2)
    return add ? launch_stream<T, true, SHIFT, 4, 512>(a, units, s) : launch_stream<T, false, SHIFT, 4, 512>(a, units, s);
  return cudaErrorInvalidValue;  // (streams() lets none through)
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
  const int units = (a.width + UNIT - 1) / UNIT;
  if (vec) return streams<T>(a, units) ? launch_streams<T, false>(a, units, s) : launch_as<T, true>(a, s);
  // rows whose arrays begin equally far behind a multiple of a unit, each of them
  const uint64_t x_at = reinterpret_cast<uintptr_t>(a.x) / sizeof(T);
  auto alike = [&](const void* p, int size, int64_t stride) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) / size - x_at) % UNIT == 0 && (stride - a.x_stride) % UNIT == 0);
  };
  constexpr int SIZE = (int)sizeof(T);
  const int most = (a.width + 2 * UNIT - 2) / UNIT;  // units, with any shift
  if (streams<T>(a, most) && alike(a.residual, SIZE, a.residual_stride) && alike(a.residual_out, SIZE, a.residual_out_stride) &&
      alike(a.normed, SIZE, a.normed_stride) && alike(a.codes, 1, a.codes_stride) &&
      (a.group == 0 || (x_at % UNIT == 0 && a.x_stride % UNIT == 0)))
    return launch_streams<T, true>(a, most, s);
  return launch_as<T, false>(a, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t s) {
  if (dtype == KV8_BF16) return launch_typed<__nv_bfloat16>(a, s);
  if (dtype == KV8_F16) return launch_typed<__half>(a, s);
  return launch_typed<float>(a, s);
}

}  // namespace kv8
