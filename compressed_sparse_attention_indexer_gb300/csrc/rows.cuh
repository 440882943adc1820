// What the kernels that write rows of a layer's type or of E4M3 codes share:
// 16-byte vectors of either type, a block's scale, and the quotient by it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace csa {

constexpr float kE4m3Max = 448.f;

template <typename T>
struct VecOf;
template <>
struct VecOf<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(float v) { return v; }
};
template <>
struct VecOf<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* f) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ __nv_bfloat16 one(float v) { return __float2bfloat16_rn(v); }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The scale of a block whose largest magnitude is m.  The quotient is the
// rounded one: the product with 1 / 448, corrected by its residual (an infinite
// m stays).
__device__ __forceinline__ float block_scale(float m) {
  constexpr float kInv = 1.f / kE4m3Max;
  const float q = m * kInv;
  return m > 0.f ? fmaxf(m < INFINITY ? fmaf(fmaf(-q, kE4m3Max, m), kInv, q) : m, 1.17549435e-38f) : 1.f;
}
// f / scale to within a rounding that almost never differs from the exact
// one's: the product with the reciprocal, corrected by its residual (one step
// of Newton's iteration for the quotient).  Rows quantised as they are have
// many values next to a border of two codes' ranges, where a quotient that is
// off in the last place takes the other code.  An infinite scale leaves 0, and
// NaN for an infinite f.
template <int E>
__device__ __forceinline__ void divide(float* f, float scale) {
  const float inv = rcp_approx(scale), d = scale < INFINITY ? scale : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float q = f[e] * inv;
    f[e] = fmaf(fmaf(-q, d, f[e]), inv, q);
  }
}

}  // namespace csa
