// Row operator before an 8-bit product or an 8-bit cache: residual addition,
// root-mean-square norm and the output in the layer's type and / or as E4M3
// codes with one fp32 scale per 128 elements.
//   s = x + residual          residual_out = s rounded to the layer's type
//   y = s * rsqrt(mean(s^2) + eps) * weight      (norm = 0: y = s)
//   scale_j = max(max|y| / 448, 2^-126) over block j of 128 elements, 1 where
//   the block is all zero; code = y / scale_j to the nearest E4M3 value
// s and y stay in fp32 registers between the load and the stores, so y is
// rounded once, from the unrounded sum.
//
// Memory bound: every input byte is read once and every output byte written
// once.  A thread holds VPT 16-byte vectors of its row; consecutive threads
// hold consecutive vectors, so a block of 128 elements sits in 16 (bf16) or
// 32 (fp32) consecutive lanes and its maximum takes 4 or 5 shuffles.  The
// sum of squares needs the whole row: a row of up to one warp's threads is
// reduced by shuffles alone, a longer one by one barrier.  Every reduction
// has a fixed order.
#include <cuda_fp8.h>

#include "csa_internal.cuh"

namespace csa {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxVec = 8;      // 16-byte vectors per thread at most
constexpr int kNormBlock = 128;     // elements that share a scale

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

// Vector v of a row of `width` elements.  kTail: the row's last vector may be
// short; elements past the row then read as zero and are not written (the row
// may be the last of its buffer: nothing behind it is touched).
template <bool kTail, typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int v, int width) {
  constexpr int E = VecOf<T>::E;
  if (!kTail || (v + 1) * E <= width) return __ldcs(reinterpret_cast<const uint4*>(row) + v);
  T t[E];
#pragma unroll
  for (int i = 0; i < E; ++i) t[i] = v * E + i < width ? row[v * E + i] : T(0.f);
  uint4 r;
  memcpy(&r, t, 16);
  return r;
}
template <bool kTail, typename T>
__device__ __forceinline__ void store_vec(T* row, int v, int width, const float* f) {
  constexpr int E = VecOf<T>::E;
  if (!kTail || (v + 1) * E <= width) {
    reinterpret_cast<uint4*>(row)[v] = VecOf<T>::pack(f);
    return;
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (v * E + i < width) row[v * E + i] = VecOf<T>::one(f[i]);
}
// E codes of a row at vector v.
template <bool kTail, int E>
__device__ __forceinline__ void store_codes(uint8_t* row, int v, int width, const float* f, float mul) {
  uint16_t c[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * mul, f[2 * i + 1] * mul), __NV_SATFINITE, __NV_E4M3);
  if (!kTail || (v + 1) * E <= width) {
    if (E == 8)
      reinterpret_cast<uint2*>(row)[v] =
          make_uint2(c[0] | (uint32_t)c[1] << 16, c[E / 2 - 2] | (uint32_t)c[E / 2 - 1] << 16);
    else
      reinterpret_cast<uint32_t*>(row)[v] = c[0] | (uint32_t)c[1] << 16;
    return;
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (v * E + i < width) row[v * E + i] = (uint8_t)(c[i / 2] >> (8 * (i & 1)));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// tpr threads per row (a divisor of 32, or the whole block); blockDim.x / tpr
// rows per block and step, rows in a grid-stride loop.  The next row's
// vectors are loaded before the current row is reduced.
// Narrow rows are bound by instructions before bytes (131072 rows of 128: 239
// per warp and step took 17.2 us), so: the weight multiplies s before the norm
// is known and the norm's factor r > 0 goes into the scale
// (max|y| = r max|s weight|, code = s weight * (r / scale)), and row pointers
// advance by additions.
template <typename T, int VPT, bool kTail>
__global__ void __launch_bounds__(kNormMaxThreads, VPT <= 2 ? 2 : 1) norm_kernel(const NormArgs a, int tpr) {
  constexpr int E = VecOf<T>::E;
  // the next row in flight and the weight held, where registers allow it
  constexpr bool kAhead = VPT <= 4;
  constexpr int kLanes = kNormBlock / E;  // lanes that share a scale
  __shared__ float part[2][32];
  const int t = threadIdx.x % tpr;
  const int rpb = blockDim.x / tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = a.width, vecs = (W + E - 1) / E;
  const float inv_width = 1.f / (float)W;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  const T* xp = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* rp = static_cast<const T*>(a.residual) + (a.residual ? row * a.residual_stride : 0);
  T* sp = static_cast<T*>(a.residual_out) + (a.residual ? row * a.residual_out_stride : 0);
  T* op = static_cast<T*>(a.out) + (a.out ? row * a.out_stride : 0);
  uint8_t* cp = a.codes + (a.codes ? row * a.codes_stride : 0);
  float* fp = a.scale + (a.codes ? row * a.scale_stride : 0);
  pdl_wait();
  pdl_trigger();
  uint4 xr[VPT], rr[VPT], wr[VPT];
  auto fetch = [&](bool have) {
    if (!have) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tpr + t;
      if (v < vecs) {
        xr[i] = load_vec<kTail>(xp, v, W);
        if (a.residual) rr[i] = load_vec<kTail>(rp, v, W);
      }
    }
    xp += step * a.x_stride;
    if (a.residual) rp += step * a.residual_stride;
  };
  if (kAhead) fetch(row < a.n);
  if (kAhead && a.weight) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tpr + t;
      if (v < vecs) wr[i] = load_vec<kTail>(static_cast<const T*>(a.weight), v, W);
    }
  }
  int buf = 0;
  // every thread of the block runs the same number of steps (barrier inside)
  for (int64_t first = (int64_t)blockIdx.x * rpb; first < a.n; first += step, row += step) {
    const bool live = row < a.n;
    if (!kAhead) fetch(live);
    float y[VPT][E];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tpr + t;
      if (live && v < vecs) {
        VecOf<T>::unpack(xr[i], y[i]);
        if (a.residual) {
          float r[E];
          VecOf<T>::unpack(rr[i], r);
#pragma unroll
          for (int e = 0; e < E; ++e) y[i][e] += r[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(y[i][e], y[i][e], sum);
    }
    if (kAhead) fetch(row + step < a.n);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        if (live && v < vecs) store_vec<kTail>(sp, v, W, y[i]);
      }
      sp += step * a.residual_out_stride;
    }
    float r = 1.f;
    if (a.norm) {
      if (tpr < 32) {
        for (int o = tpr >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (tpr > 32) {
        if (lane == 0) part[buf][warp] = sum;
        __syncthreads();
        sum = lane < (int)(blockDim.x >> 5) ? part[buf][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        buf ^= 1;  // the next step's sums go elsewhere: one barrier per row is enough
      }
      r = rsqrtf(sum * inv_width + a.eps);
      if (a.weight) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = i * tpr + t;
          if (v < vecs) {
            float w[E];
            VecOf<T>::unpack(kAhead ? wr[i] : load_vec<kTail>(static_cast<const T*>(a.weight), v, W), w);
#pragma unroll
            for (int e = 0; e < E; ++e) y[i][e] *= w[e];
          }
        }
      }
    }
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        float m = 0.f;  // NaN elements leave the maximum alone and become NaN codes
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(y[i][e]));
#pragma unroll
        for (int o = kLanes >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m *= r;
        const float scale = m > 0.f ? fmaxf(m * (1.f / kE4m3Max), 1.17549435e-38f) : 1.f;
        if (live && v < vecs) {
          store_codes<kTail, E>(cp, v, W, y[i], r * rcp_approx(scale));
          if (t % kLanes == 0) fp[v / kLanes] = scale;
        }
      }
      cp += step * a.codes_stride;
      fp += step * a.scale_stride;
    }
    if (a.out) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        if (live && v < vecs) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[i][e] *= r;
          store_vec<kTail>(op, v, W, y[i]);
        }
      }
      op += step * a.out_stride;
    }
  }
}

// The grid is what fits the device at once (or the rows, when fewer): each
// block then walks its rows with the next one in flight.
template <typename T, int VPT, bool kTail>
int launch_kind(const NormArgs& a, int tpr, int threads, int num_sms, cudaStream_t st, bool pdl) {
  static std::atomic<int> per_sm[kNormMaxThreads / 32 + 1];  // resident blocks by block size (0: not asked yet)
  int r = per_sm[threads / 32].load(std::memory_order_relaxed);
  if (r == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, norm_kernel<T, VPT, kTail>, threads, 0);
    if (e != cudaSuccess) return launch_fail("cudaOccupancyMaxActiveBlocksPerMultiprocessor", e);
    if (r < 1) r = 1;
    per_sm[threads / 32].store(r, std::memory_order_relaxed);
  }
  const int64_t rpb = threads / tpr;
  int64_t blocks = (a.n + rpb - 1) / rpb;
  if (blocks > (int64_t)num_sms * r) blocks = (int64_t)num_sms * r;
  return launch_kernel(norm_kernel<T, VPT, kTail>, dim3((unsigned)blocks), dim3(threads), 0, st, pdl, a, tpr);
}

template <typename T, int VPT>
int launch_vpt(const NormArgs& a, int tpr, int threads, int num_sms, cudaStream_t st, bool pdl) {
  return a.width % VecOf<T>::E == 0 ? launch_kind<T, VPT, false>(a, tpr, threads, num_sms, st, pdl)
                                    : launch_kind<T, VPT, true>(a, tpr, threads, num_sms, st, pdl);
}

template <typename T>
int launch_t(const NormArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  constexpr int E = VecOf<T>::E;
  const int vecs = (a.width + E - 1) / E;
  int tpr, vpt, threads;
  if (vecs <= 32) {  // a row per half warp or warp
    tpr = vecs <= kNormBlock / E ? kNormBlock / E : 32;
    vpt = 1;
    threads = 256;
  } else {
    // as few vectors per thread as the block's size allows: the shortest chain
    // per row (4097 x 1000 fp32: 7.3 us with one, 7.7 with two, 11.2 with four;
    // 16384 x 7168: the same with two and four)
    int per = 1;
    while (((vecs + per - 1) / per + 31) / 32 * 32 > kNormMaxThreads) ++per;
    tpr = ((vecs + per - 1) / per + 31) / 32 * 32;
    vpt = (vecs + tpr - 1) / tpr;
    threads = tpr;
  }
  switch (vpt) {
    case 1: return launch_vpt<T, 1>(a, tpr, threads, num_sms, st, pdl);
    case 2: return launch_vpt<T, 2>(a, tpr, threads, num_sms, st, pdl);
    case 3: return launch_vpt<T, 3>(a, tpr, threads, num_sms, st, pdl);
    case 4: return launch_vpt<T, 4>(a, tpr, threads, num_sms, st, pdl);
    case 5: return launch_vpt<T, 5>(a, tpr, threads, num_sms, st, pdl);
    case 6: return launch_vpt<T, 6>(a, tpr, threads, num_sms, st, pdl);
    case 7: return launch_vpt<T, 7>(a, tpr, threads, num_sms, st, pdl);
    default: return launch_vpt<T, 8>(a, tpr, threads, num_sms, st, pdl);
  }
}

}  // namespace

int norm_max_width(int dtype) { return kNormMaxThreads * kNormMaxVec * (dtype == CSA_DTYPE_BF16 ? 8 : 4); }

int launch_norm(const NormArgs& a, int dtype, int num_sms, cudaStream_t st, bool pdl) {
  return dtype == CSA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, num_sms, st, pdl)
                                 : launch_t<float>(a, num_sms, st, pdl);
}

}  // namespace csa
