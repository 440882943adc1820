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
//
// Measured (GB300): 16384 x 7168 bf16, residual, both outputs, in 166 us
// (6.4 TB/s, 94% of the measured copy rate); 131072 x 128 to codes in 11.8 us
// (4.3 TB/s: bound by instructions per row); 4097 x 1000 fp32 to codes in
// 6.3 us; one row of 4096 in 2.9 us (a launch).  Wide rows to codes without a
// residual are bound by each row's dependent chain, not by HBM: 10000 x 4096 bf16
// 32 us (3.8 TB/s), 80023 x 761 bf16 50 us, 24615 x 1497 fp32 53 us.
#include <cuda_fp8.h>

#include "csa_internal.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace csa {

namespace {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxVec = 8;      // 16-byte vectors per thread at most
constexpr int kNormBlock = 128;     // elements that share a scale
constexpr int kNormDepth = 2;       // rows of the shared-memory ring

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
__device__ __forceinline__ void store_codes(uint8_t* row, int v, int width, const float* f) {
  uint16_t c[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
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
// r / scale is up to 448 / max|s weight|, which for blocks below 1.3e-36 is no
// fp32 number.  So s weight is taken times kLift and r by 1 / kLift, both exactly:
// from max|s weight| = 2^-149 on 448 / (kLift max|s weight|) is one.  (A branch
// for such blocks costs registers: 40000 x 1000 bf16 36.0 us, this 33.0; the
// lift in the weight instead, 10000 x 4096 32.4, this 32.1.)
constexpr float kLift = 4294967296.f;   // 2^32
// What turns s weight into codes: r / scale, rounded (the product with the
// reciprocal, corrected by its residual; uncorrected it takes the other one of
// two neighbouring codes a fifth more often).
__device__ __forceinline__ float code_factor(float r, float scale) {
  const float inv = rcp_approx(scale), q = r * inv;
  return scale < INFINITY ? fmaf(fmaf(-q, scale, r), inv, q) : q;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void mul2(float* d, float b0, float b1) {
  uint64_t x = pack2(d[0], d[1]);
  const uint64_t y = pack2(b0, b1);
  asm("mul.rn.f32x2 %0, %0, %1;\n" : "+l"(x) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(d[0]), "=f"(d[1]) : "l"(x));
}

// tpr threads per row (a warp, or the whole block); blockDim.x / tpr rows per
// block and step, rows in a grid-stride loop.  A row's vectors are fetched
// while the rows before it are worked on: into registers, or (kRing) by
// cp.async into a ring of two rows in shared memory (four were no faster), where
// a thread reads back only what it copied itself (no barrier) and a short last vector is
// zero-filled by the copy.  The ring leaves registers to more vectors per
// thread and a tail costs nothing to load; register loads carry a
// streaming hint and do better where reads and writes are about equally
// many (see launch_t for both sides).
// Instructions bound it before bytes, so: the weight multiplies s before the
// norm is known and the norm's factor r > 0 goes into the scale
// (max|y| = r max|s weight|, code = s weight * (r / scale), see kLift), so that the
// blocks' maxima are found while the row's sum crosses the barrier.
template <typename T, int VPT, bool kTail, bool kRing>
__global__ void __launch_bounds__(kNormMaxThreads, VPT == 1 ? 2 : 1) norm_kernel(const NormArgs a, int tpr) {
  constexpr int E = VecOf<T>::E;
  // the next rows in flight and the weight held, where registers allow it
  constexpr bool kAhead = VPT <= 4;
  static_assert(kAhead || !kRing, "the ring is for rows of up to four vectors per thread");
  constexpr int kLanes = kNormBlock / E;  // lanes that share a scale
  extern __shared__ uint4 ring[];         // [slot][x, residual][vector][thread]
  __shared__ float part[2][32];
  const int t = threadIdx.x % tpr;
  const int rpb = blockDim.x / tpr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = a.width, vecs = (W + E - 1) / E;
  const float inv_width = 1.f / (float)W;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + threadIdx.x / tpr;
  const uint32_t vec_bytes = blockDim.x * 16, slot_bytes = (a.residual ? 2 : 1) * VPT * vec_bytes;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  uint32_t put = 0, get = 0;
  uint4 xr[kRing ? 1 : VPT], rr[kRing ? 1 : VPT], wr[kAhead ? VPT : 1];
  int64_t ahead = row;
  pdl_wait();
  pdl_trigger();
  auto fetch = [&]() {
    if (ahead < a.n) {
      const T* xp = static_cast<const T*>(a.x) + ahead * a.x_stride;
      const T* rp = a.residual ? static_cast<const T*>(a.residual) + ahead * a.residual_stride : nullptr;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        if (v >= vecs) continue;
        if constexpr (kRing) {
          const int bytes = kTail && (v + 1) * E > W ? (W - v * E) * (int)sizeof(T) : 16;
          const uint32_t at = mine + put + i * vec_bytes;
          cp_async16(at, xp + v * E, bytes);
          if (a.residual) cp_async16(at + VPT * vec_bytes, rp + v * E, bytes);
        } else {
          xr[i] = load_vec<kTail>(xp, v, W);
          if (a.residual) rr[i] = load_vec<kTail>(rp, v, W);
        }
      }
    }
    if constexpr (kRing) {
      cp_async_commit();
      put = put + slot_bytes == kNormDepth * slot_bytes ? 0 : put + slot_bytes;
    }
    ahead += step;
  };
  if constexpr (kRing) {
#pragma unroll
    for (int i = 0; i < kNormDepth - 1; ++i) fetch();
  } else if (kAhead) {
    fetch();
  }
  if (kAhead && a.weight) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tpr + t;
      if (v < vecs) wr[kAhead ? i : 0] = load_vec<kTail>(static_cast<const T*>(a.weight), v, W);
    }
  }
  int buf = 0;
  // every thread of the block runs the same number of steps (barrier inside)
  for (int64_t first = (int64_t)blockIdx.x * rpb; first < a.n; first += step, row += step) {
    const bool live = row < a.n;
    if (kRing || !kAhead) fetch();
    if constexpr (kRing) cp_async_wait<kNormDepth - 1>();
    float y[VPT][E];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * tpr + t;
      if (live && v < vecs) {
        const uint32_t at = mine + get + i * vec_bytes;
        VecOf<T>::unpack(kRing ? lds128(at) : xr[kRing ? 0 : i], y[i]);
        if (a.residual) {
          float r[E];
          VecOf<T>::unpack(kRing ? lds128(at + VPT * vec_bytes) : rr[kRing ? 0 : i], r);
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
    if constexpr (kRing) get = get + slot_bytes == kNormDepth * slot_bytes ? 0 : get + slot_bytes;
    else if (kAhead) fetch();
    if (a.residual) {
      T* sp = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        if (live && v < vecs) store_vec<kTail>(sp, v, W, y[i]);
      }
    }
    if (a.norm) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (tpr > 32 && lane == 0) part[buf][warp] = sum;
      if (a.weight) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int v = i * tpr + t;
          if (v < vecs) {
            float w[E];
            VecOf<T>::unpack(kAhead ? wr[kAhead ? i : 0] : load_vec<kTail>(static_cast<const T*>(a.weight), v, W), w);
#pragma unroll
            for (int e = 0; e < E; e += 2) mul2(y[i] + e, w[e], w[e + 1]);
          }
        }
      }
    }
    float top[VPT];  // NaN elements leave the maximum alone and become NaN codes
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        top[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) top[i] = fmaxf(top[i], fabsf(y[i][e]));
      }
#pragma unroll
      for (int o = kLanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < VPT; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    }
    float r = 1.f;
    if (a.norm) {
      if (tpr > 32) {
        __syncthreads();
        sum = lane < (int)(blockDim.x >> 5) ? part[buf][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        buf ^= 1;  // the next step's sums go elsewhere: one barrier per row is enough
      }
      r = rsqrtf(sum * inv_width + a.eps);
    }
    if (a.codes) {
      uint8_t* cp = a.codes + row * a.codes_stride;
      float* fp = a.scale + row * a.scale_stride;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        const float scale = block_scale(top[i] * r);
        if (live && v < vecs) {
          float z[E];
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = y[i][e];
          if (a.norm) {
            const float mul = code_factor(r * (1.f / kLift), scale);
#pragma unroll
            for (int e = 0; e < E; e += 2) mul2(z + e, kLift, kLift), mul2(z + e, mul, mul);
          } else {
            divide<E>(z, scale);
          }
          store_codes<kTail, E>(cp, v, W, z);
          if (t % kLanes == 0) fp[v / kLanes] = scale;
        }
      }
    }
    if (a.out) {
      T* op = static_cast<T*>(a.out) + row * a.out_stride;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * tpr + t;
        if (live && v < vecs) {
#pragma unroll
          for (int e = 0; e < E; e += 2) mul2(y[i] + e, r, r);
          store_vec<kTail>(op, v, W, y[i]);
        }
      }
    }
  }
}

// ---- rows of one block of codes (width <= 128: head rows, indexer keys) ----
// Sixteen (bf16) or 32 (fp32) lanes per row and kNarrowRows rows per thread,
// their chains interleaved: with a row per thread and step the kernel above
// spends 199 instructions per warp and step, most of them not on elements
// (131072 x 128 bf16 with codes: 15.5 us, this one 11.5 at the time, 11.8 now;
// two rows 13.0, one row 14.8).  Two elements per
// multiply (f32x2); both reductions run together.
constexpr int kNarrowRows = 4, kNarrowThreads = 256, kNarrowBlocks = 2;

template <typename T, bool kTail, bool kRes, bool kNorm>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowBlocks) norm_narrow_kernel(const NormArgs a) {
  constexpr int E = VecOf<T>::E, kLanes = kNormBlock / E, R = kNarrowRows;
  constexpr int kSide = kNarrowThreads / kLanes;       // rows side by side in a block
  const int t = threadIdx.x % kLanes, W = a.width;
  const bool mine = t * E < W;
  const float inv_width = 1.f / (float)W;
  pdl_wait();
  pdl_trigger();
  float w[E];
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = 1.f;
  if (kNorm && a.weight && mine) VecOf<T>::unpack(load_vec<kTail>(static_cast<const T*>(a.weight), t, W), w);
  const int64_t step = (int64_t)gridDim.x * (kSide * R);
  uint4 xr[R], rr[kRes ? R : 1];
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = at + j * kSide;
      xr[j] = make_uint4(0, 0, 0, 0);
      if (mine && row < a.n) {
        xr[j] = load_vec<kTail>(static_cast<const T*>(a.x) + row * a.x_stride, t, W);
        if constexpr (kRes) rr[j] = load_vec<kTail>(static_cast<const T*>(a.residual) + row * a.residual_stride, t, W);
      }
    }
  };
  int64_t block = (int64_t)blockIdx.x * (kSide * R);
  int64_t first = block + threadIdx.x / kLanes;
  fetch(first);
  for (; block < a.n; block += step, first += step) {  // the whole block runs the same steps
    float y[R][E], sum[R], top[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = first + j * kSide;
      VecOf<T>::unpack(xr[j], y[j]);
      if constexpr (kRes) {
        if (mine && row < a.n) {
          float r[E];
          VecOf<T>::unpack(rr[j], r);
#pragma unroll
          for (int e = 0; e < E; ++e) y[j][e] += r[e];
          store_vec<kTail>(static_cast<T*>(a.residual_out) + row * a.residual_out_stride, t, W, y[j]);
        }
      }
      if (j + 1 == R) fetch(first + step);
      sum[j] = 0.f;
      if (kNorm) {
#pragma unroll
        for (int e = 0; e < E; ++e) sum[j] = fmaf(y[j][e], y[j][e], sum[j]);
      }
      if (kNorm && a.weight) {
#pragma unroll
        for (int e = 0; e < E; e += 2) mul2(y[j] + e, w[e], w[e + 1]);
      }
      top[j] = 0.f;  // NaN elements leave the maximum alone and become NaN codes
#pragma unroll
      for (int e = 0; e < E; ++e) top[j] = fmaxf(top[j], fabsf(y[j][e]));
    }
#pragma unroll
    for (int o = kLanes >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (kNorm) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (a.codes) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t row = first + j * kSide;
      const float r = kNorm ? rsqrtf(sum[j] * inv_width + a.eps) : 1.f;
      if (!mine || row >= a.n) continue;
      if (a.codes) {
        const float scale = block_scale(top[j] * r);
        float z[E];
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = y[j][e];
        if (kNorm) {
          const float mul = code_factor(r * (1.f / kLift), scale);
#pragma unroll
          for (int e = 0; e < E; e += 2) mul2(z + e, kLift, kLift), mul2(z + e, mul, mul);
        } else {
          divide<E>(z, scale);
        }
        store_codes<kTail, E>(a.codes + row * a.codes_stride, t, W, z);
        if (t == 0) a.scale[row * a.scale_stride] = scale;
      }
      if (a.out) {
#pragma unroll
        for (int e = 0; e < E; e += 2) mul2(y[j] + e, r, r);
        store_vec<kTail>(static_cast<T*>(a.out) + row * a.out_stride, t, W, y[j]);
      }
    }
  }
}

template <typename T, bool kTail, bool kRes, bool kNorm>
int launch_narrow_kind(const NormArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  constexpr int kRowsPerBlock = kNarrowThreads / (kNormBlock / VecOf<T>::E) * kNarrowRows;
  int64_t blocks = ((int64_t)a.n + kRowsPerBlock - 1) / kRowsPerBlock;
  if (blocks > (int64_t)num_sms * kNarrowBlocks) blocks = (int64_t)num_sms * kNarrowBlocks;
  return launch_kernel(norm_narrow_kernel<T, kTail, kRes, kNorm>, dim3((unsigned)blocks), dim3(kNarrowThreads), 0, st, pdl, a);
}

template <typename T, bool kTail>
int launch_narrow(const NormArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  if (a.residual)
    return a.norm ? launch_narrow_kind<T, kTail, true, true>(a, num_sms, st, pdl)
                  : launch_narrow_kind<T, kTail, true, false>(a, num_sms, st, pdl);
  return a.norm ? launch_narrow_kind<T, kTail, false, true>(a, num_sms, st, pdl)
                : launch_narrow_kind<T, kTail, false, false>(a, num_sms, st, pdl);
}

// The grid is what fits the device at once (or the rows, when fewer): each
// block then walks its rows with the next one in flight.
template <typename T, int VPT, bool kTail, bool kRing>
int launch_kind(const NormArgs& a, int tpr, int threads, int num_sms, cudaStream_t st, bool pdl) {
  auto kern = norm_kernel<T, VPT, kTail, kRing>;
  const int depth = kRing ? kNormDepth : 0, res = a.residual ? 1 : 0;
  const size_t slot = (size_t)VPT * threads * 16 * (1 + res);
  if constexpr (kRing) {
    static PerDeviceOnce attr;
    if (const cudaError_t e = attr.run([&] { return allow_max_dynamic_smem(kern); }))
      return launch_fail("cudaFuncSetAttribute(norm_kernel)", e);
  }
  static std::atomic<int> per_sm[2][kNormMaxThreads / 32 + 1];  // resident blocks by block size (0: not asked yet)
  int r = per_sm[res][threads / 32].load(std::memory_order_relaxed);
  if (r == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, kern, threads, slot * depth);
    if (e != cudaSuccess) return launch_fail("cudaOccupancyMaxActiveBlocksPerMultiprocessor", e);
    if (r < 1) r = 1;
    per_sm[res][threads / 32].store(r, std::memory_order_relaxed);
  }
  const int64_t rpb = threads / tpr;
  int64_t blocks = (a.n + rpb - 1) / rpb;
  if (blocks > (int64_t)num_sms * r) blocks = (int64_t)num_sms * r;
  // no more slots than a block takes steps
  const int64_t steps = (a.n + blocks * rpb - 1) / (blocks * rpb);
  return launch_kernel(kern, dim3((unsigned)blocks), dim3(threads), slot * (size_t)(steps < depth ? steps : depth), st,
                       pdl, a, tpr);
}

template <typename T, int VPT>
int launch_vpt(const NormArgs& a, bool ring, int tpr, int threads, int num_sms, cudaStream_t st, bool pdl) {
  const bool tail = a.width % VecOf<T>::E != 0;
  if constexpr (VPT <= 4) {
    if (tail) return launch_kind<T, VPT, true, true>(a, tpr, threads, num_sms, st, pdl);
    if constexpr (sizeof(T) == 2) {
      if (!ring) return launch_kind<T, VPT, false, false>(a, tpr, threads, num_sms, st, pdl);
    }
    return launch_kind<T, VPT, false, true>(a, tpr, threads, num_sms, st, pdl);
  } else {
    return tail ? launch_kind<T, VPT, true, false>(a, tpr, threads, num_sms, st, pdl)
                : launch_kind<T, VPT, false, false>(a, tpr, threads, num_sms, st, pdl);
  }
}

template <typename T>
int launch_t(const NormArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  constexpr int E = VecOf<T>::E;
  const int vecs = (a.width + E - 1) / E;
  if (a.width <= kNormBlock)
    return a.width % E == 0 ? launch_narrow<T, false>(a, num_sms, st, pdl) : launch_narrow<T, true>(a, num_sms, st, pdl);
  // The ring, except for bf16 rows with a residual (1024 .. 4096 wide, both
  // outputs: 59 us from registers at 82 MB per tensor, 65 .. 67 from the ring;
  // without a residual codes take 31 us and not 38, out 28 and not 34; fp32
  // 1000 x 24615 with a residual to codes 55 and not 64; a tail from registers
  // 1.6 to 2.2 times as long).
  const bool ring = a.width % E != 0 || !a.residual || E == 4;
  auto threads_for = [&](int per) { return ((vecs + per - 1) / per + 31) / 32 * 32; };
  // Vectors per thread.  Ring: two to four, the count that leaves the fewest
  // threads idle (bf16 rows of 768: three 8.1 us, two 9.8 at 12000 rows); of
  // equals two (1497 fp32: 10.8 us with two, 12.0 with four at 4097 rows) but
  // four from 384 vectors on (bf16 4096: 37.5 and 41.5 us at 12000 rows).  One
  // row per SM or fewer: one, for the latency.
  // Registers: one where the block's size allows it, else four, so that several
  // rows share an SM (7168: 152 us with four, 176 with two at 19456 rows), or,
  // with fewer rows than SMs, as few as fit.
  int per = 1;
  if (vecs > 32) {
    if (ring && a.n >= num_sms && vecs <= 4 * kNormMaxThreads) {
      per = 2;
      for (int p = 3; p <= 4; ++p) {
        const int more = p * threads_for(p) - per * threads_for(per);
        if (more < 0 || (more == 0 && vecs > 384) || threads_for(per) > kNormMaxThreads) per = p;
      }
    } else {
      per = vecs <= kNormMaxThreads ? 1 : a.n >= num_sms ? 4 : 2;
    }
    while (threads_for(per) > kNormMaxThreads) ++per;
  }
  // a row per warp: several warps to a block (33 vectors, 4097 rows: 2.9 us with
  // four rows per block, 5.0 with one)
  const int tpr = threads_for(per), threads = vecs <= 32 ? 256 : tpr == 32 ? 128 : tpr, vpt = (vecs + tpr - 1) / tpr;
  switch (vpt) {
    case 1: return launch_vpt<T, 1>(a, ring, tpr, threads, num_sms, st, pdl);
    case 2: return launch_vpt<T, 2>(a, ring, tpr, threads, num_sms, st, pdl);
    case 3: return launch_vpt<T, 3>(a, ring, tpr, threads, num_sms, st, pdl);
    case 4: return launch_vpt<T, 4>(a, ring, tpr, threads, num_sms, st, pdl);
    case 5: return launch_vpt<T, 5>(a, ring, tpr, threads, num_sms, st, pdl);
    case 6: return launch_vpt<T, 6>(a, ring, tpr, threads, num_sms, st, pdl);
    case 7: return launch_vpt<T, 7>(a, ring, tpr, threads, num_sms, st, pdl);
    default: return launch_vpt<T, 8>(a, ring, tpr, threads, num_sms, st, pdl);
  }
}

}  // namespace

int norm_max_width(int dtype) { return kNormMaxThreads * kNormMaxVec * (dtype == CSA_DTYPE_BF16 ? 8 : 4); }

int launch_norm(const NormArgs& a, int dtype, int num_sms, cudaStream_t st, bool pdl) {
  return dtype == CSA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, num_sms, st, pdl)
                                 : launch_t<float>(a, num_sms, st, pdl);
}

}  // namespace csa
