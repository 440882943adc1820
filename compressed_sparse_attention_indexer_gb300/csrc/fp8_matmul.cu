// Matrix product of E4M3 codes with a scale for each block of 128:
//   out[m][n] = sum_kb sa[m][kb] * sb[n / 128][kb] * sum_{k in block kb} a[m][k] * b[n][k]
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, fp32
// accumulators in TMEM): one 128-byte row of the 128-byte swizzle is one
// block of 128 codes, so a pipeline stage is one block and its product lands
// in a TMEM buffer of its own.  The scales are full fp32 numbers, so the
// outer sum cannot stay in the accumulator: the epilogue warps read every
// block's product back from TMEM and add it, times its scale, to fp32
// registers, while the MMAs of the next block fill another buffer.
//
//   warps 0, 2  copies: per block one TMA box of each operand into a ring, and
//               the block's scales into another (kSwap: both by warp 0)
//   warps 1, 3  TMEM allocation; one thread each issues four K = 32 MMAs per
//               block, the blocks in turn (kSwap: warp 1 alone)
//   the rest    epilogue: thread = TMEM lane (row of P), its columns of Q
//
// The operand in the TMEM lanes (P, 128 rows per tile) and the one in its
// columns (Q, NT rows per tile) are a and b, or with `kSwap` b and a: for a
// few rows of a (M <= 64) the weights then fill the 128 lanes and only as
// many columns as there are rows are computed, and the product is bound by
// streaming the weights.
// Cluster of `split` CTAs: each takes a part of the blocks of one tile, and
// the partial sums are added through distributed shared memory in rank order,
// so that few tiles still keep every SM loading; no workspace, no atomics.
// Every mbarrier wait is bounded; one that gives up sets bit 1 of the status.
//
// Measured (GB300): 8192 x 8192 x 7168 in 456 .. 464 us (2.1 PFLOP/s, 1785 MHz under
// the power cap), 1024 x 4096 x 4096 in 22.8 us, 64 x 36864 x 1536 in 14.1 us
// (4.4 TB/s), 331 x 1100 x 7000 in 10.3 us, 1 x 8192 x 1536 in 5.8 us.  What bounds
// large tiles: about 1030 cycles per block of 256 columns and 740 of 128, of which
// the MMAs take about 290 per 128 columns; the other 450 are not explained.  It is
// not the copies or the epilogue for the larger part: with one issuing thread 406 us
// in a burst, 385 without the TMEM reads, 405 without the copies, 371 without
// either.  CTA pairs (256 x 256 tiles, half the copies per SM) came to 470 us.
// Small products: launch, the first stage's latency (0.8 us) and the output's way
// out (1.2 us) beside the stream.
#include <cudaTypedefs.h>

#include "csa_internal.cuh"
#include "mm_pipeline.h"
#include "tc5.cuh"

namespace csa {

namespace {

// One test of a barrier's phase, whose answer is used later.
__device__ __forceinline__ uint32_t bar_ask(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok;
}
struct MmSmem {
  uint64_t full[kMmMaxStages];   // the block's codes are in shared memory
  uint64_t done[kMmMaxStages];   // the block's MMAs are done: the stage is free, its product is in TMEM
  uint64_t tempty[4];            // the TMEM buffer has been read
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The same shared-memory address in the cluster's CTA `rank`, and a load from it.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// One fp32 from global to shared memory (0 when !have), and an arrival on bar
// once the thread's copies so far have landed (counted in its arrivals).
__device__ __forceinline__ void copy_f32(uint32_t dst, const float* src, bool have) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// d += a * b on two packed fp32 values.
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}

// 16 or 32 columns of the warp's TMEM lanes, asked for and (tmem_arrive) waited
// for apart, so that the sums of one chunk run while the next is on its way.
template <int N>
__device__ __forceinline__ void tmem_ask(uint32_t taddr, uint32_t* r) {
  if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_arrive(uint32_t* r) {
  if constexpr (N == 32)
    tc5::tmem_wait_ld(r);
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

template <typename T>
__device__ __forceinline__ T to_out(float v);
template <>
__device__ __forceinline__ float to_out<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void sts_u4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// 32 rows (one per lane) x kLine bytes of output from registers to out: through
// the warp's patch (16-byte chunks swizzled by the row, so that neither the
// row-wise writes nor the line-wise reads conflict), then whole lines of
// several rows per warp store.  rows / cols: how many of the patch exist.
template <typename T, int kLine>
__device__ __forceinline__ void store_patch(uint32_t patch, const float* v, int lane, T* out, int64_t stride, int rows,
                                            int cols, bool vec) {
  constexpr int E = 16 / (int)sizeof(T), C = kLine / 16;
  auto at = [&](int r, int j) { return patch + r * kLine + ((j ^ ((C == 8 ? r : r >> 2) & (C - 1))) * 16); };
#pragma unroll
  for (int j = 0; j < C; ++j) {
    T t[E];
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = to_out<T>(v[j * E + e]);
    uint4 r;
    memcpy(&r, t, 16);
    sts_u4(at(lane, j), r);
  }
  __syncwarp();
  if (vec && cols >= C * E) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int r = i * (32 / C) + lane / C, j = lane % C;
      const uint4 x = lds_u4(at(r, j));
      if (r < rows) *reinterpret_cast<uint4*>(out + r * stride + j * E) = x;
    }
  } else {
    // rows off the 16-byte boundary, or fewer columns: neighbouring lanes store
    // neighbouring elements
    constexpr int kCols = C * E;
#pragma unroll 4
    for (int i = lane; i < 32 * kCols; i += 32) {
      const int r = i / kCols, c = i % kCols;
      const uint32_t src = at(r, c / E) + (c % E) * (uint32_t)sizeof(T);
      if (r < rows && c < cols) {
        if constexpr (sizeof(T) == 2) {
          uint16_t x;
          asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(x) : "r"(src) : "memory");
          *reinterpret_cast<uint16_t*>(out + r * stride + c) = x;
        } else {
          *reinterpret_cast<float*>(out + r * stride + c) = lds_f32(src);
        }
      }
    }
  }
  __syncwarp();
}

// This rank's share of a cluster's tile: the kSplit CTAs' sums of four
// neighbouring columns added in rank order and written to out.  Every load of
// a thread is asked for before the first is used.
template <typename Sh, typename T, int kSplit>
__device__ __forceinline__ void add_sums(uint32_t base, int rank, int rows, int64_t left, T* out, int64_t stride, bool vec) {
  constexpr int kQuads = Sh::kSumCols / 4;
  constexpr int kEach = (Sh::kSumRows * kQuads / kSplit + Sh::kThreads - 1) / Sh::kThreads;
  constexpr int kStep = kEach * kSplit <= 8 ? kEach : 8 / kSplit;   // pieces in flight per thread
  const int all = rows * kQuads, i0 = rank * all / kSplit, i1 = (rank + 1) * all / kSplit;
  uint32_t from[kSplit];
#pragma unroll
  for (int x = 0; x < kSplit; ++x) from[x] = kSplit > 1 ? cluster_addr(base, x) : base;
  for (int first = i0 + threadIdx.x; first < i1; first += kStep * Sh::kThreads) {
    float4 t[kStep][kSplit];
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      const int i = first + j * Sh::kThreads, r = i / kQuads, c = i % kQuads;
      if (i < i1) {
#pragma unroll
        for (int x = 0; x < kSplit; ++x) t[j][x] = ld_cluster_f4(from[x] + r * Sh::kPitch + c * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      const int i = first + j * Sh::kThreads, r = i / kQuads, n = (i % kQuads) * 4;
      if (i >= i1) continue;
      float v[4] = {t[j][0].x, t[j][0].y, t[j][0].z, t[j][0].w};
#pragma unroll
      for (int x = 1; x < kSplit; ++x) v[0] += t[j][x].x, v[1] += t[j][x].y, v[2] += t[j][x].z, v[3] += t[j][x].w;
      T* dst = out + r * stride + n;
      T o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = to_out<T>(v[e]);
      if (vec && n + 4 <= left) {
        if constexpr (sizeof(T) == 2) {
          uint2 x;
          memcpy(&x, o, 8);
          *reinterpret_cast<uint2*>(dst) = x;
        } else {
          uint4 x;
          memcpy(&x, o, 16);
          *reinterpret_cast<uint4*>(dst) = x;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < left) dst[e] = o[e];
      }
    }
  }
}

template <int NT, bool kSwap, typename T>
__global__ void __launch_bounds__(MmShape<NT, kSwap>::kThreads, MmShape<NT, kSwap>::kCtasPerSm)
    mm_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
              const MmArgs g, int split, int ptiles, int qtiles) {
  using Sh = MmShape<NT, kSwap>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ MmSmem sm;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t scales = base + Sh::kStages * Sh::kStageBytes + Sh::kPatchBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = (g.K + kMmBlock - 1) / kMmBlock;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int kb0 = (int)((int64_t)rank * KB / split), kb1 = (int)((int64_t)(rank + 1) * KB / split);
  const int tiles = ptiles * qtiles;
  const int first = blockIdx.x / split, step = gridDim.x / split;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      tc5::mbar_init(smem_u32(&sm.full[i]), 1 + 32);  // the bulk copies, the scales of 32 lanes
      tc5::mbar_init(smem_u32(&sm.done[i]), 1);
    }
    for (int i = 0; i < Sh::kBufs; ++i) tc5::mbar_init(smem_u32(&sm.tempty[i]), Sh::kEpiWarps);
    sm.abort = 0;
    tc5::fence_mbar_init();
    tc5::prefetch_tmap(&pmap);
    tc5::prefetch_tmap(&qmap);
  }
  // Before the allocation: a kernel in front that triggers its dependents
  // before it has its own TMEM must not find it taken by a CTA that waits for
  // that kernel's end.
  pdl_wait();
  if (warp == 1) {
    tc5::tmem_alloc(smem_u32(&sm.tmem_base), Sh::kTmemCols);
    tc5::tmem_relinquish();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  pdl_trigger();

  // tile t: its P and Q tile
  auto p_of = [&](int t) { return t % ptiles; };
  auto q_of = [&](int t) { return t / ptiles; };

  const bool codes_warp = warp == 0, scales_warp = warp == (kSwap ? 0 : 2);
  if (codes_warp || scales_warp) {
    // copies: the codes (lane 0, bulk) and the scales (every lane).  (Fetched by
    // the epilogue's threads instead, each row's line by every warp, the scales
    // took longer than the sums.)  Block n's scales go to slot n % kSlots: see
    // MmShape for what orders the slot's reads before its next copy.
    constexpr int kRows = kSwap ? (NT < 32 ? 32 : NT) : 128, kParts = kSwap ? 1 : NT / 128;
    int st = 0, slot = 0, n = 0;
    uint32_t ph = 0;
    for (int t = first; t < tiles && !*abort; t += step) {
      const int64_t m0 = kSwap ? (int64_t)q_of(t) * NT : (int64_t)p_of(t) * 128;
      const int64_t nb = kSwap ? p_of(t) : (int64_t)q_of(t) * NT / 128;
      const float* src[kRows / 32];
      bool have[kRows / 32];
#pragma unroll
      for (int i = 0; i < kRows / 32; ++i) {
        const int64_t m = m0 + i * 32 + lane;
        have[i] = m < g.M;
        src[i] = g.a_scale + (have[i] ? m * g.a_scale_stride : 0);
      }
      const bool have_b = lane < kParts && (nb + lane) * 128 < g.N;
      const float* src_b = g.b_scale + (have_b ? (nb + lane) * g.b_scale_stride : 0);
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        if (n >= Sh::kStages && !tc5::mbar_wait(smem_u32(&sm.done[st]), ph ^ 1u, abort)) goto loaded;
        const uint32_t bar = smem_u32(&sm.full[st]);
        if (codes_warp && lane == 0) {
          const uint32_t dst = base + st * Sh::kStageBytes;
          tc5::mbar_expect_tx(bar, Sh::kStageBytes);
          tc5::tma_load_2d(dst, &pmap, kb * kMmBlock, p_of(t) * 128, bar);
          tc5::tma_load_2d(dst + kMmPBytes, &qmap, kb * kMmBlock, q_of(t) * NT, bar);
        }
        __syncwarp();
        if (scales_warp) {
          const uint32_t dst = scales + slot * Sh::kScaleFloats * 4;
#pragma unroll
          for (int i = 0; i < kRows / 32; ++i) copy_f32(dst + (i * 32 + lane) * 4, src[i] + kb, have[i]);
          if (lane < kParts) copy_f32(dst + (128 + lane) * 4, src_b + kb, have_b);
          copies_arrive(bar);
        }
        if (++st == Sh::kStages) st = 0, ph ^= 1u;
        if (++slot == Sh::kSlots) slot = 0;
      }
    }
  loaded:
    // copies still in flight land before the block exits
    cp_async_commit();
    cp_async_wait<0>();
    if (codes_warp)
      for (int k = n > Sh::kStages ? n - Sh::kStages : 0; k < n; ++k)
        tc5::mbar_wait_drain(smem_u32(&sm.full[k % Sh::kStages]), (k / Sh::kStages) & 1);
  } else if (warp < Sh::kAux) {
    // MMA issuers, the blocks in turn: a block's chain in its thread (two
    // barriers, four MMAs, a commit: 700 cycles measured) is longer than its
    // MMAs (280 with 128 columns).  One issuer / two, when the second came:
    // 1024 x 4096 x 4096 26.9 / 23.9 us, 331 x 1100 x 7000 11.5 / 10.5.
    if (lane == 0) {
      constexpr int kBy = Sh::kIssuers;
      struct {
        MmSmem& sm;
        volatile int* abort;
        __device__ __forceinline__ bool wait_stage(int i, uint32_t parity) { return tc5::mbar_wait(smem_u32(&sm.full[i]), parity, abort); }
        __device__ __forceinline__ bool wait_buffer(int i, uint32_t parity) { return tc5::mbar_wait(smem_u32(&sm.tempty[i]), parity, abort); }
        __device__ __forceinline__ uint32_t ask_stage(int i, uint32_t parity) { return bar_ask(smem_u32(&sm.full[i]), parity); }
        __device__ __forceinline__ uint32_t ask_buffer(int i, uint32_t parity) { return bar_ask(smem_u32(&sm.tempty[i]), parity); }
      } bars{sm, abort};
      const int blocks = first < tiles ? ((tiles - 1 - first) / step + 1) * (kb1 - kb0) : 0;
      const uint32_t idesc = tc5::idesc_e4m3_f32(128, NT);
      MmIssue<Sh> is(kBy == 1 || warp == 1 ? 0 : 1);
      int last = -1;
      for (; is.n < blocks && !*abort;) {
        if (!is.ready(bars)) break;
        tc5::fence_after_sync();
        const uint64_t pd = tc5::sdesc_k_sw128(base + is.st * Sh::kStageBytes);
        const uint64_t qd = tc5::sdesc_k_sw128(base + is.st * Sh::kStageBytes + kMmPBytes);
        const uint32_t d = tmem + is.buf * Sh::kAccCols, now = smem_u32(&sm.done[is.st]);
        last = is.n;
        is.next();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tc5::mma_e4m3(d, pd + 2 * i, qd + 2 * i, idesc, i > 0);
          if (i == 1) is.ask(bars);  // asked here, the next block's barriers answer while the MMAs are issued
        }
        tc5::mma_commit(now);  // frees the stage and hands the product to the epilogue
      }
      // MMAs still in flight finish before TMEM is freed (this thread's complete in order)
      if (last >= 0) tc5::mbar_wait_drain(smem_u32(&sm.done[last % Sh::kStages]), (last / Sh::kStages) & 1);
    }
  } else {
    // a warp reads the TMEM lanes of its number mod 4
    const int ew = warp - Sh::kAux, quarter = warp & 3, group = ew >> 2;
    const int row = quarter * 32 + lane;                 // TMEM lane: row of the P tile
    const uint32_t tcol = tmem + ((uint32_t)(quarter * 32) << 16) + group * Sh::kCols;
    int buf = 0, st = 0, slot = 0;
    uint32_t ph = 0;
    for (int t = first; t < tiles && !*abort; t += step) {
      const int64_t p0 = (int64_t)p_of(t) * 128, q0 = (int64_t)q_of(t) * NT + group * Sh::kCols;
      uint64_t acc[Sh::kCols / 2];
#pragma unroll
      for (int i = 0; i < Sh::kCols / 2; ++i) acc[i] = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!tc5::mbar_wait(smem_u32(&sm.done[st]), ph, abort)) { ok = false; break; }
        const uint32_t sc = scales + slot * Sh::kScaleFloats * 4;
        tc5::fence_after_sync();
        constexpr int kChunk = Sh::kChunk, kParts = Sh::kCols / kChunk;
        const uint32_t t0 = tcol + buf * Sh::kAccCols;
        uint32_t v[2][kChunk];
        tmem_ask<kChunk>(t0, v[0]);
        // !kSwap: one factor per thread; kSwap: the b scale for all, the a
        // scales by column
        const float sb = lds_f32(sc + (128 + (kSwap ? 0 : group * Sh::kCols / 128)) * 4);
        const float f = kSwap ? sb : sb * lds_f32(sc + row * 4);
        const uint64_t f2 = pack2(f, f);
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          tmem_arrive<kChunk>(v[x & 1]);
          if (x + 1 < kParts) tmem_ask<kChunk>(t0 + (x + 1) * kChunk, v[(x + 1) & 1]);
          if (x + 1 == kParts) {  // the buffer is read: the next block's MMAs may have it
            tc5::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc5::mbar_arrive(smem_u32(&sm.tempty[buf]));
          }
#pragma unroll
          for (int i = 0; i < kChunk; i += 4) {
            const uint32_t* r = v[x & 1] + i;
            const int at = (x * kChunk + i) / 2;
            uint64_t s01 = f2, s23 = f2;
            if (kSwap) {
              const uint4 s = lds_u4(sc + (x * kChunk + i) * 4);
              s01 = pack2(__uint_as_float(s.x) * f, __uint_as_float(s.y) * f);
              s23 = pack2(__uint_as_float(s.z) * f, __uint_as_float(s.w) * f);
            }
            fma2(acc[at], pack2(__uint_as_float(r[0]), __uint_as_float(r[1])), s01);
            fma2(acc[at + 1], pack2(__uint_as_float(r[2]), __uint_as_float(r[3])), s23);
          }
        }
        if (++buf == Sh::kBufs) buf = 0;
        if (++slot == Sh::kSlots) slot = 0;
        if (++st == Sh::kStages) st = 0, ph ^= 1u;
      }
      if (!ok) break;
      float v[Sh::kCols];
#pragma unroll
      for (int i = 0; i < Sh::kCols / 2; ++i) unpack2(acc[i], v[2 * i], v[2 * i + 1]);
      if (kSwap || split > 1) {
        // into the ring, which every copy and MMA of this CTA's only tile has left
        if (kSwap) {
          const uint32_t at = base + row * 4;
#pragma unroll
          for (int i = 0; i < Sh::kCols; ++i)
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(at + i * Sh::kPitch), "f"(v[i]) : "memory");
        } else {
          const uint32_t at = base + row * Sh::kPitch + group * Sh::kCols * 4;
#pragma unroll
          for (int i = 0; i < Sh::kCols; i += 4)
            sts_u4(at + i * 4, make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                                          __float_as_uint(v[i + 3])));
        }
      } else {
        constexpr int kStep = Sh::kLine / (int)sizeof(T);   // columns per patch
        const uint32_t patch = base + Sh::kStages * Sh::kStageBytes + ew * 32 * Sh::kLine;
        const int64_t m0 = p0 + quarter * 32;
        const int rows = (int)(g.M - m0 < 32 ? g.M - m0 : 32);
#pragma unroll
        for (int c = 0; c < Sh::kCols; c += kStep) {
          const int64_t left = g.N - q0 - c;
          if (rows > 0 && left > 0)
            store_patch<T, Sh::kLine>(patch, v + c, lane, static_cast<T*>(g.out) + m0 * g.out_stride + q0 + c, g.out_stride, rows,
                           (int)(left < kStep ? left : kStep), g.vec);
        }
      }
    }
  }
  if (kSwap || split > 1) {
    // one tile per cluster: its sums, added over the ranks in order, leave in
    // pieces of four neighbouring columns, an equal share from each rank
    if (split > 1)
      cluster_sync();
    else
      __syncthreads();
    const int64_t p0 = (int64_t)p_of(first) * 128, q0 = (int64_t)q_of(first) * NT;
    const int64_t m0 = kSwap ? q0 : p0, n0 = kSwap ? p0 : q0;
    const int rows = (int)(g.M - m0 < Sh::kSumRows ? g.M - m0 : Sh::kSumRows);
    const int64_t left = g.N - n0;
    T* out = static_cast<T*>(g.out) + m0 * g.out_stride + n0;
    switch (split) {
      case 1: add_sums<Sh, T, 1>(base, rank, rows, left, out, g.out_stride, g.vec); break;
      case 2: add_sums<Sh, T, 2>(base, rank, rows, left, out, g.out_stride, g.vec); break;
      case 4: add_sums<Sh, T, 4>(base, rank, rows, left, out, g.out_stride, g.vec); break;
      default: add_sums<Sh, T, 8>(base, rank, rows, left, out, g.out_stride, g.vec); break;
    }
    if (split > 1) cluster_sync();  // no CTA leaves while another reads its sums
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (threadIdx.x == 0 && sm.abort && g.status) set_status(g.status, kStatusTimeout);
  if (warp == 1) tc5::tmem_dealloc(tmem, Sh::kTmemCols);
}

bool make_mm_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {stride};
  cuuint32_t box[2] = {(cuuint32_t)kMmBlock, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool kSwap, typename T>
int launch_shape(const MmArgs& g, int num_sms, cudaStream_t st, bool pdl) {
  using Sh = MmShape<NT, kSwap>;
  CUtensorMap pmap, qmap;
  const bool ok = kSwap ? make_mm_map(&pmap, g.b, g.N, g.K, g.b_stride, 128) &&
                              make_mm_map(&qmap, g.a, g.M, g.K, g.a_stride, NT)
                        : make_mm_map(&pmap, g.a, g.M, g.K, g.a_stride, 128) &&
                              make_mm_map(&qmap, g.b, g.N, g.K, g.b_stride, NT);
  if (!ok) return launch_fail("cuTensorMapEncodeTiled(a, b)", cudaSuccess);
  auto kern = mm_kernel<NT, kSwap, T>;
  static PerDeviceOnce attr;
  if (const cudaError_t e = attr.run([&] { return allow_max_dynamic_smem(kern); }))
    return launch_fail("cudaFuncSetAttribute(mm_kernel)", e);
  const int ptiles = (int)(((int64_t)(kSwap ? g.N : g.M) + 127) / 128), qtiles = (int)(((int64_t)(kSwap ? g.M : g.N) + NT - 1) / NT);
  const int64_t tiles = (int64_t)ptiles * qtiles;
  if (tiles > 0x7fffffff / 8) return launch_fail("too many tiles", cudaSuccess);
  const int slots = num_sms * Sh::kCtasPerSm;
  const int KB = (g.K + kMmBlock - 1) / kMmBlock;
  // a tile's blocks over the CTAs of a cluster while that still adds CTAs
  int split = 1;
  while (split < 8 && tiles * split * 2 <= slots && KB >= split * 2 * 2) split *= 2;
  // kSwap and split tiles leave through the ring's memory: one tile per cluster
  const int64_t grid = kSwap || split > 1 ? tiles * split : (tiles < slots ? tiles : slots);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int na = 0;
  if (pdl) {
    at[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (split > 1) {
    at[na].id = cudaLaunchAttributeClusterDimension;
    at[na].val.clusterDim.x = split;
    at[na].val.clusterDim.y = 1;
    at[na++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = na;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, pmap, qmap, g, split, ptiles, qtiles);
  return e == cudaSuccess ? 1 : launch_fail("cudaLaunchKernelEx", e);
}

template <typename T>
int launch_out(const MmArgs& g, int num_sms, cudaStream_t st, bool pdl) {
  if (g.M <= 16) return launch_shape<16, true, T>(g, num_sms, st, pdl);
  if (g.M <= 32) return launch_shape<32, true, T>(g, num_sms, st, pdl);
  if (g.M <= 64) return launch_shape<64, true, T>(g, num_sms, st, pdl);
  // Columns per tile, by the SMs' turns that the tiles come to and what a tile
  // takes: one of 128 columns 0.48 (few blocks, where the output bounds it) to
  // 0.6 (many) of one of 256.  Measured (256 / 128): 8192 x 8192 x 1024 93 / 88 us,
  // 5051 x 12681 x 1408 108 / 113, 2048 x 9728 x 4096 75 / 83, 2048 x 5120 x 4096
  // 57 / 53, 2048 x 2432 x 4096 38 / 24, 1100 x 4000 x 8000 36 / 42,
  // 128 x 20000 x 7168 35 / 44.  Where those of 128 fit in one turn they are
  // taken: 331 x 1100 x 7000 13.1 / 10.5.
  const int64_t rows = ((int64_t)g.M + 127) / 128;
  auto turns = [&](int64_t tiles) { return (tiles + num_sms - 1) / num_sms; };
  const int64_t blocks = (g.K + kMmBlock - 1) / kMmBlock;
  const int64_t narrow = turns(rows * (((int64_t)g.N + 127) / 128)), wide = turns(rows * (((int64_t)g.N + 255) / 256));
  return narrow > 1 && narrow * (240 + (blocks < 12 ? blocks : 12) + (blocks < 60 ? blocks : 60)) >= wide * 500
             ? launch_shape<256, false, T>(g, num_sms, st, pdl)
             : launch_shape<128, false, T>(g, num_sms, st, pdl);
}

}  // namespace

int launch_fp8_matmul(const MmArgs& g, int out_dtype, int num_sms, cudaStream_t st, bool pdl) {
  return out_dtype == CSA_DTYPE_BF16 ? launch_out<__nv_bfloat16>(g, num_sms, st, pdl)
                                     : launch_out<float>(g, num_sms, st, pdl);
}

}  // namespace csa
