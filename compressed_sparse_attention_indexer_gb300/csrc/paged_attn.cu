// Dense causal attention of the S newest tokens of each request over its
// whole cache: grouped heads, K and V rows in (paged) pools, bf16 or E4M3
// with a scale per row and head, optional sliding window.
//   pos = L - S + s;  rows max(0, pos - win + 1) .. pos (win = 0: 0 .. pos)
//   out[s][h] = sum_r softmax_r(scale q[s][h] . k[r]) v[r],  lse = ln sum_r exp(.)
// and the same of a tree of drafted tokens (kTree), each of which sees the rows
// before the drafts and those drafts that its bit mask names.
//
// HBM bound: a K / V row is read once and serves every query row of its group
// (S * heads / kv_heads, folded into the M = 16 rows of the warp MMA), so the
// arithmetic per byte stays far below the tensor rate and the kernel is a
// stream of row copies.
//
// Split of the work.  A unit is (request, kv head, chunk of 16 MT query
// rows); its cost is its number of tiles (128 or 256 rows) and one more for
// its start and end.  The units' tiles form one list, cut evenly by cost over
// the CTAs (one per SM), so that a ragged batch or a single long request fills
// the device alike; the lengths are read on the device, so a captured graph
// follows them.  Within a tile each warp owns 16
// or 32 rows: it copies them itself (16-byte cp.async into its own ring, several
// tiles ahead, across unit boundaries), and keeps its own running maximum,
// sum and output in registers: no barrier per tile.  At the end of a unit (or
// of the CTA's share) the warps' states are joined through shared memory; a
// unit cut between CTAs leaves fp32 partials (m, l, O) in the workspace, which
// a second kernel, launched ahead as a programmatic dependent, joins in CTA
// order.
//
// Scores, maxima, sums and O are fp32.  The weights are rounded to bf16 for
// the PV product (the operand type: at most 2^-8 relative each, unbiased);
// the sum l adds the unrounded ones, so lse is exact to fp32.  E4M3 codes are f16
// values, so those pools take f16 products (a bf16 operand would cost three
// more conversions per pair of codes: 765 instead of 548 us at the time for 32
// requests of 16384 .. 32768 rows): a query row is scaled by a power of two to at most 2
// (what then lies below 2^-14 is rounded to 2^-25 of the row's maximum), and the
// weights include the V rows' scales (small ones are rounded to 2^-32 of the largest,
// see kWeightTop).
// Rows outside a query's range never reach its output: they are not loaded,
// or their scores become -inf and, where another query of the same MMA sees
// them, a NaN or infinity among their V rows is masked out (v_products_apart).
//
// Measured (GB300): 64 requests of 1024 .. 65536 rows, 32 / 4 heads of 128, bf16,
// in 685 us (6.9 TB/s, the copy rate); 32 of 16384 .. 32768 rows,
// 64 / 8 heads, E4M3, in 315 us (5.2 TB/s; about 820 instructions
// per 32 rows of 256 bytes in three warps per scheduler, a long chain each: 43% of
// the issue slots, HBM neither); 48 x 4 tokens, 16 / 8 heads of 64, in
// 63 us (4.9 TB/s); one request of 1023 rows in 8.1 us (launch, two rounds of
// dependent loads, one tile, the join of the warps and of the CTAs); 32 of 4096 ..
// 16384 rows, 16 / 4 heads of 256, in 203 us (6.1 TB/s).  Far from their floors: a
// prompt (4096 tokens of 4096 rows, 32 / 8 heads: 1963 us against 73; every chunk of
// query rows streams all rows, windows or not) and many short units (64 tokens with a
// window of 128 rows: 20 us against 5).
#include "csa_internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace csa {

namespace {

constexpr float kRescaleAbove = 8.f;  // the reference maximum moves when exceeded by this (log2 units)
// E4M3: the reference is set this far below the maximum, so that the f16 weights use
// f16's range: up to 2^15, and off by at most 2^-25, 2^-32 of the largest, where they
// are small.  (At the maximum itself rows below 2^-25 of it would vanish from the
// output, however many, while the sum counts them.)
constexpr float kWeightTop = 7.f;
// E4M3: the softmax's sum has exponentials of its own in tiles with a V scale outside
// 2^-kNear .. 2^kNear, and after one above them, which may have raised the reference.
// What the joint exponentials lose elsewhere is below 2^-(126 - 2 kNear) of the
// largest term.
constexpr float kNear = 24.f;
// Exponents count V scales down to kMinScale, 2^-126.  Next to it a sum's terms, up to
// 2^15 / |v_scale|, pass fp32's range: from a term above 2^kFarTerm on a sum is kept 2^kFar
// smaller, as a negative number, until its reference is far enough up again.
constexpr float kMinScale = 1.1754944e-38f;
constexpr float kFarTerm = 104.f, kFar = 64.f, kFarBy = 18446744073709551616.f;

template <int D, int MT, bool kFp8>
struct PaShape {
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  // three warps per scheduler where registers allow it (64-dim heads: 71 us with
  // 8 warps, 67 with 12; E4M3: 353 and 333 us, its Q fragments then in shared
  // memory): the chain of a tile, QK to PV, is long and each warp does its own
  static constexpr int kWarps = D == 256 ? 4 : kRowBytes <= 128 && MT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  // rows a warp takes per tile: short rows take 32, so that the work per tile
  // (maxima, look-ups) is spread over as many bytes
  static constexpr int kPer = kRowBytes <= 128 ? 32 : 16;
  static constexpr int kGroups = kPer / 16;
  static constexpr int kTile = kPer * kWarps;                    // rows per tile
  static constexpr int kRows = 16 * MT;                          // query rows per unit
  static constexpr int kChunks = kRowBytes / 16;                 // 16-byte chunks per row
  static constexpr int kWarpStage = 2 * kPer * kRowBytes + (kFp8 ? 2 * kPer * 4 : 0);
  static constexpr int kScaleBytes = kFp8 ? kPer * 16 : 0;       // per warp: the tile's scales as used
  static constexpr bool kQReg = MT == 1 && D <= 128 && !kFp8;    // Q fragments in registers
  static constexpr int kQBytes = kQReg ? 0 : kRows * D * 2 + (kFp8 ? kRows * 4 : 0);
  static constexpr int kSlots = kWarps < 8 ? kWarps / 2 : kFp8 && MT == 1 ? 2 : 4;
  // a slot: 16 MT rows of fp32 dims.  bf16: 8 floats of padding per row let the
  // threads' 8-byte pieces of eight rows fall on different banks; E4M3 (16-byte
  // pieces, see e4m3_piece) needs none
  static constexpr int kPitch = D + (kFp8 ? 0 : 8);
  static constexpr int kSlotFloats = kRows * kPitch;
  static constexpr int kSlotBytes = kSlots * (kSlotFloats + 2 * kRows) * 4;
  static constexpr int kRoom = (226 * 1024 - kQBytes - kSlotBytes - kWarps * kScaleBytes) / (kWarps * kWarpStage);
  static constexpr int kStages = kRoom > 6 ? 6 : kRoom;
  static constexpr int kRing = kStages * kWarps * kWarpStage;
  static constexpr int kSmem = kRing + kQBytes + kSlotBytes + kWarps * kScaleBytes;
  static_assert(kStages >= 2, "no room for two stages");
  // the costs of a block's scan (a request per thread) add up in 32 bits
  static_assert((uint64_t)kThreads * (kPagedMaxLen / kTile + 2) <= std::numeric_limits<PaCost>::max(), "sum of costs");
};

// The same with results below 2^-126 kept.
__device__ __forceinline__ float tiny_exp2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// A softmax's sum l moved to a reference maximum d higher (d <= 0 is added to the
// exponents).  E4M3: a reference holds a row's V scale, so two of them may lie as far
// apart as the scales, and l, which does not, is as much larger: in two factors, of
// which neither vanishes.
__device__ __forceinline__ float move_sum(float l, float d) {
  const float f = fast_exp2(0.5f * d);
  return l * f * f;
}
// Sums that are 2^kFar smaller where they are negative (see kFar): moved, added, the factor
// that is left of one, its logarithm.
__device__ __forceinline__ float far_move(float l, float d) {
  const bool far = l < 0.f && (d < -kFar || l > -1.f);
  return move_sum(far ? -l : l, far ? d + kFar : d);
}
struct FarSum {
  float near = 0.f, far = 0.f;
  __device__ __forceinline__ void add(float l) {
    near += l < 0.f ? 0.f : l;   // (a NaN is passed on)
    far -= l < 0.f ? l : 0.f;
  }
  __device__ __forceinline__ float sum() const { return far > 0.f ? -(far + near * (1.f / kFarBy)) : near; }
};
__device__ __forceinline__ float far_add(float a, float b) {
  FarSum x;
  x.add(a);
  x.add(b);
  return x.sum();
}
__device__ __forceinline__ float far_rest(float l) { return l < 0.f ? 1.f / kFarBy : 1.f; }
__device__ __forceinline__ float far_log2(float l) { return log2f(fabsf(l)) + (l < 0.f ? kFar : 0.f); }
// D += A(16x16 f16, row) * B(16x8 f16, col), fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kFp8>
__device__ __forceinline__ void mma16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (kFp8)
    mma_f16_16816(d, a, b0, b1);
  else
    mma_bf16_16816(d, a, b0, b1);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The power of two in (max / 2, max], 1 for zero, subnormal and non-finite max.
__device__ __forceinline__ float pow2_below(float max) {
  const uint32_t e = __float_as_uint(max) >> 23;
  return e >= 1 && e <= 254 ? __uint_as_float(e << 23) : 1.f;
}
// Two bf16 times inv (a power of two) as f16x2.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t v, float inv) {
  return pack_f16x2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv);
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f4(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_u2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Where 16-byte chunk ch of a warp's row lies in the row's shared memory.
// bf16: the eight rows of an ldmatrix at one chunk fall on different banks.
// E4M3: the quad-wise 16-byte reads of K (two neighbouring rows, four chunks
// per phase) and of V (four even or odd rows, two chunks) do.
template <bool kFp8>
__device__ __forceinline__ int swizzle(int row, int ch) {
  return kFp8 ? ch ^ ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2)) : ch ^ (row & 7);
}

// Where piece x (dims 32 c + 4 x .. + 3) of row r lies in its slot row: the
// pieces of the four threads of a quad, and of neighbouring rows, fall on
// different banks.
__device__ __forceinline__ int e4m3_piece(int r, int c, int x) { return 32 * c + ((x ^ c ^ ((r & 1) << 2)) << 2); }

// The products of a warp's weights with its V rows in shared memory (at vt):
// pv(mt, x, j, b0, b1) for each 16-row group x and n-tile j, b0 / b1 the
// fragment of V.
template <int D, int MT, bool kFp8, typename F>
__device__ __forceinline__ void v_products(uint32_t vt, int lane, F&& pv) {
  using Sh = PaShape<D, MT, kFp8>;
  constexpr int kGroups = Sh::kGroups;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int x = 0; x < kGroups; ++x) {
    if constexpr (kFp8) {
      // n-tile j holds dims 16 n + j (n = 0..7): thread g takes codes 16 g .. 16 g + 15 of its four rows
      uint32_t w[4][4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int r = x * 16 + (z >> 1) * 8 + c * 2 + (z & 1);
        const uint4 v = lds_u4(vt + r * Sh::kRowBytes + swizzle<true>(r, g) * 16);
        w[z][0] = v.x; w[z][1] = v.y; w[z][2] = v.z; w[z][3] = v.w;
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int z = 0; z < 4; z += 2) {  // dims 16 g + 4 y + z, + 1: rows interleaved pair by pair
          const uint32_t sel = z ? 0x7362 : 0x5140;
          uint32_t a0, a1, b0, b1;
          e4m3x4_to_f16x2(__byte_perm(w[0][y], w[1][y], sel), a0, a1);
          e4m3x4_to_f16x2(__byte_perm(w[2][y], w[3][y], sel), b0, b1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            pv(mt, x, y * 4 + z, a0, b0);
            pv(mt, x, y * 4 + z + 1, a1, b1);
          }
        }
      }
    } else {
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) {
        const int r = x * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), ch = dt * 2 + (lane >> 4);
        uint32_t b0, b1, b2, b3;
        ldsm_x4_trans(vt + r * Sh::kRowBytes + swizzle<false>(r, ch) * 16, b0, b1, b2, b3);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          pv(mt, x, dt * 2, b0, b1);
          pv(mt, x, dt * 2 + 1, b2, b3);
        }
      }
    }
  }
}

// O += P V where a V row that some token of the warp's tile does not see holds
// a NaN or an infinity: a pass per token that the product's query rows may
// be of (sq, ascending; S: no query row) with its own rows kept and its own query rows taken.
// Out of line, on copies of o and pf: rare, and the common path keeps its registers.
template <int D, int MT, bool kFp8, bool kTree>
__device__ __noinline__ void v_products_apart(float* o, const uint32_t* pf, const int* sq, uint32_t vt, int lane, int base,
                                              int p_first, int S, int win, const PagedArgs& a, int b) {
  using Sh = PaShape<D, MT, kFp8>;
  const int c = lane & 3;
  int t = __shfl_sync(0xffffffffu, sq[0], 0);
  if (S > t + 16 * MT) S = t + 16 * MT;
  for (; t < S; ++t) {
    const int last = p_first + t, out = kTree ? tree_outside(a, b, t, p_first, S) : 0;
    uint32_t keep[2 * Sh::kGroups];
#pragma unroll
    for (int n = 0; n < 2 * Sh::kGroups; ++n) {
      keep[n] = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = base + n * 8 + c * 2 + e;
        const bool sees = kTree ? (r < p_first ? r > out : r < p_first + S && tree_sees(a, b, t, r - p_first))
                                : r <= last && (win == 0 || r > last - win);
        if (sees) keep[n] |= e ? 0xffff0000u : 0xffffu;
      }
    }
    v_products<D, MT, kFp8>(vt, lane, [&](int mt, int x, int j, uint32_t b0, uint32_t b1) {
      float* d = o + (mt * (D / 8) + j) * 4;
      float y[4] = {d[0], d[1], d[2], d[3]};
      mma16<kFp8>(y, pf + (mt * Sh::kGroups + x) * 4, b0 & keep[2 * x], b1 & keep[2 * x + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sq[mt * 2 + (i >> 1)] == t) d[i] = y[i];
    });
  }
}

template <int D, int MT, bool kFp8, bool kTree>
__global__ void __launch_bounds__(PaShape<D, MT, kFp8>::kThreads, 1)
    paged_attn_kernel(const PagedArgs a, int chunks, int units, float* __restrict__ part, PaJoin* __restrict__ joins) {
  using Sh = PaShape<D, MT, kFp8>;
  constexpr int kTile = Sh::kTile, kPer = Sh::kPer, kGroups = Sh::kGroups;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ PaCost scan_tmp[33];
  __shared__ Cut cut_sh[2];
  // thread 0's alone, kept out of everyone's registers: the list's cost, and the
  // current unit's place in it
  __shared__ int64_t total_sh, unit_at;
  // E4M3, a warp's: its piece has had a V scale above 2^kNear (in a register: 388 us
  // instead of 320 for 32 requests of 16384 .. 32768 rows, spills) or a sum below zero
  __shared__ volatile int high_sh[Sh::kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem_raw) + warp * (Sh::kStages * Sh::kWarpStage);
  const uint32_t qsm = smem_u32(smem_raw) + Sh::kRing;
  float* slots = reinterpret_cast<float*>(smem_raw + Sh::kRing + Sh::kQBytes);
  const uint32_t rowsc = smem_u32(smem_raw) + Sh::kRing + Sh::kQBytes + Sh::kSlotBytes + warp * Sh::kScaleBytes;
  const int group = a.heads / a.kv_heads;
  const float per_group = 1.f / (float)group;
  // i / group for 0 <= i < S * heads <= 2^20 (off by less than half of 1 / group)
  auto token_of = [&](int i) { return (int)(((float)i + 0.5f) * per_group); };
  const int qrows = a.S * group;                    // query rows per kv head
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share of the list: of the costs (a unit's tiles and one
  // more for its start and end), with the cuts moved to the next whole tile
  int64_t total, G;
  if (!paged_cuts<kTile, kTree, Sh::kThreads, 1>(a, units, scan_tmp, cut_sh, total, G)) {
    if (tid == 0) joins[blockIdx.x].count = 0;
    return;
  }
  const int steps = (int)(cut_sh[1].at - cut_sh[0].at);
  if (steps == 0) {
    if (tid == 0) joins[blockIdx.x].count = 0;
    return;
  }
  Cursor<kTile, kTree> ld;  // the loader's position, several tiles ahead of the products
  ld.b = cut_sh[0].b;
  ld.sp.set(a, ld.b);
  ld.unit = cut_sh[0].unit;
  ld.tile = cut_sh[0].tile;
  if (tid == 0) total_sh = total, unit_at = cut_sh[0].first;
  Cursor<kTile, kTree> cu = ld;
  int loaded = 0;

  // ---- row copies: lane r < kPer looks up the pool row of the warp's row r one
  // tile ahead of the copies that use it.  A table's entry stays as it was
  // loaded until then, so that nothing waits for it earlier (E4M3: 329 us to 311).
  int entry = -1, within = 0;
  auto lookup = [&](const Cursor<kTile, kTree>& c) {
    const int r = (c.sp.t0 + c.tile) * kTile + warp * kPer + lane;
    within = -1;                                   // nothing to read
    if (lane < kPer && r >= c.sp.lo && r < c.sp.L) {
      if (a.table) {
        const int k = (int)((uint32_t)r / (uint32_t)a.block);
        within = r - k * a.block;
        entry = -1;
        if (k < a.table_stride) entry = a.table[(int64_t)c.b * a.table_stride + k];
      } else {
        const int64_t x = a.off[c.b] + r;
        within = 0;
        entry = x >= 0 && x < a.rows ? (int)x : -1;
      }
    }
  };
  int prow = -1;                                   // the pool row (-1: nothing to read)
  auto resolve = [&] {
    prow = -1;
    if (within >= 0) {
      const int64_t x = entry < 0 ? -1 : a.table ? (int64_t)entry * a.block + within : entry;
      if (x >= 0 && x < a.rows) prow = (int)x;
      else if (a.status) set_status(a.status, kStatusBadIndex);
    }
  };
  auto copy = [&](int stage) {
    const uint32_t kdst = ring + stage * Sh::kWarpStage, vdst = kdst + kPer * Sh::kRowBytes;
    const int h = chunks == 1 ? ld.unit : ld.unit / chunks;
    constexpr int kSpan = Sh::kChunks > 32 ? 32 : Sh::kChunks;           // lanes per row and copy
    constexpr int kAtOnce = 32 / kSpan;                                  // rows per warp-wide copy
    const int ch = lane % kSpan, r0 = lane / kSpan;
    const uint8_t* kb = static_cast<const uint8_t*>(a.k) + (h * Sh::kRowBytes + ch * 16);
    const uint8_t* vb = static_cast<const uint8_t*>(a.v) + (h * Sh::kRowBytes + ch * 16);
#pragma unroll
    for (int i = 0; i < kPer / kAtOnce; ++i) {
      const int row = i * kAtOnce + r0;
      const int p = __shfl_sync(0xffffffffu, prow, row);
      const uint32_t x = p < 0 ? 0u : (uint32_t)p, at = row * Sh::kRowBytes + swizzle<kFp8>(row, ch) * 16;
      const int bytes = p < 0 ? 0 : 16;
      cp_async16(kdst + at, kb + (uint64_t)x * (uint32_t)a.k_step, bytes);
      cp_async16(vdst + at, vb + (uint64_t)x * (uint32_t)a.v_step, bytes);
    }
    if (kFp8 && lane < kPer) {  // the rows' K scales, then their V scales
      const int64_t at = (int64_t)(prow < 0 ? 0 : prow) * a.scale_stride + h;
      const uint32_t dst = kdst + 2 * kPer * Sh::kRowBytes + lane * 4;
      cp_async4(dst, a.k_scale + at, prow < 0 ? 0 : 4);
      cp_async4(dst + kPer * 4, a.v_scale + at, prow < 0 ? 0 : 4);
    }
  };
  auto load_step = [&] {
    if (loaded < steps) {
      if (ld.sp.L > 0) {
        resolve();
        copy(loaded % Sh::kStages);
      }
      ++loaded;
      if (loaded < steps) {
        ld.next(a, units);
        lookup(ld);
      }
    }
    cp_async_commit();
  };
  lookup(ld);
#pragma unroll
  for (int i = 0; i < Sh::kStages - 1; ++i) load_step();

  // ---- per-unit state
  const int g = lane >> 2, c = lane & 3;
  uint32_t qf[Sh::kQReg ? D / 16 : 1][4];
  float qmul[MT][2];                               // E4M3: the power of two taken out of the thread's query rows
  float o[MT][D / 8][4], m[MT][2], l[MT][2];
  int seg_first = 0;                               // step at which the current piece starts
  const float scale2 = a.scale * kLog2e;

  for (int step = 0; step < steps; ++step) {
    const int h = chunks == 1 ? cu.unit : cu.unit / chunks, row0 = (cu.unit - h * chunks) * Sh::kRows;
    if (cu.sp.L <= 0) {  // a padding request: nothing to read, nothing to join
      load_step();
      for (int x = tid; x < Sh::kRows * (D / 8); x += Sh::kThreads) {
        const int i = row0 + x / (D / 8);
        if (i < qrows) {
          const int s = token_of(i), hd = h * group + i - s * group;
          const int64_t tok = (int64_t)cu.b * a.S + s;
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + tok * a.out_stride + hd * D + x % (D / 8) * 8) =
              make_uint4(0, 0, 0, 0);
          if (a.lse && x % (D / 8) == 0) a.lse[tok * a.heads + hd] = -INFINITY;
        }
      }
      if (tid == 0 && step + 1 == steps) joins[blockIdx.x].count = 0;
      if (tid == 0) unit_at += cu.sp.tiles + 1;
      cu.next(a, units);
      seg_first = step + 1;
      continue;
    }
    if (step == seg_first) {
      if (kFp8 && lane == 0) high_sh[warp] = 0;
      const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)cu.b * a.S * a.q_stride;
      auto q_at = [&](int i) {  // query row i of the unit's kv head: token i / group, head h * group + i % group
        const int s = token_of(i);
        return q0 + (int64_t)s * a.q_stride + (h * group + i - s * group) * D;
      };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[mt][e] = -INFINITY;
          l[mt][e] = 0.f;
        }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
      if constexpr (Sh::kQReg) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = row0 + g + 8 * e;
          const bool in = i < qrows;
          const __nv_bfloat16* q = q_at(in ? i : 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[ks][e] = in ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + c * 2) : 0;
            qf[ks][2 + e] = in ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + c * 2) : 0;
          }
        }
      } else {
        for (int x = tid; x < Sh::kRows * (D / 8); x += Sh::kThreads) {
          const int r = x / (D / 8), ch = x % (D / 8);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (row0 + r < qrows) v = *reinterpret_cast<const uint4*>(q_at(row0 + r) + ch * 8);
          if constexpr (kFp8) {  // D = 128: a row is 16 neighbouring lanes
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
            for (int i = 8; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            const float two = pow2_below(top);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = bf16x2_to_f16x2(w[i], 1.f / two);
            if (ch == 0) *reinterpret_cast<float*>(smem_raw + Sh::kRing + Sh::kRows * D * 2 + r * 4) = two;
          }
          *reinterpret_cast<uint4*>(smem_raw + Sh::kRing + r * D * 2 + ((ch ^ (r & 7)) * 16)) = v;
        }
        __syncthreads();
        if constexpr (kFp8) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) qmul[mt][e] = lds_f32(qsm + Sh::kRows * D * 2 + (mt * 16 + g + 8 * e) * 4);
        }
      }
    }
    load_step();
    cp_async_wait<Sh::kStages - 1>();
    __syncwarp();
    const uint32_t kt = ring + (step % Sh::kStages) * Sh::kWarpStage, vt = kt + kPer * Sh::kRowBytes;
    const int base = (cu.sp.t0 + cu.tile) * kTile + warp * kPer;   // first of the warp's rows
    if (base < cu.sp.L && base + kPer - 1 >= cu.sp.lo) {
      bool wide = false;
      if constexpr (kFp8) {
        // lane r: its row's scales as the scores and weights use them.  The
        // weight of a V row is p |v_scale|, so v_scale goes into the exponent
        // (lv) and the maximum is taken over both: the f16 weights then keep
        // their precision whatever the scales.  The softmax's own sum takes
        // the factor out again (1 / |v_scale|), or, where the weight may vanish
        // while its part of the sum does not (`wide`: see kNear), has an
        // exponential of its own.  |v_scale| below kMinScale (zero) counts as kMinScale, the
        // rest of it is kept in the sign factor.
        const uint32_t src = kt + 2 * kPer * Sh::kRowBytes + (lane % kPer) * 4;
        const float ks = lds_f32(src) * scale2, vs = lds_f32(src + kPer * 4);
        const float lv = fast_log2(fmaxf(fabsf(vs), kMinScale)), inv = fast_exp2(-lv);
        // a v_scale that is no number reaches whoever sees the row by its exponent alone
        if (fabsf(vs) < INFINITY)
          sts_f4(rowsc + (lane % kPer) * 16, ks, lv, inv, vs * inv);
        else
          sts_f4(rowsc + (lane % kPer) * 16, ks, __uint_as_float(0x7fffffffu), 1.f, 1.f);
        wide = __any_sync(0xffffffffu, !(fabsf(lv) <= kNear) || high_sh[warp] != 0);
        if (lv > kNear) high_sh[warp] = 1;   // for the tiles to come
        __syncwarp();
      }
      // ---- S = Q K^T: 16 MT query rows x kPer rows (n = 8 tiles)
      float s[MT][2 * kGroups][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int n = 0; n < 2 * kGroups; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
      auto q_frag = [&](int mt, int ks, uint32_t* f) {
        if constexpr (Sh::kQReg) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = qf[ks][i];
        } else if constexpr (kFp8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = mt * 16 + g + 8 * e, ch = (ks / 4) * 8 + c * 2 + ((ks % 4) >> 1);
            const uint2 v = lds_u2(qsm + r * D * 2 + ((ch ^ (r & 7)) * 16) + (ks & 1) * 8);
            f[e] = v.x;
            f[2 + e] = v.y;
          }
        } else {
          const int r = mt * 16 + (lane & 15), ch = ks * 2 + (lane >> 4);
          ldsm_x4(qsm + r * D * 2 + ((ch ^ (r & 7)) * 16), f[0], f[1], f[2], f[3]);
        }
      };
      if constexpr (kFp8) {
        // The order of the products over d is free: thread c of a quad takes
        // 16 consecutive codes of its row per 64 dims, four per K = 16 step
        // (q's fragments above take the same dims).
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t w[2 * kGroups][4];
#pragma unroll
          for (int n = 0; n < 2 * kGroups; ++n) {
            const int r = n * 8 + g;
            const uint4 v = lds_u4(kt + r * Sh::kRowBytes + swizzle<true>(r, j * 4 + c) * 16);
            w[n][0] = v.x; w[n][1] = v.y; w[n][2] = v.z; w[n][3] = v.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t f[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) q_frag(mt, j * 4 + i, f[mt]);
#pragma unroll
            for (int n = 0; n < 2 * kGroups; ++n) {
              uint32_t b0, b1;
              e4m3x4_to_f16x2(w[n][i], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16<true>(s[mt][n], f[mt], b0, b1);
            }
          }
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) q_frag(mt, ks, f[mt]);
#pragma unroll
          for (int x = 0; x < kGroups; ++x) {
            const int r = x * 16 + ((lane >> 4) << 3) + (lane & 7), ch = ks * 2 + ((lane >> 3) & 1);
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kt + r * Sh::kRowBytes + swizzle<false>(r, ch) * 16, b0, b1, b2, b3);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16<false>(s[mt][2 * x], f[mt], b0, b1);
              mma16<false>(s[mt][2 * x + 1], f[mt], b2, b3);
            }
          }
        }
      }
      // ---- scores in log2 units; rows outside a query's range weigh nothing
      const int p_first = cu.sp.L - (kTree ? cu.sp.n : a.S);   // the first token's position
      const bool edge = base < cu.sp.lo || base + kPer - 1 > p_first - (kTree ? 1 : 0) ||
                        (a.win > 0 && base < cu.sp.L - a.win);  // some query does not see all the rows
      uint32_t pf[MT][kGroups][4];
#pragma unroll
      for (int n = 0; n < 2 * kGroups; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ks = scale2, lv = 0.f;
          if constexpr (kFp8) {
            const float2 t = lds_f2(rowsc + (n * 8 + c * 2 + e) * 16);
            ks = t.x, lv = t.y;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float x = s[mt][n][2 * y + e];
              s[mt][n][2 * y + e] = kFp8 ? fmaf(x, ks * qmul[mt][y], lv) : x * ks;
            }
        }
      if (edge) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          int pos[2];                              // last visible row of the thread's query rows
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = row0 + mt * 16 + g + 8 * e;
            pos[e] = i < qrows ? p_first + token_of(i) : -1;
          }
          if constexpr (kTree) {
            int token[2], out[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = row0 + mt * 16 + g + 8 * e;
              token[e] = i < qrows ? token_of(i) : cu.sp.n;
              out[e] = token[e] < cu.sp.n ? tree_outside(a, cu.b, token[e], p_first, cu.sp.n) : cu.sp.L;
            }
#pragma unroll
            for (int n = 0; n < 2 * kGroups; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = base + n * 8 + c * 2 + (i & 1), s1 = token[i >> 1];
                const bool sees = r < p_first ? r > out[i >> 1]
                                              : r < cu.sp.L && s1 < cu.sp.n && tree_sees(a, cu.b, s1, r - p_first);
                if (!sees) s[mt][n][i] = -INFINITY;
              }
            continue;
          }
#pragma unroll
          for (int n = 0; n < 2 * kGroups; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = base + n * 8 + c * 2 + (i & 1), last = pos[i >> 1];
              if (r > last || (a.win > 0 && r <= last - a.win)) s[mt][n][i] = -INFINITY;
            }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]);
#pragma unroll
          for (int n = 1; n < 2 * kGroups; ++n) t = fmaxf(t, fmaxf(s[mt][n][2 * e], s[mt][n][2 * e + 1]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          top[e] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        }
        // how far the maximum may be above the reference, and where a new reference is
        constexpr float kAbove = kRescaleAbove + (kFp8 ? kWeightTop : 0.f), kBelow = kFp8 ? kWeightTop : 0.f;
        const bool grow = top[0] > m[mt][0] + kAbove || top[1] > m[mt][1] + kAbove;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (top[e] > m[mt][e] + kAbove) {
              const float to = top[e] - kBelow, f = fast_exp2(m[mt][e] - to);
              l[mt][e] = kFp8 ? far_move(l[mt][e], m[mt][e] - to) : l[mt][e] * f;
              m[mt][e] = to;
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                o[mt][j][2 * e] *= f;
                o[mt][j][2 * e + 1] *= f;
              }
            }
          }
        }
        if (kFp8 && wide) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float ref = m[mt][y] == -INFINITY ? 0.f : m[mt][y];
            float e[4 * kGroups], most = -INFINITY, sum = l[mt][y];
#pragma unroll
            for (int x = 0; x < 4 * kGroups; ++x) {
              const float lv = lds_f32(rowsc + ((x >> 1) * 8 + c * 2 + (x & 1)) * 16 + 4), t = s[mt][x >> 1][2 * y + (x & 1)];
              e[x] = t == -INFINITY ? t : t - lv - ref;
              most = fmaxf(most, e[x]);
            }
            if (most > kFarTerm && !(sum < 0.f)) {   // (see kFar; a NaN stays)
              sum *= 1.f / kFarBy;
              sum = sum < kMinScale ? -kMinScale : -sum;
            }
            const float off = sum < 0.f ? kFar : 0.f;
            if (off > 0.f) high_sh[warp] = 1;
            float to = fabsf(sum);
#pragma unroll
            for (int x = 0; x < 4 * kGroups; ++x) to += tiny_exp2(e[x] - off);
            l[mt][y] = off > 0.f ? -to : to;
          }
        }
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          float p[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float2 t = make_float2(1.f, 1.f);                 // E4M3: 1 / |v_scale| and its sign
              if constexpr (kFp8) t = lds_f2(rowsc + ((2 * x + n) * 8 + c * 2 + e) * 16 + 8);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float ref = m[mt][y] == -INFINITY ? 0.f : m[mt][y];
                const float w = fast_exp2(s[mt][2 * x + n][2 * y + e] - ref);
                if (!kFp8) l[mt][y] += w;
                else if (!wide) l[mt][y] += w * t.x;
                p[n][2 * y + e] = kFp8 ? w * t.y : w;
              }
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x0 = p[i >> 1][(i & 1) * 2], x1 = p[i >> 1][(i & 1) * 2 + 1];
            pf[mt][x][i] = kFp8 ? pack_f16x2(x0, x1) : pack_bf16x2(x0, x1);
          }
        }
      }
      // ---- O += P V
      // Tokens of one MMA may see different rows here.  A zero weight takes a
      // finite row's part out exactly; a NaN or infinity (looked for in the
      // warp's V rows) takes the way apart.  Both give the same bits.
      bool apart = edge && a.S > 1;
      if (apart) {
        bool bad = false;
        for (int x = lane; x < kPer * Sh::kChunks; x += 32) {
          const uint4 v = lds_u4(vt + x * 16);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            bad |= kFp8 ? (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0
                        : (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
        }
        apart = __any_sync(0xffffffffu, bad);
      }
      if (!apart) {
        v_products<D, MT, kFp8>(vt, lane, [&](int mt, int x, int j, uint32_t b0, uint32_t b1) {
          mma16<kFp8>(o[mt][j], pf[mt][x], b0, b1);
        });
      } else {
        float o2[MT][D / 8][4];
        uint32_t pf2[MT][kGroups][4];
        int sq2[MT][2];
        memcpy(o2, o, sizeof o2);
        memcpy(pf2, pf, sizeof pf2);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = row0 + mt * 16 + g + 8 * e;
            sq2[mt][e] = i < qrows ? token_of(i) : a.S;
          }
        v_products_apart<D, MT, kFp8, kTree>(&o2[0][0][0], &pf2[0][0][0], &sq2[0][0], vt, lane, base, p_first,
                                             kTree ? cu.sp.n : a.S, a.win, a, cu.b);
        memcpy(o, o2, sizeof o);
      }
    }
    __syncwarp();

    // ---- end of the unit or of this CTA's share: join the warps
    const bool unit_end = cu.tile + 1 == cu.sp.tiles;
    if (unit_end || step + 1 == steps) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int x = 1; x <= 2; ++x) {
            const float other = __shfl_xor_sync(0xffffffffu, l[mt][e], x);
            l[mt][e] = kFp8 ? far_add(l[mt][e], other) : l[mt][e] + other;
          }
        }
      float* so = slots + (warp % Sh::kSlots) * Sh::kSlotFloats;
      float* sml = slots + Sh::kSlots * Sh::kSlotFloats + (warp % Sh::kSlots) * 2 * Sh::kRows;
      auto put = [&] {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (row0 + mt * 16 + 8 * e >= qrows) continue;   // no query row in these eight
            const int r = mt * 16 + g + 8 * e;
            if (c == 0) sml[r] = m[mt][e], sml[Sh::kRows + r] = l[mt][e];
            if constexpr (kFp8) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {   // dims 32 c + 4 x .. + 3
                const int j = (x & 3) * 4, k = 2 * e + (x >> 2);
                *reinterpret_cast<float4*>(so + r * Sh::kPitch + e4m3_piece(r, c, x)) =
                    make_float4(o[mt][j][k], o[mt][j + 1][k], o[mt][j + 2][k], o[mt][j + 3][k]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < D / 8; ++j)
                *reinterpret_cast<float2*>(so + r * Sh::kPitch + 8 * j + 2 * c) = make_float2(o[mt][j][2 * e], o[mt][j][2 * e + 1]);
            }
          }
      };
      // warps that held rows in this piece (all of them if it had two tiles)
      const int left = (cu.sp.L - (cu.sp.t0 + cu.tile) * kTile + kPer - 1) / kPer;
      const int held = step > seg_first || left > Sh::kWarps ? Sh::kWarps : left;
      __syncthreads();   // the slots' last readers are done
      // kSlots warps at a time hand their state to the kSlots before them
#pragma unroll
      for (int from = Sh::kWarps - Sh::kSlots; from > 0; from -= Sh::kSlots) {
        if (from >= held) continue;
        if (warp >= from && warp < from + Sh::kSlots) put();
        __syncthreads();
        if (warp >= from - Sh::kSlots && warp < from) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (row0 + mt * 16 + 8 * e >= qrows) continue;
              const int r = mt * 16 + g + 8 * e;
              const float m2 = sml[r], top = fmaxf(m[mt][e], m2), ref = top == -INFINITY ? 0.f : top;
              const float f1 = fast_exp2(m[mt][e] - ref), f2 = fast_exp2(m2 - ref);
              if (kFp8)
                l[mt][e] = far_add(far_move(l[mt][e], m[mt][e] - ref), far_move(sml[Sh::kRows + r], m2 - ref));
              else
                l[mt][e] = l[mt][e] * f1 + sml[Sh::kRows + r] * f2;
              m[mt][e] = top;
              if constexpr (kFp8) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const int j = (x & 3) * 4, k = 2 * e + (x >> 2);
                  const float4 v = *reinterpret_cast<const float4*>(so + r * Sh::kPitch + e4m3_piece(r, c, x));
                  o[mt][j][k] = o[mt][j][k] * f1 + v.x * f2;
                  o[mt][j + 1][k] = o[mt][j + 1][k] * f1 + v.y * f2;
                  o[mt][j + 2][k] = o[mt][j + 2][k] * f1 + v.z * f2;
                  o[mt][j + 3][k] = o[mt][j + 3][k] * f1 + v.w * f2;
                }
              } else {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                  const float2 v = *reinterpret_cast<const float2*>(so + r * Sh::kPitch + 8 * j + 2 * c);
                  o[mt][j][2 * e] = o[mt][j][2 * e] * f1 + v.x * f2;
                  o[mt][j][2 * e + 1] = o[mt][j][2 * e + 1] * f1 + v.y * f2;
                }
              }
            }
        }
        if (from > Sh::kSlots) __syncthreads();
      }
      if (warp < Sh::kSlots) {
        __syncwarp();
        put();
      }
      __syncthreads();
      // the kSlots states, a warp per row: a lane owns D / 32 neighbouring dims
      const bool whole = unit_end && cu.tile == step - seg_first;   // the piece is the whole unit
      const float* ml = slots + Sh::kSlots * Sh::kSlotFloats;
      const int slot = seg_first == 0 ? 0 : 1;
      const int64_t pslot = (int64_t)blockIdx.x * 2 + slot;
      for (int r = warp; r < Sh::kRows && row0 + r < qrows; r += Sh::kWarps) {
        const float* row_at = slots + r * Sh::kPitch + (kFp8 ? e4m3_piece(r, lane >> 3, lane & 7) : lane * (D / 32));
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < Sh::kSlots; ++x) top = fmaxf(top, ml[x * 2 * Sh::kRows + r]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f, acc[D / 32];
        FarSum sums;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
#pragma unroll
        for (int x = 0; x < Sh::kSlots; ++x) {
          const float d = ml[x * 2 * Sh::kRows + r] - ref, f = fast_exp2(d), ls = ml[x * 2 * Sh::kRows + Sh::kRows + r];
          if (kFp8)
            sums.add(far_move(ls, d));
          else
            sum += ls * f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            acc[i] += row_at[x * Sh::kSlotFloats + i] * f;
        }
        if (kFp8) sum = sums.sum();
        if (whole) {
          const int i = row0 + r, s = token_of(i), hd = h * group + i - s * group;
          // some row weighs (a NaN is passed on)
          const bool any = sum != 0.f && (!kTree || s < cu.sp.n);
          const float inv = any ? 1.f / (kFp8 ? fabsf(sum) : sum) : 0.f, rest = kFp8 ? far_rest(sum) : 1.f;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)cu.b * a.S + s) * a.out_stride + hd * D +
                               lane * (D / 32);
#pragma unroll
          for (int x = 0; x < D / 32; x += 2)
            *reinterpret_cast<uint32_t*>(dst + x) = kTree && !any ? 0u : pack_bf16x2(acc[x] * inv * rest, acc[x + 1] * inv * rest);
          if (a.lse && lane == 0)
            a.lse[((int64_t)cu.b * a.S + s) * a.heads + hd] =
                any ? (top + (kFp8 ? far_log2(sum) : log2f(sum))) * kLn2 : -INFINITY;
        } else {
          float* dst = part + (pslot * Sh::kRows + r) * (D + 2);
#pragma unroll
          for (int x = 0; x < D / 32; ++x) dst[lane * (D / 32) + x] = acc[x];
          if (lane == 0) dst[D] = top, dst[D + 1] = sum;
        }
      }
      if (tid == 0 && step + 1 == steps) {
        // the unit starts here (in its first tile) and goes on in the next
        // CTAs: this CTA's entry names the pieces
        PaJoin j;
        j.count = 0;
        j.slot = slot;
        j.b = cu.b;
        j.unit = cu.unit;
        if (!unit_end && cu.tile == step - seg_first) {
          const int64_t last = unit_at + cu.sp.tiles;     // the unit's last tile in the list of costs
          const int64_t G = total_sh < gridDim.x ? total_sh : gridDim.x;
          j.count = (int)(((last + 1) * G - 1) / total_sh) - (int)blockIdx.x + 1;
        }
        joins[blockIdx.x] = j;
      }
      seg_first = step + 1;
      if (tid == 0) unit_at += cu.sp.tiles + 1;
    }
    cu.next(a, units);
  }
}

// Joins the pieces of the units cut between CTAs: block (x, y) does query row
// y of the unit that starts in CTA x, its warps a part of the pieces each.
constexpr int kJoinWarps = 8;
template <int D, bool kFp8, bool kTree>
__global__ void __launch_bounds__(32 * kJoinWarps)
    paged_join_kernel(const PagedArgs a, int chunks, int rows, const float* __restrict__ part,
                      const PaJoin* __restrict__ joins) {
  __shared__ float sm_o[kJoinWarps][D], sm_m[kJoinWarps], sm_l[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const PaJoin j = joins[blockIdx.x];
  if (j.count == 0) return;
  const int group = a.heads / a.kv_heads, h = j.unit / chunks, i = (j.unit - h * chunks) * rows + blockIdx.y;
  if (i >= a.S * group) return;
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  for (int p = warp; p < j.count; p += kJoinWarps) {
    const int64_t slot = p == 0 ? (int64_t)blockIdx.x * 2 + j.slot : (int64_t)(blockIdx.x + p) * 2;
    const float* src = part + (slot * rows + blockIdx.y) * (D + 2);
    const float m2 = src[D], l2 = src[D + 1];
    const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.f : top;
    const float f1 = fast_exp2(m - ref), f2 = fast_exp2(m2 - ref);
    l = kFp8 ? far_add(far_move(l, m - ref), far_move(l2, m2 - ref)) : l * f1 + l2 * f2;
    m = top;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) acc[x] = acc[x] * f1 + src[lane + 32 * x] * f2;
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int x = 0; x < D / 32; ++x) sm_o[warp][lane + 32 * x] = acc[x];
  __syncthreads();
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm_m[w]);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, f[kJoinWarps];
  FarSum sums;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    f[w] = fast_exp2(sm_m[w] - ref);
    if (kFp8)
      sums.add(far_move(sm_l[w], sm_m[w] - ref));
    else
      sum += sm_l[w] * f[w];
  }
  if (kFp8) sum = sums.sum();
  const int s = i / group, hd = h * group + i - s * group;
  const bool any = sum != 0.f && (!kTree || !a.count || s < a.count[j.b]);
  const int64_t tok = (int64_t)j.b * a.S + s;
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v += sm_o[w][d] * f[w];
    static_cast<__nv_bfloat16*>(a.out)[tok * a.out_stride + hd * D + d] = __float2bfloat16_rn(any ? v / (kFp8 ? fabsf(sum) : sum) * (kFp8 ? far_rest(sum) : 1.f) : 0.f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[tok * a.heads + hd] = any ? (top + (kFp8 ? far_log2(sum) : log2f(sum))) * kLn2 : -INFINITY;
}

template <int D, int MT, bool kFp8, bool kTree>
int launch_shape(const PagedArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  using Sh = PaShape<D, MT, kFp8>;
  auto kern = paged_attn_kernel<D, MT, kFp8, kTree>;
  static PerDeviceOnce attr;
  if (const cudaError_t e = attr.run([&] { return allow_max_dynamic_smem(kern); }))
    return launch_fail("cudaFuncSetAttribute(paged_attn_kernel)", e);
  const int qrows = a.S * (a.heads / a.kv_heads), chunks = (qrows + Sh::kRows - 1) / Sh::kRows;
  float* part = static_cast<float*>(a.workspace);
  PaJoin* joins = reinterpret_cast<PaJoin*>(part + (size_t)num_sms * 2 * Sh::kRows * (D + 2));
  // at most the tiles that the bound on the lengths allows
  const int64_t tiles = (int64_t)a.B * a.kv_heads * chunks * ((a.max_len + Sh::kTile - 1) / Sh::kTile + 1);
  const int grid = tiles < num_sms ? (int)tiles : num_sms;
  const int r = launch_kernel(kern, dim3(grid), dim3(Sh::kThreads), Sh::kSmem, st, pdl, a, chunks, a.kv_heads * chunks, part, joins);
  if (r < 0) return r;
  // a unit of one tile is never cut
  const int span = a.win > 0 && a.win + a.S - 1 < a.max_len ? a.win + a.S - 1 + Sh::kTile - 1 : a.max_len;
  if (span <= Sh::kTile) return r;
  const int rows = qrows < Sh::kRows ? qrows : Sh::kRows;
  const int r2 = launch_kernel(paged_join_kernel<D, kFp8, kTree>, dim3(grid, rows), dim3(32 * kJoinWarps), 0, st, pdl, a, chunks,
                               (int)Sh::kRows, (const float*)part, (const PaJoin*)joins);
  return r2 < 0 ? r2 : r + r2;
}

}  // namespace

// Partials of two pieces per CTA of up to 32 query rows, and the join list.
size_t paged_attn_workspace(int dim, int num_sms) {
  return (size_t)num_sms * (2 * 32 * (dim + 2) * sizeof(float) + sizeof(PaJoin));
}

template <bool kTree>
static int launch_warps(const PagedArgs& a, bool fp8, int num_sms, cudaStream_t st, bool pdl) {
  const bool two = a.S * (a.heads / a.kv_heads) > 16;
  if (fp8)
    return two ? launch_shape<128, 2, true, kTree>(a, num_sms, st, pdl) : launch_shape<128, 1, true, kTree>(a, num_sms, st, pdl);
  switch (a.dim) {
    case 64:
      return two ? launch_shape<64, 2, false, kTree>(a, num_sms, st, pdl) : launch_shape<64, 1, false, kTree>(a, num_sms, st, pdl);
    case 128:
      return two ? launch_shape<128, 2, false, kTree>(a, num_sms, st, pdl)
                 : launch_shape<128, 1, false, kTree>(a, num_sms, st, pdl);
    default: return launch_shape<256, 1, false, kTree>(a, num_sms, st, pdl);
  }
}

int launch_paged_attn(const PagedArgs& a, bool fp8, int num_sms, cudaStream_t st, bool pdl) {
  return a.tree ? launch_warps<true>(a, fp8, num_sms, st, pdl) : launch_warps<false>(a, fp8, num_sms, st, pdl);
}

}  // namespace csa
