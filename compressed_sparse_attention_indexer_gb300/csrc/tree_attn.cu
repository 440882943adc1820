// Attention of trees of drafted tokens over paged K / V pools on the fifth-
// generation tensor cores, for drafts and heads that make more query rows per kv
// head than the warps' MMA takes at once, over enough requests or long ones
// (csa_tree_attn; see launch_tree_attn for the rule).
//   out[s][h] = sum_r softmax_r(scale q[s][h] . k[r]) v[r],  lse = ln sum_r exp(.)
// over the rows before the drafts (the window's) and the drafts in s's mask.
//
// A K / V row pair serves all S * heads / kv_heads query rows of its kv head: up
// to about 290 of them the rows' bytes bound it, above that the products (and
// their exponentials).  So 128 query rows make the M of a product, and up to 256
// share a tile of 128 K / V rows.
//
// One CTA per SM takes an even share of the list of tiles (paged_cuts).  Two
// slots of tensor memory hold 128 x 128 scores each, over which their bf16 weights
// are written, and 128 x D of output.  A slot is a half of the query rows, both take
// every tile, and one slot's products run under the other's softmax (with 128 query
// rows or fewer the second slot passes the tiles on; slots that took tiles in turn
// there were no faster: 768 and 776 us for 64 x 16 drafts, 67 and 66 for windows of
// small heads, at the time).
//   warps 0-3, 4-7   softmax of slot 0 and 1: a thread per query row, its 128 scores
//                    in registers, so that maxima and sums need no exchange; the
//                    reference maximum moves only when exceeded by 2^8 (the output is
//                    then rescaled in place);
//   warp 13          copies the rows by TMA into a ring of 128-byte swizzled stages
//                    (K and V alike: V is read as an MN-major operand), several ahead,
//                    across units.  A copy takes the rows of a tile that surely lie in
//                    one page, gcd(block, 128) of them.  (Four warps of 16-byte
//                    cp.async took 1900 cycles for a chunk of 32 KB, TMA gathers of four
//                    rows 80 cycles each: 1699 and 2527 us for 64 x 16 drafts.)
//   warps 8-11       E4M3: convert the codes, which land beside the ring; bf16: look
//                    through V's rows in edge tiles;
//   warps 12, 14     issue the MMAs of slot 0 and 1: S = Q K^T, O += P V (P from tensor
//                    memory).  An issue waits for the pipe, so one warp for both slots
//                    left the pipe idle over its waits (4700 cycles for two slots'
//                    tile, of which 1900 are products);
//   warp 15          the unit's query rows.
//
// Masks.  A tile that some draft does not see whole (the window's first rows,
// the drafts') is an edge tile: each thread builds the 128 bits of its row and
// takes masked scores as -inf, whatever they hold.  V rows with a NaN or an
// infinity there are zeroed in shared memory and added by hand, to the drafts
// that see them (add_apart).
//
// Measured: 64 x 16 drafts over 1024 .. 65536 bf16 rows, 32 / 4 heads of 128, 761 us
// (6.2 TB/s: HBM); 8 x 64 drafts over 8192 .. 16384, 95 us (1000 TFLOP/s: softmax and
// products in turn); 16 x 64 drafts over E4M3 rows, 64 / 8 heads, 512 us (765 TFLOP/s:
// softmax and conversion share the issue slots and the instruction cache); 48 x 21 drafts
// with a window of 1000, 16 / 8 heads of 64, 56 us (starts of units).
//
// Scores, maxima, sums and output are fp32; the weights are rounded to bf16 for
// the product with V, E4M3 ones after they took V's scale: scales of a request may
// lie any factor apart (a row of zeros has 1), which bf16's range holds without an
// exponent per row, and f16's, as the warps' kernel has them, would not.  bf16 ends
// as low as fp32 does, so that E4M3 weights are lifted (kLift) for scales next to
// 2^-126.
#include <cudaTypedefs.h>

#include "csa_internal.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "tc5.cuh"
#include "tree_pipeline.h"

namespace csa {

namespace {

constexpr int kTtThreads = 512;
constexpr int kRowWarp = 8, kRowWarps = 4, kMmaWarp = 12, kMmaWarp2 = 14, kLoadWarp = 13;
// Registers of the softmax's threads and of the others, 2 x 128 together: E4M3's converters
// want more (8 x 64 drafts over 8192 .. 16384 rows, 32 / 4 heads: 146 us with 72, 158 with 64, 167 with 80;
// bf16 97 with 56, 95 with 48 but 64 x 16 drafts 772 instead of 760).
template <bool kFp8>
constexpr int kRegsSoftmax = kFp8 ? 184 : 200;
template <bool kFp8>
constexpr int kRegsOthers = 256 - kRegsSoftmax<kFp8>;
constexpr int kRows = 256;                 // query rows of a unit, two slots of 128
constexpr int kTile = 128;                 // K / V rows per tile
constexpr int kExtra = 2;                  // a unit's start and end, in tiles
constexpr int kSub = kTile * 128;          // 128 rows x 64 dims bf16
constexpr float kGrow = 8.f;               // the reference maximum moves when exceeded by this (log2 units)
// E4M3: V's scales are taken 2^lift larger (and the output back), so that weights with one of
// 2^-126 are normal bf16 numbers down to 2^-lift of the largest, and off by 2^-(lift + 8) of it
// below that.  Weights of up to 2^8 times codes of up to 2^9 and scales of up to 2^80 over L rows
// stay in fp32 for lift <= 30 - log2 L.  (A lift that ended with the first tile of larger
// scales, known from its converters: 579 us instead of 512 for 16 x 64 drafts; by max_len, a
// constant of the launch: 507, but bits that go with it.)
constexpr int kLift = 16;
__device__ __forceinline__ int lift_of(int L) { return min(kLift, __clz(L - 1) - 2); }
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
constexpr int kScaleTiles = kTreeScales;
constexpr int kScaleBytes = kTile * 2 * 4; // K's and V's of a tile

struct TtSmem {
  uint64_t full[8], empty[8];              // stages of the ring
  uint64_t land[8];                        // bf16 V of an edge tile, before it was looked through
  uint64_t raw_full[3], raw_empty[3];      // chunks of E4M3 codes
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t q_full, q_empty, sc_full[kScaleTiles], done[2];
  uint32_t tmem;
  int abort;
  PaCost scan[33];
  Cut cut[2];
  uint32_t bad[8][4];                      // per stage: V rows with a NaN or an infinity
  int looked[8];                           // warps that have looked through it, modulo 4
};

template <int D, bool kFp8>
struct TtShape {
  static constexpr int kSubs = D / 64;
  static constexpr int kStage = kSubs * kSub;
  static constexpr int kQBytes = kRows / 128 * kStage;
  static constexpr int kRawDepth = kFp8 ? kTreeRaw : 1;   // chunks of codes beside the ring
  static constexpr int kRaw = kFp8 ? kTile * D : 0;
  static constexpr int kScales = kFp8 ? kScaleTiles * kScaleBytes : 0;
  static constexpr int kStages = tree_stages(D, kFp8);
  static constexpr int kSmem = kQBytes + kStages * kStage + kRawDepth * kRaw + kScales + (int)sizeof(TtSmem);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kStages >= 3 && kStages <= 8, "a batch's V and K; barriers");
  static_assert(kStages / 2 + 1 < kScaleTiles, "scales");
};

// One piece: consecutive tiles of a unit that this CTA takes.
struct Piece {
  Span<kTile, true> sp;
  int b, unit, tile, nt;
  bool whole, first;                       // all of the unit's tiles; from the unit's first on
};
struct Walk {
  Cursor<kTile, true> cu;
  int left;
  __device__ __forceinline__ void init(const PagedArgs& a, const Cut* cut) {
    cu.b = cut[0].b;
    cu.sp.set(a, cu.b);
    cu.unit = cut[0].unit;
    cu.tile = cut[0].tile;
    left = (int)(cut[1].at - cut[0].at);
  }
  __device__ __forceinline__ bool next(const PagedArgs& a, int units, Piece& p) {
    if (left == 0) return false;
    p.sp = cu.sp;
    p.b = cu.b;
    p.unit = cu.unit;
    p.tile = cu.tile;
    p.nt = min(cu.sp.tiles - cu.tile, left);
    p.first = cu.tile == 0;
    p.whole = p.nt == cu.sp.tiles;
    left -= p.nt;
    cu.tile += p.nt - 1;
    if (left > 0) cu.next(a, units);
    return true;
  }
};

// Whether some draft sees only a part of tile t's rows.
__device__ __forceinline__ bool edge_tile(const PagedArgs& a, const Span<kTile, true>& sp, int t) {
  const int base = (sp.t0 + t) * kTile;
  return base < sp.lo || base + kTile > sp.L - sp.n || (a.win > 0 && base < sp.L - a.win);
}

// Bits lo .. hi - 1, either end anywhere.
__device__ __forceinline__ uint32_t ones(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return hi <= lo ? 0u : (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
}
// Rows 32 w .. of tile t that belong to the span.
__device__ __forceinline__ uint32_t span_rows(const Span<kTile, true>& sp, int t, int w) {
  const int r0 = (sp.t0 + t) * kTile + 32 * w;
  return ones(sp.lo - r0, sp.L - r0);
}

// The bits of a tile's rows, from row c0 on, for a draft: rows up to `out` are outside its
// window, the drafts start at row p and are n, `bits` are its mask's 32-bit words (their
// loads go out together).
__device__ __forceinline__ void seen_rows(uint32_t* seen, int c0, int out, int p, int n, const uint32_t* bits, int words32) {
  const int t0 = c0 - p, i0 = t0 >> 5;           // draft at the first bit, its word: rounded down
  uint32_t w[5] = {0, 0, 0, 0, 0};
  if (t0 > -kTile) {
#pragma unroll
    for (int k = 0; k < 5; ++k)
      if (i0 + k >= 0 && i0 + k < words32) w[k] = bits[i0 + k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + 32 * k, t = t0 + 32 * k;
    seen[k] = ones(out + 1 - c, p - c) | (__funnelshift_r(w[k], w[k + 1], t0 & 31) & ones(-t, n - t));
  }
}

__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  return tc5::sdesc_k_sw128(saddr) - ((uint64_t)1u << 16) + ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16);
}
__device__ __forceinline__ bool not_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7f80u) == 0x7f80u; }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// One lane of a warp that runs as one: the same lane every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_out(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A wait that a whole warp makes: true when every lane saw the phase.
__device__ __forceinline__ bool warp_wait(uint64_t& bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, tc5::mbar_wait_backoff(smem_u32(&bar), parity, abort, 64));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// The high bits of the bytes that are a NaN's E4M3 code.
__device__ __forceinline__ uint32_t e4m3_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// The place in the pool of `seg` rows of a tile, rows r .. of it, which lie in one page:
// looked up ahead of its use.
struct Spot {
  int entry, within;
  int first, last;                         // the span's rows among the segment's, [first, last)
  __device__ __forceinline__ void none() { within = -1; }
  __device__ __forceinline__ void lookup(const PagedArgs& a, const Span<kTile, true>& sp, int b, int tile, int r, int seg) {
    const int at = (sp.t0 + tile) * kTile + r;
    first = max(sp.lo - at, 0);
    last = min(sp.L - at, seg);
    within = entry = -1;
    if (first >= last) return;
    if (a.table) {
      const int k = (int)((uint32_t)at / (uint32_t)a.block);
      within = at - k * a.block;
      if (k < a.table_stride) entry = a.table[(int64_t)b * a.table_stride + k];
    } else {
      within = 0;
      // rows outside the pool may be a part of the segment: its start is kept near the pool
      const int64_t x = a.off[b] + at;
      entry = (int)(x < -kTile ? -kTile : x > a.rows ? a.rows : x);
    }
  }
  // Its pool row, `none` where it has no row to read; false when some of its rows in the
  // span are unmapped or outside the pool.
  __device__ __forceinline__ bool resolve(const PagedArgs& a, int none, int& row) const {
    row = none;
    if (within < 0) return true;
    if (a.table && entry < 0) return false;
    const int64_t x = a.table ? (int64_t)entry * a.block + within : entry;
    if (x < a.rows) row = (int)x;
    return x + first >= 0 && x + last <= a.rows;
  }
};

// The part of an edge tile's V rows that was zeroed: rows `bad` (four words), added to
// the output of the threads whose row sees them.  Rare, out of line.
template <int D, bool kFp8>
__device__ __noinline__ void add_apart(const PagedArgs& a, int b, int h, int base, const uint32_t* bad, const uint32_t* seen,
                                       uint32_t p_at, uint32_t o_at) {
#pragma unroll 1
  for (int r = 0; r < kTile; ++r) {
    if (!((bad[r >> 5] >> (r & 31)) & 1)) continue;
    const bool mine = (seen[r >> 5] >> (r & 31)) & 1;
    if (!__any_sync(0xffffffffu, mine)) continue;
    const int64_t row = pool_row(a.table, a.block, a.table_stride, a.off, b, base + r);
    if (row < 0 || row >= a.rows) continue;
    uint32_t w;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n tcgen05.wait::ld.sync.aligned;\n" : "=r"(w) : "r"(p_at + (r >> 1)) : "memory");
    const float p = __uint_as_float(r & 1 ? w & 0xffff0000u : w << 16);
    const uint8_t* v = static_cast<const uint8_t*>(a.v) + (uint64_t)row * a.v_step + (size_t)h * D * (kFp8 ? 1 : 2);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tc5::tmem_ld32(o_at + c, o);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float x;
        bool apart;
        if (kFp8) {
          apart = (v[c + i] & 0x7f) == 0x7f;
          x = __uint_as_float(0x7fffffffu);
        } else {
          const uint32_t u = reinterpret_cast<const uint16_t*>(v)[c + i];
          apart = not_finite(u);
          x = __uint_as_float(u << 16);
        }
        if (apart && mine) o[i] += p * x;
      }
      tc5::tmem_st32(o_at + c, o);
      tc5::tmem_wait_st();
    }
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kTtThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PagedArgs a, int rs, int seg, int chunks, int units, float* __restrict__ part, PaJoin* __restrict__ joins) {
  using Sh = TtShape<D, kFp8>;
  constexpr int ST = Sh::kStages;
  // (no static shared memory: the dynamic part starts on a 1024-byte boundary)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  TtSmem& sm = *reinterpret_cast<TtSmem*>(smem_raw + Sh::kSmem - sizeof(TtSmem));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t qsm = smem_u32(smem_raw);
  const uint32_t ring = qsm + Sh::kQBytes, raw = ring + ST * Sh::kStage, scales = raw + Sh::kRawDepth * Sh::kRaw;
  volatile int* abort = &sm.abort;
  const int group = a.heads / a.kv_heads, qrows = a.S * group;
  const int unit_rows = 2 * rs;            // query rows of a unit, rs of them in a slot
  pdl_wait();
  pdl_trigger();

  int64_t total, G;
  const bool share = paged_cuts<kTile, true, kTtThreads / 2, kExtra>(a, units, sm.scan, sm.cut, total, G);
  if (tid == 0) joins[blockIdx.x].count = 0;
  if (!share || sm.cut[1].at == sm.cut[0].at) return;
  if (tid == 0) {
    const Cut& c0 = sm.cut[0];
    const Cut& c1 = sm.cut[1];
    const bool same = c0.b == c1.b && c0.unit == c1.unit;
    if (c1.tile > 0 && (!same || c0.tile == 0)) {
      // a unit starts here and goes on in the next CTAs
      Span<kTile, true> sp;
      sp.set(a, c1.b);
      const int64_t last = c1.first + sp.tiles + kExtra - 1;   // its last place in the list of costs
      PaJoin j;
      j.count = (int)(((last + 1) * G - 1) / total) - (int)blockIdx.x + 1;
      j.slot = same ? 0 : 1;
      j.b = c1.b;
      j.unit = c1.unit;
      joins[blockIdx.x] = j;
    }
    sm.abort = 0;
    for (int i = 0; i < 8; ++i) {
      tc5::mbar_init(smem_u32(&sm.full[i]), kFp8 ? kRowWarps : 1);
      tc5::mbar_init(smem_u32(&sm.empty[i]), 2);   // the slots
      tc5::mbar_init(smem_u32(&sm.land[i]), 1);
      sm.looked[i] = 0;
    }
    for (int i = 0; i < 3; ++i) {
      tc5::mbar_init(smem_u32(&sm.raw_full[i]), 1);
      tc5::mbar_init(smem_u32(&sm.raw_empty[i]), kRowWarps);
    }
    for (int i = 0; i < kScaleTiles; ++i) tc5::mbar_init(smem_u32(&sm.sc_full[i]), kRowWarps);
    for (int i = 0; i < 2; ++i) {
      tc5::mbar_init(smem_u32(&sm.s_full[i]), 1);
      tc5::mbar_init(smem_u32(&sm.p_full[i]), 4);
      tc5::mbar_init(smem_u32(&sm.o_full[i]), 1);
    }
    tc5::mbar_init(smem_u32(&sm.q_full), 1);
    tc5::mbar_init(smem_u32(&sm.q_empty), 2);
    for (int i = 0; i < 2; ++i) tc5::mbar_init(smem_u32(&sm.done[i]), 1);
    tc5::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc5::tmem_alloc(smem_u32(&sm.tmem), 512);
    tc5::tmem_relinquish();
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  // i / group for 0 <= i < S * heads <= 2^20
  const float per_group = 1.f / (float)group;
  auto token_of = [&](int i) { return (int)(((float)i + 0.5f) * per_group); };

  if (warp < kRowWarp) {
    setmaxnreg_inc<kRegsSoftmax<kFp8>>();
    // ------------------------------------------------------------ softmax
    const int slot = warp >> 2, t = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + slot * 128, o_at = tmem + lanes + 256 + slot * 128;
    const float scale2 = a.scale * kLog2e;
    const int words32 = 2 * a.words;
    uint32_t n_s = 0, n_o = 0;                  // phases of s_full and o_full
    int jj = 0, seen_pieces = 0;                // tiles and pieces of the CTA before this piece
    Walk walk;
    walk.init(a, sm.cut);
    Piece pc;
    bool ok = true;
    while (ok && walk.next(a, units, pc)) {
      const int h = chunks == 1 ? pc.unit : pc.unit / chunks, row0 = (pc.unit - h * chunks) * unit_rows;
      const int i = t < rs ? row0 + slot * rs + t : qrows;   // (qrows: no row)
      const int s = i < qrows ? token_of(i) : 0, hd = h * group + i - s * group;
      const int64_t tok = (int64_t)pc.b * a.S + s;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + tok * a.out_stride + hd * D;
      const int at_piece = seen_pieces++;
      if (pc.sp.L <= 0) {                      // a padding request
        if (i < qrows) {
          for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[tok * a.heads + hd] = -INFINITY;
        }
        continue;
      }
      const int p_first = pc.sp.L - pc.sp.n;
      const bool real = i < qrows && s < pc.sp.n;
      const bool busy = row0 + slot * rs < qrows;   // the slot has rows
      float m = -INFINITY, l = 0.f;
      if (busy) {
        const int outside = real ? tree_outside(a, pc.b, s, p_first, pc.sp.n) : 0;
        const uint32_t* bits = reinterpret_cast<const uint32_t*>(a.tree + tok * a.words);
        {
          float z[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x] = 0.f;
#pragma unroll
          for (int c = 0; c < D; c += 32) tc5::tmem_st32(o_at + c, z);
        }
        for (int j = 0; j < pc.nt; ++j) {
          const int base = (pc.sp.t0 + pc.tile + j) * kTile;
          const bool edge = edge_tile(a, pc.sp, pc.tile + j);
          ok = warp_wait(sm.s_full[slot], n_s & 1, abort);
          ++n_s;
          if (!ok) break;
          tc5::fence_after_sync();
          float x[128];
          tc5::tmem_ld32x2(s_at, x, x + 32);
          tc5::tmem_ld32x2(s_at + 64, x + 64, x + 96);
          const float4* sc = nullptr;            // the tile's scales: K's, then V's
          if (kFp8) {
            const int at = jj + j;
            ok = warp_wait(sm.sc_full[at % kScaleTiles], (at / kScaleTiles) & 1, abort);
            if (!ok) break;
            sc = reinterpret_cast<const float4*>(smem_raw + (scales - qsm) + (at % kScaleTiles) * kScaleBytes);
#pragma unroll
            for (int c = 0; c < 128; c += 4) {
              const float4 k = sc[c / 4];
              f2_out(f2_mul(f2(x[c], x[c + 1]), f2(k.x, k.y)), x[c], x[c + 1]);
              f2_out(f2_mul(f2(x[c + 2], x[c + 3]), f2(k.z, k.w)), x[c + 2], x[c + 3]);
            }
          }
          uint32_t seen[4];
          if (edge) {
            if (real) {
              seen_rows(seen, base, outside, p_first, pc.sp.n, bits, words32);
            } else {
              seen[0] = seen[1] = seen[2] = seen[3] = 0u;
            }
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!((seen[c >> 5] >> (c & 31)) & 1)) x[c] = -INFINITY;
          }
          float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
          const float mul = kFp8 ? 1.f : scale2;
          const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * mul;
          const bool grow = most > m + kGrow;
          if (__any_sync(0xffffffffu, grow && m > -INFINITY)) {
            const float f = grow ? exp2f(m - most) : 1.f;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tc5::tmem_ld32(o_at + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tc5::tmem_st32(o_at + c, o);
            }
          }
          if (grow) m = most;
          const float ref = m == -INFINITY ? 0.f : m;
          uint64_t sum[2] = {0, 0};
          const uint64_t mul2 = f2(mul, mul), ref2 = f2(-ref, -ref);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
              float4 v = make_float4(1.f, 1.f, 1.f, 1.f);
              if (kFp8) v = sc[kTile / 4 + half * 16 + c / 4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float p0, p1;
                f2_out(f2_fma(f2(x[half * 64 + c + 2 * e], x[half * 64 + c + 2 * e + 1]), mul2, ref2), p0, p1);
                p0 = fast_exp2(p0), p1 = fast_exp2(p1);
                uint64_t p = f2(p0, p1);
                sum[e] = f2_add(sum[e], p);
                if (kFp8) f2_out(f2_mul(p, e ? f2(v.z, v.w) : f2(v.x, v.y)), p0, p1);
                pk[c / 2 + e] = __uint_as_float(pack_bf16x2(p0, p1));
              }
            }
            tc5::tmem_st32(s_at + 32 * half, pk);
          }
          {
            float s0, s1;
            f2_out(f2_add(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
          }
          tc5::tmem_wait_st();
          if (edge) {
            TreePlace<ST> v;
            v.set(2 * (jj + j) + 1);
            const uint32_t st = v.st;
            ok = warp_wait(sm.full[st], v.ph, abort);
            if (!ok) break;
            uint32_t bad[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) bad[w] = *(volatile uint32_t*)&sm.bad[st][w];
            if (bad[0] | bad[1] | bad[2] | bad[3]) add_apart<D, kFp8>(a, pc.b, h, base, bad, seen, s_at, o_at);
          }
          tc5::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc5::mbar_arrive(smem_u32(&sm.p_full[slot]));
        }
        if (ok) {
          ok = warp_wait(sm.o_full[slot], n_o & 1, abort);
          ++n_o;
          tc5::fence_after_sync();
        }
      }
      jj += pc.nt;
      if (busy && ok) {
        const bool any = real && (l > 0.f || l != l);
        const float down = kFp8 ? pow2(-lift_of(pc.sp.L)) : 1.f, inv = any ? 1.f / l * down : 0.f;
        const int64_t pslot = (int64_t)blockIdx.x * 2 + (at_piece == 0 ? 0 : 1);
        float* dst = part + (pslot * kRows + slot * 128 + (t & ~31)) * (D + 2) + lane;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tc5::tmem_ld32(o_at + c, o);
          if (i < qrows) {
            if (pc.whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = any ? pack_bf16x2(o[e + 2 * x] * inv, o[e + 2 * x + 1] * inv) : 0u;
                *reinterpret_cast<uint4*>(out + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) dst[(c + e) * 32] = kFp8 ? o[e] * down : o[e];
            }
          }
        }
        if (i < qrows) {
          if (!pc.whole) dst[D * 32] = m, dst[(D + 1) * 32] = l;
          else if (a.lse) a.lse[tok * a.heads + hd] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
      }
    }
    tc5::tmem_wait_st();   // a wait that gave up may have left stores under way
  } else {
    setmaxnreg_dec<kRegsOthers<kFp8>>();
    if (warp < kMmaWarp) {
      // ---------------------------------------------------------- converters, or V's readers
      const int w = warp - kRowWarp;
      bool ok = true;
      if constexpr (kFp8) {
        // A lane takes 8 codes of a row at a time, 16 lanes a row: the 16 bytes that they
        // make go to eight different places of 16 bytes in either quarter of the warp.  (16
        // codes a lane, halves exchanged so that theirs do: 541 us instead of 512 for 16 x 64
        // drafts; four loads at a time instead of eight 518.)
        const int e = lane & 15, hi = lane >> 4;
        uint32_t to[4];                        // of the warp's rows 2 i + hi, i < 4; then 1024 bytes on
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = ring + (e >> 3) * kSub + (w * 32 + 2 * i + hi) * 128 + (((e & 7) ^ ((2 * i + hi) & 7)) << 4);
        // the lane's row of the tile: its scales are fetched a tile ahead, its place two
        Cursor<kTile, true> at;
        int left;
        {
          Walk walk;
          walk.init(a, sm.cut);
          at = walk.cu;
          left = walk.left;
        }
        Spot spot;
        // of the tile looked up and of the one fetched: there is one, some draft does not see
        // it whole, the span's rows of the warp's
        bool some_ahead = false, edge_ahead = false, some = false, edge = false;
        uint32_t rows_ahead = 0, rows = 0;
        float ks = 0.f, vs = 0.f, up = 1.f;
        auto ahead = [&] {                     // `at` to the next tile with rows, its place looked up
          while (left > 0 && at.sp.L <= 0) {
            if (--left > 0) at.next(a, units);
          }
          spot.none();
          some_ahead = left > 0;
          if (left > 0) {
            spot.lookup(a, at.sp, at.b, at.tile, w * 32 + lane, 1);
            edge_ahead = edge_tile(a, at.sp, at.tile);
            rows_ahead = span_rows(at.sp, at.tile, w);
          }
        };
        auto fetch = [&] {
          some = some_ahead, edge = edge_ahead, rows = rows_ahead;
          int row;
          if (!spot.resolve(a, -1, row)) row = -1;
          const int h = chunks == 1 ? at.unit : at.unit / chunks;
          ks = vs = 0.f;
          up = pow2(lift_of(at.sp.L));
          if (row >= 0) ks = a.k_scale[(int64_t)row * a.scale_stride + h], vs = a.v_scale[(int64_t)row * a.scale_stride + h];
          if (left > 0 && --left > 0) at.next(a, units);
        };
        ahead();
        fetch();
        ahead();
        uint32_t n = 0;                        // chunks
        // chunk n to its stage: K or V (look: an edge tile's V, with the span's rows) of the CTA's `tile`
        auto convert = [&](uint32_t st, bool wait_empty, uint32_t parity, bool kv, uint32_t tile, bool look, uint32_t mask) {
              const uint32_t stage = ring + st * Sh::kStage, slot = n % Sh::kRawDepth;
              uint32_t bad = 0;
              ok = warp_wait(sm.raw_full[slot], (n / Sh::kRawDepth) & 1, abort);
              if (ok && wait_empty) ok = warp_wait(sm.empty[st], parity, abort);
              if (!ok) return;
              const uint32_t from = raw + slot * Sh::kRaw + w * 32 * D + lane * 8;
#pragma unroll 1
              for (int i0 = 0; i0 < 16; i0 += 8) {
                uint32_t c[8][2];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(c[i][0]), "=r"(c[i][1]) : "r"(from + (i0 + i) * 256) : "memory");
                if (look) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const uint32_t n0 = e4m3_nan(c[i][0]), n1 = e4m3_nan(c[i][1]);
                    if (n0 | n1) {
                      bad |= 1u << (2 * (i0 + i) + hi);
                      c[i][0] &= ~((n0 >> 7) * 0xffu);
                      c[i][1] &= ~((n1 >> 7) * 0xffu);
                    }
                  }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  uint32_t u[4];
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    uint32_t lo, hi2;
                    e4m3x4_to_f16x2(c[i][x], lo, hi2);
                    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
                    u[2 * x] = pack_bf16x2(f0.x, f0.y);
                    u[2 * x + 1] = pack_bf16x2(f1.x, f1.y);
                  }
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(to[i & 3] + st * Sh::kStage + (i0 + i) / 4 * 1024), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
                }
              }
              if (!kv) {
                // the row's scales as the scores and weights take them; a V scale that is no
                // number reaches whoever sees the row by its score
                const uint32_t to = scales + (tile % kScaleTiles) * kScaleBytes + (w * 32 + lane) * 4;
                const bool number = fabsf(vs) < INFINITY;
                asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(to), "f"(number ? ks * (a.scale * kLog2e) : __uint_as_float(0x7fffffffu)) : "memory");
                asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(to + kTile * 4), "f"(number ? vs * up : 1.f) : "memory");
              }
              if (look) {
                bad = __reduce_or_sync(0xffffffffu, bad) & mask;
                if (lane == 0) *(volatile uint32_t*)&sm.bad[st][w] = bad;
              }
              tc5::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tc5::mbar_arrive(smem_u32(&sm.full[st]));
                tc5::mbar_arrive(smem_u32(&sm.raw_empty[slot]));
                if (!kv) tc5::mbar_arrive(smem_u32(&sm.sc_full[tile % kScaleTiles]));
              }
              ++n;
        };
        // (K and V of tile after tile: pieces do not matter, which leaves registers)
        TreePlace<ST> to_ring;
        to_ring.ph = 1;                        // (of the phase before)
        for (uint32_t tile = 0; ok && some; ++tile) {
          const bool edge_now = edge;
          const uint32_t rows_now = rows;
#pragma unroll 1
          for (int kv = 0; ok && kv < 2; ++kv) {
            convert(to_ring.st, n >= ST, to_ring.ph, kv, tile, kv && edge_now, rows_now);
            to_ring.move(1);
            if (!kv) {
              fetch();
              ahead();
            }
          }
        }
      } else {
        constexpr int kSpan = D / 8, kAtOnce = 32 / kSpan, kIter = 32 / kAtOnce;   // 16 bytes of a row each
        const int ch = lane % kSpan, r0 = lane / kSpan;
        // where this thread's piece i of a chunk lies in a stage
        auto place = [&](int i) {
          const int row = w * 32 + i * kAtOnce + r0;
          return (uint32_t)((ch >> 3) * kSub + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
        };
        uint32_t parity = 0, jj = 0;           // bit st: phase of land[st]; tiles before the piece
        Walk walk;
        walk.init(a, sm.cut);
        Piece pc;
        while (ok && walk.next(a, units, pc)) {
          if (pc.sp.L <= 0) continue;
#pragma unroll 1
          for (int j = 0; j < pc.nt; ++j) {
            if (edge_tile(a, pc.sp, pc.tile + j)) {
              const uint32_t st = (2 * (jj + j) + 1) % ST, stage = ring + st * Sh::kStage;
              ok = warp_wait(sm.land[st], (parity >> st) & 1, abort);
              parity ^= 1u << st;
              if (!ok) break;
              uint32_t bad = 0;
#pragma unroll 4
              for (int i = 0; i < kIter; ++i) {
                uint32_t c[4];
                const uint32_t at = stage + place(i);
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(at) : "memory");
                bool any = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) any |= not_finite(c[x]) || not_finite(c[x] >> 16);
                if (any) {
                  bad |= 1u << (i * kAtOnce + r0);
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    c[x] &= (not_finite(c[x]) ? 0u : 0xffffu) | (not_finite(c[x] >> 16) ? 0u : 0xffff0000u);
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3]) : "memory");
                }
              }
              bad = __reduce_or_sync(0xffffffffu, bad) & span_rows(pc.sp, pc.tile + j, w);
              if (lane == 0) *(volatile uint32_t*)&sm.bad[st][w] = bad;
              tc5::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                __threadfence_block();
                if ((atomicAdd(&sm.looked[st], 1) & 3) == 3) {   // the last of the four
                  __threadfence_block();
                  tc5::mbar_arrive(smem_u32(&sm.full[st]));
                }
              }
            }
          }
          jj += pc.nt;
        }
      }
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- row loader
      // Segments of several tiles are looked up at once, a lane each (four at most, where
      // a tile has more than 32), and a block of tiles ahead of their copies: looked up
      // tile by tile, the table's latency was on everyone's way (4000 cycles a tile).
      // The code is kept short: it runs beside the others' all the time, and unrolled by
      // four (31 KB of 119) it pushed theirs out of the instruction cache (16 x 64 drafts
      // over E4M3 583 us instead of 541, windows of small heads 65 instead of 56).
      const int segs = kTile / seg, per = (segs + 31) / 32, ahead = per > 1 ? 1 : 32 / segs;   // tiles of a block
      const int none = a.rows > 0 ? (int)a.rows : 1;   // a row behind the pool reads as zeros
      if (lane == 0) {
        tc5::prefetch_tmap(&kmap);
        tc5::prefetch_tmap(&vmap);
      }
      Walk walk;
      walk.init(a, sm.cut);
      Piece next;                              // the block looked up: the first tiles of what is left of a piece
      bool more = false;
      Spot spot[4];
      int row[4] = {none, none, none, none};   // pool rows of the block's segments
      auto look = [&] {
        while ((more = walk.next(a, units, next)) && next.sp.L <= 0) {
        }
      };
      auto lookup = [&] {
#pragma unroll 1
        for (int i = 0; i < per; ++i) {
          Spot s;
          s.none();
          const int x = lane * per + i;         // segment of the block
          if (more && x < segs * min(ahead, next.nt))
            s.lookup(a, next.sp, next.b, next.tile + x / segs, x % segs * seg, seg);
          spot[i] = s;
        }
      };
      // the place in the ring, or of E4M3 codes beside it: counted up
      TreeFeed<kFp8 ? Sh::kRawDepth : ST> feed;
      bool ok = true;
      constexpr int kCopies = kFp8 ? 1 : Sh::kSubs;   // of a segment
      const int copies = segs * kCopies;
      const uint32_t to_lane = lane / kCopies * seg * 128 + lane % kCopies * kSub;
      // tile t of the block: its K or V
      auto copy = [&](int t, bool v, int h, bool edge) {
        const uint32_t at = feed.at;
        if (feed.again) ok = warp_wait(kFp8 ? sm.raw_empty[at] : sm.empty[at], feed.ph, abort);
        if (!ok) return;
        const uint32_t bar = smem_u32(kFp8 ? &sm.raw_full[at] : edge ? &sm.land[at] : &sm.full[at]);
        const uint32_t to = kFp8 ? raw + at * Sh::kRaw : ring + at * Sh::kStage;
        const CUtensorMap* map = v ? &vmap : &kmap;
        if (lane == 0) tc5::mbar_expect_tx(bar, kFp8 ? Sh::kRaw : Sh::kStage);
        __syncwarp();
        if (per == 1) {
          const int r = __shfl_sync(0xffffffffu, row[0], (t * segs + lane / kCopies) & 31);
          if (lane < copies) tc5::tma_load_2d(to + to_lane, map, h * D + 64 * (lane % kCopies), r, bar);
          if (copies > 32) {                     // 32 segments in two copies
            const int r2 = __shfl_sync(0xffffffffu, row[0], 32 / kCopies + lane / kCopies);
            tc5::tma_load_2d(to + to_lane + 32 / kCopies * seg * 128, map, h * D + 64 * (lane % kCopies), r2, bar);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < per; ++i)
#pragma unroll
            for (int c = 0; c < kCopies; ++c)
              tc5::tma_load_2d(to + (lane * per + i) * seg * 128 + c * kSub, map, h * D + 64 * c, row[i], bar);
        }
        feed.next(edge);
      };
      look();
      lookup();
      while (ok && more) {
        const Span<kTile, true> sp = next.sp;
        const int nt = min(ahead, next.nt), h = chunks == 1 ? next.unit : next.unit / chunks, tile0 = next.tile;
        bool all = true;
#pragma unroll 1
        for (int i = 0; i < per; ++i) all &= spot[i].resolve(a, none, row[i]);
        if (!all && a.status) set_status(a.status, kStatusBadIndex);
        next.tile += nt;
        next.nt -= nt;
        if (next.nt == 0) look();
        lookup();
#pragma unroll 1
        for (int t = 0; ok && t < nt; ++t) {
#pragma unroll 1
          for (int v = 0; ok && v < 2; ++v) copy(t, v, h, v && !kFp8 && edge_tile(a, sp, tile0 + t));
        }
      }
      // the copies land before the block ends, whoever gave up meanwhile
      bool landed = true;
#pragma unroll 1
      for (uint32_t i = 0; landed && i < (kFp8 ? Sh::kRawDepth : ST); ++i) {
        bool other;
        uint32_t parity;
        if (feed.last(i, other, parity))
          landed = tc5::mbar_wait_drain(smem_u32(kFp8 ? &sm.raw_full[i] : other ? &sm.land[i] : &sm.full[i]), parity);
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp2) {
      // ---------------------------------------------------------- MMA issue
      // The warp runs as one (waits, ring places: the same in every lane), a lane issues.
      // Places in the ring are counted up, not divided out: the chain from a softmax's end
      // to its slot's next products is on everyone's way.
      const int slot = __shfl_sync(0xffffffffu, warp, 0) == kMmaWarp ? 0 : 1;
      constexpr uint32_t idesc_s = tc5::idesc_bf16_f32(128, kTile);
      constexpr uint32_t idesc_o = tc5::idesc_bf16_f32(128, D) | (1u << 16);   // B MN-major
      const uint64_t dq = tc5::sdesc_k_sw128(qsm + slot * Sh::kStage);
      const uint64_t dk = tc5::sdesc_k_sw128(ring), dv = sdesc_mn_sw128(ring, kSub);
      const uint32_t s_at = tmem + slot * 128, o_at = tmem + 256 + slot * 128;
      uint32_t pph = 0, qph = 0;               // phases
      bool ok = true;
      auto wait = [&](uint64_t& bar, uint32_t parity) {
        uint32_t i = 0;
        while (ok && !tc5::mbar_try_wait(smem_u32(&bar), parity)) {
          if ((++i & 63u) == 0 && (*abort || i >= tc5::kWaitPolls)) {
            *abort = 1;
            ok = false;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        tc5::fence_after_sync();
      };
      uint32_t jj = 0;                         // tiles before the piece
      Walk walk;
      walk.init(a, sm.cut);
      Piece pc;
      while (ok && walk.next(a, units, pc)) {
        if (pc.sp.L <= 0) continue;
        const int h = chunks == 1 ? pc.unit : pc.unit / chunks, row0 = (pc.unit - h * chunks) * unit_rows;
        if (row0 + slot * rs >= qrows) {
          // no rows for this slot: what it would have read is given back
          TreePlace<ST> c;
          c.set(2 * jj);
#pragma unroll 1
          for (int i = 0; ok && i < 2 * pc.nt; ++i, c.move(1)) {
            wait(sm.full[c.st], c.ph);
            if (ok && elect_one()) tc5::mbar_arrive(smem_u32(&sm.empty[c.st]));
          }
          wait(sm.q_full, qph);
          if (ok && elect_one()) tc5::mbar_arrive(smem_u32(&sm.q_empty));
        } else {
          TreePlace<ST> k, v;                  // moved on to the next tile's
          k.set(2 * jj);
          v.set(2 * jj + 1);
          wait(sm.q_full, qph);
          // a batch: with tile j's weights the output, then the scores of the slot's next
          // tile, 16 MMAs without anything between them
#pragma unroll 1
          for (int j = -1; j < pc.nt; ++j) {
            const bool out = j >= 0, in = j + 1 < pc.nt;
            if (in) wait(sm.full[k.st], k.ph);
            if (out) {
              wait(sm.full[v.st], v.ph);
              wait(sm.p_full[slot], pph);
              pph ^= 1;
            }
            if (!ok) break;
            if (elect_one()) {
              if (out) {
                const uint64_t d = dv + ((v.st * Sh::kStage) >> 4);
#pragma unroll
                for (int x = 0; x < kTile / 16; ++x) tc5::mma_bf16_ta(o_at, s_at + 8 * x, d + ((x * 2048) >> 4), idesc_o, 1u);
              }
              if (in) {
                const uint64_t d = dk + ((k.st * Sh::kStage) >> 4);
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                  tc5::mma_bf16(s_at, dq + (((x >> 2) * kSub + (x & 3) * 32) >> 4), d + (((x >> 2) * kSub + (x & 3) * 32) >> 4),
                                idesc_s, x > 0);
                tc5::mma_commit(smem_u32(&sm.s_full[slot]));
                tc5::mma_commit(smem_u32(&sm.empty[k.st]));
                if (j + 2 >= pc.nt) tc5::mma_commit(smem_u32(&sm.q_empty));
              } else {
                tc5::mma_commit(smem_u32(&sm.o_full[slot]));
              }
              if (out) tc5::mma_commit(smem_u32(&sm.empty[v.st]));
            }
            if (in) k.move(2);
            if (out) v.move(2);
          }
        }
        qph ^= 1;
        jj += pc.nt;
      }
      if (elect_one()) tc5::mma_commit(smem_u32(&sm.done[slot]));
      tc5::mbar_wait_drain(smem_u32(&sm.done[slot]), 0);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- the units' query rows
      uint32_t n_q = 0;
      bool ok = true;
      if (lane == 0) tc5::prefetch_tmap(&qmap);
      Walk walk;
      walk.init(a, sm.cut);
      Piece pc;
      while (ok && walk.next(a, units, pc)) {
        if (pc.sp.L <= 0) continue;
        const int h = chunks == 1 ? pc.unit : pc.unit / chunks, row0 = (pc.unit - h * chunks) * unit_rows;
        if (n_q > 0) ok = warp_wait(sm.q_empty, (n_q - 1) & 1, abort);
        if (!ok) break;
        // whole tokens' heads: 128 / group tokens to a slot
        const int slots = row0 + rs < qrows ? 2 : 1, tokens = rs / group;
        if (lane == 0) {
          tc5::mbar_expect_tx(smem_u32(&sm.q_full), slots * Sh::kSubs * rs * 128);
          for (int x = 0; x < slots * Sh::kSubs; ++x)
            tma_load_3d(qsm + x * kSub, &qmap, 64 * (x % Sh::kSubs), h * group, pc.b * a.S + row0 / group + x / Sh::kSubs * tokens,
                        smem_u32(&sm.q_full));
        }
        __syncwarp();
        ++n_q;
      }
      if (n_q > 0) tc5::mbar_wait_drain(smem_u32(&sm.q_full), (n_q - 1) & 1);   // landed before the block ends
    }
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  if (warp == kMmaWarp) tc5::tmem_dealloc(tmem, 512);
  if (tid == 0 && sm.abort && a.status) set_status(a.status, kStatusTimeout);
}

// Joins the pieces of the units cut between CTAs: block (x, y, z) does query rows
// 32 y .. of the unit that starts in CTA x and dims 64 z .., a thread a row and eight dims.
// The largest of the pieces' maxima first, then their sums: a piece's loads wait for
// nothing of the piece before, four pieces' are under way (a running maximum took 1 us a
// piece: 52 us for a request of 8000 rows in 38 pieces).
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    tree_join_kernel(const PagedArgs a, int rs, int chunks, const float* __restrict__ part, const PaJoin* __restrict__ joins) {
  constexpr int kDims = 8;
  pdl_wait();
  pdl_trigger();
  const PaJoin j = joins[blockIdx.x];
  if (j.count == 0) return;
  const int lane = threadIdx.x & 31, c0 = blockIdx.z * 64 + (threadIdx.x >> 5) * kDims;
  const int group = a.heads / a.kv_heads, h = j.unit / chunks, r0 = blockIdx.y * 32;
  const int t = (r0 & 127) + lane, i = ((j.unit - h * chunks) * (kRows / 128) + (r0 >> 7)) * rs + t;
  if (t >= rs || i >= a.S * group) return;
  // piece p: the first is what its CTA has last (or alone), the others what theirs have first
  auto piece = [&](int p) {
    const int64_t slot = p == 0 ? (int64_t)blockIdx.x * 2 + j.slot : (int64_t)(blockIdx.x + p) * 2;
    return part + (slot * kRows + r0) * (D + 2) + lane;
  };
  float m = -INFINITY;
  for (int p0 = 0; p0 < j.count; p0 += 8) {
    float v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = p0 + p < j.count ? piece(p0 + p)[D * 32] : -INFINITY;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = fmaxf(m, v[p]);
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[kDims];
#pragma unroll
  for (int x = 0; x < kDims; ++x) acc[x] = 0.f;
  for (int p0 = 0; p0 < j.count; p0 += 4) {
    float v[4][kDims + 2];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float* src = piece(min(p0 + p, j.count - 1));
#pragma unroll
      for (int x = 0; x < kDims; ++x) v[p][x] = src[(c0 + x) * 32];
      v[p][kDims] = src[D * 32];
      v[p][kDims + 1] = src[(D + 1) * 32];
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p0 + p >= j.count) break;
      const float f = exp2f(v[p][kDims] - ref);
      l += v[p][kDims + 1] * f;
#pragma unroll
      for (int x = 0; x < kDims; ++x) acc[x] += v[p][x] * f;
    }
  }
  const int s = i / group, hd = h * group + i - s * group;
  const int64_t tok = (int64_t)j.b * a.S + s;
  const bool any = (l > 0.f || l != l) && (!a.count || s < a.count[j.b]);
  const float inv = any ? 1.f / l : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + tok * a.out_stride + hd * D + c0;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = any ? pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  if (a.lse && c0 == 0) a.lse[tok * a.heads + hd] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// The pool's rows, `width` elements each, copied `seg` rows of 128 bytes at a time.
bool make_pool_map(CUtensorMap* m, const void* ptr, int64_t rows, uint64_t width, uint64_t step, bool fp8, int dim, int seg) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)(rows > 0 ? rows : 1)};
  cuuint64_t strides[1] = {step};
  cuuint32_t box[2] = {fp8 ? 128u : 64u, (cuuint32_t)seg};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            // a head's row is 256 bytes of a bf16 pool of 128 dims, 128 otherwise
            !fp8 && dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries by token, head and 64 dims; a copy takes `group` heads of `tokens` tokens.
bool make_query_map(CUtensorMap* m, const PagedArgs& a, int group, int tokens) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)a.dim, (cuuint64_t)a.heads, (cuuint64_t)a.B * a.S};
  cuuint64_t strides[2] = {(cuuint64_t)a.dim * 2, (cuuint64_t)a.q_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kFp8>
int launch_rows(const PagedArgs& a, int num_sms, cudaStream_t st, bool pdl) {
  using Sh = TtShape<D, kFp8>;
  auto kern = tree_kernel<D, kFp8>;
  static PerDeviceOnce attr;
  if (const cudaError_t e = attr.run([&] {
        // the warpgroups' shares of the registers must add up to what the launch brings
        cudaFuncAttributes fa;
        const cudaError_t q = cudaFuncGetAttributes(&fa, kern);
        if (q != cudaSuccess) return q;
        if (fa.numRegs * kTtThreads < kTtThreads / 2 * (kRegsSoftmax<kFp8> + kRegsOthers<kFp8>)) return cudaErrorLaunchOutOfResources;
        return allow_max_dynamic_smem(kern);
      }))
    return launch_fail("cudaFuncSetAttribute(tree_kernel)", e);
  int seg = kTile;                               // rows of a copy: a power of two that divides a page
  while (a.table && a.block % seg != 0) seg /= 2;
  CUtensorMap kmap, vmap;
  if (!make_pool_map(&kmap, a.k, a.rows, (uint64_t)a.kv_heads * D, a.k_step, kFp8, D, seg) ||
      !make_pool_map(&vmap, a.v, a.rows, (uint64_t)a.kv_heads * D, a.v_step, kFp8, D, seg))
    return launch_fail("cuTensorMapEncodeTiled(K / V pools)", cudaErrorInvalidValue);
  const int group = a.heads / a.kv_heads, qrows = a.S * group, rs = 128 / group * group;
  const int unit_rows = 2 * rs, chunks = (qrows + unit_rows - 1) / unit_rows;
  CUtensorMap qmap;
  if (!make_query_map(&qmap, a, group, rs / group)) return launch_fail("cuTensorMapEncodeTiled(q)", cudaErrorInvalidValue);
  float* part = static_cast<float*>(a.workspace);
  PaJoin* joins = reinterpret_cast<PaJoin*>(part + (size_t)num_sms * 2 * kRows * (D + 2));
  const int64_t tiles = (int64_t)a.B * a.kv_heads * chunks * ((a.max_len + kTile - 1) / kTile + kExtra);
  const int grid = tiles < num_sms ? (int)tiles : num_sms;
  const int r = launch_kernel(kern, dim3(grid), dim3(kTtThreads), Sh::kSmem, st, pdl, qmap, kmap, vmap, a, rs, seg, chunks, a.kv_heads * chunks, part, joins);
  if (r < 0) return r;
  const int most = qrows < rs ? qrows : kRows;
  const int r2 = launch_kernel(tree_join_kernel<D>, dim3(grid, (most + 31) / 32, D / 64), dim3(kJoinThreads), 0, st, pdl, a, rs, chunks,
                               (const float*)part, (const PaJoin*)joins);
  return r2 < 0 ? r2 : r + r2;
}

}  // namespace

// Partials of two pieces per CTA of up to 256 query rows, and the join list (the warps'
// kernel needs less).
size_t tree_attn_workspace(int dim, int num_sms) {
  const size_t wide = dim == 256 ? 0 : (size_t)num_sms * (2 * 256 * (dim + 2) * sizeof(float) + sizeof(PaJoin));
  const size_t warps = paged_attn_workspace(dim, num_sms);
  return wide > warps ? wide : warps;
}

int launch_tree_attn(const PagedArgs& a, bool fp8, int num_sms, cudaStream_t st, bool pdl) {
  const int group = a.heads / a.kv_heads, qrows = a.S * group;
  // a slot takes whole tokens' heads; the coordinates of tokens are ints (a pool's rows are, see run_paged)
  if (a.dim == 256 || group > 128 || (int64_t)a.B * a.S > 0x7fffffff) return launch_paged_attn(a, fp8, num_sms, st, pdl);
  // The warps' kernel reads the rows again for every 32 query rows, this one for 256; a
  // pass over a tile takes about as long there as here (E4M3: 1 / 1.75 of it, the codes
  // need not be converted for it), but joining a request's pieces takes it longer here,
  // 0.4 us a piece, and few requests make many.  Measured, warps / here, us, 128 dims:
  //   query rows                 32         64         128        256
  //   1 x 4000, 4 kv heads       15 / 26    18 / 27    22 / 28    29 / 31
  //   1 x 16000                  22 / 34    27 / 35    39 / 36    63 / 40
  //   4 x 1000                   16 / 18    18 / 18    24 / 20    33 / 23
  //   4 x 4000                   21 / 23    29 / 23    41 / 24    68 / 29
  //   32 x 8192 .. 16384        160 / 150  319 / 152  614 / 157  1202 / 187
  //   E4M3, 1 x 16000            23 / 40    29 / 41    40 / 42    61 / 46
  //   E4M3, 4 x 4000             23 / 28    29 / 28    43 / 30    70 / 34
  //   E4M3, 32 x 8192 .. 16384  152 / 267  293 / 269  557 / 271  1074 / 283
  const int rs = 128 / group * group;
  const int passes = (qrows + 31) / 32, chunks = (qrows + 2 * rs - 1) / (2 * rs);
  const double more = passes - (fp8 ? 1.75 : 1.) * chunks;
  const int64_t span = a.win > 0 && (int64_t)a.win + a.S < a.max_len ? (int64_t)a.win + a.S : a.max_len;
  const double units = (double)a.B * a.kv_heads, tiles = units * ((span + kTile - 1) / kTile);
  if (more <= 0 || more * units * fmax(1., tiles / num_sms) < 30.) return launch_paged_attn(a, fp8, num_sms, st, pdl);
  if (fp8) return launch_rows<128, true>(a, num_sms, st, pdl);
  return a.dim == 64 ? launch_rows<64, false>(a, num_sms, st, pdl) : launch_rows<128, false>(a, num_sms, st, pdl);
}

}  // namespace csa
