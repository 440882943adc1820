// What the kernels over paged K / V pools share: the spans of the requests, the
// list of tiles and its cuts between the CTAs.
#pragma once

#include <limits>

#include "csa_internal.cuh"
#include "ptx.cuh"

namespace csa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

using PaCost = uint32_t;  // of the units of one kv head and chunk of as many requests as a block has threads

// What a CTA leaves for the join of the unit that starts in it and goes on in
// the next CTAs (count = 0: none).
struct PaJoin {
  int count;         // CTAs that hold a piece
  int slot;          // the first piece's slot in this CTA (0 or 1)
  int b, unit;
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Four E4M3 codes (low byte first) to two f16x2: every E4M3 value is an f16 value.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// Tiles of a request (at least one, so that every unit is visited and
// written): the rows any of its S queries sees are [lo, L).
// A tree's request has n of them, and none with a bad count.
template <int kTile, bool kTree>
struct Span {
  int L, lo, t0, tiles, n;
  __device__ __forceinline__ void set(const PagedArgs& a, int b) {
    const int len = a.ctx_len[b];
    L = len < 0 || len > a.max_len ? 0 : len;  // a bad length reads nothing
    n = a.S;
    if (kTree && a.count) {
      n = a.count[b];
      if (n <= 0 || n > a.S) L = 0;
    }
    const int p0 = L - n;
    lo = a.win > 0 && p0 - a.win + 1 > 0 ? p0 - a.win + 1 : 0;
    t0 = lo / kTile;
    tiles = (L + kTile - 1) / kTile - t0;
    if (tiles < 1) tiles = 1;
  }
};

// Position in the list of tiles: request b, unit (kv head, chunk), tile.
template <int kTile, bool kTree>
struct Cursor {
  int b, unit, tile;
  Span<kTile, kTree> sp;
  __device__ __forceinline__ void next(const PagedArgs& a, int units) {
    if (++tile < sp.tiles) return;
    tile = 0;
    if (++unit < units) return;
    unit = 0;
    if (++b < a.B) sp.set(a, b);
  }
};

// Whether draft s of request b sees draft t of its tree.
__device__ __forceinline__ bool tree_sees(const PagedArgs& a, int b, int s, int t) {
  return (a.tree[((int64_t)b * a.S + s) * a.words + (t >> 6)] >> (t & 63)) & 1;
}
// The last rows of the window before draft s of request b: rows up to this one are outside it
// (p: the request's first draft's row, n: its drafts).
__device__ __forceinline__ int tree_outside(const PagedArgs& a, int b, int s, int p, int n) {
  if (a.win == 0) return -1;
  const int at = a.tpos[(int64_t)b * a.S + s];
  return min(max(at, p), p + n - 1) - a.win;
}

// A cut of the list of tiles: before this tile of this unit.
struct Cut {
  int b, unit, tile;
  int64_t first, at;   // the unit's start in the list of costs, the tiles before the cut
};

// i * total / parts (a 32-bit division where that holds it).
__device__ __forceinline__ int64_t split_at(int64_t total, int i, int parts) {
  const int64_t x = total * i;
  return x < (int64_t(1) << 32) ? (int64_t)((uint32_t)x / (uint32_t)parts) : x / parts;
}

// The CTA's share of the list of units (request, kv head, chunk of query rows): of the
// costs (a unit's tiles and kExtra more for its start and end), with the cuts moved to
// the next whole tile.  total: the list's cost, G: the CTAs that share it.  False: no
// share.  Contains barriers; cut_sh is ready after it.  The lengths are scanned by the
// first kThreads threads of the block, kThreads requests at a time.
template <int kTile, bool kTree, int kThreads, int kExtra>
__device__ __forceinline__ bool paged_cuts(const PagedArgs& a, int units, PaCost* scan_tmp, Cut* cut_sh, int64_t& total,
                                           int64_t& G) {
  // the costs of a block's scan (a request per thread) add up in 32 bits
  static_assert((uint64_t)kThreads * (kPagedMaxLen / kTile + 1 + kExtra) <= std::numeric_limits<PaCost>::max(), "sum of costs");
  const int tid = threadIdx.x;
  const bool once = a.B <= kThreads;   // one request per thread: scanned once
  const int end = tid < kThreads ? a.B : 0;
  Span<kTile, kTree> sp;
  PaCost n = 0, sum, ahead = 0;
  int len = 0;
  total = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    n = 0;
    if (b0 + tid < end) len = a.ctx_len[b0 + tid], sp.set(a, b0 + tid), n = sp.tiles + kExtra;
    ahead = block_exclusive_scan(n, scan_tmp, &sum);
    total += sum;
  }
  total *= units;
  G = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= G) return false;
  const int64_t cut[2] = {split_at(total, blockIdx.x, (int)G), split_at(total, blockIdx.x + 1, (int)G)};
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    if (!once) {
      n = 0;
      if (b0 + tid < end) len = a.ctx_len[b0 + tid], sp.set(a, b0 + tid), n = sp.tiles + kExtra;
      ahead = block_exclusive_scan(n, scan_tmp, &sum);
    }
    if (blockIdx.x == 0 && a.status && b0 + tid < end &&
        (len < 0 || len > a.max_len || (kTree && a.count && (sp.n < 0 || sp.n > a.S))))
      set_status(a.status, kStatusBadIndex);
    const int64_t p = (before + (int64_t)ahead) * units;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      // (the list's end belongs to its last request)
      if (n > 0 && p <= cut[e] && (cut[e] < p + (int64_t)n * units || b0 + tid == a.B - 1)) {
        const int64_t at = cut[e] - p;
        const int unit = at < (1u << 31) ? (int)((uint32_t)at / n) : (int)(at / n);
        const int x = (int)(at - (int64_t)unit * n);
        cut_sh[e].b = b0 + tid;
        cut_sh[e].unit = unit;
        cut_sh[e].tile = x > kExtra ? x - kExtra : 0;
        cut_sh[e].first = p + (int64_t)unit * n;
        // tiles before it in the whole list
        cut_sh[e].at = p - (int64_t)(b0 + tid) * units * kExtra + (int64_t)unit * sp.tiles + cut_sh[e].tile;
      }
    before += sum;
  }
  __syncthreads();
  return true;
}

}  // namespace csa
