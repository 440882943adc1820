// The order in which tree_kernel's rows travel: a piece's chunks (K and V of its nt tiles of
// 128 rows) through the ring of stages.  Host and device (a host test runs it against
// random orders of the other warps).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CSA_HD __host__ __device__ __forceinline__
#else
#define CSA_HD inline
#endif

namespace csa {

// The slots share the tiles (kTurns = false: one ring of kStages, a stage is given back by
// both), or take them in turn (a ring of kStages / 2 for each): every full barrier is waited
// for by those alone that give its stage back, phase by phase.  (With one ring for
// slots in turn, a warp could wait for a stage's phase before the other slot's had come, or
// after it was gone, and take another phase's parity for it.)
template <bool kTurns, int kStages>
struct TreeRing {
  static constexpr int kPer = kTurns ? kStages / 2 : kStages;   // stages of a ring
  static constexpr int kStep = kTurns ? 2 : 1;                  // from one tile of a slot to its next

  // Chunks are copied in the order in which they are used: a batch of MMAs takes V of a slot's tile and
  // K of its next.  Tile and kind of a piece's chunk m < 2 nt.
  static CSA_HD int tile_of(int m, int nt, bool& v) {
    if (!kTurns || m + 1 == 2 * nt) {
      v = m & 1;
      return m >> 1;
    }
    v = m >= 2 && !(m & 1);
    return m < 2 ? m : v ? (m - 2) >> 1 : (m + 1) >> 1;
  }
  // Chunks of a piece up to and with the last K of its first `tiles` tiles.
  static CSA_HD int upto_k(int tiles) { return kTurns ? (tiles < 3 ? tiles : 2 * tiles - 2) : 2 * tiles - 1; }

  // Chunks that went through the rings before the piece.
  uint32_t base[2];
  CSA_HD void start() { base[0] = base[1] = 0; }
  CSA_HD void after(int nt) {
    base[0] += kTurns ? 2 * ((nt + 1) / 2) : 2 * nt;
    if (kTurns) base[1] += 2 * (nt / 2);
  }
  // The place of tile j's K or V: its number in its ring, stage and phase.
  struct Place {
    uint32_t c, st, ph;
  };
  CSA_HD Place at(int j, bool v) const {
    const int slot = kTurns ? j & 1 : 0;
    Place p;
    p.c = base[slot] + 2 * (kTurns ? j >> 1 : j) + (v ? 1 : 0);
    p.st = slot * kPer + p.c % kPer;
    p.ph = (p.c / kPer) & 1;
    return p;
  }
};

}  // namespace csa
