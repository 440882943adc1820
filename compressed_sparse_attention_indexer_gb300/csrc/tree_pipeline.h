// The ring of tree_kernel without its device code: how many stages it has, and the ways of
// the warps through it.  Plain C++, so that their order can be run against every order
// of copies, products and warps on the host.
//
// Chunk 2 t is K, chunk 2 t + 1 V of a block's tile t, across its pieces.  Chunk c lies in
// stage c % N, in the stage's phase c / N.  A parity tells a phase only from its
// neighbours, so a barrier may be asked for a phase only when the phase before it is known
// to be over: both slots' MMA warps wait for every chunk, in order, and give it back, a slot
// without rows too, and a softmax warp asks for a V only after the scores of its tile.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CSA_TREE_FN __host__ __device__ __forceinline__
#else
#define CSA_TREE_FN inline
#endif

namespace csa {

// Stages of the ring (E4M3: rows as bf16; their codes land in kTreeRaw chunks beside it).
constexpr int tree_stages(int dim, bool fp8) { return fp8 ? 3 : dim == 64 ? 8 : 5; }
constexpr int kTreeRaw = 3;
// Tiles whose E4M3 scales are held.  A tile's stay until its weights are made: its V then
// waits in the ring, so that the tile being written is at most N / 2 + 1 tiles ahead.
constexpr int kTreeScales = 8;

// A chunk's stage and the parity of its phase, moved on by up to N chunks at a time.
template <int N>
struct TreePlace {
  uint32_t st = 0, ph = 0;
  CSA_TREE_FN void set(uint32_t chunk) { st = chunk % N, ph = (chunk / N) & 1; }
  CSA_TREE_FN void move(uint32_t by) {
    st += by;
    if (st >= N) st -= N, ph ^= 1;
  }
};

// The loader's way through its N places (the ring's, or the codes').  A chunk lands on the
// place's barrier, or (`other`) on a second one that it has.
template <int N>
struct TreeFeed {
  uint32_t at = 0, ph = 1;            // the place, the parity of its empty barrier's phase before
  bool again = false;                 // a chunk has been there
  uint32_t others = 0, turns = 0;     // bit i: place i's last chunk was the other barrier's; that one's phases, modulo 2
  CSA_TREE_FN void next(bool other) {
    others = other ? others | 1u << at : others & ~(1u << at);
    turns ^= other ? 1u << at : 0u;
    if (++at == N) at = 0, ph ^= 1, again = true;
  }
  // The barrier and the parity of the phase in which place i's last chunk lands; false
  // when it had none.  The chunks before have landed, or the place would not have been free.
  CSA_TREE_FN bool last(uint32_t i, bool& other, uint32_t& parity) const {
    other = (others >> i) & 1;
    parity = other ? ((turns >> i) & 1) ^ 1 : i < at ? ph ^ 1 : ph;
    return again || i < at;
  }
};

}  // namespace csa
