// The product's pipeline without its device code: the shapes, and an issuer's
// way through the barriers.  Plain C++, so that the order of the waits can be
// run against every order of the other warps on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CSA_MM_FN __device__ __forceinline__
#else
#define CSA_MM_FN inline
#endif

namespace csa {

constexpr int kMmBlock = 128;                 // codes per scale, bytes per stage row
constexpr int kMmPBytes = 128 * kMmBlock;     // P tile: 128 rows
constexpr int kMmMaxStages = 12;

template <int NT, bool kSwap>
struct MmShape {
  // 64 sums per epilogue thread at most; with 256 columns sixteen warps, four
  // per scheduler, hide each other's TMEM reads
  static constexpr int kEpiWarps = kSwap ? 4 : NT == 256 ? 16 : 8;
  static constexpr int kAux = kSwap ? 2 : 4;               // warps before the epilogue's
  static constexpr int kIssuers = kSwap ? 1 : 2;
  static constexpr int kThreads = 32 * (kAux + kEpiWarps);
  static constexpr int kCols = NT / (kEpiWarps / 4);       // columns per epilogue thread
  static constexpr int kChunk = kSwap || NT == 256 ? 16 : 32;  // columns per TMEM read
  static constexpr int kAccCols = NT < 32 ? 32 : NT;       // TMEM columns per buffer
  static constexpr int kBufs = kSwap || NT == 128 ? 4 : 2;
  static constexpr int kTmemCols = kAccCols * kBufs;
  static constexpr int kStageBytes = kMmPBytes + NT * kMmBlock;
  static constexpr int kCtasPerSm = kSwap ? 2 : 1;
  // !kSwap: a patch per epilogue warp, through which the output leaves in
  // 32- or 128-byte pieces of a row
  static constexpr int kLine = NT == 256 ? 32 : 128;
  static constexpr int kPatchBytes = kSwap ? 0 : kEpiWarps * 32 * kLine;
  // scales: per block the a scales of the tile's rows of a (padded to 128) and
  // the b scales of its 128-row parts
  static constexpr int kScaleFloats = 128 + 4;
  static constexpr int kRoom = (kSwap ? 113 * 1024 : 227 * 1024) - 1024 - 1024 - kPatchBytes;
  static constexpr int kFit = (kRoom - (kBufs + 1) * kScaleFloats * 4) / (kStageBytes + kScaleFloats * 4);
  static constexpr int kStages = kFit > kMmMaxStages ? kMmMaxStages : kFit;
  // Block n's scales lie in slot n % kSlots and may be read until block n + 1's
  // buffer is given back (kSwap: the last chunk's after block n's own is).  The
  // slot's next copy, block n + kSlots, follows done(n + kBufs + 1), whose MMAs
  // waited for that buffer.
  static constexpr int kSlots = kStages + kBufs + 1;
  static constexpr int kSmem = kStages * kStageBytes + kPatchBytes + kSlots * kScaleFloats * 4 + 1024;
  // fp32 sums of the tile in the ring's memory, laid out like the output: rows
  // of kSumCols neighbouring columns of out, the pitch chosen so that neither
  // the writes nor the reads conflict
  static constexpr int kSumRows = kSwap ? NT : 128, kSumCols = kSwap ? 128 : NT;
  static constexpr int kPitch = kSumCols * 4 + (kSwap ? 0 : 16);
  static_assert(kSumRows * kPitch <= kStages * kStageBytes, "sums exceed the ring");
  static_assert(kSmem + 1024 <= (kSwap ? 113 : 227) * 1024, "shared memory");
  static_assert(kStages <= kMmMaxStages && kTmemCols <= 512 / kCtasPerSm, "ring or TMEM");
  // a buffer belongs to one issuer, and no stage comes round before the product
  // of its last block has been read (see MmIssue)
  static_assert(kBufs % kIssuers == 0 && kStages >= kBufs, "the issuers' order");
};

// One of the threads that issue MMAs: blocks which, which + kIssuers, ..; block
// n from stage n % kStages into TMEM buffer n % kBufs.  A parity tells a phase
// only from its neighbours, so a barrier may be asked for a phase only when the
// phase before it is known to be over.  A buffer is always the same issuer's:
// its phase before is one that this thread waited for.  A stage's last block,
// n - kStages, may be another issuer's, and it is the buffer that vouches for
// it: block n - kBufs has been read by every epilogue warp, which takes the
// blocks in order and so has waited for done(n - kStages), kStages >= kBufs.
// So the buffer is asked and waited for first, and an answer of the stage
// counts only with a buffer's answer before it.
template <class Sh>
struct MmIssue {
  int st, buf, n;
  uint32_t ph = 0, bph = 0;
  uint32_t okf = 0, okt = 1;   // answers for block n: its codes are there, its buffer is free
  CSA_MM_FN explicit MmIssue(int which) : st(which), buf(which), n(which) {}
  // Waits until block n may be issued; false when a wait gave up.
  template <class Bars>
  CSA_MM_FN bool ready(Bars& b) {
    if (!okt && !b.wait_buffer(buf, bph ^ 1u)) return false;
    okt = 1;
    return okf || b.wait_stage(st, ph);
  }
  CSA_MM_FN void next() {
    if ((st += Sh::kIssuers) >= Sh::kStages) st -= Sh::kStages, ph ^= 1u;
    if ((buf += Sh::kIssuers) >= Sh::kBufs) buf -= Sh::kBufs, bph ^= 1u;
    n += Sh::kIssuers;
  }
  // Asks for the block that ready() will be called for, without waiting.
  template <class Bars>
  CSA_MM_FN void ask(Bars& b) {
    okt = n < Sh::kBufs ? 1u : b.ask_buffer(buf, bph ^ 1u);
    okf = b.ask_stage(st, ph) & okt;
  }
};

}  // namespace csa
