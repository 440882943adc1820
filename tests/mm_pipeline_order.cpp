// Runs the product's pipeline (mm_pipeline.h) as a model in which every warp, every copy and every
// MMA may be as late as it likes, with mbarriers that tell a phase by its parity alone, as the
// hardware's do.  Arguments: how many random orders to run per shape, and which mistake is planted to
// see that the model finds it: "none", "stage-first" (in the issuers' walk) or "one-slot-less" (in
// the ring of the scales).
// Prints a line per shape and returns the number of shapes that went wrong.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <random>
#include <vector>

#include "mm_pipeline.h"

using namespace csa;

namespace {

// Pending arrivals of the running phase, and how many phases are over.
struct Bar {
  int count = 1, pending = 1, over = 0;
  void init(int n) { count = pending = n; }
  void arrive() { if (--pending == 0) pending = count, ++over; }
  bool test(uint32_t parity) const { return (uint32_t)(over & 1) != parity; }
};

// The same walk with the stage asked and waited for before the buffer.
template <class Sh>
struct StageFirst : MmIssue<Sh> {
  using MmIssue<Sh>::MmIssue;
  template <class Bars>
  bool ready(Bars& b) {
    if (!this->okf && !b.wait_stage(this->st, this->ph)) return false;
    this->okf = 1;
    return this->okt || b.wait_buffer(this->buf, this->bph ^ 1u);
  }
  template <class Bars>
  void ask(Bars& b) {
    this->okf = b.ask_stage(this->st, this->ph);
    this->okt = this->n < Sh::kBufs ? 1u : b.ask_buffer(this->buf, this->bph ^ 1u);
  }
};

template <class Sh, template <class> class Walk>
struct Model {
  static constexpr int kEpi = 3;                      // epilogue warps (more change nothing)
  static constexpr int kCopiers = Sh::kIssuers == 1 ? 1 : 2;
  std::mt19937 rng;
  int blocks, slots;
  const char* wrong = nullptr;
  Bar full[kMmMaxStages], done[kMmMaxStages], tempty[4];
  int holds[kMmMaxStages];                            // the block whose codes are in the stage, -1: in flux
  int product[4];                                     // the block whose product is in the buffer, -1: in flux
  std::vector<int> scales;                            // the block whose scales the slot is for, from its copy's start
  struct Landing { int block; bool codes; };
  std::vector<Landing> flight;                        // copies asked for and not landed
  struct Copier { int n = 0; } copier[2];
  struct Issuer { Walk<Sh> is; std::deque<int> mmas; bool asked = true; explicit Issuer(int i) : is(i) {} };
  std::vector<Issuer> issuer;
  struct Epilogue { int n = 0; bool late = false; } epi[kEpi];

  // what an issuer sees of the barriers: a wait that is not over is a step not taken
  bool wait_stage(int i, uint32_t p) { return full[i].test(p); }
  bool wait_buffer(int i, uint32_t p) { return tempty[i].test(p); }
  uint32_t ask_stage(int i, uint32_t p) { return full[i].test(p); }
  uint32_t ask_buffer(int i, uint32_t p) { return tempty[i].test(p); }

  Model(unsigned seed, int n, int ring) : rng(seed), blocks(n), slots(ring), scales(ring, -1) {
    for (Bar& b : full) b.init(2);                    // the codes and the scales
    for (Bar& b : tempty) b.init(kEpi);
    for (int i = 0; i < Sh::kIssuers; ++i) issuer.emplace_back(i);
    for (int& x : holds) x = -1;
    for (int& x : product) x = -1;
  }

  void copy(int who) {                                // the codes' warp, the scales' warp (or both in one)
    const int n = copier[who].n;
    if (n >= blocks) return;
    const int st = n % Sh::kStages;
    if (n >= Sh::kStages && !done[st].test((n / Sh::kStages & 1) ^ 1)) return;
    if (who == 0) {
      for (const Issuer& i : issuer)
        for (int m : i.mmas)
          if (m % Sh::kStages == st) wrong = "codes written under a running MMA";
      holds[st] = -1;
      flight.push_back({n, true});
    }
    if (who == kCopiers - 1) {
      scales[n % slots] = n;
      flight.push_back({n, false});
    }
    ++copier[who].n;
  }
  void land() {
    if (flight.empty()) return;
    const size_t i = rng() % flight.size();
    const Landing x = flight[i];
    flight.erase(flight.begin() + i);
    if (x.codes) holds[x.block % Sh::kStages] = x.block;
    full[x.block % Sh::kStages].arrive();
  }
  void issue(int who) {
    Issuer& i = issuer[who];
    if (!i.asked) {                                   // between two of the block's MMAs
      i.is.ask(*this);
      i.asked = true;
      return;
    }
    if (i.is.n >= blocks || !i.is.ready(*this)) return;
    if (holds[i.is.st] != i.is.n) wrong = "MMAs on a stage that does not hold their block";
    for (const Epilogue& e : epi)
      if (e.n + e.late <= i.is.n - Sh::kBufs) wrong = "MMAs into a buffer that has not been read";
    i.mmas.push_back(i.is.n);
    product[i.is.buf] = -1;
    i.is.next();
    i.asked = false;
  }
  void finish(int who) {
    Issuer& i = issuer[who];
    if (i.mmas.empty()) return;
    const int n = i.mmas.front();
    i.mmas.pop_front();
    product[n % Sh::kBufs] = n;
    done[n % Sh::kStages].arrive();
  }
  void read(int who) {
    Epilogue& e = epi[who];
    if (e.n >= blocks) return;
    if (e.late) {                                     // scales may be read after the buffer is given back
      if (scales[e.n % slots] != e.n) wrong = "scales read that are another block's";
      e.late = false;
      ++e.n;
      return;
    }
    if (!done[e.n % Sh::kStages].test(e.n / Sh::kStages & 1)) return;
    if (product[e.n % Sh::kBufs] != e.n) wrong = "a product read that is not its block's";
    tempty[e.n % Sh::kBufs].arrive();
    e.late = true;
  }

  const char* run() {
    // how often each actor gets a turn: some almost never, for a while
    const int actors = kCopiers + 1 + 2 * Sh::kIssuers + kEpi;
    std::vector<int> weight(actors);
    for (int turn = 0; turn < 400 * blocks && !wrong; ++turn) {
      if (turn % 64 == 0)
        for (int& w : weight) w = rng() % 4 == 0 ? 1 : 1 + rng() % 40;
      int all = 0;
      for (int w : weight) all += w;
      int x = rng() % all, a = 0;
      while (x >= weight[a]) x -= weight[a++];
      if (a < kCopiers) { copy(a); continue; }
      a -= kCopiers;
      if (a == 0) { land(); continue; }
      a -= 1;
      if (a < Sh::kIssuers) { issue(a); continue; }
      a -= Sh::kIssuers;
      if (a < Sh::kIssuers) { finish(a); continue; }
      read(a - Sh::kIssuers);
    }
    // every block goes through in the end
    for (int turn = 0; turn < 100 * blocks && !wrong; ++turn) {
      for (int i = 0; i < kCopiers; ++i) copy(i);
      land();
      for (int i = 0; i < Sh::kIssuers; ++i) issue(i), finish(i);
      for (int i = 0; i < kEpi; ++i) read(i), read(i);
    }
    for (const Epilogue& e : epi)
      if (!wrong && e.n != blocks) wrong = "a block that never came through";
    return wrong;
  }
};

template <class Sh, template <class> class Walk>
int check(const char* name, int orders, int less) {
  const char* wrong = nullptr;
  int at = -1;
  for (int i = 0; i < orders && !wrong; ++i) {
    Model<Sh, Walk> m(1000003u * i + 17, 3 + i % 60, Sh::kSlots - less);
    wrong = m.run();
    at = i;
  }
  std::printf("%s: stages %d, buffers %d, issuers %d, slots %d: %s", name, Sh::kStages, Sh::kBufs, Sh::kIssuers, Sh::kSlots - less,
              wrong ? wrong : "ok");
  if (wrong) std::printf(" (order %d)", at);
  std::printf("\n");
  return wrong != nullptr;
}

template <template <class> class Walk>
int all(int orders, int less) {
  return check<MmShape<16, true>, Walk>("16 swapped", orders, less) + check<MmShape<32, true>, Walk>("32 swapped", orders, less) +
         check<MmShape<64, true>, Walk>("64 swapped", orders, less) + check<MmShape<128, false>, Walk>("128", orders, less) +
         check<MmShape<256, false>, Walk>("256", orders, less);
}

}  // namespace

int main(int argc, char** argv) {
  const int orders = argc > 1 ? std::atoi(argv[1]) : 1000;
  const char* mistake = argc > 2 ? argv[2] : "none";
  return !std::strcmp(mistake, "stage-first") ? all<StageFirst>(orders, 0)
                                              : all<MmIssue>(orders, !std::strcmp(mistake, "one-slot-less"));
}
