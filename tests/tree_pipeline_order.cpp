// Runs the order of csrc/tree_pipeline.h against random orders of the warps that share the ring: copies that
// land late and out of order, row warps in between, two issuers and two softmaxes.  Barriers are modelled as
// the hardware has them, a phase counter whose parity alone is asked for.  Checks that every product reads the
// chunk it means (one that was overwritten too soon does not), and that every order comes to its end.
#include <stdio.h>
#include <stdlib.h>

#include <random>
#include <vector>

#include "tree_pipeline.h"

struct Bar {
  int count, pending, phase = 0;
  explicit Bar(int c) : count(c), pending(c) {}
  void arrive() {
    if (--pending == 0) pending = count, ++phase;
  }
  // test_wait.parity: the phase before the current one has this parity
  bool done(int parity) const { return (phase & 1) != parity; }
};

template <bool kTurns, int kStages>
int run(const std::vector<int>& pieces, bool converted, unsigned seed) {
  using Ring = csa::TreeRing<kTurns, kStages>;
  std::mt19937 rng(seed);
  std::vector<Bar> full(kStages, Bar(1)), empty(kStages, Bar(kTurns ? 1 : 2)), p_full(2, Bar(1)), s_full(2, Bar(1));
  std::vector<long> held(kStages, -1);                        // chunk id in a stage
  std::vector<long> flying;                                   // (stage, id) pairs on their way
  std::vector<int> fly_stage;
  auto id = [](int piece, int j, bool v) { return ((long)piece * 100000 + j) * 2 + (v ? 1 : 0); };

  // the copier
  int lp = 0, lm = 0;
  Ring lr;
  lr.start();
  // issuers: piece, step within it, what they wait for
  struct Issuer {
    int piece = 0, j = 0, stage_of = 0, pph = 0, idle = 0;
    bool fresh = true;
    Ring ring;
  } is[2];
  struct Soft {
    int todo = 0, done = 0;
  } soft[2];
  for (auto& x : is) x.ring.start();
  const int P = (int)pieces.size();
  long steps = 0, stuck = 0;
  auto slot_tiles = [&](int nt, int s) { return kTurns ? (s ? nt / 2 : (nt + 1) / 2) : nt; };
  while (is[0].piece < P || is[1].piece < P) {
    if (++steps > 4000000 || stuck > 20000) return fprintf(stderr, "stuck: pieces %d %d\n", is[0].piece, is[1].piece), 1;
    ++stuck;
    switch (rng() % 6) {
      case 0: {                                               // a copy is issued
        if (lp >= P) break;
        bool v;
        const int j = Ring::tile_of(lm, pieces[lp], v);
        const auto at = lr.at(j, v);
        if (at.c >= (uint32_t)Ring::kPer && !empty[at.st].done(at.ph ^ 1)) break;
        held[at.st] = -2;
        flying.push_back(id(lp, j, v));
        fly_stage.push_back(at.st);
        if (++lm == 2 * pieces[lp]) lr.after(pieces[lp]), lm = 0, ++lp;
        stuck = 0;
        break;
      }
      case 1: {                                               // some copy lands (converted: in order)
        if (flying.empty()) break;
        const size_t k = converted ? 0 : rng() % flying.size();
        held[fly_stage[k]] = flying[k];
        full[fly_stage[k]].arrive();
        flying.erase(flying.begin() + k);
        fly_stage.erase(fly_stage.begin() + k);
        stuck = 0;
        break;
      }
      case 2: case 3: {                                       // an issuer
        const int s = rng() % 2;
        Issuer& x = is[s];
        if (x.piece >= P) break;
        const int nt = pieces[x.piece], mine = slot_tiles(nt, s), step = Ring::kStep, first = kTurns ? s : 0;
        if (x.fresh) x.j = first - step, x.fresh = false;
        if (mine == 0) {
          x.ring.after(nt), ++x.piece, x.fresh = true, stuck = 0;
          break;
        }
        const bool out = x.j >= first, in = x.j + step < nt;
        auto landed = [&](int j, bool v) { const auto at = x.ring.at(j, v); return full[at.st].done(at.ph); };
        if (in && !landed(x.j + step, false)) break;
        if (out && (!landed(x.j, true) || !p_full[s].done(x.pph & 1))) break;
        auto use = [&](int j, bool v) {
          const auto at = x.ring.at(j, v);
          if (held[at.st] != id(x.piece, j, v)) {
            fprintf(stderr, "slot %d reads %ld for %ld\n", s, held[at.st], id(x.piece, j, v));
            return false;
          }
          empty[at.st].arrive();
          return true;
        };
        if (out) {
          ++x.pph;
          if (!use(x.j, true)) return 1;
        }
        if (in) {
          if (!use(x.j + step, false)) return 1;
          s_full[s].arrive();
          ++soft[s].todo;
        }
        x.j += step;
        if (x.j >= nt) x.ring.after(nt), ++x.piece, x.fresh = true;
        stuck = 0;
        break;
      }
      default: {                                              // a softmax
        const int s = rng() % 2;
        if (soft[s].done < soft[s].todo) ++soft[s].done, p_full[s].arrive(), stuck = 0;
      }
    }
  }
  return lp == P && flying.empty() ? 0 : (fprintf(stderr, "copies left\n"), 1);
}

int main() {
  std::mt19937 rng(7);
  for (int it = 0; it < 3000; ++it) {
    std::vector<int> pieces;
    for (int n = 1 + rng() % 6; n > 0; --n) pieces.push_back(1 + (rng() % 3 ? rng() % 4 : rng() % 40));
    const unsigned s = rng();
    if (run<true, 4>(pieces, true, s) || run<true, 6>(pieces, false, s) || run<true, 8>(pieces, false, s) || run<false, 3>(pieces, true, s) ||
        run<false, 5>(pieces, false, s) || run<false, 8>(pieces, false, s))
      return 1;
  }
  // the chunks of a piece: each once, V and K where they are looked for
  for (int nt = 1; nt < 60; ++nt) {
    std::vector<int> seen(2 * nt, 0);
    for (int m = 0; m < 2 * nt; ++m) {
      bool v;
      const int j = csa::TreeRing<true, 6>::tile_of(m, nt, v);
      if (j < 0 || j >= nt || seen[2 * j + v]++) return 2;
      if (!v && m + 1 != csa::TreeRing<true, 6>::upto_k(j + 1) && nt > 1) return 3;
      const int k = csa::TreeRing<false, 5>::tile_of(m, nt, v);
      if (k != m / 2 || v != (m & 1) || (!v && m + 1 != csa::TreeRing<false, 5>::upto_k(k + 1))) return 4;
    }
  }
  printf("ok\n");
  return 0;
}
