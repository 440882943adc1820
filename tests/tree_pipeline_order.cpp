// Runs the ring of csa_tree_attn's tcgen05 kernel (tree_pipeline.h) as a model in which every warp, every copy
// and every product may be as late as it likes, with mbarriers that tell a phase by its parity alone, as the
// hardware's do.  The warps are the kernel's, wait for wait: the loader, E4M3's converters or bf16's readers of V,
// the queries' warp, two MMA warps, two slots' softmax warps.  In half of the orders a wait gives up at some point, as
// one that ran out does, and the others' after it: nothing may be under way when the last warp is gone.  Arguments:
// how many random orders to run per shape, and which mistake is planted to see that the model finds it (see main).
// Prints a line per shape and returns the number of shapes that went wrong.
#include <coroutine>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <exception>
#include <functional>
#include <random>
#include <vector>

#include "tree_pipeline.h"

using namespace csa;

namespace {

// Pending arrivals and bytes (here: copies) of the running phase, and how many phases are over.
struct Bar {
  int count = 1, pending = 1, tx = 0, over = 0;
  void init(int n) { count = pending = n; }
  void arrive() { --pending, turn(); }
  void expect(int n) { tx += n, arrive(); }
  void landed() { --tx, turn(); }
  void turn() { if (pending == 0 && tx == 0) pending = count, ++over; }
  bool test(uint32_t parity) const { return (uint32_t)(over & 1) != parity; }
};

struct Plan {
  const char* mistake = "none";
  bool is(const char* what) const { return !std::strcmp(mistake, what); }
};

// A warp: a coroutine that stops where the kernel's waits or may be overtaken.
struct Warp {
  struct promise_type {
    Warp get_return_object() { return {std::coroutine_handle<promise_type>::from_promise(*this)}; }
    std::suspend_always initial_suspend() noexcept { return {}; }
    std::suspend_always final_suspend() noexcept { return {}; }
    void return_void() {}
    void unhandled_exception() { std::terminate(); }
    std::function<bool()> until;               // what it waits for; empty: it may go on
    bool may_give_up = false, seen = true;
  };
  std::coroutine_handle<promise_type> h;
  bool done() const { return h.done(); }
  // give_up: whether a wait that is not over gives up
  bool step(bool give_up) {
    if (h.done()) return false;
    promise_type& p = h.promise();
    p.seen = !p.until || p.until();
    if (!p.seen && !(give_up && p.may_give_up)) return false;
    p.until = nullptr;
    h.resume();
    return true;
  }
};
struct Until {
  std::function<bool()> f;
  bool may_give_up = false;
  Warp::promise_type* p = nullptr;
  bool await_ready() { return false; }
  void await_suspend(std::coroutine_handle<Warp::promise_type> h) {
    p = &h.promise();
    p->until = f, p->may_give_up = may_give_up;
  }
  bool await_resume() { return p->seen; }
};

template <int ST, bool kFp8>
struct Model {
  static constexpr int kRowWarps = 4, kSoftmax = 2;     // a slot's softmax warps (more change nothing)
  static constexpr int kParts = 2;                      // copies of a chunk
  static constexpr int kPlaces = kFp8 ? kTreeRaw : ST;
  struct Piece { int nt; bool rows[2], empty; std::vector<bool> edge; };

  std::mt19937 rng;
  Plan plan;
  int scale_slots;
  const char* wrong = nullptr;
  std::vector<Piece> pieces;
  Bar full[ST], empty[ST], land[ST], raw_full[kTreeRaw], raw_empty[kTreeRaw], sc_full[kTreeScales];
  Bar s_full[2], p_full[2], o_full[2], q_full, q_empty;
  int stage[ST][kRowWarps], bad[ST][kRowWarps];         // the chunk whose quarter is there, looked through
  int raw[kTreeRaw][kParts], scales[kTreeScales][kRowWarps], q_holds[2];
  int scores[2] = {-1, -1}, weights[2][kSoftmax], output[2] = {-1, -1}, added[2] = {0, 0}, reading[2] = {0, 0};
  int taken[2][kSoftmax] = {{-1, -1}, {-1, -1}};        // the piece whose output a warp has read
  struct Copy { Bar* bar; std::function<void()> write; };
  std::vector<Copy> flight;
  struct Batch { int slot, piece, v = -1, k = -1, tile = -1; bool last = false; std::vector<Bar*> commits; };
  std::deque<Batch> pipe[2];
  std::vector<Warp> warps;

  void fault(const char* what) { if (!wrong) wrong = what; }
  Until see(Bar& b, uint32_t parity) { return {[&b, parity] { return b.test(parity); }, true}; }
  Until drain(Bar& b, uint32_t parity) { return {[&b, parity] { return b.test(parity); }}; }
  long patience = -1;                                   // the turn from which on a wait gives up; -1: none does
  bool abort = false;
  Until pause() { return {}; }

  Model(unsigned seed, Plan p) : rng(seed), plan(p) {
    scale_slots = plan.is("few-scales") ? ST / 2 : kTreeScales;
    for (int n = 1 + rng() % 7; n > 0; --n) {
      Piece x;
      x.nt = 1 + (rng() % 4 ? rng() % 5 : rng() % 24);
      x.empty = rng() % 8 == 0;                         // a padding request: nobody's
      x.rows[0] = true, x.rows[1] = rng() % 2;
      for (int j = 0; j < x.nt; ++j) x.edge.push_back(rng() % 3 == 0);
      pieces.push_back(x);
    }
    for (int i = 0; i < ST; ++i) {
      full[i].init(kFp8 ? kRowWarps : 1), empty[i].init(plan.is("one-slot") ? 1 : 2), land[i].init(1);
      for (int w = 0; w < kRowWarps; ++w) stage[i][w] = bad[i][w] = -1;
    }
    for (int i = 0; i < kTreeRaw; ++i) raw_full[i].init(1), raw_empty[i].init(kRowWarps), raw[i][0] = raw[i][1] = -1;
    for (int i = 0; i < kTreeScales; ++i)
      for (int w = 0; w < kRowWarps; ++w) scales[i][w] = -1;
    for (Bar& b : sc_full) b.init(kRowWarps);
    for (Bar& b : p_full) b.init(kSoftmax);
    q_empty.init(2);
    q_holds[0] = q_holds[1] = -1;
    for (auto& s : weights) for (int& x : s) x = -1;
    warps.push_back(loader());
    for (int w = 0; w < kRowWarps; ++w) warps.push_back(kFp8 ? converter(w) : reader(w));
    warps.push_back(queries());
    for (int s = 0; s < 2; ++s) {
      warps.push_back(issuer(s));
      for (int w = 0; w < kSoftmax; ++w) warps.push_back(softmax(s, w));
    }
  }
  ~Model() { for (Warp& w : warps) w.h.destroy(); }

  bool holds(int st, int chunk) const {
    for (int x : stage[st]) if (x != chunk) return false;
    return true;
  }

  Warp loader() {
    TreeFeed<kPlaces> feed;
    int chunk = 0;
    bool ok = true;
    for (const Piece& p : pieces) {
      if (p.empty) continue;
      for (int c = 0; ok && c < 2 * p.nt; ++c, ++chunk) {
        const uint32_t at = feed.at;
        if (feed.again) ok = co_await see(kFp8 ? raw_empty[at] : empty[at], feed.ph);
        if (!ok) break;
        const bool look = !kFp8 && c % 2 && p.edge[c / 2];
        Bar& bar = kFp8 ? raw_full[at] : look ? land[at] : full[at];
        bar.expect(kParts);
        for (int x = 0; x < kParts; ++x)
          flight.push_back({&bar, [this, at, x, chunk] {
            if (kFp8) raw[at][x] = chunk;
            else for (int w = x; w < kRowWarps; w += kParts) stage[at][w] = chunk;
          }});
        feed.next(look);
        co_await pause();
      }
    }
    if (plan.is("no-drain")) co_return;
    for (uint32_t i = 0; i < kPlaces; ++i) {
      bool other;
      uint32_t parity;
      if (feed.last(i, other, parity)) co_await drain(kFp8 ? raw_full[i] : other ? land[i] : full[i], parity);
    }
  }

  Warp converter(int w) {
    TreePlace<ST> to;
    to.ph = 1;
    int n = 0;
    for (const Piece& p : pieces) {
      if (p.empty) continue;
      for (int c = 0; c < 2 * p.nt; ++c, ++n) {
        const int slot = n % kTreeRaw, tile = n / 2;
        if (!co_await see(raw_full[slot], (n / kTreeRaw) & 1)) co_return;
        if (n >= ST && !co_await see(empty[to.st], to.ph)) co_return;
        for (int x : raw[slot]) if (x != n) fault("codes converted that are another chunk's");
        stage[to.st][w] = -1;
        co_await pause();
        for (int x : raw[slot]) if (x != n) fault("codes overwritten while they are converted");
        stage[to.st][w] = n;
        if (c % 2 == 0) scales[tile % scale_slots][w] = tile;
        if (c % 2 && p.edge[c / 2]) bad[to.st][w] = n;
        full[to.st].arrive();
        co_await pause();
        raw_empty[slot].arrive();
        co_await pause();
        if (c % 2 == 0) sc_full[tile % kTreeScales].arrive();
        to.move(1);
        co_await pause();
      }
    }
  }

  int looked[ST] = {};
  Warp reader(int w) {
    uint32_t parity = 0;
    int jj = 0;
    for (const Piece& p : pieces) {
      if (p.empty) continue;
      for (int j = 0; j < p.nt; ++j) {
        if (!p.edge[j]) continue;
        const int v = 2 * (jj + j) + 1, st = v % ST;
        if (!co_await see(land[st], (parity >> st) & 1)) co_return;
        parity ^= 1u << st;
        if (stage[st][w] != v) fault("a V looked through that is another chunk");
        co_await pause();
        bad[st][w] = v;
        if (++looked[st] % kRowWarps == 0) full[st].arrive();
        co_await pause();
      }
      jj += p.nt;
    }
  }

  Warp queries() {
    int n_q = 0;
    for (size_t i = 0; i < pieces.size(); ++i) {
      if (pieces[i].empty) continue;
      if (n_q > 0 && !co_await see(q_empty, (n_q - 1) & 1)) break;
      const int slots = pieces[i].rows[1] ? 2 : 1;
      q_full.expect(slots);
      for (int s = 0; s < slots; ++s) flight.push_back({&q_full, [this, s, i] { q_holds[s] = (int)i; }});
      ++n_q;
      co_await pause();
    }
    if (n_q > 0) co_await drain(q_full, (n_q - 1) & 1);
  }

  Warp issuer(int slot) {
    uint32_t jj = 0, pph = 0, qph = 0;
    bool ok = true;
    for (size_t i = 0; ok && i < pieces.size(); ++i) {
      const Piece& p = pieces[i];
      if (p.empty) continue;
      if (!p.rows[slot]) {
        TreePlace<ST> c;
        c.set(2 * jj);
        for (int x = 0; ok && x < 2 * p.nt; ++x, c.move(1)) {
          if (!plan.is("unseen")) ok = co_await see(full[c.st], c.ph);
          if (ok) empty[c.st].arrive();
          co_await pause();
        }
        if (ok) ok = co_await see(q_full, qph);
        if (ok) q_empty.arrive();
      } else {
        TreePlace<ST> k, v;
        k.set(2 * jj);
        v.set(2 * jj + 1);
        ok = co_await see(q_full, qph);
        for (int j = -1; ok && j < p.nt; ++j) {
          const bool out = j >= 0, in = j + 1 < p.nt;
          if (in) ok = co_await see(full[k.st], k.ph);
          if (ok && out) ok = co_await see(full[v.st], v.ph);
          if (ok && out) ok = co_await see(p_full[slot], pph);
          if (out) pph ^= 1;
          if (!ok) break;
          Batch b;
          b.slot = slot, b.piece = (int)i;
          if (out) b.v = 2 * ((int)jj + j) + 1;
          if (in) b.k = 2 * ((int)jj + j + 1);
          if (in) {
            b.commits.push_back(&s_full[slot]);
            b.commits.push_back(&empty[k.st]);
            if (j + 2 >= p.nt) b.commits.push_back(&q_empty);
          } else {
            b.commits.push_back(&o_full[slot]);
          }
          if (out) b.commits.push_back(&empty[v.st]);
          check(b);
          pipe[slot].push_back(b);
          if (in) k.move(2);
          if (out) v.move(2);
          co_await pause();
        }
      }
      qph ^= 1;
      jj += p.nt;
    }
    co_await Until{[this, slot] { return pipe[slot].empty(); }};
  }
  // a batch's operands: when it is issued and when it is done
  void check(const Batch& b) {
    if (b.v >= 0) {
      if (!holds(b.v % ST, b.v)) fault("a product with a V that is not its tile's");
      for (int x : weights[b.slot]) if (x != b.v / 2) fault("a product with weights that are not its tile's");
    }
    if (b.k >= 0) {
      if (!holds(b.k % ST, b.k)) fault("scores of a K that is not its tile's");
      if (q_holds[b.slot] != b.piece) fault("scores of another piece's queries");
      if (reading[b.slot] && b.v < 0) fault("scores written over ones that are read");
    }
  }
  void finish(int slot) {
    if (pipe[slot].empty()) return;
    const Batch b = pipe[slot].front();
    pipe[slot].pop_front();
    check(b);
    if (b.v >= 0) {
      if (output[slot] != b.piece) {
        for (int x : taken[slot]) if (x != output[slot]) fault("an output written over one that is read");
        output[slot] = b.piece, added[slot] = 0;
      }
      ++added[slot];
    }
    if (b.k >= 0) scores[slot] = b.k / 2;
    for (Bar* x : b.commits) x->arrive();
  }

  Warp softmax(int slot, int w) {
    uint32_t n_s = 0, n_o = 0;
    int jj = 0;
    for (size_t i = 0; i < pieces.size(); ++i) {
      const Piece& p = pieces[i];
      if (p.empty) continue;
      if (p.rows[slot]) {
        for (int j = 0; j < p.nt; ++j) {
          const int at = jj + j;
          if (!co_await see(s_full[slot], n_s++ & 1)) co_return;
          ++reading[slot];
          if (scores[slot] != at) fault("scores that are another tile's");
          if (kFp8 && !co_await see(sc_full[at % kTreeScales], (at / kTreeScales) & 1)) co_return;
          for (int turn = 0; turn < 2; ++turn) {        // K's scales, later V's
            if (kFp8) for (int x : scales[at % scale_slots]) if (x != at) fault("scales that are another tile's");
            co_await pause();
          }
          weights[slot][w] = at;
          if (p.edge[j]) {
            TreePlace<ST> v;
            v.set(2 * at + 1);
            if (!plan.is("unlooked") && !co_await see(full[v.st], v.ph)) co_return;
            for (int x : bad[v.st]) if (x != 2 * at + 1) fault("a V's rows apart that are another chunk's");
          }
          --reading[slot];
          p_full[slot].arrive();
          co_await pause();
        }
        if (!co_await see(o_full[slot], n_o++ & 1)) co_return;
        if (output[slot] != (int)i || added[slot] != p.nt) fault("an output that is not its piece's");
        co_await pause();
        taken[slot][w] = (int)i;
      }
      jj += p.nt;
    }
  }

  bool turn(size_t actor) {
    if (actor < warps.size()) {
      const bool waits = !warps[actor].done() && warps[actor].h.promise().until && !warps[actor].h.promise().until();
      const bool out = abort || (patience >= 0 && turns >= patience);
      if (out && waits && warps[actor].h.promise().may_give_up) abort = true;
      return warps[actor].step(out);
    }
    actor -= warps.size();
    if (actor < 2) {
      const bool some = !pipe[actor].empty();
      finish((int)actor);
      return some;
    }
    if (flight.empty()) return false;
    const size_t i = rng() % flight.size();
    const Copy c = flight[i];
    flight.erase(flight.begin() + (long)i);
    c.write();
    c.bar->landed();
    return true;
  }
  bool over() const {
    for (const Warp& w : warps) if (!w.done()) return false;
    return true;
  }
  long turns = 0;
  const char* run() {
    if (rng() % 2) patience = rng() % 2000;
    // how often each actor gets a turn: some almost never, for a while
    const size_t actors = warps.size() + 3;
    std::vector<int> weight(actors);
    long idle = 0;
    for (; !wrong && !over(); ++turns) {
      if (turns % 64 == 0)
        for (int& w : weight) w = rng() % 4 == 0 ? 1 : 1 + rng() % 40;
      int all = 0;
      for (int w : weight) all += w;
      int x = rng() % all;
      size_t a = 0;
      while (x >= weight[a]) x -= weight[a++];
      idle = turn(a) ? 0 : idle + 1;
      if (idle > 20000) {                               // nobody gets on?
        bool some = false;
        for (size_t y = 0; y < actors; ++y) some |= turn(y);
        if (!some) fault("warps that wait for one another");
        idle = 0;
      }
    }
    if (!wrong && (!flight.empty() || !pipe[0].empty() || !pipe[1].empty())) fault("a copy or a product behind its block's end");
    return wrong;
  }
};

template <int ST, bool kFp8>
int check(const char* name, int orders, Plan plan) {
  const char* wrong = nullptr;
  int at = -1;
  for (int i = 0; i < orders && !wrong; ++i) {
    Model<ST, kFp8> m(1000003u * (unsigned)i + 17, plan);
    wrong = m.run();
    at = i;
  }
  std::printf("%s: stages %d: %s", name, ST, wrong ? wrong : "ok");
  if (wrong) std::printf(" (order %d)", at);
  std::printf("\n");
  return wrong != nullptr;
}

}  // namespace

int main(int argc, char** argv) {
  const int orders = argc > 1 ? std::atoi(argv[1]) : 1000;
  Plan plan;
  // none; unseen: a slot without rows gives back what has not come; one-slot: a stage is free when either slot is done
  // with it; no-drain: the loader leaves with copies under way; unlooked: a V's rows apart are read before it was looked through; few-scales
  if (argc > 2) plan.mistake = argv[2];
  return check<tree_stages(64, false), false>("64", orders, plan) + check<tree_stages(128, false), false>("128", orders, plan) +
         check<tree_stages(128, true), true>("128 E4M3", orders, plan);
}
