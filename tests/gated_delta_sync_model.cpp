// The chain kernels' roles as lists of steps on barriers, walked through every
// order of events. Prints "ok" if from each state every role can come to its end
// and no wait ends before its time, or what went wrong first.
//
//   gated_delta_sync_model dv STAGES ROUNDS kernel|one
//     Reverse chain: loads, value warps and the warp that stores dV, with the
//     kernel's rule for dV's barriers or with one barrier for all rounds.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <vector>

#include "gated_delta_sync.h"

using kata::gdsync::Turn;

namespace {

struct Step {
  enum Kind { kArrive, kWait } kind;
  int bar;
  unsigned parity = 0;               // of a wait, as the kernel gives it
  int phase = 0;                     // the phase it means
};
using Role = std::vector<Step>;

struct State {
  std::vector<int> at, phase;        // each role's next step, each barrier's phases completed
  bool operator<(const State &o) const { return at != o.at ? at < o.at : phase < o.phase; }
};

struct Model {
  std::vector<Role> roles;
  int bars = 0;
  void arrive(int role, int bar) { roles[role].push_back({Step::kArrive, bar}); }
  void wait(int role, int bar, unsigned parity, int phase) { roles[role].push_back({Step::kWait, bar, parity, phase}); }

  std::string walk() const {
    std::set<State> seen;
    std::vector<State> open{State{std::vector<int>(roles.size()), std::vector<int>(bars)}};
    seen.insert(open[0]);
    while (!open.empty()) {
      const State s = open.back();
      open.pop_back();
      bool moved = false, ended = true;
      for (size_t r = 0; r < roles.size(); ++r) {
        if (s.at[r] == (int)roles[r].size()) continue;
        ended = false;
        const Step &step = roles[r][s.at[r]];
        State t = s;
        ++t.at[r];
        if (step.kind == Step::kArrive) {
          ++t.phase[step.bar];
        } else {
          // a test of a parity is true if the barrier's running phase has the other one
          if ((unsigned)(s.phase[step.bar] & 1) == step.parity) continue;
          if (s.phase[step.bar] <= step.phase) return "a wait ended early";
        }
        moved = true;
        if (seen.insert(t).second) open.push_back(t);
      }
      if (!ended && !moved) return "stuck";
    }
    return "ok";
  }
};

int dv(int stages, int rounds, bool one) {
  auto ready = [&](int i) { return one ? kata::gdsync::turn(i, 1) : kata::gdsync::dv_ready(i, stages); };
  const int loaded = 0, freed = stages, stored = 2 * stages, dv_ready = 3 * stages;
  Model m;
  m.bars = 4 * stages;
  m.roles.resize(3);
  for (int i = 0; i < rounds; ++i) {
    const int st = i % stages, nth = i / stages;
    if (i >= stages) {
      m.wait(0, freed + st, (nth - 1) & 1, nth - 1);
      m.wait(0, stored + st, (nth - 1) & 1, nth - 1);
    }
    m.arrive(0, loaded + st);
    m.wait(1, loaded + st, nth & 1, nth);
    m.arrive(1, dv_ready + ready(i).place);
    m.arrive(1, freed + st);
    m.wait(2, dv_ready + ready(i).place, ready(i).parity, one ? i : nth);
    m.arrive(2, stored + st);
  }
  const std::string found = m.walk();
  puts(found.c_str());
  return 0;
}

}  // namespace

int main(int argc, char **argv) {
  if (argc == 5 && !strcmp(argv[1], "dv")) return dv(atoi(argv[2]), atoi(argv[3]), !strcmp(argv[4], "one"));
  return 2;
}
