// The chain kernels' roles as lists of steps on barriers, walked through every
// order of events. Prints "ok" if from each state every role can come to its end
// and no wait ends before its time, or what went wrong first.
//
//   gated_delta_sync_model dv STAGES ROUNDS kernel|one
//     Reverse chain: loads, value warps and the warp that stores dV, with the
//     kernel's rule for dV's barriers or with one barrier for all rounds.
//   gated_delta_sync_model CHAIN WARPS CHUNKS kernel|pass|place
//     Hand-overs from WARPS state warps to the issuers of a chain (forward,
//     forward_apart, save, effect, reverse), where any wait of a state warp may give
//     up: with the kernels' rules, with state warps that always pass, or with one
//     barrier for all hand-overs of D.
//   gated_delta_sync_model loads|own_loads STAGES ROUNDS kernel|waited|leave
//     Loads by a warp of their own, or by the warp that uses them: with the kernels'
//     rules, with loads after any wait that ended, or leaving what is in flight.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>
#include <tuple>
#include <vector>

#include "gated_delta_sync.h"

namespace gdsync = kata::gdsync;

namespace {

struct Step {
  // mbarriers: one arrival completes a phase; a wait of a role that may give up
  // goes on without it. Hardware barriers count arrivals of hand and take. A load
  // lands some time after its start and completes a phase; a drain waits
  // for it. Whether it starts: by the wait before it (`exit`), or by the role's waits.
  enum Kind { kArrive, kWait, kHand, kTake, kLoad, kDrain } kind;
  int bar;
  unsigned parity = 0;               // of a wait, as the kernel gives it
  int phase = 0;                     // the phase it means
  int exit = -1;                     // the step to go to where the wait does not allow a load
};

struct State {
  std::vector<int> at;               // each role's next step
  std::vector<int> inside;           // -1, or the generation of the hardware barrier it waits at
  std::vector<char> ok;              // none of its waits has given up
  std::vector<int> phase;            // mbarriers: phases completed
  std::vector<int> count, generation;   // hardware barriers
  std::vector<char> flying;          // mbarriers: a load is in flight
  bool aborted = false;
  bool operator<(const State &o) const {
    auto tie = [](const State &s) {
      return std::tie(s.at, s.inside, s.ok, s.phase, s.count, s.generation, s.flying, s.aborted);
    };
    return tie(*this) < tie(o);
  }
};

struct Model {
  std::vector<std::vector<Step>> roles;
  std::vector<char> gives_up;        // its waits have a limit
  int bars = 0, hardware = 0, quota = 0;
  bool (*passes)(bool) = [](bool ok) { return gdsync::passes(ok); };
  bool (*may_load)(bool, bool) = [](bool waited, bool aborted) { return gdsync::may_load(waited, aborted); };
  bool (*may_load_own)(bool) = [](bool ok) { return gdsync::may_load_own(ok); };

  void resize(int n) {
    roles.resize(n);
    gives_up.resize(n);
  }
  void arrive(int role, int bar) { roles[role].push_back({Step::kArrive, bar}); }
  void wait(int role, int bar, unsigned parity, int phase) { roles[role].push_back({Step::kWait, bar, parity, phase}); }
  void hand(int role, int bar) { roles[role].push_back({Step::kHand, bar}); }
  void take(int role, int bar) { roles[role].push_back({Step::kTake, bar}); }
  void load(int role, int bar) { roles[role].push_back({Step::kLoad, bar}); }
  void drain(int role, int bar) { roles[role].push_back({Step::kDrain, bar}); }

  // The states that role r can come to from s by one step.
  void moves(const State &s, int r, std::vector<State> &out, std::string &wrong) const {
    if (s.at[r] == (int)roles[r].size()) return;
    const Step &step = roles[r][s.at[r]];
    State t = s;
    if (step.kind == Step::kArrive) {
      ++t.at[r];
      ++t.phase[step.bar];
      out.push_back(t);
    } else if (step.kind == Step::kLoad) {
      ++t.at[r];
      if (step.exit >= 0 || may_load_own(s.ok[r])) {
        if (s.flying[step.bar]) wrong = "a load started over another";
        t.flying[step.bar] = 1;
      }
      out.push_back(t);
    } else if (step.kind == Step::kDrain) {
      if (s.flying[step.bar]) return;
      ++t.at[r];
      out.push_back(t);
    } else if (step.kind == Step::kWait) {
      // a test of a parity is true if the barrier's running phase has the other one
      const bool there = (unsigned)(s.phase[step.bar] & 1) != step.parity;
      ++t.at[r];
      if (there) {
        if (s.ok[r] && !s.aborted && s.phase[step.bar] <= step.phase) wrong = "a wait ended early";
        if (step.exit >= 0 && !may_load(true, s.aborted)) t.at[r] = step.exit;
        out.push_back(t);
      }
      if (gives_up[r] && (!there || s.aborted)) {
        t.at[r] = step.exit >= 0 && !may_load(false, true) ? step.exit : s.at[r] + 1;
        t.ok[r] = 0;
        t.aborted = true;
        out.push_back(t);
      }
    } else if (s.inside[r] >= 0) {                         // waits at a hardware barrier
      if (s.generation[step.bar] == s.inside[r]) return;
      ++t.at[r];
      t.inside[r] = -1;
      out.push_back(t);
    } else {
      const bool goes_on = step.kind == Step::kHand && passes(s.ok[r]);
      if (goes_on)
        ++t.at[r];
      else
        t.inside[r] = s.generation[step.bar];
      if (++t.count[step.bar] == quota) {
        t.count[step.bar] = 0;
        ++t.generation[step.bar];
      }
      out.push_back(t);
    }
  }

  std::string walk() const {
    State first;
    first.at.resize(roles.size());
    first.inside.assign(roles.size(), -1);
    first.ok.assign(roles.size(), 1);
    first.phase.resize(bars);
    first.flying.resize(bars);
    first.count.resize(hardware);
    first.generation.resize(hardware);
    std::set<State> seen{first};
    std::vector<State> open{first}, next;
    std::string wrong;
    while (!open.empty()) {
      const State s = open.back();
      open.pop_back();
      next.clear();
      bool ended = true;
      for (size_t r = 0; r < roles.size(); ++r) {
        ended = ended && s.at[r] == (int)roles[r].size();
        moves(s, (int)r, next, wrong);
      }
      if (!wrong.empty()) return wrong;
      for (int b = 0; b < bars; ++b)
        if (s.flying[b]) {
          if (ended) return "a load in flight at the end";
          next.push_back(s);
          next.back().flying[b] = 0;
          ++next.back().phase[b];
        }
      if (!ended && next.empty()) return "stuck";
      for (const State &t : next)
        if (seen.insert(t).second) open.push_back(t);
    }
    return "ok";
  }
};

std::string dv(int stages, int rounds, bool one) {
  auto ready = [&](int i) { return one ? gdsync::turn(i, 1) : gdsync::dv_ready(i, stages); };
  const int loaded = 0, freed = stages, stored = 2 * stages, dv_ready = 3 * stages;
  Model m;
  m.bars = 4 * stages;
  m.resize(3);
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
  return m.walk();
}

// Role 0 loads, role 1 uses the places and frees them; or role 0 does both, and has
// the next round's load in flight while it uses this one's.
std::string loads(bool own, int stages, int rounds, const std::string &rule) {
  Model m;
  m.bars = 2 * stages;
  m.resize(own ? 1 : 2);
  for (char &g : m.gives_up) g = 1;
  if (rule == "waited") m.may_load = [](bool waited, bool) { return waited; };
  if (rule == "waited") m.may_load_own = [](bool) { return true; };
  if (own) m.load(0, 0);
  for (int c = 0; c < rounds; ++c) {
    const gdsync::Turn t = gdsync::turn(c, stages);
    if (own) {
      if (c + 1 < rounds) m.load(0, (c + 1) % stages);
      m.wait(0, t.place, t.parity, c / stages);
    } else {
      if (c >= stages) m.wait(0, stages + t.place, t.parity ^ 1, c / stages - 1);
      m.load(0, t.place);
      m.wait(1, t.place, t.parity, c / stages);
      m.arrive(1, stages + t.place);
    }
  }
  const int exit = (int)m.roles[0].size();
  if (!own)
    for (Step &step : m.roles[0]) step.exit = exit;
  if (rule != "leave")
    for (int b = 0; b < stages; ++b) m.drain(0, b);
  return m.walk();
}

std::string chain(const std::string &name, int warps, int chunks, const std::string &rule) {
  Model m;
  m.quota = warps + 1;
  m.bars = m.hardware = 6;
  if (rule == "pass") m.passes = [](bool) { return true; };
  auto place = [&](int c) { return rule == "place" ? 0 : gdsync::output_place(c); };
  const bool apart = name == "forward_apart";
  m.resize(warps + 1 + apart);
  const int issuer = warps, outputs = warps + apart;       // who takes D for the outputs
  for (int w = 0; w < warps; ++w) m.gives_up[w] = 1;
  auto hand = [&](int bar) {
    for (int w = 0; w < warps; ++w) m.hand(w, bar);
  };
  auto wait = [&](int bar, int c) {
    for (int w = 0; w < warps; ++w) m.wait(w, bar, c & 1, c);
  };
  auto issue = [&](int role, int taken, int done) {
    m.take(role, taken);
    m.arrive(role, done);
  };
  if (name == "effect") {                                  // two chains; S, R, D~ of each
    hand(0), hand(1);
    for (int c = 0; c < chunks; ++c) {
      for (int part = 0; part < 3; ++part)
        for (int x = 0; x < 2; ++x) {
          wait(2 * part + x, c);
          if (part < 2) hand(2 * (part + 1) + x);
          else if (c + 1 < chunks) hand(x);
          issue(issuer, 2 * part + x, 2 * part + x);
        }
    }
  } else if (name == "reverse") {                          // S, D, Z; X is P^T dO
    m.arrive(issuer, 3);
    for (int i = 0; i < chunks; ++i) {
      hand(0), wait(3, i), wait(0, i);
      hand(1), wait(1, i);
      hand(2), wait(2, i);
      issue(issuer, 0, 0), issue(issuer, 1, 1), issue(issuer, 2, 2);
      if (i + 1 < chunks) m.arrive(issuer, 3);
    }
  } else {                                                 // S, R, D~ and, with outputs, D in two places
    const bool out = name != "save";
    for (int c = 0; c < chunks; ++c) {
      hand(0);
      if (out && !apart && c > 0) wait(3, c - 1);
      wait(0, c);
      hand(1);
      if (out && apart && c > 0) wait(3, c - 1);
      wait(1, c);
      hand(2);
      if (out) hand(3 + place(c));
      wait(2, c);
      issue(issuer, 0, 0), issue(issuer, 1, 1), issue(issuer, 2, 2);
      if (out) issue(outputs, 3 + place(c), 3);
    }
    if (out) wait(3, chunks - 1);
  }
  return m.walk();
}

}  // namespace

int main(int argc, char **argv) {
  if (argc != 5) return 2;
  const std::string name = argv[1], rule = argv[4];
  const int n = atoi(argv[2]), rounds = atoi(argv[3]);
  const bool own = name == "own_loads";
  puts((name == "dv"                    ? dv(n, rounds, rule == "one")
        : own || name == "loads" ? loads(own, n, rounds, rule)
                                 : chain(name, n, rounds, rule))
           .c_str());
  return 0;
}
