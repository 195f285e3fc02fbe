// Rules of the gated delta rule's chain kernels that decide whether a wait can
// miss what it waits for. Plain C++ as well as device code, so that a host program
// walks the kernels' roles through every order of events by the same rules.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GD_SYNC_FN __host__ __device__ constexpr
#else
#define GD_SYNC_FN constexpr
#endif

namespace kata {
namespace gdsync {

// An mbarrier tells only the parity of its last completed phase: who waits for
// phase i has to look before phase i + 1 completes. Uses that may be `places` ahead of
// their waiter therefore take `places` barriers by turns.
struct Turn {
  int place;
  uint32_t parity;
};
GD_SYNC_FN Turn turn(int use, int places) { return Turn{use % places, (uint32_t)(use / places) & 1u}; }

// Reverse chain: dV of round i lies in stage i % stages. The value warps reach round
// i + stages only behind its loads, these behind the stores of round i: they may be
// `stages` rounds ahead of the warp that stores.
GD_SYNC_FN Turn dv_ready(int round, int stages) { return turn(round, stages); }

}  // namespace gdsync
}  // namespace kata
