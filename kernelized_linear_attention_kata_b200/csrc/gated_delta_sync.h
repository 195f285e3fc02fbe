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

// Hand-overs from the state warps to an issuer, on hardware barriers: these count
// arrivals, whoever they come from, and an issuer's wait there has no limit. So no
// state warp may come twice before the issuer has come once. A warp that passes
// (arrives and goes on) next waits for the MMAs which the issuer starts behind the
// barrier. Once one of its waits has given up, that order is gone, and the warp waits
// at each further hand-over until all have come. Then all roles meet at every hand-over
// in the same order and come to their ends. Each is of another barrier than the
// one before it, so the first of them waits for what the warp passed last, too.
GD_SYNC_FN bool passes(bool ok) { return ok; }

// The one hand-over that a warp apart may take (D, for the outputs) is not followed
// by a wait for it in the same chunk: two barriers by turns, so that the hand-over of
// the next chunk is of another barrier than the one that may still be open.
GD_SYNC_FN int output_place(int chunk) { return chunk & 1; }

// Loads: a barrier takes the next one's arrival only when the one before it there has
// landed, and a block ends only when all have. That a place is free says the first as
// long as no wait has given up: a warp that went on without its load frees the place,
// too. So no load starts after an abort, and the last ones are waited for in any case.
GD_SYNC_FN bool may_load(bool waited, bool aborted) { return waited && !aborted; }
// A thread that has itself waited for the loads before knows it from its own waits.
GD_SYNC_FN bool may_load_own(bool ok) { return ok; }

}  // namespace gdsync
}  // namespace kata
