// The hand-overs of the gated delta rule's chains with the kernels' own helpers and
// roles (state warps, issuer, the warp that issues the outputs' products, loads),
// without data: an MMA round is an arrival. In each block the loads stop for good
// after `stop` chunks; a state warp's wait then runs into its 2 s limit, and every
// role has to come to its end and the block to report it. All waits but those at the
// hardware barriers are bounded, and at these all roles meet (gated_delta_sync.h,
// walked through every order of events by gated_delta_sync_model.cpp).
//
// Prints, for every block, stop, chunks, the status word, and the chunks that the
// issuers and the state warps came through; then the milliseconds it all took.
#include <cstdio>
#include <vector>

#include "common.cuh"
#include "gated_delta_tc.cuh"

namespace {

using namespace kata;
using namespace kata::gdtc;

constexpr int kChunks = 6, kStages = 2, kSeeds = 4;
enum { kLoaded = 0, kFree = 2, kKsDone = 4, kDDone, kUDone, kODone, kNumBars };
enum { kSReady = 1, kRReady, kDtReady, kDlReady };

struct Report {
  unsigned status;
  int stop, issued, outputs, walked;
};

__global__ void __launch_bounds__(kChainThreads, 1) handover_kernel(Report *reports) {
  __shared__ __align__(8) uint64_t bars[kNumBars];
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;
  Report &report = reports[blockIdx.x];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int stop = blockIdx.x % (kChunks + 1);
  const bool apart = blockIdx.x / (kChunks + 1) % 2;       // outputs awaited before or behind R
  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], i >= kFree && i < kFree + kStages ? kStateWarps : 1);
    *abort_flag = 0;
    mbar_init_fence();
    report.stop = stop;
  }
  __syncthreads();
  // warps come at uneven times, and after an abort some at once
  auto uneven = [&](int c, int place) {
    const unsigned x = (blockIdx.x * 64 + warp) * 2654435761u + (c * 8 + place) * 40503u;
    if (x >> 16 & 1) __nanosleep((x >> 8) % 3000);
  };
  if (warp < kStateWarps) {
    bool ok = true;
    for (int c = 0; c < kChunks; ++c) {
      const gdsync::Turn load = gdsync::turn(c, kStages);
      ok &= warp_wait(&bars[kLoaded + load.place], load.parity, abort_flag);
      uneven(c, 0);
      hand_over(kSReady, ok);
      if (!apart && c > 0) ok &= warp_wait(&bars[kODone], (c - 1) & 1, abort_flag);
      ok &= warp_wait(&bars[kKsDone], c & 1, abort_flag);
      uneven(c, 1);
      hand_over(kRReady, ok);
      if (apart && c > 0) ok &= warp_wait(&bars[kODone], (c - 1) & 1, abort_flag);
      ok &= warp_wait(&bars[kDDone], c & 1, abort_flag);
      uneven(c, 2);
      hand_over(kDtReady, ok);
      hand_over(kDlReady + gdsync::output_place(c), ok);
      ok &= warp_wait(&bars[kUDone], c & 1, abort_flag);
      warp_arrive(&bars[kFree + load.place]);
    }
    warp_wait(&bars[kODone], (kChunks - 1) & 1, abort_flag);
    if (lane == 0) atomicAdd(&report.walked, kChunks);
  } else if (warp == kIssuer) {
    for (int c = 0; c < kChunks; ++c) {
      for (int round = 0; round < 3; ++round) {
        take_over(kSReady + round);
        uneven(c, 3 + round);
        if (lane == 0) mbar_arrive(&bars[kKsDone + round]);
      }
      if (lane == 0) ++report.issued;
    }
  } else if (warp == kSaver) {
    for (int c = 0; c < kChunks; ++c) {
      take_over(kDlReady + gdsync::output_place(c));
      uneven(c, 6);
      if (lane == 0) mbar_arrive(&bars[kODone]);
      if (lane == 0) ++report.outputs;
    }
  } else if (warp == kLoader && lane == 0) {
    for (int c = 0; c < stop; ++c) {
      const gdsync::Turn load = gdsync::turn(c, kStages);
      if (c >= kStages && !mbar_wait(&bars[kFree + load.place], load.parity ^ 1, abort_flag)) break;
      mbar_arrive(&bars[kLoaded + load.place]);
    }
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(&report.status, kStatusDeviceTimeout);
}

}  // namespace

int main() {
  constexpr int blocks = (kChunks + 1) * 2 * kSeeds;       // at most one an SM
  static_assert(blocks <= 148, "all blocks run at once");
  Report *reports;
  cudaEvent_t start, end;
  if (cudaMalloc(&reports, blocks * sizeof(Report)) != cudaSuccess) return 1;
  if (cudaMemset(reports, 0, blocks * sizeof(Report)) != cudaSuccess) return 1;
  cudaEventCreate(&start);
  cudaEventCreate(&end);
  cudaEventRecord(start);
  handover_kernel<<<blocks, kChainThreads>>>(reports);
  cudaEventRecord(end);
  std::vector<Report> got(blocks);
  if (cudaMemcpy(got.data(), reports, blocks * sizeof(Report), cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
  for (const Report &r : got)
    printf("%d %d %u %d %d %d\n", r.stop, kChunks, r.status, r.issued, r.outputs, r.walked / kStateWarps);
  float ms = 0.f;
  cudaEventElapsedTime(&ms, start, end);
  printf("%.0f\n", ms);
  return 0;
}
