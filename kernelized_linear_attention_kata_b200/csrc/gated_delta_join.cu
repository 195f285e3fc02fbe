// Where the sequence of a head is cut into G segments: the states at the
// borders from the segments' effects, S_{j+1} = F_j S_j + B_j, first to last, and
// the state's gradients, E_{j-1} = F_j^T E_j + B'_j, last to first. `starts` and
// `ends` come with B and B' in their places and leave with the states.
//
// One block a head, 16 value columns and direction; the border's 16 columns
// stay in shared memory, and the next F (64 KB at d_k = 128) comes by
// asynchronous copies while this one is multiplied, on the fp32 kernels' TF32
// products. Bound by those copies: every block of a head reads all of its F.
#include "gated_delta.h"
#include "gated_delta_f32.cuh"
#include "profile.h"

namespace kata {
namespace {

using gd::kThreads;
constexpr int kCols = 16;

template <int DK> struct JoinSmem {
  static constexpr int LD = DK + 4, LS = kCols + 8;
  float F[2][DK * LD];
  float S[DK * LS];
};

template <int DK, bool BACK>
__device__ __forceinline__ void join(JoinSmem<DK> &s, const float *__restrict__ F, float *states, int G, int DV) {
  constexpr int LD = JoinSmem<DK>::LD, LS = JoinSmem<DK>::LS;
  using GJ = gd::Gemm<DK, kCols, BACK, false, LD, LS>;
  const int tid = threadIdx.x, steps = G - 2;
  auto segment = [&](int i) { return BACK ? G - 2 - i : 1 + i; };      // whose F is the i-th
  auto fetch = [&](int i) {
    if (i < steps) {
      const float *src = F + (size_t)(segment(i) - 1) * DK * DK;
      for (int e = tid; e < DK * DK / 4; e += kThreads)
        gd::copy16(&s.F[i & 1][e / (DK / 4) * LD + e % (DK / 4) * 4], src + 4 * e, true);
    }
    gd::copies_done();
  };
  fetch(0);
  {
    const float *first = states + (size_t)(BACK ? G - 2 : 1) * DK * DV;
    for (int e = tid; e < DK * kCols; e += kThreads)
      s.S[e / kCols * LS + e % kCols] = first[(size_t)(e / kCols) * DV + e % kCols];
  }
  for (int i = 0; i < steps; ++i) {
    fetch(i + 1);
    float *to = states + (size_t)(BACK ? segment(i) - 1 : segment(i) + 1) * DK * DV;
    float acc[GJ::TM][GJ::TN];
    if (GJ::active()) {
#pragma unroll
      for (int x = 0; x < GJ::TM; ++x)
#pragma unroll
        for (int y = 0; y < GJ::TN; ++y) acc[x][y] = to[(size_t)GJ::row(x) * DV + GJ::col(y)];
    }
    gd::copies_wait<1>();
    __syncthreads();
    GJ::run(s.F[i & 1], s.S, acc, 0, DK);
    __syncthreads();                                       // S and this F have been read
    if (GJ::active()) {
#pragma unroll
      for (int x = 0; x < GJ::TM; ++x)
#pragma unroll
        for (int y = 0; y < GJ::TN; ++y) {
          s.S[GJ::row(x) * LS + GJ::col(y)] = acc[x][y];
          to[(size_t)GJ::row(x) * DV + GJ::col(y)] = acc[x][y];
        }
    }
  }
}

template <int DK>
__global__ void __launch_bounds__(kThreads)
gd_join_kernel(const float *__restrict__ F, float *starts, float *ends, int G, int DV) {
  extern __shared__ __align__(16) float sm[];
  JoinSmem<DK> &s = *reinterpret_cast<JoinSmem<DK> *>(sm);
  const int nb = DV / kCols, bh = blockIdx.x / nb;
  const size_t at = (size_t)bh * G * DK * DV + blockIdx.x % nb * kCols;
  F += (size_t)bh * (G - 2) * DK * DK;
  if (blockIdx.y == 0)
    join<DK, false>(s, F, starts + at, G, DV);
  else
    join<DK, true>(s, F, ends + at, G, DV);
}

template <int DK> cudaError_t run(const GatedDeltaLaunch &a, int dv) {
  auto kern = gd_join_kernel<DK>;
  GD_ALLOW_SMEM(kern, sizeof(JoinSmem<DK>));
  ProfileScope prof("gd_join", a.stream);
  kern<<<dim3((unsigned)(a.BH * (dv / kCols)), a.ends_seg ? 2 : 1), kThreads, sizeof(JoinSmem<DK>), a.stream>>>(
      a.F, a.starts_seg, a.ends_seg, a.G, dv);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_tc_join(const GatedDeltaLaunch &a, int d_k, int d_v) {
  if (a.G <= 2) return cudaSuccess;                        // one border: its state is there
  return gd_padded(d_k) == 64 ? run<64>(a, gd_padded(d_v)) : run<128>(a, gd_padded(d_v));
}
cudaError_t gd_f32_join(const GatedDeltaLaunch &a, int d_k, int d_v) {
  if (a.G <= 2) return cudaSuccess;
  if (d_k <= 32) return d_k == 16 ? run<16>(a, d_v) : run<32>(a, d_v);
  return d_k == 64 ? run<64>(a, d_v) : run<128>(a, d_v);
}

}  // namespace kata
