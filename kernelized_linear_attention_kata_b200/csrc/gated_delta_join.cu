// Where the sequence of a head is cut into G segments: the states at the
// borders from the segments' effects, S_{j+1} = F_j S_j + B_j, first to last, and
// the state's gradients, E_{j-1} = F_j^T E_j + B'_j, last to first. `starts` and
// `ends` come with B and B' in their places and leave with the states.
//
// One block a head, 16 value columns and direction; the border's 16 columns
// stay in shared memory, and the next F (64 KB at d_k = 128) comes by
// asynchronous copies while this one is multiplied. A step of the walk is
// bound by the shared-memory reads: a thread's d_k / 32 rows x 2 columns take
// one 16-byte read of F a row and one of the state for 4 of the depth.
#include "gated_delta.h"
#include "profile.h"

namespace kata {
namespace {

constexpr int kCols = 16, kThreads = 256;

template <int DK> struct JoinSmem {
  static constexpr int LD = DK + 4;
  float F[2][DK * LD];
  float S[kCols * LD];               // transposed: a column's entries lie side by side
};

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

template <int DK>
__global__ void __launch_bounds__(kThreads)
gd_join_kernel(const float *__restrict__ F, float *starts, float *ends, int G, int DV) {
  extern __shared__ __align__(16) float sm[];
  JoinSmem<DK> &s = *reinterpret_cast<JoinSmem<DK> *>(sm);
  constexpr int LD = JoinSmem<DK>::LD, PER = DK / 32;
  const int nb = DV / kCols, bh = blockIdx.x / nb, c0 = blockIdx.x % nb * kCols;
  const bool back = blockIdx.y == 1;
  float *states = (back ? ends : starts) + (size_t)bh * G * DK * DV;
  const int tid = threadIdx.x, col = 2 * (tid % 8), rg = tid / 8;
  const int steps = G - 2;
  auto segment = [&](int i) { return back ? G - 2 - i : 1 + i; };      // whose F is the i-th
  auto fetch = [&](int i) {
    if (i < steps) {
      const float *src = F + ((size_t)bh * (G - 2) + segment(i) - 1) * DK * DK;
      for (int e = tid; e < DK * DK / 4; e += kThreads)
        copy16(&s.F[i & 1][e / (DK / 4) * LD + e % (DK / 4) * 4], src + 4 * e);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0);
  {
    const float *first = states + (size_t)(back ? G - 2 : 1) * DK * DV + c0;
    for (int e = tid; e < DK * kCols; e += kThreads) s.S[e % kCols * LD + e / kCols] = first[(size_t)(e / kCols) * DV + e % kCols];
  }
  for (int i = 0; i < steps; ++i) {
    fetch(i + 1);
    const int j = segment(i);
    float *to = states + (size_t)(back ? j - 1 : j + 1) * DK * DV + c0 + col;
    // rows rg + 32 x (back: PER rg + x, F is read across)
    auto row = [&](int x) { return back ? PER * rg + x : rg + 32 * x; };
    float2 acc[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) acc[x] = *reinterpret_cast<const float2 *>(to + (size_t)row(x) * DV);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float *f = s.F[i & 1], *s0 = s.S + col * LD, *s1 = s0 + LD;
#pragma unroll 4
    for (int k = 0; k < DK; k += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(s0 + k), b = *reinterpret_cast<const float4 *>(s1 + k);
      if (!back) {
#pragma unroll
        for (int x = 0; x < PER; ++x) {
          const float4 m = *reinterpret_cast<const float4 *>(f + (rg + 32 * x) * LD + k);
          acc[x].x = fmaf(m.w, a.w, fmaf(m.z, a.z, fmaf(m.y, a.y, fmaf(m.x, a.x, acc[x].x))));
          acc[x].y = fmaf(m.w, b.w, fmaf(m.z, b.z, fmaf(m.y, b.y, fmaf(m.x, b.x, acc[x].y))));
        }
      } else {
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float m[PER];
#pragma unroll
          for (int x = 0; x < PER; x += 2) {
            const float2 p = *reinterpret_cast<const float2 *>(f + (k + u) * LD + PER * rg + x);
            m[x] = p.x;
            m[x + 1] = p.y;
          }
#pragma unroll
          for (int x = 0; x < PER; ++x) {
            acc[x].x = fmaf(m[x], av[u], acc[x].x);
            acc[x].y = fmaf(m[x], bv[u], acc[x].y);
          }
        }
      }
    }
    __syncthreads();                                       // S and this F have been read
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      s.S[col * LD + row(x)] = acc[x].x;
      s.S[(col + 1) * LD + row(x)] = acc[x].y;
      *reinterpret_cast<float2 *>(to + (size_t)row(x) * DV) = acc[x];
    }
  }
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

}  // namespace kata
