// Launchers of the gated delta rule's fp32 kernels.

#include "gated_delta_f32.cuh"

namespace kata {
namespace gd {

#define GD_TRY(expr)                          \
  do {                                        \
    cudaError_t e_ = (expr);                  \
    if (e_ != cudaSuccess) return e_;         \
  } while (0)

template <int DK>
cudaError_t solve(const GatedDeltaLaunch &a) {
  auto kern = gd_solve_kernel<DK>;
  GD_ALLOW_SMEM(kern, sizeof(SolveSmem<DK>));
  ProfileScope prof("gd_f32_solve", a.stream);
  kern<<<(unsigned)(a.BH * a.N), kThreads, sizeof(SolveSmem<DK>), a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), a.g, a.beta, a.M, a.P, a.gates, a.status,
      a.H, a.Hk, a.T, a.N);
  return cudaGetLastError();
}

template <int DK, int CB, bool EFFECT>
cudaError_t chain(const GatedDeltaLaunch &a, int d_v) {
  auto kern = gd_chain_kernel<DK, CB, EFFECT>;
  constexpr size_t smem = sizeof(ChainSmem<DK, CB>);
  GD_ALLOW_SMEM(kern, smem);
  const int kind0 = (int)(a.BH * (a.G - 1) * (d_v / CB));
  const Segments sg{a.starts_seg, a.F, a.G, a.seg_chunks, kind0};
  const long long blocks = EFFECT ? kind0 + a.BH * (a.G - 2) * (DK / CB) : a.BH * a.G * (d_v / CB);
  ProfileScope prof(EFFECT ? "gd_f32_segment" : "gd_f32_chain", a.stream);
  kern<<<(unsigned)blocks, kThreads, smem, a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), static_cast<const float *>(a.v), a.gates,
      a.M, a.P, a.S0, EFFECT ? nullptr : static_cast<float *>(a.o), a.S_out, EFFECT ? nullptr : a.starts,
      EFFECT ? nullptr : a.writes, a.H, a.Hk, a.T, a.N, d_v, sg);
  return cudaGetLastError();
}

template <int DK, int CB, bool EFFECT>
cudaError_t reverse(const GatedDeltaLaunch &a, int d_v) {
  auto kern = gd_chain_reverse_kernel<DK, CB, EFFECT>;
  constexpr size_t smem = sizeof(ChainSmem<DK, CB>);
  GD_ALLOW_SMEM(kern, smem);
  const Segments sg{a.ends_seg, nullptr, a.G, a.seg_chunks, 0};
  ProfileScope prof(EFFECT ? "gd_f32_reverse_segment" : "gd_f32_chain_reverse", a.stream);
  kern<<<(unsigned)(a.BH * (EFFECT ? a.G - 1 : a.G) * (d_v / CB)), kThreads, smem, a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), static_cast<const float *>(a.dout),
      a.gates, a.M, a.P, a.dS, static_cast<float *>(a.dv), a.dR, a.ends, a.dS0, a.H, a.Hk, a.T, a.N, d_v, sg);
  return cudaGetLastError();
}

template <int DK, int CB>
cudaError_t grads(const GatedDeltaLaunch &a, int d_v) {
  auto kern = gd_grads_kernel<DK, CB>;
  constexpr size_t smem = sizeof(GradSmem<DK, CB>);
  GD_ALLOW_SMEM(kern, smem);
  ProfileScope prof("gd_f32_grads", a.stream);
  kern<<<(unsigned)(a.BH * a.N), kThreads, smem, a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), static_cast<const float *>(a.v),
      static_cast<const float *>(a.dout), a.g, a.beta, a.starts, a.ends, a.writes, a.dR,
      static_cast<float *>(a.dq), static_cast<float *>(a.dk), a.dq_part, a.dk_part, a.dg, a.dbeta, a.H, a.Hk,
      a.T, a.N, d_v);
  return cudaGetLastError();
}

// Value columns a block of the chains: the columns are independent and a block
// of 16 has half the products of one of 32, so 16 as long as all blocks still run
// at once.
bool narrow(const GatedDeltaLaunch &a, int d_v) { return d_v == 16 || a.BH * a.G * (d_v / 16) <= kGdSms; }

template <int DK>
cudaError_t effects(const GatedDeltaLaunch &a, int d_v) {
  constexpr int CB = DK == 16 ? 16 : 32;                   // F has d_k columns
  GD_TRY((d_v == 16 ? chain<DK, 16, true>(a, d_v) : chain<DK, CB, true>(a, d_v)));
  if (a.ends_seg) GD_TRY((d_v == 16 ? reverse<DK, 16, true>(a, d_v) : reverse<DK, 32, true>(a, d_v)));
  return gd_f32_join(a, DK, d_v);
}

template <int DK>
cudaError_t forward(const GatedDeltaLaunch &a, int d_v) {
  GD_TRY(solve<DK>(a));
  if (a.G > 1) GD_TRY(effects<DK>(a, d_v));
  return narrow(a, d_v) ? chain<DK, 16, false>(a, d_v) : chain<DK, 32, false>(a, d_v);
}

template <int DK>
cudaError_t backward(const GatedDeltaLaunch &a, int d_v) {
  GD_TRY(forward<DK>(a, d_v));
  GD_TRY((narrow(a, d_v) ? reverse<DK, 16, false>(a, d_v) : reverse<DK, 32, false>(a, d_v)));
  GD_TRY((d_v == 16 ? grads<DK, 16>(a, d_v) : grads<DK, 32>(a, d_v)));
  return a.dq_part ? gd_sum_groups(a, DK, false) : cudaSuccess;
}

}  // namespace gd

#define GD_DISPATCH(FN)                  \
  switch (d_k) {                         \
    case 16: return gd::FN<16>(a, d_v);  \
    case 32: return gd::FN<32>(a, d_v);  \
    case 64: return gd::FN<64>(a, d_v);  \
    case 128: return gd::FN<128>(a, d_v); \
    default: return cudaErrorNotSupported; \
  }

cudaError_t gd_f32(const GatedDeltaLaunch &a, int d_k, int d_v) { GD_DISPATCH(forward) }
cudaError_t gd_f32_backward(const GatedDeltaLaunch &a, int d_k, int d_v) { GD_DISPATCH(backward) }

// Segments a head, as for bf16 (gated_delta_tc.cu): 4.5 us a chunk of the chains
// and the effects, 5.4 of the reverse ones, 32 value columns a block. Where the blocks
// of this many segments all fit with 16 columns each, they run so (narrow), with half the products.
void gd_f32_split(long long BH, int N, int d_k, int d_v, bool gradient, int *G, int *seg_chunks) {
  const long long nb = d_v > 32 ? d_v / 32 : 1, nf = d_k > 32 ? d_k / 32 : 1;
  int best = 1;
  double least = 1e300;
  auto waves = [](long long blocks) { return (double)((blocks + kGdSms - 1) / kGdSms); };
  for (int g = 1; g <= 64 && (g == 1 || g * BH * nb <= kGdSms); ++g) {
    const int per = (N + g - 1) / g, used = per > 0 ? (N + per - 1) / per : 1;
    if (used != g) continue;
    double time = (gradient ? 9.9 : 4.5) * waves(BH * g * nb) * per;
    if (g > 1)
      time += (4.5 * waves(BH * ((g - 1) * nb + (g - 2) * nf)) + (gradient ? 5.4 * waves(BH * (g - 1) * nb) : 0.0)) * per +
              (gradient ? 14.0 : 7.0);
    if (g > 2) time += 7.0 + 4.0 * (g - 2) * waves(BH * (d_v / 16) * (gradient ? 2 : 1));
    if (time < least) {
      least = time;
      best = g;
    }
  }
  *G = best;
  *seg_chunks = (N + best - 1) / best;
}

}  // namespace kata
