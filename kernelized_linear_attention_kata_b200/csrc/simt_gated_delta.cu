// Launchers of the gated delta rule's CUDA-core kernels (fp32).

#include "simt_gated_delta.cuh"

namespace kata {
namespace gd {

template <typename K> cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

#define GD_TRY(expr)                          \
  do {                                        \
    cudaError_t e_ = (expr);                  \
    if (e_ != cudaSuccess) return e_;         \
  } while (0)

template <int DK>
cudaError_t solve(const GatedDeltaLaunch &a) {
  auto kern = gd_solve_kernel<DK>;
  GD_TRY(allow_smem(kern, sizeof(SolveSmem<DK>)));
  ProfileScope prof("simt_gd_solve", a.stream);
  kern<<<(unsigned)(a.BH * a.N), kThreads, sizeof(SolveSmem<DK>), a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), a.g, a.beta, a.M, a.P, a.H, a.Hk,
      a.T, a.N);
  return cudaGetLastError();
}

template <int DK, int CB>
cudaError_t chain(const GatedDeltaLaunch &a, int d_v) {
  auto kern = gd_chain_kernel<DK, CB>;
  constexpr size_t smem = sizeof(ChainSmem<DK, CB>);
  GD_TRY(allow_smem(kern, smem));
  ProfileScope prof("simt_gd_chain", a.stream);
  kern<<<(unsigned)(a.BH * (d_v / CB)), kThreads, smem, a.stream>>>(
      static_cast<const float *>(a.q), static_cast<const float *>(a.k), static_cast<const float *>(a.v), a.g,
      a.beta, a.M, a.P, a.S0, static_cast<float *>(a.o), a.S_out, a.starts, a.writes, a.H, a.Hk, a.T,
      a.N, d_v);
  return cudaGetLastError();
}

template <int DK, int CB>
cudaError_t backward(const GatedDeltaLaunch &a, int d_v) {
  GD_TRY((solve<DK>(a)));
  GD_TRY((chain<DK, CB>(a, d_v)));
  const float *q = static_cast<const float *>(a.q), *k = static_cast<const float *>(a.k);
  const float *dout = static_cast<const float *>(a.dout);
  {
    auto kern = gd_chain_reverse_kernel<DK, CB>;
    constexpr size_t smem = sizeof(ChainSmem<DK, CB>);
    GD_TRY(allow_smem(kern, smem));
    ProfileScope prof("simt_gd_chain_reverse", a.stream);
    kern<<<(unsigned)(a.BH * (d_v / CB)), kThreads, smem, a.stream>>>(
        q, k, dout, a.g, a.beta, a.M, a.P, a.dS, static_cast<float *>(a.dv), a.dR, a.ends, a.dS0, a.H,
        a.Hk, a.T, a.N, d_v);
    GD_TRY(cudaGetLastError());
  }
  {
    auto kern = gd_grads_kernel<DK, CB>;
    constexpr size_t smem = sizeof(GradSmem<DK, CB>);
    GD_TRY(allow_smem(kern, smem));
    ProfileScope prof("simt_gd_grads", a.stream);
    kern<<<(unsigned)(a.BH * a.N), kThreads, smem, a.stream>>>(
        q, k, static_cast<const float *>(a.v), dout, a.g, a.beta, a.starts, a.ends, a.writes, a.dR,
        static_cast<float *>(a.dq), static_cast<float *>(a.dk), a.dq_part, a.dk_part, a.dg, a.dbeta, a.H,
        a.Hk, a.T, a.N, d_v);
    GD_TRY(cudaGetLastError());
  }
  return a.dq_part ? gd_sum_groups(a, DK, false) : cudaSuccess;
}

}  // namespace gd

// Value columns a block: 32 (16 for d_v = 16). The columns are independent,
// so a narrow block fills more SMs when there are few heads.
#define GD_DISPATCH(FN)                                            \
  switch (d_k) {                                                   \
    case 16: return d_v == 16 ? FN(16, 16) : FN(16, 32);           \
    case 32: return d_v == 16 ? FN(32, 16) : FN(32, 32);           \
    case 64: return d_v == 16 ? FN(64, 16) : FN(64, 32);           \
    case 128: return d_v == 16 ? FN(128, 16) : FN(128, 32);        \
    default: return cudaErrorNotSupported;                         \
  }

template <int DK, int CB>
cudaError_t simt_gated_delta_run(const GatedDeltaLaunch &a, int d_v) {
  cudaError_t e = gd::solve<DK>(a);
  return e != cudaSuccess ? e : gd::chain<DK, CB>(a, d_v);
}

cudaError_t simt_gated_delta(const GatedDeltaLaunch &a, int d_k, int d_v) {
#define GD_RUN(DK, CB) simt_gated_delta_run<DK, CB>(a, d_v)
  GD_DISPATCH(GD_RUN)
#undef GD_RUN
}

cudaError_t simt_gated_delta_backward(const GatedDeltaLaunch &a, int d_k, int d_v) {
#define GD_RUN(DK, CB) (gd::backward<DK, CB>(a, d_v))
  GD_DISPATCH(GD_RUN)
#undef GD_RUN
}

}  // namespace kata
