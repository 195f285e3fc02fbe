// bf16 tensors to fp32 and back, for the few tokens whose bf16 gradient runs on
// the fp32 kernels (gated_delta_api.cu). A launch for all tensors each way; bound
// by the launch.
#include "common.cuh"
#include "gated_delta.h"
#include "profile.h"

namespace kata {
namespace {

template <typename From, typename To> struct Arrays {
  const From *from[4];
  To *to[4];
  size_t n[4];
};

template <typename From, typename To>
__global__ void gd_convert_kernel(const Arrays<From, To> a) {
  const From *from = a.from[blockIdx.y];
  To *to = a.to[blockIdx.y];
  const size_t n = a.n[blockIdx.y], step = (size_t)gridDim.x * blockDim.x;
  for (size_t e = (size_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += step) to[e] = from_f<To>(to_f(from[e]));
}

template <typename From, typename To>
cudaError_t run(const Arrays<From, To> &a, int count, cudaStream_t stream) {
  ProfileScope prof("gd_convert", stream);
  gd_convert_kernel<From, To><<<dim3(64, (unsigned)count), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_bf16_gradient_in_f32(const GatedDeltaLaunch &a, int d_k, int d_v) {
  const size_t keys = (size_t)(a.BH / (a.H / a.Hk)) * a.T * d_k, values = (size_t)a.BH * a.T * d_v;
  using bf16 = __nv_bfloat16;
  float *const *t = a.in_f32;                              // q, k, v, dout, dq, dk, dv
  const Arrays<bf16, float> in{{static_cast<const bf16 *>(a.q), static_cast<const bf16 *>(a.k),
                                static_cast<const bf16 *>(a.v), static_cast<const bf16 *>(a.dout)},
                               {t[0], t[1], t[2], t[3]}, {keys, keys, values, values}};
  cudaError_t e = run(in, 4, a.stream);
  if (e != cudaSuccess) return e;
  GatedDeltaLaunch f = a;
  f.q = t[0]; f.k = t[1]; f.v = t[2]; f.dout = t[3];
  f.dq = t[4]; f.dk = t[5]; f.dv = t[6];
  e = gd_f32_backward(f, d_k, d_v);
  if (e != cudaSuccess) return e;
  const Arrays<float, bf16> out{{t[4], t[5], t[6], nullptr},
                                {static_cast<bf16 *>(a.dq), static_cast<bf16 *>(a.dk), static_cast<bf16 *>(a.dv),
                                 nullptr},
                                {keys, keys, values, 0}};
  return run(out, 3, a.stream);
}

}  // namespace kata
