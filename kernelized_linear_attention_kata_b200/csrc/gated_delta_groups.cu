// dq and dk of query / key heads that several value heads share: the value
// heads' fp32 parts are added in head order (the same bits every run) and
// rounded once. Bound by the parts' bytes.
#include "common.cuh"
#include "gated_delta.h"
#include "profile.h"

namespace kata {
namespace {

template <typename Tin>
__global__ void gd_group_sum_kernel(const float *__restrict__ dq_part, const float *__restrict__ dk_part,
                                    Tin *__restrict__ dq, Tin *__restrict__ dk, int group, size_t head,
                                    size_t total) {
  const float *part = blockIdx.y ? dk_part : dq_part;
  Tin *out = blockIdx.y ? dk : dq;
  for (size_t e = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) * 4; e < total;
       e += (size_t)gridDim.x * blockDim.x * 4) {
    const float *src = part + (e / head) * group * head + e % head;    // head is a multiple of 16
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int h = 0; h < group; ++h) {
      const float4 x = *reinterpret_cast<const float4 *>(src + (size_t)h * head);
      sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
    }
    out[e] = from_f<Tin>(sum.x);
    out[e + 1] = from_f<Tin>(sum.y);
    out[e + 2] = from_f<Tin>(sum.z);
    out[e + 3] = from_f<Tin>(sum.w);
  }
}

template <typename Tin> cudaError_t run(const GatedDeltaLaunch &a, int d_k) {
  const size_t head = (size_t)a.T * d_k, total = head * (size_t)(a.BH / (a.H / a.Hk));
  const size_t want = (total / 4 + 255) / 256;
  ProfileScope prof("gd_group_sum", a.stream);
  gd_group_sum_kernel<Tin><<<dim3((unsigned)(want < 2048 ? want : 2048), 2), 256, 0, a.stream>>>(
      a.dq_part, a.dk_part, static_cast<Tin *>(a.dq), static_cast<Tin *>(a.dk), a.H / a.Hk, head, total);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_sum_groups(const GatedDeltaLaunch &a, int d_k, bool bf16) {
  return bf16 ? run<__nv_bfloat16>(a, d_k) : run<float>(a, d_k);
}

}  // namespace kata
