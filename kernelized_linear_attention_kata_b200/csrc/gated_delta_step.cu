// One token of the gated delta rule, the state updated in place:
//   S <- e^g S + k d^T,  d = beta (v - e^g S^T k),  y = S^T q.
// e^g is 0 from -104 on, the clamp of the chunked forms included: no clamp here.
// With u = S^T k and w = S^T q of the old state, y = e^g w + (k . q) d, so one
// reading of S gives both products and it stays in registers for the update:
// S moves once in and once out, which is the floor (the step is bound by that
// traffic; the arithmetic is 6 flops per 8 bytes).
//
// One block of 128 threads per head and CB = 64 value columns (all of fewer): a
// thread holds up to 16 float4 of S, four blocks an SM have 128 KB in flight, and
// the loads and stores are marked as streaming, since a state is not read again
// before the next token. 256 sequences x 16 heads at d = 128: 82.6 us, the copy
// rate; 103 with 256 threads on 32 columns and plain accesses, 92 with streaming
// alone. Rows are summed by shuffles, then across the warps.
#include "common.cuh"
#include "gated_delta.h"
#include "profile.h"

namespace kata {
namespace {

template <int DK, int CB> constexpr int step_threads() {
  return DK * CB / 4 < 128 ? DK * CB / 4 : 128;
}

template <int DK, int CB, typename Tin>
__global__ void __launch_bounds__(step_threads<DK, CB>())
gd_step_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
               const float *__restrict__ g, const float *__restrict__ beta, float *__restrict__ S,
               Tin *__restrict__ y, int H, int Hk, int DV) {
  constexpr int TH = step_threads<DK, CB>(), NC4 = CB / 4, NR = TH / NC4, PER = DK / NR;
  constexpr int NW = TH / 32;
  __shared__ float qs[DK], ks[DK];
  __shared__ float4 red[2][NW][NC4];
  const int tid = threadIdx.x, c4 = tid % NC4, r0 = tid / NC4, NB = DV / CB;
  const long long bh = blockIdx.x / NB;
  const int c0 = (blockIdx.x % NB) * CB;
  const size_t kh = (size_t)(bh / H) * Hk + (size_t)(bh % H) / (H / Hk);
  float *Sb = S + (size_t)bh * DK * DV + c0 + 4 * c4;
  float4 s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    s[i] = __ldcs(reinterpret_cast<const float4 *>(Sb + (size_t)(r0 + i * NR) * DV));
  for (int i = tid; i < DK; i += TH) {
    qs[i] = to_f(q[kh * DK + i]);
    ks[i] = to_f(k[kh * DK + i]);
  }
  const float a = expf(g[bh]), b = beta[bh];
  float vv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) vv[i] = to_f(v[(size_t)bh * DV + c0 + 4 * c4 + i]);
  __syncthreads();
  float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float x = ks[r0 + i * NR], z = qs[r0 + i * NR];
    u.x = fmaf(x, s[i].x, u.x); u.y = fmaf(x, s[i].y, u.y);
    u.z = fmaf(x, s[i].z, u.z); u.w = fmaf(x, s[i].w, u.w);
    w.x = fmaf(z, s[i].x, w.x); w.y = fmaf(z, s[i].y, w.y);
    w.z = fmaf(z, s[i].z, w.z); w.w = fmaf(z, s[i].w, w.w);
  }
#pragma unroll
  for (int off = 16; off >= NC4; off >>= 1) {
    u.x += __shfl_xor_sync(0xffffffffu, u.x, off); u.y += __shfl_xor_sync(0xffffffffu, u.y, off);
    u.z += __shfl_xor_sync(0xffffffffu, u.z, off); u.w += __shfl_xor_sync(0xffffffffu, u.w, off);
    w.x += __shfl_xor_sync(0xffffffffu, w.x, off); w.y += __shfl_xor_sync(0xffffffffu, w.y, off);
    w.z += __shfl_xor_sync(0xffffffffu, w.z, off); w.w += __shfl_xor_sync(0xffffffffu, w.w, off);
  }
  if (tid % 32 < NC4) {
    red[0][tid / 32][c4] = u;
    red[1][tid / 32][c4] = w;
  }
  __syncthreads();
  u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const float4 x = red[0][i][c4];
    u.x += x.x; u.y += x.y; u.z += x.z; u.w += x.w;
  }
  const float4 d = make_float4(b * (vv[0] - a * u.x), b * (vv[1] - a * u.y), b * (vv[2] - a * u.z),
                               b * (vv[3] - a * u.w));
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float x = ks[r0 + i * NR];
    __stcs(reinterpret_cast<float4 *>(Sb + (size_t)(r0 + i * NR) * DV),
           make_float4(fmaf(x, d.x, a * s[i].x), fmaf(x, d.y, a * s[i].y), fmaf(x, d.z, a * s[i].z),
                       fmaf(x, d.w, a * s[i].w)));
  }
  if (tid < 32) {                              // warp 0: k . q, then y
    float kq = 0.f;
    for (int i = tid; i < DK; i += 32) kq = fmaf(ks[i], qs[i], kq);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, off);
    if (tid < NC4) {
      w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float4 x = red[1][i][c4];
        w.x += x.x; w.y += x.y; w.z += x.z; w.w += x.w;
      }
      Tin *dst = y + (size_t)bh * DV + c0 + 4 * c4;
      dst[0] = from_f<Tin>(fmaf(kq, d.x, a * w.x));
      dst[1] = from_f<Tin>(fmaf(kq, d.y, a * w.y));
      dst[2] = from_f<Tin>(fmaf(kq, d.z, a * w.z));
      dst[3] = from_f<Tin>(fmaf(kq, d.w, a * w.w));
    }
  }
}

template <int DK, int CB, typename Tin>
cudaError_t launch(const GatedDeltaStep &a, int d_v) {
  ProfileScope prof("gd_step", a.stream);
  gd_step_kernel<DK, CB, Tin><<<(unsigned)(a.BH * (d_v / CB)), step_threads<DK, CB>(), 0, a.stream>>>(
      static_cast<const Tin *>(a.q), static_cast<const Tin *>(a.k), static_cast<const Tin *>(a.v), a.g,
      a.beta, a.S, static_cast<Tin *>(a.y), a.H, a.Hk, d_v);
  return cudaGetLastError();
}

}  // namespace

template <int DK, typename Tin> cudaError_t columns(const GatedDeltaStep &a, int d_v) {
  if (d_v == 16) return launch<DK, 16, Tin>(a, d_v);
  return d_v == 32 ? launch<DK, 32, Tin>(a, d_v) : launch<DK, 64, Tin>(a, d_v);
}

template <typename Tin> cudaError_t gated_delta_step(const GatedDeltaStep &a, int d_k, int d_v) {
  switch (d_k) {
    case 16: return columns<16, Tin>(a, d_v);
    case 32: return columns<32, Tin>(a, d_v);
    case 64: return columns<64, Tin>(a, d_v);
    case 128: return columns<128, Tin>(a, d_v);
    default: return cudaErrorNotSupported;
  }
}
template cudaError_t gated_delta_step<float>(const GatedDeltaStep &, int, int);
template cudaError_t gated_delta_step<__nv_bfloat16>(const GatedDeltaStep &, int, int);

}  // namespace kata
