// Launch descriptors of the gated delta rule (forward, gradient, one-token
// step), shared by its C ABI file and its kernel files.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kata {

constexpr int kGdChunk = 64;     // tokens a chunk, in every kernel of the family
// A log decay below this (a reset, -inf included) counts as this, so that sums and
// their differences stay finite. Its exponential is 0 in fp32, whose least value is
// e^-103.3 (and at half of which, e^-103.98, rounding turns to 0).
constexpr float kGdMinLogDecay = -110.f;
// SMs of a B200. Sizes the split of a sequence into segments; a constant, so that
// a workspace's size follows from the shape alone, with or without a device.
constexpr int kGdSms = 148;

// Tensors [B, heads, T, d], contiguous; value head h reads query / key head
// h / (H / Hk). BH = B * H value heads, N = ceil(T / kGdChunk) chunks.
struct GatedDeltaLaunch {
  const void *q, *k, *v;
  const float *g, *beta;
  void *o;                       // forward; null for the gradient
  const float *S0;               // nullable [BH][d_k][d_v]
  float *S_out;                  // forward: nullable
  long long BH;
  int H, Hk, T, N;
  cudaStream_t stream;
  // gradient
  const void *dout = nullptr;
  const float *dS = nullptr;     // nullable: the last state's gradient
  void *dq = nullptr, *dk = nullptr, *dv = nullptr;
  float *dg = nullptr, *dbeta = nullptr, *dS0 = nullptr;   // dS0 nullable
  // workspace regions (fp32 kernels)
  float *gates = nullptr;                       // [BH][N][3][64]
  float *M = nullptr, *P = nullptr;             // [BH][N][64][64]
  float *starts = nullptr, *ends = nullptr;     // [BH][N][d_k][d_v]: S and dS at the chunks' borders
  float *writes = nullptr, *dR = nullptr;       // [BH][T][d_v]
  float *dq_part = nullptr, *dk_part = nullptr; // [BH][T][d_k], only where heads share keys
  float *in_f32[7] = {};                        // fp32 q, k, v, dout, dq, dk, dv of a small bf16 gradient
  // G segments of seg_chunks chunks a head. A segment takes
  // a state S to F S + B and, back, its gradient E to F^T E + B'.
  unsigned *status = nullptr;
  int G = 1, seg_chunks = 0;
  float *F = nullptr;              // of segments 1 .. G - 2 [BH][G - 2]
  float *starts_seg = nullptr;     // [BH][G], 1 .. G - 1 used: B of the segment before, then the state
  float *ends_seg = nullptr;       // gradient [BH][G], 0 .. G - 2 used: B' of the segment behind, then dS
  uint8_t *img_S = nullptr, *img_D = nullptr, *img_dS = nullptr, *img_dR = nullptr;   // gradient, [BH][N]
  uint8_t *records = nullptr;      // what the solve leaves of each chunk [BH][N]
};

struct GatedDeltaStep {
  const void *q, *k, *v;
  const float *g, *beta;
  float *S;
  void *y;
  long long BH;
  int H, Hk;
  cudaStream_t stream;
};

// fp32 kernels.
cudaError_t gd_f32(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_f32_backward(const GatedDeltaLaunch &a, int d_k, int d_v);
void gd_f32_split(long long BH, int N, int d_k, int d_v, bool gradient, int *G, int *seg_chunks);
cudaError_t gd_f32_join(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_bf16_gradient_in_f32(const GatedDeltaLaunch &a, int d_k, int d_v);   // bf16 tensors
// Tensor-core forward (bf16, 16-byte aligned q, k, v, o).
// The kernels' head sizes: 64 or 128.
constexpr int gd_padded(int d) { return d <= 64 ? 64 : 128; }
#define GD_TC_DISPATCH(FN)                                                    \
  (gd_padded(d_k) == 64 ? (gd_padded(d_v) == 64 ? FN(64, 64) : FN(64, 128)) \
                        : (gd_padded(d_v) == 64 ? FN(128, 64) : FN(128, 128)))
void gd_tc_split(long long BH, int N, int d_k, int d_v, bool gradient, int *G, int *seg_chunks);
size_t gd_tc_record_bytes();
cudaError_t gd_tc_solve(const GatedDeltaLaunch &a, int d_k);
// Tensor-core gradient: the saved images of states and writes.
cudaError_t gd_tc_effect(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_save(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_reverse_effect(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_reverse(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_join(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_grads(const GatedDeltaLaunch &a, int d_k, int d_v);
cudaError_t gd_tc_grads_wide(const GatedDeltaLaunch &a, int d_k, int d_v);   // 64 < d_k
cudaError_t gd_tc_backward(const GatedDeltaLaunch &a, int d_k, int d_v);
// dq, dk of shared heads: the sums of the value heads' parts.
cudaError_t gd_sum_groups(const GatedDeltaLaunch &a, int d_k, bool bf16);
size_t gd_tc_state_image(int d_k, int d_v);
size_t gd_tc_write_image(int d_v);
cudaError_t gd_tc_forward(const GatedDeltaLaunch &a, int d_k, int d_v);
// Lets `kern` use `bytes` of dynamic shared memory on the current device; on every
// call, since a device reset forgets it.
#define GD_ALLOW_SMEM(kern, bytes)                                                                          \
  do {                                                                                                      \
    const cudaError_t e_ = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(bytes)); \
    if (e_ != cudaSuccess) return e_;                                                                       \
  } while (0)

template <typename Tin> cudaError_t gated_delta_step(const GatedDeltaStep &a, int d_k, int d_v);

}  // namespace kata
