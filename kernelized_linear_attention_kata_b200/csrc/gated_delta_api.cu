// C ABI of the gated delta rule: argument checks, workspace layout and kernel
// dispatch. The contract is in include/kata.h.
#include "../../include/kata.h"

#include <cuda_runtime.h>

#include <initializer_list>

#include "common.cuh"
#include "gated_delta.h"

using namespace kata;

namespace {

constexpr size_t kHeaderBytes = 256;   // status word + padding
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool head_size(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

kata_status_t check_shape(int B, int H_k, int H, int T, int d_k, int d_v, kata_dtype_t dtype) {
  if (B < 0 || H_k < 0 || H < 0 || T < 0) return KATA_ERR_INVALID_ARGUMENT;
  if (dtype != KATA_DTYPE_F32 && dtype != KATA_DTYPE_BF16) return KATA_ERR_UNSUPPORTED;
  if (!head_size(d_k) || !head_size(d_v)) return KATA_ERR_UNSUPPORTED;
  if (H > 0 && (H_k == 0 || H % H_k != 0)) return KATA_ERR_INVALID_ARGUMENT;
  if (T > 0x7fffffff - kGdChunk) return KATA_ERR_UNSUPPORTED;   // token indices stay in an int
  // one block per head, chunk and 16 or 32 value columns: the largest grid
  const long long N = T / kGdChunk + (T % kGdChunk != 0);
  const long long per_head = N > d_v / 16 ? N : d_v / 16;
  if ((long long)B * (H > H_k ? H : H_k) > 0x7fffffffLL / (per_head > 0 ? per_head : 1)) return KATA_ERR_UNSUPPORTED;
  return KATA_OK;
}

// Workspace: status header, then the regions of the launch descriptor in the
// order below. `bytes` counts, `place` also hands out the pointers.
struct Regions {
  unsigned char *base;
  size_t used = kHeaderBytes;
  unsigned char *take_bytes(size_t n) {
    unsigned char *p = base ? base + used : nullptr;
    used += align_up(n);
    return p;
  }
  float *take(size_t floats) { return reinterpret_cast<float *>(take_bytes(floats * sizeof(float))); }
};

// bf16 runs on the tensor cores (TMA loads make 16-byte alignment a condition),
// fp32 on kernels of its own.
bool on_tensor_cores(kata_dtype_t dtype) { return dtype == KATA_DTYPE_BF16; }

// The bf16 gradient of few tokens runs in fp32: the gradients of the gates are dots
// whose terms cancel, and with few tokens to a head nothing averages out what 16-bit
// operands leave. Of 512 heads the worst one's dg is off by 2e-2 of its norm at one
// token, 5e-5 at 4, 2.5e-5 at 16, 1.9e-5 at 32, 1e-5 from 64 on (in fp32: 1e-3,
// 2.5e-6, then 1e-6; the median head 3.5e-6 and 2e-7 at any length). A head's own
// tokens count, not the call's: a head has the same gradient in any batch. 31 tokens
// of 4 / 128 / 512 heads, d = 64: 58 / 83 / 260 us, 38 / 39 / 98 in bf16 halves.
bool few_tokens(int T) { return T < 32; }

bool aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
  return true;
}

// The tensor-core forward's regions (the gradient's first pass needs them too).
void place_chain(GatedDeltaLaunch &a, int d_k, int d_v, bool gradient, Regions &r) {
  if (a.BH > 0 && a.T > 0) gd_tc_split(a.BH, a.N, d_k, d_v, gradient, &a.G, &a.seg_chunks);
  a.records = r.take_bytes((size_t)a.BH * a.N * gd_tc_record_bytes());
  if (a.G > 1) {
    const size_t dk = gd_padded(d_k), dv = gd_padded(d_v);
    a.F = r.take((size_t)a.BH * (a.G - 2) * dk * dk);
    a.starts_seg = r.take((size_t)a.BH * a.G * dk * dv);
    if (gradient) a.ends_seg = r.take((size_t)a.BH * a.G * dk * dv);
  }
}

// The fp32 kernels' segments.
void place_segments(GatedDeltaLaunch &a, int d_k, int d_v, bool gradient, Regions &r) {
  a.seg_chunks = a.N;
  if (a.BH > 0 && a.T > 0) gd_f32_split(a.BH, a.N, d_k, d_v, gradient, &a.G, &a.seg_chunks);
  if (a.G > 1) {
    a.F = r.take((size_t)a.BH * (a.G - 2) * d_k * d_k);
    a.starts_seg = r.take((size_t)a.BH * a.G * d_k * d_v);
    if (gradient) a.ends_seg = r.take((size_t)a.BH * a.G * d_k * d_v);
  }
}

size_t place_forward(GatedDeltaLaunch &a, int d_k, int d_v, kata_dtype_t dtype, void *ws) {
  Regions r{static_cast<unsigned char *>(ws)};
  if (on_tensor_cores(dtype)) {
    place_chain(a, d_k, d_v, false, r);
    return r.used;
  }
  const size_t square = (size_t)a.BH * a.N * kGdChunk * kGdChunk;
  a.M = r.take(square);
  a.P = r.take(square);
  a.gates = r.take((size_t)a.BH * a.N * 3 * kGdChunk);
  place_segments(a, d_k, d_v, false, r);
  return r.used;
}

size_t place_backward(GatedDeltaLaunch &a, int d_k, int d_v, kata_dtype_t dtype, void *ws) {
  Regions r{static_cast<unsigned char *>(ws)};
  const size_t chunks = (size_t)a.BH * a.N, tokens = (size_t)a.BH * a.T;
  if (a.H != a.Hk) {
    a.dq_part = r.take(tokens * d_k);
    a.dk_part = r.take(tokens * d_k);
  }
  if (on_tensor_cores(dtype) && !few_tokens(a.T)) {
    place_chain(a, d_k, d_v, true, r);
    a.img_S = r.take_bytes(chunks * gd_tc_state_image(d_k, d_v));
    a.img_dS = r.take_bytes(chunks * gd_tc_state_image(d_k, d_v));
    a.img_D = r.take_bytes(chunks * gd_tc_write_image(d_v));
    a.img_dR = r.take_bytes(chunks * gd_tc_write_image(d_v));
    return r.used;
  }
  a.M = r.take(chunks * kGdChunk * kGdChunk);
  a.P = r.take(chunks * kGdChunk * kGdChunk);
  a.gates = r.take(chunks * 3 * kGdChunk);
  place_segments(a, d_k, d_v, true, r);
  a.starts = r.take(chunks * d_k * d_v);
  a.ends = r.take(chunks * d_k * d_v);
  a.writes = r.take(tokens * d_v);
  a.dR = r.take(tokens * d_v);
  if (on_tensor_cores(dtype)) {
    const size_t keys = a.H > 0 ? tokens / (a.H / a.Hk) * d_k : 0;
    const size_t n[7] = {keys, keys, tokens * d_v, tokens * d_v, keys, keys, tokens * d_v};
    for (int i = 0; i < 7; ++i) a.in_f32[i] = r.take(n[i]);
  }
  return r.used;
}

GatedDeltaLaunch describe(int B, int H_k, int H, int T) {
  GatedDeltaLaunch a{};
  a.BH = (long long)B * H;
  a.H = H;
  a.Hk = H_k;
  a.T = T;
  a.N = T / kGdChunk + (T % kGdChunk != 0);
  return a;
}

bool overlap(const float *x, const float *y, size_t floats) {
  if (!x || !y) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const uintptr_t n = floats * sizeof(float);
  return a < b + n && b < a + n;
}

// an empty sequence leaves the state (or its gradient) as it came
kata_status_t pass_state(const float *from, float *to, size_t floats, cudaStream_t stream) {
  if (!to || floats == 0) return KATA_OK;
  const size_t n = floats * sizeof(float);
  const cudaError_t e = from ? cudaMemcpyAsync(to, from, n, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(to, 0, n, stream);
  return e == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

kata_status_t check_workspace(const void *ws, size_t have, size_t need) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % kAlign != 0 || have < need) return KATA_ERR_WORKSPACE;
  return KATA_OK;
}

}  // namespace

extern "C" {

size_t kata_fwd_gated_delta_workspace_bytes(int B, int H_k, int H, int T, int d_k, int d_v,
                                            kata_dtype_t dtype) {
  if (check_shape(B, H_k, H, T, d_k, d_v, dtype) != KATA_OK) return 0;
  GatedDeltaLaunch a = describe(B, H_k, H, T);
  return place_forward(a, d_k, d_v, dtype, nullptr);
}

kata_status_t kata_fwd_gated_delta(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, void *o, int B, int H_k, int H, int T, int d_k,
                                   int d_v, kata_dtype_t dtype, const float *S0, float *S_out,
                                   void *workspace, size_t workspace_bytes, kata_stream_t stream_) {
  const kata_status_t shape = check_shape(B, H_k, H, T, d_k, d_v, dtype);
  if (shape != KATA_OK) return shape;
  GatedDeltaLaunch a = describe(B, H_k, H, T);
  const size_t need = place_forward(a, d_k, d_v, dtype, workspace);
  const kata_status_t ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != KATA_OK) return ws;
  a.stream = reinterpret_cast<cudaStream_t>(stream_);
  const size_t state = (size_t)a.BH * d_k * d_v;
  if (overlap(S0, S_out, state)) return KATA_ERR_INVALID_ARGUMENT;
  const bool tc = on_tensor_cores(dtype);
  if (a.BH > 0 && T > 0 &&
      (!q || !k || !v || !g || !beta || !o || (tc && !aligned16({q, k, v, o}))))
    return KATA_ERR_INVALID_ARGUMENT;
  const bool empty = a.BH == 0 || T == 0;                  // the fp32 kernels write the status themselves
  if ((tc || empty) && cudaMemsetAsync(workspace, 0, sizeof(unsigned), a.stream) != cudaSuccess) return KATA_ERR_CUDA;
  if (empty) return pass_state(S0, S_out, state, a.stream);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.o = o; a.S0 = S0; a.S_out = S_out;
  a.status = static_cast<unsigned *>(workspace);
  const cudaError_t e = tc ? gd_tc_forward(a, d_k, d_v) : gd_f32(a, d_k, d_v);
  return e == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

size_t kata_bwd_gated_delta_workspace_bytes(int B, int H_k, int H, int T, int d_k, int d_v,
                                            kata_dtype_t dtype) {
  if (check_shape(B, H_k, H, T, d_k, d_v, dtype) != KATA_OK) return 0;
  GatedDeltaLaunch a = describe(B, H_k, H, T);
  return place_backward(a, d_k, d_v, dtype, nullptr);
}

kata_status_t kata_bwd_gated_delta(const void *q, const void *k, const void *v, const float *g,
                                   const float *beta, const void *dout, const float *S0,
                                   const float *dS, void *dq, void *dk, void *dv, float *dg,
                                   float *dbeta, float *dS0, int B, int H_k, int H, int T, int d_k,
                                   int d_v, kata_dtype_t dtype, void *workspace,
                                   size_t workspace_bytes, kata_stream_t stream_) {
  const kata_status_t shape = check_shape(B, H_k, H, T, d_k, d_v, dtype);
  if (shape != KATA_OK) return shape;
  GatedDeltaLaunch a = describe(B, H_k, H, T);
  const size_t need = place_backward(a, d_k, d_v, dtype, workspace);
  const kata_status_t ws = check_workspace(workspace, workspace_bytes, need);
  if (ws != KATA_OK) return ws;
  a.stream = reinterpret_cast<cudaStream_t>(stream_);
  const size_t state = (size_t)a.BH * d_k * d_v;
  if (overlap(dS, dS0, state) || overlap(S0, dS0, state)) return KATA_ERR_INVALID_ARGUMENT;
  const bool tc = on_tensor_cores(dtype);
  if (a.BH > 0 && T > 0 &&
      (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta ||
       (tc && !aligned16({q, k, v, dout, dq, dk, dv}))))
    return KATA_ERR_INVALID_ARGUMENT;
  // no value heads: dq and dk are sums over none
  const size_t lone = H == 0 ? (size_t)B * H_k * T * d_k * (dtype == KATA_DTYPE_F32 ? 4 : 2) : 0;
  if (lone > 0) {
    if (!dq || !dk) return KATA_ERR_INVALID_ARGUMENT;
    if (cudaMemsetAsync(dq, 0, lone, a.stream) != cudaSuccess || cudaMemsetAsync(dk, 0, lone, a.stream) != cudaSuccess)
      return KATA_ERR_CUDA;
  }
  const bool empty = a.BH == 0 || T == 0;                  // the fp32 kernels write the status themselves
  if ((tc || empty) && cudaMemsetAsync(workspace, 0, sizeof(unsigned), a.stream) != cudaSuccess) return KATA_ERR_CUDA;
  if (empty) return pass_state(dS, dS0, state, a.stream);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0;
  a.dout = dout; a.dS = dS; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dS0 = dS0;
  a.status = static_cast<unsigned *>(workspace);
  const cudaError_t e = !tc             ? gd_f32_backward(a, d_k, d_v)
                        : few_tokens(T) ? gd_bf16_gradient_in_f32(a, d_k, d_v)
                                        : gd_tc_backward(a, d_k, d_v);
  return e == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

kata_status_t kata_gated_delta_step(const void *q, const void *k, const void *v, const float *g,
                                    const float *beta, float *S, void *y, int B, int H_k, int H,
                                    int d_k, int d_v, kata_dtype_t dtype, kata_stream_t stream_) {
  const kata_status_t shape = check_shape(B, H_k, H, 1, d_k, d_v, dtype);
  if (shape != KATA_OK) return shape;
  const long long BH = (long long)B * H;
  if (BH == 0) return KATA_OK;
  if (!q || !k || !v || !g || !beta || !S || !y) return KATA_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(S) % 16 != 0) return KATA_ERR_INVALID_ARGUMENT;
  const GatedDeltaStep a{q, k, v, g, beta, S, y, BH, H, H_k, reinterpret_cast<cudaStream_t>(stream_)};
  const cudaError_t e = dtype == KATA_DTYPE_F32 ? gated_delta_step<float>(a, d_k, d_v)
                                                : gated_delta_step<__nv_bfloat16>(a, d_k, d_v);
  return e == cudaSuccess ? KATA_OK : KATA_ERR_CUDA;
}

}  // extern "C"
