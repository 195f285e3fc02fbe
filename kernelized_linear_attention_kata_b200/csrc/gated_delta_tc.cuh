// Building blocks of the gated delta rule's tensor-core kernels: operand
// splitting, barrier waits by whole warps, bounded draining, and the chunk
// solve (I + L)^-1 of four warps.
#pragma once

#include "gated_delta.h"
#include "tc_common.cuh"

namespace kata {
namespace gdtc {

using namespace tc;

constexpr int kC = kGdChunk;         // 64 tokens a chunk
constexpr int kPanel = 8192;         // 64 rows x 128 bytes: one 64-column bf16 panel
constexpr int kLs = kC + 4;          // row stride of the solve's fp32 matrix
constexpr float kMinLogDecay = -100.f;

// An fp32 pair as two bf16 pairs, x = hi + lo up to 2^-17 of its binade. The
// tensor core multiplies bf16: an fp32 operand enters as hi + lo (q, k, v and
// dout are bf16 already and enter as they are), so that a product keeps 16
// bits of it instead of 8. The sums are fp32 throughout.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 h = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  const float2 rest = __ffma2_rn(h, make_float2(-1.f, -1.f), x);
  lo = pack_bf16x2(rest.x, rest.y);
}
__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// The bounded wait of tc_common.cuh, in line: a kernel that moves registers
// between its warpgroups makes no calls.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  if (mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity, kSuspendHintNs)) return true;
  const uint64_t start = global_ns();
  while (!mbar_try_wait(bar, parity, kSuspendHintNs)) {
    if (*abort_flag) return false;
    if (global_ns() - start > kWaitLimitNs) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// A wait by a whole warp: the result is the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}
// One arrival for a warp, after all its lanes got here.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}
// Waits (at most kWaitLimitNs) for copies or MMAs in flight after an abort.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
  const uint64_t start = global_ns();
  while (!mbar_try_wait(bar, parity, kSuspendHintNs))
    if (global_ns() - start > kWaitLimitNs) return;
}

// Byte offset of 16-byte chunk c of row r in a 128-byte-row tile, 128B swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)r * 128u + (uint32_t)((c ^ (r & 7)) << 4);
}

// A chunk's gates in shared memory. G is the running sum of the log decays in
// units of log 2, kept as two floats: their differences give the decay ratios
// to fp32 accuracy however large G grows. A ratio e^{G_t - G_s} with s in a
// block of 8 tokens before t's is taken as e^{G_t - G_a} e^{G_a - G_s}, a the
// block's last token: both exponents are <= 0 (for g <= 0), and a row needs 8
// exponentials plus those of its own block instead of 64.
struct Gates {
  float hi[kC], lo[kC];              // G_t
  float from_start[kC];              // e^{G_t}
  float to_end[kC];                  // e^{G_C - G_t}
  float to_block[kC];                // e^{G_a - G_t}, a = t | 7
  float beta[kC];
};
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float decay_ratio(const Gates &g, float hi_t, float lo_t, int s) {
  return exp2_fast((hi_t - g.hi[s]) + (lo_t - g.lo[s]));
}

// Gates of one chunk by one warp, two tokens a lane; gx, gy are their log decays.
__device__ __forceinline__ void make_gates(Gates &s, float gx, float gy, float bx, float by) {
  const int lane = threadIdx.x % 32;
  const double x = (double)(gx < kMinLogDecay ? kMinLogDecay : gx) * 1.4426950408889634;
  const double y = (double)(gy < kMinLogDecay ? kMinLogDecay : gy) * 1.4426950408889634;
  double sum = x + y;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += up;
  }
  const double last = __shfl_sync(0xffffffffu, sum, 31);
  const double block = __shfl_sync(0xffffffffu, sum, lane | 3);
  const double G[2] = {sum - y, sum};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * lane + i;
    const float hi = (float)G[i];
    s.hi[t] = hi;
    s.lo[t] = (float)(G[i] - (double)hi);
    s.from_start[t] = exp2f((float)G[i]);
    s.to_end[t] = exp2f((float)(last - G[i]));
    s.to_block[t] = exp2f((float)(block - G[i]));
    s.beta[t] = i ? by : bx;
  }
}

// Row t, columns s = 8 block .. 8 block + 7 of the causal decay matrix times
// x: e^{G_t - G_s} x_s for s <= t (STRICT: s < t), else 0. `same`: the row may
// lie in this block or before it.
template <bool STRICT, bool SAME>
__device__ __forceinline__ void decay8(const Gates &g, int t, float hi_t, float lo_t, int block,
                                       const uint32_t *x, float (&out)[8]) {
  const int rel = t / 8 - block;
  const float f = decay_ratio(g, hi_t, lo_t, 8 * block + 7);
  const float4 e0 = *reinterpret_cast<const float4 *>(&g.to_block[8 * block]);
  const float4 e1 = *reinterpret_cast<const float4 *>(&g.to_block[8 * block + 4]);
  const float e[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int s = 8 * block + j;
    float w = f * e[j];
    if (SAME) {
      const bool seen = STRICT ? s < t : s <= t;
      w = rel > 0 ? w : decay_ratio(g, hi_t, lo_t, s);
      out[j] = seen ? w * __uint_as_float(x[j]) : 0.f;
    } else {
      out[j] = w * __uint_as_float(x[j]);
    }
  }
}

// Register split of a block of four warpgroups, launched with 128 a thread.
template <int R> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Barrier of the four warps of the chunk-local group (the 128 threads after
// the eight state warps). Its callers reach it in every round, aborted or not.
__device__ __forceinline__ void intra_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// (I + L)^-1 by blocks of 32, four warps, in `Lm` (row stride kLs):
//   [[A, 0], [X, B]]^-1 = [[A', 0], [-B' X A', B']].
// Warp w < 2 inverts diagonal block w, given transposed: lane j solves column
// j in registers, and once x_s is known every later x_t takes its term (496
// independent multiply-adds a lane, a dependent chain of 32). Its own rows of
// L are all it reads, so only the warp has to have written them. Forward
// substitution and block products are as stable as the triangular solve
// itself, where repeated squaring of L would not be (powers of L grow with
// repeated keys).
__device__ __forceinline__ void invert_diagonal(float *Lm, int w) {
  const int lane = threadIdx.x % 32;
  float *blk = Lm + (32 * w) * kLs + 32 * w;
  float2 x[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) x[t] = make_float2(2 * t == lane ? 1.f : 0.f, 2 * t + 1 == lane ? 1.f : 0.f);
#pragma unroll
  for (int s = 0; s < 31; ++s) {
    const float xs = s % 2 ? -x[s / 2].y : -x[s / 2].x;
    const float2 m = make_float2(xs, xs);
#pragma unroll
    for (int t = (s + 1) / 4 * 4; t < 32; t += 4) {        // entries t <= s are zero
      const float4 l = *reinterpret_cast<const float4 *>(blk + s * kLs + t);
      x[t / 2] = __ffma2_rn(make_float2(l.x, l.y), m, x[t / 2]);
      x[t / 2 + 1] = __ffma2_rn(make_float2(l.z, l.w), m, x[t / 2 + 1]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < 32; ++t) blk[t * kLs + lane] = t % 2 ? x[t / 2].y : x[t / 2].x;
}
// 32 x 32 x 32 product by 128 threads: out = sign * A B (all row stride kLs).
__device__ __forceinline__ void block_product(const float *A, const float *B, float *out, float sign) {
  const int i = threadIdx.x % 128, r = 2 * (i / 8), c = 4 * (i % 8);
  float acc[2][4] = {};
#pragma unroll
  for (int u = 0; u < 32; u += 4) {
    const float4 a0 = *reinterpret_cast<const float4 *>(A + r * kLs + u);
    const float4 a1 = *reinterpret_cast<const float4 *>(A + (r + 1) * kLs + u);
    const float l0[4] = {a0.x, a0.y, a0.z, a0.w}, l1[4] = {a1.x, a1.y, a1.z, a1.w};
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float4 b = *reinterpret_cast<const float4 *>(B + (u + v) * kLs + c);
      acc[0][0] = fmaf(l0[v], b.x, acc[0][0]); acc[0][1] = fmaf(l0[v], b.y, acc[0][1]);
      acc[0][2] = fmaf(l0[v], b.z, acc[0][2]); acc[0][3] = fmaf(l0[v], b.w, acc[0][3]);
      acc[1][0] = fmaf(l1[v], b.x, acc[1][0]); acc[1][1] = fmaf(l1[v], b.y, acc[1][1]);
      acc[1][2] = fmaf(l1[v], b.z, acc[1][2]); acc[1][3] = fmaf(l1[v], b.w, acc[1][3]);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    *reinterpret_cast<float4 *>(out + (r + k) * kLs + c) =
        make_float4(sign * acc[k][0], sign * acc[k][1], sign * acc[k][2], sign * acc[k][3]);
}
// After both diagonal blocks (and a barrier): the lower left block. The upper
// right block, zero in L, holds the product in between.
__device__ __forceinline__ void invert_corner(float *Lm) {
  block_product(Lm + 32 * kLs, Lm, Lm + 32, 1.f);
  intra_sync();
  block_product(Lm + 32 * kLs + 32, Lm + 32, Lm + 32 * kLs, -1.f);
  intra_sync();
}

// Row `row` of a 64-column bf16 tile (hi and lo planes, 128B swizzle): 8
// values at 16-byte chunk c.
__device__ __forceinline__ void store_split8(uint8_t *hi_tile, uint8_t *lo_tile, int row, int c,
                                             const float (&x)[8]) {
  uint4 h, l;
  split2(make_float2(x[0], x[1]), h.x, l.x);
  split2(make_float2(x[2], x[3]), h.y, l.y);
  split2(make_float2(x[4], x[5]), h.z, l.z);
  split2(make_float2(x[6], x[7]), h.w, l.w);
  *reinterpret_cast<uint4 *>(hi_tile + sw128(row, c)) = h;
  *reinterpret_cast<uint4 *>(lo_tile + sw128(row, c)) = l;
}

// The inverse times diag(beta) (BETA) as bf16 hi / lo tiles, two threads a row.
template <bool BETA>
__device__ __forceinline__ void store_inverse(const float *Lm, const Gates &g, uint8_t *hi_tile,
                                              uint8_t *lo_tile) {
  const int i = threadIdx.x % 128, t = i / 2, half = i % 2;
  const bool zero = t < 32 && half == 1;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int s0 = 32 * half + 8 * c;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 m = *reinterpret_cast<const float4 *>(Lm + t * kLs + s0 + j);
      const float4 b = *reinterpret_cast<const float4 *>(&g.beta[s0 + j]);
      x[j] = zero ? 0.f : (BETA ? m.x * b.x : m.x);
      x[j + 1] = zero ? 0.f : (BETA ? m.y * b.y : m.y);
      x[j + 2] = zero ? 0.f : (BETA ? m.z * b.z : m.z);
      x[j + 3] = zero ? 0.f : (BETA ? m.w * b.w : m.w);
    }
    store_split8(hi_tile, lo_tile, t, 4 * half + c, x);
  }
}

}  // namespace gdtc
}  // namespace kata
