// Building blocks of the gated delta rule's tensor-core kernels: operand
// splitting, barrier waits by whole warps, bounded draining, bulk copies, the
// record of a chunk, and the chunk solve (I + L)^-1 of four warps.
#pragma once

#include "gated_delta.h"
#include "gated_delta_sync.h"
#include "tc_common.cuh"

namespace kata {
namespace gdtc {

using namespace tc;

constexpr int kC = kGdChunk;         // 64 tokens a chunk
constexpr int kPanel = 8192;         // 64 rows x 128 bytes: one 64-column bf16 panel
constexpr int kLs = kC + 4;          // row stride of the solve's fp32 matrix
constexpr int kSpins = 64;           // tests of a barrier before a thread suspends

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

// An fp32 pair as two bf16 pairs, x = hi + lo up to 2^-17 of its binade. The
// tensor core multiplies bf16: an fp32 operand enters as hi + lo (q, k, v and
// dout are bf16 already and enter as they are), so that a product keeps 16
// bits of it instead of 8. The sums are fp32 throughout. What this costs: S_out, dS0,
// dg and dbeta are off by 3e-6 to 6e-6 of their norm instead of 1e-7 to 4e-7; a bf16
// output lies one step beside the exact value's rounding in 0.4 % of its entries. A
// third half would need 192 columns for S where d_k = 128 has 128 of the 512 left.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(x.x, x.y);
  const float2 h = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
  const float2 rest = __ffma2_rn(h, make_float2(-1.f, -1.f), x);
  lo = pack_bf16x2(rest.x, rest.y);
}
__device__ __forceinline__ float2 as_float2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// A wait by a whole warp: the result is the same in all lanes. Most waits of the
// chains end within a few tests; a suspended thread comes back later than that.
// Once a wait has given up, all others do at once: a warp of the chains then goes
// on through its hand-overs (which it now waits for, see below) and leaves garbage
// behind, and the block reports it.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
#pragma unroll 1
  for (int i = 0; i < kSpins; ++i)
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(bar, parity, abort_flag));
}
// The chains' warps: 0-15 the state warps (four warpgroups, each a quarter of the
// columns of keys or tokens), 16 the MMA issuer, 17 the loads and the output
// stores, 18 the saves. A pass of the state warps waits for its own tensor memory,
// shared memory and conversions more than it computes: with 8 warps of twice the
// columns a pass took 1.5 times as long (1 or 2 warps a scheduler).
constexpr int kStateWarps = 16, kIssuer = 16, kLoader = 17, kSaver = 18, kChainThreads = 19 * 32;

// Hardware barrier `id` of the state warps and the issuer: the state warps pass,
// the issuer waits for them. Through an mbarrier the same takes 300 cycles
// instead of 40, three or four times a chunk. A hardware barrier counts warps, not
// which: a state warp must not come to it again before the issuer has been there.
// Its waits see to that as long as none of them has given up (`ok`: of this warp);
// from then on the warp waits at the hand-overs themselves (gated_delta_sync.h).
__device__ __forceinline__ void hand_over(int id, bool ok) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p bar.arrive %0, %1;\n\t"
      "@!p bar.sync %0, %1;\n\t}" ::"r"(id),
      "n"(32 * (kStateWarps + 1)), "r"((uint32_t)gdsync::passes(ok))
      : "memory");
}
__device__ __forceinline__ void take_over(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * (kStateWarps + 1)) : "memory");
}
// One arrival for a warp, after all its lanes got here.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}
// A place is free for the next load into it.
__device__ __forceinline__ bool free_to_load(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  const bool waited = mbar_wait(bar, parity, abort_flag);
  return gdsync::may_load(waited, *abort_flag != 0);
}
// Waits (at most kWaitLimitNs) for copies or MMAs in flight before the block ends.
static __device__ __noinline__ void drain(uint64_t *bar, uint32_t parity) {
  const uint64_t start = global_ns();
  while (!mbar_try_wait(bar, parity, kSuspendHintNs))
    if (global_ns() - start > kWaitLimitNs) return;
}

// Untiled bulk copies (16-byte aligned, multiples of 16 bytes, no multicast).
__device__ __forceinline__ void bulk_load(void *smem_dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(smem_src)), "r"(bytes)
               : "memory");
}

// What the chains need of a chunk beside q, k and v, as the solve leaves it in
// the workspace: e^{G_t}, e^{G_C - G_t} and beta_t, then 64 x 64 bf16 tiles in
// the layout of an MMA operand (128-byte rows, 128B swizzle), each as hi and
// lo: M, then P.
constexpr int kRecGates = 3 * kC * 4;
constexpr int kRecM = kRecGates, kRecP = kRecM + 2 * kPanel, kRecBytes = kRecP + 2 * kPanel;

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
  float from_start[kC];              // e^{G_t}
  float to_end[kC];                  // e^{G_C - G_t}
  float beta[kC];
  float hi[kC], lo[kC];              // G_t
  float to_block[kC];                // e^{G_a - G_t}, a = t | 7
};
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a + b as a rounded sum and its error.
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return make_float2(s, (a - (s - t)) + (b - t));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  const float l = s.y + (a.y + b.y);
  const float h = s.x + l;
  return make_float2(h, l - (h - s.x));
}
// Gates of one chunk by one warp, two tokens a lane; gx, gy are their log decays.
__device__ __forceinline__ void make_gates(Gates &s, float gx, float gy, float bx, float by) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eRest = 1.92596299112661746887e-8f;
  const int lane = threadIdx.x % 32;
  auto units = [&](float x) {                              // x / log 2 as two floats
    x = x < kGdMinLogDecay ? kGdMinLogDecay : x;
    const float h = x * kLog2e;
    return make_float2(h, fmaf(x, kLog2eRest, fmaf(x, kLog2e, -h)));
  };
  const float2 x = units(gx), y = units(gy);
  float2 sum = add2(x, y);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float2 up = make_float2(__shfl_up_sync(0xffffffffu, sum.x, off), __shfl_up_sync(0xffffffffu, sum.y, off));
    if (lane >= off) sum = add2(up, sum);
  }
  // the first token of the lane, from the sum before it: no difference of sums
  float2 before = make_float2(__shfl_up_sync(0xffffffffu, sum.x, 1), __shfl_up_sync(0xffffffffu, sum.y, 1));
  if (lane == 0) before = make_float2(0.f, 0.f);
  auto from = [&](int l) {
    return make_float2(__shfl_sync(0xffffffffu, sum.x, l), __shfl_sync(0xffffffffu, sum.y, l));
  };
  const float2 last = from(31), block = from(lane | 3);
  const float2 G[2] = {add2(before, x), sum};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = 2 * lane + i;
    s.hi[t] = G[i].x;
    s.lo[t] = G[i].y;
    s.from_start[t] = exp2_fast(G[i].x + G[i].y);
    s.to_end[t] = exp2_fast((last.x - G[i].x) + (last.y - G[i].y));
    s.to_block[t] = exp2_fast((block.x - G[i].x) + (block.y - G[i].y));
    s.beta[t] = i ? by : bx;
  }
}

// A row's part in the causal decay matrix: w[j] = e^{G_t - G_s} for the eight
// tokens s of its own block, 0 behind the row (skip = 1: and on the diagonal).
struct RowDecay {
  float hi, lo, own[8];
  int block;
};
__device__ __forceinline__ RowDecay row_decay(const Gates &g, int t, int skip) {
  RowDecay d;
  d.hi = g.hi[t];
  d.lo = g.lo[t];
  d.block = t / 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float w = exp2_fast((d.hi - g.hi[t / 8 * 8 + j]) + (d.lo - g.lo[t / 8 * 8 + j]));
    d.own[j] = j + skip <= t % 8 ? w : 0.f;
  }
  return d;
}
// Columns 8 block .. 8 block + 7 of the row times x.
__device__ __forceinline__ void decay8(const Gates &g, const RowDecay &d, int block, const uint32_t (&x)[8],
                                       float (&out)[8]) {
  const float f = exp2_fast((d.hi - g.hi[8 * block + 7]) + (d.lo - g.lo[8 * block + 7]));
  const float4 e0 = *reinterpret_cast<const float4 *>(&g.to_block[8 * block]);
  const float4 e1 = *reinterpret_cast<const float4 *>(&g.to_block[8 * block + 4]);
  const float e[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float w = block < d.block ? f * e[j] : (block == d.block ? d.own[j] : 0.f);
    out[j] = w * __uint_as_float(x[j]);
  }
}

// (I + L)^-1 of a chunk, in `Lm` (row stride kLs), by blocks of 16, 32, 64:
//   [[A, 0], [X, B]]^-1 = [[A', 0], [-B' X A', B']].
// The 16-blocks by forward substitution, the products on the warp's tensor
// instructions in three TF32 products an fp32 pair (x = hi + lo up to 2^-23):
// on the CUDA cores every operand of these small products would be a shared-
// memory broadcast, which fills the 128 B/cycle return path with one value.
// Block substitution is as stable as the triangular solve itself, where
// repeated squaring of L would not be (powers of L grow with repeated keys).
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
  // rounded half up in the bits: the conversion instruction runs at an eighth of
  // this rate (a NaN that the carry clears is still one in lo)
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));           // the tensor core drops its low bits
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc (16 x 16, two n-tiles) = A (16 x K) B (K x 16) by one warp; element (r,
// k) of A at A[r * ra + k * ca], B and the result in rows of kLs.
template <int K>
__device__ __forceinline__ void product16(const float *A, int ra, int ca, const float *B, float (&acc)[2][4]) {
  const int g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[0][i] = acc[1][i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < K; k += 8) {
    uint32_t ah[4], al[4], bh[2][2], bl[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      split_tf32(A[(g + 8 * (i & 1)) * ra + (k + t + 4 * (i >> 1)) * ca], ah[i], al[i]);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) split_tf32(B[(k + t + 4 * i) * kLs + 8 * n + g], bh[n][i], bl[n][i]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};                   // the tensor core cuts its sums: they are added here
      mma_tf32(d, al, bh[n]);
      mma_tf32(d, ah, bl[n]);
      mma_tf32(d, ah, bh[n]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] += d[i];
    }
  }
}
__device__ __forceinline__ void store16(float *out, const float (&acc)[2][4], float sign) {
  const int g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    *reinterpret_cast<float2 *>(out + g * kLs + 8 * n + 2 * t) = make_float2(sign * acc[n][0], sign * acc[n][1]);
    *reinterpret_cast<float2 *>(out + (g + 8) * kLs + 8 * n + 2 * t) =
        make_float2(sign * acc[n][2], sign * acc[n][3]);
  }
}
// One warp inverts a 32-block given transposed (entry (t, s) of L at [s][t]):
// a half warp a 16-block, lane j its column j; once x_s is known every later
// x_t takes its term. Its own rows of L are all it reads.
__device__ __forceinline__ void invert_diagonal(float *blk) {
  const int lane = threadIdx.x % 32, half = lane / 16, j = lane % 16;
  float *sub = blk + 16 * half * (kLs + 1);
  float2 x[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) x[t] = make_float2(2 * t == j ? 1.f : 0.f, 2 * t + 1 == j ? 1.f : 0.f);
#pragma unroll
  for (int s = 0; s < 15; ++s) {
    const float xs = s % 2 ? -x[s / 2].y : -x[s / 2].x;
    const float2 m = make_float2(xs, xs);
#pragma unroll
    for (int t = (s + 1) / 4 * 4; t < 16; t += 4) {        // entries t <= s are zero
      const float4 l = *reinterpret_cast<const float4 *>(sub + s * kLs + t);
      x[t / 2] = __ffma2_rn(make_float2(l.x, l.y), m, x[t / 2]);
      x[t / 2 + 1] = __ffma2_rn(make_float2(l.z, l.w), m, x[t / 2 + 1]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < 16; ++t) sub[t * kLs + j] = t % 2 ? x[t / 2].y : x[t / 2].x;
  __syncwarp();
  float acc[2][4];
  product16<16>(blk + 16, 1, kLs, blk, acc);               // X A', X transposed in the upper right
  store16(blk + 16 * kLs, acc, 1.f);
  __syncwarp();
  product16<16>(blk + 16 * (kLs + 1), kLs, 1, blk + 16 * kLs, acc);
  __syncwarp();
  store16(blk + 16 * kLs, acc, -1.f);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  *reinterpret_cast<float4 *>(blk + j * kLs + 16 + 8 * half) = zero;
  *reinterpret_cast<float4 *>(blk + j * kLs + 20 + 8 * half) = zero;
}
// After both 32-blocks (and a barrier): the lower left one, by four warps, X A'
// into the upper right block (zero in L) and then -B' times it.
__device__ __forceinline__ void invert_corner(float *Lm) {
  const int w = threadIdx.x / 32 % 4, r = 16 * (w & 1), c = 16 * (w >> 1);
#pragma unroll 1
  for (int step = 0; step < 2; ++step) {
    float acc[2][4];
    product16<32>(Lm + 32 * kLs + 32 * step + r * kLs, kLs, 1, Lm + 32 * step + c, acc);
    store16(Lm + (step ? 32 * kLs : 32) + r * kLs + c, acc, step ? -1.f : 1.f);
    __syncthreads();
  }
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

// The inverse as bf16 hi / lo tiles, two threads a row. The tiles may lie over Lm.
__device__ __forceinline__ void store_inverse(const float *Lm, uint8_t *hi_tile, uint8_t *lo_tile) {
  const int i = threadIdx.x % 128, t = i / 2, half = i % 2;
  const bool zero = t < 32 && half == 1;
  float4 m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = *reinterpret_cast<const float4 *>(Lm + t * kLs + 32 * half + 4 * j);
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 a = m[2 * c], b = m[2 * c + 1];
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = zero ? 0.f : x[j];
    store_split8(hi_tile, lo_tile, t, 4 * half + c, x);
  }
}

// 16 values of a thread's row (one TMEM lane) as an operand: a 16-deep step of
// hi, then of lo.
__device__ __forceinline__ void put16(uint32_t col, const float2 *x) {
  uint32_t y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2(x[i], y[i], y[8 + i]);
  tmem_st16(col, y);
}
// 8 x COUNT values of row `row` of a saved image (128-byte rows, 64 values a
// panel of `rows` rows), from value `first`; the hi or the lo halves.
template <int COUNT>
__device__ __forceinline__ void stage_row(uint8_t *image, int rows, int row, int first, const float2 *x, bool lo_half) {
#pragma unroll
  for (int j = 0; j < COUNT; ++j) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[4 * j + i], h[i], l[i]);
    const int at = first + 8 * j;
    *reinterpret_cast<uint4 *>(image + (size_t)(at / 64) * rows * 128 + sw128(row, at % 64 / 8)) =
        lo_half ? make_uint4(l[0], l[1], l[2], l[3]) : make_uint4(h[0], h[1], h[2], h[3]);
  }
}
__device__ __forceinline__ float2 gate2(const float *g, int i) { return *reinterpret_cast<const float2 *>(g + i); }

// Saved images of a chunk for its gradients: a state (or its gradient) [d_v
// rows][d_k] and the writes (or theirs) [d_v rows][64 tokens], hi, then lo.
constexpr size_t state_image(int dk, int dv) { return (size_t)dk * dv * 4; }
constexpr size_t write_image(int dv) { return (size_t)kC * dv * 4; }

}  // namespace gdtc
}  // namespace kata
