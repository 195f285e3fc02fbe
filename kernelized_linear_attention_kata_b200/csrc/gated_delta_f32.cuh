// The gated delta rule in fp32: solve, chain, reverse chain and gradients.
//
//   S_t = e^{g_t} S_{t-1} + k_t d_t^T,  d_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),
//   o_t = S_t^T q_t.
//
// In chunks of C = 64 tokens from the chunk's starting state S (exact), with
// G the running sum of g inside the chunk and W_ts = e^{G_t - G_s}, s <= t:
//   L_ts = beta_t W_ts k_t.k_s (s < t),  M = (I + L)^-1,  P_ts = W_ts q_t.k_s (s <= t)
//   R = beta (V - e^G K S),  D = M R,  O = e^G Q S + P D,
//   S' = e^{G_C} S + (e^{G_C - G} K)^T D.
// Gradient, from dO and dS' = dL/dS':
//   dD = P^T dO + e^{G_C - G} K dS',  dR = M^T dD,  dV = beta dR,
//   dS = e^{G_C} dS' + (e^G Q)^T dO - (e^G K)^T dV,
//   dL = -dR D^T (s < t),  dP = dO D^T (s <= t),
// and the chain rule of L, P and the decays for dq, dk, dg, dbeta.
//
// Products run on the warp tensor instructions in three TF32 products an fp32
// pair: x = hi + lo, hi rounded to 11 bits and lo cut to 11, so a product loses
// 2^-23 of its factors. On the CUDA cores the same chain took 2.8 times as
// long (204 us, now 73, at 32 heads of 1023 tokens, d = 64): a 2 x 4 register
// tile reads 12 words of shared memory for 32 FMAs.
//
// The running sums are kept in fp64 and differenced there: with strong decays
// G reaches thousands, and an fp32 difference of two such sums would lose the
// ratio's digits. Resets (kGdMinLogDecay) keep the differences finite.
//
// Kernels: solve (M, P and the decays of every chunk, all chunks at once),
// chain (one block per head, segment and CB value columns walks the chunks: the
// columns of S follow the rule on their own), chain_reverse (dS, dR, dV, last
// chunk first), grads (dq, dk, dg, dbeta, all chunks at once). Few heads are cut
// into segments as in bf16: their effects first, joined by gated_delta_join.cu.
#pragma once

#include "common.cuh"
#include "gated_delta.h"
#include "gated_delta_tc.cuh"
#include "profile.h"

namespace kata {
namespace gd {

constexpr int kC = kGdChunk;
constexpr int kThreads = 256;
constexpr int kLD = kC + 4;          // row stride of a 64 x 64 matrix
constexpr int kRec = 3 * kC;         // a chunk's gates in the workspace: e^G, e^{G_C - G}, beta

__device__ __forceinline__ float clamp_decay(float g) { return g < kGdMinLogDecay ? kGdMinLogDecay : g; }

// acc += A B for an M x N tile, operands in shared memory, 8 warps. A[m][k] at
// A[m * LDA + k] (TA: A[k * LDA + m]); B[k][n] at B[k * LDB + n] (TB: B[n * LDB
// + k]), B's rows times scale[k] if given. A warp owns 16 MT rows x 8 NT columns,
// a thread of it rows row(i) and columns col(j); col(j), j even, and the next lie
// side by side. Where there are fewer than 8 tiles, warps beyond them are idle.
template <int M, int N, bool TA, bool TB, int LDA, int LDB>
struct Gemm {
  static constexpr int kTilesM = M / 16, kTilesN = N / 8;
  static constexpr int WM = kTilesM < 8 ? kTilesM : 8;                       // warps along the rows
  static constexpr int WN = 8 / WM < kTilesN ? 8 / WM : kTilesN;
  static constexpr int MT = kTilesM / WM, NT = kTilesN / WN, TM = 2 * MT, TN = 2 * NT;
  static_assert(WM * MT * 16 == M && WN * NT * 8 == N, "tile split");
  static __device__ __forceinline__ int wm() { return threadIdx.x / 32 % WM; }
  static __device__ __forceinline__ int wn() { return threadIdx.x / 32 / WM; }
  static __device__ __forceinline__ bool active() { return WM * WN == 8 || wn() < WN; }
  static __device__ __forceinline__ int row(int i) {
    return wm() * 16 * MT + i / 2 * 16 + i % 2 * 8 + threadIdx.x % 32 / 4;
  }
  static __device__ __forceinline__ int col(int j) {
    return wn() * 8 * NT + j / 2 * 8 + threadIdx.x % 4 * 2 + j % 2;
  }
  static __device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
  }
  struct Right {
    uint32_t hi[NT][2], lo[NT][2];
  };
  static __device__ __forceinline__ void right(Right &r, const float *B, int k, const float *scale) {
    const int g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = wn() * 8 * NT + 8 * n + g, d = k + t + 4 * i;
        float x = TB ? B[c * LDB + d] : B[d * LDB + c];
        if (scale) x *= scale[d];
        gdtc::split_tf32(x, r.hi[n][i], r.lo[n][i]);
      }
  }
  static __device__ __forceinline__ void step(const float *A, int k, const Right &r, float (&acc)[TM][TN]) {
    const int g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t ah[4], al[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int a = (wm() * MT + m) * 16 + g + 8 * (i & 1), d = k + t + 4 * (i >> 1);
        gdtc::split_tf32(TA ? A[d * LDA + a] : A[a * LDA + d], ah[i], al[i]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // summed here: the tensor core cuts its sums (a chain of 24 loses 1e-6)
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        gdtc::mma_tf32(d, al, r.hi[n]);
        gdtc::mma_tf32(d, ah, r.lo[n]);
        gdtc::mma_tf32(d, ah, r.hi[n]);
        acc[2 * m][2 * n] += d[0];
        acc[2 * m][2 * n + 1] += d[1];
        acc[2 * m + 1][2 * n] += d[2];
        acc[2 * m + 1][2 * n + 1] += d[3];
      }
    }
  }
  static __device__ __forceinline__ void run(const float *A, const float *B, float (&acc)[TM][TN], int k0, int k1,
                                             const float *scale = nullptr) {
    if (!active()) return;
#pragma unroll 2
    for (int k = k0; k < k1; k += 8) {
      Right r;
      right(r, B, k, scale);
      step(A, k, r, acc);
    }
  }
  // two left operands at once
  static __device__ __forceinline__ void run2(const float *A, const float *A2, const float *B, float (&acc)[TM][TN],
                                              float (&acc2)[TM][TN], int k1) {
#pragma unroll 2
    for (int k = 0; k < k1; k += 8) {
      Right r;
      right(r, B, k, nullptr);
      step(A, k, r, acc);
      step(A2, k, r, acc2);
    }
  }
  // depths at which a warp's rows of a lower triangular 64 x 64 A (TA: its
  // transpose) are not all zero
  static __device__ __forceinline__ int from() { return TA ? wm() * 16 * MT : 0; }
  static __device__ __forceinline__ int to() { return TA ? kC : (wm() + 1) * 16 * MT; }
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(float *dst, const float *src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all groups of this thread's copies but the last PENDING have landed
template <int PENDING> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ bool aligned16(const float *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// rows [t0, t0 + 64) of a [T][d] tensor, columns [c0, c0 + W), zeros behind T,
// by asynchronous copies
template <int W, int LD>
__device__ __forceinline__ void fetch_rows(float *dst, const float *src, int t0, int T, int d, int c0) {
  if (aligned16(src)) {
    for (int e = threadIdx.x; e < kC * W / 4; e += kThreads) {
      const int t = e / (W / 4), c = e % (W / 4) * 4, row = t0 + t < T ? t0 + t : 0;
      copy16(dst + t * LD + c, src + (size_t)row * d + c0 + c, t0 + t < T);
    }
  } else {
    for (int e = threadIdx.x; e < kC * W; e += kThreads) {
      const int t = e / W, c = e % W, row = t0 + t < T ? t0 + t : 0;
      copy4(dst + t * LD + c, src + (size_t)row * d + c0 + c, t0 + t < T);
    }
  }
}
__device__ __forceinline__ void fetch_square(float *dst, const float *src) {
  for (int e = threadIdx.x; e < kC * kC / 4; e += kThreads)
    copy16(dst + e / (kC / 4) * kLD + e % (kC / 4) * 4, src + 4 * e, true);
}
__device__ __forceinline__ void fetch_gates(float *dst, const float *src) {
  if (threadIdx.x < kRec / 4) copy16(dst + 4 * threadIdx.x, src + 4 * threadIdx.x, true);
}

// Gates of a chunk: running sums G (fp64), e^G, e^{G_C - G} and beta, one
// entry a token. Tokens behind T have g = 0 and beta = 0. Warp 0 works.
struct Gates {
  float from_start[kC], to_end[kC], beta[kC];
  double G[kC];
};
__device__ __forceinline__ void load_gates(Gates &s, const float *g, const float *beta, int t0, int T) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, t = t0 + 2 * lane;
    const double x = t < T ? (double)clamp_decay(g[t]) : 0.0;
    const double y = t + 1 < T ? (double)clamp_decay(g[t + 1]) : 0.0;
    double sum = x + y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += up;
    }
    const double last = __shfl_sync(0xffffffffu, sum, 31);
    const double G[2] = {sum - y, sum};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s.G[2 * lane + i] = G[i];
      s.from_start[2 * lane + i] = expf((float)G[i]);
      s.to_end[2 * lane + i] = expf((float)(last - G[i]));
      s.beta[2 * lane + i] = t + i < T ? beta[t + i] : 0.f;
    }
  }
}

struct Where {                       // the tensors' offsets of a value head
  size_t k, v;                       // first token's row in q / k and in v / gates
  __device__ Where(long long bh, int H, int Hk, int T) {
    const long long b = bh / H, h = bh % H;
    k = (size_t)(b * Hk + h / (H / Hk)) * T;
    v = (size_t)bh * T;
  }
};

// ---------------------------------------------------------------------------
// M, P and the gates of every chunk; the inversion is that of the bf16 kernels
// (gated_delta_tc.cuh), diagonal 32-blocks of L stored transposed for it.
// ---------------------------------------------------------------------------
template <int DK>
struct SolveSmem {
  float q[kC * (DK + 4)], k[kC * (DK + 4)], L[kC * kLD];
  Gates gates;
};

template <int DK>
__global__ void __launch_bounds__(kThreads)
gd_solve_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ g,
                const float *__restrict__ beta, float *__restrict__ M, float *__restrict__ P,
                float *__restrict__ gates, unsigned *__restrict__ status, int H, int Hk, int T, int N) {
  extern __shared__ __align__(16) float sm[];
  SolveSmem<DK> &s = *reinterpret_cast<SolveSmem<DK> *>(sm);
  constexpr int LD = DK + 4;
  static_assert(kLD == gdtc::kLs, "the inversion's row stride");
  const long long bh = blockIdx.x / N;
  const int n = blockIdx.x % N, t0 = n * kC, tid = threadIdx.x;
  const Where at(bh, H, Hk, T);
  if (blockIdx.x == 0 && tid == 0) *status = 0;            // these kernels have no wait that could give up
  fetch_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
  fetch_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
  copies_done();
  load_gates(s.gates, g + at.v, beta + at.v, t0, T);
  copies_wait<0>();
  __syncthreads();
  using GT = Gemm<kC, kC, false, true, LD, LD>;
  float kk[GT::TM][GT::TN], qk[GT::TM][GT::TN];
  GT::zero(kk);
  GT::zero(qk);
  GT::run2(s.k, s.q, s.k, kk, qk, DK);
  const size_t out = (size_t)blockIdx.x * kC * kC;
#pragma unroll
  for (int i = 0; i < GT::TM; ++i)
#pragma unroll
    for (int j = 0; j < GT::TN; j += 2) {
      const int t = GT::row(i), c = GT::col(j);
      float p[2], l[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float w = c + u <= t ? expf((float)(s.gates.G[t] - s.gates.G[c + u])) : 0.f;
        p[u] = c + u <= t ? w * qk[i][j + u] : 0.f;
        l[u] = c + u < t ? s.gates.beta[t] * w * kk[i][j + u] : 0.f;
        if (t / 32 == c / 32) s.L[(c + u) * kLD + t] = l[u];
      }
      if (t / 32 != c / 32) *reinterpret_cast<float2 *>(&s.L[t * kLD + c]) = make_float2(l[0], l[1]);
      *reinterpret_cast<float2 *>(P + out + t * kC + c) = make_float2(p[0], p[1]);
    }
  if (tid < kRec) gates[(size_t)blockIdx.x * kRec + tid] = reinterpret_cast<const float *>(&s.gates)[tid];
  __syncthreads();
  if (tid < 64) gdtc::invert_diagonal(s.L + tid / 32 * 32 * (kLD + 1));
  __syncthreads();
  gdtc::invert_corner(s.L);                                // warps 4-7 do what 0-3 do
  for (int e = tid; e < kC * kC / 4; e += kThreads) {
    const int t = e / (kC / 4), c = e % (kC / 4) * 4;
    const float4 x = *reinterpret_cast<const float4 *>(&s.L[t * kLD + c]);
    *reinterpret_cast<float4 *>(M + out + 4 * e) = t < 32 && c >= 32 ? make_float4(0.f, 0.f, 0.f, 0.f) : x;
  }
}

// ---------------------------------------------------------------------------
// The chain: S through the chunks, for CB value columns. `o` and S_out for
// the forward; with `starts` the chunks' starting states and `writes` D. K and
// the gates have two buffers; of the rest the next chunk's is fetched as soon as
// this one's has been read, so that every copy has two of the three steps to land.
// ---------------------------------------------------------------------------
template <int DK, int CB>
struct ChainSmem {
  static constexpr int LD = DK + 4, LS = CB + 8;           // rows of K, Q; of what has value columns
  float k[2][kC * LD], q[kC * LD], M[kC * kLD], P[kC * kLD];
  float S[DK * LS], V[2][kC * LS], R[kC * LS], D[kC * LS], gates[2][kRec];
};

// A head's sequence may be cut into G segments of seg_chunks chunks. EFFECT: what a
// segment does to a state, S -> F S + B, without outputs: the first kind0 blocks walk
// segments 0 .. G - 2 from S = 0 (segment 0: from S0) to B, into `states` of the next
// segment, the others segments 1 .. G - 2 from S = I without V to F.
struct Segments {
  float *states, *F;
  int G, chunks, kind0;
};

template <int DK, int CB, bool EFFECT>
__global__ void __launch_bounds__(kThreads)
gd_chain_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                const float *__restrict__ gates, const float *__restrict__ M, const float *__restrict__ P,
                const float *__restrict__ S0, float *__restrict__ o, float *__restrict__ S_out,
                float *__restrict__ starts, float *__restrict__ writes, int H, int Hk, int T, int N, int DV,
                const Segments sg) {
  extern __shared__ __align__(16) float sm[];
  using Smem = ChainSmem<DK, CB>;
  Smem &s = *reinterpret_cast<Smem *>(sm);
  constexpr int LD = Smem::LD, LS = Smem::LS;
  const int tid = threadIdx.x;
  const bool to_F = EFFECT && (int)blockIdx.x >= sg.kind0;
  const int block = (int)blockIdx.x - (to_F ? sg.kind0 : 0), NB = (to_F ? DK : DV) / CB;
  const int segs = EFFECT ? sg.G - 1 - to_F : sg.G, seg = block / NB % segs + to_F;
  const long long bh = block / NB / segs;
  const int c0 = (block % NB) * CB;
  const int first = seg * sg.chunks, end = first + sg.chunks < N ? first + sg.chunks : N;
  const Where at(bh, H, Hk, T);
  const size_t state = (size_t)DK * DV, chunk0 = (size_t)bh * N;
  const float *from = seg == 0 ? (S0 ? S0 + bh * state : nullptr) : EFFECT ? nullptr : sg.states + (bh * sg.G + seg) * state;
  for (int e = tid; e < DK * CB; e += kThreads)
    s.S[(e / CB) * LS + e % CB] = to_F ? (e / CB == c0 + e % CB ? 1.f : 0.f)
                                  : from ? from[(size_t)(e / CB) * DV + c0 + e % CB]
                                         : 0.f;
  if (to_F)
    for (int e = tid; e < kC * CB; e += kThreads) s.V[0][(e / CB) * LS + e % CB] = 0.f;
  using GS = Gemm<kC, CB, false, false, LD, LS>;         // K S, Q S
  using GD = Gemm<kC, CB, false, false, kLD, LS>;        // M R, P D: the same tiles
  using GU = Gemm<DK, CB, true, false, LD, LS>;          // K^T D
  auto fetch_kqv = [&](int n) {
    if (n < end) {
      fetch_rows<DK, LD>(s.k[n & 1], k + at.k * DK, n * kC, T, DK, 0);
      if (o) fetch_rows<DK, LD>(s.q, q + at.k * DK, n * kC, T, DK, 0);
      if (!to_F) fetch_rows<CB, LS>(s.V[0], v + at.v * DV, n * kC, T, DV, c0);
      fetch_gates(s.gates[n & 1], gates + (chunk0 + n) * kRec);
    }
    copies_done();
  };
  auto fetch_tile = [&](float *dst, const float *src, int n, bool wanted) {
    if (n < end && wanted) fetch_square(dst, src + (chunk0 + n) * kC * kC);
    copies_done();
  };
  fetch_kqv(first);
  fetch_tile(s.M, M, first, true);
  for (int n = first; n < end; ++n) {
    const int t0 = n * kC;
    const float *sk = s.k[n & 1], *from_start = s.gates[n & 1], *to_end = from_start + kC, *beta = to_end + kC;
    copies_wait<1>();
    __syncthreads();                                       // K, Q, V, the gates and S are there; P has been read
    fetch_tile(s.P, P, n, o != nullptr);
    if (starts)
      for (int e = tid; e < DK * CB; e += kThreads)
        starts[(chunk0 + n) * DK * DV + (size_t)(e / CB) * DV + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
    float ks[GS::TM][GS::TN], qs[GS::TM][GS::TN];
    GS::zero(ks);
    GS::zero(qs);
    if (o)
      GS::run2(sk, s.q, s.S, ks, qs, DK);
    else
      GS::run(sk, s.S, ks, 0, DK);
#pragma unroll
    for (int i = 0; i < GS::TM; ++i)
#pragma unroll
      for (int j = 0; j < GS::TN; ++j) {
        const int t = GS::row(i), e = t * LS + GS::col(j);
        s.R[e] = beta[t] * (s.V[0][e] - from_start[t] * ks[i][j]);
      }
    copies_wait<1>();
    __syncthreads();                                       // R and M are there; Q and V have been read
    fetch_kqv(n + 1);
    float d[GD::TM][GD::TN];
    GD::zero(d);
    GD::run(s.M, s.R, d, GD::from(), GD::to());
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) {
        const int t = GD::row(i), c = GD::col(j);
        s.D[t * LS + c] = d[i][j];
        if (writes && t0 + t < T) writes[(at.v + t0 + t) * DV + c0 + c] = d[i][j];
      }
    copies_wait<1>();
    __syncthreads();                                       // D and P are there; M has been read
    fetch_tile(s.M, M, n + 1, true);
    if (o) {
      GD::zero(d);
      GD::run(s.P, s.D, d, GD::from(), GD::to());
#pragma unroll
      for (int i = 0; i < GD::TM; ++i)
#pragma unroll
        for (int j = 0; j < GD::TN; ++j) {
          const int t = GD::row(i);
          if (t0 + t < T) o[(at.v + t0 + t) * DV + c0 + GD::col(j)] = fmaf(from_start[t], qs[i][j], d[i][j]);
        }
    }
    if (GU::active()) {
      float up[GU::TM][GU::TN];
      GU::zero(up);
      GU::run(sk, s.D, up, 0, kC, to_end);
      const float whole = from_start[kC - 1];
#pragma unroll
      for (int i = 0; i < GU::TM; ++i)
#pragma unroll
        for (int j = 0; j < GU::TN; ++j) {
          float &x = s.S[GU::row(i) * LS + GU::col(j)];
          x = fmaf(whole, x, up[i][j]);
        }
    }
  }
  __syncthreads();
  float *to = nullptr;
  if (!EFFECT)
    to = S_out && seg == sg.G - 1 ? S_out + bh * state : nullptr;
  else
    to = to_F ? sg.F + (bh * (sg.G - 2) + seg - 1) * DK * DK : sg.states + (bh * sg.G + seg + 1) * state;
  const int ld = to_F ? DK : DV;
  if (to)
    for (int e = tid; e < DK * CB; e += kThreads)
      to[(size_t)(e / CB) * ld + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
}

// ---------------------------------------------------------------------------
// The reverse chain: dS through the chunks, last first, for CB value columns.
// K, dO and the gates have two buffers; Q is fetched at the chunk's beginning for
// its end. EFFECT: what segments 1 .. G - 1 pass on from dS' = 0 (the last: from dS)
// into `states` of the segment before.
// ---------------------------------------------------------------------------
template <int DK, int CB, bool EFFECT>
__global__ void __launch_bounds__(kThreads)
gd_chain_reverse_kernel(const float *__restrict__ q, const float *__restrict__ k,
                        const float *__restrict__ dout, const float *__restrict__ gates,
                        const float *__restrict__ M, const float *__restrict__ P,
                        const float *__restrict__ dS, float *__restrict__ dv, float *__restrict__ dR,
                        float *__restrict__ ends, float *__restrict__ dS0, int H, int Hk, int T, int N, int DV,
                        const Segments sg) {
  extern __shared__ __align__(16) float sm[];
  using Smem = ChainSmem<DK, CB>;
  Smem &s = *reinterpret_cast<Smem *>(sm);
  constexpr int LD = Smem::LD, LS = Smem::LS;
  const int tid = threadIdx.x, NB = DV / CB, block = (int)blockIdx.x;
  const int segs = EFFECT ? sg.G - 1 : sg.G, seg = block / NB % segs + (EFFECT ? 1 : 0);
  const long long bh = block / NB / segs;
  const int c0 = (block % NB) * CB;
  const int first = seg * sg.chunks, end = first + sg.chunks < N ? first + sg.chunks : N;
  const Where at(bh, H, Hk, T);
  const size_t state = (size_t)DK * DV, chunk0 = (size_t)bh * N;
  const float *from = seg == sg.G - 1 ? (dS ? dS + bh * state : nullptr)
                      : EFFECT        ? nullptr
                                      : sg.states + (bh * sg.G + seg) * state;
  for (int e = tid; e < DK * CB; e += kThreads)
    s.S[(e / CB) * LS + e % CB] = from ? from[(size_t)(e / CB) * DV + c0 + e % CB] : 0.f;
  using GS = Gemm<kC, CB, false, false, LD, LS>;         // K dS
  using GD = Gemm<kC, CB, true, false, kLD, LS>;         // P^T dO, M^T dD: the same tiles
  using GU = Gemm<DK, CB, true, false, LD, LS>;          // Q^T dO, K^T dV
  auto fetch_kp = [&](int i) {                           // the i-th from the end
    if (i < end - first) {
      const int n = end - 1 - i;
      fetch_rows<DK, LD>(s.k[i & 1], k + at.k * DK, n * kC, T, DK, 0);
      fetch_rows<CB, LS>(s.V[i & 1], dout + at.v * DV, n * kC, T, DV, c0);
      fetch_gates(s.gates[i & 1], gates + (chunk0 + n) * kRec);
      fetch_square(s.P, P + (chunk0 + n) * kC * kC);
    }
    copies_done();
  };
  auto fetch_m = [&](int i) {
    if (i < end - first) fetch_square(s.M, M + (chunk0 + end - 1 - i) * kC * kC);
    copies_done();
  };
  fetch_kp(0);
  fetch_m(0);
  for (int i0 = 0; i0 < end - first; ++i0) {
    const int n = end - 1 - i0, t0 = n * kC;
    const float *sk = s.k[i0 & 1], *dO = s.V[i0 & 1], *from_start = s.gates[i0 & 1], *to_end = from_start + kC,
                *beta = to_end + kC;
    copies_wait<1>();
    __syncthreads();                                       // K, dO, P, the gates and dS are there; Q has been read
    fetch_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
    copies_done();
    if (!EFFECT)
      for (int e = tid; e < DK * CB; e += kThreads)
        ends[(chunk0 + n) * DK * DV + (size_t)(e / CB) * DV + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
    float ks[GS::TM][GS::TN];
    GS::zero(ks);
    GS::run(sk, s.S, ks, 0, DK);
    float d[GD::TM][GD::TN];
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) d[i][j] = to_end[GD::row(i)] * ks[i][j];
    GD::run(s.P, dO, d, GD::from(), GD::to());             // dD
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) s.D[GD::row(i) * LS + GD::col(j)] = d[i][j];
    copies_wait<1>();
    __syncthreads();                                       // dD and M are there; P has been read
    fetch_kp(i0 + 1);
    GD::zero(d);
    GD::run(s.M, s.D, d, GD::from(), GD::to());            // dR
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) {
        const int t = GD::row(i), c = GD::col(j);
        const float x = beta[t] * d[i][j];
        s.R[t * LS + c] = -from_start[t] * x;
        if (!EFFECT && t0 + t < T) {
          dv[(at.v + t0 + t) * DV + c0 + c] = x;
          dR[(at.v + t0 + t) * DV + c0 + c] = d[i][j];
        }
      }
    copies_wait<1>();
    __syncthreads();                                       // dV and Q are there; M has been read
    fetch_m(i0 + 1);
    if (GU::active()) {
      float up[GU::TM][GU::TN];
      GU::zero(up);
      GU::run(s.q, dO, up, 0, kC, from_start);
      GU::run(sk, s.R, up, 0, kC);
      const float whole = from_start[kC - 1];
#pragma unroll
      for (int i = 0; i < GU::TM; ++i)
#pragma unroll
        for (int j = 0; j < GU::TN; ++j) {
          float &x = s.S[GU::row(i) * LS + GU::col(j)];
          x = fmaf(whole, x, up[i][j]);
        }
    }
  }
  __syncthreads();
  float *to = EFFECT ? sg.states + (bh * sg.G + seg - 1) * state : seg == 0 && dS0 ? dS0 + bh * state : nullptr;
  if (to)
    for (int e = tid; e < DK * CB; e += kThreads)
      to[(size_t)(e / CB) * DV + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
}

// ---------------------------------------------------------------------------
// dq, dk, dg and dbeta of every chunk, from the states and state gradients at
// its borders. With X = dR S^T, Y = dO S^T, Z = D dS'^T (64 x d_k):
//   dq = e^G Y + (dP W) K,
//   dk = -beta e^G X + e^{G_C - G} Z + (dP W)^T Q + (A + A^T) K,  A = dL beta W,
//   dbeta_t = dR_t . v_t - e^{G_t} k_t . X_t + sum_s dL_ts W_ts k_t.k_s,
//   dG_t = e^{G_t} (q_t . Y_t - beta_t k_t . X_t) - z_t + sum_s pairs_ts - sum_s pairs_st,
//   dg_t = sum_{u >= t} dG_u + sum_s z_s + e^{G_C} <S, dS'>,
// z_t = e^{G_C - G_t} k_t . Z_t, pairs = dP P + dL L.
// ---------------------------------------------------------------------------
template <int DK, int CB>
struct GradSmem {
  float q[kC * (DK + 4)], k[kC * (DK + 4)], pair_p[kC * kLD], pair_l[kC * kLD];
  float dO[kC * (CB + 4)], dR[kC * (CB + 4)], D[kC * (CB + 4)], S[DK * (CB + 4)], dS[DK * (CB + 4)];
  // the warps' parts of the row and column sums
  float row_v[kC], row_q[2][kC], row_k[2][kC], row_z[2][kC], row_b[2][kC], row_p[2][kC], col_p[4][kC];
  float dot[kThreads / 32];
  Gates gates;
};

// sum over four neighbouring lanes: a warp's part of a tile row
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int DK, int CB>
__global__ void __launch_bounds__(kThreads)
gd_grads_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                const float *__restrict__ dout, const float *__restrict__ g,
                const float *__restrict__ beta, const float *__restrict__ starts,
                const float *__restrict__ ends, const float *__restrict__ writes,
                const float *__restrict__ dRg, float *__restrict__ dq, float *__restrict__ dk,
                float *__restrict__ dq_part, float *__restrict__ dk_part, float *__restrict__ dg,
                float *__restrict__ dbeta, int H, int Hk, int T, int N, int DV) {
  extern __shared__ __align__(16) float sm[];
  GradSmem<DK, CB> &s = *reinterpret_cast<GradSmem<DK, CB> *>(sm);
  constexpr int LD = DK + 4, LS = CB + 4;                // value columns are read across here
  const long long bh = blockIdx.x / N;
  const int n = blockIdx.x % N, t0 = n * kC, tid = threadIdx.x;
  const Where at(bh, H, Hk, T);
  const size_t border = ((size_t)bh * N + n) * DK * DV;
  fetch_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
  fetch_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
  load_gates(s.gates, g + at.v, beta + at.v, t0, T);
  if (tid < kC) s.row_v[tid] = 0.f;

  using GX = Gemm<kC, DK, false, true, LS, LS>;      // X, Y, Z
  using GP = Gemm<kC, kC, false, true, LS, LS>;      // dP, dL
  float X[GX::TM][GX::TN], Y[GX::TM][GX::TN], Z[GX::TM][GX::TN];
  float dP[GP::TM][GP::TN], dL[GP::TM][GP::TN];
  GX::zero(X); GX::zero(Y); GX::zero(Z);
  GP::zero(dP); GP::zero(dL);
  float dot = 0.f;
  for (int c0 = 0; c0 < DV; c0 += CB) {
    __syncthreads();
    fetch_rows<CB, LS>(s.dO, dout + at.v * DV, t0, T, DV, c0);
    fetch_rows<CB, LS>(s.dR, dRg + at.v * DV, t0, T, DV, c0);
    fetch_rows<CB, LS>(s.D, writes + at.v * DV, t0, T, DV, c0);
    for (int e = tid; e < DK * CB; e += kThreads) {
      const int i = (e / CB) * LS + e % CB;
      const size_t src = border + (size_t)(e / CB) * DV + c0 + e % CB;
      s.S[i] = starts[src];
      s.dS[i] = ends[src];
      dot = fmaf(s.S[i], s.dS[i], dot);
    }
    copies_done();
    copies_wait<0>();
    __syncthreads();
    GX::run2(s.dR, s.dO, s.S, X, Y, CB);
    GX::run(s.D, s.dS, Z, 0, CB);
    GP::run2(s.dO, s.dR, s.D, dP, dL, CB);
    // dR_t . v_t: four threads a row
    const int t = tid / 4;
    float rv = 0.f;
    if (t0 + t < T)
      for (int c = tid % 4; c < CB; c += 4)
        rv = fmaf(s.dR[t * LS + c], v[(at.v + t0 + t) * DV + c0 + c], rv);
    rv = quad_sum(rv);
    if (tid % 4 == 0) s.row_v[t] += rv;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  if (tid % 32 == 0) s.dot[tid / 32] = dot;

  // row dots of q, k with Y, X, Z
  static_assert(GX::WM == 4 && GX::WN == 2 && GP::WM == 4 && GP::WN == 2, "two warps share a tile row");
  const int wn = GX::wn(), g4 = tid % 4;
#pragma unroll
  for (int i = 0; i < GX::TM; ++i) {
    float rq = 0.f, rk = 0.f, rz = 0.f;
#pragma unroll
    for (int j = 0; j < GX::TN; ++j) {
      const int e = GX::row(i) * LD + GX::col(j);
      rq = fmaf(s.q[e], Y[i][j], rq);
      rk = fmaf(s.k[e], X[i][j], rk);
      rz = fmaf(s.k[e], Z[i][j], rz);
    }
    rq = quad_sum(rq);
    rk = quad_sum(rk);
    rz = quad_sum(rz);
    if (g4 == 0) {
      s.row_q[wn][GX::row(i)] = rq;
      s.row_k[wn][GX::row(i)] = rk;
      s.row_z[wn][GX::row(i)] = rz;
    }
  }
  // the pair matrices
  using GK = Gemm<kC, kC, false, true, LD, LD>;          // K K^T, Q K^T: GP's tile map
  float kk[GK::TM][GK::TN], qk[GK::TM][GK::TN];
  GK::zero(kk);
  GK::zero(qk);
  GK::run2(s.k, s.q, s.k, kk, qk, DK);
  float pairs[GP::TM][GP::TN];
#pragma unroll
  for (int i = 0; i < GP::TM; ++i) {
    const int t = GP::row(i);
    float rb = 0.f, rp = 0.f;
#pragma unroll
    for (int j = 0; j < GP::TN; ++j) {
      const int c = GP::col(j);
      const float w = c <= t ? expf((float)(s.gates.G[t] - s.gates.G[c])) : 0.f;
      const float p = c <= t ? dP[i][j] * w : 0.f;
      const float l = c < t ? -dL[i][j] * w : 0.f;       // dL W, dL = -dR D^T
      s.pair_p[t * kLD + c] = p;
      s.pair_l[t * kLD + c] = l * s.gates.beta[t];
      rb = fmaf(l, kk[i][j], rb);
      pairs[i][j] = fmaf(p, qk[i][j], l * s.gates.beta[t] * kk[i][j]);
      rp += pairs[i][j];
    }
    rb = quad_sum(rb);
    rp = quad_sum(rp);
    if (g4 == 0) {
      s.row_b[wn][t] = rb;
      s.row_p[wn][t] = rp;
    }
  }
  // column sums of the pairs, a warp's 16 rows at a time
#pragma unroll
  for (int j = 0; j < GP::TN; ++j) {
    float cs = 0.f;
#pragma unroll
    for (int i = 0; i < GP::TM; ++i) cs += pairs[i][j];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) cs += __shfl_xor_sync(0xffffffffu, cs, off);
    if (tid % 32 < 4) s.col_p[GP::wm()][GP::col(j)] = cs;
  }
  __syncthreads();
  if (tid < 32) {
    // dG, its sum from the right, dbeta: two tokens a lane
    const int t = 2 * tid;
    float dG[2], z = 0.f;
    auto both = [](const float (&x)[2][kC], int u) { return x[0][u] + x[1][u]; };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float zt = s.gates.to_end[t + i] * both(s.row_z, t + i);
      z += zt;
      const float down = (s.col_p[0][t + i] + s.col_p[1][t + i]) + (s.col_p[2][t + i] + s.col_p[3][t + i]);
      dG[i] = s.gates.from_start[t + i] * (both(s.row_q, t + i) - s.gates.beta[t + i] * both(s.row_k, t + i)) - zt +
              both(s.row_p, t + i) - down;
      if (t0 + t + i < T)
        dbeta[at.v + t0 + t + i] =
            s.row_v[t + i] - s.gates.from_start[t + i] * both(s.row_k, t + i) + both(s.row_b, t + i);
    }
    float last = z, sum = dG[0] + dG[1];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) last += __shfl_xor_sync(0xffffffffu, last, off);
    float border_dot = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) border_dot += s.dot[w];
    last = fmaf(s.gates.from_start[kC - 1], border_dot, last);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float down = __shfl_down_sync(0xffffffffu, sum, off);
      if (tid + off < 32) sum += down;
    }
    if (t0 + t < T) dg[at.v + t0 + t] = sum + last;
    if (t0 + t + 1 < T) dg[at.v + t0 + t + 1] = sum - dG[0] + last;
  }
  // dq = e^G Y + pair_p K;  dk = ... + pair_p^T Q + (pair_l + pair_l^T) K
  using GA = Gemm<kC, DK, false, false, kLD, LD>;        // GX's tiles
  using GT = Gemm<kC, DK, true, false, kLD, LD>;
#pragma unroll
  for (int i = 0; i < GX::TM; ++i) {
    const int t = GX::row(i);
    const float f = s.gates.from_start[t], e = s.gates.to_end[t], fb = f * s.gates.beta[t];
#pragma unroll
    for (int j = 0; j < GX::TN; ++j) {
      Y[i][j] *= f;
      X[i][j] = fmaf(-fb, X[i][j], e * Z[i][j]);
    }
  }
  GA::run(s.pair_p, s.k, Y, GA::from(), GA::to());
  GA::run(s.pair_l, s.k, X, GA::from(), GA::to());
  GT::run(s.pair_l, s.k, X, GT::from(), GT::to());
  GT::run(s.pair_p, s.q, X, GT::from(), GT::to());
#pragma unroll
  for (int i = 0; i < GX::TM; ++i) {
    const int t = GX::row(i);
    if (t0 + t >= T) continue;
#pragma unroll
    for (int j = 0; j < GX::TN; ++j) {
      const int c = GX::col(j);
      if (dq_part) {
        dq_part[(at.v + t0 + t) * DK + c] = Y[i][j];
        dk_part[(at.v + t0 + t) * DK + c] = X[i][j];
      } else {
        dq[(at.k + t0 + t) * DK + c] = Y[i][j];
        dk[(at.k + t0 + t) * DK + c] = X[i][j];
      }
    }
  }
}

}  // namespace gd
}  // namespace kata
