// The gated delta rule on the CUDA cores: the path of fp32 tensors.
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
// The running sums are kept in fp64 and differenced there: with strong decays
// G reaches thousands, and an fp32 difference of two such sums would lose the
// ratio's digits. A log decay below -100 (a reset, -inf included) counts as
// -100: e^-100 is 0 in fp32, and the differences stay finite.
//
// Kernels: solve (M and P of every chunk, all chunks at once), chain (one
// block per head and kCB value columns walks the chunks: the columns of S
// follow the rule on their own), chain_reverse (dS, dR, dV, last chunk
// first), grads (dq, dk, dg, dbeta, all chunks at once).
#pragma once

#include "common.cuh"
#include "gated_delta.h"
#include "profile.h"

namespace kata {
namespace gd {

constexpr int kC = kGdChunk;
constexpr int kThreads = 256;
constexpr int kLD = kC + 4;          // row stride of a 64 x 64 matrix (float4 rows)
constexpr float kMinLogDecay = -100.f;

__device__ __forceinline__ float clamp_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// acc += A B for an M x N tile and depth K, operands in shared memory, 256
// threads. A[m][k] at A[m * LDA + k] (TA: A[k * LDA + m]); B[k][n] at
// B[k * LDB + n] (TB: B[n * LDB + k]). Thread (ty, tx) owns the rows
// ty * TM + i and the columns tx * TN + j (TB: tx + j * NX, so that lanes
// read different banks). Rows are read as float4 along the contiguous axis:
// 3 wavefronts a k-step feed 16 FMAs a thread.
template <int M, int N, int K, bool TA, bool TB, int LDA, int LDB>
struct Gemm {
  static constexpr int PER = M * N / kThreads;
  static constexpr int TN = PER >= 16 ? 4 : (PER >= 2 ? 2 : 1);
  static constexpr int TM = PER / TN;
  static constexpr int NX = N / TN;
  static_assert(PER >= 1 && TM * TN * kThreads == M * N, "tile split");
  static __device__ __forceinline__ int row(int i) { return (int)(threadIdx.x / NX) * TM + i; }
  static __device__ __forceinline__ int col(int j) {
    const int tx = threadIdx.x % NX;
    return TB ? tx + j * NX : tx * TN + j;
  }
  static __device__ __forceinline__ void zero(float (&acc)[TM][TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
  }
  static __device__ __forceinline__ void run(const float *A, const float *B, float (&acc)[TM][TN]) {
    const int r0 = row(0);
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
      float a[TM][4], b[4][TN];
      if constexpr (!TA) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const float4 x = *reinterpret_cast<const float4 *>(A + (r0 + i) * LDA + k);
          a[i][0] = x.x; a[i][1] = x.y; a[i][2] = x.z; a[i][3] = x.w;
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int i = 0; i < TM; ++i) a[i][kk] = A[(k + kk) * LDA + r0 + i];
      }
      if constexpr (TB) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const float4 x = *reinterpret_cast<const float4 *>(B + col(j) * LDB + k);
          b[0][j] = x.x; b[1][j] = x.y; b[2][j] = x.z; b[3][j] = x.w;
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const float *src = B + (k + kk) * LDB + col(0);
          if constexpr (TN == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            b[kk][0] = x.x; b[kk][1] = x.y; b[kk][2] = x.z; b[kk][3] = x.w;
          } else {
#pragma unroll
            for (int j = 0; j < TN; ++j) b[kk][j] = src[j];
          }
        }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i][kk], b[kk][j], acc[i][j]);
    }
  }
};

// rows [t0, t0 + 64) of a [T][d] tensor, columns [c0, c0 + W), zeros behind T
template <int W, int LD>
__device__ __forceinline__ void load_rows(float *dst, const float *src, int t0, int T, int d, int c0) {
  for (int e = threadIdx.x; e < kC * W; e += kThreads) {
    const int t = e / W, c = e % W;
    dst[t * LD + c] = t0 + t < T ? src[(size_t)(t0 + t) * d + c0 + c] : 0.f;
  }
}

// Gates of a chunk: running sums G (fp64), e^G, e^{G_C - G} and beta, one
// entry a token. Tokens behind T have g = 0 and beta = 0. Warp 0 works.
struct Gates {
  double G[kC];
  float from_start[kC], to_end[kC], beta[kC];
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
// M and P of every chunk. Columns of M = (I + L)^-1 are independent: thread
// j < 64 solves column j by forward substitution in registers, L's rows
// broadcast from shared memory.
// ---------------------------------------------------------------------------
template <int DK>
struct SolveSmem {
  float q[kC * (DK + 4)], k[kC * (DK + 4)], L[kC * kLD], P[kC * kLD];
  Gates gates;
};

template <int DK>
__global__ void __launch_bounds__(kThreads)
gd_solve_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ g,
                const float *__restrict__ beta, float *__restrict__ M, float *__restrict__ P, int H,
                int Hk, int T, int N) {
  extern __shared__ __align__(16) float sm[];
  SolveSmem<DK> &s = *reinterpret_cast<SolveSmem<DK> *>(sm);
  constexpr int LD = DK + 4;
  const long long bh = blockIdx.x / N;
  const int n = blockIdx.x % N, t0 = n * kC, tid = threadIdx.x;
  const Where at(bh, H, Hk, T);
  load_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
  load_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
  load_gates(s.gates, g + at.v, beta + at.v, t0, T);
  __syncthreads();
  using GT = Gemm<kC, kC, DK, false, true, LD, LD>;
  float kk[GT::TM][GT::TN], qk[GT::TM][GT::TN];
  GT::zero(kk);
  GT::zero(qk);
  GT::run(s.k, s.k, kk);
  GT::run(s.q, s.k, qk);
#pragma unroll
  for (int i = 0; i < GT::TM; ++i)
#pragma unroll
    for (int j = 0; j < GT::TN; ++j) {
      const int t = GT::row(i), c = GT::col(j);
      const float w = c <= t ? expf((float)(s.gates.G[t] - s.gates.G[c])) : 0.f;
      s.P[t * kLD + c] = c <= t ? w * qk[i][j] : 0.f;
      s.L[t * kLD + c] = c < t ? s.gates.beta[t] * w * kk[i][j] : 0.f;
    }
  __syncthreads();
  const size_t out = (size_t)blockIdx.x * kC * kC;
  if (tid < kC) {
    float x[kC];
#pragma unroll
    for (int t = 0; t < kC; ++t) {
      float a0 = t == tid ? 1.f : 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int u = 0; u < t; u += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(&s.L[t * kLD + u]);
        a0 = fmaf(-l.x, x[u], a0);
        if (u + 1 < t) a1 = fmaf(-l.y, x[u + 1], a1);
        if (u + 2 < t) a2 = fmaf(-l.z, x[u + 2], a2);
        if (u + 3 < t) a3 = fmaf(-l.w, x[u + 3], a3);
      }
      x[t] = (a0 + a1) + (a2 + a3);
    }
#pragma unroll
    for (int t = 0; t < kC; ++t) M[out + t * kC + tid] = x[t];
  }
  for (int e = tid; e < kC * kC; e += kThreads) P[out + e] = s.P[(e / kC) * kLD + e % kC];
}

// ---------------------------------------------------------------------------
// The chain: S through the chunks, for kCB value columns. `o` and S_out for
// the forward; with `starts` the chunks' starting states and `writes` D.
// ---------------------------------------------------------------------------
template <int DK, int CB>
struct ChainSmem {
  float q[kC * (DK + 4)], k[kC * (DK + 4)], M[kC * kLD], P[kC * kLD];
  float S[DK * (CB + 4)], R[kC * (CB + 4)], D[kC * (CB + 4)];
  Gates gates;
};

template <int LD>
__device__ __forceinline__ void load_square(float *dst, const float *src) {
  for (int e = threadIdx.x; e < kC * kC / 4; e += kThreads)
    *reinterpret_cast<float4 *>(dst + (e / (kC / 4)) * LD + 4 * (e % (kC / 4))) =
        reinterpret_cast<const float4 *>(src)[e];
}

template <int DK, int CB>
__global__ void __launch_bounds__(kThreads)
gd_chain_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                const float *__restrict__ g, const float *__restrict__ beta,
                const float *__restrict__ M, const float *__restrict__ P, const float *__restrict__ S0,
                float *__restrict__ o, float *__restrict__ S_out, float *__restrict__ starts,
                float *__restrict__ writes, int H, int Hk, int T, int N, int DV) {
  extern __shared__ __align__(16) float sm[];
  ChainSmem<DK, CB> &s = *reinterpret_cast<ChainSmem<DK, CB> *>(sm);
  constexpr int LD = DK + 4, LS = CB + 4;
  const int NB = DV / CB, tid = threadIdx.x;
  const long long bh = blockIdx.x / NB;
  const int c0 = (blockIdx.x % NB) * CB;
  const Where at(bh, H, Hk, T);
  const size_t state = (size_t)bh * DK * DV;
  for (int e = tid; e < DK * CB; e += kThreads)
    s.S[(e / CB) * LS + e % CB] = S0 ? S0[state + (size_t)(e / CB) * DV + c0 + e % CB] : 0.f;
  using GS = Gemm<kC, CB, DK, false, false, LD, LS>;     // K S, Q S
  using GD = Gemm<kC, CB, kC, false, false, kLD, LS>;    // M R, P D
  using GU = Gemm<DK, CB, kC, true, false, LD, LS>;      // K^T D
  for (int n = 0; n < N; ++n) {
    const int t0 = n * kC;
    __syncthreads();
    load_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
    if (o) load_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
    load_rows<CB, LS>(s.R, v + at.v * DV, t0, T, DV, c0);
    load_gates(s.gates, g + at.v, beta + at.v, t0, T);
    load_square<kLD>(s.M, M + ((size_t)bh * N + n) * kC * kC);
    if (o) load_square<kLD>(s.P, P + ((size_t)bh * N + n) * kC * kC);
    if (starts)
      for (int e = tid; e < DK * CB; e += kThreads)
        starts[((size_t)bh * N + n) * DK * DV + (size_t)(e / CB) * DV + c0 + e % CB] =
            s.S[(e / CB) * LS + e % CB];
    __syncthreads();
    float ks[GS::TM][GS::TN], qs[GS::TM][GS::TN];
    GS::zero(ks);
    GS::zero(qs);
    GS::run(s.k, s.S, ks);
    if (o) GS::run(s.q, s.S, qs);
#pragma unroll
    for (int i = 0; i < GS::TM; ++i)
#pragma unroll
      for (int j = 0; j < GS::TN; ++j) {
        const int t = GS::row(i), e = t * LS + GS::col(j);
        s.R[e] = s.gates.beta[t] * (s.R[e] - s.gates.from_start[t] * ks[i][j]);
      }
    __syncthreads();
    float d[GD::TM][GD::TN];
    GD::zero(d);
    GD::run(s.M, s.R, d);
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) {
        const int t = GD::row(i), c = GD::col(j);
        s.D[t * LS + c] = d[i][j];
        if (writes && t0 + t < T) writes[(at.v + t0 + t) * DV + c0 + c] = d[i][j];
      }
    __syncthreads();
    if (o) {
      // the tile maps of GS and GD are the same: qs and d share indices
      GD::zero(d);
      GD::run(s.P, s.D, d);
#pragma unroll
      for (int i = 0; i < GD::TM; ++i)
#pragma unroll
        for (int j = 0; j < GD::TN; ++j) {
          const int t = GD::row(i);
          if (t0 + t < T)
            o[(at.v + t0 + t) * DV + c0 + GD::col(j)] =
                (fmaf(s.gates.from_start[t], qs[i][j], d[i][j]));
        }
      __syncthreads();                                   // P D has read D
    }
    for (int e = tid; e < kC * CB; e += kThreads) s.D[(e / CB) * LS + e % CB] *= s.gates.to_end[e / CB];
    __syncthreads();
    float up[GU::TM][GU::TN];
    GU::zero(up);
    GU::run(s.k, s.D, up);
    const float whole = s.gates.from_start[kC - 1];
#pragma unroll
    for (int i = 0; i < GU::TM; ++i)
#pragma unroll
      for (int j = 0; j < GU::TN; ++j) {
        float &x = s.S[GU::row(i) * LS + GU::col(j)];
        x = fmaf(whole, x, up[i][j]);
      }
  }
  __syncthreads();
  if (S_out)
    for (int e = tid; e < DK * CB; e += kThreads)
      S_out[state + (size_t)(e / CB) * DV + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
}

// ---------------------------------------------------------------------------
// The reverse chain: dS through the chunks, last first, for CB value columns.
// ---------------------------------------------------------------------------
template <int DK, int CB>
__global__ void __launch_bounds__(kThreads)
gd_chain_reverse_kernel(const float *__restrict__ q, const float *__restrict__ k,
                        const float *__restrict__ dout, const float *__restrict__ g,
                        const float *__restrict__ beta, const float *__restrict__ M,
                        const float *__restrict__ P, const float *__restrict__ dS,
                        float *__restrict__ dv, float *__restrict__ dR, float *__restrict__ ends,
                        float *__restrict__ dS0, int H, int Hk, int T, int N, int DV) {
  extern __shared__ __align__(16) float sm[];
  ChainSmem<DK, CB> &s = *reinterpret_cast<ChainSmem<DK, CB> *>(sm);
  constexpr int LD = DK + 4, LS = CB + 4;
  const int NB = DV / CB, tid = threadIdx.x;
  const long long bh = blockIdx.x / NB;
  const int c0 = (blockIdx.x % NB) * CB;
  const Where at(bh, H, Hk, T);
  const size_t state = (size_t)bh * DK * DV;
  for (int e = tid; e < DK * CB; e += kThreads)
    s.S[(e / CB) * LS + e % CB] = dS ? dS[state + (size_t)(e / CB) * DV + c0 + e % CB] : 0.f;
  using GS = Gemm<kC, CB, DK, false, false, LD, LS>;     // K dS
  using GD = Gemm<kC, CB, kC, true, false, kLD, LS>;     // P^T dO, M^T dD
  using GU = Gemm<DK, CB, kC, true, false, LD, LS>;      // Q^T dO, K^T dV
  for (int n = N - 1; n >= 0; --n) {
    const int t0 = n * kC;
    __syncthreads();
    load_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
    load_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
    load_rows<CB, LS>(s.R, dout + at.v * DV, t0, T, DV, c0);
    load_gates(s.gates, g + at.v, beta + at.v, t0, T);
    load_square<kLD>(s.M, M + ((size_t)bh * N + n) * kC * kC);
    load_square<kLD>(s.P, P + ((size_t)bh * N + n) * kC * kC);
    for (int e = tid; e < DK * CB; e += kThreads)
      ends[((size_t)bh * N + n) * DK * DV + (size_t)(e / CB) * DV + c0 + e % CB] =
          s.S[(e / CB) * LS + e % CB];
    __syncthreads();
    float ks[GS::TM][GS::TN];
    GS::zero(ks);
    GS::run(s.k, s.S, ks);
    float d[GD::TM][GD::TN];
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) d[i][j] = s.gates.to_end[GD::row(i)] * ks[i][j];
    GD::run(s.P, s.R, d);                                // dD
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) s.D[GD::row(i) * LS + GD::col(j)] = d[i][j];
    __syncthreads();
    GD::zero(d);
    GD::run(s.M, s.D, d);                                // dR
    __syncthreads();
#pragma unroll
    for (int i = 0; i < GD::TM; ++i)
#pragma unroll
      for (int j = 0; j < GD::TN; ++j) {
        const int t = GD::row(i), c = GD::col(j);
        const float x = s.gates.beta[t] * d[i][j];
        s.D[t * LS + c] = -s.gates.from_start[t] * x;
        s.R[t * LS + c] *= s.gates.from_start[t];
        if (t0 + t < T) {
          dv[(at.v + t0 + t) * DV + c0 + c] = (x);
          dR[(at.v + t0 + t) * DV + c0 + c] = d[i][j];
        }
      }
    __syncthreads();
    float up[GU::TM][GU::TN];
    GU::zero(up);
    GU::run(s.q, s.R, up);
    GU::run(s.k, s.D, up);
    const float whole = s.gates.from_start[kC - 1];
#pragma unroll
    for (int i = 0; i < GU::TM; ++i)
#pragma unroll
      for (int j = 0; j < GU::TN; ++j) {
        float &x = s.S[GU::row(i) * LS + GU::col(j)];
        x = fmaf(whole, x, up[i][j]);
      }
  }
  __syncthreads();
  if (dS0)
    for (int e = tid; e < DK * CB; e += kThreads)
      dS0[state + (size_t)(e / CB) * DV + c0 + e % CB] = s.S[(e / CB) * LS + e % CB];
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
  float row_v[kC], row_q[kC], row_k[kC], row_z[kC], row_b[kC], row_p[kC], col_p[kC];
  float dot[kThreads / 32];
  Gates gates;
};

// sum over the NX threads that share a tile row (NX a power of two)
template <int NX> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = (NX < 32 ? NX : 32) / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
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
  constexpr int LD = DK + 4, LS = CB + 4;
  const long long bh = blockIdx.x / N;
  const int n = blockIdx.x % N, t0 = n * kC, tid = threadIdx.x;
  const Where at(bh, H, Hk, T);
  const size_t border = ((size_t)bh * N + n) * DK * DV;
  load_rows<DK, LD>(s.k, k + at.k * DK, t0, T, DK, 0);
  load_rows<DK, LD>(s.q, q + at.k * DK, t0, T, DK, 0);
  load_gates(s.gates, g + at.v, beta + at.v, t0, T);
  if (tid < kC) s.row_v[tid] = s.col_p[tid] = 0.f;

  using GX = Gemm<kC, DK, CB, false, true, LS, LS>;      // X, Y, Z
  using GP = Gemm<kC, kC, CB, false, true, LS, LS>;      // dP, dL
  float X[GX::TM][GX::TN], Y[GX::TM][GX::TN], Z[GX::TM][GX::TN];
  float dP[GP::TM][GP::TN], dL[GP::TM][GP::TN];
  GX::zero(X); GX::zero(Y); GX::zero(Z);
  GP::zero(dP); GP::zero(dL);
  float dot = 0.f;
  for (int c0 = 0; c0 < DV; c0 += CB) {
    __syncthreads();
    load_rows<CB, LS>(s.dO, dout + at.v * DV, t0, T, DV, c0);
    load_rows<CB, LS>(s.dR, dRg + at.v * DV, t0, T, DV, c0);
    load_rows<CB, LS>(s.D, writes + at.v * DV, t0, T, DV, c0);
    for (int e = tid; e < DK * CB; e += kThreads) {
      const int i = (e / CB) * LS + e % CB;
      const size_t src = border + (size_t)(e / CB) * DV + c0 + e % CB;
      s.S[i] = starts[src];
      s.dS[i] = ends[src];
      dot = fmaf(s.S[i], s.dS[i], dot);
    }
    __syncthreads();
    GX::run(s.dR, s.S, X);
    GX::run(s.dO, s.S, Y);
    GX::run(s.D, s.dS, Z);
    GP::run(s.dO, s.D, dP);
    GP::run(s.dR, s.D, dL);
    // dR_t . v_t: four threads a row
    const int t = tid / 4;
    float rv = 0.f;
    if (t0 + t < T)
      for (int c = tid % 4; c < CB; c += 4)
        rv = fmaf(s.dR[t * LS + c], v[(at.v + t0 + t) * DV + c0 + c], rv);
    rv = row_sum<4>(rv);
    if (tid % 4 == 0) s.row_v[t] += rv;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  if (tid % 32 == 0) s.dot[tid / 32] = dot;

  // row dots of q, k with Y, X, Z
  static_assert(GX::NX <= 32 && GP::NX <= 32, "a tile row lies in one warp");
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
    rq = row_sum<GX::NX>(rq);
    rk = row_sum<GX::NX>(rk);
    rz = row_sum<GX::NX>(rz);
    if (tid % GX::NX == 0) {
      s.row_q[GX::row(i)] = rq;
      s.row_k[GX::row(i)] = rk;
      s.row_z[GX::row(i)] = rz;
    }
  }
  // the pair matrices
  using GK = Gemm<kC, kC, DK, false, true, LD, LD>;      // K K^T, Q K^T: GP's tile map
  float kk[GK::TM][GK::TN], qk[GK::TM][GK::TN];
  GK::zero(kk);
  GK::zero(qk);
  GK::run(s.k, s.k, kk);
  GK::run(s.q, s.k, qk);
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
    rb = row_sum<GP::NX>(rb);
    rp = row_sum<GP::NX>(rp);
    if (tid % GP::NX == 0) {
      s.row_b[t] = rb;
      s.row_p[t] = rp;
    }
  }
  __syncthreads();
  // column sums of the pairs: through the D buffer's place, in a fixed order
  {
    constexpr int NY = kThreads / GP::NX;
    float *part = s.dO;                                  // NY x 64 floats
    static_assert(NY * kC <= 3 * kC * (CB + 4), "partial sums fit in dO, dR, D");
#pragma unroll
    for (int j = 0; j < GP::TN; ++j) {
      float cs = 0.f;
#pragma unroll
      for (int i = 0; i < GP::TM; ++i) cs += pairs[i][j];
      part[(tid / GP::NX) * kC + GP::col(j)] = cs;
    }
    __syncthreads();
    if (tid < kC) {
      float cs = 0.f;
      for (int y = 0; y < NY; ++y) cs += part[y * kC + tid];
      s.col_p[tid] = cs;
    }
  }
  __syncthreads();
  if (tid < 32) {
    // dG, its sum from the right, dbeta: two tokens a lane
    const int t = 2 * tid;
    float dG[2], z = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float zt = s.gates.to_end[t + i] * s.row_z[t + i];
      z += zt;
      dG[i] = s.gates.from_start[t + i] * (s.row_q[t + i] - s.gates.beta[t + i] * s.row_k[t + i]) - zt +
              s.row_p[t + i] - s.col_p[t + i];
      if (t0 + t + i < T)
        dbeta[at.v + t0 + t + i] =
            s.row_v[t + i] - s.gates.from_start[t + i] * s.row_k[t + i] + s.row_b[t + i];
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
  using GA = Gemm<kC, DK, kC, false, false, kLD, LD>;
  using GT = Gemm<kC, DK, kC, true, false, kLD, LD>;
  float dqa[GA::TM][GA::TN], dka[GA::TM][GA::TN];
  GA::zero(dqa);
  GA::zero(dka);
  GA::run(s.pair_p, s.k, dqa);
  GA::run(s.pair_l, s.k, dka);
  GT::run(s.pair_l, s.k, dka);
  GT::run(s.pair_p, s.q, dka);
  // X, Y, Z are spread as GX's tiles (columns strided over the threads): they
  // join the sums through q's and k's place
  __syncthreads();
#pragma unroll
  for (int i = 0; i < GX::TM; ++i)
#pragma unroll
    for (int j = 0; j < GX::TN; ++j) {
      const int t = GX::row(i), e = t * LD + GX::col(j);
      s.q[e] = s.gates.from_start[t] * Y[i][j];
      s.k[e] = fmaf(-s.gates.beta[t] * s.gates.from_start[t], X[i][j], s.gates.to_end[t] * Z[i][j]);
    }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < GA::TM; ++i) {
    const int t = GA::row(i);
    if (t0 + t >= T) continue;
#pragma unroll
    for (int j = 0; j < GA::TN; ++j) {
      const int c = GA::col(j);
      const float x = dqa[i][j] + s.q[t * LD + c], y = dka[i][j] + s.k[t * LD + c];
      if (dq_part) {
        dq_part[(at.v + t0 + t) * DK + c] = x;
        dk_part[(at.v + t0 + t) * DK + c] = y;
      } else {
        dq[(at.k + t0 + t) * DK + c] = (x);
        dk[(at.k + t0 + t) * DK + c] = (y);
      }
    }
  }
}

}  // namespace gd
}  // namespace kata
