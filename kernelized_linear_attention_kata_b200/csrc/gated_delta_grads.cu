// The gradient of the gated delta rule, second kernel: dq, dk, dg and dbeta of
// every chunk from what the chains saved at its borders (bf16; this kernel for
// d_k <= 64, padded to 64, gated_delta_grads_tc.cu above). With X = dR S^T, Y = dO
// S^T, Z = D dS'^T (64 x d_k), W_ts = e^{G_t - G_s} and dP = dO D^T, dL = -dR D^T:
//   dq = e^G Y + (dP W) K,
//   dk = -beta e^G X + e^{G_C - G} Z + (dP W)^T Q + (A + A^T) K,  A = dL beta W,
//   dbeta_t = dR_t . v_t - e^{G_t} k_t . X_t + sum_s dL_ts W_ts k_t . k_s,
//   dG_t = e^{G_t} (q_t . Y_t - beta_t k_t . X_t) - z_t + sum_s pairs_ts - sum_s pairs_st,
//   dg_t = sum_{u >= t} dG_u + sum_s z_s + e^{G_C} <S, dS'>,
// z_t = e^{G_C - G_t} k_t . Z_t, pairs = dP P + dL L.
//
// The chunks are independent: no chain, so blocks of eight warps walk them, bound
// by the products: 5 MFLOP a chunk at d_v = 64 with the operand halves, 14K
// cycles. These run on the warp tensor instructions, whose accumulators stay in
// registers through the row sums and scalings between the products; in tensor
// memory each of the seven accumulators would be read back and its operands
// written out between them, which at this size takes longer (140 us instead of
// 107 at 32 heads of 4096 tokens). fp32 operands are bf16 halves; a product takes
// hi hi, hi lo and lo hi.
//
// Warp (rt, ch): rows 16 rt .. 16 rt + 15 of every 64-row result, half ch of
// its columns. Values come in panels of 64: the tiles of dO, v, dR and D (two
// slots), then S, then dS', each loaded while the one before is used.
#include "common.cuh"
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kThreads = 256;
constexpr int DK = 64;               // one panel of keys; smaller heads are padded

template <int DV> struct Layout {
  static constexpr int NV = DV / 64;
  static constexpr int kT = 6 * kPanel;                    // dO, v, dR hi, lo, D hi, lo of 64 values
  static constexpr int kS = 2 * kPanel;                    // hi, lo of 64 values
  static constexpr int kOffT = 0;
  static constexpr int kOffS = 2 * kT;
  static constexpr int kOffDS = kOffS + kS;
  static constexpr int kOffQ = kOffDS + kS;
  static constexpr int kOffK = kOffQ + kPanel;
  static constexpr int kOffA = kOffK + kPanel;             // a 64 x 64 pair matrix, hi, lo
  static constexpr int kOffGates = kOffA + 2 * kPanel;
  static constexpr int kOffRows = kOffGates + (int)sizeof(Gates);   // row sums [6][2][64], column sums [4][64]
  static constexpr int kOffBars = kOffRows + (6 * 2 + 4) * kC * 4 + 64;
  static constexpr int kBytes = kOffBars + 128 + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};
enum { kTFull = 0, kSFull = 2, kDSFull, kQkFull, kNumBars };

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Fragments from 128-byte-row tiles (64 bf16 a row, 128B swizzle):
// left operand rows r0.., depth k0.. of a tile [row][depth] / [depth][row]
__device__ __forceinline__ void left(uint32_t (&f)[4], uint32_t tile, int r0, int k0) {
  const int l = threadIdx.x % 32, m = l / 8;
  ldsm(f, tile + sw128(r0 + l % 8 + 8 * (m & 1), k0 / 8 + (m >> 1)));
}
__device__ __forceinline__ void left_t(uint32_t (&f)[4], uint32_t tile, int r0, int k0) {
  const int l = threadIdx.x % 32, m = l / 8;
  ldsm_t(f, tile + sw128(k0 + l % 8 + 8 * (m >> 1), r0 / 8 + (m & 1)));
}
// right operand of two 8-column tiles n0.., depth k0.. of a tile [depth][column] / [column][depth]
__device__ __forceinline__ void right(uint32_t (&f)[4], uint32_t tile, int k0, int n0) {
  const int l = threadIdx.x % 32, m = l / 8;
  ldsm_t(f, tile + sw128(k0 + l % 8 + 8 * (m & 1), n0 / 8 + (m >> 1)));
}
__device__ __forceinline__ void right_n(uint32_t (&f)[4], uint32_t tile, int k0, int n0) {
  const int l = threadIdx.x % 32, m = l / 8;
  ldsm(f, tile + sw128(n0 + l % 8 + 8 * (m >> 1), k0 / 8 + (m & 1)));
}
__device__ __forceinline__ float2 unpack(uint32_t x) { return as_float2(x << 16, x & 0xffff0000u); }
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

struct Args {
  const float *g, *beta;
  const uint8_t *img_S, *img_D, *img_dS, *img_dR;
  float *dg, *dbeta, *dq_part, *dk_part;
  unsigned *status;
  int H, Hk, T, N;
  int dk;                          // the tensors' d_k, <= DK
  long long jobs;
};

template <int DV>
__global__ void __launch_bounds__(kThreads, 1)
gd_grads_warp_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo,
                     const __grid_constant__ CUtensorMap tmdq, const __grid_constant__ CUtensorMap tmdk,
                     const Args a) {
  using L = Layout<DV>;
  constexpr int NV = L::NV, NT = DK / 16, HC = DK / 2;     // column tiles, columns of a warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + kNumBars);
  Gates &gt = *reinterpret_cast<Gates *>(smem + L::kOffGates);
  float *rows = reinterpret_cast<float *>(smem + L::kOffRows), *cols = rows + 6 * 2 * kC, *dots = cols + 4 * kC;
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rt = warp % 4, ch = warp / 4, g = lane / 4, q2 = 2 * (lane % 4);
  const bool below = ch == 0 || rt >= 2;                   // its 16 x 32 pairs are not all above the diagonal

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();

  // loads, by thread 0: units are (job, value panel) in order
  auto head = [&](long long job) { return (int)(job / a.N); };
  auto load_t = [&](long long job, int vp, int slot) {
    const int bh = head(job), t0 = (int)(job % a.N) * kC;
    uint8_t *dst = smem + L::kOffT + slot * L::kT;
    mbar_arrive_expect_tx(&bars[kTFull + slot], L::kT);
    tma_load_3d(dst, &tmdo, &bars[kTFull + slot], 64 * vp, t0, bh);
    tma_load_3d(dst + kPanel, &tmv, &bars[kTFull + slot], 64 * vp, t0, bh);
#pragma unroll
    for (int lo = 0; lo < 2; ++lo) {
      const size_t at = (size_t)job * write_image(DV) + lo * (write_image(DV) / 2) + vp * kPanel;
      bulk_load(dst + (2 + lo) * kPanel, a.img_dR + at, kPanel, &bars[kTFull + slot]);
      bulk_load(dst + (4 + lo) * kPanel, a.img_D + at, kPanel, &bars[kTFull + slot]);
    }
  };
  auto load_state = [&](const uint8_t *img, long long job, int vp, int off, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, L::kS);
#pragma unroll
    for (int lo = 0; lo < 2; ++lo)
      bulk_load(smem + off + lo * kPanel,
                img + (size_t)job * state_image(DK, DV) + lo * (state_image(DK, DV) / 2) + vp * kPanel, kPanel, bar);
  };
  auto load_qk = [&](long long job) {
    const int bh = head(job), t0 = (int)(job % a.N) * kC;
    const int kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
    mbar_arrive_expect_tx(&bars[kQkFull], 2 * kPanel);
    tma_load_3d(smem + L::kOffQ, &tmq, &bars[kQkFull], 0, t0, kh);
    tma_load_3d(smem + L::kOffK, &tmk, &bars[kQkFull], 0, t0, kh);
  };
  const long long first = blockIdx.x;
  if (tid == 0 && first < a.jobs) {
    load_t(first, 0, 0);
    load_state(a.img_S, first, 0, L::kOffS, &bars[kSFull]);
    load_state(a.img_dS, first, 0, L::kOffDS, &bars[kDSFull]);
    load_qk(first);
  }

  // A wait that gave up leaves garbage behind and the abort flag up: the block
  // goes on through its barriers and reports at the end. Thread 0 loads no more then: a
  // load on each barrier starts only after its own wait for the one before.
  int unit = 0, nth = 0, sent_t = 1, sent_s = 1, sent_ds = 1, sent_qk = 1;
  bool ok = true;
  auto landed = [&](int bar, uint32_t parity) { ok &= mbar_wait(&bars[bar], parity, abort_flag); };
  auto may_load = [&]() { return tid == 0 && gdsync::may_load_own(ok); };
  for (long long job = first; job < a.jobs; job += gridDim.x, ++nth) {
    const int bh = head(job), t0 = (int)(job % a.N) * kC;
    const size_t tok = (size_t)bh * a.T + t0;
    const int left_t0 = a.T - t0;
    if (warp == 4) {                                       // it has no pairs of its own
      const int u = 2 * lane;
      make_gates(gt, u < left_t0 ? a.g[tok + u] : 0.f, u + 1 < left_t0 ? a.g[tok + u + 1] : 0.f,
                 u < left_t0 ? a.beta[tok + u] : 0.f, u + 1 < left_t0 ? a.beta[tok + u + 1] : 0.f);
    }
    float X[NT][4], Y[NT][4], Z[NT][4], dP[4][4], dL[4][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) X[n][i] = Y[n][i] = Z[n][i] = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) dP[n][i] = dL[n][i] = 0.f;
    float rv[2] = {0.f, 0.f}, dot = 0.f;

    for (int vp = 0; vp < NV; ++vp, ++unit) {
      const int slot = unit & 1;
      const long long next_job = vp + 1 < NV ? job : job + gridDim.x;
      const int next_vp = vp + 1 < NV ? vp + 1 : 0;
      const bool more = next_job < a.jobs;
      if (more && may_load()) {                            // free since the unit before ended
        load_t(next_job, next_vp, slot ^ 1);
        ++sent_t;
      }
      const uint32_t t_dO = base + L::kOffT + slot * L::kT, t_v = t_dO + kPanel, t_dR = t_dO + 2 * kPanel,
                     t_D = t_dO + 4 * kPanel;
      landed(kTFull + slot, (unit >> 1) & 1);
      landed(kSFull, unit & 1);
#pragma unroll 1
      for (int k = 0; k < 64; k += 16) {
        uint32_t fo[4], rh[4], rl[4], b[4], c[4];
        left(fo, t_dO, 16 * rt, k);
        left_t(rh, t_dR, 16 * rt, k);
        left_t(rl, t_dR + kPanel, 16 * rt, k);
        if (below) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            right(b, t_D, k, 32 * ch + 16 * n);
            right(c, t_D + kPanel, k, 32 * ch + 16 * n);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma(dP[2 * n + i], fo, b[2 * i], b[2 * i + 1]);
              mma(dP[2 * n + i], fo, c[2 * i], c[2 * i + 1]);
              mma(dL[2 * n + i], rh, b[2 * i], b[2 * i + 1]);
              mma(dL[2 * n + i], rh, c[2 * i], c[2 * i + 1]);
              mma(dL[2 * n + i], rl, b[2 * i], b[2 * i + 1]);
            }
          }
        }
        if ((k / 16 & 1) == ch) {                          // dR . v, half the depth a warp
          left(b, t_v, 16 * rt, k);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = unpack(b[i]), x = unpack(rh[i]), y = unpack(rl[i]);
            rv[i & 1] = fmaf(v.x, x.x + y.x, fmaf(v.y, x.y + y.y, rv[i & 1]));
          }
        }
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          right(b, base + L::kOffS, k, HC * ch + 16 * n);
          right(c, base + L::kOffS + kPanel, k, HC * ch + 16 * n);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma(Y[2 * n + i], fo, b[2 * i], b[2 * i + 1]);
            mma(Y[2 * n + i], fo, c[2 * i], c[2 * i + 1]);
            mma(X[2 * n + i], rh, b[2 * i], b[2 * i + 1]);
            mma(X[2 * n + i], rh, c[2 * i], c[2 * i + 1]);
            mma(X[2 * n + i], rl, b[2 * i], b[2 * i + 1]);
          }
        }
      }
      landed(kDSFull, unit & 1);
      // <S, dS'>: the tiles hold both in the same places
      for (int e = tid; e < kPanel / 16; e += kThreads) {
        const uint4 sh = *reinterpret_cast<const uint4 *>(smem + L::kOffS + 16 * e);
        const uint4 sl = *reinterpret_cast<const uint4 *>(smem + L::kOffS + kPanel + 16 * e);
        const uint4 dh = *reinterpret_cast<const uint4 *>(smem + L::kOffDS + 16 * e);
        const uint4 dl = *reinterpret_cast<const uint4 *>(smem + L::kOffDS + kPanel + 16 * e);
        auto pair = [&](uint32_t h1, uint32_t l1, uint32_t h2, uint32_t l2) {
          const float2 p = unpack(h1), q = unpack(l1), r = unpack(h2), s = unpack(l2);
          dot = fmaf(p.x + q.x, r.x + s.x, fmaf(p.y + q.y, r.y + s.y, dot));
        };
        pair(sh.x, sl.x, dh.x, dl.x);
        pair(sh.y, sl.y, dh.y, dl.y);
        pair(sh.z, sl.z, dh.z, dl.z);
        pair(sh.w, sl.w, dh.w, dl.w);
      }
      __syncthreads();                                     // S has been read
      if (more && may_load()) {
        load_state(a.img_S, next_job, next_vp, L::kOffS, &bars[kSFull]);
        ++sent_s;
      }
#pragma unroll 1
      for (int k = 0; k < 64; k += 16) {
        uint32_t dh[4], dl[4], b[4], c[4];
        left_t(dh, t_D, 16 * rt, k);
        left_t(dl, t_D + kPanel, 16 * rt, k);
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          right(b, base + L::kOffDS, k, HC * ch + 16 * n);
          right(c, base + L::kOffDS + kPanel, k, HC * ch + 16 * n);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma(Z[2 * n + i], dh, b[2 * i], b[2 * i + 1]);
            mma(Z[2 * n + i], dh, c[2 * i], c[2 * i + 1]);
            mma(Z[2 * n + i], dl, b[2 * i], b[2 * i + 1]);
          }
        }
      }
      __syncthreads();                                     // dS' and the slot have been read; the gates are there
      if (more && may_load()) {
        load_state(a.img_dS, next_job, next_vp, L::kOffDS, &bars[kDSFull]);
        ++sent_ds;
      }
    }

    // ---- pairs of tokens
    landed(kQkFull, nth & 1);
    const uint32_t t_q = base + L::kOffQ, t_k = base + L::kOffK, t_a = base + L::kOffA;
    float qk[4][4], kk[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) qk[n][i] = kk[n][i] = 0.f;
    if (below) {
#pragma unroll 1
      for (int k = 0; k < DK; k += 16) {
        uint32_t fq[4], fk[4], b[4];
        left(fq, t_q, 16 * rt, k);
        left(fk, t_k, 16 * rt, k);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          right_n(b, t_k, k, 32 * ch + 16 * n);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma(qk[2 * n + i], fq, b[2 * i], b[2 * i + 1]);
            mma(kk[2 * n + i], fk, b[2 * i], b[2 * i + 1]);
          }
        }
      }
    }
    // dP <- dP W, dL <- dL beta W; the sums over s and over t
    auto row_of = [&](int i) { return 16 * rt + g + 8 * (i >> 1); };   // of accumulator entry i
    float rb[2] = {0.f, 0.f}, rp[2] = {0.f, 0.f}, cp[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      cp[n][0] = cp[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = row_of(i), s = 32 * ch + 8 * n + q2 + (i & 1);
        const float w = s <= t ? exp2_fast((gt.hi[t] - gt.hi[s]) + (gt.lo[t] - gt.lo[s])) : 0.f;
        const float p = s <= t ? dP[n][i] * w : 0.f, l = s < t ? -dL[n][i] * w : 0.f;
        const float lb = l * gt.beta[t], pr = fmaf(p, qk[n][i], lb * kk[n][i]);
        rb[i >> 1] = fmaf(l, kk[n][i], rb[i >> 1]);
        rp[i >> 1] += pr;
        cp[n][i & 1] += pr;
        dP[n][i] = p;
        dL[n][i] = lb;
      }
    }
    // row dots of q and k with Y, X, Z, which take their factors in dq and dk on the way
    float rq[2] = {0.f, 0.f}, rk[2] = {0.f, 0.f}, rz[2] = {0.f, 0.f};
#pragma unroll
    for (int hrow = 0; hrow < 2; ++hrow) {
      const int t = 16 * rt + g + 8 * hrow;
      const float f = gt.from_start[t], e = gt.to_end[t], fb = f * gt.beta[t];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = HC * ch + 8 * n + q2;
        const uint32_t at = sw128(t, col / 8) + (col % 8) * 2;
        const float2 q = unpack(*reinterpret_cast<const uint32_t *>(smem + L::kOffQ + at));
        const float2 k = unpack(*reinterpret_cast<const uint32_t *>(smem + L::kOffK + at));
        float &x0 = X[n][2 * hrow], &x1 = X[n][2 * hrow + 1], &y0 = Y[n][2 * hrow], &y1 = Y[n][2 * hrow + 1];
        const float z0 = Z[n][2 * hrow], z1 = Z[n][2 * hrow + 1];
        rq[hrow] = fmaf(q.x, y0, fmaf(q.y, y1, rq[hrow]));
        rk[hrow] = fmaf(k.x, x0, fmaf(k.y, x1, rk[hrow]));
        rz[hrow] = fmaf(k.x, z0, fmaf(k.y, z1, rz[hrow]));
        y0 *= f;                                           // dq so far
        y1 *= f;
        x0 = fmaf(-fb, x0, e * z0);                        // dk so far
        x1 = fmaf(-fb, x1, e * z1);
      }
    }
    {
      const float sums[6][2] = {{rq[0], rq[1]}, {rk[0], rk[1]}, {rz[0], rz[1]},
                                {rb[0], rb[1]}, {rp[0], rp[1]}, {rv[0], rv[1]}};
#pragma unroll
      for (int j = 0; j < 6; ++j)
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
          const float x = quad_sum(sums[j][hrow]);
          if (lane % 4 == 0) rows[(2 * j + ch) * kC + 16 * rt + g + 8 * hrow] = x;
        }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = cp[n][i];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
          if (g == 0) cols[rt * kC + 32 * ch + 8 * n + q2 + i] = x;
        }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (lane == 0) dots[warp] = dot;
    }
    auto put_pairs = [&](const float (&m)[4][4]) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
          const int t = 16 * rt + g + 8 * hrow, s = 32 * ch + 8 * n + q2;
          uint32_t hi, lo;
          split2(make_float2(m[n][2 * hrow], m[n][2 * hrow + 1]), hi, lo);
          uint8_t *dst = smem + L::kOffA + sw128(t, s / 8) + (s % 8) * 2;
          *reinterpret_cast<uint32_t *>(dst) = hi;
          *reinterpret_cast<uint32_t *>(dst + kPanel) = lo;
        }
    };
    put_pairs(dP);
    __syncthreads();
    if (warp == 7) {                                       // dg, dbeta: two tokens a lane
      const int t = 2 * lane;
      auto sum = [&](int j, int u) { return rows[2 * j * kC + u] + rows[(2 * j + 1) * kC + u]; };
      float dG[2], z = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = t + i;
        const float zt = gt.to_end[u] * sum(2, u), fk = gt.from_start[u] * sum(1, u);
        z += zt;
        const float down = (cols[u] + cols[kC + u]) + (cols[2 * kC + u] + cols[3 * kC + u]);
        dG[i] = fmaf(gt.from_start[u], sum(0, u), -gt.beta[u] * fk) - zt + sum(4, u) - down;
        if (u < left_t0) a.dbeta[tok + u] = sum(5, u) - fk + sum(3, u);
      }
      float last = z, up = dG[0] + dG[1], border = 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) last += __shfl_xor_sync(0xffffffffu, last, off);
#pragma unroll
      for (int w = 0; w < 8; ++w) border += dots[w];
      last = fmaf(gt.from_start[kC - 1], border, last);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, up, off);
        if (lane + off < 32) up += x;
      }
      if (t < left_t0) a.dg[tok + t] = up + last;
      if (t + 1 < left_t0) a.dg[tok + t + 1] = up - dG[0] + last;
    }
    // acc (rows 16 rt.., the warp's columns) += A or A^T (hi, lo) times the rows of a q or k tile
    auto pair_product = [&](float (&acc)[NT][4], bool transposed, uint32_t tile) {
#pragma unroll 1
      for (int k = transposed ? 16 * rt : 0; k < (transposed ? 64 : 16 * rt + 16); k += 16) {
        uint32_t h[4], l[4], b[4];
        if (transposed) {
          left_t(h, t_a, 16 * rt, k);
          left_t(l, t_a + kPanel, 16 * rt, k);
        } else {
          left(h, t_a, 16 * rt, k);
          left(l, t_a + kPanel, 16 * rt, k);
        }
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          const int col = HC * ch + 16 * n;
          right(b, tile, k, col);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma(acc[2 * n + i], h, b[2 * i], b[2 * i + 1]);
            mma(acc[2 * n + i], l, b[2 * i], b[2 * i + 1]);
          }
        }
      }
    };
    pair_product(Y, false, t_k);
    pair_product(X, true, t_q);
    __syncthreads();
    put_pairs(dL);
    __syncthreads();
    pair_product(X, false, t_k);
    pair_product(X, true, t_k);
    __syncthreads();                                       // q, k and the pairs have been read
    if (a.dq_part) {
#pragma unroll
      for (int hrow = 0; hrow < 2; ++hrow) {
        const int t = 16 * rt + g + 8 * hrow;
        if (t < left_t0)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int col = HC * ch + 8 * n + q2;
            const size_t at = (tok + t) * a.dk + col;
            if (col < a.dk) {
              *reinterpret_cast<float2 *>(a.dq_part + at) = make_float2(Y[n][2 * hrow], Y[n][2 * hrow + 1]);
              *reinterpret_cast<float2 *>(a.dk_part + at) = make_float2(X[n][2 * hrow], X[n][2 * hrow + 1]);
            }
          }
      }
      if (job + gridDim.x < a.jobs && may_load()) {
        load_qk(job + gridDim.x);
        ++sent_qk;
      }
    } else {
#pragma unroll
      for (int hrow = 0; hrow < 2; ++hrow) {
        const int t = 16 * rt + g + 8 * hrow;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int col = HC * ch + 8 * n + q2;
          const uint32_t at = sw128(t, col / 8) + (col % 8) * 2;
          *reinterpret_cast<uint32_t *>(smem + L::kOffQ + at) = pack_bf16x2(Y[n][2 * hrow], Y[n][2 * hrow + 1]);
          *reinterpret_cast<uint32_t *>(smem + L::kOffK + at) = pack_bf16x2(X[n][2 * hrow], X[n][2 * hrow + 1]);
        }
      }
      fence_async_smem();
      __syncthreads();
      if (tid == 0) {
        tma_store_3d(&tmdq, smem + L::kOffQ, 0, t0, bh);
        tma_store_3d(&tmdk, smem + L::kOffK, 0, t0, bh);
        bulk_commit_group();
        bulk_wait_read_all();
        if (job + gridDim.x < a.jobs && may_load()) {
          load_qk(job + gridDim.x);
          ++sent_qk;
        }
      }
    }
  }
  if (tid == 0) {
    bulk_wait_all();
    if (first < a.jobs) {                                  // copies in flight land before the exit
      for (int u = sent_t > 2 ? sent_t - 2 : 0; u < sent_t; ++u) drain(&bars[kTFull + (u & 1)], (u >> 1) & 1);
      drain(&bars[kSFull], (sent_s - 1) & 1);
      drain(&bars[kDSFull], (sent_ds - 1) & 1);
      drain(&bars[kQkFull], (sent_qk - 1) & 1);
    }
    if (*abort_flag) flag_status(a.status, kStatusDeviceTimeout);
  }
}

template <int DV> cudaError_t launch(const GatedDeltaLaunch &a, int d_k, int d_v) {
  CUtensorMap tq, tk, tv, tdo, tdq, tdk;
  const long long BHk = a.BH / a.H * a.Hk;
  if (!make_tma_3d_bf16_box(&tq, a.q, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tk, a.k, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tv, a.v, d_v, a.T, a.BH, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdo, a.dout, d_v, a.T, a.BH, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdq, a.dq, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdk, a.dk, d_k, a.T, BHk, 64, kC, true))
    return cudaErrorInvalidValue;
  constexpr int bytes = Layout<DV>::kBytes;
  auto kern = gd_grads_warp_kernel<DV>;
  GD_ALLOW_SMEM(kern, bytes);
  const Args x{a.g, a.beta, a.img_S, a.img_D, a.img_dS, a.img_dR, a.dg, a.dbeta, a.dq_part, a.dk_part,
               a.status, a.H, a.Hk, a.T, a.N, d_k, a.BH * a.N};
  ProfileScope prof("gd_tc_grads", a.stream);
  kern<<<(unsigned)(x.jobs < kGdSms ? x.jobs : kGdSms), kThreads, bytes, a.stream>>>(tq, tk, tv, tdo, tdq, tdk, x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_tc_grads(const GatedDeltaLaunch &a, int d_k, int d_v) {
  if (gd_padded(d_k) == 128) return gd_tc_grads_wide(a, d_k, d_v);
  const cudaError_t e = gd_padded(d_v) == 64 ? launch<64>(a, d_k, d_v) : launch<128>(a, d_k, d_v);
  return e == cudaSuccess && a.dq_part ? gd_sum_groups(a, d_k, true) : e;
}

cudaError_t gd_tc_backward(const GatedDeltaLaunch &a, int d_k, int d_v) {
  cudaError_t e = gd_tc_solve(a, d_k);
  if (e == cudaSuccess) e = gd_tc_effect(a, d_k, d_v);
  if (e == cudaSuccess) e = gd_tc_reverse_effect(a, d_k, d_v);
  if (e == cudaSuccess) e = gd_tc_join(a, d_k, d_v);
  if (e == cudaSuccess) e = gd_tc_save(a, d_k, d_v);
  if (e == cudaSuccess) e = gd_tc_reverse(a, d_k, d_v);
  return e == cudaSuccess ? gd_tc_grads(a, d_k, d_v) : e;
}

}  // namespace kata
