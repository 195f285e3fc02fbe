// dq, dk, dg and dbeta of every chunk for 64 < d_k <= 128 (bf16), by tcgen05; the
// formulas are those of gated_delta_grads.cu, the kernel of the smaller heads.
//
// The chunks are independent: no chain, so blocks walk them one after another.
// Everything is transposed, keys on TMEM lanes and tokens along columns: X^T =
// S dR^T, Y^T = S dO^T and Z^T = dS' D^T have d_k rows, dP^T and dL^T (and K K^T, K
// Q^T) tokens s on the lanes and t along the columns. fp32 operands are bf16 halves;
// a product takes hi hi, lo hi and hi lo. Bound by its MMAs (144 a chunk at d_v
// = 128, 70-85 cycles each) and by the passes over tensor memory between them,
// whose loads come slowly while MMAs run: 21K cycles a chunk, where accumulators
// in registers took 28K (366 us instead of 425 at 16 heads of 16384 tokens). For
// d_k = 64 it is the other way round: 140 us against 107 at 32 heads of 4096.
//
// Warps: 0-15 the lanes' warps (four warpgroups, 16 tokens each), of which 8 (TMEM
// lanes 64-127, where there are no pairs) take dR . v and <S, dS'>; 16 the MMA
// issuer; 17 the loads and stores. Values come in panels of 64.
#include "common.cuh"
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kThreads = kLoader * 32 + 32;
constexpr int kLaneThreads = kStateWarps * 32;
constexpr uint32_t kTmemCols = 512;
// Tensor memory columns: X (then dk), Y (then dq), Z, dP, dL, K K^T and K Q^T.
constexpr uint32_t kColX = 0, kColY = 64, kColZ = 128, kColP = 192, kColL = 256, kColKK = 320, kColQK = 384;

struct RowSums {                     // by the warps that hold parts of them
  float q[4][kC], k[4][kC], z[4][kC];   // q_t . Y_t, k_t . X_t, k_t . Z_t
  float b[2][kC], p[2][kC];          // sum_s dL W k.k, sum_s pairs_ts
  float down[4][kC];                 // sum_t pairs_ts
  float v[4][kC];                    // dR_t . v_t
  float dots[8];                     // <S, dS'>
};

template <int DK, int DV> struct Layout {
  static constexpr int NP = DK / 64, NV = DV / 64;
  static constexpr int kT = 5 * kPanel;                    // dO, dR hi, lo, D hi, lo of 64 values
  static constexpr int kS = 2 * NP * kPanel;               // hi panels, lo panels of 64 values
  static constexpr int kQk = 2 * NP * kPanel;              // [K p0][Q p0][K p1][Q p1], then dk, dq
  static constexpr int kOffT = 0;
  static constexpr int kOffV = 2 * kT;
  static constexpr int kOffS = kOffV + kPanel;
  static constexpr int kOffDS = kOffS + kS;
  static constexpr int kOffQk = kOffDS + kS;
  static constexpr int kOffA = kOffQk + kQk;          // dP W hi, lo; A hi, lo
  static constexpr int kOffGates = kOffA + 4 * kPanel;
  static constexpr int kOffRows = kOffGates + 2 * (int)sizeof(Gates);
  static constexpr int kOffBars = kOffRows + (int)sizeof(RowSums);
  static constexpr int kBytes = kOffBars + 256 + 1024;
  static_assert(kBytes <= 232448, "shared memory budget");
};
// Loaded and free: tiles, v, S, dS'; q and k are loaded, dq and dk are in their
// place. Then per chunk: the pairs' products and X, Y and Z are done; the operands
// of dq and dk are ready; dq and dk are done; they have been read.
enum {
  kTFull = 0, kTFree = 2, kVFull = 4, kVFree, kSFull, kSFree, kDSFull, kDSFree, kQkFull, kOut, kPairs,
  kXyz, kReady, kDone, kRead, kEnd, kNumBars
};

__device__ __forceinline__ float2 unpack(uint32_t x) { return as_float2(x << 16, x & 0xffff0000u); }
__device__ __forceinline__ float bf16_at(const uint8_t *p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(p) << 16);
}
__device__ __forceinline__ void lane_warps_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kLaneThreads) : "memory");
}
// Sums of N columns over a warp's lanes: 32 / N neighbours return column lane / (32 / N)'s.
template <int N> __device__ __forceinline__ float sum_columns(float (&v)[N]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int half = N / 2; half >= 1; half >>= 1) {
    const int off = 32 / N * half;
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
#pragma unroll
  for (int off = 16 / N; off >= 1; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}

// The same value, of which the compiler keeps nothing over the loops: addresses
// made of it are made anew in each phase and take no registers in the others.
__device__ __forceinline__ int afresh(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

struct Args {
  const float *g, *beta;
  const uint8_t *img_S, *img_D, *img_dS, *img_dR;
  float *dg, *dbeta, *dq_part, *dk_part;
  unsigned *status;
  int H, Hk, T, N;
  int dk;                          // the tensors' d_k, <= DK
  int fold;                        // value heads a block takes one after another, adding up dq and dk
  long long units;                 // chunks, of query / key heads if fold > 1
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
gd_grads_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmdo,
                   const __grid_constant__ CUtensorMap tmdq, const __grid_constant__ CUtensorMap tmdk,
                   const Args a) {
  using L = Layout<DK, DV>;
  constexpr int NP = L::NP, NV = L::NV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Gates *gates = reinterpret_cast<Gates *>(smem + L::kOffGates);
  RowSums &rows = *reinterpret_cast<RowSums *>(smem + L::kOffRows);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int jobs = (int)((a.units - blockIdx.x + gridDim.x - 1) / gridDim.x) * a.fold;   // of this block
  // value head and chunk of the block's j-th job, as head * N + chunk
  auto job_of = [&](int j) {
    const long long unit = (long long)blockIdx.x + (long long)(j / a.fold) * gridDim.x;
    return (unit / a.N * a.fold + j % a.fold) * a.N + unit % a.N;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if (i == kTFree || i == kTFree + 1 || i == kSFree || i == kDSFree) count = 1 + kStateWarps / 2;
      if (i == kVFree) count = kStateWarps / 2;
      if (i == kReady || i == kRead || i == kOut) count = kStateWarps;
      mbar_init(&bars[i], count);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kIssuer) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp < kStateWarps) {
    const int h = warp / 4, quarter = warp % 4;            // tokens 16 h .., TMEM lanes 32 quarter ..
    const int r = 32 * quarter + lane;                     // key column; token s of the pairs (quarter < 2)
    const uint32_t col = tbase + ((uint32_t)(32 * quarter) << 16) + 16 * h;
    int unit = 0;
    for (int j = 0; j < jobs; ++j) {
      const long long job = job_of(j);
      const int bh = (int)(job / a.N), t0 = (int)(job % a.N) * kC;
      const size_t tok = (size_t)bh * a.T + t0;
      const int left = a.T - t0;
      Gates &gt = gates[j & 1];
      if (warp == 2) {
        const int u = 2 * lane;
        make_gates(gt, u < left ? a.g[tok + u] : 0.f, u + 1 < left ? a.g[tok + u + 1] : 0.f,
                   u < left ? a.beta[tok + u] : 0.f, u + 1 < left ? a.beta[tok + u + 1] : 0.f);
      }
      lane_warps_sync();                                   // the gates are there; the row sums have been read
      if (quarter >= 2) {
        // ------------------------------------------- dR . v and <S, dS'>
        const int extra = afresh(h * 64 + (quarter - 2) * 32 + lane);   // 0 .. 255
        const int t = extra % 64, part = extra / 64;
        float rv = 0.f, dot = 0.f;
        for (int p = 0; p < NV; ++p, ++unit) {
          const int slot = unit & 1;
          const uint8_t *tile = smem + L::kOffT + slot * L::kT;
          warp_wait(&bars[kTFull + slot], (unit >> 1) & 1, abort_flag);
          warp_wait(&bars[kVFull], unit & 1, abort_flag);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(smem + L::kOffV + sw128(t, 2 * part + c));
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t at = sw128(16 * part + 8 * c + i, t / 8) + (t % 8) * 2;
              const float2 pair = unpack(v[i / 2]);
              rv = fmaf(i % 2 ? pair.y : pair.x, bf16_at(tile + kPanel + at) + bf16_at(tile + 2 * kPanel + at), rv);
            }
          }
          warp_arrive(&bars[kVFree]);
          warp_arrive(&bars[kTFree + slot]);
          warp_wait(&bars[kSFull], unit & 1, abort_flag);
          warp_wait(&bars[kDSFull], unit & 1, abort_flag);
          // the tiles hold both in the same places
          for (int e = extra; e < NP * kPanel / 16; e += kLaneThreads / 2) {
            auto at = [&](int off, int lo) {
              return *reinterpret_cast<const uint4 *>(smem + off + lo * NP * kPanel + 16 * e);
            };
            const uint4 sh = at(L::kOffS, 0), sl = at(L::kOffS, 1), dh = at(L::kOffDS, 0), dl = at(L::kOffDS, 1);
            auto pair = [&](uint32_t h1, uint32_t l1, uint32_t h2, uint32_t l2) {
              const float2 p1 = unpack(h1), q1 = unpack(l1), p2 = unpack(h2), q2 = unpack(l2);
              dot = fmaf(p1.x + q1.x, p2.x + q2.x, fmaf(p1.y + q1.y, p2.y + q2.y, dot));
            };
            pair(sh.x, sl.x, dh.x, dl.x);
            pair(sh.y, sl.y, dh.y, dl.y);
            pair(sh.z, sl.z, dh.z, dl.z);
            pair(sh.w, sl.w, dh.w, dl.w);
          }
          warp_arrive(&bars[kSFree]);
          warp_arrive(&bars[kDSFree]);
        }
        rows.v[part][t] = rv;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) rows.dots[2 * h + quarter - 2] = dot;
      } else {
        // ------------------------------------------- pairs (s = r, t = 16 h ..)
        warp_wait(&bars[kPairs], j & 1, abort_flag);
        tc_fence_after();
        uint8_t *pw = smem + L::kOffA;
        const int r = afresh(32 * quarter + lane);
        const float hi = gt.hi[r], lo = gt.lo[r];
        float down = 0.f;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t dP[8], dL[8], kk[8], qk[8];
          tmem_ld8(col + kColP + 8 * half, dP);
          tmem_ld8(col + kColL + 8 * half, dL);
          tmem_ld8(col + kColKK + 8 * half, kk);
          tmem_ld8(col + kColQK + 8 * half, qk);
          tmem_wait_ld();
          // the values first, the stores after them: a load of the gates would wait
          // for the stores before it
          float b[8], p[8], x[8], y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = 16 * h + 8 * half + i;
            const float w = t >= r ? exp2_fast((gt.hi[t] - hi) + (gt.lo[t] - lo)) : 0.f;
            const float l = t > r ? -__uint_as_float(dL[i]) * w : 0.f;          // dL W, dL = -dR D^T
            const float k2 = __uint_as_float(kk[i]);
            x[i] = t >= r ? __uint_as_float(dP[i]) * w : 0.f;                   // dP W
            y[i] = l * gt.beta[t];
            b[i] = t > r ? l * k2 : 0.f;
            p[i] = t >= r ? fmaf(x[i], __uint_as_float(qk[i]), t > r ? y[i] * k2 : 0.f) : 0.f;
            down += p[i];
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            uint32_t xh, xl, yh, yl;
            split2(make_float2(x[i], x[i + 1]), xh, xl);
            split2(make_float2(y[i], y[i + 1]), yh, yl);
            const uint32_t v[4] = {xh, xl, yh, yl};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint8_t *dst = pw + sw128(16 * h + 8 * half + i + u, r / 8) + (r % 8) * 2;
#pragma unroll
              for (int w = 0; w < 4; ++w)
                *reinterpret_cast<uint16_t *>(dst + w * kPanel) = (uint16_t)(v[w] >> (16 * u));
            }
          }
          const float sb = sum_columns(b), sp = sum_columns(p);
          if (lane % 4 == 0) {
            rows.b[quarter][16 * h + 8 * half + lane / 4] = sb;
            rows.p[quarter][16 * h + 8 * half + lane / 4] = sp;
          }
        }
        rows.down[h][r] = down;
      }

      // --------------------------------------------- X, Y, Z: row dots, factors
      const uint8_t *kt = smem + L::kOffQk, *qt = kt + kPanel;
      int key = afresh(r);
      auto at_token = [&](int i) {
        return (uint32_t)(key / 64) * 2 * kPanel + (key % 8) * 2 + sw128(16 * h + i, key % 64 / 8);
      };
      warp_wait(&bars[kQkFull], j & 1, abort_flag);
      warp_wait(&bars[kXyz], j & 1, abort_flag);
      tc_fence_after();
      {
        uint32_t y[16];
        float s[16];
        tmem_ld16(col + kColY, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = bf16_at(qt + at_token(i)) * __uint_as_float(y[i]);
          y[i] = __float_as_uint(gt.from_start[16 * h + i] * __uint_as_float(y[i]));
        }
        tmem_st16(col + kColY, y);                         // dq so far
        const float sq = sum_columns(s);
        uint32_t x[16];
        tmem_ld16(col + kColX, x);
        tmem_ld16(col + kColZ, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = bf16_at(kt + at_token(i)) * __uint_as_float(x[i]);
        const float sk = sum_columns(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[i] = bf16_at(kt + at_token(i)) * __uint_as_float(y[i]);
          const float fb = gt.from_start[16 * h + i] * gt.beta[16 * h + i];
          x[i] = __float_as_uint(fmaf(-fb, __uint_as_float(x[i]), gt.to_end[16 * h + i] * __uint_as_float(y[i])));
        }
        tmem_st16(col + kColX, x);                         // dk so far
        const float sz = sum_columns(s);
        tmem_wait_st();
        if (lane % 2 == 0) {
          const int t = 16 * h + lane / 2;
          rows.q[quarter][t] = sq;
          rows.k[quarter][t] = sk;
          rows.z[quarter][t] = sz;
        }
      }
      fence_async_smem();
      tc_fence_before();
      warp_arrive(&bars[kReady]);
      lane_warps_sync();                                   // the row sums are there
      if (warp == 15) {                                    // dg, dbeta: two tokens a lane
        const int t = 2 * lane;
        auto four = [&](const float (&x)[4][kC], int u) { return (x[0][u] + x[1][u]) + (x[2][u] + x[3][u]); };
        float dG[2], z = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = t + i;
          const float zt = gt.to_end[u] * four(rows.z, u), fk = gt.from_start[u] * four(rows.k, u);
          z += zt;
          dG[i] = fmaf(gt.from_start[u], four(rows.q, u), -gt.beta[u] * fk) - zt + (rows.p[0][u] + rows.p[1][u]) -
                  four(rows.down, u);
          if (u < left) a.dbeta[tok + u] = four(rows.v, u) - fk + (rows.b[0][u] + rows.b[1][u]);
        }
        float last = z, up = dG[0] + dG[1], border = 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) last += __shfl_xor_sync(0xffffffffu, last, off);
#pragma unroll
        for (int w = 0; w < 8; ++w) border += rows.dots[w];
        last = fmaf(gt.from_start[kC - 1], border, last);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const float x = __shfl_down_sync(0xffffffffu, up, off);
          if (lane + off < 32) up += x;
        }
        if (t < left) a.dg[tok + t] = up + last;
        if (t + 1 < left) a.dg[tok + t + 1] = up - dG[0] + last;
      }

      // --------------------------------------------- dq, dk
      warp_wait(&bars[kDone], j & 1, abort_flag);
      tc_fence_after();
      key = afresh(r);
      uint32_t x[16], y[16];
      tmem_ld16(col + kColX, x);
      tmem_ld16(col + kColY, y);
      tmem_wait_ld();
      tc_fence_before();
      warp_arrive(&bars[kRead]);
      const int nth = j % a.fold;                          // of the heads that are added up
      const bool last = nth == a.fold - 1;
      if (a.dq_part && r < a.dk) {
        // parts: a value head's, or the sum so far of a query / key head's (which
        // this thread has written)
        const size_t row = ((size_t)(bh / a.fold) * a.T + t0 + 16 * h) * a.dk + r;
        if (nth > 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * h + i < left) {
              y[i] = __float_as_uint(a.dq_part[row + (size_t)i * a.dk] + __uint_as_float(y[i]));
              x[i] = __float_as_uint(a.dk_part[row + (size_t)i * a.dk] + __uint_as_float(x[i]));
            }
        }
        if (a.fold == 1 || !last) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * h + i < left) {
              a.dq_part[row + (size_t)i * a.dk] = __uint_as_float(y[i]);
              a.dk_part[row + (size_t)i * a.dk] = __uint_as_float(x[i]);
            }
        }
      }
      if (!a.dq_part || (a.fold > 1 && last)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint8_t *dst = smem + L::kOffQk + at_token(i);
          *reinterpret_cast<__nv_bfloat16 *>(dst) = __float2bfloat16_rn(__uint_as_float(x[i]));
          *reinterpret_cast<__nv_bfloat16 *>(dst + kPanel) = __float2bfloat16_rn(__uint_as_float(y[i]));
        }
        fence_async_smem();
      }
      warp_arrive(&bars[kOut]);
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_mn = idesc_bf16(128, 64, true, true);        // right operand [depth][token]
    constexpr uint32_t id_k = idesc_bf16(128, 64, true, false);        // right operand [token][depth]
    constexpr uint32_t id_kq = idesc_bf16(128, 128, false, false);
    const bool leader = lane == 0;
    const uint32_t base0 = smem_u32(smem);
    auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
    // acc (+)= A^T B over 64 of the depth; K_MAJOR: B's rows are tokens
    auto product = [&](uint32_t acc, uint64_t A, uint64_t B, bool k_major, bool first) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ss(tbase + acc, adv(A, k * 2048), adv(B, k_major ? 32 * k : 2048 * k), k_major ? id_k : id_mn,
               !first || k > 0);
    };
    int unit = 0;
    for (int j = 0; j < jobs; ++j) {
#pragma unroll 1
      for (int p = 0; p < NV; ++p, ++unit) {
        const uint32_t base = (uint32_t)afresh((int)base0), qk = base + L::kOffQk;
        const int slot = unit & 1;
        const uint32_t tile = base + L::kOffT + slot * L::kT;
        const uint64_t b_dO = smem_desc(tile, 16, 1024, kSw128), dR = smem_desc(tile + kPanel, kPanel, 1024, kSw128),
                       D = smem_desc(tile + 3 * kPanel, kPanel, 1024, kSw128);
        const uint64_t S = smem_desc(base + L::kOffS, kPanel, 1024, kSw128),
                       dS = smem_desc(base + L::kOffDS, kPanel, 1024, kSw128);
        warp_wait(&bars[kTFull + slot], (unit >> 1) & 1, abort_flag);
        tc_fence_after();
        if (leader) {                                      // the last chunk's pairs have been read (its kReady)
          product(kColP, D, b_dO, true, p == 0);
          product(kColP, adv(D, kPanel), b_dO, true, false);
          product(kColL, D, dR, false, p == 0);
          product(kColL, adv(D, kPanel), dR, false, false);
          product(kColL, D, adv(dR, kPanel), false, false);
        }
        __syncwarp();
        if (p == NV - 1) {
          warp_wait(&bars[kQkFull], j & 1, abort_flag);
          tc_fence_after();
          if (leader) {
            const uint64_t d_kq = smem_desc(qk, 16, 1024, kSw128);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
              const uint64_t d = adv(d_kq, (k / 4) * 2 * kPanel + (k % 4) * 32);
              mma_ss(tbase + kColKK, d, d, id_kq, k > 0);
            }
            mma_commit(&bars[kPairs]);
          }
          __syncwarp();
        }
        if (p == 0 && j > 0) warp_wait(&bars[kRead], (j - 1) & 1, abort_flag);
        warp_wait(&bars[kSFull], unit & 1, abort_flag);
        tc_fence_after();
        if (leader) {
          product(kColX, S, dR, false, p == 0);
          product(kColX, adv(S, NP * kPanel), dR, false, false);
          product(kColX, S, adv(dR, kPanel), false, false);
          product(kColY, S, b_dO, true, p == 0);
          product(kColY, adv(S, NP * kPanel), b_dO, true, false);
          mma_commit(&bars[kSFree]);
        }
        __syncwarp();
        warp_wait(&bars[kDSFull], unit & 1, abort_flag);
        tc_fence_after();
        if (leader) {
          product(kColZ, dS, D, false, p == 0);
          product(kColZ, adv(dS, NP * kPanel), D, false, false);
          product(kColZ, dS, adv(D, kPanel), false, false);
          mma_commit(&bars[kDSFree]);
          mma_commit(&bars[kTFree + slot]);
          if (p == NV - 1) mma_commit(&bars[kXyz]);
        }
        __syncwarp();
      }
      // dq += K^T (dP W)^T, dk += Q^T (dP W) + K^T A^T + K^T A
      warp_wait(&bars[kReady], j & 1, abort_flag);
      tc_fence_after();
      if (leader) {
        const uint32_t base = (uint32_t)afresh((int)base0), qk = base + L::kOffQk;
        const uint64_t K = smem_desc(qk, 2 * kPanel, 1024, kSw128), Q = adv(K, kPanel);
        const uint64_t pw = smem_desc(base + L::kOffA, 16, 1024, kSw128),
                       pw_mn = smem_desc(base + L::kOffA, kPanel, 1024, kSw128);
#pragma unroll
        for (int lo = 0; lo < 2; ++lo) {
          product(kColY, K, adv(pw, lo * kPanel), true, false);
          product(kColX, Q, adv(pw_mn, lo * kPanel), false, false);
          product(kColX, K, adv(pw, (2 + lo) * kPanel), true, false);
          product(kColX, K, adv(pw_mn, (2 + lo) * kPanel), false, false);
        }
        mma_commit(&bars[kDone]);
      }
      __syncwarp();
    }
    if (leader) {                                          // nothing in flight when tensor memory is given back
      mma_commit(&bars[kEnd]);
      drain(&bars[kEnd], 0);
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ loads, stores
    int unit = 0;
    bool ok = true;
    auto store = [&](int j) {                              // dq, dk of the block's j-th chunk
      ok = ok && free_to_load(&bars[kOut], j & 1, abort_flag);
      if (!ok || (a.dq_part && (a.fold == 1 || j % a.fold != a.fold - 1))) return;
      const long long job = job_of(j);
      const int bh = (int)(job / a.N), t0 = (int)(job % a.N) * kC;
      const uint8_t *src = smem + L::kOffQk;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        tma_store_3d(&tmdk, src + 2 * p * kPanel, 64 * p, t0, bh / a.fold);
        tma_store_3d(&tmdq, src + (2 * p + 1) * kPanel, 64 * p, t0, bh / a.fold);
      }
      bulk_commit_group();
      bulk_wait_read_all();
    };
    int sent_t = 0, sent_v = 0, sent_s = 0, sent_ds = 0, sent_qk = 0;
    for (int j = 0; j < jobs && ok; ++j) {
      const long long job = job_of(j);
      const int bh = (int)(job / a.N), t0 = (int)(job % a.N) * kC;
      const int kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
      for (int p = 0; p < NV; ++p, ++unit) {
        const int slot = unit & 1;
        if (unit >= 2) ok = free_to_load(&bars[kTFree + slot], ((unit >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        ++sent_t;
        uint8_t *dst = smem + L::kOffT + slot * L::kT;
        mbar_arrive_expect_tx(&bars[kTFull + slot], L::kT);
        tma_load_3d(dst, &tmdo, &bars[kTFull + slot], 64 * p, t0, bh);
#pragma unroll
        for (int lo = 0; lo < 2; ++lo) {
          const size_t at = (size_t)job * write_image(DV) + lo * (write_image(DV) / 2) + p * kPanel;
          bulk_load(dst + (1 + lo) * kPanel, a.img_dR + at, kPanel, &bars[kTFull + slot]);
          bulk_load(dst + (3 + lo) * kPanel, a.img_D + at, kPanel, &bars[kTFull + slot]);
        }
        if (unit >= 1) ok = free_to_load(&bars[kVFree], (unit - 1) & 1, abort_flag);
        if (!ok) break;
        ++sent_v;
        mbar_arrive_expect_tx(&bars[kVFull], kPanel);
        tma_load_3d(smem + L::kOffV, &tmv, &bars[kVFull], 64 * p, t0, bh);
        auto load_state = [&](const uint8_t *img, int off, uint64_t *bar) {
          mbar_arrive_expect_tx(bar, L::kS);
#pragma unroll
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int c = 0; c < NP; ++c)
              bulk_load(smem + off + (lo * NP + c) * kPanel,
                        img + (size_t)job * state_image(DK, DV) + lo * (state_image(DK, DV) / 2) +
                            (size_t)c * DV * 128 + p * kPanel,
                        kPanel, bar);
        };
        if (unit >= 1) ok = free_to_load(&bars[kSFree], (unit - 1) & 1, abort_flag);
        if (!ok) break;
        ++sent_s;
        load_state(a.img_S, L::kOffS, &bars[kSFull]);
        if (unit >= 1) ok = free_to_load(&bars[kDSFree], (unit - 1) & 1, abort_flag);
        if (!ok) break;
        ++sent_ds;
        load_state(a.img_dS, L::kOffDS, &bars[kDSFull]);
        if (p == 0) {
          if (j > 0) store(j - 1);
          if (!ok) break;
          uint64_t *bar = &bars[kQkFull];
          uint8_t *kq = smem + L::kOffQk;
          mbar_arrive_expect_tx(bar, L::kQk);
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            tma_load_3d(kq + 2 * c * kPanel, &tmk, bar, 64 * c, t0, kh);
            tma_load_3d(kq + (2 * c + 1) * kPanel, &tmq, bar, 64 * c, t0, kh);
          }
          ++sent_qk;
        }
      }
    }
    if (ok) store(jobs - 1);
    bulk_wait_all();
    // copies in flight land before the exit
    for (int u = sent_t > 2 ? sent_t - 2 : 0; u < sent_t; ++u) drain(&bars[kTFull + (u & 1)], (u >> 1) & 1);
    if (sent_v > 0) drain(&bars[kVFull], (sent_v - 1) & 1);
    if (sent_s > 0) drain(&bars[kSFull], (sent_s - 1) & 1);
    if (sent_ds > 0) drain(&bars[kDSFull], (sent_ds - 1) & 1);
    if (sent_qk > 0) drain(&bars[kQkFull], (sent_qk - 1) & 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tbase, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) flag_status(a.status, kStatusDeviceTimeout);
}

template <int DK, int DV> cudaError_t launch(const GatedDeltaLaunch &a, int d_k, int d_v, int fold) {
  CUtensorMap tq, tk, tv, tdo, tdq, tdk;
  const long long BHk = a.BH / a.H * a.Hk;
  if (!make_tma_3d_bf16_box(&tq, a.q, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tk, a.k, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tv, a.v, d_v, a.T, a.BH, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdo, a.dout, d_v, a.T, a.BH, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdq, a.dq, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdk, a.dk, d_k, a.T, BHk, 64, kC, true))
    return cudaErrorInvalidValue;
  constexpr int bytes = Layout<DK, DV>::kBytes;
  auto kern = gd_grads_tc_kernel<DK, DV>;
  GD_ALLOW_SMEM(kern, bytes);
  const Args x{a.g, a.beta, a.img_S, a.img_D, a.img_dS, a.img_dR, a.dg, a.dbeta, a.dq_part, a.dk_part,
               a.status, a.H, a.Hk, a.T, a.N, d_k, fold, a.BH * a.N / fold};
  ProfileScope prof("gd_tc_grads", a.stream);
  kern<<<(unsigned)(x.units < kGdSms ? x.units : kGdSms), kThreads, bytes, a.stream>>>(tq, tk, tv, tdo, tdq, tdk, x);
  return cudaGetLastError();
}

}  // namespace

// Where value heads share keys, a block adds up a chunk's dq and dk over them (in
// head order), as long as there are chunks enough for the blocks; otherwise the
// parts go through the workspace and a kernel of their own (8 heads of 16384 tokens,
// each shared by two: 57 us, and 90 us of writing and reading back beside it).
cudaError_t gd_tc_grads_wide(const GatedDeltaLaunch &a, int d_k, int d_v) {
  const int group = a.H / a.Hk;
  const int fold = a.dq_part && a.BH / group * a.N >= 2 * kGdSms ? group : 1;
  const cudaError_t e =
      gd_padded(d_v) == 64 ? launch<128, 64>(a, d_k, d_v, fold) : launch<128, 128>(a, d_k, d_v, fold);
  return e == cudaSuccess && a.dq_part && fold == 1 ? gd_sum_groups(a, d_k, true) : e;
}

}  // namespace kata
