// The chunk-local part of the gated delta rule, all chunks at once (bf16): M =
// (I + L)^-1 and P of each 64-token chunk as MMA operands, with its decays, into
// the workspace (the record of gated_delta_tc.cuh).
//
// One block of four warps a chunk: [K; Q] K^T by tcgen05 (K rows on TMEM lanes
// 0-63, Q rows on 64-127), thread = row; the K rows become L and are inverted
// by blocks, the Q rows become P. Six blocks share an SM and hide one
// another's latencies. Loops are kept rolled: straight code beyond 32 KB runs
// from the second instruction cache at 2.4 cycles an instruction (measured),
// and the same work unrolled to 40 KB took twice as long. Inside the chains'
// kernel, one chunk ahead, it took 10K cycles a chunk to the chain's 5K, both
// codes waiting on instructions.
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "common.cuh"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kSolveThreads = 128;

template <int DK> struct SolveLayout {
  static constexpr int NP = DK / 64;
  static constexpr int kKq = 2 * NP * kPanel;
  // K and Q, then in their place P's tiles and L, then M's tiles in L's
  static constexpr int kOffP = 0, kOffL = 2 * kPanel;
  static constexpr int kLBytes = kC * kLs * 4;
  static constexpr int kWork = kOffL + kLBytes > kKq ? kOffL + kLBytes : kKq;
  static constexpr int kOffGates = (kWork + 127) / 128 * 128;
  static constexpr int kOffBars = kOffGates + (int)sizeof(Gates);
  static constexpr int kBytes = kOffBars + 64 + 1024;
};

template <int DK>
__global__ void __launch_bounds__(kSolveThreads, 6)
gd_solve_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const float *__restrict__ g, const float *__restrict__ beta,
                   uint8_t *__restrict__ records, unsigned *__restrict__ status, int H, int Hk, int T,
                   int N) {
  using L = SolveLayout<DK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);     // loads, products
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Gates &gt = *reinterpret_cast<Gates *>(smem + L::kOffGates);
  float *Lm = reinterpret_cast<float *>(smem + L::kOffL);
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bh = blockIdx.x / N, t0 = (int)(blockIdx.x % N) * kC;
  const int kh = bh / H * Hk + bh % H / (H / Hk);

  if (threadIdx.x == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    *abort_flag = 0;
    mbar_init_fence();
    mbar_arrive_expect_tx(&bars[0], L::kKq);
#pragma unroll
    for (int p = 0; p < L::NP; ++p) {
      tma_load_3d(smem + 2 * p * kPanel, &tmk, &bars[0], 64 * p, t0, kh);
      tma_load_3d(smem + (2 * p + 1) * kPanel, &tmq, &bars[0], 64 * p, t0, kh);
    }
  }
  if (w == 2) {
    tmem_alloc(tmem_slot, 64);
    tmem_relinquish();
  }
  if (w == 3) {
    const float *gp = g + (size_t)bh * T + t0, *bp = beta + (size_t)bh * T + t0;
    const int u = 2 * lane, left = T - t0;
    make_gates(gt, u < left ? gp[u] : 0.f, u + 1 < left ? gp[u + 1] : 0.f, u < left ? bp[u] : 0.f,
               u + 1 < left ? bp[u + 1] : 0.f);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  if (threadIdx.x == 0) {
    if (mbar_wait(&bars[0], 0, abort_flag)) {
      constexpr uint32_t id = idesc_bf16(128, kC, false, false);
      const uint32_t kq = smem_u32(smem);
      tc_fence_after();
#pragma unroll 1
      for (int k = 0; k < DK / 16; ++k) {
        const uint64_t desc = smem_desc(kq + (k / 4) * 2 * kPanel + (k % 4) * 32, 16, 1024, kSw128);
        mma_ss(tbase, desc, desc, id, k > 0);
      }
    } else {
      drain(&bars[0], 0);
    }
    mma_commit(&bars[1]);
  }
  __syncwarp();
  const bool ok = warp_wait(&bars[1], 0, abort_flag);
  tc_fence_after();
  {
    const int diag = w & 1, t = 32 * diag + lane;          // token of the row
    const uint32_t row = tbase + ((uint32_t)(32 * w) << 16);
    uint8_t *tile = smem + L::kOffP;                       // P hi, lo
    const RowDecay d = row_decay(gt, t, w < 2);
    const float b_t = gt.beta[t];
    const int seen = 4 + 4 * diag;                         // blocks of 8 tokens not behind the warp's rows
#pragma unroll 1
    for (int b = 0; b < (w < 2 ? seen : 8); ++b) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (b < seen) {
        uint32_t x[8];
        tmem_ld8(row + 8 * b, x);
        tmem_wait_ld();
        decay8(gt, d, b, x, y);
      }
      if (w >= 2) {
        store_split8(tile, tile + kPanel, t, b, y);
      } else if (b / 4 == diag) {
#pragma unroll
        for (int j = 0; j < 8; ++j)                        // transposed, for the inversion
          Lm[(8 * b + j) * kLs + t] = b_t * y[j];
      } else {
        float *dst = Lm + t * kLs + 8 * b;
        *reinterpret_cast<float4 *>(dst) = make_float4(b_t * y[0], b_t * y[1], b_t * y[2], b_t * y[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(b_t * y[4], b_t * y[5], b_t * y[6], b_t * y[7]);
      }
    }
    __syncwarp();
    if (w < 2) invert_diagonal(Lm + 32 * w * (kLs + 1));
  }
  __syncthreads();
  invert_corner(Lm);
  store_inverse(Lm, smem + L::kOffL, smem + L::kOffL + kPanel);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 2) tmem_dealloc(tbase, 64);
  if (threadIdx.x == 0) {
    uint8_t *rec = records + (size_t)blockIdx.x * kRecBytes;
    bulk_store(rec, gt.from_start, kRecGates);             // from_start, to_end, beta
    bulk_store(rec + kRecP, smem + L::kOffP, 2 * kPanel);
    bulk_store(rec + kRecM, smem + L::kOffL, 2 * kPanel);
    bulk_commit_group();
    if (!ok) flag_status(status, kStatusDeviceTimeout);
    bulk_wait_read_all();
  }
}

template <int DK> cudaError_t launch(const GatedDeltaLaunch &a, int d_k) {
  using L = SolveLayout<DK>;
  CUtensorMap tq, tk;
  const long long BHk = a.BH / a.H * a.Hk;
  if (!make_tma_3d_bf16_box(&tq, a.q, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tk, a.k, d_k, a.T, BHk, 64, kC, true))
    return cudaErrorInvalidValue;
  auto kern = gd_solve_tc_kernel<DK>;
  GD_ALLOW_SMEM(kern, L::kBytes);
  ProfileScope prof("gd_tc_solve", a.stream);
  kern<<<(unsigned)(a.BH * a.N), kSolveThreads, L::kBytes, a.stream>>>(tq, tk, a.g, a.beta, a.records,
                                                                       a.status, a.H, a.Hk, a.T, a.N);
  return cudaGetLastError();
}

}  // namespace

size_t gd_tc_record_bytes() { return kRecBytes; }

cudaError_t gd_tc_solve(const GatedDeltaLaunch &a, int d_k) {
  return gd_padded(d_k) == 64 ? launch<64>(a, d_k) : launch<128>(a, d_k);
}

}  // namespace kata
