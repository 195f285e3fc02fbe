// The gradient of the gated delta rule on the tensor cores (bf16; head sizes below
// 64 or 128 are padded with zeros as in the forward): the reverse chain, then the gradients of all chunks at once.
//
// The forward chain has saved each chunk's starting state S and writes D. With
// dS' the gradient of a chunk's last state, last chunk first:
//   dD = P^T dO + e^{G_C - G} (K dS'),  dR = M^T dD,  dV = beta dR,
//   dS = e^{G_C} dS' + Q^T (e^G dO) - K^T (e^G dV).
// As in the forward chain everything with a value axis is transposed (thread =
// value column = TMEM lane), the state's gradient stays in registers, and
// fp32 operands enter as two bf16 halves:
//   K dS'      A = dS'^T (TMEM)          B = K tile, K-major
//   P^T dO     A = dO tile, MN-major     B = [P hi; P lo] tiles, MN-major
//   M^T dD     A = dD^T (TMEM)           B = [M hi; M lo], MN-major
//   Q^T (..)   A = (e^G dO)^T (TMEM)     B = Q tile, MN-major
//   K^T (..)   A = -(e^G dV)^T (TMEM)    B = K tile, MN-major
// P^T dO of the next chunk and Q^T (e^G dO) run in the gaps of the chain. dS'
// and dR are saved as bf16 halves for the second kernel. Where the sequence is
// cut into segments, a segment passes F^T dS' + B' on: F is the forward's, B' what
// the same chain leaves from dO and dS' = 0.
#include "common.cuh"
#include "gated_delta_sync.h"
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kThreads = kChainThreads + 32;            // warp 19 stores dV
constexpr uint32_t kTmemCols = 512;
// Columns: dS' operand and update accumulator; K dS', then dD; P^T dO in two
// accumulators; M^T dD in two, the first then -(e^G dV); e^G dO.
constexpr uint32_t kColS = 0, kColU = 128, kColX = 192, kColD = 320, kColG = 448;

template <int DK, int DV> struct Layout {
  static constexpr int NP = DK / 64, NV = DV / 64;
  static constexpr int kKq = 2 * NP * kPanel;              // [K p0][Q p0][K p1][Q p1]
  static constexpr int kTiles = 4 * kPanel;                // M hi, lo, P hi, lo
  static constexpr int kDo = NV * kPanel;                  // dO panels, then dV in their place
  static constexpr int kStateHalf = (int)state_image(DK, DV) / 2, kWrites = (int)write_image(DV);
  static constexpr int kSaves = kStateHalf > kWrites ? kStateHalf : kWrites;
  static constexpr int kOne = kKq + kTiles + kDo + kRecGates, kRoom = 232448 - 512 - 1024 - kSaves;
  static constexpr int NS = kRoom / kOne < 4 ? kRoom / kOne : 4;   // stages, as in the forward
  static constexpr int kOffKq = 0;
  static constexpr int kOffTiles = NS * kKq;
  static constexpr int kOffDo = kOffTiles + NS * kTiles;
  static constexpr int kOffStage = kOffDo + NS * kDo;
  static constexpr int kOffGates = kOffStage + kSaves;
  static constexpr int kOffBars = kOffGates + NS * kRecGates;
  static constexpr int kBytes = kOffBars + 512 + 1024;
  // with d_v = 64 the dO operand's lanes 64-127 (not used) read the 8 KB behind it
  static_assert(kOffDo + NS * kDo + kPanel <= kOffBars + 512, "operand rows stay in shared memory");
  static_assert(kBytes <= 232448, "shared memory budget");
};
// dV is ready: a barrier per stage, since the value warps may be as many chunks
// ahead of the storing warp as there are stages (gated_delta_sync.h).
enum {
  kLoaded = 0, kFree = 4, kStored = 8, kDvReady = 12, kXDone = 16, kUDone, kRDone, kSDone, kStaged, kSaved, kEnd,
  kNumBars
};
// hardware barriers, value warps to issuer (0 is the block's)
enum { kSReady = 1, kDReady, kZReady };
static_assert(8 * kNumBars + 8 <= 512, "barrier area");

struct Args {
  const float *dS;                 // nullable: the last state's gradient
  float *dS0;                      // nullable
  const uint8_t *records;
  uint8_t *img_dS, *img_dR;
  float *ends;                     // segments' [BH][G][DK][DV], 0 .. G - 2 used
  unsigned *status;
  int H, Hk, T, N, G, seg_chunks;
  int dk, dv;                      // the tensors' head sizes, <= DK, DV
};

// EFFECT: what segments 1 .. G - 1 add to the gradient they pass on, from dO and dS' =
// 0 (the last: from dS, which makes it the gradient itself), into `ends` of the
// segment before. Otherwise all segments, from `ends`.
template <int DK, int DV, bool EFFECT>
__global__ void __launch_bounds__(kThreads, 1)
gd_reverse_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmdo, const __grid_constant__ CUtensorMap tmdv,
                  const Args a) {
  using L = Layout<DK, DV>;
  constexpr int NP = L::NP, NV = L::NV, NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const float *gates = reinterpret_cast<const float *>(smem + L::kOffGates);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int segs = EFFECT ? a.G - 1 : a.G;
  const int bh = blockIdx.x / segs, seg = blockIdx.x % segs + (EFFECT ? 1 : 0);
  const int kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
  const int first = seg * a.seg_chunks;                    // chunks first .. first + n - 1
  const int n = a.N - first < a.seg_chunks ? a.N - first : a.seg_chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if ((i >= kFree && i < kFree + 4) || (i >= kDvReady && i < kDvReady + 4) || i == kStaged) count = kStateWarps;
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
    // ------------------------------------------------------------ value columns
    const int h = warp / 4;
    const int r = 32 * (warp % 4) + lane;
    const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
    const bool active = r < DV;
    constexpr int HK = DK / 4;
    float2 S[HK / 2];                                      // dS'
    {
      const bool given = seg == a.G - 1;                   // by the caller, in its own head sizes
      const int rows = given ? a.dk : DK, ld = given ? a.dv : DV;
      const float *src = nullptr;
      if (given)
        src = a.dS ? a.dS + (size_t)bh * rows * ld : nullptr;
      else if (!EFFECT)
        src = a.ends + ((size_t)bh * a.G + seg) * DK * DV;
      auto entry = [&](int k) { return src && r < ld && k < rows ? src[(size_t)k * ld + r] : 0.f; };
#pragma unroll
      for (int i = 0; i < HK / 2; ++i) S[i] = make_float2(entry(HK * h + 2 * i), entry(HK * h + 2 * i + 1));
    }
    const uint32_t col_s = tbase + lane_off + kColS + HK * h;
    const uint32_t col_part = tbase + lane_off + 16 * h;
    uint8_t *stage = smem + L::kOffStage;
    auto stage_free = [&](int use) -> bool {
      return use == 0 || warp_wait(&bars[kSaved], (use - 1) & 1, abort_flag);
    };
    auto staged = [&]() {
      fence_async_smem();
      warp_arrive(&bars[kStaged]);
    };
    bool ok = true;

    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      ok &= warp_wait(&bars[kLoaded + st], (i / NS) & 1, abort_flag);
      if (active) {
#pragma unroll
        for (int b = 0; b < HK / 16; ++b) put16(col_s + 16 * b, S + 8 * b);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kSReady, ok);
      if (!EFFECT) {
        ok &= stage_free(3 * i);
        if (active) stage_row<HK / 8>(stage, DV, r, HK * h, S, false);
        staged();
      }

      // e^G dO; its place in shared memory later takes dV
      const float *from_start = gates + st * (kRecGates / 4), *to_end = from_start + kC, *beta = to_end + kC;
      uint8_t *col = smem + L::kOffDo + st * L::kDo + (r / 64) * kPanel + (r % 8) * 2;
      const int chunk = r % 64 / 8;
      auto at = [&](int t) { return reinterpret_cast<uint16_t *>(col + sw128(t, chunk)); };
      if (active) {
        float2 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = 16 * h + 2 * j;
          y[j] = __fmul2_rn(gate2(from_start, t), as_float2((uint32_t)*at(t) << 16, (uint32_t)*at(t + 1) << 16));
        }
        put16(col_part + kColG, y);
      }

      // dD = P^T dO + e^{G_C - G} (K dS')
      ok &= warp_wait(&bars[kXDone], i & 1, abort_flag);
      ok &= warp_wait(&bars[kUDone], i & 1, abort_flag);
      tc_fence_after();
      if (active) {
        uint32_t x[16], y[16];
        float2 z[8];
        tmem_ld16(col_part + kColX, x);
        tmem_ld16(col_part + kColX + 64, y);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          z[j] = __fadd2_rn(as_float2(x[2 * j], x[2 * j + 1]), as_float2(y[2 * j], y[2 * j + 1]));
        tmem_ld16(col_part + kColU, x);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          z[j] = __ffma2_rn(gate2(to_end, 16 * h + 2 * j), as_float2(x[2 * j], x[2 * j + 1]), z[j]);
        put16(col_part + kColU, z);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kDReady, ok);
      if (!EFFECT) {
        ok &= stage_free(3 * i + 1);
        if (active) stage_row<HK / 8>(stage, DV, r, HK * h, S, true);
        staged();
      }

      // dR = M^T dD, dV = beta dR
      ok &= warp_wait(&bars[kRDone], i & 1, abort_flag);
      tc_fence_after();
      float2 d[8];
      if (active) {
        uint32_t x[16], y[16];
        float2 z[8];
        tmem_ld16(col_part + kColD, x);
        tmem_ld16(col_part + kColD + 64, y);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = gate2(from_start, 16 * h + 2 * j), b = gate2(beta, 16 * h + 2 * j);
          d[j] = __fadd2_rn(as_float2(x[2 * j], x[2 * j + 1]), as_float2(y[2 * j], y[2 * j + 1]));
          z[j] = __fmul2_rn(make_float2(-f.x * b.x, -f.y * b.y), d[j]);
        }
        put16(col_part + kColD, z);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kZReady, ok);
      const float whole = from_start[kC - 1];
      if (!EFFECT) {
        ok &= stage_free(3 * i + 2);
        if (active) {
          stage_row<2>(stage, DV, r, 16 * h, d, false);
          stage_row<2>(stage + (size_t)DV * 128, DV, r, 16 * h, d, true);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int t = 16 * h + 2 * j;
            *reinterpret_cast<__nv_bfloat16 *>(at(t)) = __float2bfloat16_rn(beta[t] * d[j].x);
            *reinterpret_cast<__nv_bfloat16 *>(at(t + 1)) = __float2bfloat16_rn(beta[t + 1] * d[j].y);
          }
        }
        staged();                                          // fences dV's writes too
        warp_arrive(&bars[kDvReady + gdsync::dv_ready(i, NS).place]);
      }

      // dS = e^{G_C} dS' + Q^T (e^G dO) - K^T (e^G dV)
      ok &= warp_wait(&bars[kSDone], i & 1, abort_flag);
      tc_fence_after();
      if (active) {
        const float2 w2 = make_float2(whole, whole);
#pragma unroll
        for (int b = 0; b < HK / 16; ++b) {
          uint32_t x[16];
          tmem_ld16(col_s + 16 * b, x);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            S[8 * b + j] = __ffma2_rn(w2, S[8 * b + j], as_float2(x[2 * j], x[2 * j + 1]));
        }
      }
      warp_arrive(&bars[kFree + st]);
    }
    float *dst = nullptr;
    const int rows = EFFECT ? DK : a.dk, ld = EFFECT ? DV : a.dv;
    if (EFFECT)
      dst = a.ends + ((size_t)bh * a.G + seg - 1) * DK * DV;
    else if (seg == 0 && a.dS0)
      dst = a.dS0 + (size_t)bh * rows * ld;
    if (r < ld && ok && dst) {
#pragma unroll
      for (int i = 0; i < HK / 2; ++i)
        if (HK * h + 2 * i < rows) {                       // even
          dst[(size_t)(HK * h + 2 * i) * ld + r] = S[i].x;
          dst[(size_t)(HK * h + 2 * i + 1) * ld + r] = S[i].y;
        }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_u = idesc_bf16(128, 64, false, false);       // K-major right operand
    constexpr uint32_t id_x = idesc_bf16(128, 128, true, true);        // both MN-major
    constexpr uint32_t id_r128 = idesc_bf16(128, 128, false, true), id_r64 = idesc_bf16(128, 64, false, true);
    constexpr uint32_t id_up = idesc_bf16(128, DK, false, true);
    const bool leader = lane == 0;
    const uint32_t base = smem_u32(smem);
    auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
    // P^T dO of round i, in two accumulators
    auto issue_x = [&](int i) {
      const int st = i % NS;
      warp_wait(&bars[kLoaded + st], (i / NS) & 1, abort_flag);
      tc_fence_after();
      if (leader) {
        const uint64_t d_do = smem_desc(base + L::kOffDo + st * L::kDo, kPanel, 1024, kSw128);
        const uint64_t d_p = smem_desc(base + L::kOffTiles + st * L::kTiles + 2 * kPanel, kPanel, 1024, kSw128);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tbase + kColX, adv(d_do, k * 2048), adv(d_p, k * 2048), id_x, k > 0);
        mma_commit(&bars[kXDone]);
      }
      __syncwarp();
    };
    issue_x(0);
    for (int i = 0; i < n; ++i) {
      const int st = i % NS;
      const uint64_t d_k = smem_desc(base + L::kOffKq + st * L::kKq, 16, 1024, kSw128);
      const uint64_t d_k_mn = smem_desc(base + L::kOffKq + st * L::kKq, 2 * kPanel, 1024, kSw128);
      const uint64_t d_q_mn = adv(d_k_mn, kPanel);
      const uint64_t d_m = smem_desc(base + L::kOffTiles + st * L::kTiles, kPanel, 1024, kSw128);
      take_over(kSReady);
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
            mma_ts(tbase + kColU, tbase + kColS + 16 * k + 8 * lo, adv(d_k, (k / 4) * 2 * kPanel + (k % 4) * 32),
                   id_u, lo > 0 || k > 0);
        mma_commit(&bars[kUDone]);
      }
      take_over(kDReady);
      tc_fence_after();
      if (leader) {
        // dD hi against [M hi; M lo] in two accumulators, dD lo against M hi
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tbase + kColD, tbase + kColU + 16 * k + 8 * lo, adv(d_m, k * 2048), lo ? id_r64 : id_r128,
                   lo > 0 || k > 0);
        mma_commit(&bars[kRDone]);
        // dS' has been read (its products are done, or dD would not be ready)
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tbase + kColS, tbase + kColG + 16 * k + 8 * lo, adv(d_q_mn, k * 2048), id_up, lo > 0 || k > 0);
      }
      take_over(kZReady);
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tbase + kColS, tbase + kColD + 16 * k + 8 * lo, adv(d_k_mn, k * 2048), id_up, 1);
        mma_commit(&bars[kSDone]);
      }
      __syncwarp();
      if (i + 1 < n) issue_x(i + 1);                  // in the gap before the next K dS'
    }
    if (leader) {                                          // nothing in flight when tensor memory is given back
      mma_commit(&bars[kEnd]);
      drain(&bars[kEnd], 0);
    }
  } else if (warp == kLoader) {
    if (lane == 0) {
      // ---------------------------------------------------------- loads, last chunk first
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmq);
      tma_prefetch_desc(&tmdo);
      int sent = 0;
      for (int i = 0; i < n; ++i) {
        const int st = i % NS, c = first + n - 1 - i, row = kC * c;
        if (i >= NS && (!free_to_load(&bars[kFree + st], (i / NS - 1) & 1, abort_flag) ||
                        (!EFFECT && !free_to_load(&bars[kStored + st], (i / NS - 1) & 1, abort_flag))))
          break;
        uint8_t *kq = smem + L::kOffKq + st * L::kKq, *dO = smem + L::kOffDo + st * L::kDo;
        const uint8_t *rec = a.records + ((size_t)bh * a.N + c) * kRecBytes;
        mbar_arrive_expect_tx(&bars[kLoaded + st], L::kKq + kRecGates + L::kTiles + L::kDo);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          tma_load_3d(kq + 2 * p * kPanel, &tmk, &bars[kLoaded + st], 64 * p, row, kh);
          tma_load_3d(kq + (2 * p + 1) * kPanel, &tmq, &bars[kLoaded + st], 64 * p, row, kh);
        }
#pragma unroll
        for (int p = 0; p < NV; ++p) tma_load_3d(dO + p * kPanel, &tmdo, &bars[kLoaded + st], 64 * p, row, bh);
        bulk_load(smem + L::kOffGates + st * kRecGates, rec, kRecGates, &bars[kLoaded + st]);
        bulk_load(smem + L::kOffTiles + st * L::kTiles, rec + kRecM, L::kTiles, &bars[kLoaded + st]);
        sent = i + 1;
      }
      // copies in flight land before the exit
      for (int i = sent > NS ? sent - NS : 0; i < sent; ++i) drain(&bars[kLoaded + i % NS], (i / NS) & 1);
    }
  } else if (!EFFECT && warp == kSaver) {
    if (lane == 0) {
      // ---------------------------------------------------------- saves: dS' hi, lo, dR
      for (int use = 0; use < 3 * n; ++use) {
        if (!mbar_wait(&bars[kStaged], use & 1, abort_flag)) break;
        const int part = use % 3;
        const size_t at = (size_t)bh * a.N + (first + n - 1 - use / 3);
        if (part < 2)
          bulk_store(a.img_dS + at * state_image(DK, DV) + part * L::kStateHalf, smem + L::kOffStage, L::kStateHalf);
        else
          bulk_store(a.img_dR + at * write_image(DV), smem + L::kOffStage, L::kWrites);
        bulk_commit_group();
        bulk_wait_read_all();
        mbar_arrive(&bars[kSaved]);
      }
      bulk_wait_all();
    }
  } else if (!EFFECT) {
    if (lane == 0) {
      // ---------------------------------------------------------- dV's stores
      tma_prefetch_desc(&tmdv);
      for (int i = 0; i < n; ++i) {
        const gdsync::Turn ready = gdsync::dv_ready(i, NS);
        if (!mbar_wait(&bars[kDvReady + ready.place], ready.parity, abort_flag)) break;
#pragma unroll
        for (int p = 0; p < NV; ++p)
          tma_store_3d(&tmdv, smem + L::kOffDo + i % NS * L::kDo + p * kPanel, 64 * p, kC * (first + n - 1 - i), bh);
        bulk_commit_group();
        bulk_wait_read_all();
        mbar_arrive(&bars[kStored + i % NS]);
      }
      bulk_wait_all();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tbase, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) flag_status(a.status, kStatusDeviceTimeout);
}

template <int DK, int DV, bool EFFECT> cudaError_t launch(const GatedDeltaLaunch &a, int d_k, int d_v) {
  CUtensorMap tq, tk, tdo, tdv;
  const long long BHk = a.BH / a.H * a.Hk;
  if (!make_tma_3d_bf16_box(&tq, a.q, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tk, a.k, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdo, a.dout, d_v, a.T, a.BH, 64, kC, true) ||
      !make_tma_3d_bf16_box(&tdv, a.dv, d_v, a.T, a.BH, 64, kC, true))
    return cudaErrorInvalidValue;
  constexpr int bytes = Layout<DK, DV>::kBytes;
  auto kern = gd_reverse_kernel<DK, DV, EFFECT>;
  GD_ALLOW_SMEM(kern, bytes);
  const Args x{a.dS, a.dS0, a.records, a.img_dS, a.img_dR, a.ends_seg, a.status, a.H, a.Hk, a.T, a.N, a.G,
               a.seg_chunks, d_k, d_v};
  ProfileScope prof(EFFECT ? "gd_tc_reverse_segment" : "gd_tc_reverse", a.stream);
  kern<<<(unsigned)(a.BH * (EFFECT ? a.G - 1 : a.G)), kThreads, bytes, a.stream>>>(tq, tk, tdo, tdv, x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_tc_reverse_effect(const GatedDeltaLaunch &a, int d_k, int d_v) {
  if (a.G == 1) return cudaSuccess;
#define GD_RUN(DK, DV) launch<DK, DV, true>(a, d_k, d_v)
  return GD_TC_DISPATCH(GD_RUN);
#undef GD_RUN
}
cudaError_t gd_tc_reverse(const GatedDeltaLaunch &a, int d_k, int d_v) {
#define GD_RUN(DK, DV) launch<DK, DV, false>(a, d_k, d_v)
  return GD_TC_DISPATCH(GD_RUN);
#undef GD_RUN
}

}  // namespace kata
