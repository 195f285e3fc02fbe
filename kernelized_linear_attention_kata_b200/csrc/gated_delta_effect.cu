// What a segment of the sequence does to a state, S -> F S + B, for the gated
// delta rule's chains in segments (bf16): the chain of gated_delta_tc.cu without
// outputs, walked for two states at once, one from V and S = 0 that ends as B and
// one without V from S = I that ends as F.
//
// The two chains share K, M and the decays, and each waits most of the time (for
// its MMAs, then the MMAs for its next operand): the state warps make one
// chain's operands while the tensor core works on the other's. A chunk of both
// takes 3.4 us at d_k = 64 and 4.2 at 128, where the two alone take 5.0 and 5.5. Segment 0 starts from the
// caller's state, which makes its B the next one's starting state: it needs no F.
//
// Layout, operands and warps as in gated_delta_tc.cu; tensor memory columns of
// chain x from 256 x: S operand, M R, the update (128); K S, R operand (64); D~
// operand (64).
#include "common.cuh"
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kThreads = kLoader * 32 + 32;
constexpr uint32_t kTmemCols = 512, kChain = 256, kColKS = 128, kColD = 192;

template <int DK, int DV> struct Layout {
  static constexpr int NP = DK / 64;
  static constexpr int kK = NP * kPanel, kM = 2 * kPanel, kV = kC * DV * 2;
  static constexpr int kState = DK == 128 ? DK * DK * 4 : 0;   // F's state (see below)
  static constexpr int kOne = kK + kM + kV + kRecGates, kRoom = 232448 - 512 - 1024 - kState;
  static constexpr int NS = kRoom / kOne < 4 ? kRoom / kOne : 4;   // stages of loads
  static constexpr int kOffK = 0;
  static constexpr int kOffM = NS * kK;
  static constexpr int kOffV = kOffM + NS * kM;
  static constexpr int kOffGates = kOffV + NS * kV;
  static constexpr int kOffState = kOffGates + NS * kRecGates;
  static constexpr int kOffBars = kOffState + kState;
  static constexpr int kBytes = kOffBars + 512 + 1024;
  static_assert(NS >= 2 && kBytes <= 232448, "shared memory budget");
};
// Loaded, free; then per chain: K S, M R and the update are done.
enum { kLoaded = 0, kFree = 4, kKsDone = 8, kDDone = 10, kUDone = 12, kEnd = 14, kNumBars };
// hardware barriers, state warps to issuer, + the chain
enum { kSReady = 1, kRReady = 3, kDtReady = 5 };

struct Args {
  const float *S0;                 // nullable
  float *F, *starts;
  const uint8_t *records;
  unsigned *status;
  int H, Hk, T, N, G, seg_chunks, dk, dv;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
gd_effect_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const Args a) {
  using L = Layout<DK, DV>;
  constexpr int NP = L::NP, NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const float *gates = reinterpret_cast<const float *>(smem + L::kOffGates);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int seg = blockIdx.x % (a.G - 1), bh = blockIdx.x / (a.G - 1);
  const int kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
  const int n = a.seg_chunks;                              // these segments are full
  const int t_begin = seg * n * kC;
  const bool dual = seg > 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(&bars[i], i >= kFree && i < kFree + 4 ? kStateWarps : 1);
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
    // ------------------------------------------------------------ state warps
    const int h = warp / 4;                                // quarter of the columns
    const int r = 32 * (warp % 4) + lane;                  // value column
    const uint32_t col = tbase + ((uint32_t)(32 * (warp % 4)) << 16);
    constexpr int HK = DK / 4;
    // The states, in registers; F's of d_k = 128 in shared memory [k][column]: both
    // are 64 registers, which leaves too few for the rest (spilled, the loads went
    // to the L2, and a chunk took 10.8K cycles).
    constexpr bool kInSmem = L::kState > 0;
    float2 S[2][HK / 2];
    float *Fs = reinterpret_cast<float *>(smem + L::kOffState) + HK * h * DK + r;
    {
      const float *src = seg == 0 && a.S0 ? a.S0 + (size_t)bh * a.dk * a.dv : nullptr;
      auto given = [&](int k) { return src && r < a.dv && k < a.dk ? src[(size_t)k * a.dv + r] : 0.f; };
#pragma unroll
      for (int i = 0; i < HK / 2; ++i) {
        const int k = HK * h + 2 * i;
        S[0][i] = make_float2(given(k), given(k + 1));
        const float2 one = make_float2(k == r ? 1.f : 0.f, k + 1 == r ? 1.f : 0.f);
        if (kInSmem) {
          Fs[2 * i * DK] = one.x;
          Fs[(2 * i + 1) * DK] = one.y;
        } else {
          S[1][i] = one;
        }
      }
    }
    bool ok = true;
    auto runs = [&](int x) { return x == 0 || dual; };
    auto active = [&](int x) { return r < (x == 0 ? DV : DK); };       // the same in the whole warp
    auto state16 = [&](int x, int b, float2 (&y)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = kInSmem && x == 1 ? make_float2(Fs[(16 * b + 2 * i) * DK], Fs[(16 * b + 2 * i + 1) * DK])
                                 : S[x][8 * b + i];
    };
    auto put_state = [&](int x) {
      if (active(x)) {
#pragma unroll
        for (int b = 0; b < HK / 16; ++b) {
          float2 y[8];
          state16(x, b, y);
          put16(col + kChain * x + HK * h + 16 * b, y);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kSReady + x, ok);
    };
    ok &= warp_wait(&bars[kLoaded], 0, abort_flag);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (runs(x)) put_state(x);

    for (int c = 0; c < n; ++c) {
      const int st = c % NS;
      const float *from_start = gates + st * (kRecGates / 4), *to_end = from_start + kC, *beta = to_end + kC;
      const uint16_t *v = reinterpret_cast<const uint16_t *>(smem + L::kOffV + st * L::kV) + 16 * h * DV + r;
      auto value = [&](int i) { return __uint_as_float((uint32_t)v[i * DV] << 16); };
      // R = beta (V - e^G (K S)); beta (- e^G (K S))
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!runs(x)) continue;
        ok &= warp_wait(&bars[kKsDone + x], c & 1, abort_flag);
        tc_fence_after();
        if (active(x)) {
          const uint32_t at = col + kChain * x + kColKS + 16 * h;
          uint32_t y[16];
          float2 z[8];
          tmem_ld16(at, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = gate2(from_start, 16 * h + 2 * i), b = gate2(beta, 16 * h + 2 * i);
            const float2 v2 = x == 0 ? make_float2(value(2 * i), value(2 * i + 1)) : make_float2(0.f, 0.f);
            z[i] = __fmul2_rn(b, __ffma2_rn(make_float2(-f.x, -f.y), as_float2(y[2 * i], y[2 * i + 1]), v2));
          }
          put16(at, z);
          tmem_wait_st();
        }
        tc_fence_before();
        hand_over(kRReady + x, ok);
      }
      // D~ = e^{G_C - G} D, from its two accumulators
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!runs(x)) continue;
        ok &= warp_wait(&bars[kDDone + x], c & 1, abort_flag);
        tc_fence_after();
        if (active(x)) {
          uint32_t y[16], w[16];
          float2 z[8];
          tmem_ld16(col + kChain * x + 16 * h, y);
          tmem_ld16(col + kChain * x + 64 + 16 * h, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = gate2(to_end, 16 * h + 2 * i);
            z[i] = __fmul2_rn(f, __fadd2_rn(as_float2(y[2 * i], y[2 * i + 1]), as_float2(w[2 * i], w[2 * i + 1])));
          }
          put16(col + kChain * x + kColD + 16 * h, z);
          tmem_wait_st();
        }
        tc_fence_before();
        hand_over(kDtReady + x, ok);
      }
      // S' = e^{G_C} S + K^T D~, and the next chunk's operand
      const float whole = from_start[kC - 1];
      const float2 w2 = make_float2(whole, whole);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (runs(x)) {
          ok &= warp_wait(&bars[kUDone + x], c & 1, abort_flag);
          tc_fence_after();
          if (active(x)) {
#pragma unroll
            for (int b = 0; b < HK / 16; ++b) {
              uint32_t y[16];
              tmem_ld16(col + kChain * x + HK * h + 16 * b, y);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int k = 16 * b + 2 * i;
                if (kInSmem && x == 1) {
                  Fs[k * DK] = fmaf(whole, Fs[k * DK], __uint_as_float(y[2 * i]));
                  Fs[(k + 1) * DK] = fmaf(whole, Fs[(k + 1) * DK], __uint_as_float(y[2 * i + 1]));
                } else {
                  S[x][8 * b + i] = __ffma2_rn(w2, S[x][8 * b + i], as_float2(y[2 * i], y[2 * i + 1]));
                }
              }
            }
          }
        }
        if (x == 0 && c + 1 < n) ok &= warp_wait(&bars[kLoaded + (c + 1) % NS], ((c + 1) / NS) & 1, abort_flag);
        if (x == 1) warp_arrive(&bars[kFree + st]);
        if (runs(x) && c + 1 < n) put_state(x);
      }
    }
    if (ok) {
      float *B = a.starts + ((size_t)bh * a.G + seg + 1) * DK * DV;
      float *F = a.F + ((size_t)bh * (a.G - 2) + seg - 1) * DK * DK;
#pragma unroll
      for (int i = 0; i < HK / 2; ++i) {
        const size_t k = HK * h + 2 * i;
        if (active(0)) {
          B[k * DV + r] = S[0][i].x;
          B[(k + 1) * DV + r] = S[0][i].y;
        }
        if (dual && active(1)) {
          F[k * DK + r] = kInSmem ? Fs[2 * i * DK] : S[1][i].x;
          F[(k + 1) * DK + r] = kInSmem ? Fs[(2 * i + 1) * DK] : S[1][i].y;
        }
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_64 = idesc_bf16(128, 64, false, false);      // K-major right operand
    constexpr uint32_t id_128 = idesc_bf16(128, 128, false, false);
    constexpr uint32_t id_up = idesc_bf16(128, DK, false, true);       // MN-major
    const bool leader = lane == 0;
    const uint32_t base = smem_u32(smem);
    auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
    for (int c = 0; c < n; ++c) {
      const int st = c % NS;
      const uint64_t d_k = smem_desc(base + L::kOffK + st * L::kK, 16, 1024, kSw128);
      const uint64_t d_k_mn = smem_desc(base + L::kOffK + st * L::kK, kPanel, 1024, kSw128);
      const uint64_t d_m = smem_desc(base + L::kOffM + st * L::kM, 16, 1024, kSw128);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && !dual) continue;
        const uint32_t t = tbase + kChain * x;
        take_over(kSReady + x);
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
              mma_ts(t + kColKS, t + 16 * k + 8 * lo, adv(d_k, (k / 4) * kPanel + (k % 4) * 32), id_64, lo > 0 || k > 0);
          mma_commit(&bars[kKsDone + x]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && !dual) continue;
        const uint32_t t = tbase + kChain * x;
        take_over(kRReady + x);
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(t, t + kColKS + 16 * k + 8 * lo, adv(d_m, 32 * k), lo ? id_64 : id_128, lo > 0 || k > 0);
          mma_commit(&bars[kDDone + x]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && !dual) continue;
        const uint32_t t = tbase + kChain * x;
        take_over(kDtReady + x);
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int lo = 0; lo < 2; ++lo)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(t, t + kColD + 16 * k + 8 * lo, adv(d_k_mn, k * 2048), id_up, lo > 0 || k > 0);
          mma_commit(&bars[kUDone + x]);
        }
      }
    }
    if (leader) {                                          // nothing in flight when tensor memory is given back
      mma_commit(&bars[kEnd]);
      drain(&bars[kEnd], 0);
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------ loads
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
    const uint8_t *rec = a.records + ((size_t)bh * a.N + (size_t)seg * n) * kRecBytes;
    int sent = 0;
    for (; sent < n; ++sent) {
      const int st = sent % NS, row = t_begin + kC * sent;
      if (sent >= NS && !free_to_load(&bars[kFree + st], (sent / NS - 1) & 1, abort_flag)) break;
      uint64_t *bar = &bars[kLoaded + st];
      mbar_arrive_expect_tx(bar, L::kOne);
#pragma unroll
      for (int p = 0; p < NP; ++p) tma_load_3d(smem + L::kOffK + st * L::kK + p * kPanel, &tmk, bar, 64 * p, row, kh);
      bulk_load(smem + L::kOffGates + st * kRecGates, rec + (size_t)sent * kRecBytes, kRecGates, bar);
      bulk_load(smem + L::kOffM + st * L::kM, rec + (size_t)sent * kRecBytes + kRecM, L::kM, bar);
      tma_load_3d(smem + L::kOffV + st * L::kV, &tmv, bar, 0, row, bh);
    }
    // copies in flight land before the exit
    for (int c = sent > NS ? sent - NS : 0; c < sent; ++c) drain(&bars[kLoaded + c % NS], (c / NS) & 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tbase, kTmemCols);
  if (threadIdx.x == 0 && *abort_flag) flag_status(a.status, kStatusDeviceTimeout);
}

template <int DK, int DV>
cudaError_t launch(const GatedDeltaLaunch &a, int d_k, int d_v) {
  CUtensorMap mk, mv;
  if (!make_tma_3d_bf16_box(&mk, a.k, d_k, a.T, a.BH / a.H * a.Hk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&mv, a.v, d_v, a.T, a.BH, DV, kC, false))
    return cudaErrorInvalidValue;
  const Args x{a.S0, a.F, a.starts_seg, a.records, a.status, a.H, a.Hk, a.T, a.N, a.G, a.seg_chunks, d_k, d_v};
  constexpr int bytes = Layout<DK, DV>::kBytes;
  auto kern = gd_effect_kernel<DK, DV>;
  GD_ALLOW_SMEM(kern, bytes);
  ProfileScope prof("gd_tc_segment", a.stream);
  kern<<<(unsigned)(a.BH * (a.G - 1)), kThreads, bytes, a.stream>>>(mk, mv, x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t gd_tc_effect(const GatedDeltaLaunch &a, int d_k, int d_v) {
  if (a.G == 1) return cudaSuccess;
#define GD_RUN(DK, DV) launch<DK, DV>(a, d_k, d_v)
  return GD_TC_DISPATCH(GD_RUN);
#undef GD_RUN
}

}  // namespace kata
