// The gated delta rule's chunked forward on the tensor cores (tcgen05 / TMEM /
// TMA): bf16, chunks of C = 64 tokens. Head sizes DK, DV in {64, 128}: smaller
// ones are padded by the tile loads' zero fill, and the stores leave the rest out.
//
// Per chunk, from its starting state S [d_k, d_v] (fp32), with G the running
// sum of g, W_ts = e^{G_t - G_s} (s <= t), M = (I + L)^-1, L_ts = beta_t W_ts
// k_t.k_s (s < t) and P_ts = W_ts q_t.k_s (s <= t):
//   R = beta (V - e^G (K S)),  D = M R,
//   O = e^G (Q S) + P D,  S' = e^{G_C} S + K^T (e^{G_C - G} D).
//
// Everything with a value axis is held transposed: thread r of a warpgroup
// owns value column r (one TMEM lane), and the axis of the keys or tokens
// runs along TMEM columns. Then every left operand (S^T, R^T, D^T) is written
// to tensor memory by the threads that computed it, every right operand (K,
// Q, M, P) is a shared-memory tile, and the state itself stays in registers
// from the first chunk to the last:
//   [K; Q] S      A = S^T (TMEM)           B = K, Q tiles, K-major
//   M R           A = R^T (TMEM)           B = M tile
//   K^T D~        A = (e^{G_C-G} D)^T      B = K tile, MN-major
//   P D           A = D^T                  B = P tile
// fp32 operands enter as two bf16 halves (hi + lo, 16 bits); q, k and v are
// bf16 and exact. S rounded to one bf16 per product would put 2^-9 of it into
// every later state.
//
// What bounds it: the chain S -> K S -> R -> D -> S' of one chunk, three MMA
// rounds and three passes of the value threads over the columns. What does not
// depend on S is kept off it: M, P and the decays come ready from the solve
// (gated_delta_solve.cu), and a chunk's P D runs while the state warps make S'
// and its operand, its outputs leave during the next one's K S (d_k = 64: M R).
// With fewer heads than SMs the sequence is cut into G segments: each but the
// last is first walked for its effect on a state, S_end = F S_start + B
// (gated_delta_effect.cu), a small kernel joins them, and the segments then run
// side by side. For the gradient the same kernel without outputs saves every
// chunk's S and D (gated_delta_bwd_tc.cu).
//
// An MMA takes 70-85 cycles here whatever its N (from one issuing thread or from
// two), so N is 128 wherever two tiles lie side by side: K and Q rows, the two
// 64-key panels of the update, the hi and lo tiles of M.
#include "common.cuh"
#include "gated_delta_tc.cuh"
#include "profile.h"
#include "tma_host.h"

namespace kata {
namespace {

using namespace gdtc;

constexpr int kThreads = kChainThreads;
constexpr uint32_t kTmemCols = 512;
// Tensor memory columns. Operands and accumulators share them, each thread
// rewriting only what it has read:
//   kColS     S operand; M R with M hi, with M lo; the update
//   col_ks(c) [K; Q] S, in two places by turns; R operand in K S's, then P D, which
//             with Q S stays into the next chunk
//   kColD     D~ operand;  kColDl  D operand
constexpr uint32_t kColS = 0, kColKS = 128, kColD = 384, kColDl = 448;
__device__ __forceinline__ uint32_t col_ks(int c) { return kColKS + 128 * (c & 1); }
__device__ __forceinline__ uint32_t col_qs(int c) { return col_ks(c) + 64; }

// kOut: outputs. kSave: each chunk's starting state and writes for the gradient.
enum Mode { kOut, kSave };

template <int DK, int DV, int MODE> struct Layout {
  static constexpr int NP = DK / 64;                       // panels of a K or Q tile
  static constexpr int kStride = (MODE == kOut ? 2 : 1) * kPanel;   // [K p0][Q p0][K p1][Q p1] or K alone
  static constexpr int kKq = NP * kStride;
  static constexpr int kM = 2 * kPanel, kP = MODE == kOut ? 2 * kPanel : 0;   // tiles hi, lo
  static constexpr int kV = kC * DV * 2;                   // V, then the outputs in its place
  static constexpr int kStateHalf = (int)state_image(DK, DV) / 2, kWrites = (int)write_image(DV);
  static constexpr int kSaves = MODE != kSave ? 0 : kStateHalf > kWrites ? kStateHalf : kWrites;
  // Stages of loads, as many as fit: NS of K, Q and M, which a chunk's update
  // frees, and NV of V, P and the gates, which its outputs free in the next chunk.
  static constexpr int kEarly = kKq + kM, kLate = kV + kP + kRecGates, kRoom = 232448 - 512 - 1024 - kSaves;
  static constexpr int kExtra = MODE == kOut ? 1 : 0;
  static constexpr int kFit = (kRoom - kExtra * kLate) / (kEarly + kLate);
  static constexpr int NS = kFit < 4 - kExtra ? kFit : 4 - kExtra, NV = NS + kExtra;
  static constexpr int kOffKq = 0;
  static constexpr int kOffM = NS * kKq;
  static constexpr int kOffP = kOffM + NS * kM;
  static constexpr int kOffV = kOffP + NV * kP;
  static constexpr int kOffStage = kOffV + NV * kV;        // what is being saved: half an image
  static constexpr int kOffGates = kOffStage + kSaves;
  static constexpr int kOffBars = kOffGates + NV * kRecGates;
  static constexpr int kBytes = kOffBars + 512 + 1024;     // barriers, alignment slack
  static_assert(NS >= 2 && kBytes <= 232448, "shared memory budget");
};
// Loaded: K, Q and M; V, P and the gates. Free: K, Q and M (!OUT: V and the gates
// too); V's place, which holds the chunk's outputs. The issuer waits for the
// state warps alone: they wait for the loads and fold them into their own arrivals.
enum {
  kKqFull = 0, kVFull = 4, kFree = 8, kOutputs = 12, kKsDone = 16, kDDone, kUDone, kODone, kStaged, kSaved, kEnd,
  kNumBars = kEnd + 2
};
static_assert(8 * kNumBars + 8 <= 512, "barrier area");
// hardware barriers, state warps to issuers (0 is the block's; two for D by turns)
enum { kSReady = 1, kRReady, kDtReady, kDlReady };

struct Args {
  const float *S0;
  float *S_out;
  uint8_t *img_S, *img_D;          // kSave
  const uint8_t *records;          // [BH][N]
  const float *starts;             // segments' starting states [BH][G][DK][DV], 1 .. G - 1 used
  unsigned *status;
  int H, Hk, T, N, G, seg_chunks;
  int dk, dv;                      // the tensors' head sizes, <= DK, DV
};

template <int DK, int DV, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
gd_tc_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
             const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo,
             const Args a) {
  using L = Layout<DK, DV, MODE>;
  constexpr int NP = L::NP, NS = L::NS, NV = L::NV;
  constexpr bool OUT = MODE == kOut, SAVE = MODE == kSave;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kOffBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const float *gates = reinterpret_cast<const float *>(smem + L::kOffGates);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int seg = blockIdx.x % a.G, bh = blockIdx.x / a.G;
  const int kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
  const int t_begin = seg * a.seg_chunks * kC;
  const int t_left = a.T - t_begin;
  const int nall = t_left <= 0 ? 0 : (t_left - 1) / kC + 1;
  const int n = nall < a.seg_chunks ? nall : a.seg_chunks;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if ((i >= kFree && i < kOutputs + 4) || i == kStaged) count = kStateWarps;
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

  // P D of chunk c, by a whole warp. For d_k = 64 a warp of its own issues it
  // while the issuer goes on: P D takes as long as K S, which the state warps then
  // wait for (99 us instead of 108 at 128 heads of 2048 tokens). For d_k = 128 it
  // comes after the update, which it would only slow down (778 us instead of 799 at
  // 16 heads of 131072).
  constexpr bool kOwnPd = DK == 64;
  auto issue_pd = [&](int c) {
    constexpr uint32_t id_64 = idesc_bf16(128, 64, false, false);
    const uint32_t acc = tbase + col_ks(c);
    const uint64_t d_p = smem_desc(smem_u32(smem) + L::kOffP + c % NV * L::kP, 16, 1024, kSw128);
    take_over(kDlReady + gdsync::output_place(c));
    tc_fence_after();
    if (lane == 0) {
#pragma unroll
      for (int pass = 0; pass < 3; ++pass)                 // hi hi, hi lo, lo hi
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts(acc, tbase + kColDl + 16 * k + 8 * (pass == 2),
                 d_p + (uint64_t)(((pass == 1 ? kPanel : 0) + 32 * k) >> 4), id_64, pass > 0 || k > 0);
      mma_commit(&bars[kODone]);
    }
  };

  if (warp < kStateWarps) {
    // ------------------------------------------------------------ state warps
    const int h = warp / 4;                                // quarter of the columns
    const int r = 32 * (warp % 4) + lane;                  // value column
    const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
    const bool active = r < DV;                            // the same in the whole warp
    constexpr int HK = DK / 4;                             // state entries a thread
    float2 S[HK / 2];
    {
      const float *src = nullptr;
      const bool given = seg == 0;                         // by the caller, in its own head sizes
      const int rows = given ? a.dk : DK, ld = given ? a.dv : DV;
      if (given)
        src = a.S0 ? a.S0 + (size_t)bh * rows * ld : nullptr;
      else
        src = a.starts + ((size_t)bh * a.G + seg) * DK * DV;
      auto entry = [&](int k) { return src && r < ld && k < rows ? src[(size_t)k * ld + r] : 0.f; };
#pragma unroll
      for (int i = 0; i < HK / 2; ++i) S[i] = make_float2(entry(HK * h + 2 * i), entry(HK * h + 2 * i + 1));
    }
    const uint32_t col_s = tbase + lane_off + kColS + HK * h;
    const uint32_t col_part = tbase + lane_off + 16 * h;           // + a 64-token region
    bool ok = true;

    // the staging buffer takes three parts a chunk: S hi, S lo, D
    uint8_t *stage = smem + L::kOffStage;
    auto stage_free = [&](int use) -> bool {
      return use == 0 || warp_wait(&bars[kSaved], (use - 1) & 1, abort_flag);
    };
    auto staged = [&]() {
      fence_async_smem();
      warp_arrive(&bars[kStaged]);
    };
    // outputs of chunk c, o_t = e^{G_t} (Q S)_t + (P D)_t, 16 tokens a thread,
    // into the places its values of V were read from
    auto outputs = [&](int c) {
      ok &= warp_wait(&bars[kODone], c & 1, abort_flag);
      tc_fence_after();
      if (active) {
        __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(smem + L::kOffV + c % NV * L::kV) +
                             16 * h * DV + r;
        const float *from_start = gates + c % NV * (kRecGates / 4);
        uint32_t x[16], y[16];
        tmem_ld16(col_part + col_ks(c), x);
        tmem_ld16(col_part + col_qs(c), y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 o = __ffma2_rn(gate2(from_start, 16 * h + i), as_float2(y[i], y[i + 1]), as_float2(x[i], x[i + 1]));
          dst[i * DV] = __float2bfloat16_rn(o.x);
          dst[(i + 1) * DV] = __float2bfloat16_rn(o.y);
        }
      }
      fence_async_smem();
      tc_fence_before();
      warp_arrive(&bars[kOutputs + c % NV]);
    };

    for (int c = 0; c < n; ++c) {
      const int st = c % NS, sv = c % NV;
      ok &= warp_wait(&bars[kKqFull + st], (c / NS) & 1, abort_flag);
      if (active) {
#pragma unroll
        for (int b = 0; b < HK / 16; ++b) put16(col_s + 16 * b, S + 8 * b);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kSReady, ok);
      if (OUT && !kOwnPd && c > 0) outputs(c - 1);
      if (SAVE) {
        ok &= stage_free(3 * c);
        if (active) stage_row<HK / 8>(stage, DV, r, HK * h, S, false);
        staged();
      }

      // R = beta (V - e^G (K S))
      ok &= warp_wait(&bars[kVFull + sv], (c / NV) & 1, abort_flag);
      const float *from_start = gates + sv * (kRecGates / 4), *to_end = from_start + kC, *beta = to_end + kC;
      uint32_t V[8];                                       // two tokens a register
      {
        const uint16_t *v = reinterpret_cast<const uint16_t *>(smem + L::kOffV + sv * L::kV) + 16 * h * DV + r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          V[i] = active ? (uint32_t)v[2 * i * DV] | (uint32_t)v[(2 * i + 1) * DV] << 16 : 0u;
      }
      ok &= warp_wait(&bars[kKsDone], c & 1, abort_flag);
      tc_fence_after();
      if (active) {
        uint32_t x[16];
        float2 y[8];
        tmem_ld16(col_part + col_ks(c), x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = gate2(from_start, 16 * h + 2 * i);
          y[i] = __fmul2_rn(gate2(beta, 16 * h + 2 * i),
                            __ffma2_rn(make_float2(-f.x, -f.y), as_float2(x[2 * i], x[2 * i + 1]),
                                       as_float2(V[i] << 16, V[i] & 0xffff0000u)));
        }
        put16(col_part + col_ks(c), y);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kRReady, ok);
      if (OUT && kOwnPd && c > 0) outputs(c - 1);
      if (SAVE) {
        ok &= stage_free(3 * c + 1);
        if (active) stage_row<HK / 8>(stage, DV, r, HK * h, S, true);
        staged();
      }

      // D, from its two accumulators: scaled for the update first, as it is
      // for the outputs after
      ok &= warp_wait(&bars[kDDone], c & 1, abort_flag);
      tc_fence_after();
      float2 d[8];
      if (active) {
        uint32_t x[16], y[16];
        float2 z[8];
        tmem_ld16(col_part + kColS, x);
        tmem_ld16(col_part + kColS + 64, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = __fadd2_rn(as_float2(x[2 * i], x[2 * i + 1]), as_float2(y[2 * i], y[2 * i + 1]));
          z[i] = __fmul2_rn(gate2(to_end, 16 * h + 2 * i), d[i]);
        }
        put16(col_part + kColD, z);
        tmem_wait_st();
      }
      tc_fence_before();
      hand_over(kDtReady, ok);
      const float whole = from_start[kC - 1];
      if (OUT) {
        if (active) {
          put16(col_part + kColDl, d);
          tmem_wait_st();
        }
        tc_fence_before();
        hand_over(kDlReady + gdsync::output_place(c), ok);
      }

      if (SAVE) {
        ok &= stage_free(3 * c + 2);
        if (active) {
          stage_row<2>(stage, DV, r, 16 * h, d, false);
          stage_row<2>(stage + (size_t)DV * 128, DV, r, 16 * h, d, true);
        }
        staged();
      }

      // S' = e^{G_C} S + K^T D~
      ok &= warp_wait(&bars[kUDone], c & 1, abort_flag);
      tc_fence_after();
      if (active) {
        const float2 w2 = make_float2(whole, whole);
#pragma unroll
        for (int b = 0; b < HK / 16; ++b) {
          uint32_t x[16];
          tmem_ld16(col_s + 16 * b, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            S[8 * b + i] = __ffma2_rn(w2, S[8 * b + i], as_float2(x[2 * i], x[2 * i + 1]));
        }
      }
      warp_arrive(&bars[kFree + st]);
    }
    if (OUT) {
      outputs(n - 1);
    }
    if (OUT && ok && seg == a.G - 1 && a.S_out && r < a.dv) {
      float *dst = a.S_out + (size_t)bh * a.dk * a.dv + r;
#pragma unroll
      for (int i = 0; i < HK / 2; ++i) {
        const int k = HK * h + 2 * i;
        if (k < a.dk) {                                    // even
          dst[(size_t)k * a.dv] = S[i].x;
          dst[(size_t)(k + 1) * a.dv] = S[i].y;
        }
      }
    }
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and one lane issues: descriptors and column
    // addresses are then uniform values (computed by a lane on its own they cost
    // an MMA 100 cycles). Descriptors of a stage differ only in their address
    // field (bytes / 16).
    constexpr uint32_t id_64 = idesc_bf16(128, 64, false, false);      // K-major right operand
    constexpr uint32_t id_128 = idesc_bf16(128, 128, false, false);
    constexpr uint32_t id_up = idesc_bf16(128, DK, false, true);       // MN-major
    const bool leader = lane == 0;
    const uint32_t base = smem_u32(smem);
    auto adv = [](uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); };
    for (int c = 0; c < n; ++c) {
      const int st = c % NS;
      const uint64_t d_kq = smem_desc(base + L::kOffKq + st * L::kKq, 16, 1024, kSw128);
      const uint64_t d_k_mn = smem_desc(base + L::kOffKq + st * L::kKq, L::kStride, 1024, kSw128);
      const uint64_t d_m = smem_desc(base + L::kOffM + st * L::kM, 16, 1024, kSw128);
      const uint32_t ks = tbase + col_ks(c);
      take_over(kSReady);
      tc_fence_after();
      if (leader) {
        // [K; Q] S (!OUT: K S): S^T hi and lo against the K and Q rows. An
        // operand in tensor memory takes 16 columns a 16-deep step, hi then lo.
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
            mma_ts(ks, tbase + kColS + 16 * k + 8 * lo, adv(d_kq, (k / 4) * L::kStride + (k % 4) * 32),
                   OUT ? id_128 : id_64, lo > 0 || k > 0);
        mma_commit(&bars[kKsDone]);
      }
      take_over(kRReady);
      tc_fence_after();
      if (leader) {
        // R^T hi against [M hi; M lo] (two accumulators), R^T lo against M hi
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tbase + kColS, ks + 16 * k + 8 * lo, adv(d_m, 32 * k), lo ? id_64 : id_128, lo > 0 || k > 0);
        mma_commit(&bars[kDDone]);
      }
      take_over(kDtReady);
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tbase + kColS, tbase + kColD + 16 * k + 8 * lo, adv(d_k_mn, k * 2048), id_up, lo > 0 || k > 0);
        mma_commit(&bars[kUDone]);
      }
      if (OUT && !kOwnPd) issue_pd(c);
    }
    if (leader) {                                          // nothing in flight when tensor memory is given back
      mma_commit(&bars[kEnd]);
      drain(&bars[kEnd], 0);
    }
  } else if (OUT && kOwnPd && warp == kSaver) {
    for (int c = 0; c < n; ++c) issue_pd(c);
    if (lane == 0) {
      mma_commit(&bars[kEnd + 1]);
      drain(&bars[kEnd + 1], 0);
    }
  } else if (warp == kLoader) {
    if (lane == 0) {
      // ---------------------------------------------------------- loads, output stores
      tma_prefetch_desc(&tmk);
      if (OUT) tma_prefetch_desc(&tmq);
      if (OUT) tma_prefetch_desc(&tmo);
      tma_prefetch_desc(&tmv);
      const uint8_t *rec = a.records + ((size_t)bh * a.N + (size_t)seg * a.seg_chunks) * kRecBytes;
      auto load_early = [&](int c) {
        const int st = c % NS;
        uint8_t *kq = smem + L::kOffKq + st * L::kKq;
        mbar_arrive_expect_tx(&bars[kKqFull + st], L::kEarly);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          tma_load_3d(kq + p * L::kStride, &tmk, &bars[kKqFull + st], 64 * p, t_begin + kC * c, kh);
          if (OUT) tma_load_3d(kq + p * L::kStride + kPanel, &tmq, &bars[kKqFull + st], 64 * p, t_begin + kC * c, kh);
        }
        bulk_load(smem + L::kOffM + st * L::kM, rec + (size_t)c * kRecBytes + kRecM, L::kM, &bars[kKqFull + st]);
      };
      auto load_late = [&](int c) {
        const int sv = c % NV;
        mbar_arrive_expect_tx(&bars[kVFull + sv], L::kLate);
        bulk_load(smem + L::kOffGates + sv * kRecGates, rec + (size_t)c * kRecBytes, kRecGates, &bars[kVFull + sv]);
        tma_load_3d(smem + L::kOffV + sv * L::kV, &tmv, &bars[kVFull + sv], 0, t_begin + kC * c, bh);
        if (OUT)
          bulk_load(smem + L::kOffP + sv * L::kP, rec + (size_t)c * kRecBytes + kRecP, L::kP, &bars[kVFull + sv]);
      };
      int early = 0, late = 0;                             // sent
      for (; early < n && early < NS; ++early) {
        load_early(early);
        load_late(late++);
      }
      if (OUT && late < n) load_late(late++);
      for (int c = 0; c <= n; ++c) {
        if (OUT && c > 0) {
          const int sv = (c - 1) % NV;
          if (!free_to_load(&bars[kOutputs + sv], ((c - 1) / NV) & 1, abort_flag)) break;
          tma_store_3d(&tmo, smem + L::kOffV + sv * L::kV, 0, t_begin + kC * (c - 1), bh);
          bulk_commit_group();
          if (late < n) {
            bulk_wait_read_all();                          // the outputs have left V's place
            load_late(late++);
          }
        }
        if (early < n) {
          if (!free_to_load(&bars[kFree + c % NS], (c / NS) & 1, abort_flag)) break;
          load_early(early++);
          if (!OUT) load_late(late++);
        } else if (!OUT) {
          break;
        }
      }
      bulk_wait_all();
      // copies in flight land before the exit
      for (int c = early > NS ? early - NS : 0; c < early; ++c) drain(&bars[kKqFull + c % NS], (c / NS) & 1);
      for (int c = late > NV ? late - NV : 0; c < late; ++c) drain(&bars[kVFull + c % NV], (c / NV) & 1);
    }
  } else if (SAVE && warp == kSaver) {
    if (lane == 0) {
      // ---------------------------------------------------------- saves
      const size_t first = (size_t)bh * a.N + (size_t)seg * a.seg_chunks;
      for (int use = 0; use < 3 * n; ++use) {
        if (!mbar_wait(&bars[kStaged], use & 1, abort_flag)) break;
        const int part = use % 3;
        const size_t at = first + use / 3;
        if (part < 2)
          bulk_store(a.img_S + at * state_image(DK, DV) + part * L::kStateHalf, smem + L::kOffStage, L::kStateHalf);
        else
          bulk_store(a.img_D + at * write_image(DV), smem + L::kOffStage, L::kWrites);
        bulk_commit_group();
        bulk_wait_read_all();
        mbar_arrive(&bars[kSaved]);
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

template <int DK, int DV, int MODE>
cudaError_t run_chain(const char *name, const GatedDeltaLaunch &a, const CUtensorMap *maps, const Args &x,
                      long long blocks) {
  constexpr int bytes = Layout<DK, DV, MODE>::kBytes;
  auto kern = gd_tc_kernel<DK, DV, MODE>;
  GD_ALLOW_SMEM(kern, bytes);
  ProfileScope prof(name, a.stream);
  kern<<<(unsigned)blocks, kThreads, bytes, a.stream>>>(maps[0], maps[1], maps[2], maps[3], x);
  return cudaGetLastError();
}

template <int DK, int DV, int MODE>
cudaError_t launch(const char *name, const GatedDeltaLaunch &a, int d_k, int d_v) {
  CUtensorMap m[4];
  const long long BHk = a.BH / a.H * a.Hk;
  void *o = MODE == kOut ? a.o : const_cast<void *>(a.v);  // no outputs: the map is not used
  if (!make_tma_3d_bf16_box(&m[0], a.q, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&m[1], a.k, d_k, a.T, BHk, 64, kC, true) ||
      !make_tma_3d_bf16_box(&m[2], a.v, d_v, a.T, a.BH, DV, kC, false) ||
      !make_tma_3d_bf16_box(&m[3], o, d_v, a.T, a.BH, DV, kC, false))
    return cudaErrorInvalidValue;
  const Args x{a.S0, a.S_out, a.img_S, a.img_D, a.records, a.starts_seg,
               a.status, a.H, a.Hk, a.T, a.N, a.G, a.seg_chunks, d_k, d_v};
  return run_chain<DK, DV, MODE>(name, a, m, x, a.BH * a.G);
}

}  // namespace

// Segments a head, by the time they should take. Microseconds a chunk of each
// pass as measured for d_k <= 64 and above, one block an SM; every further launch
// costs 7, a join step 4.
void gd_tc_split(long long BH, int N, int d_k, int d_v, bool gradient, int *G, int *seg_chunks) {
  struct Cost { double out, effect, save, reverse, reverse_effect; };
  const Cost us = gd_padded(d_k) == 64 ? Cost{2.8, 3.2, 2.9, 4.1, 2.8} : Cost{3.3, 4.2, 4.2, 5.4, 3.3};
  int best = 1;
  double least = 1e300;
  auto waves = [](long long blocks) { return (double)((blocks + kGdSms - 1) / kGdSms); };
  for (int g = 1; g <= 64 && (g == 1 || (long long)g * BH <= kGdSms); ++g) {
    const int per = (N + g - 1) / g, used = per > 0 ? (N + per - 1) / per : 1;
    if (used != g) continue;
    double time = (gradient ? us.save + us.reverse : us.out) * waves(BH * g) * per;
    if (g > 1)
      time += (us.effect + (gradient ? us.reverse_effect : 0.0)) * waves(BH * (g - 1)) * per + (gradient ? 14.0 : 7.0);
    if (g > 2) time += 7.0 + 4.0 * (g - 2) * waves(BH * (gd_padded(d_v) / 16) * (gradient ? 2 : 1));
    if (time < least) {
      least = time;
      best = g;
    }
  }
  *G = best;
  *seg_chunks = (N + best - 1) / best;
}

cudaError_t gd_tc_save(const GatedDeltaLaunch &a, int d_k, int d_v) {
#define GD_RUN(DK, DV) launch<DK, DV, kSave>("gd_tc_save", a, d_k, d_v)
  return GD_TC_DISPATCH(GD_RUN);
#undef GD_RUN
}
// The solve, the segments' starting states, then the outputs.
cudaError_t gd_tc_forward(const GatedDeltaLaunch &a, int d_k, int d_v) {
  cudaError_t e = gd_tc_solve(a, d_k);
  if (e == cudaSuccess) e = gd_tc_effect(a, d_k, d_v);
  if (e == cudaSuccess) e = gd_tc_join(a, d_k, d_v);
  if (e != cudaSuccess) return e;
#define GD_RUN(DK, DV) launch<DK, DV, kOut>("gd_tc_forward", a, d_k, d_v)
  return GD_TC_DISPATCH(GD_RUN);
#undef GD_RUN
}
size_t gd_tc_state_image(int d_k, int d_v) { return state_image(gd_padded(d_k), gd_padded(d_v)); }
size_t gd_tc_write_image(int d_v) { return write_image(gd_padded(d_v)); }

}  // namespace kata
