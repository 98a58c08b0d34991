// What the backward kernels share (fa_bwd.cu and fa_scored_bwd.cu, whose head comments
// describe the design): block sizes, warp roles, the register split, the layout of
// shared memory and TMEM, and small device helpers.
#pragma once

#include <math.h>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kBkB = 128;       // keys per CTA
constexpr int kBqB = 64;        // query rows per inner step
constexpr int kThreads = 512;   // 0-7 compute, 8-11 dQ reduction, 12 TMA, 13-15 MMA issuers (15: see kSplitSdp)
constexpr int kWarpDq = 8;
constexpr int kWarpCtl = 12;
constexpr int kWarpLoad = 12;
constexpr int kWarpMma = 13;     // issues dV, dK, dQ^T (and owns the TMEM allocation)
constexpr int kWarpMmaS = 14;    // issues S^T
constexpr int kWarpMmaDP = 15;   // issues dP^T when the kernel splits that issue (kSplitSdp), else idle
constexpr int kStages = 3;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
// Launch budget 128 x 512 registers: the two compute warpgroups (one 32-query
// half of a score row each) take 160, the dQ warpgroup 120, the control
// warpgroup (TMA, MMA) gives back to 72.
constexpr uint32_t kLaunchRegs = 128;
constexpr uint32_t kRegsCompute = 160;
constexpr uint32_t kRegsDq = 120;
constexpr uint32_t kRegsControl = 72;
static_assert(128 * (2 * kRegsCompute + kRegsDq + kRegsControl) <= kLaunchRegs * kThreads, "register split");

enum : uint32_t {
  kSiteBLoad = 0x111,
  kSiteBMmaKV = 0x211,
  kSiteBMmaQ = 0x212,
  kSiteBMmaC = 0x213,
  kSiteBMmaDq = 0x214,
  kSiteBMmaSd = 0x215,
  kSiteBComp = 0x311,
  kSiteBDq = 0x312,
  kSiteBEpi = 0x313,
};

template <int D>
struct BwdCfg {
  static_assert(D == 64 || D == 128, "head dim");
  static constexpr int kBoxes = D / 64;                 // 128-byte TMA boxes per bf16 row
  static constexpr int kKVBox = kBkB * 64 * 2;          // 16 KB: 128 rows x 128 B
  static constexpr int kKVTile = kBkB * D * 2;          // 32 KB (d=128), 16 KB (d=64)
  static constexpr int kQBox = kBqB * 64 * 2;           // 8 KB: 64 rows x 128 B
  static constexpr int kQTile = kBqB * D * 2;           // 16 KB (d=128), 8 KB (d=64)
  static constexpr int kStageQ = 0;
  static constexpr int kStageDO = kQTile;
  // The extra K-step's per-query tiles (64 rows x 32 bytes, 32-byte swizzle):
  // [a1 a2 a3 a1 a2 a3 a1 a2 a3 0...] with a1 + a2 + a3 = -LSE2 for S^T, then
  // [d1 d2 d3 0...] with d1 + d2 + d3 = -D for dP^T (three-term bf16 splits).
  static constexpr int kAugTile = kBqB * 32;           // 2 KB
  static constexpr int kStageAug = 2 * kQTile;
  static constexpr int kStageTx = 2 * kQTile + 2 * kAugTile;  // bytes landing per stage
  static constexpr int kStageBytes = (kStageTx + 1023) / 1024 * 1024;
  static constexpr int kDsBytes = kBkB * kBqB * 2;      // 16 KB: 128 key rows x 128 B
  // K, then (d = 64) the zero box that pads K^T to the dQ^T MMA's 128 rows, then V,
  // then the extra K-step's constant key-side tiles (128 rows x 32 bytes each):
  // [c1 c1 c1 c2 c2 c2 c3 c3 c3 0...] with c1 + c2 + c3 = 1 / (scale log2 e) for S^T
  // (so the nine products sum to (c1 + c2 + c3)(a1 + a2 + a3)), [1 1 1 0...] for dP^T.
  static constexpr int kKOff = 0;
  static constexpr int kZeroOff = kKVTile;
  static constexpr int kVOff = kKVTile + (D == 64 ? kKVBox : 0);
  static constexpr int kKAugOff = kVOff + kKVTile;
  static constexpr int kVAugOff = kKAugOff + kBkB * 32;
  static constexpr int kRingOff = kVAugOff + kBkB * 32;
  static constexpr int kDsOff = kRingOff + kStages * kStageBytes;
  static constexpr int kBarOff = kDsOff + 2 * kDsBytes;
  // kv, full[S], empty[S], sdp, sde, comp[2], dqf[2], dqe[2], dkv, epi, drain
  static constexpr int kNumBars = 1 + 2 * kStages + 1 + 1 + 2 + 2 + 2 + 1 + 1 + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  // TMEM columns: dV, dK accumulators (D columns each); one S^T, dP^T pair (fp32,
  // read once by the compute warps, then free for the next query block); two
  // 64-column buffers that hold P^T | dS^T (bf16, 32 columns each) and then dQ^T (fp32).
  static constexpr uint32_t kColDV = 0, kColDK = 128, kColS = 256, kColDP = 320;
  static __device__ __forceinline__ uint32_t col_pdq(int b) { return 384u + 64u * b; }
  static_assert(kStageTx <= kStageBytes, "stage layout");
  static_assert(kZeroOff % 1024 == 0 && kKAugOff % 1024 == 0 && kRingOff % 1024 == 0, "operand tile alignment");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ bool warp_wait_b(uint64_t* bar, uint32_t parity, const WaitCtl& wc, uint32_t site) {
  const bool ok = mbar_wait(bar, parity, wc, site);
  return __all_sync(0xffffffffu, ok);
}
// For the compute and dQ warps' long waits (S^T, dP^T ready; dQ^T ready): their polls
// suspend instead of spinning beside the MMA-issuing warps.
__device__ __forceinline__ bool warp_wait_b_suspend(uint64_t* bar, uint32_t parity, const WaitCtl& wc, uint32_t site) {
  const bool ok = mbar_wait_suspend(bar, parity, wc, site, 20000u);
  return __all_sync(0xffffffffu, ok);
}

// Deterministic dQ: fixed-point accumulation.  Every contribution of a key block
// to dQacc[i, c] is sum_j dS_ij k_jc, and the whole sum over all key blocks obeys
//   |sum_j dS_ij k_jc| <= sum_j |dS_ij| max|k| <= 2 max_j |dP_ij| max|k|
//                      <= 2 |dO_i| max_j |v_j| max|k|
// (|dS_ij| = P_ij |dP_ij - D_i| with D_i a P-weighted mean of dP_i., and
// |dP_ij| = |dO_i . v_j| <= |dO_i| |v_j|).  With a 64-row block's largest |dO_i|,
// the head's largest |v_j| and largest |k_jc|, and a 12.5 % margin for the bf16
// rounding of P and dS, the power of two 2^S below puts every partial sum of the
// block's rows under 2^22 in magnitude.  Contributions are rounded to integers
// once (x 2^S, nearest) and added as int32: integer addition does not depend on
// order, so dQ is the same bits on every run.  2^22 keeps the float-to-int step
// a single add of 1.5 * 2^23 (the rounding is the fp32 add's).
//
// NaN and infinities have no place in such sums (a NaN contribution would add an ordinary integer), so they are
// met in the maxima: a row that sees a key with an LSE, D or |dO| that is not finite gives its block an infinite
// maximum, a k or v that is not finite gives its head one, and the conversion writes NaN wherever the bound is
// not finite.  (Telling them apart contribution by contribution costs the plain kernel 4 %.)
__device__ __forceinline__ float det_bound(float dq_block_max, float vmax, float kmax) {
  return dq_block_max > 0.f ? 2.25f * dq_block_max * vmax * kmax : 0.f;  // (0 times an infinity counts as 0 there)
}
__device__ __forceinline__ int det_shift(float bound) {
  if (!(bound > 0.f)) return 100;           // all-zero block (or no data): nothing to scale
  if (!(bound < 3.0e38f)) return -100;
  int e;
  frexpf(bound, &e);                        // bound < 2^e
  return max(-100, min(100, 22 - e));
}
__device__ __forceinline__ float pow2f(int s) { return __int_as_float((s + 127) << 23); }  // -126 <= s <= 127

// Element offset of row n of head (b, h) in a strided [B, H, N, d] tensor.
__device__ __forceinline__ size_t row_offset(const Strides& st, long long bh, int H, int n) {
  return static_cast<size_t>((bh / H) * st.s[2] + (bh % H) * st.s[1] + static_cast<long long>(n) * st.s[0]);
}

// Stage this thread's D-column fp32 accumulator row as bf16 into 128-byte-swizzled
// [128 rows][64 cols] TMA boxes (D / 64 of them).
template <int D>
__device__ __forceinline__ void stage_row_bf16(uint32_t taddr_row, uint8_t* boxes, int row, float mul) {
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(taddr_row + c * 32, o);
    tmem_ld_wait32(o);
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      pk[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * mul, __uint_as_float(o[2 * i + 1]) * mul);
    uint8_t* box = boxes + (c / 2) * BwdCfg<D>::kKVBox + row * 128;
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const int chunk = (c % 2) * 4 + q4;
      *reinterpret_cast<uint4*>(box + ((chunk ^ (row & 7)) * 16)) =
          make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
    }
  }
}

}  // namespace
}  // namespace fa
