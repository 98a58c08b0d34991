// Scored attention backward for sm_103a (the gradient of fa_scored_fwd.cu), bf16.
//
//   P_ij = exp(s_ij - LSE_i) (0 where masked), dP = dO V^T, D_i = dO_i . O_i
//   dS   = P (dP - D) (1 - tanh^2)   dQ = scale dS K   dK = scale sum_h dS^T Q   dV = sum_h P^T dO
//
// The preprocess and the dQ conversion are the plain backward's (fa_bwd.cu), and so is
// the main kernel's pipeline: one CTA per 128-key block, K_j and V_j resident, 64-row
// blocks of Q and dO streaming through a TMA ring, S^T and dP^T in TMEM, P^T and dS^T
// written back as bf16 operands of dV, dK and dQ^T, dQ added to an fp32 accumulator.
// What differs:
//
//  * A CTA owns a key block of one key/value head and walks the query blocks of every
//    query head of the group, so dK and dV of shared heads are summed in the same TMEM
//    accumulators (no atomics, one rounding).
//  * Its query blocks are those between its first key's first query and its last key's
//    last query (the plan's intervals); each thread holds one key and its interval.
//  * Without a cap, LSE and D still enter through the extra K-step of S^T and dP^T. With
//    one, tanh needs the bare products: S^T goes without, and the compute warps subtract
//    LSE2 (64 fp32 values beside each query block) after the cap.
//  * Where the key blocks are few (parts_of), the steps of each are dealt out to several CTAs,
//    which leave fp32 sums of dK and dV in the workspace for bwd_join_kernel, added there in a
//    fixed order.
//  * At d = 64 dQ^T is an MMA of 64 rows, whose accumulator lies in 16 lanes of each of
//    the four dQ warps' quarters, so all four add (with K^T padded to 128 rows two do:
//    cap 50, B=2 H=32 N=8192 causal 2287 us, 2145 so).  The padding's box stays unused.
//
// Roundings: P and dS go to bf16 as MMA operands (off by at most 2^-8 of the value each), O
// comes in bf16 into D; scores, LSE, D and every sum are fp32.  Against gradients summed in
// fp32 throughout (relative error 0.0017, their own rounding to bf16) dQ and dK come to
// 0.0024-0.0036: dS's rounding adds 0.0017, O's 0.0006 where rows see many keys alike up to
// 0.002 where they see few.
//
// Bound: no pipe alone.  Per step (128 keys x 64 queries) at d = 128 the MMAs' math is 1344
// cycles, their operands from shared memory 62 % of its bandwidth, dQ's adds 53 % of the L2's;
// a step takes about 2080.  Measured, backward with its preprocess and conversion, B=2 H=16
// (4 key/value heads) N=8192 d=128 causal: 1075 us (1279 TFLOP/s; the plain backward 1205-1240),
// with a bias 1100, capped at 50 1290; d = 64, H = 32: 1746, capped 2150 (the plain 2588).
// Without dQ's adds it would take 940 (d = 128) and 1591 us (d = 64).  Tried and slower: 16
// compute warps of 16 queries a thread (1266), the two warpgroups on steps in turn with S and dP
// double (1235), dQ by TMA reductions from shared memory (1575), steps of 128 queries at d = 64
// (1909 for 1746).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "fa_bwd_common.cuh"
#include "fa_device.cuh"
#include "fa_internal.h"
#include "fa_score.cuh"

namespace fa {
namespace {

struct Params {
  MaskPlan plan;
  int causal, N, Npad, H, Hkv, group, nkb, parts, run;
  float scale, scale_log2;
  float cap_in, cap_out;  // 4 scale / softcap (products to x = 4 u), softcap log2(e)
  CapPoly poly;           // factor 1
  const float* slopes;
  const uint8_t* aug;
  float* dq_acc;
  float* part_sums;       // [parts][dV, dK][B Hkv][N][D] where parts > 1
  const float* dq_bmax;
  const float* kv_max;
  unsigned int* err_word;
  unsigned long long wait_ns;
};

// The CTA's steps: query blocks [i0, i0 + nq) of each head of the group, head by head.
struct Steps {
  int i0, nq, n;
};
__device__ __forceinline__ Steps steps_of(const Params& p, int kb, int b) {
  const int lo = queries_of(p.plan, p.causal, b, kb * kBkB, p.N).x;
  const int hi = queries_of(p.plan, p.causal, b, min(kb * kBkB + kBkB, p.N) - 1, p.N).y;
  const int i0 = lo / kBqB;
  const int nq = hi > lo ? (hi + kBqB - 1) / kBqB - i0 : 0;
  return {i0, nq, nq * p.group};
}

// MODE 0: scores as they are; 1: with a distance bias; 2: capped; 3: capped within kBoundedCap and
// biased; 4: capped beyond it and biased (its own build: the fourth way through a step would cost MODE 3 14 % at B=2
// H=16/4 N=4096 d=128, cap 20, causal: 505 us, 576 with it).
// DIVIDED: parts > 1 (its own build: the undivided one would be 1 % slower with it).
template <int D, int MODE, bool DET, bool DIVIDED>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_scored_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                      const __grid_constant__ Params p) {
  using C = BwdCfg<D>;
  // S^T and dP^T from two threads: at d = 128 their 18 MMAs a step delay each other's issue (B=2 H=16/4 N=8192
  // causal: 1075 us against 1135 from one; deterministic 1107 against 1205); at d = 64 there are 10 (H=32: 1764
  // against 1727).
  constexpr bool kSplitSdp = D == 128;
  // The deterministic form adds full query blocks without a test of every row (B=2 N=8192 causal, cap 50, d = 128,
  // H=16/4: 1641 us with the test, 1391 without; d = 64, H=32: 3390 | 2269).  The fp32 adds keep it: they take less
  // time, and in bursts hold up the compute warps' stores (d = 128: 1272 us with the test, 1337 without; d = 64: 2145 |
  // 2325).
  constexpr bool kWholeAdds = DET;
  constexpr bool kCapped = MODE >= 2, kBiased = MODE != 0 && MODE != 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + C::kKOff;
  uint8_t* sV = smem + C::kVOff;
  uint8_t* sRing = smem + C::kRingOff;
  uint8_t* sDs = smem + C::kDsOff;
  uint64_t* bar_kv = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* bar_full = bar_kv + 1;
  uint64_t* bar_empty = bar_full + kStages;
  uint64_t* bar_sdp = bar_empty + kStages;  // S^T, dP^T ready in TMEM
  uint64_t* bar_sde = bar_sdp + 1;          // S^T, dP^T read out of TMEM
  uint64_t* bar_comp = bar_sde + 1;         // [2] P^T, dS^T written
  uint64_t* bar_dqf = bar_comp + 2;         // [2] dQ^T ready in TMEM
  uint64_t* bar_dqe = bar_dqf + 2;          // [2] dQ^T read out of TMEM
  uint64_t* bar_dkv = bar_dqe + 2;
  uint64_t* bar_epi = bar_dkv + 1;
  uint64_t* bar_drain = bar_epi + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // Heads in runs of p.run: within one, key blocks in order and heads next to one another; causal key
  // blocks near the start see the most queries and go first.
  const int parts = DIVIDED ? p.parts : 1;
  const int unit = static_cast<int>(blockIdx.x) / parts, part = static_cast<int>(blockIdx.x) % parts;
  const int kvheads = static_cast<int>(gridDim.x) / parts / p.nkb;  // B Hkv
  const int run0 = unit / (p.run * p.nkb) * p.run, run = min(p.run, kvheads - run0), in_run = unit - run0 * p.nkb;
  const int kb = in_run / run, bhk = run0 + in_run % run;
  const int hk = bhk % p.Hkv, b_idx = bhk / p.Hkv;
  const int h0 = hk * p.group;               // first query head of the group
  const int bh0 = b_idx * p.H + h0;

  if (threadIdx.x == kWarpLoad * 32) {
    mbar_init(bar_kv, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    mbar_init(bar_sdp, kSplitSdp ? 2 : 1);
    mbar_init(bar_sde, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bar_comp[b], 8);
      mbar_init(&bar_dqf[b], 1);
      mbar_init(&bar_dqe[b], 4);
    }
    mbar_init(bar_dkv, 1);
    mbar_init(bar_epi, 8);
    mbar_init(bar_drain, kSplitSdp ? 3 : 2);
    *abort_flag = 0;
    fence_mbar_init();
    // K and V start at once, while the intervals are read and TMEM is allocated.
    mbar_arrive_expect_tx(bar_kv, 2 * C::kKVTile);
    for (int c = 0; c < C::kBoxes; ++c) {
      tma_load_4d(sK + c * C::kKVBox, &tm_k, bar_kv, c * 64, kb * kBkB, hk, b_idx);
      tma_load_4d(sV + c * C::kKVBox, &tm_v, bar_kv, c * 64, kb * kBkB, hk, b_idx);
    }
  }
  const Steps st = steps_of(p, kb, b_idx);
  // This part's steps: n from the first on, that one being block i_first of head head_first.
  const int first = st.n * part / parts, n = st.n * (part + 1) / parts - first;
  const int head_first = DIVIDED && n > 0 ? first / st.nq : 0, i_first = st.i0 + first - head_first * st.nq;
  auto load_q_do = [&](int slot, int g, int i) {
    uint8_t* dst = sRing + slot * C::kStageBytes;
    mbar_arrive_expect_tx(&bar_full[slot], C::kStageTx);
    for (int c = 0; c < C::kBoxes; ++c) {
      tma_load_4d(dst + C::kStageQ + c * C::kQBox, &tm_q, &bar_full[slot], c * 64, i * kBqB, h0 + g, b_idx);
      tma_load_4d(dst + C::kStageDO + c * C::kQBox, &tm_do, &bar_full[slot], c * 64, i * kBqB, h0 + g, b_idx);
    }
  };
  // Q and dO of the first steps do not wait for the preprocess either; their LSE and D follow in the producer.
  if (threadIdx.x == kWarpLoad * 32)
    for (int it = 0, g = head_first, i = i_first; it < min(n, kStages); ++it) {
      load_q_do(it, g, i);
      if (++i == st.i0 + st.nq) {
        i = st.i0;
        ++g;
      }
    }
  {
    // The extra K-step's key-side tiles (BwdCfg), one 16-byte half-row per thread.
    const int tile = threadIdx.x >> 8, krow = (threadIdx.x >> 1) & 127, half = threadIdx.x & 1;
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (tile == 0) {
      uint32_t c[3];
      split3_bf16(1.f / p.scale_log2, c);
      val = half == 0 ? make_uint4(c[0] | (c[0] << 16), c[0] | (c[1] << 16), c[1] | (c[1] << 16), c[2] | (c[2] << 16))
                      : make_uint4(c[2], 0u, 0u, 0u);
    } else if (half == 0) {
      val = make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u);  // bf16 1.0, 1.0, 1.0
    }
    uint8_t* base = smem + (tile == 0 ? C::kKAugOff : C::kVAugOff);
    *reinterpret_cast<uint4*>(base + krow * 32 + ((half ^ ((krow >> 2) & 1)) << 4)) = val;
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err_word, p.wait_ns};
  grid_release();
  grid_wait();  // the preprocess has written LSE and D and zeroed the dQ accumulator
  const size_t head_blocks = static_cast<size_t>(p.Npad / kBqB);

  if (warp >= kWarpCtl) {
    regs_decrease<kRegsControl>();
    if (warp == kWarpLoad) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        int issued = 0, g = head_first, i = i_first;
        for (int it = 0; it < n; ++it) {
          const int slot = it % kStages;
          if (!mbar_wait(&bar_empty[slot], ((it / kStages) & 1) ^ 1, wc, kSiteBLoad)) break;
          uint8_t* dst = sRing + slot * C::kStageBytes;
          if (it >= kStages) load_q_do(slot, g, i);
          bulk_load(dst + C::kStageAug, p.aug + ((bh0 + g) * head_blocks + i) * (2 * C::kAugTile), 2 * C::kAugTile,
                    &bar_full[slot]);
          ++issued;
          if (++i == st.i0 + st.nq) {
            i = st.i0;
            ++g;
          }
        }
        if (issued < n) {  // aborted: let the copies already in flight land
          mbar_wait_drain(bar_kv, 0, p.wait_ns);
          for (int t = max(0, issued - kStages); t < issued; ++t)
            mbar_wait_drain(&bar_full[t % kStages], (t / kStages) & 1, p.wait_ns);
        }
      }
      __syncwarp();
    } else if (warp == kWarpMma || warp == kWarpMmaS || (kSplitSdp && warp == kWarpMmaDP)) {
      // -------------------------------------------- MMA issuers (one thread each)
      // Hazards between the issuing threads are covered as in the plain backward.
      if (lane == 0) {
        constexpr uint32_t idesc_sdp = idesc_bf16_f32(kBkB, kBqB, 0, 0);   // keys x queries, K = d
        constexpr uint32_t idesc_dkv = idesc_bf16_f32(kBkB, D, 0, 1);      // keys x d, K = queries
        constexpr uint32_t idesc_dq = idesc_bf16_f32(D, kBqB, 1, 1);       // d x queries, K = keys
        const uint64_t k_kmaj = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t v_kmaj = sdesc_sw128(smem_u32(sV), 16, 1024);
        const uint64_t k_mn = sdesc_sw128(smem_u32(sK), C::kKVBox, 1024);
        const uint64_t ring_kmaj = sdesc_sw128(smem_u32(sRing), 16, 1024);
        const uint64_t ring_mn = sdesc_sw128(smem_u32(sRing), C::kQBox, 1024);
        const uint64_t ds_mn = sdesc_sw128(smem_u32(sDs), 16, 1024);
        const uint64_t kaug = sdesc_sw32(smem_u32(smem + C::kKAugOff));
        const uint64_t vaug = sdesc_sw32(smem_u32(smem + C::kVAugOff));
        const uint64_t ring_aug = sdesc_sw32(smem_u32(sRing + C::kStageAug));
        bool ok = n == 0 || mbar_wait(bar_kv, 0, wc, kSiteBMmaKV);
        int slot = 0;
        uint32_t stage = 0;
        if (warp != kWarpMma) {
          const bool issue_s = warp == kWarpMmaS;
          const bool issue_dp = kSplitSdp ? warp == kWarpMmaDP : warp == kWarpMmaS;
          uint32_t ring_ph = 0;
          for (int it = 0; ok && it < n; ++it) {
            if (!(ok = mbar_wait(&bar_full[slot], ring_ph, wc, kSiteBMmaQ))) break;
            if (it >= 1 && !(ok = mbar_wait(bar_sde, (it - 1) & 1, wc, kSiteBMmaSd))) break;
            tc_fence_after();
            if (issue_s) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t offa = (kk / 4) * C::kKVBox + (kk % 4) * 32;
                const uint32_t offb = (kk / 4) * C::kQBox + (kk % 4) * 32;
                mma_bf16_ss(tmem + C::kColS, sdesc_add(k_kmaj, offa), sdesc_add(ring_kmaj, stage + C::kStageQ + offb),
                            idesc_sdp, kk > 0 ? 1u : 0u);
              }
              if (!kCapped) mma_bf16_ss(tmem + C::kColS, kaug, sdesc_add(ring_aug, stage), idesc_sdp, 1u);
            }
            if (issue_dp) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t offa = (kk / 4) * C::kKVBox + (kk % 4) * 32;
                const uint32_t offb = (kk / 4) * C::kQBox + (kk % 4) * 32;
                mma_bf16_ss(tmem + C::kColDP, sdesc_add(v_kmaj, offa),
                            sdesc_add(ring_kmaj, stage + C::kStageDO + offb), idesc_sdp, kk > 0 ? 1u : 0u);
              }
              mma_bf16_ss(tmem + C::kColDP, vaug, sdesc_add(ring_aug, stage + C::kAugTile), idesc_sdp, 1u);  // - D
            }
            mma_commit(bar_sdp);
            if (++slot == kStages) {
              slot = 0;
              ring_ph ^= 1u;
              stage = 0;
            } else {
              stage += C::kStageBytes;
            }
          }
        } else {
          for (int it = 0; ok && it < n; ++it) {
            const int b = it & 1;
            if (!(ok = mbar_wait(&bar_comp[b], (it >> 1) & 1, wc, kSiteBMmaC))) break;
            tc_fence_after();
            // dV += P^T dO_i ; dK += dS^T Q_i
#pragma unroll
            for (int kk = 0; kk < kBqB / 16; ++kk)
              mma_bf16_ts(tmem + C::kColDV, tmem + C::col_pdq(b) + kk * 8,
                          sdesc_add(ring_mn, stage + C::kStageDO + kk * 2048), idesc_dkv, (it > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
            for (int kk = 0; kk < kBqB / 16; ++kk)
              mma_bf16_ts(tmem + C::kColDK, tmem + C::col_pdq(b) + 32 + kk * 8,
                          sdesc_add(ring_mn, stage + C::kStageQ + kk * 2048), idesc_dkv, (it > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&bar_empty[slot]);
            // dQ_i^T = K^T dS^T
#pragma unroll
            for (int kk = 0; kk < kBkB / 16; ++kk)
              mma_bf16_ss(tmem + C::col_pdq(b), sdesc_add(k_mn, kk * 2048),
                          sdesc_add(ds_mn, b * C::kDsBytes + kk * 2048), idesc_dq, kk > 0 ? 1u : 0u);
            mma_commit(&bar_dqf[b]);
            if (++slot == kStages) {
              slot = 0;
              stage = 0;
            } else {
              stage += C::kStageBytes;
            }
          }
          if (ok) mma_commit(bar_dkv);
        }
        // Every issued MMA of every issuing thread must finish before TMEM is released.
        mma_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0, p.wait_ns);
      }
      __syncwarp();
    }
  } else if (warp < kWarpDq) {
    regs_increase<kRegsCompute>();
    // --------------------------------------- P and dS (one key row per thread)
    const int g = warp >> 2;  // queries 32g .. 32g+31 of every block
    const int row = threadIdx.x & 127;
    const int key = kb * kBkB + row;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int2 by = key < p.N ? queries_of(p.plan, p.causal, b_idx, key, p.N) : make_int2(0, 0);
    // Queries that see every key of the block: [all_lo, all_hi); none if the block is ragged.
    const bool ragged = kb * kBkB + kBkB > p.N;
    const int all_lo = queries_of(p.plan, p.causal, b_idx, min(kb * kBkB + kBkB, p.N) - 1, p.N).x;
    const int all_hi = ragged ? 0 : queries_of(p.plan, p.causal, b_idx, kb * kBkB, p.N).y;
    // No key of the warp is seen by a query before it: |i - j| = i - j wherever it counts.
    const bool one_sided = !kBiased || __all_sync(0xffffffffu, by.x >= key || by.x >= by.y);
    bool ok = true;
    int head = head_first, i = i_first, slot = 0;
    uint32_t ring_ph = 0;
    float slope2 = kBiased && n > 0 ? __ldg(p.slopes + h0 + head) * kLog2e : 0.f;
    for (int it = 0; it < n; ++it) {
      const int b = it & 1;
      if (!(ok = warp_wait_b_suspend(bar_sdp, it & 1, wc, kSiteBComp))) break;
      tc_fence_after();
      uint32_t s[32], dp[32];
      tmem_ld32(trow + C::kColS + 32 * g, s);
      tmem_ld32(trow + C::kColDP + 32 * g, dp);
      tmem_ld_wait32(s);
      tmem_ld_wait32(dp);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sde);  // the MMA warp may now overwrite S^T, dP^T
      const int qb = i * kBqB, q0 = qb + 32 * g;
      const bool need_mask = qb < all_lo || qb + kBqB > all_hi;
      bool general = kBiased && !one_sided && qb < kb * kBkB + kBkB - 1;
      bool small = false;  // MODE 4: general, but no argument of the cap reaches 1/2
      const float4* lse4 = nullptr;
      if constexpr (kCapped) {
        uint32_t bits = 0;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 x = __fmul2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), pair(p.cap_in));
          bits = or_bits(bits, x);
          s[c] = __float_as_uint(x.x);
          s[c + 1] = __float_as_uint(x.y);
        }
        if constexpr (MODE == 4) {
          small = !__any_sync(0xffffffffu, bits & kReachesTwo);
          general = general || !small;
        } else {
          general = general || __any_sync(0xffffffffu, bits & kReachesTwo);
        }
        // LSE2 of the step's queries: the slot landed before S^T was made of it (the wait makes its
        // bytes visible here), and is refilled only after this step's dV and dK.
        if (!(ok = warp_wait_b(&bar_full[slot], ring_ph, wc, kSiteBComp))) break;
        lse4 = reinterpret_cast<const float4*>(sRing + slot * C::kStageBytes + C::kStageAug) + 8 * g;
      }
      // P^T, dS^T(it) overwrite dQ^T(it-2) (TMEM) and dS^T(it-2) (shared memory).
      if (it >= 2 && !(ok = warp_wait_b(&bar_dqe[b], ((it - 2) >> 1) & 1, wc, kSiteBComp))) break;
      tc_fence_after();
      auto write = [&](const uint32_t (&ppk)[16], const uint32_t (&dpk)[16]) {
        tmem_st16(trow + C::col_pdq(b) + 16 * g, ppk);
        tmem_st16(trow + C::col_pdq(b) + 32 + 16 * g, dpk);
        // dS row into shared memory, 128-byte swizzle: chunk ch holds queries 8ch..8ch+7.
        uint8_t* ds_row = sDs + b * C::kDsBytes + row * 128;
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          const int ch = g * 4 + c4;
          *reinterpret_cast<uint4*>(ds_row + ((ch ^ (row & 7)) * 16)) =
              make_uint4(dpk[4 * c4], dpk[4 * c4 + 1], dpk[4 * c4 + 2], dpk[4 * c4 + 3]);
        }
      };
      // P and dS of the 32 queries, written out.  Three ways, each whole (scores in registers at the
      // meeting of two ways would cost the common one a move each): every key seen by every query;
      // masked; and masked in the general form (any argument of the cap, queries on both sides).  Beyond
      // kBoundedCap a fourth: queries on both sides, but tanh in the form for small arguments.
      auto step = [&](auto masked_c, auto general_c, auto small_c) {
        constexpr bool kMasked = decltype(masked_c)::value, kGeneral = decltype(general_c)::value;
        constexpr bool kAny = kGeneral && !decltype(small_c)::value;
        const uint32_t vis = kMasked ? bits_between(by.x - q0, by.y - q0) : 0xffffffffu;
        // The bias with i >= j: -slope2 more for every query; four steps are added up, then the sum
        // starts afresh.
        const float off0 = -slope2 * static_cast<float>(q0 - key);
        float2 off = make_float2(off0, off0 - slope2);
        uint32_t ppk[16], dpk[16];
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          const float4 l4 = kCapped ? lse4[c4] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = 4 * c4 + 2 * e;
            float2 x = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            float2 dpp = make_float2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1]));
            if constexpr (kCapped) {
              const float2 t = kAny ? tanh_any(x, 1.f, pair(0.f)) : __fmul2_rn(x, tanh_over_x(x, p.poly));
              x = __ffma2_rn(t, pair(p.cap_out), e ? make_float2(-l4.z, -l4.w) : make_float2(-l4.x, -l4.y));
              dpp = __fmul2_rn(dpp, __ffma2_rn(t, make_float2(-t.x, -t.y), pair(1.f)));
            }
            const float2 mul = pair(kCapped ? 1.f : p.scale_log2);
            if constexpr (kBiased && kGeneral) {
              const float d = static_cast<float>(q0 - key);
              x = __ffma2_rn(x, mul, make_float2(-slope2 * fabsf(d + static_cast<float>(c)),
                                                 -slope2 * fabsf(d + static_cast<float>(c + 1))));
            } else if constexpr (kBiased) {
              if (c > 0)
                off = c % 8 == 0 ? make_float2(fmaf(-slope2, static_cast<float>(c), off0), fmaf(-slope2, static_cast<float>(c + 1), off0))
                                 : __fadd2_rn(off, pair(-2.f * slope2));
              x = __ffma2_rn(x, mul, off);
            } else if constexpr (!kCapped) {
              x = __fmul2_rn(x, mul);
            }
            float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            if (kMasked) pp = make_float2(vis & (1u << c) ? pp.x : 0.f, vis & (2u << c) ? pp.y : 0.f);
            float2 ds = __fmul2_rn(pp, dpp);
            // (dP of a masked pair may have overflowed.)
            if (kMasked) ds = make_float2(vis & (1u << c) ? ds.x : 0.f, vis & (2u << c) ? ds.y : 0.f);
            ppk[c / 2] = pack_bf16x2(pp.x, pp.y);
            dpk[c / 2] = pack_bf16x2(ds.x, ds.y);
          }
        }
        write(ppk, dpk);
      };
      if (need_mask && !__any_sync(0xffffffffu, bits_between(by.x - q0, by.y - q0))) {
        const uint32_t zero[16] = {};  // no key of the warp is seen by the 32 queries
        write(zero, zero);
      } else if (MODE == 4 && general && small) step(std::true_type{}, std::true_type{}, std::true_type{});
      else if (general) step(std::true_type{}, std::true_type{}, std::false_type{});
      else if (need_mask) step(std::true_type{}, std::false_type{}, std::false_type{});
      else step(std::false_type{}, std::false_type{}, std::false_type{});
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_comp[b]);
      if (++slot == kStages) {
        slot = 0;
        ring_ph ^= 1u;
      }
      if (++i == st.i0 + st.nq) {
        i = st.i0;
        ++head;
        if (kBiased && head < p.group) slope2 = __ldg(p.slopes + h0 + head) * kLog2e;
      }
    }
    // ------------------------------- dK, dV epilogue (warpgroup 0: dV, 1: dK)
    // (A block that no query sees only waits for K and V to land where its zeros go.)
    if (ok) ok = warp_wait_b(n > 0 ? bar_dkv : bar_kv, 0, wc, kSiteBEpi);
    if (DIVIDED && ok) {
      tc_fence_after();
      float* dst = p.part_sums + (((static_cast<size_t>(part) * 2 + g) * kvheads + bhk) * p.N + key) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 8) {
        uint32_t x[8] = {};
        if (n > 0) tmem_ld8_wait(trow + (g == 0 ? C::kColDV : C::kColDK) + c, x);
        if (key < p.N) {
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(dst + c + 4) = make_uint4(x[4], x[5], x[6], x[7]);
        }
      }
    } else if (ok) {
      tc_fence_after();
      if (n > 0) {
        if (g == 0) stage_row_bf16<D>(trow + C::kColDV, sV, row, 1.f);
        else stage_row_bf16<D>(trow + C::kColDK, sK, row, p.scale);
      } else {  // no query sees the block: zeros
        uint8_t* box = (g == 0 ? sV : sK) + row * 128;
        for (int c = 0; c < C::kBoxes; ++c)
          for (int q4 = 0; q4 < 8; ++q4)
            *reinterpret_cast<uint4*>(box + c * C::kKVBox + q4 * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_epi);
      if (threadIdx.x == 0 && mbar_wait(bar_epi, 0, wc, kSiteBEpi)) {
        for (int c = 0; c < C::kBoxes; ++c) {
          tma_store_4d(&tm_dv, sV + c * C::kKVBox, c * 64, kb * kBkB, hk, b_idx);
          tma_store_4d(&tm_dk, sK + c * C::kKVBox, c * 64, kb * kBkB, hk, b_idx);
        }
        tma_store_commit_and_wait_read();
      }
    }
    __syncwarp();
  } else {
    regs_decrease<kRegsDq>();
    // -------------------------------- dQ reduction (one d-row of dQ^T per thread; at d = 64 half of one)
    const int wq = warp - kWarpDq;
    const int dcol = D == 128 ? 32 * wq + lane : 16 * wq + (lane & 15), q_lane = D == 128 ? 0 : 32 * (lane >> 4);
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int head = head_first, i = i_first;
    for (int it = 0; it < n; ++it) {
      const int b = it & 1;
      const int q0 = i * kBqB, bh = bh0 + head;
      if (++i == st.i0 + st.nq) {
        i = st.i0;
        ++head;
      }
      if (!warp_wait_b_suspend(&bar_dqf[b], (it >> 1) & 1, wc, kSiteBDq)) break;
      tc_fence_after();
      uint32_t v[D / 64][32];
      if constexpr (D == 64) {
        tmem_ld16x64(trow + C::col_pdq(b), v[0]);
        tmem_ld_wait32(v[0]);
      } else {
        tmem_ld32(trow + C::col_pdq(b), v[0]);
        tmem_ld32(trow + C::col_pdq(b) + 32, v[1]);
        tmem_ld_wait32(v[0]);
        tmem_ld_wait32(v[1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_dqe[b]);
      float* dst = p.dq_acc + (static_cast<size_t>(bh) * p.N + q0 + q_lane) * D + dcol;
      const int lim = p.N - q0 - q_lane;
      float mul = 1.f;
      if constexpr (DET)
        mul = pow2f(det_shift(
            det_bound(p.dq_bmax[bh * head_blocks + q0 / kBqB], p.kv_max[2 * bhk], p.kv_max[2 * bhk + 1])));
      auto add = [&](auto whole_c) {
        constexpr bool kWhole = decltype(whole_c)::value;
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (!kWhole && hh * 32 + c >= lim) continue;
            float* at = dst + static_cast<size_t>(hh * 32 + c) * D;
            const float x = __uint_as_float(v[hh][c]);
            if constexpr (DET) {
              constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: x + kMagic rounds x to an integer in the low bits
              atomicAdd(reinterpret_cast<int*>(at), __float_as_int(fmaf(x, mul, kMagic)) - 0x4B400000);
            } else {
              atomicAdd(at, x);
            }
          }
      };
      if (kWholeAdds && q0 + kBqB <= p.N) add(std::true_type{});
      else add(std::false_type{});
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// dV and dK of divided key blocks: the parts' sums, added in order, rounded once.  One thread per 8 columns.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kernel(const float* __restrict__ part_sums, int parts, long long rows,
                                                       int N, int Hkv, __nv_bfloat16* __restrict__ dv, Strides sdv,
                                                       __nv_bfloat16* __restrict__ dk, Strides sdk, float scale) {
  grid_release();
  grid_wait();  // the parts are written
  const long long x = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 8, size = rows * D;
  if (x >= 2 * size) return;
  float acc[8] = {};
  for (int s = 0; s < parts; ++s) {
    const float4* src = reinterpret_cast<const float4*>(part_sums + s * 2 * size + x);
    const float4 a = src[0], b = src[1];
    acc[0] += a.x;
    acc[1] += a.y;
    acc[2] += a.z;
    acc[3] += a.w;
    acc[4] += b.x;
    acc[5] += b.y;
    acc[6] += b.z;
    acc[7] += b.w;
  }
  const bool is_k = x >= size;
  const long long r = (is_k ? x - size : x) / D;
  const float mul = is_k ? scale : 1.f;
  uint4 out;
  out.x = pack_bf16x2(acc[0] * mul, acc[1] * mul);
  out.y = pack_bf16x2(acc[2] * mul, acc[3] * mul);
  out.z = pack_bf16x2(acc[4] * mul, acc[5] * mul);
  out.w = pack_bf16x2(acc[6] * mul, acc[7] * mul);
  __nv_bfloat16* dst = is_k ? dk : dv;
  *reinterpret_cast<uint4*>(dst + row_offset(is_k ? sdk : sdv, r / N, Hkv, static_cast<int>(r % N)) + x % D) = out;
}

// How many CTAs share a key block's steps: up to two a SM in all, each with 8 steps or more if every
// query sees the block.  Undivided, a block's steps run one after another however many SMs are
// idle (causal, d = 128: B=2 H=16/2 N=1030 155 us, 58 divided; B=1 H=8/2 N=3737 of three documents
// 220 | 82; H=2 N=6063 109 | 67).  More parts than that cost more in sums than they gain (three a
// SM: 72 | 92 | 80), and so do shorter ones (4 steps, H=8 N=1024: 37 us for 29).
int parts_of(int B, int H, int Hkv, int N) {
  const long long blocks = static_cast<long long>((N + kBkB - 1) / kBkB) * B * Hkv;
  const long long steps = static_cast<long long>((N + kBqB - 1) / kBqB) * (H / Hkv);
  return static_cast<int>(std::max(1ll, std::min({16ll, 2 * sm_count() / blocks, steps / 8})));
}

// Key/value heads worked on together: as many as have dQ accumulators of 48 MB, which then stay in the L2 (129 MB, with
// what else passes through it) between the adds of a head's key blocks (d = 128: B=16 H=16 N=1024 causal 373 us over
// all heads at once, 297 in runs; B=2 H=16 N=8192 1185 | 1107-1132, full 2231 | 2133-2156; d = 64, H=32 N=8192 biased
// 1771 | 1688).  Where a group's alone are more (long rows of large groups), one key/value head at a time: its key
// blocks walk the query heads in the same order, so the adds of a time still fall on few of them (d = 128, B=1 H=64/8
// N=32768: full 81.6 ms over all heads, 66.0 one at a time, causal 34.7 | 33.4; N=16384 17.2 | 17.3, 8.5 | 8.5; budgeted
// by one query head instead 67.2 and 33.4).  The last run's heavy blocks start late, so only with 10 blocks an SM or
// more (6.7: B=2 H=32/8 N=8192 of eight documents 653 us, 745 in runs).
int run_of(int B, int H, int Hkv, int N, int d) {
  const long long heads = static_cast<long long>(B) * Hkv, blocks = (N + kBkB - 1) / kBkB * heads;
  if (blocks < 10ll * sm_count()) return static_cast<int>(heads);
  const long long bytes = static_cast<long long>(H / Hkv) * N * d * static_cast<long long>(sizeof(float));
  return static_cast<int>(std::max(1ll, std::min(heads, 48000000ll / bytes)));
}

template <int D, int MODE, bool DET, bool DIVIDED>
cudaError_t launch_main(const BwdArgs& a, const ScoreArgs& sc, int parts, cudaStream_t stream) {
  using C = BwdCfg<D>;
  const BwdWorkspace w = bwd_workspace_layout(a.B, a.H, a.N, a.d);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  cudaError_t e;
  CUtensorMap tq, tk, tv, tdo, tdk, tdv;
  constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if ((e = make_tmap_4d(&tq, a.q, kBf16, 2, D, a.N, a.H, a.B, a.sq.s, 64, kBqB))) return e;
  if ((e = make_tmap_4d(&tdo, a.dout, kBf16, 2, D, a.N, a.H, a.B, a.sdo.s, 64, kBqB))) return e;
  if ((e = make_tmap_4d(&tk, a.k, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sk.s, 64, kBkB))) return e;
  if ((e = make_tmap_4d(&tv, a.v, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sv.s, 64, kBkB))) return e;
  if ((e = make_tmap_4d(&tdk, a.dk, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sdk.s, 64, kBkB))) return e;
  if ((e = make_tmap_4d(&tdv, a.dv, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sdv.s, 64, kBkB))) return e;
  Params p{};
  p.plan = sc.plan;
  p.causal = sc.causal;
  p.N = a.N;
  p.Npad = w.npad;
  p.H = a.H;
  p.Hkv = sc.Hkv;
  p.group = a.group;
  p.nkb = (a.N + kBkB - 1) / kBkB;
  p.parts = parts;
  p.run = run_of(a.B, a.H, sc.Hkv, a.N, D);
  p.part_sums = reinterpret_cast<float*>(ws + w.total);
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  if (MODE >= 2) {
    p.cap_in = 4.f * a.scale / sc.softcap;
    p.cap_out = sc.softcap * kLog2e;
    p.poly = cap_poly(1.f);
  }
  p.slopes = sc.slopes;
  p.aug = ws + w.off_aug;
  p.dq_acc = reinterpret_cast<float*>(ws + w.off_dq);
  p.dq_bmax = reinterpret_cast<const float*>(ws + w.off_dqmax);
  p.kv_max = reinterpret_cast<const float*>(ws + w.off_kvmax);
  p.err_word = a.err_word;
  p.wait_ns = a.dbg.wait_limit_ns;
  auto kern = bwd_scored_kernel<D, MODE, DET, DIVIDED>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes))) return e;
  // The register split assumes the block launches with kLaunchRegs per thread.
  cudaFuncAttributes fattr;
  if ((e = cudaFuncGetAttributes(&fattr, kern))) return e;
  if (static_cast<uint32_t>(fattr.numRegs) < kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = launch_dependent(kern, static_cast<unsigned>(p.nkb * a.B * sc.Hkv * p.parts), kThreads, C::kSmemBytes, stream, tq,
                       tk, tv, tdo, tdk, tdv, p);
  if (e || !DIVIDED) return e;
  const long long rows = static_cast<long long>(a.B) * sc.Hkv * a.N;
  return launch_dependent(bwd_join_kernel<D>, static_cast<unsigned>((rows * D / 4 + 255) / 256), 256, 0, stream,
                          const_cast<const float*>(p.part_sums), p.parts, rows, a.N, sc.Hkv,
                          static_cast<__nv_bfloat16*>(a.dv), a.sdv, static_cast<__nv_bfloat16*>(a.dk), a.sdk, a.scale);
}

template <int D, int MODE>
cudaError_t launch_mode(const BwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  const int parts = parts_of(a.B, a.H, sc.Hkv, a.N);
  if (parts > 1)
    return a.deterministic ? launch_main<D, MODE, true, true>(a, sc, parts, stream)
                           : launch_main<D, MODE, false, true>(a, sc, parts, stream);
  return a.deterministic ? launch_main<D, MODE, true, false>(a, sc, parts, stream)
                         : launch_main<D, MODE, false, false>(a, sc, parts, stream);
}

template <int D>
cudaError_t launch_d(const BwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  if (sc.softcap > 0.f)
    return !sc.slopes                           ? launch_mode<D, 2>(a, sc, stream)
           : sc.softcap * kLog2e <= kBoundedCap ? launch_mode<D, 3>(a, sc, stream)
                                                : launch_mode<D, 4>(a, sc, stream);
  return sc.slopes ? launch_mode<D, 1>(a, sc, stream) : launch_mode<D, 0>(a, sc, stream);
}

}  // namespace

size_t bwd_scored_workspace(int B, int H, int Hkv, int N, int d) {
  const int parts = parts_of(B, H, Hkv, N);
  return bwd_workspace_layout(B, H, N, d).total +
         (parts > 1 ? static_cast<size_t>(parts) * 2 * B * Hkv * N * d * sizeof(float) : 0);
}

cudaError_t launch_bwd_scored(const BwdArgs& args, const ScoreArgs& sc, cudaStream_t stream) {
  BwdArgs a = args;
  a.group = a.H / sc.Hkv;
  a.raw_lse = sc.softcap > 0.f;
  a.seen_by = sc.plan.k;
  a.dependent = 1;
  cudaError_t e;
  if ((e = launch_bwd_prep(a, stream))) return e;
  if ((e = a.d == 64 ? launch_d<64>(a, sc, stream) : launch_d<128>(a, sc, stream))) return e;
  return launch_bwd_dq(a, stream);
}

}  // namespace fa
