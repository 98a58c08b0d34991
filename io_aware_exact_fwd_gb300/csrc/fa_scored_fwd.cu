// Scored attention forward for sm_103a: tanh cap, distance bias, interval masks
// (documents, prefixes), shared key/value heads.  bf16 in and out, fp32 logsumexp.
//
// The pipeline is the plain forward's (fa_fwd.cu): each unit 256 query rows of one head
// as two 128-row tiles (or one in two halves, unit_tiles); K_j, V_j stream through a TMA ring; one thread
// issues S_t = Q_t K_j^T and O_t += P_t V_j on tcgen05 with S, P and O in TMEM; two
// softmax warpgroups hold one query row per thread.  What differs:
//
//  * The keys of a tile are the blocks between its first row's first key and its last
//    row's last key (intervals of the plan, both ends nondecreasing along the rows), so
//    blocks of other documents are never loaded.  A unit streams the union of its two
//    tiles' blocks, and each tile takes part in a contiguous run of that stream.
//  * The stream runs from the last block to the first.  A causal row then meets its
//    diagonal block first, where a distance bias is smallest, so the reference maximum
//    of the first block holds for the rest (forward order would raise every row's
//    maximum in every block) and no row of a document waits masked for its first key.
//  * A unit's work depends on the mask, which only the device knows, so units are not
//    dealt out beforehand: the grid has one block per unit, heaviest rows first, and a
//    running block takes over blocks that have not started (cluster launch control), its
//    pipeline running on from unit to unit.  A scheduler warp asks for the next unit
//    while the current one runs and publishes its key blocks in shared memory.
//
// Bound, as the plain forward: two MMAs of 128 x 128 x d a score block, and beside them one
// exponential a score (with a cap 5 multiply-adds more), of which neither alone fills
// the block's time; the MMA thread and the softmax warps wait for each other.  Measured,
// B=2 H=16 (4 key/value heads) N=8192 d=128 causal: 437 us (1258 TFLOP/s; the plain kernel
// 424-438), with a bias 490, capped at 50 535, both 560; nine documents a row 160, capped 187.
// Units dealt out beforehand in zigzag order were slower (nine documents: 185 us for 166).
#include <math.h>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "fa_score.cuh"

namespace fa {
namespace {

constexpr int kTiles = 2;                       // query tiles per unit
// Warp roles.  With one part, each of the 8 softmax warps holds 32 rows of a tile, 128
// keys a thread; with two, each of 16 holds 64 keys of 32 rows, and two threads share a
// row.  Then K/V TMA, MMA, Q TMA and the scheduler, one warp each.  Capped scores take long chains of
// dependent operations, which four warps a scheduler hide better than two (B=2 H=16/4 N=8192
// causal: 582 us against 648); the other forms keep more values live than 104 registers hold and
// spill (454 us with 8 warps, 732 with 16).
template <int PARTS>
struct Roles {
  static constexpr int kSoftWarps = 8 * PARTS;
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr int kWarpLoad = kSoftWarps, kWarpMma = kSoftWarps + 1, kWarpLoadQ = kSoftWarps + 2,
                       kWarpSched = kSoftWarps + 3;
  // Registers a thread: at launch (65536 / kThreads, down to a multiple of 8), then for the softmax
  // and the control warpgroups.
  static constexpr uint32_t kRegsLaunch = 65536 / kThreads / 8 * 8;
  static constexpr uint32_t kRegsSoftmax = PARTS == 1 ? 216 : 104;
  static constexpr uint32_t kRegsControl = PARTS == 1 ? 72 : 64;
  static constexpr uint32_t kRegsNeeded = 32 * kSoftWarps * kRegsSoftmax + 128 * kRegsControl;
  static_assert(kRegsNeeded <= kRegsLaunch * kThreads, "register split exceeds the launch's registers");
};
constexpr uint32_t kTmemCols = 512;
// A block is exponentiated against the running reference without its own maximum; its
// row sum then proves that no P passed 2^60 (else the block is redone).  P is bf16 and
// everything it enters is fp32, so a reference that is off costs no precision while
// weights, sums and O stay inside the exponent's range (|v| below 2^68 / N).
constexpr float kSpeculationSumBound = 1.152921504606847e18f;
// With a cap, scores lie in [-softcap, softcap] log2(e) (plus a bias whose maximum over
// the row's keys is known): up to kBoundedCap on softcap log2(e) that maximum alone is the
// reference, with P in 2^-80 .. 2^80 (so |v| below 2^48 / N, and what is below 2^-46 of it may be lost where
// scores lie near -softcap) and no maximum taken at all (a cap of 55 at B=2 H=16/4
// N=8192 causal: 535 us; one of 56, with the running reference: 781).
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;

enum : uint32_t {
  kSiteLoadEmpty = 0x121,
  kSiteLoadQ = 0x122,
  kSiteMmaQ = 0x221,
  kSiteMmaK = 0x222,
  kSiteMmaP = 0x223,
  kSiteMmaV = 0x224,
  kSiteSoftS = 0x321,
  kSiteSoftO = 0x322,
  kSiteUnit = 0x324,
  kSiteSched = 0x325,
};

template <int D, int MODE>
struct Cfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kBoxes = kRowBytes / 128;
  static constexpr int kBoxBytes = kBlockK * 128;
  static constexpr int kTileBytes = kBlockK * kRowBytes;
  static constexpr int kKSteps = D / 16;
  static constexpr int kSlots = D == 64 ? 10 : MODE == 1 ? 4 : 5;
  // MODE 1: one more K-step of Q K^T adds the bias's growth along the block's keys: rows of 16 bf16
  // (32-byte swizzle), [s1 s2 s3 0...] with s1 + s2 + s3 = slope / scale for every query of a tile,
  // [j j j 0...] for key j of the block (0 .. 127, exact in bf16).
  static constexpr int kBiasTile = MODE == 1 ? kBlockK * 32 : 0;
  static constexpr int kQOff = 0;
  static constexpr int kRingOff = kTiles * kTileBytes;
  static constexpr int kBiasOff = kRingOff + kSlots * kTileBytes;   // the two tiles' query side, the key side
  static constexpr int kBarOff = kBiasOff + 3 * kBiasTile;
  // q_full[2], q_empty[2], full[kSlots], empty[kSlots], s_full[2], p_full[2], o_done[2], drain, unit,
  // unit_read, answer
  static constexpr int kNumBars = 2 + 2 + 2 * kSlots + 2 + 2 + 2 + 1 + 3;
  static constexpr int kMiscOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kAnswerOff = kMiscOff + 16;                  // launch control's 16-byte answer
  static constexpr int kUnitOff = kAnswerOff + 16;                  // the published unit
  static constexpr int kSmemBytes = kUnitOff + 64 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static __device__ __forceinline__ uint32_t col_s(int t) { return 128u * static_cast<uint32_t>(t); }
  static __device__ __forceinline__ uint32_t col_o(int t) { return 256u + D * static_cast<uint32_t>(t); }
};

struct Params {
  MaskPlan plan;
  int causal, N, H, group, BH, nunits;
  float scale, scale_log2;  // scale_log2 = scale log2(e)
  float cap_in;       // 4 scale / softcap: products to x = 4 u
  float cap_out;      // softcap log2(e)
  CapPoly poly;       // factor cap_out
  const float* slopes;
  __nv_bfloat16* o;
  Strides so;
  float* lse;
  unsigned int* err_word;
  unsigned long long wait_ns;
};

// A unit as the scheduler publishes it: rows u * 256 .. of head bh as two tiles, or rows u * 128 ..
// in two halves (u < 0: no more units).  Tile t attends key blocks [begin[t], end[t]) (empty: both 0),
// and every row of it sees the keys [all_lo[t], all_hi[t]).  The stream covers blocks [first, last)
// from last - 1 down; the halves of a halved unit have the same range and take its blocks in turn.
struct Unit {
  int u, bh;
  int begin[kTiles], end[kTiles], all_lo[kTiles], all_hi[kTiles];
  __device__ __forceinline__ bool has(int t) const { return end[t] > begin[t]; }
  __device__ __forceinline__ int first() const {
    return min(has(0) ? begin[0] : last(), has(1) ? begin[1] : last());
  }
  __device__ __forceinline__ int last() const { return max(end[0], end[1]); }
  // Tile t's run of the stream.
  __device__ __forceinline__ int from(int t) const { return last() - end[t]; }
  __device__ __forceinline__ int to(int t) const { return last() - begin[t]; }
};
// Block w of the grid: the last rows (the heaviest, when causal) first, heads next to one another.
template <int UNIT>
__device__ __forceinline__ Unit unit_of(const Params& p, int w) {
  Unit x;
  x.u = p.nunits - 1 - w / p.BH;
  x.bh = w % p.BH;
  const int b = x.bh / p.H;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int r0 = UNIT == 1 ? x.u * kBlockQ : x.u * 2 * kBlockQ + t * kBlockQ;
    x.begin[t] = x.end[t] = x.all_lo[t] = x.all_hi[t] = 0;
    if (r0 < p.N) {
      const int2 head = keys_of(p.plan, p.causal, b, r0, p.N);
      const int2 tail = keys_of(p.plan, p.causal, b, min(r0 + kBlockQ, p.N) - 1, p.N);
      if (tail.y > head.x) {
        x.begin[t] = head.x / kBlockK;
        x.end[t] = (tail.y + kBlockK - 1) / kBlockK;
      }
      x.all_lo[t] = tail.x;
      x.all_hi[t] = head.y;
    }
  }
  if (UNIT == 1 && x.end[1] - x.begin[1] < 2) x.begin[1] = x.end[1] = 0;
  return x;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc, uint32_t site) {
  const bool ok = mbar_wait(bar, parity, wc, site);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait_suspend(uint64_t* bar, uint32_t parity, const WaitCtl& wc, uint32_t site) {
  const bool ok = mbar_wait_suspend(bar, parity, wc, site, 20000u);
  return __all_sync(0xffffffffu, ok);
}

// The barrier of two warps, and the same with an "any".
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.red.or.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// MODE 0: scores as they are; 1: with a distance bias; 2 and 3: capped within kBoundedCap,
// without and with a bias; 4: capped beyond it (biased if slopes).
template <int MODE>
constexpr int kPartsOf = MODE == 2 || MODE == 3 ? 2 : 1;

// UNIT: tiles of a unit.
template <int D, int MODE, int UNIT>
__global__ void __launch_bounds__(Roles<kPartsOf<MODE>>::kThreads, 1)
    fwd_scored_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using C = Cfg<D, MODE>;
  constexpr int kParts = kPartsOf<MODE>;
  constexpr bool kBounded = MODE == 2 || MODE == 3;  // the fixed reference (kBoundedCap)
  using R = Roles<kParts>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::kQOff;
  uint8_t* sRing = smem + C::kRingOff;
  uint64_t* bar_q = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // [2] per tile: Q landed
  uint64_t* bar_qe = bar_q + 2;              // [2] per tile: last Q K^T of a unit done (Q slot free)
  uint64_t* bar_full = bar_qe + 2;           // [kSlots]
  uint64_t* bar_empty = bar_full + C::kSlots;
  uint64_t* bar_s = bar_empty + C::kSlots;   // [2] per tile: S ready
  uint64_t* bar_p = bar_s + 2;               // [2] per tile: P written
  uint64_t* bar_o = bar_p + 2;               // [2] per tile: last P V of a unit done
  uint64_t* bar_drain = bar_o + 2;
  uint64_t* bar_unit = bar_drain + 1;        // a unit is published
  uint64_t* bar_unit_read = bar_unit + 1;    // every role has read it
  uint64_t* bar_answer = bar_unit_read + 1;  // launch control answered
  Unit* s_unit = reinterpret_cast<Unit*>(smem + C::kUnitOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(&bar_q[t], 1);
      mbar_init(&bar_qe[t], 1);
      mbar_init(&bar_s[t], 1);
      mbar_init(&bar_p[t], 4 * kParts);
      mbar_init(&bar_o[t], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    mbar_init(bar_drain, 1);
    mbar_init(bar_unit, 1);
    mbar_init(bar_unit_read, 3 + R::kSoftWarps);  // the K/V, Q and MMA threads, the softmax warps
    mbar_init(bar_answer, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if constexpr (MODE == 1) {
    for (int x = threadIdx.x; x < 2 * kBlockK; x += R::kThreads) {  // 16-byte half rows, swizzled
      const int j = x >> 1, part = x & 1;
      const uint32_t v = pack_bf16x2(static_cast<float>(j), static_cast<float>(j));
      *reinterpret_cast<uint4*>(smem + C::kBiasOff + 2 * C::kBiasTile + j * 32 + ((part ^ ((j >> 2) & 1)) << 4)) =
          part == 0 ? make_uint4(v, v & 0xffffu, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == R::kWarpMma) tmem_alloc(tmem_slot, kTmemCols);
  if (warp == R::kWarpLoad && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl wc{abort_flag, p.err_word, p.wait_ns};
  // The k-th unit of this block, for a role that is one thread.  False: no more (or aborting).
  auto next_unit = [&](int k, Unit& x, bool& ok) -> bool {
    if (!(ok = mbar_wait(bar_unit, k & 1, wc, kSiteUnit))) return false;
    x = *s_unit;
    mbar_arrive(bar_unit_read);
    return x.u >= 0;
  };

  if (warp >= R::kSoftWarps) {
    regs_decrease<R::kRegsControl>();
    if (warp == R::kWarpSched) {
      // --------------------------------------------------------------- scheduler
      // Unit 0 is the block's own.  The next is asked for once every role has started on the
      // current one: early enough to hide the answer, late enough to keep units for others.
      if (lane == 0) {
        int w = static_cast<int>(blockIdx.x);
        for (int k = 0;; ++k) {
          Unit x{};
          x.u = -1;
          if (w >= 0) x = unit_of<UNIT>(p, w);
          if (k > 0 && !mbar_wait_suspend(bar_unit_read, (k - 1) & 1, wc, kSiteSched, 20000u)) break;
          *s_unit = x;
          mbar_arrive(bar_unit);
          if (w < 0) break;
          if (UNIT == 1) {  // (its results leave the ring and TMEM in use: one unit a block)
            w = -1;
            continue;
          }
          if (k > 0 && !mbar_wait_suspend(bar_unit_read, k & 1, wc, kSiteSched, 20000u)) break;
          mbar_arrive_expect_tx(bar_answer, 16);
          try_cancel(smem + C::kAnswerOff, bar_answer);
          if (!mbar_wait_drain(bar_answer, k & 1, p.wait_ns)) {
            record_timeout(wc, kSiteSched);
            break;
          }
          w = launch_answer(smem + C::kAnswerOff);
          fence_proxy_async_smem();  // the answer is read before the next one lands
        }
      }
      __syncwarp();
    } else if (warp == R::kWarpLoad) {
      // ------------------------------------------------------- K/V TMA producer
      if (lane == 0) {
        int issued = 0;
        bool ok = true;
        Unit x;
        for (int k = 0; ok && next_unit(k, x, ok); ++k) {
          const int b = x.bh / p.H, hk = (x.bh % p.H) / p.group;
          const int first = x.first(), last = x.last();
          // K_j, then V_j; in a halved unit K of two blocks, then V of one and K of the next but one in turn.
          for (int j = UNIT == 1 ? last + 1 : last - 1; ok && j >= first; --j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool kv = UNIT == 1 ? i == 0 : i == 1;
              const int block = UNIT == 1 && !kv ? j - 2 : j;
              if (UNIT == 1 && (block < first || block >= last)) continue;
              const int slot = issued % C::kSlots;
              if (!(ok = mbar_wait_suspend(&bar_empty[slot], ((issued / C::kSlots) & 1) ^ 1, wc, kSiteLoadEmpty, 20000u))) break;
              mbar_arrive_expect_tx(&bar_full[slot], C::kTileBytes);
              uint8_t* dst = sRing + slot * C::kTileBytes;
#pragma unroll
              for (int c = 0; c < C::kBoxes; ++c)
                tma_load_4d(dst + c * C::kBoxBytes, kv ? &tm_v : &tm_k, &bar_full[slot], c * kBoxCols, block * kBlockK,
                            hk, b);
              ++issued;
            }
          }
        }
        if (!ok)  // drain: the last (up to kSlots) issued copies may still be landing
          for (int t = max(0, issued - C::kSlots); t < issued; ++t)
            mbar_wait_drain(&bar_full[t % C::kSlots], (t / C::kSlots) & 1, p.wait_ns);
      }
      __syncwarp();
    } else if (warp == R::kWarpLoadQ) {
      // --------------------------------------------------------- Q TMA producer
      int nload[kTiles] = {0, 0};
      bool ok = true;
      for (int k = 0; (ok = warp_wait_suspend(bar_unit, k & 1, wc, kSiteUnit)); ++k) {
        const Unit x = *s_unit;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_unit_read);
        if (x.u < 0) break;
        const int b = x.bh / p.H, h = x.bh % p.H;
#pragma unroll
        for (int tt = 0; tt < kTiles; ++tt) {
          const int t = UNIT == 1 ? tt : kTiles - 1 - tt;  // the later tile's run of the stream starts first
          if (!ok || !x.has(t)) continue;
          if (nload[t] > 0 && !(ok = warp_wait_suspend(&bar_qe[t], (nload[t] - 1) & 1, wc, kSiteLoadQ))) continue;
          if constexpr (MODE == 1) {  // the head's slope for the bias's K-step
            uint32_t c[3];
            split3_bf16(__ldg(p.slopes + h) / p.scale, c);
            for (int r = lane; r < kBlockQ; r += 32) {
              uint8_t* dst = smem + C::kBiasOff + t * C::kBiasTile + r * 32;
              const int half = (r >> 2) & 1;
              *reinterpret_cast<uint4*>(dst + half * 16) = make_uint4(c[0] | (c[1] << 16), c[2], 0u, 0u);
              *reinterpret_cast<uint4*>(dst + (half ^ 1) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar_q[t], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kBoxes; ++c)
              tma_load_4d(sQ + t * C::kTileBytes + c * C::kBoxBytes, &tm_q, &bar_q[t], c * kBoxCols,
                          UNIT == 1 ? x.u * kBlockQ : x.u * 2 * kBlockQ + t * kBlockQ, h, b);
          }
          ++nload[t];
        }
        if (!ok) break;
      }
      if (!ok && lane == 0)
        for (int t = 0; t < kTiles; ++t)
          if (nload[t] > 0) mbar_wait_drain(&bar_q[t], (nload[t] - 1) & 1, p.wait_ns);
      __syncwarp();
    } else if (warp == R::kWarpMma) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kBlockQ, kBlockK, 0, 0);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kBlockQ, D, 0, 1);
        const uint64_t qdesc = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t kdesc = sdesc_sw128(smem_u32(sRing), 16, 1024);
        const uint64_t vdesc = sdesc_sw128(smem_u32(sRing), C::kBoxBytes, 1024);
        const uint64_t bias_q = sdesc_sw32(smem_u32(smem + C::kBiasOff));
        const uint64_t bias_k = sdesc_sw32(smem_u32(smem + C::kBiasOff + 2 * C::kBiasTile));
        auto qk = [&](int t, int slot) {  // S_t = Q_t K^T: both K-major, 16 columns of d per MMA
          const uint64_t qd = sdesc_add(qdesc, t * C::kTileBytes);
          const uint64_t kd = sdesc_add(kdesc, slot * C::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < C::kKSteps; ++kk) {
            const uint32_t off = (kk / 4) * C::kBoxBytes + (kk % 4) * 32;
            mma_bf16_ss(tmem + C::col_s(t), sdesc_add(qd, off), sdesc_add(kd, off), idesc_qk, kk > 0 ? 1u : 0u);
          }
          if (MODE == 1)  // + slope / scale times the key's place in the block
            mma_bf16_ss(tmem + C::col_s(t), sdesc_add(bias_q, t * C::kBiasTile), bias_k, idesc_qk, 1u);
          mma_commit(&bar_s[t]);
        };
        auto pv = [&](int t, int slot, bool accumulate) {  // O_t += P_t V: P from TMEM, V MN-major
          const uint64_t vd = sdesc_add(vdesc, slot * C::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < kBlockK / 16; ++kk)
            // With two parts, P of keys 64-127 lies over S columns 64-95, each part over its own S.
            mma_bf16_ts(tmem + C::col_o(t), tmem + C::col_s(t) + kk * 8 + (kParts == 2 ? (kk / 4) * 32 : 0),
                        sdesc_add(vd, kk * 16 * 128), idesc_pv, (accumulate || kk > 0) ? 1u : 0u);
        };
        int item = 0;  // ring index of the next K or V block to consume
        uint32_t nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;  // Q tiles and P blocks consumed so far
        bool ok = true;
        Unit x{}, nx{};
        bool have_next = false;             // nx is the next unit
        bool early0 = false, early1 = false;  // its first S of tile 0, 1 is issued
        for (int k = 0; ok; ++k) {
          if (have_next) x = nx;
          else if (!next_unit(k, x, ok)) break;
          if (x.u < 0) break;
          have_next = false;
          const int n = x.last() - x.first();
          if constexpr (UNIT == 1) {
            // Block j from the end belongs to slot j & 1; every ring item has one user.
            for (int j = -2; ok && j < n; ++j) {
              const int t = j & 1;
              if (j >= 0) {  // O_t += P_t V_j
                const int slot = item % C::kSlots;
                if (!(ok = mbar_wait(&bar_full[slot], (item / C::kSlots) & 1, wc, kSiteMmaV))) break;
                if (!(ok = mbar_wait(&bar_p[t], (j >> 1) & 1, wc, kSiteMmaP))) break;
                ++item;
                tc_fence_after();
                pv(t, slot, j >= 2);
                mma_commit(&bar_empty[slot]);
                if (j + 2 >= n) mma_commit(&bar_o[t]);
              }
              if (j + 2 < n) {  // S_t = Q K_{j + 2}^T
                const int slot = item % C::kSlots;
                if (!(ok = mbar_wait(&bar_full[slot], (item / C::kSlots) & 1, wc, kSiteMmaK))) break;
                if (j < 0 && !(ok = mbar_wait(&bar_q[t], 0, wc, kSiteMmaQ))) break;
                ++item;
                tc_fence_after();
                qk(t, slot);
                mma_commit(&bar_empty[slot]);
              }
            }
          } else
          // Stream position s: K_s is ring item 2 s, V_s item 2 s + 1 of the unit.  S_t of position
          // s is issued right after the P_t V of position s - 1 (position 0: before the loop).
          for (int s = -1; ok && s < n; ++s) {
            const int slot_v = item % C::kSlots;
            if (s >= 0) {
              if (!(ok = mbar_wait(&bar_full[slot_v], (item / C::kSlots) & 1, wc, kSiteMmaV))) break;
              ++item;
            }
            const bool has_next = s + 1 < n;
            const int slot_k = item % C::kSlots;
            const uint32_t par_k = (item / C::kSlots) & 1;
            if (has_next) ++item;
            bool k_ready = false;
#pragma unroll
            for (int tt = 0; tt < kTiles; ++tt) {
              const int t = kTiles - 1 - tt;
              const int f = x.from(t), l = x.has(t) ? x.to(t) : f;
              if (ok && s >= f && s < l) {
                if (!(ok = mbar_wait(&bar_p[t], (t ? np1 : np0) & 1, wc, kSiteMmaP))) continue;
                if (t) ++np1; else ++np0;
                tc_fence_after();
                pv(t, slot_v, s > f);
                if (s + 1 == l) mma_commit(&bar_o[t]);
              }
              if (ok && s + 1 >= f && s + 1 < l && !(s == -1 && (t ? early1 : early0))) {
                if (!k_ready) {
                  if (!(ok = mbar_wait(&bar_full[slot_k], par_k, wc, kSiteMmaK))) continue;
                  k_ready = true;
                }
                if (s + 1 == f) {
                  if (!(ok = mbar_wait(&bar_q[t], (t ? nq1 : nq0) & 1, wc, kSiteMmaQ))) continue;
                  if (t) ++nq1; else ++nq0;
                }
                tc_fence_after();
                qk(t, slot_k);
                if (s + 2 == l) mma_commit(&bar_qe[t]);
              }
              if (s == -1) (t ? early1 : early0) = false;
              // The unit's last position: tile t's first S of the next unit need not wait for the other
              // tile's last P, if all it needs has arrived.  (With one part the unit change is a smaller
              // share and the code costs more: causal 447 -> 465 us at B=2 H=16/4 N=8192 d=128.)
              if (kParts == 2 && ok && s == n - 1) {
                if (!have_next && mbar_try_wait(bar_unit, (k + 1) & 1)) have_next = next_unit(k + 1, nx, ok) || nx.u < 0;
                const int slot0 = item % C::kSlots;  // K_0 of the next unit
                if (have_next && nx.u >= 0 && nx.has(t) && nx.from(t) == 0 &&
                    mbar_try_wait(&bar_full[slot0], (item / C::kSlots) & 1) &&
                    mbar_try_wait(&bar_q[t], (t ? nq1 : nq0) & 1)) {
                  if (t) ++nq1; else ++nq0;
                  tc_fence_after();
                  qk(t, slot0);
                  if (nx.to(t) == 1) mma_commit(&bar_qe[t]);
                  (t ? early1 : early0) = true;
                }
              }
            }
            if (!ok) break;
            if (s >= 0) mma_commit(&bar_empty[slot_v]);
            if (has_next) {
              if (!k_ready && !(ok = mbar_wait(&bar_full[slot_k], par_k, wc, kSiteMmaK))) break;
              mma_commit(&bar_empty[slot_k]);
            }
          }
        }
        mma_commit(bar_drain);  // every issued MMA must finish before TMEM is released
        mbar_wait_drain(bar_drain, 0, p.wait_ns);
      }
      __syncwarp();
    }
  } else {
    regs_increase<R::kRegsSoftmax>();
    // ------------------------------------------------------ softmax warpgroups
    const int t = warp / (4 * kParts), half = kParts == 2 ? (warp >> 2) & 1 : 0;
    const int row = threadIdx.x & 127;
    const int pair_id = 1 + t * 4 + (warp & 3);  // named barrier of the two warps that share 32 rows
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t col_s = C::col_s(t) + 64 * half, col_o = C::col_o(t);
    uint32_t scnt = 0;   // S blocks consumed so far (bar_s phase)
    uint32_t nout = 0;   // units of this tile with keys (bar_o phase)
    // The warps of a pair meet at their barrier in every unit, so a warp whose wait gave up (the block
    // is aborting) carries on with whatever TMEM holds, and both leave together at the next unit.
    bool ok = true;
    // The next unit; with two parts, read (and its row's interval and slope requested) before the
    // epilogue of the current one if it is published by then.  With one part the registers that takes
    // cost more than it saves (bias 542 -> 667 us at B=2 H=16/4 N=8192 d=128).
    struct {
      int u, bh, blk0, blk1, all_lo, all_hi;
      int2 see;
      float slope2;
    } nu;
    bool have_next = false;
    struct {  // a halved unit's result in this slot
      bool done;
      float m, l;
      int nkt, bh, qrow;
    } mine{};
    auto read_unit = [&]() {
      nu.u = s_unit->u;
      nu.bh = s_unit->bh;
      nu.blk0 = s_unit->begin[t];
      nu.blk1 = s_unit->end[t];
      nu.all_lo = s_unit->all_lo[t];
      nu.all_hi = s_unit->all_hi[t];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_unit_read);
      const int qrow = (UNIT == 1 ? nu.u * kBlockQ : nu.u * 2 * kBlockQ + t * kBlockQ) + row;
      nu.see = make_int2(0, 0);
      nu.slope2 = 0.f;
      if (nu.u >= 0) {
        if (qrow < p.N) nu.see = keys_of(p.plan, p.causal, nu.bh / p.H, qrow, p.N);
        if (MODE != 0 && p.slopes) nu.slope2 = __ldg(p.slopes + nu.bh % p.H) * kLog2e;
      }
    };
    for (int k = 0;; ++k) {
      if (!have_next) ok = ok && warp_wait(bar_unit, k & 1, wc, kSiteUnit);
      if (kParts == 2 ? pair_or(pair_id, !ok) : !ok) break;
      if (!have_next) read_unit();
      have_next = false;
      if (nu.u < 0) break;
      const int bh = nu.bh, b = bh / p.H, h = bh % p.H;
      const int row0 = UNIT == 1 ? nu.u * kBlockQ : nu.u * 2 * kBlockQ + t * kBlockQ;
      if (row0 >= p.N) continue;
      const int qrow = row0 + row;
      const int2 see = nu.see;
      const float slope2 = nu.slope2;
      // Keys that every row of the tile sees: [all_lo, all_hi).
      const int all_lo = nu.all_lo, all_hi = nu.all_hi, blk1 = nu.blk1;
      const int nkt = UNIT == 1 ? (nu.blk1 - nu.blk0 - t + 1) / 2 : nu.blk1 - nu.blk0;
      // Reference maximum, log2 units (0 until the row has seen a key).  kBounded: the largest bias
      // among the row's keys: 0, at the row's own position, or for a negative slope at its farthest.
      float m_used = 0.f;
      if (MODE == 3 && slope2 < 0.f && see.x < see.y)
        m_used = -slope2 * static_cast<float>(max(qrow - see.x, see.y - 1 - qrow));
      bool seen = false;
      float l = 0.f;
      // No row of the warp sees a key right of itself: |i - j| = i - j wherever it counts.
      const bool one_sided = MODE == 0 || __all_sync(0xffffffffu, see.y <= qrow + 1);

      for (int j = 0; j < nkt; ++j, ++scnt) {
        ok = warp_wait_suspend(&bar_s[t], scnt & 1, wc, kSiteSoftS) && ok;
        tc_fence_after();
        const int kbase = (blk1 - 1 - (UNIT == 1 ? 2 * j + t : j)) * kBlockK;
        const bool need_mask = kbase < all_lo || kbase + kBlockK > all_hi;
        const bool left = one_sided || kbase + kBlockK - 1 <= row0, right = kbase >= row0 + kBlockQ - 1;
        float2 part = make_float2(0.f, 0.f);
        if constexpr (kBounded) {
          // The fixed reference: P = exp2(cap + bias - m_used), 32 columns at a time.  P of columns 32c..
          // goes over columns 16c.. of the thread's S, which are consumed.
#pragma unroll 1
          for (int c = 0; c < 4 / kParts; ++c) {
            uint32_t r[32];
            tmem_ld32(trow + col_s + c * 32, r);
            tmem_ld_wait32(r);
            const int key0 = kbase + 64 * half + c * 32;
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = __fmul2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), pair(p.cap_in));
              bits = or_bits(bits, x);
              r[i] = __float_as_uint(x.x);
              r[i + 1] = __float_as_uint(x.y);
            }
            const bool general = __any_sync(0xffffffffu, bits & kReachesTwo) || (MODE == 3 && !left);
            const uint32_t vis = bits_between(see.x - key0, see.y - key0);
            // Each way below stores its own P: scores in registers at the meeting of two ways cost the
            // common one a move each (14 % of the kernel).
            if (general) {
              // Any argument of the cap, a bias with keys right of the row: a small rolled loop from S,
              // still whole in TMEM (P of these columns trails the columns read).
#pragma unroll 1
              for (int i = 0; i < 32; i += 8) {
                uint32_t x[8], pk[4];
                tmem_ld8_wait(trow + col_s + c * 32 + i, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  float2 y = tanh_any(__fmul2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), pair(p.cap_in)),
                                      p.cap_out, pair(-m_used));
                  if (MODE == 3) {
                    const float off = static_cast<float>(key0 + i + e - qrow);
                    y.x = fmaf(-slope2, fabsf(off), y.x);
                    y.y = fmaf(-slope2, fabsf(off + 1.f), y.y);
                  }
                  const uint32_t v = vis >> (i + e);
                  const float2 w = make_float2(v & 1u ? ex2_approx(y.x) : 0.f, v & 2u ? ex2_approx(y.y) : 0.f);
                  part = __fadd2_rn(part, w);
                  pk[e / 2] = pack_bf16x2(w.x, w.y);
                }
                tmem_st4(trow + col_s + c * 16 + i / 2, pk);
              }
              continue;
            }
            // The bias on the row's left: slope2 more for every key; four steps are added up, then the
            // sum starts afresh.
            const float off0 = MODE == 3 ? fmaf(slope2, static_cast<float>(key0 - qrow), -m_used) : -m_used;
            float2 off = make_float2(off0, MODE == 3 ? off0 + slope2 : off0);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]));
              if (MODE == 3 && i > 0)
                off = i % 8 == 0 ? make_float2(fmaf(slope2, static_cast<float>(i), off0), fmaf(slope2, static_cast<float>(i + 1), off0))
                                 : __fadd2_rn(off, pair(2.f * slope2));
              const float2 y = __ffma2_rn(x, tanh_over_x(x, p.poly), off);
              r[i] = __float_as_uint(y.x);
              r[i + 1] = __float_as_uint(y.y);
            }
            uint32_t pk[16];
            if (need_mask) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = make_float2(vis & (1u << (2 * i)) ? ex2_approx(__uint_as_float(r[2 * i])) : 0.f,
                                             vis & (2u << (2 * i)) ? ex2_approx(__uint_as_float(r[2 * i + 1])) : 0.f);
                part = __fadd2_rn(part, e);
                pk[i] = pack_bf16x2(e.x, e.y);
              }
              tmem_st16(trow + col_s + c * 16, pk);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = make_float2(ex2_approx(__uint_as_float(r[2 * i])), ex2_approx(__uint_as_float(r[2 * i + 1])));
                part = __fadd2_rn(part, e);
                pk[i] = pack_bf16x2(e.x, e.y);
              }
              tmem_st16(trow + col_s + c * 16, pk);
            }
          }
        }
        if constexpr (!kBounded) {
        // The general form of the scores (any argument of the cap, a bias with keys right of the row),
        // eight columns at a time in place in TMEM before they are loaded: a small rolled loop, because
        // it is rare, the kernel's speed depends on its code fitting the instruction caches, and a
        // second form of 128 scores in registers would cost the common one a move for each.
        const bool biased = MODE == 1 || (MODE == 4 && p.slopes != nullptr);
        bool pre = biased && !left, far = false;  // far: an argument of the cap reaches 1/2
        if constexpr (MODE == 4) {
          uint32_t bits = 0;
#pragma unroll 1
          for (int c = 0; c < kBlockK; c += 8) {
            uint32_t x[8];
            tmem_ld8_wait(trow + col_s + c, x);
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              bits = or_bits(bits, __fmul2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), pair(p.cap_in)));
          }
          far = __any_sync(0xffffffffu, bits & kReachesTwo);
          pre = pre || far;
        }
        if (pre) {
#pragma unroll 1
          for (int c = 0; c < kBlockK; c += 8) {
            uint32_t x[8];
            tmem_ld8_wait(trow + col_s + c, x);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              float2 a = make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
              if constexpr (MODE == 4) {
                a = __fmul2_rn(a, pair(p.cap_in));
                a = far ? tanh_any(a, p.cap_out, pair(0.f)) : __fmul2_rn(a, tanh_over_x(a, p.poly));
              } else {  // the K-step's slope times the key's place is taken out again
                a = __ffma2_rn(pair(-slope2), make_float2(static_cast<float>(c + i), static_cast<float>(c + i + 1)),
                               __fmul2_rn(a, pair(p.scale_log2)));
              }
              const float off = static_cast<float>(kbase + c + i - qrow);
              x[i] = __float_as_uint(fmaf(-slope2, fabsf(off), a.x));
              x[i + 1] = __float_as_uint(fmaf(-slope2, fabsf(off + 1.f), a.y));
            }
            tmem_st8(trow + col_s + c, x);
          }
          tmem_st_wait();
        }
        if (MODE != 4 && need_mask) {  // in TMEM as well: -inf stays -inf below (its factor is positive)
#pragma unroll 1
          for (int c = 0; c < kBlockK; c += 32) {
            uint32_t x[32];
            tmem_ld32(trow + col_s + c, x);
            tmem_ld_wait32(x);
            const uint32_t vis = bits_between(see.x - kbase - c, see.y - kbase - c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(vis & (1u << i))) x[i] = __float_as_uint(-INFINITY);
            tmem_st32(trow + col_s + c, x);
          }
          tmem_st_wait();
        }
        uint32_t r[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(trow + col_s + c * 32, r[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait32(r[c]);
        // The score less the reference, in log2 units, is r mul + base.  On the row's left, base has the
        // bias of the block's first key; its growth from there is in S (MODE 1).
        const float first = slope2 * static_cast<float>(kbase - qrow);
        const float mul = MODE == 4 || pre ? 1.f : p.scale_log2;
        float base = MODE == 0 || MODE == 4 || pre ? -m_used : first - m_used;
        if constexpr (MODE == 4) {  // the cap and the bias, in place; the identity where `pre` has made the scores
          CapPoly poly = p.poly;
          if (pre) {
            poly.c[0] = pair(1.f);
            poly.c[1] = poly.c[2] = poly.c[3] = pair(0.f);
          }
          const float in = pre ? 1.f : p.cap_in, step = pre ? 0.f : slope2;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // step more for every key: four steps are added up, then the sum starts afresh.
            const float off0 = pre ? 0.f : fmaf(step, 32.f * c, first);
            float2 off = pair(off0);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              off = i % 8 == 0 ? make_float2(fmaf(step, static_cast<float>(i), off0), fmaf(step, static_cast<float>(i + 1), off0))
                               : __fadd2_rn(off, pair(2.f * step));
              const float2 x = __fmul2_rn(make_float2(__uint_as_float(r[c][i]), __uint_as_float(r[c][i + 1])), pair(in));
              const float2 y = __ffma2_rn(x, tanh_over_x(x, poly), off);
              r[c][i] = __float_as_uint(y.x);
              r[c][i + 1] = __float_as_uint(y.y);
            }
            if (need_mask) {
              const uint32_t vis = bits_between(see.x - kbase - c * 32, see.y - kbase - c * 32);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(vis & (1u << i))) r[c][i] = __float_as_uint(-INFINITY);
            }
          }
        }
        // P = exp2(r mul + base), packed bf16 over the S columns.  The row's reference is its first block's
        // maximum.  Later blocks are first taken against the reference as it is, and taken again
        // against their own maximum if a P may have overflowed, or if they hold the row's first
        // visible keys.  A bias that falls with distance makes the maxima grow while the blocks lie
        // right of the rows: there the maximum comes first, too.
        bool own_max = j == 0 || (MODE != 0 && slope2 > 0.f && right && !one_sided);
        while (true) {
          if (own_max) {
            float mc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float a[11];
#pragma unroll
              for (int i = 0; i < 10; ++i)
                a[i] = max3(__uint_as_float(r[c][3 * i]), __uint_as_float(r[c][3 * i + 1]),
                            __uint_as_float(r[c][3 * i + 2]));
              a[10] = fmaxf(__uint_as_float(r[c][30]), __uint_as_float(r[c][31]));
              mc[c] = fmaxf(max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), max3(a[6], a[7], a[8])),
                            fmaxf(a[9], a[10]));
            }
            const float mt = fmaf(fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])), mul, base);  // mul > 0
            // The reference moves by mt where that is up, or the row's first.
            const bool first = !seen && mt > -INFINITY;
            const bool up = first || (seen && mt > 0.f);
            const float delta = up ? mt : 0.f;
            const float alpha = up && seen ? ex2_approx(-delta) : 1.f;
            const bool scale_o = up && seen;
            m_used += delta;
            seen = seen || first;
            l *= alpha;
            base -= delta;
            // O_t holds P V of the earlier blocks (Q K^T of this block was issued after them).
            if (j > 0 && __any_sync(0xffffffffu, scale_o)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 8) {
                uint32_t o[8];
                tmem_ld8_wait(trow + col_o + c, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st8(trow + col_o + c, o);
              }
            }
          }
          part = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(r[c][2 * i]), __uint_as_float(r[c][2 * i + 1])),
                                          pair(mul), pair(base));
              const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
              part = __fadd2_rn(part, e);
              pk[i] = pack_bf16x2(e.x, e.y);
            }
            tmem_st16(trow + col_s + c * 16, pk);
          }
          if (own_max) break;
          const float sum = part.x + part.y;
          const bool bad = !(sum <= kSpeculationSumBound) ||  // also inf and NaN
                           (!seen && see.x < kbase + kBlockK && see.y > kbase && see.x < see.y);
          if (!__any_sync(0xffffffffu, bad)) break;
          tmem_st_wait();  // the speculative P has landed before it is overwritten
          own_max = true;
        }
        }
        l += part.x + part.y;
        if (kParts == 2 && j == nkt - 1) {
          // The two halves of the row sum, swapped through S column 56 of each half (consumed, and not
          // P's), before the last P lets the next unit's S overwrite it.
          tmem_st1(trow + col_s + 56, l);
          tmem_st_wait();
          tc_fence_before();
          pair_sync(pair_id);
          tc_fence_after();
          l += tmem_ld1_wait(trow + (col_s ^ 64) + 56);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[t]);
      }

      // ------------------------------------------------------------ epilogue
      if (kParts == 2 && ok && __all_sync(0xffffffffu, mbar_try_wait(bar_unit, (k + 1) & 1))) {
        read_unit();
        have_next = true;
      }
      if (nkt > 0) {
        ok = warp_wait(&bar_o[t], nout & 1, wc, kSiteSoftO) && ok;
        ++nout;
        tc_fence_after();
      }
      if (!ok) continue;
      if constexpr (UNIT == 1) {
        mine = {true, m_used, l, nkt, bh, qrow};
        continue;
      }
      // O straight to memory, 16 bytes a store: staging it for a TMA store would need 32 KB that the
      // two tiles share, so one tile's epilogue would wait for the other's, and it costs ring slots.
      const bool any_key = l != 0.f;  // a row without keys has exactly 0; a NaN sum is a NaN result
      const float inv_l = any_key ? 1.f / l : 0.f;
      uint4* orow = reinterpret_cast<uint4*>(p.o + b * p.so.s[2] + h * p.so.s[1] + static_cast<int64_t>(qrow) * p.so.s[0]);
#pragma unroll 1
      for (int c = half * (D / 64); c < (kParts == 2 ? (half + 1) * (D / 64) : D / 32); ++c) {
        uint32_t o[32];
        if (nkt > 0) {
          tmem_ld32(trow + col_o + c * 32, o);
          tmem_ld_wait32(o);
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {  // a row without keys is 0 whatever the accumulator holds
          const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), pair(inv_l));
          pk[i] = any_key ? pack_bf16x2(y.x, y.y) : 0u;
        }
        if (qrow < p.N) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            orow[c * 4 + q4] = make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
        }
      }
      tc_fence_before();
      if (half == 0 && qrow < p.N)
        p.lse[static_cast<size_t>(bh) * p.N + qrow] = any_key ? (m_used + log2f(l)) * kLn2 : -INFINITY;
    }
    if constexpr (UNIT == 1) {
      // The two slots' softmaxes of the same rows, joined: slot 1 leaves m and l (where its Q was) and O (column
      // by column in the ring, which both slots' products have finished with), slot 0 writes the rows. Every
      // softmax thread comes to the barrier, whatever it met before.
      float2* ml = reinterpret_cast<float2*>(sQ + C::kTileBytes);
      float* other = reinterpret_cast<float*>(sRing);
      constexpr int kChunks = D / 32 / kParts;  // of 32 columns of this thread
      if (t == 1) {
        if (mine.nkt > 0) mine.done = mine.done && warp_wait(&bar_o[0], 0, wc, kSiteSoftO);
        if (mine.done && mine.nkt > 0) {
          tc_fence_after();
#pragma unroll 1
          for (int c = half * kChunks; c < (half + 1) * kChunks; ++c) {
            uint32_t o[32];
            tmem_ld32(trow + col_o + c * 32, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) other[(c * 32 + i) * kBlockQ + row] = __uint_as_float(o[i]);
          }
          tc_fence_before();
        }
        if (half == 0) ml[row] = mine.done ? make_float2(mine.m, mine.l) : make_float2(0.f, 0.f);
      }
      asm volatile("bar.sync 15, %0;" ::"n"(32 * R::kSoftWarps) : "memory");
      if (t == 0 && mine.done) {
        tc_fence_after();
        const float2 b1 = ml[row];
        const bool any0 = mine.l != 0.f, any1 = b1.y != 0.f;  // (a NaN counts)
        const float m = any0 && any1 ? fmaxf(mine.m, b1.x) : any0 ? mine.m : b1.x;
        const float a0 = any0 ? ex2_approx(mine.m - m) : 0.f, a1 = any1 ? ex2_approx(b1.x - m) : 0.f;
        const float l = a0 * mine.l + a1 * b1.y;
        const bool any_key = any0 || any1;
        const float f0 = any0 ? a0 / l : 0.f, f1 = any1 ? a1 / l : 0.f;
        uint4* orow = reinterpret_cast<uint4*>(p.o + mine.bh / p.H * p.so.s[2] + mine.bh % p.H * p.so.s[1] +
                                               static_cast<int64_t>(mine.qrow) * p.so.s[0]);
#pragma unroll 1
        for (int c = half * kChunks; c < (half + 1) * kChunks; ++c) {
          uint32_t o[32];
          if (mine.nkt > 0) {
            tmem_ld32(trow + col_o + c * 32, o);
            tmem_ld_wait32(o);
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {  // (a slot without keys counts as 0 whatever it holds)
            float2 y = any0 ? __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), pair(f0))
                            : make_float2(0.f, 0.f);
            if (any1)
              y = __ffma2_rn(make_float2(other[(c * 32 + 2 * i) * kBlockQ + row], other[(c * 32 + 2 * i + 1) * kBlockQ + row]),
                             pair(f1), y);
            pk[i] = pack_bf16x2(y.x, y.y);
          }
          if (mine.qrow < p.N) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4)
              orow[c * 4 + q4] = make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]);
          }
        }
        tc_fence_before();
        if (half == 0 && mine.qrow < p.N)
          p.lse[static_cast<size_t>(mine.bh) * p.N + mine.qrow] = any_key ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Halved units of one tile (1) or units of two (2).  A halved unit takes its blocks in 0.6 of the time of one
// of two tiles, which has twice the rows: better where its longest unit sets the time.  That is so
// while all run at once (full, d = 128, H=2 N=6063: 93 us in units of two tiles, 55 halved), and where the mask
// makes units of long rows differ also in twice as many (causal, H=16 N=2048 35.8 | 27.8; H=6 N=4096 64.3 | 39.0;
// three documents, H=8 N=3737 59.0 | 35.3).  With shorter rows or more units the throughput counts (causal, B=2 H=16
// N=964 d=64 19.6 | 20.5; B=6 H=32 N=7 12.3 | 15.0; B=8 H=16 N=300 17.2 | 23.8; H=32 N=4096 124 | 154).
int unit_tiles(const FwdArgs& a, const ScoreArgs& sc) {
  const long long tiles = static_cast<long long>((a.N + kBlockQ - 1) / kBlockQ) * a.B * a.H;
  return tiles <= ((sc.causal || sc.plan.q) && a.N > 8 * kBlockK ? 2 : 1) * sm_count() ? 1 : 2;
}

template <int D, int MODE, int UNIT>
cudaError_t launch(const FwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  using C = Cfg<D, MODE>;
  using R = Roles<kPartsOf<MODE>>;
  CUtensorMap tq, tk, tv;
  cudaError_t e;
  constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if ((e = make_tmap_4d(&tq, a.q, kBf16, 2, D, a.N, a.H, a.B, a.sq.s, kBoxCols, kBlockQ))) return e;
  if ((e = make_tmap_4d(&tk, a.k, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sk.s, kBoxCols, kBlockK))) return e;
  if ((e = make_tmap_4d(&tv, a.v, kBf16, 2, D, a.N, sc.Hkv, a.B, a.sv.s, kBoxCols, kBlockK))) return e;
  Params p{};
  p.plan = sc.plan;
  p.causal = sc.causal;
  p.N = a.N;
  p.H = a.H;
  p.group = a.H / sc.Hkv;
  p.BH = a.B * a.H;
  p.nunits = (a.N + UNIT * kBlockQ - 1) / (UNIT * kBlockQ);
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  if (MODE >= 2) {
    p.cap_in = 4.f * a.scale / sc.softcap;
    p.cap_out = sc.softcap * kLog2e;
    p.poly = cap_poly(p.cap_out);
  }
  p.slopes = sc.slopes;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.so = a.so;
  p.lse = a.lse;
  p.err_word = a.err_word;
  p.wait_ns = a.dbg.wait_limit_ns;
  auto kern = fwd_scored_kernel<D, MODE, UNIT>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes))) return e;
  // setmaxnreg.inc can only draw on the registers the block was launched with.
  cudaFuncAttributes fattr;
  if ((e = cudaFuncGetAttributes(&fattr, kern))) return e;
  if (static_cast<uint32_t>(fattr.numRegs) * R::kThreads < R::kRegsNeeded) return cudaErrorInvalidConfiguration;
  kern<<<static_cast<unsigned>(p.nunits) * static_cast<unsigned>(p.BH), R::kThreads, C::kSmemBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

template <int D, int UNIT>
cudaError_t launch_unit(const FwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  if (sc.softcap > 0.f)
    return sc.softcap * kLog2e > kBoundedCap ? launch<D, 4, UNIT>(a, sc, stream)
           : sc.slopes                       ? launch<D, 3, UNIT>(a, sc, stream)
                                             : launch<D, 2, UNIT>(a, sc, stream);
  return sc.slopes ? launch<D, 1, UNIT>(a, sc, stream) : launch<D, 0, UNIT>(a, sc, stream);
}

template <int D>
cudaError_t launch_d(const FwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  return unit_tiles(a, sc) == 1 ? launch_unit<D, 1>(a, sc, stream) : launch_unit<D, 2>(a, sc, stream);
}

}  // namespace

cudaError_t launch_fwd_scored(const FwdArgs& a, const ScoreArgs& sc, cudaStream_t stream) {
  return a.d == 64 ? launch_d<64>(a, sc, stream) : launch_d<128>(a, sc, stream);
}

}  // namespace fa
