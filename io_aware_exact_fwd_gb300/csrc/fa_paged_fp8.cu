// The paged key/value cache held in e4m3 codes, with a scale for each block of 16 tokens
// of one head: appending new tokens, and attention of one token a sequence over the
// cache (include/fa.h states both).
//
// The scales are powers of two, 2^e with e the smallest integer such that the block's
// largest value is at most 448 * 2^e.  e4m3 being floating point, that costs no relative
// precision, scaling is exact, and a block whose scale has to grow because a later token is
// larger has its older codes re-coded without loss (a code loses bits only where it falls
// below the type's normal range).
#include "fa_paged.cuh"

namespace fa {
namespace {

// Two codes (low byte first) as fp16, exactly.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}

// ------------------------------------------------------------------------------
// Append.  The tokens of one block and head, new and old, have one scale, so one warp writes them: it reads the
// block's new rows (16 bytes a lane and row part) into registers, finds their largest value, and if the block held
// tokens whose scale is smaller, re-codes those.  A unit is a run of consecutive new tokens and one head of K or
// V; the lanes look the tokens' places up, one each, and a token that is the first new one of its block stands for
// the block.  With few tokens, or many sequences with few each, the runs are of one token, so that blocks do not wait for
// each other; else of up to 31, so that the look-ups are not done for every token that stands for none.  Bound by HBM: 2 bytes read and 1 written a
// value.  Measured, in a graph: 16 prompts, 35k tokens of 8 heads x 128, in 37 us, 5.8 TB/s (runs of 16 tokens 39.7; the next block's rows
// fetched into registers while one is coded 43.8: fewer warps an SM); 64 tokens in 3.1; 2000 sequences a token each in 26.  The time grows with the
// idle sequences between two that a run spans: 35k tokens in the first and the last of 2 sequences 31 us, of 1000 75, of 4000 252.
template <bool FP16>
__device__ __forceinline__ float2 widen(uint32_t two) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&two));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&two));
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// 2^-e of a scale's e, -126 <= e <= 127.
__device__ __forceinline__ float inverse_of_two(int e) { return e == 127 ? 0x1p-127f : power_of_two(-e); }
// The codes of a block's older tokens (rows `row`, row + step, ... below `held`, eight codes a lane) times `by`, each rounded as
// the exact product is: where `by` has 24 bits (a scale that is no power of two) fp32's product would already be rounded,
// so it is cut off, with the last bit set if anything was lost.  A call: blocks that held tokens are few, and in line
// it cost the append of 35k tokens of 8 heads x 128 a tenth of its time (40.7 us for 36.9; 36.5 with fp32's rounding).
__device__ __noinline__ void recode(uint8_t* at, int64_t stride, int row, int step, int held, float by) {
  for (int r = row; r < held; r += step) {
    uint2* place = reinterpret_cast<uint2*>(at + r * stride);
    const uint2 c = *place;
    const uint32_t in[2] = {c.x, c.y};
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 p = widen<true>(codes_to_half2(in[j])), q = widen<true>(codes_to_half2(in[j] >> 16));
      const float x[4] = {p.x, p.y, q.x, q.y};
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = __fmul_rz(x[i], by);
        if (fmaf(x[i], by, -y[i]) != 0.f) y[i] = __uint_as_float(__float_as_uint(y[i]) | 1u);
      }
      out[j] = e4m3x2_bits(y[0], y[1]) | (e4m3x2_bits(y[2], y[3]) << 16);
    }
    *place = make_uint2(out[0], out[1]);
  }
}
// The smallest e >= -126 with top <= 448 * 2^e; top finite and not negative.
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t bits = __float_as_uint(top);
  return max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -126);  // 448 = 1.75 * 2^8
}

template <int D, bool FP16>
__global__ void __launch_bounds__(128, D == 128 ? 6 : 8) append_fp8_kernel(const __grid_constant__ PagedAppendArgs a, int run) {
  constexpr int kLanes = D / 8;             // lanes of a row, 16 bytes of new values each
  constexpr int kRows = 32 / kLanes;        // rows at once
  constexpr int kPasses = 16 / kRows;
  constexpr uint32_t kFinite = FP16 ? 0x7c00u : 0x7f80u;  // |x| below it as bits
  const int lane = threadIdx.x & 31;
  const long long unit = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int sides = 2 * a.c.Hkv;
  const long long line = quotient(unit, sides), first = line * run;
  if (first >= a.T) return;
  const int side = static_cast<int>(unit - line * sides), head = side >> 1;
  const bool is_v = side & 1;
  // Lane x < run: the place of token first + x, if it stands for its block.
  int page = -1, off = 0, count = 0;
  int lo = 0, hi = a.c.B + 1;  // the number of offsets <= first, by the whole warp: 32 probes at once
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step - 1;
    const int k = __popc(__ballot_sync(0xffffffffu, probe < hi && __ldg(a.cu_new + probe) <= first));
    hi = min(hi, lo + (k + 1) * step - 1);
    lo += k * step;
  }
  if (lane < run && first + lane < a.T) {
    const int t = static_cast<int>(first) + lane;
    // From there to the number of offsets <= t: a few further on, and one for every idle sequence between.
    while (lo <= a.c.B && __ldg(a.cu_new + lo) <= t) ++lo;
    if (lo != 0 && lo != a.c.B + 1) {  // (else a row of no sequence)
      const int b = lo - 1, end = __ldg(a.cu_new + lo);
      const long long pos = static_cast<long long>(a.c.seq_lens[b]) - (static_cast<long long>(end) - t);
      const bool stands = (pos & 15) == 0 || t == __ldg(a.cu_new + b);
      if (stands && pos >= 0 && pos < static_cast<long long>(a.c.max_pages) * a.c.page_size) {
        const int place = a.c.per_page(static_cast<int>(pos));
        off = static_cast<int>(pos) - place * a.c.page_size;
        page = a.c.page_table[b * a.c.table_stride + place];
        if (page >= a.c.n_pages) page = -1;
        count = min(16 - (off & 15), min(end, a.T) - t);
      }
    }
  }
  const Strides& sx = is_v ? a.sv : a.sk;
  const Strides& sc = is_v ? a.c.sv : a.c.sk;
  const int row = lane / kLanes, col = lane % kLanes * 8;
  const uint16_t* x = static_cast<const uint16_t*>(is_v ? a.v : a.k) + head * sx.s[0] + col;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + head * sc.s[1] + col;
  float* scales = is_v ? a.c.v_scales : a.c.k_scales;
  const int per_page = a.c.page_size >> 4;
  for (uint32_t todo = __ballot_sync(0xffffffffu, page >= 0); todo; todo &= todo - 1) {
    const int from = __ffs(todo) - 1;
    const int pg = __shfl_sync(0xffffffffu, page, from), of = __shfl_sync(0xffffffffu, off, from),
              n = __shfl_sync(0xffffffffu, count, from);
    const long long t0 = first + from;
    float* scale_at = scales + (static_cast<long long>(pg) * a.c.Hkv + head) * per_page + (of >> 4);
    uint4 v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + row;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < n) v[i] = *reinterpret_cast<const uint4*>(x + (t0 + r) * sx.s[1]);
    }
    const int held = of & 15;  // (the block's new tokens start here: what is before them is older)
    const uint32_t old_bits = held ? __float_as_uint(*scale_at) : 0u;
    // The largest |x|, as the bits of the 16-bit type; infinities and NaN do not count.
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                     __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
    uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
    if (top >= kFinite) {
      top = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
          top = max(top, max(lo < kFinite ? lo : 0u, hi < kFinite ? hi : 0u));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    int e = exponent_for(widen<FP16>(top).x);
    bool grows = false;
    if (held) {
      // A scale that is no power of two (not one of this kernel's) counts as the next larger one, up to 2^127.
      const int e_old = min(static_cast<int>((old_bits >> 23) & 0xffu) - 127 + ((old_bits & 0x7fffffu) ? 1 : 0), 127);
      grows = e > e_old || (old_bits & 0x7fffffu);
      e = max(e, max(e_old, -126));
    }
    if (grows)
      recode(cache + pg * sc.s[2] + (of & ~15) * sc.s[0], sc.s[0], row, kRows, held, __uint_as_float(old_bits) * inverse_of_two(e));
    const float inv = inverse_of_two(e);
    uint8_t* dst = cache + pg * sc.s[2] + of * sc.s[0];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kRows + row;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = widen<FP16>(w[j]);
        c[j] = e4m3x2_bits(f.x * inv, f.y * inv);
      }
      if (r < n) *reinterpret_cast<uint2*>(dst + r * sc.s[0]) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    __syncwarp();  // every lane has the old scale
    if (lane == 0) *scale_at = power_of_two(e);
  }
}

// ------------------------------------------------------------------------------
// Decode: as the 16-bit cache's (fa_paged.cu has the division of the work, the ring and the join), with half the
// bytes to read a token and so half the time for the arithmetic on it.
//
// Products are m16n8k16 instructions in fp16 with the codes widened to fp16 (exact, one instruction for two).  The 16 rows
// are K's tokens and V's columns, the 8 columns the heads, S^T = K Q^T and O^T += V^T P^T: with heads as rows, as in the
// 16-bit decode, half of a product and of the softmax is for rows of zeros where up to 8 heads share a key/value head, and the tensor
// instructions (11 cycles each and scheduler) would take half the time that HBM leaves.  (The 8-bit m16n8k32 form is no way
// round the widening: it takes 29 cycles here, conversions and two fp16 products.)
//
// q, whatever its type, comes in as fp16 times a power of two of its head, with its largest entry in [2^14, 2^15) (below that in rows
// under 2^-112), so that entries down to 2^-28 of the largest keep all their bits.  K's scale multiplies the finished scores of its block.  V's
// cannot follow its products, which sum over blocks: it goes into the weights.  A head therefore has two running references: m
// for its scores, under which l sums the weights, and mv for scores + log2 of the block's V scale, under which the
// weights are rounded to fp16 for P V.  Both are only raised when they have to be: a tile's weights are made under the old
// ones and kept if those for P V sum up to 2^15 at most and those for l to 2^60; else the maxima are found (shuffles over 8 lanes) and
// mv set 7 below its own.  So weights times scales keep all their bits down to 2^-21 of the largest, and none above 2^-32 is
// lost.  O goes back to the reference m where a segment ends.
//
// Fragments.  An 8 x 8 matrix of 16-bit units that ldmatrix loads is one of 8 tokens x 16 codes.  For K a thread gets four
// neighbouring codes of a token, columns 4t .. 4t + 3 of 16: the products take them as their columns {2t, 2t + 1} and
// {2t + 8, 2t + 9}, and Q's fragments are put in the same order.  For V, transposed, it gets two codes of two tokens: a
// byte shuffle makes pairs of tokens, of the even column 2g (row g of the product) and the odd one (row g + 8).  The weights
// come out with a token's heads side by side and go in with a head's tokens side by side: movmatrix transposes them.
//
// A warp's part of a tile is 32 tokens for 8 or 16 query heads; where two key/value heads are a unit, half of the warps
// have the one and half the other.  More heads a key/value head are chunks of 16, head units of their
// own, whose tiles come from L2 for all but the first.  (Two or three groups of four warps that work on the same stages, so
// that the cache is read once, ran at 3.6 TB/s of codes with 32 heads and 1.9 with 40: no more than chunks reach
// with nothing in L2, for their arithmetic is the same and one CTA an SM hides less of it.)
//
// Measured, in a graph: 64 sequences of 1 .. 16384 tokens (0.96 GB), H=32 over 8 heads, d=128, capped: 148-151 us, 6.4-6.5 TB/s (heads
// as rows 197); one of 131072 tokens, 16 heads of d=64 beside each other, biased: 52-57 us, 4.8-5.2 TB/s; 24 of 2000 .. 8000 tokens, 40 heads over one: 25.3 (chunks of 8 heads 26.5, and 147
// for 90 at 32000 tokens each); one of 900 tokens, H=16 over 4: 7.5, two launches and three waits on memory.
enum : uint32_t { kSite8Load = 0x141, kSite8Full = 0x341 };

template <int D, int NH, bool TWO>
struct Dec8Cfg {
  static constexpr int kWarpHeads = 8 * NH;                  // query heads of a warp
  static constexpr int kHeads = TWO ? 16 : kWarpHeads;       // of a unit: a chunk, or (TWO) eight of each of two key/value heads
  static constexpr int kRow = TWO && D == 64 ? 128 : D;      // bytes of a tile's row: a token's codes of one head, or of both
  static constexpr int kTile = TWO && D == 128 ? 64 : 128;   // tokens per tile
  static constexpr int kPart = kTile / (TWO ? 2 : 4);        // of a warp
  static constexpr int kBlocksOfTile = kTile / 16;
  static constexpr int kHalf = kTile * D * (TWO ? 2 : 1);    // K or V of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kPerSm = NH * D <= 128 ? 3 : 2;
  static constexpr int kStages = (kPerSm == 3 ? 65536 : 98304) / kStage;
  static constexpr int kORow = D + (NH == 1 ? 8 : 0);        // of a head's O; 8 more: fewer bank conflicts, where a stage has the room
  static constexpr int kO = 4 * kWarpHeads * kORow * 4;      // the warps' O, in a segment's last stage
  static constexpr int kQStride = D * 2 + 32;                // bytes; 8-byte loads of 4 rows meet every bank once
  static constexpr int kSets = TWO ? 4 : 2;                  // of scales: K's and V's, of one head and the other
  static constexpr int kScaleLanes = kSets * kBlocksOfTile;
  static constexpr int kScaleOff = kStages * kStage;         // the scales of each stage
  static constexpr int kQOff = kScaleOff + kStages * kScaleLanes * 4;
  static constexpr int kQsOff = kQOff + kHeads * kQStride;   // q's powers of two
  static constexpr int kMlOff = kQsOff + kHeads * 4;         // (m, l) of each warp's heads
  static constexpr int kBarOff = kMlOff + 4 * kWarpHeads * 8;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kSmemBytes = kMiscOff + 64 + 1024;
  static_assert(!TWO || NH == 1, "a warp has heads of one key/value head");
  static_assert(kO <= kStage, "the warps' O fits a stage");
  static_assert(kQOff % 16 == 0 && kQsOff % 16 == 0 && kMlOff % 8 == 0 && kBarOff % 8 == 0 && kScaleLanes <= 32, "layout");
};

// mma16816 in fp16 of registers alone: the compiler may move it.
__device__ __forceinline__ void mma_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit numbers, two neighbours of row lane / 4 a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float2 ex2_pair(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ float2 max_pair(float2 x, float2 y) { return make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y)); }
__device__ __forceinline__ float2 minus(float2 x, float2 y) { return __fadd2_rn(x, make_float2(-y.x, -y.y)); }

// Where the 16-byte piece `chunk` of a row stands in a tile whose rows of 64 or 128 bytes TMA swizzled in spans of their length.
template <int ROW>
__device__ __forceinline__ uint32_t piece_of(int row, int chunk) {
  if constexpr (ROW == 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
  else return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <int D, int NH, bool TWO, bool FP16>
__global__ void __launch_bounds__(kDecThreads, Dec8Cfg<D, NH, TWO>::kPerSm)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ DecParams p) {
  using C = Dec8Cfg<D, NH, TWO>;
  constexpr int kTile = C::kTile, kHeads = C::kHeads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* bar_empty = bar_full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  long long* s_sums = reinterpret_cast<long long*>(smem + C::kMlOff);
  int* s_start = reinterpret_cast<int*>(smem + C::kMiscOff + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = units_of(p);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_full[s], 1 + C::kScaleLanes);
      mbar_init(&bar_empty[s], kConsumers);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  Place<kTile> at;
  long long w0, w1;
  const int cta = static_cast<int>(blockIdx.x);
  if (!share_of_tiles<kConsumers + 1>(p, units, s_sums, s_start, at, w0, w1)) return;
  const WaitCtl wc{abort_flag, p.err_word, p.wait_ns};

  if (warp == kConsumers) {
    // ------------------------------------------------------------- producer warp
    // Lane x: a block of the tile, of K or V, of the unit's one head or of the other.  It fetches the block's scale, and
    // if a piece (the tokens of one page in the tile) starts with its block, the piece's codes, unless they come with the other
    // head's in one row.  Past the sequence's end, and for a page index outside the cache, the page coordinate n_pages, out of
    // bounds, fills the piece with zeros; such a block's scale is 0.
    const bool mine = lane < C::kScaleLanes, is_v = (lane / C::kBlocksOfTile) & 1;
    const int block = lane % C::kBlocksOfTile, per_page = p.c.page_size >> 4, second = lane / (2 * C::kBlocksOfTile);
    const float* scales = is_v ? p.c.v_scales : p.c.k_scales;
    auto page_at = [&](const Place<kTile>& x, int& row) -> int {
      const int tok = x.t * kTile + block * 16;
      const int place = p.c.per_page(tok);
      row = tok - place * p.c.page_size;
      int page = p.c.n_pages;
      if (mine && tok < x.n) page = p.c.page_table[x.b * p.c.table_stride + place];
      return page < 0 || page >= p.c.n_pages ? p.c.n_pages : page;
    };
    const bool starts = mine && block * 16 % p.piece == 0 && (C::kRow == D || second == 0);
    int issued = 0, row;
    int page = page_at(at, row);
    bool ok = true;
    for (long long w = w0; w < w1; ++w, ++issued) {
      const int slot = issued % C::kStages;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_empty[slot], ((issued / C::kStages) & 1) ^ 1, wc, kSite8Load))))
        break;
      if (lane == 0) mbar_arrive_expect_tx(&bar_full[slot], C::kStage);
      __syncwarp();
      const int hk = TWO ? 2 * at.u + second : at.u / p.chunks;
      if (starts)
        tma_load_4d(smem + slot * C::kStage + (is_v ? C::kHalf : 0) + (second * kTile + block * 16) * C::kRow, is_v ? &tm_v : &tm_k,
                    &bar_full[slot], 0, row, C::kRow == D ? hk : at.u, page);
      if (mine) {
        const bool real = page < p.c.n_pages;
        const float* src = scales + (real ? (static_cast<long long>(page) * p.c.Hkv + hk) * per_page + (row >> 4) : 0);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         smem_u32(smem + C::kScaleOff + (slot * C::kScaleLanes + lane) * 4)),
                     "l"(src), "r"(real ? 4 : 0)
                     : "memory");
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bar_full[slot])) : "memory");
      }
      if (w + 1 < w1) {
        if (++at.t == at.T) at.next_unit(p.c, units);
        page = page_at(at, row);
      }
    }
    if (!ok || *abort_flag)  // the copies in flight land before the block's shared memory goes
      for (int t = max(0, issued - C::kStages); t < issued; ++t)
        mbar_wait_drain(&bar_full[t % C::kStages], (t / C::kStages) & 1, p.wait_ns);
    __syncwarp();
    return;
  }

  // ---------------------------------------------------------------- consumer warps
  const uint32_t ring = smem_u32(smem);
  // TWO: warps 0 and 1 have the unit's first key/value head, 2 and 3 the second.
  constexpr int kWarpHeads = C::kWarpHeads;
  const int kv = TWO ? warp >> 1 : 0, row0 = 8 * kv, part0 = C::kPart * (TWO ? warp & 1 : warp);  // first row and token in the tile
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMlOff);  // [warp][head]
  float* s_qs = reinterpret_cast<float*>(smem + C::kQsOff);
  uint8_t* s_q = smem + C::kQOff;
  // In fragments of scores this thread has tokens gr and gr + 8 of 16 and heads gc and gc + 1 of 8.
  const int gr = lane >> 2, gc = 2 * (lane & 3);
  int slot = 0;
  uint32_t phase = 0;
  bool first_segment = true;
  // A segment's Q rows (those past the group's heads: zeros) and slopes, fetched into registers while
  // the segment before it ends.
  constexpr int kPieces = kHeads * (D / 8);             // of 16 bytes
  constexpr int kQPer = (kPieces + 127) / 128;          // a thread
  uint4 q_next[kQPer];
  float2 slope_next[NH];
  // The query head of row r of a unit, or -1.  (TWO: eight rows for each of the two key/value heads, p.group of them real.)
  auto head_of = [&](const Place<kTile>& x, int r) {
    if constexpr (TWO) return (r & 7) < p.group ? (2 * x.u + (r >> 3)) * p.group + (r & 7) : -1;
    const int in_group = (x.u % p.chunks) * kHeads + r;
    return in_group < p.group ? (x.u / p.chunks) * p.group + in_group : -1;
  };
  auto fetch_q = [&](const Place<kTile>& x) {
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int y = threadIdx.x + i * 128, r = y / (D / 8), c = y % (D / 8);
      const int head = y < kPieces ? head_of(x, r) : -1;
      q_next[i] = make_uint4(0u, 0u, 0u, 0u);
      if (head >= 0) q_next[i] = *reinterpret_cast<const uint4*>(p.q + x.b * p.sq.s[1] + head * p.sq.s[0] + c * 8);
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      slope_next[h] = pair(0.f);
      if (p.slopes) {
        const int one = head_of(x, row0 + 8 * h + gc), two = head_of(x, row0 + 8 * h + gc + 1);
        if (one >= 0) slope_next[h].x = p.slopes[one] * -kLog2e;
        if (two >= 0) slope_next[h].y = p.slopes[two] * -kLog2e;
      }
    }
  };
  fetch_q(at);
  for (long long w = w0; w < w1;) {
    // ---- a segment: tiles [at.t, at.t + count) of one head unit
    const int count = static_cast<int>(min(static_cast<long long>(at.T - at.t), w1 - w));
    const bool whole = count == at.T;
    float2 slope2[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) slope2[h] = slope_next[h];
    // Q to fp16 in [2^14, 2^15) of its row's largest entry.
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int y = threadIdx.x + i * 128, r = y / (D / 8), c = y % (D / 8);
      const uint32_t in[4] = {q_next[i].x, q_next[i].y, q_next[i].z, q_next[i].w};
      float2 f[4];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[j] = widen<FP16>(in[j]);
        top = fmaxf(top, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
      }
#pragma unroll
      for (int x = 1; x < D / 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -126);
      const float by = power_of_two(-e);
      uint4 out;
      out.x = pack2<true>(f[0].x * by, f[0].y * by);
      out.y = pack2<true>(f[1].x * by, f[1].y * by);
      out.z = pack2<true>(f[2].x * by, f[2].y * by);
      out.w = pack2<true>(f[3].x * by, f[3].y * by);
      if (y < kPieces) {
        *reinterpret_cast<uint4*>(s_q + r * C::kQStride + c * 16) = out;
        if (c == 0) s_qs[r] = power_of_two(e);
      }
    }
    consumers_sync();
    // B fragments of Q^T in the order of K's codes: four neighbouring columns of head gr.
    auto load_q = [&](int h, int kk) {
      return *reinterpret_cast<const uint2*>(s_q + (row0 + 8 * h + gr) * C::kQStride + kk * 32 + 4 * gc);
    };
    constexpr bool kHoldQ = NH * D <= 128;  // in registers
    uint2 qf[kHoldQ ? NH : 1][kHoldQ ? D / 16 : 1];
    if constexpr (kHoldQ) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) qf[h][kk] = load_q(h, kk);
    }
    float o[D / 16][NH][4];  // columns 2 gr and 2 gr + 1 of 16 for heads gc, gc + 1: {even, head gc}, {even, gc + 1}, {odd, gc}, ...
    float2 m[NH], mv[NH], l[NH], to_log2[NH];  // of heads gc and gc + 1; l over this thread's tokens
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      m[h] = mv[h] = pair(kNoScore);
      l[h] = pair(0.f);
      to_log2[h] = __fmul2_rn(pair(p.cap_out > 0.f ? p.cap_in : p.scale_log2), make_float2(s_qs[row0 + 8 * h + gc], s_qs[row0 + 8 * h + gc + 1]));
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[c][h][0] = o[c][h][1] = o[c][h][2] = o[c][h][3] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      // A wait that gave up (the block is aborting) skips the tile but stays in step with the other
      // warps, which it meets at barriers.
      const bool landed = __all_sync(0xffffffffu, mbar_wait(&bar_full[slot], phase, wc, kSite8Full));
      // The warp's head: a tile of its own, or the row's second half.
      const uint32_t kb = ring + slot * C::kStage + (TWO && C::kRow == D ? kv * kTile * C::kRow : 0), vb = kb + C::kHalf;
#pragma unroll 1
      for (int sub = 0; sub < C::kPart; sub += 32) {
        const int key0 = (at.t + i) * kTile + part0 + sub;  // 32 tokens from here
        if (!landed || key0 >= at.n) break;
        const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff) + slot * C::kScaleLanes +
                          2 * kv * C::kBlocksOfTile + (part0 + sub) / 16;
        // What this lane addresses for ldmatrix.
        const int frow = part0 + sub + (lane & 15), fchunk = (lane >> 4) + (C::kRow == D ? 0 : 4 * kv);
        // S^T = K Q^T of two blocks of 16 tokens.
        float s[2][NH][4] = {};
#pragma unroll
        for (int c2 = 0; c2 < D / 32; ++c2) {
          uint32_t b4[2][4];
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) ldsm4(b4[nb], kb + piece_of<C::kRow>(frow + 16 * nb, 2 * c2 + fchunk));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int kk = 2 * c2 + half;
            uint2 b[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) b[h] = kHoldQ ? qf[kHoldQ ? h : 0][kHoldQ ? kk : 0] : load_q(h, kk);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
              const uint32_t x = b4[nb][2 * half], y = b4[nb][2 * half + 1];
              const uint32_t a4[4] = {codes_to_half2(x), codes_to_half2(y), codes_to_half2(x >> 16), codes_to_half2(y >> 16)};
#pragma unroll
              for (int h = 0; h < NH; ++h) mma_half(s[nb][h], a4, b[h].x, b[h].y);
            }
          }
        }
        // Scales; a block past the end has whatever its page holds there.
        const bool ragged = key0 + 32 > at.n;
        float ks[2], lgv[2];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          const bool inside = key0 + 16 * nb < at.n;
          ks[nb] = inside ? sc[nb] : 0.f;
          lgv[nb] = inside ? __log2f(sc[C::kBlocksOfTile + nb]) : 0.f;
        }
        // Scores in log2 units: x[block][h][token gr or gr + 8], of heads gc and gc + 1.
        float2 x[2][NH][2];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float2 f = __fmul2_rn(to_log2[h], pair(ks[nb]));
            x[nb][h][0] = __fmul2_rn(make_float2(s[nb][h][0], s[nb][h][1]), f);
            x[nb][h][1] = __fmul2_rn(make_float2(s[nb][h][2], s[nb][h][3]), f);
          }
        if (p.cap_out > 0.f) {
          // As in the 16-bit decode: relative to the score while |x| < 2.
          uint32_t bits = 0;
#pragma unroll
          for (int y = 0; y < 4 * NH; ++y) bits = or_bits(bits, x[y & 1][y >> 2][(y >> 1) & 1]);
          const bool any_far = __any_sync(0xffffffffu, bits & kReachesTwo);
#pragma unroll
          for (int y = 0; y < 4 * NH; ++y) {
            float2& u = x[y & 1][y >> 2][(y >> 1) & 1];
            float2 z = __fmul2_rn(u, tanh_over_x(u, p.poly));
            if (any_far) {
              const float2 far = tanh_any(u, p.cap_out, pair(0.f));
              z = make_float2(fabsf(u.x) < 2.f ? z.x : far.x, fabsf(u.y) < 2.f ? z.y : far.y);
            }
            u = z;
          }
        }
        if (p.slopes) {
          const float back = static_cast<float>(at.n - 1 - key0 - gr);
#pragma unroll
          for (int y = 0; y < 4 * NH; ++y) {
            float2& u = x[y & 1][y >> 2][(y >> 1) & 1];
            u = __ffma2_rn(slope2[y >> 2], pair(back - (16 * (y & 1) + 8 * ((y >> 1) & 1))), u);
          }
        }
        if (ragged) {
#pragma unroll
          for (int y = 0; y < 4 * NH; ++y)
            if (key0 + gr + 16 * (y & 1) + 8 * ((y >> 1) & 1) >= at.n) x[y & 1][y >> 2][(y >> 1) & 1] = pair(-INFINITY);
        }
        // Weights under the references so far: for l, and times 2^(lgv + m - mv) for P V.  That factor stays below 2^100, so that a
        // weight that is 0 in fp32 would be under 2^-26 in P V.
        uint32_t pf[2][NH][2];
        float2 sum[NH];
        bool fits = true;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float2 sum_v = pair(0.f);
          sum[h] = pair(0.f);
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            const float2 to_v = __fadd2_rn(minus(m[h], mv[h]), pair(lgv[nb])), by = ex2_pair(to_v);
            fits = fits && to_v.x <= 100.f && to_v.y <= 100.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = ex2_pair(minus(x[nb][h][e], m[h])), v = __fmul2_rn(y, by);
              sum[h] = __fadd2_rn(sum[h], y);
              sum_v = __fadd2_rn(sum_v, v);
              pf[nb][h][e] = pack2<true>(v.x, v.y);
            }
          }
          fits = fits && fmaxf(sum_v.x, sum_v.y) <= 32768.f && fmaxf(sum[h].x, sum[h].y) <= 0x1p60f;
        }
        if (!__all_sync(0xffffffffu, fits)) {
          // New references, O and l brought to them, and the weights again, each kind from the scores.
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            float2 mx = pair(-INFINITY), mxv = pair(-INFINITY);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
              const float2 top = max_pair(x[nb][h][0], x[nb][h][1]);
              mx = max_pair(mx, top);
              mxv = max_pair(mxv, __fadd2_rn(top, pair(lgv[nb])));
            }
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) {
              mx = max_pair(mx, make_float2(__shfl_xor_sync(0xffffffffu, mx.x, y), __shfl_xor_sync(0xffffffffu, mx.y, y)));
              mxv = max_pair(mxv, make_float2(__shfl_xor_sync(0xffffffffu, mxv.x, y), __shfl_xor_sync(0xffffffffu, mxv.y, y)));
            }
            mx = max_pair(mx, m[h]);
            mxv = max_pair(__fadd2_rn(mxv, pair(-7.f)), mv[h]);
            const float2 alpha = ex2_pair(minus(m[h], mx)), alpha_v = ex2_pair(minus(mv[h], mxv));
            m[h] = mx;
            mv[h] = mxv;
            l[h] = __fmul2_rn(l[h], alpha);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][h][0] *= alpha_v.x;
              o[c][h][1] *= alpha_v.y;
              o[c][h][2] *= alpha_v.x;
              o[c][h][3] *= alpha_v.y;
            }
            sum[h] = pair(0.f);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                sum[h] = __fadd2_rn(sum[h], ex2_pair(minus(x[nb][h][e], mx)));
                const float2 v = ex2_pair(__fadd2_rn(x[nb][h][e], minus(pair(lgv[nb]), mxv)));
                pf[nb][h][e] = pack2<true>(v.x, v.y);
              }
          }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          l[h] = __fadd2_rn(l[h], sum[h]);
#pragma unroll
          for (int nb = 0; nb < 2; ++nb) {
            pf[nb][h][0] = transposed(pf[nb][h][0]);
            pf[nb][h][1] = transposed(pf[nb][h][1]);
          }
        }
        // O^T += V^T P^T.  Tokens past the end: their weight is 0, but what the page holds there may be anything.
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          const int left = at.n - (key0 + 16 * nb + gc);
          const uint32_t keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
          const uint32_t keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
#pragma unroll
          for (int c2 = 0; c2 < D / 32; ++c2) {
            uint32_t b4[4];
            ldsm4_t(b4, vb + piece_of<C::kRow>(frow + 16 * nb, 2 * c2 + fchunk));
            if (ragged) {
              b4[0] &= keep0;
              b4[1] &= keep1;
              b4[2] &= keep0;
              b4[3] &= keep1;
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t u = __byte_perm(b4[2 * half], 0, 0x3120), v = __byte_perm(b4[2 * half + 1], 0, 0x3120);
              const uint32_t a4[4] = {codes_to_half2(u), codes_to_half2(u >> 16), codes_to_half2(v), codes_to_half2(v >> 16)};
#pragma unroll
              for (int h = 0; h < NH; ++h) mma_half(o[2 * c2 + half][h], a4, pf[nb][h][0], pf[nb][h][1]);
            }
          }
        }
      }
      if (i + 1 < count) {  // the segment's last stage is kept for the warps' meeting below
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_empty[slot]);
        if (++slot == C::kStages) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }

    Place<kTile> next = at;
    if (w + count < w1) {
      next.next_unit(p.c, units);
      fetch_q(next);
    }
    // ---- the four warps' parts, joined
    float* s_o = reinterpret_cast<float*>(smem + slot * C::kStage);  // [warp][head][kORow]
    const int part_rows = TWO ? p.part_rows : kHeads;
    float* part = p.part + static_cast<size_t>(2 * cta + (first_segment ? 0 : 1)) * part_rows * (D + 2);
    consumers_sync();  // every warp is done with the stage
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float2 all = l[h];
#pragma unroll
      for (int y = 4; y < 32; y <<= 1)
        all = __fadd2_rn(all, make_float2(__shfl_xor_sync(0xffffffffu, all.x, y), __shfl_xor_sync(0xffffffffu, all.y, y)));
      const int head = warp * kWarpHeads + 8 * h + gc;
      if (gr == 0) {
        s_ml[head] = make_float2(m[h].x, all.x);
        s_ml[head + 1] = make_float2(m[h].y, all.y);
      }
      const float2 back = ex2_pair(minus(mv[h], m[h]));
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float* dst = s_o + head * C::kORow + 16 * c + 2 * gr;
        const float(&x)[4] = o[c][h];
        *reinterpret_cast<float2*>(dst) = make_float2(x[0] * back.x, x[2] * back.x);
        *reinterpret_cast<float2*>(dst + C::kORow) = make_float2(x[1] * back.y, x[3] * back.y);
      }
    }
    consumers_sync();
    constexpr int kThreadsOfRow = 128 / kHeads;
    const int r = threadIdx.x / kThreadsOfRow, in_row = threadIdx.x % kThreadsOfRow;
    const int head = head_of(at, r);
    if (head >= 0) {
      // The row's parts: all four warps', or (TWO) those of its key/value head's two.
      constexpr int kParts = TWO ? 2 : 4;
      const int from = TWO ? (r >> 3) * 2 * kWarpHeads + (r & 7) : r;
      const int part_row = TWO ? (r >> 3) * p.group + (r & 7) : r;
      float M = kNoScore, L = 0.f, wgt[kParts];
#pragma unroll
      for (int x = 0; x < kParts; ++x) M = fmaxf(M, s_ml[x * kWarpHeads + from].x);
#pragma unroll
      for (int x = 0; x < kParts; ++x) {
        const float2 ml = s_ml[x * kWarpHeads + from];
        wgt[x] = ex2_approx(ml.x - M);
        L += ml.y * wgt[x];
      }
      const float inv = whole ? 1.f / L : 1.f;
#pragma unroll
      for (int c = 0; c < D / (4 * kThreadsOfRow); ++c) {
        const int col = 4 * (in_row + kThreadsOfRow * c);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
          const float4 v = *reinterpret_cast<const float4*>(s_o + (x * kWarpHeads + from) * C::kORow + col);
          acc.x = fmaf(wgt[x], v.x, acc.x);
          acc.y = fmaf(wgt[x], v.y, acc.y);
          acc.z = fmaf(wgt[x], v.z, acc.z);
          acc.w = fmaf(wgt[x], v.w, acc.w);
        }
        if (whole)
          *reinterpret_cast<uint2*>(p.o + at.b * p.so.s[1] + head * p.so.s[0] + col) =
              make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
        else
          *reinterpret_cast<float4*>(part + part_row * D + col) = acc;
      }
      if (in_row == 0) {
        if (whole)
          p.lse[static_cast<size_t>(at.b) * p.H + head] = (M + log2f(L)) * kLn2;
        else
          *reinterpret_cast<float2*>(part + part_rows * D + 2 * part_row) = make_float2(M, L);
      }
    }
    fence_proxy_async_smem();  // the stage goes back to the TMA producer
    consumers_sync();          // (also: s_ml and Q are free)
    if (lane == 0) mbar_arrive(&bar_empty[slot]);
    if (++slot == C::kStages) {
      slot = 0;
      phase ^= 1u;
    }
    w += count;
    first_segment = false;
    at = next;
  }
}

// Rows of a part: the heads of a unit (TWO: those that there are).
template <class C, bool TWO>
int part_rows_of(int group) {
  return TWO ? 2 * group : C::kHeads;
}

template <int D, int NH, bool TWO, bool FP16>
cudaError_t launch_decode8(const PagedDecodeArgs& a, cudaStream_t stream) {
  using C = Dec8Cfg<D, NH, TWO>;
  DecParams p = decode_params(a, C::kHeads, C::kTile, part_rows_of<C, TWO>(a.H / a.c.Hkv), C::kPerSm);
  p.two = TWO;
  CUtensorMap tk, tv;
  cudaError_t e;
  constexpr auto kSwizzle = C::kRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // L2 fetches no more than a row where the rows of a head lie apart (fa_paged.cu).
  auto map = [&](CUtensorMap* t, const void* x, const Strides& s) {
    constexpr bool kBoth = C::kRow != D;
    const auto fetch = s.s[0] == C::kRow ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                       : C::kRow == 128  ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                         : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    const int64_t strides[3] = {s.s[0], kBoth ? 2 * s.s[1] : s.s[1], s.s[2]};
    return make_tmap_4d(t, x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, C::kRow, a.c.page_size, kBoth ? a.c.Hkv / 2 : a.c.Hkv,
                        a.c.n_pages, strides, C::kRow, p.piece, kSwizzle, fetch);
  };
  if ((e = map(&tk, a.c.k, a.c.sk))) return e;
  if ((e = map(&tv, a.c.v, a.c.sv))) return e;
  auto kern = decode_fp8_kernel<D, NH, TWO, FP16>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes))) return e;
  kern<<<static_cast<unsigned>(sm_count() * C::kPerSm), kDecThreads, C::kSmemBytes, stream>>>(tk, tv, p);
  if ((e = cudaGetLastError())) return e;
  return launch_join<D, FP16>(p, C::kHeads, stream);
}

template <int D, bool FP16>
cudaError_t launch_decode8_heads(const PagedDecodeArgs& a, cudaStream_t stream) {
  if (a.H / a.c.Hkv > 8) return launch_decode8<D, 2, false, FP16>(a, stream);
  // Rows that lie apart, each beside the next head's: two heads a unit, so that HBM is asked for both at once (64 sequences
  // of 1 .. 16384 tokens, 8 heads x 128: 152 us, 161 one by one; 131072 tokens of 16 heads x 64: 52, 91 one by one).
  const Strides &k = a.c.sk, &v = a.c.sv;
  if (a.c.Hkv % 2 == 0 && k.s[1] == D && v.s[1] == D && k.s[0] >= 2 * D && v.s[0] >= 2 * D)
    return launch_decode8<D, 1, true, FP16>(a, stream);
  return launch_decode8<D, 1, false, FP16>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append_fp8(const PagedAppendArgs& a, cudaStream_t stream) {
  const long long sides = 2LL * a.c.Hkv;
  // About two blocks a warp (each sequence's tokens are a block for every 16, and one more), one where there are few.
  const int run = a.T * sides <= 64LL * sm_count() ? 1 : std::max(1, static_cast<int>(32LL * a.T / (a.T + 16LL * a.c.B)));
  const long long warps = (a.T + run - 1LL) / run * sides;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  auto kern = a.c.d == 64 ? (a.fp16 ? append_fp8_kernel<64, true> : append_fp8_kernel<64, false>)
                          : (a.fp16 ? append_fp8_kernel<128, true> : append_fp8_kernel<128, false>);
  kern<<<grid, 128, 0, stream>>>(a, run);
  return cudaGetLastError();
}

// Whatever the cache's layout.  Both d have the same builds' rows, but for groups past 8.
size_t paged_decode_fp8_workspace(int B, int H, int Hkv, int d) {
  const int group = H / Hkv;
  using One = Dec8Cfg<128, 1, false>;
  using Two = Dec8Cfg<128, 1, true>;
  static_assert(One::kPerSm == Dec8Cfg<64, 1, false>::kPerSm && Two::kPerSm == Dec8Cfg<64, 1, true>::kPerSm, "as said");
  int rows;
  if (group > 8) rows = d == 64 ? Dec8Cfg<64, 2, false>::kPerSm * 16 : Dec8Cfg<128, 2, false>::kPerSm * 16;
  else rows = std::max(One::kPerSm * One::kHeads, Hkv % 2 == 0 ? Two::kPerSm * part_rows_of<Two, true>(group) : 0);
  return decode_workspace(rows, B, d);
}

cudaError_t launch_paged_decode_fp8(const PagedDecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return a.fp16 ? launch_decode8_heads<64, true>(a, stream) : launch_decode8_heads<64, false>(a, stream);
  return a.fp16 ? launch_decode8_heads<128, true>(a, stream) : launch_decode8_heads<128, false>(a, stream);
}

}  // namespace fa
