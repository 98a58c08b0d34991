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
// the block.  With few tokens the runs are of one token, so that blocks do not wait for each other; with many of 16, so
// that the look-ups are not done for every token that stands for none.  Bound by HBM: 2 bytes read and 1 written a
// value.
template <bool FP16>
__device__ __forceinline__ float2 widen(uint32_t two) {
  if constexpr (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&two));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&two));
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The smallest e >= -126 with top <= 448 * 2^e; top finite and not negative.
__device__ __forceinline__ int exponent_for(float top) {
  const uint32_t bits = __float_as_uint(top);
  return max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -126);  // 448 = 1.75 * 2^8
}

template <int D, bool FP16>
__global__ void __launch_bounds__(128) append_fp8_kernel(const __grid_constant__ PagedAppendArgs a, int run) {
  constexpr int kLanes = D / 8;             // lanes of a row, 16 bytes of new values each
  constexpr int kRows = 32 / kLanes;        // rows at once
  constexpr int kPasses = 16 / kRows;
  constexpr uint32_t kFinite = FP16 ? 0x7c00u : 0x7f80u;  // |x| below it as bits
  const int lane = threadIdx.x & 31;
  const long long unit = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  const int sides = 2 * a.c.Hkv;
  const long long first = unit / sides * run;
  if (first >= a.T) return;
  const int side = static_cast<int>(unit % sides), head = side >> 1;
  const bool is_v = side & 1;
  // Lane x < run: the place of token first + x, if it stands for its block.
  int page = -1, off = 0, count = 0;
  const int t = static_cast<int>(first) + lane;
  if (lane < run && t < a.T) {
    int lo = 0, hi = a.c.B + 1;  // the number of offsets <= t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.cu_new + mid) <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo != 0 && lo != a.c.B + 1) {  // (else a row of no sequence)
      const int b = lo - 1, end = __ldg(a.cu_new + lo);
      const long long pos = static_cast<long long>(a.c.seq_lens[b]) - (static_cast<long long>(end) - t);
      const bool stands = (pos & 15) == 0 || t == __ldg(a.cu_new + b);
      if (stands && pos >= 0 && pos < static_cast<long long>(a.c.max_pages) * a.c.page_size) {
        off = static_cast<int>(pos) % a.c.page_size;
        page = a.c.page_table[b * a.c.table_stride + static_cast<int>(pos) / a.c.page_size];
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
    if (held) {
      // A scale that is no power of two (not one of this kernel's) counts as the next larger one.
      const int e_old = min(static_cast<int>((old_bits >> 23) & 0xffu) - 127 + ((old_bits & 0x7fffffu) ? 1 : 0), 126);
      const bool grows = e > e_old || (old_bits & 0x7fffffu);
      e = max(e, max(e_old, -126));
      if (grows) {
        const float by = __uint_as_float(old_bits) * power_of_two(-e);
        for (int r = row; r < held; r += kRows) {
          uint2* at = reinterpret_cast<uint2*>(cache + pg * sc.s[2] + ((of & ~15) + r) * sc.s[0]);
          uint2 c = *at;
          uint32_t out[2];
          const uint32_t in[2] = {c.x, c.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 p = widen<true>(codes_to_half2(in[j])), q = widen<true>(codes_to_half2(in[j] >> 16));
            out[j] = e4m3x2_bits(p.x * by, p.y * by) | (e4m3x2_bits(q.x * by, q.y * by) << 16);
          }
          *at = make_uint2(out[0], out[1]);
        }
      }
    }
    const float inv = power_of_two(-e);
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
// Products are m16n8k16 instructions in fp16 with the codes widened to fp16 (exact, one instruction for two): q, whatever
// its type, comes in as fp16 times a power of two of its head, with its largest entry in [2^14, 2^15), so that entries
// down to 2^-29 of the largest keep all their bits.  K's scale multiplies the finished scores of its block.  V's cannot
// follow its products, which sum over blocks: it goes into the weights.  A row therefore has two running references: m
// for its scores, under which l sums the weights, and mv for scores + log2 of the block's V scale, under which the
// weights are rounded to fp16 for P V.  mv stands 15 below its maximum, so weights times scales keep all their bits down to
// 2^-29 of the largest and none above 2^-40 is lost.  O goes back to the reference m where a segment ends.
//
// Fragments.  An 8 x 8 matrix of 16-bit units that ldmatrix loads is one of 8 tokens x 16 codes.  For K a thread gets four
// neighbouring codes of a token, columns 4t .. 4t + 3 of 16: the products take them as their columns {2t, 2t + 1} and
// {2t + 8, 2t + 9}, and Q's fragments are put in the same order.  For V, transposed, it gets two codes of two tokens: a
// byte shuffle makes pairs of tokens, for the even columns of 16 and for the odd ones, whose products are kept apart
// until O is written.
enum : uint32_t { kSite8Load = 0x141, kSite8Full = 0x341 };

template <int D, int MT>
struct Dec8Cfg {
  static constexpr int kRows = 16 * MT;                      // query heads per chunk
  static constexpr int kTile = 128;                          // tokens per tile
  static constexpr int kBlocksOfTile = kTile / 16;
  static constexpr int kBlocks = kBlocksOfTile / kConsumers; // of a warp
  static constexpr int kHalf = kTile * D;                    // K or V of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = (MT == 1 ? 98304 : 196608) / kStage;  // two CTAs per SM, or one
  static constexpr int kQStride = D * 2 + 32;                // bytes; 8-byte loads of 4 rows meet every bank once
  static constexpr int kScaleOff = kStages * kStage;         // K's and V's scales of each stage
  static constexpr int kQOff = kScaleOff + kStages * 2 * kBlocksOfTile * 4;
  static constexpr int kQsOff = kQOff + kRows * kQStride;    // q's powers of two
  static constexpr int kMlOff = kQsOff + kRows * 4;          // (m, l) of each warp's rows
  static constexpr int kBarOff = kMlOff + kConsumers * kRows * 8;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kSmemBytes = kMiscOff + 64 + 1024;
  static constexpr float kHeadroom = 15.f;
  static constexpr int kScaleLanes = 2 * kBlocksOfTile;
  static_assert(kConsumers * 16 * D * 4 <= kStage, "the warps' O of 16 heads fit a stage");
  static_assert(kQOff % 16 == 0 && kQsOff % 16 == 0 && kMlOff % 8 == 0 && kBarOff % 8 == 0 && kScaleLanes <= 32, "layout");
};

// Where the 16-byte piece `chunk` of a row of D codes stands in a tile that TMA swizzled in spans of min(D, 128) bytes.
template <int D>
__device__ __forceinline__ uint32_t piece_of(int row, int chunk) {
  if constexpr (D == 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
  else return row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

template <int D, int MT, bool FP16>
__global__ void __launch_bounds__(kDecThreads, MT == 1 ? 2 : 1)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ DecParams p) {
  using C = Dec8Cfg<D, MT>;
  constexpr int kTile = C::kTile, NB = C::kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* bar_empty = bar_full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  long long* s_sums = reinterpret_cast<long long*>(smem + C::kMlOff);
  int* s_start = reinterpret_cast<int*>(smem + C::kMiscOff + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.c.Hkv * p.chunks;

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
  if (!share_of_tiles(p, units, s_sums, s_start, at, w0, w1)) return;
  const WaitCtl wc{abort_flag, p.err_word, p.wait_ns};

  if (warp == kConsumers) {
    // ------------------------------------------------------------- producer warp
    // Lane x: block x mod 8 of the tile, of K (x < 8) or V.  It fetches the block's scale, and if a piece (the tokens
    // of one page in the tile) starts with its block, the piece's codes.  Past the sequence's end, and for a page index
    // outside the cache, the page coordinate n_pages, out of bounds, fills the piece with zeros; such a
    // block's scale is 0.
    const bool mine = lane < C::kScaleLanes, is_v = lane >= C::kBlocksOfTile;
    const int block = lane % C::kBlocksOfTile, per_page = p.c.page_size >> 4;
    const float* scales = is_v ? p.c.v_scales : p.c.k_scales;
    auto page_at = [&](const Place<kTile>& x, int& row) -> int {
      const int tok = x.t * kTile + block * 16;
      row = tok % p.c.page_size;
      int page = p.c.n_pages;
      if (mine && tok < x.n) page = p.c.page_table[x.b * p.c.table_stride + tok / p.c.page_size];
      return page < 0 || page >= p.c.n_pages ? p.c.n_pages : page;
    };
    const bool starts = mine && block * 16 % p.piece == 0;
    int issued = 0, row;
    int page = page_at(at, row);
    bool ok = true;
    for (long long w = w0; w < w1; ++w, ++issued) {
      const int slot = issued % C::kStages;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_empty[slot], ((issued / C::kStages) & 1) ^ 1, wc, kSite8Load))))
        break;
      if (lane == 0) mbar_arrive_expect_tx(&bar_full[slot], C::kStage);
      __syncwarp();
      const int hk = at.u / p.chunks;
      if (starts)
        tma_load_4d(smem + slot * C::kStage + (is_v ? C::kHalf : 0) + block * 16 * D, is_v ? &tm_v : &tm_k, &bar_full[slot],
                    0, row, hk, page);
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
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMlOff);  // [warp][row]
  float* s_qs = reinterpret_cast<float*>(smem + C::kQsOff);
  const int gr = lane >> 2, gc = 2 * (lane & 3);  // fragment row and first column of this thread
  int slot = 0;
  uint32_t phase = 0;
  bool first_segment = true;
  // A segment's Q rows (those past the group's heads: zeros) and slopes, fetched into registers while
  // the segment before it ends.
  constexpr int kQPer = C::kRows * (D / 8) / (32 * kConsumers);  // 16-byte pieces a thread
  uint4 q_next[kQPer];
  float slope_next[MT][2];
  auto fetch_q = [&](const Place<kTile>& x) {
    const int chunk = x.u % p.chunks, head0 = (x.u / p.chunks) * p.group + chunk * C::kRows;
    const int rows = min(p.group - chunk * C::kRows, C::kRows);
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int y = threadIdx.x + i * 32 * kConsumers, r = y / (D / 8), c = y % (D / 8);
      q_next[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        q_next[i] = *reinterpret_cast<const uint4*>(p.q + x.b * p.sq.s[1] + (head0 + r) * p.sq.s[0] + c * 8);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 16 * mt + gr + 8 * e;
        slope_next[mt][e] = p.slopes && r < rows ? p.slopes[head0 + r] * kLog2e : 0.f;
      }
  };
  fetch_q(at);
  for (long long w = w0; w < w1;) {
    // ---- a segment: tiles [at.t, at.t + count) of one head unit
    const int hk = at.u / p.chunks, chunk = at.u % p.chunks;
    const int head0 = hk * p.group + chunk * C::kRows;
    const int rows = min(p.group - chunk * C::kRows, C::kRows);
    const int count = static_cast<int>(min(static_cast<long long>(at.T - at.t), w1 - w));
    const bool whole = count == at.T;
    float slope2[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      slope2[mt][0] = slope_next[mt][0];
      slope2[mt][1] = slope_next[mt][1];
    }
    // Q to fp16 in [2^14, 2^15) of its row's largest entry.
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int y = threadIdx.x + i * 32 * kConsumers, r = y / (D / 8), c = y % (D / 8);
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
      *reinterpret_cast<uint4*>(smem + C::kQOff + r * C::kQStride + c * 16) = out;
      if (c == 0) s_qs[r] = power_of_two(e);
    }
    consumers_sync();
    // A fragments of Q in the order of K's codes: four neighbouring columns a thread.
    auto load_q = [&](uint32_t (&f)[4], int mt, int kk) {
      const uint8_t* at_q = smem + C::kQOff + (16 * mt + gr) * C::kQStride + kk * 32 + 4 * gc;
      const uint2 x = *reinterpret_cast<const uint2*>(at_q), y = *reinterpret_cast<const uint2*>(at_q + 8 * C::kQStride);
      f[0] = x.x;
      f[1] = y.x;
      f[2] = x.y;
      f[3] = y.y;
    };
    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) load_q(qf[kk], 0, kk);
    }
    float o[MT][D / 8][4], m[MT][2], mv[MT][2], l[MT][2], to_log2[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = mv[mt][0] = mv[mt][1] = kNoScore;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        to_log2[mt][e] = (p.cap_out > 0.f ? p.cap_in : p.scale_log2) * s_qs[16 * mt + gr + 8 * e];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) o[mt][c][0] = o[mt][c][1] = o[mt][c][2] = o[mt][c][3] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      // A wait that gave up (the block is aborting) skips the tile but stays in step with the other
      // warps, which it meets at barriers.
      const bool landed = __all_sync(0xffffffffu, mbar_wait(&bar_full[slot], phase, wc, kSite8Full));
      const uint32_t kb = ring + slot * C::kStage, vb = kb + C::kHalf;
      const int key0 = (at.t + i) * kTile + 16 * NB * warp;  // this warp's first token
      if (landed && key0 < at.n) {
        const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff) + slot * C::kScaleLanes + NB * warp;
        const int frow = 16 * NB * warp + (lane & 15), fchunk = lane >> 4;  // what this lane addresses for ldmatrix
        float s[MT][2 * NB][4] = {};
#pragma unroll
        for (int c2 = 0; c2 < D / 32; ++c2) {
          uint32_t b4[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) ldsm4(b4[nb], kb + piece_of<D>(frow + 16 * nb, 2 * c2 + fchunk));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int kk = 2 * c2 + half;
            uint32_t kf[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              kf[nb][0] = codes_to_half2(b4[nb][2 * half]);
              kf[nb][1] = codes_to_half2(b4[nb][2 * half] >> 16);
              kf[nb][2] = codes_to_half2(b4[nb][2 * half + 1]);
              kf[nb][3] = codes_to_half2(b4[nb][2 * half + 1] >> 16);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t a4[4];
              if constexpr (MT > 1) load_q(a4, mt, kk);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                  if constexpr (MT == 1) mma16816<true>(s[mt][2 * nb + nt], qf[kk], kf[nb][2 * nt], kf[nb][2 * nt + 1]);
                  else mma16816<true>(s[mt][2 * nb + nt], a4, kf[nb][2 * nt], kf[nb][2 * nt + 1]);
                }
            }
          }
        }
        // Scales; a block past the end has whatever its page holds there.
        float ks[NB], lgv[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const bool inside = key0 + 16 * nb < at.n;
          ks[nb] = inside ? sc[nb] : 0.f;
          lgv[nb] = inside ? __log2f(sc[C::kBlocksOfTile + nb]) : 0.f;
        }
        // Scores in log2 units, and the running softmax of the warp's rows.
        uint32_t pf[MT][NB][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t bits = 0;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float f[2] = {to_log2[mt][0] * ks[nb], to_log2[mt][1] * ks[nb]};
#pragma unroll
            for (int nt = 2 * nb; nt < 2 * nb + 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[mt][nt][e] *= f[e >> 1];
                bits |= __float_as_uint(s[mt][nt][e]);
              }
          }
          if (p.cap_out > 0.f) {
            // As in the 16-bit decode: relative to the score while |x| < 2.
            const bool any_far = __any_sync(0xffffffffu, bits & kReachesTwo);
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
              for (int e = 0; e < 4; e += 2) {
                const float2 x = make_float2(s[mt][nt][e], s[mt][nt][e + 1]);
                float2 y = __fmul2_rn(x, tanh_over_x(x, p.poly));
                if (any_far) {
                  const float2 far = tanh_any(x, p.cap_out, pair(0.f));
                  y = make_float2(fabsf(x.x) < 2.f ? y.x : far.x, fabsf(x.y) < 2.f ? y.y : far.y);
                }
                s[mt][nt][e] = y.x;
                s[mt][nt][e + 1] = y.y;
              }
          }
          float mx[2] = {-INFINITY, -INFINITY}, mxv[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 2 * nb; nt < 2 * nb + 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + 8 * nt + gc + (e & 1);
                float x = fmaf(-slope2[mt][e >> 1], static_cast<float>(at.n - 1 - key), s[mt][nt][e]);
                x = key < at.n ? x : -INFINITY;
                s[mt][nt][e] = x;
                top[e >> 1] = fmaxf(top[e >> 1], x);
              }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[e] = fmaxf(mx[e], top[e]);
              mxv[e] = fmaxf(mxv[e], top[e] + lgv[nb]);
            }
          }
          float alpha[2], alpha_v[2];
          bool up = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mxv[e] = fmaxf(mxv[e], __shfl_xor_sync(0xffffffffu, mxv[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            mxv[e] = fmaxf(mxv[e], __shfl_xor_sync(0xffffffffu, mxv[e], 2));
            const float mn = fmaxf(m[mt][e], mx[e]), mvn = fmaxf(mv[mt][e], mxv[e] - C::kHeadroom);
            alpha[e] = ex2_approx(m[mt][e] - mn);
            alpha_v[e] = ex2_approx(mv[mt][e] - mvn);
            up |= mn > m[mt][e] || mvn > mv[mt][e];
            m[mt][e] = mn;
            mv[mt][e] = mvn;
          }
          if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) l[mt][e] *= alpha[e];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              o[mt][c][0] *= alpha_v[0];
              o[mt][c][1] *= alpha_v[0];
              o[mt][c][2] *= alpha_v[1];
              o[mt][c][3] *= alpha_v[1];
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float to_v[2] = {lgv[nb] - mv[mt][0], lgv[nb] - mv[mt][1]};
            float pr[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = s[mt][2 * nb + nt][e];
                l[mt][e >> 1] += ex2_approx(x - m[mt][e >> 1]);  // this thread's columns; summed over the quad at the end
                pr[nt][e] = ex2_approx(x + to_v[e >> 1]);
              }
            pf[mt][nb][0] = pack2<true>(pr[0][0], pr[0][1]);
            pf[mt][nb][1] = pack2<true>(pr[0][2], pr[0][3]);
            pf[mt][nb][2] = pack2<true>(pr[1][0], pr[1][1]);
            pf[mt][nb][3] = pack2<true>(pr[1][2], pr[1][3]);
          }
        }
        // O += P V: B fragments of 16 tokens x the even or the odd columns of 16.
        const bool ragged = key0 + 16 * NB > at.n;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // Tokens past the end: their weight is 0, but what the page holds there may be anything.
          const int left = at.n - (key0 + 16 * nb + gc);
          const uint32_t keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
          const uint32_t keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
#pragma unroll
          for (int c2 = 0; c2 < D / 32; ++c2) {
            uint32_t b4[4];
            ldsm4_t(b4, vb + piece_of<D>(frow + 16 * nb, 2 * c2 + fchunk));
            if (ragged) {
              b4[0] &= keep0;
              b4[1] &= keep1;
              b4[2] &= keep0;
              b4[3] &= keep1;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) b4[j] = __byte_perm(b4[j], 0, 0x3120);  // columns 2g of both tokens, then 2g + 1
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t x = b4[2 * half], y = b4[2 * half + 1];
              const uint32_t even[2] = {codes_to_half2(x), codes_to_half2(y)};
              const uint32_t odd[2] = {codes_to_half2(x >> 16), codes_to_half2(y >> 16)};
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<true>(o[mt][4 * c2 + 2 * half], pf[mt][nb], even[0], even[1]);
                mma16816<true>(o[mt][4 * c2 + 2 * half + 1], pf[mt][nb], odd[0], odd[1]);
              }
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
    // ---- the four warps' parts, joined through the segment's last stage
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 1);
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 2);
        if ((lane & 3) == 0) s_ml[warp * C::kRows + 16 * mt + gr + 8 * e] = make_float2(m[mt][e], l[mt][e]);
      }
    float* s_o = reinterpret_cast<float*>(smem + slot * C::kStage);  // [warp][16][D]
    float* part = p.part + static_cast<size_t>(2 * cta + (first_segment ? 0 : 1)) * C::kRows * (D + 2);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      consumers_sync();  // every warp is done with the stage (or with the previous 16 rows)
      const float back[2] = {ex2_approx(mv[mt][0] - m[mt][0]), ex2_approx(mv[mt][1] - m[mt][1])};
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        float* dst = s_o + (warp * 16 + gr) * D + 16 * c + 2 * gc;
        const float(&x)[4] = o[mt][2 * c], (&y)[4] = o[mt][2 * c + 1];
        *reinterpret_cast<float4*>(dst) = make_float4(x[0] * back[0], y[0] * back[0], x[1] * back[0], y[1] * back[0]);
        *reinterpret_cast<float4*>(dst + 8 * D) = make_float4(x[2] * back[1], y[2] * back[1], x[3] * back[1], y[3] * back[1]);
      }
      consumers_sync();
      const int r = threadIdx.x >> 3, gl = 16 * mt + r;  // 8 threads a row
      if (gl < rows) {
        float M = kNoScore, L = 0.f, wgt[kConsumers];
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, s_ml[x * C::kRows + gl].x);
#pragma unroll
        for (int x = 0; x < kConsumers; ++x) {
          const float2 ml = s_ml[x * C::kRows + gl];
          wgt[x] = ex2_approx(ml.x - M);
          L += ml.y * wgt[x];
        }
        const float inv = whole ? 1.f / L : 1.f;
        const int head = head0 + gl;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const int col = 4 * ((threadIdx.x & 7) + 8 * c);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < kConsumers; ++x) {
            const float4 v = *reinterpret_cast<const float4*>(s_o + (x * 16 + r) * D + col);
            acc.x = fmaf(wgt[x], v.x, acc.x);
            acc.y = fmaf(wgt[x], v.y, acc.y);
            acc.z = fmaf(wgt[x], v.z, acc.z);
            acc.w = fmaf(wgt[x], v.w, acc.w);
          }
          if (whole)
            *reinterpret_cast<uint2*>(p.o + at.b * p.so.s[1] + head * p.so.s[0] + col) =
                make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
          else
            *reinterpret_cast<float4*>(part + gl * D + col) = acc;
        }
        if ((threadIdx.x & 7) == 0) {
          if (whole)
            p.lse[static_cast<size_t>(at.b) * p.H + head] = (M + log2f(L)) * kLn2;
          else
            *reinterpret_cast<float2*>(part + C::kRows * D + 2 * gl) = make_float2(M, L);
        }
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

template <int D, int MT, bool FP16>
cudaError_t launch_decode8(const PagedDecodeArgs& a, cudaStream_t stream) {
  using C = Dec8Cfg<D, MT>;
  const DecParams p = decode_params(a, C::kRows, C::kTile);
  CUtensorMap tk, tv;
  cudaError_t e;
  constexpr auto kSwizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  // L2 fetches no more than a row where the rows of a head lie apart (fa_paged.cu).
  auto map = [&](CUtensorMap* t, const void* x, const Strides& s) {
    const auto fetch = s.s[0] == D ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                   : D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    return make_tmap_4d(t, x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, a.c.page_size, a.c.Hkv, a.c.n_pages, s.s, D, p.piece,
                        kSwizzle, fetch);
  };
  if ((e = map(&tk, a.c.k, a.c.sk))) return e;
  if ((e = map(&tv, a.c.v, a.c.sv))) return e;
  auto kern = decode_fp8_kernel<D, MT, FP16>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes))) return e;
  kern<<<static_cast<unsigned>(paged_decode_ctas(p.group)), kDecThreads, C::kSmemBytes, stream>>>(tk, tv, p);
  if ((e = cudaGetLastError())) return e;
  return launch_dependent(decode_join_kernel<D, FP16>, static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.H), 128, 0,
                          stream, p, C::kRows);
}

template <int D, bool FP16>
cudaError_t launch_decode8_mt(const PagedDecodeArgs& a, cudaStream_t stream) {
  return paged_decode_mt(a.H / a.c.Hkv) == 1 ? launch_decode8<D, 1, FP16>(a, stream) : launch_decode8<D, 2, FP16>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append_fp8(const PagedAppendArgs& a, cudaStream_t stream) {
  const long long sides = 2LL * a.c.Hkv;
  const int run = a.T * sides > 64LL * sm_count() ? 16 : 1;
  const long long warps = (a.T + run - 1LL) / run * sides;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  auto kern = a.c.d == 64 ? (a.fp16 ? append_fp8_kernel<64, true> : append_fp8_kernel<64, false>)
                          : (a.fp16 ? append_fp8_kernel<128, true> : append_fp8_kernel<128, false>);
  kern<<<grid, 128, 0, stream>>>(a, run);
  return cudaGetLastError();
}

cudaError_t launch_paged_decode_fp8(const PagedDecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return a.fp16 ? launch_decode8_mt<64, true>(a, stream) : launch_decode8_mt<64, false>(a, stream);
  return a.fp16 ? launch_decode8_mt<128, true>(a, stream) : launch_decode8_mt<128, false>(a, stream);
}

}  // namespace fa
