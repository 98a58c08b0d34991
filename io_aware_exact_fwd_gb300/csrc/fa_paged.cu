// The paged key/value cache: appending new tokens, and attention of one token a
// sequence over the cache (include/fa.h states both).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "fa_device.cuh"
#include "fa_internal.h"
#include "fa_score.cuh"

namespace fa {
namespace {

__device__ __forceinline__ int tokens_of(const PagedCache& c, int b) {
  return min(max(c.seq_lens[b], 0), c.max_pages * c.page_size);
}

// Append: a warp takes as many consecutive new tokens as make up to 128 pieces of 16 bytes of K (one if there are
// few), up to four pieces of K and of V a lane in flight while its first lanes look the tokens' places up, a token
// each.  Bound by HBM: the new rows are read once and written once.  Measured with 8 heads x 128: 35k tokens in 45.6
// us, 6.3 TB/s; 64 tokens in 4.1 us, a launch and three dependent loads; 29k tokens of one head x 128 in 5.2 us, 5.8
// TB/s.  (One 16-byte piece a thread, each with its own look-up: 49.1 us for the first; one token a warp: 11.6 for the
// last.)
template <bool ONE>  // per_warp is 1
__global__ void __launch_bounds__(128) paged_append_kernel(PagedAppendArgs a, int per_warp) {
  const long long first = ((static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5) * per_warp;
  if (first >= a.T) return;
  const int t0 = static_cast<int>(first), lane = threadIdx.x & 31, tokens = min(per_warp, a.T - t0);
  const int shift = a.c.d == 64 ? 3 : 4, row = a.c.Hkv << shift;  // pieces of a head's row: 8 or 16; of a token's
  const int pieces = tokens * row;
  const uint16_t* ks = static_cast<const uint16_t*>(a.k) + t0 * a.sk.s[1];
  const uint16_t* vs = static_cast<const uint16_t*>(a.v) + t0 * a.sv.s[1];
  // Piece x: token t, head h, column col.
  auto piece = [&](int x, int& t, int& h, int& col) {
    t = ONE ? 0 : x / row;
    x -= t * row;
    h = x >> shift;
    col = (x & ((1 << shift) - 1)) * 8;
  };
  uint4 kv[4], vv[4];
  auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = p0 + 32 * i;
      int t, h, col;
      piece(x, t, h, col);
      if (x < pieces) {
        kv[i] = *reinterpret_cast<const uint4*>(ks + t * a.sk.s[1] + h * a.sk.s[0] + col);
        vv[i] = *reinterpret_cast<const uint4*>(vs + t * a.sv.s[1] + h * a.sv.s[0] + col);
      }
    }
  };
  load(lane);  // in flight while the places are looked up
  int page = -1, off = 0;
  if (ONE || lane < tokens) {
    const int t = ONE ? t0 : t0 + lane;
    int lo = 0, hi = a.c.B + 1;  // the number of offsets <= t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.cu_new + mid) <= t) lo = mid + 1;
      else hi = mid;
    }
    if (lo != 0 && lo != a.c.B + 1) {  // (else a row of no sequence)
      const int b = lo - 1;
      const long long pos = static_cast<long long>(a.c.seq_lens[b]) - (static_cast<long long>(a.cu_new[lo]) - t);
      if (pos >= 0 && pos < static_cast<long long>(a.c.max_pages) * a.c.page_size) {
        off = static_cast<int>(pos) % a.c.page_size;
        page = a.c.page_table[b * a.c.table_stride + static_cast<int>(pos) / a.c.page_size];
        if (page >= a.c.n_pages) page = -1;
      }
    }
  }
  if (ONE && page < 0) return;
  long long k_at = page * a.c.sk.s[2] + off * a.c.sk.s[0], v_at = page * a.c.sv.s[2] + off * a.c.sv.s[0];
  for (int p0 = lane; ONE ? p0 < pieces : p0 - lane < pieces; p0 += 128) {
    if (p0 != lane) load(p0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = p0 + 32 * i;
      int t, h, col;
      piece(x, t, h, col);
      bool here = x < pieces;
      if (!ONE) {
        const int pg = __shfl_sync(0xffffffffu, page, t), r = __shfl_sync(0xffffffffu, off, t);
        here = here && pg >= 0;
        k_at = pg * a.c.sk.s[2] + r * a.c.sk.s[0];
        v_at = pg * a.c.sv.s[2] + r * a.c.sv.s[0];
      }
      if (here) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.k) + k_at + h * a.c.sk.s[1] + col) = kv[i];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c.v) + v_at + h * a.c.sv.s[1] + col) = vv[i];
      }
    }
  }
}

// ------------------------------------------------------------------------------
// Decode: one token a sequence, softmax over its whole cache.  Bound by HBM: K and V are
// read once for all G query heads that share them (4 d bytes against 4 G d flops a
// token).
//
// Work.  A tile is 64 tokens (d = 128) or 128 (d = 64) of one (sequence, key/value head,
// chunk of 16 MT query heads); the tiles of all of them stand in one line (sequence by
// sequence, head by head, token by token) and every CTA takes the same number of
// consecutive ones (down to one: two at least made 900 tokens take 10.7 us for 9.3), so
// ragged lengths balance without the host knowing them.  A run of tiles of one head
// inside a CTA's share is a segment: a segment that covers the head's tokens is written
// out at once, any other leaves its (m, l, O) in the workspace for the join kernel.  A
// CTA has at most two such segments, its first and its last, so the workspace depends
// on the number of CTAs alone.
//
// A CTA is four consumer warps and a producer warp.  The producer's lanes each fetch one
// piece of a tile (the tokens of one page in it) with TMA into a ring of stages.
// Consumer warp w takes the w-th quarter of every tile's tokens and keeps its own running
// maximum, sum and O (16 MT heads x d in registers), so the warps meet only at a
// segment's end.  Its products are m16n8k16 tensor instructions with the heads as rows
// (S = Q K^T, O += P V; with fewer than 16 heads the other rows are zeros): at most 1/7
// of their rate is used, and a tcgen05 tile of 128 rows would waste more.
//
// Measured: 64 sequences of 1 .. 16384 tokens (1.9 GB), H=32 over 8 heads, d=128, capped,
// 64-token pages: 295-303 us, 6.4 TB/s; one of 131072 tokens, 16 heads of d=64 beside each
// other, biased: 92-101 us, 5.3-5.8 TB/s (86 us where each head's tokens lie together); one
// of 900 tokens, H=16 over 4: 9.3 us in a graph, two launches and two waits on memory.
constexpr int kConsumers = 4;     // consumer warps
constexpr int kDecThreads = 32 * (kConsumers + 1);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;
// The reference of a row before its first token, and where every score so far is -inf (a key with an infinite entry):
// finite, so that such tokens weigh 0 and a part that holds no others joins with weight 0.
constexpr float kNoScore = -3.0e38f;

enum : uint32_t { kSiteDecLoad = 0x131, kSiteDecFull = 0x331 };

template <int D, int MT, bool FP16>
struct DecCfg {
  static constexpr int kRows = 16 * MT;                   // query heads per chunk
  static constexpr int kTile = 8192 / D;                  // tokens per tile: K and V of one are 32 KB
  static constexpr int kBlocks = kTile / (16 * kConsumers);  // 16-token blocks of a warp in a tile
  static constexpr int kBoxes = D / 64;                   // 128-byte TMA boxes per row
  static constexpr int kHalf = kTile * D * 2;             // K or V of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 3;                       // two CTAs per SM
  static constexpr int kQStride = D * 2 + 16;             // bytes; 16 apart from a multiple of 128: no bank conflicts
  static constexpr int kQOff = kStages * kStage;
  static constexpr int kMlOff = kQOff + kRows * kQStride; // (m, l) of each warp's rows
  static constexpr int kBarOff = kMlOff + kConsumers * kRows * 8;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kSmemBytes = kMiscOff + 64 + 1024;
  // A row's reference stands this far below its maximum, in log2 units.  P is rounded to the cache's
  // type; fp16 holds 2^-14 .. 2^15 with all its bits, so with P up to 2^15 weights keep them down to 2^-29 of the
  // largest and none above 2^-40 is lost (a million tokens of 2^-25 together are 3 % of the one they
  // follow).  bf16 has fp32's range.  The factor is in l too and cancels.
  static constexpr float kHeadroom = FP16 ? 15.f : 0.f;
  static_assert(kConsumers * 16 * D * 4 <= kStage, "the warps' O of 16 heads fit a stage");
};

struct DecParams {
  PagedCache c;
  const uint16_t* q;
  uint16_t* o;
  Strides sq, so;
  float* lse;
  float* part;               // [2 CTAs][rows][D + 2]: O, then m and l
  long long* offsets;        // [B + 1] tiles before each sequence, then the share
  int H, group, chunks, piece;
  float scale_log2, cap_in, cap_out;
  CapPoly poly;              // factor cap_out
  const float* slopes;
  unsigned int* err_word;
  unsigned long long wait_ns;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool FP16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (FP16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (FP16) {
    const __half2 x = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory"); }
__device__ __forceinline__ int tiles_of(const PagedCache& c, int b, int tile) {
  return (tokens_of(c, b) + tile - 1) / tile;
}

// A place in the line of tiles: tile t of head unit u (key/value head and chunk) of
// sequence b, with n tokens in T tiles.
template <int TILE>
struct Place {
  int b, u, t, n, T;
  __device__ __forceinline__ void sequence(const PagedCache& c) {
    n = tokens_of(c, b);
    T = (n + TILE - 1) / TILE;
  }
  // To the next head unit (the next sequence with tokens after the last one).
  __device__ __forceinline__ void next_unit(const PagedCache& c, int units) {
    t = 0;
    if (++u < units) return;
    u = 0;
    do {
      ++b;
      if (b >= c.B) return;
      sequence(c);
    } while (T == 0);
  }
};

template <int D, int MT, bool FP16>
__global__ void __launch_bounds__(kDecThreads, MT == 1 ? 2 : 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ DecParams p) {
  using C = DecCfg<D, MT, FP16>;
  constexpr int kTile = C::kTile, NB = C::kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* bar_empty = bar_full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  long long* s_sums = reinterpret_cast<long long*>(smem + C::kMlOff);  // scratch of the scan, before any segment
  int* s_start = reinterpret_cast<int*>(smem + C::kMiscOff + 8);       // sequence, then tiles into it (two words)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.c.Hkv * p.chunks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], kConsumers);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // Tiles before each sequence: a thread sums a run of sequences, the block scans the sums.
  const int per = (p.c.B + kDecThreads - 1) / kDecThreads;
  const int b_lo = min(static_cast<int>(threadIdx.x) * per, p.c.B), b_hi = min(b_lo + per, p.c.B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += static_cast<long long>(tiles_of(p.c, b, kTile)) * units;
  long long before = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, w);
    if (lane >= w) before += x;
  }
  if (lane == 31) s_sums[warp] = before;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w <= kConsumers; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  before -= mine;
  const int G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const long long share = (total + G - 1) / G;  // down to one tile: a block's tile costs more than its join
  const long long w0 = cta * share, w1 = min(w0 + share, total);
  const long long after = before + mine;
  if (cta == 0) {  // for the join
    for (int b = b_lo; b < b_hi; ++b) {
      p.offsets[b] = before;
      before += static_cast<long long>(tiles_of(p.c, b, kTile)) * units;
    }
    if (threadIdx.x == 0) {
      p.offsets[p.c.B] = total;
      p.offsets[p.c.B + 1] = share;
    }
    before = after - mine;
  }
  if (w0 < total && before <= w0 && w0 < after) {  // this thread's run holds the CTA's first tile
    int b = b_lo;
    for (;; ++b) {
      const long long x = static_cast<long long>(tiles_of(p.c, b, kTile)) * units;
      if (w0 < before + x) break;
      before += x;
    }
    s_start[0] = b;
    *reinterpret_cast<long long*>(s_start + 2) = w0 - before;
  }
  __syncthreads();
  grid_release();
  if (w0 >= total) return;
  Place<kTile> at;
  at.b = s_start[0];
  at.sequence(p.c);
  {
    const long long into = *reinterpret_cast<const long long*>(s_start + 2);
    at.u = static_cast<int>(into / at.T);
    at.t = static_cast<int>(into % at.T);
  }
  const WaitCtl wc{abort_flag, p.err_word, p.wait_ns};

  if (warp == kConsumers) {
    // ------------------------------------------------------------- producer warp
    // Lane x < pieces: the tokens [x piece, (x + 1) piece) of a tile, one page's; past the
    // sequence's end (and for a page index outside the cache) the page coordinate n_pages,
    // out of bounds, fills the piece with zeros.
    const int pieces = kTile / p.piece;
    auto page_at = [&](const Place<kTile>& x, int& row) -> int {
      const int tok = x.t * kTile + lane * p.piece;
      row = tok % p.c.page_size;
      int page = p.c.n_pages;
      if (lane < pieces && tok < x.n) page = p.c.page_table[x.b * p.c.table_stride + tok / p.c.page_size];
      return page < 0 || page >= p.c.n_pages ? p.c.n_pages : page;
    };
    int issued = 0, row;
    int page = page_at(at, row);
    bool ok = true;
    for (long long w = w0; w < w1; ++w, ++issued) {
      const int slot = issued % C::kStages;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bar_empty[slot], ((issued / C::kStages) & 1) ^ 1, wc, kSiteDecLoad))))
        break;
      if (lane == 0) mbar_arrive_expect_tx(&bar_full[slot], C::kStage);
      __syncwarp();
      if (lane < pieces) {
        uint8_t* dst = smem + slot * C::kStage + lane * p.piece * 128;
        const int hk = at.u / p.chunks;
#pragma unroll
        for (int c = 0; c < C::kBoxes; ++c) {
          tma_load_4d(dst + c * kTile * 128, &tm_k, &bar_full[slot], c * 64, row, hk, page);
          tma_load_4d(dst + C::kHalf + c * kTile * 128, &tm_v, &bar_full[slot], c * 64, row, hk, page);
        }
      }
      if (w + 1 < w1) {
        if (++at.t == at.T) at.next_unit(p.c, units);
        page = page_at(at, row);
      }
    }
    if ((!ok || *abort_flag) && lane == 0)  // the copies in flight land before the block's shared memory goes
      for (int t = max(0, issued - C::kStages); t < issued; ++t)
        mbar_wait_drain(&bar_full[t % C::kStages], (t / C::kStages) & 1, p.wait_ns);
    __syncwarp();
    return;
  }

  // ---------------------------------------------------------------- consumer warps
  const uint32_t ring = smem_u32(smem), sq = smem_u32(smem + C::kQOff);
  float2* s_ml = reinterpret_cast<float2*>(smem + C::kMlOff);  // [warp][row]
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
#pragma unroll
    for (int i = 0; i < kQPer; ++i) {
      const int y = threadIdx.x + i * 32 * kConsumers, r = y / (D / 8), c = y % (D / 8);
      *reinterpret_cast<uint4*>(smem + C::kQOff + r * C::kQStride + c * 16) = q_next[i];
    }
    consumers_sync();
    // A fragments of Q: lanes 0-15 address rows, lanes 16-31 the same rows 8 columns on.
    const uint32_t q_addr = sq + (lane & 15) * C::kQStride + (lane >> 4) * 16;
    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) ldsm4(qf[kk], q_addr + kk * 32);
    }
    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt][0] = m[mt][1] = kNoScore;
      l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) o[mt][c][0] = o[mt][c][1] = o[mt][c][2] = o[mt][c][3] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      // A wait that gave up (the block is aborting) skips the tile but stays in step with the other
      // warps, which it meets at barriers.
      const bool landed = __all_sync(0xffffffffu, mbar_wait(&bar_full[slot], phase, wc, kSiteDecFull));
      const uint32_t kb = ring + slot * C::kStage, vb = kb + C::kHalf;
      const int key0 = (at.t + i) * kTile + 16 * NB * warp;  // this warp's first token
      if (landed && key0 < at.n) {
        // S = Q K^T: B fragments of 16 tokens x 16 columns: matrices (tokens 0-7, 8-15) x (two column halves).
        float s[MT][2 * NB][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const int ch = 2 * kk + ((lane >> 3) & 1);
          uint32_t b4[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int krow = 16 * (NB * warp + nb) + (lane & 7) + ((lane & 16) >> 1);
            ldsm4(b4[nb], kb + (ch >> 3) * (kTile * 128) + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4));
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t a4[4];
            if constexpr (MT > 1) ldsm4(a4, q_addr + mt * 16 * C::kQStride + kk * 32);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if constexpr (MT == 1) {
                mma16816<FP16>(s[mt][2 * nb], qf[kk], b4[nb][0], b4[nb][1]);
                mma16816<FP16>(s[mt][2 * nb + 1], qf[kk], b4[nb][2], b4[nb][3]);
              } else {
                mma16816<FP16>(s[mt][2 * nb], a4, b4[nb][0], b4[nb][1]);
                mma16816<FP16>(s[mt][2 * nb + 1], a4, b4[nb][2], b4[nb][3]);
              }
            }
          }
        }
        // Scores in log2 units, and the running softmax of the warp's rows.
        uint32_t pf[MT][NB][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float mx[2] = {-INFINITY, -INFINITY};
          if (p.cap_out > 0.f) {
            // As in the forward: relative to the score while |x| < 2, so that a cap far above the scores costs
            // them no bits; the other form only where an argument of the warp needs it.
            uint32_t bits = 0;
#pragma unroll
            for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                s[mt][nt][e] *= p.cap_in;
                bits |= __float_as_uint(s[mt][nt][e]);
              }
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
#pragma unroll
          for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 8 * nt + gc + (e & 1);
              float x = p.cap_out > 0.f ? s[mt][nt][e] : s[mt][nt][e] * p.scale_log2;
              x = fmaf(-slope2[mt][e >> 1], static_cast<float>(at.n - 1 - key), x);
              x = key < at.n ? x : -INFINITY;
              s[mt][nt][e] = x;
              mx[e >> 1] = fmaxf(mx[e >> 1], x);
            }
          float alpha[2];
          bool up = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            const float mn = fmaxf(m[mt][e], mx[e] - C::kHeadroom);
            alpha[e] = ex2_approx(m[mt][e] - mn);
            up |= mn > m[mt][e];
            m[mt][e] = mn;
          }
          if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) l[mt][e] *= alpha[e];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              o[mt][c][0] *= alpha[0];
              o[mt][c][1] *= alpha[0];
              o[mt][c][2] *= alpha[1];
              o[mt][c][3] *= alpha[1];
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float pr[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                pr[nt][e] = ex2_approx(s[mt][2 * nb + nt][e] - m[mt][e >> 1]);
                l[mt][e >> 1] += pr[nt][e];  // this thread's columns; summed over the quad at the end
              }
            pf[mt][nb][0] = pack2<FP16>(pr[0][0], pr[0][1]);
            pf[mt][nb][1] = pack2<FP16>(pr[0][2], pr[0][3]);
            pf[mt][nb][2] = pack2<FP16>(pr[1][0], pr[1][1]);
            pf[mt][nb][3] = pack2<FP16>(pr[1][2], pr[1][3]);
          }
        }
        // O += P V: B fragments (16 tokens x 16 columns) by transposing loads.
        const bool ragged = key0 + 16 * NB > at.n;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int vrow = 16 * (NB * warp + nb) + (lane & 15);
          // Tokens past the end: their weight is 0, but what the page holds there may be anything.
          const int left = at.n - (key0 + 16 * nb + gc);
          const uint32_t keep0 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
          const uint32_t keep1 = (left > 8 ? 0xffffu : 0u) | (left > 9 ? 0xffff0000u : 0u);
#pragma unroll
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t b4[4];
            const int ch = 2 * cc + (lane >> 4);
            ldsm4_t(b4, vb + (ch >> 3) * (kTile * 128) + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4));
            if (ragged) {
              b4[0] &= keep0;
              b4[1] &= keep1;
              b4[2] &= keep0;
              b4[3] &= keep1;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<FP16>(o[mt][2 * cc], pf[mt][nb], b4[0], b4[1]);
              mma16816<FP16>(o[mt][2 * cc + 1], pf[mt][nb], b4[2], b4[3]);
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
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float* dst = s_o + (warp * 16 + gr) * D + 8 * c + gc;
        *reinterpret_cast<float2*>(dst) = make_float2(o[mt][c][0], o[mt][c][1]);
        *reinterpret_cast<float2*>(dst + 8 * D) = make_float2(o[mt][c][2], o[mt][c][3]);
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

// Joins the parts of heads whose tiles lie in several CTAs' shares, and writes the
// result of empty sequences.  One block per (sequence, query head): warp x takes parts
// x, x + 4, ...
template <int D, bool FP16>
__global__ void __launch_bounds__(128) decode_join_kernel(const __grid_constant__ DecParams p, int rows_per_part) {
  __shared__ float2 s_ml[4];
  __shared__ __align__(16) float s_o[4][D];
  grid_wait();  // the parts are written
  const int b = blockIdx.x / p.H, head = blockIdx.x % p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = D / 32;
  const int hk = head / p.group, in_group = head % p.group;
  const int u = hk * p.chunks + in_group / rows_per_part, row = in_group % rows_per_part;
  const long long first = p.offsets[b], tiles = (p.offsets[b + 1] - first) / (p.c.Hkv * p.chunks);
  const long long share = p.offsets[p.c.B + 1];
  const long long w0 = first + u * tiles;
  uint16_t* dst = p.o + b * p.so.s[1] + head * p.so.s[0];
  float* lse = p.lse + static_cast<size_t>(b) * p.H + head;
  if (tiles == 0) {
    if (threadIdx.x < D / 8) *reinterpret_cast<uint4*>(dst + 8 * threadIdx.x) = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) *lse = -INFINITY;
    return;
  }
  const int c0 = static_cast<int>(w0 / share), c1 = static_cast<int>((w0 + tiles - 1) / share);
  if (c0 == c1) return;  // one CTA had the whole head and wrote it
  float m = kNoScore, l = 0.f, acc[E] = {};
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += 4) {
    // A CTA's first segment has slot 0; only the first part can be another segment of its CTA.
    const int slot = 2 * c + (c * share >= w0 ? 0 : 1);
    const float* part = p.part + static_cast<size_t>(slot) * rows_per_part * (D + 2);
    const float2 ml = *reinterpret_cast<const float2*>(part + rows_per_part * D + 2 * row);
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = part[row * D + lane + 32 * e];
    const float mn = fmaxf(m, ml.x), wa = ex2_approx(m - mn), wb = ex2_approx(ml.x - mn);
    l = l * wa + ml.y * wb;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * wa + v[e] * wb;
    m = mn;
  }
  if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float M = kNoScore, L = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) M = fmaxf(M, s_ml[x].x);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float wgt = ex2_approx(s_ml[x].x - M);
      L += s_ml[x].y * wgt;
      sum.x = fmaf(s_o[x][2 * threadIdx.x], wgt, sum.x);
      sum.y = fmaf(s_o[x][2 * threadIdx.x + 1], wgt, sum.y);
    }
    reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = pack2<FP16>(sum.x / L, sum.y / L);
    if (threadIdx.x == 0) *lse = (M + log2f(L)) * kLn2;
  }
}

// Query heads per chunk (16 MT) and the CTAs of the decode.  Up to 16 heads share a key/value head
// in most models, and two CTAs an SM with 16 rows each keep more loads in flight than one with 32
// (64 sequences of 4000-8000 tokens, one head of d=128: 40.5 us against 46.5); larger groups read
// the cache once a chunk, so chunks of 32 pay (32 heads: 49.2 us against 54.0).
int decode_mt(int group) { return group <= 16 ? 1 : 2; }
int decode_ctas(int group) { return sm_count() * (decode_mt(group) == 1 ? 2 : 1); }

size_t part_bytes(int group, int d) {
  return (static_cast<size_t>(2) * decode_ctas(group) * 16 * decode_mt(group) * (d + 2) * sizeof(float) + 255) / 256 * 256;
}

template <int D, int MT, bool FP16>
cudaError_t launch_decode(const PagedDecodeArgs& a, cudaStream_t stream) {
  using C = DecCfg<D, MT, FP16>;
  DecParams p{};
  p.c = a.c;
  p.q = static_cast<const uint16_t*>(a.q);
  p.o = static_cast<uint16_t*>(a.o);
  p.sq = a.sq;
  p.so = a.so;
  p.lse = a.lse;
  p.H = a.H;
  p.group = a.H / a.c.Hkv;
  p.chunks = (p.group + C::kRows - 1) / C::kRows;
  p.part = static_cast<float*>(a.workspace);
  p.offsets = reinterpret_cast<long long*>(static_cast<uint8_t*>(a.workspace) + part_bytes(p.group, D));
  // The tokens of one page inside a tile: the largest power of two that divides both.
  p.piece = std::min(C::kTile, a.c.page_size & -a.c.page_size);
  p.scale_log2 = a.scale * kLog2e;
  if (a.softcap > 0.f) {
    p.cap_in = 4.f * a.scale / a.softcap;  // products to x = 4 u (fa_score.cuh)
    p.cap_out = a.softcap * kLog2e;
    p.poly = cap_poly(p.cap_out);
  }
  p.slopes = a.slopes;
  p.err_word = a.err_word;
  p.wait_ns = a.dbg.wait_limit_ns;
  CUtensorMap tk, tv;
  cudaError_t e;
  // L2 fetches a row of one head at a time: with heads beside each other a 256-byte fetch of a
  // 128-byte row (d = 64) reads the next head's row too, for a block that wants it later (8 sequences
  // of 32768 tokens, 32 heads: 464 us against 362).
  constexpr auto kFetch = D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  constexpr auto kType = FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if ((e = make_tmap_4d(&tk, a.c.k, kType, 2, D, a.c.page_size, a.c.Hkv, a.c.n_pages, a.c.sk.s, 64, p.piece,
                        CU_TENSOR_MAP_SWIZZLE_128B, kFetch)))
    return e;
  if ((e = make_tmap_4d(&tv, a.c.v, kType, 2, D, a.c.page_size, a.c.Hkv, a.c.n_pages, a.c.sv.s, 64, p.piece,
                        CU_TENSOR_MAP_SWIZZLE_128B, kFetch)))
    return e;
  auto kern = decode_kernel<D, MT, FP16>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes))) return e;
  kern<<<static_cast<unsigned>(decode_ctas(p.group)), kDecThreads, C::kSmemBytes, stream>>>(tk, tv, p);
  if ((e = cudaGetLastError())) return e;
  return launch_dependent(decode_join_kernel<D, FP16>, static_cast<unsigned>(a.c.B) * static_cast<unsigned>(a.H), 128, 0,
                          stream, p, C::kRows);
}

template <int D, bool FP16>
cudaError_t launch_decode_mt(const PagedDecodeArgs& a, cudaStream_t stream) {
  return decode_mt(a.H / a.c.Hkv) == 1 ? launch_decode<D, 1, FP16>(a, stream) : launch_decode<D, 2, FP16>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  // More than one token a warp only past 16 warps an SM (64 tokens of one head: 2.7 us, 3.4 with eight a warp).
  const int per_warp = std::max(1, std::min(128 / (a.c.Hkv * (a.c.d / 8)), a.T / (16 * sm_count())));
  const long long warps = (static_cast<long long>(a.T) + per_warp - 1) / per_warp;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  if (per_warp == 1) paged_append_kernel<true><<<grid, 128, 0, stream>>>(a, per_warp);
  else paged_append_kernel<false><<<grid, 128, 0, stream>>>(a, per_warp);
  return cudaGetLastError();
}

size_t paged_decode_workspace(int B, int H, int Hkv, int d) {
  return part_bytes(H / Hkv, d) + (static_cast<size_t>(B) + 2) * sizeof(long long);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return a.fp16 ? launch_decode_mt<64, true>(a, stream) : launch_decode_mt<64, false>(a, stream);
  return a.fp16 ? launch_decode_mt<128, true>(a, stream) : launch_decode_mt<128, false>(a, stream);
}

}  // namespace fa
