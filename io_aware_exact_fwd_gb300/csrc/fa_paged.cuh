// Device pieces that the paged cache's kernels share: how the tiles of all sequences are
// dealt out to the CTAs of a decode, and the join of a head's parts.
#pragma once

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

constexpr int kConsumers = 4;     // consumer warps
constexpr int kDecThreads = 32 * (kConsumers + 1);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;
// The reference of a row before its first token, and where every score so far is -inf (a key with an infinite entry):
// finite, so that such tokens weigh 0 and a part that holds no others joins with weight 0.
constexpr float kNoScore = -3.0e38f;

struct DecParams {
  PagedCache c;
  const uint16_t* q;
  uint16_t* o;
  Strides sq, so;
  float* lse;
  float* part;               // [2 CTAs][part_rows][D + 2]: O, then m and l
  long long* offsets;        // [B + 1] tiles before each sequence, then the share
  int H, group, chunks, piece;
  int two;                   // 1: a head unit is two key/value heads (8-bit cache, rows of up to 8 query heads for each)
  float scale_log2, cap_in, cap_out;
  CapPoly poly;              // factor cap_out
  const float* slopes;
  unsigned int* err_word;
  unsigned long long wait_ns;
  int part_rows;             // even, so that parts start on 16 bytes
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

// a / b for a >= 0, b > 0: in 32 bits where a allows it (a division in 64 takes some hundred cycles).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ int units_of(const DecParams& p) { return p.two ? p.c.Hkv / 2 : p.c.Hkv * p.chunks; }

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

// The CTA's share [w0, w1) of the line of tiles, and the place of its first one; false if
// it has none.  Every thread of the block, of WARPS warps, calls it, once; s_sums (WARPS words
// of 8 bytes) and s_start (16 bytes, 8-byte aligned) are scratch until then.
template <int WARPS, int TILE>
__device__ __forceinline__ bool share_of_tiles(const DecParams& p, int units, long long* s_sums, int* s_start,
                                               Place<TILE>& at, long long& w0, long long& w1) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Tiles before each sequence: a thread sums a run of sequences, the block scans the sums.
  const int per = (p.c.B + 32 * WARPS - 1) / (32 * WARPS);
  const int b_lo = min(static_cast<int>(threadIdx.x) * per, p.c.B), b_hi = min(b_lo + per, p.c.B);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += static_cast<long long>(tiles_of(p.c, b, TILE)) * units;
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
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  before -= mine;
  const int G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const long long share = quotient(total + G - 1, G);  // down to one tile: a block's tile costs more than its join
  w0 = cta * share;
  w1 = min(w0 + share, total);
  const long long after = before + mine;
  if (cta == 0) {  // for the join
    for (int b = b_lo; b < b_hi; ++b) {
      p.offsets[b] = before;
      before += static_cast<long long>(tiles_of(p.c, b, TILE)) * units;
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
      const long long x = static_cast<long long>(tiles_of(p.c, b, TILE)) * units;
      if (w0 < before + x) break;
      before += x;
    }
    s_start[0] = b;
    *reinterpret_cast<long long*>(s_start + 2) = w0 - before;
  }
  __syncthreads();
  grid_release();
  if (w0 >= total) return false;
  at.b = s_start[0];
  at.sequence(p.c);
  {
    const long long into = *reinterpret_cast<const long long*>(s_start + 2);
    at.u = static_cast<int>(quotient(into, at.T));
    at.t = static_cast<int>(into - static_cast<long long>(at.u) * at.T);
  }
  return true;
}

// Where the tiles of one sequence's query head are: CTAs c0 to c1 had them.
struct HeadParts {
  int b, head, row, c0, c1;  // row: of a part's
  long long w0, share;
  bool empty;
  __device__ __forceinline__ HeadParts(const DecParams& p, int rows_per_unit, int x) {
    b = x / p.H;
    head = x - b * p.H;
    const int hk = head / p.group, in_group = head % p.group;
    const int u = p.two ? hk / 2 : hk * p.chunks + in_group / rows_per_unit;
    row = p.two ? (hk & 1) * p.group + in_group : in_group % rows_per_unit;
    const long long first = p.offsets[b], tiles = quotient(p.offsets[b + 1] - first, units_of(p));
    share = p.offsets[p.c.B + 1];
    w0 = first + u * tiles;
    empty = tiles == 0;
    c0 = empty ? 0 : static_cast<int>(quotient(w0, share));
    c1 = empty ? 0 : static_cast<int>(quotient(w0 + tiles - 1, share));
  }
  // Not written yet by the one CTA that had all of it.
  __device__ __forceinline__ bool open() const { return empty || c0 != c1; }
};

// A block joins one head's parts: warp x takes parts x, x + 4, ...
template <int D, bool FP16>
__device__ __forceinline__ void join_head(const DecParams& p, const HeadParts& h, float2 (&s_ml)[4], float (&s_o)[4][D]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int E = D / 32;
  uint16_t* dst = p.o + h.b * p.so.s[1] + h.head * p.so.s[0];
  float* lse = p.lse + static_cast<size_t>(h.b) * p.H + h.head;
  if (h.empty) {
    if (threadIdx.x < D / 8) *reinterpret_cast<uint4*>(dst + 8 * threadIdx.x) = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) *lse = -INFINITY;
    return;
  }
  float m = kNoScore, l = 0.f, acc[E] = {};
#pragma unroll 4
  for (int c = h.c0 + warp; c <= h.c1; c += 4) {
    // A CTA's first segment has slot 0; only the first part can be another segment of its CTA.
    const int slot = 2 * c + (c * h.share >= h.w0 ? 0 : 1);
    const float* part = p.part + static_cast<size_t>(slot) * p.part_rows * (D + 2);
    const float2 ml = *reinterpret_cast<const float2*>(part + p.part_rows * D + 2 * h.row);
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = part[h.row * D + lane + 32 * e];
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

// Joins the parts of heads whose tiles lie in several CTAs' shares, and writes the
// result of empty sequences.  A block per (sequence, query head); where these would be more than 16 an SM, a block has every
// gridDim-th and each thread looks first at one, whether there is something to do: most of so many heads are whole (the 8-bit decode of
// 109 sequences with 9 .. 18 tokens, 192 heads: 47 us with a block each, 30 so), or of idle sequences, whose results that thread writes
// (1000 places of which one has 3000 tokens, 32 heads, 16-bit: 31.5 us with a block each, 42.9 with a block's turn
// each, 16.0 so).
template <int D, bool FP16>
__global__ void __launch_bounds__(128) decode_join_kernel(const __grid_constant__ DecParams p, int rows_per_unit) {
  __shared__ float2 s_ml[4];
  __shared__ __align__(16) float s_o[4][D];
  __shared__ uint32_t s_open[4];
  grid_wait();  // the parts are written
  const int all = p.c.B * p.H, step = gridDim.x;
  if (all == step) {
    const HeadParts h(p, rows_per_unit, blockIdx.x);
    if (h.open()) join_head<D, FP16>(p, h, s_ml, s_o);
    return;
  }
  for (long long first = blockIdx.x; first < all; first += 128LL * step) {
    const long long mine = first + static_cast<long long>(threadIdx.x) * step;
    bool open = false;
    if (mine < all) {
      const HeadParts h(p, rows_per_unit, static_cast<int>(mine));
      open = !h.empty && h.open();
      if (h.empty) {  // of an idle sequence: there may be thousands
        uint16_t* dst = p.o + h.b * p.so.s[1] + h.head * p.so.s[0];
#pragma unroll
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
        p.lse[static_cast<size_t>(h.b) * p.H + h.head] = -INFINITY;
      }
    }
    const uint32_t some = __ballot_sync(0xffffffffu, open);
    if ((threadIdx.x & 31) == 0) s_open[threadIdx.x >> 5] = some;
    __syncthreads();
    for (int w = 0; w < 4; ++w)
      for (uint32_t todo = s_open[w]; todo; todo &= todo - 1) {
        const int x = static_cast<int>(first + static_cast<long long>(32 * w + __ffs(todo) - 1) * step);
        join_head<D, FP16>(p, HeadParts(p, rows_per_unit, x), s_ml, s_o);
        __syncthreads();  // (s_ml and s_o are free)
      }
    __syncthreads();
  }
}
template <int D, bool FP16>
cudaError_t launch_join(const DecParams& p, int rows_per_unit, cudaStream_t stream) {
  const unsigned heads = static_cast<unsigned>(p.c.B) * static_cast<unsigned>(p.H), most = static_cast<unsigned>(sm_count()) * 16;
  return launch_dependent(decode_join_kernel<D, FP16>, heads < most ? heads : most, 128, 0, stream, p, rows_per_unit);
}

// The parts of a decode: two a CTA.
inline size_t part_bytes(int rows_per_sm, int d) {
  return (static_cast<size_t>(2) * rows_per_sm * sm_count() * (d + 2) * sizeof(float) + 255) / 256 * 256;
}
// With the tiles before each sequence and the share.
inline size_t decode_workspace(int rows_per_sm, int B, int d) {
  return part_bytes(rows_per_sm, d) + (static_cast<size_t>(B) + 2) * sizeof(long long);
}

// Of units of `rows` heads, in `per_sm` CTAs an SM.
inline DecParams decode_params(const PagedDecodeArgs& a, int rows, int tile, int part_rows, int per_sm) {
  DecParams p{};
  p.c = a.c;
  p.q = static_cast<const uint16_t*>(a.q);
  p.o = static_cast<uint16_t*>(a.o);
  p.sq = a.sq;
  p.so = a.so;
  p.lse = a.lse;
  p.H = a.H;
  p.group = a.H / a.c.Hkv;
  p.chunks = (p.group + rows - 1) / rows;
  p.part_rows = part_rows;
  p.part = static_cast<float*>(a.workspace);
  p.offsets = reinterpret_cast<long long*>(static_cast<uint8_t*>(a.workspace) + part_bytes(per_sm * part_rows, a.c.d));
  // The tokens of one page inside a tile: the largest power of two that divides both.
  p.piece = std::min(tile, a.c.page_size & -a.c.page_size);
  p.scale_log2 = a.scale * kLog2e;
  if (a.softcap > 0.f) {
    p.cap_in = 4.f * a.scale / a.softcap;  // products to x = 4 u (fa_score.cuh)
    p.cap_out = a.softcap * kLog2e;
    p.poly = cap_poly(p.cap_out);
  }
  p.slopes = a.slopes;
  p.err_word = a.err_word;
  p.wait_ns = a.dbg.wait_limit_ns;
  return p;
}

}  // namespace
}  // namespace fa
