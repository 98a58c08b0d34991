// Queries and keys of a layer as attention takes them (include/fa.h, fa_qk_norm_rope): the
// norm of every head's row, its weights, and the rotation by the token's position, in one pass
// over q and k together; and the gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  pairs (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c),
//   c, s = cos, sin(position * inv_freq)
// and back, with g the outputs' gradient turned by the opposite angles and h = w g:
//   dx = r (h - x r mean(h x r)),  dw = sum over rows of g x r.
//
// Bound by HBM: 4 bytes a value forward, 6 backward, against 10 to 20 operations.
//
// Work.  A warp takes a token (or, where there are few heads, some) with all its heads, q's and then k's: the angles' sines and
// cosines, the costliest part, are made once for them and stay in registers, as do the weights.  Rows stream through the warp: each lane
// copies its pieces of the next rows into places of its own in shared memory (cp.async: HBM's latency at full rate takes
// more bytes on the way than registers could wait for), over the ends of sides and tokens.  Measured: 16384 tokens of 40 heads
// x 128 in 55 us, 6.1 TB/s; the gradient, 32 heads, in 67, 6.0 TB/s; 16 tokens of 10 heads x 64 in 3.7.  In neighbouring pairs, which do
// not go through the packed products of two values, 76 and 104; half of each head rotated, in halves, 67 and 87.  Times in a graph.  (A block that
// shares its tokens' angles in shared memory and reads them for every row: 62 and 82 us, the reads' bank conflicts being
// most of it; rows kept in registers alone: 76 and 89.)
//
// Angles.  position * inv_freq in fp32 would lose all but a few bits of the angle at far positions.  An angle counts only
// modulo one turn, so the frequency is held in turns a token as a 64-bit fraction, made from inv_freq (a 24-bit integer times
// a power of two) and 1 / 2 pi to 128 bits: the product with the position, modulo 2^64, is the angle with an error below 2^-32 of a
// turn for every 32-bit position, for four integer products a pair.
//
// A row of d = 64 or 128 lies in d / 16 lanes, 16 values each: two pieces of 16 bytes, chosen so that a rotated pair is in one lane
// (halves: pieces l and l + rot / 16, neighbours: pieces 2l and 2l + 1), and sums over a row are three or two shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kQkThreads = 256;

// inv_freq / 2 pi modulo 1, as a 64-bit fraction, of a finite |inv_freq| < 2^64.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
  // 1 / 2 pi = 0x0.28be60db9391054a7f09d5f47d4d3770...
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;
  const uint32_t bits = __float_as_uint(inv_freq);
  const int field = (bits >> 23) & 0xff;
  const uint64_t m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);  // |inv_freq| = m 2^(max(field, 1) - 150)
  // m / 2 pi in 128 bits behind the point and 64 before it.
  const uint64_t p0 = m * kLo, carry = __umul64hi(m, kLo), p1 = m * kHi + carry;
  const uint64_t p2 = __umul64hi(m, kHi) + (p1 < carry ? 1 : 0);
  const int shift = 64 + 150 - max(field, 1);  // down, to 64 bits behind the point: 214 - field
  uint64_t f;
  if (shift >= 192) f = 0;
  else if (shift >= 128) f = p2 >> (shift - 128);
  else if (shift >= 64) f = shift == 64 ? p1 : (p1 >> (shift - 64)) | (p2 << (128 - shift));
  else if (shift >= 1) f = (p0 >> shift) | (p1 << (64 - shift));
  else f = p0;  // (past the documented range)
  return (bits >> 31) ? 0ull - f : f;
}

// cos and sin of position * frequency.
__device__ __forceinline__ float2 turn(uint64_t turns, int position) {
  const uint64_t angle = turns * static_cast<uint64_t>(static_cast<int64_t>(position)) + 0x80000000ull;
  const float half_turns = static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f;
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// Eight 16-bit values as four pairs.
template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& u, float2* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FP16) x[j] = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    else x[j] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]));
  }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float2* x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FP16) {
      const __half2 h = __floats2half2_rn(x[j].x, x[j].y);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[j] = pack_bf16x2(x[j].x, x[j].y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == 0) return __ldg(static_cast<const float*>(w) + i);
  const uint16_t u = __ldg(static_cast<const uint16_t*>(w) + i);
  if (type == 1) return __uint_as_float(static_cast<uint32_t>(u) << 16);
  return __half2float(__ushort_as_half(u));
}

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int w = 1; w < D / 16; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
  return x;
}
__device__ __forceinline__ float dot16(const float2 (&x)[8], const float2 (&y)[8]) {
  float2 s = __fmul2_rn(x[0], y[0]), t = __fmul2_rn(x[1], y[1]);
#pragma unroll
  for (int j = 2; j < 8; j += 2) {
    s = __ffma2_rn(x[j], y[j], s);
    t = __ffma2_rn(x[j + 1], y[j + 1], t);
  }
  s = __fadd2_rn(s, t);
  return s.x + s.y;
}

// How the rows are divided: a warp takes at once `heads` heads (a power of two) of 32 / (D / 16) / heads tokens; the warps of one
// token's slices take its heads in turns.
struct QkGrid {
  int heads, slices;
  Div per_row;    // by N
  int step;       // heads * slices
  int rows[2];    // of q's and k's heads that a slice takes, at most: heads / step, rounded up
  long long x_step[2], dy_step[2], out_step[2];  // elements from a warp's row to its next
};
// The rows of a side that this block takes: where there are few tokens, blocks are for q (blockIdx.y = 0) or for k.
__device__ __forceinline__ int rows_of(const QkGrid& g, int side) {
  return gridDim.y == 1 || static_cast<int>(blockIdx.y) == side ? g.rows[side] : 0;
}

// Cosines, sines and their negatives of this lane's eight pairs, in pairs.
struct Angles {
  float2 c[4], s[4], ns[4];
};
// x[8] of a lane turned by them: the pairs are its first piece's values with its second's, or with PAIRS the two of
// each x[j].  Where not all columns are rotated (PART), a lane past those that are (turned false) leaves its values alone:
// times 1 and 0 an infinity would make the value beside it NaN.  A build of its own: with the choice in every row's
// way the gradient of 16384 tokens of 32 heads x 128, whole heads rotated, took 69.9 us for 66.7.
template <bool PAIRS, bool PART>
__device__ __forceinline__ void rotate(float2 (&x)[8], const Angles& g, bool turned) {
  if (PART && !turned) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (PAIRS) {
      float2 &u = x[2 * j], &v = x[2 * j + 1];
      u = make_float2(u.x * g.c[j].x - u.y * g.s[j].x, u.x * g.s[j].x + u.y * g.c[j].x);
      v = make_float2(v.x * g.c[j].y - v.y * g.s[j].y, v.x * g.s[j].y + v.y * g.c[j].y);
    } else {
      const float2 u = x[j], v = x[4 + j];
      x[j] = __ffma2_rn(v, g.ns[j], __fmul2_rn(u, g.c[j]));
      x[4 + j] = __ffma2_rn(u, g.s[j], __fmul2_rn(v, g.c[j]));
    }
  }
}

// 16 bytes of a row (bytes = 16) or of zeros (0) to this lane's own place in shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this lane's copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Rows of a warp in the ring, the one that is worked on among them.  16384 tokens of 40 heads x 128 forward, of 32
// backward: 55.0 and 67.0 us; two rows 65.7 and 74.5, four 59.8 and 67.9 (HBM serves fewer streams at once better).
constexpr int kDepth = 3;
constexpr int kForwardBlocksPerSm = 2, kBackBlocksPerSm = 2;

// This thread's part: its place in its row's lanes and the columns of its two pieces; its row's head and token among the warp's.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 16, kGroups = 32 / kLanes;  // lanes of a row, rows of a warp
  int lane, c0, c1, head, token;
  bool turned;  // its columns are among the rotated (rot is a multiple of 16: all of them or none)
  __device__ __forceinline__ Lane(const QkArgs& a, const QkGrid& g) {
    const int x = threadIdx.x & 31, group = x / kLanes;
    lane = x % kLanes;
    turned = lane < a.rot / 16;
    if (a.pairs || !turned) {
      c0 = 16 * lane;  // (past the rotated columns the pieces of both kinds follow each other)
      c1 = c0 + 8;
    } else {
      c0 = 8 * lane;
      c1 = c0 + a.rot / 2;
    }
    head = group & (g.heads - 1);
    token = group / g.heads;
  }
};

// The rows that a warp takes, in order: token by token (of a step between them), side by side (q, k), heads in steps.
// Fetching runs kDepth - 1 rows ahead of the work.
template <int D, bool BACK>
struct Fetch {
  static constexpr int kParts = BACK ? 4 : 2;  // pieces a lane: of x, and of the gradient
  static constexpr uint32_t kSlot = kParts * kQkThreads * 16;
  const QkArgs& a;
  const QkGrid& g;
  const Lane<D>& me;
  uint32_t begin, to;      // shared memory: this lane's place of slot 0, and of the slot to fill
  int all, token_step, head;
  int token, side;         // of the rows to fetch next
  int left, real;          // of this side: rows that the warp takes, and rows that this lane has
  const uint16_t *x, *dy;  // the next one's first piece
  __device__ __forceinline__ Fetch(const QkArgs& a_, const QkGrid& g_, const Lane<D>& me_, const void* ring, int first, int step,
                                   int slice)
      : a(a_), g(g_), me(me_), begin(smem_u32(ring) + threadIdx.x * 16), to(begin), all(a_.B * a_.N), token_step(step),
        head(slice * g_.heads + me_.head), token(first + me_.token), side(-1) {
    next_side();
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) row();
  }
  __device__ __forceinline__ void next_side() {
    do {
      if (++side == 2) {
        side = 0;
        token += token_step;
      }
      left = rows_of(g, side);
    } while (left == 0);  // (a block without rows does not come here)
    // Heads head, head + step, ... of this side: as many rows as the warp takes, or one less.
    real = token < all ? left - (head + (left - 1) * g.step < (side ? a.Hkv : a.H) ? 0 : 1) : 0;
    const int at = min(token, all - 1), b = g.per_row(at), n = at - b * a.N;
    auto start = [&](const void* base, const Strides& s) {
      return static_cast<const uint16_t*>(base) + (b * s.s[2] + n * s.s[0] + head * s.s[1] + me.c0);
    };
    if (!BACK || a.norm) x = side ? start(a.k, a.sk) : start(a.q, a.sq);
    if constexpr (BACK) dy = side ? start(a.dk_in, a.sdk_in) : start(a.dq_in, a.sdq_in);
  }
  // Asks for a row (for zeros where this lane has none) and goes to the next.
  __device__ __forceinline__ void row() {
    const uint32_t bytes = real > 0 ? 16 : 0;
    if (!BACK || a.norm) {
      copy16(to, x, bytes);
      copy16(to + 16 * kQkThreads, x + (me.c1 - me.c0), bytes);
      x += side ? g.x_step[1] : g.x_step[0];
    }
    if constexpr (BACK) {
      copy16(to + 32 * kQkThreads, dy, bytes);
      copy16(to + 48 * kQkThreads, dy + (me.c1 - me.c0), bytes);
      dy += side ? g.dy_step[1] : g.dy_step[0];
    }
    copies_end();
    to = to == begin + (kDepth - 1) * kSlot ? begin : to + kSlot;
    --real;
    if (--left == 0) next_side();
  }
};

// The angles of a warp's tokens: each lane makes those of one or two pairs, all read theirs.
template <int D>
struct Turns {
  static constexpr int kPairs = D / 2, kOwn = kPairs / 32;
  uint64_t turns[kOwn];
  __device__ __forceinline__ explicit Turns(const QkArgs& a) {
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      const int i = (threadIdx.x & 31) + 32 * k;
      turns[k] = i < a.rot / 2 ? turns_of(__ldg(a.inv_freq + i)) : 0;
    }
  }
  template <bool BACK>
  __device__ __forceinline__ Angles of(const QkArgs& a, const QkGrid& g, const Lane<D>& me, float2* mine, int first) const {
    constexpr int kMost = Lane<D>::kGroups;
    const int all = a.B * a.N, tokens = kMost / g.heads, lane = threadIdx.x & 31;
    int pos[kMost];
#pragma unroll
    for (int t = 0; t < kMost; ++t) {
      const int at = min(first + t, all - 1);
      if (t < tokens) pos[t] = a.positions ? __ldg(a.positions + at) : at - g.per_row(at) * a.N;
    }
    __syncwarp();  // every lane has read the angles before
#pragma unroll
    for (int t = 0; t < kMost; ++t)
      if (t < tokens) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) mine[t * kPairs + lane + 32 * k] = turn(turns[k], pos[t]);
      }
    __syncwarp();
    const float4* from = reinterpret_cast<const float4*>(mine + me.token * kPairs + 8 * me.lane);
    Angles r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 y = from[j];
      r.c[j] = make_float2(y.x, y.z);
      r.s[j] = BACK ? make_float2(-y.y, -y.w) : make_float2(y.y, y.w);
      r.ns[j] = make_float2(-r.s[j].x, -r.s[j].y);
    }
    return r;
  }
};

// The weights (1 without) in shared memory, and this lane's.
template <int D>
__device__ __forceinline__ void make_weights(float (&w)[2][D], const QkArgs& a) {
  for (int x = threadIdx.x; x < 2 * D; x += kQkThreads) {
    const void* from = x < D ? a.q_weight : a.k_weight;
    w[x / D][x % D] = from ? weight_at(from, a.weight_type, x % D) : 1.f;
  }
}
template <int D>
__device__ __forceinline__ void load_weights(const float (&in)[2][D], const Lane<D>& me, int side, float2 (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float4 x = *reinterpret_cast<const float4*>(&in[side][j < 4 ? me.c0 + 2 * j : me.c1 + 2 * (j - 4)]);
    w[j] = make_float2(x.x, x.y);
    w[j + 1] = make_float2(x.z, x.w);
  }
}

// This lane's first piece of its slice's first head in token first + me.token (the last there is, if none) of an output.
template <int D>
__device__ __forceinline__ uint16_t* out_row(const QkArgs& a, const QkGrid& g, const Lane<D>& me, int first, int side, int slice) {
  const int at = min(first + me.token, a.B * a.N - 1), b = g.per_row(at), n = at - b * a.N;
  const Strides& s = side ? a.sk_out : a.sq_out;
  return static_cast<uint16_t*>(side ? a.k_out : a.q_out) +
         (b * s.s[2] + n * s.s[0] + (slice * g.heads + me.head) * s.s[1] + me.c0);
}

// Where a warp begins and what it takes.
struct Share {
  int slice, begin, step;
  bool any;
  __device__ __forceinline__ Share(const QkGrid& g, int tokens, int all) {
    const int unit = blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5), units = gridDim.x * (kQkThreads / 32);
    const int lines = units / g.slices;  // warps that take the same slice
    begin = unit / g.slices;
    slice = unit - begin * g.slices;
    any = begin < lines;
    begin *= tokens;
    step = lines * tokens;
    any = any && begin < all && (rows_of(g, 0) > 0 || rows_of(g, 1) > 0);
  }
};

template <int D, bool FP16, bool PAIRS, bool PART>
__global__ void __launch_bounds__(kQkThreads, kForwardBlocksPerSm)
    qk_forward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkGrid g) {
  __shared__ __align__(16) float2 angles[kQkThreads / 32][Lane<D>::kGroups * D / 2];
  __shared__ __align__(16) float weights[2][D];
  extern __shared__ uint4 ring[];
  if (a.norm) {
    make_weights<D>(weights, a);
    __syncthreads();
  }
  const Lane<D> me(a, g);
  const int all = a.B * a.N;
  const Share mine(g, Lane<D>::kGroups / g.heads, all);
  if (!mine.any) return;
  Fetch<D, false> fetch(a, g, me, ring, mine.begin, mine.step, mine.slice);
  const Turns<D> turns(a);
  uint32_t slot = threadIdx.x;
  for (int first = mine.begin; first < all; first += mine.step) {
    const Angles turn_by = turns.template of<false>(a, g, me, angles[threadIdx.x >> 5], first);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int heads = side ? a.Hkv : a.H, rows = rows_of(g, side);
      if (rows == 0) continue;
      uint16_t* out = out_row<D>(a, g, me, first, side, mine.slice);
      const long long out_step = side ? g.out_step[1] : g.out_step[0];
      int h = first + me.token < all ? mine.slice * g.heads + me.head : heads;  // (no token: no head)
      float2 w[8];
      if (a.norm) load_weights<D>(weights, me, side, w);
      for (int left = rows; left > 0; --left, h += g.step, out += out_step) {
        copies_wait<kDepth - 2>();
        const uint4* from = ring + slot;
        slot = slot == (kDepth - 1) * 2 * kQkThreads + threadIdx.x ? threadIdx.x : slot + 2 * kQkThreads;
        float2 x[8];
        unpack8<FP16>(from[0], x);
        unpack8<FP16>(from[kQkThreads], x + 4);
        fetch.row();   // into the place of the row before this one
        if (a.norm) {  // (the root comes last: the rotation does not wait for it)
          const float2 r = twice(rsqrtf(row_sum<D>(dot16(x, x)) * (1.f / D) + a.eps));
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __fmul2_rn(x[j], w[j]);
          rotate<PAIRS, PART>(x, turn_by, me.turned);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __fmul2_rn(x[j], r);
        } else {
          rotate<PAIRS, PART>(x, turn_by, me.turned);
        }
        if (h < heads) {
          *reinterpret_cast<uint4*>(out) = pack8<FP16>(x);
          *reinterpret_cast<uint4*>(out + (me.c1 - me.c0)) = pack8<FP16>(x + 4);
        }
      }
    }
  }
}

// The gradient.  Blocks stay on the GPU and their warps take tokens in turn, so that the weights' gradients add up in a thread; each
// block's sums go to the workspace and a second kernel adds them in order: the same bits on every run.  A thread's sums of the side that
// it is not at lie in shared memory: 16 registers less.
template <int D, bool FP16, bool PAIRS, bool PART>
__global__ void __launch_bounds__(kQkThreads, 2) qk_backward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkGrid g) {
  __shared__ __align__(16) float2 angles[kQkThreads / 32][Lane<D>::kGroups * D / 2];
  __shared__ __align__(16) float weights[2][D];
  extern __shared__ float4 sums[];  // [2][4][kQkThreads], then the ring
  uint4* ring = reinterpret_cast<uint4*>(sums + 8 * kQkThreads);
  const Lane<D> me(a, g);
  const int all = a.B * a.N;
  const Share mine(g, Lane<D>::kGroups / g.heads, all);
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[i * kQkThreads + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.norm) {
    make_weights<D>(weights, a);
    __syncthreads();
  }
  if (mine.any) {
    Fetch<D, true> fetch(a, g, me, ring, mine.begin, mine.step, mine.slice);
    const Turns<D> turns(a);
    uint32_t slot = threadIdx.x;
    for (int first = mine.begin; first < all; first += mine.step) {
      const Angles turn_by = turns.template of<true>(a, g, me, angles[threadIdx.x >> 5], first);
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        const int heads = side ? a.Hkv : a.H, rows = rows_of(g, side);
        if (rows == 0) continue;
        uint16_t* out = out_row<D>(a, g, me, first, side, mine.slice);
        const long long out_step = side ? g.out_step[1] : g.out_step[0];
        int h = first + me.token < all ? mine.slice * g.heads + me.head : heads;  // (no token: no head)
        float2 w[8], dw[8];
        if (a.norm) load_weights<D>(weights, me, side, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 s = sums[(4 * side + i) * kQkThreads + threadIdx.x];
          dw[2 * i] = make_float2(s.x, s.y);
          dw[2 * i + 1] = make_float2(s.z, s.w);
        }
        for (int left = rows; left > 0; --left, h += g.step, out += out_step) {
          copies_wait<kDepth - 2>();
          const uint4* from = ring + slot;
          slot = slot == (kDepth - 1) * 4 * kQkThreads + threadIdx.x ? threadIdx.x : slot + 4 * kQkThreads;
          float2 x[8], y[8];
          unpack8<FP16>(from[2 * kQkThreads], y);
          unpack8<FP16>(from[3 * kQkThreads], y + 4);
          if (a.norm) {
            unpack8<FP16>(from[0], x);
            unpack8<FP16>(from[kQkThreads], x + 4);
          }
          fetch.row();  // into the place of the row before this one
          rotate<PAIRS, PART>(y, turn_by, me.turned);
          if (a.norm) {
            const float2 r = twice(rsqrtf(row_sum<D>(dot16(x, x)) * (1.f / D) + a.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              x[j] = __fmul2_rn(x[j], r);
              dw[j] = __ffma2_rn(y[j], x[j], dw[j]);
              y[j] = __fmul2_rn(y[j], w[j]);
            }
            const float2 dot = twice(row_sum<D>(dot16(x, y)) * (-1.f / D));
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fmul2_rn(__ffma2_rn(dot, x[j], y[j]), r);
          }
          if (h < heads) {
            *reinterpret_cast<uint4*>(out) = pack8<FP16>(y);
            *reinterpret_cast<uint4*>(out + (me.c1 - me.c0)) = pack8<FP16>(y + 4);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sums[(4 * side + i) * kQkThreads + threadIdx.x] = make_float4(dw[2 * i].x, dw[2 * i].y, dw[2 * i + 1].x, dw[2 * i + 1].y);
      }
    }
  }
  grid_release();
  if (!a.dq_weight && !a.dk_weight) return;
  // This block's sums: column i of a side over all rows' lanes.
  __syncthreads();
  float* part = static_cast<float*>(a.workspace) + static_cast<size_t>(blockIdx.y * gridDim.x + blockIdx.x) * 2 * D;
  for (int x = threadIdx.x; x < 2 * D; x += kQkThreads) {
    const int side = x / D, i = x % D;
    // The lane and place whose pieces hold the column.
    int lane, j;
    if (a.pairs || i >= a.rot) {
      lane = i / 16;
      j = i % 16;
    } else {
      const int half = i >= a.rot / 2, k = i - half * (a.rot / 2);
      lane = k / 8;
      j = k % 8 + 8 * half;
    }
    const float* from = reinterpret_cast<const float*>(sums + (4 * side + j / 4) * kQkThreads) + j % 4;
    float sum = 0.f;
#pragma unroll 8
    for (int k = lane; k < kQkThreads; k += Lane<D>::kLanes) sum += from[4 * k];
    part[x] = sum;
  }
}

// The blocks' sums: one block for q's weights and one for k's, a thread a column and every 1024 / D-th part.
template <int D>
__global__ void __launch_bounds__(1024) qk_weights_kernel(const __grid_constant__ QkArgs a, int parts) {
  __shared__ float s_sum[1024 / D][D];
  grid_wait();
  const int side = blockIdx.x, col = threadIdx.x % D, from = threadIdx.x / D;
  float* out = side ? a.dk_weight : a.dq_weight;
  if (!out) return;
  const float* part = static_cast<const float*>(a.workspace) + side * D + col;
  float x = 0.f;
#pragma unroll 8
  for (int i = from; i < parts; i += 1024 / D) x += part[static_cast<size_t>(i) * 2 * D];
  s_sum[from][col] = x;
  __syncthreads();
  if (from == 0) {
#pragma unroll
    for (int k = 1; k < 1024 / D; ++k) x += s_sum[k][col];
    out[col] = x;
  }
}

constexpr size_t kFetched = kDepth * 2 * kQkThreads * sizeof(uint4);  // the forward's; the backward's is twice that
constexpr size_t kSums = 8 * kQkThreads * sizeof(float4);

// As many heads at once as keep at most an eighth more rows than there are (few heads: more tokens instead), as long as there
// are tokens for `most` warps; and slices of the heads where there are fewer.
template <int D>
QkGrid grid_of(const QkArgs& a, long long most, dim3* blocks) {
  constexpr int kGroups = Lane<D>::kGroups, kWarps = kQkThreads / 32;
  const long long all = static_cast<long long>(a.B) * a.N;
  int heads = kGroups;
  auto steps = [](int n, int step) { return (n + step - 1) / step; };
  auto rows = [&](int n) { return (steps(a.H, n) + steps(a.Hkv, n)) * n; };
  auto units = [&](int n) { return std::max(1LL, (all + kGroups / n - 1) / (kGroups / n)); };
  while (heads > 1 && 8 * rows(heads) > 9 * (a.H + a.Hkv) && units(heads / 2) >= most) heads /= 2;
  QkGrid g{};
  g.heads = heads;
  g.slices = static_cast<int>(std::max(1LL, std::min<long long>(std::max(steps(a.H, heads), steps(a.Hkv, heads)), most / units(heads))));
  g.per_row = Div(std::max(a.N, 1));
  g.step = heads * g.slices;
  g.rows[0] = steps(a.H, g.step);
  g.rows[1] = steps(a.Hkv, g.step);
  const Strides* each[3][2] = {{&a.sq, &a.sk}, {&a.sdq_in, &a.sdk_in}, {&a.sq_out, &a.sk_out}};
  for (int side = 0; side < 2; ++side) {
    g.x_step[side] = each[0][side]->s[1] * g.step;
    g.dy_step[side] = each[1][side]->s[1] * g.step;
    g.out_step[side] = each[2][side]->s[1] * g.step;
  }
  // The same number of tokens to every warp.
  const long long lines = units(heads) * g.slices, rounds = (lines + most - 1) / most;
  *blocks = dim3(static_cast<unsigned>(((lines + rounds - 1) / rounds + kWarps - 1) / kWarps), 2 * lines <= most ? 2 : 1);
  return g;
}

template <int D, bool FP16, bool PAIRS, bool PART>
cudaError_t launch_forward(const QkArgs& a, cudaStream_t stream) {
  dim3 blocks;
  const QkGrid g = grid_of<D>(a, static_cast<long long>(sm_count()) * kForwardBlocksPerSm * (kQkThreads / 32), &blocks);
  qk_forward_kernel<D, FP16, PAIRS, PART><<<blocks, kQkThreads, kFetched, stream>>>(a, g);  // (48 KB with what is static: no attribute)
  return cudaGetLastError();
}

template <int D, bool FP16, bool PAIRS, bool PART>
cudaError_t launch_backward(const QkArgs& a, cudaStream_t stream) {
  dim3 blocks;
  const QkGrid g = grid_of<D>(a, static_cast<long long>(sm_count()) * kBackBlocksPerSm * (kQkThreads / 32), &blocks);
  auto kern = qk_backward_kernel<D, FP16, PAIRS, PART>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSums + 2 * kFetched));
  if (e) return e;
  kern<<<blocks, kQkThreads, kSums + 2 * kFetched, stream>>>(a, g);
  e = cudaGetLastError();
  if (e || (!a.dq_weight && !a.dk_weight)) return e;
  return launch_dependent(qk_weights_kernel<D>, 2, 1024, 0, stream, a, static_cast<int>(blocks.x * blocks.y));
}

template <int D, bool FP16, bool PAIRS>
cudaError_t launch(const QkArgs& a, bool back, cudaStream_t stream) {
  if (a.rot < D) return back ? launch_backward<D, FP16, PAIRS, true>(a, stream) : launch_forward<D, FP16, PAIRS, true>(a, stream);
  return back ? launch_backward<D, FP16, PAIRS, false>(a, stream) : launch_forward<D, FP16, PAIRS, false>(a, stream);
}
template <int D, bool FP16>
cudaError_t launch(const QkArgs& a, bool back, cudaStream_t stream) {
  return a.pairs ? launch<D, FP16, true>(a, back, stream) : launch<D, FP16, false>(a, back, stream);
}
cudaError_t launch(const QkArgs& a, bool back, cudaStream_t stream) {
  if (a.d == 64) return a.fp16 ? launch<64, true>(a, back, stream) : launch<64, false>(a, back, stream);
  return a.fp16 ? launch<128, true>(a, back, stream) : launch<128, false>(a, back, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs& a, cudaStream_t stream) { return launch(a, false, stream); }
size_t qk_norm_rope_bwd_workspace(int d) {
  return static_cast<size_t>(sm_count()) * kBackBlocksPerSm * 2 * d * sizeof(float);
}
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, cudaStream_t stream) { return launch(a, true, stream); }

}  // namespace fa
