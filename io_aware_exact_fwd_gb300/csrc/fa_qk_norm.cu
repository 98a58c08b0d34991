// Queries and keys of a layer as attention takes them (include/fa.h, fa_qk_norm_rope): the
// norm of every head's row, its weights, and the rotation by the token's position, in one pass
// over q and k together; and the gradient.
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r w,  pairs (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c),
//   c, s = cos, sin(position * inv_freq)
// and back, with g the outputs' gradient turned by the opposite angles and h = w g:
//   dx = r (h - x r mean(h x r)),  dw = sum over rows of g x r.
//
// Bound by HBM: 4 bytes a value forward, 6 backward, against 10 to 20 operations.  The angles are what could cost more: a sine and a cosine
// for each pair and token, so a block makes them once for its tokens, in shared memory, for all their heads.
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

// x / n for 0 <= x < 2^31 by a product: with s the least number such that n <= 2^s, ceil(2^(31 + s) / n) has 32 bits.
struct Div {
  uint32_t by, shift;
  Div() = default;
  explicit Div(int n) {
    int s = 0;
    while ((1ll << s) < n) ++s;
    shift = static_cast<uint32_t>(31 + s);
    by = static_cast<uint32_t>(((1ull << shift) + n - 1) / n);
  }
  __device__ __forceinline__ int operator()(int x) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(x)) * by >> shift);
  }
};

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

template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 f;
    if constexpr (FP16) f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]));
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (FP16) {
      const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float weight_at(const void* w, int type, int i) {
  if (type == 0) return static_cast<const float*>(w)[i];
  const uint16_t u = static_cast<const uint16_t*>(w)[i];
  if (type == 1) return __uint_as_float(static_cast<uint32_t>(u) << 16);
  return __half2float(__ushort_as_half(u));
}

// A row's layout in its lanes.
template <int D>
struct Rows {
  static constexpr int kLanes = D / 16;                  // of a row
  static constexpr int kGroups = kQkThreads / kLanes;    // rows at once
  int lane, group, c0, c1;                               // this thread's place in its row, its row, the columns of its two pieces
  bool turned;
  __device__ __forceinline__ explicit Rows(const QkArgs& a) {
    lane = threadIdx.x % kLanes;
    group = threadIdx.x / kLanes;
    turned = lane < a.rot / 16;
    if (a.pairs || !turned) {
      c0 = 16 * lane;  // (past the rotated columns the pieces of both kinds follow each other)
      c1 = c0 + 8;
    } else {
      c0 = 8 * lane;
      c1 = c0 + a.rot / 2;
    }
  }
};

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int w = 1; w < D / 16; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
  return x;
}

// x[16] of a lane: the pairs (x[j], x[8 + j]), or with PAIRS (x[2j], x[2j + 1]), turned by (c[j], s[j]).
template <bool PAIRS>
__device__ __forceinline__ void rotate(float (&x)[16], const float (&c)[8], const float (&s)[8], float sign) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float &a = x[PAIRS ? 2 * j : j], &b = x[PAIRS ? 2 * j + 1 : 8 + j];
    const float sj = sign * s[j], y = a * c[j] - b * sj;
    b = a * sj + b * c[j];
    a = y;
  }
}

constexpr int kMostTokens = 8;  // of a tile

template <int D>
struct Angles {
  float c[kMostTokens][D / 2], s[kMostTokens][D / 2];
};
// Of tokens first .. first + tokens of the line of all.
template <int D>
__device__ __forceinline__ void make_angles(Angles<D>& x, const QkArgs& a, const Div& per_row, int first, int tokens) {
  const int half = a.rot / 2;
  for (int y = threadIdx.x; y < tokens * half; y += kQkThreads) {
    const int t = y / half, i = y % half, at = first + t;
    const int pos = a.positions ? __ldg(a.positions + at) : at - per_row(at) * a.N;
    const float2 cs = turn(turns_of(__ldg(a.inv_freq + i)), pos);
    x.c[t][i] = cs.x;
    x.s[t][i] = cs.y;
  }
}
template <int D>
__device__ __forceinline__ void angles_of(const Angles<D>& x, const Rows<D>& me, int t, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 y = *reinterpret_cast<const float4*>(&x.c[t][8 * me.lane + j]);
    const float4 z = *reinterpret_cast<const float4*>(&x.s[t][8 * me.lane + j]);
    c[j] = me.turned ? y.x : 1.f;
    c[j + 1] = me.turned ? y.y : 1.f;
    c[j + 2] = me.turned ? y.z : 1.f;
    c[j + 3] = me.turned ? y.w : 1.f;
    s[j] = me.turned ? z.x : 0.f;
    s[j + 1] = me.turned ? z.y : 0.f;
    s[j + 2] = me.turned ? z.z : 0.f;
    s[j + 3] = me.turned ? z.w : 0.f;
  }
}

template <int D>
__device__ __forceinline__ void make_weights(float (&w)[2][D], const QkArgs& a) {
  for (int x = threadIdx.x; x < 2 * D; x += kQkThreads) {
    const void* from = x < D ? a.q_weight : a.k_weight;
    w[x / D][x % D] = from ? weight_at(from, a.weight_type, x % D) : 1.f;
  }
}
template <int D>
__device__ __forceinline__ void weights_of(const float (&in)[2][D], const Rows<D>& me, int side, float (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 x = *reinterpret_cast<const float4*>(&in[side][me.c0 + j]);
    const float4 y = *reinterpret_cast<const float4*>(&in[side][me.c1 + j]);
    w[j] = x.x;
    w[j + 1] = x.y;
    w[j + 2] = x.z;
    w[j + 3] = x.w;
    w[8 + j] = y.x;
    w[9 + j] = y.y;
    w[10 + j] = y.z;
    w[11 + j] = y.w;
  }
}

// How the grid divides the rows: tiles of `tokens` tokens and (forward) `heads` heads of q's and k's in one line.
struct QkGrid {
  int tokens, heads, slices;
  bool heads_first;  // rows that follow each other are heads of a token
  Div per_row;       // by N
};

// The rows of a tile and some heads, kGroups at a time: this thread's place among them, with no division after the first.
struct Walk {
  int minor, major, minors, majors, step_minor, step_major;
  __device__ __forceinline__ void start(int group, int groups, int tokens, int heads, bool heads_first) {
    minors = heads_first ? heads : tokens;
    majors = heads_first ? tokens : heads;
    minor = group % minors;
    major = group / minors;
    step_minor = groups % minors;
    step_major = groups / minors;
  }
  __device__ __forceinline__ void step() {
    minor += step_minor;
    major += step_major;
    if (minor >= minors) {
      minor -= minors;
      ++major;
    }
  }
  __device__ __forceinline__ bool real() const { return major < majors; }
};

__device__ __forceinline__ long long row_at(const Strides& s, int b, int n, int h) {
  return b * s.s[2] + n * s.s[0] + h * s.s[1];
}

// Two pieces of a row.
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ Raw load_row(const void* base, long long at, int c0, int c1) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  return Raw{__ldcs(reinterpret_cast<const uint4*>(p + c0)), __ldcs(reinterpret_cast<const uint4*>(p + c1))};
}

// The forward.  A block's rows stream through its threads, the next ones' loads in flight while this one is worked on; the
// first are requested before the angles are made.
template <int D, bool FP16, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads, 4) qk_forward_kernel(const __grid_constant__ QkArgs a, const QkGrid g) {
  __shared__ __align__(16) Angles<D> angles;
  __shared__ __align__(16) float weights[2][D];
  using R = Rows<D>;
  const R me(a);
  const int tile = blockIdx.x / g.slices, first = tile * g.tokens, tokens = min(g.tokens, a.B * a.N - first);
  const int h0 = (blockIdx.x - tile * g.slices) * g.heads, heads = min(g.heads, a.H + a.Hkv - h0);
  Walk at;
  at.start(me.group, R::kGroups, tokens, heads, g.heads_first);
  // A row: its token in the tile, whether it is k's, its head there; and its pieces.
  struct Row {
    int t, side, head, b, n;
    bool real;
  };
  auto here = [&]() {
    Row r;
    r.real = at.real();
    const int minor = r.real ? at.minor : 0, major = r.real ? at.major : 0;
    r.t = g.heads_first ? major : minor;
    const int h = h0 + (g.heads_first ? minor : major);
    r.side = h >= a.H;
    r.head = r.side ? h - a.H : h;
    r.b = g.per_row(first + r.t);
    r.n = first + r.t - r.b * a.N;
    return r;
  };
  auto load = [&](const Row& r) {
    return load_row(r.side ? a.k : a.q, row_at(r.side ? a.sk : a.sq, r.b, r.n, r.head), me.c0, me.c1);
  };
  Row row = here();
  Raw raw = load(row);
  make_angles<D>(angles, a, g.per_row, first, tokens);
  make_weights<D>(weights, a);
  __syncthreads();
  for (int r0 = 0, rows = tokens * heads; r0 < rows; r0 += R::kGroups) {  // (a whole warp goes through: the sums are shuffles)
    at.step();
    const Row next = here();
    Raw ahead = raw;
    if (r0 + R::kGroups < rows) ahead = load(next);
    float x[16];
    unpack8<FP16>(raw.a, x);
    unpack8<FP16>(raw.b, x + 8);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
      const float r_norm = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
      float w[16];
      weights_of<D>(weights, me, row.side, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= r_norm * w[j];
    }
    float c[8], s[8];
    angles_of<D>(angles, me, row.t, c, s);
    rotate<PAIRS>(x, c, s, 1.f);
    if (row.real) {
      uint16_t* out = static_cast<uint16_t*>(row.side ? a.k_out : a.q_out) +
                      row_at(row.side ? a.sk_out : a.sq_out, row.b, row.n, row.head);
      *reinterpret_cast<uint4*>(out + me.c0) = pack8<FP16>(x);
      *reinterpret_cast<uint4*>(out + me.c1) = pack8<FP16>(x + 8);
    }
    row = next;
    raw = ahead;
  }
}

// The gradient.  Blocks stay on the GPU and take tiles of tokens in turn, so that the weights' gradients add up in a thread; each block's
// sums go to the workspace and a second kernel adds them in order: the same bits on every run.  Rows stream as in the forward, over the
// ends of sides (q, then k) and tiles too.  A thread's sums of the side that it is not at lie in shared memory: 16 registers less.
template <int D, bool FP16, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads, 2) qk_backward_kernel(const __grid_constant__ QkArgs a, const QkGrid g) {
  __shared__ __align__(16) Angles<D> angles[2];
  __shared__ __align__(16) float weights[2][D];
  __shared__ float4 sums[2][4][kQkThreads];
  using R = Rows<D>;
  const R me(a);
  const int all = a.B * a.N, tiles = (all + g.tokens - 1) / g.tokens;
  // The place of the rows that are being loaded: a tile, a side, a pass of the walk through its rows.
  struct Place {
    int tile, side, left;  // passes left
    Walk at;
    int t, head, b, n;
    bool real;
  } ahead;
  auto enter = [&]() {  // to the first pass of (tile, side), or of the next that has rows
    for (; ahead.tile < tiles; ahead.tile += gridDim.x, ahead.side = 0)
      for (; ahead.side < 2; ++ahead.side) {
        const int tokens = min(g.tokens, all - ahead.tile * g.tokens), heads = ahead.side ? a.Hkv : a.H;
        ahead.left = (tokens * heads + R::kGroups - 1) / R::kGroups;
        if (ahead.left == 0) continue;
        ahead.at.start(me.group, R::kGroups, tokens, heads, g.heads_first);
        return;
      }
  };
  Raw raw_x, raw_g;
  auto load = [&]() {
    if (ahead.tile >= tiles) return;
    ahead.real = ahead.at.real();
    ahead.t = !ahead.real ? 0 : g.heads_first ? ahead.at.major : ahead.at.minor;
    ahead.head = !ahead.real ? 0 : g.heads_first ? ahead.at.minor : ahead.at.major;
    const int at = ahead.tile * g.tokens + ahead.t;
    ahead.b = g.per_row(at);
    ahead.n = at - ahead.b * a.N;
    const bool k = ahead.side;
    raw_x = raw_g = Raw{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (ahead.real) {  // (a row that is none: zeros, which add nothing to the sums)
      raw_g = load_row(k ? a.dk_in : a.dq_in, row_at(k ? a.sdk_in : a.sdq_in, ahead.b, ahead.n, ahead.head), me.c0, me.c1);
      if (a.norm) raw_x = load_row(k ? a.k : a.q, row_at(k ? a.sk : a.sq, ahead.b, ahead.n, ahead.head), me.c0, me.c1);
    }
  };
  ahead.tile = blockIdx.x;
  ahead.side = 0;
  enter();
  load();
  make_weights<D>(weights, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[i / 4][i % 4][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  int buffer = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buffer ^= 1) {
    make_angles<D>(angles[buffer], a, g.per_row, tile * g.tokens, min(g.tokens, all - tile * g.tokens));
    __syncthreads();  // (and the buffer of the tile before the last is free)
    for (int side = 0; side < 2; ++side) {
      if (ahead.tile != tile || ahead.side != side) continue;  // no rows on this side
      uint16_t* outs = static_cast<uint16_t*>(side ? a.k_out : a.q_out);
      const Strides& so = side ? a.sk_out : a.sq_out;
      float dw[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(dw + 4 * i) = sums[side][i][threadIdx.x];
      for (bool last = false; !last;) {
        float x[16], y[16], c[8], s[8];
        unpack8<FP16>(raw_g.a, y);
        unpack8<FP16>(raw_g.b, y + 8);
        unpack8<FP16>(raw_x.a, x);
        unpack8<FP16>(raw_x.b, x + 8);
        const bool real = ahead.real;
        const int t = ahead.t;
        uint16_t* out = outs + row_at(so, ahead.b, ahead.n, ahead.head);
        last = --ahead.left == 0;
        if (last) {
          ++ahead.side;
          enter();
        } else {
          ahead.at.step();
        }
        load();
        angles_of<D>(angles[buffer], me, t, c, s);
        rotate<PAIRS>(y, c, s, -1.f);
        if (a.norm) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
          const float r_norm = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
          float w[16], dot = 0.f;
          weights_of<D>(weights, me, side, w);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            x[j] *= r_norm;
            dw[j] = fmaf(y[j], x[j], dw[j]);
            y[j] *= w[j];
            dot = fmaf(y[j], x[j], dot);
          }
          dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = r_norm * fmaf(-dot, x[j], y[j]);
        }
        if (real) {
          *reinterpret_cast<uint4*>(out + me.c0) = pack8<FP16>(y);
          *reinterpret_cast<uint4*>(out + me.c1) = pack8<FP16>(y + 8);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[side][i][threadIdx.x] = *reinterpret_cast<float4*>(dw + 4 * i);
    }
  }
  grid_release();
  if (!a.dq_weight && !a.dk_weight) return;
  // This block's sums: column i of a side over all groups of lanes.
  __syncthreads();
  float* part = static_cast<float*>(a.workspace) + static_cast<size_t>(blockIdx.x) * 2 * D;
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
    const float* from = reinterpret_cast<const float*>(&sums[side][j / 4][0]) + j % 4;
    float sum = 0.f;
#pragma unroll 8
    for (int k = 0; k < R::kGroups; ++k) sum += from[4 * (k * R::kLanes + lane)];
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

constexpr int kBackBlocksPerSm = 2;

bool heads_first(const QkArgs& a) { return a.sq.s[1] < a.sq.s[0]; }

template <int D, bool FP16, bool PAIRS>
cudaError_t launch_forward(const QkArgs& a, cudaStream_t stream) {
  constexpr int kGroups = Rows<D>::kGroups;
  const long long all = static_cast<long long>(a.B) * a.N;
  const int sms = sm_count(), heads = a.H + a.Hkv;
  QkGrid g{kMostTokens, heads, 1, heads_first(a), Div(a.N)};
  while (g.tokens > 1 && (all + g.tokens - 1) / g.tokens < 4LL * sms) g.tokens /= 2;
  if (g.tokens == 1) {
    // Too few tokens for the SMs: their heads in slices of one row a group at least.
    const long long want = std::max(1LL, 4LL * sms / all);
    g.slices = static_cast<int>(std::min<long long>(want, (heads + kGroups - 1) / kGroups));
    g.heads = (heads + g.slices - 1) / g.slices;
    g.slices = (heads + g.heads - 1) / g.heads;
  }
  const long long blocks = (all + g.tokens - 1) / g.tokens * g.slices;
  qk_forward_kernel<D, FP16, PAIRS><<<static_cast<unsigned>(blocks), kQkThreads, 0, stream>>>(a, g);
  return cudaGetLastError();
}

template <int D, bool FP16, bool PAIRS>
cudaError_t launch_backward(const QkArgs& a, cudaStream_t stream) {
  const long long all = static_cast<long long>(a.B) * a.N;
  const int most = sm_count() * kBackBlocksPerSm;
  QkGrid g{kMostTokens, 0, 1, heads_first(a), Div(a.N)};
  while (g.tokens > 1 && (all + g.tokens - 1) / g.tokens < most) g.tokens /= 2;
  const int blocks = static_cast<int>(std::max(1LL, std::min<long long>(most, (all + g.tokens - 1) / g.tokens)));
  qk_backward_kernel<D, FP16, PAIRS><<<blocks, kQkThreads, 0, stream>>>(a, g);
  cudaError_t e = cudaGetLastError();
  if (e || (!a.dq_weight && !a.dk_weight)) return e;
  return launch_dependent(qk_weights_kernel<D>, 2, 1024, 0, stream, a, blocks);
}

template <int D, bool FP16>
cudaError_t launch(const QkArgs& a, bool back, cudaStream_t stream) {
  if (a.pairs) return back ? launch_backward<D, FP16, true>(a, stream) : launch_forward<D, FP16, true>(a, stream);
  return back ? launch_backward<D, FP16, false>(a, stream) : launch_forward<D, FP16, false>(a, stream);
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
