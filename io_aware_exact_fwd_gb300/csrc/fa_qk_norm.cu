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

// A row's layout in its lanes, and one block's tokens.
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

template <int D>
struct QkShared {
  float c[8][D / 2], s[8][D / 2];        // of the block's tokens
  float w[2][D];                         // q's and k's weights
  long long in[8][2], out[8][2], g[8][2];  // where the tokens' rows start in q and k
};

// The places and angles of tokens first .. first + tokens of the line of all.
template <int D, bool BACK>
__device__ __forceinline__ void make_tokens(QkShared<D>& sh, const QkArgs& a, long long first, int tokens) {
  const int half = a.rot / 2;
  if (threadIdx.x < tokens) {
    const long long at = first + threadIdx.x;
    const int b = static_cast<int>(at / a.N), n = static_cast<int>(at % a.N);
    auto place = [&](const Strides& s) { return b * s.s[2] + n * s.s[0]; };
    sh.in[threadIdx.x][0] = place(a.sq);
    sh.in[threadIdx.x][1] = place(a.sk);
    sh.out[threadIdx.x][0] = place(a.sq_out);
    sh.out[threadIdx.x][1] = place(a.sk_out);
    if constexpr (BACK) {
      sh.g[threadIdx.x][0] = place(a.sdq_in);
      sh.g[threadIdx.x][1] = place(a.sdk_in);
    }
  }
  for (int x = threadIdx.x; x < tokens * half; x += kQkThreads) {
    const int t = x / half, i = x % half;
    const long long at = first + t;
    const int pos = a.positions ? __ldg(a.positions + at) : static_cast<int>(at % a.N);
    const float2 cs = turn(turns_of(__ldg(a.inv_freq + i)), pos);
    sh.c[t][i] = cs.x;
    sh.s[t][i] = cs.y;
  }
}

template <int D>
__device__ __forceinline__ void make_weights(QkShared<D>& sh, const QkArgs& a) {
  for (int x = threadIdx.x; x < 2 * D; x += kQkThreads) {
    const void* w = x < D ? a.q_weight : a.k_weight;
    sh.w[x / D][x % D] = w ? weight_at(w, a.weight_type, x % D) : 1.f;
  }
}

template <int D>
__device__ __forceinline__ void angles_of(const QkShared<D>& sh, const Rows<D>& me, int t, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    const float4 x = *reinterpret_cast<const float4*>(&sh.c[t][8 * me.lane + j]);
    const float4 y = *reinterpret_cast<const float4*>(&sh.s[t][8 * me.lane + j]);
    c[j] = me.turned ? x.x : 1.f;
    c[j + 1] = me.turned ? x.y : 1.f;
    c[j + 2] = me.turned ? x.z : 1.f;
    c[j + 3] = me.turned ? x.w : 1.f;
    s[j] = me.turned ? y.x : 0.f;
    s[j + 1] = me.turned ? y.y : 0.f;
    s[j + 2] = me.turned ? y.z : 0.f;
    s[j + 3] = me.turned ? y.w : 0.f;
  }
}
template <int D>
__device__ __forceinline__ void weights_of(const QkShared<D>& sh, const Rows<D>& me, int side, float (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = sh.w[side][me.c0 + j];
    w[8 + j] = sh.w[side][me.c1 + j];
  }
}

// How the grid divides the rows: blocks of `tokens` tokens and `heads` heads (of q's and k's in one line).
struct QkGrid {
  int tokens, heads, slices;
  bool heads_first;  // rows that follow each other are heads of a token
};

template <int D, bool FP16, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads) qk_forward_kernel(const __grid_constant__ QkArgs a, const QkGrid g) {
  __shared__ __align__(16) QkShared<D> sh;
  using R = Rows<D>;
  const R me(a);
  const long long all = static_cast<long long>(a.B) * a.N, first = static_cast<long long>(blockIdx.x / g.slices) * g.tokens;
  const int tokens = static_cast<int>(min(static_cast<long long>(g.tokens), all - first));
  const int h0 = (blockIdx.x % g.slices) * g.heads, heads = min(g.heads, a.H + a.Hkv - h0);
  make_tokens<D, false>(sh, a, first, tokens);
  make_weights<D>(sh, a);
  __syncthreads();
  const int rows = tokens * heads;
  for (int r0 = 0; r0 < rows; r0 += R::kGroups) {  // (a whole warp goes through: the sums are shuffles)
    const int r = r0 + me.group;
    const bool real = r < rows;
    const int t = !real ? 0 : g.heads_first ? r / heads : r % tokens, h = h0 + (!real ? 0 : g.heads_first ? r % heads : r / tokens);
    const int side = h >= a.H;
    const long long head = side ? h - a.H : h;
    const uint16_t* in = static_cast<const uint16_t*>(side ? a.k : a.q) + sh.in[t][side] + head * (side ? a.sk : a.sq).s[1];
    float x[16];
    unpack8<FP16>(*reinterpret_cast<const uint4*>(in + me.c0), x);
    unpack8<FP16>(*reinterpret_cast<const uint4*>(in + me.c1), x + 8);
    if (a.norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
      const float r_norm = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
      float w[16];
      weights_of<D>(sh, me, side, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= r_norm * w[j];
    }
    float c[8], s[8];
    angles_of<D>(sh, me, t, c, s);
    rotate<PAIRS>(x, c, s, 1.f);
    uint16_t* out = static_cast<uint16_t*>(side ? a.k_out : a.q_out) + sh.out[t][side] + head * (side ? a.sk_out : a.sq_out).s[1];
    if (real) {
      *reinterpret_cast<uint4*>(out + me.c0) = pack8<FP16>(x);
      *reinterpret_cast<uint4*>(out + me.c1) = pack8<FP16>(x + 8);
    }
  }
}

// The gradient.  Blocks stay on the GPU and take tiles of tokens in turn, so that the weights' gradients add up in registers; each block's sums go
// to the workspace and a second kernel adds them in order: the same bits on every run.
template <int D, bool FP16, bool PAIRS>
__global__ void __launch_bounds__(kQkThreads) qk_backward_kernel(const __grid_constant__ QkArgs a, const QkGrid g) {
  __shared__ __align__(16) QkShared<D> sh;
  __shared__ float s_dw[kQkThreads / 32][D];
  using R = Rows<D>;
  const R me(a);
  const long long all = static_cast<long long>(a.B) * a.N, tiles = (all + g.tokens - 1) / g.tokens;
  make_weights<D>(sh, a);
  float dw[2][16] = {};
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long first = tile * g.tokens;
    const int tokens = static_cast<int>(min(static_cast<long long>(g.tokens), all - first));
    __syncthreads();
    make_tokens<D, true>(sh, a, first, tokens);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = side ? a.Hkv : a.H, rows = tokens * heads;
      const uint16_t *xs = static_cast<const uint16_t*>(side ? a.k : a.q),
                     *gs = static_cast<const uint16_t*>(side ? a.dk_in : a.dq_in);
      uint16_t* os = static_cast<uint16_t*>(side ? a.k_out : a.q_out);
      const long long hx = (side ? a.sk : a.sq).s[1], hg = (side ? a.sdk_in : a.sdq_in).s[1], ho = (side ? a.sk_out : a.sq_out).s[1];
      float w[16];
      weights_of<D>(sh, me, side, w);
      for (int r0 = 0; r0 < rows; r0 += R::kGroups) {
        const int r = r0 + me.group;
        const bool real = r < rows;
        const int t = !real ? 0 : g.heads_first ? r / heads : r % tokens, h = !real ? 0 : g.heads_first ? r % heads : r / tokens;
        const uint16_t* grow = gs + sh.g[t][side] + h * hg;
        float y[16], c[8], s[8];
        unpack8<FP16>(*reinterpret_cast<const uint4*>(grow + me.c0), y);
        unpack8<FP16>(*reinterpret_cast<const uint4*>(grow + me.c1), y + 8);
        angles_of<D>(sh, me, t, c, s);
        if (a.norm) {
          const uint16_t* in = xs + sh.in[t][side] + h * hx;
          float x[16];
          unpack8<FP16>(*reinterpret_cast<const uint4*>(in + me.c0), x);
          unpack8<FP16>(*reinterpret_cast<const uint4*>(in + me.c1), x + 8);
          rotate<PAIRS>(y, c, s, -1.f);
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
          const float r_norm = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            x[j] *= r_norm;
            if (real) dw[side][j] = fmaf(y[j], x[j], dw[side][j]);
            y[j] *= w[j];
            dot = fmaf(y[j], x[j], dot);
          }
          dot = row_sum<D>(dot) * (1.f / D);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = r_norm * fmaf(-dot, x[j], y[j]);
        } else {
          rotate<PAIRS>(y, c, s, -1.f);
        }
        uint16_t* out = os + sh.out[t][side] + h * ho;
        if (real) {
          *reinterpret_cast<uint4*>(out + me.c0) = pack8<FP16>(y);
          *reinterpret_cast<uint4*>(out + me.c1) = pack8<FP16>(y + 8);
        }
      }
    }
  }
  grid_release();
  if (!a.dq_weight && !a.dk_weight) return;
  // This block's sums: over a warp's rows by shuffles, over the warps in shared memory.
  float* part = static_cast<float*>(a.workspace) + static_cast<size_t>(blockIdx.x) * 2 * D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float x = dw[side][j];
#pragma unroll
      for (int m = R::kLanes; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
      if (lane < R::kLanes) s_dw[warp][(j < 8 ? me.c0 : me.c1 - 8) + j] = x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kQkThreads) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < kQkThreads / 32; ++k) x += s_dw[k][i];
      part[side * D + i] = x;
    }
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

constexpr int kBackBlocksPerSm = 3;

bool heads_first(const QkArgs& a) { return a.sq.s[1] < a.sq.s[0]; }

template <int D, bool FP16, bool PAIRS>
cudaError_t launch_forward(const QkArgs& a, cudaStream_t stream) {
  constexpr int kGroups = Rows<D>::kGroups;
  const long long all = static_cast<long long>(a.B) * a.N;
  const int sms = sm_count(), heads = a.H + a.Hkv;
  QkGrid g{8, heads, 1, heads_first(a)};
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
  QkGrid g{8, 0, 1, heads_first(a)};
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
