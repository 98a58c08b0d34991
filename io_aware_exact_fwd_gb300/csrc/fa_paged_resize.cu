// The paged cache's bookkeeping (include/fa.h, fa_paged_resize): from the changes of the
// sequences' lengths their new lengths, pages taken from or given back to the list of
// free ones, the rows of the new tokens, and each new token's position and slot.
//
// One block scans the sequences: how many pages each takes (grow) or gives back (drop) and how many tokens are new, and the
// sums of these before each sequence.  All or nothing: if pages are missing or a length does not fit, nothing changes.
// The rest needs no order: page k of all that are taken, page r of all that come back and new token t each find
// their sequence in those sums, a warp for 32 neighbours together.  Pages that come back are written behind the free ones, and the
// pages taken are the last of that longer list, so a page may come back and be taken in one call: its taker reads it from the table of
// the sequence that gave it.  A token's page, if it is a taken one, is found in the same way and not in the table, so
// nothing waits for the table's new entries.
//
// Bound by latency: a launch, two dependent loads of the lengths, the scan; then, for many tokens, by the instructions of
// their look-ups.  The second part runs in the same block, with the sums in shared memory, where there is little of it, and as a
// dependent launch over the GPU where there is more.  Measured, in a graph: 64 sequences a token longer each 3.9-4.1 us, 1000 of them
// 6.6 (each row stepping through the sums by itself: 4.7 and 14.8); 1000 sequences, 600 of them longer by 750k tokens
// together, the others shorter, 14 (9.7 MB written).
#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kScanThreads = 1024, kSpreadPerSm = 5;

// The workspace, int32: pages taken before each sequence [B + 1], pages given back before each [B + 1], then the list's
// length on entry.
struct Sums {
  int32_t* grow;
  int32_t* drop;
  int32_t* count;
};
__host__ __device__ inline Sums sums_of(void* workspace, int B) {
  int32_t* p = static_cast<int32_t*>(workspace);
  return Sums{p, p + B + 1, p + 2 * (B + 1)};
}

__device__ __forceinline__ int pages_of(const PagedResizeArgs& a, int n) { return a.per_page(n + a.page_size - 1); }  // n up to 2^30

// What one sequence does.
struct Change {
  int after, had, has;
  bool fits;
};
__device__ __forceinline__ Change change_of(const PagedResizeArgs& a, int b) {
  Change c;
  const int n = a.seq_lens[b], most = a.max_pages * a.page_size;
  const long long after = static_cast<long long>(n) + a.delta[b];
  c.fits = n >= 0 && n <= most && after >= 0 && after <= most;
  c.after = c.fits ? static_cast<int>(after) : 0;
  c.had = c.fits ? pages_of(a, n) : 0;
  c.has = c.fits ? pages_of(a, c.after) : 0;
  return c;
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, w);
    if (lane >= w) x += y;
  }
  return x;
}

// The last place of sums[0 .. B] (sums[0] = 0, sums[B] > x) whose value is at most x.
__device__ __forceinline__ int owner_of(const int32_t* sums, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// The same by a whole warp, for an x of the warp's: 32 probes at once.
__device__ __forceinline__ int owner_of_warp(const int32_t* sums, int B, int x, int lane) {
  int lo = 0, hi = B;  // sums[lo] <= x < sums[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, probe = lo + (lane + 1) * step;
    const int k = __popc(__ballot_sync(0xffffffffu, probe < hi && sums[probe] <= x));
    hi = min(hi, lo + (k + 1) * step);
    lo += k * step;
  }
  return lo;
}

// The same for rows of 32 rising numbers x, one a lane, of which none is before place `from`: 32 sums behind it at once, in
// registers for as long as they do, and bisection among the lanes.
struct Owners {
  const int32_t* sums;
  int B, lane, from, next;
  __device__ __forceinline__ Owners(const int32_t* sums_, int B_, int lane_, int from_) : sums(sums_), B(B_), lane(lane_), from(from_) {
    load();
  }
  __device__ __forceinline__ void load() { next = from + 1 + lane < B ? sums[from + 1 + lane] : 0x7fffffff; }
  __device__ __forceinline__ int of(int x) {
    int mine = from;
    while (true) {
      if (__shfl_sync(0xffffffffu, next, 0) > __shfl_sync(0xffffffffu, x, 31)) return mine;
      int k = 0;  // how many of them are at most x
#pragma unroll
      for (int w = 16; w > 0; w >>= 1)
        if (__shfl_sync(0xffffffffu, next, k + w - 1) <= x) k += w;
      k += __shfl_sync(0xffffffffu, next, k) <= x ? 1 : 0;
      if (mine == from) mine += k;
      if (!__any_sync(0xffffffffu, mine == from + 32)) return mine;
      from += 32;
      load();
    }
  }
};

// What the second part goes by: the sums, the new lengths, and the list's length on entry.
struct Plan {
  const int32_t *grow, *drop, *cu, *lens;
  int count;
};

// Where page r of those given back, and page k of those taken, stand.
__device__ __forceinline__ const int32_t* given_back(const PagedResizeArgs& a, const Plan& p, int r) {
  const int b = owner_of(p.drop, a.B, r);
  return a.page_table + (b * a.table_stride + pages_of(a, p.lens[b]) + (r - p.drop[b]));
}
__device__ __forceinline__ const int32_t* taken(const PagedResizeArgs& a, const Plan& p, int k) {
  const int place = p.count + p.drop[a.B] - 1 - k;
  return place >= p.count ? given_back(a, p, place - p.count) : a.free_pages + place;
}

// The second part: thread `at` of `all`, of whole warps.  (After a refusal there are no pages and no new tokens.)  A warp takes
// UNROLL x 32 pages or rows after each other: the first one's sequence by all lanes, the others' from there on; their loads
// together.
template <int UNROLL>
__device__ __forceinline__ void pages(const PagedResizeArgs& a, const Plan& p, int at, int all) {
  const int grow = p.grow[a.B], drop = p.drop[a.B], lane = at & 31;
  const long long start = static_cast<long long>(at - lane) * UNROLL, step = static_cast<long long>(all) * UNROLL;
  for (long long r0 = start; r0 < drop; r0 += step) {
    Owners owners(p.drop, a.B, lane, owner_of_warp(p.drop, a.B, static_cast<int>(r0), lane));
    const int32_t* from[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      from[i] = nullptr;
      if (r0 + 32 * i >= drop) continue;
      const long long r = r0 + 32 * i + lane;
      const int own = owners.of(static_cast<int>(min(r, drop - 1LL)));
      if (r < drop) from[i] = a.page_table + (own * a.table_stride + pages_of(a, p.lens[own]) + (r - p.drop[own]));
    }
    int page[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) page[i] = from[i] ? *from[i] : 0;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
      if (from[i]) a.free_pages[p.count + r0 + 32 * i + lane] = page[i];
  }
  for (long long k0 = start; k0 < grow; k0 += step) {
    Owners owners(p.grow, a.B, lane, owner_of_warp(p.grow, a.B, static_cast<int>(k0), lane));
    const int32_t* from[UNROLL];
    int32_t* to[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      from[i] = nullptr;
      if (k0 + 32 * i >= grow) continue;
      const long long k = k0 + 32 * i + lane;
      const int own = owners.of(static_cast<int>(min(k, grow - 1LL)));
      if (k < grow) {
        const int had = pages_of(a, p.lens[own]) - (p.grow[own + 1] - p.grow[own]);
        to[i] = a.page_table + (own * a.table_stride + had + (k - p.grow[own]));
        from[i] = taken(a, p, static_cast<int>(k));
      }
    }
    int page[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) page[i] = from[i] ? *from[i] : 0;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
      if (from[i]) *to[i] = page[i];
  }
}
template <int UNROLL>
__device__ __forceinline__ void tokens(const PagedResizeArgs& a, const Plan& p, int at, int all) {
  const int total = p.cu[a.B], lane = at & 31;
  for (long long t0 = static_cast<long long>(at - lane) * UNROLL; t0 < a.T; t0 += static_cast<long long>(all) * UNROLL) {
    Owners owners(p.cu, a.B, lane, t0 < total ? owner_of_warp(p.cu, a.B, static_cast<int>(t0), lane) : 0);
    const int32_t* from[UNROLL];
    int pos[UNROLL], row[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      pos[i] = -1;
      from[i] = nullptr;
      if (t0 + 32 * i >= total) continue;
      const long long t = t0 + 32 * i + lane;
      const int own = owners.of(static_cast<int>(min(t, total - 1LL)));
      if (t >= total || t >= a.T) continue;
      pos[i] = p.lens[own] - (p.cu[own + 1] - static_cast<int>(t));
      if (!a.slots) continue;
      const int place = a.per_page(pos[i]), had = pages_of(a, p.lens[own]) - (p.grow[own + 1] - p.grow[own]);
      row[i] = pos[i] - place * a.page_size;
      from[i] = place < had ? a.page_table + (own * a.table_stride + place) : taken(a, p, p.grow[own] + place - had);
    }
    int page[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) page[i] = from[i] ? *from[i] : 0;
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const long long t = t0 + 32 * i + lane;
      if (t >= a.T) continue;
      if (a.slots) a.slots[t] = from[i] ? static_cast<long long>(page[i]) * a.page_size + row[i] : -1;
      if (a.positions) a.positions[t] = pos[i];
    }
  }
}

__global__ void __launch_bounds__(kScanThreads) resize_scan_kernel(const __grid_constant__ PagedResizeArgs a, int alone) {
  __shared__ long long s_part[3][32];
  __shared__ int s_unfit;
  __shared__ int32_t s_sums[3][kScanThreads / 4 + 1], s_lens[kScanThreads / 4];  // for the second part, if it is this block's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_unfit = 0;
  __syncthreads();
  const int count = min(max(*a.free_count, 0), a.capacity);
  const int per = (a.B + kScanThreads - 1) / kScanThreads;
  const int lo = min(static_cast<int>(threadIdx.x) * per, a.B), hi = min(lo + per, a.B);
  long long mine[3] = {0, 0, 0};  // pages taken, given back, new tokens
  int unfit = 0;
  for (int b = lo; b < hi; ++b) {
    const Change c = change_of(a, b);
    unfit += !c.fits;
    mine[0] += max(c.has - c.had, 0);
    mine[1] += max(c.had - c.has, 0);
    mine[2] += c.fits ? max(a.delta[b], 0) : 0;
  }
  long long before[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    before[i] = warp_scan(mine[i], lane);
    if (lane == 31) s_part[i][warp] = before[i];
  }
  if (unfit) atomicAdd(&s_unfit, unfit);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const long long x = warp_scan(s_part[i][lane], lane);
    total[i] = __shfl_sync(0xffffffffu, x, 31);
    before[i] += __shfl_sync(0xffffffffu, x, warp) - s_part[i][warp] - mine[i];
  }
  // Pages that come back have to have room in the list, the new tokens' rows to be numbers of 32 bits.
  const long long longer = count + total[1], missing = max(total[0] - longer, 0LL);
  const int bad = s_unfit + (longer > a.capacity ? 1 : 0) + (total[2] > 0x7fffffffLL ? 1 : 0);
  const bool done = bad == 0 && missing == 0;
  const Sums s = sums_of(a.workspace, a.B);
  for (int b = lo; b < hi; ++b) {
    const Change c = change_of(a, b);
    const int new_tokens = max(a.delta[b], 0), length = a.seq_lens[b];
    const int now[4] = {done ? static_cast<int>(before[0]) : 0, done ? static_cast<int>(before[1]) : 0,
                        done ? static_cast<int>(before[2]) : 0, done ? c.after : length};
    a.cu_new[b] = now[2];
    a.lens_out[b] = now[3];  // (may be seq_lens: this thread alone reads entry b)
    if (alone) {
      s_sums[0][b] = now[0];
      s_sums[1][b] = now[1];
      s_sums[2][b] = now[2];
      s_lens[b] = now[3];
    } else {
      s.grow[b] = now[0];
      s.drop[b] = now[1];
    }
    before[0] += max(c.has - c.had, 0);
    before[1] += max(c.had - c.has, 0);
    before[2] += new_tokens;
  }
  if (threadIdx.x == 0) {
    const int now[3] = {done ? static_cast<int>(total[0]) : 0, done ? static_cast<int>(total[1]) : 0,
                        done ? static_cast<int>(total[2]) : 0};
    a.cu_new[a.B] = now[2];
    if (alone) {
      s_sums[0][a.B] = now[0];
      s_sums[1][a.B] = now[1];
      s_sums[2][a.B] = now[2];
    } else {
      s.grow[a.B] = now[0];
      s.drop[a.B] = now[1];
      *s.count = count;
    }
    *a.count_out = done ? static_cast<int>(longer - total[0]) : *a.free_count;
    a.status[0] = static_cast<int>(min(missing, 0x7fffffffLL));
    a.status[1] = bad;
  }
  if (!alone) return;
  __syncthreads();
  // Half of the block for the pages, half for the tokens: each waits for loads that depend on each other.
  const Plan p{s_sums[0], s_sums[1], s_sums[2], s_lens, count};
  constexpr int kHalf = kScanThreads / 2;
  if (threadIdx.x < kHalf) pages<4>(a, p, threadIdx.x, kHalf);
  else tokens<1>(a, p, threadIdx.x - kHalf, kHalf);
}

// The rows go to all warps, in groups of 32, UNROLL at a time.
// (The sums copied to each block's shared memory first did not pay: with rows that each stepped through them, 12.7 us for 1000 sequences and
// 750k new tokens against 13.1.)
template <int UNROLL>
__global__ void __launch_bounds__(256, kSpreadPerSm) resize_spread_kernel(const __grid_constant__ PagedResizeArgs a) {
  grid_wait();
  const Sums s = sums_of(a.workspace, a.B);
  const Plan p{s.grow, s.drop, a.cu_new, a.lens_out, *s.count};
  const int at = static_cast<int>(blockIdx.x * 256 + threadIdx.x), all = static_cast<int>(gridDim.x * 256);
  tokens<UNROLL>(a, p, at, all);
  pages<1>(a, p, all - 32 - (at & ~31) + (at & 31), all);  // (from the other end: the last blocks have fewer tokens)
}

}  // namespace

size_t paged_resize_workspace(int B) { return (2 * (static_cast<size_t>(B) + 1) + 1) * sizeof(int32_t); }

cudaError_t launch_paged_resize(const PagedResizeArgs& a, cudaStream_t stream) {
  // One block where that is quicker most of the time: 64 sequences a token longer each 3.9 us, 4.7 with the second launch.  Many
  // pages take longer so, 0.5 us for 1000 of them, but each is taken and comes back once for 16 or more such steps: 256 sequences of
  // 131072 tokens in pages of 16 that all end, 2 million pages, 1.1 ms (257 of them, by two launches, 15 us); 64 prompts of 4000
  // tokens without slots or positions 16.6 us, with slots 8.4.
  const int alone = a.T <= 2 * kScanThreads && a.B <= kScanThreads / 4;
  resize_scan_kernel<<<1, kScanThreads, 0, stream>>>(a, alone);
  const cudaError_t e = cudaGetLastError();
  if (e || alone) return e;
  // More than 32 rows a warp: four groups at a time (1000 sequences, 750k rows: 14 us, 17.8 one by one); else one group, for
  // there may be many sequences with few rows each (1000 of one: 6.6 us, 9.7 in fours).
  const unsigned blocks = static_cast<unsigned>(sm_count()) * kSpreadPerSm;
  const auto kern = static_cast<unsigned>(a.T) > blocks * 256 ? resize_spread_kernel<4> : resize_spread_kernel<1>;
  return launch_dependent(kern, blocks, 256, 0, stream, a);
}

}  // namespace fa
