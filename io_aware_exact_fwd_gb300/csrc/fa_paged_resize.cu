// The paged cache's bookkeeping (include/fa.h, fa_paged_resize): from the changes of the
// sequences' lengths their new lengths, pages taken from or given back to the list of
// free ones, the rows of the new tokens, and each new token's position and slot.
//
// One block scans the sequences: how many pages each takes (grow) or gives back (drop) and how many tokens are new, and the
// sums of these before each sequence.  All or nothing: if pages are missing or a length does not fit, nothing changes.
// The rest needs no order: page k of all that are taken, page r of all that come back and new token t each find
// their sequence by bisection in those sums.  Pages that come back are written behind the free ones, and the pages taken are
// the last of that longer list, so a page may come back and be taken in one call: its taker reads it from the table of
// the sequence that gave it.  A token's page, if it is a taken one, is found in the same way and not in the table, so
// nothing waits for the table's new entries.
//
// Bound by latency: a launch, two dependent loads of the lengths, the scan.  The second part runs in the same block, with the
// sums in shared memory, where there is little of it, and as a dependent launch over the GPU where there is more.
#include "fa_device.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kScanThreads = 1024;

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

__device__ __forceinline__ int pages_of(long long n, int page) { return static_cast<int>((n + page - 1) / page); }

// What one sequence does.
struct Change {
  long long after;
  int had, has;
  bool fits;
};
__device__ __forceinline__ Change change_of(const PagedResizeArgs& a, int b) {
  Change c;
  const long long n = a.seq_lens[b], most = static_cast<long long>(a.max_pages) * a.page_size;
  c.after = n + a.delta[b];
  c.fits = n >= 0 && n <= most && c.after >= 0 && c.after <= most;
  c.had = c.fits ? pages_of(n, a.page_size) : 0;
  c.has = c.fits ? pages_of(c.after, a.page_size) : 0;
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

// What the second part goes by: the sums, the new lengths, and the list's length on entry.
struct Plan {
  const int32_t *grow, *drop, *cu, *lens;
  int count;
};

// Page r of those given back, and page k of those taken.
__device__ __forceinline__ int given_back(const PagedResizeArgs& a, const Plan& p, int r) {
  const int b = owner_of(p.drop, a.B, r);
  return a.page_table[b * a.table_stride + pages_of(p.lens[b], a.page_size) + (r - p.drop[b])];
}
__device__ __forceinline__ int taken(const PagedResizeArgs& a, const Plan& p, int k) {
  const int place = p.count + p.drop[a.B] - 1 - k;
  return place >= p.count ? given_back(a, p, place - p.count) : a.free_pages[place];
}

// The second part: thread `at` of `all`, of whole warps.  (After a refusal there are no pages and no new tokens.)
__device__ __forceinline__ void spread(const PagedResizeArgs& a, const Plan& p, int at, int all) {
  const int grow = p.grow[a.B], drop = p.drop[a.B], total = p.cu[a.B], lane = at & 31;
  for (long long r = at; r < drop; r += all) a.free_pages[p.count + r] = given_back(a, p, static_cast<int>(r));
  for (long long k = at; k < grow; k += all) {
    const int b = owner_of(p.grow, a.B, static_cast<int>(k));
    const int had = pages_of(p.lens[b], a.page_size) - (p.grow[b + 1] - p.grow[b]);
    a.page_table[b * a.table_stride + had + (k - p.grow[b])] = taken(a, p, static_cast<int>(k));
  }
  // 32 rows a warp: the first one's sequence by all lanes, the others' from there on.
  for (long long t0 = at - lane; t0 < a.T; t0 += all) {
    long long pos = -1, slot = -1;
    const long long t = t0 + lane;
    if (t0 < total) {
      int b = owner_of_warp(p.cu, a.B, static_cast<int>(t0), lane);
      if (t < total && t < a.T) {
        while (p.cu[b + 1] <= t) ++b;
        pos = p.lens[b] - (p.cu[b + 1] - t);
        if (a.slots) {
          const int place = static_cast<int>(pos) / a.page_size, more = p.grow[b + 1] - p.grow[b];
          const int had = pages_of(p.lens[b], a.page_size) - more;
          const int page = place < had ? a.page_table[b * a.table_stride + place] : taken(a, p, p.grow[b] + place - had);
          slot = static_cast<long long>(page) * a.page_size + (static_cast<int>(pos) - place * a.page_size);
        }
      }
    }
    if (t < a.T) {
      if (a.slots) a.slots[t] = slot;
      if (a.positions) a.positions[t] = static_cast<int>(pos);
    }
  }
}

__global__ void __launch_bounds__(kScanThreads) resize_scan_kernel(const __grid_constant__ PagedResizeArgs a, int alone) {
  __shared__ long long s_part[3][32];
  __shared__ int s_unfit;
  __shared__ int32_t s_sums[3][kScanThreads + 1], s_lens[kScanThreads];  // for the second part, if it is this block's
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
                        done ? static_cast<int>(before[2]) : 0, done ? static_cast<int>(c.after) : length};
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
  spread(a, Plan{s_sums[0], s_sums[1], s_sums[2], s_lens, count}, threadIdx.x, kScanThreads);
}

__global__ void __launch_bounds__(256) resize_spread_kernel(const __grid_constant__ PagedResizeArgs a) {
  grid_wait();
  const Sums s = sums_of(a.workspace, a.B);
  spread(a, Plan{s.grow, s.drop, a.cu_new, a.lens_out, *s.count}, static_cast<int>(blockIdx.x * 256 + threadIdx.x),
         static_cast<int>(gridDim.x * 256));
}

}  // namespace

size_t paged_resize_workspace(int B) { return (2 * (static_cast<size_t>(B) + 1) + 1) * sizeof(int32_t); }

cudaError_t launch_paged_resize(const PagedResizeArgs& a, cudaStream_t stream) {
  const int alone = a.T <= 4 * kScanThreads && a.B <= kScanThreads;
  resize_scan_kernel<<<1, kScanThreads, 0, stream>>>(a, alone);
  const cudaError_t e = cudaGetLastError();
  if (e || alone) return e;
  return launch_dependent(resize_spread_kernel, static_cast<unsigned>(sm_count()) * 8, 256, 0, stream, a);
}

}  // namespace fa
