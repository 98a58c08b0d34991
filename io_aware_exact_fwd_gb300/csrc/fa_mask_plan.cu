// Scored attention: the mask plan (the intervals that include/fa.h describes).
#include "fa_internal.h"

namespace fa {
namespace {

// Two intervals a position say the whole mask, because a document's positions see one run of
// keys and are seen by one run of queries; the attention kernels read two of them a tile and
// need no search.  Bound by a launch: 2 x 8192 or 8 x 16384 positions of 9 or 20 documents
// take 4.1 us.
//
// One thread per position.  Position i of row b: the last document that starts at or
// before i (binary search in the offsets) holds it if it ends after i.  Padding gets
// empty intervals that keep both ends nondecreasing along the row: at the first
// document's start before it, else at the end of the document before it.  Everything
// is clamped to [0, N], so offsets that break the contract still give intervals inside
// the row.
__global__ void __launch_bounds__(256) mask_plan_kernel(const int32_t* __restrict__ cu_docs,
                                                        const int32_t* __restrict__ prefix, int n_docs,
                                                        int2* __restrict__ qi, int2* __restrict__ ki, int N,
                                                        long long rows, int causal) {
  const long long r = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  const int b = static_cast<int>(r / N), i = static_cast<int>(r % N);
  int s = 0, e = N, p = 0;
  if (cu_docs) {
    const int32_t* cu = cu_docs + static_cast<size_t>(b) * (n_docs + 1);
    int lo = 0, hi = n_docs + 1;  // the number of offsets <= i
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (cu[mid] <= i) lo = mid + 1;
      else hi = mid;
    }
    if (lo == 0) {
      s = e = min(max(cu[0], 0), N);
    } else if (lo == n_docs + 1) {
      s = e = min(max(cu[n_docs], 0), N);
    } else {
      s = min(max(cu[lo - 1], 0), N);
      e = min(max(cu[lo], s), N);
      if (prefix) p = max(prefix[static_cast<size_t>(b) * n_docs + lo - 1], 0);
    }
  } else if (prefix) {
    p = max(prefix[b], 0);
  }
  if (s >= e) {
    qi[r] = ki[r] = make_int2(s, s);
    return;
  }
  const int reach = p >= e - s ? e : s + p;  // the prefix's end
  qi[r] = make_int2(s, causal ? max(i + 1, reach) : e);
  ki[r] = make_int2(causal && i >= reach ? i : s, e);
}

}  // namespace

cudaError_t launch_mask_plan(const int32_t* cu_docs, const int32_t* prefix, int n_docs, void* plan, int B, int N,
                             int causal, cudaStream_t stream) {
  const long long rows = static_cast<long long>(B) * N;
  int2* qi = static_cast<int2*>(plan);
  mask_plan_kernel<<<static_cast<unsigned>((rows + 255) / 256), 256, 0, stream>>>(cu_docs, prefix, n_docs, qi,
                                                                                  qi + rows, N, rows, causal);
  return cudaGetLastError();
}

}  // namespace fa
