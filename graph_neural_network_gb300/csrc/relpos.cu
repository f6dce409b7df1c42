// Buckets of relative node positions, prepared once per graph and position
// vector: for every edge j -> i the bucket of pos[j] - pos[i], as one byte, in
// the order of the CSR and again in the order of the cached CSC transpose, so
// that the attention kernels read it next to the edge's node id in whichever
// direction they walk.
//
// The rule is a table of ascending lower bounds of the distance |pos[j] - pos[i]|,
// bucket b holding bounds[b] <= distance < bounds[b + 1] and the last bucket
// everything from its bound on.  Whole-number bounds make the bucket exact at
// every border, which a logarithm in floating point does not.  Two-sided
// rules give positive differences (source after destination) a second set of
// buckets; one-sided rules put them all into bucket 0.
//
// Bound: per edge 4 bytes of node id, a 4-byte gather of pos (N * 4 bytes, in L2
// for any graph in use here) and a byte written.  A block takes 4 * kThreads
// consecutive edges: one thread finds the rows that they span by bisection,
// every thread bisects within that span for the first of its four edges and
// walks on from there.  6M edges over 300k nodes: 40 us for each of the two edge
// orders, where the ids and bytes alone would take 4.5 us at the copy rate; the
// gathers and the dependent bisections bound it, once per graph and positions.
#include <math.h>
#include <string.h>

#include "device.cuh"

namespace gnn {
namespace {

struct Bounds {
  int32_t v[kMaxBuckets];
};

// The row of edge e: the largest r in [lo, hi] with ptr[r] <= e.
__device__ __forceinline__ int row_of(const int32_t* ptr, int lo, int hi, int e) {
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (__ldg(ptr + mid) <= e)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// transpose: rows of ptr are sources (CSC), otherwise destinations.
__global__ void __launch_bounds__(kThreads)
    rel_buckets(const int32_t* ptr, const int32_t* idx, int n, int64_t e_total,
                const int32_t* pos, const __grid_constant__ Bounds bounds, int nb, int two_sided,
                int transpose, uint8_t* out) {
  __shared__ int32_t sb[kMaxBuckets];
  __shared__ int span[2];
  const int64_t first = int64_t(blockIdx.x) * (4 * kThreads);
  const int64_t last = (first + 4 * kThreads < e_total ? first + 4 * kThreads : e_total) - 1;
  if (threadIdx.x < nb) sb[threadIdx.x] = bounds.v[threadIdx.x];
  if (threadIdx.x == 0) span[0] = row_of(ptr, 0, n - 1, int(first));
  if (threadIdx.x == 32) span[1] = row_of(ptr, 0, n - 1, int(last));
  __syncthreads();
  const int64_t e0 = first + 4 * int64_t(threadIdx.x);
  if (e0 >= e_total) return;
  int r = row_of(ptr, span[0], span[1], int(e0));
  int end = __ldg(ptr + r + 1);
  int own = __ldg(pos + r);
  uint32_t word = 0;
  for (int u = 0; u < 4 && e0 + u < e_total; ++u) {
    if (e0 + u >= end) {
      do end = __ldg(ptr + ++r + 1);
      while (e0 + u >= end);
      own = __ldg(pos + r);
    }
    const int other = __ldg(pos + __ldg(idx + e0 + u));
    const int64_t d = transpose ? int64_t(own) - other : int64_t(other) - own;
    const uint32_t dist = uint32_t(d < 0 ? -d : (two_sided ? d : 0));  // < 2^32
    int lo = 0, hi = nb - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (uint32_t(sb[mid]) <= dist)
        lo = mid;
      else
        hi = mid - 1;
    }
    word |= uint32_t(lo + (two_sided && d > 0 ? nb : 0)) << (8 * u);
  }
  if (e0 + 4 <= e_total) {
    *reinterpret_cast<uint32_t*>(out + e0) = word;
  } else {
    for (int u = 0; e0 + u < e_total; ++u) out[e0 + u] = uint8_t(word >> (8 * u));
  }
}

// Non-negative whole numbers of up to 64 * 32 bits, for the bounds of the
// logarithmic rule: products of at most 64 factors below 2^31.
struct Big {
  uint32_t w[66];
  int n = 1;
  Big() { w[0] = 1; }
  void mul(uint32_t f) {
    uint64_t carry = 0;
    for (int k = 0; k < n; ++k) {
      carry += uint64_t(w[k]) * f;
      w[k] = uint32_t(carry);
      carry >>= 32;
    }
    if (carry) w[n++] = uint32_t(carry);
  }
  bool at_least(const Big& o) const {
    if (n != o.n) return n > o.n;
    for (int k = n - 1; k >= 0; --k)
      if (w[k] != o.w[k]) return w[k] > o.w[k];
    return true;
  }
};

Big power(uint32_t base, int e) {
  Big r;
  for (int k = 0; k < e; ++k) r.mul(base);
  return r;
}

}  // namespace

// Buckets below m = n / 2 hold one distance each; bucket m + k holds the
// distances t with floor((n - m) log(t / m) / log(max_distance / m)) = k, so
// its bound is the smallest t with t^(n - m) >= max_distance^k m^(n - m - k).
void rel_log_bounds(int n, int max_distance, int32_t* bounds) {
  const int m = n / 2, rest = n - m;
  for (int b = 0; b < m; ++b) bounds[b] = b;
  for (int k = 0; k < rest; ++k) {
    Big need = power(uint32_t(max_distance), k);
    for (int x = 0; x < rest - k; ++x) need.mul(uint32_t(m));
    // a guess in floating point, then to the exact border
    const double guess = m * pow(double(max_distance) / m, double(k) / rest);
    int64_t t = int64_t(guess);
    if (t < m) t = m;
    if (t > max_distance) t = max_distance;
    while (t > m && power(uint32_t(t - 1), rest).at_least(need)) --t;
    while (!power(uint32_t(t), rest).at_least(need)) ++t;
    bounds[m + k] = int32_t(t);
  }
}

cudaError_t launch_rel_buckets(const gnn_graph* g, const int32_t* pos, const int32_t* bounds,
                               int nb, int two_sided, uint8_t* csr, uint8_t* csc,
                               cudaStream_t st) {
  if (g->e == 0) return cudaSuccess;
  Bounds b{};
  memcpy(b.v, bounds, size_t(nb) * sizeof(int32_t));
  const unsigned blocks = unsigned((g->e + 4 * kThreads - 1) / (4 * kThreads));
  rel_buckets<<<blocks, kThreads, 0, st>>>(g->csr.ptr, g->csr.idx, int(g->n), g->e, pos, b, nb,
                                           two_sided, 0, csr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  rel_buckets<<<blocks, kThreads, 0, st>>>(g->csc.ptr, g->csc.idx, int(g->n), g->e, pos, b, nb,
                                           two_sided, 1, csc);
  return cudaGetLastError();
}

}  // namespace gnn
