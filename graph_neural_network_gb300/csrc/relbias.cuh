// The learned relative position bias inside an attention kernel: its table in
// shared memory, the buckets of a batch of edges, and the bias gradient's tables.
#pragma once

#include "device.cuh"

namespace gnn {

// The bias table [buckets][H] in base-2 score units.  A barrier must follow.
__device__ __forceinline__ float* stage_bias(const float* bias, int entries, unsigned char* to) {
  float* t = reinterpret_cast<float*>(to);
  for (int x = threadIdx.x; x < entries; x += kThreads) t[x] = bias[x] * kLog2e;
  return t;
}

// Gradient tables: per warp [buckets][32 / hv], the column a lane's head group, so
// that the lanes leading a head add without atomics or conflicts.  A column adds
// hundreds to thousands of edges one after the other, and plain float32 sums of
// that length lose more than the edges' own rounding (1e-6 of the gradient on a
// graph of 6M edges, against 2e-7 to 3e-7).  So an entry is a float2, the sum and
// what its additions left over (Kahan), as long as two blocks stay on an SM: 839 us
// instead of 831 in pass 2 of that graph, 920 instead of 904 from checkpoints.
// Wider tables, of many buckets and heads as narrow as a lane, hold sums alone.
constexpr size_t kPairBytes = 72 * 1024;  // and up to 32 KB of biases and own rows a block

__host__ __device__ inline size_t grad_columns(const Shape& s, int buckets) {
  return size_t(kWarps) * buckets << (5 - s.hv_log2);
}
__host__ __device__ inline bool grad_pairs(const Shape& s, int buckets) {
  return grad_columns(s, buckets) * 8 <= kPairBytes;
}
__host__ __device__ inline size_t grad_tables_bytes(const Shape& s, int buckets) {
  return grad_columns(s, buckets) * (grad_pairs(s, buckets) ? 8 : 4);
}

// Clears the block's tables (a barrier must follow) and returns this lane's column.
__device__ __forceinline__ float* clear_grad_tables(float* tables, const Shape& s,
                                                    const Lane<1>& L, int buckets) {
  const int words = int(grad_tables_bytes(s, buckets) / 4);
  for (int x = threadIdx.x; x < words; x += kThreads) tables[x] = 0.f;
  const int at = ((threadIdx.x >> 5) * buckets << (5 - s.hv_log2)) + (L.lane >> s.hv_log2);
  return tables + (grad_pairs(s, buckets) ? 2 * at : at);
}

// Adds de to a bucket of the lane's column, on the lanes that lead a head; the
// others go along and store nothing (a branch around it: 903 us instead of 839).
// kPair: grad_pairs of the call.  A sum that overflows becomes NaN in a pair.
template <bool kPair>
__device__ __forceinline__ void add_grad(float* column, const Shape& s, bool leads, int bucket,
                                         float de) {
  const int at = bucket << (5 - s.hv_log2);
  if (kPair) {
    float2* const c = reinterpret_cast<float2*>(column) + at;
    const float2 was = *c;
    const float add = de + was.y, sum = was.x + add;
    if (leads) *c = make_float2(sum, add - (sum - was.x));
  } else if (leads) {
    column[at] += de;
  }
}

// This block's share [buckets][H] of the bias gradient: a lane adds the columns of
// one table (at most 32), eight lanes the tables of the warps, in float64 and in a
// fixed order.  Called by every thread of the block.
template <bool kPair>
__device__ __forceinline__ void fold_grad_tables(const float* tables, const Shape& s,
                                                 const Lane<1>& L, int buckets, double* part) {
  static_assert(kWarps == 8, "eight lanes an entry");
  const int H = s.H;
  const int cols_log2 = 5 - s.hv_log2;             // columns of a table
  const int heads_log2 = s.lpr_log2 - s.hv_log2;   // columns of a sub-group
  const int w = threadIdx.x & 7;
  __syncthreads();
  for (int x0 = 0; x0 < buckets * H; x0 += kThreads / 8) {
    const int x = x0 + (threadIdx.x >> 3);
    const bool ok = x < buckets * H;
    const int b = ok ? x / H : 0, k = ok ? x - b * H : 0;
    const int t = ((w * buckets + b) << cols_log2) + k;
    double sum = 0.0;
    for (int g = 0; g < L.G; ++g) {
      const int at = t + (g << heads_log2);
      sum += kPair ? double(tables[2 * at]) + double(tables[2 * at + 1]) : double(tables[at]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (ok && w == 0) part[int64_t(blockIdx.x) * buckets * H + x] = sum;
  }
}

}  // namespace gnn
