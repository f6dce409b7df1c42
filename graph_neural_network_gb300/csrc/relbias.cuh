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

// Gradient tables: per warp [buckets][32 / hv] floats, the column a lane's head
// group, so that the lanes leading a head add without atomics or conflicts.
__host__ __device__ inline size_t grad_tables_bytes(const Shape& s, int buckets) {
  return size_t(kWarps) * buckets * 4 << (5 - s.hv_log2);
}

// Clears the block's tables (a barrier must follow) and returns this lane's column.
__device__ __forceinline__ float* clear_grad_tables(float* tables, const Shape& s,
                                                    const Lane<1>& L, int buckets) {
  const int cols_log2 = 5 - s.hv_log2;
  for (int x = threadIdx.x; x < kWarps * buckets << cols_log2; x += kThreads) tables[x] = 0.f;
  return tables + (((threadIdx.x >> 5) * buckets) << cols_log2) + (L.lane >> s.hv_log2);
}

__device__ __forceinline__ void add_grad(float* column, const Shape& s, int bucket, float de) {
  column[bucket << (5 - s.hv_log2)] += de;
}

// This block's share [buckets][H] of the bias gradient: a lane adds the columns of
// one table (at most 32, in float32), eight lanes the tables of the warps in
// float64, both in a fixed order.  Called by every thread of the block.
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
    const float* t = tables + ((w * buckets + b) << cols_log2) + k;
    float f = 0.f;
    for (int g = 0; g < L.G; ++g) f += t[g << heads_log2];
    double sum = double(f);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (ok && w == 0) part[int64_t(blockIdx.x) * buckets * H + x] = sum;
  }
}

}  // namespace gnn
