// The learned relative position bias inside an attention kernel: its table in
// shared memory, softmax weights that stay right beside a bias of any size, and the
// bias gradient's tables.
#pragma once

#include "device.cuh"

namespace gnn {

// How a kernel forms its scores.
enum class Bias {
  kNone,     // dot products alone
  kOrdinary, // every finite entry within +-kOrdinaryBias: dot + bias in one float
  kAny       // a pair of both (SoftRef<Bias::kAny>)
};
constexpr float kOrdinaryBias = 16.f;

// Softmax weights depend on differences of scores.  A sum of dot product and bias in one
// float32 keeps them to 2^-19 while biases stay within 16; beside a bias of 1e6 it would
// lose the dot product (and the row's lse, one float, the sum of the weights), and the
// type's lowest value, a common mask, would overflow in base 2.  So a table with a larger
// finite entry is used another way: each block finds out while it stages the table, every
// block and both passes of a call the same.  Ordinary tables pay one barrier for it (pairs
// throughout: 2,133 instead of 2,058 us for the training step on the 300k-node graph, 589
// instead of 501 us on the 100k-node one in float32).  With a large entry in the table
// the passes of the former take 682, 855 and 928 us instead of 512, 662 and 910.
//
// Stages the table [buckets][H]: as given for kAny, in base-2 units otherwise.  Returns
// whether it is kAny, to every thread of the block.  A barrier must follow.
__device__ __forceinline__ bool stage_bias(const float* bias, int entries, float* t) {
  bool large = false;
  for (int x = threadIdx.x; x < entries; x += kThreads) {
    const float b = bias[x];
    t[x] = b;
    large |= fabsf(b) > kOrdinaryBias && fabsf(b) < INFINITY;
  }
  const bool any = __syncthreads_or(large);
  if (!any)
    for (int x = threadIdx.x; x < entries; x += kThreads) t[x] *= kLog2e;
  return any;
}

// f as the factor of dot products beside a bias y.  A bias of 2^60 or more outweighs them:
// they count for nothing, as in the sum evaluated in 64 bits, so that a row whose edges all
// carry the type's lowest value has equal weights.  (Not 0: infinities stay.)
__device__ __forceinline__ float beside(float y, float f) {
  return fabsf(y) >= 0x1p60f ? f * 0x1p-100f : f;
}

// The reference of an online softmax in one float m (base 2).
template <Bias kBias>
struct SoftRef {
  float m;
  static constexpr int kFloats = 1;

  __device__ __forceinline__ void clear() { m = -INFINITY; }
  // t[u] = log2 of the weights of a batch (-infinity where not ok), its dot products
  // scaled by f * per[u], relative to the highest score so far.  l: the sum of the row's
  // weights so far; where the reference moves, rescale(r) scales l and what else the row
  // has summed up.
  template <int U, int M, class F>
  __device__ __forceinline__ void weigh(float (&t)[M], float f, const float (&per)[U],
                                        const float (&y)[U], const bool (&ok)[U], const float& l,
                                        const F& rescale) {
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      t[u] = kBias == Bias::kNone ? t[u] * (f * per[u]) : fmaf(t[u], f * per[u], y[u]);
      if (!ok[u]) t[u] = -INFINITY;
      top = fmaxf(top, t[u]);
    }
    if (top > m) {
      rescale(ex2(m - top));
      m = top;
    }
    const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] -= mr;
  }
  // Takes N stored sums z[n] with their references in: r[n] scales the stored sums.
  template <int N, class F>
  __device__ __forceinline__ void join(float l, const float (&z)[N], const float (&ref)[1][N],
                                       const F& rescale, float (&r)[N]) {
    float top = m;
#pragma unroll
    for (int n = 0; n < N; ++n) top = fmaxf(top, ref[0][n]);
    if (top > m) {
      rescale(ex2(m - top));
      m = top;
    }
    const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = ex2(ref[0][n] - mr);
  }
  __device__ __forceinline__ void put(float* p) const { p[0] = m; }
  __device__ __forceinline__ float lse(float l) const { return (m + __log2f(l)) * kLn2; }
};

// The same as a pair: a scaled dot product d (base 2) and a bias b (as given), so that a
// weight is 2^((x - d) + log2(e) (y - b)).  The difference of the biases is exact where
// they are equal and off by half a step of itself where they are not: a row's weights are as
// accurate under a bias of -1e9 as under none.  A batch whose highest score lies within
// 2^16 of the reference shifts its d; one farther off (the row's first, mostly, or where
// its biases change over) sets the pair to that of its highest edge.  (A score of -infinity or
// NaN is no reference.)
template <>
struct SoftRef<Bias::kAny> {
  float d, b;
  static constexpr int kFloats = 2;

  __device__ __forceinline__ void clear() { d = b = 0.f; }
  __device__ __forceinline__ float above(float x, float y) const {
    return fmaf(y - b, kLog2e, x - d);
  }
  template <int U, int M, class F>
  __device__ __forceinline__ void weigh(float (&t)[M], float f, const float (&per)[U],
                                        const float (&y)[U], const bool (&ok)[U], const float& l,
                                        const F& rescale) {
    float dot[U], top = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) dot[u] = t[u];
    const auto weights = [&] {
      const float now = beside(b, f);
#pragma unroll
      for (int u = 0; u < U; ++u)
        t[u] = ok[u] ? fmaf(y[u] - b, kLog2e, fmaf(dot[u], now * per[u], -d)) : -INFINITY;
    };
    weights();
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, t[u]);
    if (!(top > 0.f || l == 0.f)) return;
    if (fabsf(top) <= 16.f) {
      rescale(ex2(-top));
      d += top;
#pragma unroll
      for (int u = 0; u < U; ++u) t[u] -= top;
      return;
    }
    const SoftRef was = *this;
    bool any = l != 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float x = dot[u] * beside(y[u], f * per[u]);
      if (ok[u] && x > -INFINITY && (!any || above(x, y[u]) > 0.f)) {
        any = true;
        d = x;
        b = y[u];
      }
    }
    if (l != 0.f) rescale(ex2(above(was.d, was.b)));
    weights();
  }
  template <int N, class F>
  __device__ __forceinline__ void join(float l, const float (&z)[N], const float (&ref)[2][N],
                                       const F& rescale, float (&r)[N]) {
    const SoftRef was = *this;
    bool any = l != 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (z[n] != 0.f && (!any || above(ref[0][n], ref[1][n]) > 0.f)) {
        any = true;
        d = ref[0][n];
        b = ref[1][n];
      }
    if (l != 0.f) rescale(ex2(above(was.d, was.b)));
#pragma unroll
    for (int n = 0; n < N; ++n)
      r[n] = z[n] != 0.f ? ex2(above(ref[0][n], ref[1][n])) : 0.f;
  }
  __device__ __forceinline__ void put(float* p) const {
    p[0] = d;
    p[1] = b;
  }
  __device__ __forceinline__ float lse(float l) const { return fmaf(d + __log2f(l), kLn2, b); }
};

// Gradient tables: per warp [buckets][32 / hv], the column a lane's head group, so
// that the lanes leading a head add without atomics or conflicts.  A column adds
// hundreds to thousands of edges one after the other, and plain float32 sums of
// that length lose more than the edges' own rounding (1e-6 of the gradient on a
// graph of 6M edges, against 2e-7 to 3e-7).  So an entry is a float2, the sum and
// what its additions left over (Kahan), as long as two blocks stay on an SM: 839 us
// instead of 831 in pass 2 of that graph, 920 instead of 904 from checkpoints.
// Wider tables, of many buckets and heads as narrow as a lane, hold sums alone (6M edges:
// 6e-7 of the gradient for H8 D16 bf16 with 128 buckets, 1.5e-6 for H32 D8 with 64).
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
