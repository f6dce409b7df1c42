// Rotary positions: the first dim elements of every head vector are pairs (a, b)
// that turn by t = pos * freq, a' = m (a cos t - b sin t), b' = m (a sin t + b cos t);
// the gradient turns by -t.
//
// Angle: frequencies are fractions of a turn in 64 bits, so pos * freq modulo
// 2^64 is the exact fraction of a turn left over (whole turns wrap away); its top
// 32 bits, as a signed fraction of half a turn, go to sincospif.  The error is the
// conversion's to float32, 2^-25 of half a turn at most, at position 2^31 as at 1:
// a float32 product would have lost the angle at 2^20.
//
// Bound: HBM, 2 s bytes an element (and 4 a node).  A node's angles serve all its
// heads and tensors, so a thread keeps the sines and cosines of its pairs (of two
// accesses of `width` bytes) and walks heads with them, two vectors a head, four
// heads in flight.  The threads of a node stand beside each other over the pairs
// and then over heads, far enough that their accesses are whole lines, and
// over more heads where there are too few nodes for the GPU.
#include "device.cuh"

namespace gnn {
namespace {

struct RopeArgs {
  int64_t items;         // nodes * per
  uint64_t div_per;      // ceil(2^64 / per): item * div_per / 2^64 is the node (items * per < 2^62)
  uint32_t per, slots;   // threads of a node, and of one of its heads
  int turned;            // slots of the rotated part; the others copy
  int half, dim, D;      // elements
  int lanes;             // heads of a node side by side
  int count;
  int interleaved;
  float amplitude, sine; // sine: the amplitude with the direction's sign
  const int32_t* pos;
  gnn_rope_rows t[kRopeMax];
  uint64_t turns[GNN_ROPE_MAX_DIM / 2];
};

// kB bytes of memory (not the read-only path: y may be x).
template <int kB>
struct Access;
template <>
struct Access<16> { using type = uint4; };
template <>
struct Access<8> { using type = uint2; };
template <>
struct Access<4> { using type = uint32_t; };
template <>
struct Access<2> { using type = uint16_t; };

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int kB>
struct RopeVec {
  static constexpr int n = kB / int(sizeof(T));
  union {
    typename Access<kB>::type raw;
    T e[n];
  };
  __device__ __forceinline__ RopeVec() {}
  __device__ __forceinline__ void get(float (&x)[n]) const {
#pragma unroll
    for (int c = 0; c < n; ++c) x[c] = widen(e[c]);
  }
  __device__ __forceinline__ void set(const float (&x)[n]) {
#pragma unroll
    for (int c = 0; c < n; ++c) e[c] = T(x[c]);
  }
};

constexpr int kRopeUnroll = 4;

template <typename T, int kB>
__global__ void __launch_bounds__(kThreads) rope_rows(const __grid_constant__ RopeArgs A) {
  using Vec = RopeVec<T, kB>;
  using Raw = typename Access<kB>::type;
  constexpr int V = Vec::n;
  __shared__ uint64_t turns[GNN_ROPE_MAX_DIM / 2];
  for (int i = threadIdx.x; i < A.half; i += kThreads) turns[i] = A.turns[i];
  const int64_t item = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const bool on = item < A.items;
  const int64_t node =
      !on ? 0 : A.per == 1 ? item : int64_t(__umul64hi(uint64_t(item), A.div_per));
  const uint32_t r = on ? uint32_t(item - node * A.per) : 0u;
  const int lane = int(r / A.slots), slot = int(r - uint32_t(lane) * A.slots);
  const int32_t p = __ldg(A.pos + node);
  __syncthreads();
  if (!on) return;
  // the two accesses of a slot, as elements of the head vector: b < 0 where there is none
  int a, b;
  const bool turn = slot < A.turned;
  if (turn) {
    a = A.interleaved ? 2 * slot * V : slot * V;
    b = A.interleaved ? a + V : a + A.half;
  } else {
    a = A.dim + 2 * (slot - A.turned) * V;
    b = a + V < A.D ? a + V : -1;
  }
  float co[V], si[V];
  if (turn) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const uint64_t left = uint64_t(int64_t(p)) * turns[slot * V + c];
      const float x = float(int32_t(uint32_t(left >> 32))) * 4.656612873077393e-10f;  // 2^-31
      sincospif(x, &si[c], &co[c]);
      co[c] *= A.amplitude;
      si[c] *= A.sine;
    }
  }
  int k = 0, h = 0;  // the next tensor and its head for lane 0 (the same in every thread)
  while (k < A.count) {
    Vec va[kRopeUnroll], vb[kRopeUnroll];
    T* to[kRopeUnroll];
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      to[u] = nullptr;
      if (k < A.count) {
        const gnn_rope_rows& t = A.t[k];
        const int head = h + lane;
        if (head < t.H && (turn || t.x != t.y)) {
          const T* x = static_cast<const T*>(t.x) + node * t.x_node + head * t.x_head;
          to[u] = static_cast<T*>(t.y) + node * t.y_node + head * t.y_head;
          va[u].raw = *reinterpret_cast<const Raw*>(x + a);
          if (b >= 0) vb[u].raw = *reinterpret_cast<const Raw*>(x + b);
        }
        h += A.lanes;
        if (h >= t.H) {
          h = 0;
          ++k;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      if (!to[u]) continue;
      if (turn) {
        float x[V], y[V], f[V], g[V];
        va[u].get(x);
        vb[u].get(y);
        if (A.interleaved && V > 1) {
          // pairs (0, 1), (2, 3) .. of the first access, then of the second
#pragma unroll
          for (int c = 0; c + 1 < V; c += 2) {
            const int d = c / 2, e = (V + c) / 2;
            f[c] = x[c] * co[d] - x[c + 1] * si[d];
            f[c + 1] = x[c] * si[d] + x[c + 1] * co[d];
            g[c] = y[c] * co[e] - y[c + 1] * si[e];
            g[c + 1] = y[c] * si[e] + y[c + 1] * co[e];
          }
        } else {
#pragma unroll
          for (int c = 0; c < V; ++c) {
            f[c] = x[c] * co[c] - y[c] * si[c];
            g[c] = x[c] * si[c] + y[c] * co[c];
          }
        }
        va[u].set(f);
        vb[u].set(g);
      }
      *reinterpret_cast<Raw*>(to[u] + a) = va[u].raw;
      if (b >= 0) *reinterpret_cast<Raw*>(to[u] + b) = vb[u].raw;
    }
  }
}

template <typename T, int kB>
cudaError_t launch(RopeArgs& A, int64_t n, int most_heads, int sm_count, cudaStream_t st) {
  constexpr int V = RopeVec<T, kB>::n;
  A.turned = A.half / V;
  A.slots = uint32_t(A.turned + (A.D - A.dim + 2 * V - 1) / (2 * V));
  // Heads side by side: whole lines (eight threads take 256 bytes of a tensor), and
  // enough threads for the GPU as long as there are heads.
  const int64_t full = int64_t(sm_count) * 1024;
  int lanes = 1;
  while (lanes < most_heads && (A.slots * lanes < 8 || n * A.slots * lanes < full)) lanes *= 2;
  A.lanes = lanes < most_heads ? lanes : most_heads;
  A.per = A.slots * uint32_t(A.lanes);
  A.div_per = A.per == 1 ? 0 : ~uint64_t(0) / A.per + 1;
  A.items = n * A.per;
  const int64_t blocks = (A.items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  rope_rows<T, kB><<<unsigned(blocks), kThreads, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const gnn_rope& rope, int inverse, int64_t n, int D, const int32_t* pos,
                        int count, const gnn_rope_rows* t, gnn_dtype dt, int width, int sm_count,
                        cudaStream_t st) {
  RopeArgs A{};
  A.half = rope.dim / 2;
  A.dim = rope.dim;
  A.D = D;
  A.count = count;
  A.interleaved = rope.layout == GNN_ROPE_INTERLEAVED;
  A.amplitude = rope.amplitude;
  A.sine = inverse ? -rope.amplitude : rope.amplitude;
  A.pos = pos;
  int most = 1;
  for (int k = 0; k < count; ++k) {
    A.t[k] = t[k];
    most = t[k].H > most ? t[k].H : most;
  }
  for (int i = 0; i < A.half; ++i) A.turns[i] = rope.turns[i];
  if (dt == GNN_F32)
    return width == 16  ? launch<float, 16>(A, n, most, sm_count, st)
           : width == 8 ? launch<float, 8>(A, n, most, sm_count, st)
                        : launch<float, 4>(A, n, most, sm_count, st);
  return width == 16  ? launch<__nv_bfloat16, 16>(A, n, most, sm_count, st)
         : width == 8 ? launch<__nv_bfloat16, 8>(A, n, most, sm_count, st)
         : width == 4 ? launch<__nv_bfloat16, 4>(A, n, most, sm_count, st)
                      : launch<__nv_bfloat16, 2>(A, n, most, sm_count, st);
}

}  // namespace gnn
