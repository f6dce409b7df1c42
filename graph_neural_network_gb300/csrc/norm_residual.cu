// The per-node half of a transformer layer between two blocks: the norm after
// a block, its gate and residual scale, the sum, and the norm before the next
// block, in one pass over the rows (and one for the gradients).
//
// Forward, for a row x (residual stream), o (the block's output), gate g:
//   n = norm(o) w_post + b_post,  y = x + scale * sigmoid(g) * n,
//   z = norm(y) w_pre + b_pre
// with norm(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) (layer) or
// v / sqrt(mean(v^2) + eps) (rms).  Backward, given dy (what reaches y past the
// next norm) and dz, with ^ for the normed row:
//   dx = dy + rstd_y (dz w_pre - [mean(dz w_pre)] - y^ mean(dz w_pre y^))
//   u = dx scale sigmoid(g):  dgate = u n (1 - sigmoid(g)),
//   do = rstd_o (u w_post - [mean(u w_post)] - o^ mean(u w_post o^))
//   dw_post = sum u o^, db_post = sum u, dscale = sum dx sigmoid(g) n,
//   dw_pre = sum dz y^, db_pre = sum dz  over the rows
// (the bracketed terms for layer only).  Means, variances and all sums are
// float32 (parameter sums: float32 per thread over its own rows, float64 over
// threads and blocks); a layer variance is the mean of squared differences from
// the mean, not a difference of squares.  Outputs are rounded once.  z comes
// from the unrounded y; the backward takes y as stored and recomputes both
// rows' statistics, which costs arithmetic under a memory-bound pass and no
// state between the calls.
//
// Bound: HBM.  Every element is read once and written once: s bytes (4 + 1
// with a gate per element) forward, (6 + 2) backward.
//
// A thread holds one 16-byte vector of a row, so a row of rv vectors takes the
// next power of two of them: up to 32 a sub-group of a warp, above that two or
// four warps of the block, joined through shared memory.  Rows are dealt to
// the groups in a fixed stride, and the parameter sums are added in a fixed
// order: results are bitwise reproducible.
#include "device.cuh"

namespace gnn {
namespace {

struct NrArgs {
  int64_t n;
  int F, rv;          // elements and 16-byte vectors of a row
  int tpr_log2;       // threads per row
  int post, pre;      // gnn_rownorm
  int gate_width;     // 0, 1 or F
  float eps, inv_f;
  const void *x, *o, *gate, *dy, *dz;   // x holds y in the backward pass
  gnn_norm_params p;
  void *y, *z, *dx, *dout, *dgate;
  double* part;       // [blocks][5][F]
  int blocks;
};

enum { kDwPost, kDbPost, kDscale, kDwPre, kDbPre, kParams };

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t at) {
  return float(reinterpret_cast<const T*>(p)[at]);
}

__device__ __forceinline__ float sigmoid(float g) {
  // 1 / (1 + 2^(-g log2 e)); the exponential overflows to infinity and the
  // quotient to 0 where the sigmoid is below the smallest float
  return __fdividef(1.f, 1.f + ex2(-g * kLog2e));
}

// Sums of each element of v over the threads of a row, on every thread of it.
// WPR: warps per row (1: sub-groups of a warp).  buf: [2][kWarps][N], used in turn.
template <int WPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int tpr_log2, float* buf, int& turn) {
  if (WPR == 1) {
    for (int o = 1; o < (1 << tpr_log2); o <<= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(kFull, v[k], o);
    return;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(kFull, v[k], o);
  const int wid = threadIdx.x >> 5;
  float* b = buf + (turn & 1) * kWarps * 4;
  ++turn;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) b[wid * 4 + k] = v[k];
  __syncthreads();  // the buffer of the next turn is the other one: one barrier a turn
  const int w0 = wid & ~(WPR - 1);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v[k] += b[(w0 + w) * 4 + k];
  }
}

// This thread's vector of its rows, and the rows the grid takes in one turn.
struct Place {
  int vec;
  bool in;
  int64_t stride;
  __device__ __forceinline__ explicit Place(const NrArgs& A) {
    vec = threadIdx.x & ((1 << A.tpr_log2) - 1);
    in = vec < A.rv;
    stride = int64_t(gridDim.x) * (kThreads >> A.tpr_log2);
  }
};

template <typename T>
__device__ __forceinline__ void load_vec(const void* p, int64_t at, bool ok,
                                         float (&x)[VecOf<T>::n]) {
  unpack<T>(ok ? ld16(reinterpret_cast<const char*>(p) + 16 * at) : make_uint4(0, 0, 0, 0), x);
}

template <typename T>
__device__ __forceinline__ void load_param(const float* p, const Place& P, float none,
                                           float (&w)[VecOf<T>::n]) {
  constexpr int V = VecOf<T>::n;
#pragma unroll
  for (int c = 0; c < V; ++c) w[c] = p && P.in ? __ldg(p + P.vec * V + c) : none;
}

template <typename T>
__device__ __forceinline__ void load_gate(const NrArgs& A, const Place& P, int64_t row, bool ok,
                                          float (&s)[VecOf<T>::n]) {
  constexpr int V = VecOf<T>::n;
  if (A.gate_width == 0) {
#pragma unroll
    for (int c = 0; c < V; ++c) s[c] = 1.f;
  } else if (A.gate_width == 1) {
    const float t = ok ? sigmoid(load1<T>(A.gate, row)) : 1.f;
#pragma unroll
    for (int c = 0; c < V; ++c) s[c] = t;
  } else {
    load_vec<T>(A.gate, row * A.rv + P.vec, ok, s);
#pragma unroll
    for (int c = 0; c < V; ++c) s[c] = sigmoid(s[c]);
  }
}

template <int V>
__device__ __forceinline__ float total(const float (&x)[V]) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < V; ++c) s += x[c];
  return s;
}

// x becomes (x - mean) * rstd (rows of `kind`), rstd returned.
template <typename T, int WPR>
__device__ __forceinline__ float norm_row(const NrArgs& A, const Place& P, int kind, float* buf,
                                          int& turn, float (&x)[VecOf<T>::n]) {
  constexpr int V = VecOf<T>::n;
  if (kind == GNN_ROWNORM_NONE) return 1.f;
  if (kind == GNN_ROWNORM_LAYER) {
    float m[1] = {total<V>(x)};
    row_sums<WPR, 1>(m, A.tpr_log2, buf, turn);
    const float mean = m[0] * A.inv_f;
#pragma unroll
    for (int c = 0; c < V; ++c) x[c] = P.in ? x[c] - mean : 0.f;
  }
  float q[1] = {dot<V>(x, x)};
  row_sums<WPR, 1>(q, A.tpr_log2, buf, turn);
  const float rstd = rsqrtf(fmaf(q[0], A.inv_f, A.eps));
  scale<V>(x, rstd);
  return rstd;
}

template <typename T, int WPR>
__global__ void __launch_bounds__(kThreads) nr_fwd(const NrArgs A) {
  constexpr int V = VecOf<T>::n;
  __shared__ float buf[2 * kWarps * 4];
  int turn = 0;
  const Place P(A);
  float wp[V], bp[V], sc[V], wn[V], bn[V];
  load_param<T>(A.p.w_post, P, 1.f, wp);
  load_param<T>(A.p.b_post, P, 0.f, bp);
  load_param<T>(A.p.scale, P, 1.f, sc);
  load_param<T>(A.p.w_pre, P, 1.f, wn);
  load_param<T>(A.p.b_pre, P, 0.f, bn);
  // every thread of the block makes the same number of turns (barriers)
  for (int64_t r0 = int64_t(blockIdx.x) * (kThreads >> A.tpr_log2); r0 < A.n; r0 += P.stride) {
    const int64_t row = r0 + (threadIdx.x >> A.tpr_log2);
    const bool ok = P.in && row < A.n;
    const int64_t at = row * A.rv + P.vec;
    float o[V], y[V], s[V];
    load_vec<T>(A.o, at, ok, o);
    load_vec<T>(A.x, at, ok, y);
    load_gate<T>(A, P, row, ok, s);
    norm_row<T, WPR>(A, P, A.post, buf, turn, o);
#pragma unroll
    for (int c = 0; c < V; ++c) y[c] = fmaf(sc[c] * s[c], fmaf(o[c], wp[c], bp[c]), y[c]);
    if (!ok) zero<V>(y);
    if (ok) st16(reinterpret_cast<char*>(A.y) + 16 * at, pack<T>(y));
    if (A.pre != GNN_ROWNORM_NONE) {
      norm_row<T, WPR>(A, P, A.pre, buf, turn, y);
#pragma unroll
      for (int c = 0; c < V; ++c) y[c] = fmaf(y[c], wn[c], bn[c]);
      if (ok) st16(reinterpret_cast<char*>(A.z) + 16 * at, pack<T>(y));
    }
  }
}

// g becomes rstd (g - [mean(g)] - hat mean(g hat)): the gradient of the norm.
// extra: one more value summed over the row along with them.
template <typename T, int WPR>
__device__ __forceinline__ void norm_grad(const NrArgs& A, const Place& P, int kind, float rstd,
                                          const float (&hat)[VecOf<T>::n], float* buf, int& turn,
                                          float (&g)[VecOf<T>::n], float& extra) {
  constexpr int V = VecOf<T>::n;
  float c[3] = {dot<V>(g, hat), total<V>(g), extra};
  if (!P.in) c[0] = c[1] = c[2] = 0.f;
  row_sums<WPR, 3>(c, A.tpr_log2, buf, turn);
  extra = c[2];
  if (kind == GNN_ROWNORM_NONE) return;
  const float a = c[0] * A.inv_f, b = kind == GNN_ROWNORM_LAYER ? c[1] * A.inv_f : 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) g[k] = rstd * (g[k] - b - hat[k] * a);
}

template <typename T, int WPR>
__global__ void __launch_bounds__(kThreads) nr_bwd(const NrArgs A) {
  constexpr int V = VecOf<T>::n;
  __shared__ float buf[2 * kWarps * 4];
  extern __shared__ float sums[];  // [groups of the block][F], one parameter at a time
  int turn = 0;
  const Place P(A);
  float wp[V], bp[V], sc[V], wn[V];
  load_param<T>(A.p.w_post, P, 1.f, wp);
  load_param<T>(A.p.b_post, P, 0.f, bp);
  load_param<T>(A.p.scale, P, 1.f, sc);
  load_param<T>(A.p.w_pre, P, 1.f, wn);
  float acc[kParams][V];
#pragma unroll
  for (int k = 0; k < kParams; ++k) zero<V>(acc[k]);
  for (int64_t r0 = int64_t(blockIdx.x) * (kThreads >> A.tpr_log2); r0 < A.n; r0 += P.stride) {
    const int64_t row = r0 + (threadIdx.x >> A.tpr_log2);
    const bool ok = P.in && row < A.n;
    const int64_t at = row * A.rv + P.vec;
    float o[V], y[V], s[V], d[V], g[V];
    load_vec<T>(A.o, at, ok, o);
    load_vec<T>(A.dy, at, ok, d);
    load_gate<T>(A, P, row, ok, s);
    float none = 0.f;
    if (A.pre != GNN_ROWNORM_NONE) {
      load_vec<T>(A.x, at, ok, y);
      load_vec<T>(A.dz, at, ok, g);
      const float rstd = norm_row<T, WPR>(A, P, A.pre, buf, turn, y);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        acc[kDwPre][c] = fmaf(g[c], y[c], acc[kDwPre][c]);
        acc[kDbPre][c] += g[c];
        g[c] *= wn[c];
      }
      norm_grad<T, WPR>(A, P, A.pre, rstd, y, buf, turn, g, none);
#pragma unroll
      for (int c = 0; c < V; ++c) d[c] += g[c];
    }
    if (!ok) zero<V>(d);
    if (ok) st16(reinterpret_cast<char*>(A.dx) + 16 * at, pack<T>(d));
    const float rstd = norm_row<T, WPR>(A, P, A.post, buf, turn, o);
    float dg[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float n = fmaf(o[c], wp[c], bp[c]);
      const float ds = d[c] * s[c];
      const float u = ds * sc[c];
      acc[kDscale][c] = fmaf(ds, n, acc[kDscale][c]);
      acc[kDwPost][c] = fmaf(u, o[c], acc[kDwPost][c]);
      acc[kDbPost][c] += u;
      dg[c] = u * n * (1.f - s[c]);
      g[c] = u * wp[c];
    }
    float all = total<V>(dg);
    norm_grad<T, WPR>(A, P, A.post, rstd, o, buf, turn, g, all);
    if (ok) {
      st16(reinterpret_cast<char*>(A.dout) + 16 * at, pack<T>(g));
      if (A.gate_width == 1) {
        if (P.vec == 0) reinterpret_cast<T*>(A.dgate)[row] = T(all);
      } else if (A.gate_width > 1) {
        st16(reinterpret_cast<char*>(A.dgate) + 16 * at, pack<T>(dg));
      }
    }
  }
  // the block's parameter sums, its row slots added in order in float64
  const int slots = kThreads >> A.tpr_log2;
#pragma unroll
  for (int k = 0; k < kParams; ++k) {
    __syncthreads();
    if (P.in)
#pragma unroll
      for (int c = 0; c < V; ++c) sums[(threadIdx.x >> A.tpr_log2) * A.F + P.vec * V + c] = acc[k][c];
    __syncthreads();
    for (int f = threadIdx.x; f < A.F; f += kThreads) {
      double t = 0.0;
      for (int x = 0; x < slots; ++x) t += double(sums[x * A.F + f]);
      A.part[(int64_t(blockIdx.x) * kParams + k) * A.F + f] = t;
    }
  }
}

// Parameter gradients: column f of parameter k summed over the blocks, 32
// columns and 32 slices of blocks at a time, in a fixed order.
__global__ void __launch_bounds__(1024) nr_sum(const double* part, int blocks, int F,
                                               float* dw_post, float* db_post, float* dscale,
                                               float* dw_pre, float* db_pre) {
  __shared__ double t[32][33];
  float* out[kParams] = {dw_post, db_post, dscale, dw_pre, db_pre};
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  const int cols = kParams * F;
  double s = 0.0;
  if (col < cols)
    for (int b = slice; b < blocks; b += 32) s += part[int64_t(b) * cols + col];
  t[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && col < cols) {
    double a = 0.0;
    for (int x = 0; x < 32; ++x) a += t[x][threadIdx.x];
    float* o = out[col / F];
    if (o) o[col % F] = float(a);
  }
}

int tpr_log2(int rv) {
  int l = 0;
  while ((1 << l) < rv) ++l;
  return l;
}

// Blocks of the backward pass: at most four on each of 152 SMs, at least 16
// rows a slot before its sums are folded.
constexpr int kBwdBlocks = 4 * 152;
int bwd_blocks(int64_t n, int rv) {
  const int64_t slots = kThreads >> tpr_log2(rv);
  const int64_t want = (n + slots * 16 - 1) / (slots * 16);
  return want < 1 ? 1 : want < kBwdBlocks ? int(want) : kBwdBlocks;
}

NrArgs nr_args(const gnn_norm_residual& d, gnn_dtype dt) {
  NrArgs A{};
  A.n = d.n;
  A.F = d.F;
  A.rv = d.F * (dt == GNN_F32 ? 4 : 2) / 16;
  A.tpr_log2 = tpr_log2(A.rv);
  A.post = d.post;
  A.pre = d.pre;
  A.gate_width = d.gate_width;
  A.eps = d.eps;
  A.inv_f = 1.f / float(d.F);
  A.p = d.params;
  return A;
}

template <typename T>
cudaError_t fwd_t(const NrArgs& A, int sm_count, cudaStream_t st) {
  const int wpr = A.tpr_log2 <= 5 ? 1 : 1 << (A.tpr_log2 - 5);
  auto kernel = wpr == 1 ? nr_fwd<T, 1> : wpr == 2 ? nr_fwd<T, 2> : nr_fwd<T, 4>;
  const int64_t slots = kThreads >> A.tpr_log2;
  const int64_t want = (A.n + slots - 1) / slots;
  const int64_t cap = persistent_blocks(kernel, 0, sm_count);
  kernel<<<unsigned(want < cap ? want : cap), kThreads, 0, st>>>(A);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const NrArgs& A, const gnn_norm_grads& d, cudaStream_t st) {
  const int wpr = A.tpr_log2 <= 5 ? 1 : 1 << (A.tpr_log2 - 5);
  auto kernel = wpr == 1 ? nr_bwd<T, 1> : wpr == 2 ? nr_bwd<T, 2> : nr_bwd<T, 4>;
  const size_t smem = size_t(kThreads >> A.tpr_log2) * A.F * 4;
  kernel<<<unsigned(A.blocks), kThreads, smem, st>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  nr_sum<<<unsigned((kParams * A.F + 31) / 32), 1024, 0, st>>>(
      A.part, A.blocks, A.F, d.dw_post, d.db_post, d.dscale, d.dw_pre, d.db_pre);
  return cudaGetLastError();
}

}  // namespace

size_t norm_residual_ws_bytes(int64_t n, int F, gnn_dtype dt) {
  const int rv = F * (dt == GNN_F32 ? 4 : 2) / 16;
  return align_up(size_t(bwd_blocks(n, rv)) * kParams * F * 8, 256);
}

cudaError_t launch_norm_residual_forward(const gnn_norm_residual& d, gnn_dtype dt, const void* x,
                                         const void* o, const void* gate, void* y, void* z,
                                         int sm_count, cudaStream_t st) {
  NrArgs A = nr_args(d, dt);
  A.x = x;
  A.o = o;
  A.gate = gate;
  A.y = y;
  A.z = z;
  return dt == GNN_F32 ? fwd_t<float>(A, sm_count, st) : fwd_t<__nv_bfloat16>(A, sm_count, st);
}

cudaError_t launch_norm_residual_backward(const gnn_norm_residual& d, gnn_dtype dt, const void* y,
                                          const void* o, const void* gate, const void* dy,
                                          const void* dz, const gnn_norm_grads& grads, char* ws,
                                          cudaStream_t st) {
  NrArgs A = nr_args(d, dt);
  A.x = y;
  A.o = o;
  A.gate = gate;
  A.dy = dy;
  A.dz = dz;
  A.dx = grads.dx;
  A.dout = grads.dout;
  A.dgate = grads.dgate;
  A.part = reinterpret_cast<double*>(ws);
  A.blocks = bwd_blocks(d.n, A.rv);
  return dt == GNN_F32 ? bwd_t<float>(A, grads, st) : bwd_t<__nv_bfloat16>(A, grads, st);
}

}  // namespace gnn
