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
//   dw_pre = sum dz y^, db_pre = sum dz  over the rows.
// A channel's parameters leave the sums over rows: with a = sum dx sigmoid(g) o^ and
// b = sum dx sigmoid(g), dw_post = scale a, db_post = scale b and dscale = w_post a +
// b_post b.  So the kernels carry four sums per channel, and the rows need only
// scale w_post, scale b_post and w_pre
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
  double* part;       // [blocks][kSums][F]
  int blocks;
};

// Sums over the rows, per channel: a and b above, dw_pre, db_pre.
enum { kSumA, kSumB, kSumW, kSumC, kSums };
static_assert(kSums == 4, "nr_sum takes them in two pairs");

// A gate's e = 2^(-g log2 e), from which s = sigmoid(g) = 1 / (1 + e) and 1 - s, both
// accurate relative to themselves: 1 - s = e s where the gate is open (the difference has
// lost it at g = 17), the difference where s is at most two thirds (it has fewer
// roundings).  e overflows to infinity and s to 0 where the sigmoid is below the smallest
// float.
__device__ __forceinline__ float gate_e(float g) { return ex2(-kLog2e * g); }
__device__ __forceinline__ float sigmoid_of(float e) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float complement_of(float e, float s) {
  return e < 0.5f ? e * s : 1.f - s;
}

// Element-wise arithmetic on a thread's vector, two floats an instruction.
// d = a * b + c
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V],
                                     const float (&c)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    float x = c[k], y = c[k + 1];
    fma2(x, y, a[k], a[k + 1], b[k], b[k + 1]);
    d[k] = x;
    d[k + 1] = y;
  }
}
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 2) mul2v(d[k], d[k + 1], a[k], a[k + 1], b[k], b[k + 1]);
}
template <int V>
__device__ __forceinline__ void vadd(float (&d)[V], const float (&a)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 2) add2(d[k], d[k + 1], d[k], d[k + 1], a[k], a[k + 1]);
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

__device__ __forceinline__ uint4 load_raw(const void* p, int64_t at, bool ok) {
  return ok ? ld16(reinterpret_cast<const char*>(p) + 16 * at) : make_uint4(0, 0, 0, 0);
}

// w[c] = a[c] * b[c] of the thread's channels; a null factor counts as `none`.
template <int V>
__device__ __forceinline__ void load_product(const float* a, float none_a, const float* b,
                                             const Place& P, float (&w)[V]) {
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int f = P.vec * V + c;
    w[c] = P.in ? (a ? __ldg(a + f) : none_a) * (b ? __ldg(b + f) : 1.f) : 0.f;
  }
}

// The gate of a row as loaded: this thread's vector of it (width F) or the row's
// value as a float's bits (width 1).
template <typename T>
__device__ __forceinline__ uint4 load_gate(const NrArgs& A, const Place& P, int64_t row, bool ok) {
  if (A.gate_width == 1)
    return make_uint4(ok ? __float_as_uint(float(reinterpret_cast<const T*>(A.gate)[row])) : 0u, 0,
                      0, 0);
  return load_raw(A.gate, row * A.rv + P.vec, ok && A.gate_width > 1);
}

// The gates' e (0 without a gate).
template <typename T>
__device__ __forceinline__ void open_gate(const NrArgs& A, const uint4& raw,
                                          float (&e)[VecOf<T>::n]) {
  constexpr int V = VecOf<T>::n;
  if (A.gate_width > 1) {
    unpack<T>(raw, e);
#pragma unroll
    for (int c = 0; c < V; ++c) e[c] = gate_e(e[c]);
  } else {
    const float t = A.gate_width == 1 ? gate_e(__uint_as_float(raw.x)) : 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) e[c] = t;
  }
}

// e becomes the gates' sigmoids.
template <int V>
__device__ __forceinline__ void sigmoids(float (&e)[V]) {
#pragma unroll
  for (int c = 0; c < V; ++c) e[c] = sigmoid_of(e[c]);
}

template <int V>
__device__ __forceinline__ float total(const float (&x)[V]) {
  float a = x[0], b = x[1];
#pragma unroll
  for (int c = 2; c < V; c += 2) add2(a, b, a, b, x[c], x[c + 1]);
  return a + b;
}

// x += s over a thread's vector.
template <int V>
__device__ __forceinline__ void shift(float (&x)[V], float s) {
#pragma unroll
  for (int c = 0; c < V; c += 2) add2(x[c], x[c + 1], x[c], x[c + 1], s, s);
}

// x becomes (x - mean) * rstd (rows of `kind`), rstd returned.  kLayer: a kind of
// the call is the layer norm.
template <typename T, int WPR, bool kLayer>
__device__ __forceinline__ float norm_row(const NrArgs& A, const Place& P, int kind, float* buf,
                                          int& turn, float (&x)[VecOf<T>::n]) {
  constexpr int V = VecOf<T>::n;
  if (kind == GNN_ROWNORM_NONE) return 1.f;
  if (kLayer && kind == GNN_ROWNORM_LAYER) {
    float m[1] = {total<V>(x)};
    row_sums<WPR, 1>(m, A.tpr_log2, buf, turn);
    shift<V>(x, P.in ? -m[0] * A.inv_f : 0.f);
  }
  float q[1] = {dot<V>(x, x)};
  row_sums<WPR, 1>(q, A.tpr_log2, buf, turn);
  const float rstd = rsqrtf(fmaf(q[0], A.inv_f, A.eps));
  scale<V>(x, rstd);
  return rstd;
}

// Blocks per SM the kernels are compiled for.  Each thread loads the next row's
// vectors before it works on the present one's, so that loads are always in
// flight; the registers of a bfloat16 vector (eight channels of parameters and,
// backward, of sums) leave room for three blocks forward and two backward.
template <typename T>
struct NrBlocks {
  static constexpr int fwd = sizeof(T) == 4 ? 4 : 3;
};
constexpr int kBwdPerSm = 2;

// Rows of float32 whose parameter sums a thread of the backward pass keeps in
// registers before it adds them to its sums in shared memory: two levels of
// additions lose with the roots of 64 and of the number of parts, not with that of
// all rows (400k rows of 512: 1.7e-7 of the gradient instead of 4.9e-7; 100k rows of
// 128: 79.6 us instead of 79.3).  In bfloat16, eight channels a thread, the same spills (492 us instead of 398
// on 600k rows of 256), and the rows carry 2^-9 each: one level, 3.7e-7 on 1M rows.
constexpr int kKeepRows = 64;

template <typename T, int WPR, bool kLayer>
__global__ void __launch_bounds__(kThreads, NrBlocks<T>::fwd) nr_fwd(const NrArgs A) {
  constexpr int V = VecOf<T>::n;
  __shared__ float buf[2 * kWarps * 4];
  int turn = 0;
  const Place P(A);
  float wp[V], bp[V], wn[V], bn[V];
  load_product<V>(A.p.w_post, 1.f, A.p.scale, P, wp);
  load_product<V>(A.p.b_post, 0.f, A.p.scale, P, bp);
  load_product<V>(A.p.w_pre, 1.f, nullptr, P, wn);
  load_product<V>(A.p.b_pre, 0.f, nullptr, P, bn);
  // every thread of the block makes the same number of turns (barriers)
  int64_t r0 = int64_t(blockIdx.x) * (kThreads >> A.tpr_log2);
  int64_t row = r0 + (threadIdx.x >> A.tpr_log2);
  bool ok = P.in && row < A.n;
  uint4 ro = load_raw(A.o, row * A.rv + P.vec, ok), rx = load_raw(A.x, row * A.rv + P.vec, ok);
  uint4 rg = load_gate<T>(A, P, row, ok);
  for (; r0 < A.n; r0 += P.stride) {
    float o[V], y[V], s[V];
    unpack<T>(ro, o);
    unpack<T>(rx, y);
    open_gate<T>(A, rg, s);
    sigmoids<V>(s);
    const int64_t at = row * A.rv + P.vec;
    const bool now = ok;
    row += P.stride;
    ok = P.in && row < A.n;
    ro = load_raw(A.o, row * A.rv + P.vec, ok);
    rx = load_raw(A.x, row * A.rv + P.vec, ok);
    rg = load_gate<T>(A, P, row, ok);
    norm_row<T, WPR, kLayer>(A, P, A.post, buf, turn, o);
    vfma<V>(o, o, wp, bp);
    vfma<V>(y, s, o, y);
    if (now) st16(reinterpret_cast<char*>(A.y) + 16 * at, pack<T>(y));
    if (A.pre != GNN_ROWNORM_NONE) {
      norm_row<T, WPR, kLayer>(A, P, A.pre, buf, turn, y);
      vfma<V>(y, y, wn, bn);
      if (now) st16(reinterpret_cast<char*>(A.z) + 16 * at, pack<T>(y));
    }
  }
}

// Both rows of the backward pass at once: a and b become their normed rows (kinds ka,
// kb), ra and rb their rstd (1 without a norm).  Half the chain of row sums of two
// calls of norm_row: the pass waits for shuffles as much as for memory.
template <typename T, int WPR, bool kLayer>
__device__ __forceinline__ void norm_rows(const NrArgs& A, const Place& P, int ka, int kb,
                                          float* buf, int& turn, float (&a)[VecOf<T>::n],
                                          float (&b)[VecOf<T>::n], float& ra, float& rb) {
  constexpr int V = VecOf<T>::n;
  if (kLayer) {
    float m[2] = {total<V>(a), total<V>(b)};
    row_sums<WPR, 2>(m, A.tpr_log2, buf, turn);
    shift<V>(a, P.in && ka == GNN_ROWNORM_LAYER ? -m[0] * A.inv_f : 0.f);
    shift<V>(b, P.in && kb == GNN_ROWNORM_LAYER ? -m[1] * A.inv_f : 0.f);
  }
  float q[2] = {dot<V>(a, a), dot<V>(b, b)};
  row_sums<WPR, 2>(q, A.tpr_log2, buf, turn);
  ra = ka == GNN_ROWNORM_NONE ? 1.f : rsqrtf(fmaf(q[0], A.inv_f, A.eps));
  rb = kb == GNN_ROWNORM_NONE ? 1.f : rsqrtf(fmaf(q[1], A.inv_f, A.eps));
  scale<V>(a, ra);
  scale<V>(b, rb);
}

// g becomes rstd (g - [mean(g)] - hat mean(g hat)): the gradient of the norm.
// kExtra: `extra` is summed over the row along with them.
template <typename T, int WPR, bool kLayer, bool kExtra>
__device__ __forceinline__ void norm_grad(const NrArgs& A, int kind, float rstd,
                                          const float (&hat)[VecOf<T>::n], float* buf, int& turn,
                                          float (&g)[VecOf<T>::n], float& extra) {
  constexpr int V = VecOf<T>::n;
  if (!kExtra && kind == GNN_ROWNORM_NONE) return;
  constexpr int N = 1 + kLayer + kExtra;
  float c[N];
  c[0] = dot<V>(g, hat);
  if (kLayer) c[1] = total<V>(g);
  if (kExtra) c[N - 1] = extra;
  row_sums<WPR, N>(c, A.tpr_log2, buf, turn);
  if (kExtra) extra = c[N - 1];
  if (kind == GNN_ROWNORM_NONE) return;
  // rstd g + (-rstd mean(g hat)) hat + (-rstd mean(g))
  const float a = -rstd * A.inv_f * c[0];
  const float b = kLayer && kind == GNN_ROWNORM_LAYER ? -rstd * A.inv_f * c[1] : 0.f;
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    float x = b, y = b;
    fma2(x, y, hat[k], hat[k + 1], a, a);
    fma2(x, y, g[k], g[k + 1], rstd, rstd);
    g[k] = x;
    g[k + 1] = y;
  }
}

// kRow: the gate is one number per row.
template <typename T, int WPR, bool kLayer, bool kRow>
__global__ void __launch_bounds__(kThreads, kBwdPerSm) nr_bwd(const NrArgs A) {
  constexpr int V = VecOf<T>::n;
  __shared__ float buf[2 * kWarps * 4];
  // [kSums][row slots of the block][F], or one sum at a time (bfloat16)
  extern __shared__ __align__(16) float sums[];
  int turn = 0;
  const Place P(A);
  const bool pre = A.pre != GNN_ROWNORM_NONE;
  float wp[V], bp[V], wn[V];
  load_product<V>(A.p.w_post, 1.f, A.p.scale, P, wp);
  load_product<V>(A.p.b_post, 0.f, A.p.scale, P, bp);
  load_product<V>(A.p.w_pre, 1.f, nullptr, P, wn);
  float acc[kSums][V];
  constexpr bool kTwo = sizeof(T) == 4;  // levels of sums (kKeepRows)
  // Adds acc to the thread's shared sums.  (Its index is read anew here, so that no
  // register holds a place over the loop.)
  const auto keep = [&] {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    const int vec = t & ((1 << A.tpr_log2) - 1);
    if (vec >= A.rv) return;
    float* at = sums + (t >> A.tpr_log2) * A.F + vec * V;
#pragma unroll
    for (int k = 0; k < kSums; ++k, at += (kThreads >> A.tpr_log2) * A.F)
#pragma unroll
      for (int c = 0; c < V; c += 4) {
        float4 v = *reinterpret_cast<float4*>(at + c);
        v.x += acc[k][c];
        v.y += acc[k][c + 1];
        v.z += acc[k][c + 2];
        v.w += acc[k][c + 3];
        *reinterpret_cast<float4*>(at + c) = v;
      }
  };
  int rows_left = kKeepRows;
#pragma unroll
  for (int k = 0; k < kSums; ++k) zero<V>(acc[k]);
  if (kTwo) {
    for (int x = threadIdx.x; x < kSums * (kThreads >> A.tpr_log2) * A.F; x += kThreads)
      sums[x] = 0.f;
    __syncthreads();
  }
  int64_t r0 = int64_t(blockIdx.x) * (kThreads >> A.tpr_log2);
  int64_t row = r0 + (threadIdx.x >> A.tpr_log2);
  uint4 ro, rd, rg, ry, rz;
  bool ok;
  const auto load = [&] {
    ok = P.in && row < A.n;
    const int64_t at = row * A.rv + P.vec;
    ry = load_raw(A.x, at, ok && pre);
    rz = load_raw(A.dz, at, ok && pre);
    rd = load_raw(A.dy, at, ok);
    ro = load_raw(A.o, at, ok);
    rg = load_gate<T>(A, P, row, ok);
  };
  load();
  for (; r0 < A.n; r0 += P.stride) {
    float o[V], y[V], e[V], d[V], g[V];
    unpack<T>(ry, y);
    unpack<T>(rz, g);
    unpack<T>(rd, d);
    unpack<T>(ro, o);
    open_gate<T>(A, rg, e);
    const int64_t this_row = row, at = row * A.rv + P.vec;
    const bool now = ok;
    row += P.stride;
    load();
    float rstd_y, rstd_o;
    norm_rows<T, WPR, kLayer>(A, P, A.pre, A.post, buf, turn, y, o, rstd_y, rstd_o);
    if (pre) {
      vfma<V>(acc[kSumW], g, y, acc[kSumW]);
      vadd<V>(acc[kSumC], g);
      vmul<V>(g, g, wn);
      float none = 0.f;
      norm_grad<T, WPR, kLayer, false>(A, A.pre, rstd_y, y, buf, turn, g, none);
      vadd<V>(d, g);
    }
    if (now) st16(reinterpret_cast<char*>(A.dx) + 16 * at, pack<T>(d));
    // d becomes dx sigmoid(g) (0 on a thread without a vector or a row: it adds
    // nothing to the sums), y the gate's gradient d n (1 - sigmoid(g)), g = d wp
    float s[V];
#pragma unroll
    for (int c = 0; c < V; ++c) s[c] = now ? sigmoid_of(e[c]) : 0.f;
    vmul<V>(d, d, s);
    vfma<V>(acc[kSumA], d, o, acc[kSumA]);
    vadd<V>(acc[kSumB], d);
    vmul<V>(g, d, wp);
    float all = 0.f;
    if (A.gate_width > 0) {
      vfma<V>(y, o, wp, bp);
      vmul<V>(y, y, d);
#pragma unroll
      for (int c = 0; c < V; ++c) s[c] = complement_of(e[c], s[c]);
      vmul<V>(y, y, s);
      if (kRow) all = total<V>(y);
    }
    norm_grad<T, WPR, kLayer, kRow>(A, A.post, rstd_o, o, buf, turn, g, all);
    if (now) {
      st16(reinterpret_cast<char*>(A.dout) + 16 * at, pack<T>(g));
      if (kRow) {
        if (P.vec == 0) reinterpret_cast<T*>(A.dgate)[this_row] = T(all);
      } else if (A.gate_width > 0) {
        st16(reinterpret_cast<char*>(A.dgate) + 16 * at, pack<T>(y));
      }
    }
    if (kTwo && --rows_left == 0) {
      keep();
      rows_left = kKeepRows;
#pragma unroll
      for (int k = 0; k < kSums; ++k) zero<V>(acc[k]);
    }
  }
  let_next_start();
  // the block's sums, its row slots added in order in float64
  const int slots = kThreads >> A.tpr_log2;
  if (kTwo) keep();
#pragma unroll
  for (int k = 0; k < kSums; ++k) {
    if (!kTwo) {
      __syncthreads();
      if (P.in)
#pragma unroll
        for (int c = 0; c < V; ++c)
          sums[(threadIdx.x >> A.tpr_log2) * A.F + P.vec * V + c] = acc[k][c];
    }
    if (!kTwo || k == 0) __syncthreads();
    const float* from = sums + (kTwo ? k * slots * A.F : 0);
    for (int f = threadIdx.x; f < A.F; f += kThreads) {
      double t = 0.0;
      for (int x = 0; x < slots; ++x) t += double(from[x * A.F + f]);
      A.part[(int64_t(blockIdx.x) * kSums + k) * A.F + f] = t;
    }
  }
}

// Parameter gradients from the blocks' sums, in a fixed order: a block takes 16
// channels and two of their four sums (a and b, blockIdx.y 0, or dw_pre and
// db_pre), in 32 slices of blocks, every load of a slice in flight at once.
constexpr int kSlices = 32, kLoads = 10;  // 320 blocks at once
__global__ void __launch_bounds__(kSlices * 32)
    nr_sum(const double* part, int blocks, int F, const gnn_norm_params p,
           const gnn_norm_grads d) {
  __shared__ double t[kSlices][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int f = blockIdx.x * 16 + (lane & 15), k = 2 * blockIdx.y + (lane >> 4);
  double s = 0.0;
  grid_wait();
  if (f < F) {
    const double* at = part + k * F + f;
    const int64_t step = int64_t(kSums) * F;
    for (int b = slice; b < blocks; b += kLoads * kSlices) {
      double v[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        v[u] = b + u * kSlices < blocks ? at[(b + u * kSlices) * step] : 0.0;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) s += v[u];
    }
  }
  t[slice][lane] = s;
  __syncthreads();
  if (slice != 0) return;
  double first = 0.0;
#pragma unroll
  for (int x = 0; x < kSlices; ++x) first += t[x][lane];
  const double second = __shfl_down_sync(kFull, first, 16);
  if (lane >= 16 || f >= F) return;
  if (blockIdx.y == 0) {
    const double sc = p.scale ? p.scale[f] : 1.0, w = p.w_post ? p.w_post[f] : 1.0,
                 c = p.b_post ? p.b_post[f] : 0.0;
    if (d.dw_post) d.dw_post[f] = float(sc * first);
    if (d.db_post) d.db_post[f] = float(sc * second);
    if (d.dscale) d.dscale[f] = float(w * first + c * second);
  } else {
    if (d.dw_pre) d.dw_pre[f] = float(first);
    if (d.db_pre) d.db_pre[f] = float(second);
  }
}

int tpr_log2(int rv) {
  int l = 0;
  while ((1 << l) < rv) ++l;
  return l;
}

// Blocks of the backward pass: what fits on a GB300's 152 SMs, at least 16 rows a slot
// before its sums are folded.  (A constant, as the workspace query asks no device.)
int bwd_blocks(int64_t n, int rv) {
  const int cap = 152 * kBwdPerSm;
  const int64_t slots = kThreads >> tpr_log2(rv);
  const int64_t want = (n + slots * 16 - 1) / (slots * 16);
  return want < 1 ? 1 : want < cap ? int(want) : cap;
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

bool any_layer(const NrArgs& A) {
  return A.post == GNN_ROWNORM_LAYER || A.pre == GNN_ROWNORM_LAYER;
}

template <typename T, int WPR>
cudaError_t fwd_w(const NrArgs& A, int sm_count, cudaStream_t st) {
  auto kernel = any_layer(A) ? nr_fwd<T, WPR, true> : nr_fwd<T, WPR, false>;
  const int64_t slots = kThreads >> A.tpr_log2;
  const int64_t want = (A.n + slots - 1) / slots;
  const int64_t cap = int64_t(sm_count) * NrBlocks<T>::fwd;  // what the launch bounds allow
  kernel<<<unsigned(want < cap ? want : cap), kThreads, 0, st>>>(A);
  return cudaGetLastError();
}

template <typename T, int WPR>
cudaError_t bwd_w(const NrArgs& A, const gnn_norm_grads& d, cudaStream_t st) {
  const bool row = A.gate_width == 1;
  auto kernel = any_layer(A) ? (row ? nr_bwd<T, WPR, true, true> : nr_bwd<T, WPR, true, false>)
                             : (row ? nr_bwd<T, WPR, false, true> : nr_bwd<T, WPR, false, false>);
  const int sums = sizeof(T) == 4 ? kSums : 1;
  const size_t smem = size_t(kThreads >> A.tpr_log2) * A.F * sums * 4;  // at most 16 KB
  kernel<<<unsigned(A.blocks), kThreads, smem, st>>>(A);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(nr_sum, dim3(unsigned((A.F + 15) / 16), 2), kSlices * 32, 0, st, A.part,
                      A.blocks, A.F, A.p, d);
}

// Warps per row from the threads per row: 1 (a part or all of one), 2 or 4.
template <typename T>
cudaError_t fwd_t(const NrArgs& A, int sm_count, cudaStream_t st) {
  return A.tpr_log2 <= 5   ? fwd_w<T, 1>(A, sm_count, st)
         : A.tpr_log2 == 6 ? fwd_w<T, 2>(A, sm_count, st)
                           : fwd_w<T, 4>(A, sm_count, st);
}

template <typename T>
cudaError_t bwd_t(const NrArgs& A, const gnn_norm_grads& d, cudaStream_t st) {
  return A.tpr_log2 <= 5   ? bwd_w<T, 1>(A, d, st)
         : A.tpr_log2 == 6 ? bwd_w<T, 2>(A, d, st)
                           : bwd_w<T, 4>(A, d, st);
}

}  // namespace

size_t norm_residual_ws_bytes(int64_t n, int F, gnn_dtype dt) {
  const int rv = F * (dt == GNN_F32 ? 4 : 2) / 16;
  return align_up(size_t(bwd_blocks(n, rv)) * kSums * F * 8, 256);
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
