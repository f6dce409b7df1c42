// Backward pass of the graph-transformer attention from 8-bit checkpoints.
//
// q, key and val are given as the forward call's 8-bit checkpoints (pack8.cu):
// integers q8, k8, v8 with a scale per head vector, standing for
// q^ = q8 qs, k^ = k8 ks, v^ = v8 vs.  The result is the gradient of the attention at
// that point, exactly: its softmax statistics are those of the checkpoints, not
// the forward call's (whose log-sum-exp would leave weights that do not sum to
// one), so no statistic is kept from the forward either.
//
//   pass 1, destination side (CSR), one streaming pass with an online softmax
//     over e_ij = scale q^_i . k^_j (+ bias): with p = exp(e - m) it carries
//     l = sum p, D = sum p da, P = sum p da k^_j, Q = sum p k^_j (da = dout_i . v^_j)
//     and ends with Delta_i = D / l, lse_i = m + log l,
//     dq_i = scale (P - Delta_i Q) / l.  Record {lse, Delta, qs} to the workspace.
//   pass 2, source side (CSC), as for transformer_agg_backward:
//     dkey_j = scale sum_i de_ij q^_i, dval_j = sum_i alpha_ij dout_i.
//
// The scores' dot products are sums of byte products by the four-way integer
// dot instruction: whole numbers below 2^23, exact in float32 as well, scaled
// once.  The other products need a gathered byte as a float (widen8).
//
// Bound: gathers.  Per edge pass 1 reads 2 F bytes and two scales per head, pass 2
// F (1 + s) bytes and a record per head; half to three quarters of what the
// 16-bit pass gathers.  A lane holds kE = 16 (or 8, 4 for narrow heads) elements:
// per-edge work that does not depend on them is then shared by more.
//
// Lane geometry: a Shape whose "16-byte vector" is kE elements.  Work items,
// masks, buckets and the bias gradient as in transformer.cu.
#include "relbias.cuh"

namespace gnn {
namespace {

constexpr int kGrab = 4;

struct T8Dir {
  const int32_t* ptr;
  const int32_t* idx;
  const uint8_t* buckets;  // of the edges in this direction, or null
  const int32_t* light;
  int64_t n_light;
  const int4* items;
  int64_t n_items;
  const int4* hubs;
  int64_t n_hubs;
  int col_off;             // bytes of shared memory before the warps' partial sums
};

struct T8Args {
  Shape s;                 // in kE-element vectors
  T8Dir csr, csc;
  const int8_t *q8, *k8, *v8;
  const float *qs, *ks, *vs;   // [N][H]
  float scale, scale2;     // natural units, base 2
  const void* dout;
  void *dq, *dkey, *dval;
  float4* stats;           // [N][H] {lse (base 2), Delta, qs, -}
  float* d_part;           // [CSR hub chunks][dst floats]
  float* s_part;           // [CSC hub chunks][src floats]
  const float* bias;
  int buckets;
  int rel_off;
  double* db_part;         // [pass 2 blocks][buckets][H]
  int* ctr;
  int32_t* err;
};

// ---- lane vectors of kE elements ---------------------------------------------

template <int kE>
struct Raw8 {
  uint32_t w[kE / 4];
};

template <int kE>
__device__ __forceinline__ Raw8<kE> ld8(const int8_t* p, int64_t node, const Shape& s,
                                        const Lane<1>& L, bool ok) {
  Raw8<kE> r;
  const int8_t* at = p + (node * s.rv + L.q[0]) * kE;
  if constexpr (kE == 16) {
    const uint4 t = ok ? ld16(at) : make_uint4(0, 0, 0, 0);
    r.w[0] = t.x;
    r.w[1] = t.y;
    r.w[2] = t.z;
    r.w[3] = t.w;
  } else if constexpr (kE == 8) {
    const uint2 t = ok ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0, 0);
    r.w[0] = t.x;
    r.w[1] = t.y;
  } else {
    r.w[0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(at)) : 0u;
  }
  return r;
}

template <int kE>
__device__ __forceinline__ float dot8(const Raw8<kE>& a, const Raw8<kE>& b) {
  int d = 0;
#pragma unroll
  for (int k = 0; k < kE / 4; ++k) d = __dp4a(int(a.w[k]), int(b.w[k]), d);
  return float(d);
}

template <int kE>
__device__ __forceinline__ void widen(const Raw8<kE>& r, float (&x)[kE]) {
#pragma unroll
  for (int k = 0; k < kE / 4; ++k) widen8(r.w[k], x + 4 * k);
}

// kE elements of a row of T, as loaded.
template <typename T, int kE>
struct RawT {
  uint4 v[kE * int(sizeof(T)) / 16];
};

template <typename T, int kE>
__device__ __forceinline__ RawT<T, kE> ldT(const void* p, int64_t node, const Shape& s,
                                           const Lane<1>& L, bool ok) {
  RawT<T, kE> r;
  constexpr int n = kE * int(sizeof(T)) / 16;
  const char* at = reinterpret_cast<const char*>(p) + (node * s.rv + L.q[0]) * (kE * sizeof(T));
#pragma unroll
  for (int k = 0; k < n; ++k) r.v[k] = ok ? ld16(at + 16 * k) : make_uint4(0, 0, 0, 0);
  return r;
}

template <typename T, int kE>
__device__ __forceinline__ void widenT(const RawT<T, kE>& r, float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
#pragma unroll
  for (int k = 0; k < kE / V; ++k) unpack<T>(r.v[k], *reinterpret_cast<float(*)[V]>(x + V * k));
}

template <typename T, int kE>
__device__ __forceinline__ void storeT(void* p, int64_t node, const Shape& s, const Lane<1>& L,
                                       const float (&x)[kE]) {
  constexpr int V = VecOf<T>::n;
  char* at = reinterpret_cast<char*>(p) + (node * s.rv + L.q[0]) * (kE * sizeof(T));
#pragma unroll
  for (int k = 0; k < kE / V; ++k)
    st16(at + 16 * k, pack<T>(*reinterpret_cast<const float(*)[V]>(x + V * k)));
}

// Edges in flight per lane.
template <int kE>
struct Unroll8 {
  static constexpr int value = kE == 16 ? 2 : 4;
};

// ---------------------------------------------------------------------------
// pass 1: destination side
// ---------------------------------------------------------------------------

template <typename T, int kE_, bool kRel>
struct DstPass {
  static constexpr int kE = kE_;
  static constexpr int U = Unroll8<kE>::value;
  const T8Args& A;
  const Lane<1>& L;
  const float* sb;
  // the node
  Raw8<kE> q8;
  float qsc;        // qs_i
  float g[kE];
  // its sums; m is in base 2
  float m, l, d, P[kE], Q[kE];

  __device__ __forceinline__ DstPass(const T8Args& a, const Lane<1>& lane) : A(a), L(lane) {}
  // floats of a partial state: P, Q, then m, l, d per head
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE + 3 * s.H; }
  static __device__ __forceinline__ const T8Dir& dir(const T8Args& A) { return A.csr; }

  __device__ __forceinline__ void zero_sums() {
    m = -INFINITY;
    l = d = 0.f;
    zero<kE>(P);
    zero<kE>(Q);
  }
  __device__ __forceinline__ void begin(int i) {
    q8 = ld8<kE>(A.q8, i, A.s, L, L.ok[0]);
    qsc = L.ok[0] ? __ldg(A.qs + int64_t(i) * A.s.H + L.k[0]) : 0.f;
    widenT<T, kE>(ldT<T, kE>(A.dout, i, A.s, L, L.ok[0]), g);
    zero_sums();
  }
  __device__ __forceinline__ void rescale(float mn) {
    const float s0 = ex2(m - mn);
    l *= s0;
    d *= s0;
    scale<kE>(P, s0);
    scale<kE>(Q, s0);
    m = mn;
  }

  template <bool kFixed>
  __device__ __forceinline__ void edges(const int32_t* cols, int colbase, int beg, int end, int sg,
                                        int SG, int step, int trips, int (&jn)[U]) {
    const int H = A.s.H;
    const float qk = qsc * A.scale2;
    int bn[U];
    if (kRel) batch_buckets<U>(A.csr.buckets, beg, end, sg, SG, bn);
    int base = beg;
    for (int t = 0; kFixed ? t < trips : base < end; ++t, base += step) {
      int j[U];
#pragma unroll
      for (int u = 0; u < U; ++u) j[u] = jn[u];
      float bs[U];
      if (kRel) edge_bias<U>(sb, A.s, L, bn, j, bs);
      Raw8<kE> rk[U], rv[U];
      float ks[U], vs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = j[u] >= 0 && L.ok[0];
        rk[u] = ld8<kE>(A.k8, j[u], A.s, L, ok);
        rv[u] = ld8<kE>(A.v8, j[u], A.s, L, ok);
        ks[u] = ok ? __ldg(A.ks + int64_t(j[u]) * H + L.k[0]) : 0.f;
        vs[u] = ok ? __ldg(A.vs + int64_t(j[u]) * H + L.k[0]) : 0.f;
      }
      if (kFixed ? t + 1 < trips : base + step < end) {
        batch_ids<U>(cols, colbase, base + step, end, sg, SG, jn);
        if (kRel) batch_buckets<U>(A.csr.buckets, base + step, end, sg, SG, bn);
      }
      float red[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[kE];
        red[u] = dot8<kE>(rk[u], q8);
        widen<kE>(rv[u], x);
        red[U + u] = dot<kE>(x, g);
      }
      head_sums<2 * U>(red, A.s.hv_log2);
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        red[u] = kRel ? fmaf(red[u], qk * ks[u], bs[u]) : red[u] * (qk * ks[u]);
        if (j[u] < 0) red[u] = -INFINITY;
        top = fmaxf(top, red[u]);
      }
      if (top > m) rescale(top);
      const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float p = ex2(red[u] - mr);
        // an absent edge may face an own row that holds anything
        const float pd = j[u] < 0 ? 0.f : p * (red[U + u] * vs[u]);
        l += p;
        d += pd;
        float x[kE];
        widen<kE>(rk[u], x);
        axpy<kE>(P, pd * ks[u], x);
        axpy<kE>(Q, p * ks[u], x);
      }
    }
  }

  // adds another partial state of the same node
  __device__ __forceinline__ void add(float mb, float lb, float db, const float (&Pb)[kE],
                                      const float (&Qb)[kE]) {
    const float M = fmaxf(m, mb), Mr = M == -INFINITY ? 0.f : M;
    const float sa = ex2(m - Mr), sb_ = ex2(mb - Mr);
    l = l * sa + lb * sb_;
    d = d * sa + db * sb_;
    scale<kE>(P, sa);
    axpy<kE>(P, sb_, Pb);
    scale<kE>(Q, sa);
    axpy<kE>(Q, sb_, Qb);
    m = M;
  }
  __device__ __forceinline__ void join_subgroups() {
    for (int o = A.s.lpr; o < 32; o <<= 1) {
      const float mb = __shfl_xor_sync(kFull, m, o), lb = __shfl_xor_sync(kFull, l, o),
                  db = __shfl_xor_sync(kFull, d, o);
      float Pb[kE], Qb[kE];
#pragma unroll
      for (int c = 0; c < kE; ++c) {
        Pb[c] = __shfl_xor_sync(kFull, P[c], o);
        Qb[c] = __shfl_xor_sync(kFull, Q[c], o);
      }
      add(mb, lb, db, Pb, Qb);
    }
  }
  __device__ __forceinline__ void put(float* to) const {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
#pragma unroll
    for (int c = 0; c < kE; ++c) {
      to[at + c] = P[c];
      to[row + at + c] = Q[c];
    }
    if (L.head_leader(A.s, 0)) {
      float* h = to + 2 * row + 3 * L.k[0];
      h[0] = m;
      h[1] = l;
      h[2] = d;
    }
  }
  __device__ __forceinline__ void take(const float* from) {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
    float Pb[kE], Qb[kE];
#pragma unroll
    for (int c = 0; c < kE; ++c) {
      Pb[c] = from[at + c];
      Qb[c] = from[row + at + c];
    }
    const float* h = from + 2 * row + 3 * L.k[0];
    add(h[0], h[1], h[2], Pb, Qb);
  }
  __device__ __forceinline__ float* chunk(int slot) const {
    return A.d_part + int64_t(slot) * floats(A.s);
  }
  __device__ __forceinline__ void finish(int i) {
    const bool any = l != 0.f;  // a NaN stays one
    const float inv = any ? __frcp_rn(l) : 0.f;
    const float delta = d * inv;
    const float f = A.scale * inv;
#pragma unroll
    for (int c = 0; c < kE; ++c) P[c] = f * fmaf(-delta, Q[c], P[c]);
    storeT<T, kE>(A.dq, i, A.s, L, P);
    if (L.head_leader(A.s, 0))
      A.stats[int64_t(i) * A.s.H + L.k[0]] =
          make_float4(any ? m + __log2f(l) : 0.f, delta, __ldg(A.qs + int64_t(i) * A.s.H + L.k[0]),
                      0.f);
  }
};

// ---------------------------------------------------------------------------
// pass 2: source side
// ---------------------------------------------------------------------------

template <typename T, int kE_, bool kRel>
struct SrcPass {
  static constexpr int kE = kE_;
  static constexpr int U = Unroll8<kE>::value;
  const T8Args& A;
  const Lane<1>& L;
  const float* sb;
  float* hist;      // this lane's column of its warp's gradient table
  Raw8<kE> k8;
  float ksc, vsc;
  float v[kE];      // v8_j as floats
  float dk[kE], dv[kE];

  __device__ __forceinline__ SrcPass(const T8Args& a, const Lane<1>& lane) : A(a), L(lane) {}
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE; }
  static __device__ __forceinline__ const T8Dir& dir(const T8Args& A) { return A.csc; }

  __device__ __forceinline__ void zero_sums() {
    zero<kE>(dk);
    zero<kE>(dv);
  }
  __device__ __forceinline__ void begin(int j) {
    k8 = ld8<kE>(A.k8, j, A.s, L, L.ok[0]);
    widen<kE>(ld8<kE>(A.v8, j, A.s, L, L.ok[0]), v);
    ksc = L.ok[0] ? __ldg(A.ks + int64_t(j) * A.s.H + L.k[0]) : 0.f;
    vsc = L.ok[0] ? __ldg(A.vs + int64_t(j) * A.s.H + L.k[0]) : 0.f;
    zero_sums();
  }

  template <bool kFixed>
  __device__ __forceinline__ void edges(const int32_t* cols, int colbase, int beg, int end, int sg,
                                        int SG, int step, int trips, int (&in)[U]) {
    const int H = A.s.H;
    const float kq = ksc * A.scale2;
    int bn[U];
    if (kRel) batch_buckets<U>(A.csc.buckets, beg, end, sg, SG, bn);
    int base = beg;
    for (int t = 0; kFixed ? t < trips : base < end; ++t, base += step) {
      int i[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) i[u] = in[u];
      float bs[U];
      if (kRel) {
#pragma unroll
        for (int u = 0; u < U; ++u) b[u] = bn[u];
        edge_bias<U>(sb, A.s, L, bn, i, bs);
      }
      Raw8<kE> rq[U];
      RawT<T, kE> rg[U];
      float4 st[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = i[u] >= 0 && L.ok[0];
        rq[u] = ld8<kE>(A.q8, i[u], A.s, L, ok);
        rg[u] = ldT<T, kE>(A.dout, i[u], A.s, L, ok);
        st[u] = ok ? ld16f(A.stats + int64_t(i[u]) * H + L.k[0]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (kFixed ? t + 1 < trips : base + step < end) {
        batch_ids<U>(cols, colbase, base + step, end, sg, SG, in);
        if (kRel) batch_buckets<U>(A.csc.buckets, base + step, end, sg, SG, bn);
      }
      float red[2 * U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[kE];
        red[u] = dot8<kE>(rq[u], k8);
        widenT<T, kE>(rg[u], x);
        red[U + u] = dot<kE>(x, v);
      }
      head_sums<2 * U>(red, A.s.hv_log2);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float e = kRel ? fmaf(red[u], kq * st[u].z, bs[u]) : red[u] * (kq * st[u].z);
        const float al = i[u] >= 0 ? ex2(e - st[u].x) : 0.f;
        const float de = i[u] >= 0 ? al * fmaf(red[U + u], vsc, -st[u].y) : 0.f;
        if (kRel && i[u] >= 0 && L.head_leader(A.s, 0)) add_grad(hist, A.s, b[u], de);
        float x[kE];
        widen<kE>(rq[u], x);
        axpy<kE>(dk, de * A.scale * st[u].z, x);
        widenT<T, kE>(rg[u], x);
        axpy<kE>(dv, al, x);
      }
    }
  }

  __device__ __forceinline__ void join_subgroups() {
    subgroup_sums<kE>(dk, A.s);
    subgroup_sums<kE>(dv, A.s);
  }
  __device__ __forceinline__ void put(float* to) const {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
#pragma unroll
    for (int c = 0; c < kE; ++c) {
      to[at + c] = dk[c];
      to[row + at + c] = dv[c];
    }
  }
  __device__ __forceinline__ void take(const float* from) {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
#pragma unroll
    for (int c = 0; c < kE; ++c) {
      dk[c] += from[at + c];
      dv[c] += from[row + at + c];
    }
  }
  __device__ __forceinline__ float* chunk(int slot) const {
    return A.s_part + int64_t(slot) * floats(A.s);
  }
  __device__ __forceinline__ void finish(int j) {
    storeT<T, kE>(A.dkey, j, A.s, L, dk);
    storeT<T, kE>(A.dval, j, A.s, L, dv);
  }
};

// ---------------------------------------------------------------------------
// the walk over the nodes of one direction
// ---------------------------------------------------------------------------

// Block items first, then light nodes: a sub-group each where a warp holds
// several (kSub), a warp otherwise.  kStatic: work goes to blocks and warps by
// index (sums across nodes stay reproducible), else by the counters.
template <class P, bool kSub, bool kStatic>
__device__ __forceinline__ void walk(P& p, const T8Args& A, unsigned char* smem, int* ctr) {
  constexpr int U = P::U;
  const T8Dir& D = P::dir(A);
  const Lane<1>& L = p.L;
  const int wid = threadIdx.x >> 5;
  __shared__ int s_item;
  if (D.n_items > 0) {
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem);
    int32_t* cols = reinterpret_cast<int32_t*>(smem + 16);
    float* wbuf = reinterpret_cast<float*>(smem + D.col_off);  // [kWarps][floats]
    const int nf = P::floats(A.s);
    uint32_t parity = 0;
    if (threadIdx.x == 0) mbar_init(bar, 1);
    for (int turn = 0;; ++turn) {
      if (!kStatic && threadIdx.x == 0) s_item = atomicAdd(ctr, 1);
      __syncthreads();
      const int64_t n = kStatic ? blockIdx.x + int64_t(turn) * gridDim.x : s_item;
      if (n >= D.n_items) break;
      const int4 it = D.items[n];
      if (!stage_edges(cols, D.idx, it.y, it.z, bar, parity, A.err)) return;
      // batches of U * G edges dealt to the warps in turn
      const int beg = it.y + wid * U * L.G, base = it.y & ~3;
      int jn[U];
      batch_ids<U>(cols, base, beg, it.z, L.g, L.G, jn);
      p.begin(it.x);
      p.template edges<false>(cols, base, beg, it.z, L.g, L.G, kWarps * U * L.G, 0, jn);
      p.join_subgroups();
      if (L.g == 0 && L.ok[0]) p.put(wbuf + wid * nf);
      __syncthreads();
      if (wid == 0 && L.g == 0 && L.ok[0]) {
        for (int w = 1; w < kWarps; ++w) p.take(wbuf + w * nf);
        if (it.w < 0)
          p.finish(it.x);
        else
          p.put(p.chunk(it.w));
      }
      __syncthreads();
    }
  }
  // nodes a warp takes at a time: one sub-group's share is four where a warp
  // holds two sub-groups, two otherwise
  const int R = !kSub ? kGrab : L.G >= 32 ? 1 : (L.G == 2 ? 4 : 2);
  const int npull = kSub ? R * L.G : R;
  for (int64_t turn = 0;; ++turn) {
    int64_t t0 = 0;
    if (kStatic) {
      t0 = (turn * gridDim.x * kWarps + int64_t(wid) * gridDim.x + blockIdx.x) * npull;
    } else {
      int t = 0;
      if (L.lane == 0) t = atomicAdd(ctr + 1, npull);
      t0 = __shfl_sync(kFull, t, 0);
    }
    if (t0 >= D.n_light) break;
    int my_n = -1, my_b = 0, my_e = 0;
    if (L.lane < npull && t0 + L.lane < D.n_light) {
      my_n = D.light[t0 + L.lane];
      my_b = D.ptr[my_n];
      my_e = D.ptr[my_n + 1];
    }
    for (int r = 0; r < R; ++r) {
      const int from = kSub ? r * L.G + L.g : r;
      const int i = __shfl_sync(kFull, my_n, from);
      const int beg = __shfl_sync(kFull, my_b, from);
      const int e0 = __shfl_sync(kFull, my_e, from);
      const int end = i >= 0 ? e0 : beg;
      if (!__any_sync(kFull, i >= 0)) break;
      int jn[U];
      if (kSub) {
        int trips = (end - beg + U - 1) / U;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) trips = max(trips, __shfl_xor_sync(kFull, trips, o));
        batch_ids<U>(D.idx, 0, beg, end, 0, 1, jn);
        p.begin(i >= 0 ? i : 0);
        p.template edges<true>(D.idx, 0, beg, end, 0, 1, U, trips, jn);
        if (i >= 0 && L.ok[0]) p.finish(i);
      } else {
        batch_ids<U>(D.idx, 0, beg, end, L.g, L.G, jn);
        p.begin(i);
        p.template edges<false>(D.idx, 0, beg, end, L.g, L.G, U * L.G, 0, jn);
        p.join_subgroups();
        if (L.g == 0 && L.ok[0]) p.finish(i);
      }
    }
  }
}

template <typename T, int kE, bool kSub, bool kRel>
__global__ void __launch_bounds__(kThreads, 2) t8_dst_main(const __grid_constant__ T8Args A) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  DstPass<T, kE, kRel> p(A, L);
  p.sb = kRel ? stage_bias(A.bias, A.buckets * A.s.H, smem + A.rel_off) : nullptr;
  walk<DstPass<T, kE, kRel>, kSub, false>(p, A, smem, A.ctr);
}

template <typename T, int kE, bool kSub, bool kRel>
__global__ void __launch_bounds__(kThreads, 2) t8_src_main(const __grid_constant__ T8Args A) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  SrcPass<T, kE, kRel> p(A, L);
  float* tables = nullptr;
  p.sb = nullptr;
  p.hist = nullptr;
  if (kRel) {
    tables = reinterpret_cast<float*>(smem + A.rel_off) + A.buckets * A.s.H;
    p.hist = clear_grad_tables(tables, A.s, L, A.buckets);
    p.sb = stage_bias(A.bias, A.buckets * A.s.H, smem + A.rel_off);
  }
  walk<SrcPass<T, kE, kRel>, kSub, kRel>(p, A, smem, A.ctr + 2);
  if (kRel) fold_grad_tables(tables, A.s, L, A.buckets, A.db_part);
}

// Hubs: their chunks' partial states added in chunk order, one warp each.
template <class P>
__global__ void __launch_bounds__(kThreads) t8_merge(const __grid_constant__ T8Args A) {
  const Lane<1> L(A.s);
  const T8Dir& D = P::dir(A);
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= D.n_hubs || L.g != 0 || !L.ok[0]) return;
  const int4 hb = D.hubs[t];
  P p(A, L);
  p.zero_sums();
  for (int c = 0; c < hb.z; ++c) p.take(p.chunk(hb.y + c));
  p.finish(hb.x);
}

int rel_blocks8(int sm_count) { return 2 * (sm_count > 0 ? sm_count : 1); }

template <typename K>
cudaError_t launch_main(K kernel, const T8Args& A, const T8Dir& D, size_t smem, int sm_count,
                        int* blocks, cudaStream_t st) {
  *blocks = 0;
  if (D.n_items + D.n_light == 0) return cudaSuccess;
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem))) !=
          cudaSuccess)
    return e;
  const int64_t work = D.n_items + (D.n_light + kWarps * kGrab - 1) / (kWarps * kGrab);
  int64_t cap = persistent_blocks(kernel, smem, sm_count);
  if (cap > rel_blocks8(sm_count)) cap = rel_blocks8(sm_count);
  *blocks = int(work < cap ? work : cap);
  kernel<<<unsigned(*blocks), kThreads, smem, st>>>(A);
  return cudaGetLastError();
}

template <typename T, int kE, bool kRel>
cudaError_t bwd8_t(T8Args A, float* dbias, int sm_count, cudaStream_t st) {
  cudaError_t e;
  if ((e = cudaMemsetAsync(A.ctr, 0, kCounters * sizeof(int), st)) != cudaSuccess) return e;
  const bool sub = A.s.lpr < 32;
  const size_t table = kRel ? size_t(A.buckets) * A.s.H * 4 : 0;
  int blocks = 0;
  using Dst = DstPass<T, kE, kRel>;
  using Src = SrcPass<T, kE, kRel>;
  size_t smem = size_t(A.csr.col_off) + size_t(kWarps) * Dst::floats(A.s) * 4;
  A.rel_off = int(smem);
  if ((e = launch_main(sub ? t8_dst_main<T, kE, true, kRel> : t8_dst_main<T, kE, false, kRel>, A,
                       A.csr, smem + table, sm_count, &blocks, st)) != cudaSuccess)
    return e;
  if (A.csr.n_hubs > 0) {
    t8_merge<Dst><<<unsigned((A.csr.n_hubs + kWarps - 1) / kWarps), kThreads, 0, st>>>(A);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  smem = size_t(A.csc.col_off) + size_t(kWarps) * Src::floats(A.s) * 4;
  A.rel_off = int(smem);
  if (kRel) smem += table + grad_tables_bytes(A.s, A.buckets);
  if ((e = launch_main(sub ? t8_src_main<T, kE, true, kRel> : t8_src_main<T, kE, false, kRel>, A,
                       A.csc, smem, sm_count, &blocks, st)) != cudaSuccess)
    return e;
  if (A.csc.n_hubs > 0) {
    t8_merge<Src><<<unsigned((A.csc.n_hubs + kWarps - 1) / kWarps), kThreads, 0, st>>>(A);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return kRel ? launch_dbias_sum(A.db_part, blocks, A.buckets * A.s.H, dbias, st) : cudaSuccess;
}

template <typename T, int kE>
cudaError_t bwd8_rel(const T8Args& A, float* dbias, int sm_count, cudaStream_t st) {
  return A.buckets > 0 ? bwd8_t<T, kE, true>(A, dbias, sm_count, st)
                       : bwd8_t<T, kE, false>(A, dbias, sm_count, st);
}

// Elements of a lane vector: 16 where a head has as many.
int lane_elems(int D) { return D >= 16 ? 16 : D; }

// The row geometry of `s` (valid: a head is a power of two of 16-byte vectors)
// in vectors of lane_elems(D) elements.
Shape shape8(const Shape& s) {
  Shape w = s;
  const int e = lane_elems(s.D);
  w.hv = s.D / e;
  w.rv = s.H * w.hv;
  w.nv = 1;
  w.hv_log2 = 0;
  while ((1 << w.hv_log2) < w.hv) ++w.hv_log2;
  w.lpr_log2 = 0;
  while ((1 << w.lpr_log2) < w.rv) ++w.lpr_log2;
  w.lpr = 1 << w.lpr_log2;
  return w;
}

T8Dir t8_dir(const Dir& d, const uint8_t* buckets) {
  T8Dir a{};
  a.ptr = d.ptr;
  a.idx = d.idx;
  a.buckets = buckets;
  a.light = d.light;
  a.n_light = d.n_light;
  a.items = d.items;
  a.n_items = d.n_items;
  a.hubs = d.hubs;
  a.n_hubs = d.n_hubs;
  a.col_off = int(16 + align_up(size_t(d.max_item + 4) * 4, 16));
  return a;
}

struct T8Layout {
  size_t ctr, stats, d_part, s_part, db_part, total;
};

T8Layout t8_layout(const gnn_graph* g, const Shape& s, int buckets) {
  const size_t row = size_t(s.H) * s.D;
  T8Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t r = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  L.ctr = take(kCounters * 4);
  L.stats = take(size_t(g->n) * s.H * 16);
  L.d_part = take(size_t(g->csr.n_hub_chunks) * (2 * row + 3 * s.H) * 4);
  L.s_part = take(size_t(g->csc.n_hub_chunks) * 2 * row * 4);
  L.db_part = take(size_t(rel_blocks8(g->sm_count)) * buckets * s.H * 8);
  L.total = off;
  return L;
}

}  // namespace

size_t transformer8_ws_bytes(const gnn_graph* g, const Shape& s, int buckets) {
  return t8_layout(g, s, buckets).total;
}

cudaError_t launch_transformer8_backward(const gnn_graph* g, const gnn_rel* rel, const Shape& s,
                                         gnn_dtype dt, const gnn_packed8& q,
                                         const gnn_packed8& key, const gnn_packed8& val,
                                         float scale, const float* bias, const void* dout,
                                         void* dq, void* dkey, void* dval, float* dbias, char* ws,
                                         cudaStream_t st) {
  const T8Layout W = t8_layout(g, s, rel ? rel->buckets : 0);
  T8Args A{};
  A.s = shape8(s);
  A.csr = t8_dir(g->csr, rel ? rel->csr : nullptr);
  A.csc = t8_dir(g->csc, rel ? rel->csc : nullptr);
  A.q8 = q.values;
  A.k8 = key.values;
  A.v8 = val.values;
  A.qs = q.scale;
  A.ks = key.scale;
  A.vs = val.scale;
  A.scale = scale;
  A.scale2 = scale * kLog2e;
  A.dout = dout;
  A.dq = dq;
  A.dkey = dkey;
  A.dval = dval;
  A.stats = reinterpret_cast<float4*>(ws + W.stats);
  A.d_part = reinterpret_cast<float*>(ws + W.d_part);
  A.s_part = reinterpret_cast<float*>(ws + W.s_part);
  A.bias = bias;
  A.buckets = rel ? rel->buckets : 0;
  A.db_part = reinterpret_cast<double*>(ws + W.db_part);
  A.ctr = reinterpret_cast<int*>(ws + W.ctr);
  A.err = g->err;
  const int e = lane_elems(s.D), sms = g->sm_count;
  if (dt == GNN_F32)
    return e == 16  ? bwd8_rel<float, 16>(A, dbias, sms, st)
           : e == 8 ? bwd8_rel<float, 8>(A, dbias, sms, st)
                    : bwd8_rel<float, 4>(A, dbias, sms, st);
  return e == 16 ? bwd8_rel<__nv_bfloat16, 16>(A, dbias, sms, st)
                 : bwd8_rel<__nv_bfloat16, 8>(A, dbias, sms, st);
}

}  // namespace gnn
