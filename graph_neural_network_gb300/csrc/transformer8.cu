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
//     over e_ij = scale q^_i . k^_j (+ bias): with p = exp(e - m) (SoftRef) it carries
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
// Bound: instruction issue and the latency of gathers together (issue 50 to 60 % of
// cycles).  Per edge pass 1 gathers 2 F bytes and two scales per head, pass 2 F (1 + s)
// bytes and a record per head: half to three quarters of what the passes over
// 16-bit rows gather, while widening bytes costs more than widening bfloat16.  A lane
// holds 16 elements (8 or 4 of narrow heads), so that what an edge costs whatever its
// width is shared by more.  300k nodes, 6M edges, H4 D64 bf16 with the bias: 0.81 and
// 0.91 ms, against 0.67 and 0.85 from the rows themselves; 100k nodes, 1.7M edges, H4
// D32 f32 without: 0.11 and 0.17 ms.  What the checkpoints save is memory: a byte
// instead of two or four per element of q, key and val, and lse.
//
// Masks, biases of any size and the bias gradient as in transformer_rel.cu; the work is cut as
// edgewalk.cuh says.
#include "edgewalk.cuh"
#include "lanevec.cuh"

namespace gnn {
namespace {

struct T8Args {
  Shape s;                 // in kE-element vectors
  Walk walk;
  WalkDir dir;
  const int8_t *q8, *k8, *v8;
  const float *qs, *ks, *vs;   // [N][H]
  float scale, scale2;     // natural units, base 2
  const void* dout;
  void *dq, *dkey, *dval;
  // [N][H] {lse (base 2), Delta, qs, 0}, or {log2 of the sum, Delta, qs, the reference's
  // bias} (Bias::kAny)
  float4* stats;
  const float* bias;
  int buckets;
  double* db_part;         // [pass 2 blocks][buckets][H]
};

// ---- lane vectors of kE elements ---------------------------------------------

template <int kE>
struct Raw8 {
  uint32_t w[kE / 4];
};

template <int kE>
__device__ __forceinline__ Raw8<kE> ld8(const char* at) {
  Raw8<kE> r;
  if constexpr (kE == 16) {
    const uint4 t = ld16(at);
    r.w[0] = t.x;
    r.w[1] = t.y;
    r.w[2] = t.z;
    r.w[3] = t.w;
  } else if constexpr (kE == 8) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(at));
    r.w[0] = t.x;
    r.w[1] = t.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
  }
  return r;
}

// The number of head k (base points to it) of a node in a [N][H] array.
template <typename X>
__device__ __forceinline__ X of_head(const X* base, int node, const Shape& s) {
  return __ldg(base + uint64_t(uint32_t(node)) * uint32_t(s.H));
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

// Edges in flight per lane: pass 1 gathers 32 bytes of an edge and keeps four in
// flight (300k-node graph, both passes: 1,700 us; with three 1,746, with five
// 1,743); pass 2 gathers three to five times as much and keeps two (with three
// 1,735 us; 100k nodes in float32 272 us, with three 320).
// Half as many beside large biases, where that costs the ordinary form nothing
// (transformer_rel.cu).
template <int kE, Bias kBias>
struct Edges {
  static constexpr bool any = kBias == Bias::kAny;
  static constexpr int dst = any ? 2 : 4, src = kE < 16 ? 4 : any ? 1 : 2;
};

// ---------------------------------------------------------------------------
// pass 1: destination side
// ---------------------------------------------------------------------------

template <typename T, int kE_, Bias kBias>
struct DstPass {
  static constexpr int kE = kE_;
  static constexpr bool kRel = kBias != Bias::kNone;
  static constexpr int U = Edges<kE, kBias>::dst;
  static constexpr bool kBuckets = kRel;
  const T8Args& A;
  const Lane<1>& L;
  const LanePlace<kE> place;                      // in rows of bytes
  const LanePlace<kE * int(sizeof(T))> rows;      // in rows of T
  const LaneRows<kE> r0, r1;  // the gathered rows
  const float* sb;            // the bias table
  // the node
  Raw8<kE> q8;
  float qsc;        // qs_i
  HeldT<T, kE> g;   // dout_i
  // its sums
  SoftRef<kBias> ref;
  float l, d, P[kE], Q[kE];

  __device__ __forceinline__ DstPass(const T8Args& a, const Lane<1>& lane)
      : A(a), L(lane), place(a.s, lane), rows(a.s, lane), r0(a.k8, place), r1(a.v8, place) {}
  // floats of a partial state: P, Q, then l, d and the reference per head
  static constexpr int kHead = 2 + SoftRef<kBias>::kFloats;
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE + kHead * s.H; }

  __device__ __forceinline__ void clear() {
    ref.clear();
    l = d = 0.f;
    zero<kE>(P);
    zero<kE>(Q);
  }
  __device__ __forceinline__ void begin(int i) {
    q8 = ld8<kE>(place.of(A.q8, i));
    qsc = of_head(A.qs + L.k[0], i, A.s);
    g.fetch(rows.of(A.dout, i));
    clear();
  }
  __device__ __forceinline__ void rescale(float r) {
    l *= r;
    d *= r;
    scale<kE>(P, r);
    scale<kE>(Q, r);
  }

  template <class F>
  __device__ __forceinline__ void batch(const int (&j)[U], const int (&b)[U], int cnt,
                                        const F& sent) {
    Raw8<kE> rk[U], rv[U];
    float ks[U], vs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rk[u] = ld8<kE>(r0.at(j[u]));
      rv[u] = ld8<kE>(r1.at(j[u]));
      ks[u] = of_head(A.ks + L.k[0], j[u], A.s);
      vs[u] = of_head(A.vs + L.k[0], j[u], A.s);
    }
    float bs[U];
    bool ok[U];  // there, and not masked for the lane's head
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bs[u] = kRel ? sb[b[u] * A.s.H] : 0.f;
      ok[u] = u < cnt && (!kRel || bs[u] != -INFINITY);
    }
    sent();
    const float qk = qsc * A.scale2;
    float red[2 * U];
    {
      float own[kE];
      held_ready();
      widenT<T, kE>(g.get(), own);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[kE];
        red[u] = dot8<kE>(rk[u], q8);
        widen<kE>(rv[u], x);
        red[U + u] = dot<kE>(x, own);
      }
    }
    head_sums<2 * U>(red, A.s.hv_log2);
    ref.template weigh<U>(red, qk, ks, bs, ok, l, [&](float r) { rescale(r); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      const float p = ex2(red[u]);
      const float pd = p * (red[U + u] * vs[u]);
      l += p;
      d += pd;
      float x[kE];
      widen<kE>(rk[u], x);
      axpy<kE>(P, pd * ks[u], x);
      axpy<kE>(Q, p * ks[u], x);
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
      float* h = to + 2 * row + kHead * L.k[0];
      h[0] = l;
      h[1] = d;
      ref.put(h + 2);
    }
  }
  template <int N>
  __device__ __forceinline__ void take(const float* from, int step) {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
    float lb[N], db[N], ref_b[SoftRef<kBias>::kFloats][N], r[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float* h = from + n * step + 2 * row + kHead * L.k[0];
      lb[n] = part_load(h);
      db[n] = part_load(h + 1);
#pragma unroll
      for (int c = 0; c < SoftRef<kBias>::kFloats; ++c) ref_b[c][n] = part_load(h + 2 + c);
    }
    ref.template join<N>(l, lb, ref_b, [&](float by) { rescale(by); }, r);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      l = fmaf(lb[n], r[n], l);
      d = fmaf(db[n], r[n], d);
    }
    float x[N][kE];
#pragma unroll
    for (int n = 0; n < N; ++n) part_row<kE>(from + n * step + at, x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) axpy<kE>(P, r[n], x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) part_row<kE>(from + n * step + row + at, x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) axpy<kE>(Q, r[n], x[n]);
  }
  __device__ __forceinline__ void finish(int i) {
    const bool any = l != 0.f;  // a NaN stays one
    const float inv = any ? reciprocal(l) : 0.f;
    const float delta = d * inv;
    minus_scaled<kE>(P, Q, delta, A.scale * inv);
    storeT<T, kE>(const_cast<char*>(rows.of(A.dq, i)), P);
    if (!L.head_leader(A.s, 0)) return;
    float4 r = make_float4(0.f, delta, qsc, 0.f);
    if constexpr (kBias == Bias::kAny) {  // (a row without weights: pass 2 gives it none)
      r.x = any ? ref.d + __log2f(l) : 0.f;
      r.w = any ? ref.b : INFINITY;
    } else if (any) {
      r.x = ref.m + __log2f(l);
    }
    A.stats[int64_t(i) * A.s.H + L.k[0]] = r;
  }
};

// ---------------------------------------------------------------------------
// pass 2: source side
// ---------------------------------------------------------------------------

// kPair: the form of the bias gradient's tables.
template <typename T, int kE_, Bias kBias, bool kPair>
struct SrcPass {
  static constexpr int kE = kE_;
  static constexpr bool kRel = kBias != Bias::kNone;
  static constexpr int U = Edges<kE, kBias>::src;
  static constexpr bool kBuckets = kRel;
  const T8Args& A;
  const Lane<1>& L;
  const LanePlace<kE> place;                      // in rows of bytes
  const LanePlace<kE * int(sizeof(T))> rows;      // in rows of T
  const LaneRows<kE> r0;      // the gathered rows
  const LaneRows<kE * int(sizeof(T))> r1;
  const float* sb;            // the bias table
  float* hist;      // this lane's column of its warp's gradient table
  Raw8<kE> k8;
  float ksc, vsc;
  Raw8<kE> v8;
  bool fresh;              // v8 not widened yet (begin waits for no load)
  // v8_j, exact in bfloat16 too, where both halves of the product stay packed (300k-node
  // graph: 1,699 us a call, 1,730 with floats)
  HeldT<T, kE> v;
  float dk[kE], dv[kE];

  __device__ __forceinline__ SrcPass(const T8Args& a, const Lane<1>& lane)
      : A(a), L(lane), place(a.s, lane), rows(a.s, lane), r0(a.q8, place), r1(a.dout, rows) {}
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE; }

  __device__ __forceinline__ void clear() {
    zero<kE>(dk);
    zero<kE>(dv);
  }
  __device__ __forceinline__ void begin(int j) {
    k8 = ld8<kE>(place.of(A.k8, j));
    v8 = ld8<kE>(place.of(A.v8, j));
    fresh = true;
    ksc = of_head(A.ks + L.k[0], j, A.s);
    vsc = of_head(A.vs + L.k[0], j, A.s);
    clear();
  }

  template <class F>
  __device__ __forceinline__ void batch(const int (&i)[U], const int (&b)[U], int cnt,
                                        const F& sent) {
    Raw8<kE> rq[U];
    RawT<T, kE> rg[U];
    float4 st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rq[u] = ld8<kE>(r0.at(i[u]));
      rg[u] = ldT<T, kE>(r1.at(i[u]));
      // (no __ldg: pass 1 may still be writing when this kernel starts)
      st[u] = A.stats[L.k[0] + uint64_t(uint32_t(i[u])) * uint32_t(A.s.H)];
    }
    float bs[U];
    int bk[U];
    bool ok[U];  // there, and not masked for the lane's head
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bk[u] = kRel ? b[u] : 0;
      bs[u] = kRel ? sb[bk[u] * A.s.H] : 0.f;
      ok[u] = u < cnt && (!kRel || bs[u] != -INFINITY);
    }
    sent();
    const float kq = ksc * A.scale2;
    if (fresh) {
      float x[kE];
      widen<kE>(v8, x);
      v.put(x);
      fresh = false;
    }
    const RawT<T, kE> own = v.get();
    float red[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      red[u] = dot8<kE>(rq[u], k8);
      red[U + u] = dotT<kE>(own, rg[u]);
    }
    head_sums<2 * U>(red, A.s.hv_log2);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float e;
      if (kBias == Bias::kAny)
        e = fmaf(bs[u] - st[u].w, kLog2e, fmaf(red[u], beside(st[u].w, kq * st[u].z), -st[u].x));
      else
        e = (kRel ? fmaf(red[u], kq * st[u].z, bs[u]) : red[u] * (kq * st[u].z)) - st[u].x;
      if (!ok[u]) continue;
      const float al = ex2(e);
      const float de = al * fmaf(red[U + u], vsc, -st[u].y);
      if (kRel) add_grad<kPair>(hist, A.s, L.head_leader(A.s, 0), bk[u], de);
      float x[kE];
      widen<kE>(rq[u], x);
      axpy<kE>(dk, de * A.scale * st[u].z, x);
      widenT<T, kE>(rg[u], x);
      axpy<kE>(dv, al, x);
    }
  }
  __device__ __forceinline__ void put(float* to) const {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
#pragma unroll
    for (int c = 0; c < kE; ++c) {
      to[at + c] = dk[c];
      to[row + at + c] = dv[c];
    }
  }
  template <int N>
  __device__ __forceinline__ void take(const float* from, int step) {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
    take_rows<kE, N>(dk, from + at, step);
    take_rows<kE, N>(dv, from + row + at, step);
  }
  __device__ __forceinline__ void finish(int j) {
    storeT<T, kE>(const_cast<char*>(rows.of(A.dkey, j)), dk);
    storeT<T, kE>(const_cast<char*>(rows.of(A.dval, j)), dv);
  }
};

constexpr int kPerSm = 2;  // resident blocks

template <typename T, int kE, bool kRel>
__global__ void __launch_bounds__(kThreads, kPerSm) t8_dst(const __grid_constant__ T8Args A) {
  let_next_start();
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  __shared__ __align__(16) unsigned char held[kWarps * HeldT<T, kE>::kBytes];
  const auto pass = [&](auto p, float* table) {
    p.g.place(held + (threadIdx.x >> 5) * HeldT<T, kE>::kBytes, L.lane);
    p.sb = table;
    walk(p, A.walk, A.dir, A.s, L);
  };
  if constexpr (kRel) {
    float* table = reinterpret_cast<float*>(smem);
    if (stage_bias(A.bias, A.buckets * A.s.H, table))
      pass(DstPass<T, kE, Bias::kAny>(A, L), table + L.k[0]);
    else
      pass(DstPass<T, kE, Bias::kOrdinary>(A, L), table + L.k[0]);
  } else {
    pass(DstPass<T, kE, Bias::kNone>(A, L), nullptr);
  }
}

template <typename T, int kE, bool kRel, bool kPair>
__global__ void __launch_bounds__(kThreads, kPerSm) t8_src(const __grid_constant__ T8Args A) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  __shared__ __align__(16) unsigned char held[kWarps * HeldT<T, kE>::kBytes];
  const auto pass = [&](auto p, float* table, float* column) {
    p.v.place(held + (threadIdx.x >> 5) * HeldT<T, kE>::kBytes, L.lane);
    p.sb = table;
    p.hist = column;
    walk(p, A.walk, A.dir, A.s, L);
  };
  if constexpr (kRel) {
    float* tables = reinterpret_cast<float*>(smem);
    float* column = clear_grad_tables(tables, A.s, L, A.buckets);
    float* table = reinterpret_cast<float*>(smem + grad_tables_bytes(A.s, A.buckets));
    if (stage_bias(A.bias, A.buckets * A.s.H, table))
      pass(SrcPass<T, kE, Bias::kAny, kPair>(A, L), table + L.k[0], column);
    else
      pass(SrcPass<T, kE, Bias::kOrdinary, kPair>(A, L), table + L.k[0], column);
    let_next_start();
    fold_grad_tables<kPair>(tables, A.s, L, A.buckets, A.db_part);
  } else {
    pass(SrcPass<T, kE, Bias::kNone, kPair>(A, L), nullptr, nullptr);
  }
}

// after: launched behind the first pass of the same call (launch_after).
cudaError_t launch(void (*kernel)(T8Args), const T8Args& A, int blocks, size_t smem,
                   cudaStream_t st, bool after = false) {
  cudaError_t e;
  // (the default limit, 48 KB, counts the kernels' static 16 KB too)
  if ((e = allow_smem(kernel, smem, 32 * 1024)) != cudaSuccess) return e;
  if (after) return launch_after(kernel, dim3(unsigned(blocks)), kThreads, smem, st, A);
  kernel<<<unsigned(blocks), kThreads, smem, st>>>(A);
  return cudaGetLastError();
}

template <typename T, int kE, bool kRel>
cudaError_t bwd8_t(T8Args A, const gnn_graph* g, const gnn_rel* rel, const WalkPlan& p,
                   float* dbias, cudaStream_t st) {
  const Walk src = make_walk(p, g->n, g->csc.max_deg, A.walk.arrived + p.workers, A.walk.part);
  cudaError_t e;
  // the counters of both passes
  if ((A.walk.cuts || src.cuts) &&
      (e = cudaMemsetAsync(A.walk.arrived, 0, size_t(p.workers) * 2 * sizeof(int), st)) !=
          cudaSuccess)
    return e;
  const size_t table = kRel ? size_t(A.buckets) * A.s.H * 4 : 0;
  if ((e = launch(t8_dst<T, kE, kRel>, A, p.blocks, table, st)) != cudaSuccess) return e;
  A.dir = WalkDir{g->csc.ptr, g->csc.idx, rel ? rel->csc : nullptr};
  A.walk = src;
  const size_t grads = kRel ? grad_tables_bytes(A.s, A.buckets) : 0;
  const auto src_pass = kRel && grad_pairs(A.s, A.buckets) ? t8_src<T, kE, kRel, kRel>
                                                           : t8_src<T, kE, kRel, false>;
  if ((e = launch(src_pass, A, p.blocks, table + grads, st, true)) != cudaSuccess) return e;
  return kRel ? launch_dbias_sum(A.db_part, p.blocks, A.buckets * A.s.H, dbias, st) : cudaSuccess;
}

template <typename T, int kE>
cudaError_t bwd8_rel(const T8Args& A, const gnn_graph* g, const gnn_rel* rel, const WalkPlan& p,
                     float* dbias, cudaStream_t st) {
  return rel ? bwd8_t<T, kE, true>(A, g, rel, p, dbias, st)
             : bwd8_t<T, kE, false>(A, g, rel, p, dbias, st);
}

// Elements of a lane vector: 16 where a head has as many and dout's rows can be read
// 32 bytes at a time, else those of 16 bytes of dout.
int lane_elems(const Shape& s, bool aligned) {
  if (!aligned) return 16 / s.esize;
  return s.D >= 16 ? 16 : s.D;
}

struct T8Layout {
  size_t arrived, part, stats, db_part, total;
  WalkPlan plan;  // the same for both directions: n and e are
};

T8Layout t8_layout(const gnn_graph* g, const Shape& s, int buckets, int elems) {
  T8Layout L{};
  L.plan = walk_plan(g->n, g->e, lane_shape(s, elems), kPerSm, g->sm_count);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t r = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  L.arrived = take(size_t(L.plan.workers) * 2 * sizeof(int));
  L.part = take(size_t(L.plan.workers) * 2 * (2 * size_t(s.H) * s.D + 4 * s.H) * 4);
  L.stats = take(size_t(g->n) * s.H * 16);
  L.db_part = take(size_t(L.plan.blocks) * buckets * s.H * 8);
  L.total = off;
  return L;
}

}  // namespace

size_t transformer8_ws_bytes(const gnn_graph* g, const Shape& s, int buckets) {
  const size_t a = t8_layout(g, s, buckets, lane_elems(s, true)).total;
  const size_t b = t8_layout(g, s, buckets, lane_elems(s, false)).total;
  return a > b ? a : b;
}

cudaError_t launch_transformer8_backward(const gnn_graph* g, const gnn_rel* rel, const Shape& s,
                                         gnn_dtype dt, const gnn_packed8& q,
                                         const gnn_packed8& key, const gnn_packed8& val,
                                         float scale, const float* bias, const void* dout,
                                         void* dq, void* dkey, void* dval, float* dbias, char* ws,
                                         cudaStream_t st) {
  const int e = lane_elems(s, aligned32(dout));
  const T8Layout W = t8_layout(g, s, rel ? rel->buckets : 0, e);
  T8Args A{};
  A.s = lane_shape(s, e);
  A.walk = make_walk(W.plan, g->n, g->csr.max_deg, reinterpret_cast<int*>(ws + W.arrived),
                     reinterpret_cast<float*>(ws + W.part));
  A.dir = WalkDir{g->csr.ptr, g->csr.idx, rel ? rel->csr : nullptr};
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
  A.bias = bias;
  A.buckets = rel ? rel->buckets : 0;
  A.db_part = reinterpret_cast<double*>(ws + W.db_part);
  if (dt == GNN_F32)
    return e == 16  ? bwd8_rel<float, 16>(A, g, rel, W.plan, dbias, st)
           : e == 8 ? bwd8_rel<float, 8>(A, g, rel, W.plan, dbias, st)
                    : bwd8_rel<float, 4>(A, g, rel, W.plan, dbias, st);
  return e == 16 ? bwd8_rel<__nv_bfloat16, 16>(A, g, rel, W.plan, dbias, st)
                 : bwd8_rel<__nv_bfloat16, 8>(A, g, rel, W.plan, dbias, st);
}

}  // namespace gnn
