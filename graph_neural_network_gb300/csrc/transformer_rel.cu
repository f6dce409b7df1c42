// Graph-transformer attention with a learned relative position bias, forward and
// backward.  As transformer.cu, with
//   e_ij = scale * q_i[k] . key_j[k] + bias[b_ij][k],
// the bucket b_ij read next to the edge's node id from the prepared bucket bytes
// (relpos.cu) of the direction being walked, and the bias table in shared
// memory.  An entry of -infinity masks its edges for that head: the lanes of the head
// skip them like absent ones, so what their rows hold enters no sum.  Tables with large
// finite entries take another form of the scores (Bias), within the same kernels.
//
// Forward: one pass over the CSR with an online softmax whose reference moves
// only when a score passes it.  Backward pass 1 (CSR): Delta, P = sum alpha da
// key_j, Q = sum alpha key_j, dq_i = scale (P - Delta Q), record {lse, Delta}.  (Beside
// large biases lse, one number, has lost what the weights need: there the pass is an online
// softmax of its own and records the sum and the reference apart.)  Pass 2 (CSC): dkey,
// dval, and dbias[b][k] = sum of de_ij over the edges of bucket b, de_ij = alpha_ij
// (da_ij - Delta_i) being known per edge there: each lane that leads a head adds into a
// column of its own of its warp's table in shared memory (no atomics, no bank conflicts),
// the block adds its tables in a fixed order in float64, and dbias_sum adds the blocks.
//
// Bound: latency of the gathers, 2 rows an edge and pass (edgewalk.cuh, which also
// says how the work is cut and what it measured).  A lane holds 32 bytes of a row
// (16 where a head has no more), so that what an edge costs whatever its width
// (ids, bucket, bias, score, exponential, addresses) is shared by more elements;
// both dot products of bfloat16 rows multiply the packed halves.
#include <type_traits>

#include "edgewalk.cuh"
#include "lanevec.cuh"

namespace gnn {
namespace {

struct RelArgs {
  Shape s;                 // in kE-element vectors
  Walk walk;
  WalkDir dir;
  const void *q, *key, *val;
  float scale, scale2;     // natural units, base 2
  const float* bias;       // [buckets][H]
  int buckets;
  void* out;
  float* lse;
  const float* lse_in;
  const void* dout;
  void *dq, *dkey, *dval;
  // [N][H] {lse (base 2), Delta}, or {log2 of the sum, Delta, the reference's bias,
  // factor of the dot products} (Bias::kAny)
  void* stats;
  double* db_part;         // [pass 2 blocks][buckets][H]
};

// Edges in flight per lane, for lane vectors of 32 bytes (twice as many of 16): as
// many as the registers of 16 warps an SM hold beside the accumulators, of which
// float32 lanes have half as many.  Training step on the 300k-node bfloat16 graph when
// these were compared (2,026 us now): 2,044 us; forward with three edges 2,083, with five
// 2,060; pass 1 with two 2,162, with four 2,216; pass 2 with three 2,088.  On the 100k-node
// float32 graph: 499 us; pass 2 with two 524, with four 642; pass 1 with two 562, with
// five 518.
// Beside large biases, whose form needs more registers, as many or fewer: with more the
// compiler also schedules the ordinary form of the same kernel worse (forward 593 instead
// of 514 us; pass 2 with 16-byte vectors, 200k nodes H8 D4 float32, 235 instead of 221).
template <typename T, int kE, Bias kBias, int kBf16, int kF32, bool kHalve = true>
struct RelEdges {
  static constexpr int full = 32 / (kE * int(sizeof(T)));  // 1: vectors of 32 bytes
  static constexpr int all = (sizeof(T) == 4 ? kF32 : kBf16) * full;
  static constexpr int any = full == 2 ? 2 : kHalve ? (all + 1) / 2 : all;
  static constexpr int value = kBias == Bias::kAny ? any : all;
};
constexpr int kFwdEdges = 4, kDstEdges = 3, kDstEdgesF32 = 3, kSrcEdges = 2, kSrcEdgesF32 = 3;

// ---- forward -----------------------------------------------------------------

template <typename T, int kE_, Bias kBias>
struct RelFwd {
  static constexpr int kE = kE_;
  static constexpr int U = RelEdges<T, kE, kBias, kFwdEdges, kFwdEdges>::value;
  static constexpr int kRow = kE * int(sizeof(T));
  static constexpr bool kBuckets = true;
  const RelArgs& A;
  const Lane<1>& L;
  const LanePlace<kRow> place;
  const LaneRows<kRow> r0, r1;  // the gathered rows
  const float* sb;    // the bias table
  HeldT<T, kE> q;
  SoftRef<kBias> ref;
  float l, acc[kE];

  __device__ __forceinline__ RelFwd(const RelArgs& a, const Lane<1>& lane)
      : A(a), L(lane), place(a.s, lane), r0(a.key, place), r1(a.val, place) {}
  static constexpr int kHead = 1 + SoftRef<kBias>::kFloats;  // l, the reference
  static __host__ __device__ int floats(const Shape& s) { return s.rv * kE + kHead * s.H; }

  __device__ __forceinline__ void clear() {
    ref.clear();
    l = 0.f;
    zero<kE>(acc);
  }
  __device__ __forceinline__ void rescale(float by) {
    l *= by;
    scale<kE>(acc, by);
  }
  __device__ __forceinline__ void begin(int i) {
    q.fetch(place.of(A.q, i));
    clear();
  }
  template <class F>
  __device__ __forceinline__ void batch(const int (&j)[U], const int (&b)[U], int cnt,
                                        const F& sent) {
    RawT<T, kE> rk[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rk[u] = ldT<T, kE>(r0.at(j[u]));
      rv[u] = ldT<T, kE>(r1.at(j[u]));
    }
    float bs[U];
    bool ok[U];  // there, and not masked for the lane's head
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bs[u] = sb[b[u] * A.s.H];
      ok[u] = u < cnt && bs[u] != -INFINITY;
    }
    sent();
    held_ready();
    float sc[U];
    const RawT<T, kE> own = q.get();
#pragma unroll
    for (int u = 0; u < U; ++u) sc[u] = dotT<kE>(own, rk[u]);
    head_sums<U>(sc, A.s.hv_log2);
    float one[U];
#pragma unroll
    for (int u = 0; u < U; ++u) one[u] = 1.f;
    ref.template weigh<U>(sc, A.scale2, one, bs, ok, l, [&](float by) { rescale(by); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      const float p = ex2(sc[u]);
      l += p;
      float x[kE];
      widenT<T, kE>(rv[u], x);
      axpy<kE>(acc, p, x);
    }
  }
  __device__ __forceinline__ void put(float* to) const {
#pragma unroll
    for (int c = 0; c < kE; ++c) to[L.q[0] * kE + c] = acc[c];
    if (L.head_leader(A.s, 0)) {
      float* h = to + A.s.rv * kE + kHead * L.k[0];
      h[0] = l;
      ref.put(h + 1);
    }
  }
  template <int N>
  __device__ __forceinline__ void take(const float* from, int step) {
    float lb[N], ref_b[SoftRef<kBias>::kFloats][N], r[N], x[N][kE];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float* h = from + n * step + A.s.rv * kE + kHead * L.k[0];
      lb[n] = part_load(h);
#pragma unroll
      for (int c = 0; c < SoftRef<kBias>::kFloats; ++c) ref_b[c][n] = part_load(h + 1 + c);
    }
    ref.template join<N>(l, lb, ref_b, [&](float by) { rescale(by); }, r);
#pragma unroll
    for (int n = 0; n < N; ++n) part_row<kE>(from + n * step + L.q[0] * kE, x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      l = fmaf(lb[n], r[n], l);
      axpy<kE>(acc, r[n], x[n]);
    }
  }
  __device__ __forceinline__ void finish(int i) {
    const bool any = l != 0.f;  // a NaN stays one
    scale<kE>(acc, any ? reciprocal(l) : 0.f);
    storeT<T, kE>(const_cast<char*>(place.of(A.out, i)), acc);
    if (L.head_leader(A.s, 0))
      A.lse[int64_t(i) * A.s.H + L.k[0]] = any ? ref.lse(l) : -INFINITY;
  }
};

// ---- backward pass 1: destination side ---------------------------------------

template <typename T, int kE_, Bias kBias>
struct RelDst {
  static constexpr int kE = kE_;
  static constexpr int U = RelEdges<T, kE, kBias, kDstEdges, kDstEdgesF32>::value;
  static constexpr int kRow = kE * int(sizeof(T));
  static constexpr bool kBuckets = true;
  const RelArgs& A;
  const Lane<1>& L;
  const LanePlace<kRow> place;
  const LaneRows<kRow> r0, r1;  // the gathered rows
  const float* sb;    // the bias table
  HeldT<T, kE> q, g;
  static constexpr bool kAny = kBias == Bias::kAny;
  float lse2;          // ordinary biases: weights are relative to it
  SoftRef<kBias> ref;  // any: weights to be divided by their sum l
  float l;
  float delta, P[kE], Q[kE];

  __device__ __forceinline__ RelDst(const RelArgs& a, const Lane<1>& lane)
      : A(a), L(lane), place(a.s, lane), r0(a.key, place), r1(a.val, place) {}
  static constexpr int kHead = kAny ? 4 : 1;  // Delta, l, the reference
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE + kHead * s.H; }

  __device__ __forceinline__ void clear() {
    ref.clear();
    l = delta = 0.f;
    zero<kE>(P);
    zero<kE>(Q);
  }
  __device__ __forceinline__ void rescale(float by) {
    l *= by;
    delta *= by;
    scale<kE>(P, by);
    scale<kE>(Q, by);
  }
  __device__ __forceinline__ void begin(int i) {
    q.fetch(place.of(A.q, i));
    g.fetch(place.of(A.dout, i));
    if (!kAny) lse2 = __ldg(A.lse_in + int64_t(i) * A.s.H + L.k[0]) * kLog2e;
    clear();
  }
  template <class F>
  __device__ __forceinline__ void batch(const int (&j)[U], const int (&b)[U], int cnt,
                                        const F& sent) {
    RawT<T, kE> rk[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rk[u] = ldT<T, kE>(r0.at(j[u]));
      rv[u] = ldT<T, kE>(r1.at(j[u]));
    }
    float bs[U];
    bool ok[U];  // there, and not masked for the lane's head
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bs[u] = sb[b[u] * A.s.H];
      ok[u] = u < cnt && bs[u] != -INFINITY;
    }
    sent();
    held_ready();
    float red[2 * U];
    {
      const RawT<T, kE> own = g.get();
#pragma unroll
      for (int u = 0; u < U; ++u) red[U + u] = dotT<kE>(own, rv[u]);
    }
    {
      const RawT<T, kE> own = q.get();
#pragma unroll
      for (int u = 0; u < U; ++u) red[u] = dotT<kE>(own, rk[u]);
    }
    head_sums<2 * U>(red, A.s.hv_log2);
    if (kAny) {
      float one[U];
#pragma unroll
      for (int u = 0; u < U; ++u) one[u] = 1.f;
      ref.template weigh<U>(red, A.scale2, one, bs, ok, l, [&](float by) { rescale(by); });
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) red[u] = fmaf(red[u], A.scale2, bs[u]) - lse2;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      const float al = ex2(red[u]);
      const float ad = al * red[U + u];
      if (kAny) l += al;
      delta += ad;
      float x[kE];
      widenT<T, kE>(rk[u], x);
      axpy<kE>(P, ad, x);
      axpy<kE>(Q, al, x);
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
      h[0] = delta;
      if (kAny) {
        h[1] = l;
        ref.put(h + 2);
      }
    }
  }
  template <int N>
  __device__ __forceinline__ void take(const float* from, int step) {
    const int row = A.s.rv * kE, at = L.q[0] * kE;
    float db[N], lb[N], ref_b[SoftRef<kBias>::kFloats][N], r[N], x[N][kE];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float* h = from + n * step + 2 * row + kHead * L.k[0];
      db[n] = part_load(h);
      r[n] = 1.f;
      if (!kAny) continue;
      lb[n] = part_load(h + 1);
#pragma unroll
      for (int c = 0; c < SoftRef<kBias>::kFloats; ++c) ref_b[c][n] = part_load(h + 2 + c);
    }
    if (kAny) {
      ref.template join<N>(l, lb, ref_b, [&](float by) { rescale(by); }, r);
#pragma unroll
      for (int n = 0; n < N; ++n) l = fmaf(lb[n], r[n], l);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) part_row<kE>(from + n * step + at, x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      delta = fmaf(db[n], r[n], delta);
      axpy<kE>(P, r[n], x[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) part_row<kE>(from + n * step + row + at, x[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) axpy<kE>(Q, r[n], x[n]);
  }
  __device__ __forceinline__ void finish(int i) {
    const bool any = l != 0.f;  // a NaN stays one
    const float inv = !kAny ? 1.f : any ? reciprocal(l) : 0.f;
    if (kAny) delta *= inv;
    minus_scaled<kE>(P, Q, delta, A.scale * inv);
    storeT<T, kE>(const_cast<char*>(place.of(A.dq, i)), P);
    if (!L.head_leader(A.s, 0)) return;
    const int64_t to = int64_t(i) * A.s.H + L.k[0];
    if constexpr (kAny)  // (a row without weights: no edge gets one in pass 2 either)
      static_cast<float4*>(A.stats)[to] =
          make_float4(any ? ref.d + __log2f(l) : 0.f, delta, any ? ref.b : INFINITY,
                      beside(ref.b, A.scale2));
    else
      static_cast<float2*>(A.stats)[to] = make_float2(lse2, delta);
  }
};

// ---- backward pass 2: source side --------------------------------------------

template <typename T, int kE_, bool kPair, Bias kBias>
struct RelSrc {
  static constexpr int kE = kE_;
  static constexpr int U = RelEdges<T, kE, kBias, kSrcEdges, kSrcEdgesF32, false>::value;
  static constexpr int kRow = kE * int(sizeof(T));
  static constexpr bool kBuckets = true;
  const RelArgs& A;
  const Lane<1>& L;
  const LanePlace<kRow> place;
  const LaneRows<kRow> r0, r1;  // the gathered rows
  const float* sb;    // the bias table
  float* hist;  // this lane's column of its warp's gradient table
  HeldT<T, kE> k, v;
  float dk[kE], dv[kE];

  __device__ __forceinline__ RelSrc(const RelArgs& a, const Lane<1>& lane)
      : A(a), L(lane), place(a.s, lane), r0(a.q, place), r1(a.dout, place) {}
  static __host__ __device__ int floats(const Shape& s) { return 2 * s.rv * kE; }

  __device__ __forceinline__ void clear() {
    zero<kE>(dk);
    zero<kE>(dv);
  }
  __device__ __forceinline__ void begin(int j) {
    k.fetch(place.of(A.key, j));
    v.fetch(place.of(A.val, j));
    clear();
  }
  template <class F>
  __device__ __forceinline__ void batch(const int (&i)[U], const int (&b)[U], int cnt,
                                        const F& sent) {
    RawT<T, kE> rq[U], rg[U];
    using Stats = std::conditional_t<kBias == Bias::kAny, float4, float2>;
    Stats st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rq[u] = ldT<T, kE>(r0.at(i[u]));
      rg[u] = ldT<T, kE>(r1.at(i[u]));
      // (no __ldg: pass 1 may still be writing when this kernel starts)
      st[u] = static_cast<const Stats*>(
          A.stats)[L.k[0] + uint64_t(uint32_t(i[u])) * uint32_t(A.s.H)];
    }
    float bs[U];
    int bk[U];
    bool ok[U];  // there, and not masked for the lane's head
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bk[u] = b[u];
      bs[u] = sb[bk[u] * A.s.H];
      ok[u] = u < cnt && bs[u] != -INFINITY;
    }
    sent();
    held_ready();
    float red[2 * U];
    {
      const RawT<T, kE> own = k.get();
#pragma unroll
      for (int u = 0; u < U; ++u) red[u] = dotT<kE>(own, rq[u]);
    }
    {
      const RawT<T, kE> own = v.get();
#pragma unroll
      for (int u = 0; u < U; ++u) red[U + u] = dotT<kE>(own, rg[u]);
    }
    head_sums<2 * U>(red, A.s.hv_log2);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ok[u]) continue;
      float t;
      if constexpr (kBias == Bias::kAny)
        t = fmaf(bs[u] - st[u].z, kLog2e, fmaf(red[u], st[u].w, -st[u].x));
      else
        t = fmaf(red[u], A.scale2, bs[u]) - st[u].x;
      const float al = ex2(t);
      const float de = al * (red[U + u] - st[u].y);
      add_grad<kPair>(hist, A.s, L.head_leader(A.s, 0), bk[u], de);
      float x[kE];
      widenT<T, kE>(rq[u], x);
      axpy<kE>(dk, de, x);
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
    scale<kE>(dk, A.scale);
    storeT<T, kE>(const_cast<char*>(place.of(A.dkey, j)), dk);
    storeT<T, kE>(const_cast<char*>(place.of(A.dval, j)), dv);
  }
};

// ---- kernels -----------------------------------------------------------------

constexpr int kPerSm = 2;  // resident blocks

template <typename T, int kE>
__global__ void __launch_bounds__(kThreads, kPerSm) rel_fwd(const __grid_constant__ RelArgs A) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  __shared__ __align__(16) unsigned char held[kWarps * HeldT<T, kE>::kBytes];
  float* table = reinterpret_cast<float*>(smem);
  const bool any = stage_bias(A.bias, A.buckets * A.s.H, table);
  const auto pass = [&](auto p) {
    p.q.place(held + (threadIdx.x >> 5) * HeldT<T, kE>::kBytes, L.lane);
    p.sb = table + L.k[0];
    walk(p, A.walk, A.dir, A.s, L);
  };
  if (any)
    pass(RelFwd<T, kE, Bias::kAny>(A, L));
  else
    pass(RelFwd<T, kE, Bias::kOrdinary>(A, L));
}

template <typename T, int kE>
__global__ void __launch_bounds__(kThreads, kPerSm) rel_dst(const __grid_constant__ RelArgs A) {
  let_next_start();
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  __shared__ __align__(16) unsigned char held[2 * kWarps * HeldT<T, kE>::kBytes];
  float* table = reinterpret_cast<float*>(smem);
  const bool any = stage_bias(A.bias, A.buckets * A.s.H, table);
  const auto pass = [&](auto p) {
    p.q.place(held + (threadIdx.x >> 5) * HeldT<T, kE>::kBytes, L.lane);
    p.g.place(held + (kWarps + (threadIdx.x >> 5)) * HeldT<T, kE>::kBytes, L.lane);
    p.sb = table + L.k[0];
    walk(p, A.walk, A.dir, A.s, L);
  };
  if (any)
    pass(RelDst<T, kE, Bias::kAny>(A, L));
  else
    pass(RelDst<T, kE, Bias::kOrdinary>(A, L));
}

template <typename T, int kE, bool kPair>
__global__ void __launch_bounds__(kThreads, kPerSm) rel_src(const __grid_constant__ RelArgs A) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<1> L(A.s);
  __shared__ __align__(16) unsigned char held[2 * kWarps * HeldT<T, kE>::kBytes];
  float* tables = reinterpret_cast<float*>(smem);
  float* column = clear_grad_tables(tables, A.s, L, A.buckets);
  float* table = reinterpret_cast<float*>(smem + grad_tables_bytes(A.s, A.buckets));
  const bool any = stage_bias(A.bias, A.buckets * A.s.H, table);
  const auto pass = [&](auto p) {
    p.k.place(held + (threadIdx.x >> 5) * HeldT<T, kE>::kBytes, L.lane);
    p.v.place(held + (kWarps + (threadIdx.x >> 5)) * HeldT<T, kE>::kBytes, L.lane);
    p.hist = column;
    p.sb = table + L.k[0];
    walk(p, A.walk, A.dir, A.s, L);
  };
  if (any)
    pass(RelSrc<T, kE, kPair, Bias::kAny>(A, L));
  else
    pass(RelSrc<T, kE, kPair, Bias::kOrdinary>(A, L));
  let_next_start();
  fold_grad_tables<kPair>(tables, A.s, L, A.buckets, A.db_part);
}

// dbias[x] = sum over the blocks of pass 2, one warp per entry.
__global__ void __launch_bounds__(kThreads) dbias_sum(const double* part, int blocks, int entries,
                                                      float* dbias) {
  const int x = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (x >= entries) return;
  grid_wait();
  double sum = 0.0;
  for (int b = threadIdx.x & 31; b < blocks; b += 32) sum += part[int64_t(b) * entries + x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if ((threadIdx.x & 31) == 0) dbias[x] = float(sum);
}

// ---- host side ---------------------------------------------------------------

// Elements of a lane vector: 32 bytes where a head has as many and the gathered
// rows start on 32-byte boundaries, else 16 bytes.  Loads of 32 bytes halve the
// requests to the L1 cache, three quarters busy with 16-byte ones: 529 instead of
// 567 us forward, 681 instead of 708 in pass 1 on the 300k-node graph.
int lane_elems(const Shape& s, bool aligned) {
  return aligned && s.D * s.esize >= 32 ? 32 / s.esize : 16 / s.esize;
}

struct RelLayout {
  size_t arrived, part, stats, db_part, total;
  WalkPlan plan;  // the same for both directions: n and e are
};

RelLayout rel_layout(const gnn_graph* g, const Shape& s, int buckets, bool aligned) {
  const size_t row = size_t(s.H) * s.D;
  RelLayout L{};
  L.plan = walk_plan(g->n, g->e, lane_shape(s, lane_elems(s, aligned)), kPerSm, g->sm_count);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t r = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  L.arrived = take(size_t(L.plan.workers) * 2 * sizeof(int));
  // at least every pass's state: two rows and four numbers per head in pass 1
  const size_t state = 2 * row + 4 * s.H;
  L.part = take(size_t(L.plan.workers) * 2 * state * 4);
  L.stats = take(size_t(g->n) * s.H * 16);
  L.db_part = take(size_t(L.plan.blocks) * buckets * s.H * 8);
  L.total = off;
  return L;
}

// after: launched behind the first pass of the same call (launch_after).
cudaError_t launch(void (*kernel)(RelArgs), const RelArgs& A, int blocks, size_t smem,
                   cudaStream_t st, bool after = false) {
  cudaError_t e;
  // (the default limit, 48 KB, counts the kernels' static 16 KB too)
  if ((e = allow_smem(kernel, smem, 32 * 1024)) != cudaSuccess) return e;
  if (after) return launch_after(kernel, dim3(unsigned(blocks)), kThreads, smem, st, A);
  kernel<<<unsigned(blocks), kThreads, smem, st>>>(A);
  return cudaGetLastError();
}

template <typename T, int kE>
cudaError_t fwd_t(const RelArgs& A, const WalkPlan& p, cudaStream_t st) {
  cudaError_t e;
  if (A.walk.cuts && (e = cudaMemsetAsync(A.walk.arrived, 0, size_t(p.workers) * sizeof(int),
                                            st)) != cudaSuccess)
    return e;
  return launch(rel_fwd<T, kE>, A, p.blocks, size_t(A.buckets) * A.s.H * 4, st);
}

template <typename T, int kE>
cudaError_t bwd_t(RelArgs A, const gnn_graph* g, const gnn_rel* rel, const WalkPlan& p,
                  float* dbias, cudaStream_t st) {
  const Walk src = make_walk(p, g->n, g->csc.max_deg, A.walk.arrived + p.workers, A.walk.part);
  cudaError_t e;
  // the counters of both passes
  if ((A.walk.cuts || src.cuts) &&
      (e = cudaMemsetAsync(A.walk.arrived, 0, size_t(p.workers) * 2 * sizeof(int), st)) !=
          cudaSuccess)
    return e;
  const size_t table = size_t(A.buckets) * A.s.H * 4;
  if ((e = launch(rel_dst<T, kE>, A, p.blocks, table, st)) != cudaSuccess) return e;
  A.dir = WalkDir{g->csc.ptr, g->csc.idx, rel->csc};
  A.walk = src;
  const auto src_pass =
      grad_pairs(A.s, A.buckets) ? rel_src<T, kE, true> : rel_src<T, kE, false>;
  if ((e = launch(src_pass, A, p.blocks, table + grad_tables_bytes(A.s, A.buckets), st, true)) !=
      cudaSuccess)
    return e;
  return launch_dbias_sum(A.db_part, p.blocks, A.buckets * A.s.H, dbias, st);
}

RelArgs rel_args(const gnn_graph* g, const gnn_rel* rel, const Shape& s, const void* q,
                 const void* key, const void* val, float scale, const float* bias,
                 const RelLayout& W, const WalkPlan& p, int elems, char* ws) {
  RelArgs A{};
  A.s = lane_shape(s, elems);
  A.walk = make_walk(p, g->n, g->csr.max_deg, reinterpret_cast<int*>(ws + W.arrived),
                     reinterpret_cast<float*>(ws + W.part));
  A.dir = WalkDir{g->csr.ptr, g->csr.idx, rel->csr};
  A.q = q;
  A.key = key;
  A.val = val;
  A.scale = scale;
  A.scale2 = scale * kLog2e;
  A.bias = bias;
  A.buckets = rel->buckets;
  A.stats = ws + W.stats;
  A.db_part = reinterpret_cast<double*>(ws + W.db_part);
  return A;
}

}  // namespace

cudaError_t launch_dbias_sum(const double* part, int blocks, int entries, float* dbias,
                             cudaStream_t st) {
  return launch_after(dbias_sum, dim3(unsigned((entries + kWarps - 1) / kWarps)), kThreads, 0, st,
                      part, blocks, entries, dbias);
}

size_t transformer_rel_ws_bytes(const gnn_graph* g, const Shape& s, int buckets) {
  const size_t a = rel_layout(g, s, buckets, true).total;
  const size_t b = rel_layout(g, s, buckets, false).total;
  return a > b ? a : b;
}

cudaError_t launch_transformer_rel_forward(const gnn_graph* g, const gnn_rel* rel, const Shape& s,
                                           gnn_dtype dt, const void* q, const void* key,
                                           const void* val, float scale, const float* bias,
                                           void* out, float* lse, char* ws, cudaStream_t st) {
  const bool aligned = aligned32(key) && aligned32(val);
  const int e = lane_elems(s, aligned);
  const RelLayout W = rel_layout(g, s, rel->buckets, aligned);
  RelArgs A = rel_args(g, rel, s, q, key, val, scale, bias, W, W.plan, e, ws);
  A.out = out;
  A.lse = lse;
  if (dt == GNN_F32)
    return e == 8 ? fwd_t<float, 8>(A, W.plan, st) : fwd_t<float, 4>(A, W.plan, st);
  return e == 16 ? fwd_t<__nv_bfloat16, 16>(A, W.plan, st) : fwd_t<__nv_bfloat16, 8>(A, W.plan, st);
}

cudaError_t launch_transformer_rel_backward(const gnn_graph* g, const gnn_rel* rel,
                                            const Shape& s, gnn_dtype dt, const void* q,
                                            const void* key, const void* val, float scale,
                                            const float* bias, const float* lse,
                                            const void* dout, void* dq, void* dkey, void* dval,
                                            float* dbias, char* ws, cudaStream_t st) {
  const bool aligned = aligned32(q) && aligned32(key) && aligned32(val) && aligned32(dout);
  const int e = lane_elems(s, aligned);
  const RelLayout W = rel_layout(g, s, rel->buckets, aligned);
  RelArgs A = rel_args(g, rel, s, q, key, val, scale, bias, W, W.plan, e, ws);
  A.lse_in = lse;
  A.dout = dout;
  A.dq = dq;
  A.dkey = dkey;
  A.dval = dval;
  if (dt == GNN_F32)
    return e == 8 ? bwd_t<float, 8>(A, g, rel, W.plan, dbias, st)
                  : bwd_t<float, 4>(A, g, rel, W.plan, dbias, st);
  return e == 16 ? bwd_t<__nv_bfloat16, 16>(A, g, rel, W.plan, dbias, st)
                 : bwd_t<__nv_bfloat16, 8>(A, g, rel, W.plan, dbias, st);
}

}  // namespace gnn
