// The walk of the transformer passes with a bias or from checkpoints over the
// edges of one direction, cut into equal pieces of work whatever the degrees.
//
// Every node costs kNodeCost units and every edge one; laid out node by node
// (edges first, then the node's own cost) that is a line of E + kNodeCost n units,
// and worker w takes units [w seg, (w + 1) seg) of it: a path through row
// pointers and edges cut at equal steps (Merrill and Garland, "Merge-based
// parallel sparse matrix-vector multiplication", SC 2016).  A cut that falls into a
// node of at most `split` units moves to the node's end; only longer nodes are cut.
// A worker is a sub-group of a warp, as wide as a feature row.  It finds its two ends
// by bisection, finishes the nodes that lie whole inside, and leaves partial states
// of the long node that it begins in the middle (its head) and of the one that it
// leaves unfinished (its tail) in the workspace.  Whoever brings the last piece of
// a node (a counter per node, no waiting) adds its pieces in worker order and
// finishes it, so results do not depend on timing, and sums across nodes
// that a block keeps (the bias gradient) depend on the grid alone.  (Cutting every
// node costs two pieces a worker, each with a fence and a counter: 153 instead of
// 110 us for pass 1 of 100k nodes of 17 edges from checkpoints, 20 instead of 9 us
// for a forward pass over 512 nodes.)
//
// Why: on the power-law graphs more than half of the edges belong to nodes that
// the degree buckets give to whole blocks, each with a staged edge list and three
// barriers around about a hundred edges a warp, and the reproducible bias
// gradient needs a fixed assignment, which those items balance badly.  300k
// nodes, 6M edges, H4 D64 bf16: forward 0.85 ms by degree buckets, 0.52 by this walk
// (with 32-byte lane vectors), pass 1 1.02 and 0.67 ms, pass 2 1.97 and 0.85 ms.
//
// Bound: per SM 16 warps wait about 1,700 cycles a batch for gathered rows and issue for
// about half of the time; gathers alone would run at twice the rate (nodes of 300
// edges, everything in L2: 333 us forward, 458 pass 1, 572 pass 2).  What did not help:
// a ring of asynchronous copies to shared memory (no waits left, but a third more
// instructions: 982 to 1,106 us a kernel), prefetches to L2, more warps with fewer
// registers (spills), more and smaller segments (1.02 to 1.1 times the time).
#pragma once

#include "relbias.cuh"

namespace gnn {

constexpr int kNodeCost = 3;   // of a node, in edges: its own rows, its result
constexpr int kMinSeg = 32;    // units of a worker on small graphs

struct WalkDir {
  const int32_t* ptr;
  const int32_t* idx;
  const uint8_t* buckets;  // of the edges in this direction, or null
};

struct Walk {
  int n;
  int64_t total, seg;      // units, and units of a worker
  int split;               // units of the longest node that is not cut
  bool cuts;               // there are longer ones (else the counters are not used)
  int* arrived;            // [workers] pieces of the node whose first piece is the worker's
  float* part;             // [workers][head, tail][state floats]
};

// a, b = how many nodes start at or below units d0 and d1: two bisections side by
// side, three probes a step, so that n nodes take log4(n) dependent loads.
__device__ __forceinline__ void nodes_from(const int32_t* ptr, int n, int64_t d0, int64_t d1,
                                           int& a, int& b) {
  int lo[2] = {0, 0}, hi[2] = {n, n};
  const int64_t d[2] = {d0, d1};
  while (lo[0] < hi[0] || lo[1] < hi[1]) {
    bool in[2][3];
    int m[2][3];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        m[k][x] = lo[k] + int((int64_t(hi[k] - lo[k]) * (x + 1)) >> 2);
        const int at = m[k][x] < n ? m[k][x] : n - 1;
        in[k][x] = int64_t(__ldg(ptr + at)) + int64_t(kNodeCost) * at <= d[k];
      }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (lo[k] < hi[k]) {
        if (!in[k][0]) {
          hi[k] = m[k][0];
        } else if (!in[k][1]) {
          lo[k] = m[k][0] + 1;
          hi[k] = m[k][1];
        } else if (!in[k][2]) {
          lo[k] = m[k][1] + 1;
          hi[k] = m[k][2];
        } else {
          lo[k] = m[k][2] + 1;
        }
      }
  }
  a = lo[0];
  b = lo[1];
}

// Partial states pass between workers through L2.
__device__ __forceinline__ float part_load(const float* p) { return __ldcg(p); }
template <int kE>
__device__ __forceinline__ void part_row(const float* p, float (&x)[kE]) {
#pragma unroll
  for (int c = 0; c < kE; ++c) x[c] = __ldcg(p + c);
}
template <int kE>
__device__ __forceinline__ void add_row(float (&a)[kE], const float (&x)[kE]) {
#pragma unroll
  for (int c = 0; c < kE; c += 2) add2(a[c], a[c + 1], a[c], a[c + 1], x[c], x[c + 1]);
}
// a += the N rows at p, p + step, ... in that order.
template <int kE, int N>
__device__ __forceinline__ void take_rows(float (&a)[kE], const float* p, int step) {
  float x[N][kE];
#pragma unroll
  for (int n = 0; n < N; ++n) part_row<kE>(p + n * step, x[n]);
#pragma unroll
  for (int n = 0; n < N; ++n) add_row<kE>(a, x[n]);
}

// Called by every thread of a block that has written its tables to shared memory
// (the walk begins with the barrier that ends those writes).  P holds a node's own
// rows and its partial state:
//   begin(i)         loads the rows of node i and clears the state
//   clear()          clears the state
//   batch(j, b, cnt, f)  adds the edges to j[u] with buckets b[u], u < cnt (the
//                    others name some node, whose rows may be loaded but enter
//                    nowhere); calls f(), which overwrites j and b, once its
//                    gathers are on their way
//   finish(i)        writes node i's results from the state; the rows of begin(i)
//                    are still there unless the node has no edges
//   put(p)           stores the state, P::floats(s) numbers
//   take<N>(p, d)    adds the N stored states at p, p + d, ... in that order
template <class P>
__device__ __forceinline__ void walk(P& p, const Walk& W, const WalkDir& D, const Shape& s,
                                     const Lane<1>& L) {
  constexpr int U = P::U;
  const int64_t worker = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * L.G + L.g;
  const int64_t d0 = worker * W.seg < W.total ? worker * W.seg : W.total;
  const int64_t d1 = d0 + W.seg < W.total ? d0 + W.seg : W.total;
  bool live = d0 < d1;
  const unsigned mine = (s.lpr == 32 ? kFull : ((1u << s.lpr) - 1u)) << (L.g << s.lpr_log2);
  int i = 0, e = 0, i1 = 0, e1 = 0, row_end = 0, ahead = 0;
  bool cont = false;  // node i has edges before this segment
  if (live) {
    int c0, c1;
    nodes_from(D.ptr, W.n, d0, d1, c0, c1);
    // the cut at unit d of the line, node k being the last that starts there or
    // before: (node, edge) from which the work goes on
    const auto cut = [&](int64_t d, int k, int& node, int& edge) {
      const int from = __ldg(D.ptr + k), to = __ldg(D.ptr + k + 1);
      const int64_t in = d - (int64_t(from) + int64_t(kNodeCost) * k);  // units into the node
      if (to - from > W.split - kNodeCost) {
        node = k;
        edge = in < to - from ? from + int(in) : to;
      } else {
        node = in > 0 ? k + 1 : k;
        edge = in > 0 ? to : from;
      }
    };
    cut(d0, c0 - 1, i, e);
    if (d1 < W.total) {
      cut(d1, c1 - 1, i1, e1);
    } else {
      i1 = W.n;
      e1 = __ldg(D.ptr + W.n);
    }
    live = i < i1 || e < e1;
    cont = live && i < W.n && e > __ldg(D.ptr + i);
  }
  if (live) {
    row_end = __ldg(D.ptr + i + 1);
    ahead = __ldg(D.ptr + (i + 2 < W.n ? i + 2 : W.n));
  }
  __syncthreads();  // the block's tables are staged
  grid_wait();      // and the pass before, whose results batch() may read, is complete
  const int nf = P::floats(s);

  // Hands over a piece of node i; the last to arrive finishes the node.
  const auto piece = [&](int side) {
    const int64_t first = (int64_t(__ldg(D.ptr + i)) + int64_t(kNodeCost) * i) / W.seg;
    const int64_t last = (int64_t(__ldg(D.ptr + i + 1)) + int64_t(kNodeCost) * (i + 1) - 1) / W.seg;
    if (L.ok[0]) p.put(W.part + (2 * worker + side) * nf);
    __threadfence();
    __syncwarp(mine);
    int before = 0;
    if (L.p == 0) before = atomicAdd(W.arrived + first, 1);
    before = __shfl_sync(mine, before, L.g << s.lpr_log2);
    if (before == int(last - first)) {
      __threadfence();
      p.clear();
      if (L.ok[0]) {
        // tails first .. last - 1, then the head of the last: four loads at a time
        const float* from = W.part + (2 * first + 1) * nf;
        int more = int(last - first);
        for (; more >= 4; more -= 4, from += 8 * nf) p.template take<4>(from, 2 * nf);
        for (; more > 0; --more, from += 2 * nf) p.template take<1>(from, 0);
        p.template take<1>(W.part + 2 * last * nf, 0);
        p.finish(i);
      }
    }
  };

  int lim = i < i1 ? row_end : e1;  // edges of node i in this segment end here
  p.begin(live ? i : 0);  // without a segment i may be past the last node
  // Node ids (and buckets) of the next batch: the segment's next U edges, also
  // where they belong to the next node.
  int jn[U], bn[U];
  const int32_t* ip = D.idx + e;
  const uint8_t* bp = P::kBuckets ? D.buckets + e : nullptr;
  int left = live ? e1 - e : 0;
  const auto ids = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      jn[u] = u < left ? __ldg(ip + u) : 0;
      if (P::kBuckets) bn[u] = u < left ? int(__ldg(bp + u)) : 0;
    }
  };
  ids();
  while (__any_sync(kFull, live)) {
    const int rest = lim - e;
    const int cnt = live ? (rest < U ? rest : U) : 0;
    e += cnt;
    ip += cnt;
    if (P::kBuckets) bp += cnt;
    left -= cnt;
    p.batch(jn, bn, cnt, ids);
    if (live && e == lim) {
      for (;;) {
        if (i == i1) {  // the segment ends inside node i
          piece(1);
          live = false;
          break;
        }
        if (cont)
          piece(0);
        else if (L.ok[0])
          p.finish(i);
        cont = false;
        ++i;
        if (i == i1 && e == e1) {  // ... or between two nodes
          live = false;
          break;
        }
        row_end = ahead;
        ahead = __ldg(D.ptr + (i + 2 < W.n ? i + 2 : W.n));
        lim = i < i1 ? row_end : e1;
        if (lim > e) {
          p.begin(i);
          break;
        }
        p.clear();  // a node without edges: straight to its result
      }
    }
  }
}

// ---- host side ---------------------------------------------------------------

struct WalkPlan {
  int64_t total, seg;
  int64_t workers;
  int blocks;
};

// The grid of a walk over n nodes and e edges for a kernel of which `per_sm`
// blocks are resident, and rows of `s`.
inline WalkPlan walk_plan(int64_t n, int64_t e, const Shape& s, int per_sm, int sm_count) {
  WalkPlan p{};
  p.total = e + int64_t(kNodeCost) * n;
  const int64_t per_block = int64_t(kWarps) * (32 >> s.lpr_log2);
  const int64_t most = int64_t(per_sm) * (sm_count > 0 ? sm_count : 1) * per_block;
  p.seg = (p.total + most - 1) / most;
  if (p.seg < kMinSeg) p.seg = kMinSeg;
  p.blocks = int((p.total + p.seg * per_block - 1) / (p.seg * per_block));
  p.workers = int64_t(p.blocks) * per_block;
  return p;
}

// max_deg: of the direction walked.
inline Walk make_walk(const WalkPlan& p, int64_t n, int max_deg, int* arrived, float* part) {
  Walk w{};
  // at most a sixteenth of a segment more or less; on small graphs, where the
  // latency of a few nodes is all there is, two segments
  w.split = int(p.seg / 16 > 2 * kMinSeg ? (p.seg / 16 < (1 << 30) ? p.seg / 16 : (1 << 30))
                                        : 2 * kMinSeg);
  w.cuts = max_deg > w.split - kNodeCost;
  w.n = int(n);
  w.total = p.total;
  w.seg = p.seg;
  w.arrived = arrived;
  w.part = part;
  return w;
}

}  // namespace gnn
