// The walk of the transformer passes with a bias or from checkpoints over the
// edges of one direction, cut into equal pieces of work whatever the degrees.
//
// Every node costs kNodeCost units and every edge one; laid out node by node
// (edges first, then the node's own cost) that is a line of E + kNodeCost n units,
// and worker w takes units [w seg, (w + 1) seg) of it: a path through row
// pointers and edges cut at equal steps (Merrill and Garland, "Merge-based
// parallel sparse matrix-vector multiplication", SC 2016).  A worker is a
// sub-group of a warp, as wide as a feature row.  It finds its two ends by
// bisection, finishes the nodes that lie whole inside, and leaves partial states
// of the node that it begins in the middle (its head) and of the one that it
// leaves unfinished (its tail) in the workspace.  Whoever brings the last piece of
// a node (a counter per node, no waiting) adds its pieces in worker order and
// finishes it, so results do not depend on timing, and sums across nodes
// that a block keeps (the bias gradient) depend on the grid alone.
//
// Why: on the power-law graphs more than half of the edges belong to nodes that
// the degree buckets give to whole blocks, each with a staged edge list and three
// barriers around about a hundred edges a warp, and the reproducible bias
// gradient needs a fixed assignment, which those items balance badly.  300k
// nodes, 6M edges, H4 D64 bf16, degree buckets -> this walk: WALKTIMES.
#pragma once

#include "relbias.cuh"

namespace gnn {

constexpr int kNodeCost = 3;   // of a node, in edges: its own rows, its result
constexpr int kMinSeg = 16;    // units of a worker on small graphs
constexpr int kWaves = 1;      // segments per resident sub-group on large ones

struct WalkDir {
  const int32_t* ptr;
  const int32_t* idx;
  const uint8_t* buckets;  // of the edges in this direction, or null
};

struct Walk {
  int n;
  int64_t total, seg;      // units, and units of a worker
  int* arrived;            // [workers] pieces of the node whose first piece is the worker's
  float* part;             // [workers][head, tail][state floats]
};

// Nodes whose units all lie below d.
__device__ __forceinline__ int nodes_below(const int32_t* ptr, int n, int64_t d) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (int64_t(__ldg(ptr + mid + 1)) + int64_t(kNodeCost) * (mid + 1) <= d)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// Partial states pass between workers through L2.
__device__ __forceinline__ float part_load(const float* p) { return __ldcg(p); }

// P holds a node's own rows and its partial state:
//   begin(i)         loads the rows of node i and clears the state
//   clear()          clears the state
//   batch(j, b, cnt, f)  adds the edges to j[u] with buckets b[u], u < cnt (the
//                    others name some node, whose rows may be loaded but enter
//                    nowhere); calls f(), which overwrites j and b, once its
//                    gathers are on their way
//   finish(i)        writes node i's results from the state; the rows of begin(i)
//                    are still there unless the node has no edges
//   put(p), take(p)  stores the state, adds a stored one; P::floats(s) of them
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
    i = nodes_below(D.ptr, W.n, d0);
    i1 = nodes_below(D.ptr, W.n, d1);
    row_end = __ldg(D.ptr + i + 1);
    const int64_t at = d0 - int64_t(kNodeCost) * i;
    e = int(at < row_end ? at : row_end);
    const int end1 = __ldg(D.ptr + (i1 < W.n ? i1 + 1 : W.n));
    const int64_t at1 = d1 - int64_t(kNodeCost) * i1;
    e1 = int(at1 < end1 ? at1 : end1);
    cont = e > __ldg(D.ptr + i);
    ahead = __ldg(D.ptr + (i + 2 < W.n ? i + 2 : W.n));
  }
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
        for (int64_t w = first; w < last; ++w) p.take(W.part + (2 * w + 1) * nf);
        p.take(W.part + 2 * last * nf);
        p.finish(i);
      }
    }
  };

  int lim = i < i1 ? row_end : e1;  // edges of node i in this segment end here
  p.begin(i);  // (node 0 where there is no segment)
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
  const int64_t most = int64_t(kWaves) * per_sm * (sm_count > 0 ? sm_count : 1) * per_block;
  p.seg = (p.total + most - 1) / most;
  if (p.seg < kMinSeg) p.seg = kMinSeg;
  p.blocks = int((p.total + p.seg * per_block - 1) / (p.seg * per_block));
  p.workers = int64_t(p.blocks) * per_block;
  return p;
}

inline Walk make_walk(const WalkPlan& p, int64_t n, int* arrived, float* part) {
  Walk w{};
  w.n = int(n);
  w.total = p.total;
  w.seg = p.seg;
  w.arrived = arrived;
  w.part = part;
  return w;
}

}  // namespace gnn
