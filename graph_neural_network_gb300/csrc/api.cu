// C-ABI entry points: argument checks, workspace layout, dispatch.
#include <new>

#include "internal.h"

namespace gnn {

bool make_shape(int H, int D, gnn_dtype dt, Shape* s) {
  if (H < 1 || D < 1 || H > 4096 || D > 4096) return false;
  if (dt != GNN_F32 && dt != GNN_BF16) return false;
  s->H = H;
  s->D = D;
  s->esize = dt == GNN_F32 ? 4 : 2;
  const int head_bytes = D * s->esize;
  if (head_bytes % 16) return false;
  s->hv = head_bytes / 16;
  if (s->hv > 32 || (s->hv & (s->hv - 1))) return false;
  const int64_t rv = int64_t(H) * s->hv;
  if (rv * 16 > 2048) return false;
  s->rv = int(rv);
  if (s->rv <= 32) {
    s->lpr = 1;
    while (s->lpr < s->rv) s->lpr <<= 1;
    s->nv = 1;
  } else {
    s->lpr = 32;
    s->nv = (s->rv + 31) / 32;
    if (s->nv == 3) s->nv = 4;
  }
  s->hv_log2 = 0;
  while ((1 << s->hv_log2) < s->hv) ++s->hv_log2;
  s->lpr_log2 = 0;
  while ((1 << s->lpr_log2) < s->lpr) ++s->lpr_log2;
  return true;
}

bool make_wide_shape(const Shape& s, Shape* w) {
  if (s.hv < 2 || s.rv > 64) return false;
  *w = s;
  w->rv = s.rv / 2;
  w->hv = s.hv / 2;
  w->lpr = 1;
  while (w->lpr < w->rv) w->lpr <<= 1;
  w->nv = 1;
  w->hv_log2 = s.hv_log2 - 1;
  w->lpr_log2 = 0;
  while ((1 << w->lpr_log2) < w->lpr) ++w->lpr_log2;
  return true;
}

WsLayout ws_layout(const gnn_graph* g, const Shape& s) {
  WsLayout L;
  const size_t HD = size_t(s.H) * s.D;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t r = off;
    off += align_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  // forward: work counters, hub chunk partials of the CSR direction
  L.fwd_ctr = take(kCounters * 4);
  L.fwd_scores = take(size_t(g->n) * s.H * 8);  // s_src [N][H] then s_dst [N][H]
  L.fwd_acc = take(size_t(g->csr.n_hub_chunks) * HD * 4);
  L.fwd_ml = take(size_t(g->csr.n_hub_chunks) * s.H * 8);
  L.fwd_total = off;
  // backward
  off = 0;
  L.bwd_ctr = take(kCounters * 4);
  L.bwd_scores = take(size_t(g->n) * s.H * 8);
  L.stats = take(size_t(g->n) * s.H * 16);
  L.ds_src = take(size_t(g->n) * s.H * 4);
  L.dst_part = take(size_t(g->csr.n_hub_chunks) * s.H * 16);
  L.src_acc = take(size_t(g->csc.n_hub_chunks) * HD * 4);
  L.src_sum = take(size_t(g->csc.n_hub_chunks) * s.H * 4);
  // attention-vector partial sums: up to 8 blocks per SM, each warp summing
  // at least 16 nodes before its block's float64 fold
  const int64_t cap = int64_t(g->sm_count > 0 ? g->sm_count : 1) * 8;
  int64_t blocks = (g->n + 127) / 128;
  if (blocks < 1) blocks = 1;
  if (blocks > cap) blocks = cap;
  L.da_blocks = int(blocks);
  L.da_part = take(size_t(blocks) * 2 * HD * 8);
  L.bwd_total = off;
  return L;
}

}  // namespace gnn

using gnn::Shape;
using gnn::WsLayout;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool tiling_ok(const gnn_tiling& t) {
  return t.light_max_deg >= GNN_LIGHT_AUTO && t.cta_max_deg >= 0 &&
         t.cta_max_deg >= t.light_max_deg && t.cta_max_deg <= 16384 && t.hub_chunk >= 1 &&
         t.hub_chunk <= 16384;
}

// The tiling that bounds the prepared graph's buffers: an automatic light
// threshold is never below its floor (or cta_max_deg), and fewer light nodes
// only mean more block items, which the bound covers.
gnn_tiling bound_tiling(gnn_tiling t) {
  if (t.light_max_deg == GNN_LIGHT_AUTO)
    t.light_max_deg = t.cta_max_deg < gnn::kLightAutoMin ? t.cta_max_deg : gnn::kLightAutoMin;
  return t;
}

gnn_tiling resolve_tiling(const gnn_tiling* t) {
  gnn_tiling r;
  gnn_default_tiling(&r);
  if (t) r = *t;
  return r;
}

bool sizes_ok(int64_t n, int64_t e) {
  return n >= 0 && e >= 0 && n < (int64_t(1) << 31) - 1 && e < (int64_t(1) << 31) - 1;
}

gnn_status check_call(const gnn_graph* g, int H, int D, gnn_dtype dt, Shape* s) {
  if (!g) return GNN_ERR_INVALID_ARG;
  if (dt != GNN_F32 && dt != GNN_BF16) return GNN_ERR_INVALID_ARG;
  if (H < 1 || D < 1) return GNN_ERR_INVALID_ARG;
  if (!gnn::make_shape(H, D, dt, s)) return GNN_ERR_UNSUPPORTED;
  return GNN_OK;
}

// The status of a call's launches.  A refused one (cudaLaunchKernelEx, an attribute) also
// stays as the thread's last error, which the next call's cudaGetLastError would take for
// its own: it is taken here.
gnn_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return GNN_OK;
  (void)cudaGetLastError();
  return GNN_ERR_CUDA;
}

}  // namespace

extern "C" {

void gnn_default_tiling(gnn_tiling* t) {
  if (!t) return;
  t->light_max_deg = GNN_LIGHT_AUTO;
  t->cta_max_deg = 4096;
  t->hub_chunk = 2048;
}

int gnn_abi_version(void) { return GNNAGG_ABI_VERSION; }

const char* gnn_status_string(gnn_status s) {
  switch (s) {
    case GNN_OK: return "ok";
    case GNN_ERR_INVALID_ARG: return "invalid argument";
    case GNN_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case GNN_ERR_INVALID_GRAPH: return "invalid CSR graph";
    case GNN_ERR_WORKSPACE_TOO_SMALL: return "buffer or workspace too small";
    case GNN_ERR_CUDA: return "CUDA error";
    case GNN_ERR_DEVICE_ASSERT: return "device-side consistency check failed";
    case GNN_ERR_TIMEOUT: return "a bounded device wait timed out";
  }
  return "unknown status";
}

size_t gnn_graph_buffer_bytes(int64_t n_nodes, int64_t n_edges, const gnn_tiling* tiling) {
  const gnn_tiling t = resolve_tiling(tiling);
  if (!sizes_ok(n_nodes, n_edges) || !tiling_ok(t)) return 0;
  return gnn::graph_buffer_bytes(n_nodes, n_edges, bound_tiling(t));
}

size_t gnn_graph_scratch_bytes(int64_t n_nodes, int64_t n_edges) {
  if (!sizes_ok(n_nodes, n_edges)) return 0;
  return gnn::graph_scratch_bytes(n_nodes, n_edges);
}

gnn_status gnn_graph_prepare(int64_t n_nodes, int64_t n_edges, const int32_t* row_ptr_d,
                             const int32_t* col_idx_d, void* buffer_d, size_t buffer_bytes,
                             void* scratch_d, size_t scratch_bytes, const gnn_tiling* tiling,
                             void* stream, gnn_graph** out) {
  if (!out) return GNN_ERR_INVALID_ARG;
  *out = nullptr;
  const gnn_tiling t = resolve_tiling(tiling);
  if (!sizes_ok(n_nodes, n_edges) || !tiling_ok(t)) return GNN_ERR_INVALID_ARG;
  if (!row_ptr_d || !buffer_d || !scratch_d || (n_edges > 0 && !col_idx_d))
    return GNN_ERR_INVALID_ARG;
  if (!aligned(row_ptr_d, 4) || !aligned(col_idx_d, 16) || !aligned(buffer_d, 256) ||
      !aligned(scratch_d, 256))
    return GNN_ERR_INVALID_ARG;
  if (buffer_bytes < gnn::graph_buffer_bytes(n_nodes, n_edges, bound_tiling(t)) ||
      scratch_bytes < gnn::graph_scratch_bytes(n_nodes, n_edges))
    return GNN_ERR_WORKSPACE_TOO_SMALL;
  gnn_graph* g = new (std::nothrow) gnn_graph;
  if (!g) return GNN_ERR_INVALID_ARG;
  g->n = n_nodes;
  g->e = n_edges;
  g->tiling = t;
  if (cudaGetDevice(&g->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&g->sm_count, cudaDevAttrMultiProcessorCount, g->device) !=
          cudaSuccess) {
    delete g;
    return GNN_ERR_CUDA;
  }
  if (t.light_max_deg == GNN_LIGHT_AUTO)
    g->tiling.light_max_deg = gnn::auto_light_max(n_edges, g->sm_count, t.cta_max_deg);
  const gnn_status s =
      gnn::prepare_graph(g, row_ptr_d, col_idx_d, static_cast<char*>(buffer_d), buffer_bytes,
                         static_cast<char*>(scratch_d), scratch_bytes,
                         static_cast<cudaStream_t>(stream));
  if (s != GNN_OK) {
    delete g;
    return s;
  }
  *out = g;
  return GNN_OK;
}

gnn_status gnn_graph_destroy(gnn_graph* g) {
  delete g;
  return GNN_OK;
}

gnn_status gnn_graph_stats(const gnn_graph* g, int64_t* st, int n) {
  if (!g || !st || n < 16) return GNN_ERR_INVALID_ARG;
  st[0] = g->n;
  st[1] = g->e;
  const gnn::Dir* d[2] = {&g->csr, &g->csc};
  for (int k = 0; k < 2; ++k) {
    int64_t* o = st + 2 + 6 * k;
    o[0] = d[k]->n_light;
    o[1] = d[k]->n_items;
    o[2] = d[k]->n_hubs;
    o[3] = d[k]->n_hub_chunks;
    o[4] = d[k]->max_deg;
    o[5] = d[k]->max_item;
  }
  st[14] = g->tiling.light_max_deg;
  st[15] = g->tiling.cta_max_deg;
  for (int k = 16; k < n; ++k) st[k] = 0;
  return GNN_OK;
}

gnn_status gnn_graph_arrays(const gnn_graph* g, const void** p, int n) {
  if (!g || !p || n < 8) return GNN_ERR_INVALID_ARG;
  p[0] = g->csc.ptr;
  p[1] = g->csc.idx;
  p[2] = g->csr.light;
  p[3] = g->csr.items;
  p[4] = g->csr.hubs;
  p[5] = g->csc.light;
  p[6] = g->csc.items;
  p[7] = g->csc.hubs;
  for (int k = 8; k < n; ++k) p[k] = nullptr;
  return GNN_OK;
}

size_t gat_agg_workspace_bytes(const gnn_graph* g, int H, int D, gnn_dtype dtype) {
  Shape s;
  if (check_call(g, H, D, dtype, &s) != GNN_OK) return 0;
  const WsLayout L = gnn::ws_layout(g, s);
  return L.fwd_total > L.bwd_total ? L.fwd_total : L.bwd_total;
}

gnn_status gat_agg_forward_timed(const gnn_graph* g, int H, int D, gnn_dtype dtype, const void* h,
                                 const float* a_src, const float* a_dst, float slope, void* out,
                                 float* lse, void* ws, size_t ws_bytes, void* stream,
                                 void* const* events, int n_events) {
  if (events && n_events < 4) return GNN_ERR_INVALID_ARG;
  Shape s;
  gnn_status r = check_call(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!h || !a_src || !a_dst || !out || !lse) return GNN_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(out, 16) || !aligned(a_src, 16) || !aligned(a_dst, 16) ||
      !aligned(lse, 4))
    return GNN_ERR_INVALID_ARG;
  const WsLayout L = gnn::ws_layout(g, s);
  if (ws_bytes < L.fwd_total) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_forward(g, s, dtype, h, a_src, a_dst, slope, out, lse,
                                       static_cast<char*>(ws), L,
                                       static_cast<cudaStream_t>(stream),
                                       reinterpret_cast<const cudaEvent_t*>(events)));
}

gnn_status gat_agg_forward(const gnn_graph* g, int H, int D, gnn_dtype dtype, const void* h,
                           const float* a_src, const float* a_dst, float slope, void* out,
                           float* lse, void* ws, size_t ws_bytes, void* stream) {
  return gat_agg_forward_timed(g, H, D, dtype, h, a_src, a_dst, slope, out, lse, ws, ws_bytes,
                               stream, nullptr, 0);
}

}  // extern "C"

namespace {

gnn_status backward_call(const gnn_graph* g, int H, int D, gnn_dtype dtype, const void* h,
                         const float* a_src, const float* a_dst, float slope, const float* lse,
                         const void* dout, void* dh, float* da_src, float* da_dst, void* ws,
                         size_t ws_bytes, void* stream, void* const* events, int n_events,
                         bool reuse_scores) {
  if (events && n_events < 8) return GNN_ERR_INVALID_ARG;
  Shape s;
  gnn_status r = check_call(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (!a_src || !a_dst || !da_src || !da_dst) return GNN_ERR_INVALID_ARG;
  if (!aligned(a_src, 16) || !aligned(a_dst, 16) || !aligned(da_src, 4) || !aligned(da_dst, 4))
    return GNN_ERR_INVALID_ARG;
  if (g->n > 0) {
    if (!h || !lse || !dout || !dh) return GNN_ERR_INVALID_ARG;
    if (!aligned(h, 16) || !aligned(dout, 16) || !aligned(dh, 16) || !aligned(lse, 4))
      return GNN_ERR_INVALID_ARG;
  }
  const WsLayout L = gnn::ws_layout(g, s);
  if (ws_bytes < L.bwd_total) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  // both calls keep the per-node scores at the same offset of ws
  if (reuse_scores && L.fwd_scores != L.bwd_scores) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_backward(g, s, dtype, h, a_src, a_dst, slope, lse, dout, dh,
                                        da_src, da_dst, static_cast<char*>(ws), L,
                                        static_cast<cudaStream_t>(stream),
                                        reinterpret_cast<const cudaEvent_t*>(events),
                                        reuse_scores));
}

}  // namespace

extern "C" {

gnn_status gat_agg_backward_timed(const gnn_graph* g, int H, int D, gnn_dtype dtype,
                                  const void* h, const float* a_src, const float* a_dst,
                                  float slope, const float* lse, const void* dout, void* dh,
                                  float* da_src, float* da_dst, void* ws, size_t ws_bytes,
                                  void* stream, void* const* events, int n_events) {
  return backward_call(g, H, D, dtype, h, a_src, a_dst, slope, lse, dout, dh, da_src, da_dst,
                       ws, ws_bytes, stream, events, n_events, false);
}

gnn_status gat_agg_backward_reuse(const gnn_graph* g, int H, int D, gnn_dtype dtype,
                                  const void* h, const float* a_src, const float* a_dst,
                                  float slope, const float* lse, const void* dout, void* dh,
                                  float* da_src, float* da_dst, void* ws, size_t ws_bytes,
                                  void* stream, void* const* events, int n_events) {
  return backward_call(g, H, D, dtype, h, a_src, a_dst, slope, lse, dout, dh, da_src, da_dst,
                       ws, ws_bytes, stream, events, n_events, true);
}

gnn_status gat_agg_backward(const gnn_graph* g, int H, int D, gnn_dtype dtype, const void* h,
                            const float* a_src, const float* a_dst, float slope,
                            const float* lse, const void* dout, void* dh, float* da_src,
                            float* da_dst, void* ws, size_t ws_bytes, void* stream) {
  return gat_agg_backward_timed(g, H, D, dtype, h, a_src, a_dst, slope, lse, dout, dh, da_src,
                                da_dst, ws, ws_bytes, stream, nullptr, 0);
}

}  // extern "C"

// ---- SpMM-family propagation ---------------------------------------------

namespace {

// A row of F elements as F * size / 16 one-vector "heads".
gnn_status spmm_shape(const gnn_graph* g, int F, gnn_dtype dt, Shape* s) {
  if (!g || F < 1 || (dt != GNN_F32 && dt != GNN_BF16)) return GNN_ERR_INVALID_ARG;
  const int64_t bytes = int64_t(F) * (dt == GNN_F32 ? 4 : 2);
  if (bytes % 16 || bytes > 2048) return GNN_ERR_UNSUPPORTED;
  return gnn::make_shape(int(bytes / 16), dt == GNN_F32 ? 4 : 8, dt, s) ? GNN_OK
                                                                         : GNN_ERR_UNSUPPORTED;
}

gnn_status spmm_call(const gnn_graph* g, int F, gnn_dtype dt, gnn_norm norm, const void* x,
                     void* out, void* ws, size_t ws_bytes, void* stream, bool transpose) {
  Shape s;
  gnn_status r = spmm_shape(g, F, dt, &s);
  if (r != GNN_OK) return r;
  if (norm != GNN_NORM_SUM && norm != GNN_NORM_MEAN && norm != GNN_NORM_SYM)
    return GNN_ERR_INVALID_ARG;
  if (g->n == 0) return GNN_OK;
  if (!x || !out || !aligned(x, 16) || !aligned(out, 16)) return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::spmm_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_spmm(g, s, dt, int(norm), transpose, x, out,
                                    static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t gcn_agg_workspace_bytes(const gnn_graph* g, int F, gnn_dtype dtype) {
  Shape s;
  if (spmm_shape(g, F, dtype, &s) != GNN_OK) return 0;
  return gnn::spmm_ws_bytes(g, s);
}

gnn_status gcn_agg_forward(const gnn_graph* g, int F, gnn_dtype dtype, gnn_norm norm,
                           const void* x, void* out, void* ws, size_t ws_bytes, void* stream) {
  return spmm_call(g, F, dtype, norm, x, out, ws, ws_bytes, stream, false);
}

gnn_status gcn_agg_backward(const gnn_graph* g, int F, gnn_dtype dtype, gnn_norm norm,
                            const void* dout, void* dx, void* ws, size_t ws_bytes,
                            void* stream) {
  return spmm_call(g, F, dtype, norm, dout, dx, ws, ws_bytes, stream, true);
}

}  // extern "C"

namespace {

gnn_status gatv2_shape(const gnn_graph* g, int H, int D, gnn_dtype dt, Shape* s) {
  gnn_status r = check_call(g, H, D, dt, s);
  if (r != GNN_OK) return r;
  return s->nv == 1 ? GNN_OK : GNN_ERR_UNSUPPORTED;
}

// The current device is the graph's (a launch on another device's stream, or on
// memory of another device, would fail after the call has returned).
bool device_ok(const gnn_graph* g) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == g->device;
}

bool current_sms(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

gnn_status pack8_shape(int64_t n, int H, int D, gnn_dtype dt, Shape* s) {
  if (n < 0 || n >= (int64_t(1) << 31) || (dt != GNN_F32 && dt != GNN_BF16) || H < 1 || D < 1)
    return GNN_ERR_INVALID_ARG;
  return gnn::make_shape(H, D, dt, s) ? GNN_OK : GNN_ERR_UNSUPPORTED;
}

bool packed_ok(const gnn_packed8* p) {
  return p && p->values && p->scale && aligned(p->values, 16) && aligned(p->scale, 4);
}

gnn_status norm_residual_check(const gnn_norm_residual* d, gnn_dtype dt) {
  if (!d || (dt != GNN_F32 && dt != GNN_BF16) || d->n < 0 || d->n >= (int64_t(1) << 31) ||
      d->F < 1)
    return GNN_ERR_INVALID_ARG;
  const auto known = [](gnn_rownorm k) {
    return k == GNN_ROWNORM_NONE || k == GNN_ROWNORM_RMS || k == GNN_ROWNORM_LAYER;
  };
  const gnn_norm_params& p = d->params;
  if (!known(d->post) || !known(d->pre) || !(d->eps > 0.f) || d->eps > 3.0e38f ||
      (d->gate_width != 0 && d->gate_width != 1 && d->gate_width != d->F))
    return GNN_ERR_INVALID_ARG;
  if ((d->post == GNN_ROWNORM_NONE && (p.w_post || p.b_post)) ||
      (d->pre == GNN_ROWNORM_NONE && (p.w_pre || p.b_pre)))
    return GNN_ERR_INVALID_ARG;
  if (!aligned(p.w_post, 4) || !aligned(p.b_post, 4) || !aligned(p.scale, 4) ||
      !aligned(p.w_pre, 4) || !aligned(p.b_pre, 4))
    return GNN_ERR_INVALID_ARG;
  const int64_t bytes = int64_t(d->F) * (dt == GNN_F32 ? 4 : 2);
  return bytes % 16 || bytes > 2048 ? GNN_ERR_UNSUPPORTED : GNN_OK;
}

// A gate or its gradient: null exactly where there is no gate, aligned.
bool gate_ok(const gnn_norm_residual* d, gnn_dtype dt, const void* gate) {
  if (d->gate_width == 0) return !gate;
  return gate && aligned(gate, d->gate_width == 1 ? (dt == GNN_F32 ? 4 : 2) : 16);
}

gnn_status rel_shape(const gnn_graph* g, const gnn_rel* rel, int H, int D, gnn_dtype dt,
                     Shape* s) {
  if (!g || !rel || rel->g != g || rel->n != g->n || rel->e != g->e) return GNN_ERR_INVALID_ARG;
  return gatv2_shape(g, H, D, dt, s);
}

}  // namespace

extern "C" {

size_t gatv2_agg_workspace_bytes(const gnn_graph* g, int H, int D, gnn_dtype dtype) {
  Shape s;
  if (gatv2_shape(g, H, D, dtype, &s) != GNN_OK) return 0;
  return gnn::gatv2_ws_bytes(g, s);
}

gnn_status gatv2_agg_forward(const gnn_graph* g, int H, int D, gnn_dtype dtype, const void* xl,
                             const void* xr, const float* att, float slope, void* out,
                             float* lse, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  gnn_status r = gatv2_shape(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!xl || !xr || !att || !out || !lse) return GNN_ERR_INVALID_ARG;
  if (!aligned(xl, 16) || !aligned(xr, 16) || !aligned(att, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::gatv2_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_gatv2_forward(g, s, dtype, xl, xr, att, slope, out, lse,
                                             static_cast<char*>(ws),
                                             static_cast<cudaStream_t>(stream)));
}

gnn_status gatv2_agg_backward(const gnn_graph* g, int H, int D, gnn_dtype dtype,
                              const void* xl, const void* xr, const float* att, float slope,
                              const float* lse, const void* dout, void* dxl, void* dxr,
                              float* datt, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  gnn_status r = gatv2_shape(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (!att || !datt || !aligned(att, 16) || !aligned(datt, 4)) return GNN_ERR_INVALID_ARG;
  if (g->n > 0) {
    if (!xl || !xr || !lse || !dout || !dxl || !dxr) return GNN_ERR_INVALID_ARG;
    if (!aligned(xl, 16) || !aligned(xr, 16) || !aligned(dout, 16) || !aligned(dxl, 16) ||
        !aligned(dxr, 16) || !aligned(lse, 4))
      return GNN_ERR_INVALID_ARG;
  }
  if (ws_bytes < gnn::gatv2_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_gatv2_backward(g, s, dtype, xl, xr, att, slope, lse, dout, dxl,
                                              dxr, datt, static_cast<char*>(ws),
                                              static_cast<cudaStream_t>(stream)));
}

size_t transformer_agg_workspace_bytes(const gnn_graph* g, int H, int D, gnn_dtype dtype) {
  Shape s;
  if (gatv2_shape(g, H, D, dtype, &s) != GNN_OK) return 0;
  return gnn::transformer_ws_bytes(g, s);
}

gnn_status transformer_agg_forward(const gnn_graph* g, int H, int D, gnn_dtype dtype,
                                   const void* q, const void* key, const void* val, float scale,
                                   void* out, float* lse, void* ws, size_t ws_bytes,
                                   void* stream) {
  Shape s;
  gnn_status r = gatv2_shape(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!q || !key || !val || !out || !lse) return GNN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(val, 16) || !aligned(out, 16) ||
      !aligned(lse, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::transformer_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_transformer_forward(g, s, dtype, q, key, val, scale, out, lse,
                                                   static_cast<char*>(ws),
                                                   static_cast<cudaStream_t>(stream)));
}

gnn_status transformer_agg_backward(const gnn_graph* g, int H, int D, gnn_dtype dtype,
                                    const void* q, const void* key, const void* val, float scale,
                                    const float* lse, const void* dout, void* dq, void* dkey,
                                    void* dval, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  gnn_status r = gatv2_shape(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!q || !key || !val || !lse || !dout || !dq || !dkey || !dval) return GNN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(val, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dkey, 16) || !aligned(dval, 16) || !aligned(lse, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::transformer_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_transformer_backward(g, s, dtype, q, key, val, scale, lse, dout,
                                                    dq, dkey, dval, static_cast<char*>(ws),
                                                    static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_rel_log_bounds(int n_bounds, int max_distance, int32_t* bounds) {
  if (!bounds || n_bounds < 2 || n_bounds > gnn::kMaxBuckets || max_distance <= n_bounds / 2)
    return GNN_ERR_INVALID_ARG;
  gnn::rel_log_bounds(n_bounds, max_distance, bounds);
  return GNN_OK;
}

size_t gnn_rel_buffer_bytes(const gnn_graph* g) {
  return g ? 2 * gnn::align_up(size_t(g->e) + 1, 256) : 0;
}

gnn_status gnn_rel_prepare(const gnn_graph* g, const int32_t* pos_d, const int32_t* bounds,
                           int n_bounds, int two_sided, void* buffer_d, size_t buffer_bytes,
                           void* stream, gnn_rel** out) {
  if (!out) return GNN_ERR_INVALID_ARG;
  *out = nullptr;
  if (!g || !bounds || n_bounds < 1 || (two_sided != 0 && two_sided != 1) ||
      n_bounds > gnn::kMaxBuckets / (two_sided ? 2 : 1))
    return GNN_ERR_INVALID_ARG;
  if (bounds[0] != 0) return GNN_ERR_INVALID_ARG;
  for (int b = 1; b < n_bounds; ++b)
    if (bounds[b] < bounds[b - 1]) return GNN_ERR_INVALID_ARG;
  if ((g->n > 0 && !pos_d) || !aligned(pos_d, 4) || !buffer_d || !aligned(buffer_d, 256))
    return GNN_ERR_INVALID_ARG;
  if (buffer_bytes < gnn_rel_buffer_bytes(g)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!device_ok(g)) return GNN_ERR_INVALID_ARG;
  gnn_rel* r = new (std::nothrow) gnn_rel;
  if (!r) return GNN_ERR_INVALID_ARG;
  uint8_t* csr = static_cast<uint8_t*>(buffer_d);
  uint8_t* csc = csr + gnn::align_up(size_t(g->e) + 1, 256);
  r->g = g;
  r->n = g->n;
  r->e = g->e;
  r->csr = csr;
  r->csc = csc;
  r->buckets = n_bounds * (two_sided ? 2 : 1);
  if (gnn::launch_rel_buckets(g, pos_d, bounds, n_bounds, two_sided, csr, csc,
                              static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    delete r;
    return GNN_ERR_CUDA;
  }
  *out = r;
  return GNN_OK;
}

gnn_status gnn_rel_destroy(gnn_rel* r) {
  delete r;
  return GNN_OK;
}

gnn_status gnn_rel_arrays(const gnn_rel* r, const void** p, int n) {
  if (!r || !p || n < 2) return GNN_ERR_INVALID_ARG;
  p[0] = r->csr;
  p[1] = r->csc;
  for (int k = 2; k < n; ++k) p[k] = nullptr;
  return GNN_OK;
}

int gnn_rel_buckets(const gnn_rel* r) { return r ? r->buckets : 0; }

size_t transformer_rel_workspace_bytes(const gnn_graph* g, const gnn_rel* rel, int H, int D,
                                       gnn_dtype dtype) {
  Shape s;
  if (rel_shape(g, rel, H, D, dtype, &s) != GNN_OK) return 0;
  return gnn::transformer_rel_ws_bytes(g, s, rel->buckets);
}

gnn_status transformer_rel_forward(const gnn_graph* g, const gnn_rel* rel, int H, int D,
                                   gnn_dtype dtype, const void* q, const void* key,
                                   const void* val, float scale, const float* bias, void* out,
                                   float* lse, void* ws, size_t ws_bytes, void* stream) {
  Shape s;
  gnn_status r = rel_shape(g, rel, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!q || !key || !val || !bias || !out || !lse) return GNN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(val, 16) || !aligned(out, 16) ||
      !aligned(bias, 4) || !aligned(lse, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::transformer_rel_ws_bytes(g, s, rel->buckets))
    return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256) || !device_ok(g)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_transformer_rel_forward(
      g, rel, s, dtype, q, key, val, scale, bias, out, lse, static_cast<char*>(ws),
      static_cast<cudaStream_t>(stream)));
}

gnn_status transformer_rel_backward(const gnn_graph* g, const gnn_rel* rel, int H, int D,
                                    gnn_dtype dtype, const void* q, const void* key,
                                    const void* val, float scale, const float* bias,
                                    const float* lse, const void* dout, void* dq, void* dkey,
                                    void* dval, float* dbias, void* ws, size_t ws_bytes,
                                    void* stream) {
  Shape s;
  gnn_status r = rel_shape(g, rel, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (!dbias || !aligned(dbias, 4)) return GNN_ERR_INVALID_ARG;
  if (g->n == 0) {
    if (!device_ok(g)) return GNN_ERR_INVALID_ARG;
    return from_cuda(cudaMemsetAsync(dbias, 0, size_t(rel->buckets) * H * sizeof(float),
                                     static_cast<cudaStream_t>(stream)));
  }
  if (!q || !key || !val || !bias || !lse || !dout || !dq || !dkey || !dval)
    return GNN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(key, 16) || !aligned(val, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dkey, 16) || !aligned(dval, 16) || !aligned(lse, 4) ||
      !aligned(bias, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::transformer_rel_ws_bytes(g, s, rel->buckets))
    return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256) || !device_ok(g)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_transformer_rel_backward(
      g, rel, s, dtype, q, key, val, scale, bias, lse, dout, dq, dkey, dval, dbias,
      static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_norm_residual_forward(const gnn_norm_residual* d, gnn_dtype dtype, const void* x,
                                     const void* o, const void* gate, void* y, void* z,
                                     void* stream) {
  const gnn_status r = norm_residual_check(d, dtype);
  if (r != GNN_OK) return r;
  if ((d->pre == GNN_ROWNORM_NONE) != !z && d->n > 0) return GNN_ERR_INVALID_ARG;
  if (d->n == 0) return GNN_OK;
  if (!x || !o || !y || !gate_ok(d, dtype, gate)) return GNN_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(o, 16) || !aligned(y, 16) || !aligned(z, 16))
    return GNN_ERR_INVALID_ARG;
  int sms = 0;
  if (!current_sms(&sms)) return GNN_ERR_CUDA;
  return from_cuda(gnn::launch_norm_residual_forward(*d, dtype, x, o, gate, y, z, sms,
                                                     static_cast<cudaStream_t>(stream)));
}

size_t gnn_norm_residual_workspace_bytes(const gnn_norm_residual* d, gnn_dtype dtype) {
  if (norm_residual_check(d, dtype) != GNN_OK) return 0;
  return gnn::norm_residual_ws_bytes(d->n, d->F, dtype);
}

gnn_status gnn_norm_residual_backward(const gnn_norm_residual* d, gnn_dtype dtype, const void* y,
                                      const void* o, const void* gate, const void* dy,
                                      const void* dz, const gnn_norm_grads* grads, void* ws,
                                      size_t ws_bytes, void* stream) {
  const gnn_status r = norm_residual_check(d, dtype);
  if (r != GNN_OK) return r;
  if (!grads) return GNN_ERR_INVALID_ARG;
  const gnn_norm_grads& g = *grads;
  if (d->n > 0) {
    const bool pre = d->pre != GNN_ROWNORM_NONE;
    if (!o || !dy || !g.dx || !g.dout || pre != (y != nullptr) || pre != (dz != nullptr) ||
        !gate_ok(d, dtype, gate) || !gate_ok(d, dtype, g.dgate))
      return GNN_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(o, 16) || !aligned(dy, 16) || !aligned(dz, 16) ||
        !aligned(g.dx, 16) || !aligned(g.dout, 16))
      return GNN_ERR_INVALID_ARG;
  }
  if (!aligned(g.dw_post, 4) || !aligned(g.db_post, 4) || !aligned(g.dscale, 4) ||
      !aligned(g.dw_pre, 4) || !aligned(g.db_pre, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::norm_residual_ws_bytes(d->n, d->F, dtype))
    return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_norm_residual_backward(*d, dtype, y, o, gate, dy, dz, g,
                                                      static_cast<char*>(ws),
                                                      static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_pack8(int count, int64_t n, int H, int D, gnn_dtype dtype, const void* const* x,
                     int8_t* const* values, float* const* scale, void* stream) {
  Shape s;
  const gnn_status r = pack8_shape(n, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if (count < 1 || count > gnn::kPack8Max || !x || !values || !scale) return GNN_ERR_INVALID_ARG;
  if (n == 0) return GNN_OK;
  for (int k = 0; k < count; ++k)
    if (!x[k] || !values[k] || !scale[k] || !aligned(x[k], 16) || !aligned(values[k], 16) ||
        !aligned(scale[k], 4))
      return GNN_ERR_INVALID_ARG;
  int sms = 0;
  if (!current_sms(&sms)) return GNN_ERR_CUDA;
  return from_cuda(gnn::launch_pack8(count, n * s.rv, s.hv_log2, dtype, x, values, scale, sms,
                                     static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_unpack8(int64_t n, int H, int D, gnn_dtype dtype, const gnn_packed8* p, void* x,
                       void* stream) {
  // what either type packs reads back as either type
  Shape s;
  if (dtype != GNN_F32 && dtype != GNN_BF16) return GNN_ERR_INVALID_ARG;
  gnn_status r = pack8_shape(n, H, D, GNN_F32, &s);
  if (r == GNN_ERR_UNSUPPORTED) r = pack8_shape(n, H, D, GNN_BF16, &s);
  if (r != GNN_OK) return r;
  if (n == 0) return GNN_OK;
  if (!packed_ok(p) || !x || !aligned(x, 16)) return GNN_ERR_INVALID_ARG;
  int sms = 0;
  if (!current_sms(&sms)) return GNN_ERR_CUDA;
  return from_cuda(gnn::launch_unpack8(p->values, p->scale, n, H, D, dtype, x, sms,
                                       static_cast<cudaStream_t>(stream)));
}

size_t transformer_packed8_workspace_bytes(const gnn_graph* g, const gnn_rel* rel, int H, int D,
                                           gnn_dtype dtype) {
  Shape s;
  if ((rel ? rel_shape(g, rel, H, D, dtype, &s) : gatv2_shape(g, H, D, dtype, &s)) != GNN_OK)
    return 0;
  return gnn::transformer8_ws_bytes(g, s, rel ? rel->buckets : 0);
}

gnn_status transformer_packed8_backward(const gnn_graph* g, const gnn_rel* rel, int H, int D,
                                        gnn_dtype dtype, const gnn_packed8* q,
                                        const gnn_packed8* key, const gnn_packed8* val,
                                        float scale, const float* bias, const void* dout,
                                        void* dq, void* dkey, void* dval, float* dbias, void* ws,
                                        size_t ws_bytes, void* stream) {
  Shape s;
  const gnn_status r =
      rel ? rel_shape(g, rel, H, D, dtype, &s) : gatv2_shape(g, H, D, dtype, &s);
  if (r != GNN_OK) return r;
  if ((rel != nullptr) != (dbias != nullptr) || !aligned(dbias, 4)) return GNN_ERR_INVALID_ARG;
  if (!device_ok(g)) return GNN_ERR_INVALID_ARG;
  if (g->n == 0)
    return rel ? from_cuda(cudaMemsetAsync(dbias, 0, size_t(rel->buckets) * H * sizeof(float),
                                           static_cast<cudaStream_t>(stream)))
               : GNN_OK;
  if (!packed_ok(q) || !packed_ok(key) || !packed_ok(val) || !dout || !dq || !dkey || !dval ||
      (rel != nullptr) != (bias != nullptr))
    return GNN_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(dq, 16) || !aligned(dkey, 16) || !aligned(dval, 16) ||
      !aligned(bias, 4))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::transformer8_ws_bytes(g, s, rel ? rel->buckets : 0))
    return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_transformer8_backward(
      g, rel, s, dtype, *q, *key, *val, scale, bias, dout, dq, dkey, dval, dbias,
      static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
}

size_t reduce_agg_workspace_bytes(const gnn_graph* g, int F, gnn_dtype dtype) {
  Shape s;
  if (spmm_shape(g, F, dtype, &s) != GNN_OK) return 0;
  return gnn::reduce_ws_bytes(g, s);
}

gnn_status reduce_agg_forward(const gnn_graph* g, int F, gnn_dtype dtype, gnn_reduce_op op,
                              const void* x, void* out, int32_t* arg, void* ws, size_t ws_bytes,
                              void* stream) {
  Shape s;
  gnn_status r = spmm_shape(g, F, dtype, &s);
  if (r != GNN_OK) return r;
  if (op != GNN_REDUCE_MAX && op != GNN_REDUCE_MIN) return GNN_ERR_INVALID_ARG;
  if (g->n == 0) return GNN_OK;
  if (!x || !out || !arg || !aligned(x, 16) || !aligned(out, 16) || !aligned(arg, 16))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::reduce_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_reduce_forward(g, s, dtype, int(op), x, out, arg,
                                              static_cast<char*>(ws),
                                              static_cast<cudaStream_t>(stream)));
}

gnn_status reduce_agg_backward(const gnn_graph* g, int F, gnn_dtype dtype, const int32_t* arg,
                               const void* dout, void* dx, void* ws, size_t ws_bytes,
                               void* stream) {
  Shape s;
  gnn_status r = spmm_shape(g, F, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!arg || !dout || !dx || !aligned(arg, 16) || !aligned(dout, 16) || !aligned(dx, 16))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::reduce_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_reduce_backward(g, s, dtype, arg, dout, dx,
                                               static_cast<char*>(ws),
                                               static_cast<cudaStream_t>(stream)));
}

gnn_status reduce_agg_backward_ordered(const gnn_graph* g, int F, gnn_dtype dtype,
                                       const int32_t* arg, const void* dout, void* dx, void* ws,
                                       size_t ws_bytes, void* stream) {
  Shape s;
  gnn_status r = spmm_shape(g, F, dtype, &s);
  if (r != GNN_OK) return r;
  if (g->n == 0) return GNN_OK;
  if (!arg || !dout || !dx || !aligned(arg, 16) || !aligned(dout, 16) || !aligned(dx, 16))
    return GNN_ERR_INVALID_ARG;
  if (ws_bytes < gnn::reduce_ws_bytes(g, s)) return GNN_ERR_WORKSPACE_TOO_SMALL;
  if (!ws || !aligned(ws, 256)) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_reduce_backward_ordered(g, s, dtype, arg, dout, dx,
                                                       static_cast<char*>(ws),
                                                       static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_wait_selftest(const gnn_graph* g, int polls, void* stream) {
  if (!g || !g->err || polls < 1 || polls > 1000000) return GNN_ERR_INVALID_ARG;
  return from_cuda(gnn::launch_wait_selftest(g, polls, static_cast<cudaStream_t>(stream)));
}

gnn_status gnn_check_device_error(const gnn_graph* g, void* stream, int32_t* info) {
  if (!g || !g->err) return GNN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t w = 0;
  if (cudaStreamSynchronize(st) != cudaSuccess) return GNN_ERR_CUDA;
  if (cudaMemcpy(&w, g->err, sizeof w, cudaMemcpyDeviceToHost) != cudaSuccess) return GNN_ERR_CUDA;
  if (w != 0 && cudaMemset(g->err, 0, sizeof w) != cudaSuccess) return GNN_ERR_CUDA;
  if (info) *info = w;
  if (w & gnn::DEVERR_TIMEOUT) return GNN_ERR_TIMEOUT;
  if (w) return GNN_ERR_DEVICE_ASSERT;
  return GNN_OK;
}

}  // extern "C"
