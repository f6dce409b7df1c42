"""IO-aware fused GAT neighbour aggregation on GB300 (sm_103a).

Python front end of the C-ABI library ``libgnnagg.so`` (``include/gnnagg.h``).
torch supplies device memory and the current stream; the library's CUDA
kernels do all the work.

    g = Graph(row_ptr, col_idx)                    # once per graph (CSR, int32, cuda)
    out, lse = gat_forward(g, h, a_src, a_dst, 0.2)
    dh, da_src, da_dst = gat_backward(g, h, a_src, a_dst, 0.2, lse, dout)

``GATAggregate`` wraps the pair as a torch.autograd.Function.

The SpMM-family propagation of GCN / GraphConv layers (out = A~ x, norm
"sum", "mean" or "sym") runs on the same prepared graph:

    out = gcn_forward(g, x, "sym")                 # x [N, F]
    dx = gcn_backward(g, dout, "sym")              # A~^T dout over the cached CSC

the GATv2 attention (score att . LeakyReLU(xr_i + xl_j), value xl_j):

    out, lse = gatv2_forward(g, xl, xr, att, 0.2)
    dxl, dxr, datt = gatv2_backward(g, xl, xr, att, 0.2, lse, dout)

the graph-transformer attention (score scale * q_i . key_j, value val_j):

    out, lse = transformer_forward(g, q, key, val)     # scale defaults to 1/sqrt(D)
    dq, dkey, dval = transformer_backward(g, q, key, val, lse, dout)

the same with a learned relative position bias (bias [buckets, H], pos [N] int32):

    rel = RelPos(g, pos, 32, 128)                      # once per position vector
    out, lse = transformer_rel_forward(g, rel, q, key, val, bias)
    dq, dkey, dval, dbias = transformer_rel_backward(g, rel, q, key, val, bias, lse, dout)

the attention's backward pass from 8-bit checkpoints of q, key and val:

    q8, key8, val8 = pack8(q, key, val)                # int8 values, a scale per head vector
    dq, dkey, dval = transformer_backward8(g, q8, key8, val8, dout)   # rel=, bias= too

the norms, gate and residual scale between two blocks of a layer:

    y, z = norm_residual_forward(x, o, gate, w_post, scale=scale, w_pre=w_pre)
    grads = norm_residual_backward(y, o, dy, dz, gate, w_post, scale=scale, w_pre=w_pre)

``transformer_layer`` runs a layer between its projections with autograd: the
attention (bias and 8-bit checkpoints if asked for), the output projection that
the caller gives, and the norms, gate and residual.

and the max / min neighbourhood reduction with its winners:

    out, arg = reduce_forward(g, x, "max")         # arg [N, F] int32, -1 if no in-edges
    dx = reduce_backward(g, arg, dout)

The autograd Functions' backward passes are kernels without derivatives of their own: a
second derivative through them raises an error.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _native
from ._native import GnnError, Tiling

__all__ = ["Graph", "gat_forward", "gat_backward", "GATAggregate", "GnnError", "Tiling",
           "check_device_error", "default_tiling", "gcn_forward", "gcn_backward",
           "GCNAggregate", "reduce_forward", "reduce_backward", "ReduceAggregate",
           "gatv2_forward", "gatv2_backward", "GATv2Aggregate", "transformer_forward",
           "transformer_backward", "TransformerAggregate", "RelPos", "transformer_rel_forward",
           "transformer_rel_backward", "TransformerRelAggregate", "norm_residual_forward",
           "norm_residual_backward", "NormResidual", "Packed8", "pack8", "unpack8",
           "transformer_backward8", "TransformerCheckpoint8", "transformer_layer"]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(dt):
    if dt == torch.float32:
        return _native.F32
    if dt == torch.bfloat16:
        return _native.BF16
    raise TypeError(f"features must be float32 or bfloat16, got {dt}")


def default_tiling() -> Tiling:
    return _native.default_tiling()


class Graph:
    """A CSR graph prepared for aggregation (CSC transpose and degree buckets).

    row_ptr [N+1] and col_idx [E] are int32 CUDA tensors; row i lists the
    sources j of the edges j -> i.  They are referenced, not copied, and kept
    alive by this object.
    """

    def __init__(self, row_ptr: torch.Tensor, col_idx: torch.Tensor, tiling: Tiling | None = None,
                 stream=None):
        lib = _native.load()
        if row_ptr.dtype != torch.int32 or col_idx.dtype != torch.int32:
            raise TypeError("row_ptr and col_idx must be int32")
        if not (row_ptr.is_cuda and col_idx.is_cuda):
            raise ValueError("row_ptr and col_idx must be CUDA tensors")
        self.row_ptr = row_ptr.contiguous()
        self.col_idx = col_idx.contiguous()
        self.device = row_ptr.device
        self.n = self.row_ptr.numel() - 1
        self.e = self.col_idx.numel()
        self.tiling = tiling if tiling is not None else default_tiling()
        tref = ctypes.byref(self.tiling)
        nb = lib.gnn_graph_buffer_bytes(self.n, self.e, tref)
        ns = lib.gnn_graph_scratch_bytes(self.n, self.e)
        if nb == 0 or ns == 0:
            raise GnnError(_native.ERR_INVALID_ARG, "graph sizes or tiling")
        self.buffer = torch.empty(nb, dtype=torch.uint8, device=self.device)
        scratch = torch.empty(ns, dtype=torch.uint8, device=self.device)
        handle = ctypes.c_void_p()
        col = self.col_idx if self.e > 0 else torch.empty(4, dtype=torch.int32, device=self.device)
        rc = lib.gnn_graph_prepare(self.n, self.e, _ptr(self.row_ptr), _ptr(col),
                                   _ptr(self.buffer), nb, _ptr(scratch), ns, tref,
                                   _stream(stream, self.device), ctypes.byref(handle))
        _native.check(rc, "gnn_graph_prepare")
        self._col_keepalive = col
        self.handle = handle
        self._lib = lib

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.gnn_graph_destroy(h)
            self.handle = None

    def stats(self) -> dict:
        arr = (ctypes.c_int64 * 16)()
        _native.check(self._lib.gnn_graph_stats(self.handle, arr, 16), "gnn_graph_stats")
        v = list(arr)
        keys = ["light", "items", "hubs", "hub_chunks", "max_deg", "max_item"]
        return dict(n=v[0], e=v[1], csr=dict(zip(keys, v[2:8])), csc=dict(zip(keys, v[8:14])),
                    light_max_deg=v[14], cta_max_deg=v[15])

    def arrays(self) -> dict:
        """Views (into this graph's buffer) of the prepared structures."""
        ptrs = (ctypes.c_void_p * 8)()
        _native.check(self._lib.gnn_graph_arrays(self.handle, ptrs, 8), "gnn_graph_arrays")
        st = self.stats()
        base = self.buffer.data_ptr()

        def view(p, count, width):
            off = p - base
            assert 0 <= off and off + 4 * width * count <= self.buffer.numel()
            return self.buffer[off:off + 4 * width * count].view(torch.int32).view(count, width) \
                if width > 1 else self.buffer[off:off + 4 * count].view(torch.int32)

        def nitems(d):
            return d["items"]
        return dict(
            col_ptr=view(ptrs[0], self.n + 1, 1), row_idx=view(ptrs[1], self.e, 1),
            csr_light=view(ptrs[2], st["csr"]["light"], 1),
            csr_items=view(ptrs[3], nitems(st["csr"]), 4),
            csr_hubs=view(ptrs[4], st["csr"]["hubs"], 4),
            csc_light=view(ptrs[5], st["csc"]["light"], 1),
            csc_items=view(ptrs[6], nitems(st["csc"]), 4),
            csc_hubs=view(ptrs[7], st["csc"]["hubs"], 4))

    def workspace_bytes(self, H: int, D: int, dtype: torch.dtype) -> int:
        return int(self._lib.gat_agg_workspace_bytes(self.handle, H, D, _dtype_code(dtype)))

    def workspace(self, H: int, D: int, dtype: torch.dtype) -> torch.Tensor:
        n = self.workspace_bytes(H, D, dtype)
        if n == 0:
            raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
        return torch.empty(n, dtype=torch.uint8, device=self.device)


def _check_tensor(g: Graph, t, name: str, shape, dtype=None, floating=False):
    """Raise before any pointer reaches the library unless t is a contiguous
    tensor of the given shape (and dtype) on the graph's CUDA device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if floating and not t.is_floating_point():
        raise TypeError(f"{name} must be a floating-point tensor, got {t.dtype}")
    if not t.is_cuda or t.device != g.device:
        raise ValueError(f"{name} must be on the graph's device {g.device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _check_features(g: Graph, x: torch.Tensor, name: str):
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or x.shape[0] != g.n:
        raise ValueError(f"{name} must be [N, H, D] with N = {g.n}")
    _dtype_code(x.dtype)
    _check_tensor(g, x, name, None)


def _att(g: Graph, a, name: str, H: int, D: int) -> torch.Tensor:
    """An attention vector [H, D] on the graph's device, widened to float32."""
    _check_tensor(g, a, name, (H, D), floating=True)
    return a.to(torch.float32).contiguous()


def _given(g: Graph, t, name: str, shape, dtype, make):
    """A caller-supplied output (checked) or a new one."""
    return make() if t is None else _check_tensor(g, t, name, shape, dtype)


def _check_ws(g: Graph, ws):
    if ws is not None:
        _check_tensor(g, ws, "ws", None, torch.uint8)
        if ws.dim() != 1:
            raise ValueError("ws must be a one-dimensional uint8 tensor")
    return ws


def gat_forward(g: Graph, h: torch.Tensor, a_src: torch.Tensor, a_dst: torch.Tensor,
                slope: float = 0.2, out=None, lse=None, ws=None, stream=None):
    """out [N,H,D] (h's dtype) and lse [N,H] float32."""
    _check_features(g, h, "h")
    N, H, D = h.shape
    dt = _dtype_code(h.dtype)
    a_src = _att(g, a_src, "a_src", H, D)
    a_dst = _att(g, a_dst, "a_dst", H, D)
    out = _given(g, out, "out", h.shape, h.dtype, lambda: torch.empty_like(h))
    lse = _given(g, lse, "lse", (N, H), torch.float32,
                 lambda: torch.empty((N, H), dtype=torch.float32, device=h.device))
    if _check_ws(g, ws) is None:
        ws = g.workspace(H, D, h.dtype)
    rc = g._lib.gat_agg_forward(g.handle, H, D, dt, _ptr(h), _ptr(a_src), _ptr(a_dst),
                                float(slope), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                _stream(stream, h.device))
    _native.check(rc, "gat_agg_forward")
    return out, lse


def gat_backward(g: Graph, h: torch.Tensor, a_src: torch.Tensor, a_dst: torch.Tensor,
                 slope: float, lse: torch.Tensor, dout: torch.Tensor, dh=None, da_src=None,
                 da_dst=None, ws=None, stream=None, reuse_scores=False):
    """dh [N,H,D] (h's dtype), da_src and da_dst [H,D] float32.

    reuse_scores: ws is the workspace the gat_forward call on the same h,
    a_src, a_dst used, untouched since; the backward then takes the per-node
    scores that call left there instead of computing them again."""
    _check_features(g, h, "h")
    _check_features(g, dout, "dout")
    if dout.dtype != h.dtype:
        raise TypeError("dout must have h's dtype")
    N, H, D = h.shape
    dt = _dtype_code(h.dtype)
    a_src = _att(g, a_src, "a_src", H, D)
    a_dst = _att(g, a_dst, "a_dst", H, D)
    _check_tensor(g, lse, "lse", (N, H), torch.float32)
    dh = _given(g, dh, "dh", h.shape, h.dtype, lambda: torch.empty_like(h))
    da_src = _given(g, da_src, "da_src", (H, D), torch.float32,
                    lambda: torch.empty((H, D), dtype=torch.float32, device=h.device))
    da_dst = _given(g, da_dst, "da_dst", (H, D), torch.float32,
                    lambda: torch.empty((H, D), dtype=torch.float32, device=h.device))
    if _check_ws(g, ws) is None:
        if reuse_scores:
            raise ValueError("reuse_scores needs the forward call's workspace")
        ws = g.workspace(H, D, h.dtype)
    if reuse_scores:
        rc = g._lib.gat_agg_backward_reuse(g.handle, H, D, dt, _ptr(h), _ptr(a_src), _ptr(a_dst),
                                           float(slope), _ptr(lse), _ptr(dout), _ptr(dh),
                                           _ptr(da_src), _ptr(da_dst), _ptr(ws), ws.numel(),
                                           _stream(stream, h.device), None, 0)
    else:
        rc = g._lib.gat_agg_backward(g.handle, H, D, dt, _ptr(h), _ptr(a_src), _ptr(a_dst),
                                     float(slope), _ptr(lse), _ptr(dout), _ptr(dh), _ptr(da_src),
                                     _ptr(da_dst), _ptr(ws), ws.numel(), _stream(stream, h.device))
    _native.check(rc, "gat_agg_backward")
    return dh, da_src, da_dst


def _row_width(g: Graph, x: torch.Tensor, name: str) -> int:
    if not isinstance(x, torch.Tensor) or x.dim() < 2 or x.shape[0] != g.n:
        raise ValueError(f"{name} must be a tensor [N, ...] with N = {g.n}")
    _check_tensor(g, x, name, None)
    F = 1
    for d in x.shape[1:]:
        F *= d
    return F


def _gcn_call(fname, g, x, norm, out, ws, stream, what):
    F = _row_width(g, x, "features")
    dt = _dtype_code(x.dtype)
    if norm not in _native.NORMS:
        raise ValueError(f"norm must be one of {sorted(_native.NORMS)}")
    out = _given(g, out, "out", x.shape, x.dtype, lambda: torch.empty_like(x))
    if _check_ws(g, ws) is None:
        n = g._lib.gcn_agg_workspace_bytes(g.handle, F, dt)
        if n == 0:
            raise GnnError(_native.ERR_UNSUPPORTED, f"(F={F}, {x.dtype})")
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    fn = getattr(g._lib, fname)
    rc = fn(g.handle, F, dt, _native.NORMS[norm], _ptr(x), _ptr(out), _ptr(ws), ws.numel(),
            _stream(stream, x.device))
    _native.check(rc, what)
    return out


def gcn_forward(g: Graph, x: torch.Tensor, norm: str = "sym", out=None, ws=None, stream=None):
    """out = A~ x (x [N, ...] float32 or bfloat16, features flattened per node)."""
    return _gcn_call("gcn_agg_forward", g, x, norm, out, ws, stream, "gcn_agg_forward")


def gcn_backward(g: Graph, dout: torch.Tensor, norm: str = "sym", dx=None, ws=None, stream=None):
    """dx = A~^T dout."""
    return _gcn_call("gcn_agg_backward", g, dout, norm, dx, ws, stream, "gcn_agg_backward")


class GCNAggregate(torch.autograd.Function):
    """out = GCNAggregate.apply(graph, x, norm)."""

    @staticmethod
    def forward(ctx, g, x, norm):
        ctx.g = g
        ctx.norm = norm
        return gcn_forward(g, x.contiguous(), norm)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        return None, gcn_backward(ctx.g, dout.contiguous(), ctx.norm), None


def _gatv2_ws(g, H, D, dtype, ws, device):
    if ws is not None:
        return ws
    n = g._lib.gatv2_agg_workspace_bytes(g.handle, H, D, _dtype_code(dtype))
    if n == 0:
        raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def gatv2_forward(g: Graph, xl: torch.Tensor, xr: torch.Tensor, att: torch.Tensor,
                  slope: float = 0.2, out=None, lse=None, ws=None, stream=None):
    """out [N,H,D] (xl's dtype) and lse [N,H] float32."""
    _check_features(g, xl, "xl")
    _check_features(g, xr, "xr")
    if xr.shape != xl.shape or xr.dtype != xl.dtype:
        raise ValueError("xr must match xl in shape and dtype")
    N, H, D = xl.shape
    att = _att(g, att, "att", H, D)
    out = _given(g, out, "out", xl.shape, xl.dtype, lambda: torch.empty_like(xl))
    lse = _given(g, lse, "lse", (N, H), torch.float32,
                 lambda: torch.empty((N, H), dtype=torch.float32, device=xl.device))
    ws = _gatv2_ws(g, H, D, xl.dtype, _check_ws(g, ws), xl.device)
    rc = g._lib.gatv2_agg_forward(g.handle, H, D, _dtype_code(xl.dtype), _ptr(xl), _ptr(xr),
                                  _ptr(att), float(slope), _ptr(out), _ptr(lse), _ptr(ws),
                                  ws.numel(), _stream(stream, xl.device))
    _native.check(rc, "gatv2_agg_forward")
    return out, lse


def gatv2_backward(g: Graph, xl: torch.Tensor, xr: torch.Tensor, att: torch.Tensor,
                   slope: float, lse: torch.Tensor, dout: torch.Tensor, dxl=None, dxr=None,
                   datt=None, ws=None, stream=None):
    """dxl, dxr [N,H,D] (xl's dtype) and datt [H,D] float32."""
    _check_features(g, xl, "xl")
    _check_features(g, xr, "xr")
    _check_features(g, dout, "dout")
    if xr.shape != xl.shape or dout.shape != xl.shape or dout.dtype != xl.dtype:
        raise ValueError("xr and dout must match xl")
    N, H, D = xl.shape
    att = _att(g, att, "att", H, D)
    _check_tensor(g, lse, "lse", (N, H), torch.float32)
    dxl = _given(g, dxl, "dxl", xl.shape, xl.dtype, lambda: torch.empty_like(xl))
    dxr = _given(g, dxr, "dxr", xl.shape, xl.dtype, lambda: torch.empty_like(xl))
    datt = _given(g, datt, "datt", (H, D), torch.float32,
                  lambda: torch.empty((H, D), dtype=torch.float32, device=xl.device))
    ws = _gatv2_ws(g, H, D, xl.dtype, _check_ws(g, ws), xl.device)
    rc = g._lib.gatv2_agg_backward(g.handle, H, D, _dtype_code(xl.dtype), _ptr(xl), _ptr(xr),
                                   _ptr(att), float(slope), _ptr(lse), _ptr(dout),
                                   _ptr(dxl), _ptr(dxr), _ptr(datt), _ptr(ws), ws.numel(),
                                   _stream(stream, xl.device))
    _native.check(rc, "gatv2_agg_backward")
    return dxl, dxr, datt


class GATv2Aggregate(torch.autograd.Function):
    """out = GATv2Aggregate.apply(graph, xl, xr, att, slope)."""

    @staticmethod
    def forward(ctx, g, xl, xr, att, slope):
        xl, xr = xl.contiguous(), xr.contiguous()
        out, lse = gatv2_forward(g, xl, xr, att, slope)
        ctx.g, ctx.slope = g, slope
        ctx.save_for_backward(xl, xr, att, lse)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        xl, xr, att, lse = ctx.saved_tensors
        dxl, dxr, datt = gatv2_backward(ctx.g, xl, xr, att, ctx.slope, lse, dout.contiguous())
        return None, dxl, dxr, datt.to(att.dtype), None


def _gt_ws(g, H, D, dtype, ws, device):
    if ws is not None:
        return ws
    n = g._lib.transformer_agg_workspace_bytes(g.handle, H, D, _dtype_code(dtype))
    if n == 0:
        raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _gt_inputs(g, q, key, val):
    for name, x in (("q", q), ("key", key), ("val", val)):
        _check_features(g, x, name)
        if x.shape != q.shape or x.dtype != q.dtype:
            raise ValueError("q, key and val must share shape and dtype")
    return q.shape


def transformer_forward(g: Graph, q: torch.Tensor, key: torch.Tensor, val: torch.Tensor,
                        scale: float | None = None, out=None, lse=None, ws=None, stream=None):
    """out [N,H,D] (q's dtype) and lse [N,H] float32; scale defaults to 1/sqrt(D)."""
    N, H, D = _gt_inputs(g, q, key, val)
    scale = D ** -0.5 if scale is None else float(scale)
    out = _given(g, out, "out", q.shape, q.dtype, lambda: torch.empty_like(q))
    lse = _given(g, lse, "lse", (N, H), torch.float32,
                 lambda: torch.empty((N, H), dtype=torch.float32, device=q.device))
    ws = _gt_ws(g, H, D, q.dtype, _check_ws(g, ws), q.device)
    rc = g._lib.transformer_agg_forward(g.handle, H, D, _dtype_code(q.dtype), _ptr(q), _ptr(key),
                                        _ptr(val), scale, _ptr(out), _ptr(lse), _ptr(ws),
                                        ws.numel(), _stream(stream, q.device))
    _native.check(rc, "transformer_agg_forward")
    return out, lse


def transformer_backward(g: Graph, q: torch.Tensor, key: torch.Tensor, val: torch.Tensor,
                         lse: torch.Tensor, dout: torch.Tensor, scale: float | None = None,
                         dq=None, dkey=None, dval=None, ws=None, stream=None):
    """dq, dkey, dval [N,H,D] (q's dtype)."""
    N, H, D = _gt_inputs(g, q, key, val)
    _check_features(g, dout, "dout")
    if dout.shape != q.shape or dout.dtype != q.dtype:
        raise ValueError("dout must match q")
    scale = D ** -0.5 if scale is None else float(scale)
    _check_tensor(g, lse, "lse", (N, H), torch.float32)
    dq = _given(g, dq, "dq", q.shape, q.dtype, lambda: torch.empty_like(q))
    dkey = _given(g, dkey, "dkey", q.shape, q.dtype, lambda: torch.empty_like(q))
    dval = _given(g, dval, "dval", q.shape, q.dtype, lambda: torch.empty_like(q))
    ws = _gt_ws(g, H, D, q.dtype, _check_ws(g, ws), q.device)
    rc = g._lib.transformer_agg_backward(g.handle, H, D, _dtype_code(q.dtype), _ptr(q),
                                         _ptr(key), _ptr(val), scale, _ptr(lse),
                                         _ptr(dout), _ptr(dq), _ptr(dkey), _ptr(dval), _ptr(ws),
                                         ws.numel(), _stream(stream, q.device))
    _native.check(rc, "transformer_agg_backward")
    return dq, dkey, dval


class TransformerAggregate(torch.autograd.Function):
    """out = TransformerAggregate.apply(graph, q, key, val, scale)."""

    @staticmethod
    def forward(ctx, g, q, key, val, scale):
        q, key, val = q.contiguous(), key.contiguous(), val.contiguous()
        out, lse = transformer_forward(g, q, key, val, scale)
        ctx.g, ctx.scale = g, scale
        ctx.save_for_backward(q, key, val, lse)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, key, val, lse = ctx.saved_tensors
        dq, dk, dv = transformer_backward(ctx.g, q, key, val, lse, dout.contiguous(), ctx.scale)
        return None, dq, dk, dv, None


def _on_stream(fn):
    """Lets a call take stream=: it then runs with that stream as torch's own, so
    that what it allocates belongs to the stream that uses it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        device = next((a.device for a in args if hasattr(a, "device")), stream.device)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the arguments on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _launch(fn, what: str, device, *args):
    """fn(*args, the device's current stream), with the device current."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != _native.OK:
        raise GnnError(rc, what)


def _at(t):
    return None if t is None else t.data_ptr()


def _plain_tensor(t, name, shape, dtype, device):
    """Raise unless t is a contiguous tensor of that shape, dtype and device."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and \
            t.device == device and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous and on {device}")


def _output(t, name, shape, dtype, device):
    """A caller-supplied output (checked) or a new one."""
    return torch.empty(shape, dtype=dtype, device=device) if t is None else \
        _plain_tensor(t, name, shape, dtype, device)


def _like(t, name, x):
    """_output of x's shape, dtype and device (x contiguous)."""
    return torch.empty_like(x) if t is None else _plain_tensor(t, name, x.shape, x.dtype, x.device)


class RelPos:
    """Buckets of the relative positions of a graph's edges.

    pos [N] int32: the nodes' positions.  An edge j -> i falls into the bucket
    of pos[j] - pos[i].  The default rule gives small distances a bucket each
    and lets the others grow by equal ratios up to max_distance; bidirectional
    gives half of the buckets to sources after the destination, otherwise these
    all share bucket 0 with distance 0.  bounds: the lower bounds of one side's
    buckets (ascending whole numbers from 0) instead of that rule.  At most
    128 buckets.  Prepare it once per position vector; pos is not kept.
    """

    @_on_stream
    def __init__(self, g: Graph, pos: torch.Tensor, num_buckets: int = 32,
                 max_distance: int = 128, bidirectional: bool = True, bounds=None):
        lib = _native.load()
        _check_tensor(g, pos, "pos", (g.n,), torch.int32)
        if bounds is None:
            if bidirectional and num_buckets % 2:
                raise ValueError("a bidirectional rule needs an even number of buckets")
            if not 0 < max_distance < 2 ** 31:
                raise ValueError("max_distance must be a positive 32-bit number")
            side = num_buckets // 2 if bidirectional else num_buckets
            table = (ctypes.c_int32 * max(side, 1))()
            _native.check(lib.gnn_rel_log_bounds(side, int(max_distance), table),
                          "gnn_rel_log_bounds")
        else:
            if not all(0 <= b < 2 ** 31 for b in bounds):
                raise ValueError("bounds must be whole numbers of 32 bits, not negative")
            table = (ctypes.c_int32 * len(bounds))(*bounds)
        self.graph = g
        self.bounds = list(table)
        self.bidirectional = bool(bidirectional)
        handle = ctypes.c_void_p()
        n = lib.gnn_rel_buffer_bytes(g.handle)
        self.buffer = torch.empty(n, dtype=torch.uint8, device=g.device)

        def prepare(s):
            return lib.gnn_rel_prepare(g.handle, _at(pos), table, len(table),
                                       int(self.bidirectional), _at(self.buffer), n, s,
                                       ctypes.byref(handle))

        _launch(prepare, "gnn_rel_prepare", g.device)
        self.handle = handle
        self._lib = lib
        self._ws = {}  # workspace bytes by (H, D, dtype)
        self.buckets = lib.gnn_rel_buckets(handle)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self._lib.gnn_rel_destroy(h)
            self.handle = None

    def workspace(self, H: int, D: int, dtype: torch.dtype) -> torch.Tensor:
        """A workspace that serves transformer_rel_forward, transformer_rel_backward
        and transformer_backward8 with this plan (one call at a time)."""
        dt = _dtype_code(dtype)
        n = max(f(self.graph.handle, self.handle, H, D, dt) for f in (
            self._lib.transformer_rel_workspace_bytes,
            self._lib.transformer_packed8_workspace_bytes))
        if n == 0:
            raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
        return torch.empty(n, dtype=torch.uint8, device=self.graph.device)

    def arrays(self):
        """The buckets of the edges, uint8 [E], in CSR and in CSC order (views)."""
        ptrs = (ctypes.c_void_p * 2)()
        _native.check(self._lib.gnn_rel_arrays(self.handle, ptrs, 2), "gnn_rel_arrays")
        at = [p - self.buffer.data_ptr() for p in ptrs]
        return tuple(self.buffer[o:o + self.graph.e] for o in at)


def _rel_bias(g: Graph, rel: RelPos, bias, H: int):
    if not isinstance(rel, RelPos):
        raise TypeError(f"rel must be a RelPos, got {type(rel).__name__}")
    if rel.graph is not g:
        raise ValueError("rel was prepared for another graph")
    _check_tensor(g, bias, "bias", (rel.buckets, H), floating=True)
    if bias.dtype == torch.float64:  # finite entries stay finite: an infinity masks
        top = torch.finfo(torch.float32).max
        bias = torch.where(bias.isinf(), bias, bias.clamp(-top, top))
    return bias if bias.dtype == torch.float32 else bias.to(torch.float32)


def _rel_qkv(g: Graph, q, key, val):
    _check_features(g, q, "q")
    _plain_tensor(key, "key", q.shape, q.dtype, g.device)
    _plain_tensor(val, "val", q.shape, q.dtype, g.device)
    return q.shape


def _rel_ws(g, rel, H, D, dtype, ws):
    if _check_ws(g, ws) is not None:
        return ws
    n = rel._ws.get((H, D, dtype))
    if n is None:
        n = g._lib.transformer_rel_workspace_bytes(g.handle, rel.handle, H, D, _dtype_code(dtype))
        if n == 0:
            raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
        rel._ws[H, D, dtype] = n
    return torch.empty(n, dtype=torch.uint8, device=g.device)


@_on_stream
def transformer_rel_forward(g: Graph, rel: RelPos, q: torch.Tensor, key: torch.Tensor,
                            val: torch.Tensor, bias: torch.Tensor, scale: float | None = None,
                            out=None, lse=None, ws=None):
    """transformer_forward with bias [buckets, H] added to the scores by the
    bucket of each edge: out [N,H,D] (q's dtype) and lse [N,H] float32.  An
    entry of -inf masks its bucket; finite entries may have any size (a row
    whose edges all carry the same one has the weights that it has without)."""
    N, H, D = _rel_qkv(g, q, key, val)
    bias = _rel_bias(g, rel, bias, H)
    out = _like(out, "out", q)
    lse = _output(lse, "lse", (N, H), torch.float32, g.device)
    ws = _rel_ws(g, rel, H, D, q.dtype, ws)
    _launch(g._lib.transformer_rel_forward, "transformer_rel_forward", g.device, g.handle,
            rel.handle, H, D, _dtype_code(q.dtype), _at(q), _at(key), _at(val),
            D ** -0.5 if scale is None else float(scale), _at(bias), _at(out), _at(lse), _at(ws),
            ws.numel())
    return out, lse


@_on_stream
def transformer_rel_backward(g: Graph, rel: RelPos, q: torch.Tensor, key: torch.Tensor,
                             val: torch.Tensor, bias: torch.Tensor, lse: torch.Tensor,
                             dout: torch.Tensor, scale: float | None = None, dq=None, dkey=None,
                             dval=None, dbias=None, ws=None):
    """dq, dkey, dval [N,H,D] (q's dtype) and dbias [buckets,H] float32."""
    N, H, D = shape = _rel_qkv(g, q, key, val)
    _plain_tensor(dout, "dout", shape, q.dtype, g.device)
    _plain_tensor(lse, "lse", (N, H), torch.float32, g.device)
    bias = _rel_bias(g, rel, bias, H)
    dq = _like(dq, "dq", q)
    dkey = _like(dkey, "dkey", q)
    dval = _like(dval, "dval", q)
    dbias = _like(dbias, "dbias", bias)
    ws = _rel_ws(g, rel, H, D, q.dtype, ws)
    _launch(g._lib.transformer_rel_backward, "transformer_rel_backward", g.device, g.handle,
            rel.handle, H, D, _dtype_code(q.dtype), _at(q), _at(key), _at(val),
            D ** -0.5 if scale is None else float(scale), _at(bias), _at(lse), _at(dout), _at(dq),
            _at(dkey), _at(dval), _at(dbias), _at(ws), ws.numel())
    return dq, dkey, dval, dbias


class TransformerRelAggregate(torch.autograd.Function):
    """out = TransformerRelAggregate.apply(graph, rel, q, key, val, bias, scale)."""

    @staticmethod
    def forward(ctx, g, rel, q, key, val, bias, scale):
        q, key, val, bias = (t.contiguous() for t in (q, key, val, bias))
        out, lse = transformer_rel_forward(g, rel, q, key, val, bias, scale)
        ctx.g, ctx.rel, ctx.scale = g, rel, scale
        ctx.save_for_backward(q, key, val, bias, lse)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, key, val, bias, lse = ctx.saved_tensors
        dq, dk, dv, db = transformer_rel_backward(ctx.g, ctx.rel, q, key, val, bias, lse,
                                                  dout.contiguous(), ctx.scale)
        return None, None, dq, dk, dv, db.to(bias.dtype), None


class Packed8(NamedTuple):
    """An activation [N, H, D] in 8 bits: int8 values of that shape and a
    float32 scale [N, H], standing for values * scale[..., None]."""

    values: torch.Tensor
    scale: torch.Tensor

    @property
    def device(self):
        return self.values.device


@_on_stream
def pack8(*xs: torch.Tensor, out=None):
    """8-bit checkpoints of up to 8 tensors [N, H, D] of one shape and dtype, in
    one launch: a Packed8 for each.  Every head vector has its own scale, the
    largest magnitude over 127; values are rounded to nearest, ties to even.
    out: the Packed8s to write."""
    if not 1 <= len(xs) <= 8:
        raise ValueError("pack8 takes 1 to 8 tensors")
    x = xs[0]
    if not isinstance(x, torch.Tensor) or x.dim() != 3 or not x.is_cuda:
        raise ValueError("pack8 takes CUDA tensors [N, H, D]")
    shape, device = x.shape, x.device
    dt = _dtype_code(x.dtype)
    for t in xs:
        _plain_tensor(t, "every tensor", shape, x.dtype, device)
    N, H, D = shape
    if out is None:
        line = (N, H)
        out = tuple([Packed8(torch.empty(shape, dtype=torch.int8, device=device),
                             torch.empty(line, dtype=torch.float32, device=device)) for _ in xs])
    else:
        out = tuple(out)
        if len(out) != len(xs):
            raise ValueError("out must have a Packed8 for every tensor")
        for p in out:
            _packed(p, "out", shape, device)
    rows = _native.PTRS[len(xs)]
    _launch(_native.load().gnn_pack8, "gnn_pack8", device, len(xs), N, H, D, dt,
            rows(*[t.data_ptr() for t in xs]), rows(*[p[0].data_ptr() for p in out]),
            rows(*[p[1].data_ptr() for p in out]))
    return out


def _packed(p, name, shape, device) -> _native.Packed8:
    if not isinstance(p, Packed8):
        raise TypeError(f"{name} must be a Packed8, got {type(p).__name__}")
    _plain_tensor(p.values, f"{name}.values", shape, torch.int8, device)
    _plain_tensor(p.scale, f"{name}.scale", shape[:2], torch.float32, device)
    return _native.Packed8(p.values.data_ptr(), p.scale.data_ptr())


@_on_stream
def unpack8(p: Packed8, dtype: torch.dtype = torch.float32, out=None):
    """values * scale, rounded to dtype (float32 or bfloat16)."""
    if not isinstance(p, Packed8) or not isinstance(p.values, torch.Tensor) or \
            p.values.dim() != 3 or not p.values.is_cuda:
        raise ValueError("unpack8 takes a Packed8 of CUDA tensors")
    dt = _dtype_code(dtype)
    shape, device = p.values.shape, p.values.device
    c = _packed(p, "p", shape, device)
    out = _output(out, "out", shape, dtype, device)
    _launch(_native.load().gnn_unpack8, "gnn_unpack8", device, *shape, dt, ctypes.byref(c),
            _at(out))
    return out


@_on_stream
def transformer_backward8(g: Graph, q: Packed8, key: Packed8, val: Packed8, dout: torch.Tensor,
                          scale: float | None = None, rel: RelPos | None = None, bias=None,
                          dq=None, dkey=None, dval=None, dbias=None, ws=None):
    """The gradients of the graph-transformer attention from 8-bit checkpoints
    of q, key and val, taken at the values that these stand for (its softmax is
    computed there too; no lse is needed): dq, dkey, dval (dout's dtype) and,
    with rel and bias, dbias [buckets,H] float32."""
    _check_features(g, dout, "dout")
    shape, device, dtype = dout.shape, g.device, dout.dtype
    N, H, D = shape
    cq, ck, cv = (_packed(q, "q", shape, device), _packed(key, "key", shape, device),
                  _packed(val, "val", shape, device))
    if (rel is None) != (bias is None):
        raise ValueError("rel and bias go together")
    if rel is not None:
        bias = _rel_bias(g, rel, bias, H)
        dbias = _like(dbias, "dbias", bias)
    elif dbias is not None:
        raise ValueError("there is no dbias without a bias")
    dq = _like(dq, "dq", dout)
    dkey = _like(dkey, "dkey", dout)
    dval = _like(dval, "dval", dout)
    handle = None if rel is None else rel.handle
    dt = _dtype_code(dtype)
    if _check_ws(g, ws) is None:
        n = g._lib.transformer_packed8_workspace_bytes(g.handle, handle, H, D, dt)
        if n == 0:
            raise GnnError(_native.ERR_UNSUPPORTED, f"(H={H}, D={D}, {dtype})")
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    _launch(g._lib.transformer_packed8_backward, "transformer_packed8_backward", device, g.handle,
            handle, H, D, dt, ctypes.byref(cq), ctypes.byref(ck), ctypes.byref(cv),
            D ** -0.5 if scale is None else float(scale), _at(bias), _at(dout), _at(dq), _at(dkey),
            _at(dval), _at(dbias), _at(ws), ws.numel())
    return (dq, dkey, dval) if rel is None else (dq, dkey, dval, dbias)


class TransformerCheckpoint8(torch.autograd.Function):
    """out = TransformerCheckpoint8.apply(graph, rel, q, key, val, bias, scale):
    the graph-transformer attention (rel and bias None, or both given) that
    keeps only 8-bit checkpoints of q, key and val for its backward pass."""

    @staticmethod
    def forward(ctx, g, rel, q, key, val, bias, scale):
        if (rel is None) != (bias is None):
            raise ValueError("rel and bias go together")
        q, key, val = q.contiguous(), key.contiguous(), val.contiguous()
        if rel is None:
            out, _ = transformer_forward(g, q, key, val, scale)
        else:
            bias = bias.contiguous()
            out, _ = transformer_rel_forward(g, rel, q, key, val, bias, scale)
        packed = pack8(q, key, val)
        ctx.g, ctx.rel, ctx.scale = g, rel, scale
        ctx.save_for_backward(*(t for p in packed for t in p), bias)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        *flat, bias = ctx.saved_tensors
        c = [Packed8(*flat[k:k + 2]) for k in (0, 2, 4)]
        d = transformer_backward8(ctx.g, *c, dout.contiguous(), ctx.scale, ctx.rel, bias)
        return None, None, *d[:3], None if ctx.rel is None else d[3].to(bias.dtype), None


_NORM_PARAMS = ("w_post", "b_post", "scale", "w_pre", "b_pre")
_NORM_GRADS = ("dx", "do", "dgate") + tuple("d" + k for k in _NORM_PARAMS)


def _norm_desc(o, gate, params, kind, eps):
    """The call's gnn_norm_residual, the float32 parameters it points to (to be
    kept until the launch) and whether there is a norm before the next block."""
    if not isinstance(o, torch.Tensor) or o.dim() < 2:
        raise ValueError("o must be a tensor [N, ...]")
    shape, dtype, device = o.shape, o.dtype, o.device
    _dtype_code(dtype)
    if not o.is_cuda or not o.is_contiguous():
        raise ValueError("o must be a contiguous CUDA tensor")
    post, pre = (kind, kind) if isinstance(kind, str) else kind
    post, pre = _native.ROWNORMS.get(post), _native.ROWNORMS.get(pre)
    if post is None or pre is None:
        raise ValueError(f"kind must be one of {sorted(_native.ROWNORMS)}, or a pair of them "
                         "(after the block, before the next)")
    n = shape[0]
    F = math.prod(shape[1:])
    width = 0
    if gate is not None:
        width = F if isinstance(gate, torch.Tensor) and gate.shape == shape else 1
        _plain_tensor(gate, "gate", shape if width == F else (n, 1), dtype, device)
    kept, at, line = [], [], (F,)
    for k, t in zip(_NORM_PARAMS, params):
        if t is None:
            at.append(None)
        else:
            if not isinstance(t, torch.Tensor) or not t.is_floating_point():
                raise TypeError(f"{k} must be a floating-point tensor")
            if t.dtype is not torch.float32:
                t = t.to(torch.float32)
            if t.shape != line or t.device != device or not t.is_contiguous():
                _plain_tensor(t, k, line, torch.float32, device)
            at.append(t.data_ptr())
        kept.append(t)
    return _native.NormResidual(n, F, post, pre, width, eps, *at), kept, pre != 0


@_on_stream
def norm_residual_forward(x: torch.Tensor, o: torch.Tensor, gate=None, w_post=None, b_post=None,
                          scale=None, w_pre=None, b_pre=None, kind="rms", eps: float = 1e-6,
                          y=None, z=None):
    """y = x + scale * sigmoid(gate) * (norm(o) w_post + b_post) and
    z = norm(y) w_pre + b_pre, for x, o [N, ...] (a node's features flattened).

    kind: "rms", "layer" or "none" for both norms, or a pair (after the block,
    before the next).  gate: None, [N, 1] or o's shape (before its sigmoid).
    Parameters have one entry per feature; None leaves a factor or a sum out.
    z is None where the second norm is "none"."""
    d, kept, pre = _norm_desc(o, gate, (w_post, b_post, scale, w_pre, b_pre), kind, eps)
    _plain_tensor(x, "x", o.shape, o.dtype, o.device)
    if z is not None and not pre:
        raise ValueError("there is no z without a norm before the next block")
    y = _like(y, "y", o)
    if pre:
        z = _like(z, "z", o)
    _launch(_native.load().gnn_norm_residual_forward, "gnn_norm_residual_forward", o.device,
            ctypes.byref(d), _dtype_code(o.dtype), _at(x), _at(o), _at(gate), _at(y), _at(z))
    return y, z


@_on_stream
def norm_residual_backward(y, o: torch.Tensor, dy: torch.Tensor, dz=None, gate=None, w_post=None,
                           b_post=None, scale=None, w_pre=None, b_pre=None, kind="rms",
                           eps: float = 1e-6, ws=None, grads=None):
    """The gradients of norm_residual_forward, as a dict: dx, do, dgate (o's
    dtype; dgate None without a gate) and dw_post, db_post, dscale, dw_pre,
    db_pre (float32; None where the parameter is).  y is the forward's y, dy the
    gradient that reaches it past the second norm and dz that of z; y and dz are
    None where that norm is "none".  grads: outputs to write, by those names."""
    d, kept, pre = _norm_desc(o, gate, (w_post, b_post, scale, w_pre, b_pre), kind, eps)
    device = o.device
    like = (o.shape, o.dtype, device)
    _plain_tensor(dy, "dy", *like)
    for name, t in (("y", y), ("dz", dz)):
        if pre:
            _plain_tensor(t, name, *like)
        elif t is not None:
            raise ValueError(f"there is no {name} without a norm before the next block")
    got = {}
    for name, t in zip(_NORM_GRADS, (o, o, gate, *kept)):
        given = None if grads is None else grads.get(name)
        if t is not None:
            got[name] = _like(given, name, t)
        elif given is None:
            got[name] = None
        else:
            raise ValueError(f"there is no {name} in this call")
    if grads is not None and not grads.keys() <= got.keys():
        raise ValueError(f"unknown gradients {sorted(grads.keys() - got.keys())}")
    lib = _native.load()
    dt = _dtype_code(o.dtype)
    if ws is None:
        ws = torch.empty(lib.gnn_norm_residual_workspace_bytes(ctypes.byref(d), dt),
                         dtype=torch.uint8, device=device)
    elif not isinstance(ws, torch.Tensor) or ws.dtype != torch.uint8 or ws.dim() != 1 or \
            ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a one-dimensional uint8 tensor on {device}")
    c = _native.NormGrads(*map(_at, got.values()))
    _launch(lib.gnn_norm_residual_backward, "gnn_norm_residual_backward", device, ctypes.byref(d),
            dt, _at(y), _at(o), _at(gate), _at(dy), _at(dz), ctypes.byref(c), _at(ws), ws.numel())
    return got


class NormResidual(torch.autograd.Function):
    """y, z = NormResidual.apply(x, o, gate, w_post, b_post, scale, w_pre, b_pre,
    kind, eps)."""

    @staticmethod
    def forward(ctx, x, o, gate, w_post, b_post, scale, w_pre, b_pre, kind, eps):
        x, o, gate = (None if t is None else t.contiguous() for t in (x, o, gate))
        params = [None if t is None else t.contiguous()
                  for t in (w_post, b_post, scale, w_pre, b_pre)]
        y, z = norm_residual_forward(x, o, gate, *params, kind=kind, eps=eps)
        ctx.kind, ctx.eps = kind, eps
        ctx.save_for_backward(None if z is None else y, o, gate, *params)
        return y, z

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dz):
        y, o, gate, *params = ctx.saved_tensors
        dz = None if y is None else dz.contiguous()
        g = norm_residual_backward(y, o, dy.contiguous(), dz, gate, *params, kind=ctx.kind,
                                   eps=ctx.eps)
        return (g["dx"], g["do"], g["dgate"],
                *(None if t is None else g["d" + k].to(t.dtype)
                  for k, t in zip(_NORM_PARAMS, params)), None, None)


def transformer_layer(g: Graph, x: torch.Tensor, q: torch.Tensor, key: torch.Tensor,
                      val: torch.Tensor, rel: RelPos | None = None, bias=None, gate=None,
                      w_post=None, b_post=None, res_scale=None, w_pre=None, b_pre=None,
                      project=None, scale: float | None = None, kind="rms", eps: float = 1e-6,
                      checkpoint8: bool = False):
    """One graph-transformer layer between its input projections and the next
    layer's, with autograd: attention of q, key, val [N,H,D] over g (with rel and
    bias, if given), `project` (the output projection, a function of the
    attention's [N,H,D] returning x's shape; None where H*D is x's width), then
    norm, gate, residual scale and sum with x, and the norm before the next
    layer.  Returns (y, z) as norm_residual_forward does.  checkpoint8: the
    attention keeps 8-bit checkpoints of q, key and val for its backward pass
    instead of the tensors.  To capture a training step into a CUDA graph, let no
    eager autograd graph of the same leaves be alive (torch would order the
    captured gradients behind the eager stream)."""
    if (rel is None) != (bias is None):
        raise ValueError("rel and bias go together")
    if checkpoint8:
        out = TransformerCheckpoint8.apply(g, rel, q, key, val, bias, scale)
    elif rel is not None:
        out = TransformerRelAggregate.apply(g, rel, q, key, val, bias, scale)
    else:
        out = TransformerAggregate.apply(g, q, key, val, scale)
    o = out.reshape(x.shape) if project is None else project(out)
    return NormResidual.apply(x, o, gate, w_post, b_post, res_scale, w_pre, b_pre, kind, eps)


def _reduce_ws(g, F, dt, ws, device):
    if ws is not None:
        return ws
    n = g._lib.reduce_agg_workspace_bytes(g.handle, F, dt)
    if n == 0:
        raise GnnError(_native.ERR_UNSUPPORTED, f"(F={F})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def reduce_forward(g: Graph, x: torch.Tensor, op: str = "max", out=None, arg=None, ws=None,
                   stream=None):
    """out [N, ...] (x's dtype) = max or min over in-neighbours, feature by
    feature; arg int32 of the same shape = the winning source (-1: none)."""
    F = _row_width(g, x, "x")
    dt = _dtype_code(x.dtype)
    if op not in _native.REDUCE_OPS:
        raise ValueError(f"op must be one of {sorted(_native.REDUCE_OPS)}")
    out = _given(g, out, "out", x.shape, x.dtype, lambda: torch.empty_like(x))
    arg = _given(g, arg, "arg", x.shape, torch.int32,
                 lambda: torch.empty(x.shape, dtype=torch.int32, device=x.device))
    ws = _reduce_ws(g, F, dt, _check_ws(g, ws), x.device)
    rc = g._lib.reduce_agg_forward(g.handle, F, dt, _native.REDUCE_OPS[op], _ptr(x), _ptr(out),
                                   _ptr(arg), _ptr(ws), ws.numel(), _stream(stream, x.device))
    _native.check(rc, "reduce_agg_forward")
    return out, arg


def reduce_backward(g: Graph, arg: torch.Tensor, dout: torch.Tensor, dx=None, ws=None,
                    stream=None, ordered=False):
    """dx = the gradient of sum(out * dout) w.r.t. x, from the forward's arg.

    ordered: gather the terms over the cached CSC in a fixed order instead of
    adding them with atomics (bitwise reproducible, more bytes moved)."""
    F = _row_width(g, dout, "dout")
    _check_tensor(g, arg, "arg", dout.shape, torch.int32)
    dt = _dtype_code(dout.dtype)
    dx = _given(g, dx, "dx", dout.shape, dout.dtype, lambda: torch.empty_like(dout))
    ws = _reduce_ws(g, F, dt, _check_ws(g, ws), dout.device)
    fn = g._lib.reduce_agg_backward_ordered if ordered else g._lib.reduce_agg_backward
    rc = fn(g.handle, F, dt, _ptr(arg), _ptr(dout), _ptr(dx), _ptr(ws), ws.numel(),
            _stream(stream, dout.device))
    _native.check(rc, "reduce_agg_backward_ordered" if ordered else "reduce_agg_backward")
    return dx


class ReduceAggregate(torch.autograd.Function):
    """out = ReduceAggregate.apply(graph, x, op)."""

    @staticmethod
    def forward(ctx, g, x, op):
        out, arg = reduce_forward(g, x.contiguous(), op)
        ctx.g = g
        ctx.save_for_backward(arg)
        ctx.mark_non_differentiable(arg)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (arg,) = ctx.saved_tensors
        return None, reduce_backward(ctx.g, arg, dout.contiguous()), None


def check_device_error(g: Graph, stream=None) -> int:
    """Synchronise and read the graph's device status word (raises on error)."""
    info = ctypes.c_int32(0)
    rc = g._lib.gnn_check_device_error(g.handle, _stream(stream, g.device), ctypes.byref(info))
    _native.check(rc, "gnn_check_device_error")
    return info.value


class GATAggregate(torch.autograd.Function):
    """out = GATAggregate.apply(graph, h, a_src, a_dst, slope)."""

    @staticmethod
    def forward(ctx, g, h, a_src, a_dst, slope):
        h = h.contiguous()
        ws = g.workspace(h.shape[1], h.shape[2], h.dtype)
        out, lse = gat_forward(g, h, a_src, a_dst, slope, ws=ws)
        ctx.g = g
        ctx.slope = slope
        ctx.ws = ws  # its per-node scores serve the backward; nothing else writes it
        ctx.save_for_backward(h, a_src, a_dst, lse)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        h, a_src, a_dst, lse = ctx.saved_tensors
        dh, da_s, da_d = gat_backward(ctx.g, h, a_src, a_dst, ctx.slope, lse, dout.contiguous(),
                                      ws=ctx.ws, reuse_scores=True)
        return None, dh, da_s.to(a_src.dtype), da_d.to(a_dst.dtype), None
