"""The norms before and after a block with its gate and residual scale: the
CUDA path against a plain float64 implementation, with bounds propagated
through its formulas (layer_ref)."""
import ctypes

import numpy as np
import pytest
import torch

import layer_ref
import workload
from gpu_util import to_device, to_f64

PARAMS = ("w_post", "b_post", "scale", "w_pre", "b_pre")


def data(n, F, dtype, gate, seed=1, offset=0.0, params=PARAMS):
    def draw(stream, *shape):
        x = workload.normal_f32(seed, stream, shape, 1.0)
        return x

    a = {k: draw(s, n, F) for s, k in enumerate(("x", "o", "dy", "dz"), 1)}
    a["o"] = (3 * a["o"] + np.float32(offset)).astype(np.float32)
    a["x"] = (a["x"] - np.float32(offset)).astype(np.float32)
    a["gate"] = {"none": None, "row": draw(5, n, 1), "element": 4 * draw(5, n, F)}[gate]
    if dtype == "bf16":
        a = {k: None if t is None else workload.f32_to_bf16_bits(t) for k, t in a.items()}
    p = {k: workload.normal_f32(seed, 10 + s, (F,), 0.2) + np.float32(k[0] != "b")
         for s, k in enumerate(PARAMS) if k in params}
    return a, p


def wide(x):
    if x is None:
        return None
    return (workload.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def run(a, p, dtype, kind, eps=1e-6, **kw):
    import graph_neural_network_gb300 as gnn
    t = {k: None if v is None else to_device(v, dtype) for k, v in a.items()}
    pt = {k: torch.from_numpy(v).cuda() for k, v in p.items()}
    y, z = gnn.norm_residual_forward(t["x"], t["o"], t["gate"], kind=kind, eps=eps, **pt, **kw)
    has = z is not None
    g = gnn.norm_residual_backward(y if has else None, t["o"], t["dy"], t["dz"] if has else None,
                                   t["gate"], kind=kind, eps=eps, **pt, **kw)
    torch.cuda.synchronize()
    return y, z, g


def check(n, F, dtype, kind, gate, seed=1, offset=0.0, params=PARAMS, what="", eps=1e-6):
    a, p = data(n, F, dtype, gate, seed, offset, params)
    kinds = (kind, kind) if isinstance(kind, str) else kind
    if kinds[0] == "none":
        p = {k: v for k, v in p.items() if not k.endswith("_post")}
    if kinds[1] == "none":
        p = {k: v for k, v in p.items() if not k.endswith("_pre")}
    y, z, g = run(a, p, dtype, kind, eps)
    w = {k: wide(v) for k, v in a.items()}
    half = layer_ref.HALF[dtype]
    ry, by, rz, bz = layer_ref.norm_residual(w["x"], w["o"], w["gate"], p, kinds, eps)
    layer_ref.hold(to_f64(y), ry, by + half * np.abs(ry) * (1 + half) + 1e-37, what + " y")
    if rz is None:
        assert z is None
    else:
        layer_ref.hold(to_f64(z), rz, bz + half * (np.abs(rz) + bz) + 1e-37, what + " z")
    ref = layer_ref.norm_residual_grads(to_f64(y), w["o"], w["gate"], w["dy"], w["dz"], p, kinds,
                                        eps)
    for k, (v, b) in ref.items():
        if k[1:] in PARAMS and k[1:] not in p:
            assert g[k] is None
            continue
        h = 0.0 if k[1:] in PARAMS else half
        layer_ref.hold(to_f64(g[k]), v, b + h * (np.abs(v) + b) + 2 * layer_ref.U * np.abs(v)
                       + 1e-37, f"{what} {k}")
    return y, z, g


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("kind", ["rms", "layer", ("none", "rms"), ("layer", "none"),
                                  ("rms", "layer"), ("none", "none")], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_kinds_and_gates(dtype, kind, gate):
    check(333, 64, dtype, kind, gate, what=f"{kind} {gate}")


@pytest.mark.gpu
@pytest.mark.parametrize("n, F, dtype", [
    (1, 4, "f32"), (1, 8, "bf16"), (7, 12, "f32"), (1000, 20, "f32"), (513, 40, "bf16"),
    (300, 128, "f32"), (300, 132, "f32"), (65, 256, "bf16"), (65, 264, "bf16"),
    (33, 512, "f32"), (33, 260, "f32"), (17, 1024, "bf16"), (129, 520, "bf16"),
    (20_011, 8, "bf16"), (60_001, 24, "bf16"), (40_000, 320, "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sizes(n, F, dtype, kind):
    check(n, F, dtype, kind, "element", seed=F, what=f"{n} {F}")


@pytest.mark.gpu
@pytest.mark.parametrize("params", [(), ("scale",), ("w_post", "w_pre"), ("b_post", "b_pre")],
                         ids=lambda p: "+".join(p) or "none")
def test_parameters_left_out(params):
    check(200, 48, "f32", "layer", "row", params=params, what=str(params))


@pytest.mark.gpu
def test_rows_far_from_zero():
    """A layer norm of rows whose mean is a thousand times their spread."""
    check(500, 128, "f32", "layer", "element", offset=3000.0, what="offset")


@pytest.mark.gpu
def test_constant_and_zero_rows_and_saturated_gates():
    import graph_neural_network_gb300 as gnn
    x = torch.zeros(4, 16, device="cuda")
    o = torch.tensor([0.0, 2.0, -1.0, 5.0], device="cuda")[:, None].expand(4, 16).contiguous()
    gate = torch.tensor([-200.0, 200.0, float("inf"), float("-inf")], device="cuda")[:, None]
    gate = gate.contiguous()
    y, z = gnn.norm_residual_forward(x, o, gate, kind="layer")
    assert not y.any() and not z.any()          # differences from the mean are zero
    y, z = gnn.norm_residual_forward(x, o, gate, kind=("none", "rms"))
    assert not y[0].any() and torch.equal(y[1], o[1]) and torch.equal(y[2], o[2])
    assert not y[3].any() and torch.isfinite(z).all()
    g = gnn.norm_residual_backward(y, o, x + 1, x + 1, gate, kind=("none", "rms"))
    for k in ("dx", "do", "dgate"):
        assert torch.isfinite(g[k]).all(), k
    assert not g["dgate"].any()


@pytest.mark.gpu
def test_no_rows():
    import graph_neural_network_gb300 as gnn
    x = torch.zeros(0, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    y, z = gnn.norm_residual_forward(x, x, w_post=w)
    g = gnn.norm_residual_backward(y, x, x, x, w_post=w,
                                   grads={"dw_post": torch.full((32,), 5.0, device="cuda")})
    assert y.shape == z.shape == (0, 32) and not g["dw_post"].any()


@pytest.mark.gpu
def test_reproducible_streams_and_capture():
    a, p = data(50_000, 96, "bf16", "element")
    first = run(a, p, "bf16", "rms")
    again = run(a, p, "bf16", "rms")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = run(a, p, "bf16", "rms", stream=side)
    import graph_neural_network_gb300 as gnn
    t = {k: to_device(v, "bf16") for k, v in a.items()}
    pt = {k: torch.from_numpy(v).cuda() for k, v in p.items()}
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        y, z = gnn.norm_residual_forward(t["x"], t["o"], t["gate"], **pt)
        g = gnn.norm_residual_backward(y, t["o"], t["dy"], t["dz"], t["gate"], **pt)
    cg.replay()
    cg.replay()
    torch.cuda.synchronize()
    for b in (again, other, (y, z, g)):
        assert torch.equal(first[0], b[0]) and torch.equal(first[1], b[1])
        for k in first[2]:
            assert torch.equal(first[2][k], b[2][k]), k


@pytest.mark.gpu
def test_autograd_and_differences():
    """Through autograd the gradients are the direct call's; a central
    difference with step h differs from them by h^2 / 6 times the third
    derivative (at most 64 / std^3 times the magnitudes here, std >= 0.5) and by
    the sums' rounding over h."""
    import graph_neural_network_gb300 as gnn
    a, p = data(6, 16, "f32", "element", seed=5)
    t = {k: to_device(v, "f32").requires_grad_(True) for k, v in a.items()}
    pt = {k: torch.from_numpy(v).cuda().requires_grad_(True) for k, v in p.items()}
    args = [t["x"], t["o"], t["gate"]] + [pt[k] for k in PARAMS]
    y, z = gnn.NormResidual.apply(*args, "layer", 1e-6)
    got = torch.autograd.grad([y, z], args, [t["dy"].detach(), t["dz"].detach()])
    _, _, g = run(a, p, "f32", "layer")
    for name, v in zip(("dx", "do", "dgate") + tuple("d" + k for k in PARAMS), got):
        assert torch.equal(v, g[name].reshape(v.shape)), name
    w = {k: wide(v) for k, v in a.items()}

    def loss(**over):
        v = {**w, **over}
        y, _, z, _ = layer_ref.norm_residual(v["x"], v["o"], v["gate"], p, ("layer",) * 2, 1e-6)
        return float((y * w["dy"] + z * w["dz"]).sum())

    h = 2.0 ** -12   # in float64: h^2 terms about 1e-5 of the magnitudes, rounding 1e-12
    for name, key in (("x", "dx"), ("o", "do"), ("gate", "dgate")):
        for at in ((0, 0), (3, 7), (5, 15)):
            f = []
            for s in (h, -h):
                v = w[name].copy()
                v[at] += s
                f.append(loss(**{name: v}))
            want = (f[0] - f[1]) / (2 * h)
            mag = np.abs(w["dy"][at[0]]).max() + np.abs(w["dz"][at[0]]).max()
            assert abs(float(g[key][at]) - want) <= h * h / 6 * 64 * 8 * mag + 2e-5 * mag



def test_refusals_on_the_host():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build, _native
    build.build()
    lib = _native.load()
    P = ctypes.c_void_p
    a, ws = P(256), 1 << 30

    def desc(**kw):
        return _native.NormResidual(**{**dict(n=4, F=16, post=1, pre=1, gate_width=0, eps=1e-6),
                                       **kw})

    def fwd(d, gate=None, z=a, dt=0, x=a):
        return lib.gnn_norm_residual_forward(ctypes.byref(d), dt, x, a, gate, a, z, None)

    assert lib.gnn_norm_residual_forward(None, 0, a, a, None, a, a, None) == 1
    for bad in (dict(n=-1), dict(F=0), dict(post=3), dict(pre=-1), dict(gate_width=2),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(post=0, w_post=256), dict(post=0, b_post=256), dict(w_post=258)):
        assert fwd(desc(**bad)) == _native.ERR_INVALID_ARG, bad
    for bad in (dict(pre=0, w_pre=256), dict(pre=0)):                # a z without its norm
        assert fwd(desc(**bad)) == _native.ERR_INVALID_ARG, bad
    assert fwd(desc(), dt=2) == _native.ERR_INVALID_ARG
    assert fwd(desc(), gate=a) == _native.ERR_INVALID_ARG            # a gate of width 0
    assert fwd(desc(gate_width=16)) == _native.ERR_INVALID_ARG       # no gate
    assert fwd(desc(), z=None) == _native.ERR_INVALID_ARG
    assert fwd(desc(), x=None) == _native.ERR_INVALID_ARG
    assert fwd(desc(), x=P(264)) == _native.ERR_INVALID_ARG          # misaligned
    for F, dt in ((6, 0), (12, 1), (516, 0), (1032, 1)):
        assert fwd(desc(F=F), dt=dt) == _native.ERR_UNSUPPORTED, (F, dt)
        assert lib.gnn_norm_residual_workspace_bytes(ctypes.byref(desc(F=F)), dt) == 0
    d = desc()
    need = lib.gnn_norm_residual_workspace_bytes(ctypes.byref(d), 0)
    assert need > 0
    gr = _native.NormGrads(dx=256, dout=256)

    def bwd(d=d, y=a, gate=None, dz=a, gr=gr, ws=a, size=need):
        return lib.gnn_norm_residual_backward(ctypes.byref(d), 0, y, a, gate, a, dz,
                                              None if gr is None else ctypes.byref(gr), ws, size,
                                              None)

    assert bwd(size=need - 1) == _native.ERR_WORKSPACE_TOO_SMALL
    assert bwd(ws=P(264)) == _native.ERR_INVALID_ARG
    assert bwd(gr=None) == _native.ERR_INVALID_ARG
    assert bwd(gr=_native.NormGrads(dx=256)) == _native.ERR_INVALID_ARG
    assert bwd(gr=_native.NormGrads(dx=256, dout=256, dgate=256)) == _native.ERR_INVALID_ARG
    assert bwd(gr=_native.NormGrads(dx=256, dout=256, dscale=258)) == _native.ERR_INVALID_ARG
    assert bwd(y=None) == _native.ERR_INVALID_ARG
    assert bwd(dz=None) == _native.ERR_INVALID_ARG
    # the binding: host tensors, kinds, shapes
    x = torch.zeros(4, 16)
    for call in (lambda: gnn.norm_residual_forward(x, x), lambda: gnn.norm_residual_forward(x, 3),
                 lambda: gnn.norm_residual_backward(x, x, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        gnn.norm_residual_forward(x, x.double())


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import graph_neural_network_gb300 as gnn
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    for kw, err in ((dict(kind="batch"), ValueError), (dict(gate=x[:, :2]), ValueError),
                    (dict(gate=x.bfloat16()), TypeError), (dict(w_post=w[:8]), ValueError),
                    (dict(w_post=w.int()), TypeError), (dict(y=x[:2]), ValueError),
                    (dict(kind=("rms", "none"), z=x), ValueError),
                    (dict(kind=("none", "rms"), w_post=w), gnn.GnnError),
                    (dict(eps=0.0), gnn.GnnError), (dict(scale=w.cpu()), ValueError)):
        with pytest.raises(err):
            gnn.norm_residual_forward(x, x, **kw)
    with pytest.raises(ValueError):
        gnn.norm_residual_forward(x, x.t().contiguous().t())
    with pytest.raises(ValueError):
        gnn.norm_residual_backward(x, x, x, x, grads={"dgate": x})
    with pytest.raises(ValueError):
        gnn.norm_residual_backward(x, x, x, x, grads={"dnothing": x})
    with pytest.raises(TypeError):
        gnn.norm_residual_backward(x, x, x, None)


@pytest.mark.gpu
def test_parameter_sums_over_many_rows():
    """400k rows, some 660 of them a thread.  The terms of db_pre are dz itself, so its
    error is that of the additions alone.  An addition into a partial sum of k
    random terms is off by u / sqrt(3) of it at most on average, so m of them in a row
    by u sqrt(m / 6) of their sum: 3.3 u for 64, 1.3 u for the 11 parts after them,
    3.6 u together (one chain of 660: 10.5 u, and the partial sums of a thread lie
    anywhere in their binades, which takes a third off each)."""
    import graph_neural_network_gb300 as gnn
    n, F = 400_000, 512
    gen = torch.Generator("cuda").manual_seed(3)
    o, y, dy, dz = (torch.randn(n, F, generator=gen, device="cuda") for _ in range(4))
    w = torch.ones(F, device="cuda")
    got = gnn.norm_residual_backward(y, o, dy, dz, None, w, w_pre=w, b_pre=w)["db_pre"].double()
    want = torch.stack([t.double().sum(0) for t in dz.split(50_000)]).sum(0)
    error = (got - want).norm() / want.norm()
    assert error <= 4 * 2.0 ** -24, float(error)
