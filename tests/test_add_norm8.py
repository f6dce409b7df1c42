"""The sum with the residual and its root-mean-square norm in 8 bits: the CUDA path
against a plain float64 implementation.

y is a float32 sum rounded to the type: exact.  The 8-bit values are decided by the exact
quotient of the float32 t = y w and its group's scale s: exact too.  U = 2^-24:

scale.  A row's sum of squares is added in float32 over at most 8 elements, 4 vectors, 5
levels of a warp and 16 warps, each square rounded with its addition: a relative error
of 33 U at most, half of it in the root, and rsqrtf is within 2 units of its last
place (4 U); eps and the mean add 2 U and two products 2 U.  So 25 U.

backward.  rstd as above, 25 U; y^ = y rstd 26 U.  mean(g y^): products and sums as
for the squares, 35 U of the sum of magnitudes, and the factors' 27 U.  dx's two terms
are then off by 28 U rstd |g| and (26 + 27 + 35 + 25 + 4) U rstd |y^| mean |g y^|, and its
additions by 3 U of what is added.  dw: 27 U a term, a thread's sum of its m rows m U, the
threads' and the blocks' sums (float64 or compensated, 2 U, each rounded) 4 U."""
import ctypes

import numpy as np
import pytest
import torch

import layer_ref
import workload
from gpu_util import to_device, to_f64

U = 2.0 ** -24
TOP = {"int8": 127.0, "e4m3": 448.0}
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def draw(seed, *shape, dtype="f32", std=1.0):
    x = workload.normal_f32(seed, 1, shape, std)
    return workload.f32_to_bf16_bits(x) if dtype == "bf16" else x


def wide(x):
    return workload.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x


def eight(fmt, q):
    """q (float64) rounded to the nearest value of the format, ties to even."""
    if fmt == "int8":
        return np.rint(q)
    a = np.abs(q)
    lo = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 125)
    below, above = a - E4M3[lo], E4M3[lo + 1] - a
    return np.copysign(E4M3[lo + ((above < below) | ((above == below) & (lo % 2 == 1)))], q)


def reference(x, o, w, fmt, group, eps):
    """y, values, and the scales in float64, from float32 x, o, w."""
    y = x if o is None else x + o
    t = (y if w is None else y * w).reshape(len(x), -1, group)
    assert t.dtype == np.float32
    s = (np.abs(t).max(-1).astype(np.float64) / TOP[fmt]).astype(np.float32)
    s = np.maximum(s, np.float32(2.0 ** -126)).astype(np.float64)
    values = eight(fmt, t.astype(np.float64) / s[..., None])
    rstd = 1 / np.sqrt((y.astype(np.float64) ** 2).mean(-1) + eps)
    return y, values, s * rstd[:, None]


def run(x, o, w, dtype, fmt, group, eps=1e-6, **kw):
    import graph_neural_network_gb300 as gnn
    t = [None if a is None else to_device(a, dtype) for a in (x, o)]
    wt = None if w is None else torch.from_numpy(w).cuda()
    return gnn.add_norm8_forward(*t, wt, fmt=fmt, group=group, eps=eps, **kw)


def values_of(z8):
    return z8.values.to(torch.float32).double().cpu().numpy()


def check_forward(x, o, w, dtype, fmt, group, eps=1e-6, what=""):
    import graph_neural_network_gb300 as gnn
    y, z8 = run(x, o, w, dtype, fmt, group, eps)
    ry, rv, rs = reference(wide(x), None if o is None else wide(o), w, fmt, group or x.shape[1],
                           eps)
    if o is None:
        assert y is None
    else:
        want = torch.from_numpy(ry).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        assert np.array_equal(to_f64(y), to_f64(want)), what
    assert np.array_equal(values_of(z8), rv), what
    layer_ref.hold(to_f64(z8.scale), rs, 25 * U * rs + 2.0 ** -149, what + " scale")
    for dt in (torch.float32, torch.bfloat16):
        if z8.values.shape[2] % (4 if dt == torch.float32 else 8) == 0:
            back = gnn.unpack8(z8, dt)
            assert torch.equal(back, (z8.values.float() * z8.scale[..., None]).to(dt)), what
    return y, z8


SHAPES = [  # n, F, group, dtype
    (1, 4, None, "f32"), (1, 8, None, "bf16"), (3, 12, 4, "f32"), (1000, 20, None, "f32"),
    (77, 40, 8, "bf16"), (333, 64, 32, "f32"), (129, 128, 128, "f32"), (65, 256, 64, "bf16"),
    (130, 264, None, "bf16"), (70, 512, 256, "bf16"), (31, 520, 8, "bf16"), (50, 512, None, "f32"),
    (9, 516, 4, "f32"), (40, 1024, 128, "bf16"), (5, 1032, None, "bf16"), (17, 2048, 16, "bf16"),
    (4, 2056, None, "bf16"), (6, 4096, 256, "bf16"), (3, 4104, None, "bf16"),
    (3, 4104, 8, "bf16"), (2, 8192, 128, "f32"), (3, 8188, None, "f32"), (2, 16384, 128, "bf16"),
    (1, 16376, None, "bf16"), (40_003, 8, None, "bf16"), (30_001, 96, 32, "bf16")]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n, F, group, dtype", SHAPES)
def test_forward(n, F, group, dtype, fmt):
    w = (1 + draw(3, F, std=0.3)).astype(np.float32)
    x, o = draw(1, n, F, dtype=dtype, std=2.0), draw(2, n, F, dtype=dtype)
    check_forward(x, o, w, dtype, fmt, group, what=f"{n} {F}")
    check_forward(x, None, None, dtype, fmt, group, what=f"{n} {F} alone")


@pytest.mark.gpu
@pytest.mark.parametrize("F", [32, 2112])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_quotients_next_to_a_border(F, fmt):
    """Rows whose elements lie on the borders between neighbouring 8-bit values times a
    scale, and one unit of their last place to either side."""
    values = np.arange(128.0) if fmt == "int8" else E4M3
    border = (values[1:] + values[:-1]) / 2
    rng = np.random.default_rng(1)
    rows = []
    for k in range(400):
        s = np.float32(2.0 ** rng.uniform(-20, 20)) if k % 2 else np.float32(2.0 ** (k % 9))
        b = np.float32(rng.choice(border, F) * np.float64(s))
        b = np.nextafter(b, np.float32(rng.choice([0.0, np.inf])) if k % 3 else b)
        b *= rng.choice([-1, 1], F).astype(np.float32)
        b[rng.integers(F)] = np.float32(TOP[fmt]) * s
        rows.append(b)
    x = np.array(rows, np.float32)
    check_forward(x, None, None, "f32", fmt, None, what="borders")
    check_forward(x, None, None, "f32", fmt, 32, what="borders, groups")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("F, group", [(16, None), (64, 16), (4096, None), (4096, 64)])
def test_zeros_extremes_and_numbers_that_are_none(F, group, fmt):
    """Zero rows, denormal rows, rows whose squares overflow or vanish, beside rows of
    their own warp that do not; infinities and NaN read back as NaN in their row alone."""
    import graph_neural_network_gb300 as gnn
    scales = [0.0, 1e-42, 1e-30, 1.0, 1e15, 3e19, 1e30, 5e37]
    x = draw(5, len(scales), F) * np.array(scales, np.float32)[:, None]
    x = np.clip(x, -3e38, 3e38).astype(np.float32)
    y, z8 = check_forward(x, None, None, "f32", fmt, group, what="sizes")
    assert not values_of(z8)[0].any()
    for bad in (np.inf, -np.inf, np.nan):
        b = x.copy()
        b[3, F - 1] = bad
        _, z = run(b, None, None, "f32", fmt, group)
        back = gnn.unpack8(z).reshape(len(x), F)
        assert torch.isnan(back[3]).all() and not z.values[3].float().any()
        keep = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(back[keep], gnn.unpack8(z8).reshape(len(x), F)[keep])
    # a sum that overflows, and a product that does (its group's alone)
    big = np.full((1, F), 3e38, np.float32)
    y, z = run(big, big, None, "f32", fmt, group)
    assert torch.isinf(y).all() and torch.isnan(z.scale).all()
    w = np.ones(F, np.float32)
    w[0] = 10.0
    _, z = run(big, None, w, "f32", fmt, group)
    assert torch.isnan(z.scale[0, 0]) and torch.isfinite(z.scale[0, 1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("F", [64, 520, 4096])
def test_in_place(F):
    """The sum written over x or o, rows whose squares overflow among them."""
    import graph_neural_network_gb300 as gnn
    x, o = (to_device(draw(s, 9, F, dtype="bf16"), "bf16") for s in (1, 2))
    x[4] *= 1e25
    want, z = gnn.add_norm8_forward(x, o, fmt="e4m3")
    assert torch.isfinite(z.scale).all()
    for k in (0, 1):
        t = [x.clone(), o.clone()]
        y, z8 = gnn.add_norm8_forward(*t, fmt="e4m3", y=t[k])
        assert y is t[k] and torch.equal(y, want) and torch.equal(z8.scale, z.scale)
        assert torch.equal(z8.values.view(torch.uint8), z.values.view(torch.uint8))


@pytest.mark.gpu
def test_values_are_those_of_pack8():
    import graph_neural_network_gb300 as gnn
    x, o = (to_device(draw(s, 500, 4 * 32, dtype="bf16"), "bf16") for s in (1, 2))
    _, z8 = gnn.add_norm8_forward(x.float(), o.float(), group=32)
    (p,) = gnn.pack8((x.float() + o.float()).view(500, 4, 32))
    assert torch.equal(z8.values, p.values)


@pytest.mark.gpu
def test_rows_of_several_dimensions_and_weights_in_another_type():
    import graph_neural_network_gb300 as gnn
    x, o, dz = (to_device(draw(s, 30, 4, 16), "f32") for s in (1, 2, 3))
    w = torch.from_numpy(1 + draw(4, 64, std=0.1)).cuda().double()
    y, z = gnn.add_norm8_forward(x, o, w, group=16)
    y2, z2 = gnn.add_norm8_forward(x.view(30, 64), o.view(30, 64), w.float(), group=16)
    assert y.shape == x.shape and torch.equal(y.view(30, 64), y2)
    assert z.values.shape == (30, 4, 16) and torch.equal(z.values, z2.values)
    dx, dw = gnn.add_norm8_backward(y, None, dz, w)
    assert dx.shape == x.shape and dw.dtype == torch.float32
    leaf = w.clone().requires_grad_(True)
    out = gnn.AddNorm8.apply(x, o, leaf, "int8", 16, 1e-6)
    (g,) = torch.autograd.grad(out[1], leaf, dz)
    assert out[1].shape == x.shape and g.dtype == torch.float64 and torch.equal(g, dw.double())


def check_backward(n, F, dtype, with_dy=True, with_w=True, std=2.0, what=""):
    import graph_neural_network_gb300 as gnn
    a = [draw(s, n, F, dtype=dtype, std=sd) for s, sd in ((1, std), (2, 1.0), (3, 1.0))]
    w = (1 + draw(4, F, std=0.3)).astype(np.float32) if with_w else None
    t = [to_device(v, dtype) for v in a]
    if not with_dy:
        t[1] = None
    wt = None if w is None else torch.from_numpy(w).cuda()
    dx, dw = gnn.add_norm8_backward(*t, wt)
    y, dy, dz = (wide(v).astype(np.float64) for v in a)
    if not with_dy:
        dy = 0 * dy
    w64 = 1.0 if w is None else w.astype(np.float64)
    rstd = 1 / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6)
    hat, g = y * rstd, dz * w64
    ref = dy + rstd * (g - hat * (g * hat).mean(-1, keepdims=True))
    mag = rstd * (np.abs(g) + np.abs(hat) * np.abs(g * hat).mean(-1, keepdims=True))
    bound = (117 + 6) * U * mag + 3 * U * np.abs(dy)
    half = layer_ref.HALF[dtype]
    layer_ref.hold(to_f64(dx), ref, bound + half * (np.abs(ref) + bound) + 1e-37, what + " dx")
    if w is None:
        assert dw is None
        return dx, dw
    rows = n  # of a thread: all of them at most
    layer_ref.hold(to_f64(dw), (dz * hat).sum(0),
                   (31 + min(rows, 400)) * U * np.abs(dz * hat).sum(0) + 1e-37, what + " dw")
    return dx, dw


@pytest.mark.gpu
@pytest.mark.parametrize("n, F, dtype", sorted({(n, F, d) for n, F, _, d in SHAPES}) + [
    (1500, 4104, "bf16"), (700, 8192, "f32"), (701, 16384, "bf16"), (20_000, 256, "f32"),
    (900, 2048, "bf16")])
def test_backward(n, F, dtype):
    check_backward(n, F, dtype, what=f"{n} {F}")


@pytest.mark.gpu
@pytest.mark.parametrize("with_dy, with_w", [(False, True), (True, False), (False, False)])
def test_backward_without(with_dy, with_w):
    for n, F, dtype in ((50, 24, "f32"), (50, 1032, "bf16")):
        check_backward(n, F, dtype, with_dy, with_w, what=f"{with_dy} {with_w}")


@pytest.mark.gpu
def test_backward_of_large_rows():
    """Rows whose squares overflow beside others of their warp: 1 / y is their factor."""
    import graph_neural_network_gb300 as gnn
    for F in (16, 2048):
        y = torch.from_numpy(draw(1, 6, F)).cuda()
        dz = torch.from_numpy(draw(2, 6, F)).cuda()
        y[1::2] *= 2.0 ** 100
        dx, _ = gnn.add_norm8_backward(y, None, dz)
        y[1::2] /= 2.0 ** 100
        want, _ = gnn.add_norm8_backward(y, None, dz, eps=1e-30)
        # scaled by powers of two; without eps the gradient scales with 1 / y
        a, b = dx[1::2].double() * 2.0 ** 100, want[1::2].double()
        assert (a - b).norm() <= 1e-6 * b.norm()
        assert torch.isfinite(dx).all() and dx[1::2].any()


@pytest.mark.gpu
def test_parameter_sums_over_many_rows():
    """400,000 rows, some 660 of them a thread.  An addition into a partial sum of k random
    terms is off by U / sqrt(3) of it at most on average, so m of them in a row by U sqrt(m / 6)
    of their sum: 3.3 U for 64, 1.3 U for the 11 parts after them; the terms themselves, products
    with y^, have errors of 1 U that are common to a row (rstd: they add up like the terms) and 1 U
    that are not: 1 U of the sum each at most.  Together, as squares: 3.9 U (one chain of 660:
    10.6 U)."""
    import graph_neural_network_gb300 as gnn
    n, F = 400_000, 512
    gen = torch.Generator("cuda").manual_seed(3)
    y, dz = (torch.randn(n, F, generator=gen, device="cuda") for _ in range(2))
    _, dw = gnn.add_norm8_backward(y, None, dz, torch.ones(F, device="cuda"))
    want = 0
    for a, b in zip(y.split(50_000), dz.split(50_000)):
        a = a.double()
        want = want + (b.double() * a * (a.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()).sum(0)
    error = (dw.double() - want).norm() / want.norm()
    assert error <= 4 * U, float(error)


@pytest.mark.gpu
def test_autograd_and_differences():
    """Straight through: the gradients are those of the norm itself, whose central
    differences in float64 agree to h^2 and the rounding of dx."""
    import graph_neural_network_gb300 as gnn
    n, F = 5, 24
    x, o, dy, dz = (torch.from_numpy(draw(s, n, F)).cuda() for s in range(1, 5))
    w = torch.from_numpy((1 + draw(9, F, std=0.2)).astype(np.float32)).cuda()
    leaves = [t.clone().requires_grad_(True) for t in (x, o, w)]
    y, z = gnn.AddNorm8.apply(*leaves, "e4m3", 8, 1e-6)
    y2, z8 = gnn.add_norm8_forward(x, o, w, fmt="e4m3", group=8)
    assert torch.equal(y, y2) and torch.equal(z, gnn.unpack8(z8).view(n, F))
    gx, go, gw = torch.autograd.grad([y, z], leaves, [dy, dz])
    dx, dw = gnn.add_norm8_backward(y2, dy, dz, w)
    assert torch.equal(gx, dx) and torch.equal(go, dx) and torch.equal(gw, dw)
    alone = gnn.AddNorm8.apply(leaves[0], None, None, "int8", None, 1e-6)
    (g1,) = torch.autograd.grad(alone, leaves[0], dz)
    assert torch.equal(g1, gnn.add_norm8_backward(x, None, dz)[0])
    x64, o64, w64, dy64, dz64 = (t.double().cpu() for t in (x, o, w, dy, dz))

    def loss(x_, w_):
        y_ = x_ + o64
        z_ = y_ * w_ / ((y_ * y_).mean(-1, keepdim=True) + 1e-6).sqrt()
        return float((y_ * dy64 + z_ * dz64).sum())

    h = 2.0 ** -12
    mag = float(dy.abs().max() + dz.abs().max())
    for at in ((0, 0), (2, 7), (4, 23)):
        d = torch.zeros_like(x64)
        d[at] = h
        diff = (loss(x64 + d, w64) - loss(x64 - d, w64)) / (2 * h)
        assert abs(float(dx[at]) - diff) <= h * h / 6 * 64 * 8 * mag + 2e-5 * mag
    d = torch.zeros_like(w64)
    d[3] = h
    diff = (loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * h)
    assert abs(float(dw[3]) - diff) <= 2e-5 * n * mag     # linear in w


@pytest.mark.gpu
def test_reproducible_streams_and_capture():
    import graph_neural_network_gb300 as gnn
    for n, F in ((20_001, 96), (600, 4104)):
        x, o, dz = (to_device(draw(s, n, F, dtype="bf16"), "bf16") for s in (1, 2, 3))
        w = torch.from_numpy(1 + draw(4, F, std=0.1)).cuda()

        def both(**kw):
            y, z = gnn.add_norm8_forward(x, o, w, fmt="e4m3", **kw)
            return (y, z.values.float(), z.scale, *gnn.add_norm8_backward(y, x, dz, w, **kw))

        first = both()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = both(stream=side)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            kept = both()
        cg.replay()
        cg.replay()
        torch.cuda.synchronize()
        for r in (both(), other, kept):
            assert all(torch.equal(a, b) for a, b in zip(first, r))


@pytest.mark.gpu
def test_no_rows():
    import graph_neural_network_gb300 as gnn
    x, w = torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, z = gnn.add_norm8_forward(x, x, w, group=16)
    assert y.shape == (0, 64) and z.values.shape == (0, 4, 16) and z.scale.shape == (0, 4)
    assert gnn.unpack8(z).shape == (0, 4, 16)
    dx, dw = gnn.add_norm8_backward(x, x, x, w, dw=torch.full((64,), 3.0, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    import graph_neural_network_gb300 as gnn
    n, F = (1 << 31) // 4096 + 9, 4096
    x = torch.zeros(n, F, dtype=torch.bfloat16, device="cuda")
    x[-32:] = to_device(draw(1, 32, F, dtype="bf16"), "bf16")
    w = torch.ones(F, device="cuda")
    y, z = gnn.add_norm8_forward(x, x, w, group=128)
    y1, z1 = gnn.add_norm8_forward(x[-32:], x[-32:], w, group=128)
    assert torch.equal(y[-32:], y1) and torch.equal(z.values[-32:], z1.values)
    assert torch.equal(z.scale[-32:], z1.scale)
    back = gnn.unpack8(z, torch.bfloat16)
    assert torch.equal(back[-32:], gnn.unpack8(z1, torch.bfloat16))
    dx, _ = gnn.add_norm8_backward(y, y, x, w)
    assert torch.equal(dx[-32:], gnn.add_norm8_backward(y1, y1, x[-32:], w)[0])


def test_refusals_on_the_host():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build, _native
    build.build()
    lib = _native.load()
    P = 4096
    bad, no = _native.ERR_INVALID_ARG, _native.ERR_UNSUPPORTED

    def desc(**kw):
        return _native.AddNorm8(**{**dict(n=4, F=64, group=64, fmt=0, eps=1e-6), **kw})

    def fwd(d, dt=0, x=P, o=P, w=None, y=P, v=P, s=P):
        return lib.gnn_add_norm8_forward(ctypes.byref(d), dt, x, o, w, y, v, s, None)

    assert lib.gnn_add_norm8_forward(None, 0, P, P, None, P, P, P, None) == bad
    assert fwd(desc(n=0)) == _native.OK
    for kw in (dict(n=-1), dict(F=0), dict(group=0), dict(group=128), dict(group=48),
               dict(fmt=2), dict(fmt=-1), dict(eps=0.0), dict(eps=1e-31),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert fwd(desc(**kw)) == bad, kw
    for kw, dt in ((dict(F=6, group=6), 0), (dict(F=12, group=12), 1),
                   (dict(F=8196, group=8196), 0), (dict(F=16392, group=16392), 1),
                   (dict(F=96, group=12), 0), (dict(F=64, group=2), 0), (dict(F=512, group=256), 0),
                   (dict(F=64, group=4), 1)):
        assert fwd(desc(**kw), dt) == no, kw
        assert lib.gnn_add_norm8_workspace_bytes(ctypes.byref(desc(**kw)), dt) == 0
    assert fwd(desc(), dt=2) == bad
    for kw in (dict(x=None), dict(o=None), dict(y=None), dict(v=None), dict(s=None),
               dict(x=P + 8), dict(o=P + 8), dict(y=P + 8), dict(v=P + 8), dict(s=P + 2),
               dict(w=P + 4)):
        assert fwd(desc(), **kw) == bad, kw
    need = lib.gnn_add_norm8_workspace_bytes(ctypes.byref(desc()), 0)
    assert need > 0

    def bwd(d=None, y=P, dy=P, dz=P, w=P, dx=P, dw=P, ws=P, size=need):
        return lib.gnn_add_norm8_backward(ctypes.byref(d or desc()), 0, y, dy, dz, w, dx, dw, ws,
                                          size, None)

    assert bwd(size=need - 1) == _native.ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(y=None), dict(dz=None), dict(dx=None), dict(ws=None), dict(ws=P + 16),
               dict(y=P + 8), dict(dy=P + 8), dict(dw=P + 2), dict(w=P + 4)):
        assert bwd(**kw) == bad, kw

    def unpack(groups=4, group=64, fmt=0, dt=0, v=P, s=P, x=P):
        return lib.gnn_unpack8_groups(groups, group, fmt, dt, v, s, x, None)

    assert unpack(groups=0) == _native.OK and unpack(group=6) == no and unpack(group=12, dt=1) == no
    for kw in (dict(groups=-1), dict(group=0), dict(fmt=2), dict(dt=2), dict(v=None),
               dict(s=None), dict(x=None), dict(x=P + 8), dict(v=P + 2), dict(group=1 << 25),
               dict(groups=1 << 40)):
        assert unpack(**kw) == bad, kw
    x = torch.zeros(4, 64)
    for call in (lambda: gnn.add_norm8_forward(x), lambda: gnn.add_norm8_backward(x, x, x),
                 lambda: gnn.add_norm8_forward(3)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import graph_neural_network_gb300 as gnn
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for kw, err in ((dict(fmt="int4"), ValueError), (dict(group=48), ValueError),
                    (dict(group=0), ValueError), (dict(group=2), gnn.GnnError),
                    (dict(o=x[:2]), ValueError), (dict(o=x.bfloat16()), TypeError),
                    (dict(y=x), ValueError), (dict(w=w[:8]), ValueError),
                    (dict(w=w.int()), TypeError), (dict(w=w.cpu()), ValueError),
                    (dict(eps=0.0), gnn.GnnError), (dict(out=x), TypeError),
                    (dict(out=gnn.Packed8(x, x)), ValueError)):
        with pytest.raises(err):
            gnn.add_norm8_forward(x, **kw)
    with pytest.raises(ValueError):
        gnn.add_norm8_forward(x.t())
    with pytest.raises(TypeError):
        gnn.add_norm8_forward(x.double())
    for args, kw, err in (((x, x[:1], x), {}, ValueError), ((x, x, None), {}, TypeError),
                          ((x, x, x), dict(dw=w), ValueError),
                          ((x, x, x, w), dict(ws=w), ValueError),
                          ((x, x, x, w), dict(ws=torch.empty(16, dtype=torch.uint8,
                                                             device="cuda")), gnn.GnnError)):
        with pytest.raises(err):
            gnn.add_norm8_backward(*args, **kw)
    with pytest.raises(TypeError):
        gnn.unpack8(gnn.Packed8(x.view(4, 8, 8).half(), x[:, :8]))
