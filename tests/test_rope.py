"""Rotary positions: the CUDA path against a plain float64 implementation whose angles
are exact fractions.

Bounds, U = 2^-24.  An angle's fraction of a turn is cut at 2^-32 and converted to
float32: off by at most pi 2^-25 + 2 pi 2^-32 < 1.7 U.  Sine and cosine add a unit of
their last place, 2 U at most, and the product with the amplitude m another U m: 4.7 U m
each.  a cos t - b sin t rounds a product and a sum: 2 U m (|a| + |b|) more.  So an
output is off by at most 7 U m (|a| + |b|), and the rounding of the type."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import layer_ref
import workload
from gpu_util import to_device, to_f64

U = 2.0 ** -24
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def angles(pos, freqs):
    """pos * freq less whole turns, in exact fractions, as float64 [n, half]."""
    f = [Fraction(x) for x in freqs]
    return np.array([[float((int(p) * x) % TWO_PI) for x in f] for p in pos]).reshape(
        len(pos), len(f))


def rotated(x, t, dim, layout, m, sign=1.0):
    """x [n, H, D] float64; the rotation and its bound before the type's rounding."""
    out, bound = x.copy(), np.zeros_like(x)
    at = (slice(0, dim // 2), slice(dim // 2, dim)) if layout == "half" else \
        (slice(0, dim, 2), slice(1, dim, 2))
    a, b = x[..., at[0]], x[..., at[1]]
    c, s = m * np.cos(t)[:, None], sign * m * np.sin(t)[:, None]
    out[..., at[0]], out[..., at[1]] = a * c - b * s, a * s + b * c
    bound[..., at[0]] = bound[..., at[1]] = 7 * U * abs(m) * (abs(a) + abs(b))
    return out, bound


def draw(seed, *shape, dtype="f32"):
    x = workload.normal_f32(seed, 1, shape, 1.0)
    return workload.f32_to_bf16_bits(x) if dtype == "bf16" else x


def wide(x):
    return (workload.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def check(xs, pos, rope, dtype, got, inverse=False, what=""):
    t = angles(pos, rope.freqs)
    for k, (x, y) in enumerate(zip(xs, got)):
        ref, bound = rotated(wide(x), t, rope.dim, rope.layout, rope.amplitude,
                             -1.0 if inverse else 1.0)
        half = layer_ref.HALF[dtype]
        rest = np.zeros_like(bound)
        rest[..., :rope.dim] = half * (np.abs(ref) + bound)[..., :rope.dim]
        layer_ref.hold(to_f64(y), ref, bound + rest + 1e-37 * (bound > 0), f"{what} {k}")


def positions(n, seed=3, lo=-2 ** 31, hi=2 ** 31 - 1):
    p = np.random.default_rng(seed).integers(lo, hi, n, dtype=np.int64)
    p[:4] = (0, hi, lo, 1)[:len(p[:4])]
    return p.astype(np.int32)


# ---- host ---------------------------------------------------------------------------

def test_frequencies_of_the_rules():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build
    build.build()
    plain = gnn.Rope(64)
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert np.allclose(plain.freqs, want, rtol=1e-15) and plain.amplitude == 1.0
    assert np.allclose(gnn.Rope(64, scaling="linear", factor=4.0).freqs, np.array(want) / 4,
                       rtol=1e-15)
    base = 10000.0 * 4.0 ** (64 / 62)
    ntk = gnn.Rope(64, scaling="ntk", factor=4.0).freqs
    assert np.allclose(ntk, [base ** (-2 * i / 64) for i in range(32)], rtol=1e-14)
    assert abs(ntk[-1] * 4 / want[-1] - 1) < 1e-12          # the slowest pair: as if linear
    yarn = gnn.Rope(64, scaling="yarn", factor=16.0, length=4096)
    low = math.floor(64 * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(1e4)))
    high = math.ceil(64 * math.log(4096 / (2 * math.pi)) / (2 * math.log(1e4)))
    r = np.array(yarn.freqs) / want
    assert np.allclose(r[:low + 1], 1, rtol=1e-15) and np.allclose(r[high:], 1 / 16, rtol=1e-14)
    assert (np.diff(r[low:high + 1]) < 0).all()
    assert yarn.amplitude == np.float32(0.1 * math.log(16) + 1)
    own = gnn.Rope(6, freqs=[0.5, -2.0, 0.0], amplitude=0.25)
    assert own.freqs == [0.5, -2.0, 0.0] and own.amplitude == 0.25
    # a fraction of a turn in 64 bits; a negative frequency's complement
    for f, w in zip(own.freqs, own._c.turns):
        off = (Fraction(w, 2 ** 64) - (Fraction(f) / TWO_PI) % 1) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 62)


def test_refusals_on_the_host():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build, _native
    build.build()
    lib = _native.load()
    for kw in (dict(dim=3), dict(dim=0), dict(dim=258), dict(dim=8, layout="full"),
               dict(dim=8, scaling="cubic"), dict(dim=8, factor=2.0),
               dict(dim=8, scaling="yarn", factor=2.0), dict(dim=8, freqs=[1.0]),
               dict(dim=2, freqs=[1.0], scaling="linear")):
        with pytest.raises(ValueError):
            gnn.Rope(**kw)
    for kw in (dict(dim=8, base=1.0), dict(dim=8, base=float("inf")),
               dict(dim=8, scaling="linear", factor=0.5), dict(dim=2, scaling="ntk", factor=2.0),
               dict(dim=8, scaling="yarn", factor=2.0, length=0.0),
               dict(dim=8, scaling="yarn", factor=2.0, length=64, fast=1.0),
               dict(dim=2, freqs=[float("nan")]), dict(dim=2, freqs=[2.0 ** 31]),
               dict(dim=2, amplitude=float("inf"))):
        with pytest.raises(gnn.GnnError):
            gnn.Rope(**kw)
    rope = gnn.Rope(8)
    P = 4096

    assert ctypes.sizeof(_native.RopeRows) == 56

    def packed(rows):    # as the binding lays them out
        whole = _native.ROPE_ROWS[len(rows)]()
        ctypes.memmove(whole, (_native.RopeRows * len(rows))(*rows), ctypes.sizeof(whole))
        return whole

    one = _native.RopeRows(1, 2, 3, 4, 5, 6, 7)
    assert list(packed([one])) == [1, 2, 3, 4, 5, 6, 7]

    def call(rows=None, n=4, D=16, pos=P, count=None, dt=0, inverse=0, c=rope._c):
        rows = [_native.RopeRows(P, 2 * P, 32, 16, 32, 16, 2)] if rows is None else rows
        return lib.gnn_rope_apply(None if c is None else ctypes.byref(c), inverse, n, D, pos,
                                  len(rows) if count is None else count,
                                  packed(rows), dt, None)

    bad = _native.ERR_INVALID_ARG
    assert call(n=0) == _native.OK and call(n=0, pos=None) == _native.OK
    assert call(c=None) == bad and call(n=-1) == bad and call(n=2 ** 31) == bad
    assert call(D=6) == bad and call(D=65537) == bad and call(dt=2) == bad
    assert call(inverse=2) == bad and call(pos=None) == bad and call(pos=P + 2) == bad
    assert call(count=0) == bad and call(count=9) == bad
    R = _native.RopeRows
    for row in (R(None, P, 32, 16, 32, 16, 2), R(P, None, 32, 16, 32, 16, 2),
                R(P + 2, P, 32, 16, 32, 16, 2), R(P, P + 2, 32, 16, 32, 16, 2),
                R(P, 2 * P, 32, 16, 32, 16, 0), R(P, 2 * P, 32, 16, 32, 16, 65537),
                R(P, 2 * P, 32, 16, 0, 16, 2), R(P, 2 * P, 32, 16, 31, 16, 2),
                R(P, 2 * P, 32, 16, 32, 15, 2), R(P, 2 * P, 32, 16, 16, 63, 2),
                R(P, 2 * P, 2 ** 60, 16, 32, 16, 2), R(P, P, 64, 16, 32, 16, 2)):
        assert call([row]) == bad
    twice = R(P, 2 * P, 32, 16, 32, 16, 2)
    assert call([twice, twice]) == bad
    # an output that is another tensor's input: both calls would read what the other writes
    there, back = R(P, 2 * P, 32, 16, 32, 16, 2), R(2 * P, P, 32, 16, 32, 16, 2)
    assert call([there, back]) == bad and call([R(P, P, 32, 16, 32, 16, 2), there]) == bad
    broken = _native.Rope.from_buffer_copy(rope._c)
    broken.dim = 7
    assert call(c=broken) == bad
    x = torch.zeros(4, 2, 16)
    with pytest.raises(ValueError):
        gnn.rope_forward(rope, torch.zeros(4, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        gnn.rope_forward(rope, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError):
        gnn.rope_forward(None, torch.zeros(4, dtype=torch.int32), x)


# ---- GPU ----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n, heads, D, dim, dtype", [
    (1, (1,), 2, 2, "f32"), (1, (32, 8), 128, 128, "bf16"), (5, (3, 1), 16, 16, "f32"),
    (33, (4, 4), 64, 32, "bf16"), (7, (2,), 10, 6, "bf16"), (9, (5,), 20, 20, "bf16"),
    (6, (3,), 80, 40, "bf16"), (6, (3,), 36, 4, "f32"), (3, (2, 7), 6, 2, "f32"),
    (17, (2,), 256, 256, "f32"), (4, (1,), 300, 256, "bf16"), (300, (1,) * 8, 16, 8, "f32"),
    (3, (2,), 2048, 16, "f32"), (2, (1, 3), 4098, 6, "bf16"), (20_011, (12, 3), 64, 48, "bf16"),
    (30_001, (5, 1, 2), 64, 64, "f32"), (70_001, (2, 1), 8, 8, "bf16")])
def test_sizes(n, heads, D, dim, dtype, layout):
    import graph_neural_network_gb300 as gnn
    rope = gnn.Rope(dim, layout, amplitude=1.25)
    pos = positions(n) if n < 10_000 else positions(n, hi=400, lo=-400)
    if n > 10_000:   # angles once for each position
        pos = np.sort(pos)
    xs = [draw(10 + k, n, H, D, dtype=dtype) for k, H in enumerate(heads)]
    ts = [to_device(x, dtype) for x in xs]
    pt = torch.from_numpy(pos).cuda()
    got = gnn.rope_forward(rope, pt, *ts)
    back = gnn.rope_backward(rope, pt, *ts)
    torch.cuda.synchronize()
    if n > 10_000:
        pick = np.r_[0:40, n // 2:n // 2 + 40, n - 40:n]
        xs, pos = [x[pick] for x in xs], pos[pick]
        got, back = [y[pick] for y in got], [y[pick] for y in back]
    check(xs, pos, rope, dtype, got, what="forward")
    check(xs, pos, rope, dtype, back, True, what="backward")
    for x, y in zip(xs, got):
        assert np.array_equal(to_f64(y)[..., dim:], wide(x)[..., dim:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 24])
def test_views_and_in_place(dtype, dim):
    """Views of fused projections, head-major tensors, rows that start anywhere, and a
    rotation in place give what contiguous tensors give; nothing else is written."""
    import graph_neural_network_gb300 as gnn
    n, H, D = 37, 3, 64
    rope = gnn.Rope(dim, scaling="ntk", factor=3.0)
    pt = torch.from_numpy(positions(n)).cuda()
    flat = to_device(draw(4, n * 3 * H * D + 1, dtype=dtype), dtype)
    views = {"projection": flat[:-1].view(n, 3, H, D)[:, 1],
             "heads": flat[:-1].view(n, H, 3, D)[:, :, 2],
             "head-major": flat[:n * H * D].view(H, n, D).transpose(0, 1),
             "odd start": flat[1:1 + n * H * D].view(n, H, D),
             "part of a row": flat[:n * 2 * H * D].view(n, H, 2 * D)[..., 3:3 + D],
             "one row for all": flat[:H * D].view(1, H, D).expand(n, H, D)}
    for name, v in views.items():
        (want,) = gnn.rope_forward(rope, pt, v.contiguous())
        (got,) = gnn.rope_forward(rope, pt, v)
        assert torch.equal(got, want), name
        if name == "one row for all":
            with pytest.raises(gnn.GnnError):
                gnn.rope_forward(rope, pt, v.contiguous(), out=[v])
            continue
        whole = flat.clone()
        place = torch.as_strided(whole, v.shape, v.stride(), v.storage_offset())
        gnn.rope_forward(rope, pt, place, out=[place])
        assert torch.equal(place, want), name
        place.copy_(v)
        assert torch.equal(whole, flat), name


@pytest.mark.gpu
def test_two_views_of_one_tensor_in_place():
    """q and key of a fused projection, rotated where they lie in one call."""
    import graph_neural_network_gb300 as gnn
    n, H, D = 45, 3, 32
    rope = gnn.Rope(16, "interleaved")
    pt = torch.from_numpy(positions(n)).cuda()
    qkv = to_device(draw(4, n, 3, H, D, dtype="bf16"), "bf16")
    want = gnn.rope_forward(rope, pt, qkv[:, 0], qkv[:, 1])
    val = qkv[:, 2].clone()
    got = gnn.rope_forward(rope, pt, qkv[:, 0], qkv[:, 1], out=[qkv[:, 0], qkv[:, 1]])
    assert got[0].data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, 0], want[0]) and torch.equal(qkv[:, 1], want[1])
    assert torch.equal(qkv[:, 2], val)


@pytest.mark.gpu
def test_scores_depend_on_the_difference_of_positions():
    """q at p and key at p - d: their product turns by d alone, wherever p lies."""
    import graph_neural_network_gb300 as gnn
    n, D = 64, 128
    for layout in ("half", "interleaved"):
        rope = gnn.Rope(D, layout)
        q, k = (to_device(draw(s, 1, 1, D), "f32").expand(n, 1, D) for s in (1, 2))
        p = torch.arange(n, dtype=torch.int32, device="cuda") * 33_000_000
        a, b = (gnn.rope_forward(rope, p - d, t)[0].double() for t, d in ((q, 0), (k, 71)))
        score = (a * b).sum(-1).flatten()
        mag = (q.double().norm(dim=-1) * k.double().norm(dim=-1)).flatten()
        # each side's vector is off by 7 U (|a| + |b|) an element: 14 U of its norm
        assert ((score - score[0]).abs() <= 2 * 2 * 14 * U * mag).all()


@pytest.mark.gpu
def test_autograd_streams_capture_and_differences():
    import graph_neural_network_gb300 as gnn
    n, D = 21, 32
    rope = gnn.Rope(16, "interleaved", scaling="yarn", factor=4.0, length=64)
    pt = torch.from_numpy(positions(n, lo=0, hi=500)).cuda()
    qkv = to_device(draw(7, n, 3, 2, D), "f32").requires_grad_(True)
    q, k = gnn.RotaryPositions.apply(rope, pt, qkv[:, 0], qkv[:, 1])
    dq, dk = (to_device(draw(8 + s, n, 2, D), "f32") for s in (0, 1))
    (g,) = torch.autograd.grad([q, k], qkv, [dq, dk])
    want = gnn.rope_backward(rope, pt, dq, dk)
    assert torch.equal(g[:, 0], want[0]) and torch.equal(g[:, 1], want[1]) and not g[:, 2].any()
    # the map is linear: its gradient along a direction is the difference itself, and
    # the two sums agree but for the rounding of both rotations
    x = to_device(draw(9, n, 2, D), "f32")
    (y,) = gnn.rope_forward(rope, pt, x)
    left, right = (y.double() * dq.double()).sum(), (x.double() * want[0].double()).sum()
    mag = 2 * rope.amplitude * float(x.double().norm() * dq.double().norm())
    assert abs(float(left - right)) <= 2 * 14 * U * mag
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = gnn.rope_forward(rope, pt, x, dq, stream=side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        kept = gnn.rope_forward(rope, pt, x, dq)
    cg.replay()
    cg.replay()
    torch.cuda.synchronize()
    assert torch.equal(other[0], y) and torch.equal(kept[0], y) and torch.equal(kept[1], other[1])


@pytest.mark.gpu
def test_no_nodes_and_refusals_of_the_binding():
    import graph_neural_network_gb300 as gnn
    rope = gnn.Rope(8)
    x = torch.zeros(4, 2, 8, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert gnn.rope_forward(rope, pos[:0], x[:0])[0].shape == (0, 2, 8)
    for args, err in (((rope, pos.long(), x), TypeError), ((rope, pos[:3], x), ValueError),
                      ((rope, pos.cpu(), x), ValueError), ((rope, pos, x.half()), TypeError),
                      ((rope, pos, x[..., :6]), ValueError), ((rope, pos, x[:, :0]), ValueError),
                      ((rope, pos, x[..., ::2].expand(4, 2, 4)), ValueError),
                      ((rope, pos, x, x.bfloat16()), TypeError),
                      ((rope, pos, x, x[:3]), ValueError), ((rope, pos, *[x] * 9), ValueError),
                      ((rope, pos, x.transpose(1, 2).contiguous().transpose(1, 2)), ValueError)):
        with pytest.raises(err):
            gnn.rope_forward(*args)
    with pytest.raises(ValueError):
        gnn.rope_forward(rope, pos, x, out=[x, x])
    with pytest.raises(ValueError):
        gnn.rope_forward(rope, pos, x, out=[x[:, :1]])
    y = torch.empty_like(x)
    with pytest.raises(gnn.GnnError):
        gnn.rope_forward(rope, pos, x, x, out=[y, y])
    with pytest.raises(ValueError):
        gnn.transformer_layer(None, x, x, x, x, rope=rope)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last nodes of tensors of more than 2^31 elements, strided and contiguous."""
    import graph_neural_network_gb300 as gnn
    n, D = (1 << 31) // (3 * 256) + 5, 256
    rope = gnn.Rope(128)
    x = torch.empty(n, 3, 1, D, dtype=torch.bfloat16, device="cuda")
    tail = to_device(draw(2, 64, 3, 1, D, dtype="bf16"), "bf16")
    x[-64:] = tail
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    (y,) = gnn.rope_forward(rope, pos, x[:, 2])
    (want,) = gnn.rope_forward(rope, pos[-64:], tail[:, 2])
    assert torch.equal(y[-64:], want)
    gnn.rope_forward(rope, pos, x[:, 2], out=[x[:, 2]])
    assert torch.equal(x[-64:, 2], want) and torch.equal(x[-64:, :2], tail[:, :2])


@pytest.mark.gpu
def test_in_a_layer():
    """transformer_layer's rotation is RotaryPositions before it, forward and backward."""
    import graph_neural_network_gb300 as gnn
    from workload import testgraphs
    from gpu_util import device_graph
    rp, ci = testgraphs.with_in_degrees([3] * 40, n_nodes=40, seed=1)
    g = device_graph(dict(row_ptr=rp, col=ci))
    n, H, D = 40, 2, 16
    rope = gnn.Rope(8, scaling="linear", factor=2.0)
    pos = torch.from_numpy(positions(n, lo=0, hi=10_000)).cuda()
    grads = []
    for inside in (True, False):
        qkv = to_device(draw(5, n, 3, H, D), "f32").requires_grad_(True)
        x = to_device(draw(6, n, H * D), "f32").requires_grad_(True)
        q, k, v = qkv.unbind(1)
        if inside:
            y, z = gnn.transformer_layer(g, x, q, k, v, rope=rope, pos=pos)
        else:
            q, k = gnn.RotaryPositions.apply(rope, pos, q, k)
            y, z = gnn.transformer_layer(g, x, q, k, v)
        grads.append(torch.autograd.grad((y * z).sum(), [qkv, x]) + (y, z))
    for a, b in zip(*grads):
        assert torch.equal(a, b)
