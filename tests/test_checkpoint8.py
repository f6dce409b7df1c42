"""8-bit activation checkpoints and the attention's backward pass from them:
packing against the exact rounding of the quotient, the backward pass against a
plain float64 implementation at the values the checkpoints stand for
(layer_ref)."""
import ctypes

import numpy as np
import pytest
import torch

import layer_ref
import workload
from workload import testgraphs
from gpu_util import device_graph, to_device, to_f64
from test_rel_attention import DEGREES, edge_buckets, features, positions, wide

NAMES = ("dq", "dkey", "dval")


def exact_pack(x):
    """Integers and scales of x [..., D] (float64 holding float32 values): the
    scale is one division rounded to float32; the quotient's nearest integer is
    decided on residues, which float64 holds exactly (24 + 7 bits)."""
    s = np.maximum((np.abs(x).max(-1) / 127.0).astype(np.float32), np.float32(2.0 ** -126))
    s = s.astype(np.float64)[..., None]
    down = np.floor(x / s)
    down -= (x - down * s) < 0          # the quotient may have been rounded up to a whole number
    below, above = x - down * s, (down + 1) * s - x
    up = (above < below) | ((above == below) & (down % 2 != 0))
    return (down + up).astype(np.int8), s[..., 0].astype(np.float32)


def borderline(n, H, D, seed):
    """Float32 vectors whose entries lie next to the halves of their scale."""
    rng = np.random.default_rng(seed)
    top = rng.uniform(0.5, 2.0, (n, H, 1)).astype(np.float32)
    top *= np.float32(2.0) ** rng.integers(-20, 20, (n, H, 1)).astype(np.float32)
    s = (top.astype(np.float64) / 127).astype(np.float32).astype(np.float64)
    x = (s * (rng.integers(-127, 127, (n, H, D)) + 0.5)).astype(np.float32)
    x = np.nextafter(x, x + rng.integers(-1, 2, x.shape).astype(np.float32) * np.abs(x))
    x[..., 0] = top[..., 0]
    return np.clip(x, -top, top).astype(np.float32)


def pack(x, dtype):
    import graph_neural_network_gb300 as gnn
    (p,) = gnn.pack8(to_device(x, dtype))
    torch.cuda.synchronize()
    return p


@pytest.mark.gpu
@pytest.mark.parametrize("n, H, D, dtype", [
    (1, 1, 4, "f32"), (1, 1, 8, "bf16"), (3, 5, 8, "f32"), (1001, 4, 32, "f32"),
    (77, 1, 128, "f32"), (501, 8, 16, "bf16"), (333, 4, 64, "bf16"), (41, 1, 256, "bf16"),
    (9, 127, 4, "f32"), (2, 8, 128, "bf16"), (300_001, 2, 8, "bf16")])
def test_pack_is_the_exact_rounding(n, H, D, dtype):
    import graph_neural_network_gb300 as gnn
    x = features(n, H, D, dtype, n + D, streams=(1,))[0]
    p = pack(x, dtype)
    want, s = exact_pack(wide(x))
    assert np.array_equal(p.values.cpu().numpy(), want)
    assert np.array_equal(p.scale.cpu().numpy(), s)
    v = want * s.astype(np.float64)[..., None]
    for dt, h in ((torch.float32, layer_ref.U), (torch.bfloat16, 2.0 ** -8)):
        layer_ref.hold(to_f64(gnn.unpack8(p, dt)), v, h * np.abs(v) * (1 + 2.0 ** -20), str(dt))
    assert np.all(np.abs(v - wide(x)) <= s.astype(np.float64)[..., None] / 2)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [4, 16, 128])
def test_pack_next_to_the_halves(D):
    x = borderline(20_000, 1, D, D)
    p = pack(x, "f32")
    want, s = exact_pack(x.astype(np.float64))
    assert np.array_equal(p.scale.cpu().numpy(), s)
    assert np.array_equal(p.values.cpu().numpy(), want)


@pytest.mark.gpu
def test_pack_special_values():
    import graph_neural_network_gb300 as gnn
    tiny, big = np.float32(1e-44), np.float32(3.4e38)
    rows = [[0, 0, 0, 0], [tiny, -tiny, 0, 0], [1e-38, 5e-39, -3e-40, 0], [big, -big, 1, 0],
            [np.inf, 1, 2, 3], [1, np.nan, 2, 3], [-np.inf, np.nan, 0, 0], [127, 0.5, 1.5, -2.5]]
    x = np.array(rows, np.float32).reshape(8, 1, 4)
    p = pack(x, "f32")
    v, s = p.values.cpu().numpy()[:, 0], p.scale.cpu().numpy()[:, 0]
    good = [0, 1, 2, 3, 7]
    want, ws = exact_pack(x[good].astype(np.float64))
    assert np.array_equal(v[good], want[:, 0]) and np.array_equal(s[good], ws[:, 0])
    assert v[7].tolist() == [127, 0, 2, -2]     # ties to even
    assert np.isnan(s[4:7]).all() and not v[4:7].any()
    back = gnn.unpack8(p).cpu().numpy()
    assert np.isnan(back[4:7]).all() and np.isfinite(back[good]).all()


@pytest.mark.gpu
def test_pack_several_and_streams_and_capture():
    import graph_neural_network_gb300 as gnn
    xs = [to_device(x, "bf16") for x in features(999, 3, 16, "bf16", 5)]
    one = [gnn.pack8(x)[0] for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    many = gnn.pack8(*xs, *xs, stream=side)
    side.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        cap = gnn.pack8(*xs)
        back = gnn.unpack8(cap[0], torch.bfloat16)
    cg.replay()
    torch.cuda.synchronize()
    for a, b in zip(one * 2 + one, many + cap):
        assert torch.equal(a.values, b.values) and torch.equal(a.scale, b.scale)
    assert torch.equal(back, gnn.unpack8(one[0], torch.bfloat16))
    given = tuple(gnn.Packed8(torch.empty_like(p.values), torch.empty_like(p.scale)) for p in one)
    assert gnn.pack8(*xs, out=given) == given and torch.equal(given[1].values, one[1].values)
    empty = torch.zeros(0, 3, 16, device="cuda")
    assert gnn.unpack8(gnn.pack8(empty)[0]).shape == (0, 3, 16)


def backward(g, packed, dout, dtype, rel=None, bias=None, **kw):
    import graph_neural_network_gb300 as gnn
    b = None if bias is None else torch.from_numpy(bias).cuda()
    got = gnn.transformer_backward8(g, *packed, to_device(dout, dtype), rel=rel, bias=b, **kw)
    torch.cuda.synchronize()
    assert gnn.check_device_error(g) == 0
    return dict(zip(NAMES + ("dbias",), got))


def check(rp, ci, H, D, dtype, tiling=None, with_rel=True, seed=3, bias=None, pos=None, what=""):
    import graph_neural_network_gb300 as gnn
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci), tiling)
    q, k, v, dout = features(n, H, D, dtype, seed)
    packed = gnn.pack8(*(to_device(x, dtype) for x in (q, k, v)))
    at = [p.values.cpu().numpy() * p.scale.cpu().numpy().astype(np.float64)[..., None]
          for p in packed]
    rel = bucket = None
    if with_rel:
        pos = positions(n, seed, 300) if pos is None else pos
        rel = gnn.RelPos(g, torch.from_numpy(pos).cuda())
        bucket = edge_buckets(rp, ci, pos, rel.bounds, True)
        bias = workload.normal_f32(seed, 7, (32, H), 1.0) if bias is None else bias
    got = backward(g, packed, dout, dtype, rel, bias)
    ref = layer_ref.attention(rp, ci, *at, D ** -0.5, bias, bucket, wide(dout))
    layer_ref.hold_attention({x: to_f64(t) for x, t in got.items()}, ref, dtype, what, list(got))
    return g, rel, packed, dout, bias, got


@pytest.mark.gpu
@pytest.mark.parametrize("with_rel", [False, True], ids=["plain", "rel"])
@pytest.mark.parametrize("tiling", [(64, 4096, 2048), (8, 64, 16), (0, 0, 1)],
                         ids=lambda t: "t%d_%d_%d" % t)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_bucket_path(dtype, tiling, with_rel):
    rp, ci = testgraphs.with_in_degrees(DEGREES, n_nodes=1500, seed=7)
    check(rp, ci, 4, 8 if dtype == "f32" else 16, dtype, tiling, with_rel, what=f"{tiling}")


@pytest.mark.gpu
@pytest.mark.parametrize("with_rel", [False, True], ids=["plain", "rel"])
@pytest.mark.parametrize("H, D, dtype", [
    (1, 4, "f32"), (32, 4, "f32"), (3, 8, "f32"), (4, 32, "f32"), (1, 128, "f32"), (1, 8, "bf16"),
    (32, 8, "bf16"), (5, 16, "bf16"), (16, 16, "bf16"), (3, 64, "bf16"), (4, 64, "bf16"),
    (1, 256, "bf16")])
def test_shapes(H, D, dtype, with_rel):
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=500, seed=H * 100 + D)
    check(rp, ci, H, D, dtype, (8, 64, 16), with_rel, seed=17, what=f"{H} {D}")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[[0]], [[], [], []], [[1], []], [[0, 0, 0]]],
                         ids=["one", "no edges", "two", "multi-edge"])
def test_smallest_graphs(rows):
    rp, ci = testgraphs.csr_from_rows(rows)
    check(rp, ci, 2, 8, "bf16", what="small")


@pytest.mark.gpu
@pytest.mark.parametrize("H, D, dtype", [(2, 16, "f32"), (8, 16, "bf16"), (1, 128, "bf16")])
def test_masked_buckets_with_anything_behind_them(H, D, dtype):
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 1, 2, 9, 70, 300, 700], n_nodes=300, seed=11)
    n = len(rp) - 1
    pos = np.random.default_rng(2).permutation(n).astype(np.int32)
    last = int(np.argmax(pos))
    ci = np.where(ci == last, (last + 1) % n, ci).astype(np.int32)
    dst = np.repeat(np.arange(n), np.diff(rp))
    ci[::7] = np.where(dst[::7] != last, last, ci[::7])
    bias = workload.normal_f32(3, 7, (32, H), 1.0)
    bias[16:] = -np.inf
    bias[3, 0] = -np.inf
    g, rel, packed, dout, bias, clean = check(rp, ci, H, D, dtype, (8, 64, 16), bias=bias,
                                              pos=pos, what="masked")
    for p in packed[1:]:                      # the key and value that only masked edges reach
        p.scale[last] = float("nan")
    got = backward(g, packed, dout, dtype, rel, bias)
    for x in got:
        assert torch.equal(got[x], clean[x]), x


@pytest.mark.gpu
def test_a_nan_stays_visible():
    """A checkpoint of a NaN poisons the gradients of every row that uses it."""
    rp, ci = testgraphs.csr_from_rows([[1, 2], [0, 1], [0, 1]])
    g, _, packed, dout, _, _ = check(rp, ci, 1, 16, "f32", with_rel=False, what="clean")
    packed[1].scale[2] = float("nan")         # key of node 2: row 0 attends to it
    got = backward(g, packed, dout, "f32")
    assert torch.isnan(got["dq"][0]).all() and torch.isfinite(got["dq"][1:]).all()
    assert torch.isnan(got["dval"][1]).any() and torch.isnan(got["dkey"][2]).all()
    assert torch.isfinite(got["dval"][0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1.0, 30.0])
def test_power_law_reproducible_streams_capture(spread):
    """Also with scores spread over hundreds, where the running maximum moves."""
    import graph_neural_network_gb300 as gnn
    rp, ci = workload.chung_lu(20_000, 2.1, 15.0, 6_000.0, 29)
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci))
    q, k, v, dout = features(n, 2, 16, "f32", 9)
    packed = gnn.pack8(*(to_device(x, "f32") for x in (q * np.float32(spread), k, v)))
    at = [p.values.cpu().numpy() * p.scale.cpu().numpy().astype(np.float64)[..., None]
          for p in packed]
    first = backward(g, packed, dout, "f32")
    ref = layer_ref.attention(rp, ci, *at, 0.25, dout=wide(dout))
    layer_ref.hold_attention({x: to_f64(t) for x, t in first.items()}, ref, "f32", "power",
                             list(NAMES))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = backward(g, packed, dout, "f32", stream=side)
    d = to_device(dout, "f32")
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        cap = dict(zip(NAMES, gnn.transformer_backward8(g, *packed, d)))
    cg.replay()
    cg.replay()
    torch.cuda.synchronize()
    for got in (other, cap, backward(g, packed, dout, "f32")):
        for x in NAMES:
            assert torch.equal(first[x], got[x]), x


@pytest.mark.gpu
def test_autograd_keeps_only_checkpoints():
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=400, seed=5)
    g, rel, packed, dout, bias, got = check(rp, ci, 2, 16, "f32", what="autograd")
    feats = features(400, 2, 16, "f32", 3)
    q, k, v = (to_device(x, "f32").requires_grad_(True) for x in feats[:3])
    b = torch.from_numpy(bias).cuda().requires_grad_(True)
    y = gnn.TransformerCheckpoint8.apply(g, rel, q, k, v, b, None)
    want, _ = gnn.transformer_rel_forward(g, rel, q.detach(), k.detach(), v.detach(), b.detach())
    assert torch.equal(y.detach(), want)
    y.backward(to_device(dout, "f32"))
    for x, t in zip(NAMES + ("dbias",), (q, k, v, b)):
        assert torch.equal(got[x], t.grad), x
    y = gnn.TransformerCheckpoint8.apply(g, None, q, k, v, None, None)
    d = torch.autograd.grad(y, (q, k, v), to_device(dout, "f32"))
    plain = backward(g, packed, dout, "f32")
    for x, t in zip(NAMES, d):
        assert torch.equal(plain[x], t), x


def test_refusals_on_the_host():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build, _native
    build.build()
    lib = _native.load()
    P = ctypes.c_void_p
    a, BAD, UNS = P(256), _native.ERR_INVALID_ARG, _native.ERR_UNSUPPORTED
    two = (P * 2)(256, 512)

    def pk(count=2, n=4, H=2, D=16, dt=0, x=two, v=two, s=two):
        return lib.gnn_pack8(count, n, H, D, dt, x, v, s, None)

    for kw in (dict(count=0), dict(count=9), dict(n=-1), dict(H=0), dict(dt=2), dict(x=None),
               dict(v=None), dict(s=None), dict(x=(P * 2)(256, None)),
               dict(x=(P * 2)(256, 264)), dict(v=(P * 2)(256, 264)), dict(s=(P * 2)(256, 258))):
        assert pk(**kw) == BAD, kw
    for kw in (dict(D=6), dict(D=48), dict(D=4, dt=1), dict(H=40)):
        assert pk(**kw) == UNS, kw
    assert pk(n=0) == _native.OK
    p = _native.Packed8(256, 512)
    assert lib.gnn_unpack8(4, 2, 16, 0, None, a, None) == BAD
    assert lib.gnn_unpack8(4, 2, 16, 0, ctypes.byref(_native.Packed8(256, None)), a, None) == BAD
    assert lib.gnn_unpack8(4, 2, 16, 0, ctypes.byref(_native.Packed8(264, 256)), a, None) == BAD
    assert lib.gnn_unpack8(4, 2, 16, 0, ctypes.byref(p), P(8), None) == BAD
    assert lib.transformer_packed8_workspace_bytes(None, None, 1, 16, 0) == 0
    r = ctypes.byref(p)
    assert lib.transformer_packed8_backward(None, None, 1, 16, 0, r, r, r, 1.0, None, a, a, a, a,
                                            None, a, 1 << 20, None) == BAD
    x = torch.zeros(4, 2, 16)
    for call in (lambda: gnn.pack8(), lambda: gnn.pack8(*[x] * 9), lambda: gnn.pack8(x),
                 lambda: gnn.pack8(x[0]), lambda: gnn.unpack8(gnn.Packed8(x, x)),
                 lambda: gnn.unpack8(x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([2] * 6, n_nodes=6, seed=5)
    g = device_graph(dict(row_ptr=rp, col=ci))
    x = torch.zeros(6, 2, 16, device="cuda")
    (p,) = gnn.pack8(x)
    rel = gnn.RelPos(g, torch.arange(6, dtype=torch.int32, device="cuda"))
    b = torch.zeros(32, 2, device="cuda")
    ok = (p, p, p, x)
    half = gnn.Packed8(p.values[:3], p.scale[:3])
    for args, kw, err in (
            ((x, p, p, x), {}, TypeError), ((half, p, p, x), {}, ValueError),
            ((gnn.Packed8(p.values.int(), p.scale), p, p, x), {}, TypeError),
            ((gnn.Packed8(p.values, p.scale[:, :1]), p, p, x), {}, ValueError),
            (ok, dict(rel=rel), ValueError), (ok, dict(bias=b), ValueError),
            (ok, dict(dbias=b), ValueError), (ok, dict(rel=rel, bias=b[:8]), ValueError),
            (ok, dict(dq=x[:2]), ValueError), ((p, p, p, x[:2]), {}, ValueError),
            (ok, dict(ws=torch.zeros(256, dtype=torch.uint8, device="cuda")), gnn.GnnError)):
        with pytest.raises(err):
            gnn.transformer_backward8(g, *args, **kw)
    with pytest.raises(ValueError):
        gnn.pack8(x, x, out=[p])
    with pytest.raises(TypeError):
        gnn.pack8(x, x.bfloat16())
    with pytest.raises(TypeError):
        gnn.unpack8(p, torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("H, D, dtype", [(32, 4, "f32"), (8, 16, "bf16"), (1, 8, "bf16"),
                                         (4, 64, "bf16")])
def test_most_buckets(H, D, dtype):
    """Tables of the bias gradient of every size, the widest one included."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=500, seed=H + D)
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci), (8, 64, 16))
    q, k, v, dout = features(n, H, D, dtype, 23)
    packed = gnn.pack8(*(to_device(x, dtype) for x in (q, k, v)))
    at = [p.values.cpu().numpy() * p.scale.cpu().numpy().astype(np.float64)[..., None]
          for p in packed]
    pos = positions(n, 23, 900)
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), 128, 1000)
    bucket = edge_buckets(rp, ci, pos, rel.bounds, True)
    bias = workload.normal_f32(23, 7, (128, H), 1.0)
    got = backward(g, packed, dout, dtype, rel, bias)
    ref = layer_ref.attention(rp, ci, *at, D ** -0.5, bias, bucket, wide(dout))
    layer_ref.hold_attention({x: to_f64(t) for x, t in got.items()}, ref, dtype, "128", list(got))
