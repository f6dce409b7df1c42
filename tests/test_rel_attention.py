"""Graph-transformer attention with a learned relative position bias: the CUDA
path against a plain float64 implementation, with bounds derived from the
rounding of its sums (layer_ref)."""
import numpy as np
import pytest
import torch

import layer_ref
import workload
from workload import testgraphs
from gpu_util import device_graph, to_device, to_f64

pytestmark = pytest.mark.gpu

DEGREES = [0, 1, 2, 3, 7, 8, 9, 16, 17, 63, 64, 65, 129, 257, 1000, 2049, 4097]
NAMES = ("out", "lse", "dq", "dkey", "dval", "dbias")


def features(n, H, D, dtype, seed, streams=(1, 5, 6, 4)):
    arrs = [workload.normal_f32(seed, s, (n, H, D), 1.0) for s in streams]
    return [workload.f32_to_bf16_bits(x) for x in arrs] if dtype == "bf16" else arrs


def wide(x):
    return (workload.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def positions(n, seed, span):
    return np.random.default_rng(seed).integers(-span, span, n, dtype=np.int32)


def edge_buckets(rp, ci, pos, bounds, two_sided):
    dst = np.repeat(np.arange(len(rp) - 1), np.diff(rp))
    return layer_ref.bucket_of(pos[ci].astype(np.int64) - pos[dst], bounds, two_sided)


def run(g, rel, feats, bias, dtype, scale=None):
    import graph_neural_network_gb300 as gnn
    q, k, v, dout = (to_device(x, dtype) for x in feats)
    b = torch.from_numpy(bias).cuda()
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b, scale)
    grads = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, dout, scale)
    torch.cuda.synchronize()
    assert gnn.check_device_error(g) == 0
    return dict(zip(NAMES, (out, lse) + grads))


def check(rp, ci, H, D, dtype, tiling=None, buckets=32, dist=128, two=True, bounds=None, seed=3,
          bias=None, feats=None, pos=None, what=""):
    import graph_neural_network_gb300 as gnn
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci), tiling)
    pos = positions(n, seed, 3 * dist) if pos is None else pos
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), buckets, dist, two, bounds=bounds)
    bucket = edge_buckets(rp, ci, pos, rel.bounds, two)
    csr, csc = rel.arrays()
    assert np.array_equal(csr.cpu().numpy(), bucket)
    if bias is None:
        bias = workload.normal_f32(seed, 7, (rel.buckets, H), 1.0)
    feats = features(n, H, D, dtype, seed) if feats is None else feats
    got = run(g, rel, feats, bias, dtype)
    q, k, v, dout = (wide(x) for x in feats)
    ref = layer_ref.attention(rp, ci, q, k, v, D ** -0.5, bias, bucket, dout)
    layer_ref.hold_attention({x: to_f64(t) for x, t in got.items()}, ref, dtype, what, NAMES)
    return g, rel, got, feats, bias


@pytest.mark.parametrize("tiling", [(64, 4096, 2048), (8, 64, 16), (0, 0, 1)],
                         ids=lambda t: "t%d_%d_%d" % t)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_bucket_path(dtype, tiling):
    rp, ci = testgraphs.with_in_degrees(DEGREES, n_nodes=1500, seed=7)
    check(rp, ci, 4, 8 if dtype == "f32" else 16, dtype, tiling, what=f"{tiling}")


SHAPES = [(1, 4, "f32", 32), (3, 4, "f32", 6), (32, 4, "f32", 128), (4, 32, "f32", 2),
          (1, 128, "f32", 64), (1, 8, "bf16", 128), (32, 8, "bf16", 128), (5, 16, "bf16", 32),
          (3, 64, "bf16", 18), (4, 64, "bf16", 64), (1, 256, "bf16", 32)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "H%d_D%d_%s_B%d" % s)
def test_shapes(shape):
    H, D, dtype, B = shape
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=500, seed=H * 100 + D)
    one = B == 2
    check(rp, ci, H, D, dtype, (8, 64, 16), buckets=B, two=not one, dist=200, seed=17, what=f"{shape}")


def test_one_sided_and_given_bounds():
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=400, seed=5)
    check(rp, ci, 2, 16, "f32", buckets=17, dist=90, two=False, what="one-sided")
    check(rp, ci, 2, 16, "f32", two=True, bounds=[0], what="the sign alone")
    check(rp, ci, 2, 16, "f32", two=False, bounds=[0, 1, 1, 4, 40], what="an empty bucket")


def test_extreme_positions():
    rp, ci = testgraphs.with_in_degrees([3] * 40, n_nodes=60, seed=5)
    far = np.array([-2**31, 2**31 - 1, 0, 1, -1, 2**30], np.int32)
    pos = far[np.random.default_rng(1).integers(0, len(far), 60)]
    check(rp, ci, 2, 16, "f32", pos=pos, buckets=64, dist=2**31 - 1, what="far")


@pytest.mark.parametrize("rows", [[[0]], [[], [], []], [[1], []], [[0, 0, 0]]],
                         ids=["one", "no edges", "two", "multi-edge"])
def test_smallest_graphs(rows):
    rp, ci = testgraphs.csr_from_rows(rows)
    check(rp, ci, 2, 8, "bf16", what="small")


def test_no_nodes():
    import graph_neural_network_gb300 as gnn
    g = device_graph(dict(row_ptr=np.zeros(1, np.int32), col=np.zeros(0, np.int32)))
    rel = gnn.RelPos(g, torch.zeros(0, dtype=torch.int32, device="cuda"))
    x = torch.zeros(0, 2, 8, device="cuda")
    b = torch.zeros(32, 2, device="cuda")
    out, lse = gnn.transformer_rel_forward(g, rel, x, x, x, b)
    db = torch.full((32, 2), 7.0, device="cuda")
    gnn.transformer_rel_backward(g, rel, x, x, x, b, lse, x, dbias=db)
    assert out.shape == (0, 2, 8) and lse.shape == (0, 2) and not db.any()


@pytest.mark.parametrize("H,D,dtype", [(2, 16, "f32"), (8, 16, "bf16"), (1, 128, "bf16")])
def test_masked_buckets_with_anything_behind_them(H, D, dtype):
    """Every bucket of later sources masked: rows of early nodes are left with
    nothing, and rows that only masked edges reach hold infinities and NaN."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 1, 2, 9, 70, 300, 700], n_nodes=300, seed=11)
    n = len(rp) - 1
    pos = np.random.default_rng(2).permutation(n).astype(np.int32)
    last = int(np.argmax(pos))                     # as a source, later than all others
    ci = np.where(ci == last, (last + 1) % n, ci).astype(np.int32)
    dst = np.repeat(np.arange(n), np.diff(rp))
    ci[::7] = np.where(dst[::7] != last, last, ci[::7])
    bias = workload.normal_f32(3, 7, (32, H), 1.0)
    bias[16:] = -np.inf
    bias[3, 0] = -np.inf                           # and one bucket of one head alone
    feats = features(n, H, D, dtype, 5)
    g, rel, clean, _, _ = check(rp, ci, H, D, dtype, (8, 64, 16), feats=feats, pos=pos, bias=bias,
                                dist=128, what="masked")
    bad = [x.copy() for x in feats]
    nan, inf = (0x7FC0, 0xFF80) if dtype == "bf16" else (np.nan, -np.inf)
    bad[1][last], bad[2][last, :, ::2], bad[2][last, :, 1::2] = nan, inf, nan
    got = run(g, rel, bad, bias, dtype)
    for x in NAMES:
        if x == "dq":   # its own row of keys enters nowhere either
            pass
        assert torch.equal(got[x], clean[x]), x
    assert torch.isneginf(got["lse"]).any()


def test_all_masked():
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=400, seed=5)
    bias = np.full((32, 2), -np.inf, np.float32)
    _, _, got, _, _ = check(rp, ci, 2, 16, "f32", (8, 64, 16), bias=bias, what="all masked")
    assert not got["out"].any() and not got["dval"].any() and not got["dbias"].any()


def test_zero_bias_is_the_plain_attention():
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300, 5000], n_nodes=900, seed=5)
    g, rel, got, feats, _ = check(rp, ci, 4, 32, "bf16", bias=np.zeros((32, 4), np.float32),
                                  what="zero")
    q, k, v, dout = (to_device(x, "bf16") for x in feats)
    out, lse = gnn.transformer_forward(g, q, k, v)
    dq, dk, dv = gnn.transformer_backward(g, q, k, v, lse, dout)
    C = 2.0 ** -7   # two roundings to bfloat16, each half a step
    for a, b in ((got["out"], out), (got["dq"], dq), (got["dkey"], dk), (got["dval"], dv)):
        assert float((a.float() - b.float()).abs().max()) <= C * float(b.float().abs().max())


def test_reproducible_streams_and_capture():
    import graph_neural_network_gb300 as gnn
    rp, ci = workload.chung_lu(20_000, 2.1, 15.0, 6_000.0, 29)
    g, rel, a, feats, bias = check(rp, ci, 2, 16, "f32", seed=9, what="power law")
    for _ in range(3):
        b = run(g, rel, feats, bias, "f32")
        for x in NAMES:
            assert torch.equal(a[x], b[x]), x
    q, k, v, dout = (to_device(x, "f32") for x in feats)
    bt = torch.from_numpy(bias).cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, bt, stream=side)
    gr = gnn.transformer_rel_backward(g, rel, q, k, v, bt, lse, dout, stream=side)
    side.synchronize()
    for x, t in zip(NAMES, (out, lse) + gr):
        assert torch.equal(a[x], t), x
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, bt)
        gr = gnn.transformer_rel_backward(g, rel, q, k, v, bt, lse, dout)
    for _ in range(2):
        cg.replay()
    torch.cuda.synchronize()
    for x, t in zip(NAMES, (out, lse) + gr):
        assert torch.equal(a[x], t), x


def test_autograd_and_differences():
    """Central differences of a float64 sum of the outputs: with step h the
    quotient is off by h^2 / 6 times the third derivative (products of at most
    three softmax weights and the values: below 8 times the gradient's own
    magnitude sum) and by the outputs' rounding over 2 h."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([4] * 30, n_nodes=30, seed=5)
    g = device_graph(dict(row_ptr=rp, col=ci))
    pos = positions(30, 1, 20)
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), 8, 16, True)
    feats = features(30, 2, 8, "f32", 3)
    q, k, v, dout = (to_device(x, "f32").requires_grad_(True) for x in feats)
    b = torch.from_numpy(workload.normal_f32(3, 7, (8, 2), 1.0)).cuda().requires_grad_(True)
    y = gnn.TransformerRelAggregate.apply(g, rel, q, k, v, b, None)
    y.backward(dout.detach())
    bucket = edge_buckets(rp, ci, pos, rel.bounds, True)
    ref = layer_ref.attention(rp, ci, *(wide(x) for x in feats[:3]), 8 ** -0.5,
                              b.detach().cpu().numpy(), bucket, wide(feats[3]))
    got = dict(dq=q.grad, dkey=k.grad, dval=v.grad, dbias=b.grad)
    layer_ref.hold_attention({x: to_f64(t) for x, t in got.items()}, ref, "f32", "autograd",
                             list(got))
    h = 2.0 ** -6
    noise = ref["C"] * float((ref["out_mag"] * np.abs(wide(feats[3]))).sum())
    with torch.no_grad():
        for at in [(0, 0), (3, 1), (7, 0)]:
            f = []
            for sign in (h, -h):
                bb = b.detach().clone()
                bb[at] += sign
                f.append(float((gnn.transformer_rel_forward(g, rel, q, k, v, bb)[0].double()
                                * dout.double()).sum()))
            bound = h * h / 6 * 8 * ref["dbias_mag"][at] + noise / h
            assert abs((f[0] - f[1]) / (2 * h) - ref["dbias"][at]) <= bound


def test_refusals():
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([2] * 6, n_nodes=6, seed=5)
    g, g2 = (device_graph(dict(row_ptr=rp, col=ci)) for _ in range(2))
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    for kw, err in ((dict(num_buckets=7), ValueError), (dict(num_buckets=130), gnn.GnnError),
                    (dict(num_buckets=32, max_distance=8), gnn.GnnError),
                    (dict(bounds=[1, 2]), gnn.GnnError), (dict(bounds=[0, 3, 2]), gnn.GnnError),
                    (dict(bounds=[]), gnn.GnnError),
                    (dict(bounds=list(range(65))), gnn.GnnError)):
        with pytest.raises(err):
            gnn.RelPos(g, pos, **kw)
    rel = gnn.RelPos(g, pos)
    x = torch.zeros(6, 2, 8, device="cuda")
    b = torch.zeros(32, 2, device="cuda")
    with pytest.raises(ValueError):
        gnn.transformer_rel_forward(g2, rel, x, x, x, b)
    with pytest.raises(ValueError):
        gnn.transformer_rel_forward(g, rel, x, x, x, b[:, :1])
    with pytest.raises(gnn.GnnError):
        gnn.transformer_rel_forward(g, rel, x, x, x, b,
                                    ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    wide_row = torch.zeros(6, 1, 256, device="cuda")
    with pytest.raises(gnn.GnnError):
        gnn.transformer_rel_forward(g, rel, wide_row, wide_row, wide_row, b[:, :1].contiguous())


@pytest.mark.parametrize("H,D,dtype", [(4, 32, "f32"), (4, 64, "bf16"), (2, 8, "f32")])
def test_rows_on_odd_16_byte_boundaries(H, D, dtype):
    """Tensors that start 16 bytes past a 32-byte boundary give the same within
    the bounds (both are held to them), and the workspace serves either."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([0, 5, 70, 300], n_nodes=500, seed=5)
    g, rel, got, feats, bias = check(rp, ci, H, D, dtype, (8, 64, 16), what="aligned")
    n = len(rp) - 1

    def moved(x):
        t = to_device(x, dtype)
        pad = 16 // t.element_size()
        room = torch.empty(t.numel() + pad, dtype=t.dtype, device="cuda")
        v = room[pad:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    q, k, v, dout = (moved(x) for x in feats)
    b = torch.from_numpy(bias).cuda()
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
    gr = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, dout)
    bucket = rel.arrays()[0].cpu().numpy()
    ref = layer_ref.attention(rp, ci, *(wide(x) for x in feats[:3]), D ** -0.5, bias, bucket,
                              wide(feats[3]))
    layer_ref.hold_attention({x: to_f64(t) for x, t in zip(NAMES, (out, lse) + gr)}, ref, dtype,
                             "odd", NAMES)
    packed = gnn.pack8(q, k, v)
    at = [p.values.cpu().numpy() * p.scale.cpu().numpy().astype(np.float64)[..., None]
          for p in packed]
    g8 = gnn.transformer_backward8(g, *packed, dout, rel=rel, bias=b)
    ref = layer_ref.attention(rp, ci, *at, D ** -0.5, bias, bucket, wide(feats[3]))
    names = ("dq", "dkey", "dval", "dbias")
    layer_ref.hold_attention({x: to_f64(t) for x, t in zip(names, g8)}, ref, dtype, "odd 8", names)


@pytest.mark.parametrize("make", [testgraphs.star_in, testgraphs.star_out], ids=["in", "out"])
def test_one_node_with_every_edge(make):
    """A node whose edges run through all workers, as destination and as source."""
    rp, ci = make(30_000)
    check(rp, ci, 2, 16, "f32", what="star")
    check(rp, ci, 4, 64, "bf16", what="star")


def test_positions_and_bounds_outside_32_bits_are_refused():
    import graph_neural_network_gb300 as gnn
    g = device_graph(dict(row_ptr=np.zeros(7, np.int32), col=np.zeros(0, np.int32)))
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    for kw in (dict(bounds=[0, 2 ** 32 + 5]), dict(bounds=[0, -1]), dict(max_distance=2 ** 32 + 64),
               dict(max_distance=0)):
        with pytest.raises(ValueError):
            gnn.RelPos(g, pos, **kw)


def test_bias_gradient_is_no_worse_than_its_terms():
    """Six million edges, most into 2 x 4 sums: the error stays that of the terms, however
    long the columns that add them.  A term de = alpha (da - Delta) carries the
    rounding of a dot product of 64 products in each factor, of the exponential
    and of two subtractions, all of random sign: under ten half steps in the root
    of the mean square, which N independent terms keep as sqrt(sum de^2)."""
    import graph_neural_network_gb300 as gnn
    n, deg, H, D = 300_000, 20, 4, 64
    gen = torch.Generator("cuda").manual_seed(5)
    rp = torch.arange(0, n * deg + 1, deg, dtype=torch.int32, device="cuda")
    ci = torch.randint(n, (n * deg,), generator=gen, device="cuda", dtype=torch.int32)
    pos = torch.randint(1 << 16, (n,), generator=gen, device="cuda", dtype=torch.int32)
    g = gnn.Graph(rp, ci)
    rel = gnn.RelPos(g, pos, 32, 128)          # nearly every edge in the two last buckets
    q, k, v, d = (torch.randn(n, H, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
    b = torch.randn(32, H, generator=gen, device="cuda")
    _, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
    got = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, d)[3].double()
    bucket = rel.arrays()[0].long().view(n, deg)
    want, square = (torch.zeros(32, H, dtype=torch.float64, device="cuda") for _ in range(2))
    step = 25_000
    for r in range(0, n, step):
        at, j = bucket[r:r + step], ci.view(n, deg)[r:r + step].long()
        for h in range(H):
            own = lambda t: t[r:r + step, None, h].double()  # noqa: E731
            e = (own(q) * k[:, h].double()[j]).sum(-1) * D ** -0.5 + b[:, h].double()[at]
            al = torch.softmax(e, 1)
            da = (own(d) * v[:, h].double()[j]).sum(-1)
            de = al * (da - (al * da).sum(1, keepdim=True))
            want[:, h].index_add_(0, at.reshape(-1), de.reshape(-1))
            square[:, h].index_add_(0, at.reshape(-1), (de * de).reshape(-1))
    error = (got - want).norm() / square.sum().sqrt()
    assert error <= 10 * 2.0 ** -24, float(error)
