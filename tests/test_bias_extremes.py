"""Finite biases of any size: the attention with a learned relative position bias
and its backward pass from checkpoints, against float64 with bounds that do not
grow with the bias or with lse.

Softmax weights depend on differences of scores only.  The reference takes the
biases of a row relative to the row's largest one before anything is rounded,
so it is exact to float64 at every bias; where a bias is 2^60 or more the score
beside it counts as 0, as evaluating their sum in float64 gives.

Bounds, with u = 2^-24, per edge e of row i, S_e = |scale| sum |q_c k_c|, B_i the
row's largest bias.  The scaled score carries (D + 6) u S_e, the difference from
the reference edge 4 u |b_e - B_i| (its rounding and that of log2(e)), the joining
of the two 2 u max S, the stored logarithm of the sum 2 u (max S + log2 deg).  The
sum of deg weights adds (deg + 8) u and its own terms' errors, the hardware's
exponentials and logarithm 2^-21.  A weight is therefore off by a factor 1 + w,
    w_e = x_e + max over the row of x + (deg + 8) u + 2^-21,
    x_e = u ((D + 6) S_e + 4 |b_e - B_i| + 4 max S + 2 log2 deg),
and everything after it adds D u for a dot product and one u per addition.  Where no bias
of the table is above 16, dot product and bias may be one float and so may lse: x_e has
4 u (|b_e| + |lse|) more, at most 4 u (32 + S + log deg).
"""
import numpy as np
import pytest
import torch

import layer_ref
import workload
from workload import testgraphs
from gpu_util import device_graph, to_device, to_f64
from test_rel_attention import edge_buckets, features, positions, run, wide

U = 2.0 ** -24
BIG = 2.0 ** 60
F32 = float(np.finfo(np.float32).max)
BF16 = 3.3895313892515355e38
VALUES = [-F32, -BF16, -1e30, -1e9, -1e6, -1e4, -1e2, -17.0, -16.0, 16.0, 17.0, 1e4, 1e9, 2.4e38,
          F32]
NAMES = ("dq", "dkey", "dval", "dbias")


def reference(rp, ci, q, k, v, dout, scale, bias, bucket):
    """{name: (value, bound)} of out, lse and the gradients, in float64."""
    n, H, D = q.shape
    i, j = np.repeat(np.arange(n), np.diff(rp)), np.asarray(ci, np.int64)
    heads = []
    for h in range(H):
        b = bias[bucket, h].astype(np.float64)
        keep = b > -np.inf
        I, J, B = i[keep], j[keep], b[keep]                    # noqa: E741
        qh, kh, vh, gh = q[:, h], k[:, h], v[:, h], dout[:, h]

        def over(idx, x, op=np.add, start=0.0):
            r = np.full((n,) + x.shape[1:], start)
            op.at(r, idx, x)
            return r

        deg, odeg = np.bincount(I, minlength=n), np.bincount(J, minlength=n)
        base = over(I, B, np.maximum, -np.inf)
        S = np.abs(scale) * np.abs(qh[I] * kh[J]).sum(-1)
        d = np.where(np.abs(B) >= BIG, 0.0, scale * (qh[I] * kh[J]).sum(-1))
        e = d + (B - base[I])
        top = over(I, e, np.maximum, -np.inf)
        p = np.exp(e - top[I])
        z = over(I, p)
        a = p / z[I]
        Smax = over(I, S, np.maximum, 0.0)[I]
        x = U * ((D + 6) * S + 4 * np.abs(B - base[I]) + 4 * Smax + 2 * np.log2(deg[I] + 1))
        if np.abs(bias[np.isfinite(bias)]).max(initial=0.0) <= 16:
            x = x + 4 * U * (32 + Smax + np.log(deg[I] + 1))
        # an edge below 2^-130 is flushed to zero (the absolute 1e-36 of hold())
        x = np.where(a > 2.0 ** -130, x, 0.0)
        w = x + over(I, x, np.maximum, 0.0)[I] + (deg[I] + 8) * U + 2.0 ** -21
        add = lambda idx, t: over(idx, t)                      # noqa: E731
        with np.errstate(divide="ignore"):
            lse = np.where(z > 0, np.log(np.where(z > 0, z, 1.0)) + np.where(
                z > 0, top + base, 0.0), -np.inf)
        r = {"lse": (lse, over(I, w, np.maximum, 0.0) + 2 * U * np.abs(np.where(z > 0, lse, 0)))}
        A, W = a[:, None], w[:, None]
        r["out"] = (add(I, A * vh[J]), add(I, (W + (deg[I] + 4)[:, None] * U) * A * np.abs(vh[J])))
        da, da_m = (gh[I] * vh[J]).sum(-1), np.abs(gh[I] * vh[J]).sum(-1)
        delta, delta_m = add(I, a * da), add(I, a * da_m)
        delta_e = add(I, a * da_m * (w + (deg[I] + D + 6) * U))
        de, de_m = a * (da - delta[I]), a * (da_m + delta_m[I])
        de_e = de_m * (w + (D + deg[I] + 8) * U) + a * delta_e[I]
        sc = np.abs(scale)
        for name, idx, row, m, nd in (("dq", I, kh[J], I, deg), ("dkey", J, qh[I], J, odeg)):
            r[name] = (scale * add(idx, de[:, None] * row), sc * add(
                idx, (de_e + (nd[m] + 6) * U * de_m)[:, None] * np.abs(row)))
        r["dval"] = (add(J, A * gh[I]),
                     add(J, (W + (odeg[J] + 4)[:, None] * U) * A * np.abs(gh[I])))
        nb = len(bias)
        count = np.bincount(bucket[keep], minlength=nb)[bucket[keep]]
        db, db_e = np.zeros(nb), np.zeros(nb)
        np.add.at(db, bucket[keep], de)
        np.add.at(db_e, bucket[keep], de_e + (count + 8) * U * de_m)
        r["dbias"] = (db, db_e)
        heads.append(r)
    return {x: tuple(np.stack([r[x][t] for r in heads], 1) for t in (0, 1)) for x in heads[0]}


def hold(got, ref, dtype, what, names):
    for x in names:
        value, bound = ref[x]
        half = 0.0 if x in ("lse", "dbias") else layer_ref.HALF[dtype]
        size = np.where(np.isinf(value), 0.0, np.abs(value))
        layer_ref.hold(got[x], value, bound + half * size * (1 + half) + 1e-36, f"{what} {x}")


def graph(seed):
    """Rows of 17 edges, shorter ones, and rows long enough to be cut."""
    return testgraphs.with_in_degrees([17] * 60 + [0, 1, 2, 63, 64, 65, 300, 700], n_nodes=300,
                                      seed=seed)


def check_both(rp, ci, H, D, dtype, bias, pos, what, seed=5, rel_args=()):
    import graph_neural_network_gb300 as gnn
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci))
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), *rel_args)
    bucket = edge_buckets(rp, ci, pos, rel.bounds, rel.bidirectional)
    feats = features(n, H, D, dtype, seed)
    got = run(g, rel, feats, bias, dtype)
    ref = reference(rp, ci, *(wide(x) for x in feats), D ** -0.5, bias, bucket)
    hold({x: to_f64(t) for x, t in got.items()}, ref, dtype, what, ("out", "lse") + NAMES)
    q, k, v, dout = (to_device(x, dtype) for x in feats)
    packed = gnn.pack8(q, k, v)
    at = [p.values.cpu().numpy() * p.scale.cpu().numpy().astype(np.float64)[..., None]
          for p in packed]
    got = gnn.transformer_backward8(g, *packed, dout, rel=rel, bias=torch.from_numpy(bias).cuda())
    ref = reference(rp, ci, *at, wide(feats[3]), D ** -0.5, bias, bucket)
    hold({x: to_f64(t) for x, t in zip(NAMES, got)}, ref, dtype, what + " checkpoints", NAMES)


@pytest.mark.gpu
@pytest.mark.parametrize("H, D, dtype", [(2, 16, "f32"), (4, 64, "bf16"), (3, 8, "bf16")])
@pytest.mark.parametrize("value", VALUES, ids=lambda v: f"{v:.3g}")
def test_every_edge_carries_it(value, H, D, dtype):
    rp, ci = graph(3)
    check_both(rp, ci, H, D, dtype, np.full((32, H), value, np.float32),
               positions(len(rp) - 1, 3, 300), f"{value}")


@pytest.mark.gpu
@pytest.mark.parametrize("H, D, dtype", [(2, 16, "f32"), (4, 64, "bf16")])
@pytest.mark.parametrize("value", VALUES, ids=lambda v: f"{v:.3g}")
def test_beside_ordinary_ones(value, H, D, dtype):
    """Half of the buckets (sources after the destination) carry the value, one other bucket
    -infinity; positions descend along the rows of the CSR, so that rows have every mix."""
    rp, ci = graph(4)
    n = len(rp) - 1
    bias = workload.normal_f32(3, 7, (32, H), 1.0)
    bias[16:] = value
    bias[4, 0] = -np.inf
    check_both(rp, ci, H, D, dtype, bias, np.arange(n, 0, -1, dtype=np.int32), f"{value}")
    check_both(rp, ci, H, D, dtype, bias, np.arange(n, dtype=np.int32), f"{value} up")


@pytest.mark.gpu
@pytest.mark.parametrize("H, D, dtype, buckets", [
    (1, 4, "f32", 32), (32, 4, "f32", 128), (3, 8, "f32", 40), (4, 32, "f32", 64),
    (1, 128, "f32", 32), (1, 8, "bf16", 128), (32, 8, "bf16", 128), (5, 16, "bf16", 32),
    (1, 256, "bf16", 32)])
def test_shapes(H, D, dtype, buckets):
    """Every lane width and form of the gradient tables, with a mask value in one bucket of
    each side and one head."""
    rp, ci = graph(H + D)
    n = len(rp) - 1
    bias = workload.normal_f32(3, 7, (buckets, H), 1.0)
    bias[1], bias[buckets // 2 + 1] = -1e9, -F32
    bias[2, H - 1] = 1e5
    check_both(rp, ci, H, D, dtype, bias, positions(n, 3, 300), f"{H} {D}",
               rel_args=(buckets, 400))


@pytest.mark.gpu
def test_reproducible_captured_and_masked():
    """A power-law graph with every kind of bias: the same bits again, on another stream and
    from a CUDA graph, and with NaN and infinities in the rows that only masked edges reach."""
    import graph_neural_network_gb300 as gnn
    rp, ci = workload.chung_lu(20_000, 2.1, 15.0, 6_000.0, 29)
    n = len(rp) - 1
    ci = np.where(ci == 17, 18, ci).astype(np.int32)
    dst = np.repeat(np.arange(n), np.diff(rp))
    ci[::50] = np.where(dst[::50] != 17, 17, ci[::50])      # node 17: a source far after all
    pos = np.random.default_rng(1).integers(0, 100, n).astype(np.int32)
    pos[17] = 10_000
    g = device_graph(dict(row_ptr=rp, col=ci))
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), 32, 128)
    b = torch.from_numpy(workload.normal_f32(3, 7, (32, 2), 1.0)).cuda()
    b[2], b[20], b[5, 1], b[31] = -1e9, 1e4, -F32, -float("inf")
    q, k, v, dout = (to_device(x, "f32") for x in features(n, 2, 16, "f32", 9))

    def step(k, v, packed, **kw):
        out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b, **kw)
        return ((out, lse) + gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, dout, **kw)
                + gnn.transformer_backward8(g, *packed, dout, rel=rel, bias=b, **kw))

    packed = gnn.pack8(q, k, v)
    first = step(k, v, packed)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    runs = [step(k, v, packed), step(k, v, packed, stream=side)]
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        runs.append(step(k, v, packed))
    cg.replay()
    cg.replay()
    bad_k, bad_v = k.clone(), v.clone()
    bad_k[17], bad_v[17, :, ::2], bad_v[17, :, 1::2] = float("nan"), -float("inf"), float("nan")
    runs.append(step(bad_k, bad_v, gnn.pack8(q, bad_k, bad_v)))
    torch.cuda.synchronize()
    own = np.flatnonzero(dst == 17)                          # its own row reads only others' keys
    assert len(own) and (b[rel.arrays()[0][torch.from_numpy(own).cuda()].long()] > -1e38).any()
    for r in runs:
        for a, c in zip(first, r):
            assert torch.isfinite(a).logical_or(torch.isneginf(a)).all() and torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("order", [1, -1], ids=["last", "first"])
@pytest.mark.parametrize("value", [-F32, -1e9, -1e4, 2.4e38], ids=lambda v: f"{v:.3g}")
def test_a_long_row_that_changes_over(value, order):
    """One destination of 3000 edges, of which the first (or last) tenth carries an
    ordinary bias and the others the value: pieces of the row that hold only one
    kind are joined with those that hold the other."""
    n = 3001
    src = np.arange(1, n)[::order]
    rp = np.concatenate([[0], np.full(n, n - 1)]).astype(np.int32)
    pos = np.zeros(n, np.int32)
    pos[src[:300]] = -1            # distance 1 before the destination: bucket 1
    bias = np.array([[value, value], [0.25, -0.5]], np.float32)
    check_both(rp, src.astype(np.int32), 2, 16, "f32", bias, pos, f"{value} {order}",
               rel_args=(2, 2, False))


@pytest.mark.gpu
def test_scores_of_minus_infinity_and_masked_rows():
    """A key of -infinity gives its edge weight 0 under a finite bias too, at any place
    of the row; a row of nothing else stays 0 with lse -infinity, in the gradients as
    well."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.csr_from_rows([[1, 2, 3], [3, 1, 2], [3, 3], [0, 1]])
    g = device_graph(dict(row_ptr=rp, col=ci))
    rel = gnn.RelPos(g, torch.arange(4, dtype=torch.int32, device="cuda"), 4, 2)
    q = torch.ones(4, 1, 16, device="cuda")
    k = torch.linspace(-1, 1, 64, device="cuda").view(4, 1, 16).contiguous()
    k[3] = -float("inf")
    v = torch.arange(64.0, device="cuda").view(4, 1, 16).contiguous()
    b = torch.full((4, 1), -1e9, device="cuda")
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
    w = torch.softmax(torch.tensor([float(k[1].sum()), float(k[2].sum())]).double() / 4, 0)
    want = (w[0] * v[1].double().cpu() + w[1] * v[2].double().cpu())
    for row in (0, 1):
        assert float((out[row].double().cpu() - want).abs().max()) <= 64 * 2.0 ** -20
    assert not out[2].any() and torch.isneginf(lse[2]).all() and torch.isfinite(lse[3]).all()
    *_, dval, _ = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, torch.ones_like(q))
    assert not dval[3].any() and torch.isfinite(dval).all()
    # ... and under the lowest value, beside which finite scores count for nothing
    b.fill_(torch.finfo(torch.float32).min)
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
    want = (v[1] + v[2]).double().cpu() / 2
    for row in (0, 1):
        assert float((out[row].double().cpu() - want).abs().max()) <= 64 * 2.0 ** -20
    assert not out[2].any() and torch.isneginf(lse[2]).all()
    *_, dval, _ = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, torch.ones_like(q))
    assert not dval[3].any() and torch.isfinite(dval).all()


@pytest.mark.gpu
def test_a_float64_table_keeps_its_finite_entries_finite():
    """float64's lowest value is not representable in float32; it stays a bias, and only
    -infinity masks."""
    import graph_neural_network_gb300 as gnn
    rp, ci = graph(3)
    n = len(rp) - 1
    g = device_graph(dict(row_ptr=rp, col=ci))
    rel = gnn.RelPos(g, torch.from_numpy(positions(n, 3, 300)).cuda())
    q, k, v, dout = (to_device(x, "f32") for x in features(n, 2, 16, "f32", 3))
    for low, high in ((-np.inf, F32), (-F32, 0.5), (-F32, F32)):
        b32 = torch.full((32, 2), low, device="cuda")
        b32[8:, 1] = high
        b64 = b32.double()
        b64[b32 == -F32] = torch.finfo(torch.float64).min
        b64[b32 == F32] = torch.finfo(torch.float64).max
        want = gnn.transformer_rel_forward(g, rel, q, k, v, b32)
        got = gnn.transformer_rel_forward(g, rel, q, k, v, b64)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = gnn.transformer_rel_backward(g, rel, q, k, v, b32, got[1], dout)
        got = gnn.transformer_rel_backward(g, rel, q, k, v, b64, got[1], dout)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.isfinite(got[0]).all()


def test_the_reference_agrees_with_the_plain_one():
    """At ordinary biases it is the reference of the other tests."""
    rp, ci = graph(3)
    n, H, D = len(rp) - 1, 2, 8
    q, k, v, dout = (x.astype(np.float64) for x in features(n, H, D, "f32", 3))
    bias = workload.normal_f32(3, 7, (32, H), 1.0)
    bias[5] = -np.inf
    bucket = edge_buckets(rp, ci, positions(n, 3, 300), list(range(16)), True)
    a = reference(rp, ci, q, k, v, dout, 0.3, bias, bucket)
    b = layer_ref.attention(rp, ci, q, k, v, 0.3, bias, bucket, dout)
    for x in ("out", "lse") + NAMES:
        assert np.allclose(a[x][0], b[x], rtol=1e-10, atol=1e-12), x
