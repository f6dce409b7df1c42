"""Tokens in the order of their experts and back: the CUDA path against a plain
implementation in whole numbers and float64.

The plan's arrays are whole numbers and a dispatched row is a copy: exact.  U = 2^-24.
A combined element rounds each of its K products with an addition: (K + 1) U of the sum of
magnitudes.  dys is one product: U of it.  dweights adds, per lane, V / 2 products of a
vector of V elements, a vector a turn (rv / 32 of the row's rv at most), then 5 levels of a
warp and 8 warps: (V / 2 + rv / 32 + 16) U of the sum of magnitudes at most.  Then each
result's own rounding."""
import ctypes

import numpy as np
import pytest
import torch

import layer_ref
import workload
from gpu_util import to_device, to_f64

U = 2.0 ** -24


def draw(seed, *shape, dtype="f32"):
    x = workload.normal_f32(seed, 1, shape, 1.0)
    return workload.f32_to_bf16_bits(x) if dtype == "bf16" else x


def wide(x):
    return (workload.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def order_of(ids, E, align):
    """offsets, counts, order and slots by the definition."""
    flat = ids.reshape(-1).astype(np.int64)
    pairs = len(flat)
    rows = (pairs + min(E, pairs) * (align - 1)) // align * align
    kept = (flat >= 0) & (flat < E)
    counts = np.bincount(flat[kept], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    by = np.flatnonzero(kept)[np.argsort(flat[kept], kind="stable")]
    rank = np.arange(len(by)) - np.repeat(np.cumsum(counts) - counts, counts)
    at = offsets[flat[by]] + rank
    order = np.full(rows, -1, np.int64)
    order[at] = by
    slots = np.full(pairs, -1, np.int64)
    slots[by] = at
    return offsets, counts, order, slots.reshape(ids.shape if ids.ndim == 2 else (-1, 1))


def choose(n, K, E, seed=1, kind="even", dtype=np.int64):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full((n, K), E - 1, dtype)
    if kind == "none":
        return np.full((n, K), -1, dtype)
    if kind == "skewed":
        ids = (E * rng.random((n, K)) ** 6).astype(dtype)
    else:
        ids = rng.integers(0, E, (n, K)).astype(dtype)
    if kind == "dropped":
        bad = np.array([-1, E, np.iinfo(dtype).max, np.iinfo(dtype).min, -E], dtype)
        ids = np.where(rng.random((n, K)) < 0.4, rng.choice(bad, (n, K)), ids)
    return ids


def check_plan(ids, E, align):
    import graph_neural_network_gb300 as gnn
    plan = gnn.Experts(torch.from_numpy(ids).cuda(), E, align)
    for name, want in zip(("offsets", "counts", "order", "slots"), order_of(ids, E, align)):
        got = getattr(plan, name).cpu().numpy()
        assert got.shape == want.shape and np.array_equal(got, want), (name, ids.shape, E, align)
    assert plan.rows == len(order_of(ids, E, align)[2])
    return plan


@pytest.mark.gpu
@pytest.mark.parametrize("n, K, E", [
    (0, 2, 4), (1, 1, 1), (1, 8, 64), (31, 1, 3), (33, 3, 5), (512, 8, 64), (1024, 8, 256),
    (4096, 2, 257), (1025, 8, 64), (2731, 3, 1024), (2048, 1, 64), (683, 3, 700), (100, 64, 1000), (40_000, 2, 8),
    (300_007, 1, 1), (200_001, 4, 64), (150_000, 3, 300), (90_001, 8, 1024), (700_001, 5, 100)])
@pytest.mark.parametrize("kind", ["even", "skewed", "dropped", "one", "none"])
def test_plan(n, K, E, kind):
    for align, dtype in ((1, np.int64), (16, np.int32), (100, np.int64)):
        check_plan(choose(n, K, E, n + K, kind, dtype), E, align)


@pytest.mark.gpu
def test_plan_of_many_pairs():
    """More than a block's turn of pairs in each of the most blocks; ids of one dimension."""
    check_plan(choose(6_000_011, 1, 64, 3, "dropped", np.int32)[:, 0].copy(), 64, 128)
    check_plan(choose(1_500_001, 8, 1024, 4, "skewed", np.int32), 1024, 1)


def check_rows(n, F, E, K, dtype, align=1, kind="dropped", seed=2):
    import graph_neural_network_gb300 as gnn
    ids = choose(n, K, E, seed, kind)
    plan = check_plan(ids, E, align)
    _, _, order, slots = order_of(ids, E, align)
    m, kept = plan.rows, slots >= 0
    x, res, dy = (draw(s, n, F, dtype=dtype) for s in (1, 2, 3))
    ys, dxs = (draw(s, m, F, dtype=dtype) for s in (4, 5))
    w = draw(6, n, K)
    t = {k: to_device(v, dtype) for k, v in dict(x=x, res=res, dy=dy, ys=ys, dxs=dxs).items()}
    wt = torch.from_numpy(w).cuda()
    half = layer_ref.HALF[dtype]
    what = f"{n} {F} {E} {K} {kind}"

    xs = torch.full((m, F), float("nan"), dtype=t["x"].dtype, device="cuda")
    gnn.expert_dispatch_forward(plan, t["x"], out=xs)
    want = np.where((order >= 0)[:, None], wide(x)[np.maximum(order, 0) // K], 0.0)
    assert np.array_equal(to_f64(xs), want), what

    def summed(rows, weights, base):
        g = np.where(kept[..., None], wide(rows)[np.maximum(slots, 0)], 0.0) * \
            weights[..., None].astype(np.float64)
        return base + g.sum(1), np.abs(base) + np.abs(g).sum(1)

    for name, got, (ref, mag) in (
            ("combine", gnn.expert_combine_forward(plan, t["ys"], wt, t["res"]),
             summed(ys, w, wide(res))),
            ("combine alone", gnn.expert_combine_forward(plan, t["ys"], wt),
             summed(ys, w, 0 * wide(res))),
            ("dispatch backward", gnn.expert_dispatch_backward(plan, t["dxs"]),
             summed(dxs, np.ones_like(w), 0 * wide(res)))):
        bound = (K + 1) * U * mag
        layer_ref.hold(to_f64(got), ref, bound + half * (np.abs(ref) + bound) + 1e-37,
                       what + " " + name)
    place = t["res"].clone()
    gnn.expert_combine_forward(plan, t["ys"], wt, place, out=place)
    assert torch.equal(place, gnn.expert_combine_forward(plan, t["ys"], wt, t["res"]))

    dys = torch.full((m, F), float("nan"), dtype=t["x"].dtype, device="cuda")
    _, dw = gnn.expert_combine_backward(plan, t["dy"], t["ys"], wt, dys=dys)
    ref = np.zeros((m, F))
    at = slots[kept]
    tok = np.nonzero(kept)[0]
    ref[at] = w[kept][:, None].astype(np.float64) * wide(dy)[tok]
    layer_ref.hold(to_f64(dys), ref, (U + half * (1 + U)) * np.abs(ref) + 1e-37, what + " dys")
    terms = np.where(kept[..., None], wide(dy)[:, None] * wide(ys)[np.maximum(slots, 0)], 0.0)
    V = 4 if dtype == "f32" else 8
    layer_ref.hold(to_f64(dw), terms.sum(-1),
                   (V / 2 + F / V / 32 + 16) * U * np.abs(terms).sum(-1) + 1e-37, what + " dw")
    plain, none = gnn.expert_combine_backward(plan, t["dy"])
    assert none is None
    assert torch.equal(plain, gnn.expert_dispatch_forward(plan, t["dy"]))


@pytest.mark.gpu
@pytest.mark.parametrize("n, F, E, K, dtype", [
    (1, 4, 1, 1, "f32"), (1, 8, 4, 2, "bf16"), (5, 12, 3, 2, "f32"), (64, 2048, 64, 8, "bf16"),
    (300, 64, 16, 2, "f32"), (1001, 40, 7, 3, "bf16"), (513, 128, 8, 1, "f32"),
    (200, 132, 8, 5, "f32"), (77, 256, 300, 6, "bf16"), (50, 264, 8, 4, "bf16"),
    (33, 520, 9, 9, "bf16"), (3000, 520, 9, 2, "f32"), (9, 4104, 5, 3, "bf16"),
    (2600, 1032, 16, 5, "bf16"), (20, 4, 10, 64, "f32"), (5000, 8, 30, 4, "bf16")])
@pytest.mark.parametrize("align", [1, 24])
def test_rows(n, F, E, K, dtype, align):
    check_rows(n, F, E, K, dtype, align)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one", "none", "even"])
def test_rows_of_odd_choices(kind):
    """Every token at one expert (each choice the same), none at any, all kept."""
    check_rows(70, 96, 6, 3, "bf16", 8, kind)
    check_rows(70, 1024, 6, 3, "f32", 1, kind)


@pytest.mark.gpu
def test_rows_that_are_not_read():
    """NaN and infinities in padding rows, and weights of dropped choices that are NaN, reach
    no result; a kept row's do."""
    import graph_neural_network_gb300 as gnn
    for F in (16, 2048):
        ids = choose(40, 3, 5, 2, "dropped")
        plan = check_plan(ids, 5, 16)
        _, _, order, slots = order_of(ids, 5, 16)
        ys = to_device(draw(1, plan.rows, F), "f32")
        w, dy = to_device(draw(2, 40, 3), "f32"), to_device(draw(3, 40, F), "f32")
        bad, wbad = ys.clone(), w.clone()
        bad[torch.from_numpy(order).cuda() < 0] = float("nan")
        wbad[torch.from_numpy(slots).cuda() < 0] = float("nan")
        for a, b in zip((gnn.expert_combine_forward(plan, ys, w),
                         *gnn.expert_combine_backward(plan, dy, ys, w)),
                        (gnn.expert_combine_forward(plan, bad, wbad),
                         *gnn.expert_combine_backward(plan, dy, bad, wbad))):
            assert torch.equal(a, b)
        t, k = np.argwhere(slots >= 0)[0]
        bad[slots[t, k], 1] = float("inf")
        y = gnn.expert_combine_forward(plan, bad, w)
        assert torch.isinf(y[t, 1]) and torch.isfinite(y).sum() == y.numel() - 1


@pytest.mark.gpu
def test_no_tokens():
    import graph_neural_network_gb300 as gnn
    plan = check_plan(np.zeros((0, 2), np.int64), 4, 8)
    x, w = torch.zeros(0, 3, 16, device="cuda"), torch.zeros(0, 2, device="cuda")
    assert gnn.expert_dispatch_forward(plan, x).shape == (0, 3, 16)
    assert gnn.expert_combine_forward(plan, x, w, x).shape == (0, 3, 16)
    assert gnn.expert_dispatch_backward(plan, x).shape == (0, 3, 16)
    dys, dw = gnn.expert_combine_backward(plan, x, x, w)
    assert dys.shape == (0, 3, 16) and dw.shape == (0, 2)


@pytest.mark.gpu
def test_one_choice_and_rows_of_several_dimensions():
    """ids and weights [N], rows [N, H, D], weights in another type."""
    import graph_neural_network_gb300 as gnn
    ids = torch.from_numpy(choose(60, 1, 5, 3, "dropped")[:, 0].copy()).cuda()
    x = to_device(draw(1, 60, 4, 8), "f32")
    w = torch.from_numpy(draw(2, 60)).cuda().bfloat16()
    one, two = gnn.Experts(ids, 5, align=4), gnn.Experts(ids[:, None].contiguous(), 5, align=4)
    xs = gnn.expert_dispatch_forward(one, x)
    assert xs.shape == (one.rows, 4, 8) and one.slots.shape == (60, 1)
    assert torch.equal(xs.view(-1, 32), gnn.expert_dispatch_forward(two, x.view(60, 32)))
    y = gnn.expert_combine_forward(one, xs, w, x)
    want = gnn.expert_combine_forward(two, xs.view(-1, 32), w.float()[:, None].contiguous(),
                                      x.view(60, 32))
    assert y.shape == x.shape and torch.equal(y.view(60, 32), want)
    dys, dw = gnn.expert_combine_backward(one, x, xs, w)
    assert dys.shape == xs.shape and dw.shape == (60,) and dw.dtype == torch.float32
    leaf = w.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(gnn.ExpertCombine.apply(one, xs, leaf, None), leaf, x)
    assert g.dtype == torch.bfloat16 and torch.equal(g, dw.bfloat16())


@pytest.mark.gpu
def test_packed_rows():
    """Rows in 8 bits go with their scales."""
    import graph_neural_network_gb300 as gnn
    for F, group, fmt in ((4104, 8, "int8"), (64, None, "e4m3"), (20, None, "int8")):
        x = to_device(draw(1, 90, F), "f32")
        plan = check_plan(choose(90, 2, 7, 3, "dropped"), 7, 4)
        _, z8 = gnn.add_norm8_forward(x, fmt=fmt, group=group)
        got = gnn.expert_dispatch_forward(plan, z8)
        assert got.values.dtype == z8.values.dtype
        want = gnn.expert_dispatch_forward(plan, gnn.unpack8(z8))
        assert torch.equal(gnn.unpack8(got), want)
        again = gnn.expert_dispatch_forward(plan, z8, out=got)
        assert again.values is got.values


@pytest.mark.gpu
def test_autograd_differences_streams_and_capture():
    import graph_neural_network_gb300 as gnn
    n, F, E, K = 50, 24, 6, 3
    ids = torch.from_numpy(choose(n, K, E, 5, "dropped")).cuda()
    x, res, dy = (to_device(draw(s, n, F), "f32").requires_grad_(s < 3) for s in (1, 2, 3))
    w = torch.from_numpy(draw(4, n, K)).cuda().requires_grad_(True)
    m = to_device(draw(5, E, F, F), "f32").requires_grad_(True)
    plan = gnn.Experts(ids, E, align=4)

    def products(xs, p):
        at = p.offsets.tolist()
        rows = [xs[at[e]:at[e + 1]] @ m[e] for e in range(E)]
        return torch.cat(rows + [xs[at[E]:] * 0])

    y = gnn.expert_layer(plan, x, products, w, res)
    got = torch.autograd.grad(y, [x, w, res, m], dy)
    # the same in float64 by autograd, token by token
    x6, w6, r6, m6 = leaves = [t.detach().double().cpu().requires_grad_(True)
                               for t in (x, w, res, m)]
    y6 = [r6[t] + sum(w6[t, k] * (x6[t] @ m6[int(e)]) for k, e in enumerate(ids[t].tolist())
                      if 0 <= e < E) for t in range(n)]
    y6 = torch.stack(y6)
    want = torch.autograd.grad(y6, leaves, dy.double().cpu())
    for a, b in zip((y, *got), (y6, *want)):
        assert (a.double().cpu() - b).norm() <= 1e-5 * b.norm()
    # differences in float64: linear in x and in w
    assert torch.equal(got[2], dy)
    h = 0.5
    for leaf, g, at in ((x6, got[0], (3, 5)), (w6, got[1], (7, 1)), (w6, got[1], (9, 2))):
        d = torch.zeros_like(leaf)
        d[at] = h

        def loss(sign):
            x_, w_ = (t + sign * d if t is leaf else t for t in (x6, w6))
            return sum(float((dy[t].double().cpu() * w_[t, k] * (x_[t] @ m6[int(e)])).sum())
                       for t in range(n) for k, e in enumerate(ids[t].tolist()) if 0 <= e < E)

        diff = (loss(1) - loss(-1)) / (2 * h)
        assert abs(float(g[at]) - diff) <= 1e-4 * (1 + abs(diff))

    def calls(**kw):
        p = gnn.Experts(ids, E, align=4, **kw)
        ys = gnn.expert_dispatch_forward(p, x.detach(), **kw)
        return (p.offsets, p.order, p.slots, ys,
                gnn.expert_combine_forward(p, ys, w.detach(), res.detach(), **kw),
                *gnn.expert_combine_backward(p, dy, ys, w.detach(), **kw),
                gnn.expert_dispatch_backward(p, ys, **kw))

    first = calls()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = calls(stream=side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        kept = calls()
    cg.replay()
    moved = ids.roll(1, 0).contiguous()
    ids.copy_(moved)          # new choices under the captured calls
    cg.replay()
    torch.cuda.synchronize()
    fresh = calls()
    for a, b, c, d in zip(first, other, kept, fresh):
        assert torch.equal(a, b) and torch.equal(c, d)


@pytest.mark.gpu
def test_a_large_plan_is_captured():
    """Two kernels of a plan, the second started early, in a graph replayed twice."""
    import graph_neural_network_gb300 as gnn
    a, b = (torch.from_numpy(choose(60_000, 4, 64, s, "skewed")).cuda() for s in (1, 2))
    ids = a.clone()
    gnn.Experts(ids, 64)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        plan = gnn.Experts(ids, 64, align=8)
    for t in (a, b, a):
        ids.copy_(t)
        cg.replay()
        torch.cuda.synchronize()
        want = order_of(t.cpu().numpy(), 64, 8)
        assert np.array_equal(plan.slots.cpu().numpy(), want[3])
        assert np.array_equal(plan.order.cpu().numpy(), want[2])


@pytest.mark.gpu
def test_offsets_past_32_bits():
    import graph_neural_network_gb300 as gnn
    n, F, K = (1 << 30) // 4096 + 3, 4096, 2
    ids = torch.zeros(n, K, dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    plan = gnn.Experts(ids, 2)
    x = torch.zeros(n, F, dtype=torch.bfloat16, device="cuda")
    x[-8:] = to_device(draw(1, 8, F, dtype="bf16"), "bf16")
    xs = gnn.expert_dispatch_forward(plan, x)
    assert xs.numel() > 1 << 31 and torch.equal(xs[-8:], x[-8:]) and torch.equal(xs[n - 8:n], x[-8:])
    w = torch.full((n, K), 0.5, device="cuda")
    assert torch.equal(gnn.expert_combine_forward(plan, xs, w)[-8:], x[-8:])
    dys, dw = gnn.expert_combine_backward(plan, x, xs, w)
    assert torch.equal(dys[-8:].float(), x[-8:].float() / 2)
    want = (x[-8:].double() ** 2).sum(-1, keepdim=True)
    assert ((dw[-8:].double() - want).abs() <= 36 * U * want).all()


def test_refusals_on_the_host():
    import graph_neural_network_gb300 as gnn
    from graph_neural_network_gb300 import build, _native
    build.build()
    lib = _native.load()
    P = 4096
    bad, no = _native.ERR_INVALID_ARG, _native.ERR_UNSUPPORTED
    assert lib.gnn_experts_rows(10, 2, 4, 1) == 20
    assert lib.gnn_experts_rows(10, 2, 4, 8) == (20 + 28) // 8 * 8
    assert lib.gnn_experts_rows(1, 1, 100, 16) == 16 and lib.gnn_experts_rows(0, 3, 4, 8) == 0
    for size in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1),
                 (1, 1, 1, 0), (1, 1, 1, 65537), (1 << 31, 1, 1, 1), (1 << 26, 64, 1, 1),
                 ((1 << 31) - 2, 1, 1000, 8)):
        assert lib.gnn_experts_rows(*size) == -1, size
        assert lib.gnn_experts_buffer_bytes(*size) == 0, size
    out = _native.Experts()
    need = lib.gnn_experts_buffer_bytes(10, 2, 4, 1)

    def prepare(ids=P, width=4, size=(10, 2, 4, 1), buf=P, nb=need, to=out):
        return lib.gnn_experts_prepare(ids, width, *size, buf, nb, None,
                                       None if to is None else ctypes.byref(to))

    for kw in (dict(ids=None), dict(ids=P + 2), dict(ids=P + 4, width=8), dict(width=2),
               dict(buf=None), dict(buf=P + 16), dict(size=(10, 2, 4, 0)), dict(to=None)):
        assert prepare(**kw) == bad, kw
    assert prepare(nb=need - 1) == _native.ERR_WORKSPACE_TOO_SMALL
    plan = _native.Experts(10, 20, 2, 4, 1, P, P, P, P)

    def ref(**kw):
        p = _native.Experts.from_buffer_copy(plan)
        for k, v in kw.items():
            setattr(p, k, v)
        return ctypes.byref(p)

    assert lib.gnn_expert_dispatch(ref(tokens=0, rows=0), 16, None, None, None) == _native.OK
    for kw in (dict(rows=21), dict(tokens=-1), dict(offsets=None), dict(slots=None)):
        assert lib.gnn_expert_dispatch(ref(**kw), 16, P, P, None) == bad, kw
        assert lib.gnn_expert_combine(ref(**kw), 16, 0, P, None, None, P, None) == bad, kw
    assert lib.gnn_expert_dispatch(None, 16, P, P, None) == bad
    assert lib.gnn_expert_dispatch(ref(), 0, P, P, None) == bad
    assert lib.gnn_expert_dispatch(ref(), 6, P, P, None) == no
    assert lib.gnn_expert_dispatch(ref(), (1 << 20) + 16, P, P, None) == no
    for x, xs in ((None, P), (P, None), (P + 8, P), (P, P + 8)):
        assert lib.gnn_expert_dispatch(ref(), 32, x, xs, None) == bad
    for F, dt, r in ((6, 0, no), (12, 1, no), (1 << 19, 0, no), (16, 2, bad), (0, 0, bad)):
        assert lib.gnn_expert_combine(ref(), F, dt, P, None, None, P, None) == r
        assert lib.gnn_expert_combine_backward(ref(), F, dt, P, P, None, P, None, None) == r
    for ys, w, res, y in ((None, None, None, P), (P, None, None, None), (P + 8, None, None, P),
                          (P, P + 2, None, P), (P, None, P + 8, P), (P, None, None, P + 8)):
        assert lib.gnn_expert_combine(ref(), 16, 0, ys, w, res, y, None) == bad
    for dy, ys, w, dys, dw in ((None, P, P, P, P), (P, None, P, P, P), (P, P, P, None, P),
                               (P + 8, P, P, P, P), (P, P + 8, P, P, P), (P, P, P + 2, P, P),
                               (P, P, P, P + 8, P), (P, P, P, P, P + 2)):
        assert lib.gnn_expert_combine_backward(ref(), 16, 0, dy, ys, w, dys, dw, None) == bad
    for call in (lambda: gnn.Experts(torch.zeros(4, 2, dtype=torch.int64), 4),
                 lambda: gnn.Experts(None, 4)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    import graph_neural_network_gb300 as gnn
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    for args, err in (((ids.int().short(), 4), TypeError), ((ids.t(), 4), ValueError),
                      ((ids[None], 4), ValueError), ((ids, 0), ValueError),
                      ((ids, 2000), ValueError), ((ids, 4, 0), ValueError)):
        with pytest.raises(err):
            gnn.Experts(*args)
    plan = gnn.Experts(ids, 4)
    x = torch.zeros(4, 16, device="cuda")
    ys = torch.zeros(8, 16, device="cuda")
    w = torch.ones(4, 2, device="cuda")
    for call, err in ((lambda: gnn.expert_dispatch_forward(plan, ys), ValueError),
                      (lambda: gnn.expert_dispatch_forward(plan, x.cpu()), ValueError),
                      (lambda: gnn.expert_dispatch_forward(plan, x[:, ::2]), ValueError),
                      (lambda: gnn.expert_dispatch_forward(None, x), TypeError),
                      (lambda: gnn.expert_dispatch_forward(plan, x, out=x), ValueError),
                      (lambda: gnn.expert_dispatch_forward(plan, x[:, :3].contiguous().half()),
                       gnn.GnnError),
                      (lambda: gnn.expert_combine_forward(plan, x), ValueError),
                      (lambda: gnn.expert_combine_forward(plan, ys.half()), TypeError),
                      (lambda: gnn.expert_combine_forward(plan, ys, w[:, :1]), ValueError),
                      (lambda: gnn.expert_combine_forward(plan, ys, w.long()), TypeError),
                      (lambda: gnn.expert_combine_forward(plan, ys, w, x[:2]), ValueError),
                      (lambda: gnn.expert_combine_forward(plan, ys, w, x.bfloat16()), TypeError),
                      (lambda: gnn.expert_combine_backward(plan, ys, ys, w), ValueError),
                      (lambda: gnn.expert_combine_backward(plan, x, None, w), TypeError),
                      (lambda: gnn.expert_combine_backward(plan, x, dweights=w), ValueError),
                      (lambda: gnn.expert_dispatch_backward(plan, x), ValueError)):
        with pytest.raises(err):
            call()
