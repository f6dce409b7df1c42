"""The operators of a graph-transformer layer run together as they are used: two
layers with projections, forward and backward, against torch's autograd of the
same formulas in float64; and one training step captured into a CUDA graph."""
import numpy as np
import pytest
import torch

import workload
from workload import testgraphs
from gpu_util import device_graph
from test_rel_attention import edge_buckets, positions

pytestmark = pytest.mark.gpu

N, H, D = 300, 2, 16
F = H * D


def setup(seed=3):
    rp, ci = testgraphs.with_in_degrees([0, 1, 5, 70, 200], n_nodes=N, seed=seed)
    g = device_graph(dict(row_ptr=rp, col=ci), (8, 64, 16))
    pos = positions(N, seed, 60)
    import graph_neural_network_gb300 as gnn
    rel = gnn.RelPos(g, torch.from_numpy(pos).cuda(), 16, 32)

    def t(stream, *shape, std=1.0):
        return torch.from_numpy(workload.normal_f32(seed, stream, shape, std)).cuda()

    x = t(1, N, F)
    par = {}
    for layer in range(2):
        b = 20 * layer
        par[layer] = dict(wqkv=t(b + 2, F, 3 * F, std=F ** -0.5), wo=t(b + 3, F, F, std=F ** -0.5),
                          wg=t(b + 4, F, F, std=F ** -0.5), bias=t(b + 5, 16, H),
                          w_post=1 + t(b + 6, F, std=0.1), b_post=t(b + 7, F, std=0.1),
                          res_scale=0.5 + t(b + 8, F, std=0.1), w_pre=1 + t(b + 9, F, std=0.1),
                          b_pre=t(b + 10, F, std=0.1))
    bucket = edge_buckets(rp, ci, pos, rel.bounds, True)
    return g, rel, x, par, (rp, ci, bucket), t(60, N, F), t(61, N, F)


def forward(g, rel, x, par, checkpoint8):
    import graph_neural_network_gb300 as gnn
    y, z = x, x
    for p in par.values():
        q, k, v = ((z @ p["wqkv"]).view(N, 3, H, D).unbind(1))
        gate = z @ p["wg"]
        wo = p["wo"]
        y, z = gnn.transformer_layer(
            g, y, q, k, v, rel=rel, bias=p["bias"], gate=gate, w_post=p["w_post"],
            b_post=p["b_post"], res_scale=p["res_scale"], w_pre=p["w_pre"], b_pre=p["b_pre"],
            project=lambda out: out.reshape(N, F) @ wo, kind="layer", checkpoint8=checkpoint8)
    return y, z


def plain(x, par, graph):
    rp, ci, bucket = graph
    dst = torch.from_numpy(np.repeat(np.arange(N), np.diff(rp)))
    src, bk = torch.from_numpy(ci.astype(np.int64)), torch.from_numpy(bucket)
    y, z = x, x
    for p in par.values():
        q, k, v = (z @ p["wqkv"]).view(N, 3, H, D).unbind(1)
        e = (q[dst] * k[src]).sum(-1) * D ** -0.5 + p["bias"][bk]
        w = torch.exp(e - e.detach().max())
        l = torch.zeros(N, H, dtype=torch.float64).index_add(0, dst, w)
        o = torch.zeros(N, H, D, dtype=torch.float64).index_add(0, dst, w[..., None] * v[src])
        o = o / torch.where(l > 0, l, torch.ones_like(l))[..., None]
        o = torch.nn.functional.layer_norm(o.reshape(N, F) @ p["wo"], (F,), p["w_post"],
                                           p["b_post"], 1e-6)
        y = y + p["res_scale"] * torch.sigmoid(z @ p["wg"]) * o
        z = torch.nn.functional.layer_norm(y, (F,), p["w_pre"], p["b_pre"], 1e-6)
    return y, z


def leaves(x, par):
    return [x] + [par[a][k] for a in sorted(par) for k in sorted(par[a])]


def grads(fn, x, par, dy, dz):
    par = {a: {k: v.detach().requires_grad_(True) for k, v in p.items()} for a, p in par.items()}
    x = x.detach().requires_grad_(True)
    y, z = fn(x, par)
    return (y.detach(), z.detach()), torch.autograd.grad([y, z], leaves(x, par), [dy, dz])


def rel_err(a, b):
    b = b.double().cpu()
    return float((a.double().cpu() - b).norm() / b.norm())


def test_two_layers_against_float64():
    """Every step adds a relative error of at most the row bound G = 32 u, the
    attention's C (about 2^-13 here: scores below 32, degrees up to 200) or a
    product's (F + 2) u; two layers forward and backward chain 12 such steps, and a
    nearly constant row magnifies what enters a norm by at most 16 (its row's
    length over its spread): 12 * 16 * 2^-13 is the bound of the norm of the error
    over the norm of the result, far below what a wrong term would give (order 1)."""
    g, rel, x, par, graph, dy, dz = setup()
    (y, z), got = grads(lambda a, p: forward(g, rel, a, p, False), x, par, dy, dz)
    cpu = {a: {k: v.double().cpu() for k, v in p.items()} for a, p in par.items()}
    (ry, rz), ref = grads(lambda a, p: plain(a, p, graph), x.double().cpu(), cpu,
                          dy.double().cpu(), dz.double().cpu())
    bound = 12 * 16 * 2.0 ** -13
    assert rel_err(y, ry) <= bound and rel_err(z, rz) <= bound
    for a, b in zip(got, ref):
        assert rel_err(a, b) <= bound


def test_checkpoints_change_the_gradients_by_their_rounding_only():
    """The forward pass is the same bit for bit.  A packed element is off by at
    most s / 2 = max / 254, so a score by D * scale * max^2 / 127: below 0.2 here;
    gradients then differ by that order, and those that do not pass through the
    attention of their layer (the last layer's norms) not at all."""
    g, rel, x, par, graph, dy, dz = setup()
    (y, z), a = grads(lambda b, p: forward(g, rel, b, p, False), x, par, dy, dz)
    (y8, z8), b = grads(lambda c, p: forward(g, rel, c, p, True), x, par, dy, dz)
    assert torch.equal(y, y8) and torch.equal(z, z8)
    names = ["x"] + [f"{layer}.{k}" for layer in sorted(par) for k in sorted(par[layer])]
    for name, s, t in zip(names, a, b):
        if name in ("1.w_post", "1.b_post", "1.res_scale", "1.w_pre", "1.b_pre", "1.wo", "1.wg"):
            assert torch.equal(s, t), name
        else:
            assert 0 < rel_err(t, s) < 0.2, name


@pytest.mark.parametrize("checkpoint8", [False, True])
def test_training_step_in_a_cuda_graph(checkpoint8):
    """A step captured on a side stream while no eager graph of its leaves lives
    replays to the eager step's bits, twice."""
    g, rel, x, par, graph, dy, dz = setup()
    fn = lambda a, p: forward(g, rel, a, p, checkpoint8)  # noqa: E731
    eager = grads(fn, x, par, dy, dz)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(fn, x, par, dy, dz)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        static = grads(fn, x, par, dy, dz)
    for _ in range(2):
        cg.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager[0] + eager[1], static[0] + static[1]):
        assert torch.equal(a, b)


def test_no_gate_no_bias_no_projection():
    import graph_neural_network_gb300 as gnn
    g, rel, x, par, graph, dy, dz = setup()
    q, k, v = (x.view(N, H, D).clone().requires_grad_(True) for _ in range(3))
    y, z = gnn.transformer_layer(g, x, q, k, v, kind=("none", "rms"), checkpoint8=True)
    out, _ = gnn.transformer_forward(g, q.detach(), k.detach(), v.detach())
    want, wz = gnn.norm_residual_forward(x, out.view(N, F), kind=("none", "rms"))
    assert torch.equal(y.detach(), want) and torch.equal(z.detach(), wz)
    z.sum().backward()
    assert all(torch.isfinite(t.grad).all() for t in (q, k, v))
    with pytest.raises(ValueError):
        gnn.transformer_layer(g, x, q, k, v, rel=rel)


def test_offsets_past_32_bits():
    """A ring of 8.5M nodes with 512-byte rows: every row has one edge, so the
    attention copies its source's value and the gradients are known; rows beyond
    the first 4 GB go through every operator."""
    import graph_neural_network_gb300 as gnn
    n, D = 8_500_001, 128
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of free device memory")
    rp = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    ci = torch.roll(torch.arange(n, dtype=torch.int32, device="cuda"), -1)
    g = gnn.Graph(rp, ci)
    rel = gnn.RelPos(g, torch.arange(n, dtype=torch.int32, device="cuda") % 1000)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, 1, D, generator=gen, device="cuda")
    bias = torch.ones(32, 1, device="cuda")
    out, lse = gnn.transformer_rel_forward(g, rel, x, x, x, bias)
    assert torch.equal(out, torch.roll(x, -1, 0))
    dq, dk, dv, db = gnn.transformer_rel_backward(g, rel, x, x, x, bias, lse, x)
    # one weight a row: exp(e - lse) with both rounded, e below 32: 2^-17 covers it
    top = float(x.abs().max())
    assert float((dv - torch.roll(x, 1, 0)).abs().max()) <= 2.0 ** -17 * top
    del dq, dk, dv, out
    (p,) = gnn.pack8(x)
    tail = slice(n - 1000, n)
    (q,) = gnn.pack8(x[tail].contiguous())
    assert torch.equal(p.values[tail], q.values) and torch.equal(p.scale[tail], q.scale)
    dq, dk, dv = gnn.transformer_backward8(g, p, p, p, x)
    assert float((dv - torch.roll(x, 1, 0)).abs().max()) <= 2.0 ** -17 * top
    del dq, dk, dv
    rows = x.view(n, D)
    y, z = gnn.norm_residual_forward(rows, rows, rows)
    ty, tz = gnn.norm_residual_forward(*(rows[tail].contiguous(),) * 3)
    assert torch.equal(y[tail], ty) and torch.equal(z[tail], tz)
    del z
    gr = gnn.norm_residual_backward(y, rows, rows, rows, rows)
    tr = gnn.norm_residual_backward(ty, *(rows[tail].contiguous(),) * 4)
    for k in ("dx", "do", "dgate"):
        assert torch.equal(gr[k][tail], tr[k]), k


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    import graph_neural_network_gb300 as gnn
    rp, ci = workload.chung_lu(50_000, 2.1, 20.0, 10_000.0, 3)
    g = device_graph(dict(row_ptr=rp, col=ci))
    n = len(rp) - 1
    rel = gnn.RelPos(g, torch.arange(n, dtype=torch.int32, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(1)
    sets = [[torch.randn(n, 4, 32, generator=gen, device="cuda") for _ in range(4)]
            for _ in range(2)]
    bias = torch.randn(32, 4, generator=gen, device="cuda")

    def step(a, **kw):
        q, k, v, d = a
        out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, bias, **kw)
        r = gnn.transformer_rel_backward(g, rel, q, k, v, bias, lse, d, **kw)
        p = gnn.pack8(q, k, v, **kw)
        return (out, lse) + r + tuple(gnn.transformer_backward8(g, *p, d, rel=rel, bias=bias, **kw))

    alone = [step(a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        both = [step(a, stream=s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            assert all(torch.equal(a, b) for a, b in zip(x, y))


def test_rel_and_bias_go_together_in_autograd():
    import graph_neural_network_gb300 as gnn
    g, rel, x, par, graph, dy, dz = setup()
    q = x.view(N, H, D)
    with pytest.raises(ValueError):
        gnn.TransformerCheckpoint8.apply(g, None, q, q, q, par[0]["bias"], None)
    with pytest.raises(ValueError):
        gnn.TransformerCheckpoint8.apply(g, rel, q, q, q, None, None)


def test_autograd_without_the_second_norm():
    import graph_neural_network_gb300 as gnn
    g, rel, x, par, graph, dy, dz = setup()
    a, o, w = (t.clone().requires_grad_(True) for t in (x, dz, par[0]["w_post"]))
    y, z = gnn.NormResidual.apply(a, o, None, w, None, None, None, None, ("rms", "none"), 1e-6)
    assert z is None
    got = torch.autograd.grad(y, (a, o, w), dy)
    want = gnn.norm_residual_backward(None, dz, dy, w_post=par[0]["w_post"], kind=("rms", "none"))
    for t, k in zip(got, ("dx", "do", "dw_post")):
        assert torch.equal(t, want[k]), k


def test_nothing_is_allocated_with_outputs_and_workspaces_given():
    import graph_neural_network_gb300 as gnn
    g, rel, x, par, graph, dy, dz = setup()
    q, k, v, d = (t.view(N, H, D) for t in (x, dy, dz, x))
    b, w = par[0]["bias"], par[0]["w_post"]
    ws = rel.workspace(H, D, torch.float32)
    out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b, ws=ws)
    dq, dk, dv, db = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, d, ws=ws)
    packed = gnn.pack8(q, k, v)
    back = gnn.unpack8(packed[0])
    y, z = gnn.norm_residual_forward(x, dy, dz, w, w_pre=w)
    grads = gnn.norm_residual_backward(y, dy, dy, dz, dz, w, w_pre=w)
    nws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in (out, lse, dq, dk, dv, db, back, y, z)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    gnn.transformer_rel_forward(g, rel, q, k, v, b, out=out, lse=lse, ws=ws)
    gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, d, dq=dq, dkey=dk, dval=dv, dbias=db,
                                 ws=ws)
    gnn.pack8(q, k, v, out=packed)
    gnn.unpack8(packed[0], out=back)
    gnn.norm_residual_forward(x, dy, dz, w, w_pre=w, y=y, z=z)
    gnn.norm_residual_backward(y, dy, dy, dz, dz, w, w_pre=w, grads=grads, ws=nws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    for a, c in zip(want, (out, lse, dq, dk, dv, db, back, y, z)):
        assert torch.equal(a, c)
    # the comparisons above allocate their own results
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    gnn.transformer_backward8(g, *packed, d, rel=rel, bias=b, dq=dq, dkey=dk, dval=dv, dbias=db,
                              ws=ws)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    with pytest.raises(gnn.GnnError):
        rel.workspace(1, 256, torch.float32)
