"""The operators round a layer's projections run together as a layer runs them: the 8-bit
norm before the projections, rotary positions on views of their result, the attention and
its norms, and a feed-forward half of experts; eagerly, captured, and from several host
threads.

Tolerance of the float32 layer against float64: a stage's result is off by 2^-20 of its norm
at most (its own tests; the library's float32 products of 64 terms likewise), a softmax over
scores of size 8 multiplies what enters it by 8 at most, the other stages by 2, and there are
8 of them before the gradient's 8: 16 * 2^-20 * 8 < 1.3e-4 of the norm."""
import threading

import pytest
import torch

from workload import testgraphs
from gpu_util import device_graph

pytestmark = pytest.mark.gpu

N, H, D, E, K = 96, 2, 32, 4, 2
F = H * D


def setup(seed=1):
    rp, ci = testgraphs.with_in_degrees([0, 1, 7] + [5] * (N - 3), n_nodes=N, seed=2)
    g = device_graph(dict(row_ptr=rp, col=ci))
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    t = dict(x=normal(N, F), o=normal(N, F), w=1 + normal(F, std=0.1),
             wqkv=normal(F, 3 * F, std=F ** -0.5), wo=normal(F, F, std=F ** -0.5),
             w_pre=1 + normal(F, std=0.1), up=normal(E, F, F, std=F ** -0.5),
             weights=torch.rand(N, K, generator=gen, device="cuda"))
    pos = torch.randint(0, 100_000, (N,), generator=gen, device="cuda").int()
    ids = torch.randint(-1, E, (N, K), generator=gen, device="cuda")
    return g, t, pos, ids


def layer(g, t, pos, ids, rope, at):
    """at: the first rows of the experts' segments, on the host."""
    import graph_neural_network_gb300 as gnn
    y, z = gnn.AddNorm8.apply(t["x"], t["o"], t["w"], "int8", 32, 1e-6)
    q, k, v = (z @ t["wqkv"]).view(N, 3, H, D).unbind(1)
    y, z = gnn.transformer_layer(g, y, q, k, v, w_pre=t["w_pre"], kind=("none", "rms"),
                                 project=lambda a: a.flatten(1) @ t["wo"], rope=rope, pos=pos)

    def products(xs, plan):
        rows = [torch.tanh(xs[at[e]:at[e + 1]] @ t["up"][e]) for e in range(E)]
        return torch.cat(rows + [xs[at[E]:]])

    plan = gnn.Experts(ids, E, align=8)
    return gnn.expert_layer(plan, z, products, t["weights"], y)


def plain(g, t, pos, ids, rope):
    """The same in float64, the rounding to 8 bits as the library decided it."""
    import graph_neural_network_gb300 as gnn
    _, z8 = gnn.add_norm8_forward(t["x"].float().detach(), t["o"].float().detach(),
                                  t["w"].float().detach(), group=32)
    rp, src = g.row_ptr.long(), g.col_idx.long()
    dst = torch.repeat_interleave(torch.arange(N, device="cuda"), rp.diff())

    def norm(a, w):
        return a * torch.rsqrt((a * a).mean(-1, keepdim=True) + 1e-6) * w

    y = t["x"] + t["o"]
    z = norm(y, t["w"])
    z = z + (gnn.unpack8(z8).view(N, F).double() - z).detach()
    q, k, v = (z @ t["wqkv"]).view(N, 3, H, D).unbind(1)
    angle = pos.double()[:, None] * torch.tensor(rope.freqs, dtype=torch.float64, device="cuda")
    c, s = (rope.amplitude * f(angle)[:, None] for f in (torch.cos, torch.sin))

    def turn(a):
        h = rope.dim // 2
        u, w = a[..., :h], a[..., h:2 * h]
        return torch.cat([u * c - w * s, u * s + w * c, a[..., 2 * h:]], -1)

    q, k = turn(q), turn(k)
    e = torch.exp((q[dst] * k[src]).sum(-1) * D ** -0.5)
    total = torch.zeros(N, H, dtype=torch.float64, device="cuda").index_add(0, dst, e)
    out = torch.zeros(N, H, D, dtype=torch.float64, device="cuda").index_add(
        0, dst, e[..., None] * v[src])
    out = out / torch.where(total > 0, total, 1.0)[..., None]
    y = y + out.flatten(1) @ t["wo"]
    z = norm(y, t["w_pre"])
    for k_ in range(K):
        for e_ in range(E):
            mine = torch.nonzero(ids[:, k_] == e_).squeeze(1)
            y = y.index_add(0, mine, t["weights"][mine, k_, None]
                            * torch.tanh(z[mine] @ t["up"][e_]))
    return y


def test_a_layer_and_its_gradients():
    import graph_neural_network_gb300 as gnn
    g, t, pos, ids = setup()
    rope = gnn.Rope(D // 2, scaling="yarn", factor=8.0, length=2048)
    at = gnn.Experts(ids, E, align=8).offsets.tolist()
    dy = torch.randn(N, F, generator=torch.Generator("cuda").manual_seed(9), device="cuda")
    mine = {k: v.clone().requires_grad_(True) for k, v in t.items()}
    ref = {k: v.double().requires_grad_(True) for k, v in t.items()}
    y = layer(g, mine, pos, ids, rope, at)
    got = torch.autograd.grad(y, list(mine.values()), dy)
    y6 = plain(g, ref, pos, ids, rope)
    want = torch.autograd.grad(y6, list(ref.values()), dy.double())
    for name, a, b in zip(["y", *t], (y, *got), (y6, *want)):
        assert (a.double() - b).norm() <= 1.3e-4 * b.norm(), name


def test_serving_rows_captured():
    """Norm, 8-bit rows by expert, their combination and the next positions in one graph,
    replayed on new inputs: as called eagerly."""
    import graph_neural_network_gb300 as gnn
    g, t, pos, ids = setup()
    rope = gnn.Rope(D)
    b = {k: v.bfloat16() for k, v in t.items() if k in ("x", "o")}
    w, weights = t["w"], t["weights"]

    def step():
        y, z8 = gnn.add_norm8_forward(b["x"], b["o"], w, fmt="e4m3")
        plan = gnn.Experts(ids, E)
        rows = gnn.expert_dispatch_forward(plan, z8)
        y = gnn.expert_combine_forward(plan, gnn.unpack8(rows, torch.bfloat16).view(-1, F),
                                       weights, y)
        return y, *gnn.rope_forward(rope, pos, y.view(N, H, D))

    step()
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        kept = step()
    for seed in (3, 4):
        _, new, p, i = setup(seed)
        for k in b:
            b[k].copy_(new[k])
        pos.copy_(p)
        ids.copy_(i)
        weights.copy_(new["weights"])
        cg.replay()
        torch.cuda.synchronize()
        for a, c in zip(kept, step()):
            assert torch.equal(a, c)


def test_second_derivatives_are_refused():
    import graph_neural_network_gb300 as gnn
    _, t, pos, ids = setup()
    x = t["x"].clone().requires_grad_(True)
    plan = gnn.Experts(ids, E)
    for fn in (lambda: gnn.RotaryPositions.apply(gnn.Rope(D), pos, x.view(N, H, D))[0],
               lambda: gnn.AddNorm8.apply(x, None, None, "int8", None, 1e-6),
               lambda: gnn.ExpertDispatch.apply(plan, x),
               lambda: gnn.ExpertCombine.apply(plan, gnn.ExpertDispatch.apply(plan, x),
                                               t["weights"], None)):
        (first,) = torch.autograd.grad((fn() ** 2).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable|differentiated twice"):
            ((first * first).sum() + (x * x).sum()).backward()


def test_several_threads():
    """Calls whose kernels need different amounts of shared memory and blocks, each thread
    on its own stream."""
    import graph_neural_network_gb300 as gnn
    gen = torch.Generator("cuda").manual_seed(1)

    def work(width, seed):
        n = 300
        y, dy, dz = (torch.randn(n, width, generator=gen, device="cuda") for _ in range(3))
        w = torch.ones(width, device="cuda")
        ids = torch.randint(0, seed + 3, (n, 2), generator=gen, device="cuda")
        wt = torch.rand(n, 2, generator=gen, device="cuda")
        pos = torch.arange(n, dtype=torch.int32, device="cuda") * 7

        def call(**kw):
            plan = gnn.Experts(ids, seed + 3, align=4, **kw)
            xs = gnn.expert_dispatch_forward(plan, y, **kw)
            return (*gnn.add_norm8_backward(y, dy, dz, w, **kw),
                    gnn.add_norm8_forward(y, dy, w, **kw)[1].values, plan.order, xs,
                    gnn.expert_combine_forward(plan, xs, wt, **kw),
                    *gnn.rope_forward(gnn.Rope(16), pos, y.view(n, width // 32, 32), **kw))
        return call

    calls = [work(wd, s) for s, wd in enumerate((64, 256, 1024, 2048, 4096, 8192))]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        stream = torch.cuda.Stream()
        for _ in range(20):
            got = calls[k](stream=stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                bad.append(k)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(calls))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad
