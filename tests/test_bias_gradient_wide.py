"""The bias gradient where its tables hold float32 sums alone (many buckets and heads as
narrow as a lane): six million edges, most into two buckets.

A term de = alpha (da - Delta) is off by under ten half steps u = 2^-24 in the root of the mean
square (a dot product in each factor, an exponential, two subtractions), which N independent
terms keep as sqrt(sum de^2).  A column of m terms of random sign adds one after the
other: an addition is off by at most u / sqrt(3) of the partial sum on average, in the root of
the mean square, and that grows as the root of the number of terms, so the column is off by
u sqrt(m / 6) of its own sqrt(sum de^2).  Every warp has `columns` of them a head, over 2
blocks of 8 warps an SM, and all of the edges may lie in one bucket.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H, D, dtype, buckets, columns", [
    (32, 8, torch.bfloat16, 64, 1), (8, 16, torch.bfloat16, 128, 4),
    (32, 4, torch.float32, 128, 1)])
def test_sums_over_six_million_edges(H, D, dtype, buckets, columns):
    import graph_neural_network_gb300 as gnn
    n, deg = 300_000, 20
    gen = torch.Generator("cuda").manual_seed(5)
    rp = torch.arange(0, n * deg + 1, deg, dtype=torch.int32, device="cuda")
    ci = torch.randint(n, (n * deg,), generator=gen, device="cuda", dtype=torch.int32)
    pos = torch.randint(1 << 16, (n,), generator=gen, device="cuda", dtype=torch.int32)
    g = gnn.Graph(rp, ci)
    rel = gnn.RelPos(g, pos, buckets, 128)
    q, k, v, d = (torch.randn(n, H, D, generator=gen, device="cuda").to(dtype) for _ in range(4))
    b = torch.randn(buckets, H, generator=gen, device="cuda")
    _, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
    got = gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, d)[3].double()
    bucket = rel.arrays()[0].long().view(n, deg)
    want, square = (torch.zeros(buckets, H, dtype=torch.float64, device="cuda") for _ in range(2))
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
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    m = n * deg / (sms * 2 * 8 * columns)
    error = float((got - want).norm() / square.sum().sqrt())
    assert error <= (10 ** 2 + m / 6) ** 0.5 * 2.0 ** -24, error * 2 ** 24
