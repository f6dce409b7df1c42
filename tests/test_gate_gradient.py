"""The gradient of nearly open and nearly closed gates.

dgate = u n (1 - sigmoid(g)) with u = dy scale sigmoid(g); without norms n = o and
dgate = dy scale o s c, s = 1 / (1 + e), c = e s, e = exp(-g): four products and
two factors that are accurate relative to themselves.  e is 2^t of t = -g log2(e),
whose rounded constant and product put it off by 2 u |g| relative, the
exponential by 2^-22 = 4 u, the reciprocal by 2 u, the sum and the products by u
each: below (2 |g| + 16) u in all, u = 2^-24, and the sum over a row of F terms of
one sign adds (F / 4 + 5) u at most (a vector in sequence, then a tree).
"""
import numpy as np
import pytest
import torch

from layer_ref import U

pytestmark = pytest.mark.gpu
GATES = [-80.0, -40.0, -20.0, -9.5, -3.0, -0.5, 0.0, 0.5, 3.0, 7.0, 10.0, 12.0, 15.0, 17.0, 20.0,
         28.0, 40.0, 60.0, 80.0]


def factor(g):
    """sigmoid(g) (1 - sigmoid(g)) in float64, without a difference."""
    return np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))) ** 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_element_gates(dtype):
    import graph_neural_network_gb300 as gnn
    n, F = 200, 64
    gen = torch.Generator("cuda").manual_seed(1)
    o, dy = (torch.randn(n, F, generator=gen, device="cuda").to(dtype) for _ in range(2))
    scale = torch.randn(F, generator=gen, device="cuda")
    g = torch.tensor(GATES, device="cuda").to(dtype)[
        torch.randint(len(GATES), (n, F), generator=gen, device="cuda")]
    got = gnn.norm_residual_backward(None, o, dy, gate=g, scale=scale, kind="none")["dgate"]
    g64 = g.double().cpu().numpy()
    want = (dy.double() * scale.double() * o.double()).cpu().numpy() * factor(g64)
    half = 0.0 if dtype == torch.float32 else 2.0 ** -8
    err = np.abs(got.double().cpu().numpy() - want)
    bound = ((2 * np.abs(g64) + 16) * U * (1 + half) + half) * np.abs(want) + 1e-37
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("F", [8, 512])
def test_row_gates(F):
    """Terms of one sign, so that the sum is as accurate as they are."""
    import graph_neural_network_gb300 as gnn
    n = 10 * len(GATES)
    gen = torch.Generator("cuda").manual_seed(2)
    o, dy = (torch.rand(n, F, generator=gen, device="cuda") + 0.5 for _ in range(2))
    g = torch.tensor(GATES * 10, device="cuda")[:, None].contiguous()
    got = gnn.norm_residual_backward(None, o, dy, gate=g, kind="none")["dgate"]
    g64 = g.double().cpu().numpy()
    want = (dy.double() * o.double()).sum(1, keepdim=True).cpu().numpy() * factor(g64)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = (2 * np.abs(g64) + 21 + F / 4) * U * np.abs(want) + 1e-37
    assert (err <= bound).all(), float((err / bound).max())


def test_with_norms():
    """The normed row is off by 20 u of itself (its sums, square root and product) besides,
    relative to its largest element (layer norm: the mean's error); gates of either end."""
    import graph_neural_network_gb300 as gnn
    n, F = 150, 48
    gen = torch.Generator("cuda").manual_seed(3)
    o, dy = (torch.randn(n, F, generator=gen, device="cuda") for _ in range(2))
    g = torch.tensor(GATES, device="cuda")[
        torch.randint(len(GATES), (n, F), generator=gen, device="cuda")]
    for kind in ("rms", "layer"):
        got = gnn.norm_residual_backward(None, o, dy, gate=g, kind=(kind, "none"))["dgate"]
        x = o.double().cpu().numpy()
        if kind == "layer":
            x = x - x.mean(1, keepdims=True)
        hat = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6)
        g64 = g.double().cpu().numpy()
        f = np.abs(dy.double().cpu().numpy()) * factor(g64)
        err = np.abs(got.double().cpu().numpy() - np.sign(dy.cpu().numpy()) * f * hat)
        bound = f * U * ((2 * np.abs(g64) + 36) * np.abs(hat) +
                         20 * np.abs(hat).max(1, keepdims=True)) + 1e-37
        assert (err <= bound).all(), (kind, float((err / bound).max()))
