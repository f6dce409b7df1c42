"""Two graph-transformer layers against float64, close enough to miss no term.

A step of the layer (a projection, the attention, a norm, the sum) rounds each element by
the sum of at most 64 products, roundings of either sign: sqrt(64) half steps of
float32, 2^-21 of the step's result in the norm.  Two layers forward and backward chain 12
of them, and a nearly constant row magnifies what enters a norm by at most 16 (its length
over its spread): 12 * 16 * 2^-21 of the norm of each result.  What that bound must not
miss is shown on the CPU: one edge of one row left out of the attention, or a hundredth of
what the norms' means add to their gradients, lies outside it.
"""
import numpy as np
import pytest
import torch

import test_transformer_layer as layer
import workload
from workload import testgraphs

BOUND = 12 * 16 * 2.0 ** -21
N, H, D, F = layer.N, layer.H, layer.D, layer.F


def host_setup(seed=3):
    """setup()'s inputs on the CPU in float64 (its buckets from the same rule)."""
    rp, ci = testgraphs.with_in_degrees([0, 1, 5, 70, 200], n_nodes=N, seed=seed)
    pos = layer.positions(N, seed, 60)
    import layer_ref
    bucket = layer.edge_buckets(rp, ci, pos, layer_ref.log_bounds(8, 32), True)

    def t(stream, *shape, std=1.0):
        return torch.from_numpy(workload.normal_f32(seed, stream, shape, std)).double()

    par = {}
    for a in range(2):
        b = 20 * a
        par[a] = dict(wqkv=t(b + 2, F, 3 * F, std=F ** -0.5), wo=t(b + 3, F, F, std=F ** -0.5),
                      wg=t(b + 4, F, F, std=F ** -0.5), bias=t(b + 5, 16, H),
                      w_post=1 + t(b + 6, F, std=0.1), b_post=t(b + 7, F, std=0.1),
                      res_scale=0.5 + t(b + 8, F, std=0.1), w_pre=1 + t(b + 9, F, std=0.1),
                      b_pre=t(b + 10, F, std=0.1))
    return t(1, N, F), par, (rp, ci, bucket), t(60, N, F), t(61, N, F)


def outside(got, want):
    return [k for k, (a, b) in enumerate(zip(got, want)) if not layer.rel_err(a, b) <= BOUND]


def test_the_bound_sees_one_edge_and_one_term(monkeypatch):
    x, par, (rp, ci, bucket), dy, dz = host_setup()
    whole = layer.grads(lambda a, p: layer.plain(a, p, (rp, ci, bucket)), x, par, dy, dz)
    for e in (int(rp[4]), int(rp[5]) - 1, int(rp[-1]) - 1):  # of the row of 200 and of a short one
        rp2 = rp.copy()
        row = int(np.searchsorted(rp, e, side="right")) - 1
        rp2[row + 1:] -= 1
        less = layer.grads(lambda a, p: layer.plain(a, p, (rp2, np.delete(ci, e),
                                                           np.delete(bucket, e))), x, par, dy, dz)
        assert outside(less[0], whole[0]) and len(outside(less[1], whole[1])) > 10
    true_norm = torch.nn.functional.layer_norm

    def no_mean(t, shape, w, b, eps):
        mean = t.mean(-1, keepdim=True)                      # adds 0, and a gradient
        return true_norm(t, shape, w, b, eps) + (mean.detach() - mean) * 0.01

    monkeypatch.setattr(torch.nn.functional, "layer_norm", no_mean)
    wrong = layer.grads(lambda a, p: layer.plain(a, p, (rp, ci, bucket)), x, par, dy, dz)
    assert not outside(wrong[0], whole[0]) and len(outside(wrong[1], whole[1])) > 10


@pytest.mark.gpu
def test_two_layers():
    g, rel, x, par, graph, dy, dz = layer.setup()
    assert rel.bounds and np.array_equal(graph[2], host_setup()[2][2])
    got = layer.grads(lambda a, p: layer.forward(g, rel, a, p, False), x, par, dy, dz)
    hx, hpar, hgraph, hdy, hdz = host_setup()
    want = layer.grads(lambda a, p: layer.plain(a, p, hgraph), hx, hpar, hdy, hdz)
    assert not outside(got[0], want[0]), [layer.rel_err(a, b) for a, b in zip(got[0], want[0])]
    assert not outside(got[1], want[1]), [layer.rel_err(a, b) for a, b in zip(got[1], want[1])]
