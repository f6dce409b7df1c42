"""The backward passes are kernels without a derivative of their own: asking for one is an
error, not a gradient with terms missing."""
import pytest
import torch

from workload import testgraphs
from gpu_util import device_graph

pytestmark = pytest.mark.gpu


def cases():
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([3] * 10, n_nodes=10, seed=1)
    g = device_graph(dict(row_ptr=rp, col=ci))
    rel = gnn.RelPos(g, torch.arange(10, dtype=torch.int32, device="cuda"), 8, 8)
    gen = torch.Generator("cuda").manual_seed(1)

    def leaf(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").requires_grad_(True)

    x, q, k, v, b = leaf(10, 16), leaf(10, 1, 16), leaf(10, 1, 16), leaf(10, 1, 16), leaf(8, 1)
    a, c = leaf(1, 16), leaf(1, 16)
    return {
        "rel": (lambda: gnn.TransformerRelAggregate.apply(g, rel, q, k, v, b, None), q),
        "checkpoint": (lambda: gnn.TransformerCheckpoint8.apply(g, rel, q, k, v, b, None), q),
        "norms": (lambda: gnn.NormResidual.apply(x, q.view(10, 16), None, None, None, None, None,
                                                 None, "rms", 1e-6)[1], q),
        "layer": (lambda: gnn.transformer_layer(g, x, q, k, v, rel=rel, bias=b)[1], q),
        "transformer": (lambda: gnn.TransformerAggregate.apply(g, q, k, v, None), q),
        "gat": (lambda: gnn.GATAggregate.apply(g, q, a, c, 0.2), q),
        "gatv2": (lambda: gnn.GATv2Aggregate.apply(g, q, k, a, 0.2), q),
        "gcn": (lambda: gnn.GCNAggregate.apply(g, x, "sym"), x),
        "reduce": (lambda: gnn.ReduceAggregate.apply(g, x, "max"), x),
    }


@pytest.mark.parametrize("name", ["rel", "checkpoint", "norms", "layer", "transformer", "gat",
                                  "gatv2", "gcn", "reduce"])
def test_a_second_derivative_is_refused(name):
    fn, leaf = cases()[name]
    y = fn()
    (first,) = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
    plain = torch.autograd.grad((fn() ** 2).sum(), leaf)[0]
    assert torch.equal(first.detach(), plain)
    # a gradient penalty beside a term that does have a second derivative
    with pytest.raises(RuntimeError, match="once_differentiable|differentiated twice"):
        ((first * first).sum() + (leaf * leaf).sum()).backward()
