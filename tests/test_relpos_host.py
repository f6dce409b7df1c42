"""Relative position buckets, host side (CPU only): the bounds of the
logarithmic rule against whole-number arithmetic, and the refusals that come
before any GPU work."""
import ctypes

import pytest
import torch

import layer_ref


@pytest.fixture(scope="module")
def lib():
    from graph_neural_network_gb300 import build, _native
    build.build()
    return _native.load()


@pytest.mark.parametrize("n, dist", [(2, 2), (2, 2**31 - 1), (3, 2), (16, 128), (16, 64),
                                     (17, 100), (32, 128), (64, 33), (128, 65), (127, 10**9),
                                     (128, 2**31 - 1), (32, 8192)])
def test_log_bounds_are_exact(lib, n, dist):
    table = (ctypes.c_int32 * n)()
    assert lib.gnn_rel_log_bounds(n, dist, table) == 0
    assert list(table) == layer_ref.log_bounds(n, dist)


def test_log_bounds_powers_of_two(lib):
    # 16 buckets to distance 128: the borders 8 * 2^(k/2), whole at even k
    table = (ctypes.c_int32 * 16)()
    assert lib.gnn_rel_log_bounds(16, 128, table) == 0
    assert list(table) == [0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91]


@pytest.mark.parametrize("n, dist", [(1, 10), (0, 10), (129, 1000), (16, 8), (2, 1), (16, -5)])
def test_log_bounds_refusals(lib, n, dist):
    table = (ctypes.c_int32 * 256)()
    assert lib.gnn_rel_log_bounds(n, dist, table) == 1
    assert lib.gnn_rel_log_bounds(16, 128, None) == 1


def test_calls_without_a_graph_are_refused(lib):
    P = ctypes.c_void_p
    out = P()
    table = (ctypes.c_int32 * 4)(0, 1, 2, 3)
    assert lib.gnn_rel_prepare(None, P(16), table, 4, 1, P(256), 1 << 20, None,
                               ctypes.byref(out)) == 1
    assert lib.gnn_rel_prepare(None, P(16), table, 4, 1, P(256), 1 << 20, None, None) == 1
    assert lib.gnn_rel_buffer_bytes(None) == 0
    assert lib.gnn_rel_buckets(None) == 0
    assert lib.gnn_rel_arrays(None, None, 2) == 1
    assert lib.gnn_rel_destroy(None) == 0
    assert lib.transformer_rel_workspace_bytes(None, None, 1, 16, 0) == 0
    a = [P(256)] * 3
    assert lib.transformer_rel_forward(None, None, 1, 16, 0, *a, 1.0, *[P(256)] * 4, 1 << 20,
                                       None) == 1
    assert lib.transformer_rel_backward(None, None, 1, 16, 0, *a, 1.0, *[P(256)] * 8, 1 << 20,
                                        None) == 1


class _FakeGraph:
    n = 6
    device = torch.device("cuda", 0)


def test_binding_checks_positions_and_rel(lib):
    import graph_neural_network_gb300 as gnn
    g = _FakeGraph()
    for pos, err in ((torch.zeros(5, dtype=torch.int32), ValueError),     # short
                     (torch.zeros(6, dtype=torch.int64), TypeError),
                     (torch.zeros(6, dtype=torch.int32), ValueError),     # a host tensor
                     ([0] * 6, TypeError)):
        with pytest.raises(err):
            gnn.RelPos(g, pos)
    with pytest.raises(TypeError):
        gnn._rel_bias(g, "rel", torch.zeros(32, 2), 2)
    rel = object.__new__(gnn.RelPos)
    rel.graph, rel.buckets = g, 32
    for bias, err in ((torch.zeros(32, 3), ValueError), (torch.zeros(31, 2), ValueError),
                      (torch.zeros(32, 2, dtype=torch.int32), TypeError),
                      (torch.zeros(32, 2), ValueError)):                  # a host tensor
        with pytest.raises(err):
            gnn._rel_bias(g, rel, bias, 2)
    with pytest.raises(ValueError):
        gnn._rel_bias(_FakeGraph(), rel, torch.zeros(32, 2), 2)         # another graph
