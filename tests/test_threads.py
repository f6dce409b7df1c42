"""Calls of several host threads at once, each on a stream of its own.  Their kernels are the
same functions with tables of different sizes in shared memory; the size that one thread's
call needs must not limit another's."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from workload import testgraphs
from gpu_util import device_graph

pytestmark = pytest.mark.gpu

# Waits 1 ms after a function's limit of shared memory (attribute 8) is set, so that another
# thread's call falls between that and the launch.
SLOW = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <unistd.h>
static int refusing;
void refuse(int on) { refusing = on; }
int cudaFuncSetAttribute(const void* f, int attr, int value) {
  static int (*real)(const void*, int, int);
  if (!real) {
    void* h = dlopen("libcudart.so.13", RTLD_LAZY | RTLD_NOLOAD);
    real = (int (*)(const void*, int, int))dlsym(h, "cudaFuncSetAttribute");
  }
  const int r = real(f, attr, attr == 8 && refusing ? 1 << 30 : value);
  if (attr == 8) usleep(1000);
  return r;
}
"""


def backward_calls(checkpoints):
    """Backward calls of 128, 40 and 64 buckets (147, 46 and 74 KB of shared memory in the
    same kernel), with everything that they write given."""
    import graph_neural_network_gb300 as gnn
    rp, ci = testgraphs.with_in_degrees([5] * 60, n_nodes=64, seed=1)
    g = device_graph(dict(row_ptr=rp, col=ci))
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v, d = (torch.randn(64, 1, 8, generator=gen, device="cuda").bfloat16()
                  for _ in range(4))
    packed = gnn.pack8(q, k, v)

    def call(buckets):
        rel = gnn.RelPos(g, pos, buckets, 200)
        bias = torch.linspace(-1, 1, buckets, device="cuda")[:, None].contiguous()
        ws = rel.workspace(1, 8, torch.bfloat16)
        got = dict(dq=torch.empty_like(q), dkey=torch.empty_like(q), dval=torch.empty_like(q),
                   dbias=torch.empty_like(bias))
        _, lse = gnn.transformer_rel_forward(g, rel, q, k, v, bias)
        if checkpoints:
            return lambda **kw: gnn.transformer_backward8(g, *packed, d, rel=rel, bias=bias, ws=ws,
                                                          **got, **kw)
        return lambda **kw: gnn.transformer_rel_backward(g, rel, q, k, v, bias, lse, d, ws=ws,
                                                         **got, **kw)

    return [call(b) for b in (128, 40, 64)]


def aggregation_calls(name):
    """Forward calls over nodes of 13,000, 14,500 and 16,000 edges that each go to one block
    with its edge list (52 to 64 KB of shared memory in the same kernel)."""
    import graph_neural_network_gb300 as gnn

    def call(deg):
        rp = torch.tensor([0] + [deg] * 64, dtype=torch.int32, device="cuda")
        ci = torch.arange(deg, dtype=torch.int32, device="cuda") % 64
        g = gnn.Graph(rp, ci, gnn.Tiling(64, 16384, 2048))
        x = torch.linspace(-1, 1, 64 * 32, device="cuda").view(64, 1, 32).contiguous()
        out, lse = torch.empty_like(x), torch.empty(64, 1, device="cuda")
        a = torch.linspace(-1, 1, 32, device="cuda")[None]
        arg = torch.empty(64, 32, dtype=torch.int32, device="cuda")
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        return {
            "gat": lambda **kw: gnn.gat_forward(g, x, a, a, out=out, lse=lse, ws=ws, **kw),
            "gatv2": lambda **kw: gnn.gatv2_forward(g, x, x, a, out=out, lse=lse, ws=ws, **kw),
            "transformer": lambda **kw: gnn.transformer_forward(g, x, x, x, out=out, lse=lse,
                                                                ws=ws, **kw),
            "gcn": lambda **kw: (gnn.gcn_forward(g, x[:, 0], "sum", out=out[:, 0], ws=ws, **kw),),
            "max": lambda **kw: gnn.reduce_forward(g, x[:, 0], "max", out=out[:, 0], arg=arg,
                                                   ws=ws, **kw),
        }[name]

    return [call(d) for d in (16_000, 13_000, 14_500)]


def run_at_once(calls, turns):
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    failed = []

    def work(c):
        stream = torch.cuda.Stream()
        try:
            for turn in range(turns):
                c(stream=stream)
                if turn % 100 == 0:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c(), w))


@pytest.mark.parametrize("checkpoints", [False, True], ids=["rows", "checkpoints"])
def test_backward_passes_with_different_bucket_counts(checkpoints):
    run_at_once(backward_calls(checkpoints), 1000)


def child(tmp_path, code):
    """Runs code in a process where setting a limit takes a millisecond."""
    src, lib = tmp_path / "slow.c", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src), "-ldl"], check=True)
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=os.pathsep.join(
        [here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", f"SHIM = {str(lib)!r}\n{code}\nprint('done')\n"],
                       env=env, cwd=os.path.dirname(here), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("checkpoints", [False, True], ids=["rows", "checkpoints"])
def test_a_call_between_another_ones_limit_and_launch(tmp_path, checkpoints):
    child(tmp_path, "import test_threads as t\n"
                    f"t.run_at_once(t.backward_calls({checkpoints}), 60)")


@pytest.mark.parametrize("name", ["gat", "gatv2", "transformer", "gcn", "max"])
def test_the_same_in_the_aggregations(tmp_path, name):
    child(tmp_path, f"import test_threads as t\nt.run_at_once(t.aggregation_calls({name!r}), 60)")


def test_a_refused_launch_leaves_no_error_behind(tmp_path):
    """A call whose kernel cannot be launched raises; the next call, whose kernels can, does
    not find that error.  (The host refuses a limit far above the device's.)"""
    child(tmp_path, """
import ctypes
import pytest
import torch
import graph_neural_network_gb300 as gnn
import test_threads as t
big = t.backward_calls(False)[0]
shim = ctypes.CDLL(SHIM)
x = torch.ones(8, 16, device="cuda")
want = gnn.norm_residual_forward(x, x)[0]
# (a fresh kernel: the limit of the first one is set already)
shim.refuse(1)
with pytest.raises(gnn.GnnError):
    t.backward_calls(True)[0]()
shim.refuse(0)
assert torch.equal(gnn.norm_residual_forward(x, x)[0], want)
big()
torch.cuda.synchronize()
""")
