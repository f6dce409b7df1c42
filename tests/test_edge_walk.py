"""The cut line of nodes and edges that the attention passes with a bias and from
checkpoints walk: every edge counted once, wherever a cut falls.

The inputs make an edge visible by itself.  Scores are zero (queries live in the
upper half of a head's channels, keys in the lower) and so is the bias: a row of
deg edges has weights 1 / deg.  The rows of val, key, q and dout are one-hot (val and
dout with one more channel), dout times its row's degree, so that an element of a
result is a count of the edges of one class, or a short sum of such counts.  A result
is held to 2^-17 of the magnitude of its terms (scores and biases are exact; weights
1 / deg carry the rounding of a logarithm below 16 and an exponential: 2^-19, and Delta
another; a sum of m terms one after the other, m below 2,000 in a segment and in the
joining of pieces, adds roundings of either sign, sqrt(m) u of it = 2^-18).
One edge lost or counted twice moves some element by at least 2^-15 of that: the test
on the CPU takes edges out of the reference to show it.
"""
import numpy as np
import pytest
import torch

from workload import testgraphs

REL = 2.0 ** -17
NAMES = ("out", "dq", "dkey", "dval", "dbias")


def one_hot(n, H, D, channels, order, device, per_head=True):
    """Rows [n, H, D] with a one in the channel of `channels` that belongs to the node's
    place in `order`, so that every channel gets equally many nodes; in every head, or in
    one head of H times as many classes."""
    x = torch.zeros(n, H, D, device=device)
    c = torch.as_tensor(channels, device=device)
    at = order.to(device) * (len(channels) * (1 if per_head else H)) // n
    row = torch.arange(n, device=device)
    if per_head:
        x[row, :, c[at]] = 1.0
    else:
        x[row, at // len(channels), c[at % len(channels)]] = 1.0
    return x


def inputs(rp, H, D, device, seed=1):
    """q, key, val and dout (float32).  The last channel of val is 1 or 2 by the node's
    parity and that of dout the degree, so that every edge has a dout . val of its own."""
    n = len(rp) - 1
    gen = torch.Generator().manual_seed(seed)
    place = torch.arange(n)
    shuffled = torch.randperm(n, generator=gen)
    deg = torch.from_numpy(np.diff(rp).astype(np.float32)).to(device)
    val = one_hot(n, H, D, range(D - 1), place, device, False)
    val[:, :, D - 1] = 1.0 + torch.arange(n, device=device)[:, None] % 2
    dout = one_hot(n, H, D, range(D - 1), shuffled, device, False)
    dout[:, :, D - 1] = 1.0
    return (one_hot(n, H, D, range(D // 2, D), shuffled, device),
            one_hot(n, H, D, range(D // 2), place, device), val, dout * deg[:, None, None])


def expected(rp, ci, q, k, v, dout, bucket, buckets, scale, skip=()):
    """{name: (value, magnitude of its terms)} at weights 1 / deg, in float64 on q's device.
    skip: edges left out of the sums (their rows keep their weights)."""
    dev = q.device
    rp, ci = (torch.as_tensor(t, device=dev).long() for t in (rp, ci))
    n, H, D = q.shape
    deg = rp[1:] - rp[:-1]
    dst = torch.repeat_interleave(torch.arange(n, device=dev), deg)
    keep = torch.ones(len(ci), dtype=torch.bool, device=dev)
    keep[list(skip)] = False
    a = torch.where(keep, 1.0 / deg[dst].double(), 0.0)
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    res = {x: (zero(n, H, D), zero(n, H, D)) for x in NAMES[:4]}
    res["dbias"] = (zero(buckets, H), zero(buckets, H))
    delta = zero(n, H)
    step = max(1, (1 << 26) // (H * D))
    parts = [slice(s, s + step) for s in range(0, len(ci), step)]
    for s in parts:
        i, j = dst[s], ci[s]
        delta.index_add_(0, i, a[s, None] * (dout[i] * v[j]).sum(-1).double())
    for s in parts:
        i, j, w = dst[s], ci[s], a[s]
        da = (dout[i] * v[j]).sum(-1).double()
        de, mag = w[:, None] * (da - delta[i]), w[:, None] * (da.abs() + delta[i].abs())

        def put(name, at, value, size):
            res[name][0].index_add_(0, at, value)
            res[name][1].index_add_(0, at, size)
        t = w[:, None, None] * v[j].double()
        put("out", i, t, t)
        t = w[:, None, None] * dout[i].double()
        put("dval", j, t, t)
        put("dq", i, scale * de[..., None] * k[j].double(), scale * mag[..., None] * k[j].double())
        put("dkey", j, scale * de[..., None] * q[i].double(),
            scale * mag[..., None] * q[i].double())
        put("dbias", bucket[s], de, mag)
    return res


def outside(got, want, half=0.0):
    """Names of the results with an element outside its bound, with the worst."""
    bad = {}
    for x, t in got.items():
        value, mag = want[x]
        err = (t.double().to(value.device) - value).abs() - half * value.abs()
        over = ~(err <= REL * mag)
        if over.any():
            bad[x] = (int(over.sum()), float(err.max()))
    return bad


def buckets_of(rp, ci, device):
    return torch.as_tensor(np.asarray(ci, np.int64) % 2, device=device)


@pytest.mark.parametrize("make", [testgraphs.star_in, testgraphs.star_out], ids=["in", "out"])
def test_the_bounds_see_one_edge(make):
    """On the CPU: the reference without one edge, or with it counted twice, lies outside
    the bounds, for edges all over the hub's list."""
    rp, ci = make(30_000)
    H, D = 2, 16
    x = inputs(rp, H, D, "cpu")
    bucket = buckets_of(rp, ci, "cpu")
    want = expected(rp, ci, *x, bucket, 2, 0.25)
    assert not outside({k: v[0] for k, v in want.items()}, want)
    hub = np.flatnonzero(np.repeat(np.arange(len(rp) - 1), np.diff(rp)) == 0) \
        if make is testgraphs.star_in else np.flatnonzero(ci == 0)
    seen = set(["out", "dq"] if make is testgraphs.star_in else ["dval", "dkey"])
    rng = np.random.default_rng(1)
    for e in rng.choice(hub, 6, replace=False):
        for sign in (1, -1):
            wrong = expected(rp, ci, *x, bucket, 2, 0.25, skip=[int(e)])
            off = {k: want[k][0] + sign * (wrong[k][0] - want[k][0]) for k in seen}
            assert set(outside(off, want)) == seen, (e, sign)


def run(rp, ci, H, D, dtype=torch.float32, odd=False):
    """Both passes and the checkpoint pass on the GPU against expected(), without a bias and
    with one that every edge carries (weights stay; scores are then pairs)."""
    import graph_neural_network_gb300 as gnn
    n = len(rp) - 1
    g = gnn.Graph(torch.as_tensor(rp, device="cuda").int(),
                  torch.as_tensor(ci, device="cuda").int())
    pos = torch.arange(n, dtype=torch.int32, device="cuda") % 2
    rel = gnn.RelPos(g, pos, bounds=[0], bidirectional=True)
    bucket = rel.arrays()[0].long()
    x = [t.to(dtype) for t in inputs(rp, H, D, "cuda")]
    if odd:  # rows that start 16 bytes past a 32-byte boundary: 16-byte lane vectors
        def move(t):
            pad = 16 // t.element_size()
            room = torch.empty(t.numel() + pad, dtype=t.dtype, device="cuda")
            room[pad:].copy_(t.reshape(-1))
            return room[pad:].view(t.shape)
        x = [move(t) for t in x]
    q, k, v, d = x
    half = 0.0 if dtype == torch.float32 else 2.0 ** -8
    names = NAMES if dtype == torch.float32 else ("out", "dval")
    scale = D ** -0.5
    want = expected(rp, ci, *(t.float() for t in x), bucket, 2, scale)
    packed = gnn.pack8(q, k, v)
    at = [gnn.unpack8(p) for p in packed]
    want8 = expected(rp, ci, *at, d.float(), bucket, 2, scale)
    deg = (g.row_ptr[1:] - g.row_ptr[:-1]).double()
    for value in (0.0, -1e9):
        b = torch.full((2, H), value, device="cuda")
        out, lse = gnn.transformer_rel_forward(g, rel, q, k, v, b)
        got = dict(zip(NAMES, (out,) + gnn.transformer_rel_backward(g, rel, q, k, v, b, lse, d)))
        assert not outside({n_: got[n_] for n_ in names}, want, half), f"bias {value}"
        if value == 0.0:
            off = lse[deg > 0] - deg[deg > 0].log()[:, None]
            assert float(off.abs().max()) <= 16 * 2.0 ** -22
        got = dict(zip(NAMES[1:], gnn.transformer_backward8(g, *packed, d, rel=rel, bias=b)))
        assert not outside({n_: got[n_] for n_ in names if n_ in got}, want8, half), f"8, {value}"
    got = dict(zip(NAMES[1:], gnn.transformer_backward8(g, *packed, d)))
    assert not outside({n_: got[n_] for n_ in names if n_ in got}, want8, half), "checkpoints"
    return g


@pytest.mark.gpu
@pytest.mark.parametrize("make", [testgraphs.star_in, testgraphs.star_out], ids=["in", "out"])
@pytest.mark.parametrize("H, D, dtype", [(2, 16, "f32"), (4, 32, "f32"), (1, 128, "f32"),
                                         (4, 64, "bf16")])
def test_stars(make, H, D, dtype):
    """In bfloat16 a channel counts 119 edges, so that one is more than the rounding."""
    rp, ci = make(30_000)
    run(rp, ci, H, D, torch.float32 if dtype == "f32" else torch.bfloat16)


def cut_places(degs, seg, split):
    """What the cuts at the multiples of seg meet, on the line of a node's edges and its three
    own units: {"short": inside a node that stays whole, and of longer nodes "start", "first"
    (behind its first edge), "last" (before its last), "end" (behind it), "own" (in its own
    units), "within" (two cuts in one node)}."""
    degs = np.asarray(degs)
    start = np.concatenate([[0], np.cumsum(degs + 3)])
    cuts = np.arange(seg, start[-1], seg)
    k = np.searchsorted(start, cuts, side="right") - 1
    at, deg = cuts - start[k], degs[k]
    lng = deg > split - 3
    met = {"short": ~lng & (at > 0), "start": lng & (at == 0), "first": lng & (at == 1),
           "last": lng & (at == deg - 1), "end": lng & (at == deg), "own": lng & (at > deg),
           "within": np.append(k[1:] == k[:-1], False) & lng}
    return {x for x, m in met.items() if m.any()}


def degrees_near(split, lengths, rng):
    """Runs of nodes of 0 edges, nodes about the longest uncut length and longer ones."""
    d = []
    for t in lengths:
        d += [0] * int(rng.integers(0, 40)) + [int(t)] + [int(x) for x in
                                                         rng.integers(0, 5, rng.integers(0, 9))]
    return d + [split - 3] * 7 + [split - 2] * 7 + [0] * 70


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_cuts_at_the_smallest_segments(seed):
    """Segments of 32 units, nodes of up to 64 whole: degrees on both sides of 61, cuts on
    a node's first and last edge and in its own three units, segments that a whole node
    leaves empty and segments wholly inside one."""
    rng = np.random.default_rng(seed)
    near = list(range(26, 36)) + list(range(57, 68)) + list(range(88, 100)) + [127, 128, 129, 500]
    degs = degrees_near(64, rng.permutation(near * 8), rng)
    rp = np.concatenate([[0], np.cumsum(degs)]).astype(np.int32)
    n = len(degs)
    ci = rng.integers(0, n, rp[-1]).astype(np.int32)
    ci[rng.random(rp[-1]) < 0.3] = 5                        # a long node of the other direction
    assert cut_places(degs, 32, 64) == {"short", "start", "first", "last", "end", "own", "within"}
    run(rp, ci, 2, 16)
    run(rp, ci, 1, 128, odd=True)


@pytest.mark.gpu
@pytest.mark.parametrize("reverse", [False, True], ids=["rows", "columns"])
def test_cuts_at_long_segments(reverse):
    """Segments of over 1,024 units, where nodes of up to a sixteenth of one stay whole:
    degrees just below and above it among bulk nodes, and a few that span segments."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    workers = 2 * sms * 8                                   # 512-byte rows in 16-byte lanes
    n = 60_000
    rng = np.random.default_rng(7)
    degs = rng.integers(0, 80, n)
    at = rng.choice(n, 600, replace=False)
    near, seg = rng.integers(-2, 3, 500), 0
    degs[at[500:]] = rng.integers(600, 5000, 100)
    for _ in range(4):                                       # (degrees move the segment)
        seg = -(-(int(degs.sum()) + 3 * n) // workers)
        degs[at[:500]] = seg // 16 - 3 + near                # 0: the longest whole node
    assert seg == -(-(int(degs.sum()) + 3 * n) // workers) and seg > 1040
    assert {"short", "own", "within"} <= cut_places(degs, seg, seg // 16)
    rp = np.concatenate([[0], np.cumsum(degs)]).astype(np.int32)
    ci = rng.integers(0, n, rp[-1]).astype(np.int32)
    if reverse:                                              # the same degrees on the source side
        dst = np.repeat(np.arange(n), degs)
        order = np.argsort(ci, kind="stable")
        rp = np.concatenate([[0], np.cumsum(np.bincount(ci, minlength=n))]).astype(np.int32)
        ci = dst[order].astype(np.int32)
    run(rp, ci, 1, 128, odd=True)
