"""The graph-transformer layer's operators between its projections: attention
with a learned relative position bias, 8-bit activation checkpoints and the
backward pass from them, and the norms, gate and residual scale round a block.

``listed()`` and ``draw()`` give cases, ``prepare()`` their inputs, ``run()``
one pass: the framework's kernels where ``own`` is set, plain torch operations
in 32 bits otherwise.  ``exact()`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    def att(name, op, n, deg, kind, H, D, dtype, buckets=32, dist=128, two=True, mask=False,
            rel=True):
        return dict(name=name, op=op, n=n, deg=deg, graph=kind, H=H, D=D, dtype=dtype,
                    buckets=buckets, dist=dist, two=two, mask=mask, rel=rel)

    def node(name, op, n, F, dtype, kind, gate, bias):
        return dict(name=name, op=op, n=n, F=F, dtype=dtype, kind=kind, gate=gate, bias=bias)

    return [
        # one small molecule- or sentence-sized batch: latency counts
        att("rel fwd 512 f32", "rel_fwd", 512, 8, "uniform", 1, 16, "f32"),
        # inference over a power-law graph whose hubs span several blocks
        att("rel fwd 200k bf16", "rel_fwd", 200_000, 20, "power", 8, 16, "bf16"),
        # a training step on a graph of nearly equal degrees, in float32, with
        # a one-sided table that masks its farthest bucket
        att("rel train 100k f32", "rel_train", 100_000, 17, "uniform", 4, 32, "f32", 16, 64, False,
            True),
        # a training step on a large power-law graph
        att("rel train 300k bf16", "rel_train", 300_000, 20, "power", 4, 64, "bf16"),
        # checkpoints of a small batch, and the values read back for a weight gradient
        dict(name="pack 2k f32", op="pack8", n=2_000, H=2, D=16, dtype="f32"),
        # checkpoints of a large layer's q, key and val
        dict(name="pack 1m bf16", op="pack8", n=1_000_003, H=8, D=16, dtype="bf16"),
        # the backward pass of attention from its checkpoints, without a bias
        att("bwd8 100k f32", "bwd8", 100_000, 17, "uniform", 4, 32, "f32", rel=False),
        # ... and of the large training step above, with its bias gradient
        att("bwd8 300k bf16", "bwd8", 300_000, 20, "power", 4, 64, "bf16"),
        # the norms, gate and residual of a small batch at inference
        node("nr fwd 512 f32", "nr_fwd", 512, 64, "f32", "layer", "row", True),
        # ... of a large graph at inference
        node("nr fwd 1m bf16", "nr_fwd", 1_000_003, 128, "bf16", "rms", "element", False),
        # backward passes: layer norms with their biases, and root mean squares
        node("nr bwd 100k f32", "nr_bwd", 100_000, 128, "f32", "layer", "element", True),
        node("nr bwd 600k bf16", "nr_bwd", 600_001, 256, "bf16", "rms", "element", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rel_fwd", "rel_train", "pack8", "bwd8", "nr_fwd", "nr_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("nr_fwd", "nr_bwd"):
        step = 4 if dtype == "f32" else 8
        F = step * _log_int(rng, 1, 512 // step)
        n = _log_int(rng, 1, min(1_000_000, 150_000_000 // F))
        return dict(op=op, n=n, F=F, dtype=dtype, kind=rng.choice(["rms", "layer"]),
                    gate=rng.choice(["none", "row", "element"]), bias=rng.random() < 0.5)
    # rows of at most 512 bytes, heads of 16 bytes times a power of two
    if dtype == "f32":
        D = rng.choice([4, 8, 16, 32, 64, 128])
        H = rng.randint(1, 128 // D)
    else:
        D = rng.choice([8, 16, 32, 64, 128, 256])
        H = rng.randint(1, 256 // D)
    if op == "pack8":
        return dict(op=op, n=_log_int(rng, 1, 120_000_000 // (H * D)), H=H, D=D, dtype=dtype)
    deg = rng.randint(4, 24)
    n = _log_int(rng, 64, min(300_000, 1_400_000_000 // (deg * H * D)))
    two = rng.random() < 0.5
    return dict(op=op, n=n, deg=deg, graph=rng.choice(["uniform", "power"]), H=H, D=D, dtype=dtype,
                buckets=rng.randint(2, 32) * 2, dist=_log_int(rng, 40, 4000), two=two,
                mask=rng.random() < 0.3, rel=op != "bwd8" or rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _graph(case, gen):
    """CSR of n * deg edges.  "uniform": deg random sources a node; "power":
    both ends drawn from weights (r + 1)^(-1 / 1.1) over random node ids, so
    some nodes have thousands of in-edges and many have none."""
    n, deg = case["n"], case["deg"]
    e = n * deg
    if case["graph"] == "uniform":
        dst = torch.arange(n, device=DEV).repeat_interleave(deg)
        src = torch.randint(0, n, (e,), generator=gen, device=DEV)
    else:
        w = torch.arange(1, n + 1, device=DEV, dtype=torch.float64).pow(-1 / 1.1)
        w = w.clamp(max=float(w.sum()) * 20_000 / e)
        cum = w.cumsum(0)
        cum = cum / cum[-1]
        ids = [torch.randperm(n, generator=gen, device=DEV) for _ in range(2)]
        pick = [torch.searchsorted(cum, torch.rand(e, generator=gen, device=DEV,
                                                   dtype=torch.float64)).clamp(max=n - 1)
                for _ in range(2)]
        key, _ = torch.sort(ids[0][pick[0]] * n + ids[1][pick[1]])
        dst, src = key // n, key % n
    row_ptr = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    row_ptr[1:] = torch.bincount(dst, minlength=n).cumsum(0)
    return row_ptr, dst, src


def _bounds(case):
    """The smallest distance of each bucket of one side, as whole numbers:
    distances below half the buckets have one each, the others grow by equal
    ratios up to dist."""
    nb = case["buckets"] // 2 if case["two"] else case["buckets"]
    exact_to = nb // 2
    rest = nb - exact_to
    low = list(range(exact_to))
    for k in range(rest):
        # smallest t with (t / exact_to)^rest >= (dist / exact_to)^k, in whole numbers
        need = case["dist"] ** k * exact_to ** (rest - k)
        t = max(1, int(exact_to * (case["dist"] / exact_to) ** (k / rest)) - 2)
        while t ** rest < need:
            t += 1
        low.append(t)
    return low


def _bucket(case, delta):
    """The bucket of each signed distance."""
    low = torch.tensor(_bounds(case), device=DEV)
    if case["two"]:
        side = (delta > 0) * (case["buckets"] // 2)
        return side + torch.searchsorted(low, delta.abs(), right=True) - 1
    return torch.searchsorted(low, (-delta).clamp(min=0), right=True) - 1


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    st = {"case": case, "dt": dt}
    n = case["n"]
    if case["op"] in ("nr_fwd", "nr_bwd"):
        F = case["F"]
        f32 = torch.float32
        st["x"], st["o"] = normal(n, F), normal(n, F, std=3.0)
        st["gate"] = (normal(n, F) if case["gate"] == "element" else
                      normal(n, 1) if case["gate"] == "row" else None)
        st["w_post"], st["w_pre"] = 1 + normal(F, std=0.1, dtype=f32), 1 + normal(F, std=0.1,
                                                                                  dtype=f32)
        st["scale"] = 0.5 + normal(F, std=0.1, dtype=f32)
        st["b_post"] = normal(F, std=0.1, dtype=f32) if case["bias"] else None
        st["b_pre"] = normal(F, std=0.1, dtype=f32) if case["bias"] else None
        if case["op"] == "nr_bwd":
            st["y"] = normal(n, F, std=1.5)  # the stored sum that the next norm took
            st["dy"], st["dz"] = normal(n, F), normal(n, F)
            del st["x"]
        return st
    H, D = case["H"], case["D"]
    st["q"], st["key"], st["val"] = (normal(n, H, D) for _ in range(3))
    if case["op"] == "pack8":
        return st
    row_ptr, dst, src = _graph(case, gen)
    st["row_ptr"], st["dst"], st["src"] = row_ptr.int(), dst, src
    st["att_scale"] = D ** -0.5
    if case["rel"]:
        # positions along sequences a few times longer than the farthest bucket
        st["pos"] = torch.randint(0, 4 * case["dist"], (n,), generator=gen, device=DEV).int()
        st["bias"] = normal(case["buckets"], H, dtype=torch.float32)
        if case["mask"]:
            st["bias"][case["buckets"] - 1] = -INF
        pos = st["pos"].long()
        st["bucket"] = _bucket(case, pos[src] - pos[dst])
    if case["op"] != "rel_fwd":
        st["dout"] = normal(n, H, D)
    if case["op"] == "bwd8":
        for k in ("q", "key", "val"):
            st[k + "8"] = _plain_pack(st.pop(k))
    if own:
        import graph_neural_network_gb300 as gnn
        st["g"] = gnn.Graph(st["row_ptr"], src.int())
        if case["rel"]:
            st["rel"] = gnn.RelPos(st["g"], st["pos"], case["buckets"], case["dist"], case["two"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"rel_fwd": _plain_rel, "rel_train": _plain_rel, "pack8": _plain_pack8,
            "bwd8": _plain_bwd8, "nr_fwd": _plain_nr_fwd, "nr_bwd": _plain_nr_bwd}[st["case"]["op"]](st)


def _own(st):
    import graph_neural_network_gb300 as gnn
    op = st["case"]["op"]
    if op == "pack8":
        packed = gnn.pack8(st["q"], st["key"], st["val"])
        return [(gnn.unpack8(p, st["dt"]), p.scale) for p in packed]
    if op == "bwd8":
        c = [gnn.Packed8(*st[k]) for k in ("q8", "key8", "val8")]
        return gnn.transformer_backward8(st["g"], *c, st["dout"], rel=st.get("rel"),
                                         bias=st.get("bias"))
    if op in ("rel_fwd", "rel_train"):
        q, k, v, b = st["q"], st["key"], st["val"], st["bias"]
        out, lse = gnn.transformer_rel_forward(st["g"], st["rel"], q, k, v, b)
        if op == "rel_fwd":
            return out, lse
        return (out, lse) + tuple(gnn.transformer_rel_backward(st["g"], st["rel"], q, k, v, b, lse,
                                                               st["dout"]))
    par = {k: st[k] for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")}
    kind = st["case"]["kind"]
    if op == "nr_fwd":
        return gnn.norm_residual_forward(st["x"], st["o"], kind=kind, eps=EPS, **par)
    return {k: v for k, v in gnn.norm_residual_backward(
        st["y"], st["o"], st["dy"], st["dz"], kind=kind, eps=EPS, **par).items() if v is not None}


EPS = 1e-6


def _sum_rows(idx, x, n):
    return torch.zeros(n, *x.shape[1:], dtype=x.dtype, device=DEV).index_add_(0, idx, x)


def _scores(st, q, k):
    e = (q[st["dst"]] * k[st["src"]]).sum(-1) * st["att_scale"]
    if st["case"]["rel"]:
        e = e + st["bias"][st["bucket"]]
    return e


def _softmax(st, e):
    """The edges' softmax weights and each row's log of the sum."""
    n, H = st["case"]["n"], e.shape[1]
    at = st["dst"][:, None].expand(-1, H)
    top = torch.full((n, H), -INF, device=DEV).scatter_reduce(0, at, e, "amax")
    top = torch.where(top == -INF, 0.0, top)
    p = torch.exp(e - top[st["dst"]])
    total = _sum_rows(st["dst"], p, n)
    lse = torch.log(total) + top
    return p / torch.where(total == 0, 1.0, total)[st["dst"]], lse


def _attention_backward(st, q, k, v, alpha):
    n, dst, src, sc = st["case"]["n"], st["dst"], st["src"], st["att_scale"]
    g = st["dout"].float()[dst]
    da = (g * v[src]).sum(-1)
    delta = _sum_rows(dst, alpha * da, n)
    de = alpha * (da - delta[dst])
    dval = _sum_rows(src, alpha[..., None] * g, n)
    del g
    dq = _sum_rows(dst, de[..., None] * k[src], n) * sc
    dkey = _sum_rows(src, de[..., None] * q[dst], n) * sc
    grads = [t.to(st["dt"]) for t in (dq, dkey, dval)]
    if st["case"]["rel"]:
        # a sum over millions of edges into a few numbers: in 64 bits
        B, H = st["bias"].shape
        at = st["bucket"][:, None] * H + torch.arange(H, device=DEV)
        grads.append(torch.bincount(at.reshape(-1), weights=de.double().reshape(-1),
                                    minlength=B * H).reshape(B, H).float())
    return grads


def _plain_rel(st):
    q, k, v = (st[x].float() for x in ("q", "key", "val"))
    alpha, lse = _softmax(st, _scores(st, q, k))
    out = _sum_rows(st["dst"], alpha[..., None] * v[st["src"]], st["case"]["n"]).to(st["dt"])
    if st["case"]["op"] == "rel_fwd":
        return out, lse
    return (out, lse) + tuple(_attention_backward(st, q, k, v, alpha))


def _plain_pack(x):
    x = x.float()
    # in 64 bits: a quotient next to a half would round the other way
    s = (x.abs().amax(-1).double() / 127).float().clamp(min=2.0 ** -126)
    return torch.round(x.double() / s.double()[..., None]).to(torch.int8), s


def _plain_pack8(st):
    packed = [_plain_pack(st[k]) for k in ("q", "key", "val")]
    return [((x8.float() * s[..., None]).to(st["dt"]), s) for x8, s in packed]


def _plain_bwd8(st):
    q, k, v = (st[x][0].float() * st[x][1][..., None] for x in ("q8", "key8", "val8"))
    alpha, _ = _softmax(st, _scores(st, q, k))
    return _attention_backward(st, q, k, v, alpha)


def _normed(x, layer):
    mean = x.mean(-1, keepdim=True) if layer else 0.0
    x = x - mean
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * rstd, rstd


def _norm_backward(g, hat, rstd, layer):
    d = g - hat * (g * hat).mean(-1, keepdim=True)
    if layer:
        d = d - g.mean(-1, keepdim=True)
    return d * rstd


def _affine(hat, w, b):
    return hat * w if b is None else hat * w + b


def _plain_nr_fwd(st):
    layer = st["case"]["kind"] == "layer"
    x, o = st["x"].float(), st["o"].float()
    n = _affine(_normed(o, layer)[0], st["w_post"], st["b_post"])
    if st["gate"] is not None:
        n = n * torch.sigmoid(st["gate"].float())
    y = x + st["scale"] * n
    z = _affine(_normed(y, layer)[0], st["w_pre"], st["b_pre"])
    return y.to(st["dt"]), z.to(st["dt"])


def _plain_nr_bwd(st):
    case, dt = st["case"], st["dt"]
    layer = case["kind"] == "layer"
    sig = 1.0 if st["gate"] is None else torch.sigmoid(st["gate"].float())
    ohat, orstd = _normed(st["o"].float(), layer)
    yhat, yrstd = _normed(st["y"].float(), layer)
    n = _affine(ohat, st["w_post"], st["b_post"])

    def total(t):  # over all rows, in 64 bits
        return t.sum(0, dtype=torch.float64).float()

    dz = st["dz"].float()
    dx = st["dy"].float() + _norm_backward(dz * st["w_pre"], yhat, yrstd, layer)
    dn = dx * st["scale"] * sig
    do = _norm_backward(dn * st["w_post"], ohat, orstd, layer)
    got = {"dx": dx.to(dt), "do": do.to(dt), "dw_post": total(dn * ohat),
           "dscale": total(dx * sig * n), "dw_pre": total(dz * yhat)}
    if st["gate"] is not None:
        dgate = dn * n * (1 - sig)
        got["dgate"] = (dgate.sum(-1, keepdim=True) if case["gate"] == "row" else dgate).to(dt)
    if case["bias"]:
        got["db_post"], got["db_pre"] = total(dn), total(dz)
    return got


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    s = 4 if case["dtype"] == "f32" else 2
    n, op = case["n"], case["op"]
    if op in ("nr_fwd", "nr_bwd"):
        F = case["F"]
        gate = {"none": 0, "row": 1, "element": F}[case["gate"]]
        if op == "nr_fwd":  # x, o, gate; y, z
            return {"bytes": n * s * (4 * F + gate) + 12 * F, "flops": 15 * n * F}
        # y, o, gate, dy, dz; dx, do, dgate
        return {"bytes": n * s * (6 * F + 2 * gate) + 24 * F, "flops": 45 * n * F}
    H, D = case["H"], case["D"]
    F = H * D
    if op == "pack8":
        # q, key, val; their values read back, and the scales
        return {"bytes": 3 * n * (2 * F * s + 4 * H), "flops": 9 * n * F}
    e = n * case["deg"]
    index = 4 * (n + 1) + 4 * e + (e + 4 * case["buckets"] * H if case["rel"] else 0)
    if op == "rel_fwd":  # q, key, val; out, lse
        return {"bytes": index + 4 * n * F * s + 4 * n * H, "flops": 4 * e * F}
    if op == "rel_train":  # and dout; dq, dkey, dval, dbias
        return {"bytes": index + 8 * n * F * s + 4 * n * H, "flops": 14 * e * F}
    # the checkpoints, dout; dq, dkey, dval, dbias
    return {"bytes": index + 3 * n * (F + 4 * H) + 4 * n * F * s, "flops": 12 * e * F}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pack8":
        return [_exact_pack(st[k]) for k in ("q", "key", "val")]
    if case["op"] in ("nr_fwd", "nr_bwd"):
        return _exact_nr(st)
    return _exact_attention(st)


def _exact_pack(x):
    """The nearest multiples of a hundred-and-twenty-seventh of the largest
    magnitude, found by comparing the two whole numbers next to each quotient."""
    x = x.double()
    s = torch.linalg.vector_norm(x, INF, -1).div(127.0).float().clamp(min=2.0 ** -126).double()
    s_ = s.unsqueeze(-1)
    down = torch.floor(x / s_)
    below, above = x - down * s_, (down + 1) * s_ - x
    up = (above < below) | ((above == below) & (down % 2 != 0))
    return (down + up) * s_, s


def _exact_attention(st):
    """Head by head: autograd of the definition over the edges whose bias is
    not minus infinity."""
    case = st["case"]
    n, H = case["n"], case["H"]
    train = case["op"] != "rel_fwd"
    if case["op"] == "bwd8":
        q, k, v = (st[x][0].double() * st[x][1].double().unsqueeze(-1)
                   for x in ("q8", "key8", "val8"))
    else:
        q, k, v = (st[x].double() for x in ("q", "key", "val"))
    outs, lses, grads, dbias = [], [], [], []
    for h in range(H):
        i, j = st["dst"], st["src"]
        qh, kh, vh = (t[:, h].contiguous().requires_grad_(train) for t in (q, k, v))
        leaves = [qh, kh, vh]
        b = None
        if case["rel"]:
            bh = st["bias"][:, h].double().requires_grad_(train)
            leaves.append(bh)
            seen = torch.nonzero(bh.detach()[st["bucket"]] > -INF).squeeze(1)
            i, j = i[seen], j[seen]
            b = bh.index_select(0, st["bucket"][seen])
        e = torch.einsum("ed,ed->e", qh.index_select(0, i), kh.index_select(0, j)) / math.sqrt(
            case["D"])
        e = e if b is None else e + b
        peak = torch.zeros(n, dtype=torch.float64, device=DEV).index_reduce(
            0, i, e.detach(), "amax", include_self=False)
        w = (e - peak[i]).exp()
        z = torch.zeros(n, dtype=torch.float64, device=DEV).index_add(0, i, w)
        some = z.detach() > 0
        out = torch.zeros(n, case["D"], dtype=torch.float64, device=DEV).index_add(
            0, i, w.unsqueeze(1) * vh.index_select(0, j))
        out = out / torch.where(some, z, torch.ones_like(z)).unsqueeze(1)
        outs.append(out.detach())
        lses.append(torch.where(some, z.detach().log() + peak, torch.full_like(peak, -INF)))
        if train:
            got = torch.autograd.grad(out, leaves, st["dout"][:, h].double())
            grads.append(got[:3])
            dbias.append(got[3] if case["rel"] else None)
    head = [torch.stack(outs, 1), torch.stack(lses, 1)]
    if not train:
        return tuple(head)
    tail = [torch.stack([g[t] for g in grads], 1) for t in range(3)]
    if case["rel"]:
        tail.append(torch.stack(dbias, 1))
    return tail if case["op"] == "bwd8" else tuple(head + tail)


def _exact_nr(st):
    """The layer norm or root mean square written out, and autograd through
    the two halves: z from the stored y, and y from x, o and the gate."""
    case = st["case"]
    layer = case["kind"] == "layer"
    train = case["op"] == "nr_bwd"
    n, F = st["o"].shape

    def norm(t, w, b):
        var, mean = (torch.var_mean(t, -1, correction=0, keepdim=True) if layer else
                     (t.pow(2).mean(-1, keepdim=True), 0.0))
        r = (t - mean) / (var + EPS).sqrt() * w
        return r if b is None else r + b

    par = {k: None if st[k] is None else st[k].double().requires_grad_(train)
           for k in ("w_post", "b_post", "scale", "w_pre", "b_pre")}
    parts, sums = [], {}
    rows = max(1, (1 << 27) // F)
    for r in range(0, n, rows):
        at = slice(r, r + rows)
        o = st["o"][at].double().requires_grad_(train)
        gate = st["gate"][at].double().requires_grad_(train) if st["gate"] is not None else None
        add = norm(o, par["w_post"], par["b_post"]) * par["scale"]
        add = add if gate is None else add * gate.sigmoid()
        if not train:
            y = st["x"][at].double() + add
            parts.append((y, norm(y, par["w_pre"], par["b_pre"])))
            continue
        y = st["y"][at].double().requires_grad_()
        z = norm(y, par["w_pre"], par["b_pre"])
        after = {"dw_pre": par["w_pre"], "db_pre": par["b_pre"]}
        after = {k: t for k, t in after.items() if t is not None}
        dy, *rest = torch.autograd.grad(z, [y, *after.values()], st["dz"][at].double())
        dy = dy + st["dy"][at].double()
        before = {"do": o, "dgate": gate, "dw_post": par["w_post"], "db_post": par["b_post"],
                  "dscale": par["scale"]}
        before = {k: t for k, t in before.items() if t is not None}
        got = dict(zip(before, torch.autograd.grad(add, list(before.values()), dy)),
                   **dict(zip(after, rest)), dx=dy)
        for k in ("dw_post", "db_post", "dscale", "dw_pre", "db_pre"):
            if k in got:
                sums[k] = sums.get(k, 0) + got.pop(k)
        parts.append(got)
    if not train:
        return tuple(torch.cat(p) for p in zip(*parts))
    return dict({k: torch.cat([p[k] for p in parts]) for k in parts[0]}, **sums)
