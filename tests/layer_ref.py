"""Plain float64 references of the graph-transformer layer's operators and the
rounding bounds that the GPU tests hold them to.

Bounds.  u = 2^-24 is the half step of float32; a result stored in type t adds
h(t) |value| with h = finfo(t).eps / 2.  Inputs are exact.

Attention.  S = max over edges of scale * sum_c |q_c k_c| + |bias|.  A score is
a float32 sum of D products, scaled: off by at most (D + 4) u S, in base-2
units 1.5 times that; lse comes from such scores and deg terms.  So a weight
alpha = exp(e - lse) is off by a factor 1 + w with
    |w| <= 2 * ((D + 4) u S + (|lse| + deg + 8) u) + 2^-21
(2^-21: the hardware's exponential and logarithm, and the base-2 conversion).
A sum of deg weighted terms t is off by at most (w + (deg + 4) u) sum |t|, and
the factors inside a term (dout_i . val_j: D products; Delta_i: a sum of deg of
those with weights) add their own relative error to sums of magnitudes.  Every
attention bound is therefore C * mag with mag the sum of the terms' magnitudes,
|da| taken as sum_c |dout_c val_c| and |Delta| as its weighted mean, and
    C = 3 |w| + (deg + 2 D + 16) u.
The hardware's exponential flushes results below 2^-126 to zero: a weight may
also be off by 2^-126 itself, whatever it multiplies.  A sum of terms alpha t is
then off by another 2^-126 sum |t|; in de = alpha (da - Delta) the factor is |da|
+ |Delta|, and Delta, a sum over the row, is off by 2^-126 sum |da| at alpha <= 1.
*_one holds these sums, counted twice (2^-125) for products of two such errors.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}   # rounding of the result (float32 sums: in C)


def attention(rp, ci, q, k, v, scale, bias=None, bucket=None, dout=None):
    """Values (and with dout gradients) in float64, head by head, with each
    result's magnitude sum.  Arrays are float64; bucket [E] int in CSR order.
    Masked edges (bias -inf) are left out.  Returns a dict; *_mag beside each
    of out, dq, dkey, dval, dbias, and "C"."""
    rp = np.asarray(rp, np.int64)
    n, H, D = q.shape
    dst = torch.from_numpy(np.repeat(np.arange(n), np.diff(rp)))
    src = torch.from_numpy(np.asarray(ci, np.int64))
    t = lambda a: torch.from_numpy(np.asarray(a, np.float64))  # noqa: E731
    q, k, v = t(q), t(k), t(v)
    g = None if dout is None else t(dout)
    r = {x: [] for x in ("out", "lse", "out_mag", "out_one")}
    if g is not None:
        r.update({x + y: [] for x in ("dq", "dkey", "dval") for y in ("", "_mag", "_one")})
        if bias is not None:
            r.update(dbias=[], dbias_mag=[], dbias_one=[])
    S, lse_top = 0.0, 0.0
    for h in range(H):
        i, j, b = dst, src, None
        if bias is not None:
            bh = t(bias)[:, h]
            b = torch.from_numpy(np.asarray(bucket, np.int64))
            seen = bh[b] > -math.inf
            i, j, b = i[seen], j[seen], b[seen]
        qh, kh, vh = q[:, h], k[:, h], v[:, h]
        e = scale * (qh[i] * kh[j]).sum(-1)
        mag_e = abs(scale) * (qh[i] * kh[j]).abs().sum(-1)
        if b is not None:
            e = e + bh[b]
            mag_e = mag_e + bh[b].abs()
        top = torch.full((n,), -math.inf, dtype=torch.float64).scatter_reduce(0, i, e, "amax")
        top0 = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        p = torch.exp(e - top0[i])
        z = torch.zeros(n, dtype=torch.float64).index_add(0, i, p)
        a = p / z[i]
        lse = torch.where(z > 0, torch.log(z) + top0, torch.full_like(z, -math.inf))
        add = lambda idx, x: torch.zeros(n, *x.shape[1:],  # noqa: E731
                                         dtype=torch.float64).index_add(0, idx, x)
        r["out"].append(add(i, a[:, None] * vh[j]))
        r["out_mag"].append(add(i, a[:, None] * vh[j].abs()))
        r["out_one"].append(add(i, vh[j].abs()))
        r["lse"].append(lse)
        if len(e):
            S = max(S, float(mag_e.max()))
            lse_top = max(lse_top, float(lse[torch.isfinite(lse)].abs().max()))
        if g is None:
            continue
        gi = g[:, h][i]
        da, da_m = (gi * vh[j]).sum(-1), (gi * vh[j]).abs().sum(-1)
        delta, delta_m = add(i, a * da), add(i, a * da_m)
        de, de_m = a * (da - delta[i]), a * (da_m + delta_m[i])
        de_1 = da_m + delta_m[i] + add(i, da_m)[i]
        sc = abs(scale)
        r["dq_one"].append(sc * add(i, de_1[:, None] * kh[j].abs()))
        r["dkey_one"].append(sc * add(j, de_1[:, None] * qh[i].abs()))
        r["dval_one"].append(add(j, gi.abs()))
        r["dq"].append(scale * add(i, de[:, None] * kh[j]))
        r["dq_mag"].append(sc * add(i, de_m[:, None] * kh[j].abs()))
        r["dkey"].append(scale * add(j, de[:, None] * qh[i]))
        r["dkey_mag"].append(sc * add(j, de_m[:, None] * qh[i].abs()))
        r["dval"].append(add(j, a[:, None] * gi))
        r["dval_mag"].append(add(j, a[:, None] * gi.abs()))
        if b is not None:
            nb = len(bh)
            r["dbias"].append(torch.zeros(nb, dtype=torch.float64).index_add(0, b, de))
            r["dbias_mag"].append(torch.zeros(nb, dtype=torch.float64).index_add(0, b, de_m))
            r["dbias_one"].append(torch.zeros(nb, dtype=torch.float64).index_add(0, b, de_1))
    out = {x: torch.stack(y, 1).numpy() for x, y in r.items()}
    deg = max(int(np.diff(rp).max(initial=0)),
              int(np.bincount(np.asarray(ci, np.int64), minlength=1).max(initial=0)))
    w = 2 * ((D + 4) * U * S + (lse_top + deg + 8) * U) + 2.0 ** -21
    out["C"] = 3 * w + (deg + 2 * D + 16) * U
    out["lse_bound"] = (D + 4) * U * S + (lse_top + deg + 8) * U + 2.0 ** -21
    return out


def hold(got, ref, bound, what):
    """|got - ref| <= bound element by element; the same infinities."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, ref))
    bad = ~(err <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(np.isnan(err), np.inf, err / bound)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; worst {at}: "
                             f"{got[at]!r} for {ref[at]!r}, bound "
                             f"{np.broadcast_to(bound, err.shape)[at]!r}")


def hold_attention(got, ref, dtype, what, names):
    """names of `got` (numpy, float64) against attention()'s result."""
    for x in names:
        if x == "lse":
            hold(got[x], ref[x], ref["lse_bound"], f"{what} lse")
            continue
        half = 0.0 if x == "dbias" else HALF[dtype]
        hold(got[x], ref[x], ref["C"] * ref[x + "_mag"] + half * np.abs(ref[x]) +
             2.0 ** -125 * ref[x + "_one"] + 1e-37, f"{what} {x}")


def bucket_of(d, bounds, two_sided):
    """The bucket of whole differences d, straight from the definition."""
    out = []
    for x in np.asarray(d).tolist():
        dist = abs(x) if two_sided else max(-x, 0)
        b = max(k for k in range(len(bounds)) if bounds[k] <= dist)
        out.append(b + (len(bounds) if two_sided and x > 0 else 0))
    return np.array(out, np.int64)


def log_bounds(n, max_distance):
    """The logarithmic rule's bounds in Python's whole numbers."""
    m = n // 2
    rest = n - m
    out = list(range(m))
    for k in range(rest):
        need = max_distance ** k * m ** (rest - k)
        lo, hi = m, max_distance
        while lo < hi:
            mid = (lo + hi) // 2
            if mid ** rest >= need:
                hi = mid
            else:
                lo = mid + 1
        out.append(lo)
    return out


# ---------------------------------------------------------------------------
# norms, gate and residual scale
# ---------------------------------------------------------------------------
#
# Bounds.  A sum over a row (at most 1024 elements: eight in a thread, then a
# tree) makes at most 20 roundings: relative to its magnitude sum, G = 32 u with
# the products and the division.  A layer mean is then off by e = G max|x|, a
# normed value by E = e rstd + |hat| (G + e rstd) (rms: e = 0).  The sigmoid is
# off by 2^-21 + 2 u |g| relative (exponential 2^-22, its argument g log2(e) with
# a rounded constant and product, sum and quotient).  The rest is the product rule, each operation adding u; parameter sums add R u
# for the R rows that a thread adds in sequence.

G = 32 * U
SIG = 2.0 ** -21


def _norm(x, kind, eps):
    """hat, rstd, and the bounds of hat (absolute) and rstd (relative)."""
    if kind == "none":
        return x, np.ones((len(x), 1)), np.zeros_like(x), 0.0
    mean = x.mean(-1, keepdims=True) if kind == "layer" else 0.0
    e = G * np.abs(x).max(-1, keepdims=True) if kind == "layer" else 0.0
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    hat = (x - mean) * rstd
    rho = G + e * rstd
    return hat, rstd, e * rstd + np.abs(hat) * rho, rho


def _params(p, F):
    one, nil = np.ones(F), np.zeros(F)
    return [np.asarray(p.get(k), np.float64) if p.get(k) is not None else d for k, d in
            (("w_post", one), ("b_post", nil), ("scale", one), ("w_pre", one), ("b_pre", nil))]


def _sig(gate, like):
    if gate is None:
        return np.ones_like(like), 0.0
    return (np.broadcast_to(1 / (1 + np.exp(-gate)), like.shape),
            np.broadcast_to(SIG + 2 * U * np.abs(gate), like.shape))


def norm_residual(x, o, gate, p, kinds, eps):
    """y, z and their bounds (without the rounding of the result)."""
    wp, bp, sc, wn, bn = _params(p, x.shape[1])
    oh, _, Eo, _ = _norm(o, kinds[0], eps)
    sig, serr = _sig(gate, x)
    n = oh * wp + bp
    dn = np.abs(wp) * Eo + 3 * U * (np.abs(oh * wp) + np.abs(bp))
    y = x + sc * sig * n
    by = np.abs(sc * sig) * dn + (serr + 4 * U) * np.abs(sc * sig * n) + U * np.abs(y)
    if kinds[1] == "none":
        return y, by, None, None
    yh, rstd, Ey, _ = _norm(y, kinds[1], eps)
    # an error d of y moves the normed row by rstd (d - mean d) and by its length
    move = rstd * (by + by.mean(-1, keepdims=True)) + np.abs(yh) * rstd * np.sqrt(
        (by ** 2).mean(-1, keepdims=True))
    z = yh * wn + bn
    bz = np.abs(wn) * (Ey + move) + 3 * U * (np.abs(yh * wn) + np.abs(bn))
    return y, by, z, bz


def _norm_back(g, dg, hat, E, rstd, rho, kind):
    if kind == "none":
        return g, dg
    m = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    c0, b0 = m(g * hat), m(dg * np.abs(hat) + np.abs(g) * E) + G * m(np.abs(g * hat))
    c1, b1 = (m(g), m(dg) + G * m(np.abs(g))) if kind == "layer" else (0.0, 0.0)
    d = rstd * (g - c1 - hat * c0)
    return d, np.abs(d) * rho + rstd * (dg + b1 + np.abs(c0) * E + np.abs(hat) * b0 + 4 * U * (
        np.abs(g) + np.abs(c1) + np.abs(hat * c0)))


def norm_residual_grads(y, o, gate, dy, dz, p, kinds, eps):
    """{name: (value, bound)} of the gradients, from y as given."""
    n_rows, F = o.shape
    wp, bp, sc, wn, _ = _params(p, F)
    oh, ro, Eo, rho_o = _norm(o, kinds[0], eps)
    got = {}
    R = 32 + n_rows / 600
    def total(a, da): return a.sum(0), da.sum(0) + R * U * np.abs(a).sum(0)  # noqa: E704
    if kinds[1] == "none":
        dx, bx = dy, np.zeros_like(dy)
    else:
        yh, ry, Ey, rho_y = _norm(y, kinds[1], eps)
        t, bt = _norm_back(dz * wn, U * np.abs(dz * wn), yh, Ey, ry, rho_y, kinds[1])
        dx = dy + t
        bx = bt + U * np.abs(dx)
        got["dw_pre"] = total(dz * yh, np.abs(dz) * Ey + U * np.abs(dz * yh))
        got["db_pre"] = total(dz, 0 * dz)
    got["dx"] = dx, bx
    sig, serr = _sig(gate, o)
    n = oh * wp + bp
    bn = np.abs(wp) * Eo + 3 * U * (np.abs(oh * wp) + np.abs(bp))
    u = dx * sc * sig
    bu = bx * np.abs(sc * sig) + (serr + 3 * U) * np.abs(u)
    got["dscale"] = total(dx * sig * n, np.abs(sig) * (bx * np.abs(n) + np.abs(dx) * bn) +
                          (serr + 3 * U) * np.abs(dx * sig * n))
    got["dw_post"] = total(u * oh, bu * np.abs(oh) + np.abs(u) * Eo + U * np.abs(u * oh))
    got["db_post"] = total(u, bu)
    if gate is not None:
        dg = u * n * (1 - sig)
        bg = (bu * np.abs(n) + np.abs(u) * bn) * (1 - sig) + np.abs(u * n) * (
            serr * sig + 2 * U) + 4 * U * np.abs(dg)
        if gate.shape[1] == 1 and F != 1:
            dg, bg = dg.sum(-1, keepdims=True), (bg + G * np.abs(dg)).sum(-1, keepdims=True)
        got["dgate"] = dg, bg
    got["do"] = _norm_back(u * wp, bu * np.abs(wp) + U * np.abs(u * wp), oh, Eo, ro, rho_o,
                           kinds[0])
    return got
