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
    r = {x: [] for x in ("out", "lse", "out_mag")}
    if g is not None:
        r.update({x: [] for x in ("dq", "dkey", "dval", "dq_mag", "dkey_mag", "dval_mag")})
        if bias is not None:
            r.update(dbias=[], dbias_mag=[])
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
        sc = abs(scale)
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
        hold(got[x], ref[x], ref["C"] * ref[x + "_mag"] + half * np.abs(ref[x]) + 1e-37,
             f"{what} {x}")


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
