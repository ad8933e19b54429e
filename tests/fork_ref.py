"""Plain 64-bit implementations of the operators of a fork batch's step (CPU, written from the formulas)."""
import math

import numpy as np
import torch


# ---- norms around a block ------------------------------------------------------------------------
def _rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def block_norm(h, y, pre_w, post_w, gate, scale, eps):
    """(x, n, and the magnitudes that rounding errors of the two are relative to)."""
    h, y, pre_w = h.double(), y.double(), pre_w.double()
    z = y if post_w is None else post_w.double() * y * _rms(y, eps)
    if gate is not None:
        z = z * torch.sigmoid(gate.double())
    if scale is not None:
        z = z * scale.double()
    x = h + z
    s = _rms(x, eps)
    n = pre_w * x * s
    A = h.abs() + z.abs()
    more = _spread(A, x)
    return x, n, A, pre_w.abs() * A * s + n.abs() * more


def _spread(A, x):
    """How much larger the terms of x are than x, row by row (1 where nothing cancels)."""
    a, b = A.square().sum(-1, keepdim=True).sqrt(), x.square().sum(-1, keepdim=True).sqrt()
    return torch.where(b > 0, a / b.clamp(min=1e-300), torch.ones_like(a))


def block_norm_grad(h, y, pre_w, post_w, gate, scale, eps, dn, dh_out):
    """({name: gradient}, {name: magnitudes of its errors}), by the formula."""
    f = lambda t: None if t is None else t.double()   # noqa: E731
    h, y, pre_w, post_w, gate, scale, dn, dh_out = map(f, (h, y, pre_w, post_w, gate, scale, dn, dh_out))
    one = torch.ones((), dtype=torch.float64)
    g = one if gate is None else torch.sigmoid(gate)
    sc = one if scale is None else scale
    pw = one if post_w is None else post_w
    r = one if post_w is None else _rms(y, eps)
    z = pw * y * r
    x, n, A, _ = block_norm(h, y, pre_w, post_w, gate, scale, eps)
    s, k = _rms(x, eps), _spread(A, x)
    wdn = pre_w * dn
    dx = s * (wdn - x * s * s * (wdn * x).mean(-1, keepdim=True))
    mx = k ** 3 * s * (wdn.abs() + A * s * s * (wdn.abs() * A).mean(-1, keepdim=True))
    if dh_out is not None:
        dx, mx = dx + dh_out, mx + dh_out.abs()
    dz, mz = dx * sc * g, mx * sc.abs() * g
    rows = tuple(range(h.dim() - 1))
    out = dict(dh=dx, dpre_w=(dn * x * s).sum(rows))
    mag = dict(dh=mx, dpre_w=(dn.abs() * A * s * k).sum(rows))
    if post_w is None:
        out["dy"], mag["dy"] = dz, mz
    else:
        out["dy"] = r * (pw * dz - y * r * r * (pw * dz * y).mean(-1, keepdim=True))
        mag["dy"] = r * (pw.abs() * mz + y.abs() * r * r * (pw.abs() * mz * y.abs()).mean(-1, keepdim=True))
        out["dpost_w"], mag["dpost_w"] = (dz * y * r).sum(rows), (mz * y.abs() * r).sum(rows)
    if scale is not None:
        out["dscale"], mag["dscale"] = (dx * g * z).sum(rows), (mx * g * z.abs()).sum(rows)
    if gate is not None:
        out["dgate"] = dx * sc * z * g * (1 - g)
        mag["dgate"] = mx * sc.abs() * z.abs() * g
    return out, mag


# ---- sampling ------------------------------------------------------------------------------------
def weights(logits, temperature):
    """w = e^((l - max) / T) of one row in float64 (nan: none; +inf: all the weight; T = 0: the first largest)."""
    x = np.asarray(logits, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    if not (x > -np.inf).any():
        return np.zeros_like(x)
    if temperature == 0:
        w = np.zeros_like(x)
        w[int(np.argmax(x))] = 1.0
        return w
    if np.isposinf(x).any():
        return np.where(np.isposinf(x), 1.0, 0.0)
    with np.errstate(over="ignore", under="ignore"):
        return np.where(x > -np.inf, np.exp((x - x.max()) / float(temperature)), 0.0)


def kept(logits, temperature, top_k=0, top_p=1.0, min_p=0.0, off=0.0):
    """Truth values of the tokens that the filters leave; `off` moves the border of top_p by so much of the
    mass (how far sums may be off)."""
    x = np.asarray(logits, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    w = weights(x, temperature)
    there = w > 0 if temperature == 0 or np.isposinf(x).any() else x > -np.inf
    order = np.argsort(-x, kind="stable")
    order = order[there[order]]
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1 and len(order) and temperature > 0:
        before = np.concatenate([[0.0], np.cumsum(w[order])[:-1]])
        total = math.fsum(w[order])
        order = order[:max(1, int((before < float(top_p) * total + off * total).sum()))]
    if min_p > 0 and temperature > 0:
        order = order[w[order] >= float(min_p)]
    out = np.zeros(len(x), bool)
    out[order] = True
    return out


def drawn(w, u, off=0.0):
    """The tokens that u may draw from the weights w where running sums are off by at most `off`."""
    if not (w > 0).any():
        return {-1}
    total, sums = math.fsum(w), np.cumsum(w)
    got = set()
    for t in (-off, 0.0, off):
        over = np.nonzero((sums > u * total + t) & (w > 0))[0]
        got.add(int(over[0]) if len(over) else int(np.nonzero(w)[0][-1]))
    lo, hi = min(got), max(got)
    return {i for i in range(lo, hi + 1) if w[i] > 0}
