"""Plain 64-bit implementations of the attention-layer operators (CPU, written from the formulas)."""
import math

import numpy as np
import torch


# ---- q/k norm + rotation -------------------------------------------------------------------------
def rotation(pos, inv_freq, D, interleaved):
    """cos, signed sin and partner index of every element: out = y cos + y[partner] sin."""
    ang = pos.double()[..., None] * inv_freq.double()
    R2 = ang.shape[-1]
    cos = torch.ones(*pos.shape, D, dtype=torch.float64)
    sin = torch.zeros_like(cos)
    partner = list(range(D))
    for j in range(R2):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + R2)
        cos[..., lo] = cos[..., hi] = torch.cos(ang[..., j])
        sin[..., lo], sin[..., hi] = -torch.sin(ang[..., j]), torch.sin(ang[..., j])
        partner[lo], partner[hi] = hi, lo
    return cos[:, :, None], sin[:, :, None], partner


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """(out, scale): scale bounds the magnitudes that rounding errors of out are relative to."""
    x = x.double()
    cos, sin, partner = rotation(pos, inv_freq, x.shape[-1], interleaved)
    y = w.double() * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y * cos + y[..., partner] * sin, y.abs() + y[..., partner].abs()


def norm_rope_grad(x, w, pos, inv_freq, eps, interleaved, dout):
    """(dx, dw, and the magnitudes their errors are relative to), by the formula."""
    x, w, dout = x.double(), w.double(), dout.double()
    cos, sin, partner = rotation(pos, inv_freq, x.shape[-1], interleaved)
    dy = dout * cos + (dout * sin)[..., partner]
    mag = dout.abs() + dout.abs()[..., partner]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dx = r * (w * dy - x * r * r * (w * dy * x).mean(-1, keepdim=True))
    sx = r * (w.abs() * mag + x.abs() * r * r * (w.abs() * mag * x.abs()).mean(-1, keepdim=True))
    dw = (dy * x * r).sum((0, 1, 2))
    return dx, dw, sx, (mag * x.abs() * r).sum((0, 1, 2))


# ---- verification --------------------------------------------------------------------------------
def verify_row(tokens, parents, n, p, q, u, u_next):
    """One row, by normalised residuals in float64: (path, next token)."""
    if n == 0:
        return [], -1
    clean = lambda r: np.where(r > 0, r, 0.0)  # noqa: E731
    V = p.shape[1]
    path, cur = [0], 0
    while True:
        r, Z = clean(p[cur].astype(np.float64)), 1.0
        draft = clean(q[cur].astype(np.float64)) if q is not None else None
        taken = None
        for i in range(cur + 1, n):
            t = int(tokens[i])
            if parents[i] != cur or not 0 <= t < V:
                continue
            if float(u[i]) * (draft[t] if draft is not None else 1.0) * Z < r[t]:
                taken = i
                break
            if draft is not None:
                left = np.maximum(r / Z - draft, 0.0)
                if left.sum() > 0:
                    r, Z = left, math.fsum(left)
            else:
                Z -= r[t]
                r[t] = 0.0
        if taken is None:
            break
        path.append(taken)
        cur = taken
    if not r.sum() > 0:
        r = clean(p[cur].astype(np.float64))
    if not r.sum() > 0:
        return path, -1
    cdf = np.cumsum(r)
    over = np.nonzero(cdf > float(u_next) * cdf[-1])[0]
    return path, int(over[0]) if len(over) else int(np.nonzero(r)[0][-1])


# ---- pages ---------------------------------------------------------------------------------------
class Pool:
    """Tables, counts and cache entries as lists and arrays."""

    def __init__(self, k, v, table, ctx, refs):
        self.k, self.v = k.clone(), v.clone()
        self.table, self.ctx, self.refs = table.tolist(), ctx.tolist(), refs.tolist()
        self.page, self.M = k.shape[2], table.shape[1]

    def free_pages(self):
        return [e for e, r in enumerate(self.refs) if r == 0]

    def release(self, row):
        for e in self.table[row]:
            if e >= 0:
                self.refs[e] -= 1
        self.table[row], self.ctx[row] = [-1] * self.M, 0

    def reserve(self, rows, extra):
        free = self.free_pages()
        for r in rows:
            have = next((m for m, e in enumerate(self.table[r]) if e < 0), self.M)
            need = max(0, -(-(self.ctx[r] + extra) // self.page) - have)
            if need > len(free):
                free = []
                continue
            for m in range(need):
                self.table[r][have + m] = free.pop(0)
                self.refs[self.table[r][have + m]] += 1

    def fork(self, src, dst):
        for d in dst:
            self.release(d)
        free = self.free_pages()
        for s, d in zip(src, dst):
            full, part = divmod(self.ctx[s], self.page)
            row = self.table[s][:full]
            if part:
                if not free:
                    continue
                e, f = free.pop(0), self.table[s][full]
                self.k[:, e, :part], self.v[:, e, :part] = self.k[:, f, :part], self.v[:, f, :part]
                row = row + [e]
            for e in row:
                self.refs[e] += 1
            self.table[d], self.ctx[d] = row + [-1] * (self.M - len(row)), self.ctx[s]

    def slot(self, row, at):
        return self.table[row][at // self.page], at % self.page

    def compact(self, path, n_path):
        out = []
        for b, n in enumerate(n_path):
            old = [(self.k[(slice(None), *self.slot(b, self.ctx[b] + i))].clone(),
                    self.v[(slice(None), *self.slot(b, self.ctx[b] + i))].clone()) for i in path[b][:n]]
            for i in range(n):
                e, o = self.slot(b, self.ctx[b] + i)
                self.k[:, e, o], self.v[:, e, o] = old[i]
            out.append(self.ctx[b] + n)
        return out


# ---- attention -----------------------------------------------------------------------------------
def tree_attn(q, k_pages, v_pages, table, ctx, lengths, see, scale):
    """(o, lse, A, E): A = sum_j p_j |v_j| and E = max_j scale sum_d |q_d k_jd| set the errors' size.
    see [B, N, N] truth values among nodes; unseen positions are left out of every sum."""
    B, N, Hq, D = q.shape
    page, Hk = k_pages.shape[1:3]
    o = torch.zeros(B, N, Hq, D, dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    A, E = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n, c = int(lengths[b]), int(ctx[b])
        at = torch.arange(c + n)
        if c + n == 0:
            continue
        pages = table[b].long()[at // page]
        k, v = k_pages[pages, at % page].double(), v_pages[pages, at % page].double()   # [c + n, Hk, D]
        for i in range(n):
            vis = torch.cat([torch.ones(c, dtype=torch.bool), see[b, i, :n]])
            if not vis.any():
                continue
            ki, vi = k[vis], v[vis]
            for h in range(Hq):
                kh, vh = ki[:, h // (Hq // Hk)], vi[:, h // (Hq // Hk)]
                s = kh @ q[b, i, h].double() * scale
                lse[b, i, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                o[b, i, h], A[b, i, h] = p @ vh, p @ vh.abs()
                E[b, i, h] = (kh.abs() @ q[b, i, h].double().abs()).max() * scale
    return o, lse, A, E
