"""The operators of a speculative decoding step, as a program calls them, and their plain forms.

Four operators of the softmax-attention layers that stand beside the gated delta rule layers of a
hybrid model, over a cache of pages that forked rows share:

  norm_rope   norms of queries and keys for each head with the position rotation (forward; forward
              that leaves k and v in the cache's pages; gradient)
  attn        attention of a tree (or a chain) of drafted tokens over the cache
  verify      verification of drafted tokens against the target's probabilities
  fork,       a fork of rows that share the full pages of their source, and the move of an accepted
  compact     path's entries to the front of its row

listed() and draw() give cases, prepare() what a program holds before the call, run() one pass:
the plain form where `own` is false, the framework's calls where it is true; work() the bytes and
operations a pass cannot do without; exact() the same results from the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
_GOLDEN = 0.6180339887498949


# --------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------
def listed():
    return [
        # one new token of one short sequence: latency alone
        dict(name="attn one token", op="attn", B=1, N=1, Hq=16, Hk=4, D=128, ctx=700, page=64, tree=False),
        # an ordinary serving batch: small trees over ragged contexts, an odd node count
        dict(name="attn batch of trees", op="attn", B=16, N=13, Hq=32, Hk=8, D=128, ctx=8192, page=64, tree=True),
        # wide trees: 512 query rows for each key head, bound by the products
        dict(name="attn wide trees", op="attn", B=8, N=64, Hq=32, Hk=4, D=128, ctx=16384, page=64, tree=True),
        # two long contexts in small pages, heads of 256
        dict(name="attn long contexts", op="attn", B=2, N=7, Hq=16, Hk=2, D=256, ctx=131072, page=16, tree=True),
        # one decode step's q, k, v out of the fused projection, k and v into the pages
        dict(name="norm_rope one token", op="append", B=24, N=1, Hq=16, Hk=4, D=128, R=128, page=64, ctx=900,
             interleaved=False, fused=True),
        # a training or prefill row
        dict(name="norm_rope row", op="norm_rope", B=1, N=8192, Hq=32, Hk=8, D=128, R=128, f32=False,
             interleaved=False, fused=False),
        # the gradient of short rows of an odd length, a quarter of each head rotated
        dict(name="norm_rope gradient", op="norm_rope_grad", B=3, N=2731, Hq=16, Hk=2, D=256, R=64, f32=False,
             interleaved=False, fused=False),
        # a chain of five drafts for one sequence: latency
        dict(name="verify chain", op="verify", B=1, N=6, V=32000, width=1, drawn=True),
        # a batch of trees, up to three drafts of each node, a large vocabulary
        dict(name="verify trees", op="verify", B=48, N=24, V=131072, width=3, drawn=True),
        # the framework's own fork batch: 256 forks of a few trunks, four layers' caches
        dict(name="fork 256", op="fork", F=256, trunks=8, layers=4, Hk=4, D=128, ctx=2048, page=64),
        # a few forks of one row: latency
        dict(name="fork few", op="fork", F=3, trunks=1, layers=2, Hk=2, D=128, ctx=500, page=64),
        # the accepted paths of a batch, eight layers' caches
        dict(name="compact batch", op="compact", B=64, N=32, layers=8, Hk=4, D=128, ctx=1024, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "norm_rope", "norm_rope_grad", "verify", "verify", "fork",
                     "compact"])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "attn":
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
        tree = rng.random() < 0.7
        N = 1 if rng.random() < 0.2 else _log(rng, 2, 100)
        B = _log(rng, 1, 48)
        most = min(131072, int(1e8 / (B * Hk * D)), int(2e10 / (B * Hq * N * D)))
        return dict(op=op, B=B, N=N, Hq=Hq, Hk=Hk, D=D, ctx=_log(rng, 1, max(2, most)), page=page, tree=tree)
    if op in ("append", "norm_rope", "norm_rope_grad"):
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5])
        R = rng.choice([r for r in (16, 32, 48, 64, 128, 256) if r <= D])
        more = dict(Hq=Hq, Hk=Hk, D=D, R=R, interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
        if op == "append":
            return dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 33), page=page, ctx=_log(rng, 1, 4000), **more)
        B = rng.choice([1, 2, 3])
        most = int(4e7 / (B * (Hq + Hk) * D))
        return dict(op=op, B=B, N=_log(rng, 1, max(2, min(8192, most))), f32=rng.random() < 0.4, **more)
    if op == "verify":
        B, N = _log(rng, 1, 48), _log(rng, 1, 32)
        V = _log(rng, 1000, max(1001, min(131072, int(1.4e8 / (B * N)))))
        return dict(op=op, B=B, N=N, V=V, width=rng.choice([1, 2, 3, 4]), drawn=rng.random() < 0.6)
    layers, Hk = rng.choice([1, 2, 4]), rng.choice([1, 2, 4])
    if op == "fork":
        F = _log(rng, 1, 256)
        return dict(op=op, F=F, trunks=min(F, _log(rng, 1, 16)), layers=layers, Hk=Hk, D=D, ctx=_log(rng, 1, 2048),
                    page=min(page, 64))
    return dict(op=op, B=_log(rng, 1, 64), N=_log(rng, 1, 40), layers=layers, Hk=Hk, D=D, ctx=_log(rng, 1, 1024),
                page=min(page, 64))


def _spread(most, n):
    """n lengths in (0, most], the longest first: most itself, then spread over (most / 4, most]."""
    return [max(1, int(most * (1.0 - 0.75 * ((i * _GOLDEN) % 1.0)))) for i in range(n)]


def _nodes(case):
    """Valid nodes of each row: N for a single row or token, else up to a quarter fewer."""
    B, N = case["B"], case["N"]
    return [max(1, N - (i * 5) % max(1, N // 4 + 1)) if B > 1 else N for i in range(B)]


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _parents(g, B, N, width):
    """Random trees in topological order: parents[:, i] < i (-1 at the root), chains for width 1."""
    u = torch.rand(B, N, generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    back = (u * torch.clamp(i, max=1 if width == 1 else 2 * width)).floor().long() + 1
    return torch.where(i > 0, i - torch.minimum(back, i), torch.full_like(i, -1)).int()


def _ancestors(parents):
    """[B, N, N] truth values: node j is node i or one of its ancestors."""
    B, N = parents.shape
    see = torch.zeros(B, N, N, dtype=torch.bool, device=parents.device)
    rows = torch.arange(B, device=parents.device)
    for i in range(N):
        if i:
            see[:, i] = see[rows, parents[:, i].long()]
        see[:, i, i] = True
    return see


def _pack(see):
    """[B, N, N] truth values as [B, N, ceil(N / 64)] int64 words, bit j of word w for node 64 w + j."""
    B, N, _ = see.shape
    W = (N + 63) // 64
    full = torch.zeros(B, N, W * 64, dtype=torch.int64, device=see.device)
    full[..., :N] = see.long()
    return (full.view(B, N, W, 64) << torch.arange(64, device=see.device)).sum(-1)


def _pages(g, rows, page, spare=3):
    """A page table for rows of so many positions: distinct pages in a random order, -1 past a row's own."""
    need = [-(-r // page) for r in rows]
    P, M = sum(need) + spare, max(need)
    order = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.full((len(rows), M), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, P


def _inv_freq(R):
    return 10000000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)


def _shuffled(g, values):
    order = torch.randperm(len(values), generator=g, device="cuda")
    return torch.tensor(values, dtype=torch.int32, device="cuda")[order]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "attn":
        B, N, Hq, Hk, D, page = (case[k] for k in ("B", "N", "Hq", "Hk", "D", "page"))
        s["ctx"] = _shuffled(g, _spread(case["ctx"], B))
        s["lengths"] = _shuffled(g, _nodes(case))
        s["table"], P = _pages(g, [c + N for c in s["ctx"].tolist()], page)
        s["q"] = _randn(g, B, N, Hq, D, dtype=torch.bfloat16, scale=1.5)
        s["k_pages"] = _randn(g, P, page, Hk, D, dtype=torch.bfloat16)
        s["v_pages"] = _randn(g, P, page, Hk, D, dtype=torch.bfloat16)
        s["mask"] = _pack(_ancestors(_parents(g, B, N, 3))) if case["tree"] else None
    elif op in ("append", "norm_rope", "norm_rope_grad"):
        B, N, Hq, Hk, D, R = (case[k] for k in ("B", "N", "Hq", "Hk", "D", "R"))
        dtype = torch.float32 if case.get("f32") else torch.bfloat16
        heads = Hq + 2 * Hk
        x = _randn(g, B, N, heads, D, dtype=dtype, scale=2.0)  # the projection, q | k | v
        s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (s[n].contiguous() for n in "qkv")
        s["q_w"], s["k_w"] = 1.0 + _randn(g, D, scale=0.1), 1.0 + _randn(g, D, scale=0.1)
        s["inv_freq"] = _inv_freq(R)
        if op == "append":
            s["ctx"] = _shuffled(g, _spread(case["ctx"], B))
            s["pos"] = s["ctx"][:, None] + torch.arange(N, device="cuda", dtype=torch.int32)
            s["table"], P = _pages(g, [c + N for c in s["ctx"].tolist()], case["page"])
            s["k_pages"] = _randn(g, P, case["page"], Hk, D, dtype=torch.bfloat16)
            s["v_pages"] = _randn(g, P, case["page"], Hk, D, dtype=torch.bfloat16)
        else:
            first = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda", dtype=torch.int32)
            s["pos"] = first + torch.arange(N, device="cuda", dtype=torch.int32)
        if op == "norm_rope_grad":
            s["dq_out"] = _randn(g, B, N, Hq, D, dtype=dtype)
            s["dk_out"] = _randn(g, B, N, Hk, D, dtype=dtype)
    elif op == "verify":
        B, N, V = case["B"], case["N"], case["V"]
        s["parents"] = _parents(g, B, N, case["width"])
        s["lengths"] = _shuffled(g, _nodes(case))
        logits = _randn(g, B, N, V, scale=3.0)
        s["p"] = torch.softmax(logits, -1)
        q = torch.softmax(logits.add_(_randn(g, B, N, V, scale=0.7)), -1)
        del logits
        rows = torch.arange(B, device="cuda")
        tokens = torch.zeros(B, N, dtype=torch.int32, device="cuda")
        if case["drawn"]:  # children drawn from the draft model's distribution at their parent
            s["q"] = q
            u = torch.rand(B, N, generator=g, device="cuda")
            for i in range(1, N):
                cdf = q[rows, s["parents"][:, i].long()].cumsum(-1)
                at = torch.searchsorted(cdf, (u[:, i] * cdf[:, -1])[:, None], right=True)
                tokens[:, i] = at[:, 0].clamp(max=V - 1).int()
        else:  # the draft model's best tokens at their parent, in order
            s["q"] = None
            for i in range(1, N):
                nth = (s["parents"][:, :i] == s["parents"][:, i:i + 1]).sum(1)
                best = q[rows, s["parents"][:, i].long()].topk(min(V, 64), -1).indices
                tokens[:, i] = best.gather(1, nth.clamp(max=63)[:, None])[:, 0].int()
        s["tokens"] = tokens
        s["u"] = torch.rand(B, N, generator=g, device="cuda")
        s["u_next"] = torch.rand(B, generator=g, device="cuda")
    elif op == "fork":
        F, T, page = case["F"], case["trunks"], case["page"]
        ctx = _shuffled(g, _spread(case["ctx"], T)).tolist()
        table, P = _pages(g, ctx, page, spare=F + 5)
        s["table"] = torch.cat([table, torch.full((F, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        s["ctx"] = torch.tensor(ctx + [0] * F, dtype=torch.int32, device="cuda")
        s["refs"] = torch.zeros(P, dtype=torch.int32, device="cuda")
        s["refs"][table[table >= 0].long()] = 1
        s["src"] = torch.randint(0, T, (F,), generator=g, device="cuda", dtype=torch.int32)
        s["dst"] = T + torch.randperm(F, generator=g, device="cuda").int()
        shape = (case["layers"], P, page, case["Hk"], case["D"])
        s["k_cache"], s["v_cache"] = (_randn(g, *shape, dtype=torch.bfloat16) for _ in "kv")
    elif op == "compact":
        B, N, page = case["B"], case["N"], case["page"]
        s["ctx"] = _shuffled(g, _spread(case["ctx"], B))
        s["table"], P = _pages(g, [c + N for c in s["ctx"].tolist()], page)
        shape = (case["layers"], P, page, case["Hk"], case["D"])
        s["k_cache"], s["v_cache"] = (_randn(g, *shape, dtype=torch.bfloat16) for _ in "kv")
        # accepted paths: the root, then each node with an even chance, up to nine of them
        keep = torch.rand(B, N, generator=g, device="cuda") < 0.5
        keep[:, 0] = True
        keep &= keep.long().cumsum(1) <= 9
        s["n_path"] = keep.sum(1).int()
        order = torch.argsort((~keep).int(), dim=1, stable=True).int()
        s["path"] = torch.where(torch.arange(N, device="cuda") < s["n_path"][:, None], order, -1)
    return s


# --------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------
def _rows_of(pages, table, length):
    """The first `length` positions of every row of a page table: [B, length, Hk, D] in 32 bits."""
    got = pages[table.long().clamp(min=0)]
    return got.reshape(table.shape[0], -1, *pages.shape[2:])[:, :length].float()


def _plain_attn(q, k_pages, v_pages, table, ctx, lengths, mask):
    B, N, Hq, D = q.shape
    Hk, G = k_pages.shape[2], Hq // k_pages.shape[2]
    length = table.shape[1] * k_pages.shape[1]
    k, v = (_rows_of(x, table, length) for x in (k_pages, v_pages))
    s = torch.matmul(q.float().view(B, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, N * G, D),
                     k.permute(0, 2, 3, 1)).view(B, Hk, N, G, length) * D ** -0.5
    node = torch.arange(length, device=q.device) - ctx[:, None]  # [B, length]: below 0 in the context
    i = torch.arange(N, device=q.device)
    if mask is None:
        see = node[:, None, :] <= i[:, None]
    else:
        word = mask.gather(2, (node.clamp(0, N - 1) // 64)[:, None, :].expand(B, N, length))
        see = (node[:, None, :] < 0) | ((word >> (node.clamp(0, N - 1) % 64)[:, None, :]) & 1 > 0)
    see = see & (node < lengths[:, None])[:, None, :] & (i < lengths[:, None])[:, :, None]
    s = s.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.clamp(min=-3e38))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hk, N * G, length), v.permute(0, 2, 1, 3)).view(B, Hk, N, G, D)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(q.dtype),
            lse.permute(0, 2, 1, 3).reshape(B, N, Hq))


def _angles(inv_freq, pos):
    """cos and sin of position times frequency, [B, N, 1, R / 2] in 32 bits, from angles in 64."""
    a = pos.double()[..., None] * inv_freq
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _turn(y, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    if interleaved:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., R:]], -1)


def _plain_norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    return _turn(w * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS), cos, sin, interleaved)


def _plain_norm_rope_grad(x, w, dout, cos, sin, interleaved):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dy = _turn(dout.float(), cos, -sin, interleaved)
    dw = (dy * x * r).sum((0, 1, 2))
    wdy = w * dy
    return r * (wdy - x * r.square() * (wdy * x).mean(-1, keepdim=True)), dw


def _slots(table, at, page):
    """The slot of position `at` [B, n] of each row in the cache's pages laid end to end."""
    at = at.long()
    return table.long().gather(1, at // page) * page + at % page


def _plain_verify(tokens, parents, lengths, p, q, u, u_next):
    """Walks every tree at once, one node after the other: an accepted node becomes the current one,
    and later nodes whose parent is the current one are its candidates. A refused candidate takes the
    residual on: max(p - c q, 0) with c grown by the residual's own sum (drafts drawn from q), or p
    without the token (drafts given)."""
    B, N, V = p.shape
    rows = torch.arange(B, device=p.device)
    zero = torch.zeros((), dtype=torch.float64, device=p.device)
    rest, cur = p[:, 0].double(), torch.zeros(B, dtype=torch.long, device=p.device)
    mass = torch.ones(B, dtype=torch.float64, device=p.device)
    c = torch.zeros(B, dtype=torch.float64, device=p.device)
    alive = lengths > 0
    path = torch.full((B, N), -1, dtype=torch.int32, device=p.device)
    path[:, 0] = torch.where(alive, 0, -1)
    count = alive.long()
    for i in range(1, N):
        t = tokens[:, i].long()
        cand = (i < lengths) & (parents[:, i] == cur)
        here = rest[rows, t]
        qt = q[rows, cur, t].double() if q is not None else 1.0
        yes = cand & (u[:, i].double() * qt * mass < here)
        no = cand & ~yes
        if q is not None:
            pc, qc = p[rows, cur].double(), q[rows, cur].double()
            grown = c + mass
            left = (pc - grown[:, None] * qc).clamp(min=0)
            total = left.sum(-1)
            no = no & (total > 0)
            c, mass = torch.where(no, grown, c), torch.where(no, total, mass)
            rest = torch.where(no[:, None], left, rest)
        else:
            rest = rest.clone()
            rest[rows, t] = torch.where(no, zero, here)
            mass = torch.where(no, mass - here, mass)
        path[rows, count.clamp(max=N - 1)] = torch.where(yes, i, path[rows, count.clamp(max=N - 1)])
        count = count + yes
        cur = torch.where(yes, i, cur)
        rest = torch.where(yes[:, None], p[:, i].double(), rest)
        c, mass = torch.where(yes, zero, c), torch.where(yes, 1.0, mass)
    none = ~(rest.sum(-1) > 0)
    rest = torch.where(none[:, None], p[rows, cur].double(), rest)
    cdf = rest.cumsum(-1)
    token = (cdf <= u_next.double()[:, None] * cdf[:, -1:]).sum(-1)
    last = V - 1 - (rest.flip(-1) > 0).int().argmax(-1)
    token = torch.where(cdf[:, -1] > 0, torch.minimum(token, last), -1)
    return path, count.int(), torch.where(alive, token, -1).int()


def _plain_fork(k_cache, v_cache, table, ctx, refs, src, dst):
    page, M = k_cache.shape[2], table.shape[1]
    src, dst = src.long(), dst.long()
    old = table[dst]  # what the forked rows held goes back first
    refs.index_add_(0, old.clamp(min=0).reshape(-1).long(), -(old >= 0).reshape(-1).int())
    n = ctx[src]
    full, part = n // page, n % page
    free = torch.argsort((refs != 0).int(), stable=True).int()  # free pages, the lowest first
    new = free[((part > 0).long().cumsum(0) - 1).clamp(min=0)]
    at, cols = table[src], torch.arange(M, device=table.device)
    row = torch.where(cols < full[:, None], at, torch.where((cols == full[:, None]) & (part > 0)[:, None],
                                                            new[:, None], -1))
    table[dst], ctx[dst] = row, n
    refs.index_add_(0, row.clamp(min=0).reshape(-1).long(), (row >= 0).reshape(-1).int())
    a = at.gather(1, full.clamp(max=M - 1).long()[:, None])[:, 0]  # the source's last, partly filled page
    a = torch.where(part > 0, a, at[:, 0]).long()
    b = torch.where(part > 0, new, at[:, 0]).long()
    copied = (torch.arange(page, device=table.device) < part[:, None])[None, :, :, None, None]
    k_cache[:, b] = torch.where(copied, k_cache[:, a], k_cache[:, b])
    v_cache[:, b] = torch.where(copied, v_cache[:, a], v_cache[:, b])


def _plain_compact(k_cache, v_cache, table, ctx, path, n_path):
    page = k_cache.shape[2]
    i = torch.arange(path.shape[1], device=path.device)
    node = torch.where(i < n_path[:, None], path, i)
    a = _slots(table, ctx[:, None] + node, page)
    b = _slots(table, ctx[:, None] + i, page)
    k, v = (x.view(x.shape[0], -1, *x.shape[3:]) for x in (k_cache, v_cache))
    k[:, b], v[:, b] = k[:, a], v[:, a]
    return ctx + n_path


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from gated_deltanet_rule_gb300 import gdr
    if op == "attn":
        args = (s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"])
        if own:
            return gdr.gdr_tree_attn(*args, lengths=s["lengths"], mask=s["mask"], want_lse=True)
        return _plain_attn(*args, s["lengths"], s["mask"])
    if op == "append":
        if own:
            q = gdr.gdr_qk_norm_rope_append(s["q"], s["k"], s["v"], s["q_w"], s["k_w"], s["inv_freq"], s["pos"],
                                            s["k_pages"], s["v_pages"], s["table"], s["ctx"], eps=EPS,
                                            interleaved=case["interleaved"])
        else:
            turn = (*_angles(s["inv_freq"], s["pos"]), case["interleaved"])
            q = _plain_norm_rope(s["q"], s["q_w"], *turn).to(s["q"].dtype)
            k = _plain_norm_rope(s["k"], s["k_w"], *turn).to(s["k_pages"].dtype)
            page = case["page"]
            i = torch.arange(case["N"], device=q.device)
            at = _slots(s["table"], s["ctx"][:, None] + i, page)
            s["k_pages"].view(-1, *k.shape[2:])[at] = k
            s["v_pages"].view(-1, *k.shape[2:])[at] = s["v"]
        return q, s["k_pages"], s["v_pages"]
    if op == "norm_rope":
        if own:
            return gdr.gdr_qk_norm_rope(s["q"], s["k"], s["q_w"], s["k_w"], s["inv_freq"], s["pos"], eps=EPS,
                                        interleaved=case["interleaved"])
        turn = (*_angles(s["inv_freq"], s["pos"]), case["interleaved"])
        return (_plain_norm_rope(s["q"], s["q_w"], *turn).to(s["q"].dtype),
                _plain_norm_rope(s["k"], s["k_w"], *turn).to(s["k"].dtype))
    if op == "norm_rope_grad":
        if own:
            return gdr.gdr_qk_norm_rope_backward(s["q"], s["k"], s["q_w"], s["k_w"], s["inv_freq"], s["pos"],
                                                 s["dq_out"], s["dk_out"], eps=EPS, interleaved=case["interleaved"])
        turn = (*_angles(s["inv_freq"], s["pos"]), case["interleaved"])
        dq, dq_w = _plain_norm_rope_grad(s["q"], s["q_w"], s["dq_out"], *turn)
        dk, dk_w = _plain_norm_rope_grad(s["k"], s["k_w"], s["dk_out"], *turn)
        return dq, dk, dq_w, dk_w
    if op == "verify":
        args = (s["tokens"], s["parents"], s["lengths"], s["p"], s["q"], s["u"], s["u_next"])
        return gdr.gdr_verify_draft(*args) if own else _plain_verify(*args)
    if op == "fork":
        args = (s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["refs"], s["src"], s["dst"])
        gdr.gdr_cache_fork(*args) if own else _plain_fork(*args)
        return args[:5]
    args = (s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["path"], s["n_path"])
    new_ctx = gdr.gdr_cache_compact(*args) if own else _plain_compact(*args)
    return s["k_cache"], s["v_cache"], new_ctx


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "attn":
        B, N, Hq, Hk, D = (case[k] for k in ("B", "N", "Hq", "Hk", "D"))
        ctx, n = _spread(case["ctx"], B), sum(_nodes(case)) / B
        keys = sum(ctx) + B * n
        return dict(bytes=keys * Hk * D * 4 + B * n * Hq * D * 4 + B * N * Hq * 4 + B * N * ((N + 63) // 64) * 8,
                    flops=4 * n * Hq * D * keys)
    if op in ("append", "norm_rope", "norm_rope_grad"):
        heads = case["B"] * case["N"] * case["D"]
        size = 4 if case.get("f32") else 2
        q, k = heads * case["Hq"], heads * case["Hk"]
        if op == "append":
            return dict(bytes=2 * size * (q + 2 * k), flops=8 * (q + k))
        if op == "norm_rope":
            return dict(bytes=2 * size * (q + k), flops=8 * (q + k))
        return dict(bytes=(2 * size + 4) * (q + k), flops=16 * (q + k))
    if op == "verify":
        rows = case["B"] * case["V"]  # the distributions at one node of each row: p, and q where it is given
        return dict(bytes=rows * 4 * (2 if case["drawn"] else 1), flops=rows * 3)
    entry = case["layers"] * case["Hk"] * case["D"] * 2 * 2  # bytes of one position, k and v
    if op == "fork":
        page, ctx = case["page"], _spread(case["ctx"], case["trunks"])
        part = sum(c % page for c in ctx) / len(ctx)
        pages = sum(-(-c // page) for c in ctx) / len(ctx)
        return dict(bytes=case["F"] * (2 * part * entry + pages * 16), flops=case["F"] * pages)
    moved = sum(min(8, 0.5 * (case["N"] - 1)) for _ in range(case["B"]))
    return dict(bytes=2 * moved * entry + case["B"] * case["N"] * 4 + 1, flops=0)


# --------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------
def _exact_attn(s):
    q, ctx, lengths, table = s["q"].double(), s["ctx"].tolist(), s["lengths"].tolist(), s["table"].long()
    B, N, Hq, D = q.shape
    Hk = s["k_pages"].shape[2]
    o = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n, c, page = lengths[b], ctx[b], s["k_pages"].shape[1]
        own_pages = table[b, :-(-(c + n) // page)]
        see = torch.zeros(n, c + n, dtype=torch.bool, device=q.device)
        see[:, :c] = True
        for j in range(n):
            if s["mask"] is None:
                see[j:, c + j] = True
            else:
                see[:, c + j] = (s["mask"][b, :n, j // 64] >> (j % 64)) % 2 == 1
        for h in range(Hq):
            hk = h // (Hq // Hk)
            k = s["k_pages"][own_pages, :, hk].reshape(-1, D)[:c + n].double()
            v = s["v_pages"][own_pages, :, hk].reshape(-1, D)[:c + n].double()
            a = (q[b, :n, h] @ k.T) / math.sqrt(D)
            a[~see] = -math.inf
            lse[b, :n, h] = torch.logsumexp(a, -1)
            o[b, :n, h] = torch.softmax(a, -1) @ v
    return o, lse


def _rotation(s, interleaved, D):
    """The rotations of every position as matrices would act: index of the partner and the factors."""
    a = s["pos"].double()[..., None] * s["inv_freq"]
    half = a.shape[-1]
    cos = torch.ones(*a.shape[:2], D, dtype=torch.float64, device=a.device)
    sin = torch.zeros_like(cos)
    partner = torch.arange(D, device=a.device)
    j = torch.arange(half, device=a.device)
    lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    cos[..., lo], cos[..., hi] = torch.cos(a), torch.cos(a)
    sin[..., lo], sin[..., hi] = -torch.sin(a), torch.sin(a)
    partner[lo], partner[hi] = hi, lo
    return cos[:, :, None], sin[:, :, None], partner


def _exact_norm_rope(x, w, rot):
    cos, sin, partner = rot
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    return y * cos + y[..., partner] * sin


def _exact_norm_rope_grad(x, w, dout, rot):
    """By the chain rule through automatic differentiation of the definition."""
    x = x.double().detach().clone().requires_grad_(True)
    w = w.double().detach().clone().requires_grad_(True)
    y = _exact_norm_rope(x, w, rot)
    return torch.autograd.grad(y, (x, w), dout.double())


def _exact_verify(s):
    tokens, parents, lengths = s["tokens"].tolist(), s["parents"].tolist(), s["lengths"].tolist()
    u, u_next = s["u"].double().tolist(), s["u_next"].double().tolist()
    B, N, V = s["p"].shape
    paths, counts, nexts = [], [], []
    for b in range(B):
        path, cur = [0], 0
        children = {}
        for i in range(1, lengths[b]):
            children.setdefault(parents[b][i], []).append(i)
        while True:
            r = s["p"][b, cur].double()
            draft = s["q"][b, cur].double() if s["q"] is not None else None
            whole, gone, taken = 1.0, None, None
            for i in children.get(cur, []):
                t = tokens[b][i]
                if u[b][i] * (float(draft[t]) if draft is not None else 1.0) * whole < float(r[t]):
                    taken = i
                    break
                if draft is not None:
                    # the residual of the normalised rest against the draft distribution
                    rest = torch.relu(r / whole - draft)
                    if float(rest.sum()) > 0:
                        r, whole = rest, float(rest.sum())
                else:
                    r = r.clone()
                    whole -= float(r[t])
                    r[t] = 0.0
            if taken is None:
                break
            path.append(taken)
            cur = taken
        if not float(r.sum()) > 0:
            r = s["p"][b, cur].double()
        cdf = torch.cumsum(r, 0)
        above = torch.nonzero(cdf > u_next[b] * float(cdf[-1]))
        nexts.append(int(above[0]) if len(above) else int(torch.nonzero(r)[-1]))
        counts.append(len(path))
        paths.append(path + [-1] * (N - len(path)))
    back = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(paths, **back), torch.tensor(counts, **back), torch.tensor(nexts, **back)


def _exact_fork(s):
    k, v = s["k_cache"].double(), s["v_cache"].double()
    table, ctx, refs = s["table"].tolist(), s["ctx"].tolist(), s["refs"].tolist()
    page = k.shape[2]
    for row in s["dst"].tolist():
        for e in table[row]:
            if e >= 0:
                refs[e] -= 1
        table[row] = [-1] * len(table[row])
    taken, free = [], iter([e for e, r in enumerate(refs) if r == 0])
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        full, part = divmod(ctx[a], page)
        mine = table[a][:full]
        if part:
            e = next(free)
            k[:, e, :part], v[:, e, :part] = k[:, table[a][full], :part], v[:, table[a][full], :part]
            mine = mine + [e]
        taken += mine
        table[b], ctx[b] = mine + [-1] * (len(table[b]) - len(mine)), ctx[a]
    for e in taken:
        refs[e] += 1
    back = dict(dtype=torch.int32, device="cuda")
    return k, v, torch.tensor(table, **back), torch.tensor(ctx, **back), torch.tensor(refs, **back)


def _exact_compact(s):
    k, v = s["k_cache"].double(), s["v_cache"].double()
    page, table, ctx = k.shape[2], s["table"].tolist(), s["ctx"].tolist()
    frm, to = [], []
    for b, (path, n) in enumerate(zip(s["path"].tolist(), s["n_path"].tolist())):
        for i, node in enumerate(path[:n]):
            for at, into in ((ctx[b] + node, frm), (ctx[b] + i, to)):
                into.append(table[b][at // page] * page + at % page)
    frm, to = torch.tensor(frm, device=k.device), torch.tensor(to, device=k.device)
    for x in (k, v):
        x = x.view(x.shape[0], -1, *x.shape[3:])
        x[:, to] = x[:, frm].clone()
    return k, v, s["ctx"] + s["n_path"]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "attn":
        return _exact_attn(s)
    if op in ("append", "norm_rope", "norm_rope_grad"):
        rot = _rotation(s, case["interleaved"], case["D"])
        if op == "norm_rope_grad":
            dq, dq_w = _exact_norm_rope_grad(s["q"], s["q_w"], s["dq_out"], rot)
            dk, dk_w = _exact_norm_rope_grad(s["k"], s["k_w"], s["dk_out"], rot)
            return dq, dk, dq_w, dk_w
        q, k = _exact_norm_rope(s["q"], s["q_w"], rot), _exact_norm_rope(s["k"], s["k_w"], rot)
        if op == "norm_rope":
            return q, k
        kp, vp, page = s["k_pages"].double(), s["v_pages"].double(), case["page"]
        table = s["table"].tolist()
        for b, c in enumerate(s["ctx"].tolist()):
            for i in range(case["N"]):
                e, at = table[b][(c + i) // page], (c + i) % page
                kp[e, at], vp[e, at] = k[b, i], s["v"][b, i].double()
        return q, kp, vp
    return {"verify": _exact_verify, "fork": _exact_fork, "compact": _exact_compact}[op](s)
