"""The operators of a step that decodes many forks of a few trunks, as a program calls them, and their plain forms.

  fork_attn   attention of forked rows over the pages that they share with their trunk, read once for all
              of them, and over their own
  sample      tokens from logits with temperature, top-k, top-p and min-p and given uniform numbers, and the
              probabilities that a verification of drafts compares
  block_norm  what stands between two blocks of a layer: the norm after the one, its gate and residual
              scale, the sum into the residual, and the norm before the other (forward and gradient)

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
        # three samples of one short prompt: latency alone
        dict(name="fork_attn few forks", op="fork_attn", B=3, T=1, N=1, Hq=16, Hk=4, D=128, shared=448, more=60, page=64,
             tree=False),
        # the framework's own fork batch, decoding: 256 forks of a few trunks
        dict(name="fork_attn batch", op="fork_attn", B=256, T=8, N=1, Hq=32, Hk=8, D=128, shared=8192, more=256, page=64,
             tree=False),
        # one long trunk in small pages, heads of 256
        dict(name="fork_attn long trunk", op="fork_attn", B=64, T=1, N=1, Hq=16, Hk=2, D=256, shared=65536, more=128,
             page=16, tree=False),
        # the fork pass itself: forks of up to 64 tokens each after their trunk, right-padded
        dict(name="fork_attn tokens of forks", op="fork_attn", B=64, T=4, N=64, Hq=16, Hk=4, D=128, shared=8192, more=63,
             page=64, tree=False),
        # one sequence's next token, all filters: latency
        dict(name="sample one token", op="sample", R=1, V=32000, f32=True, top_k=True, top_p=True, min_p=False,
             draws=True, probs=False, wide=False),
        # the forks' next tokens from the head's bfloat16 logits, top-p alone (ties by the thousand)
        dict(name="sample forks", op="sample", R=256, V=131072, f32=False, top_k=False, top_p=True, min_p=False,
             draws=True, probs=False, wide=False),
        # a draft's tokens with the probabilities that its verification needs, an odd vocabulary in padded rows
        dict(name="sample draft", op="sample", R=48, V=49999, f32=True, top_k=True, top_p=True, min_p=True, draws=True,
             probs=True, wide=True),
        # the target's probabilities at every node of small trees, no token drawn
        dict(name="sample target", op="sample", R=96, V=131072, f32=True, top_k=False, top_p=True, min_p=True,
             draws=False, probs=True, wide=False),
        # one decode step's tokens between two blocks
        dict(name="block_norm one token", op="block_norm", rows=24, C=2048, f32=False, gate=True, post=True, scale=True,
             fused=True),
        # a training or prefill row
        dict(name="block_norm row", op="block_norm", rows=8192, C=4096, f32=False, gate=True, post=True, scale=True,
             fused=False),
        # the gradient of such a row
        dict(name="block_norm gradient", op="block_norm_grad", rows=8192, C=4096, f32=False, gate=True, post=True,
             scale=True, fused=False),
        # the gradient without gate and post norm, float32, odd rows
        dict(name="block_norm plain gradient", op="block_norm_grad", rows=2731, C=2560, f32=True, gate=False, post=False,
             scale=False, fused=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fork_attn", "fork_attn", "fork_attn", "sample", "sample", "sample", "block_norm",
                     "block_norm_grad"])
    if op == "fork_attn":
        D = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
        N = 1 if rng.random() < 0.6 else _log(rng, 2, 64)
        B = _log(rng, 1, min(256, 4096 // N))
        T = min(B, _log(rng, 1, 8))
        more = _log(rng, 1, 300)
        most = min(65536, int(2e10 / (B * N * Hq * 128)) * 128, int(2e8 / (T * Hk * D)))
        return dict(op=op, B=B, T=T, N=N, Hq=Hq, Hk=Hk, D=D, shared=_log(rng, page, max(page + 1, min(most, int(5e8 / (B * N * Hq))))),
                    more=more, page=page, tree=N > 1 and rng.random() < 0.5)
    if op == "sample":
        R = _log(rng, 1, 256)
        draws = rng.random() < 0.8
        return dict(op=op, R=R, V=_log(rng, 1000, max(1001, min(131072, int(1.2e7 / R)))), f32=rng.random() < 0.6,
                    top_k=rng.random() < 0.5, top_p=rng.random() < 0.6, min_p=rng.random() < 0.4, draws=draws,
                    probs=not draws or rng.random() < 0.4, wide=rng.random() < 0.3)
    C = 8 * _log(rng, 16, 1024)
    return dict(op=op, rows=_log(rng, 1, max(2, min(8192, int(3e7 / C)))), C=C, f32=rng.random() < 0.4, gate=rng.random() < 0.6,
                post=rng.random() < 0.6, scale=rng.random() < 0.6, fused=rng.random() < 0.4)


def _spread(most, n):
    """n lengths in (0, most], the longest first: most itself, then spread over (most / 4, most]."""
    return [max(1, int(most * (1.0 - 0.75 * ((i * _GOLDEN) % 1.0)))) for i in range(n)]


def _nodes(case):
    """Valid nodes of each row: N for single tokens, else up to a quarter fewer."""
    B, N = case["B"], case["N"]
    return [max(1, N - (i * 5) % max(1, N // 4 + 1)) if B > 1 else N for i in range(B)]


def _trunks(case):
    """Bounds of the trunks' rows (uneven groups) and the positions that each of them shares, in whole pages."""
    B, T, page = case["B"], case["T"], case["page"]
    first = [0] + [(t * B) // T + (t % 2 if B >= 4 * T else 0) for t in range(1, T)] + [B]
    return first, [max(1, s // page) * page for s in _spread(case["shared"], T)]


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _shuffled(g, values):
    order = torch.randperm(len(values), generator=g, device="cuda")
    return torch.tensor(values, dtype=torch.int32, device="cuda")[order]


def _tree_masks(g, B, N):
    """Random trees, packed: bit j of a node's words says that it is node j or one of its descendants."""
    u = torch.rand(B, N, generator=g, device="cuda")
    i = torch.arange(N, device="cuda")
    parents = torch.where(i > 0, i - torch.minimum((u * i.clamp(max=6)).floor().long() + 1, i), torch.full_like(i, -1))
    see = torch.zeros(B, N, N, dtype=torch.bool, device="cuda")
    rows = torch.arange(B, device="cuda")
    for n in range(N):
        if n:
            see[:, n] = see[rows, parents[:, n]]
        see[:, n, n] = True
    W = (N + 63) // 64
    full = torch.zeros(B, N, W * 64, dtype=torch.int64, device="cuda")
    full[..., :N] = see.long()
    return (full.view(B, N, W, 64) << torch.arange(64, device="cuda")).sum(-1)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "fork_attn":
        B, T, N, Hq, Hk, D, page = (case[k] for k in ("B", "T", "N", "Hq", "Hk", "D", "page"))
        first, shared = _trunks(case)
        more = _shuffled(g, _spread(case["more"], B))
        group = torch.tensor([t for t in range(T) for _ in range(first[t], first[t + 1])], device="cuda")
        s["bounds"], s["first"] = (first, shared), torch.tensor(first, dtype=torch.int32, device="cuda")
        s["shared"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
        s["ctx"] = s["shared"][group] + more
        s["lengths"] = _shuffled(g, _nodes(case))
        # pages in a random order: the trunks' shared ones, then each row's own
        own_pages = [-(-(m + N) // page) for m in more.tolist()]
        P = sum(shared) // page + sum(own_pages) + 3
        M = max(shared) // page + max(own_pages)
        order = torch.randperm(P, generator=g, device="cuda").int()
        s["table"] = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        at = 0
        for t in range(T):
            n = shared[t] // page
            s["table"][first[t]:first[t + 1], :n] = order[at:at + n]
            at += n
            for b in range(first[t], first[t + 1]):
                s["table"][b, n:n + own_pages[b]] = order[at:at + own_pages[b]]
                at += own_pages[b]
        s["q"] = _randn(g, B, N, Hq, D, dtype=torch.bfloat16, scale=1.5)
        s["k_pages"] = _randn(g, P, page, Hk, D, dtype=torch.bfloat16)
        s["v_pages"] = _randn(g, P, page, Hk, D, dtype=torch.bfloat16)
        s["mask"] = _tree_masks(g, B, N) if case["tree"] else None
    elif op == "sample":
        R, V = case["R"], case["V"]
        wide = V + 17 if case["wide"] else V  # the head's rows are padded: the vocabulary is a slice of them
        logits = _randn(g, R, wide, scale=2.5)
        # a few likely tokens in each row, as a trained model's, and tokens that a grammar forbids
        logits += 9.0 * (torch.rand(R, wide, generator=g, device="cuda") < 12.0 / V)
        banned = torch.rand(R, wide, generator=g, device="cuda") < 0.02
        logits[banned] = -math.inf
        s["logits"] = logits.to(torch.float32 if case["f32"] else torch.bfloat16)[:, :V]
        u = torch.rand(R, 4, generator=g, device="cuda")
        row = torch.arange(R, device="cuda")
        s["temperature"] = torch.where(row % 16 == 15, 0.0, 0.4 + u[:, 0])  # some rows take the best token
        s["top_k"] = torch.where(row % 8 == 7, 0, (5 + 95 * u[:, 1]).int()).int() if case["top_k"] else None
        s["top_p"] = torch.where(row % 8 == 6, 1.0, 0.75 + 0.24 * u[:, 2]) if case["top_p"] else None
        s["min_p"] = torch.where(row % 8 == 5, 0.0, 0.1 * u[:, 3]) if case["min_p"] else None
        s["u"] = torch.rand(R, generator=g, device="cuda") if case["draws"] else None
    else:
        rows, C = case["rows"], case["C"]
        dtype = torch.float32 if case["f32"] else torch.bfloat16
        s["h"] = _randn(g, rows, C, dtype=dtype, scale=2.0)
        both = _randn(g, rows, 2 * C, dtype=dtype)  # a projection that gives the block's output and its gate
        s["y"], s["gate"] = both[:, :C], both[:, C:] if case["gate"] else None
        if not case["fused"]:
            s["y"], s["gate"] = s["y"].contiguous(), None if s["gate"] is None else s["gate"].contiguous()
        s["pre_w"] = 1.0 + _randn(g, C, scale=0.1)
        s["post_w"] = 1.0 + _randn(g, C, scale=0.1) if case["post"] else None
        s["scale"] = 0.5 + _randn(g, C, scale=0.05) if case["scale"] else None
        if op == "block_norm_grad":
            s["dh_out"] = _randn(g, rows, C)
            s["dn"] = _randn(g, rows, C, dtype=dtype)
    return s


# --------------------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------------------
def _plain_fork_attn(s):
    q, k_pages, v_pages, table, mask = (s[n] for n in ("q", "k_pages", "v_pages", "table", "mask"))
    B, N, Hq, D = q.shape
    page, Hk = k_pages.shape[1:3]
    G = Hq // Hk
    o, lse = torch.empty_like(q), torch.empty(B, N, Hq, device=q.device)
    i = torch.arange(N, device=q.device)
    first, shared = s["bounds"]
    for t, most in enumerate(shared):
        a, b = first[t], first[t + 1]
        if a == b:
            continue
        F, n_shared = b - a, most // page
        k0, v0 = (x[table[a, :n_shared].long()].reshape(most, Hk, D).float() for x in (k_pages, v_pages))
        rest = table[a:b, n_shared:].long().clamp(min=0)
        length = rest.shape[1] * page
        k1, v1 = (x[rest].reshape(F, length, Hk, D).float() for x in (k_pages, v_pages))
        x = q[a:b].float().view(F, N, Hk, G, D).permute(2, 0, 1, 3, 4).reshape(Hk, F, N * G, D)
        # scores over what is shared, one product for all rows, and over each row's own positions
        s0 = torch.matmul(x.reshape(Hk, F * N * G, D), k0.permute(1, 2, 0)).view(Hk, F, N * G, most)
        s1 = torch.matmul(x, k1.permute(2, 0, 3, 1))
        node = torch.arange(length, device=q.device) + most - s["ctx"][a:b, None]
        if mask is None:
            see = node[:, None, :] <= i[:, None]
        else:
            word = mask[a:b].gather(2, (node.clamp(0, N - 1) // 64)[:, None, :].expand(F, N, length))
            see = (node[:, None, :] < 0) | ((word >> (node.clamp(0, N - 1) % 64)[:, None, :]) & 1 > 0)
        live = i < s["lengths"][a:b, None]
        see = see & (node < s["lengths"][a:b, None])[:, None, :] & live[:, :, None]
        s1 = s1.masked_fill(~see.repeat_interleave(G, 1), -math.inf)
        z = torch.cat([s0, s1], -1).mul_(D ** -0.5)
        del s0, s1
        top = z.amax(-1, keepdim=True)
        e = z.sub_(top).exp_()
        total = e.sum(-1, keepdim=True)
        out = torch.matmul(e[..., :most].reshape(Hk, F * N * G, most), v0.permute(1, 0, 2)).view(Hk, F, N * G, D)
        out = (out + torch.matmul(e[..., most:], v1.permute(2, 0, 1, 3))) / total
        back = out.view(Hk, F, N, G, D).permute(1, 2, 0, 3, 4).reshape(F, N, Hq, D)
        o[a:b] = torch.where(live[..., None, None], back, 0.0).to(q.dtype)
        l = (top + torch.log(total)).view(Hk, F, N, G).permute(1, 2, 0, 3).reshape(F, N, Hq)
        lse[a:b] = torch.where(live[..., None], l, -math.inf)
    return o, lse


def _plain_sample(s):
    """Weights, sums and borders in 64 bits: they decide whole numbers."""
    x = s["logits"].double()
    R, V = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    best = s["temperature"] == 0
    t = torch.where(best, 1.0, s["temperature"].double())[:, None]
    down, order = torch.sort(x, dim=-1, descending=True, stable=True)
    w = torch.exp((down - down[:, :1].clamp(min=-1.7e308)) / t)
    rank = torch.arange(V, device=x.device)
    most = torch.full((R,), V, device=x.device) if s["top_k"] is None else torch.where(s["top_k"] == 0, V, s["top_k"])
    keep = rank < torch.where(best, 1, most)[:, None]
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        mass = (w * keep).cumsum(-1)
        keep &= (mass - w < p * mass[:, -1:]) | (p >= 1) | (rank == 0)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    w = torch.zeros_like(x).scatter_(1, order, w * keep)
    total = w.sum(-1, keepdim=True)
    out = []
    if s["u"] is not None:
        over = w.cumsum(-1) > s["u"].double()[:, None] * total
        last = torch.where(w > 0, rank, -1).amax(-1)
        out.append(torch.where(over.any(-1), over.int().argmax(-1), last).int())
    if s["case"]["probs"]:
        out.append((w / torch.where(total > 0, total, 1.0)).float())
    return out


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_block_norm(s):
    h, y = s["h"].float(), s["y"].float()
    z = y if s["post_w"] is None else s["post_w"] * y * _rms(y)
    if s["gate"] is not None:
        z = z * torch.sigmoid(s["gate"].float())
    if s["scale"] is not None:
        z = z * s["scale"]
    x = h + z
    return x.to(s["h"].dtype), (s["pre_w"] * x * _rms(x)).to(s["h"].dtype)


def _plain_block_norm_grad(s):
    h, y, dn = s["h"].float(), s["y"].float(), s["dn"].float()
    scale = 1.0 if s["scale"] is None else s["scale"]
    gate = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"].float())
    r = None if s["post_w"] is None else _rms(y)
    z = y if r is None else s["post_w"] * y * r
    x = h + scale * gate * z
    rx = _rms(x)
    wdn = s["pre_w"] * dn
    dx = s["dh_out"] + rx * (wdn - x * rx.square() * (wdn * x).mean(-1, keepdim=True))
    out = dict(dh=dx, dpre_w=(dn * x * rx).sum(0))
    dz = dx * scale * gate
    if s["scale"] is not None:
        out["dscale"] = (dx * gate * z).sum(0)
    if s["gate"] is not None:
        out["dgate"] = (dx * scale * z * gate * (1 - gate)).to(s["h"].dtype)
    if r is None:
        out["dy"] = dz.to(s["h"].dtype)
    else:
        out["dpost_w"] = (dz * y * r).sum(0)
        wdz = s["post_w"] * dz
        out["dy"] = (r * (wdz - y * r.square() * (wdz * y).mean(-1, keepdim=True))).to(s["h"].dtype)
    return out


def _own(s):
    from gated_deltanet_rule_gb300 import gdr
    op = s["case"]["op"]
    if op == "fork_attn":
        return gdr.gdr_fork_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx"], s["first"], s["shared"],
                                 s["lengths"], s["mask"], want_lse=True)
    if op == "sample":
        token, probs = gdr.gdr_sample(s["logits"], s["temperature"], s["u"], s["top_k"], s["top_p"], s["min_p"],
                                      want_probs=s["case"]["probs"])
        return [t for t in (token, probs) if t is not None]
    if op == "block_norm":
        return gdr.gdr_block_norm(s["h"], s["y"], s["pre_w"], s["post_w"], s["gate"], s["scale"], eps=EPS)
    dh, dy, dgate, dpre_w, dpost_w, dscale = gdr.gdr_block_norm_backward(
        s["h"], s["y"], s["pre_w"], s["post_w"], s["gate"], s["scale"], s["dn"], s["dh_out"], eps=EPS)
    out = dict(dh=dh, dpre_w=dpre_w, dscale=dscale, dgate=dgate, dpost_w=dpost_w, dy=dy)
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return {"fork_attn": _plain_fork_attn, "sample": _plain_sample, "block_norm": _plain_block_norm,
            "block_norm_grad": _plain_block_norm_grad}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "fork_attn":
        B, N, Hq, Hk, D = (case[k] for k in ("B", "N", "Hq", "Hk", "D"))
        first, shared = _trunks(case)
        n, more = sum(_nodes(case)) / B, sum(_spread(case["more"], B)) / B
        keys = sum(shared) + B * (more + n)
        pairs = sum(s * (b - a) for s, a, b in zip(shared, first, first[1:])) * n + B * n * (more + (n + 1) / 2)
        return dict(bytes=keys * Hk * D * 4 + 2 * B * n * Hq * D * 2 + B * N * Hq * 4, flops=4 * pairs * Hq * D)
    if op == "sample":
        n = case["R"] * case["V"]
        return dict(bytes=n * (4 if case["f32"] else 2) + (4 * n if case["probs"] else 0), flops=3 * n)
    n, size = case["rows"] * case["C"], 4 if case["f32"] else 2
    if op == "block_norm":
        return dict(bytes=n * size * (5 if case["gate"] else 4), flops=10 * n)
    return dict(bytes=n * (size * (6 if case["gate"] else 4) + 8), flops=30 * n)


# --------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------------
def _exact_fork_attn(s):
    """Row by row over the row's own table, as if nothing were shared."""
    q, table = s["q"].double(), s["table"].long()
    ctx, lengths = s["ctx"].tolist(), s["lengths"].tolist()
    B, N, Hq, D = q.shape
    page, Hk = s["k_pages"].shape[1:3]
    G = Hq // Hk
    o = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n, c = lengths[b], ctx[b]
        mine = table[b, :-(-(c + n) // page)]
        k = s["k_pages"][mine].reshape(-1, Hk, D)[:c + n].double().transpose(0, 1)
        v = s["v_pages"][mine].reshape(-1, Hk, D)[:c + n].double().transpose(0, 1)
        hide = torch.zeros(n, c + n, dtype=torch.bool, device=q.device)
        for j in range(n):
            if s["mask"] is None:
                hide[:j, c + j] = True
            else:
                hide[:, c + j] = (s["mask"][b, :n, j // 64] >> (j % 64)) % 2 == 0
        x = q[b, :n].view(n, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * n, D)
        a = torch.bmm(x, k.transpose(1, 2)) / math.sqrt(D)
        a.view(Hk, G, n, c + n).masked_fill_(hide, -math.inf)
        lse[b, :n] = torch.logsumexp(a, -1).view(Hq, n).T
        o[b, :n] = torch.bmm(torch.softmax(a, -1), v).view(Hq, n, D).transpose(0, 1)
    return o, lse


def _exact_sample(s):
    """Row by row: the tokens in order of their logits, and those that the filters leave one after the other."""
    R, V = s["logits"].shape
    tokens, rows = [], []
    for r in range(R):
        x = s["logits"][r].double()
        t = float(s["temperature"][r])
        x = torch.nan_to_num(x, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
        order = torch.argsort(-x, stable=True)
        k = int(s["top_k"][r]) if s["top_k"] is not None else 0
        order = order[:1] if t == 0 else order[:k] if k else order
        w = torch.exp((x[order] - x[order[0]]) / (t or 1.0))
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            part = torch.cat([w.new_zeros(1), torch.cumsum(w, 0)[:-1]]) / w.sum()
            n = max(1, int((part < float(s["top_p"][r])).sum()))
            order, w = order[:n], w[:n]
        if s["min_p"] is not None:
            n = int((w >= float(s["min_p"][r])).sum())
            order, w = order[:n], w[:n]
        p = torch.zeros(V, dtype=torch.float64, device=x.device)
        p[order] = w / w.sum()
        rows.append(p)
        if s["u"] is not None:
            at, turn = torch.sort(order)
            run_ = torch.cumsum(w[turn], 0)
            passed = torch.nonzero(run_ > float(s["u"][r]) * float(run_[-1]))
            tokens.append(int(at[passed[0, 0]]) if len(passed) else int(at[-1]))
    out = [torch.tensor(tokens, dtype=torch.int32, device="cuda")] if s["u"] is not None else []
    return out + ([torch.stack(rows)] if s["case"]["probs"] else [])


def _exact_block_norm(h, y, gate, post_w, scale, pre_w):
    def norm(x, w):
        return w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    z = norm(y, post_w) if post_w is not None else y
    if gate is not None:
        z = z / (1 + torch.exp(-gate))
    x = h + (z * scale if scale is not None else z)
    return x, norm(x, pre_w)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "fork_attn":
        return _exact_fork_attn(s)
    if op == "sample":
        return _exact_sample(s)
    names = ("h", "y", "gate", "post_w", "scale", "pre_w")
    a = {n: None if s[n] is None else s[n].double() for n in names}
    if op == "block_norm":
        return _exact_block_norm(**a)
    # by the chain rule through automatic differentiation of the definition
    there = [n for n in names if a[n] is not None]
    a = {n: None if a[n] is None else a[n].detach().clone().requires_grad_(True) for n in names}
    x, n_out = _exact_block_norm(**a)
    got = torch.autograd.grad((x, n_out), [a[n] for n in there], (s["dh_out"].double(), s["dn"].double()))
    return {"d" + n: d for n, d in zip(there, got)}
