"""The example of sampled forks: its caches, states and logits against a plain float64 pass over the tokens it drew, and
its tokens against the distributions of its own logits."""
import importlib.util
import math
import os

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr
from tests import fork_ref as ref

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "sampled_forks", os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples", "sampled_forks.py"))
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)


def _delta(q, k, v, g, beta):
    """The gated delta rule over [L, heads, D] in float64, one token at a time: (o, S)."""
    r = v.shape[1] // k.shape[1]
    k = (k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(r, 1)
    q = (q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(r, 1) * ex.D ** -0.5
    S, out = torch.zeros(v.shape[1], ex.D, ex.D, dtype=torch.float64), []
    for t in range(len(q)):
        S = S * g[t].exp()[:, None, None]
        S = S + k[t][:, :, None] * (beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1)))[:, None]
        out.append((q[t][:, :, None] * S).sum(1))
    return torch.stack(out), S


def _plain(m, tokens):
    """The model over tokens in float64 on the CPU: (keys and values of the attention layers, states of the delta layers,
    logits)."""
    f = lambda t: t.double().cpu()  # noqa: E731
    x, L = f(m.embed)[tokens], len(tokens)
    ang = torch.arange(L, dtype=torch.float64)[:, None] * f(m.inv_freq)
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    norm = lambda y, w: y / torch.sqrt((y * y).mean(-1, keepdim=True) + ex.EPS) * f(w)  # noqa: E731

    def rope(y, w):
        a, b, rest = norm(y, w).split([32, 32, 64], -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    caches, states = [], []
    for layer, kind in enumerate(ex.LAYERS):
        h = norm(x, m.pre_w[layer])
        y = (h @ f(m.proj[layer])).unflatten(-1, (-1, ex.D))
        if kind == ex.DELTA:
            q, k, v = y.split([2, 2, 4], 1)
            a, b = (h @ f(m.gates[layer])).split(4, -1)
            o, S = _delta(q, k, v, -torch.nn.functional.softplus(a), torch.sigmoid(b))
            states.append(S)
        else:
            q, k, v = y.split([ex.ATTN_Q, ex.ATTN_K, ex.ATTN_K], 1)
            q, k = rope(q, m.q_w), rope(k, m.k_w)
            caches.append((k, v))
            r = ex.ATTN_Q // ex.ATTN_K
            s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(r, 1)) / math.sqrt(ex.D)
            s = s.masked_fill(torch.ones(L, L).triu(1).bool(), -math.inf)
            o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v.repeat_interleave(r, 1))
        z = norm(o.flatten(1) @ f(m.out[layer]), m.post_w[layer])
        x = x + f(m.scale[layer]) * torch.sigmoid(h @ f(m.gate_w[layer])) * z
    return caches, states, norm(x, m.pre_w[-1]) @ f(m.head)


# Each of the four layers rounds to bf16 its input, its projection, the operator's operands and output, the output product
# and the gate, and its result adds to the residual of those before: at most 4 layers of 7 roundings, each relative 2^-8
# of a vector's norm; the head rounds its input and its product.
TOL = 30 * 2.0 ** -8


def test_caches_states_and_logits_follow_the_drawn_tokens():
    prompt = torch.randint(0, ex.VOCAB, (70,), generator=torch.Generator().manual_seed(3)).tolist()
    s, out, steps = ex.generate(prompt, samples=20, steps=5, seed=5)
    assert len({tuple(t) for t in out}) > 10
    assert s.ctx.tolist() == [len(t) - 1 for t in out]
    full = len(prompt[:-1]) // ex.PAGE
    assert (s.table[:, :full] == s.table[0, :full]).all() and (s.refs[s.table[0, :full].long()] == 20).all()
    for b in (0, 7, 19):
        tokens = out[b]
        caches, states, logits = _plain(s.model, tokens[:-1])
        n = len(tokens) - 1
        slots = s.table[b, :-(-n // ex.PAGE)].long()
        for at, (k, v) in enumerate(caches):
            for got, want in ((s.k_cache, k), (s.v_cache, v)):
                got = got[at, slots].flatten(0, 1)[:n].double().cpu()
                assert (got - want).norm() <= TOL * want.norm()
        for at, S in enumerate(states):
            assert (s.states[at, b].double().cpu() - S).norm() <= TOL * S.norm()
        for i, (_, _, got, _) in enumerate(steps):
            want = logits[len(prompt) - 1 + i]
            assert (got[b].double().cpu() - want).norm() <= TOL * want.norm()
    s.close()
    gdr.gdr_sync_status()
    assert not s.refs.any() and (s.table == -1).all() and not s.ctx.any()


def test_tokens_are_drawn_from_the_logits():
    prompt = torch.randint(0, ex.VOCAB, (40,), generator=torch.Generator().manual_seed(4)).tolist()
    _, _, steps = ex.generate(prompt, samples=40, steps=3, seed=6)
    for kw, u, logits, tokens in steps:
        x, kw = logits.double().cpu().numpy(), {k: v.tolist() for k, v in kw.items()}
        for b in range(len(tokens)):
            args = kw["temperature"][b], kw["top_k"][b], kw["top_p"][b], kw["min_p"][b]
            off = 2.0 ** -35
            may = set()
            for o in (0.0, -off, off):   # (a border of top_p may fall to either side)
                w = ref.weights(x[b], args[0]) * ref.kept(x[b], *args, off=o)
                may |= ref.drawn(w, float(u[b]), off * w.sum())
            assert int(tokens[b]) in may
