"""The speculative example: its caches and states against a plain float64 pass over the tokens it kept."""
import importlib.util
import math
import os

import pytest
import torch

from gated_deltanet_rule_gb300 import gdr

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "speculative_step", os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples", "speculative_step.py"))
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
    """The model over committed tokens in float64 on the CPU: (keys and values of the attention layers,
    states of the delta layers)."""
    f = lambda t: t.double().cpu()  # noqa: E731
    x, L = f(m.embed)[tokens], len(tokens)
    ang = torch.arange(L, dtype=torch.float64)[:, None] * f(m.inv_freq)
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]

    def rope(y, w):
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + ex.EPS) * f(w)
        a, b, rest = y.split([32, 32, 64], -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)

    caches, states = [], []
    for layer, kind in enumerate(ex.LAYERS):
        h = x / torch.sqrt((x * x).mean(-1, keepdim=True) + ex.EPS)
        y = (h @ f(m.proj[layer])).unflatten(-1, (-1, ex.D))
        if kind == ex.DELTA:
            q, k, v = y.split([ex.DELTA_K, ex.DELTA_K, ex.DELTA_V], 1)
            a, b = (h @ f(m.gates[layer])).split(ex.DELTA_V, -1)
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
        x = x + o.flatten(1) @ f(m.out[layer])
    return caches, states


# Each of the four layers rounds to bf16 its input, its projection, the operator's operands and output and
# the output product, and its result adds to the residual of those before: at most 4 layers of 6 roundings,
# each relative 2^-8 of a vector's norm.
TOL = 24 * 2.0 ** -8


def test_caches_and_states_hold_the_accepted_tokens():
    prompt = torch.randint(0, ex.VOCAB, (70,), generator=torch.Generator().manual_seed(3)).tolist()
    session, out = ex.generate(prompt, samples=3, steps=6, seed=5)
    assert len({tuple(t) for t in out}) > 1 and any(len(t) > len(prompt) + 6 for t in out)   # drafts were taken
    assert session.ctx.tolist() == [len(t) - 1 for t in out]
    shared = session.table[:, :len(prompt[:-1]) // ex.PAGE]
    assert (shared == shared[0]).all()                                                     # the prompt's full pages
    for b, tokens in enumerate(out):
        assert tokens[:70] == prompt
        caches, states = _plain(session.model, tokens[:-1])
        n = len(tokens) - 1
        slots = session.table[b, :-(-n // ex.PAGE)].long()
        for at, (k, v) in enumerate(caches):
            for got, want in ((session.k_cache, k), (session.v_cache, v)):
                got = got[at, slots].flatten(0, 1)[:n].double().cpu()
                assert (got - want).norm() <= TOL * want.norm()
                assert ((got - want).flatten(1).norm(dim=1) <= 2 * TOL * want.flatten(1).norm(dim=1)).all()
        for at, S in enumerate(states):
            got = session.states[at, b].double().cpu()
            assert (got - S).norm() <= TOL * S.norm()
    session.close()
    gdr.gdr_sync_status()
    assert not session.refs.any() and (session.table == -1).all() and not session.ctx.any()
