"""Speculative decoding with trees on a hybrid of gated delta rule and softmax-attention layers.

A model with random weights generates several samples of one prompt:

  prefill    gdr_chunk_fwd for the delta layers; gdr_cache_reserve, gdr_qk_norm_rope_append and
             gdr_tree_attn (no mask: a chain) for the attention layers
  samples    the prompt's row is forked: gdr_cache_fork shares its full pages, the delta states are copied
  one step   a tree of drafted tokens a sample; the delta layers run its root-to-leaf paths as forks of
             the sample's state (gdr_fork_fwd), the attention layers the whole tree at once over the
             pages; gdr_verify_draft accepts a path; gdr_cache_compact moves its entries to the front and
             gdr_chunk_fwd with lengths takes the delta states along it
  at the end gdr_cache_free

Projections, MLPs and the head are plain matrix products. Run: python examples/speculative_step.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_rule_gb300 import gdr  # noqa: E402

PARENTS = [-1, 0, 0, 1, 1, 2, 3, 5]                      # every node after its parent; node 0 the last token
PATHS = [[0, 1, 3, 6], [0, 1, 4], [0, 2, 5, 7]]          # root to leaf
HID, VOCAB, D = 256, 512, 128
DELTA_K, DELTA_V, ATTN_Q, ATTN_K = 2, 4, 8, 2            # heads
PAGE, EPS = 16, 1e-6
DELTA, ATTN = 0, 1
LAYERS = [DELTA, ATTN, DELTA, ATTN]


class Model:
    """Random weights. Each layer adds its mixer's output to the residual; bf16 in, float32 residual."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(rows, cols, scale=1.0):
            return (scale / math.sqrt(rows) * torch.randn(rows, cols, generator=g)).to(device, torch.bfloat16)

        self.device = device
        self.embed, self.head = w(VOCAB, HID, math.sqrt(VOCAB)), w(HID, VOCAB, 2.0)
        self.bigram = 2 * torch.randn(VOCAB, VOCAB, generator=g).to(device)   # the draft: next token from this one
        self.proj, self.out, self.gates = [], [], []
        for kind in LAYERS:
            heads = 2 * DELTA_K + DELTA_V if kind == DELTA else ATTN_Q + 2 * ATTN_K
            self.proj.append(w(HID, heads * D))
            self.out.append(w((DELTA_V if kind == DELTA else ATTN_Q) * D, HID))
            self.gates.append(w(HID, 2 * DELTA_V) if kind == DELTA else None)
        self.q_w = 1 + 0.1 * torch.randn(D, generator=g).to(device)
        self.k_w = 1 + 0.1 * torch.randn(D, generator=g).to(device)
        self.inv_freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).to(device)   # 64 of 128 turn

    def normed(self, x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)).to(torch.bfloat16)

    def delta_inputs(self, layer, h, live):
        """q, k, v and the gates [rows, L, ...] of a delta layer; positions that are not live are pads."""
        q, k, v = (h @ self.proj[layer]).unflatten(-1, (-1, D)).split([DELTA_K, DELTA_K, DELTA_V], 2)
        a, b = (h @ self.gates[layer]).float().split(DELTA_V, -1)
        g = torch.where(live[..., None], -torch.nn.functional.softplus(a), 0.0)
        beta = torch.where(live[..., None], torch.sigmoid(b), 0.0)
        return q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), beta.contiguous()

    def logits(self, x):
        return (self.normed(x) @ self.head).float()


class Session:
    """The samples of one prompt: their pages, delta states and last tokens."""

    def __init__(self, model, samples, most=512, pages=256):
        m, dev = model, model.device
        self.model, self.samples = m, samples
        attn, delta = LAYERS.count(ATTN), LAYERS.count(DELTA)
        self.k_cache = torch.zeros(attn, pages, PAGE, ATTN_K, D, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.full((samples, most // PAGE), -1, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(samples, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.states = torch.zeros(delta, samples, DELTA_V, D, D, device=dev)
        self.last = torch.zeros(samples, dtype=torch.int32, device=dev)
        self.rows = torch.arange(samples, dtype=torch.int32, device=dev)

        N = len(PARENTS)
        see = torch.eye(N, dtype=torch.bool)
        for i, p in enumerate(PARENTS):
            if p >= 0:
                see[i] |= see[p]
        self.depth = (see.sum(1) - 1).to(dev, torch.int32)
        self.mask = (see.long() << torch.arange(N)).sum(1)[None, :, None].to(dev).expand(samples, N, 1).contiguous()
        self.parents = torch.tensor(PARENTS, dtype=torch.int32, device=dev).expand(samples, N).contiguous()
        # the paths as forks: node of every (path, step), which (path, step) gives a node, pads beyond a leaf
        F, L = len(PATHS), max(map(len, PATHS))
        self.path_node = torch.tensor([p + [p[-1]] * (L - len(p)) for p in PATHS], device=dev)
        self.path_live = torch.tensor([[i < len(p) for i in range(L)] for p in PATHS], device=dev)
        first = {n: (f, i) for f, p in reversed(list(enumerate(PATHS))) for i, n in enumerate(p)}
        self.node_at = torch.tensor([first[n][0] * L + first[n][1] for n in range(N)], device=dev)
        self.fork_of = torch.arange(samples, device=dev).repeat_interleave(F)

    def attend(self, layer, at, h, pos, rows, lengths=None, mask=None):
        """An attention layer: h's keys and values into the pages, and the nodes' attention over them."""
        m, table, ctx = self.model, self.table[rows].contiguous(), self.ctx[rows].contiguous()
        q, k, v = (h @ m.proj[layer]).unflatten(-1, (-1, D)).split([ATTN_Q, ATTN_K, ATTN_K], 2)
        kp, vp = self.k_cache[at], self.v_cache[at]
        q = gdr.gdr_qk_norm_rope_append(q, k, v, m.q_w, m.k_w, m.inv_freq, pos, kp, vp, table, ctx, lengths, EPS)
        return gdr.gdr_tree_attn(q, kp, vp, table, ctx, lengths, mask)

    def prefill(self, prompt):
        """prompt: a list of tokens. All but the last are committed; the samples share their pages."""
        m, dev = self.model, self.model.device
        tokens = torch.tensor(prompt[:-1], device=dev)[None]
        n = tokens.shape[1]
        gdr.gdr_cache_reserve(self.table, self.ctx, self.refs, self.rows[:1], n, PAGE)
        x, live = m.embed[tokens].float(), torch.ones(1, n, dtype=torch.bool, device=dev)
        pos = torch.arange(n, dtype=torch.int32, device=dev)[None]
        seen = [0, 0]
        for layer, kind in enumerate(LAYERS):
            h, at = m.normed(x), seen[kind]
            if kind == DELTA:
                o, S = gdr.gdr_chunk_fwd(*m.delta_inputs(layer, h, live))
                self.states[at] = S       # every sample starts from it
            else:
                o = self.attend(layer, at, h, pos, slice(0, 1))
            x = x + (o.flatten(2) @ m.out[layer]).float()
            seen[kind] += 1
        self.ctx[0] = n
        gdr.gdr_cache_fork(self.k_cache, self.v_cache, self.table, self.ctx, self.refs,
                           torch.zeros_like(self.rows[1:]), self.rows[1:])
        self.last.fill_(prompt[-1])

    def step(self, gen):
        """One speculative step of every sample: (accepted nodes' tokens [B, N], their number [B])."""
        m, B, N = self.model, self.samples, len(PARENTS)
        tokens = self.last[:, None].repeat(1, N)
        q = torch.empty(B, N, VOCAB, device=m.device)
        for i, p in enumerate(PARENTS):   # children drawn from the draft's distribution at their parent
            if p >= 0:
                tokens[:, i] = torch.multinomial(q[:, p], 1, generator=gen)[:, 0].int()
            q[:, i] = torch.softmax(m.bigram[tokens[:, i].long()], -1)

        gdr.gdr_cache_reserve(self.table, self.ctx, self.refs, self.rows, N, PAGE)
        x, pos = m.embed[tokens.long()].float(), self.ctx[:, None] + self.depth
        kept, seen = [], [0, 0]
        for layer, kind in enumerate(LAYERS):
            h, at = m.normed(x), seen[kind]
            if kind == DELTA:
                paths = h[:, self.path_node].flatten(0, 1)                       # [B F, L, HID]
                o, _ = gdr.gdr_fork_fwd(*m.delta_inputs(layer, paths, self.path_live.repeat(B, 1)), self.states[at],
                                        self.fork_of, keep=False)
                o = o.view(B, -1, DELTA_V, D)[:, self.node_at]
                kept.append((layer, h))
            else:
                o = self.attend(layer, at, h, pos, slice(None), mask=self.mask)
            x = x + (o.flatten(2) @ m.out[layer]).float()
            seen[kind] += 1

        p = torch.softmax(m.logits(x), -1)
        u, u_next = torch.rand(B, N, device=m.device, generator=gen), torch.rand(B, device=m.device, generator=gen)
        lengths = torch.full_like(self.ctx, N)
        path, n_path, nxt = gdr.gdr_verify_draft(tokens, self.parents, lengths, p, q, u, u_next)

        at = path.clamp(min=0).long()
        live = torch.arange(N, device=m.device) < n_path[:, None]
        for d, (layer, h) in enumerate(kept):
            h = h.gather(1, at[..., None].expand(-1, -1, HID))
            _, self.states[d] = gdr.gdr_chunk_fwd(*m.delta_inputs(layer, h, live), self.states[d], lengths=n_path)
        self.ctx = gdr.gdr_cache_compact(self.k_cache, self.v_cache, self.table, self.ctx, path, n_path)
        self.last = nxt
        return tokens.gather(1, at), n_path

    def close(self):
        gdr.gdr_cache_free(self.table, self.ctx, self.refs, self.rows)


def generate(prompt, samples=3, steps=8, seed=0):
    """(session, the samples' tokens with the prompt): the last token of each is not in the caches yet."""
    session = Session(Model(seed), samples)
    session.prefill(prompt)
    gen = torch.Generator("cuda").manual_seed(seed)
    out = [list(prompt[:-1]) for _ in range(samples)]
    for _ in range(steps):
        tokens, n = session.step(gen)
        gdr.gdr_sync_status()
        for b in range(samples):
            out[b] += tokens[b, :n[b]].tolist()
    for b in range(samples):
        out[b].append(int(session.last[b]))
    return session, out


def main():
    prompt = torch.randint(0, VOCAB, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    session, out = generate(prompt)
    for b, tokens in enumerate(out):
        print(f"sample {b}: {len(tokens) - len(prompt)} tokens in 8 steps: {tokens[len(prompt):]}")
    used = int((session.refs > 0).sum())
    session.close()
    gdr.gdr_sync_status()
    print(f"{used} pages in use before the end, {int((session.refs > 0).sum())} after")


if __name__ == "__main__":
    main()
