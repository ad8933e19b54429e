"""Many samples of one prompt on a hybrid of gated delta rule and softmax-attention layers, token by token.

  prefill    the prompt's row: gdr_chunk_fwd for the delta layers; gdr_cache_reserve, gdr_qk_norm_rope_append and
             gdr_tree_attn (a chain) for the attention layers
  samples    forks of that row: gdr_cache_fork shares its full pages, the delta states are copied
  one step   every sample's last token: gdr_decode_step in the delta layers; in the attention layers
             gdr_qk_norm_rope_append and gdr_fork_attn, which reads the prompt's pages once for all samples;
             gdr_block_norm between the blocks (norm, gate, residual scale, sum, norm); gdr_sample draws the next
             tokens from given uniform numbers
  at the end gdr_cache_free

Projections, gates and the head are plain matrix products. Run: python examples/sampled_forks.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from speculative_step import (ATTN, ATTN_K, ATTN_Q, D, DELTA, EPS, HID, LAYERS, PAGE, VOCAB, Model, gdr)  # noqa: E402


class Hybrid(Model):
    """The speculative example's mixers with a norm before and after each, a gate and a residual scale."""

    def __init__(self, seed=0, device="cuda"):
        super().__init__(seed, device)
        g = torch.Generator().manual_seed(seed + 1)
        near = lambda mean: (mean + 0.1 * torch.randn(HID, generator=g)).to(device)   # noqa: E731
        self.pre_w = [near(1.0) for _ in range(len(LAYERS) + 1)]   # (the last one: before the head)
        self.post_w, self.scale = [near(1.0) for _ in LAYERS], [near(0.7) for _ in LAYERS]
        self.gate_w = [(torch.randn(HID, HID, generator=g) / math.sqrt(HID)).to(device, torch.bfloat16) for _ in LAYERS]

    def run(self, tokens, mixer):
        """The bfloat16 logits [B, L, VOCAB] after tokens [B, L]; mixer(layer, kind, number of its kind, its input) -> [B, L, heads, D]."""
        x = self.embed[tokens.long()].float()
        x, n = gdr.gdr_block_norm(x, torch.zeros_like(x), self.pre_w[0], eps=EPS)
        seen = [0, 0]
        for layer, kind in enumerate(LAYERS):
            h = n.to(torch.bfloat16)
            y = (mixer(layer, kind, seen[kind], h).flatten(2) @ self.out[layer]).float()
            gate = (h @ self.gate_w[layer]).float()
            x, n = gdr.gdr_block_norm(x, y, self.pre_w[layer + 1], self.post_w[layer], gate, self.scale[layer], EPS, h_out=x)
            seen[kind] += 1
        return n.to(torch.bfloat16) @ self.head


class Samples:
    """A prompt's samples: their pages, delta states and last tokens."""

    def __init__(self, model, samples, most=512, pages=512):
        dev = model.device
        self.model, self.samples = model, samples
        attn, delta = LAYERS.count(ATTN), LAYERS.count(DELTA)
        self.k_cache = torch.zeros(attn, pages, PAGE, ATTN_K, D, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.table = torch.full((samples, most // PAGE), -1, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(samples, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=dev)
        self.states = torch.zeros(delta, samples, 4, D, D, device=dev)
        self.last = torch.zeros(samples, dtype=torch.int32, device=dev)
        self.rows = torch.arange(samples, dtype=torch.int32, device=dev)

    def keys(self, layer, at, h, pos, rows):
        """q, with the keys and values of h in the pages."""
        m, table, ctx = self.model, self.table[rows].contiguous(), self.ctx[rows].contiguous()
        q, k, v = (h @ m.proj[layer]).unflatten(-1, (-1, D)).split([ATTN_Q, ATTN_K, ATTN_K], 2)
        return gdr.gdr_qk_norm_rope_append(q, k, v, m.q_w, m.k_w, m.inv_freq, pos, self.k_cache[at], self.v_cache[at], table, ctx,
                                           eps=EPS), table, ctx

    def prefill(self, prompt):
        """prompt: a list of tokens. All but the last are committed; the samples share their full pages."""
        m, dev = self.model, self.model.device
        tokens = torch.tensor(prompt[:-1], device=dev)[None]
        n = tokens.shape[1]
        gdr.gdr_cache_reserve(self.table, self.ctx, self.refs, self.rows[:1], n, PAGE)
        pos, live = torch.arange(n, dtype=torch.int32, device=dev)[None], torch.ones(1, n, dtype=torch.bool, device=dev)

        def mixer(layer, kind, at, h):
            if kind == DELTA:
                o, S = gdr.gdr_chunk_fwd(*m.delta_inputs(layer, h, live))
                self.states[at] = S       # every sample starts from it
                return o
            q, table, ctx = self.keys(layer, at, h, pos, slice(0, 1))
            return gdr.gdr_tree_attn(q, self.k_cache[at], self.v_cache[at], table, ctx)

        m.run(tokens, mixer)
        self.ctx[0] = n
        gdr.gdr_cache_fork(self.k_cache, self.v_cache, self.table, self.ctx, self.refs, torch.zeros_like(self.rows[1:]), self.rows[1:])
        self.last.fill_(prompt[-1])
        # one group of rows, which share the prompt's full pages
        self.first = torch.tensor([0, self.samples], dtype=torch.int32, device=dev)
        self.shared = torch.tensor([n // PAGE * PAGE], dtype=torch.int32, device=dev)

    def step(self, temperature, u, top_k=None, top_p=None, min_p=None):
        """The samples' next tokens [B] from the uniform numbers u [B]; the logits that they were drawn from."""
        m = self.model
        gdr.gdr_cache_reserve(self.table, self.ctx, self.refs, self.rows, 1, PAGE)
        live = torch.ones(self.samples, 1, dtype=torch.bool, device=m.device)

        def mixer(layer, kind, at, h):
            if kind == DELTA:
                return gdr.gdr_decode_step(*m.delta_inputs(layer, h, live), self.states[at])
            q, table, ctx = self.keys(layer, at, h, self.ctx[:, None].contiguous(), slice(None))
            return gdr.gdr_fork_attn(q, self.k_cache[at], self.v_cache[at], table, ctx, self.first, self.shared)

        logits = m.run(self.last[:, None], mixer)[:, 0]
        self.last, _ = gdr.gdr_sample(logits, temperature, u, top_k, top_p, min_p)
        self.ctx += 1
        return self.last, logits

    def close(self):
        gdr.gdr_cache_free(self.table, self.ctx, self.refs, self.rows)


def generate(prompt, samples=24, steps=12, seed=0):
    """(the samples, their tokens with the prompt, and for each step its parameters, numbers and logits)"""
    s = Samples(Hybrid(seed), samples)
    s.prefill(prompt)
    gen = torch.Generator("cuda").manual_seed(seed)
    full = lambda x, dtype=torch.float32: torch.full((samples,), x, dtype=dtype, device="cuda")   # noqa: E731
    kw = dict(temperature=full(0.9), top_k=full(40, torch.int32), top_p=full(0.95), min_p=full(0.01))
    out, steps_made = [list(prompt) for _ in range(samples)], []
    for _ in range(steps):
        u = torch.rand(samples, device="cuda", generator=gen)
        tokens, logits = s.step(u=u, **kw)
        gdr.gdr_sync_status()
        steps_made.append((kw, u, logits, tokens))
        for b, t in enumerate(tokens.tolist()):
            out[b].append(t)
    return s, out, steps_made


def main():
    prompt = torch.randint(0, VOCAB, (100,), generator=torch.Generator().manual_seed(1)).tolist()
    s, out, _ = generate(prompt)
    for b, tokens in enumerate(out[:4]):
        print(f"sample {b}: {tokens[len(prompt):]}")
    used = int((s.refs > 0).sum())
    s.close()
    gdr.gdr_sync_status()
    print(f"{len({tuple(t) for t in out})} different samples, {used} pages in use before the end, {int((s.refs > 0).sum())} after")


if __name__ == "__main__":
    main()
