"""Speculative decoding of a small hybrid stack (random weights, synthetic prompts).

One recurrent mixer layer and one full-attention layer over a paged 8-bit cache,
run as a serving loop runs them: the prompts in one packed pass (prefill,
kv_append, kv_attention), then steps in which T drafted tokens of every sequence
are verified at once (decode with kept intermediate states, kv_append,
kv_attention, accept_drafts) and the accepted ones stay (decode_commit; the
cache's lengths move back over the others, whose rows the next step overwrites).
The drafts come from the stack without its two layers.

    python examples/speculative_hybrid.py [--sequences N] [--steps S] [--drafts T]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_mixer_gb300 as gdn  # noqa: E402


def _cu(counts):
    """Prefix sums of per-sequence token counts, on the device and on the host."""
    host = torch.tensor([0, *counts], dtype=torch.int32).cumsum(0, dtype=torch.int32)
    return host.cuda(), host


def _norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


class Stack:
    """Embedding, mixer layer, attention layer, output projection: bf16, random weights."""

    def __init__(self, vocab=1000, hidden=256, max_len=4096, cache="int8", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols, gain=1.0):
            return (torch.randn(rows, cols, generator=g, device="cuda") * (gain / rows ** 0.5)).bfloat16()

        self.vocab, self.hidden = vocab, hidden
        self.mix = gdn.Dims(2, 4, 128, 128, 4, torch.bfloat16)
        self.att = gdn.KVDims(8, 2, 128, page_size=32, cache=cache, rope_dim=64)
        d, a = self.mix, self.att
        self.params = gdn.Params(torch.randn(d.conv_dim, d.conv_k, generator=g, device="cuda") * 0.5,
                                 torch.zeros(d.n_v_heads, device="cuda"),
                                 torch.full((d.gate_width,), -2.0, device="cuda"),
                                 torch.ones(d.d_v, device="cuda"))
        vd = d.n_v_heads * d.d_v
        self.mix_in = [weight(hidden, n) for n in (d.conv_dim, vd, d.gate_width, d.n_v_heads)]
        self.mix_out = weight(vd, hidden, 0.5)
        self.qkv = weight(hidden, (a.n_q_heads + 2 * a.n_kv_heads) * a.head_dim)
        self.att_out = weight(a.n_q_heads * a.head_dim, hidden)
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda").bfloat16()
        self.head = weight(hidden, vocab, 2.0)
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, a.rope_dim, 2, device="cuda") / a.rope_dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).contiguous()

    def mixer_inputs(self, h):
        x = _norm(h)
        return [x @ w for w in self.mix_in]

    def attention(self, h, cache, cu, kv_lens, block_table):
        """h [T, hidden] plus the attention layer's output; the tokens' keys and values are cached."""
        a = self.att
        heads = (_norm(h) @ self.qkv).view(h.shape[0], -1, a.head_dim)
        q, k, v = heads.split([a.n_q_heads, a.n_kv_heads, a.n_kv_heads], 1)  # views: strides are free
        q = gdn.kv_append(a, cache, cu, kv_lens, block_table, k, v, q=q, rope=self.rope)
        o = gdn.kv_attention(a, cache, cu, kv_lens, block_table, q)
        return h + o.view(h.shape[0], -1) @ self.att_out

    def logits(self, h):
        return _norm(h) @ self.head


class Session:
    """Sequences being decoded: recurrent state and conv history, pages, lengths, last tokens."""

    def __init__(self, stack: Stack, prompts, room: int, temperature=1.0, seed=1):
        s, n = stack, len(prompts)
        self.stack, self.n = s, n
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.temperature = torch.full((n,), float(temperature), device="cuda")
        lengths = [len(p) for p in prompts]
        pages = -(-(max(lengths) + room) // s.att.page_size)
        self.cache = gdn.KVCache.empty(s.att, n * pages)
        self.block_table = torch.randperm(n * pages, generator=self.g, device="cuda").view(n, pages).int()
        d = s.mix
        self.state = torch.empty(n, d.n_v_heads, d.d_k, d.d_v, device="cuda")
        self.conv_state = torch.empty(n, d.conv_dim, d.conv_k - 1, dtype=d.dtype, device="cuda")
        self.kv_lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")

        cu = _cu(lengths)
        h = s.embedding[torch.cat([torch.as_tensor(p) for p in prompts]).cuda()]
        h = h + gdn.prefill(d, s.params, cu, *s.mixer_inputs(h), final_state=self.state,
                            conv_state_out=self.conv_state) @ s.mix_out
        h = s.attention(h, self.cache, cu, self.kv_lens, self.block_table)
        last = s.logits(h[cu[0][1:].long() - 1]).view(n, 1, -1)
        none = torch.empty(n, 0, dtype=torch.int32, device="cuda")
        _, tokens = gdn.accept_drafts(none, last, None, none.float(), self.noise(), form="logits",
                                      temperature=self.temperature)
        self.last = tokens[:, 0].long()

    def noise(self):
        return torch.empty(self.n, self.stack.vocab, device="cuda").exponential_(generator=self.g)

    def draft(self, count: int):
        """count tokens after the last one, each drawn from the logits that its row holds."""
        x = self.last
        tokens = torch.empty(self.n, count, dtype=torch.int32, device="cuda")
        rows = torch.empty(self.n, count, self.stack.vocab, dtype=torch.bfloat16, device="cuda")
        greedy = (self.temperature == 0)[:, None]
        for i in range(count):
            rows[:, i] = self.stack.logits(self.stack.embedding[x])
            row = rows[:, i].float()
            p = torch.softmax(row / torch.where(greedy, 1.0, self.temperature[:, None]), -1)
            x = torch.where(greedy, row, p / self.noise()).argmax(-1)
            tokens[:, i] = x
        return tokens, rows

    def step(self, drafts: int):
        """One speculative step.  Returns accepted [n] and tokens [n, drafts + 1] (-1 after the last)."""
        s, n, t = self.stack, self.n, drafts + 1
        guess, guess_logits = self.draft(drafts)
        h = s.embedding[torch.cat([self.last[:, None], guess.long()], 1)].view(n * t, -1)
        inputs = [i.view(n, t, -1) for i in s.mixer_inputs(h)]
        d = s.mix
        inter = torch.empty(n, t, d.n_v_heads, d.d_k, d.d_v, device="cuda")
        y = gdn.decode(d, s.params, *inputs, self.state, self.conv_state, inter)
        h = h + y.view(n * t, -1) @ s.mix_out
        self.kv_lens += t
        h = s.attention(h, self.cache, _cu([t] * n), self.kv_lens, self.block_table)
        uniforms = torch.rand(n, drafts, generator=self.g, device="cuda")
        accepted, tokens = gdn.accept_drafts(guess, s.logits(h).view(n, t, -1), guess_logits, uniforms,
                                             self.noise(), form="logits", temperature=self.temperature)
        # the last token and the accepted drafts stay; the token drawn after them is the next step's first
        gdn.decode_commit(d, accepted + 1, inputs[0], inter, self.state, self.conv_state)
        self.kv_lens -= drafts - accepted
        self.last = tokens.gather(1, accepted[:, None].long())[:, 0].long()
        gdn.sync_status()
        return accepted, tokens


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--sequences", type=int, default=8)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--drafts", type=int, default=3)
    a = p.parse_args()
    stack = Stack()
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(stack.vocab, (50 + 37 * i,), generator=g) for i in range(a.sequences)]
    session = Session(stack, prompts, room=(a.steps + 1) * (a.drafts + 1))
    kept = sum(int(session.step(a.drafts)[0].sum()) for _ in range(a.steps))
    total = a.sequences * a.steps
    print(f"{a.sequences} sequences, {a.steps} steps: {kept} of {total * a.drafts} drafts accepted, "
          f"{(kept + total) / total:.2f} tokens a step")


if __name__ == "__main__":
    main()
