"""Serving one pair of blocks of a hybrid model: a KDA block and a softmax
attention block, with random weights.

The KDA block keeps a fixed state per sequence (a slot of the state pool), the
attention block an 8-bit paged cache that grows.  The example takes a batch of
prompts through both, generates tokens one at a time, verifies a draft window,
takes back its rejected tokens, and evicts the pages that received the least
attention once a sequence is over its budget:

    python examples/hybrid_serving.py

``run`` returns the outputs of every step, and with ``check`` compares the
attention block's with a plain torch form over the cache's stored values.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_delta_rule_decode_gb300 import attn, kda  # noqa: E402


class HybridPair:
    """Weights and per-sequence storage of the two blocks."""

    def __init__(self, hidden=512, kda_heads=4, q_heads=8, kv_heads=2, d=128, seqs=3, pages_per_seq=8, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(rows)).bfloat16()
        self.hidden, self.kda_heads, self.q_heads, self.kv_heads, self.d, self.seqs = (
            hidden, kda_heads, q_heads, kv_heads, d, seqs)
        # q, k, v, decay and beta of the KDA block; its output; q, k, v of the attention block; its output
        self.kda_in = w(hidden, kda_heads * (4 * d + 1))
        self.kda_out = w(kda_heads * d, hidden)
        self.qkv = w(hidden, (q_heads + 2 * kv_heads) * d)
        self.attn_out = w(q_heads * d, hidden)
        self.pool = torch.zeros(seqs, kda_heads, d, d, device="cuda")
        self.slots = torch.arange(seqs, dtype=torch.int32, device="cuda")
        self.cache = attn.alloc_cache(seqs * pages_per_seq, kv_heads, d)
        self.table = torch.randperm(seqs * pages_per_seq, generator=g, device="cuda").int().view(seqs, pages_per_seq)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.weight = torch.zeros(seqs, pages_per_seq, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _kda_inputs(self, x):
        H, d = self.kda_heads, self.d
        y = (x @ self.kda_in).view(x.shape[0], H, 4 * d + 1)
        q, k, v = (y[..., i * d:(i + 1) * d].contiguous() for i in range(3))
        g = torch.nn.functional.logsigmoid(y[..., 3 * d:4 * d].float() + 3).contiguous()
        return q, k, v, g, y[..., 4 * d].contiguous()

    def _qkv(self, x):
        """The slices of the fused projection, as they lie."""
        y = (x @ self.qkv).view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.d)
        return y[:, :self.q_heads], y[:, self.q_heads:-self.kv_heads], y[:, -self.kv_heads:]

    def prompt(self, x, lens):
        """Packed prompts x [T, hidden] of the given lengths, one per sequence."""
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        out = kda.prefill_chunked(*self._kda_inputs(x), cu, self.slots, self.pool, err_flag=self.err)
        x = x + out.flatten(1) @ self.kda_out
        q, k, v = self._qkv(x)
        out = attn.prefill(q, k, v, cu, err_flag=self.err)
        attn.append(self.cache, k, v, cu, self.lens, self.table, err_flag=self.err)
        self.lens = cu[1:] - cu[:-1]
        return x + out.flatten(1) @ self.attn_out, (q, k, v, out)

    def window(self, x, weights=False):
        """D tokens per sequence, x [B, D, hidden], through the attention block only (the verify of a draft)."""
        B, D, _ = x.shape
        q, k, v = self._qkv(x.reshape(B * D, -1))
        cu = torch.arange(0, B * D + 1, D, dtype=torch.int32, device="cuda")
        attn.append(self.cache, k, v, cu, self.lens, self.table, err_flag=self.err)
        self.lens = self.lens + D
        q = q.unflatten(0, (B, D))
        out = attn.decode(q, self.cache, self.lens, self.table, err_flag=self.err,
                          **(dict(weight_in=self.weight, weight_out=self.weight) if weights else {}))
        out = out[0] if weights else out
        return x + out.flatten(2) @ self.attn_out, (q, out)

    def step(self, x):
        """One token per sequence through both blocks, x [B, hidden]."""
        out = kda.decode(*self._kda_inputs(x), self.slots, self.pool, err_flag=self.err)
        x = x + out.flatten(1) @ self.kda_out
        y, seen = self.window(x[:, None], weights=True)
        return y[:, 0], seen

    def take_back(self, tokens):
        """The last tokens of a window were rejected: their places are overwritten by the next ones."""
        self.lens = self.lens - tokens

    def evict(self, budget, sink=1, recent=2):
        r = attn.evict(self.lens, self.table, self.weight, budget, sink, recent, err_flag=self.err)
        # the freed pages go to the ends of their rows, for the tokens to come
        past = self.table.shape[1] - r.freed_count[:, None]
        col = torch.arange(self.table.shape[1], device="cuda")
        back = r.freed.gather(1, (col - past).clamp(min=0).long())
        self.lens, self.weight = r.seq_lens, r.weight
        self.table = torch.where(col < past, r.block_table, back).contiguous()
        return r


def stored_attention(pair: HybridPair, q):
    """Plain attention of windows q [B, D, Hq, d] over the values that the cache stands for."""
    B, D, Hq, d = q.shape
    c, G = pair.cache, Hq // pair.kv_heads
    out = torch.zeros(B, D, Hq, d, device="cuda", dtype=torch.float64)
    for n in range(B):
        length = int(pair.lens[n])
        ids = pair.table[n, :-(-length // attn.PAGE_TOKENS)].long()
        k = c.k_pages.view(torch.uint8)[ids].view(c.k_pages.dtype).double() * c.k_scale[ids].double()[..., None, None]
        v = c.v_pages.view(torch.uint8)[ids].view(c.v_pages.dtype).double() * c.v_scale[ids].double()[..., None, None]
        k = k.transpose(0, 1).flatten(1, 2)[:, :length]
        v = v.permute(1, 0, 3, 2).flatten(1, 2)[:, :length]
        for t in range(D):
            end = length - D + 1 + t
            s = torch.einsum("hgd,hld->hgl", q[n, t].double().view(-1, G, d), k[:, :end]) / math.sqrt(d)
            out[n, t] = torch.einsum("hgl,hld->hgd", s.softmax(-1), v[:, :end]).reshape(Hq, d)
    return out


def run(prompts=(300, 64, 129), steps=4, draft=5, accepted=2, budget=4, check=False, **sizes):
    """The whole course; a list of (what, output) in order."""
    pair = HybridPair(seqs=len(prompts), **sizes)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    seen = []

    def note(what, out, q=None, got=None):
        seen.append((what, out))
        if check and q is not None:
            want = stored_attention(pair, q)
            far = float((got.double() - want).abs().max() / want.abs().max())
            if not far < 1e-2:  # bf16 outputs
                raise AssertionError(f"{what}: attention is {far:.2g} off the stored values' form")

    x = torch.randn(sum(prompts), pair.hidden, generator=g, device="cuda").bfloat16()
    y, _ = pair.prompt(x, list(prompts))
    note("prompt", y)
    last = torch.cumsum(torch.tensor(prompts), 0).cuda() - 1
    x = y[last]
    for i in range(steps):
        x, (q, out) = pair.step(x)
        note(f"step {i}", x, q, out)
    y, (q, out) = pair.window(torch.randn(len(prompts), draft, pair.hidden, generator=g, device="cuda").bfloat16())
    note("window", y, q, out)
    pair.take_back(draft - accepted)
    x = y[:, accepted - 1]
    r = pair.evict(budget)
    note("evicted", r.freed_count)
    for i in range(steps):
        x, (q, out) = pair.step(x)
        note(f"step after eviction {i}", x, q, out)
    if check and int(pair.err):
        raise AssertionError(f"device errors {int(pair.err)}")
    return seen


if __name__ == "__main__":
    for what, out in run(check=True):
        print(what, tuple(out.shape), "freed pages: %s" % out.tolist() if what == "evicted" else
              "mean |x| %.4f" % float(out.float().abs().mean()))
