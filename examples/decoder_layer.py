"""A decoder layer served from a paged cache: the Engram read into the residual stream, then attention.

Prompts of unequal length go through the layer at once, then every sequence decodes token by token:

    h += gate * (Engram rows @ W_out)                        engram_forward
    q | k | v = rmsnorm(h) @ W_qkv
    q, k normed and rotated, k and v into the cache          engram_kv_append
    h += attention(q, cache) @ W_o                           engram_paged_attention

The same tokens given as one long prompt must lead to the same residuals; the example checks it.

    python examples/decoder_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import engram_gram_hash_gb300 as eg  # noqa: E402
from synth import device as sd  # noqa: E402
from synth.configs import CONFIGS, default_seeds  # noqa: E402

PAGE = 64


class Pages:
    """The layer's cache and a block table per sequence; pages are handed out as sequences grow."""

    def __init__(self, n_pages, n_seqs, kv_heads, dim, max_tokens, device):
        shape = (n_pages, PAGE, kv_heads, dim)
        self.cache = eg.kv_cache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                                 torch.empty(shape, dtype=torch.bfloat16, device=device))
        self.table = torch.zeros((n_seqs, -(-max_tokens // PAGE)), dtype=torch.int32, device=device)
        self.length = [0] * n_seqs
        self.free = list(range(n_pages))

    def grow(self, new):
        """Makes room for new[s] tokens of every sequence; returns the step's batch and its seq_offsets."""
        for s, n in enumerate(new):
            have, need = -(-self.length[s] // PAGE), -(-(self.length[s] + n) // PAGE)
            for p in range(have, need):
                self.table[s, p] = self.free.pop()
            self.length[s] += n
        offsets = torch.tensor([0] + list(new)).cumsum(0).to(self.table.device)
        kv_len = torch.tensor(self.length, dtype=torch.int32, device=self.table.device)
        return eg.kv_batch(offsets, kv_len, self.table, sum(new)), offsets


class Layer:
    def __init__(self, cfg, heads, kv_heads, dim, max_tokens, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * rows**-0.5).to(torch.bfloat16)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.engram = eg.make_config(cfg.V, cfg.R, cfg.d, default_seeds())
        self.tables = torch.empty((48, cfg.R, 256), dtype=torch.uint8, device=device)
        self.scales = torch.empty((48, cfg.R), dtype=torch.float32, device=device)
        sd.fill_tables(self.tables, cfg.seed)
        sd.fill_scales(self.scales, cfg.seed)
        self.w_out = torch.empty((512, cfg.d), dtype=torch.bfloat16, device=device)
        self.gate = torch.empty(cfg.d, dtype=torch.bfloat16, device=device)
        sd.fill_w_out(self.w_out, cfg.seed)
        sd.fill_g(self.gate, cfg.seed)
        self.attn = eg.make_attn_config(heads, kv_heads, dim)
        self.rope = eg.rope_table(max_tokens, dim, device=device)
        self.w_qkv = weight(cfg.d, (heads + 2 * kv_heads) * dim)
        self.w_o = weight(heads * dim, cfg.d)
        self.w_q = torch.ones(dim, dtype=torch.bfloat16, device=device)
        self.w_k = torch.ones(dim, dtype=torch.bfloat16, device=device)

    def __call__(self, h, pages, new, tokens, token_offsets, last_n):
        """One step in place on h [sum(new), d]: tokens holds each sequence's ids up to its last new one (at
        least the three before them), last_n the queries per sequence (0: all of them)."""
        batch, _ = pages.grow(new)
        eg.engram_forward(self.engram, tokens, token_offsets, self.tables, self.scales, self.w_out, self.gate, h,
                          last_n=last_n, n_query=h.shape[0])
        x = h.float()
        x = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
        q, k, v = (x @ self.w_qkv).split([self.heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim], 1)
        q, k, v = (t.unflatten(1, (-1, self.dim)) for t in (q, k, v))
        q = eg.engram_kv_append(self.attn, pages.cache, batch, k, v, self.rope, w_k=self.w_k, q=q, w_q=self.w_q)
        out = eg.engram_paged_attention(self.attn, pages.cache, batch, q)
        h += out.flatten(1) @ self.w_o
        return h


def ids_of(seqs, device):
    """Packed ids and their offsets."""
    flat = torch.cat(seqs).to(torch.int32).to(device)
    return flat, torch.tensor([0] + [len(s) for s in seqs]).cumsum(0).to(device)


def run(prompts=(300, 17, 1000, 64), steps=8, heads=8, kv_heads=2, dim=128, device="cuda", seed=0):
    """The residuals [n_seqs, steps, d] of the last `steps` tokens: decoded one by one, and as one prompt."""
    cfg = CONFIGS["tiny"].with_(d=1024)
    g = torch.Generator().manual_seed(seed)
    total = [p + steps for p in prompts]
    seqs = [torch.randint(0, cfg.V, (t,), generator=g) for t in total]
    rows = [torch.randn((t, cfg.d), generator=g).to(torch.bfloat16).to(device) for t in total]
    n, longest = len(prompts), max(total)
    layer = Layer(cfg, heads, kv_heads, dim, longest, device, seed)
    n_pages = sum(-(-t // PAGE) for t in total)

    # the prompts at once, then a token of every sequence per step
    pages = Pages(n_pages, n, kv_heads, dim, longest, device)
    layer(torch.cat([r[:p] for r, p in zip(rows, prompts)]), pages, list(prompts),
          *ids_of([s[:p] for s, p in zip(seqs, prompts)], device), last_n=0)
    decoded = []
    for i in range(steps):
        h = torch.stack([r[p + i] for r, p in zip(rows, prompts)])
        ids = ids_of([s[max(0, p + i - 3):p + i + 1] for s, p in zip(seqs, prompts)], device)
        decoded.append(layer(h, pages, [1] * n, *ids, last_n=1))
    decoded = torch.stack(decoded, 1)

    # everything as one prompt
    whole = layer(torch.cat(rows), Pages(n_pages, n, kv_heads, dim, longest, device), total, *ids_of(seqs, device), last_n=0)
    whole = torch.stack([w[-steps:] for w in whole.split(total)])
    assert eg.engram_last_error() == 0
    return decoded, whole


def main():
    decoded, whole = run()
    a, b = decoded.double(), whole.double()
    worst = ((a - b).abs() / b.abs().clamp(min=1.0)).max().item()
    print(f"{decoded.shape[0]} sequences, {decoded.shape[1]} decoded tokens each: "
          f"largest scaled difference from the whole prompt {worst:.2e}")
    return worst


if __name__ == "__main__":
    sys.exit(0 if main() <= 4e-2 else 1)
