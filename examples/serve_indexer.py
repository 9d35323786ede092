"""One layer of a model with sparse attention that answers: prompts of several
sequences, then tokens one by one, from 8-bit caches.

Each step takes the new tokens' hidden states and
  - projects queries, keys and values and, for the indexer, queries, a key and
    head weights; norms and rotates both (qk_norm_rope_fwd);
  - writes keys and values, and the indexer's key, into their caches
    (cache_write);
  - reads the indexer's keys back, scores them (indexer_fwd) and selects the
    best positions of each token;
  - attends to those (cache_attention).

Random weights and synthetic states; prints how near the selected attention
comes to the attention over all positions.

    python examples/serve_indexer.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_bwd_gb300 as ibwd  # noqa: E402


class Layer:
    """Projections and caches of one layer; `length` the most tokens that a sequence can have."""

    def __init__(self, sequences, length, width=512, heads=8, kv_heads=2, dim=128, index_heads=16, index_dim=64, page=64,
                 code=torch.float8_e4m3fn, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def matrix(n):
            return (torch.randn((width, n), device=device, generator=g) / width ** 0.5).bfloat16()

        self.heads, self.kv_heads, self.dim, self.index_heads, self.index_dim = heads, kv_heads, dim, index_heads, index_dim
        self.w_qkv = matrix((heads + 2 * kv_heads) * dim)
        self.w_index = matrix((index_heads + 1) * index_dim)
        self.w_weight = matrix(index_heads).float() / index_heads ** 0.5
        self.gamma = [torch.ones(n, device=device) for n in (dim, dim, index_dim)]
        self.beta = torch.zeros(index_dim, device=device)
        self.freq = [10000.0 ** (-torch.arange(n, device=device, dtype=torch.float64) / n) for n in (dim // 2, index_dim // 4)]
        pages = -(-length // page)
        # a page in no order, as an allocator would give them
        self.table = torch.randperm(sequences * pages, device=device, generator=g).view(sequences, pages).int()
        self.length = length

        def cache(n_heads, n_dim):
            return (torch.zeros((sequences * pages, n_heads, page, n_dim), device=device, dtype=torch.uint8).view(code),
                    torch.zeros((sequences * pages, n_heads), device=device))

        (self.k, self.k_scale), (self.v, self.v_scale) = cache(kv_heads, dim), cache(kv_heads, dim)
        self.index, self.index_scale = cache(1, index_dim)
        self.lens = torch.zeros(sequences, device=device, dtype=torch.int32)

    def step(self, h, counts=None):
        """New tokens' hidden states [tokens, width], counts[b] of sequence b (one each without), through norm,
        rotation and caches: (queries, index queries, head weights, offsets)."""
        cu = None
        if counts is None:
            self.lens += 1
            positions = self.lens - 1
        else:
            counts = torch.tensor(counts, device=h.device, dtype=torch.int32)
            cu = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
            self.lens += counts
            seq = torch.repeat_interleave(torch.arange(len(counts), device=h.device), counts)
            positions = (torch.arange(len(h), device=h.device) - cu[seq] + (self.lens - counts)[seq]).int()
        d, n = self.dim, self.heads
        qkv = (h @ self.w_qkv).unflatten(1, (-1, d))
        q, k, v = qkv[:, :n], qkv[:, n:n + self.kv_heads], qkv[:, n + self.kv_heads:]
        q, k = ibwd.qk_norm_rope_fwd(q, k, positions, self.freq[0], q_gamma=self.gamma[0], k_gamma=self.gamma[1])
        ibwd.cache_write(k, v, self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens, cu=cu)
        index = (h @ self.w_index).unflatten(1, (-1, self.index_dim))
        iq, ik = ibwd.qk_norm_rope_fwd(index[:, :-1], index[:, -1:], positions, self.freq[1], q_norm="none", k_norm="layer",
                                       k_gamma=self.gamma[2], k_beta=self.beta)
        ibwd.cache_write(ik, None, self.index, None, self.index_scale, None, self.table, self.lens, cu=cu)
        return q, iq, h.float() @ self.w_weight, cu

    def select(self, iq, weight, kept):
        """The `kept` best positions of each sequence's last token, -1 where it has fewer: [sequences, kept] int32."""
        keys = ibwd.cache_read(self.index, self.index_scale, self.table, self.lens, self.length)[:, :, 0]
        at = torch.arange(self.length, device=keys.device, dtype=torch.int32)
        every = torch.where(at < self.lens[:, None], at, -1)[:, None].contiguous()
        scores = ibwd.indexer_fwd(iq[:, None].contiguous(), keys, weight[:, None].contiguous(), every)[:, 0]
        best = torch.topk(torch.where(every[:, 0] >= 0, scores, -torch.inf), kept, dim=1)
        return torch.where(best.values > -torch.inf, best.indices, -1).int()

    def attend(self, q, cu=None, select=None):
        return ibwd.cache_attention(q, self.k, self.v, self.k_scale, self.v_scale, self.table, self.lens, cu=cu, select=select)


def main(steps=8, prompts=(300, 17, 129, 500), kept=128, length=1024, device="cuda"):
    layer = Layer(len(prompts), length, device=device)
    g = torch.Generator(device=device).manual_seed(1)
    q, _, _, cu = layer.step(torch.randn((sum(prompts), 512), device=device, generator=g).bfloat16(), prompts)
    layer.attend(q, cu)
    far = []
    for i in range(steps):
        q, iq, weight, _ = layer.step(torch.randn((len(prompts), 512), device=device, generator=g).bfloat16())
        chosen = layer.select(iq, weight, kept)
        some, _ = layer.attend(q, select=chosen)
        every, _ = layer.attend(q)
        far.append(((some.float() - every.float()).norm() / every.float().norm()).item())
        print(f"step {i:3d}  lengths {layer.lens.tolist()}  selected against all positions: {far[-1]:.3f}")
    status = ibwd.indexer_bwd_last_device_status()
    assert status == ibwd.IBWD_OK, ibwd.status_string(status)
    return far


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=8)
    main(p.parse_args().steps)
