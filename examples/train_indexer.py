"""One training loop of a sparse-attention indexer beside a language model head.

Each step takes a batch of hidden states and
  - projects the indexer's keys and normalises them (layer_norm_fwd), scores
    the selected keys (indexer_fwd), brings the attention target's gradient
    back (indexer_backward) and through the key norm (layer_norm_bwd) to the
    projections;
  - keeps a teacher's top logits (token_logprobs_fwd), and gives the student's
    head the distillation loss and its gradient in one call (distill_grad).

Synthetic data; prints the two losses of every step.

    python examples/train_indexer.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_bwd_gb300 as ibwd  # noqa: E402


class Indexer:
    """Projections of hidden states to the indexer's queries, keys and head weights, fp32 masters."""

    def __init__(self, width, heads, dim, device):
        g = torch.Generator(device=device).manual_seed(1)
        self.heads, self.dim = heads, dim
        self.wq = torch.randn((width, heads * dim), device=device, generator=g) / (8 * width ** 0.5)
        self.wk = torch.randn((width, dim), device=device, generator=g) / width ** 0.5
        self.ww = torch.randn((width, heads), device=device, generator=g) / (width * heads) ** 0.5
        self.gamma = torch.ones(dim, device=device)
        self.beta = torch.zeros(dim, device=device)

    def step(self, h, idx, target, lr):
        """One step towards the attention target; returns its KL divergence (before the step)."""
        B, S, _ = h.shape
        q = (h @ self.wq.to(h.dtype)).view(B, S, self.heads, self.dim)
        raw = h @ self.wk.to(h.dtype)
        k, mean, rstd = ibwd.layer_norm_fwd(raw, self.gamma, self.beta, eps=1e-6)
        w = h.float() @ self.ww
        scores = ibwd.indexer_fwd(q, k, w, idx)
        logp = torch.log_softmax(torch.where(idx >= 0, scores, -torch.inf), -1)
        loss = torch.where(target > 0, target * (target.log() - logp), 0.0).sum(-1).mean()
        dq, dw, dk = ibwd.indexer_backward(q, k, w, scores, target.clone(), idx, dk_mode=ibwd.IBWD_DK_DETERMINISTIC)
        draw, dgamma, dbeta = ibwd.layer_norm_bwd(dk, raw, mean, rstd, self.gamma)
        flat = h.reshape(B * S, -1).float()
        self.wq -= lr * flat.T @ dq.view(B * S, -1)
        self.wk -= lr * flat.T @ draw.view(B * S, -1).float()
        self.ww -= lr * flat.T @ dw.view(B * S, -1)
        self.gamma -= lr * dgamma
        self.beta -= lr * dbeta
        return loss


class Head:
    """The student's vocabulary projection."""

    def __init__(self, width, vocab, device):
        self.w = torch.zeros((width, vocab), device=device)

    def step(self, h, teacher_logits, tokens, weight, top, lr):
        """One step towards the teacher's `top` logits of each position; returns (loss, the teacher's mean log
        probability of the tokens)."""
        flat = h.reshape(-1, h.shape[-1])
        logprob, _, _, ids, kept = ibwd.token_logprobs_fwd(teacher_logits, tokens, top_n=top)
        logits = flat @ self.w.to(flat.dtype)
        # the logits are not needed afterwards: their gradient takes their place
        loss, dlogits = ibwd.distill_grad(logits, ids, kept, weight, out=logits)
        self.w -= lr * flat.float().T @ dlogits.float()
        return (loss * weight).sum(), logprob.mean()


def data(B, S, width, vocab, topk, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    h = torch.randn((B, S, width), device=device, generator=g).bfloat16()
    # distinct random causal keys, -1 where a row has fewer
    order = torch.rand((B, S, S), device=device, generator=g)
    t = torch.arange(S, device=device)
    order.masked_fill_((t[None, :] > t[:, None])[None], 2.0)
    val, idx = torch.topk(order, topk, dim=-1, largest=False)
    idx = torch.where(val <= 1.0, idx, -1).to(torch.int32)
    # what the attention gives the selected keys: a function of the hidden states, so that it can be learned
    a = torch.randn((width, 32), device=device, generator=g) / width ** 0.5
    z = h.float() @ a
    score = torch.einsum("bsd,btd->bst", z, z).gather(2, idx.clamp(min=0).long())
    target = torch.softmax(torch.where(idx >= 0, score, -torch.inf), -1)
    teacher = (h.reshape(B * S, width).float() @ torch.randn((width, vocab), device=device, generator=g)
               * (4 / width ** 0.5)).bfloat16()
    tokens = torch.randint(0, vocab, (B * S,), device=device, generator=g, dtype=torch.int32)
    weight = (torch.rand(B * S, device=device, generator=g) < 0.8).float() / (B * S)  # prompts carry no loss
    return h, idx, target, teacher, tokens, weight


def main(steps=20, B=2, S=512, width=256, vocab=5003, heads=16, dim=64, topk=128, top=32, device="cuda"):
    h, idx, target, teacher, tokens, weight = data(B, S, width, vocab, topk, device)
    indexer, head = Indexer(width, heads, dim, device), Head(width, vocab, device)
    losses = []
    for i in range(steps):
        kl = indexer.step(h, idx, target, lr=0.05)
        distill, _ = head.step(h, teacher, tokens, weight, top, lr=15.0)
        losses.append((kl.item(), distill.item()))
        print(f"step {i:3d}  indexer KL {losses[-1][0]:.4f}  distillation {losses[-1][1]:.4f}")
    status = ibwd.indexer_bwd_last_device_status()
    assert status == ibwd.IBWD_OK, ibwd.status_string(status)
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    main(p.parse_args().steps)
