"""A serving loop over a small random model that uses the whole step: drafting,
the target's pass over the drafts with attention over the paged cache,
verification, log probabilities of what was emitted, accumulated attention
weights, the cache's commit and its eviction, and a gradient step that teaches
the drafter the emitted tokens.

    python examples/serving_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_13_gb300 as sv  # noqa: E402


class Loop:
    """B requests, k drafts each, a target of `layers` attention layers without
    feed-forward blocks, and a drafter that is one matrix."""

    def __init__(self, B=4, k=3, layers=2, q_heads=8, kv_heads=2, dim=64, vocab=512, page=16,
                 budget=48, sinks=2, recent=8, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.g, self.dev, self.dtype = g, device, dtype
        self.B, self.k, self.layers = B, k, layers
        self.q_heads, self.kv_heads, self.dim, self.vocab = q_heads, kv_heads, dim, vocab
        self.budget, self.sinks, self.recent = budget, sinks, recent
        d, E = q_heads * dim, kv_heads * dim

        def weight(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=g) * rows ** -0.5).to(dtype)

        self.embed = torch.randn(vocab, d, device=device, generator=g).to(dtype)
        self.wqkv = [weight(d, d + 2 * E) for _ in range(layers)]
        self.wo = [weight(d, d) for _ in range(layers)]
        self.unembed = weight(d, vocab)
        self.drafter = torch.zeros(d, vocab, device=device, dtype=torch.float32)
        # every request owns the pages for its budget and one commit past it
        pages = -(-(budget + k + 1) // page)
        self.cache = torch.zeros(B * pages, layers, 2, page, E, dtype=dtype, device=device)
        self.table = torch.randperm(B * pages, device=device, generator=g).int().view(B, pages)
        i32 = dict(dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(B, **i32)
        self.k_per_req = torch.full((B,), k, **i32)
        self.score = torch.zeros(B, pages * page, device=device)
        self.temperature = torch.ones(B, device=device)
        self.last = torch.randint(0, vocab, (B,), device=device, generator=g).int()
        self.spec = torch.zeros(B, k + 1, layers, 2, E, dtype=dtype, device=device)

    def draft(self):
        """k drafts a request, one after the other, and the logits they are drawn from, in
        the type that verification takes: it compares with the distribution of the draw."""
        u = torch.rand(self.B, self.k, device=self.dev, generator=self.g)
        one = torch.ones_like(self.k_per_req)
        tokens, logits, last = [], [], self.last
        for i in range(self.k):
            x = (self.embed[last.long()].float() @ self.drafter).to(self.dtype)
            last = sv.draft_sample(x, one, self.temperature, u[:, i].contiguous())[0]
            tokens.append(last.clone())
            logits.append(x)
        return torch.stack(tokens, 1), torch.stack(logits, 1)

    def target(self, tokens):
        """Logits of the last token and the drafts, and each layer's q and lse."""
        rows = self.B * (self.k + 1)
        h = self.embed[tokens.reshape(-1).long()]
        d, E = h.shape[1], self.kv_heads * self.dim
        kept = []
        for i in range(self.layers):
            x = h * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + 1e-5).to(self.dtype)
            qkv = x @ self.wqkv[i]
            self.spec[:, :, i] = qkv[:, d:].view(self.B, self.k + 1, 2, E)
            q = qkv[:, :d].unflatten(1, (self.q_heads, self.dim))   # a slice: strides are free
            out, lse = sv.attention(q, self.cache, i, self.kv_len, self.table, self.k_per_req,
                                    self.spec)
            kept.append((q, lse))
            h = h + out.view(rows, d) @ self.wo[i]
        x = h * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + 1e-5).to(self.dtype)
        return (x @ self.unembed).contiguous(), kept

    def step(self, rate=0.05):
        drafts, draft_logits = self.draft()
        logits, kept = self.target(torch.cat([self.last[:, None], drafts], 1))
        uniforms = torch.rand(logits.shape[0], device=self.dev, generator=self.g)
        accept, tokens = sv.verify(logits, draft_logits.reshape(-1, self.vocab),
                                   drafts.reshape(-1), self.k_per_req, self.temperature, uniforms)
        scored = sv.logprobs(logits, tokens, n_top=4)   # -1 past the last emitted: skipped
        for i, (q, lse) in enumerate(kept):
            sv.attention_weights(q, self.cache, i, self.kv_len, self.table, self.k_per_req, lse,
                                 self.score, self.spec, accept)
        sv.kv_commit(self.cache, self.spec, accept, self.k_per_req, self.kv_len, self.table)
        sv.kv_evict(self.cache, self.score, self.kv_len, self.table, self.budget, self.sinks,
                    self.recent)
        # the drafter learns the emitted tokens: gradient of the sum of their log probabilities
        emitted = tokens.view(self.B, self.k + 1)
        before = torch.cat([self.last[:, None], emitted[:, :-1]], 1)
        x = self.learnt_from = self.embed[before.clamp_min(0).reshape(-1).long()].float()
        own = x @ self.drafter
        learnt = sv.logprobs(own, tokens)
        count = (tokens >= 0).float()
        d = sv.logprobs_grad(own, tokens, learnt.max, learnt.logsum, learnt.entropy, count)
        self.drafter += rate * (x.T @ d) / x.shape[1]
        self.last = emitted.gather(1, accept.clamp_min(0)[:, None].long())[:, 0]
        return accept, tokens, scored, learnt


def main(steps=40):
    loop = Loop()
    for i in range(steps):
        accept, tokens, scored, learnt = loop.step()
        if i % 8 == 0 or i == steps - 1:
            ok = tokens >= 0
            print(f"step {i:3d}  accepted {accept.tolist()}  cached {loop.kv_len.tolist()}  "
                  f"target {scored.logprob[ok].mean().item():.3f}  "
                  f"drafter {learnt.logprob[ok].mean().item():.3f}  "
                  f"entropy {scored.entropy[ok].mean().item():.3f}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
