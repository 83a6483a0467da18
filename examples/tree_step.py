"""A serving loop over a small random model whose drafter proposes trees: prompts
are admitted (pages from the pool, slots, attention over the packed prompts, keys
and values into their slots), every step verifies a tree of drafts a request
against the target's choices and commits the accepted path, and requests that end
give their pages back.

    python examples/tree_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_13_gb300 as sv  # noqa: E402


class Model:
    """`layers` attention layers without feed-forward blocks; positions are rotated in."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, dim=64, vocab=512, dtype=torch.bfloat16,
                 seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.layers, self.q_heads, self.kv_heads, self.dim = layers, q_heads, kv_heads, dim
        self.vocab, self.dtype, self.dev = vocab, dtype, device
        d, E = q_heads * dim, kv_heads * dim

        def weight(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=g) * rows ** -0.5).to(dtype)

        self.embed = torch.randn(vocab, d, device=device, generator=g).to(dtype)
        self.wqkv = [weight(d, d + 2 * E) for _ in range(layers)]
        self.wo = [weight(d, d) for _ in range(layers)]
        self.unembed = weight(d, vocab).T.contiguous()      # [vocab, d]

    def norm(self, h):
        return h * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + 1e-5).to(self.dtype)

    def rotate(self, x, position):
        half = self.dim // 2
        f = 10000.0 ** (-torch.arange(half, device=self.dev) / half)
        a = position[:, None, None].float() * f
        lo, hi = x[..., :half].float(), x[..., half:].float()
        return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()],
                         -1).to(self.dtype)

    def qkv(self, i, h, position):
        """q [rows, q_heads, dim], k and v [rows, kv_heads, dim] of layer i."""
        x = (self.norm(h) @ self.wqkv[i]).unflatten(1, (-1, self.dim))
        q, k, v = x.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        return self.rotate(q, position), self.rotate(k, position), v

    def choice(self, h):
        """The target's argmax of every row."""
        x = self.norm(h).contiguous()
        if self.dtype is torch.bfloat16:   # the logits stay in the product's epilogue
            ones = torch.ones(x.shape[0], device=self.dev)
            return sv.lmhead_stats(x, self.unembed, ones)[2]
        return (x @ self.unembed.T).argmax(1).int()


class Server:
    """B places for requests over a pool of pages."""

    def __init__(self, model, B=4, pages=64, page=16, cols=16, chain=3):
        self.m, self.B, self.page, self.chain = model, B, page, chain
        # the tree: three chains that begin with a request's three likeliest next tokens
        self.nodes = nodes = 3 * chain + 1
        dev = model.dev
        E = model.kv_heads * model.dim
        i32 = dict(dtype=torch.int32, device=dev)
        self.cache = torch.zeros(pages, model.layers, 2, page, E, dtype=model.dtype, device=dev)
        self.table = torch.full((B, cols), -1, **i32)
        self.held, self.kv_len = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.free = torch.arange(pages, device=dev).int()
        self.free_count = torch.full((1,), pages, **i32)
        self.spec = torch.zeros(B, nodes, model.layers, 2, E, dtype=model.dtype, device=dev)
        parent = [-1] + [0 if j % chain == 0 else j for j in range(3 * chain)]
        self.parent = torch.tensor(parent * B, **i32)
        self.k = torch.full((B,), 3 * chain, **i32)
        depth = [0]
        for p in parent[1:]:
            depth.append(depth[p] + 1)
        self.depth = torch.tensor(depth, **i32)
        self.last = torch.zeros(B, **i32)
        self.tokens = [[] for _ in range(B)]

    def reserve(self, lengths):
        sv.kv_reserve(self.table, self.held, lengths, self.free, self.free_count, self.page)

    def admit(self, prompts):
        """Prompts (lists of tokens, empty: nothing new) for the places; the first new token."""
        m = self.m
        count = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=m.dev)
        self.kv_len = torch.where(count > 0, 0, self.kv_len)
        self.reserve(torch.where(count > 0, count, self.kv_len))
        rows = sum(len(p) for p in prompts)
        at = sv.kv_slots(self.table, torch.zeros_like(count), count, rows, self.page)
        h = m.embed[torch.tensor([t for p in prompts for t in p], device=m.dev)]
        for i in range(m.layers):
            q, k, v = m.qkv(i, h, at.position)
            out, _ = sv.prompt_attention(q, k, v, at.offsets)
            sv.kv_write(self.cache, i, k, v, at.slots)
            h = h + out.flatten(1) @ m.wo[i]
        first = m.choice(h)
        new = count > 0
        ends = (at.offsets[1:] - 1).clamp_min(0).long()
        self.last = torch.where(new, first[ends], self.last)
        self.kv_len = torch.where(new, count, self.kv_len)
        for b, p in enumerate(prompts):
            if p:
                self.tokens[b] = list(p) + [int(self.last[b])]

    def drafts(self):
        """Tokens of nodes 1 .. of every request's tree, from the embeddings alone."""
        near = (self.m.embed[self.last.long()].float() @ self.m.unembed.float().T)
        tokens = near.topk(3, 1)[1]                              # [B, 3]
        out = [tokens]
        for _ in range(self.chain - 1):
            tokens = (self.m.embed[tokens].float() @ self.m.unembed.float().T).argmax(-1)
            out.append(tokens)
        return torch.stack(out, 2).flatten(1).int()              # chain by chain

    def step(self, drafts=None):
        """One verification; drafts [B, nodes - 1] instead of the drafter's."""
        m, N = self.m, self.nodes
        drafts = self.drafts() if drafts is None else drafts
        self.reserve(self.kv_len + N)
        h = m.embed[torch.cat([self.last[:, None], drafts], 1).reshape(-1).long()]
        position = (self.kv_len[:, None] + self.depth).reshape(-1)
        for i in range(m.layers):
            q, k, v = m.qkv(i, h, position)
            self.spec[:, :, i] = torch.stack([k.flatten(1), v.flatten(1)], 1).unflatten(
                0, (self.B, N))
            out, _ = sv.tree_attention(q, self.cache, i, self.kv_len, self.table, self.k,
                                       self.parent, self.spec)
            h = h + out.flatten(1) @ m.wo[i]
        accept, emitted, path = sv.verify_tree_greedy(m.choice(h), drafts.reshape(-1).contiguous(),
                                                      self.parent, self.k, m.vocab)
        sv.kv_commit(self.cache, self.spec, accept, self.k, self.kv_len, self.table, path=path)
        self.last = emitted.view(self.B, N).gather(1, accept.clamp_min(0)[:, None].long())[:, 0]
        for b, row in enumerate(emitted.view(self.B, N).tolist()):
            self.tokens[b] += [t for t in row if t >= 0]
        return accept

    def end(self, places):
        """Requests that are done give their pages back."""
        gone = torch.zeros(self.B, dtype=torch.bool, device=self.m.dev)
        gone[places] = True
        self.kv_len = torch.where(gone, 0, self.kv_len)
        self.reserve(self.kv_len)


def main(steps=12):
    g = torch.Generator().manual_seed(0)
    server = Server(Model())
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (5, 40, 17, 1)]
    server.admit(prompts)
    for i in range(steps):
        accept = server.step()
        if i == steps // 2:   # one ends, another takes its place
            server.end([1])
            server.admit([[], prompts[2][:9], [], []])
        print(f"step {i:2d}  accepted {accept.tolist()}  cached {server.kv_len.tolist()}  "
              f"free pages {server.free_count.item()}")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 12)
