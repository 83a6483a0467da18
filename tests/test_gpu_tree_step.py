"""The serving loop of examples/tree_step.py: prompts, tables, trees and their
verification used together emit what the target alone emits."""

import os
import sys

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def alone(model, tokens, n):
    """n tokens after `tokens` by the target's choice, the whole sequence each time, in torch."""
    tokens = list(tokens)
    for _ in range(n):
        h = model.embed[torch.tensor(tokens, device=model.dev)]
        T = len(tokens)
        position = torch.arange(T, device=model.dev)
        mask = position[None] > position[:, None]
        for i in range(model.layers):
            q, k, v = model.qkv(i, h, position)
            G = model.q_heads // model.kv_heads
            k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
            s = torch.einsum("ihd,jhd->hij", q, k) * model.dim ** -0.5
            w = torch.softmax(s.masked_fill(mask, -torch.inf), -1)
            h = h + torch.einsum("hij,jhd->ihd", w, v).flatten(1) @ model.wo[i]
        tokens.append(int(model.choice(h[-1:])[0]))
    return tokens


def test_trees_emit_what_the_target_alone_emits():
    import tree_step
    model = tree_step.Model(dtype=torch.float32, vocab=60, dim=32, seed=4)
    server = tree_step.Server(model, pages=20, cols=8)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 60, (n,), generator=g).tolist() for n in (3, 20, 33, 1)]
    truth = [alone(model, p, 30) for p in prompts]
    server.admit(prompts)
    errors = (sv.kv_reserve_error, sv.kv_slots_error, sv.prompt_attention_error, sv.kv_write_error,
              sv.tree_attention_error, sv.verify_tree_greedy_error, sv.kv_commit_error)
    accepted = 0
    for step in range(7):
        drafts = server.drafts()
        # the right tokens in one of the chains, of another length every time
        for b in range(4):
            done = len(server.tokens[b])
            n = (step + b) % (server.chain + 1)
            right = torch.tensor(truth[b][done:done + n], dtype=torch.int32)
            lo = (step % 3) * server.chain
            drafts[b, lo:lo + len(right)] = right.to(drafts.device)
        accept = server.step(drafts)
        for error in errors:
            assert error()[0] == 0
        assert all(int(accept[b]) >= min((step + b) % (server.chain + 1),
                                         server.chain) or len(server.tokens[b]) >= 30
                   for b in range(4))
        accepted += int(accept.sum())
        for b in range(4):
            n = min(len(server.tokens[b]), len(truth[b]))
            assert server.tokens[b][:n] == truth[b][:n]
            assert int(server.kv_len[b]) == len(server.tokens[b]) - 1
    assert accepted > 10
    # places change hands and the pool comes back whole
    server.end([1, 2])
    assert int(server.free_count) == 20 - int(server.held.sum()) and not server.held[1:3].any()
    server.admit([[], prompts[0], [], []])
    server.step()
    assert server.tokens[1][:4] == truth[0][:4]
    server.end([0, 1, 2, 3])
    assert int(server.free_count) == 20
    assert sorted(server.free.tolist()) == list(range(20))
    assert (server.table == -1).all() and (server.held == 0).all()


def test_loop_in_bf16_runs():
    import tree_step
    tree_step.main(4)
    for error in (sv.kv_reserve_error, sv.prompt_attention_error, sv.tree_attention_error,
                  sv.kv_commit_error):
        assert error()[0] == 0
