"""The serving loop of examples/serving_step.py: its parts fit together."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_loop_keeps_its_budget_and_its_sums():
    import serving_step
    import speculative_decoding_verification_13_gb300 as sv
    loop = serving_step.Loop(budget=32, recent=6, seed=3)
    total = 0
    for _ in range(14):
        before = loop.kv_len.clone()
        mass = loop.score.double().sum(1)
        accept, tokens, scored, learnt = loop.step()
        assert (accept >= 0).all()
        for error in (sv.attention_error, sv.attention_weights_error, sv.kv_commit_error,
                      sv.kv_evict_error):
            assert error()[0] == 0
        grown = before + accept + 1
        assert torch.equal(loop.kv_len, grown.clamp_max(32))
        total += int((accept + 1).sum())
        kept = grown <= 32
        # a token gives one unit of weight per head and layer
        gain = loop.score.double().sum(1) - mass
        want = (accept + 1).double() * loop.q_heads * loop.layers
        if kept.any():
            assert ((gain - want)[kept].abs() <= 2e-3 * want[kept]).all()
        beyond = torch.arange(loop.score.shape[1], device="cuda")[None] >= loop.kv_len[:, None]
        assert (loop.score[beyond] == 0).all()
        ok = tokens >= 0
        assert torch.equal(torch.isnan(scored.logprob), ~ok)
        assert int(ok.sum()) == int((accept + 1).sum())
        assert (scored.top_logprobs[ok][:, 0] >= scored.logprob[ok]).all()
    assert total >= 14 * loop.B and (loop.kv_len == 32).any()


def test_a_gradient_step_raises_the_emitted_tokens():
    import serving_step
    import speculative_decoding_verification_13_gb300 as sv
    loop = serving_step.Loop(seed=1)
    for _ in range(5):
        _, tokens, _, learnt = loop.step(rate=0.1)
        ok = tokens >= 0
        again = sv.logprobs(loop.learnt_from @ loop.drafter, tokens)
        assert again.logprob[ok].sum() > learnt.logprob[ok].sum()


def test_drafts_come_from_the_logits_that_verification_gets(monkeypatch):
    # acceptance compares the target with the distribution the drafts were drawn from
    import serving_step
    import speculative_decoding_verification_13_gb300 as sv
    loop = serving_step.Loop(seed=2)
    drawn, verified = [], []
    sample, verify = sv.draft_sample, sv.verify

    def sample_and_note(logits, *a, **kw):
        drawn.append(logits.float().clone())
        return sample(logits, *a, **kw)

    def verify_and_note(target, draft, *a, **kw):
        verified.append(draft.float().clone())
        return verify(target, draft, *a, **kw)

    monkeypatch.setattr(sv, "draft_sample", sample_and_note)
    monkeypatch.setattr(sv, "verify", verify_and_note)
    for _ in range(3):
        loop.step(rate=0.3)
        seen = torch.stack(drawn, 1).reshape(-1, loop.vocab)
        assert torch.equal(seen, verified[-1])
        drawn.clear()
    assert verified[-1].abs().max() > 0
