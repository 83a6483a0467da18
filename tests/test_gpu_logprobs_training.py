"""Log probabilities in a training step with autograd: their gradient is handed to
the logits' backward next to the loss's other terms."""

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_the_gradient_goes_to_the_logits_backward_with_the_loss_s_other_terms():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(9, 32, device=DEV, generator=g)
    w = torch.randn(32, 501, device=DEV, generator=g).requires_grad_()
    tok = torch.randint(0, 501, (9,), dtype=torch.int32, device=DEV, generator=g)
    gl, gh = torch.randn(9, device=DEV, generator=g), torch.randn(9, device=DEV, generator=g)
    logits = x @ w
    r = sv.logprobs(logits, tok)
    assert not any(t.requires_grad for t in r[:4])
    d = sv.logprobs_grad(logits, tok, r.max, r.logsum, r.entropy, gl, gh)
    assert not d.requires_grad
    torch.autograd.backward([w.square().sum(), logits], [None, d])
    w64 = w.detach().double().requires_grad_()
    lp = torch.log_softmax(x.double() @ w64, 1)
    entropy = -(lp.exp() * lp).sum(1)
    picked = lp.gather(1, tok.long()[:, None])[:, 0]
    ((picked * gl).sum() + (entropy * gh).sum() + w64.square().sum()).backward()
    # 32-bit logits of 32 products of up to 12 each, their gradient, 9 rows summed
    tol = 1e-4 * (1 + w64.grad.abs())
    assert ((w.grad.double() - w64.grad).abs() <= tol).all()
