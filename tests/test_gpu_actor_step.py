"""The training step of examples/actor_step.py: its gradients against the same step in
64-bit autograd on the dequantized weights, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

from actor_ref import D, decode, token_loss

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("actor_step", os.path.join(ROOT, "examples", "actor_step.py"))
A = importlib.util.module_from_spec(spec)
spec.loader.exec_module(A)


def inputs(tokens, hidden, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    res = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    return res, (0.3 * torch.randn(tokens, hidden, generator=g, device="cuda")).to(torch.bfloat16)


def test_step_gradients():
    tokens, hidden, ffn, vocab = 200, 256, 512, 1024
    actor = A.Actor(hidden, ffn, vocab)
    res, delta = inputs(tokens, hidden)
    batch = A.rollout(actor, res, delta, seed=3)
    loss, (dw, dgamma, dres) = A.step(actor, res, delta, batch)
    A.rlq.check()

    w = {}
    for k, (q, s) in actor.q.items():
        v = decode(q) * s.to(D).repeat_interleave(128, 0).repeat_interleave(128, 1)
        w[k] = v.requires_grad_(True)
    gamma = {k: v.to(D).requires_grad_(True) for k, v in actor.gamma.items()}
    r = res.to(D).requires_grad_(True)
    norm = lambda h, g: h * (h.square().mean(1, keepdim=True) + A.EPS).rsqrt() * g  # noqa: E731
    h1 = r + delta.to(D)
    gu = norm(h1, gamma["ffn"]) @ w["gate_up"].t()
    a = torch.nn.functional.silu(gu[:, :ffn]) * gu[:, ffn:]
    h2 = h1 + a @ w["down"].t()
    logits = norm(h2, gamma["final"]) @ w["head"].t()
    targets, old, adv, weight = batch
    lp = torch.log_softmax(logits, 1).gather(1, targets[:, None])[:, 0]
    c = lambda t: t.to(D)  # noqa: E731
    want = token_loss(lp, c(old), c(adv), c(weight), c(old), c(old), None, 0.2, 0.28, 2.0, 0.01).sum()
    want.backward()

    # E4M3 holds a value to 2^-4 at most, 0.026 of a tensor's norm as rounded here (half
    # a step is uniform over [0, 2^-4] of the value); a gradient passes through at most
    # eight such roundings (two operands of each product, the checkpoint), independent of
    # one another, so their norms add in squares: 0.026 * sqrt(8) = 0.074, and one and a
    # half times that for how unevenly the tokens weigh
    def close(got, ref, what):
        off = float((got.to(D) - ref).norm() / ref.norm())
        assert off <= 0.11, (what, off)

    for k in dw:
        close(dw[k], w[k].grad, k)
    for k in dgamma:
        close(dgamma[k], gamma[k].grad, k)
    close(dres, r.grad, "res")


def test_steps_lower_the_loss():
    actor = A.Actor(512, 1024, 2048)
    res, delta = inputs(700, 512, seed=1)
    batch = A.rollout(actor, res, delta, seed=2)
    losses = [float(A.step(actor, res, delta, batch, lr=0.5)[0]) for _ in range(6)]
    A.rlq.check()
    assert losses[-1] < losses[0], losses
