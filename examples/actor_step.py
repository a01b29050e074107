"""One training step of an actor's last feed-forward sublayer, head and policy loss.

The residual stream goes through the residual norm, the gated feed-forward block, the
down projection, the final norm and the head; the policy loss gives the gradient of the
logits, and the backward pass returns to the residual stream, with FP8 codes as the only
activations kept between the passes:

    h1 = res + delta            x1 = rmsnorm(h1) g1         (codes, both groupings)
    a  = silu(x1 Wg^T) * (x1 Wu^T)                          (codes, 8-bit checkpoint)
    y  = a Wd^T
    h2 = h1 + y                 x2 = rmsnorm(h2) g2         (codes, both groupings)
    logits = x2 Wv^T            loss, dlogits

Every product runs in the library's FP8 GEMMs; weights are kept in bf16 and quantized
after each update.  Run on a GPU:

    python examples/actor_step.py --tokens 2048 --hidden 2048 --ffn 8192 --vocab 32000 --steps 5
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_block_scaled_quantize_gb300 import rlq  # noqa: E402

EPS = 1e-6


class Actor:
    """Weights of the sublayer and the head, in bf16 and as FP8 codes."""

    def __init__(self, hidden: int, ffn: int, vocab: int, seed: int = 0):
        if vocab % 128:
            raise ValueError("vocab must be a multiple of 128 (pad the head)")
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16)

        self.w = {"gate_up": weight(2 * ffn, hidden), "down": weight(hidden, ffn), "head": weight(vocab, hidden)}
        self.gamma = {"ffn": torch.ones(hidden, dtype=torch.bfloat16, device="cuda"),
                      "final": torch.ones(hidden, dtype=torch.bfloat16, device="cuda")}
        self.quantize()

    def quantize(self):
        self.q = {k: rlq.quant_weight_128x128(w)[:2] for k, w in self.w.items()}

    def forward(self, res, delta):
        """Logits, and what the backward pass needs."""
        h1, *x1, r1 = rlq.add_rmsnorm_quant_act_1x128(res, delta, self.gamma["ffn"], EPS, colwise=True)
        aq, as_, guq, gus = rlq.gemm_gated_fprop(x1[0], x1[1], *self.q["gate_up"], checkpoint=True)
        y = rlq.gemm_fprop(aq, as_, *self.q["down"])
        h2, *x2, r2 = rlq.add_rmsnorm_quant_act_1x128(h1, y, self.gamma["final"], EPS, colwise=True)
        logits = rlq.gemm_fprop(x2[0], x2[1], *self.q["head"])
        return logits, {"h1": h1, "x1T": x1[2:], "r1": r1, "gu": (guq, gus), "h2": h2, "x2T": x2[2:], "r2": r2}

    def backward(self, dlogits, kept):
        """Gradients of the weights, the norm weights and the residual stream."""
        dw, dgamma = {}, {}
        q, s, qT, sc = rlq.quant_act_1x128(dlogits, colwise=True)
        dw["head"] = rlq.gemm_wgrad(qT, sc, *kept["x2T"])
        dx2 = rlq.gemm_dgrad(q, s, *self.q["head"], transposed=False)
        dh2, dgamma["final"] = rlq.rmsnorm_backward(dx2, kept["h2"], kept["r2"], self.gamma["final"])
        # dh2 is the gradient of the down projection's output and, past it, of h1
        q, s, qT, sc = rlq.quant_act_1x128(dh2, colwise=True)
        da = rlq.gemm_dgrad(q, s, *self.q["down"], transposed=False)
        gq, gs, gqT, gsc, aT, ac = rlq.gated_backward(da, *kept["gu"])
        dw["down"] = rlq.gemm_wgrad(qT, sc, aT, ac)
        dw["gate_up"] = rlq.gemm_wgrad(gqT, gsc, *kept["x1T"])
        dx1 = rlq.gemm_dgrad(gq, gs, *self.q["gate_up"], transposed=False)
        dres, dgamma["ffn"] = rlq.rmsnorm_backward(dx1, kept["h1"], kept["r1"], self.gamma["ffn"], dres=dh2,
                                                   inplace=True)
        return dw, dgamma, dres

    def update(self, dw, dgamma, lr):
        for k, g in dw.items():
            self.w[k].add_(g, alpha=-lr)
        for k, g in dgamma.items():
            self.gamma[k].add_(g.to(torch.bfloat16), alpha=-lr)
        self.quantize()


def rollout(actor, res, delta, seed):
    """Sampled tokens, their log probabilities and advantages, as a rollout hands them over."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    logits, _ = actor.forward(res, delta)
    targets = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=g)[:, 0]
    lp, _ = rlq.token_logprobs(logits, targets)
    adv = torch.randn(res.shape[0], generator=g, device="cuda")
    weight = (torch.rand(res.shape[0], generator=g, device="cuda") < 0.9).float()
    return targets, lp, adv, weight / weight.sum().clamp(min=1)


def step(actor, res, delta, batch, lr=None):
    """One forward and backward pass; with ``lr`` an update.  Returns (loss, gradients)."""
    targets, lp_old, adv, weight = batch
    logits, kept = actor.forward(res, delta)
    loss, _, dlogits = rlq.policy_loss(logits, targets, lp_old, adv, weight, logp_behav=lp_old, logp_ref=lp_old,
                                       eps_lo=0.2, eps_hi=0.28, kl_beta=0.01, inplace=True)
    grads = actor.backward(dlogits, kept)
    if lr is not None:
        actor.update(grads[0], grads[1], lr)
    return loss.sum(), grads


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=8192)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    actor = Actor(a.hidden, a.ffn, a.vocab)
    res = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    delta = (0.3 * torch.randn(a.tokens, a.hidden, device="cuda")).to(torch.bfloat16)
    batch = rollout(actor, res, delta, seed=1)
    for i in range(a.steps):
        loss, _ = step(actor, res, delta, batch, lr=a.lr)
        print(f"step {i}: loss {float(loss):+.6f}")
    rlq.check()


if __name__ == "__main__":
    main()
