"""Bounds of the policy loss's gradient, element by element and in proportion to each
(shared by the GPU tests and the CPU test of the bounds themselves; test infrastructure only)."""
import torch

from actor_ref import D, U
from test_gpu_actor import HYP, loss_reference, row_sensitivity


def gradient_bounds(st, temperature, hyp=HYP):
    """(rows to look at, gradient, its bound)."""
    live, lp, _, grad, elp = loss_reference(st, temperature, hyp)
    _, edlp = row_sensitivity(st, lp, elp, temperature, hyp)
    T, V = grad.shape
    cast = lambda k: None if st[k] is None else st[k].to(D)  # noqa: E731
    old, adv, behav, ref, hi = (cast(k) for k in ("logp_old", "adv", "logp_behav", "logp_ref", "clip_hi"))
    hi = torch.full_like(old, 1 + hyp["eps_hi"]) if hi is None else hi
    lo = 1 - hyp["eps_lo"]
    rho = (lp - old).exp()
    # rows within the ratio's error of a clip bound may take either branch
    sure = live & ((rho - hi).abs() > 1e-4) & ((rho - lo).abs() > 1e-4)
    w = torch.ones_like(rho) if behav is None else (old - behav).exp().clamp(max=hyp["tis_cap"])
    pg = torch.where(rho * adv <= torch.minimum(rho.clamp(min=lo), hi) * adv, -w * adv * rho, torch.zeros_like(rho))
    dlp = pg if ref is None else pg - hyp["kl_beta"] * torch.expm1(ref - lp)
    dlp, edlp = (cast("weight") * dlp).abs()[:, None], edlp[:, None]

    z = st["logits"].to(D) / temperature
    p = torch.softmax(z, 1)
    delta = z.amax(1, keepdim=True) - z
    # an exponential: its argument is five roundings of a product with the distance from the
    # maximum, the instruction within 2^-21
    e = (8 + 6 * delta) * U
    # the row's sum: its terms' errors in proportion to their share; the additions of a
    # thread (512 of them, two sums each, 64 elements a pass at least) and of three trees;
    # a rescaling for each pass of 16384 elements that raises the maximum, and three joins
    s = (p * e).sum(1, keepdim=True) + (V / 1024 + 64 + 20 + 9 * (V / 16384 + 1) + 3 * 9) * U
    target = torch.zeros_like(p, dtype=torch.bool)
    target[torch.arange(T, device=p.device), st["targets"].clamp(0, V - 1)] = True
    off = p * (edlp + dlp * (e + s + 6 * U))  # -dlp p, the quotient's and the products' roundings
    own = torch.where(target, edlp * (1 - p) + dlp * (p * (e + s + 6 * U) + 4 * U * (1 - p)), off) / temperature
    # an exponential below 2^-126 is flushed; results below the normal range round to the
    # type's smallest step
    bf16 = st["logits"].dtype == torch.bfloat16
    own = own + 2.0 ** -126 * dlp / temperature
    step = 2.0 ** -8 if bf16 else U
    return sure, grad, own + step * (grad.abs() + own) + (2.0 ** -134 if bf16 else 2.0 ** -150)


def check_gradient(st, d, temperature):
    """``st`` holds the logits as they were before the call."""
    sure, grad, tol = gradient_bounds(st, temperature)
    assert bool(sure.any())
    bad = ((d.to(D) - grad).abs() > tol) & sure[:, None]
    assert not bad.any(), f"{int(bad.sum())} gradients off, first at {bad.nonzero()[0].tolist()}"
