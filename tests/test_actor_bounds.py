"""CPU test of the bounds that the policy loss's gradient is held to: the formula in 32-bit
torch is within them, the same with a mistake in it is not."""
import pytest
import torch

import actor_bounds as B
import test_gpu_actor as A

TEMPERATURE = 0.9


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(A, "DEV", "cpu")


def formula(st, hyp=A.HYP):
    """The gradient in 32 bits, step by step as a kernel forms it."""
    x, old = st["logits"].float(), st["logp_old"]
    c = torch.tensor(1.4426950408889634) / torch.tensor(TEMPERATURE)
    m = x.amax(1, keepdim=True)
    e = torch.exp2((x - m) * c)
    total = e.sum(1, keepdim=True)
    t = st["targets"][:, None]
    lp = (0.6931471805599453 * ((x.gather(1, t) - m) * c - torch.log2(total)))[:, 0]
    rho = (lp - old).exp()
    w = torch.ones_like(rho) if st["logp_behav"] is None else (old - st["logp_behav"]).exp().clamp(max=hyp["tis_cap"])
    plain = rho * st["adv"]
    clipped = rho.clamp(1 - hyp["eps_lo"], 1 + hyp["eps_hi"]) * st["adv"]
    dlp = torch.where(plain > clipped, torch.zeros_like(rho), -w * plain)
    if st["logp_ref"] is not None:
        dlp = dlp - hyp["kl_beta"] * torch.expm1(st["logp_ref"] - lp)
    dz = (dlp * st["weight"] / TEMPERATURE)[:, None]
    return (e * (-dz / total)).scatter_add_(1, t, dz)


MISTAKES = {
    "last logit left out": lambda d: torch.cat((d[:, :-1], torch.zeros_like(d[:, :1])), 1),
    "second half left out": lambda d: torch.cat((d[:, :d.shape[1] // 2], 0 * d[:, d.shape[1] // 2:]), 1),
    "2% too large": lambda d: 1.02 * d,
    "one column off": lambda d: d.roll(1, 1),
    "sign": lambda d: -d,
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(40, 7), (40, 1001), (6, 32001), (4, 151936)])
def test_bounds(T, V, dtype):
    st = A.loss_inputs(T, V, dtype, T + V)
    d = formula(st)
    B.check_gradient(st, d.to(dtype), TEMPERATURE)
    for what, mistake in MISTAKES.items():
        with pytest.raises(AssertionError, match="gradients off"):
            B.check_gradient(st, mistake(d).to(dtype), TEMPERATURE)
            pytest.fail(f"{what}: not seen")
