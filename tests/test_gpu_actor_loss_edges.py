"""GPU tests of the policy loss where a factor overflows in 32 bits and the term that it
belongs to does not count: the formula's value is finite, and so is the operator's."""
import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_actor import HYP, loss_inputs

pytestmark = pytest.mark.gpu


def call(st, **hyp):
    return rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                           logp_behav=st["logp_behav"], logp_ref=st["logp_ref"], **{**HYP, **hyp})


@pytest.mark.parametrize("V", [500, 40001])
def test_no_advantage_and_a_ratio_that_overflows(V):
    """An advantage of 0 times exp(lp - lp_old) beyond the type's range is 0, as for any
    other ratio; the KL term stays.  An infinite or NaN lp_old stays what the formula makes of it."""
    st = loss_inputs(6, V, torch.bfloat16, 3)
    st["weight"][:] = 1 / 6
    st["logp_behav"] = None
    st["adv"][1:4] = 0
    want = call(st)
    for r in (1, 2, 3):
        st["logp_old"][r] = (-200.0, -1e4, -3e38)[r - 1]
    got = call(st)
    for a, b in zip(got, want):  # without an advantage the old probability does not matter
        assert torch.equal(a, b)
    st["logp_old"][2] = float("nan")
    assert bool(torch.isnan(call(st)[0][2]))


@pytest.mark.parametrize("V", [500, 40001])
def test_no_kl_weight_and_a_reference_far_above(V):
    """kl_beta = 0 switches the KL term off whatever exp(lp_ref - lp) is, a target of
    probability 0 included; a NaN in lp_ref is still seen."""
    st = loss_inputs(6, V, torch.bfloat16, 5)
    st["weight"][:] = 1 / 6
    st["logits"][4, st["targets"][4]] = float("-inf")
    st["logp_ref"][:] = 500.0
    got = call(st, kl_beta=0.0)
    st["logp_ref"] = None
    for a, b in zip(got, call(st)):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isfinite(got[2]).all())
    st["logp_ref"] = torch.full((6,), float("nan"), device="cuda")
    assert bool(torch.isnan(call(st, kl_beta=0.0)[0]).all())
