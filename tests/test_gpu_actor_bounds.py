"""GPU tests of the policy loss's gradient, element by element, with bounds in proportion to
each element, and of the residual norm's codes where everything is far below the normal range."""
import pytest
import torch

import actor_ref as R
from actor_bounds import check_gradient
from actor_ref import D
from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_actor import HYP, gen, loss_inputs, norm_reference, normal

pytestmark = pytest.mark.gpu


def gradient(st, temperature, inplace=False):
    return rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                           logp_behav=st["logp_behav"], logp_ref=st["logp_ref"], clip_hi=st["clip_hi"],
                           temperature=temperature, inplace=inplace, **HYP)[2]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pitch,offset", [(40, 7, 0, 0), (40, 8, 3, 1), (40, 1001, 0, 3), (9, 4096, 8, 0),
                                              (20, 32001, 0, 0), (20, 50257, 0, 5), (9, 70001, 6, 2), (7, 151936, 0, 0),
                                              (6, 262136, 0, 0), (700, 33001, 1, 3), (300, 100001, 0, 0)])
def test_gradient_of_every_logit(T, V, pitch, offset, dtype):
    for temperature in (0.9, 1.0):
        st = loss_inputs(T, V, dtype, T + V, pitch, offset, clip=temperature == 1.0)
        check_gradient(st, gradient(st, temperature), temperature)


@pytest.mark.parametrize("T,V", [(3, 524280), (2, 1200007)])
def test_gradient_of_long_rows(T, V):
    st = loss_inputs(T, V, torch.bfloat16, 4)
    st["weight"][:] = 1 / T
    check_gradient(st, gradient(st, 0.9), 0.9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pitch", [(12, 999, 1), (12, 40000, 1), (12, 140000, 1), (900, 5003, 0)])
def test_gradient_in_place(T, V, pitch, dtype):
    st = loss_inputs(T, V, dtype, V, pitch=pitch)
    before = st["logits"].clone()
    d = gradient(st, 0.9, inplace=True)
    assert d is st["logits"]
    check_gradient({**st, "logits": before}, d, 0.9)


def test_gradient_past_32_bits():
    T, V = 17003, 128256
    g = gen(13)
    logits = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    logits.normal_(0, 2, generator=g)
    assert T * V > 2 ** 31
    st = {"logits": logits, "targets": torch.randint(0, V, (T,), generator=g, device="cuda")}
    st["logp_old"] = rlq.token_logprobs(logits, st["targets"])[0] + 0.01
    st["adv"] = torch.randn(T, generator=g, device="cuda")
    st["weight"] = torch.ones(T, device="cuda")
    st.update(logp_behav=None, logp_ref=None, clip_hi=None)
    pick = torch.cat((torch.arange(6), torch.arange(T - 6, T))).cuda()
    few = {k: None if v is None else v[pick].clone() for k, v in st.items()}
    check_gradient(few, gradient(st, 1.0, inplace=True)[pick], 1.0)


@pytest.mark.parametrize("exponent", [-103, -112, -126, -131])
@pytest.mark.parametrize("add", [True, False])
def test_add_rmsnorm_far_below_the_normal_range(exponent, add):
    """Weights that put x between 2^-134 and 2^-100: scales from 2^-112 down to the last
    subnormals, on both groupings."""
    g = gen(200 - exponent)
    M, K = 140, 512
    res, delta = normal(g, M, K), normal(g, M, K, std=0.3)
    gamma = (torch.randn(K, generator=g, device="cuda").sign() * 2.0 ** exponent).to(torch.bfloat16)
    h, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(res, delta if add else None, gamma, 1e-6, colwise=True)
    assert torch.equal(h, (res.float() + delta.float()).to(torch.bfloat16) if add else res)
    r, x, rtol, err = norm_reference(h, gamma, 1e-6)
    assert bool(((rstd.to(D) - r).abs() <= rtol * r).all())
    assert 0 < float(x.abs().amax()) < 2.0 ** (exponent + 4)
    # a product and a scale each round to a multiple of 2^-149 at worst, a scale counting
    # for up to 448 of its codes
    err = err + 2.0 ** -150 + 448 * 2.0 ** -150
    R.check_rows(q, s, x, err, "rows")
    R.check_cols(qT, sc, x, err, "columns")


@pytest.mark.parametrize("std", [1e-30, 1e-18])
def test_add_rmsnorm_of_a_stream_of_almost_nothing(std):
    """h^2 far below eps: rstd is 1 / sqrt(eps), and x keeps h's relative size."""
    g = gen(17)
    h = normal(g, 60, 512, std=std)
    gamma = (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(torch.bfloat16)
    _, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(h, None, gamma, 1e-6, colwise=True)
    r, x, rtol, err = norm_reference(h, gamma, 1e-6)
    assert bool(((rstd.to(D) - r).abs() <= rtol * r).all())
    R.check_rows(q, s, x, err, "rows")
    R.check_cols(qT, sc, x, err, "columns")
