"""GPU tests of FP8 groups whose largest value is so small that its 448th part rounds to
zero: codes stay numbers, and what they stand for stays within the smallest positive one."""
import pytest
import torch

import actor_ref as R
from actor_ref import D
from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_actor import DEV, gate_reference, gen, norm_reference, normal

pytestmark = pytest.mark.gpu

# a product rounds to a multiple of 2^-149; a scale is at least 2^-149, which 448 codes
# can count (a code's own half step of it is in the checks' subnormal term)
TINY = 448 * 2.0 ** -149


@pytest.mark.parametrize("M", [1, 9, 200])
def test_add_rmsnorm(M):
    """Weights of the smallest bf16 number, and a stream far below eps: x down to 2^-149 and
    to zeros between them."""
    g = gen(M)
    K = 384
    h = normal(g, M, K)
    h[::2] *= 2.0 ** -21
    h[:, ::3] = 0
    gamma = torch.full((K,), 2.0 ** -133, device=DEV).to(torch.bfloat16)
    assert float(gamma[0]) > 0
    _, q, s, qT, sc, _ = rlq.add_rmsnorm_quant_act_1x128(h, None, gamma, 1e-6, colwise=True)
    _, x, _, err = norm_reference(h, gamma, 1e-6)
    assert 0 < float(x[0].abs().amax()) < 448 * 2.0 ** -150
    R.check_rows(q, s, x, err + TINY, "rows")
    R.check_cols(qT, sc, x, err + TINY, "columns")
    assert bool((s > 0).all()) and bool((sc > 0).all())
    # in the even rows 2^-149 is the scale, and a code the value in units of it: off by the
    # product's half unit and half a code's step
    x, got = x[::2], (R.decode(q) * R.rows_scale(s, K))[::2]
    assert bool((s[:, ::2] == 2.0 ** -149).all())
    unit = 2.0 ** -150
    assert bool(((got - x).abs() <= unit + (x.abs() + unit) * 2.0 ** -4 + err[::2] + 2.0 ** -159).all())


@pytest.mark.parametrize("M", [1, 130, 300])
def test_gated_backward(M):
    """Gradients of the smallest bf16 number through nearly closed gates."""
    g = gen(M)
    F = 256
    gu = normal(g, M, 2 * F).float()
    gu[:, :128] = -6.0 - gu[:, :128].abs()
    gu[:, F:F + 128] *= 2.0 ** -9
    guq, gus = R.quant_rows(gu)
    da = torch.full((M, F), 2.0 ** -133, device=DEV).to(torch.bfloat16)
    da[:, ::5] = 0
    q, s, qT, sc, aT, ac = rlq.gated_backward(da, guq, gus)
    dg, du, a, edg, edu, ea = gate_reference(da, guq, gus)
    assert 0 < float(dg[:, :128].abs().amax()) < 448 * 2.0 ** -150
    # dg is three products deep: each may round to the smallest step, times at most 8
    d, e = torch.cat((dg, du), 1), torch.cat((edg, edu), 1) + TINY + 24 * 2.0 ** -149
    R.check_rows(q, s, d, e, "rows")
    R.check_cols(qT, sc, d, e, "columns")
    R.check_cols(aT, ac, a, ea, "a's columns")
    assert bool((s > 0).all()) and bool((sc > 0).all())


@pytest.mark.parametrize("M", [1, 8, 40, 300])  # the few-token kernel, single CTAs, CTA pairs
def test_gated_fprop(M):
    """Projections of about 2^-145, and their product far below: from activations and
    weights whose scales are themselves tiny."""
    g = gen(M + 50)
    F, K = 256, 256
    xq, xs = R.quant_rows(normal(g, M, K))
    wq, ws = R.quant_blocks(normal(g, 2 * F, K, std=0.05))
    ws[1] *= 2.0 ** -140  # the second 128 gate columns
    ws[3] *= 2.0 ** -10   # and the up projection's beside them
    ws[1] = torch.where(ws[1] == 0, torch.full_like(ws[1], 2.0 ** -149), ws[1])
    aq, as_, guq, gus = rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=True)
    rlq.check()
    assert bool((R.decode(aq).abs() <= 448).all()) and bool((R.decode(guq).abs() <= 448).all())
    assert bool((as_ > 0).all()) and bool((gus > 0).all())
    assert float((R.decode(aq)[:, 128:].abs() * as_[1][:, None].to(D)).amax()) < 2.0 ** -120
