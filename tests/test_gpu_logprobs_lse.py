"""GPU tests of the log-sum-exp that the forward pass records: how far it is rounded, and the gradient
that is formed from it."""
import math

import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_logprobs import D, DEV, DTYPES, U, forward_bounds, fp32, gen, gradient

pytestmark = pytest.mark.gpu


def half_ulp(x):
    """Half an fp32 step at 64-bit x."""
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 0.96, 0.93, 1.57, 0.06, 0.9, 3.0, 1e-30, 1e30])
def test_lse_of_one_logit_is_rounded_once(temperature, dtype):
    """A row of one logit: lse = x / temperature, nothing added.  The reciprocal is known to 2^-48 of
    itself and its low part's product is 2^-24 of the result, rounded: 2^-46 beside the last step's half."""
    g = gen(7)
    T = 4096
    x = torch.randn(T, 1, generator=g, device=DEV)
    x = (x * torch.exp2(torch.randint(-3, 12, (T, 1), generator=g, device=DEV).float())).to(DTYPES[dtype])
    targets = torch.zeros(T, dtype=torch.int64, device=DEV)
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets, temperature=temperature)
    want = x[:, 0].to(D) / fp32(temperature)
    tol = torch.maximum(half_ulp(want), half_ulp(lse.to(D))) + 2.0 ** -46 * want.abs()
    off = (lse.to(D) - want).abs()
    assert bool((off <= tol).all()), f"{float((off / tol).max()):.2f} of the bound"
    assert not lp.any() and not H.any()


@pytest.mark.parametrize("V", [2, 40, 600])
@pytest.mark.parametrize("temperature", [0.96, 0.93, 1.57, 0.9])
def test_gradient_of_rows_whose_lse_is_off_zero(temperature, V):
    """Rows with |lse| of 100 .. 256: their probabilities are off by the lse's last rounding, the sum's
    own error and what the gradient adds."""
    g = gen(V)
    T = 300
    shift = torch.linspace(100, 250, T, device=DEV) * temperature
    shift[1::2] *= -1
    x = torch.randn(T, V, generator=g, device=DEV) + shift[:, None]
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    a, h = torch.randn(T, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV) * 0.1
    _, lse, H, _, _ = rlq.token_logprobs_top(x, targets, temperature=temperature)
    d = rlq.token_logprobs_backward(x, targets, lse, H, dlp=a, dentropy=h, temperature=temperature)
    exact = torch.logsumexp(x.to(D) / fp32(temperature), 1)
    want, tol = gradient(x, targets, exact, H, a, h, temperature)
    _, _, _, sum_error = forward_bounds(x, targets, temperature)
    off_lse = torch.maximum(half_ulp(exact), half_ulp(lse.to(D))) + sum_error
    assert bool(((lse.to(D) - exact).abs() <= off_lse).all())
    lg = x.to(D) / fp32(temperature) - exact[:, None]
    size = a.to(D).abs()[:, None] + h.to(D).abs()[:, None] * (lg.abs() + H.to(D)[:, None] + 1)
    tol = tol + 1.01 * off_lse[:, None] * lg.exp() * size / fp32(temperature)
    rows = (lse.abs() >= 100) & (lse.abs() <= 256)
    assert int(rows.sum()) >= 250
    off = (d.to(D) - want).abs()
    assert bool((off <= tol)[rows].all()), f"{float((off / tol)[rows].max()):.2f} of the bound"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lse_beyond_fp32(dtype):
    """x / temperature out of fp32's range is an infinity of its sign, and a NaN only where the row has one."""
    big = torch.finfo(DTYPES[dtype]).max
    x = torch.tensor([[big, 0.0, -big], [-big, -big, -big], [-big, -math.inf, -big], [-math.inf] * 3, [math.inf, 0, 1],
                      [math.nan, big, 0], [1e3, 1e3, 0]], dtype=DTYPES[dtype], device=DEV)
    targets = torch.zeros(7, dtype=torch.int64, device=DEV)
    for temperature in (1e-30, 0.96, 0.93, 0.06, 1.2e-38):
        lse = rlq.token_logprobs_top(x, targets, temperature=temperature)[1]
        z = torch.logsumexp(x[[0, 1, 2, 6]].to(D) / fp32(temperature), 1)
        got = lse[[0, 1, 2, 6]]
        want = z.float()
        # (a chain of three terms: 4 U of z covers the last rounding, 1e-6 the sum's logarithm)
        assert bool(((got == want) | ((got.to(D) - z).abs() <= 4 * U * z.abs() + 1e-6)).all())
        assert float(lse[3]) == -math.inf and bool(torch.isnan(lse[4:6]).all())
