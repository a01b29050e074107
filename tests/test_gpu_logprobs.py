"""GPU tests of the token log probabilities with entropy and alternatives, and of their gradient,
against the formulas in 64 bits."""
import math

import pytest
import torch

import mx_ref as R
from fp8_block_scaled_quantize_gb300 import rlq

pytestmark = pytest.mark.gpu
D = torch.float64
DEV = "cuda"
U = 2.0 ** -24  # half an fp32 step, relative
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def logits_of(g, T, V, dtype, std=2.0, ld=None):
    buf = torch.randn(T, ld or V, generator=g, device=DEV).mul_(std).to(DTYPES[dtype])
    return buf[:, :V], torch.randint(0, V, (T,), generator=g, device=DEV)


def fp32(temperature):
    """The temperature as the calls take it."""
    return float(torch.tensor(temperature, dtype=torch.float32))


def reference(x, targets, top, temperature):
    z = x.to(D) / fp32(temperature)
    # (from the maximum: next to a logit of 1e38 a log-sum is nothing in 64 bits either)
    m = z.amax(1)
    log_s = torch.logsumexp(z - m[:, None], 1)
    lse = m + log_s
    lg = (z - m[:, None]) - log_s[:, None]
    p = lg.exp()
    H = -torch.where(p == 0, torch.zeros_like(p), p * lg).sum(1)
    ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top]
    return lg.gather(1, targets[:, None])[:, 0], lse, H, ids, lg.gather(1, ids)


def forward_bounds(x, targets, temperature):
    """Bounds of lse, lp and H.  t = (z - max) log2(e) is three roundings off; a sum is a chain of
    at most V / 512 + 8 additions a thread, some 40 more to join them, and 2 ulp an exponential:
    S is then within r of itself, W = sum e t within r and the exponents' part."""
    z = x.to(D) / temperature
    V = x.shape[1]
    top = z.amax(1, keepdim=True)
    d = (top - z)
    p = torch.softmax(z, 1)
    d1, d2 = (torch.where(p == 0, torch.zeros_like(p), p * d ** k).sum(1) for k in (1, 2))
    chain = (V / 512 + 8 + 48) * U
    log_s = 3 * U * d1 + chain
    lse = log_s + 4 * U * (top[:, 0].abs() + math.log(V))
    dt = d.gather(1, targets[:, None])[:, 0]
    lp = log_s + 4 * U * (dt + math.log(V))
    H = log_s + 4 * U * math.log(V) + d1 * (2 * chain + 8 * U) + 3 * U * (d2 + d1)
    return lse, lp, H, log_s + 4 * U * math.log(V)


def check_forward(x, targets, top, temperature, got, rows=slice(None)):
    lp, lse, H, ids, top_lp = (t[rows] for t in got)
    x, targets = x[rows], targets[rows]
    want = reference(x, targets, top, temperature)
    b_lse, b_lp, b_H, b_s = forward_bounds(x, targets, temperature)
    assert torch.equal(ids, want[3])
    for name, a, b, tol in (("lse", lse, want[1], b_lse), ("lp", lp, want[0], b_lp), ("H", H, want[2], b_H)):
        same = a.to(D) == b  # infinities
        off = (a.to(D) - b).abs()
        assert bool((same | (off <= tol)).all()), f"{name}: {float((off / tol)[~same].max()):.2f} of the bound"
    if top:
        dt = (x.to(D).amax(1, keepdim=True) - x.to(D).gather(1, ids)) / temperature
        tol = b_s[:, None] + 4 * U * dt
        # (equal infinities; a value beyond fp32's range is one)
        assert bool(((top_lp == want[4].float()) | ((top_lp.to(D) - want[4]).abs() <= tol)).all())
    assert bool((H >= 0).all())


CASES = [(1, 1, 1), (1, 2, 2), (3, 7, 3), (2, 64, 64), (5, 100, 5), (2, 255, 20), (1, 1000, 64), (300, 513, 4),
         (7, 4097, 20), (64, 32001, 20), (700, 2048, 10), (1, 151936, 20), (40, 128256, 64), (5, 128256, 0), (700, 33000, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", CASES)
def test_forward(T, V, top, dtype):
    g = gen(T + V)
    x, targets = logits_of(g, T, V, dtype)
    got = rlq.token_logprobs_top(x, targets, top=top, temperature=0.8)
    assert got[3].shape == (T, top) and got[3].dtype == torch.int64 and got[4].shape == (T, top)
    check_forward(x, targets, top, 0.8, got)
    # the call without alternatives: lp and lse of the same kind
    lp, lse = rlq.token_logprobs(x, targets, temperature=0.8)
    b_lse, b_lp, _, _ = forward_bounds(x, targets, 0.8)
    assert bool(((lp.to(D) - got[0].to(D)).abs() <= 2 * b_lp).all())
    assert bool(((lse.to(D) - got[1].to(D)).abs() <= 2 * b_lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ld,shift", [(1001, 0), (1007, 3), (1024, 1)])
def test_forward_rows_off_16_bytes(dtype, ld, shift):
    g = gen(ld)
    T, V = 9, 1000
    x = torch.randn(T * ld + shift, generator=g, device=DEV).mul_(3).to(DTYPES[dtype])[shift:].as_strided((T, V), (ld, 1))
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    check_forward(x, targets, 17, 1.3, rlq.token_logprobs_top(x, targets, top=17, temperature=1.3))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(6, 700), (6, 128256), (700, 9000)])
def test_forward_masks_and_ties(dtype, T, V):
    """Rows with few tokens left, with none, with ties of every extent, with the type's lowest value as a mask."""
    g = gen(V)
    x, targets = logits_of(g, T, V, dtype)
    x[0] = 0.25  # every token alike
    x[1] = -math.inf
    x[1, targets[1]] = 1.0
    x[2] = -math.inf
    x[2, [5, V // 2, V - 1]] = torch.tensor([1.0, 2.0, 1.0], dtype=x.dtype, device=DEV)
    targets[2] = V // 2
    x[3] = -math.inf  # nothing left
    x[4] = torch.randint(0, 3, (V,), generator=g, device=DEV).to(x.dtype)  # thousands alike
    x[5] = torch.where(torch.rand(V, generator=g, device=DEV) < 0.01, x[5], torch.finfo(x.dtype).min)
    x[5, targets[5]] = 3.0
    for top in (20, 64):
        got = rlq.token_logprobs_top(x, targets, top=top)
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[3] = False
        check_forward(x, targets, top, 1.0, got, keep)
        lp, lse, H, ids, top_lp = got
        assert float(lp[3]) == -math.inf and float(lse[3]) == -math.inf and float(H[3]) == 0
        assert torch.equal(ids[3], torch.arange(top, device=DEV)) and bool((top_lp[3] == -math.inf).all())
        assert abs(float(H[0]) - math.log(V)) <= 1e-5 * math.log(V)
        assert float(H[1]) == 0 and float(lp[1]) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_lists_that_overflow(dtype):
    """Thousands of candidates: equal maxima in every thread; all finite logits in the units of few
    threads; and zeros of both signs, which are equal."""
    g = gen(77)
    T, V = 600, 40000  # (a CTA a row)
    x, targets = logits_of(g, T, V, dtype)
    x[0, ::13] = 50.0
    x[1, 1::7] = 50.0
    x[1, 30000] = 51.0
    x[1, 39999] = 52.0
    n = 8 if dtype == "bf16" else 4
    far = torch.arange(V, device=DEV) // n % 256 >= 5
    x[2, far] = -math.inf
    targets[2] = 0
    x[3, far] = -1000.0
    x[4] = torch.where(torch.rand(V, generator=g, device=DEV) < 0.5, -0.0, 0.0).to(x.dtype)
    x[5] = torch.where(torch.rand(V, generator=g, device=DEV) < 0.5, -0.0, -1.0).to(x.dtype)
    x[6] = torch.linspace(0, 5, V, device=DEV).to(x.dtype)  # in order, and
    x[7] = torch.linspace(5, 0, V, device=DEV).to(x.dtype)  # against it
    for top in (1, 20, 64):
        check_forward(x, targets, top, 1.0, rlq.token_logprobs_top(x, targets, top=top))


def test_forward_empty_rows_and_values_that_are_no_numbers():
    g = gen(3)
    x, targets = logits_of(g, 8, 5000, "f32")
    targets[1], targets[2] = -1, 5000
    x[1], x[2] = float("nan"), float("inf")  # not read
    x[4, 77] = float("nan")
    x[5, 78] = float("inf")
    x[6] = float("nan")
    lp, lse, H, ids, top_lp = rlq.token_logprobs_top(x, targets, top=6)
    for r in (1, 2):
        assert not lp[r] and not lse[r] and not H[r] and (ids[r] == -1).all() and not top_lp[r].any()
    for r in (4, 5, 6):
        assert bool(torch.isnan(torch.stack((lp[r], lse[r], H[r]))).all())
    fine = torch.tensor([0, 3, 7], device=DEV)
    check_forward(x, targets, 6, 1.0, (lp, lse, H, ids, top_lp), fine)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_rows_of_masks_only(dtype):
    """Masks that are numbers: a row of nothing else is uniform, with -inf beside them too."""
    V = 5000
    x = torch.zeros(4, V, dtype=DTYPES[dtype], device=DEV)
    x[0] = torch.finfo(x.dtype).min
    x[1] = -1e9
    x[2] = torch.finfo(x.dtype).min
    x[2, ::2] = -math.inf
    x[3] = torch.finfo(x.dtype).max
    targets = torch.full((4,), 7, device=DEV)
    got = rlq.token_logprobs_top(x, targets, top=5)
    check_forward(x, targets, 5, 1.0, got)
    n = torch.tensor([V, V, V / 2, V], device=DEV)
    assert bool(((got[2] - n.log()).abs() <= 1e-5).all())
    # the gradient's probabilities are uniform too, although the lse holds no log V next to 1e9
    one = torch.ones(4, device=DEV)
    d = rlq.token_logprobs_backward(x, targets, got[1], got[2], dlp=one, dentropy=one)
    want, tol = gradient_of_rows(x, targets, got[2], one, one, 1.0)
    assert bool(((d.to(D) - want).abs() <= tol).all())


def test_forward_far_offsets():
    """Rows beyond 2^31 elements from the first one."""
    ld, V, T = (1 << 30) + 8, 3000, 4
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((T, V), (ld, 1))
    x.copy_(torch.randn(T, V, generator=gen(2), device=DEV) * 2)
    targets = torch.tensor([1, 2, 3, 2999], device=DEV)
    got = rlq.token_logprobs_top(x, targets, top=20)
    check_forward(x, targets, 20, 1.0, got)
    want = rlq.token_logprobs_backward(x.contiguous(), targets, got[1], got[2], dlp=got[0], dentropy=got[2])
    d = rlq.token_logprobs_backward(x, targets, got[1], got[2], dlp=got[0], dentropy=got[2], inplace=True)
    assert d is x and torch.equal(x, want)


# ---------------------------------------------------------------- gradient ---

def gradient(x, targets, lse, H, dlp, dH, temperature):
    """The gradient in 64 bits from the given lse and H, and its bound."""
    c = 1 / fp32(temperature)
    z = x.to(D) * c
    lg = z - lse.to(D)[:, None]
    p = lg.exp()
    lg = torch.where(p == 0, torch.zeros_like(lg), lg)
    zero = torch.zeros(len(lse), 1, dtype=D, device=x.device)
    a = (zero if dlp is None else dlp.to(D)[:, None])
    h = (zero if dH is None else dH.to(D)[:, None])
    Hc = zero if H is None else H.to(D)[:, None]
    d = -p * (a + h * (lg + Hc)) * c
    at = torch.zeros_like(p).scatter_(1, targets[:, None], 1.0) * a * c
    # log2 p: two roundings of the result, and c and L as sums of two floats 2^-48 off; the
    # exponential 2 ulp; four roundings behind
    # (a logit of -inf has p = 0, and p times its part of the bound is 0: not 0 x inf)
    far = torch.where(p == 0, torch.zeros_like(p), (z.abs() + lse.to(D).abs()[:, None]) * 1.4427)
    t = lg.abs() * 1.4427
    err_t = 4 * U * t + 8 * U * U * far
    size = (a.abs() + h.abs() * (lg.abs() + Hc.abs())) * c
    tol = p * (size * (0.7 * err_t + 12 * U) + h.abs() * c * 0.7 * err_t) + 4 * U * at.abs()
    # probabilities below 2^-126 are zero
    tol = tol + 2.0 ** -125 * (a.abs() + h.abs() * (100 + Hc.abs())) * c
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -23
    return d + at, tol + half * ((d + at).abs() + tol) + 2.0 ** -133


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(1, 1), (2, 9), (3, 100), (5, 2048), (3, 16385), (50, 32001), (4, 151936), (600, 4000)])
@pytest.mark.parametrize("which", ["both", "lp", "entropy"])
def test_gradient(T, V, dtype, which):
    g = gen(T * V)
    x, targets = logits_of(g, T, V, dtype)
    if V > 50:
        x[0, 7::3] = -math.inf
        x[0, targets[0]] = 0.5
    temperature = 0.7
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets, temperature=temperature)
    dlp = torch.randn(T, generator=g, device=DEV) if which != "entropy" else None
    dH = torch.randn(T, generator=g, device=DEV) * 0.1 if which != "lp" else None
    if T > 2:
        for v in (dlp, dH):
            if v is not None:
                v[1] = 0  # an empty row
    d = rlq.token_logprobs_backward(x, targets, lse, H if dH is not None else None, dlp=dlp, dentropy=dH, temperature=temperature)
    want, tol = gradient(x, targets, lse, H, dlp, dH, temperature)
    off = (d.to(D) - want).abs()
    assert bool((off <= tol).all()), f"{float((off / tol).max()):.2f} of the bound"
    if T > 2:
        assert not d[1].any()
    # in place, and rows that share no 16-byte phase: the same bits
    y = x.clone()
    assert rlq.token_logprobs_backward(y, targets, lse, H, dlp=dlp, dentropy=dH, temperature=temperature, inplace=True) is y
    assert torch.equal(y, d)
    far = torch.full((T, V + 3), 9.0, dtype=x.dtype, device=DEV)
    rlq.rlq_token_logprobs_backward(x.data_ptr(), 0 if dtype == "bf16" else 1, max(x.stride(0), V), T, V, targets.data_ptr(),
                                    temperature, lse.data_ptr(), H.data_ptr(), dlp.data_ptr() if dlp is not None else None,
                                    dH.data_ptr() if dH is not None else None, far.data_ptr(), V + 3,
                                    torch.cuda.current_stream().cuda_stream)
    assert torch.equal(far[:, :V], d) and bool((far[:, V:] == 9).all())


@pytest.mark.parametrize("dtype,V,top", [("bf16", 64, 64), ("bf16", 115, 64), ("bf16", 249, 33), ("f32", 64, 64), ("f32", 130, 50),
                                         ("bf16", 700, 64), ("f32", 40000, 64)])
def test_empty_rows_have_every_alternative_empty(dtype, V, top):
    """Also where a short row has fewer threads than alternatives."""
    g = gen(52)
    x, targets = logits_of(g, 6, V, dtype)
    targets[::2] = torch.tensor([-1, V, -100], device=DEV)
    for _ in range(2):  # (what an output's memory held before is not what is found there)
        junk = [torch.full((6, top), 77, dtype=torch.int64, device=DEV), torch.full((6, top), 77.0, device=DEV)]
        del junk
        lp, lse, H, ids, top_lp = rlq.token_logprobs_top(x, targets, top=top)
        assert bool((ids[::2] == -1).all()) and not top_lp[::2].any()
        assert not lp[::2].any() and not lse[::2].any() and not H[::2].any()
        assert torch.equal(ids[1::2], torch.sort(x.float(), dim=1, descending=True, stable=True)[1][1::2, :top])


@pytest.mark.parametrize("dtype,left,V,ld", [("bf16", 0, 1000, 4096), ("bf16", 3, 1001, 4099), ("f32", 1, 37, 2050)])
def test_gradient_of_a_part_of_wide_rows(dtype, left, V, ld):
    """The gradient's rows are no wider than their phases need, and the columns beside the part are not read."""
    g = gen(51)
    T = 9
    wide = torch.full((T, ld), float("nan"), dtype=DTYPES[dtype], device=DEV)
    x = wide[:, left:left + V]
    x.copy_(torch.randn(T, V, generator=g, device=DEV) * 3)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    a, h = torch.randn(T, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV)
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets)
    d = rlq.token_logprobs_backward(x, targets, lse, H, dlp=a, dentropy=h)
    n = 16 // x.element_size()
    assert d.shape == x.shape and d.stride(1) == 1
    assert V <= d.stride(0) < V + n and (d.stride(0) - ld) % n == 0
    want, tol = gradient(x, targets, lse, H, a, h, 1.0)
    assert bool(((d.to(D) - want).abs() <= tol).all())
    y = x.contiguous()
    assert torch.equal(rlq.token_logprobs_backward(y, targets, lse, H, dlp=a, dentropy=h), d)


def gradient_of_rows(x, targets, H, dlp, dH, temperature):
    """The gradient in 64 bits from the rows' own sums (H as given), and the bound where the kernel forms them."""
    c = 1 / fp32(temperature)
    V = x.shape[1]
    m = x.to(D).amax(1, keepdim=True).clamp(min=-3.5e38)
    z = (x.to(D) - m) * c
    lg = z - z.exp().sum(1, keepdim=True).log()
    p = lg.exp()
    lg = torch.where(p < 2.0 ** -200, torch.zeros_like(lg), lg)
    a, h, Hc = dlp.to(D)[:, None], dH.to(D)[:, None], H.to(D)[:, None]
    at = torch.zeros_like(p).scatter_(1, targets[:, None], 1.0) * a * c
    d = at - p * (a + h * (lg + Hc)) * c
    # log2 p: the difference to the maximum, its product, the sum's logarithm and their sum; the sum: at
    # most V / 256 + 16 terms one after the other, 13 joined, each an exponential 2 ulp off
    t = lg.abs() * 1.4427
    err_t = 6 * U * t + 4 * U * math.log2(V + 1) + 1.4427 * (V / 256 + 35) * U
    size = (a.abs() + h.abs() * (lg.abs() + Hc.abs())) * c
    tol = p * (size * (0.7 * err_t + 12 * U) + h.abs() * c * 0.7 * err_t) + 4 * U * at.abs()
    tol = tol + 2.0 ** -125 * (a.abs() + h.abs() * (100 + Hc.abs())) * c
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -23
    return d, tol + half * (d.abs() + tol) + 2.0 ** -133


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,temperature", [(1, 1.0), (6, 0.3), (47, 0.3), (1000, 1.0), (5000, 0.3), (40000, 2.0), (40001, 0.3)])
def test_gradient_of_rows_far_from_zero(V, temperature, dtype):
    """Logits whose lse, or whose lse's logarithm of a sum, fp32 does not hold."""
    g = gen(53)
    T = 10
    x, targets = logits_of(g, T, V, dtype)
    low = torch.finfo(x.dtype).min
    x[0] = -1e9
    x[1] = low
    x[2, 1:] = low
    x[3] = torch.finfo(x.dtype).max
    x[4] = (x[4].float() + 1e6).to(x.dtype)
    x[5] *= 1e4
    x[6] = -1e9
    x[6, 1::2] = -math.inf
    x[7] -= 700
    x[8] = -math.inf
    targets[6] = 0
    a, h = torch.randn(T, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV) * 0.1
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets, temperature=temperature)
    d = rlq.token_logprobs_backward(x, targets, lse, H, dlp=a, dentropy=h, temperature=temperature)
    want, tol = gradient_of_rows(x, targets, H, a, h, temperature)
    rows = [r for r in range(T) if r != 8 and float(lse[r].abs()) > 256]
    off = (d.to(D) - want).abs()[rows]
    assert len(rows) >= 5 and bool((off <= tol[rows]).all())
    assert not d[8].any()
    y = x.clone()
    rlq.token_logprobs_backward(y, targets, lse, H, dlp=a, dentropy=h, temperature=temperature, inplace=True)
    assert torch.equal(y, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_takes_an_lse_that_is_not_the_rows(dtype):
    """A part of a vocabulary has the lse of the whole one, near to 0 or far from it."""
    g = gen(54)
    T, V = 5, 3000
    x, targets = logits_of(g, T, V, dtype)
    x[1] += 1000
    x[2] -= 1000
    a, h = torch.randn(T, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV) * 0.1
    _, lse, H, _, _ = rlq.token_logprobs_top(x, targets)
    for shift in (0.5, 3.0, 200.0):
        d = rlq.token_logprobs_backward(x, targets, lse + shift, H, dlp=a, dentropy=h)
        want, tol = gradient(x, targets, lse + shift, H, a, h, 1.0)
        assert bool(((d.to(D) - want).abs() <= tol).all())


def test_gradient_against_differences():
    """A loss of both outputs, differentiated numerically in 64 bits."""
    g = gen(50)
    T, V, temperature = 4, 300, 0.9
    x, targets = logits_of(g, T, V, "f32")
    a, h = torch.randn(T, generator=g, device=DEV), torch.randn(T, generator=g, device=DEV)

    def loss(x):
        lp, _, H, _, _ = reference(x, targets, 0, temperature)
        return a.to(D) * lp + h.to(D) * H

    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets, temperature=temperature)
    d = rlq.token_logprobs_backward(x, targets, lse, H, dlp=a, dentropy=h, temperature=temperature)
    step = 1e-5
    for v in torch.randint(0, V, (20,), generator=g, device=DEV).tolist() + targets.tolist():
        e = torch.zeros(T, V, dtype=D, device=DEV)
        e[:, v] = step
        diff = (loss(x.to(D) + e) - loss(x.to(D) - e)) / (2 * step)
        # the difference's own error: step^2 and 1e-16 / step
        assert bool(((d[:, v].to(D) - diff).abs() <= 2e-6 * (1 + diff.abs())).all())


def test_gradient_empty_rows_and_values_that_are_no_numbers():
    g = gen(8)
    x, targets = logits_of(g, 7, 3001, "bf16")
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets)
    one = torch.ones(7, device=DEV)
    a, h = one.clone(), 0.1 * one
    x[1] = float("nan")
    targets[1] = 3001
    x[2] = float("nan")
    a[2] = h[2] = 0  # not read
    x[3] = -math.inf
    lse[3], H[3] = -math.inf, 0
    lse[4] = float("nan")
    d = rlq.token_logprobs_backward(x, targets, lse, H, dlp=a, dentropy=h)
    assert not d[1:4].any() and bool(torch.isnan(d[4]).all())
    rows = torch.tensor([0, 5, 6], device=DEV)
    want, tol = gradient(x[rows], targets[rows], lse[rows], H[rows], a[rows], h[rows], 1.0)
    assert bool(((d[rows].to(D) - want).abs() <= tol).all())


def test_streams_and_graphs():
    g = gen(60)
    x, targets = logits_of(g, 48, 50000, "bf16")
    want = rlq.token_logprobs_top(x, targets, top=10)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rlq.token_logprobs_top(x, targets, top=10, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = rlq.token_logprobs_backward(x, targets, want[1], want[2], dlp=want[0], dentropy=want[2])
    static = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rlq.token_logprobs_top(static, targets, top=10)
        dg = rlq.token_logprobs_backward(static, targets, out[1], out[2], dlp=out[0], dentropy=out[2])
    static.copy_(x)
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(dg, d)


def test_nothing_to_do_and_refusals():
    x, targets = torch.zeros(0, 9, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    lp, lse, H, ids, top_lp = rlq.token_logprobs_top(x, targets, top=3)
    assert lp.shape == lse.shape == H.shape == (0,) and ids.shape == top_lp.shape == (0, 3)
    assert rlq.token_logprobs_backward(x, targets, lse, H, dlp=lp).shape == (0, 9)
    x, targets = torch.zeros(2, 100, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    assert rlq.token_logprobs_top(x[:, :5], targets, top=64)[3].shape == (2, 5)  # no more than there are
    for top in (-1, 65):
        with pytest.raises(rlq.RlqError):
            rlq.token_logprobs_top(x, targets, top=top)
    lp, lse, H, _, _ = rlq.token_logprobs_top(x, targets)
    with pytest.raises(rlq.RlqError):
        rlq.token_logprobs_backward(x, targets, lse, H)  # neither derivative
    with pytest.raises(rlq.RlqError):
        rlq.token_logprobs_backward(x, targets, lse, dentropy=lp)  # no entropy
    with pytest.raises(TypeError):
        rlq.token_logprobs_top(x, targets.int())
    with pytest.raises(ValueError):
        rlq.token_logprobs_backward(x, targets, lse[:1], H, dlp=lp)


def test_calls_on_two_streams_and_repeats():
    """Lists are filled in any order; what comes of them is the same every time."""
    g = gen(70)
    x, targets = logits_of(g, 96, 40000, "bf16")
    want = rlq.token_logprobs_top(x, targets, top=64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append(rlq.token_logprobs_top(x, targets, top=64))
        torch.cuda.synchronize()
        for per in got:
            assert all(torch.equal(a, b) for a, b in zip(per, want))


@pytest.mark.parametrize("temperature", [1e-3, 0.05, 50.0, 1e4])
def test_temperatures(temperature):
    """From nearly one token to nearly uniform, with a mask."""
    g = gen(71)
    x, targets = logits_of(g, 20, 3001, "f32")
    x[3, 100:] = -math.inf
    x[4, 5:] = torch.finfo(torch.float32).min
    targets[3:5] = 2
    got = rlq.token_logprobs_top(x, targets, top=7, temperature=temperature)
    check_forward(x, targets, 7, temperature, got)
    a, h = torch.randn(20, generator=g, device=DEV), torch.randn(20, generator=g, device=DEV)
    d = rlq.token_logprobs_backward(x, targets, got[1], got[2], dlp=a, dentropy=h, temperature=temperature)
    # (far from 0 the rows' own sums count, not the lse's rounding of them)
    far = (got[1].abs() > 256)[:, None]
    given, own = gradient(x, targets, got[1], got[2], a, h, temperature), gradient_of_rows(x, targets, got[2], a, h, temperature)
    want, tol = (torch.where(far, o, e) for o, e in zip(own, given))
    assert bool(((d.to(D) - want).abs() <= tol).all())


# ------------------------------------------------------------ the 4-bit head ---

def test_rollout_in_four_bits_and_its_gradient():
    """The operators together: hidden states quantized, the head's product, what is recorded of
    its logits, and a loss of log probabilities and entropy back through both products, against
    64-bit autograd on the values that the codes stand for."""
    g = gen(90)
    T, K, V = 70, 256, 1024
    h = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(V, K, generator=g, device=DEV) * 0.2).to(torch.bfloat16)
    hq, hs, hqT, hsT = rlq.quant_mxfp4(h, colwise=True)
    wq, ws, wqT, wsT = rlq.quant_mxfp4(w, colwise=True)
    logits = rlq.gemm_mxfp4(hq, hs, wq, ws, out_dtype=torch.float32)
    a, b = rlq.dequant_mxfp4(hq, hs).to(D), rlq.dequant_mxfp4(wq, ws).to(D)
    mag = a.abs() @ b.abs().t()
    assert bool(((logits.to(D) - a @ b.t()).abs() <= 12 * 2.0 ** -21 * mag).all())
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    lp, lse, H, ids, top_lp = rlq.token_logprobs_top(logits, targets, top=8, temperature=0.9)
    check_forward(logits, targets, 8, 0.9, (lp, lse, H, ids, top_lp))
    dlp, dH = -torch.ones(T, device=DEV) / T, -0.01 * torch.ones(T, device=DEV) / T
    z = logits.to(D).requires_grad_()
    lg = torch.log_softmax(z / 0.9, 1)
    ((lg.gather(1, targets[:, None])[:, 0] * dlp).sum() + (-(lg.exp() * lg).sum(1) * dH).sum()).backward()
    d = rlq.token_logprobs_backward(logits, targets, lse, H, dlp=dlp, dentropy=dH, temperature=0.9).to(torch.bfloat16)
    # bf16 rounding, and lse and H as the forward pass rounded them (below 1e-5)
    assert bool(((d.to(D) - z.grad).abs() <= 2.0 ** -8 * z.grad.abs() + 1e-5 / T).all())
    dq, ds, dqT, dsT = rlq.quant_mxfp4(d, colwise=True)
    dh = rlq.gemm_mxfp4(dq, ds, wqT, wsT).to(D)
    dw = rlq.gemm_mxfp4(dqT, dsT, hqT, hsT, out_dtype=torch.float32).to(D)
    val = lambda q, s, c: rlq.dequant_mxfp4(q, s, cols=c).to(D)  # noqa: E731
    want = val(dq, ds, V) @ val(wqT, wsT, V).t()
    assert bool(((dh - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5 * (val(dq, ds, V).abs() @ val(wqT, wsT, V).abs().t())).all())
    want = val(dqT, dsT, T) @ val(hqT, hsT, T).t()
    assert bool(((dw - want).abs() <= 1e-5 * (val(dqT, dsT, T).abs() @ val(hqT, hsT, T).abs().t())).all())
    assert R.untile(ds, T).shape[1] == V // 32
