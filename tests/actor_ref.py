"""Plain 64-bit forms of the actor's feed-forward sublayer and loss, and the checks
of FP8 outputs against them (shared by the GPU tests; test infrastructure only)."""
import torch

D = torch.float64
U = 2.0 ** -24  # half an fp32 step, relative


def decode(codes):
    return codes.contiguous().view(torch.float8_e4m3fn).to(D)


def quant_rows(x):
    """uint8 1x128 codes of x [M, K] and scales [K/128, M] (fp32), by torch."""
    M, K = x.shape
    g = x.float().reshape(M, K // 128, 128)
    a = g.abs().amax(2)
    s = torch.where(a == 0, torch.ones_like(a), a / 448)
    return (g / s[:, :, None]).reshape(M, K).to(torch.float8_e4m3fn).view(torch.uint8), s.t().contiguous()


def quant_blocks(w):
    N, K = w.shape
    b = w.float().reshape(N // 128, 128, K // 128, 128)
    a = b.abs().amax((1, 3))
    s = torch.where(a == 0, torch.ones_like(a), a / 448)
    return (b / s[:, None, :, None]).reshape(N, K).to(torch.float8_e4m3fn).view(torch.uint8), s


def rows_scale(s, K):
    """[M, K] per-element scales of 1x128 scales s [K/128, M]."""
    return s.to(D).t().repeat_interleave(128, 1)[:, :K]


def check_groups(codes, scales, x, err, what):
    """codes [R, G, n] and scales [R, G] against groups x [R, G, n] that the kernel knows to
    within err (same shape, absolute).

    The scale is amax / 448 of values off by at most err (one more rounding for the
    division); a decoded value is within half an E4M3 step of a value off by at most
    err (2^-4 of it, or 2^-10 of the scale among the subnormals), plus the 2 ulp of the
    quotient; and only values within err of a rounding boundary may have another code
    than the exact quotient's, which the half step covers."""
    codes, scales = codes.to(D), scales.to(D)
    amax = x.abs().amax(2)
    slack = err.amax(2) + 2 * U * amax
    want = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
    off = (scales - want).abs()
    # (a group whose exact values are all below the error may round to all zeros: scale 1)
    bad = (off > slack / 448 * (1 + 4 * U)) & ~((amax <= slack) & (scales == 1))
    assert not bad.any(), f"{what}: {int(bad.sum())} scales off, worst {float((off / want).max()):.2e}"
    assert bool((codes.abs() <= 448).all()), f"{what}: a NaN code"
    got = codes * scales[:, :, None]
    tol = torch.maximum((x.abs() + err) * 2.0 ** -4, scales[:, :, None] * 2.0 ** -10) * (1 + 4 * U) + err + 4 * U * x.abs()
    # the largest value of a group saturates at 448 where the scale rounded down
    worst = ((got - x).abs() / tol.clamp(min=1e-300)).max()
    assert worst <= 1, f"{what}: a value is {float(worst):.3f} of the bound off"


def check_rows(q, s, x, err, what):
    """1x128 codes q [M, K] (uint8), scales s [K/128, M]."""
    M, K = x.shape
    sh = (M, K // 128, 128)
    check_groups(decode(q).reshape(sh), s.t(), x.reshape(sh), err.reshape(sh), what)


def check_cols(qT, sc, x, err, what):
    """128x1 codes qT [K, M] (uint8), scales sc [ceil(M/128), K]."""
    M, K = x.shape
    assert tuple(qT.shape) == (K, M) and tuple(sc.shape) == (-(-M // 128), K)
    q = decode(qT).t()
    for b, m in enumerate(range(0, M, 128)):
        e = slice(m, min(m + 128, M))
        check_groups(q[e].t()[:, None], sc[b][:, None], x[e].t()[:, None], err[e].t()[:, None], f"{what} block {b}")


def token_loss(lp, old, adv, weight, behav, ref, clip_hi, eps_lo, eps_hi, cap, beta):
    """Per-token loss, written for autograd in 64 bits."""
    rho = (lp - old).exp()
    w = torch.ones_like(old) if behav is None else (old - behav).exp().clamp(max=cap)
    hi = torch.full_like(old, 1 + eps_hi) if clip_hi is None else clip_hi
    loss = -w * torch.minimum(rho * adv, torch.minimum(rho.clamp(min=1 - eps_lo), hi) * adv)
    if ref is not None:
        d = ref - lp
        loss = loss + beta * (d.exp() - 1 - d)
    return weight * loss
