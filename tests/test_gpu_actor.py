"""GPU tests of the residual norm, the gated feed-forward block, its backward pass and
the policy loss against plain forms in 64 bits."""
import math

import pytest
import torch

import actor_ref as R
from actor_ref import D, U
from fp8_block_scaled_quantize_gb300 import rlq

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def pitched(t, extra):
    """The same values in rows of a longer pitch."""
    buf = torch.zeros((t.shape[0], t.shape[1] + extra), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


# ------------------------------------------------------------------ norm ---

def norm_reference(h, gamma, eps):
    f = h.to(D)
    rstd = 1 / (f.square().mean(1) + eps).sqrt()
    x = f * rstd[:, None] * gamma.to(D)
    # the sum of squares is a chain of at most 64 fp32 additions and two trees (errors
    # halved by the root), then the mean, eps, the root, the reciprocal: rstd within
    # 48 half-steps; two more products for x
    return rstd, x, 48 * U, 50 * U * x.abs()


@pytest.mark.parametrize("M,K,pitch", [(1, 128, 0), (1, 4096, 0), (3, 1152, 8), (130, 384, 16), (257, 5120, 0),
                                       (200, 8192, 0), (160, 8320, 0), (170, 16384, 0), (1, 16384, 0), (128, 256, 0)])
@pytest.mark.parametrize("add", [True, False])
def test_add_rmsnorm(M, K, pitch, add):
    g = gen(M * 7 + K)
    res = normal(g, M, K)
    res[:, :: 97] *= 20
    if M > 2:
        res[1] = 0  # a row of zeros
    delta = normal(g, M, K, std=0.3) if add else None
    if add and M > 2:
        delta[1] = 0
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    if pitch:
        res, delta = pitched(res, pitch), (pitched(delta, 2 * pitch) if add else None)
    h, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(res, delta, gamma, 1e-6, colwise=True)
    want = (res.float() + delta.float()).to(torch.bfloat16) if add else res
    assert torch.equal(h, want)
    r, x, rtol, err = norm_reference(h, gamma, 1e-6)
    assert bool(((rstd.to(D) - r).abs() <= rtol * r).all())
    R.check_rows(q, s, x, err, "rows")
    R.check_cols(qT, sc, x, err, "columns")
    # without the columns: the same bits; in place: the same bits
    h2, q2, s2, _, _, r2 = rlq.add_rmsnorm_quant_act_1x128(res, delta, gamma, 1e-6)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(rstd, r2)
    rc = res.clone()
    h3, q3, s3, qT3, sc3, _ = rlq.add_rmsnorm_quant_act_1x128(rc, delta, gamma, 1e-6, colwise=True, inplace=True)
    assert h3 is rc and torch.equal(h3, want) and torch.equal(q, q3) and torch.equal(qT, qT3) and torch.equal(sc, sc3)


def test_add_rmsnorm_tiny_and_large_values():
    g = gen(5)
    for scale in (1e-30, 1e15):
        h = normal(g, 40, 512, std=scale)
        gamma = normal(g, 512, std=1e-32 if scale < 1 else 1.0)
        _, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(h, None, gamma, 0.0 if scale > 1 else 1e-6, colwise=True)
        r, x, _, err = norm_reference(h, gamma, 0.0 if scale > 1 else 1e-6)
        # scales far below the normal range are rounded to a multiple of 2^-149
        err = err + (2.0 ** -148 * 448 if scale < 1 else 0.0)
        keep = x.abs().amax() > 2.0 ** -120
        if keep:
            R.check_rows(q, s, x, err, "rows")
            R.check_cols(qT, sc, x, err, "columns")
        else:
            assert bool((R.decode(q).abs() <= 448).all())


def test_scales_and_codes_are_the_rule_of_the_values():
    """From the kernel's own rstd the fp32 values are known bit for bit: every scale is the
    IEEE quotient of its group's maximum, every code that of value * RN(1 / scale)."""
    g = gen(31)
    M, K = 1031, 4096
    h = normal(g, M, K)
    h[::7] *= torch.exp2(torch.randint(-20, 20, (h[::7].shape[0], 1), generator=g, device=DEV)).to(torch.bfloat16)
    # weights from 2^-126 to 2^60: scales from far below the normal range's end to large ones
    step = torch.linspace(-126, 60, K // 128, device=DEV).round().repeat_interleave(128)
    gamma = (torch.randn(K, generator=g, device=DEV).sign() * (1 + torch.rand(K, generator=g, device=DEV)) *
             torch.exp2(step)).to(torch.bfloat16)
    _, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(h, None, gamma, 1e-6, colwise=True)
    h, gamma, rstd = h.cpu().float(), gamma.cpu().float(), rstd.cpu()
    x = (h * rstd[:, None]) * gamma

    def rule(x, dim):  # x with its groups along dim: scales, codes
        amax = x.abs().amax(dim, keepdim=True)
        s = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
        pre = torch.where(s < 2.0 ** -100, torch.full_like(s, 2.0 ** 64), torch.ones_like(s))
        v = (x * pre) * (1 / (s * pre))
        return s, v.clamp(-448, 448).to(torch.float8_e4m3fn)

    ws, wq = rule(x.view(M, K // 128, 128), 2)
    assert torch.equal(s.cpu(), ws[:, :, 0].t())
    assert torch.equal(q.cpu(), wq.view(M, K).view(torch.uint8))
    xp = torch.nn.functional.pad(x, (0, 0, 0, -M % 128))
    ws, wq = rule(xp.view(-1, 128, K), 1)
    assert torch.equal(sc.cpu(), ws[:, 0])
    assert torch.equal(qT.cpu(), wq.view(-1, K)[:M].t().contiguous().view(torch.uint8))


def norm_bwd_reference(dx, h, rstd, gamma, dres):
    dx, xh, g, r = dx.to(D), h.to(D) * rstd.to(D)[:, None], gamma.to(D), rstd.to(D)[:, None]
    K = dx.shape[1]
    c = (dx * g * xh).mean(1, keepdim=True)
    cerr = (dx * g * xh).abs().mean(1, keepdim=True) * 80 * U  # products, a chain of 32 and two trees
    body = dx * g - xh * c
    dh = r * body + (dres.to(D) if dres is not None else 0)
    mag = r * ((dx * g).abs() + (xh * c).abs())
    err = 8 * U * mag + r * xh.abs() * cerr + 2 * U * dh.abs()
    M = dx.shape[0]
    dgamma = (dx * xh).sum(0)
    gerr = (M + 24) * U * (dx * xh).abs().sum(0)
    return dh, err + 2.0 ** -8 * (dh.abs() + err), dgamma, gerr


@pytest.mark.parametrize("M,K", [(1, 128), (2, 256), (5, 4096), (153, 1152), (700, 640), (1300, 4096), (333, 8192),
                                 (161, 8320), (200, 16384)])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_backward(M, K, residual):
    g = gen(M + 3 * K)
    h, dx = normal(g, M, K), normal(g, M, K, std=1e-3)
    dres = pitched(normal(g, M, K, std=1e-3), 8) if residual else None
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dh, dgamma = rlq.rmsnorm_backward(dx, h, rstd, gamma, dres=dres)
    want, err, wg, gerr = norm_bwd_reference(dx, h, rstd, gamma, dres)
    assert bool(((dh.to(D) - want).abs() <= err).all())
    assert bool(((dgamma.to(D) - wg).abs() <= gerr).all())
    again = rlq.rmsnorm_backward(dx, h, rstd, gamma, dres=dres)
    assert torch.equal(dh, again[0]) and torch.equal(dgamma, again[1])
    if residual:
        d2, g2 = rlq.rmsnorm_backward(dx, h, rstd, gamma, dres=dres, inplace=True)
        assert d2 is dres and torch.equal(d2, dh) and torch.equal(g2, dgamma)


def test_rmsnorm_backward_against_differences():
    """Central differences of the 64-bit forward form, along random directions."""
    g = gen(11)
    M, K = 6, 256
    h, dx = normal(g, M, K), normal(g, M, K)
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    rstd = 1 / (h.to(D).square().mean(1) + 1e-6).sqrt()
    dh, dgamma = rlq.rmsnorm_backward(dx, h, rstd.float(), gamma)

    def f(hh, gg):
        return (hh * (hh.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gg * dx.to(D)).sum()

    for k in range(4):
        v, w = normal(g, M, K, dtype=D), normal(g, K, dtype=D)
        e = 1e-5
        dif = (f(h.to(D) + e * v, gamma.to(D)) - f(h.to(D) - e * v, gamma.to(D))) / (2 * e)
        got = (dh.to(D) * v).sum()
        # dh's rounding to bf16, each element's half step, and the differences' own error
        assert abs(float(got - dif)) <= float((2.0 ** -8 * dh.to(D).abs() * v.abs()).sum()) + 1e-6 * float(dif.abs() + 1)
        dif = (f(h.to(D), gamma.to(D) + e * w) - f(h.to(D), gamma.to(D) - e * w)) / (2 * e)
        assert abs(float((dgamma.to(D) * w).sum() - dif)) <= 1e-5 * float((dgamma.to(D) * w).abs().sum() + 1)


def test_rmsnorm_backward_no_rows():
    dh, dgamma = rlq.rmsnorm_backward(*(torch.zeros((0, 256), dtype=torch.bfloat16, device=DEV),) * 2,
                                      torch.zeros(0, device=DEV), torch.ones(256, dtype=torch.bfloat16, device=DEV))
    assert dh.shape == (0, 256) and bool((dgamma == 0).all())


# ----------------------------------------------------------- gated block ---

def gated_reference(xq, xs, wq, ws):
    """g, u in 64 bits and the error that fp32 accumulation allows each."""
    M, K = xq.shape
    F2 = wq.shape[0]
    x = R.decode(xq) * R.rows_scale(xs, K)
    w = R.decode(wq) * ws.to(D).repeat_interleave(128, 0).repeat_interleave(128, 1)
    gu = x @ w.t()
    # 128 products summed by the tensor cores (each addition within one fp32 step), the
    # block's scale product, one fused multiply-add per block
    err = (x.abs() @ w.abs().t()) * (2 * 128 + 4 + K // 128) * U
    return gu[:, :F2 // 2], gu[:, F2 // 2:], err[:, :F2 // 2], err[:, F2 // 2:]


@pytest.mark.parametrize("M,F,K", [(1, 128, 128), (1, 14336, 256), (2, 384, 1024), (5, 1280, 3584), (16, 256, 384),
                                   (17, 256, 384), (33, 640, 128), (64, 512, 2048), (127, 256, 640), (128, 128, 128),
                                   (200, 384, 512), (256, 256, 256), (300, 1152, 1024), (1000, 640, 384)])
@pytest.mark.parametrize("checkpoint", [False, True])
def test_gated_fprop(M, F, K, checkpoint):
    g = gen(M + F + K)
    xq, xs = R.quant_rows(normal(g, M, K))
    wq, ws = R.quant_blocks(normal(g, 2 * F, K, std=2.0 / math.sqrt(K)))
    aq, as_, guq, gus = rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=checkpoint)
    rlq.check()
    gg, u, eg, eu = gated_reference(xq, xs, wq, ws)
    sg = torch.sigmoid(gg)
    a = gg * sg * u
    # |silu'| <= 1.1; the sigmoid within 8 half-steps plus its argument's rounding
    err = 1.1 * eg * (u.abs() + eu) + (gg * sg).abs() * eu + (12 + gg.abs()) * U * a.abs()
    R.check_rows(aq, as_, a, err, "a")
    if checkpoint:
        R.check_rows(guq, gus, torch.cat((gg, u), 1), torch.cat((eg, eu), 1), "g and u")
    else:
        assert guq is None and gus is None
    again = rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=checkpoint)
    assert torch.equal(aq, again[0]) and torch.equal(as_, again[1])
    if checkpoint:  # the product does not depend on whether the checkpoint is kept
        plain = rlq.gemm_gated_fprop(xq, xs, wq, ws)
        assert torch.equal(aq, plain[0]) and torch.equal(as_, plain[1])


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_gated_fprop_extreme_gates(M):
    """Gates far from zero: silu is 0 below and the gate itself above; rows of zeros."""
    g = gen(M)
    F, K = 256, 256
    x = normal(g, M, K)
    if M > 2:
        x[2] = 0
    xq, xs = R.quant_rows(x)
    wq, ws = R.quant_blocks(torch.cat((normal(g, F, K, std=30.0), normal(g, F, K))))
    aq, as_, _, _ = rlq.gemm_gated_fprop(xq, xs, wq, ws)
    rlq.check()
    gg, u, eg, eu = gated_reference(xq, xs, wq, ws)
    assert float(gg.min()) < -200 and float(gg.max()) > 200
    a = gg * torch.sigmoid(gg) * u
    err = 1.1 * eg * (u.abs() + eu) + (gg * torch.sigmoid(gg)).abs() * eu + (12 + gg.abs()) * U * a.abs() + 1e-36
    R.check_rows(aq, as_, a, err, "a")
    if M > 2:
        assert bool((as_[:, 2] == 1).all()) and bool((R.decode(aq)[2] == 0).all())


def test_gated_fprop_pitches():
    """Operands and outputs as parts of wider buffers; what lies beside them stays."""
    g = gen(77)
    for M in (3, 70, 290):
        F, K = 384, 512
        xq, xs = R.quant_rows(normal(g, M, K))
        wq, ws = R.quant_blocks(normal(g, 2 * F, K, std=0.05))
        want = rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=True)
        xp, wp = pitched(xq, 16), pitched(wq, 48)
        xsp, wsp = pitched(xs, 3), pitched(ws, 1)
        aq = torch.full((M, F + 32), 7, dtype=torch.uint8, device=DEV)
        gu = torch.full((M, 2 * F + 16), 9, dtype=torch.uint8, device=DEV)
        as_, gus = torch.full((F // 128, M + 5), 3.0, device=DEV), torch.full((2 * F // 128, M + 1), 3.0, device=DEV)
        rlq.rlq_gemm_gated_fprop(xp.data_ptr(), K + 16, xsp.data_ptr(), M + 3, wp.data_ptr(), K + 48, wsp.data_ptr(),
                                 K // 128 + 1, aq.data_ptr(), F + 32, as_.data_ptr(), M + 5, gu.data_ptr(), 2 * F + 16,
                                 gus.data_ptr(), M + 1, M, F, K, torch.cuda.current_stream().cuda_stream)
        rlq.check()
        assert torch.equal(aq[:, :F], want[0]) and torch.equal(as_[:, :M], want[1])
        assert torch.equal(gu[:, :2 * F], want[2]) and torch.equal(gus[:, :M], want[3])
        assert bool((aq[:, F:] == 7).all()) and bool((gu[:, 2 * F:] == 9).all())
        assert bool((as_[:, M:] == 3).all()) and bool((gus[:, M:] == 3).all())


def gate_reference(da, guq, gus):
    M, F = da.shape
    gu = R.decode(guq) * R.rows_scale(gus, 2 * F)
    g, u, d = gu[:, :F], gu[:, F:], da.to(D)
    sg = torch.sigmoid(g)
    dg, du, a = d * u * sg * (1 + g * (1 - sg)), d * g * sg, g * sg * u
    # the sigmoid is within 8 half-steps plus its argument's rounding, relative; dg's last
    # factor is a sum of sg and g sg (1 - sg), each with that error
    rel = (16 + g.abs()) * U
    edg = rel * (d * u).abs() * (sg + 2 * (g * sg).abs())
    return dg, du, a, edg, rel * du.abs(), rel * a.abs()


@pytest.mark.parametrize("M,F", [(1, 128), (2, 1280), (16, 384), (127, 256), (128, 128), (129, 512), (333, 640),
                                 (1024, 256)])
def test_gated_backward(M, F):
    g = gen(M + F)
    guq, gus = R.quant_rows(normal(g, M, 2 * F, std=2.0))
    da = normal(g, M, F, std=1e-3)
    if M > 2:
        da[1] = 0
    q, s, qT, sc, aT, ac = rlq.gated_backward(pitched(da, 8), pitched(guq, 16), pitched(gus, 1))
    dg, du, a, edg, edu, ea = gate_reference(da, guq, gus)
    d, e = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    R.check_rows(q, s, d, e, "rows")
    R.check_cols(qT, sc, d, e, "columns")
    R.check_cols(aT, ac, a, ea, "a's columns")


def test_gated_backward_against_differences():
    """The decoded gradient against central differences of a = silu(g) u."""
    g = gen(3)
    M, F = 130, 256
    guq, gus = R.quant_rows(normal(g, M, 2 * F, std=2.0))
    da = normal(g, M, F)
    q, s, *_ = rlq.gated_backward(da, guq, gus)
    gu = R.decode(guq) * R.rows_scale(gus, 2 * F)

    def f(gu):
        return (torch.nn.functional.silu(gu[:, :F]) * gu[:, F:] * da.to(D)).sum()

    got = R.decode(q) * R.rows_scale(s, 2 * F)
    for _ in range(4):
        v = normal(g, M, 2 * F, dtype=D)
        dif = (f(gu + 1e-5 * v) - f(gu - 1e-5 * v)) / 2e-5
        # half an E4M3 step of each element, or of the group's scale among the subnormals
        step = torch.maximum(2.0 ** -4 / (1 - 2.0 ** -4) * got.abs(), 2.0 ** -10 * R.rows_scale(s, 2 * F))
        assert abs(float((got * v).sum() - dif)) <= float((step * v.abs()).sum())


# ------------------------------------------------------------------ loss ---

HYP = {"eps_lo": 0.2, "eps_hi": 0.28, "tis_cap": 2.0, "kl_beta": 0.05}


def loss_inputs(T, V, dtype, seed, pitch=0, offset=0, behav=True, kl=True, clip=False):
    g = gen(seed)
    ld = V + pitch
    buf = torch.randn(T * ld + offset, generator=g, device=DEV).mul_(2).to(dtype)
    logits = buf[offset:].view(T, ld)[:, :V]
    targets = torch.randint(0, V, (T,), generator=g, device=DEV)
    rows = torch.arange(T, device=DEV)
    logits[rows, targets] += 3
    lp = torch.log_softmax(logits.to(D), 1)[rows, targets].float()
    n = lambda s: s * torch.randn(T, generator=g, device=DEV)  # noqa: E731
    st = {"logits": logits, "targets": targets, "logp_old": lp + n(0.2), "adv": n(1.0),
          "weight": (torch.rand(T, generator=g, device=DEV) < 0.8).float() / T}
    st["weight"][0] = 1.0 / T
    st["logp_behav"] = st["logp_old"] + n(0.3) if behav else None
    st["logp_ref"] = lp + n(0.3) if kl else None
    st["clip_hi"] = 1 + torch.rand(T, generator=g, device=DEV) if clip else None
    return st


def loss_reference(st, temperature, hyp=HYP):
    """(lp, loss, dlogits) in 64 bits by autograd, and the error bounds of each."""
    z = st["logits"].to(D).clone().requires_grad_(True)
    T, V = z.shape
    live = (st["weight"] != 0) & (st["targets"] >= 0) & (st["targets"] < V)
    t = st["targets"].clamp(0, V - 1)
    zt = torch.where(live[:, None], z, torch.zeros_like(z)) / temperature
    lp = torch.log_softmax(zt, 1).gather(1, t[:, None])[:, 0]
    cast = lambda k: None if st[k] is None else st[k].to(D)  # noqa: E731
    loss = R.token_loss(lp, cast("logp_old"), cast("adv"), torch.where(live, cast("weight"), 0.0), cast("logp_behav"),
                        cast("logp_ref"), cast("clip_hi"), hyp["eps_lo"], hyp["eps_hi"], hyp["tis_cap"], hyp["kl_beta"])
    loss.sum().backward()
    lp, loss, grad = lp.detach(), loss.detach(), z.grad
    top = zt.detach().amax(1)
    drop = (top - zt.detach().gather(1, t[:, None])[:, 0]).abs()
    # the exponentials within 2^-21, chains of at most 128 additions and three trees; the
    # target's distance from the maximum is three roundings, and lp one more
    elp = (8 + 128 + 20) * U + 6 * U * (drop + lp.abs())
    return live, lp, loss, grad, elp


def row_sensitivity(st, lp, elp, temperature, hyp=HYP):
    """Errors of the loss and of dloss/dlp that lp's error and their own roundings allow."""
    rho = (lp - st["logp_old"].to(D)).exp()
    w = torch.ones_like(rho) if st["logp_behav"] is None else (st["logp_old"] - st["logp_behav"]).to(D).exp().clamp(
        max=hyp["tis_cap"])
    e = elp + 16 * U + 4 * U * (lp.abs() + st["logp_old"].to(D).abs())
    wt = st["weight"].to(D).abs()
    b = w * st["adv"].to(D).abs() * rho
    k = torch.zeros_like(rho)
    if st["logp_ref"] is not None:
        d = st["logp_ref"].to(D) - lp
        k = hyp["kl_beta"] * (d.exp() + 1)
    ew = 8 * U * w  # the importance weight's own exponential
    eloss = wt * ((b * 2 + k) * e + ew * st["adv"].to(D).abs() * rho.clamp(max=4))
    edlp = wt * ((b + k) * e + 2 * ew * st["adv"].to(D).abs() * rho)
    return eloss, edlp


def check_loss(st, temperature=0.9, hyp=HYP, inplace=False):
    live, lp, loss, grad, elp = loss_reference(st, temperature, hyp)
    bf16 = st["logits"].dtype == torch.bfloat16
    got_loss, got_lp, d = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                                          logp_behav=st["logp_behav"], logp_ref=st["logp_ref"], clip_hi=st["clip_hi"],
                                          temperature=temperature, inplace=inplace, **hyp)
    assert (d is st["logits"]) == inplace and d.dtype == st["logits"].dtype
    assert bool((got_lp[~live] == 0).all()) and bool((got_loss[~live] == 0).all()) and bool((d[~live] == 0).all())
    assert bool(((got_lp.to(D) - lp).abs() <= elp)[live].all())
    eloss, edlp = row_sensitivity(st, lp, elp, temperature, hyp)
    # rows within the ratio's error of a clip bound may take either branch
    rho = (lp - st["logp_old"].to(D)).exp()
    hi = st["clip_hi"].to(D) if st["clip_hi"] is not None else 1 + hyp["eps_hi"]
    near = ((rho - hi).abs() < 1e-4) | ((rho - (1 - hyp["eps_lo"])).abs() < 1e-4)
    sure = live & ~near
    assert bool(((got_loss.to(D) - loss).abs() <= eloss)[sure].all())
    p = torch.softmax(st["logits"].to(D) / temperature, 1) if not inplace else None
    dlp = grad.abs().sum(1) / 2 * temperature  # |dloss/dlp| (1 - p_t), enough for a bound of p's error
    tol = edlp[:, None] / temperature * (1 if p is None else torch.maximum(p, (torch.arange(
        p.shape[1], device=DEV)[None] == st["targets"][:, None]).to(D)))
    tol = tol + grad.abs() * (256 * U) + 256 * U * dlp[:, None] * (grad.abs() > 0)
    tol = tol + (2.0 ** -8 if bf16 else U) * (grad.abs() + tol) + 2.0 ** -134
    bad = ((d.to(D) - grad).abs() > tol) & sure[:, None]
    assert not bad.any(), f"{int(bad.sum())} gradients off"
    return d


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pitch,offset", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 3, 1), (9, 1000, 0, 0), (33, 1001, 0, 3),
                                              (4, 4096, 8, 0), (6, 32001, 0, 0), (5, 50257, 0, 5), (3, 70001, 6, 2),
                                              (4, 151936, 0, 0), (2, 262136, 0, 0)])
def test_policy_loss(T, V, pitch, offset, dtype):
    check_loss(loss_inputs(T, V, dtype, T + V, pitch, offset))


@pytest.mark.parametrize("behav,kl,clip", [(False, False, False), (True, False, True), (False, True, False),
                                           (True, True, True)])
def test_policy_loss_options(behav, kl, clip):
    for dtype in (torch.bfloat16, torch.float32):
        check_loss(loss_inputs(64, 3001, dtype, 9, pitch=7, behav=behav, kl=kl, clip=clip), temperature=1.0)


@pytest.mark.parametrize("T,V", [(2, 524280), (1, 1200007)])
def test_policy_loss_long_rows(T, V):
    check_loss(loss_inputs(T, V, torch.bfloat16, 4))


@pytest.mark.parametrize("V", [999, 40000, 140000])
def test_policy_loss_in_place_and_without_gradient(V):
    st = loss_inputs(12, V, torch.bfloat16, V, pitch=1)
    before = st["logits"].clone()
    want = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                           logp_ref=st["logp_ref"], **HYP)
    none = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                           logp_ref=st["logp_ref"], grad=False, **HYP)
    # (another launch shape, so another order of the row's sums)
    assert none[2] is None and torch.equal(st["logits"], before)
    live, lp, loss, _, elp = loss_reference({**st, "logp_behav": None}, 1.0)
    eloss, _ = row_sensitivity({**st, "logp_behav": None}, lp, elp, 1.0)
    rho = (lp - st["logp_old"].to(D)).exp()
    sure = live & ((rho - 1.28).abs() > 1e-4) & ((rho - 0.8).abs() > 1e-4)
    assert bool(((none[1].to(D) - lp).abs() <= elp)[live].all())
    assert bool(((none[0].to(D) - loss).abs() <= eloss)[sure].all())
    over = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                           logp_ref=st["logp_ref"], inplace=True, **HYP)
    assert over[2] is st["logits"] and all(torch.equal(a, b) for a, b in zip(over, want))


@pytest.mark.parametrize("V", [500, 40001, 140000])
def test_policy_loss_empty_and_masked_rows(V):
    """Weight 0 and targets outside the row hide NaN; -inf logits have probability 0; a row
    of -inf only is empty; a row of the type's lowest value is uniform."""
    for dtype in (torch.bfloat16, torch.float32):
        st = loss_inputs(8, V, dtype, 21, pitch=3)
        st["weight"][:] = 0.125
        x = st["logits"]
        st["weight"][1] = 0
        x[1] = float("nan")
        st["targets"][2], st["targets"][3] = -100, V
        x[2], x[3] = float("nan"), float("inf")
        x[4, torch.arange(V, device=DEV) != st["targets"][4]] = float("-inf")  # the target is certain
        x[5] = float("-inf")
        x[6] = torch.finfo(dtype).min
        x[7, V // 2:] = float("-inf")
        st["targets"][7] = V // 4
        loss, lp, d = rlq.policy_loss(x, st["targets"], st["logp_old"], st["adv"], st["weight"], **HYP)
        for r in (1, 2, 3):
            assert float(loss[r]) == 0 and float(lp[r]) == 0 and bool((d[r] == 0).all())
        assert abs(float(lp[4])) <= 1e-6 and bool((d[4].abs() <= 1e-6).all())
        assert float(lp[5]) == -math.inf and float(loss[5]) == 0 and bool((d[5] == 0).all())
        assert abs(float(lp[6]) + math.log(V)) <= 2e-5
        assert bool((d[7, V // 2:] == 0).all()) and bool(torch.isfinite(d).all())
        keep = torch.tensor([0, 7], device=DEV)
        ref = torch.log_softmax(x[keep].to(D), 1).gather(1, st["targets"][keep, None])[:, 0]
        assert bool(((lp[keep].to(D) - ref).abs() <= 1e-5 * (1 + ref.abs())).all())
        l2, lse = rlq.token_logprobs(x, st["targets"])
        for r in (2, 3):
            assert float(l2[r]) == 0 and float(lse[r]) == 0
        assert math.isnan(float(l2[1])) and float(lse[5]) == -math.inf
        assert bool(((l2[keep].to(D) - ref).abs() <= 1e-5 * (1 + ref.abs())).all())


@pytest.mark.parametrize("V", [500, 40001])
def test_policy_loss_keeps_nan(V):
    """A NaN among a row's inputs reaches its loss and its gradient, and no other row's."""
    st = loss_inputs(6, V, torch.bfloat16, 23)
    st["weight"][:] = 1 / 6
    nan = float("nan")
    st["logits"][0, V // 3] = nan
    st["logp_old"][1] = nan
    st["adv"][2] = nan
    behav = st["logp_old"].clone()
    behav[1] = 0
    behav[3] = nan
    hi = torch.full((6,), 1.3, device=DEV)
    hi[4] = nan
    loss, _, d = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                                 logp_behav=behav, clip_hi=hi)
    for r in range(5):
        assert math.isnan(float(loss[r])), r
        if r < 4:
            assert bool(torch.isnan(d[r]).any()), r
    assert math.isfinite(float(loss[5])) and bool(torch.isfinite(d[5]).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pitch,offset", [(1, 1, 0, 0), (7, 333, 0, 1), (64, 32001, 0, 0), (3, 128256, 0, 0)])
def test_token_logprobs(T, V, pitch, offset, dtype):
    st = loss_inputs(T, V, dtype, 2 * V + T, pitch, offset)
    for temperature in (1.0, 0.7):
        lp, lse = rlq.token_logprobs(st["logits"], st["targets"], temperature=temperature)
        z = st["logits"].to(D) / temperature
        want = torch.logsumexp(z, 1)
        top = z.amax(1)
        zt = z.gather(1, st["targets"][:, None])[:, 0]
        tol = 156 * U + 6 * U * ((top - zt).abs() + (zt - want).abs())
        assert bool(((lp.to(D) - (zt - want)).abs() <= tol).all())
        assert bool(((lse.to(D) - want).abs() <= 156 * U + 6 * U * (top.abs() + want.abs())).all())


def test_policy_loss_against_differences():
    """The gradient against central differences of the 64-bit loss at single logits."""
    T, V, temperature = 6, 50, 0.8
    st = loss_inputs(T, V, torch.float32, 31, clip=True)
    st["weight"][:] = 1.0
    _, lp, d = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"],
                               logp_behav=st["logp_behav"], logp_ref=st["logp_ref"], clip_hi=st["clip_hi"],
                               temperature=temperature, **HYP)
    rho = (lp - st["logp_old"]).exp()
    far = ((rho - st["clip_hi"]).abs() > 1e-3) & ((rho - 0.8).abs() > 1e-3)
    assert bool(far.any())

    def f(x):
        q = torch.log_softmax(x / temperature, 1).gather(1, st["targets"][:, None])[:, 0]
        c = lambda k: st[k].to(D)  # noqa: E731
        return R.token_loss(q, c("logp_old"), c("adv"), c("weight"), c("logp_behav"), c("logp_ref"), c("clip_hi"),
                            HYP["eps_lo"], HYP["eps_hi"], HYP["tis_cap"], HYP["kl_beta"])

    x, e = st["logits"].to(D), 1e-5
    for v in range(V):
        step = torch.zeros_like(x)
        step[:, v] = e
        dif = (f(x + step) - f(x - step)) / (2 * e)
        assert bool(((d[:, v].to(D) - dif).abs() <= 1e-5 * (1 + dif.abs()))[far].all())


# --------------------------------------------------- streams and graphs ---

@pytest.mark.parametrize("M", [5, 70, 300])  # the few-token kernel, single CTAs, CTA pairs
def test_another_stream_and_a_graph(M):
    g = gen(8)
    F, K = 256, 512
    res, delta = normal(g, M, K), normal(g, M, K, std=0.3)
    gamma = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    wq, ws = R.quant_blocks(normal(g, 2 * F, K, std=0.05))
    da = normal(g, M, F, std=1e-3)
    st = loss_inputs(M, 40001, torch.bfloat16, 1)

    def step():
        h, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(res, delta, gamma, 1e-6, colwise=True)
        aq, as_, guq, gus = rlq.gemm_gated_fprop(q, s, wq, ws, checkpoint=True)
        back = rlq.gated_backward(da, guq, gus)
        dh, dgamma = rlq.rmsnorm_backward(delta, h, rstd, gamma, dres=res)
        loss, lp, d = rlq.policy_loss(st["logits"], st["targets"], st["logp_old"], st["adv"], st["weight"], **HYP)
        return [h, q, s, qT, sc, rstd, aq, as_, guq, gus, *back, dh, dgamma, loss, lp, d]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for handle in (side, side.cuda_stream):  # named instead of made current
        dh, dgamma = rlq.rmsnorm_backward(delta, want[0], want[5], gamma, dres=res, stream=handle)
        aq, as_, _, _ = rlq.gemm_gated_fprop(want[1], want[2], wq, ws, stream=handle)
        side.synchronize()
        assert torch.equal(dh, want[16]) and torch.equal(dgamma, want[17])
        assert torch.equal(aq, want[6]) and torch.equal(as_, want[7])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    res2 = normal(g, M, K)
    keep = res.clone()
    res.copy_(res2)
    graph.replay()
    want2 = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want2))
    res.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rlq.check()


@pytest.mark.parametrize("call", ["gated", "backward"])
def test_wait_that_runs_out_is_reported(call):
    """With the stall diagnostic armed nothing arrives for the first block or tile: the
    bounded waits run out, the kernel leaves, the check reports it, and the same call then
    gives the bits that it gave before."""
    M, F, K = 700, 4096, 1024  # 192 tiles: some CTAs have a second one in flight
    if call == "gated":
        g = gen(41)
        x, w = normal(g, M, K), normal(g, 2 * F, K, std=K ** -0.5)
        xq, xs, _, _ = rlq.quant_act_1x128(x)
        wq, ws, _ = rlq.quant_weight_128x128(w)
        run = lambda: rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=True)  # noqa: E731
    else:
        g = gen(42)
        da = normal(g, M, F, std=1e-3)
        guq, gus, _, _ = rlq.quant_act_1x128(normal(g, M, 2 * F))
        run = lambda: rlq.gated_backward(da, guq, gus)  # noqa: E731
    want = run()
    rlq.check()
    rlq.rlq_diag_arm_gemm_stall()
    run()
    with pytest.raises(rlq.RlqError) as e:
        rlq.check()
    assert e.value.status == 5 and "ran out" in str(e.value)
    rlq.check()
    got = run()
    rlq.check()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("scale", [1e-30, 1e-38])
def test_gated_backward_tiny_gradients(scale):
    """Groups whose scales are subnormal (their reciprocals overflow) beside ordinary ones."""
    g = gen(6)
    M, F = 150, 256
    guq, gus = R.quant_rows(normal(g, M, 2 * F))
    da = normal(g, M, F).float()
    da[:, 128:] *= scale
    da[128:, :128] *= scale
    da = da.to(torch.bfloat16)
    q, s, qT, sc, aT, ac = rlq.gated_backward(da, guq, gus)
    dg, du, a, edg, edu, ea = gate_reference(da, guq, gus)
    # products and scales below the normal range round to a multiple of 2^-149, a scale
    # counting 448 of them
    tiny = 4 * 448 * 2.0 ** -149
    d, e = torch.cat((dg, du), 1), torch.cat((edg, edu), 1) + tiny
    R.check_rows(q, s, d, e, "rows")
    R.check_cols(qT, sc, d, e, "columns")
    R.check_cols(aT, ac, a, ea, "a's columns")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,pitch,offset", [(6000, 515, 2, 1), (700, 33001, 1, 3), (300, 100001, 0, 0)])
def test_policy_loss_many_rows(T, V, pitch, offset, dtype):
    """More rows than are resident at once, cut units at different places from row to row,
    runs of empty rows."""
    st = loss_inputs(T, V, dtype, T + V, pitch, offset)
    st["weight"][T // 3: T // 3 + 40] = 0
    st["targets"][T // 2: T // 2 + 9] = -1
    check_loss(st)
    lp, lse = rlq.token_logprobs(st["logits"], st["targets"], temperature=0.9)
    assert torch.equal(lp, rlq.token_logprobs(st["logits"], st["targets"], temperature=0.9)[0])
    keep = st["targets"] >= 0
    z = st["logits"].to(D) / 0.9
    want = torch.log_softmax(z, 1).gather(1, st["targets"].clamp(min=0)[:, None])[:, 0]
    drop = z.amax(1) - z.gather(1, st["targets"].clamp(min=0)[:, None])[:, 0]
    assert bool(((lp.to(D) - want).abs() <= 156 * U + 6 * U * (drop + want.abs()))[keep].all())
    assert bool((lp[~keep] == 0).all()) and bool((lse[~keep] == 0).all())


# ------------------------------------------------ offsets past 32 bits ---

def tail_and_head(M, n):
    return torch.cat((torch.arange(n, device=DEV), torch.arange(M - n, M, device=DEV)))


def test_norm_past_32_bits():
    """M K beyond 2^31: the last rows and their column group against the 64-bit form."""
    M, K = 300003, 8192
    g = gen(12)
    res = torch.randint(-120, 121, (M, K), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    gamma = torch.ones(K, dtype=torch.bfloat16, device=DEV)
    delta = res.clone()
    h, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(res, delta, gamma, 1e-6, colwise=True, inplace=True)
    assert h is res and M * K > 2 ** 31
    last = (M - 1) // 128 * 128  # the last column group's first row
    rows = slice(last, M)
    assert torch.equal(h[rows], 2 * delta[rows])
    r, x, rtol, err = norm_reference(h[rows], gamma, 1e-6)
    assert bool(((rstd[rows].to(D) - r).abs() <= rtol * r).all())
    R.check_rows(q[rows], s[:, rows].contiguous(), x, err, "rows")
    R.check_cols(qT[:, rows], sc[-1:], x, err, "columns")
    del q, qT
    dh, dgamma = rlq.rmsnorm_backward(delta, h, rstd, gamma)
    want, e, _, _ = norm_bwd_reference(delta[rows], h[rows], rstd[rows], gamma, None)
    assert bool(((dh[rows].to(D) - want).abs() <= e).all())
    sums = torch.zeros(K, dtype=D, device=DEV)
    mags = torch.zeros(K, dtype=D, device=DEV)
    for a in range(0, M, 20000):
        v = delta[a:a + 20000].to(D) * (h[a:a + 20000].to(D) * rstd[a:a + 20000].to(D)[:, None])
        sums += v.sum(0)
        mags += v.abs().sum(0)
    # the sums run over at most 500 rows a team, then over teams and CTAs
    assert bool(((dgamma.to(D) - sums).abs() <= (M // 500 + 600 + 24) * U * mags).all())


def test_loss_past_32_bits():
    T, V = 17003, 128256
    g = gen(13)
    logits = torch.empty((T, V), dtype=torch.bfloat16, device=DEV)
    logits.normal_(0, 2, generator=g)
    assert T * V > 2 ** 31
    st = {"logits": logits, "targets": torch.randint(0, V, (T,), generator=g, device=DEV)}
    st["logp_old"] = rlq.token_logprobs(logits, st["targets"])[0]
    st["adv"] = torch.randn(T, generator=g, device=DEV)
    st["weight"] = torch.ones(T, device=DEV)
    pick = tail_and_head(T, 6)
    few = {k: v[pick].clone() for k, v in st.items()} | {"logp_behav": None, "logp_ref": None, "clip_hi": None}
    loss, lp, d = rlq.policy_loss(logits, st["targets"], st["logp_old"], st["adv"], st["weight"], temperature=1.0,
                                  inplace=True, **HYP)
    live, wlp, wloss, grad, elp = loss_reference(few, 1.0)
    eloss, edlp = row_sensitivity(few, wlp, elp, 1.0)
    assert bool(((lp[pick].to(D) - wlp).abs() <= elp).all()) and bool(((loss[pick].to(D) - wloss).abs() <= eloss).all())
    tol = edlp[:, None] + grad.abs() * (512 * U)
    assert bool(((d[pick].to(D) - grad).abs() <= tol + 2.0 ** -8 * (grad.abs() + tol)).all())


def test_gate_past_32_bits():
    """Codes [M, 2F] of more than 2^31 bytes, forward and backward: the last rows against
    the same rows alone (each row's codes depend on that row only)."""
    M, F, K = 75001, 14336, 128
    g = gen(14)
    xq, xs = R.quant_rows(normal(g, M, K))
    wq, ws = R.quant_blocks(normal(g, 2 * F, K, std=0.1))
    aq, as_, guq, gus = rlq.gemm_gated_fprop(xq, xs, wq, ws, checkpoint=True)
    rlq.check()
    assert guq.numel() > 2 ** 31
    rows = slice((M - 1) // 128 * 128, M)  # the last token group
    # (through the same tile shape: 300 rows that end with these)
    part = slice(M - 300, M)
    one = rlq.gemm_gated_fprop(xq[part], xs[:, part].contiguous(), wq, ws, checkpoint=True)
    for a, b in ((aq[part], one[0]), (as_[:, part], one[1]), (guq[part], one[2]), (gus[:, part], one[3])):
        assert torch.equal(a, b)
    del aq, one
    da = normal(g, M, F)
    q, s, qT, sc, aT, ac = rlq.gated_backward(da, guq, gus)
    two = rlq.gated_backward(da[rows], guq[rows], gus[:, rows].contiguous())
    assert torch.equal(q[rows], two[0]) and torch.equal(s[:, rows], two[1]) and torch.equal(qT[:, rows], two[2])
    assert torch.equal(sc[-1:], two[3]) and torch.equal(aT[:, rows], two[4]) and torch.equal(ac[-1:], two[5])
