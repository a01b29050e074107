"""Workloads of the actor's feed-forward sublayer and its loss.

Six operators, each in a plain form (elementary torch operations in 32 bits) and through the
library's calls (``own``):

* ``norm``       residual addition, RMSNorm and the 1x128 (and 128x1) FP8 quantizer
* ``norm_bwd``   the norm's gradient with the residual's, and the norm weight's gradient
* ``gated``      both projections of the gated feed-forward block, SiLU and product, FP8 in and
                 out, with or without the 8-bit checkpoint of the two projections
* ``gated_bwd``  the gate's gradient from that checkpoint, quantized for DGrad and WGrad
* ``logprobs``   log probabilities of given tokens from logits
* ``loss``       clipped policy loss with a KL term, and its gradient with respect to the logits

FP8 codes are returned as float8 values beside their fp32 scales.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one token's residual and norm between two layers of an 8B model, as a rollout calls it
        {"name": "norm_one_token", "op": "norm", "M": 1, "K": 4096, "colwise": False},
        # a rollout batch on a 32B model's hidden size
        {"name": "norm_prefill_odd", "op": "norm", "M": 1001, "K": 5120, "colwise": False},
        # the 8B training step: the weight gradient needs the 128x1 codes too
        {"name": "norm_train", "op": "norm", "M": 8192, "K": 4096, "colwise": True},
        # the norm's gradient in a ragged micro-batch of a 7B model
        {"name": "norm_bwd_odd", "op": "norm_bwd", "M": 777, "K": 3584, "residual": True},
        # and in the 8B training step
        {"name": "norm_bwd_train", "op": "norm_bwd", "M": 8192, "K": 4096, "residual": True},
        # one new token through an 8B block's gate and up projections
        {"name": "gated_one_token", "op": "gated", "M": 1, "F": 14336, "K": 4096, "checkpoint": False},
        # a rollout batch of 64 sequences on the 7B block
        {"name": "gated_rollout", "op": "gated", "M": 64, "F": 18944, "K": 3584, "checkpoint": False},
        # the 8B training step's forward pass, with the checkpoint
        {"name": "gated_train", "op": "gated", "M": 8192, "F": 14336, "K": 4096, "checkpoint": True},
        # the gate's gradient: a ragged micro-batch
        {"name": "gated_bwd_odd", "op": "gated_bwd", "M": 333, "F": 18944},
        # and the 8B training step's
        {"name": "gated_bwd_train", "op": "gated_bwd", "M": 8192, "F": 14336},
        # log probabilities of a batch's tokens under the reference policy, fp32 logits
        {"name": "logprobs_f32", "op": "logprobs", "T": 600, "V": 32001, "dtype": "f32"},
        # the training step's loss and gradient over a large vocabulary
        {"name": "loss_train", "op": "loss", "T": 4096, "V": 128256, "dtype": "bf16", "kl": True, "behav": True,
         "grad": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gated", "gated_bwd", "logprobs", "loss"])
    if op in ("norm", "norm_bwd"):
        c = {"op": op, "M": _log_int(rng, 1, 8192), "K": 128 * _log_int(rng, 1, 32)}
        c["colwise" if op == "norm" else "residual"] = rng.random() < 0.5
        return c
    if op == "gated":
        return {"op": op, "M": _log_int(rng, 1, 8192), "F": 128 * _log_int(rng, 1, 112),
                "K": 128 * _log_int(rng, 1, 32), "checkpoint": rng.random() < 0.5}
    if op == "gated_bwd":
        return {"op": op, "M": _log_int(rng, 1, 8192), "F": 128 * _log_int(rng, 1, 112)}
    c = {"op": op, "T": _log_int(rng, 1, 2048), "V": _log_int(rng, 64, 128256), "dtype": rng.choice(["bf16", "f32"])}
    if op == "loss":
        c.update(kl=rng.random() < 0.5, behav=rng.random() < 0.5, grad=rng.random() < 0.8)
    return c


# ---------------------------------------------------------------- inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _scale(amax):
    return torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)


def _rows_1x128(x):
    """FP8 values [M, K] and scales [K/128, M] of the 1x128 groups of x."""
    M, K = x.shape
    g = x.view(M, K // 128, 128)
    s = _scale(g.abs().amax(2))
    return (g / s[:, :, None]).view(M, K).to(FP8), s.t().contiguous()


def _cols_128x1(x):
    """FP8 values, transposed [K, M], and scales [ceil(M/128), K] of the 128x1 groups of x."""
    M, K = x.shape
    nb = -(-M // 128)
    g = torch.nn.functional.pad(x, (0, 0, 0, nb * 128 - M)).view(nb, 128, K)
    s = _scale(g.abs().amax(1))
    return (g / s[:, None, :]).view(nb * 128, K)[:M].to(FP8).t().contiguous(), s


def _block_128x128(w):
    """FP8 values [N, K] and scales [N/128, K/128] of the 128x128 blocks of w."""
    N, K = w.shape
    b = w.view(N // 128, 128, K // 128, 128)
    s = _scale(b.abs().amax((1, 3)))
    return (b / s[:, None, :, None]).view(N, K).to(FP8), s


def _padded(codes):
    """uint8 codes [rows, cols] in rows of 16-byte-aligned pitch, as the library takes them."""
    rows, cols = codes.shape
    buf = torch.zeros((rows, -(-cols // 16) * 16), dtype=torch.uint8, device="cuda")
    buf[:, :cols] = codes.view(torch.uint8)
    return buf[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op in ("norm", "norm_bwd"):
        M, K = case["M"], case["K"]
        # a residual stream with a few large channels, as trained models have
        big = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        res = (torch.randn(M, K, generator=g, device="cuda") * big).to(torch.bfloat16)
        st["gamma"] = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        if op == "norm":
            st.update(res=res, delta=_normal(g, M, K, std=0.3))
        else:
            st.update(h=res, rstd=torch.rsqrt(res.float().square().mean(1) + EPS), dx=_normal(g, M, K, std=1e-3),
                      dres=_normal(g, M, K, std=1e-3) if case["residual"] else None)
    elif op == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        xq, xs = _rows_1x128(_normal(g, M, K).float())
        wq, ws = _block_128x128(_normal(g, 2 * F, K, std=0.02).float())
        st.update(xq=xq.view(torch.uint8), xs=xs, wq=wq.view(torch.uint8), ws=ws)
    elif op == "gated_bwd":
        M, F = case["M"], case["F"]
        guq, gus = _rows_1x128(_normal(g, M, 2 * F, std=1.3).float())
        st.update(da=_normal(g, M, F, std=1e-3), guq=_padded(guq), gus=gus)
    else:
        T, V = case["T"], case["V"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # rows start on 16 bytes, as an LM head with a padded vocabulary writes them
        ld = -(-V // 8) * 8
        logits = torch.randn(T, ld, generator=g, device="cuda").mul_(2.0).to(dt)[:, :V]
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        rows = torch.arange(T, device="cuda")
        # sampled tokens are likely ones
        logits[rows, targets] = (2.0 * math.log(V) / 3 + 3.0 + torch.randn(T, generator=g, device="cuda")).to(dt)
        st.update(logits=logits, targets=targets)
        if op == "loss":
            lp = logits[rows, targets].float() - torch.logsumexp(logits.float(), 1)
            noise = lambda s: s * torch.randn(T, generator=g, device="cuda")  # noqa: E731
            st["lp_old"] = lp + noise(0.15)
            st["lp_behav"] = st["lp_old"] + noise(0.1) if case["behav"] else None
            st["lp_ref"] = lp + noise(0.2) if case["kl"] else None
            st["adv"] = torch.randn(T, generator=g, device="cuda")
            # prompt and padding tokens weigh nothing; the loss is a mean over the others
            st["weight"] = (torch.rand(T, generator=g, device="cuda") < 0.85).float() / T
    return st


# ------------------------------------------------------------------ runs ---

LOSS = {"eps_lo": 0.2, "eps_hi": 0.28, "tis_cap": 2.0, "kl_beta": 0.05, "temperature": 0.9}


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from fp8_block_scaled_quantize_gb300 import rlq

    op = st["op"]
    if op == "norm":
        h, q, s, qT, sc, rstd = rlq.add_rmsnorm_quant_act_1x128(st["res"], st["delta"], st["gamma"], EPS,
                                                                colwise=st["colwise"])
        out = {"h": h, "rstd": rstd, "q": q.view(FP8), "s": s}
        if st["colwise"]:
            out.update(qT=qT.view(FP8), sc=sc)
        return out
    if op == "norm_bwd":
        dh, dgamma = rlq.rmsnorm_backward(st["dx"], st["h"], st["rstd"], st["gamma"], dres=st["dres"])
        return {"dh": dh, "dgamma": dgamma}
    if op == "gated":
        aq, s, guq, gus = rlq.gemm_gated_fprop(st["xq"], st["xs"], st["wq"], st["ws"], checkpoint=st["checkpoint"])
        out = {"aq": aq.view(FP8), "as": s}
        if st["checkpoint"]:
            out.update(guq=guq.view(FP8), gus=gus)
        return out
    if op == "gated_bwd":
        q, s, qT, sc, aT, ac = rlq.gated_backward(st["da"], st["guq"], st["gus"])
        return {"q": q.view(FP8), "s": s, "qT": qT.view(FP8), "sc": sc, "aT": aT.view(FP8), "ac": ac}
    if op == "logprobs":
        lp, lse = rlq.token_logprobs(st["logits"], st["targets"], temperature=LOSS["temperature"])
        return {"lp": lp, "lse": lse}
    loss, lp, dlogits = rlq.policy_loss(st["logits"], st["targets"], st["lp_old"], st["adv"], st["weight"],
                                        logp_behav=st["lp_behav"], logp_ref=st["lp_ref"], grad=st["grad"], **LOSS)
    return {"loss": loss, "lp": lp, "dlogits": dlogits} if st["grad"] else {"loss": loss, "lp": lp}


def _dequant(st):
    """x [M, K] and w [2F, K] in fp32 from their codes and scales."""
    xq, wq = st["xq"].view(FP8).float(), st["wq"].view(FP8).float()
    x = xq * st["xs"].t().repeat_interleave(128, 1)
    w = wq * st["ws"].repeat_interleave(128, 0).repeat_interleave(128, 1)
    return x, w


def _gate_grads(da, g, u):
    sg = 1 / (1 + torch.exp(-g))
    return da * u * sg * (1 + g * (1 - sg)), da * g * sg, g * sg * u


def _run_plain(st):
    op = st["op"]
    if op == "norm":
        h = (st["res"].float() + st["delta"].float()).to(torch.bfloat16)
        f = h.float()
        rstd = 1 / torch.sqrt(f.square().mean(1) + EPS)
        x = f * rstd[:, None] * st["gamma"].float()
        q, s = _rows_1x128(x)
        out = {"h": h, "rstd": rstd, "q": q, "s": s}
        if st["colwise"]:
            out["qT"], out["sc"] = _cols_128x1(x)
        return out
    if op == "norm_bwd":
        xh = st["h"].float() * st["rstd"][:, None]
        dx = st["dx"].float()
        dg = dx * st["gamma"].float()
        dh = st["rstd"][:, None] * (dg - xh * (dg * xh).mean(1, keepdim=True))
        if st["dres"] is not None:
            dh = dh + st["dres"].float()
        return {"dh": dh.to(torch.bfloat16), "dgamma": (dx * xh).sum(0)}
    if op == "gated":
        x, w = _dequant(st)
        gu = x @ w.t()
        g, u = gu[:, :st["F"]], gu[:, st["F"]:]
        q, s = _rows_1x128(g / (1 + torch.exp(-g)) * u)
        out = {"aq": q, "as": s}
        if st["checkpoint"]:
            out["guq"], out["gus"] = _rows_1x128(gu)
        return out
    if op == "gated_bwd":
        gu = st["guq"].view(FP8).float() * st["gus"].t().repeat_interleave(128, 1)
        dg, du, a = _gate_grads(st["da"].float(), gu[:, :st["F"]], gu[:, st["F"]:])
        d = torch.cat((dg, du), 1)
        q, s = _rows_1x128(d)
        qT, sc = _cols_128x1(d)
        aT, ac = _cols_128x1(a.contiguous())
        return {"q": q, "s": s, "qT": qT, "sc": sc, "aT": aT, "ac": ac}
    z = st["logits"].float() / LOSS["temperature"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1)
    zt = z.gather(1, st["targets"][:, None])
    lp = (zt - top)[:, 0] - torch.log(total)
    if op == "logprobs":
        return {"lp": lp, "lse": top[:, 0] + torch.log(total)}
    loss, dlp = _token_loss(st, lp)
    # a row of weight 0 has no loss, no log probability and no gradient
    lp = torch.where(st["weight"] == 0, torch.zeros_like(lp), lp)
    if not st["grad"]:
        return {"loss": loss, "lp": lp}
    d = e.mul_((-dlp / LOSS["temperature"] / total)[:, None])
    d.scatter_add_(1, st["targets"][:, None], (dlp / LOSS["temperature"])[:, None])
    return {"loss": loss, "lp": lp, "dlogits": d.to(st["logits"].dtype)}


def _token_loss(st, lp):
    """Each token's loss and its derivative with respect to lp, in lp's type."""
    t = lp.dtype
    old, adv, weight = st["lp_old"].to(t), st["adv"].to(t), st["weight"].to(t)
    rho = torch.exp(lp - old)
    is_w = torch.ones_like(lp) if st["lp_behav"] is None else torch.clamp(torch.exp(old - st["lp_behav"].to(t)),
                                                                          max=LOSS["tis_cap"])
    plain, clipped = rho * adv, torch.clamp(rho, 1 - LOSS["eps_lo"], 1 + LOSS["eps_hi"]) * adv
    loss = -is_w * torch.minimum(plain, clipped)
    dlp = torch.where(plain <= clipped, -is_w * plain, torch.zeros_like(lp))
    if st["lp_ref"] is not None:
        d = st["lp_ref"].to(t) - lp
        loss = loss + LOSS["kl_beta"] * (torch.expm1(d) - d)
        dlp = dlp - LOSS["kl_beta"] * torch.expm1(d)
    return weight * loss, weight * dlp


# ------------------------------------------------------- work and 64 bits ---

def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        cw = M * K + 4 * -(-M // 128) * K if case["colwise"] else 0
        return {"bytes": M * K * (2 + 2 + 2 + 1) + M * K // 32 + 4 * M + 2 * K + cw, "flops": 8 * M * K}
    if op == "norm_bwd":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (8 if case["residual"] else 6) + 4 * M + 6 * K, "flops": 9 * M * K}
    if op == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        codes = M * K + 2 * F * K + M * F + (2 * M * F if case["checkpoint"] else 0)
        scales = M * K // 32 + 8 * F * K // 16384 + M * F // 32 + (M * F // 16 if case["checkpoint"] else 0)
        return {"bytes": codes + scales, "flops": 4 * M * F * K}
    if op == "gated_bwd":
        M, F = case["M"], case["F"]
        return {"bytes": M * F * (2 + 2 + 2 + 2 + 1) + 2 * (M * F // 16) + 12 * -(-M // 128) * F, "flops": 20 * M * F}
    T, V = case["T"], case["V"]
    e = 2 if case["dtype"] == "bf16" else 4
    grad = op == "loss" and case["grad"]
    return {"bytes": T * V * e * (2 if grad else 1) + 36 * T, "flops": T * V * (8 if grad else 4)}


def _exact_rows(x):
    """Unrounded values of the 1x128 codes (x / s) and the scales."""
    M, K = x.shape
    g = x.reshape(M, K // 128, 128)
    a = g.abs().amax(2)
    s = torch.where(a == 0, torch.ones_like(a), a / 448)
    return (g / s[:, :, None]).reshape(M, K), s.t().contiguous()


def _exact_cols(x):
    v, s = [], []
    for m in range(0, x.shape[0], 128):
        b = x[m:m + 128]
        a = b.abs().amax(0)
        s.append(torch.where(a == 0, torch.ones_like(a), a / 448))
        v.append(b / s[-1])
    return torch.cat(v).t().contiguous(), torch.stack(s)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "norm":
        h = st["res"].to(D) + st["delta"].to(D)
        f = h.to(torch.bfloat16).to(D)  # the stream is held in bf16, and the norm is of what is held
        rstd = (f.pow(2).sum(1) / case["K"] + EPS).rsqrt()
        x = f * rstd[:, None] * st["gamma"].to(D)
        q, s = _exact_rows(x)
        out = {"h": h, "rstd": rstd, "q": q, "s": s}
        if case["colwise"]:
            out["qT"], out["sc"] = _exact_cols(x)
        return out
    if op == "norm_bwd":
        h, r, dx, w = st["h"].to(D), st["rstd"].to(D)[:, None], st["dx"].to(D), st["gamma"].to(D)
        dot = (dx * w * h).sum(1, keepdim=True)
        dh = r * dx * w - r.pow(3) / case["K"] * dot * h
        return {"dh": dh if st["dres"] is None else dh + st["dres"].to(D), "dgamma": (dx * h * r).sum(0)}
    if op == "gated":
        M, F, K = case["M"], case["F"], case["K"]
        if M * F * K > 2 ** 39:
            return None
        gu = torch.zeros(M, 2 * F, dtype=D, device="cuda")
        for k in range(K // 128):
            c = slice(128 * k, 128 * k + 128)
            part = st["xq"][:, c].view(FP8).to(D) @ st["wq"][:, c].contiguous().view(FP8).to(D).t()
            gu += part * st["xs"][k].to(D)[:, None] * st["ws"][:, k].to(D).repeat_interleave(128)
        g, u = gu[:, :F], gu[:, F:]
        q, s = _exact_rows(g * torch.sigmoid(g) * u)
        out = {"aq": q, "as": s}
        if case["checkpoint"]:
            out["guq"], out["gus"] = _exact_rows(gu)
        return out
    if op == "gated_bwd":
        M, F = case["M"], case["F"]
        gu = (st["guq"].view(FP8).to(D).reshape(M, 2 * F // 128, 128) * st["gus"].to(D).t()[:, :, None]).reshape(M, 2 * F)
        g, u, da = gu[:, :F], gu[:, F:], st["da"].to(D)
        sg = torch.sigmoid(g)
        d = torch.cat((da * u * (sg + g * sg * (1 - sg)), da * g * sg), 1)
        q, s = _exact_rows(d)
        qT, sc = _exact_cols(d)
        aT, ac = _exact_cols(g * sg * u)
        return {"q": q, "s": s, "qT": qT, "sc": sc, "aT": aT, "ac": ac}
    T, V = case["T"], case["V"]
    lps, lses, losses, grads = [], [], [], []
    names = ("lp_old", "lp_behav", "lp_ref", "adv", "weight")
    for a in range(0, T, 256):
        z = st["logits"][a:a + 256].to(D) / LOSS["temperature"]
        t = st["targets"][a:a + 256, None]
        lse = torch.logsumexp(z, 1)
        lp = z.gather(1, t)[:, 0] - lse
        lses.append(lse)
        if op == "logprobs":
            lps.append(lp)
            continue
        old, behav, ref, adv, weight = (None if st[n] is None else st[n][a:a + 256].to(D) for n in names)
        rho = (lp - old).exp()
        w = torch.ones_like(lp) if behav is None else (old - behav).exp().clamp(max=LOSS["tis_cap"])
        # the clipped branch is the smaller one above the range for a gain, below it for a loss
        out = ((adv > 0) & (rho > 1 + LOSS["eps_hi"])) | ((adv < 0) & (rho < 1 - LOSS["eps_lo"]))
        loss = -w * adv * torch.where(out, rho.clamp(1 - LOSS["eps_lo"], 1 + LOSS["eps_hi"]), rho)
        dlp = torch.where(out, torch.zeros_like(rho), -w * adv * rho)
        if ref is not None:
            loss = loss + LOSS["kl_beta"] * ((ref - lp).exp() - (ref - lp) - 1)
            dlp = dlp + LOSS["kl_beta"] * (1 - (ref - lp).exp())
        losses.append(weight * loss)
        lps.append(torch.where(weight == 0, torch.zeros_like(lp), lp))
        if case["grad"]:
            p = (z - lse[:, None]).exp()
            grads.append((weight * dlp / LOSS["temperature"])[:, None] * (torch.zeros_like(p).scatter_(1, t, 1.0) - p))
    if op == "logprobs":
        return {"lp": torch.cat(lps), "lse": torch.cat(lses)}
    out = {"loss": torch.cat(losses), "lp": torch.cat(lps)}
    if case["grad"]:
        out["dlogits"] = torch.cat(grads)
    return out
