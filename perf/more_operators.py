"""Workloads of the 4-bit rollout: microscaled layers, and what is recorded and trained of their logits.

Five operators, each in a plain form (elementary torch operations in 32 bits) and through the
library's calls (``own``):

* ``quant``       MXFP4 quantization (E2M1 elements, one power-of-two scale per 32 of them) along
                  the rows, and along the columns too, and the values read back
* ``linear``      a linear layer's forward pass: bf16 activations quantized, FP4 x FP4 product
* ``linear_bwd``  its backward pass: the output gradient quantized both ways, and both products
* ``top``         log probabilities of given tokens, with entropy and the most likely alternatives
* ``top_bwd``     gradient of any loss of log probabilities and entropy with respect to the logits

Weights, and the activations that a backward pass reads, are held as packed codes beside their
scales, as a user's program holds them.
"""
import math

import torch

own = False

TEMPERATURE = 0.9


def listed():
    return [
        # an 8B model's gate weight after an optimizer step, for the forward and the backward product
        {"name": "quant_weight", "op": "quant", "M": 14336, "K": 4096, "colwise": True},
        # a ragged micro-batch's activations in front of a 7B model's down projection
        {"name": "quant_odd", "op": "quant", "M": 333, "K": 18944, "colwise": False},
        # one new token through an 8B model's up projection
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 14336, "K": 4096, "dtype": "bf16"},
        # a rollout batch of 64 sequences through the 7B down projection: few outputs, a long sum
        {"name": "linear_rollout", "op": "linear", "M": 64, "N": 3584, "K": 18944, "dtype": "bf16"},
        # the same batch's logits
        {"name": "linear_head", "op": "linear", "M": 64, "N": 128256, "K": 4096, "dtype": "f32"},
        # the 8B training step's forward pass, or a long prompt's
        {"name": "linear_train", "op": "linear", "M": 8192, "N": 14336, "K": 4096, "dtype": "bf16"},
        # a ragged micro-batch's backward pass through a 7B up projection
        {"name": "linear_bwd_odd", "op": "linear_bwd", "M": 1001, "N": 18944, "K": 3584},
        # a rollout step of 64 sequences over a large vocabulary, with 20 alternatives recorded
        {"name": "top_rollout", "op": "top", "T": 64, "V": 151936, "dtype": "bf16", "top": 20, "masked": False},
        # decoding under a grammar: in some rows few tokens are allowed
        {"name": "top_grammar", "op": "top", "T": 600, "V": 32001, "dtype": "f32", "top": 5, "masked": True},
        # scoring a training batch
        {"name": "top_batch", "op": "top", "T": 2048, "V": 128256, "dtype": "bf16", "top": 20, "masked": False},
        # the entropy bonus of a small batch, fp32 logits
        {"name": "top_bwd_f32", "op": "top_bwd", "T": 600, "V": 32001, "dtype": "f32", "lp": False, "entropy": True},
        # the training step's gradient: a loss of log probabilities with an entropy bonus
        {"name": "top_bwd_train", "op": "top_bwd", "T": 4096, "V": 128256, "dtype": "bf16", "lp": True,
         "entropy": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear_bwd", "top", "top_bwd"])
    if op == "quant":
        return {"op": op, "M": _log_int(rng, 1, 8192), "K": 32 * _log_int(rng, 1, 448), "colwise": rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 8, 14336), "K": 32 * _log_int(rng, 1, 128),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "linear_bwd":
        return {"op": op, "M": _log_int(rng, 1, 4096), "N": 32 * _log_int(rng, 1, 448), "K": 32 * _log_int(rng, 1, 128)}
    c = {"op": op, "T": _log_int(rng, 1, 2048), "V": _log_int(rng, 64, 128256), "dtype": rng.choice(["bf16", "f32"])}
    if op == "top":
        c.update(top=rng.choice([0, 1, 5, 20, 64]), masked=rng.random() < 0.3)
    else:
        c["lp"] = rng.random() < 0.7
        c["entropy"] = not c["lp"] or rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs ---

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _activations(g, M, K):
    """A layer's input: normal values with a few large channels, as trained models have."""
    big = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return (torch.randn(M, K, generator=g, device="cuda") * big).to(torch.bfloat16)


MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the E2M1 codes 0 .. 7


def _quant(x):
    """E2M1 codes [R, C] (sign in bit 3) and scale exponents [R, ceil(C / 32)] of the groups of 32 along x's rows."""
    R, C = x.shape
    nb = -(-C // 32)
    g = torch.nn.functional.pad(x.float(), (0, nb * 32 - C)).view(R, nb, 32)
    amax = g.abs().amax(2)
    # amax = m 2^k with m in [1/2, 1): the largest element's exponent is k - 1, and E2M1's largest is 2
    e = torch.where(amax == 0, -127, torch.frexp(amax)[1] - 3).clamp(-127, 127)
    v = torch.ldexp(g, -e[:, :, None])  # a power of two: exact
    a = v.abs()
    # to the nearest magnitude; a tie goes to the even code
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5
    code += 8 * torch.signbit(v).to(torch.uint8)
    return code.view(R, nb * 32)[:, :C], e


def _pack(code):
    """Two codes a byte, the even one in the low bits, rows of 16-byte-aligned pitch."""
    R, C = code.shape
    buf = torch.zeros((R, -(-C // 32) * 32), dtype=torch.uint8, device="cuda")
    buf[:, :C] = code
    return (buf[:, ::2] | buf[:, 1::2] << 4)[:, :(C + 1) // 2]


def _tiled(e):
    """Scale bytes (exponent + 127) in tiles of 128 rows x 4 groups: [row tile, group tile, row % 32,
    row % 128 / 32, group % 4]."""
    R, nb = e.shape
    rt, ct = -(-R // 128), -(-nb // 4)
    s = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device="cuda")
    s[:R, :nb] = (e + 127).to(torch.uint8)
    return s.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous()


def _held(x):
    """Packed codes and tiled scales of x's rows."""
    code, e = _quant(x)
    return _pack(code), _tiled(e)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case)
    if op == "quant":
        st["x"] = _activations(g, case["M"], case["K"])
    elif op == "linear":
        st["x"] = _activations(g, case["M"], case["K"])
        st["wq"], st["ws"] = _held(_normal(g, case["N"], case["K"], std=0.02))
    elif op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        st["dy"] = _normal(g, M, N, std=1e-3)
        # the weight's and the forward pass's activations' codes along the columns
        st["wTq"], st["wTs"] = _held(_normal(g, K, N, std=0.02))
        st["xTq"], st["xTs"] = _held(_activations(g, M, K).t().contiguous())
    else:
        T, V = case["T"], case["V"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # rows start on 16 bytes, as a head with a padded vocabulary writes them
        ld = -(-V // 8) * 8
        logits = torch.randn(T, ld, generator=g, device="cuda").mul_(2.0).to(dt)[:, :V]
        targets = torch.randint(0, V, (T,), generator=g, device="cuda")
        rows = torch.arange(T, device="cuda")
        # sampled tokens are likely ones
        logits[rows, targets] = (2.0 * math.log(V) / 3 + 3.0 + torch.randn(T, generator=g, device="cuda")).to(dt)
        if op == "top" and case["masked"]:
            # a third of the rows: one token in 8 allowed, or one in 4096, the sampled one among them
            u = torch.rand(T, generator=g, device="cuda")
            keep = torch.where(u < 0.15, 1 / 4096, torch.where(u < 0.33, 1 / 8, 2.0))
            allowed = torch.rand(T, V, generator=g, device="cuda") < keep[:, None]
            allowed[rows, targets] = True
            logits.masked_fill_(~allowed, -math.inf)
        st.update(logits=logits, targets=targets)
        if op == "top_bwd":
            z = logits.double() / TEMPERATURE
            lse = torch.logsumexp(z, 1)
            st["H"] = (lse - (torch.exp(z - lse[:, None]) * z).sum(1)).float()
            st["lse"] = lse.float()
            # prompt and padding tokens weigh nothing; the loss is a mean over the others
            weight = (torch.rand(T, generator=g, device="cuda") < 0.85).float() / T
            st["dlp"] = weight * torch.randn(T, generator=g, device="cuda") if case["lp"] else None
            st["dH"] = -0.01 * weight if case["entropy"] else None
    return st


# ------------------------------------------------------------------ runs ---

def run(st):
    return (_run_own if own else _run_plain)(st)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _run_own(st):
    from fp8_block_scaled_quantize_gb300 import rlq

    op = st["op"]
    if op == "quant":
        q, s, qT, sT = rlq.quant_mxfp4(st["x"], colwise=st["colwise"])
        out = {"x": rlq.dequant_mxfp4(q, s)}
        if st["colwise"]:
            out["xT"] = rlq.dequant_mxfp4(qT, sT, cols=st["M"])
        return out
    if op == "linear":
        q, s, _, _ = rlq.quant_mxfp4(st["x"])
        return {"y": rlq.gemm_mxfp4(q, s, st["wq"], st["ws"], out_dtype=_dtype(st["dtype"]))}
    if op == "linear_bwd":
        q, s, qT, sT = rlq.quant_mxfp4(st["dy"], colwise=True)
        return {"dx": rlq.gemm_mxfp4(q, s, st["wTq"], st["wTs"]), "dw": rlq.gemm_mxfp4(qT, sT, st["xTq"], st["xTs"])}
    if op == "top":
        lp, lse, H, ids, top_lp = rlq.token_logprobs_top(st["logits"], st["targets"], top=st["top"],
                                                         temperature=TEMPERATURE)
        return {"lp": lp, "lse": lse, "H": H, "ids": ids, "top_lp": top_lp}
    return {"dlogits": rlq.token_logprobs_backward(st["logits"], st["targets"], st["lse"], st["H"], dlp=st["dlp"],
                                                   dentropy=st["dH"], temperature=TEMPERATURE)}


def _values(q, s, C):
    """fp32 values [R, C] of packed codes and tiled scales."""
    R = q.shape[0]
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")
    code = torch.stack((q & 15, q >> 4), 2).view(R, -1)[:, :C]
    e = s.permute(0, 3, 2, 1, 4).reshape(s.shape[0] * 128, -1)[:R, :-(-C // 32)].int() - 127
    return torch.ldexp(table[code.int()], e.repeat_interleave(32, 1)[:, :C])


def _rounded(x):
    """x's rows as MXFP4 holds them, in fp32."""
    code, e = _quant(x)
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")
    return torch.ldexp(table[code.int()], e.repeat_interleave(32, 1)[:, :x.shape[1]])


def _run_plain(st):
    op = st["op"]
    if op == "quant":
        out = {"x": _rounded(st["x"]).to(torch.bfloat16)}
        if st["colwise"]:
            out["xT"] = _rounded(st["x"].t().contiguous()).to(torch.bfloat16)
        return out
    if op == "linear":
        return {"y": (_rounded(st["x"]) @ _values(st["wq"], st["ws"], st["K"]).t()).to(_dtype(st["dtype"]))}
    if op == "linear_bwd":
        dx = _rounded(st["dy"]) @ _values(st["wTq"], st["wTs"], st["N"]).t()
        dw = _rounded(st["dy"].t().contiguous()) @ _values(st["xTq"], st["xTs"], st["M"]).t()
        return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}
    z = st["logits"].float() / TEMPERATURE
    if op == "top":
        top = z.amax(1, keepdim=True)
        z = z - top
        e = torch.exp(z)
        total = e.sum(1)
        log_total = torch.log(total)
        H = log_total - torch.where(e == 0, torch.zeros_like(e), e * z).sum(1) / total
        lp = z.gather(1, st["targets"][:, None])[:, 0] - log_total
        k = min(st["top"], st["V"])
        # the largest logits; among equal ones the lowest token
        ids = torch.sort(st["logits"], dim=1, descending=True, stable=True)[1][:, :k]
        return {"lp": lp, "lse": top[:, 0] + log_total, "H": H, "ids": ids,
                "top_lp": z.gather(1, ids) - log_total[:, None]}
    logp = z - st["lse"][:, None]
    p = torch.exp(logp)
    zero = torch.zeros_like(st["lse"])
    dlp = zero if st["dlp"] is None else st["dlp"]
    d = -dlp[:, None] * p
    if st["dH"] is not None:
        d -= st["dH"][:, None] * torch.where(p == 0, torch.zeros_like(p), p * (logp + st["H"][:, None]))
    d.scatter_add_(1, st["targets"][:, None], dlp[:, None])
    return {"dlogits": (d / TEMPERATURE).to(st["logits"].dtype)}


# ------------------------------------------------------- work and 64 bits ---

def _held_bytes(R, C):
    return R * -(-C // 2) + R * -(-C // 32)


def work(case):
    op = case["op"]
    if op == "quant":
        M, K = case["M"], case["K"]
        ways = 2 if case["colwise"] else 1
        # x read once; codes and scales written, and read to write the values
        codes = _held_bytes(M, K) + (_held_bytes(K, M) if case["colwise"] else 0)
        return {"bytes": 2 * M * K + 2 * codes + ways * 2 * M * K, "flops": ways * 4 * M * K}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + _held_bytes(N, K) + M * N * (2 if case["dtype"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * N + _held_bytes(K, N) + _held_bytes(K, M) + 2 * M * K + 2 * N * K,
                "flops": 4 * M * N * K}
    T, V = case["T"], case["V"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "top":
        return {"bytes": T * V * e + T * (20 + 12 * min(case["top"], V)), "flops": 6 * T * V}
    return {"bytes": 2 * T * V * e + 24 * T, "flops": 8 * T * V}


def _exact_round(x):
    """x's rows as the definition rounds them: 2^floor(log2 amax) is four units, steps of 1/2 below 2,
    of 1 below 4, of 2 above, halves to even, at most 6."""
    R, C = x.shape
    nb = -(-C // 32)
    g = torch.zeros(R, nb * 32, dtype=torch.float64, device="cuda")
    g[:, :C] = x
    g = g.view(R, nb, 32)
    a = g.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(a))  # may be one off next to a power of two
    e += (torch.exp2(e + 1) <= a).to(e.dtype) - (torch.exp2(e) > a).to(e.dtype)
    u = torch.exp2(torch.where(a > 0, e - 2, torch.full_like(a, -127.0)).clamp_(-127, 127))
    v = g / u
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(torch.float64)
    return ((torch.round(v / step) * step).clamp_(-6, 6) * u).view(R, nb * 32)[:, :C]


def _exact_values(q, s, C):
    table = torch.tensor([(1 - 2 * (c >> 3)) * MAGNITUDES[c & 7] for c in range(16)], dtype=torch.float64, device="cuda")
    out = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device="cuda")
    out[:, 0::2] = table[(q % 16).long()]
    out[:, 1::2] = table[(q // 16).long()]
    out = out[:, :C]
    r = torch.arange(q.shape[0], device="cuda")[:, None]
    b = torch.arange(C, device="cuda")[None, :] // 32
    return out * torch.exp2(s[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].double() - 127)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    D = torch.float64
    if op == "quant":
        out = {"x": _exact_round(st["x"].to(D))}
        if case["colwise"]:
            out["xT"] = _exact_round(st["x"].to(D).t())
        return out
    if op == "linear":
        return {"y": _exact_round(st["x"].to(D)) @ _exact_values(st["wq"], st["ws"], case["K"]).t()}
    if op == "linear_bwd":
        dy = st["dy"].to(D)
        return {"dx": _exact_round(dy) @ _exact_values(st["wTq"], st["wTs"], case["N"]).t(),
                "dw": _exact_round(dy.t()) @ _exact_values(st["xTq"], st["xTs"], case["M"]).t()}
    T, V = case["T"], case["V"]
    parts = []
    for a in range(0, T, 256):
        x, t = st["logits"][a:a + 256], st["targets"][a:a + 256, None]
        z = x.to(D) / TEMPERATURE
        if op == "top":
            lse = torch.logsumexp(z, 1, keepdim=True)
            lg = z - lse
            ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :min(case["top"], V)]
            parts.append((lg.gather(1, t)[:, 0], lse[:, 0], -torch.special.xlogy(lg.exp(), lg.exp()).sum(1), ids,
                          lg.gather(1, ids)))
            continue
        p = torch.exp(z - st["lse"][a:a + 256, None].to(D))
        d = torch.zeros_like(p)
        if st["dlp"] is not None:
            d += st["dlp"][a:a + 256, None].to(D) * (torch.zeros_like(p).scatter_(1, t, 1.0) - p)
        if st["dH"] is not None:
            d -= st["dH"][a:a + 256, None].to(D) * (torch.special.xlogy(p, p) + p * st["H"][a:a + 256, None].to(D))
        parts.append((d / TEMPERATURE,))
    cat = [torch.cat(c) for c in zip(*parts)]
    if op == "top":
        return dict(zip(("lp", "lse", "H", "ids", "top_lp"), cat))
    return {"dlogits": cat[0]}
