"""CPU-side checks of the residual norm, gated block and loss entry points: every refusal
comes from the host before anything is launched (no GPU needed)."""
import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq

FAKE = 0x10000  # an aligned fake device address: validation never dereferences it
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


def status(fn, args):
    try:
        fn(*args)
        return 0
    except rlq.RlqError as e:
        return e.status


def refusals(fn, ok, cases):
    for change, want in cases:
        args = list(ok)
        for i, v in change.items():
            args[i] = v
        assert status(fn, args) == want, (fn.__name__, change)


def test_add_rmsnorm_refusals():
    #     res  ldr  delta ldd  M  K    gamma eps  h    ldh  rstd  q   ldq  s   lds qT  ldqT sc  ldsc stream
    ok = (FAKE, 256, FAKE, 256, 4, 256, FAKE, 1e-6, FAKE, 256, FAKE, FAKE, 256, FAKE, 4, FAKE, 16, FAKE, 256, None)
    refusals(rlq.rlq_add_rmsnorm_quant_act_1x128, ok, [
        ({4: -1}, INVALID), ({5: 200}, UNSUPPORTED), ({5: 16512}, UNSUPPORTED), ({4: 1 << 31}, UNSUPPORTED),
        ({0: None}, INVALID), ({1: 255}, INVALID), ({0: FAKE + 2}, MISALIGNED), ({1: 260}, MISALIGNED),
        ({3: 128}, INVALID), ({2: FAKE + 8}, MISALIGNED), ({6: None}, INVALID), ({6: FAKE + 4}, MISALIGNED),
        ({7: -1.0}, INVALID), ({7: float("nan")}, INVALID), ({8: None}, INVALID), ({9: 264, 8: FAKE}, INVALID),
        ({8: FAKE + 64, 9: 128}, INVALID), ({10: None}, INVALID), ({10: FAKE + 2}, MISALIGNED), ({11: None}, INVALID),
        ({12: 264}, MISALIGNED), ({14: 3}, INVALID), ({15: None}, INVALID), ({17: None}, INVALID), ({16: 3}, INVALID),
        ({16: 8}, MISALIGNED), ({18: 255}, INVALID)])
    # the sum written over delta needs delta's pitch
    refusals(rlq.rlq_add_rmsnorm_quant_act_1x128, ok, [({0: 4 * FAKE, 9: 264}, INVALID)])
    empty = (None, 0, None, 0, 0, 256, None, 0.0, None, 0, None, None, 0, None, 0, None, 0, None, 0, None)
    assert status(rlq.rlq_add_rmsnorm_quant_act_1x128, empty) == 0


def test_rmsnorm_backward_refusals():
    #     dx   lddx  h    ldh  rstd  gamma dres lddres dh  lddh dgamma M  K   ws  bytes stream
    ok = (FAKE, 256, FAKE, 256, FAKE, FAKE, FAKE, 256, FAKE, 256, FAKE, 4, 256, FAKE, 1 << 30, None)
    refusals(rlq.rlq_rmsnorm_backward, ok, [
        ({11: -1}, INVALID), ({12: 100}, UNSUPPORTED), ({12: 32768}, UNSUPPORTED), ({0: None}, INVALID),
        ({1: 248}, INVALID), ({2: FAKE + 2}, MISALIGNED), ({4: None}, INVALID), ({5: None}, INVALID),
        ({5: FAKE + 8}, MISALIGNED), ({7: 250}, INVALID), ({8: None}, INVALID), ({9: 264}, INVALID),
        ({10: None}, INVALID), ({10: FAKE + 4}, MISALIGNED), ({13: FAKE + 4}, MISALIGNED), ({14: -1}, INVALID)])
    assert rlq.rlq_rmsnorm_backward_workspace_bytes(0, 256) == 0
    with pytest.raises(rlq.RlqError):
        rlq.rlq_rmsnorm_backward_workspace_bytes(4, 100)


def test_gated_fprop_refusals():
    #     xq   ldxq  xs   ldxs wq   ldwq  ws  ldws aq   ldaq  as  ldas guq  ldguq gus ldgus M  F    K   stream
    ok = (FAKE, 256, FAKE, 4, FAKE, 256, FAKE, 2, FAKE, 128, FAKE, 4, FAKE, 256, FAKE, 4, 4, 128, 256, None)
    refusals(rlq.rlq_gemm_gated_fprop, ok, [
        ({16: -1}, INVALID), ({17: 100}, UNSUPPORTED), ({18: 100}, UNSUPPORTED), ({18: 0}, UNSUPPORTED),
        ({17: 1 << 30}, UNSUPPORTED), ({0: None}, INVALID), ({1: 128}, INVALID), ({1: 264}, MISALIGNED),
        ({3: 3}, INVALID), ({4: FAKE + 8}, MISALIGNED), ({5: 240}, INVALID), ({7: 1}, INVALID), ({8: None}, INVALID),
        ({9: 112}, INVALID), ({11: 3}, INVALID), ({12: None}, INVALID), ({14: None}, INVALID), ({13: 128}, INVALID),
        ({15: 3}, INVALID), ({10: FAKE + 2}, MISALIGNED)])
    assert status(rlq.rlq_gemm_gated_fprop, (None, 0) * 8 + (0, 128, 128, None)) == 0


def test_gated_backward_refusals():
    #     da  ldda guq  ldguq gus ldgus q   ldq  s   lds qT  ldqT sc  ldsc aT  ldaT ac  ldac M  F  stream
    ok = (FAKE, 128, FAKE, 256, FAKE, 4, FAKE, 256, FAKE, 4, FAKE, 16, FAKE, 256, FAKE, 16, FAKE, 128, 4, 128, None)
    refusals(rlq.rlq_gated_backward, ok, [
        ({18: -1}, INVALID), ({19: 64}, UNSUPPORTED), ({19: 1 << 30}, UNSUPPORTED), ({0: None}, INVALID),
        ({1: 120}, INVALID), ({2: FAKE + 1}, MISALIGNED), ({3: 128}, INVALID), ({5: 3}, INVALID), ({6: None}, INVALID),
        ({7: 240}, INVALID), ({9: 3}, INVALID), ({10: None}, INVALID), ({11: 20}, MISALIGNED), ({13: 255}, INVALID),
        ({14: None}, INVALID), ({15: 2}, INVALID), ({16: None}, INVALID), ({17: 127}, INVALID)])
    assert status(rlq.rlq_gated_backward, (None, 0) * 9 + (0, 128, None)) == 0


def test_loss_refusals():
    lp = rlq.rlq_token_logprobs
    #     logits dt ld   rows V  targets temp lp   lse stream
    ok = (FAKE, 0, 100, 4, 100, FAKE, 1.0, FAKE, FAKE, None)
    bad = [({1: 2}, INVALID), ({3: -1}, INVALID), ({4: 0}, INVALID), ({4: 1 << 30, 2: 1 << 31}, UNSUPPORTED), ({3: 1 << 28}, UNSUPPORTED), ({0: None}, INVALID),
           ({2: 99}, INVALID), ({0: FAKE + 1}, MISALIGNED), ({1: 1, 0: FAKE + 2}, MISALIGNED), ({5: None}, INVALID),
           ({5: FAKE + 4}, MISALIGNED), ({6: 0.0}, INVALID), ({6: float("inf")}, INVALID), ({6: -1.0}, INVALID)]
    refusals(lp, ok, bad + [({7: None}, INVALID), ({8: FAKE + 2}, MISALIGNED)])
    assert status(lp, (None, 0, 100, 0, 100, None, 1.0, None, None, None)) == 0
    pl = rlq.rlq_policy_loss
    #     0..6 as above, old adv weight behav ref clip eps_lo eps_hi cap beta loss lp dlogits ldd stream
    ok = ok[:7] + (FAKE,) * 6 + (0.2, 0.2, 2.0, 0.1, FAKE, FAKE, FAKE + 64, 100, None)
    refusals(pl, ok, bad + [
        ({7: None}, INVALID), ({8: None}, INVALID), ({9: None}, INVALID), ({10: FAKE + 1}, MISALIGNED),
        ({11: FAKE + 2}, MISALIGNED), ({12: FAKE + 2}, MISALIGNED), ({13: -0.1}, INVALID), ({13: 1.5}, INVALID),
        ({13: float("nan")}, INVALID), ({14: -1.0}, INVALID), ({14: float("inf")}, INVALID), ({15: 0.0}, INVALID),
        ({15: float("nan")}, INVALID), ({16: -1.0}, INVALID), ({17: None}, INVALID), ({18: None}, INVALID),
        ({20: 99}, INVALID), ({19: FAKE + 1}, MISALIGNED), ({19: FAKE, 20: 104}, INVALID)])


def test_subnormal_temperature_is_refused():
    """Its reciprocal would overflow."""
    ok = (FAKE, 0, 100, 4, 100, FAKE, 1.0, FAKE, FAKE, None)
    refusals(rlq.rlq_token_logprobs, ok, [({6: 1e-40}, INVALID), ({6: -1e-40}, INVALID), ({6: float("nan")}, INVALID)])


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU, so that the checks behind that one are reached."""

    is_cuda = True


def test_helpers_refuse_wrong_tensors():
    """Types, shapes, strides and CPU tensors are refused by name before a pointer is taken."""
    gpu = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)  # noqa: E731
    bf, f32, u8 = (gpu(4, 256, dtype=d) for d in (torch.bfloat16, torch.float32, torch.uint8))
    gamma, rstd, t64 = gpu(256, dtype=torch.bfloat16), gpu(4), gpu(4, dtype=torch.int64)
    gu, gus = gpu(4, 512, dtype=torch.uint8), gpu(4, 4)
    w, ws, xs = gpu(256, 256, dtype=torch.uint8), gpu(2, 2), gpu(2, 4)
    cpu = lambda t: torch.zeros(t.shape, dtype=t.dtype)  # noqa: E731
    for name, call in (("delta", lambda: rlq.add_rmsnorm_quant_act_1x128(bf, f32, gamma, 1e-6)),
                       ("res", lambda: rlq.add_rmsnorm_quant_act_1x128(f32, bf, gamma, 1e-6)),
                       ("gamma", lambda: rlq.add_rmsnorm_quant_act_1x128(bf, bf, gamma.float(), 1e-6)),
                       ("h", lambda: rlq.rmsnorm_backward(bf, f32, rstd, gamma)),
                       ("rstd", lambda: rlq.rmsnorm_backward(bf, bf, rstd.double(), gamma)),
                       ("xs", lambda: rlq.gemm_gated_fprop(u8, xs.double(), w, ws)),
                       ("da", lambda: rlq.gated_backward(f32, gu, gus)),
                       ("guq", lambda: rlq.gated_backward(bf, gu.float(), gus)),
                       ("logits", lambda: rlq.token_logprobs(bf.half(), t64)),
                       ("targets", lambda: rlq.token_logprobs(bf, t64.int())),
                       ("logp_old", lambda: rlq.policy_loss(bf, t64, rstd.double(), rstd, rstd))):
        with pytest.raises(TypeError, match=name):
            call()
    for name, call in (("delta", lambda: rlq.add_rmsnorm_quant_act_1x128(bf, bf[:2], gamma, 1e-6)),
                       ("gamma", lambda: rlq.add_rmsnorm_quant_act_1x128(bf, bf, gamma[:128], 1e-6)),
                       ("res", lambda: rlq.add_rmsnorm_quant_act_1x128(bf.t(), None, gamma[:4], 1e-6)),
                       ("res", lambda: rlq.add_rmsnorm_quant_act_1x128(bf[0], None, gamma, 1e-6)),
                       ("h", lambda: rlq.rmsnorm_backward(bf, bf[:, :128], rstd, gamma)),
                       ("rstd", lambda: rlq.rmsnorm_backward(bf, bf, rstd[:3], gamma)),
                       ("wq", lambda: rlq.gemm_gated_fprop(u8, xs, w[:, :128], ws)),
                       ("xs", lambda: rlq.gemm_gated_fprop(u8, xs[:1], w, ws)),
                       ("ws", lambda: rlq.gemm_gated_fprop(u8, xs, w, ws[:1])),
                       ("guq", lambda: rlq.gated_backward(bf, gu[:, :256], gus)),
                       ("gus", lambda: rlq.gated_backward(bf, gu, gus[:2])),
                       ("targets", lambda: rlq.token_logprobs(bf, t64[:3])),
                       ("logits", lambda: rlq.token_logprobs(bf[0], t64)),
                       ("logits", lambda: rlq.token_logprobs(bf.t(), gpu(256, dtype=torch.int64))),
                       ("logp_ref", lambda: rlq.policy_loss(bf, t64, rstd, rstd, rstd, logp_ref=rstd[:2])),
                       ("res", lambda: rlq.add_rmsnorm_quant_act_1x128(cpu(bf), bf, gamma, 1e-6)),
                       ("gamma", lambda: rlq.add_rmsnorm_quant_act_1x128(bf, bf, cpu(gamma), 1e-6)),
                       ("dres", lambda: rlq.rmsnorm_backward(bf, bf, rstd, gamma, dres=cpu(bf))),
                       ("ws", lambda: rlq.gemm_gated_fprop(u8, xs, w, cpu(ws))),
                       ("gus", lambda: rlq.gated_backward(bf, gu, cpu(gus))),
                       ("targets", lambda: rlq.token_logprobs(bf, cpu(t64))),
                       ("adv", lambda: rlq.policy_loss(bf, t64, rstd, cpu(rstd), rstd))):
        with pytest.raises(ValueError, match=name + " must"):
            call()
