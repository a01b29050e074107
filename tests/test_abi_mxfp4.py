"""CPU-side checks of the MXFP4 entry points: every refusal comes from the host before anything
is launched (no GPU needed), and the reference form against a second statement of the rule."""
import pytest
import torch

import mx_ref as R
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


def test_quant_refusals():
    #     x    M  K    ldx  q    ldq s     qT   ldqT sT   stream
    ok = (FAKE, 5, 128, 128, FAKE, 64, FAKE, FAKE, 16, FAKE, None)
    refusals(rlq.rlq_quant_mxfp4, ok, [
        ({1: -1}, INVALID), ({2: -32}, INVALID), ({2: 100}, UNSUPPORTED), ({1: 1 << 31}, UNSUPPORTED),
        ({0: None}, INVALID), ({3: 120}, INVALID), ({0: FAKE + 8}, MISALIGNED), ({3: 132}, MISALIGNED),
        ({4: None}, INVALID), ({5: 48}, INVALID), ({5: 72}, MISALIGNED), ({4: FAKE + 4}, MISALIGNED),
        ({6: None}, INVALID), ({6: FAKE + 8}, MISALIGNED), ({7: None}, INVALID), ({9: None}, INVALID),
        ({8: 2}, INVALID), ({8: 24}, MISALIGNED), ({7: FAKE + 1}, MISALIGNED), ({9: FAKE + 8}, MISALIGNED)])
    assert status(rlq.rlq_quant_mxfp4, (None, 0, 128, 0, None, 0, None, None, 0, None, None)) == 0


def test_dequant_refusals():
    #     q    ldq s     rows cols x    ldx stream
    ok = (FAKE, 32, FAKE, 5, 45, FAKE, 48, None)
    refusals(rlq.rlq_dequant_mxfp4, ok, [
        ({3: -1}, INVALID), ({4: -1}, INVALID), ({3: 1 << 31}, UNSUPPORTED), ({0: None}, INVALID), ({1: 16}, INVALID),
        ({1: 40}, MISALIGNED), ({0: FAKE + 1}, MISALIGNED), ({2: None}, INVALID), ({2: FAKE + 4}, MISALIGNED),
        ({5: None}, INVALID), ({6: 40}, INVALID), ({6: 47}, MISALIGNED), ({5: FAKE + 2}, MISALIGNED)])
    assert status(rlq.rlq_dequant_mxfp4, (None, 0, None, 0, 45, None, 0, None)) == 0


def test_gemm_refusals():
    #     xq   ldx xs    wq   ldw ws    y    dtype ldy M N K  stream
    ok = (FAKE, 32, FAKE, FAKE, 32, FAKE, FAKE, 0, 9, 5, 9, 64, None)
    refusals(rlq.rlq_gemm_mxfp4, ok, [
        ({9: -1}, INVALID), ({10: -1}, INVALID), ({11: -1}, INVALID), ({7: 2}, INVALID), ({11: 1 << 31}, UNSUPPORTED),
        ({0: None}, INVALID), ({1: 16}, INVALID), ({1: 40}, MISALIGNED), ({0: FAKE + 8}, MISALIGNED),
        ({2: None}, INVALID), ({2: FAKE + 8}, MISALIGNED), ({3: None}, INVALID), ({4: 16}, INVALID),
        ({4: 33}, MISALIGNED), ({3: FAKE + 8}, MISALIGNED), ({5: None}, INVALID), ({5: FAKE + 1}, MISALIGNED),
        ({6: None}, INVALID), ({8: 8}, INVALID), ({6: FAKE + 1}, MISALIGNED), ({7: 1, 6: FAKE + 2}, MISALIGNED)])
    assert status(rlq.rlq_gemm_mxfp4, (None, 0, None, None, 0, None, None, 0, 0, 0, 9, 64, None)) == 0
    assert status(rlq.rlq_gemm_mxfp4, (None, 0, None, None, 0, None, None, 0, 0, 5, 0, 64, None)) == 0


def test_helpers_refuse_before_the_library():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rlq.quant_mxfp4(cpu)
    with pytest.raises(TypeError):
        rlq.quant_mxfp4(cpu.float())
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        rlq.quant_mxfp4(cpu[0])
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(rlq.mxfp4_scales_shape(4, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        rlq.dequant_mxfp4(q, s)
    with pytest.raises(TypeError):
        rlq.gemm_mxfp4(q.float(), s, q, s)


def test_scales_shape():
    assert rlq.mxfp4_scales_shape(1, 32) == (1, 1, 32, 4, 4)
    assert rlq.mxfp4_scales_shape(129, 4096) == (2, 32, 32, 4, 4)
    assert rlq.mxfp4_scales_shape(0, 160) == (0, 2, 32, 4, 4)


def test_reference_rule_and_layout():
    """The 64-bit form against the rule stated by distances: no E2M1 value is nearer than the one
    taken, and a tie has an even code; the tiles' formula element by element."""
    x = torch.cat((torch.arange(-40, 41) / 5.0, torch.arange(-33, 34) / 4.0, torch.randn(44)))[:192].view(2, 96)
    x[0, 32:64] *= 2.0 ** -30
    code, s = R.quantize(x)
    v = R.values(code, s)
    e = (s.int() - 127).repeat_interleave(32, 1)
    amax = x.abs().view(2, 3, 32).amax(2).repeat_interleave(32, 1)
    assert bool((2.0 ** (e + 2.0) <= amax).all()) and bool((amax < 2.0 ** (e + 3.0)).all())
    grid = torch.tensor(R.MAGNITUDES + [-m for m in R.MAGNITUDES], dtype=torch.float64) * 2.0 ** e[:, :, None].double()
    dist = (x[:, :, None].double() - grid).abs()
    mine = (x.double() - v).abs()
    assert bool((mine <= dist.amin(2)).all())
    ties = (dist == mine[:, :, None]).sum(2) - (v == 0).int()  # (both zeros are as near)
    assert bool((code[ties > 1] % 2 == 0).all()) and bool((ties > 1).any())
    s = torch.randint(0, 255, (300, 9), dtype=torch.uint8)
    t = R.tile(s).view(-1)
    for m, b in ((0, 0), (31, 3), (32, 4), (127, 8), (128, 0), (299, 7)):
        at = ((m // 128) * 3 + b // 4) * 512 + (m % 32) * 16 + (m % 128) // 32 * 4 + b % 4
        assert t[at] == s[m, b]
    assert torch.equal(R.untile(R.tile(s), 300)[:, :9], s)
    c = torch.randint(0, 16, (5, 33), dtype=torch.uint8)
    assert torch.equal(R.unpack(R.pack(c), 33), c)
