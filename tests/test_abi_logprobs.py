"""CPU-side checks of the log probabilities with entropy and alternatives and of their gradient:
every refusal comes from the host before anything is launched (no GPU needed)."""
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


def test_top_refusals():
    #     logits dtype ld rows V targets temp top lp lse H  ids  top_lp stream
    ok = (FAKE, 0, 100, 5, 100, FAKE, 1.0, 7, FAKE, FAKE, FAKE, FAKE, FAKE, None)
    refusals(rlq.rlq_token_logprobs_top, ok, [
        ({1: 2}, INVALID), ({3: -1}, INVALID), ({4: 0}, INVALID), ({4: 1 << 30}, UNSUPPORTED), ({3: 1 << 28}, UNSUPPORTED),
        ({6: 0.0}, INVALID), ({6: float("nan")}, INVALID), ({6: 1e-40}, INVALID), ({0: None}, INVALID), ({2: 99}, INVALID),
        ({0: FAKE + 1}, MISALIGNED), ({1: 1, 0: FAKE + 2}, MISALIGNED), ({5: None}, INVALID), ({5: FAKE + 4}, MISALIGNED),
        ({7: -1}, INVALID), ({7: 101}, INVALID), ({7: 65}, UNSUPPORTED), ({8: None}, INVALID), ({9: None}, INVALID),
        ({10: None}, INVALID), ({8: FAKE + 2}, MISALIGNED), ({10: FAKE + 1}, MISALIGNED), ({11: None}, INVALID),
        ({11: FAKE + 4}, MISALIGNED), ({12: None}, INVALID), ({12: FAKE + 2}, MISALIGNED)])
    assert status(rlq.rlq_token_logprobs_top, (None, 0, 0, 0, 100, None, 1.0, 7, None, None, None, None, None, None)) == 0


def test_backward_refusals():
    #     logits dtype ld rows V targets temp lse  H   dlp  dH  dlogits ldd stream
    ok = (FAKE, 1, 100, 5, 100, FAKE, 1.0, FAKE, FAKE, FAKE, FAKE, 4 * FAKE, 104, None)
    refusals(rlq.rlq_token_logprobs_backward, ok, [
        ({1: -1}, INVALID), ({3: -1}, INVALID), ({6: -1.0}, INVALID), ({0: None}, INVALID), ({5: None}, INVALID),
        ({9: None, 10: None}, INVALID), ({7: None}, INVALID), ({8: None}, INVALID), ({7: FAKE + 2}, MISALIGNED),
        ({8: FAKE + 1}, MISALIGNED), ({9: FAKE + 2}, MISALIGNED), ({10: FAKE + 2}, MISALIGNED), ({11: None}, INVALID),
        ({12: 99}, INVALID), ({11: FAKE + 2}, MISALIGNED), ({11: FAKE}, INVALID)])  # (in place with another pitch)
    assert status(rlq.rlq_token_logprobs_backward,
                  (None, 0, 0, 0, 100, None, 1.0, None, None, None, None, None, 0, None)) == 0


def test_helpers_refuse_before_the_library():
    z, t, f = torch.zeros(3, 10), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        rlq.token_logprobs_top(z, t)
    with pytest.raises(TypeError):
        rlq.token_logprobs_top(z.half(), t)
    with pytest.raises(ValueError, match="CUDA"):
        rlq.token_logprobs_backward(z, t, f, dlp=f)
