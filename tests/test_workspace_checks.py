"""CPU checks of a workspace that the caller brings: the kernels write all of its bytes as
plain device memory, so anything else is refused before its address is taken."""
import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq
from test_stream_scratch import OnGpu, gpu

BAD = {
    "on the CPU": torch.zeros(1 << 20, dtype=torch.uint8),
    "more elements than memory": torch.zeros(16, dtype=torch.uint8).as_subclass(OnGpu).expand(1 << 16, 16),
    "gaps that are others'": torch.zeros((64, 1 << 15), dtype=torch.uint8).as_subclass(OnGpu)[:, :1 << 14],
}


def norm_backward(ws):
    x = gpu(4, 256, dtype=torch.bfloat16)
    rlq.rmsnorm_backward(x, x, gpu(4), gpu(256, dtype=torch.bfloat16), workspace=ws)


def wgrad(ws):
    rlq.gemm_wgrad_accumulate_(gpu(128, 256), gpu(128, 512, dtype=torch.uint8), gpu(4, 128),
                               gpu(256, 512, dtype=torch.uint8), gpu(4, 256), workspace=ws)


def fprop(ws):
    rlq.gemm_fprop(gpu(4, 256, dtype=torch.uint8), gpu(2, 4), gpu(128, 256, dtype=torch.uint8), gpu(1, 2),
                   out=gpu(4, 128, dtype=torch.bfloat16), split_k=True, workspace=ws)


@pytest.mark.parametrize("call", [norm_backward, wgrad, fprop])
@pytest.mark.parametrize("what", BAD)
def test_workspace_is_refused(call, what, monkeypatch):
    def launched(*args):
        raise AssertionError("reached the library")

    monkeypatch.setattr(rlq, "_call", launched)
    with pytest.raises(ValueError, match="workspace must be"):
        call(BAD[what])
