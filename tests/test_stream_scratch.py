"""CPU checks of where a helper's own scratch comes from: the pool of the stream that the
call names.  From the current stream's pool it could still be in use by work queued there."""
import contextlib

import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq

SCRATCH = 4096  # bytes that the faked plans ask for


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""

    is_cuda = True


@pytest.fixture
def pools(monkeypatch):
    """Pools (stream handles, None: the current stream's) that scratch was taken from."""
    made, active = [], [None]
    empty = torch.empty

    @contextlib.contextmanager
    def stream(handle):
        active.append(handle)
        yield
        active.pop()

    def record(size, *args, **kw):
        if size == SCRATCH:
            made.append(active[-1])
        return empty(size, *args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", record)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 7, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(rlq, "_norm_workspace_bytes", lambda *shape: SCRATCH)
    monkeypatch.setattr(rlq, "rlq_gemm_splitk_workspace_bytes", lambda *shape: SCRATCH)
    monkeypatch.setattr(rlq, "_call", lambda name, *args: 0)
    return made


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


def norm_backward(stream):
    x = gpu(4, 256, dtype=torch.bfloat16)
    rlq.rmsnorm_backward(x, x, gpu(4), gpu(256, dtype=torch.bfloat16), stream=stream)


def split_k(name):
    a, b, sa, sb = gpu(128, 256, dtype=torch.uint8), gpu(128, 256, dtype=torch.uint8), gpu(2, 128), gpu(2, 256)
    if name == "gemm_wgrad_accumulate_":
        return lambda stream: rlq.gemm_wgrad_accumulate_(gpu(128, 128), a, sa, b, sb, stream=stream)
    if name == "gemm_nvfp4_weight_only":
        return lambda stream: rlq.gemm_nvfp4_weight_only(gpu(4, 512, dtype=torch.bfloat16), a, sa, sb, split_k=True,
                                                         stream=stream)
    return lambda stream: getattr(rlq, name)(a, sa, b, sb, split_k=True, stream=stream)


CALLS = {"rmsnorm_backward": norm_backward}
CALLS.update((n, split_k(n)) for n in ("gemm_fprop", "gemm_dgrad", "gemm_wgrad", "gemm_fprop_per_channel",
                                       "gemm_wgrad_accumulate_", "gemm_nvfp4_weight_only"))


@pytest.mark.parametrize("name", CALLS)
def test_scratch_is_the_named_streams(name, pools):
    CALLS[name](None)
    CALLS[name](0x5000)
    CALLS[name](0)  # the default stream's handle
    assert pools == [None, 0x5000, "default"]
