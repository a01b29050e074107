"""GPU tests of helpers that bring their own scratch, called on two streams at once."""
import pytest
import torch

import actor_ref as R
from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_actor import DEV, gen, normal

pytestmark = pytest.mark.gpu


def norm_backward():
    M, K = 2048, 4096
    sets = []
    for seed in (1, 2):
        g = gen(seed)
        h, dx = normal(g, M, K), normal(g, M, K)
        sets.append((dx, h, torch.rsqrt(h.float().square().mean(1)), torch.ones(K, dtype=torch.bfloat16, device=DEV)))
    return lambda i, stream: rlq.rmsnorm_backward(*sets[i], stream=stream)


def split_k():
    M, N, K = 64, 4096, 14336
    wq, ws = R.quant_blocks(normal(gen(3), N, K))
    sets = [R.quant_rows(normal(gen(4 + i), M, K)) for i in range(2)]
    assert rlq.rlq_gemm_splitk_workspace_bytes(rlq.GEMM_FPROP, M, N, K) > 0
    return lambda i, stream: (rlq.gemm_fprop(*sets[i], wq, ws, split_k=True, stream=stream),)


@pytest.mark.parametrize("make", [norm_backward, split_k])
def test_two_streams_at_once(make):
    """Calls of the same shapes on the current stream and on a named one, nothing between
    them: each result is that of the call alone.  (All outputs are kept until the end, so
    that no block of one is another's.)"""
    call = make()
    want = [call(i, None) for i in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        got = [(call(0, None), call(1, handle)) for _ in range(20)]
        torch.cuda.synchronize()
        for a, b in got:
            assert all(map(torch.equal, a, want[0])) and all(map(torch.equal, b, want[1]))


def test_the_default_streams_handle():
    call = norm_backward()
    want = call(0, None)
    got = call(0, 0)
    torch.cuda.synchronize()
    assert all(map(torch.equal, want, got))
