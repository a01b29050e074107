"""GPU tests of the operators around the layer where the launch itself changes: shared
memory beyond what a kernel has unasked, host threads that call at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_actor import D, DEV, gen, norm_bwd_reference, normal

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_norm_backward(M, K):
    g = gen(M + 3 * K)
    h, dx, dres = normal(g, M, K), normal(g, M, K, std=1e-3), normal(g, M, K, std=1e-3)
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dh, dgamma = rlq.rmsnorm_backward(dx, h, rstd, gamma, dres=dres)
    want, err, wg, gerr = norm_bwd_reference(dx, h, rstd, gamma, dres)
    assert bool(((dh.to(D) - want).abs() <= err).all())
    assert bool(((dgamma.to(D) - wg).abs() <= gerr).all())


# the column sums and the rows' partials together pass 48 KB between 12160 and 12416
@pytest.mark.parametrize("K", [12160, 12288, 12416])
def test_rmsnorm_backward_is_the_first_call_of_a_process(K):
    """No earlier call has raised the kernel's shared memory limit."""
    code = f"import sys; sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]; " \
           f"from test_gpu_actor_limits import check_norm_backward as f; f(3, {K}); f(160, {K})"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("K", [12160, 12288, 12416])
@pytest.mark.parametrize("M", [1, 5, 200])
def test_rmsnorm_backward_around_48_kb(M, K):
    check_norm_backward(M, K)


def test_rmsnorm_backward_from_two_host_threads():
    """One thread's smaller K leaves the other's larger one launchable.  (Through the bare
    entry point, which runs without the interpreter's lock.)"""
    fn, errors = rlq.lib().rlq_rmsnorm_backward, []

    def calls(K):
        dx = torch.ones((2, K), dtype=torch.bfloat16, device=DEV)
        dh, dgamma = torch.empty_like(dx), torch.empty(K, device=DEV)
        gamma, rstd = torch.ones(K, dtype=torch.bfloat16, device=DEV), torch.ones(2, device=DEV)
        ws = torch.empty(2 * K * 4, dtype=torch.uint8, device=DEV)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        args = (dx.data_ptr(), K, dx.data_ptr(), K, rstd.data_ptr(), gamma.data_ptr(), None, 0, dh.data_ptr(), K,
                dgamma.data_ptr(), 2, K, ws.data_ptr(), ws.numel(), s.cuda_stream)
        errors.extend(st for st in (fn(*args) for _ in range(20000)) if st)
        s.synchronize()

    threads = [threading.Thread(target=calls, args=(K,)) for K in (16384, 12416)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, (len(errors), errors[0])
