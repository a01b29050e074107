"""The MXFP4 and log probability entry points where no CUDA device is to be had: an error status of
the call, whatever the sizes, and a process that goes on."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.path.insert(0, sys.argv[1])
from fp8_block_scaled_quantize_gb300 import rlq
F = 0x10000  # an aligned fake device address: nothing is launched
for args in {calls}:
    try:
        rlq.{name}(*args)
        print("ok")
    except rlq.RlqError as e:
        print(e.status)
"""
CUDA = "4"  # RLQ_ERR_CUDA


def statuses(name, calls):
    # (a process of its own, which sees no device on any machine)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(name=name, calls=calls), ROOT], capture_output=True, text=True,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), timeout=300)
    assert r.returncode == 0, f"exit {r.returncode}: {r.stderr[-500:]}"
    return r.stdout.split()


def test_product_of_every_size():
    calls = [f"(F, 2048, F, F, 2048, F, F, {dt}, 4096, {M}, {N}, {K}, None)" for M in (1, 64, 128, 129, 300, 8192)
             for N in (9, 16, 4096) for K in (0, 33, 4096) for dt in (0, 1)]
    assert statuses("rlq_gemm_mxfp4", "[" + ", ".join(calls) + "]") == [CUDA] * len(calls)


@pytest.mark.parametrize("name,calls", [
    ("rlq_quant_mxfp4", "[(F, 300, 128, 128, F, 64, F, F, 160, F, None), (F, 1, 128, 128, F, 64, F, None, 0, None, None)]"),
    ("rlq_dequant_mxfp4", "[(F, 32, F, 500, 45, F, 48, None), (F, 32, F, 1, 1, F, 48, None)]"),
    ("rlq_token_logprobs_top", "[(F, d, 100, r, 100, F, 1.0, 7, F, F, F, F, F, None) for d in (0, 1) for r in (1, 5000)]"),
    ("rlq_token_logprobs_backward", "[(F, d, 100, r, 100, F, 1.0, F, F, F, F, F, 100, None) for d in (0, 1) for r in (1, 5000)]")])
def test_operators_beside_it(name, calls):
    got = statuses(name, calls)
    assert got == [CUDA] * len(got) and len(got) >= 2
