"""The element helpers' scale and reciprocal, formed by correction steps, against the
correctly rounded operations for every finite value (2^31 of them)."""
import os
import subprocess

import pytest

from fp8_block_scaled_quantize_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_scale_and_reciprocal(tmp_path):
    exe = str(tmp_path / "scale_rule")
    flags = [f for f in build.NVCC_FLAGS if f not in ("-Xptxas", "-v")]  # the library's own, no fast-math
    r = subprocess.run([build._nvcc(), *build.ARCH, *flags, "-I", build.CSRC,
                        os.path.join(HERE, "scale_rule", "scale_rule.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split() == ["0", "0"], "differences (scales, reciprocals): " + r.stdout
