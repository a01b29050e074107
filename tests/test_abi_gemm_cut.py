"""CPU-side checks of the diagnostic that tells how a product is cut."""
import pytest

from fp8_block_scaled_quantize_gb300 import rlq

INVALID, UNSUPPORTED = 1, 2


def test_refusals():
    for args, status in (((0, 8, 8, 0, 1), INVALID), ((8, -1, 8, 0, 1), INVALID), ((8, 8, 0, 0, 1), INVALID),
                         ((8, 8, 8, 2, 1), INVALID), ((1 << 31, 8, 8, 0, 1), UNSUPPORTED), ((8, 8, 1 << 31, 1, 0), UNSUPPORTED)):
        with pytest.raises(rlq.RlqError) as e:
            rlq.rlq_diag_gemm_mxfp4_cut(*args)
        assert e.value.status == status
    with pytest.raises(rlq.RlqError) as e:
        rlq._call("rlq_diag_gemm_mxfp4_cut", 8, 8, 8, 0, 1, None)
    assert e.value.status == INVALID


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 4096), (64, 300, 20000), (300, 5001, 64), (8192, 14336, 4096)])
@pytest.mark.parametrize("dtype", [rlq.DTYPE_BF16, rlq.DTYPE_F32])
def test_every_size_has_a_cut(M, N, K, dtype):
    """Also without a device, whose SMs are counted as one."""
    for aligned in (False, True):
        pair, staged, tile, splits, two, per = rlq.rlq_diag_gemm_mxfp4_cut(M, N, K, dtype, aligned)
        assert pair in (0, 1) and staged in (0, pair) and two in (0, 1)
        assert 1 <= tile <= 256 and 1 <= splits <= 8 and per >= 1
        assert aligned or not staged
