"""GPU tests of the MXFP4 product on CTA pairs, every width of tile with either way out, and of which
cuts the product's shapes take on the device that the tests run on."""
import os
import subprocess
import sys

import pytest
import torch

import mx_ref as R
from fp8_block_scaled_quantize_gb300 import rlq
from test_gpu_mxfp4 import CLUSTERS, CUTS, SHAPES

pytestmark = pytest.mark.gpu
D = torch.float64
DEV = "cuda"
DTYPES = {"bf16": (torch.bfloat16, rlq.DTYPE_BF16, 8), "f32": (torch.float32, rlq.DTYPE_F32, 4)}

# Pairs: tiles of 128, 192 and 256, one, two and three or more of them a pair, rows of y on 16-byte
# boundaries (staged, stored by TMA) and off them (stored by the lanes), for either type.
PAIRS = [(4924, 136, 287), (7063, 520, 769), (5204, 129, 513), (150, 14650, 1452), (140, 22005, 1091), (4886, 136, 551),
         (6430, 520, 1569), (316, 8095, 1504), (132, 20533, 1482), (137, 10256, 1549), (258, 9792, 1081), (259, 20368, 788),
         (257, 6552, 2492), (257, 20352, 1879), (389, 4867, 1853), (130, 19459, 2459), (267, 20466, 1852), (6520, 259, 2711),
         (6534, 529, 1641), (282, 19486, 2149), (265, 7328, 663), (260, 15568, 519), (289, 20848, 32), (258, 7368, 816),
         (331, 9780, 42), (261, 19820, 146), (7376, 257, 793), (194, 20171, 2268), (389, 19718, 1908), (7405, 259, 1625),
         (385, 13673, 2318), (396, 19798, 2729), (1001, 6145, 2048), (2048, 8193, 1024)]


def cut(M, N, K, dtype):
    """The cut of a product into a contiguous output."""
    _, code, unit = DTYPES[dtype]
    return rlq.rlq_diag_gemm_mxfp4_cut(M, N, K, code, N % unit == 0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_shapes_take_every_cut(dtype):
    """What the parametrised shapes of the product's tests cover, asked of the library, so that a
    change of the cost model that drops a way is seen."""
    pairs, singles, several = set(), set(), set()
    for shape in SHAPES + CUTS + CLUSTERS + PAIRS:
        pair, staged, tile, splits, two, per = cut(*shape, dtype)
        if pair:
            pairs.add((staged, tile, min(per, 3)))
        else:
            singles.add((64 if tile <= 64 else 128 if tile <= 128 else 256, splits))
            if splits == 1 and per > 1:
                several.add(two)
    want = {(staged, tile, per) for staged in (0, 1) for tile in (128, 192, 256) for per in (1, 2, 3)}
    # (no shape has three staged tiles of 128 a pair: wider ones are cheaper by then)
    missing = want - {(1, 128, 3)} - pairs
    assert not missing, f"pairs (staged, tile, tiles a pair): {sorted(missing)}"
    missing = {(tile, splits) for tile in (64, 128) for splits in range(1, 9)} | {(256, 1), (256, 2)}
    missing -= singles
    assert not missing, f"single CTAs (tile, CTAs that share it): {sorted(missing)}"
    assert 1 in several


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_pairs_exact_sums(M, N, K, dtype):
    """As the other products: scales of 2^-1 .. 2^1, sums of multiples of 2^-4 that fp32 holds in whatever
    order.  Into contiguous rows, and into rows off 16-byte boundaries beside which nothing is written."""
    g = gen(M + 3 * N + K)
    t, code, unit = DTYPES[dtype]
    xq, xs, x = R.operand(g, M, K, -1, 1)
    wq, ws, w = R.operand(g, N, K, -1, 1)
    assert float((x.abs() @ w.abs().t()).max()) < 2.0 ** 20  # (units of 2^-4 below 2^24)
    want = (x @ w.t()).float().to(t)
    got = rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=t)
    rlq.check()
    assert torch.equal(got, want)
    buf = torch.full((M + 1, N + 1 + N % 2), 7.0, dtype=t, device=DEV)
    rlq.gemm_mxfp4(xq, xs, wq, ws, out=buf[:M, :N])
    rlq.check()
    assert buf.stride(0) % unit  # (odd: stored by the lanes)
    assert torch.equal(buf[:M, :N], want)
    assert bool((buf[:, N:] == 7).all()) and bool((buf[M] == 7).all())


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


_MODE_SCRIPT = """
import sys, torch
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import mx_ref as R
from fp8_block_scaled_quantize_gb300 import rlq
g = torch.Generator(device="cuda")
g.manual_seed(5)
for M, N, K in ((258, 9792, 1081), (7405, 259, 1625), (2100, 1024, 1056)):
    xq, xs, x = R.operand(g, M, K, -1, 1)
    wq, ws, w = R.operand(g, N, K, -1, 1)
    y = rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
    rlq.check()
    assert torch.equal(y.double(), x @ w.t())
    print(rlq.rlq_diag_gemm_mxfp4_cut(M, N, K, rlq.DTYPE_F32, N % 4 == 0)[0])
"""


@pytest.mark.parametrize("mode,pairs", [("0", {"0"}), ("1", {"1"})])
def test_no_pairs_where_the_environment_says_so(mode, pairs):
    """RLQ_GEMM_PAIR=0 (no CTA pairs) holds for this product as for the others, and the sums are the same."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _MODE_SCRIPT, root], env=dict(os.environ, RLQ_GEMM_PAIR=mode), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert set(r.stdout.split()) == pairs


@pytest.mark.parametrize("M,N,K,dtype", [(2100, 1024, 1056, "f32"), (2100, 5120, 512, "bf16"), (7405, 259, 1625, "f32"),
                                         (258, 9792, 1081, "bf16"), (1000, 3000, 64, "bf16"), (132, 20533, 1482, "f32")])
def test_a_pairs_bounded_wait_runs_out_and_the_next_call_is_right(M, N, K, dtype):
    """The diagnostic withholds both CTAs' first loads: one tile a pair and several, either way out, a
    ring that fills up and one that does not.  Every wait ends, the copies in flight are waited for,
    the error is reported once, and the next call is right."""
    g = gen(31)
    t = DTYPES[dtype][0]
    assert cut(M, N, K, dtype)[0] == 1
    xq, xs, x = R.operand(g, M, K, -1, 1)
    wq, ws, w = R.operand(g, N, K, -1, 1)
    want = (x @ w.t()).float().to(t)
    rlq.rlq_diag_arm_gemm_stall()
    rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=t)
    with pytest.raises(rlq.RlqError) as e:
        rlq.check()
    assert e.value.status == 5 and "MXFP4" in str(e.value)
    rlq.check()
    for _ in range(2):
        assert torch.equal(rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=t), want)
        rlq.check()
