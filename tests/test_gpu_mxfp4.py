"""GPU tests of the MXFP4 quantizer, dequantizer and product against the definition in 64 bits."""
import pytest
import torch

import mx_ref as R
from fp8_block_scaled_quantize_gb300 import rlq

pytestmark = pytest.mark.gpu
D = torch.float64
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------- quantizer ---

def difficult(g, M, K):
    """bf16 [M, K]: blocks 2^-133 .. 2^120 apart, zeros of both signs, ties of every size."""
    x = torch.randn(M, K, generator=g, device=DEV)
    nb = K // 32
    e = torch.randint(-20, 20, (M, nb), generator=g, device=DEV).float()
    far = torch.rand(M, nb, generator=g, device=DEV)
    e = torch.where(far < 0.05, e - 110, torch.where(far > 0.95, e + 100, e))
    x = x * torch.exp2(e).repeat_interleave(32, 1)
    # multiples of a quarter up to 8, times a power of two: every midpoint between codes
    t = torch.randint(-32, 33, (M, K), generator=g, device=DEV).float() / 4
    pick = (torch.rand(M, nb, generator=g, device=DEV) < 0.4).repeat_interleave(32, 1)
    x = torch.where(pick, t * torch.exp2(e.clamp(-120, 118)).repeat_interleave(32, 1), x)
    x = torch.where(torch.rand(M, K, generator=g, device=DEV) < 0.02, -torch.zeros_like(x), x)
    x = torch.where((torch.rand(M, nb, generator=g, device=DEV) < 0.03).repeat_interleave(32, 1), torch.zeros_like(x), x)
    return x.to(torch.bfloat16)


def check_codes(q, s, x, what):
    """Packed codes and scale tiles against the definition, the padding of the last tile too."""
    code, sb = R.quantize(x.cpu())
    nb = sb.shape[1]
    got = R.untile(s.cpu(), x.shape[0])
    assert torch.equal(got[:, :nb], sb), f"{what}: scales"
    assert not got[:, nb:].any(), f"{what}: scales past the row's end"
    fine = (sb != 255).repeat_interleave(32, 1)[:, :x.shape[1]]
    have = R.unpack(q.cpu(), x.shape[1])
    assert torch.equal(have[fine], code[fine]), f"{what}: codes"
    if x.shape[1] % 2:
        assert not (q.cpu()[:, -1] >> 4).any(), f"{what}: the last byte's high nibble"


@pytest.mark.parametrize("M,K,pitch", [(1, 32, 0), (1, 4096, 0), (2, 96, 8), (5, 128, 0), (31, 160, 0), (33, 288, 16),
                                       (64, 1024, 0), (97, 3584, 0), (128, 128, 0), (129, 256, 0), (200, 5120, 8),
                                       (255, 64, 0), (300, 18944, 0), (1001, 416, 0)])
def test_quantizer(M, K, pitch):
    g = gen(M * 3 + K)
    x = difficult(g, M, K)
    if pitch:
        buf = torch.full((M, K + pitch), 7.0, dtype=torch.bfloat16, device=DEV)
        buf[:, :K] = x
        x = buf[:, :K]
    q, s, qT, sT = rlq.quant_mxfp4(x, colwise=True)
    check_codes(q, s, x, "rows")
    check_codes(qT, sT, x.t(), "columns")
    q2, s2, none, none2 = rlq.quant_mxfp4(x)
    assert none is None and none2 is None
    assert torch.equal(q2, q)
    nb = K // 32
    assert torch.equal(R.untile(s2, M)[:, :nb], R.untile(s, M)[:, :nb])
    check_codes(q2, s2, x, "rows alone")
    # read back: the values themselves
    code, sb = R.quantize(x.cpu())
    assert torch.equal(rlq.dequant_mxfp4(q, s).cpu().to(D), R.values(code, sb))
    code, sb = R.quantize(x.t().cpu())
    assert torch.equal(rlq.dequant_mxfp4(qT, sT, cols=M).cpu().to(D), R.values(code, sb))


def test_quantizer_every_exponent_and_values_that_are_no_numbers():
    """A block for every bf16 exponent with each pattern of the leading bits; infinities and NaN
    make their block's scale 255 and its values NaN, the blocks beside it stay."""
    f = torch.arange(0, 255, device=DEV)
    bits = (f[:, None] << 7) + (torch.arange(0, 128, 4, device=DEV))[None, :]
    x = torch.cat((bits.to(torch.int16).view(torch.bfloat16), (bits | 0x8000).to(torch.int32).to(torch.int16).view(torch.bfloat16)), 1)
    q, s, qT, sT = rlq.quant_mxfp4(x, colwise=True)
    check_codes(q, s, x, "rows")
    check_codes(qT, sT, x.t(), "columns")
    y = torch.randn(70, 128, generator=gen(1), device=DEV).to(torch.bfloat16)
    y[3, 40] = float("nan")
    y[4, 0] = float("inf")
    y[35, 127] = float("-inf")
    q, s, qT, sT = rlq.quant_mxfp4(y, colwise=True)
    check_codes(q, s, y, "rows")
    check_codes(qT, sT, y.t(), "columns")
    v = rlq.dequant_mxfp4(q, s)
    bad = torch.zeros(70, 4, dtype=torch.bool, device=DEV)
    bad[3, 1] = bad[4, 0] = bad[35, 3] = True
    assert torch.equal(torch.isnan(v), bad.repeat_interleave(32, 1))


def test_quantizer_writes_nothing_beside_its_outputs():
    """Bytes between rows, past the last row and past the scale tiles stay as they were."""
    M, K = 77, 160
    x = difficult(gen(4), M, K)
    ldq, ldT = K // 2 + 16, 64
    bufs = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in (M * ldq + 64, 2 * 512 + 64, K * ldT + 64,
                                                                            2 * 512 + 64)]
    q, s, qT, sT = bufs
    rlq.rlq_quant_mxfp4(x.data_ptr(), M, K, K, q.data_ptr(), ldq, s.data_ptr(), qT.data_ptr(), ldT, sT.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    assert (q[:M * ldq].view(M, ldq)[:, K // 2:] == 0xA5).all() and (q[M * ldq:] == 0xA5).all()
    assert (s[1024:] == 0xA5).all() and (sT[1024:] == 0xA5).all()
    rows = qT[:K * ldT].view(K, ldT)
    assert (rows[:, (M + 1) // 2:] == 0xA5).all() and (qT[K * ldT:] == 0xA5).all()
    check_codes(q[:M * ldq].view(M, ldq)[:, :K // 2], s[:1024].view(1, 2, 32, 4, 4), x, "rows")
    check_codes(rows[:, :(M + 1) // 2], sT[:1024].view(2, 1, 32, 4, 4), x.t(), "columns")


def test_dequantizer_writes_nothing_beside_its_output():
    q, s, v = R.operand(gen(2), 9, 45, -3, 3)
    out = torch.full((9 * 64 + 32,), 5.0, dtype=torch.bfloat16, device=DEV)
    rlq.rlq_dequant_mxfp4(q.data_ptr(), q.stride(0), s.data_ptr(), 9, 45, out.data_ptr(), 64,
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out[:9 * 64].view(9, 64)[:, :45].to(D), v)
    assert (out[:9 * 64].view(9, 64)[:, 45:] == 5).all() and (out[9 * 64:] == 5).all()


# --------------------------------------------------------------- product ---

SHAPES = [(1, 128, 256), (1, 1, 32), (1, 1000, 4096), (2, 100, 64), (3, 129, 96), (16, 256, 512), (17, 384, 288),
          (64, 3584, 1024), (64, 200, 8192), (100, 129, 1000), (112, 256, 320), (113, 256, 320), (128, 130, 160),
          (129, 512, 352), (200, 257, 1001), (255, 127, 33), (256, 1024, 256), (257, 256, 256), (300, 700, 1),
          (384, 255, 416), (511, 513, 2048), (513, 1000, 777), (1000, 3000, 64), (2100, 5120, 512), (700, 20000, 288),
          (1001, 3584, 352), (600, 14300, 160), (450, 1024, 2048), (1001, 1024, 2048), (520, 900, 1120), (5000, 130, 96)]


# One shape for every way in which a product is cut: pairs with tiles of 128, 192 and 256, their
# outputs by TMA or by the lanes, one tile a pair or several; single CTAs with tiles of up to 64,
# 128 and 256 tokens, one tile each or several, alone or in clusters of 2, 4 and 8, one or two an SM.
CUTS = [(270, 10029, 1034), (5117, 130, 266), (129, 6636, 849), (6970, 568, 779), (5192, 136, 36), (134, 7144, 282),
        (263, 10138, 808), (129, 19471, 1328), (6007, 129, 258), (130, 7085, 520), (273, 10544, 258), (143, 19704, 836),
        (5738, 136, 36), (136, 7984, 286), (271, 11771, 281), (129, 21211, 263), (6132, 133, 269), (132, 6473, 257),
        (281, 10768, 38), (130, 22960, 35), (1377, 712, 33), (196, 5448, 35), (115, 19509, 567), (119, 10181, 524),
        (122, 4949, 3936), (4872, 1, 4353), (115, 2537, 2810), (2464, 1, 3664), (132, 1555, 3682), (1248, 1, 7334),
        (601, 12877, 2816), (226, 10333, 10550), (6643, 523, 1801), (225, 5604, 7753), (4923, 129, 9780),
        (226, 2709, 6165), (4930, 1, 12051), (229, 1340, 12052), (1238, 133, 15595), (1, 39803, 35), (65, 23684, 33),
        (1, 9981, 3124), (4947, 1, 3169), (67, 1, 33), (1, 5022, 6214), (1, 1, 1281), (4737, 1, 6527), (67, 1, 2079),
        (1, 1, 12291), (1, 1, 1565), (68, 1, 12354), (68, 1, 1537), (1, 1, 3586), (67, 1, 3627)]


# clusters of 2 .. 8 CTAs: one or two tokens (also with two CTAs on an SM), a narrow tile, several of them, a wide one
CLUSTERS = [(2, 6410, 1350), (67, 5467, 2331), (270, 1111, 1873), (2, 10, 1124), (129, 4044, 3140), (67, 2948, 2155),
            (200, 2554, 2840), (67, 5, 1519), (1, 5266, 1054), (5, 26, 1177), (129, 2462, 4050), (270, 1025, 3629),
            (2, 4103, 1592), (3, 27, 1833), (129, 1805, 3222), (67, 1589, 2255), (200, 1386, 3076), (300, 11, 2498),
            (2, 2956, 2113), (2, 18, 2261), (129, 1746, 2872), (67, 1153, 2808), (256, 1063, 5411), (200, 2, 2913),
            (2, 2537, 2628), (64, 5, 2731), (129, 1426, 4695), (67, 770, 3365), (200, 686, 8226), (2, 1554, 3180),
            (67, 1, 3172), (17, 1, 3345), (129, 1374, 4014), (256, 649, 7574), (1, 1549, 3607), (115, 3, 5457)]


@pytest.mark.parametrize("M,N,K", SHAPES + CUTS + CLUSTERS)
def test_product_exact_sums(M, N, K):
    """Scales within 2^-1 .. 2^1: every product is a multiple of 2^-4 and at most 144, and
    where the magnitudes' sum stays below 2^24 of those units, as it is checked to, fp32 holds
    every partial sum exactly in whatever order: the result is the exact sum."""
    g = gen(M + 7 * N + K)
    xq, xs, x = R.operand(g, M, K, -1, 1)
    wq, ws, w = R.operand(g, N, K, -1, 1)
    want = x @ w.t()
    assert float((x.abs() @ w.abs().t()).max()) < 2.0 ** 20  # (units of 2^-4 below 2^24)
    got = rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
    rlq.check()
    assert got.shape == (M, N) and got.dtype == torch.float32
    assert torch.equal(got.to(D), want)
    assert torch.equal(rlq.gemm_mxfp4(xq, xs, wq, ws), want.float().to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (5, 4096, 14336), (64, 1000, 2048), (130, 384, 1001), (600, 700, 5120)])
def test_product_rounding(M, N, K):
    """Scales 2^-12 .. 2^12.  The hardware adds a product's 64 terms and the accumulator in fp32 with
    at most a few bits of each lost to alignment: every one of the K / 64 additions is off by at
    most 2^-21 of the sum of magnitudes so far, a split's parts by 8 more."""
    g = gen(K + M)
    xq, xs, x = R.operand(g, M, K, -12, 12)
    wq, ws, w = R.operand(g, N, K, -12, 12)
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    got = rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32).to(D)
    tol = (-(-K // 64) + 8) * 2.0 ** -21 * mag
    assert bool(((got - want).abs() <= tol).all())
    # and in the mean far nearer: rounding errors of both signs
    assert float((got - want).norm() / want.norm()) < 1e-5
    b = rlq.gemm_mxfp4(xq, xs, wq, ws).to(D)
    assert bool(((b - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


def test_product_extreme_scales():
    """The ends of the scales' range: 2^-127 x 2^127 is 1; 6 x 2^127 x 2^-3 overflows nowhere."""
    for ex, ew in ((-127, 127), (127, -127), (127, -3), (-60, -60)):
        code = torch.full((40, 256), 7, dtype=torch.uint8, device=DEV)
        code[:, 1::2] = 15  # 6 and -6 in turn: sums of zero
        code[:, 0] = 4
        sx = torch.full((40, 8), ex + 127, dtype=torch.uint8, device=DEV)
        sw = torch.full((40, 8), ew + 127, dtype=torch.uint8, device=DEV)
        one = torch.zeros(40, 256, dtype=torch.uint8, device=DEV)
        one[:, 0] = 2  # 1
        y = rlq.gemm_mxfp4(R.pack(code), R.tile(sx), R.pack(one), R.tile(sw), out_dtype=torch.float32)
        assert bool((y.to(D) == 2.0 * 2.0 ** (ex + ew)).all())


def test_product_nan_scales_stay_in_their_rows():
    g = gen(9)
    for M in (20, 300):
        xq, xs, x = R.operand(g, M, 512, -1, 1)
        wq, ws, w = R.operand(g, 200, 512, -1, 1)
        xs[0, 1, 5, 0, 2] = 255  # row 5, block 6
        ws[1, 0, 3, 1, 0] = 255  # row 128 + 35
        y = rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
        nan = torch.zeros(M, 200, dtype=torch.bool, device=DEV)
        nan[5] = True
        nan[:, 163] = True
        assert torch.equal(torch.isnan(y), nan)
        assert torch.equal(y.to(D)[~nan], (x @ w.t())[~nan])


def test_scales_of_rows_that_do_not_exist_are_not_used():
    """The tiles' bytes of rows past the last one are unspecified: 255 there changes nothing."""
    g = gen(10)
    for M, N in ((3, 70), (290, 300)):
        xq, xs, x = R.operand(g, M, 256, -1, 1)
        wq, ws, w = R.operand(g, N, 256, -1, 1)
        for s, rows in ((xs, M), (ws, N)):
            r = torch.arange(s.shape[0] * 128, device=DEV).view(-1, 4, 32).permute(0, 2, 1)
            s[(r >= rows)[:, None, :, :, None].expand_as(s)] = 255
        assert torch.equal(rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32).to(D), x @ w.t())


def test_product_outputs_and_pitches():
    """Every kind of output: contiguous, pitched, off 16-byte boundaries; nothing beside it is written."""
    g = gen(12)
    for M, N, K in ((5, 131, 320), (290, 131, 320)):
        xq, xs, x = R.operand(g, M, K, -1, 1)
        wq, ws, w = R.operand(g, N, K, -1, 1)
        want = x @ w.t()
        for dt in (torch.bfloat16, torch.float32):
            buf = torch.full((M + 2, N + 9), 3.0, dtype=dt, device=DEV)
            out = buf[1:1 + M, 5:5 + N]
            assert rlq.gemm_mxfp4(xq, xs, wq, ws, out=out) is out
            assert torch.equal(out, want.float().to(dt))
            buf[1:1 + M, 5:5 + N] = 3.0
            assert (buf == 3).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,ldy", [(300, 5681, 64, 5696), (300, 5682, 64, 5688), (300, 5683, 64, 5692), (301, 5685, 33, 5688),
                                       (300, 5687, 64, 5688), (300, 5684, 64, 5688), (700, 2499, 40, 2504), (261, 4100, 600, 4104),
                                       (129, 8129, 90, 8136), (200, 4893, 494, 4896), (200, 4909, 594, 4912)])
def test_product_leaves_the_elements_beside_its_rows(M, N, K, ldy, dtype):
    """Rows that end anywhere inside 16 bytes, at pitches that are multiples of them (and of 8 bytes only)."""
    g = gen(M + N)
    xq, xs, x = R.operand(g, M, K, -1, 1)
    wq, ws, w = R.operand(g, N, K, -1, 1)
    buf = torch.full((M + 1, ldy), 7.0, dtype=dtype, device=DEV)
    rlq.gemm_mxfp4(xq, xs, wq, ws, out=buf[:M, :N])
    rlq.check()
    assert torch.equal(buf[:M, :N], (x @ w.t()).float().to(dtype))
    assert bool((buf[:, N:] == 7).all()) and bool((buf[M] == 7).all())


def test_product_empty_contraction_and_empty_outputs():
    u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    y = rlq.gemm_mxfp4(u8(5, 0), u8(1, 0, 32, 4, 4), u8(7, 0), u8(1, 0, 32, 4, 4))
    assert y.shape == (5, 7) and not y.any()
    y = torch.full((3, 9), 2.0, device=DEV)
    rlq.gemm_mxfp4(u8(3, 0), u8(1, 0, 32, 4, 4), u8(9, 0), u8(1, 0, 32, 4, 4), out=y)
    assert not y.any()
    assert rlq.gemm_mxfp4(u8(0, 16), u8(0, 1, 32, 4, 4), u8(7, 16), u8(1, 1, 32, 4, 4)).shape == (0, 7)
    assert rlq.gemm_mxfp4(u8(7, 16), u8(1, 1, 32, 4, 4), u8(0, 16), u8(0, 1, 32, 4, 4)).shape == (7, 0)
    q, s, qT, sT = rlq.quant_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), colwise=True)
    assert q.shape == (0, 32) and s.shape == (0, 1, 32, 4, 4) and qT.shape == (64, 0) and sT.shape == (1, 0, 32, 4, 4)


def test_layer_forward_and_backward_passes():
    """A layer's three passes on one pair of quantizations, ragged tokens, and the gradients of
    the layer as it was rounded against autograd in 64 bits."""
    g = gen(21)
    M, N, K = 333, 352, 288
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(N, K, generator=g, device=DEV) * 0.05).to(torch.bfloat16)
    dy = (torch.randn(M, N, generator=g, device=DEV) * 1e-3).to(torch.bfloat16)
    xq, xs, xqT, xsT = rlq.quant_mxfp4(x, colwise=True)
    wq, ws, wqT, wsT = rlq.quant_mxfp4(w, colwise=True)
    dq, ds, dqT, dsT = rlq.quant_mxfp4(dy, colwise=True)
    y = rlq.gemm_mxfp4(xq, xs, wq, ws)
    dx = rlq.gemm_mxfp4(dq, ds, wqT, wsT)
    dw = rlq.gemm_mxfp4(dqT, dsT, xqT, xsT, out_dtype=torch.float32)
    val = lambda q, s, c: rlq.dequant_mxfp4(q, s, cols=c).to(D)  # noqa: E731
    # each pass is the gradient of the bilinear form <dy, x w^T> in its rounded operands
    a, b = val(xq, xs, K), val(wq, ws, K)
    assert bool(((y.to(D) - a @ b.t()).abs() <= 2.0 ** -8 * (a @ b.t()).abs() + 1e-5 * (a.abs() @ b.abs().t())).all())
    p = torch.zeros(M, K, dtype=D, device=DEV, requires_grad=True)
    (val(dq, ds, N) * (p @ val(wqT, wsT, N))).sum().backward()
    mag = val(dq, ds, N).abs() @ val(wqT, wsT, N).abs().t()
    assert bool(((dx.to(D) - p.grad).abs() <= 2.0 ** -8 * p.grad.abs() + 1e-5 * mag).all())
    p = torch.zeros(N, K, dtype=D, device=DEV, requires_grad=True)
    (val(dqT, dsT, M).t() * (val(xqT, xsT, M).t() @ p.t())).sum().backward()
    mag = val(dqT, dsT, M).abs() @ val(xqT, xsT, M).abs().t()
    assert bool(((dw.to(D) - p.grad).abs() <= 1e-5 * mag).all())


def test_streams_graphs_and_repeatability():
    g = gen(30)
    M, N, K = 48, 640, 4096
    xq, xs, x = R.operand(g, M, K, -12, 12)
    wq, ws, w = R.operand(g, N, K, -12, 12)
    want = rlq.gemm_mxfp4(xq, xs, wq, ws)
    for _ in range(3):
        assert torch.equal(rlq.gemm_mxfp4(xq, xs, wq, ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = rlq.gemm_mxfp4(xq, xs, wq, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    xb = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    eager = rlq.gemm_mxfp4(*rlq.quant_mxfp4(xb)[:2], wq, ws)
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(xb)
    with torch.cuda.graph(graph):
        q, s, _, _ = rlq.quant_mxfp4(static)
        out = rlq.gemm_mxfp4(q, s, wq, ws)
    static.copy_(xb)
    graph.replay()
    graph.replay()
    assert torch.equal(out, eager)


def test_bounded_wait_runs_out_and_the_next_call_is_right():
    """The diagnostic withholds every CTA's first loads: the wait runs out, the call ends, the
    error is reported once, and the next call is right."""
    g = gen(31)
    for M, K in ((8, 256), (8, 4096), (300, 512)):
        xq, xs, x = R.operand(g, M, K, -1, 1)
        wq, ws, w = R.operand(g, 300, K, -1, 1)
        rlq.rlq_diag_arm_gemm_stall()
        rlq.gemm_mxfp4(xq, xs, wq, ws)
        with pytest.raises(rlq.RlqError) as e:
            rlq.check()
        assert e.value.status == 5 and "MXFP4" in str(e.value)
        rlq.check()
        assert torch.equal(rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32).to(D), x @ w.t())


def test_far_offsets():
    """Rows of every matrix beyond 2^31 bytes and elements from the first one."""
    g = gen(40)
    ld = (1 << 30) + 64
    rows, K = 4, 352
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((rows, K), (ld, 1))
    x.copy_(difficult(g, rows, K))
    q, s, qT, sT = rlq.quant_mxfp4(x, colwise=True)
    check_codes(q, s, x, "rows")
    check_codes(qT, sT, x.t(), "columns")
    code, sb = R.quantize(x.cpu())
    rlq.rlq_dequant_mxfp4(q.data_ptr(), q.stride(0), s.data_ptr(), rows, K, x.data_ptr(), ld,
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(x.cpu().to(D), R.values(code, sb))
    # codes and outputs in the same rows, a quarter apart
    bytes_ = big.view(torch.uint8)
    far = bytes_[1 << 20:].as_strided((rows, K // 2), (2 * ld, 1))
    rlq.rlq_quant_mxfp4(x.data_ptr(), rows, K, ld, far.data_ptr(), 2 * ld, s.data_ptr(), None, 0, None,
                        torch.cuda.current_stream().cuda_stream)
    xq, xs, xv = R.operand(g, rows, K, -1, 1)
    far.copy_(xq)
    wq, ws, w = R.operand(g, 300, K, -1, 1)
    y = big[1 << 20:].as_strided((rows, 300), (ld, 1))
    assert rlq.gemm_mxfp4(far, xs, wq, ws, out=y) is y
    assert torch.equal(y, (xv @ w.t()).float().to(torch.bfloat16))
    yT = rlq.gemm_mxfp4(wq, ws, far, xs)  # the far codes as the second operand
    assert torch.equal(yT, (w @ xv.t()).float().to(torch.bfloat16))


def test_operands_in_longer_rows():
    """Codes as views of longer rows, for single CTAs and pairs."""
    g = gen(41)
    for M, N, K in ((20, 200, 512), (700, 600, 1000)):
        xq, xs, x = R.operand(g, M, K, -1, 1)
        wq, ws, w = R.operand(g, N, K, -1, 1)
        bx = torch.randint(0, 255, (M, xq.shape[1] // 16 * 16 + 64), generator=g, device=DEV).to(torch.uint8)
        bw = torch.randint(0, 255, (N, wq.shape[1] // 16 * 16 + 48), generator=g, device=DEV).to(torch.uint8)
        bx[:, :xq.shape[1]], bw[:, :wq.shape[1]] = xq, wq
        got = rlq.gemm_mxfp4(bx[:, :xq.shape[1]], xs, bw[:, :wq.shape[1]], ws, out_dtype=torch.float32)
        assert torch.equal(got.to(D), x @ w.t())


def test_calls_on_two_streams_at_once():
    """Products of every kind of cut side by side: nothing is shared between calls."""
    g = gen(42)
    shapes = [(4, 1024, 4096), (64, 640, 8192), (300, 1024, 2048), (600, 2000, 512)]
    ops = [(R.operand(g, M, K, -1, 1), R.operand(g, N, K, -1, 1)) for M, N, K in shapes]
    want = [(a[2] @ b[2].t()).float() for a, b in ops]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[] for _ in streams]
    for i in range(12):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                a, b = ops[(i + j) % len(ops)]
                got[j].append(((i + j) % len(ops), rlq.gemm_mxfp4(a[0], a[1], b[0], b[1], out_dtype=torch.float32)))
    torch.cuda.synchronize()
    rlq.check()
    for per in got:
        for k, y in per:
            assert torch.equal(y, want[k])


def test_helpers_refuse_wrong_operands():
    g = gen(43)
    xq, xs, _ = R.operand(g, 5, 64, -1, 1)
    wq, ws, _ = R.operand(g, 7, 64, -1, 1)
    with pytest.raises(ValueError, match="contraction"):
        rlq.gemm_mxfp4(xq, xs, wq[:, :16], ws)
    with pytest.raises(ValueError, match="scales"):
        rlq.gemm_mxfp4(xq, xs[:, :, :16], wq, ws)
    with pytest.raises(TypeError):
        rlq.gemm_mxfp4(xq, xs.int(), wq, ws)
    with pytest.raises(TypeError):
        rlq.gemm_mxfp4(xq, xs, wq, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        rlq.gemm_mxfp4(xq, xs, wq, ws, out=torch.empty(5, 8, device=DEV))
    with pytest.raises(ValueError):
        rlq.gemm_mxfp4(xq, xs.cpu(), wq, ws)
    with pytest.raises(ValueError, match="contiguous rows"):
        rlq.quant_mxfp4(torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV).t()[:, :32])
    with pytest.raises(rlq.RlqError):
        rlq.quant_mxfp4(torch.zeros(4, 48, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="cols"):
        rlq.dequant_mxfp4(xq, xs, cols=62)
