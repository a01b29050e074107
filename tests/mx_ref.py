"""Plain 64-bit forms of the MXFP4 quantizer and the layouts it writes (shared by the tests;
test infrastructure only)."""
import torch

D = torch.float64
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantize(x):
    """Codes [R, C] (0 .. 15) and scale bytes [R, ceil(C / 32)] of the blocks of 32 along x's rows,
    by the definition; x on the CPU."""
    R, C = x.shape
    nb = -(-C // 32)
    g = torch.zeros(R, nb * 32, dtype=D)
    g[:, :C] = x.to(D)
    g = g.view(R, nb, 32)
    bad = ~torch.isfinite(g).all(2)
    a = torch.where(bad[:, :, None], torch.ones_like(g), g).abs().amax(2)
    # a = m 2^k, m in [1/2, 1)
    e = torch.where(a > 0, torch.frexp(a)[1] - 3, torch.full_like(a, -127, dtype=torch.int32)).clamp(-127, 127)
    v = torch.ldexp(g, -e[:, :, None].to(D))
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(D)
    mag = (torch.round(v.abs() / step) * step).clamp(max=6)
    code = torch.zeros_like(mag, dtype=torch.uint8)
    for i, m in enumerate(MAGNITUDES):
        code[mag == m] = i
    code += 8 * torch.signbit(v).to(torch.uint8)
    s = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return code.view(R, nb * 32)[:, :C], s


def pack(code):
    R, C = code.shape
    full = torch.zeros(R, 2 * -(-C // 2), dtype=torch.uint8, device=code.device)
    full[:, :C] = code
    return full[:, ::2] | full[:, 1::2] << 4


def unpack(q, C):
    return torch.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)[:, :C]


def tile(s):
    """Scale bytes [R, nb] in the tiles that the library reads (rows past R: 0)."""
    R, nb = s.shape
    rt, ct = -(-R // 128), -(-nb // 4)
    t = torch.zeros(rt * 128, ct * 4, dtype=torch.uint8, device=s.device)
    t[:R, :nb] = s
    return t.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous()


def untile(t, R):
    """All of the tiles' scale bytes of R rows [R, 4 ceil(nb / 4)]."""
    return t.permute(0, 3, 2, 1, 4).reshape(t.shape[0] * 128, t.shape[1] * 4)[:R]


def values(code, s):
    """64-bit values of codes [R, C] and scale bytes [R, nb]."""
    m = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], dtype=D, device=code.device)[code.long()]
    scale = torch.ldexp(torch.ones_like(s, dtype=D), s.to(D) - 127)
    scale = torch.where(s == 255, torch.full_like(scale, float("nan")), scale)
    return m * scale.repeat_interleave(32, 1)[:, :code.shape[1]]


def operand(g, R, C, lo, hi, device="cuda"):
    """A random operand, any of the 16 codes, scale exponents lo .. hi: (packed codes in rows of
    16-byte pitch, scale tiles, 64-bit values)."""
    code = torch.randint(0, 16, (R, C), generator=g, device=device, dtype=torch.uint8)
    s = torch.randint(lo + 127, hi + 128, (R, -(-C // 32)), generator=g, device=device).to(torch.uint8)
    p = pack(code)
    q = torch.zeros(R, -(-p.shape[1] // 16) * 16, dtype=torch.uint8, device=device)[:, :p.shape[1]]
    q.copy_(p)
    return q, tile(s), values(code, s)
