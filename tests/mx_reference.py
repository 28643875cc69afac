"""MXFP4 in 64 bits on the CPU, from the format's definition: what the tests of the MXFP4 operators and of the
expert layer compare with."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize(x):
    """(codes [..., M, Kp / 2], scales [..., Kp / 128, M, 4]) of rows x [..., M, K], by comparison with the borders
    between neighbouring magnitudes; a magnitude on a border goes to the even code."""
    x = x.detach().cpu().double()
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % 128))
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent + 124, torch.zeros_like(top, dtype=torch.int32)).clamp_min(0)   # floor(log2) + 125
    a = b.abs() * torch.exp2(127.0 - e.double())[..., None]
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += ((a >= border) if up else (a > border)).to(torch.uint8)
    code += 8 * torch.signbit(b).to(torch.uint8)
    code = torch.where(bad[..., None], torch.zeros_like(code), code).reshape(*x.shape[:-1], -1, 2)
    scales = torch.where(bad, torch.full_like(e, 255), e).to(torch.uint8)
    scales = scales.reshape(*scales.shape[:-1], scales.shape[-1] // 4, 4).transpose(-3, -2).contiguous()
    return code[..., 0] + 16 * code[..., 1], scales


def values(q, s):
    """Their values in 64 bits, [..., M, Kp]."""
    q, s = q.cpu(), s.cpu()
    n = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], 2 * q.shape[-1]).long()
    v = GRID[n & 7] * torch.where(n >= 8, -1.0, 1.0).double()
    b = s.transpose(-3, -2).reshape(*q.shape[:-1], q.shape[-1] // 16)
    unit = torch.where(b == 255, torch.full(b.shape, float("nan"), dtype=torch.float64), torch.exp2(b.double() - 127.0))
    return v * unit.repeat_interleave(32, dim=-1)


def random_matrix(g, *shape):
    """Codes and scales of random rows, every code and scale bytes within 16 of 1.0's."""
    *lead, M, Kp = shape
    q = torch.randint(0, 256, (*lead, M, Kp // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(119, 135, (*lead, Kp // 128, M, 4), generator=g, dtype=torch.uint8)
    return q, s


def check_product(y, x, w, bias=None, what=""):
    """y against x w^T (+ bias) of 64-bit values. A block's 32 products are multiples of 1/4 of its scale units below
    2^11, so their sum is exact in 32 bits; K / 32 block sums are added, up to two more for partial sums, and the bias, each
    addition off by at most a unit in the last place, 2^-23, of a partial sum that is at most the sum of the magnitudes;
    then one rounding to the output type, half a step."""
    ref = x @ w.T
    mag = x.abs() @ w.abs().T
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    tol = (x.shape[-1] / 32 + 3) * 2.0 ** -23 * mag
    tol = tol + (ref.abs() + tol) * torch.finfo(y.dtype).eps / 2
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25                            # half a step of its subnormal numbers
    got = y.detach().cpu().double()
    over = torch.isfinite(ref) & (ref.abs() > torch.finfo(y.dtype).max * (1 - torch.finfo(y.dtype).eps))
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    off = torch.where(torch.isnan(ref) | over, torch.zeros_like(ref), (got - ref).abs() - tol)
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} past the tolerance"
