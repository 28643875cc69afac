"""MXFP4 on the GPU: the quantizer bit for bit against the format's definition, its inverse, and the products of two
MXFP4 matrices, with one weight and with one per expert, against sums in 64 bits."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import decode_tile_interleaved_rans_amd as ep
import mx_reference as mx

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same_codes(x, q, s):
    """Codes and scales equal the definition's; the sign of a zero is x's."""
    rq, rs = mx.quantize(x)
    assert q.dtype == s.dtype == torch.uint8 and q.shape == rq.shape and s.shape == rs.shape
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)


# ---------------------------------------------------------------------------------------- quantizer
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 127), (16, 128), (17, 129), (4, 136), (33, 511), (64, 512),
                                 (19, 1000), (2, 8192), (300, 640)])
def test_quantize_sizes(dtype, M, K):
    x = (torch.randn((M, K), generator=gen(M * 1000 + K)) * torch.exp(2 * torch.randn((M, 1), generator=gen(K)))).to(dtype).cuda()
    same_codes(x, *ep.quantize_rows_mxfp4(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_every_16_bit_value(dtype):
    """Every finite 16-bit value, under the block maximum of its own magnitude and of four binades above."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[torch.isfinite(v)]
    for lift in (1.0, 1.75, 16.0):
        top = (v.float() * lift).to(dtype)
        top = torch.where(torch.isfinite(top), top, v)
        x = torch.zeros((v.numel(), 32), dtype=dtype)
        x[:, 3], x[:, 17], x[:, 30] = v, top, -v
        same_codes(x, *ep.quantize_rows_mxfp4(x.cuda()))


def test_quantize_borders_of_every_scale():
    """FP32 magnitudes on every rounding border and one step beside it, for scales over the whole range."""
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    rows = []
    for e in range(-149, 126):
        t = (borders.double() * 2.0 ** e).float()
        big = torch.tensor([4.0 * 2.0 ** e, 7.999 * 2.0 ** e], dtype=torch.float64).float()
        t = torch.cat([t, torch.nextafter(t, torch.tensor(0.0)), torch.nextafter(t, torch.tensor(float("inf")))])
        rows.append(torch.cat([t, -t[:3], big[:1 + (e % 2)], torch.zeros(1 - (e % 2))]))
    x = torch.stack(rows)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    same_codes(x, *ep.quantize_rows_mxfp4(x.cuda()))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_infinities_and_nans(dtype):
    """A block with an infinity or a NaN gets scale byte 255 and codes 0; its neighbours are untouched."""
    x = torch.randn((9, 200), generator=gen(1)).to(dtype)
    x[0, 0], x[2, 40], x[2, 41], x[5, 199], x[7, 64] = float("inf"), float("nan"), 1.0, float("-inf"), float("nan")
    x[8] = 0.0
    x[3, 32:64] = -0.0
    q, s = ep.quantize_rows_mxfp4(x.cuda())
    same_codes(x, q, s)
    assert (s == 255).sum() == 4


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strides_and_alignment(dtype):
    """Rows further apart than their width, at odd addresses, and the experts' matrices."""
    base = torch.randn((40, 333), generator=gen(2)).to(dtype).cuda()
    for x in (base[:, 1:300], base[::3, 5:133], base[:, 2:258], base[7:8, 3:]):
        same_codes(x, *ep.quantize_rows_mxfp4(x))
    w = torch.randn((5, 19, 200), generator=gen(3)).to(dtype).cuda()
    q, s = ep.quantize_rows_mxfp4(w)
    same_codes(w, q, s)
    for e in range(5):
        qe, se = ep.quantize_rows_mxfp4(w[e])
        assert torch.equal(q[e], qe) and torch.equal(s[e], se)


def test_quantize_empty():
    for shape in ((0, 64), (3, 0), (0, 5, 64), (5, 0, 64), (2, 3, 0)):
        q, s = ep.quantize_rows_mxfp4(torch.empty(shape, device="cuda"))
        *lead, M, K = shape
        assert q.shape == (*lead, M, (K + 127) // 128 * 64) and s.shape == (*lead, (K + 127) // 128, M, 4)
        assert ep.dequantize_rows_mxfp4(q, s, columns=K).shape == shape


# ------------------------------------------------------------------------------------------ inverse
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape,K", [((1, 128), 1), ((3, 256), 131), ((17, 384), 384), ((4, 5, 512), 509), ((2, 3, 128), None)])
def test_dequantize(dtype, shape, K):
    q, s = mx.random_matrix(gen(shape[-1]), *shape)
    y = ep.dequantize_rows_mxfp4(q.cuda(), s.cuda(), dtype, columns=K)
    ref = mx.values(q, s)[..., :K].to(dtype)                                # to() rounds to nearest even
    assert y.dtype == dtype and y.shape == ref.shape and torch.equal(y.cpu(), ref)


def test_dequantize_every_code_and_scale():
    q = torch.arange(16, dtype=torch.uint8).repeat(4)[None].repeat(64, 1)    # [64, 64]: low nibbles 0 .. 15
    q = q + 16 * q
    s = torch.arange(256, dtype=torch.uint8).view(64, 4)[None]
    for dtype in TYPES:
        y, ref = ep.dequantize_rows_mxfp4(q.cuda(), s.cuda(), dtype).cpu(), mx.values(q, s)
        assert torch.equal(torch.isnan(y), torch.isnan(ref))
        fits = ~torch.isnan(ref) & (ref.abs() <= torch.finfo(dtype).max)
        assert torch.equal(y[fits], ref.to(dtype)[fits])


# ----------------------------------------------------------------------------------------- products
SIZES = [(1, 1, 128), (1, 64, 256), (2, 3, 128), (5, 130, 384), (15, 65, 640), (16, 64, 512), (17, 515, 1152), (33, 96, 128), (64, 200, 2048),
         (65, 70, 256), (100, 1000, 896), (130, 129, 384), (257, 260, 640), (300, 515, 1280), (513, 768, 256), (600, 1100, 512)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K):
    g = gen(M + N + K)
    (xq, xs), (wq, ws) = mx.random_matrix(g, M, K), mx.random_matrix(g, N, K)
    bias = torch.randn(N, generator=g).to(torch.bfloat16)
    x, w = mx.values(xq, xs), mx.values(wq, ws)
    dev = [t.cuda() for t in (xq, xs, wq, ws)]
    for dtype, b in ((torch.float32, None), (torch.bfloat16, bias), (torch.float16, bias)):
        y = ep.gemm_mxfp4(*dev, b.cuda() if b is not None else None, out_dtype=dtype)
        assert y.shape == (M, N) and y.dtype == dtype
        mx.check_product(y, x, w, b, f"{M} x {N} x {K} {dtype}")
        assert torch.equal(y, ep.gemm_mxfp4(*dev, b.cuda() if b is not None else None, out_dtype=dtype))


def test_product_empty():
    u8 = lambda *shape: torch.empty(shape, dtype=torch.uint8, device="cuda")
    b = torch.randn(5, device="cuda").to(torch.bfloat16)
    assert ep.gemm_mxfp4(u8(0, 64), u8(1, 0, 4), u8(5, 64), u8(1, 5, 4)).shape == (0, 5)
    assert ep.gemm_mxfp4(u8(5, 64), u8(1, 5, 4), u8(0, 64), u8(1, 0, 4)).shape == (5, 0)
    assert torch.equal(ep.gemm_mxfp4(u8(3, 0), u8(0, 3, 4), u8(5, 0), u8(0, 5, 4), b), b.expand(3, 5))
    assert torch.equal(ep.gemm_mxfp4(u8(3, 0), u8(0, 3, 4), u8(5, 0), u8(0, 5, 4)), torch.zeros((3, 5), device="cuda").bfloat16())


@pytest.mark.parametrize("M,N,K", [(7, 70, 384), (140, 200, 640)])
def test_product_scales_far_apart(M, N, K):
    """Scale bytes over the whole range of one operand, the middle of the other's; blocks of zeros beside large ones."""
    g = gen(9)
    (xq, xs), (wq, ws) = mx.random_matrix(g, M, K), mx.random_matrix(g, N, K)
    xs = torch.randint(20, 230, xs.shape, generator=g, dtype=torch.uint8)
    xq[:, 16:32] = 0
    y = ep.gemm_mxfp4(*(t.cuda() for t in (xq, xs, wq, ws)), out_dtype=torch.float32)
    mx.check_product(y, mx.values(xq, xs), mx.values(wq, ws))


@pytest.mark.parametrize("M", [20, 150])
def test_product_nan_blocks(M):
    """A NaN block makes its own row (or column) NaN and no other, whatever the codes."""
    g = gen(10)
    (xq, xs), (wq, ws) = mx.random_matrix(g, M, 512), mx.random_matrix(g, 90, 512)
    xq[3, 16 * 5:16 * 6] = 0
    xs[1, 3, 1] = 255
    xs[3, M - 1, 3] = 255
    ws[0, 41, 0] = 255
    y = ep.gemm_mxfp4(*(t.cuda() for t in (xq, xs, wq, ws)))
    mx.check_product(y, mx.values(xq, xs), mx.values(wq, ws))
    assert torch.isnan(y).sum() == 2 * 90 + M - 2


def test_product_of_misaligned_codes():
    g = gen(11)
    (xq, xs), (wq, ws) = mx.random_matrix(g, 30, 256), mx.random_matrix(g, 50, 256)

    def moved(t, by):
        room = torch.empty(t.numel() + by, dtype=torch.uint8, device="cuda")
        room[by:] = t.cuda().reshape(-1)
        return room[by:].view(t.shape)

    want = ep.gemm_mxfp4(*(t.cuda() for t in (xq, xs, wq, ws)))
    assert torch.equal(ep.gemm_mxfp4(moved(xq, 1), moved(xs, 3), moved(wq, 8), moved(ws, 1)), want)
    assert torch.equal(ep.dequantize_rows_mxfp4(moved(xq, 1), moved(xs, 3)), ep.dequantize_rows_mxfp4(xq.cuda(), xs.cuda()))


@pytest.mark.parametrize("counts,behind,N,K", [
    ([3], 0, 70, 128), ([0, 5, 0, 1, 17], 0, 130, 384), ([2, 0, 0, 40], 9, 64, 256), ([200, 1, 130, 0, 90], 3, 515, 640),
    ([0, 0, 0], 6, 33, 128), ([1] * 70, 2, 66, 256), ([0] * 127 + [300], 0, 129, 384), ([700, 650], 0, 300, 512),
    ([300, 515, 1, 700], 5, 200, 640), ([300, 515, 128, 640], 130, 8192, 256)])
def test_product_of_experts(counts, behind, N, K):
    g = gen(len(counts) + N)
    E, R = len(counts), sum(counts) + behind
    (xq, xs), (wq, ws) = mx.random_matrix(g, R, K), mx.random_matrix(g, E, N, K)
    bias = torch.randn((E, N), generator=g).to(torch.bfloat16)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    dev = [t.cuda() for t in (xq, xs, wq, ws, offsets)]
    x = mx.values(xq, xs)
    for dtype, b in ((torch.float32, None), (torch.bfloat16, bias)):
        y = ep.gemm_mxfp4_experts(*dev, b.cuda() if b is not None else None, out_dtype=dtype)
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            mx.check_product(y[lo:hi], x[lo:hi], mx.values(wq[e], ws[e]), None if b is None else b[e], f"expert {e}")
        assert not y[offsets[-1]:].any()


def test_wrong_offsets_stay_in_bounds():
    """Offsets outside the rows are clamped; what lies before and behind the result stays."""
    g = gen(12)
    (xq, xs), (wq, ws) = mx.random_matrix(g, 40, 128), mx.random_matrix(g, 3, 64, 128)
    for offsets in ([0, 50, 20, 40], [-5, 10, 1000, 7], [0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]):
        y = ep.gemm_mxfp4_experts(*(t.cuda() for t in (xq, xs, wq, ws)), torch.tensor(offsets, dtype=torch.int32).cuda())
        assert y.shape == (40, 64)


# --------------------------------------------------------------------------------- as they are used
def test_layer_against_the_unquantized_values():
    """Activations and weight quantized, multiplied: the product of the quantized values."""
    g = gen(13)
    x, w = torch.randn((45, 500), generator=g).to(torch.bfloat16), torch.randn((77, 500), generator=g)
    (xq, xs), (wq, ws) = ep.quantize_rows_mxfp4(x.cuda()), ep.quantize_rows_mxfp4(w.cuda())
    mx.check_product(ep.gemm_mxfp4(xq, xs, wq, ws), mx.values(*mx.quantize(x)), mx.values(*mx.quantize(w)))


def test_decoded_weight_in_mxfp4():
    """A compressed weight decoded to BF16 and kept in MXFP4."""
    from decode_tile_interleaved_rans_amd import workloads as W
    stream, _ = ep.compress(W.gaussian_with_outliers(64, 512, seed=3), 4.5)
    w = ep.decompress(stream)
    x = torch.randn((20, 512), generator=gen(14)).to(torch.bfloat16).cuda()
    y = ep.gemm_mxfp4(*ep.quantize_rows_mxfp4(x), *ep.quantize_rows_mxfp4(w))
    mx.check_product(y, mx.values(*mx.quantize(x)), mx.values(*mx.quantize(w)))


@pytest.mark.parametrize("T,k,E,N,K", [(9, 2, 4, 70, 200), (150, 3, 6, 129, 384)])
def test_expert_layer(T, k, E, N, K):
    """Tokens sorted, quantized, multiplied by their experts and summed back."""
    g = gen(T)
    x = torch.randn((T, K), generator=g).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    ids[1, 0] = -1
    weights = torch.rand((T, k), generator=g)
    wq, ws = ep.quantize_rows_mxfp4(torch.randn((E, N, K), generator=g).cuda())
    rows, offsets, pos = ep.sort_tokens(x.cuda(), ids.cuda(), E)
    ys = ep.gemm_mxfp4_experts(*ep.quantize_rows_mxfp4(rows), wq, ws, offsets, out_dtype=torch.float32)
    y = ep.combine_tokens(ys, pos, weights.cuda()).cpu().double()
    xv, wv = mx.values(*mx.quantize(x)), mx.values(wq, ws)
    ref, mag = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                ref[t] += weights[t, j].double() * (wv[ids[t, j]] @ xv[t])
                mag[t] += weights[t, j].double() * (wv[ids[t, j]].abs() @ xv[t].abs())
    # the product's additions (check_product), its weight and the sum over the choices, each off by 2^-23 at most
    assert ((y - ref).abs() <= (wv.shape[-1] / 32 + 3 + k + 1) * 2.0 ** -23 * mag).all()


def test_other_stream():
    g = gen(15)
    x = torch.randn((64, 1024), generator=g).cuda().to(torch.bfloat16)
    w = torch.randn((256, 1024), generator=g).cuda()
    wq, ws = ep.quantize_rows_mxfp4(w)
    xq, xs = ep.quantize_rows_mxfp4(x)
    want = ep.gemm_mxfp4(xq, xs, wq, ws)
    side = torch.cuda.Stream()
    for _ in range(3):
        q2, s2 = ep.quantize_rows_mxfp4(x, stream=side)
        with torch.cuda.stream(side):
            y = ep.gemm_mxfp4(q2, s2, wq, ws)
            v = ep.dequantize_rows_mxfp4(q2, s2)
        z = ep.gemm_mxfp4(xq, xs, wq, ws, stream=side)
        side.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want) and torch.equal(v, ep.dequantize_rows_mxfp4(xq, xs))


def test_captured_and_replayed():
    """A layer in a graph: every replay, with new inputs and eager work between, gives the eager result."""
    g = gen(16)
    E, k = 4, 2
    x = torch.randn((50, 384), generator=g).cuda().to(torch.bfloat16)
    ids = torch.randint(0, E, (50, k), generator=g).cuda()
    wq, ws = ep.quantize_rows_mxfp4(torch.randn((E, 96, 384), generator=g).cuda())

    def layer():
        rows, offsets, pos = ep.sort_tokens(x, ids, E)
        return ep.combine_tokens(ep.gemm_mxfp4_experts(*ep.quantize_rows_mxfp4(rows), wq, ws, offsets), pos)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for i in range(4):
        x.copy_(torch.randn((50, 384), generator=g).to(torch.bfloat16))
        ids.copy_(torch.randint(0, E, (50, k), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer()), i


def test_refusals_of_tensors():
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")
    ok = (u8(4, 64), u8(1, 4, 4), u8(6, 64), u8(1, 6, 4))
    ep.gemm_mxfp4(*ok)
    bad = [
        (u8(4, 63), *ok[1:]), (ok[0], u8(1, 4, 3), *ok[2:]), (ok[0], u8(4, 4), *ok[2:]), (ok[0].to(torch.int8), *ok[1:]),
        (ok[0].cpu(), *ok[1:]), (ok[0], ok[1].cpu(), *ok[2:]), (ok[0], ok[1], u8(6, 128), u8(2, 6, 4)), (*ok[:2], u8(2, 6, 64), u8(2, 1, 6, 4)),
        (u8(64, 4).t(), *ok[1:]), (*ok[:3], u8(1, 5, 4)),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            ep.gemm_mxfp4(*args)
    with pytest.raises(ValueError):
        ep.gemm_mxfp4(*ok, torch.zeros(6, device="cuda"))
    with pytest.raises(ValueError):
        ep.gemm_mxfp4(*ok, out_dtype=torch.int8)
    with pytest.raises(ValueError):
        ep.gemm_mxfp4_experts(*ok, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ep.gemm_mxfp4_experts(*ok[:2], u8(2, 6, 64), u8(2, 1, 6, 4), torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ep.quantize_rows_mxfp4(torch.zeros((4, 64), dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        ep.quantize_rows_mxfp4(torch.zeros((2, 4, 64), device="cuda")[:, :, :32])
    with pytest.raises(ValueError):
        ep.quantize_rows_mxfp4(torch.zeros(64, device="cuda"))
    with pytest.raises(ValueError):
        ep.dequantize_rows_mxfp4(*ok[:2], columns=129)
    with pytest.raises(ValueError):
        ep.dequantize_rows_mxfp4(*ok[:2], torch.int8)


def test_threads():
    """Calls from several threads at once, each on a stream of its own."""
    g = gen(17)
    sets = []
    for i in range(4):
        x, w = torch.randn((70 + i, 640), generator=g).cuda().to(torch.bfloat16), torch.randn((130, 640), generator=g).cuda()
        sets.append((x, *ep.quantize_rows_mxfp4(w)))
    layer = lambda i: ep.gemm_mxfp4(*ep.quantize_rows_mxfp4(sets[i][0]), *sets[i][1:])
    want = [layer(i) for i in range(4)]
    side = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(side[i]):
            return [layer(i) for _ in range(20)]

    with ThreadPoolExecutor(4) as pool:
        done = list(pool.map(work, range(4)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(4) for y in done[i])


# ---------------------------------------------------------------------------- offsets past 32 bits
def repeats(y, rows):
    """All rows of y (its first dimension) repeat the first `rows`, bit for bit."""
    v = y.view(torch.int16) if y.dtype == torch.bfloat16 else y
    return bool((v.reshape(-1, rows, *v.shape[1:]) == v[:rows]).all())


def test_many_rows():
    """9.2e9 elements, 4.6e9 bytes of codes: rows that repeat give codes, values and products that repeat."""
    base = torch.randn((1000, 65536), generator=gen(18)).to(torch.bfloat16).cuda()
    x = base.repeat(140, 1)
    q, s = ep.quantize_rows_mxfp4(x)
    assert q.numel() > 2 ** 32 and repeats(q, 1000) and repeats(s.transpose(0, 1), 1000)
    q0, s0 = ep.quantize_rows_mxfp4(base)
    assert torch.equal(q[:1000], q0) and torch.equal(s[:, :1000], s0)
    same_codes(base[:50], *ep.quantize_rows_mxfp4(base[:50]))
    del x
    v = ep.dequantize_rows_mxfp4(q, s)
    assert repeats(v, 1000) and torch.equal(v[:1000], ep.dequantize_rows_mxfp4(q0, s0))
    del v
    wq, ws = mx.random_matrix(gen(19), 64, 65536)
    y = ep.gemm_mxfp4(q, s, wq.cuda(), ws.cuda())
    assert repeats(y, 1000)
    mx.check_product(y[:50], mx.values(q[:50], s[:, :50]), mx.values(wq, ws))


def test_many_outputs():
    """4.9e9 outputs."""
    (xq, xs), (wq, ws) = mx.random_matrix(gen(20), 1000, 128), mx.random_matrix(gen(21), 16384, 128)
    y = ep.gemm_mxfp4(xq.cuda().repeat(300, 1), xs.cuda().repeat(1, 300, 1), wq.cuda(), ws.cuda())
    assert y.numel() > 2 ** 32 and repeats(y, 1000)
    mx.check_product(y[:200, -300:], mx.values(xq[:200], xs[:, :200]), mx.values(wq[-300:], ws[:, -300:]))


def test_experts_past_32_bits():
    """5.4e9 bytes of the experts' codes."""
    E, N, K = 20, 8192, 65536
    (xq, xs), (wq, ws) = mx.random_matrix(gen(22), 5, K), mx.random_matrix(gen(23), N, K)
    allq, alls = (torch.zeros((E, *t.shape), dtype=torch.uint8, device="cuda") for t in (wq, ws))
    allq[E - 1], alls[E - 1] = wq.cuda(), ws.cuda()
    assert allq[:E - 1].numel() > 2 ** 32
    offsets = torch.tensor([0] * E + [5], dtype=torch.int32).cuda()
    y = ep.gemm_mxfp4_experts(xq.cuda(), xs.cuda(), allq, alls, offsets)
    mx.check_product(y[:, -40:], mx.values(xq, xs), mx.values(wq[-40:], ws[:, -40:]))


def test_longest_rows():
    """K = 2^22, the limit, in a small tile and, by the experts' product, in tiles of 256 rows: rows that repeat."""
    K = 2 ** 22
    (xq, xs), (wq, ws) = mx.random_matrix(gen(24), 1, K), mx.random_matrix(gen(25), 1, K)
    x, w = mx.values(xq, xs), mx.values(wq, ws)
    mx.check_product(ep.gemm_mxfp4(*(t.cuda() for t in (xq, xs, wq, ws))), x, w)
    many = [xq.cuda().repeat(300, 1), xs.cuda().repeat(1, 300, 1), wq.cuda().repeat(260, 1)[None], ws.cuda().repeat(1, 260, 1)[None]]
    y = ep.gemm_mxfp4_experts(*many, torch.tensor([0, 300], dtype=torch.int32).cuda(), out_dtype=torch.float32)
    assert (y == y[0, 0]).all()
    mx.check_product(y[:1, :1], x, w)
    v = torch.randn((2, K), generator=gen(26))
    same_codes(v, *ep.quantize_rows_mxfp4(v.cuda()))


def test_most_rows():
    """2^27 rows, the limit, of one block."""
    base = torch.randn((4096, 32), generator=gen(27)).to(torch.bfloat16)
    q, s = ep.quantize_rows_mxfp4(base.cuda().repeat(2 ** 15, 1))
    assert repeats(q, 4096) and repeats(s[0], 4096)
    same_codes(base, q[:4096], s[:, :4096])
    wq, ws = mx.random_matrix(gen(28), 3, 128)
    y = ep.gemm_mxfp4(q, s, wq.cuda(), ws.cuda())
    assert repeats(y, 4096)
    mx.check_product(y[:4096], mx.values(*mx.quantize(base)), mx.values(wq, ws))
