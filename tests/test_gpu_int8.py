"""The INT8 products on the GPU: the row quantizer, the product with a scale per token and per channel,
the same per expert, and the compressed linear layer's INT8 forward.

References are computed in 64 bits. The quantizer must give the same codes and scales bit for bit: its
rounding is decided exactly, and 127 x / a in fp64 can neither reach nor leave a rounding border (127 x
is exact, and a quotient of two fp32 numbers that is not on a border is at least 2^-33 of itself away
from it). The products' int32 sums are exact, so an output differs from the reference by fp32 steps
only: the sum's conversion, two scale products and the bias, each at most 2^-24 relative, then the
output type's rounding (half of finfo.eps)."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
import decode_tile_interleaved_rans_amd as ep
from decode_tile_interleaved_rans_amd import workloads as W

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def reference_codes(x):
    x64 = x.double()
    a = x64.abs().amax(1, keepdim=True)
    a = torch.where(a > 0, a.clamp_min(2.0 ** -100), a)
    q = torch.where(a > 0, 127.0 * x64 / torch.where(a > 0, a, 1.0), 0.0).round()
    return q.to(torch.int8), (a[:, 0] / 127.0).float()


def same_codes(x):
    q, s = ep.quantize_rows_int8(x)
    wq, ws = reference_codes(x)
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    assert torch.equal(s, ws)
    assert torch.equal(q, wq), f"{(q != wq).sum().item()} codes differ"
    return q, s


# ------------------------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 17), (5, 64), (2, 513), (7, 1000), (4, 1024), (3, 1025), (2, 2048),
                                 (9, 4096), (1, 8192), (2, 10240), (3, 16384), (2, 16392), (2, 20001), (300, 24)])
def test_quantizer_codes(M, K, dtype):
    g = gen(M * 1000 + K)
    x = torch.randn((M, K), generator=g, device="cuda") * torch.exp(torch.randn((M, 1), generator=g, device="cuda"))
    same_codes(x.to(dtype))


@pytest.mark.parametrize("K", [24, 1027, 4096])
def test_quantizer_at_rounding_borders(K):
    # ties ((k + 1/2) a / 127 exactly) and the fp32 neighbours of every border, rows of differing maximum
    rng = np.random.default_rng(K)
    rows = []
    for a in [127.0, 127.0 * 2 ** -30, 1.0, 3.0, 0.7, 1e30, 1e-20, 3.4e38]:
        a = np.float32(a)
        k = rng.integers(-127, 127, K)
        x = ((k + 0.5) * (float(a) / 127.0)).astype(np.float32)
        step = rng.integers(-2, 3, K)
        for _ in range(2):
            x = np.where(step > 0, np.nextafter(x, np.float32(np.inf)), np.where(step < 0, np.nextafter(x, np.float32(-np.inf)), x))
            step = step - np.sign(step)
        x[0] = a
        rows.append(np.clip(x, -a, a))
    x = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    same_codes(x)
    for t in (torch.bfloat16, torch.float16):
        same_codes(x[:5].to(t))                               # the rows that fp16 can hold


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [40, 1001, 4096])
def test_quantizer_special_rows(K, dtype):
    x = torch.randn((8, K), generator=gen(3), device="cuda").to(dtype)
    tiny = torch.finfo(dtype).smallest_normal / 64 if dtype != torch.float32 else 2.0 ** -149
    x[1] = 0
    x[2, K // 2] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = float("-inf")
    x[5] = 0
    x[5, 3] = tiny                                            # a subnormal row maximum
    x[6] = -0.0
    x[7, 1] = torch.finfo(dtype).max
    q, s = ep.quantize_rows_int8(x)
    fine = torch.tensor([0, 1, 5, 6, 7], device="cuda")
    wq, ws = reference_codes(x[fine])
    assert torch.equal(q[fine], wq) and torch.equal(s[fine], ws)
    for r in (2, 3, 4):
        assert torch.isnan(s[r]) and not q[r].any()
    assert s[1] == 0 and s[6] == 0


@pytest.mark.parametrize("K", [1, 7, 8, 9, 511, 1025, 2049, 8193, 16385, 40003])
def test_quantizer_clears_its_own_rows(K):
    # zero rows and rows without a scale between ordinary ones, in memory that held something else
    M = 9
    x = torch.randn((M, K), generator=gen(K), device="cuda").to(torch.bfloat16)
    x[1:3] = 0
    x[5, K - 1], x[7, 0] = float("nan"), float("inf")
    held = torch.full((M * K + 64,), 77, dtype=torch.int8, device="cuda")
    s = torch.full((M,), 5.0, device="cuda")
    q = held[32:32 + M * K].view(M, K)
    ep._check(ep.lib().ep_quantize_rows_int8(x.data_ptr(), ep.BF16, M, K, K, q.data_ptr(), s.data_ptr(),
                                             torch.cuda.current_stream().cuda_stream), "ep_quantize_rows_int8")
    good = [0, 3, 4, 6, 8]
    wq, ws = reference_codes(x[good])
    assert torch.equal(q[good], wq) and torch.equal(s[good], ws)
    assert not q[[1, 2, 5, 7]].any() and not s[1:3].any() and s[[5, 7]].isnan().all()
    assert (held[:32] == 77).all() and (held[32 + M * K:] == 77).all()


def test_quantizer_longest_row():
    # 2^31 - 1 elements: a step behind the last of them leaves 32 bits
    K = 2 ** 31 - 1
    x = torch.zeros((1, K), dtype=torch.bfloat16, device="cuda")
    held = torch.full((K + 1 + 64,), 77, dtype=torch.int8, device="cuda")
    s = torch.full((1,), 5.0, device="cuda")
    for last in (0.0, float("inf"), -3.0):
        held.fill_(77)
        x[0, K - 1] = last
        ep._check(ep.lib().ep_quantize_rows_int8(x.data_ptr(), ep.BF16, 1, K, K, held.data_ptr() + 32, s.data_ptr(),
                                                 torch.cuda.current_stream().cuda_stream), "ep_quantize_rows_int8")
        assert int(held[32 + K - 1]) == (-127 if last == -3.0 else 0) and not held[32:32 + K - 1].any()
        assert (held[:32] == 77).all() and (held[32 + K:] == 77).all()
        assert s.isnan().all() if last == float("inf") else float(s) == float(np.float32(abs(last)) / np.float32(127))


def test_quantizer_row_strides_and_offsets():
    base = torch.randn((20, 3000), generator=gen(4), device="cuda").to(torch.bfloat16)
    for x in (base[:, 8:1032], base[:, 3:1000], base[::2, :512], base[4:5, 1:9], base[:, :1]):
        q, s = ep.quantize_rows_int8(x)
        wq, ws = reference_codes(x)
        assert torch.equal(q, wq) and torch.equal(s, ws)


# ------------------------------------------------------------------------------------ product
def operands(M, N, K, seed, full=False):
    g = gen(seed)
    lim = 128 if full else 127
    xq = torch.randint(-lim, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-lim, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.exp(torch.randn(M, generator=g, device="cuda")) * 1e-3
    ws = torch.exp(torch.randn(N, generator=g, device="cuda")) * 1e-3
    b = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16)
    return xq, xs, wq, ws, b


def product64(xq, wq):
    return torch.mm(xq.double(), wq.double().t().contiguous())


def check_product(y, acc, xs, ws, b):
    v = acc * xs.double()[:, None] * ws.double()[None, :]
    ref = v if b is None else v + b.double()
    fp32 = 4 * U * (v.abs() + (0 if b is None else b.double().abs()))
    half = torch.finfo(y.dtype).eps / 2
    tiny = 2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -134       # half a subnormal step
    tol = fp32 + half * (ref.abs() + fp32) + tiny
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), f"largest excess {(err - tol).max().item():.3g} at {int((err - tol).argmax())}"


SHAPES = [(1, 1, 16), (1, 17, 32), (2, 64, 128), (5, 100, 144), (16, 48, 1024), (17, 33, 4112), (31, 130, 256), (33, 20, 512),
          (64, 257, 2048), (65, 63, 640), (100, 500, 96), (128, 128, 128), (200, 1000, 1040), (257, 300, 16), (130, 4100, 272),
          (700, 1300, 400), (1030, 2050, 256), (4100, 4099, 144), (1000, 11500, 272), (1000, 7001, 144), (333, 5003, 272),
          (2048, 8190, 144), (64, 8190, 144), (16, 11520, 144)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, out):
    xq, xs, wq, ws, b = operands(M, N, K, M + N + K)
    acc = product64(xq, wq)
    check_product(ep.gemm_int8(xq, xs, wq, ws, out_dtype=out), acc, xs, ws, None)
    check_product(ep.gemm_int8(xq, xs, wq, ws, b, out_dtype=out), acc, xs, ws, b)


@pytest.mark.parametrize("M,N,K", [(1, 5, 1), (3, 70, 15), (40, 33, 17), (90, 65, 127), (300, 401, 1001),
                                   (200, 130, 1500), (20, 50, 4097), (3, 4, 130945), (2, 5, 131041)])
def test_product_of_any_width(M, N, K):
    xq, xs, wq, ws, b = operands(M, N, K, K)
    check_product(ep.gemm_int8(xq, xs, wq, ws, b), product64(xq, wq), xs, ws, b)
    # codes laid out once by the program give the same bits
    xp, wp = ep.pad_rows_int8(xq), ep.pad_rows_int8(wq)
    assert xp.shape[1] % 16 == 0 and torch.equal(xp[:, :K], xq) and not xp[:, K:].any()
    assert torch.equal(ep.gemm_int8(xp, xs, wp, ws, b), ep.gemm_int8(xq, xs, wq, ws, b))


def test_product_misaligned_codes():
    xq, xs, wq, ws, b = operands(50, 70, 256, 7)
    flat = torch.zeros(50 * 256 + 3, dtype=torch.int8, device="cuda")
    off = flat[3:].view(50, 256)
    off.copy_(xq)
    assert torch.equal(ep.gemm_int8(off, xs, wq, ws, b), ep.gemm_int8(xq, xs, wq, ws, b))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_longest_sum_does_not_overflow(M):
    # every product 2^14: the largest sum an int8 row of 131056 codes can reach, and its negative
    K = 131056
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((20, K), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    xs, ws = torch.ones(M, device="cuda"), torch.ones(20, device="cuda")
    y = ep.gemm_int8(xq, xs, wq, ws, out_dtype=torch.float32)
    assert (y[:, 0] == float(np.float32(K * 16384))).all() and (y[:, 1] == float(np.float32(-K * 128 * 127))).all()


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_empty_sum_and_empty_sides(M):
    xq, xs, wq, ws, b = operands(M, 40, 16, 1)
    e = torch.empty
    y = ep.gemm_int8(e((M, 0), dtype=torch.int8, device="cuda"), xs, e((40, 0), dtype=torch.int8, device="cuda"), ws, b)
    assert torch.equal(y, b.expand(M, 40))
    assert ep.gemm_int8(xq[:0], xs[:0], wq, ws).shape == (0, 40)
    assert ep.gemm_int8(xq, xs, wq[:0], ws[:0]).shape == (M, 0)


def test_widest_product_and_the_first_refused():
    # 131056 codes are the longest row whose laid-out width keeps the sums within int32; the next are refused
    # before anything is copied
    for K in (131055, 131056):
        xq, xs, wq, ws, b = operands(3, 5, K, 1, full=True)
        check_product(ep.gemm_int8(xq, xs, wq, ws, b), product64(xq, wq), xs, ws, b)
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    for K in (131057, 131071, 131072):
        xq, xs, wq, ws, b = operands(3, 5, K, 1)
        for call in (lambda: ep.gemm_int8(xq, xs, wq, ws), lambda: ep.gemm_int8_experts(xq, xs, wq[None], ws[None], off)):
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            with pytest.raises(ep.EPError, match="131056"):
                call()
            assert torch.cuda.max_memory_allocated() - before < K


def test_bad_rows_stay_bad():
    # a row with a NaN has scale NaN: its outputs are NaN and no other row's are
    x = torch.randn((70, 128), generator=gen(6), device="cuda").to(torch.bfloat16)
    x[13, 5] = float("nan")
    x[44, 0] = float("inf")
    _, _, wq, ws, _ = operands(1, 90, 128, 8)
    q, s = ep.quantize_rows_int8(x)
    y = ep.gemm_int8(q, s, wq, ws)
    nan = torch.isnan(y)
    assert nan[13].all() and nan[44].all() and int(nan.sum()) == 180


@pytest.mark.parametrize("K", [1024, 1040, 272])
@pytest.mark.parametrize("which", ["x", "w", "both"])
def test_only_misaligned_codes_are_copied(which, K):
    E, R, N = 4, 20, 512
    xq, xs, _, _, _ = operands(R, 1, K, 5)
    wq, ws, b = zip(*(operands(1, N, K, 6 + e)[2:] for e in range(E)))
    wq, ws, b = torch.stack(wq), torch.stack(ws), torch.stack(b)
    off = torch.tensor([0, 3, 3, 11, 20], dtype=torch.int32, device="cuda")

    def moved(t):
        flat = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:] = t.reshape(-1)
        return flat[3:].view(t.shape)

    x2, w2 = moved(xq) if which != "w" else xq, moved(wq) if which != "x" else wq
    want, one = ep.gemm_int8_experts(xq, xs, wq, ws, off, b), ep.gemm_int8(xq, xs, wq[1], ws[1], b[1])
    small, large = xq.numel(), wq.numel()
    for call, ref, weight in ((lambda: ep.gemm_int8_experts(x2, xs, w2, ws, off, b), want, large),
                              (lambda: ep.gemm_int8(x2, xs, w2[1], ws[1], b[1]), one, large // E)):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        assert torch.equal(call(), ref)
        used = torch.cuda.max_memory_allocated() - before
        room = 2 * ref.numel() + ref.numel() + 8192            # the output, its comparison, the allocator's units
        assert used <= room + (small if which != "w" else 0) + (weight if which != "x" else 0)
        assert used >= (weight if which != "x" else 0)


def test_rows_do_not_depend_on_their_batch():
    # exact sums: a row's outputs are the same bits whatever the other rows and the kernel chosen
    xq, xs, wq, ws, b = operands(4200, 1100, 528, 12)
    y = ep.gemm_int8(xq, xs, wq, ws, b)
    for M in (1, 16, 20, 64, 65, 300, 1500):
        assert torch.equal(ep.gemm_int8(xq[:M], xs[:M], wq, ws, b), y[:M]), M


# ------------------------------------------------------------------------------------ experts
def expert_case(counts, N, K, R, seed):
    E = len(counts)
    g = gen(seed)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    xq = torch.randint(-127, 128, (R, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.exp(torch.randn(R, generator=g, device="cuda")) * 1e-3
    ws = torch.exp(torch.randn((E, N), generator=g, device="cuda")) * 1e-3
    b = torch.randn((E, N), generator=g, device="cuda").to(torch.bfloat16)
    return off, xq, xs, wq, ws, b


COUNTS = [[1], [0], [0, 3, 0], [16, 17, 1, 0, 64], [5] * 100, [0] * 70 + [9] + [0] * 200, [300, 0, 1, 129], [1000, 7, 513, 64],
          [2500, 2600], [40] * 60]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("N,K", [(100, 144), (520, 512)])
def test_experts(counts, N, K, out):
    R = sum(counts) + 21                                      # rows behind the last expert's
    off, xq, xs, wq, ws, b = expert_case(counts, N, K, R, sum(counts) + N)
    for bias in (None, b):
        y = ep.gemm_int8_experts(xq, xs, wq, ws, off, bias, out_dtype=out)
        assert not y[sum(counts):].any()
        a = 0
        for e, c in enumerate(counts):
            if c:
                check_product(y[a:a + c], product64(xq[a:a + c], wq[e]), xs[a:a + c], ws[e], None if bias is None else b[e])
                assert torch.equal(y[a:a + c], ep.gemm_int8(xq[a:a + c], xs[a:a + c], wq[e], ws[e],
                                                            None if bias is None else b[e], out_dtype=out))
            a += c


# tiles of 128 x 192, 128 x 256, 128 x 128 and 128 x 64
@pytest.mark.parametrize("counts,N", [([700, 0, 129, 1, 900], 4001), ([100] * 19 + [191], 4000), ([33, 64, 40, 1, 60], 7000),
                                      ([30] * 20, 1000)], ids=["192", "256", "128", "64"])
def test_experts_that_fill_the_chip(counts, N):
    K, R = 272, sum(counts) + 150
    off, xq, xs, wq, ws, b = expert_case(counts, N, K, R, N)
    y = ep.gemm_int8_experts(xq, xs, wq, ws, off, b)
    assert not y[sum(counts):].any()
    a = 0
    for e, c in enumerate(counts):
        if c:
            check_product(y[a:a + c], product64(xq[a:a + c], wq[e]), xs[a:a + c], ws[e], b[e])
        a += c


def test_experts_any_width_and_no_rows():
    off, xq, xs, wq, ws, b = expert_case([3, 0, 40], 33, 75, 43, 5)
    y = ep.gemm_int8_experts(xq, xs, wq, ws, off, b)
    check_product(y[:3], product64(xq[:3], wq[0]), xs[:3], ws[0], b[0])
    check_product(y[3:], product64(xq[3:], wq[2]), xs[3:], ws[2], b[2])
    assert ep.gemm_int8_experts(xq[:0], xs[:0], wq, ws, torch.zeros_like(off), b).shape == (0, 33)


def test_experts_wrong_offsets_stay_inside():
    # offsets out of range or order give wrong rows, never an access outside: rows that are written
    # belong to the result and everything around it keeps its values
    off, xq, xs, wq, ws, b = expert_case([8, 8, 8], 64, 128, 24, 9)
    for bad in ([0, 100, 5, 24], [0, -7, 12, 9], [0, 24, 24, 2 ** 31 - 1], [-2 ** 31, 0, 0, 0]):
        o = torch.tensor(bad, dtype=torch.int64, device="cuda").to(torch.int32)
        assert ep.gemm_int8_experts(xq, xs, wq, ws, o, b).shape == (24, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("R", [40, 300])
@pytest.mark.parametrize("out", TYPES)
def test_experts_wrong_offsets_write_nothing_outside(R, out):
    # Y in the middle of a larger buffer: whatever the offsets say, no row before or behind it changes, and the
    # calls after them are right again
    E, N, K, guard = 3, 100, 64, 96
    xq, xs, wq, ws, b = operands(R, E * N, K, 8)
    held = torch.full((guard + R + guard, N), 7.0, dtype=out, device="cuda")
    y, code = held[guard:guard + R], {torch.bfloat16: ep.BF16, torch.float16: ep.F16, torch.float32: ep.F32}[out]

    def call(offs):
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        ep._check(ep.lib().ep_gemm_int8_experts(xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), off.data_ptr(), E, R,
                                                N, K, b.data_ptr(), code, y.data_ptr(), torch.cuda.current_stream().cuda_stream),
                  "ep_gemm_int8_experts")
        assert (held[:guard] == 7).all() and (held[guard + R:] == 7).all()

    top = 2 ** 31 - 1
    for offs in ([0, 5, 3, R], [0, R + 50, 7, 20], [-5, 1, 2, 3], [0, 0, 0, top], [R - 1, R + 1, R + 60, R + 95], [top] * 4,
                 [-top - 1, -1, top, -top], [R, R, R, R], [20, 10, 5, 0]):
        call(offs)
    call([0, 11, 11, R - 4])
    for e, (a, z) in enumerate(((0, 11), (11, 11), (11, R - 4))):
        if z > a:
            part = slice(e * N, (e + 1) * N)
            check_product(y[a:z], product64(xq[a:z], wq[part]), xs[a:z], ws[part], b[part])
    assert not y[R - 4:].any()


def test_experts_take_new_offsets_in_a_captured_graph():
    off, xq, xs, wq, ws, b = expert_case([10, 0, 30, 8], 200, 256, 64, 15)
    y = ep.gemm_int8_experts(xq, xs, wq, ws, off, b)           # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ep.gemm_int8_experts(xq, xs, wq, ws, off, b)
    for counts in ([10, 0, 30, 8], [0, 0, 0, 0], [64, 0, 0, 0], [1, 1, 1, 61], [16, 16, 16, 16]):
        off.copy_(torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32))
        xq.copy_(torch.roll(xq, 1, 0))
        graph.replay()
        want = ep.gemm_int8_experts(xq, xs, wq, ws, off, b)    # eager work between replays
        torch.cuda.synchronize()
        assert torch.equal(y, want), counts


def test_large_result_offsets():
    # more than 2^31 bytes and more than 2^31 / 2 elements of output: 64-bit addresses in the epilogue
    M, N, K = 70000, 32768, 16
    xq, xs, wq, ws, _ = operands(M, N, K, 3)
    y = ep.gemm_int8(xq, xs, wq, ws)
    for r in (0, 32768, 65535, M - 100):
        check_product(y[r:r + 100], product64(xq[r:r + 100], wq), xs[r:r + 100], ws, None)
    del y


def test_experts_weights_past_32_bit_offsets():
    # 4.8e9 codes of weights: the last experts lie past 2^31 and 2^32 bytes
    E, N, K = 72, 8192, 8192
    wq = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    for e in range(E):
        wq[e] = torch.randint(-127, 128, (N, K), generator=gen(e), device="cuda", dtype=torch.int8)
    counts = [0] * E
    counts[3], counts[35], counts[E - 1] = 5, 70, 9
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    R = sum(counts)
    xq = torch.randint(-127, 128, (R, K), generator=gen(99), device="cuda", dtype=torch.int8)
    xs, ws = torch.full((R,), 1e-3, device="cuda"), torch.full((E, N), 1e-3, device="cuda")
    y = ep.gemm_int8_experts(xq, xs, wq, ws, off)
    for e, a, b in ((3, 0, 5), (35, 5, 75), (E - 1, 75, 84)):
        check_product(y[a:b], product64(xq[a:b], wq[e]), xs[a:b], ws[e], None)


def test_layer_files_and_model_replacement_in_int8(tmp_path):
    from decode_tile_interleaved_rans_amd import plan
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(256, 192), torch.nn.GELU(), torch.nn.Linear(192, 64)).cuda()
    a = ep.CompressedLinear.from_linear(model[0], 5.0, compute="int8")
    a.save(tmp_path / "a.npz")
    x = torch.randn((33, 256), generator=gen(2), device="cuda").to(torch.bfloat16)
    y = a(x)
    assert torch.equal(ep.CompressedLinear.load(tmp_path / "a.npz", compute="int8")(x), y)
    assert torch.equal(a(x.view(3, 11, 256)), y.view(3, 11, 192))
    streams = {n: ep.compress(model[int(n)].weight, 5.0, layout=ep.ROW_LAYOUT, prob_bits=11)[0] for n in ("0", "2")}
    originals = plan.replace_linears(model, streams, compute="int8")
    assert torch.equal(model[0](x), y) and model(x).shape == (33, 64)
    plan.restore_linears(model, originals)


def test_other_stream():
    xq, xs, wq, ws, b = operands(300, 400, 512, 31)
    x = torch.randn((300, 512), generator=gen(32), device="cuda").to(torch.bfloat16)
    want_y, (want_q, want_s) = ep.gemm_int8(xq, xs, wq, ws, b), ep.quantize_rows_int8(x)
    s = torch.cuda.Stream()
    for _ in range(3):
        big = torch.randn((4096, 4096), device="cuda")
        big = big @ big                                        # keeps the current stream busy
        x2 = x + 0                                             # made on it
        y = ep.gemm_int8(xq + 0, xs, wq, ws, b, stream=s)
        q, sc = ep.quantize_rows_int8(x2, stream=s)
        del x2
        s.synchronize()
        assert torch.equal(y, want_y) and torch.equal(q, want_q) and torch.equal(sc, want_s)


# ------------------------------------------------------------------------------------ compressed layer
@pytest.mark.parametrize("layout", [0, ep.ROW_LAYOUT])
@pytest.mark.parametrize("M", [1, 16, 33, 64, 65, 300])
def test_compressed_forward(M, layout):
    N, K = 300, 1040
    s, _ = ep.compress(W.student_t(N, K, 5), 4.5, dtype=ep.BF16, layout=layout, prob_bits=11)
    bias = torch.randn(N, generator=gen(5), device="cuda").to(torch.bfloat16)
    layer = ep.CompressedLinear(s, bias, compute="int8")
    xb = W.activations(M, K, 6)
    x = torch.from_numpy(xb.view(np.int16)).view(torch.bfloat16).cuda()
    y = layer(x)
    layer.handle.check()
    cq, cs = oracle.decompress(s, oracle.I8)
    xq, xs = reference_codes(x)
    wq, ws = torch.from_numpy(cq.view(np.int8)).cuda(), torch.from_numpy(cs).cuda()   # the oracle returns bytes
    check_product(y, product64(xq, wq), xs, ws, bias)
    # the same bits as the parts called one by one
    dq, ds = layer.handle.decompress(torch.int8)
    assert torch.equal(dq, wq) and torch.equal(ds, ws)
    assert torch.equal(y, ep.gemm_int8(*ep.quantize_rows_int8(x), dq, ds, bias))
    assert torch.equal(ep.linear_forward_many([layer, layer], x)[1], y)


@pytest.mark.parametrize("M", [1, 16, 40, 64, 65])
def test_layers_that_share_an_input(M):
    K = 784
    layers = []
    for i, N in enumerate((300, 16, 1000)):
        s, _ = ep.compress(W.student_t(N, K, 40 + i), 4.5, dtype=ep.BF16, layout=ep.ROW_LAYOUT, prob_bits=11)
        b = torch.randn(N, generator=gen(i), device="cuda").to(torch.bfloat16) if i != 1 else None
        layers.append(ep.CompressedLinear(s, b, compute="int8"))
    s0, _ = ep.compress(W.student_t(64, K, 50), 4.5, dtype=ep.BF16, layout=0, prob_bits=11)
    x = torch.randn((M, K), generator=gen(M), device="cuda").to(torch.bfloat16)
    for group in (layers, layers[:1], layers + [ep.CompressedLinear(s0, compute="int8")]):   # the last not fused
        for y, l in zip(ep.linear_forward_many(group, x), group):
            assert torch.equal(y, l(x))
            l.handle.check()


def test_compressed_forward_on_two_slices():
    # a weight of more than one 128 MiB slice, 128 MiB / K rows each
    N, K, M = 9000, 16384, 70
    w = W.gpu_student_t(N, K, 3)
    s, _ = ep.compress_device(w, 3.0, layout=ep.ROW_LAYOUT, prob_bits=11)
    layer = ep.CompressedLinear(s, compute="int8")
    x = torch.randn((M, K), generator=gen(8), device="cuda").to(torch.bfloat16)
    dq, ds = layer.handle.decompress(torch.int8)
    assert torch.equal(layer(x), ep.gemm_int8(*ep.quantize_rows_int8(x), dq, ds))


def layer_of(N, K, seed, compute):
    s, _ = ep.compress_device(W.gpu_student_t(N, K, seed), 4.0, layout=ep.ROW_LAYOUT, prob_bits=11)
    return ep.CompressedLinear(s, None, compute)


@pytest.mark.parametrize("compute", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("M", [20, 100])                       # fused, and slices with a product
def test_captured_forwards_keep_their_workspace(M, compute):
    """A graph holds the address of its stream's workspace. Later forwards that need a larger one, or evict the
    stream's from the pool, must not hand that memory to others."""
    layer, large = layer_of(200, 1040, M, compute), layer_of(512, 2048, M, compute)
    x, xl = torch.empty((M, 1040), dtype=torch.bfloat16, device="cuda"), torch.zeros((9000, 2048), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    x.normal_(generator=gen(M))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        layer(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        y = layer(x)
    if M == 100:
        with torch.cuda.stream(st):
            large(xl)                                          # grows the stream's workspace
        torch.cuda.synchronize()
    held = []
    for i in range(6):                                         # more streams than the pool keeps entries
        with torch.cuda.stream(torch.cuda.Stream()):
            large(xl)
        torch.cuda.synchronize()
        held.append(torch.full((1 << 24,), i, dtype=torch.uint8, device="cuda"))
        x.normal_(generator=gen(10 + i))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x)), i
    for i, t in enumerate(held):
        assert (t == i).all()
    layer.handle.check()


@pytest.mark.parametrize("compute", ["fp8", "int8"])
def test_capture_that_has_to_allocate(compute):
    # a workspace that is too small, then none, for the stream: the capture takes a new one, and the one that it
    # replaces is freed by later eager calls
    layer = layer_of(64, 4096, 1, compute)
    x = torch.empty((30000, 4096), dtype=torch.bfloat16, device="cuda")          # 117 MiB of codes
    st, graphs = torch.cuda.Stream(), []
    for warm in (True, False):
        if warm:
            layer(x.normal_(generator=gen(1)))                 # the library's handles and plans
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                layer(x[:100])
            torch.cuda.synchronize()
        else:
            st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            y = layer(x)
        graphs.append((graph, y))
    for i in range(3):
        x.normal_(generator=gen(5 + i))
        for s in [st] + [torch.cuda.Stream() for _ in range(5)]:
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                layer(x[:2000 + i])
        want = layer(x)
        torch.cuda.synchronize()
        for graph, y in graphs:
            y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), i


def test_c_abi_refusals_reach_python():
    L = ep.lib()
    x = torch.zeros((4, 32), dtype=torch.int8, device="cuda")
    f = torch.zeros(4, device="cuda")
    y = torch.zeros((4, 4), device="cuda")
    p = lambda t, o=0: C.c_void_p(t.data_ptr() + o)
    st = C.c_void_p(0)
    assert L.ep_gemm_int8(p(x), p(f), p(x, 4), p(f), 4, 3, 16, None, ep.F32, p(y), st) == -1     # W misaligned
    assert L.ep_gemm_int8(p(x), p(f), p(x), p(f), 4, 4, 32, None, ep.F32, p(y, 2), st) == -1     # Y misaligned
    assert L.ep_quantize_rows_int8(p(f, 2), ep.F32, 1, 1, 1, p(x), p(f), st) == -1
