"""Mixture-of-experts layers of compressed experts (linear_forward_experts, ep_linear_forward_experts): every
row must have the bits of its expert's own forward, whether the expert shared a fused launch (up to 64
rows in the row layout) or ran its own; the sums over a token's experts are checked in 64 bits, where fp32
steps (k fused multiply-adds of 2^-24) and the BF16 rounding (half of finfo.eps) are allowed."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
import decode_tile_interleaved_rans_amd as ep
from decode_tile_interleaved_rans_amd import workloads as W

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def experts(E, N, K, compute, layout=lambda e: ep.ROW_LAYOUT, bits=lambda e: 11, target=4.5, bias=True):
    out = []
    for e in range(E):
        s, _ = ep.compress(W.student_t(N, K, 100 + e), target, dtype=ep.BF16, layout=layout(e), prob_bits=bits(e))
        b = torch.randn(N, generator=gen(e), device="cuda").to(torch.bfloat16) if bias and e % 3 else None
        out.append(ep.CompressedLinear(s, b, compute))
    return out


def tokens(T, K, seed):
    return torch.from_numpy(W.activations(T, K, seed).view(np.int16)).view(torch.bfloat16).cuda()


def check(layers, x, ids, w):
    y = ep.linear_forward_experts(layers, x, ids, w)
    rows, off, pos = ep.sort_tokens(x, ids, len(layers))
    off = off.tolist()
    own = torch.zeros((rows.shape[0], layers[0].out_features), dtype=torch.bfloat16, device="cuda")
    for e, l in enumerate(layers):
        if off[e + 1] > off[e]:
            own[off[e]:off[e + 1]] = l(rows[off[e]:off[e + 1]])
    for l in layers:
        l.handle.check()
    assert torch.equal(y, ep.combine_tokens(own, pos, w))      # the same rows, bit for bit
    p = pos.long()
    w64 = torch.ones(p.shape, dtype=torch.float64, device="cuda") if w is None else w.double()
    part = torch.where((p >= 0)[..., None], w64[..., None] * own.double()[p.clamp_min(0)], 0.0)
    ref, mag = part.sum(1), part.abs().sum(1)
    fp32 = p.shape[1] * U * mag
    tol = fp32 + torch.finfo(torch.bfloat16).eps / 2 * (ref.abs() + fp32) + 2.0 ** -134
    assert ((y.double() - ref).abs() <= tol).all()
    return y


@pytest.mark.parametrize("compute", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("T", [0, 1, 5, 40, 300])
def test_experts_of_one_layer(T, compute):
    E, k, N, K = 6, 2, 200, 1040
    layers = experts(E, N, K, compute)
    ids = torch.randint(0, E, (T, k), generator=gen(T), device="cuda")
    if T > 4:
        ids[3] = -1                                           # a token without experts
        ids[:, 1] = torch.where(ids[:, 1] == 2, 7, ids[:, 1])  # an expert that the second choice drops
    w = torch.rand((T, k), generator=gen(T + 1), device="cuda")
    y = check(layers, tokens(T, K, T), ids, w)
    if T > 4:
        assert not y[3].any()
    check(layers, tokens(T, K, T), ids.to(torch.int32), None)


@pytest.mark.parametrize("compute", ["bf16", "fp8", "int8"])
def test_mixed_layouts_precisions_and_group_sizes(compute):
    # more experts than one launch takes, two probability precisions, some in layout 0, one with more
    # than 64 rows, some without any
    E, N, K, T = 70, 48, 528, 200
    layers = experts(E, N, K, compute, layout=lambda e: 0 if e % 9 == 4 else ep.ROW_LAYOUT, bits=lambda e: 10 + e % 2)
    ids = torch.randint(0, E, (T, 3), generator=gen(5), device="cuda")
    ids[:90, 0] = 7
    ids = torch.where(ids == 20, -1, ids)
    check(layers, tokens(T, K, 3), ids, torch.rand((T, 3), generator=gen(6), device="cuda"))


@pytest.mark.parametrize("compute", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("N,K", [(200, 1040), (201, 528), (512, 8192)])    # the last: up to 255 rows the own kernel
def test_experts_of_many_rows(N, K, compute):
    E, T = 40, 3000
    layers = experts(E, N, K, compute, layout=lambda e: e % 2)
    ids = torch.randint(0, E, (T, 2), generator=gen(5), device="cuda")
    ids[:400, 0] = 11
    ids = torch.where((ids == 20) | (ids == 3), -1, ids)
    check(layers, tokens(T, K, 3), ids, torch.rand((T, 2), generator=gen(6), device="cuda"))


def test_row_counts_beyond_the_plan_cache():
    # more distinct row counts than hipBLASLt plans are kept: the first one again gives the same bits
    N, K = 128, 128
    wq, ws = ep.quantize_rows_fp8(torch.randn((N, K), generator=gen(1), device="cuda").to(torch.bfloat16))
    xq, xs = ep.quantize_rows_fp8(torch.randn((1650, K), generator=gen(2), device="cuda").to(torch.bfloat16))
    x64, w64 = (q.view(torch.float8_e4m3fn).float().double() * s[:, None].double() for q, s in ((xq, xs), (wq, ws)))
    first = ep.gemm_fp8(xq[:600], xs[:600], wq, ws)
    for M in range(600, 1650):
        y = ep.gemm_fp8(xq[:M], xs[:M], wq, ws)
        if M % 150 == 0:
            want, room = x64[:M] @ w64.T, x64[:M].abs() @ w64.T.abs()
            # bf16 output: 2^-8 of the value; fp32 sums of 128 products: 2^-16 of the sum of magnitudes
            assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * room).all()
    assert torch.equal(ep.gemm_fp8(xq[:600], xs[:600], wq, ws), first)


def test_int8_experts_beyond_one_chunk():
    # 256 MiB of codes per expert, 256 MiB at a time: three experts in a chunk each, one without rows
    N, K, T = 16384, 16384, 150
    s, _ = ep.compress_device(W.gpu_student_t(N, K, 3), 3.0, layout=ep.ROW_LAYOUT, prob_bits=11)
    layers = [ep.CompressedLinear(s, None, "int8") for _ in range(4)]
    layers[3].bias = torch.randn(N, generator=gen(1), device="cuda").to(torch.bfloat16)
    ids = torch.tensor([0, 1, 3], device="cuda")[torch.arange(T, device="cuda") % 3][:, None]
    ids[:70] = 1
    check(layers, tokens(T, K, 4), ids, None)


def test_int8_chunks_of_several_experts():
    # 4 MiB of codes per expert, 64 experts to a chunk: three chunks, in each some experts without rows, some with
    # a bias, one of many rows in the last
    E, N, K, T = 150, 2048, 2048, 600
    streams = [ep.compress_device(W.gpu_student_t(N, K, 3 + i), 3.0, layout=i % 2, prob_bits=11)[0] for i in range(3)]
    layers = [ep.CompressedLinear(streams[e % 3], None, "int8") for e in range(E)]
    for e in range(0, E, 7):
        layers[e].bias = torch.randn(N, generator=gen(e), device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, 2), generator=gen(5), device="cuda")
    ids = torch.where((ids % 11 == 3) | ((ids >= 60) & (ids < 70)), -1, ids)
    ids[:90, 0] = 140
    check(layers, tokens(T, K, 3), ids, torch.rand((T, 2), generator=gen(6), device="cuda"))


def test_int8_chunks_take_the_tile_of_their_own_rows():
    # three chunks of 64 experts with 8 rows each: the same product of every chunk, so the same kernel on the same
    # grid, whatever the chunks before it held
    E, N, K = 192, 2048, 2048
    s, _ = ep.compress_device(W.gpu_student_t(N, K, 3), 3.0, layout=0, prob_bits=11)
    layers = [ep.CompressedLinear(s, None, "int8")] * E
    x = tokens(8 * E, K, 4)
    ids = torch.arange(8 * E, device="cuda")[:, None] % E
    want = layers[0](x)
    ep.linear_forward_experts(layers, x, ids)                  # the workspace
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        y = ep.linear_forward_experts(layers, x, ids)
        torch.cuda.synchronize()
    assert torch.equal(y, want)
    kernels = [e.name for e in prof.events()]
    if not any("quantize_rows_i8" in n for n in kernels):
        pytest.skip("the profiler records no kernels here")
    products = [n for n in kernels if "gemm_i8" in n]
    assert len(products) == 3 and len(set(products)) == 1, products


def test_wide_values_divide_in_int8():
    # rows whose largest |q| passes 127 (large targets): the INT8 container divides them
    E, N, K = 2, 64, 1024
    layers = experts(E, N, K, "int8", target=9.0)
    x = tokens(20, K, 9)
    ids = torch.arange(20, device="cuda")[:, None] % E
    check(layers, x, ids, None)
    cq, cs = oracle.decompress(layers[0].stream, oracle.I8)
    alone = layers[1]
    dq, ds = alone.handle.decompress(torch.int8)
    q, s = ep.quantize_rows_int8(x)
    assert torch.equal(alone(x), ep.gemm_int8(q, s, dq, ds, alone.bias))
    assert (cs > 0).all() and np.abs(cq.view(np.int8)).max() > 64
    # many divisors: rows of growing outliers, against the decode kernel's integer rounding
    w = W.student_t(400, 512, 77).astype(np.uint16)
    f = W.bf16_bits_to_f32(w).copy()
    f[:, 7] *= np.linspace(1.0, 400.0, 400)
    st, _ = ep.compress(f.astype(np.float32), 9.0, layout=ep.ROW_LAYOUT, prob_bits=11)
    lay = ep.CompressedLinear(st, compute="int8")
    dq, ds = lay.handle.decompress(torch.int8)
    eye = torch.eye(512, device="cuda").to(torch.bfloat16)     # unit rows: the products are the codes themselves
    for r0 in range(0, 512, 64):
        q, sc = ep.quantize_rows_int8(eye[r0:r0 + 64])
        assert torch.equal(lay(eye[r0:r0 + 64]), ep.gemm_int8(q, sc, dq, ds))
    qs = lay.handle.decode_symbols().abs().amax(1).int()
    assert len(((qs + 126) // 127).unique()) > 30              # the case covers what it is for


def test_router_gradient():
    E, k, N, K, T = 4, 2, 96, 512, 30
    layers = experts(E, N, K, "int8")
    x = tokens(T, K, 2)
    ids = torch.randint(0, E, (T, k), generator=gen(1), device="cuda")
    w = torch.rand((T, k), generator=gen(2), device="cuda").requires_grad_(True)
    y = ep.linear_forward_experts(layers, x, ids, w)
    dy = torch.randn((T, N), generator=gen(3), device="cuda").to(torch.bfloat16)
    (dw,) = torch.autograd.grad(y, w, dy)
    own = torch.stack([torch.stack([layers[int(e)](x[t:t + 1])[0] for e in ids[t]]) for t in range(T)]).double()
    prod = own * dy.double()[:, None, :]
    assert ((dw.double() - prod.sum(2)).abs() <= (N + 8) * U * prod.abs().sum(2)).all()
    with pytest.raises(ValueError, match="detach"):
        ep.linear_forward_experts(layers, x.clone().requires_grad_(True), ids, w)


def test_other_stream():
    layers = experts(3, 64, 512, "int8")
    x, ids = tokens(50, 512, 4), torch.randint(0, 3, (50, 2), generator=gen(4), device="cuda")
    want = ep.linear_forward_experts(layers, x, ids)
    s = torch.cuda.Stream()
    got = ep.linear_forward_experts(layers, x + 0, ids + 0, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    a, b = experts(1, 32, 512, "int8")[0], experts(1, 32, 256, "int8")[0]
    x, ids = tokens(4, 512, 1), torch.zeros((4, 1), dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="share"):
        ep.linear_forward_experts([a, b], x, ids)
    with pytest.raises(ValueError, match="share"):
        ep.linear_forward_experts([a, ep.CompressedLinear(a.stream)], x, ids)
    with pytest.raises(ValueError, match="bfloat16"):
        ep.linear_forward_experts([a], x.float(), ids)
    L, st = ep.lib(), C.c_void_p(torch.cuda.current_stream().cuda_stream)
    hs = (C.c_void_p * 2)(a.handle.ptr.value, a.handle.ptr.value)
    y = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    f = lambda offs, h=hs, px=x.data_ptr(), d=torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"): \
        L.ep_linear_forward_experts(h, 2, ep.I8, px, (C.c_int64 * 3)(*offs), None if d is None else d.data_ptr(), None,
                                    y.data_ptr(), st)
    assert f([0, 3, 2]) == -1 and f([1, 2, 3]) == -1 and f([0, 1, 2 ** 31]) == -4
    assert f([0, 1, 2], px=x.data_ptr() + 2) == -1
    assert f([0, 1, 2], h=(C.c_void_p * 2)(a.handle.ptr.value, b.handle.ptr.value)) == -1
    assert f([0, 2, 4], d=None) == -1
    assert f([0, 0, 0]) == 0 and f([0, 2, 4]) == 0
