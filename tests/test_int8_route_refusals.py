"""Refusals of the INT8 products and the expert routing, on the CPU: arguments are checked before any
device work, in the binding for tensors and in the C ABI for sizes, so no GPU is needed. And the
arithmetic of the fused INT8 forward's rounding, over every coordinate and divisor."""
import ctypes as C

import numpy as np
import pytest
import torch

import decode_tile_interleaved_rans_amd as ep

P = C.c_void_p(1 << 20)               # an aligned address that no call here may reach
ODD = C.c_void_p((1 << 20) + 1)
N0 = None
EINVAL, EUNSUPPORTED, ERANGE = -1, -3, -4
I31 = 2 ** 31


@pytest.mark.parametrize("rc,args", [
    (EINVAL, (P, ep.BF16, -1, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 1, -8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 2, 8, 7, P, P)),            # rows overlap
    (EINVAL, (N0, ep.BF16, 1, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 1, 8, 8, N0, P)),
    (EINVAL, (P, ep.BF16, 1, 8, 8, P, N0)),
    (EINVAL, (ODD, ep.BF16, 1, 8, 8, P, P)),
    (EUNSUPPORTED, (P, ep.I8, 1, 8, 8, P, P)),
    (EUNSUPPORTED, (P, 77, 1, 8, 8, P, P)),
    (ERANGE, (P, ep.BF16, I31, 8, 8, P, P)),
    (ERANGE, (P, ep.BF16, 1, I31, I31, P, P)),
    (ERANGE, (P, ep.BF16, 2 ** 30, 8, 2 ** 40, P, P)),
    (0, (N0, ep.BF16, 0, 8, 8, N0, N0)),
])
def test_quantizer(rc, args):
    assert ep.lib().ep_quantize_rows_int8(*args, None) == rc


@pytest.mark.parametrize("rc,M,N,K,out,xq,wq,y", [
    (EINVAL, -1, 4, 16, ep.BF16, P, P, P),
    (EINVAL, 4, 4, 24, ep.BF16, P, P, P),
    (EINVAL, 4, 4, 16, ep.BF16, ODD, P, P),
    (EINVAL, 4, 4, 16, ep.BF16, P, ODD, P),
    (EINVAL, 4, 4, 16, ep.BF16, P, P, ODD),
    (EINVAL, 4, 4, 16, ep.BF16, N0, P, P),
    (EINVAL, 4, 4, 16, ep.BF16, P, P, N0),
    (EUNSUPPORTED, 4, 4, 16, ep.I8, P, P, P),
    (ERANGE, 4, 4, 131072, ep.BF16, P, P, P),          # the sums could leave int32
    (ERANGE, I31, 4, 16, ep.BF16, P, P, P),
    (ERANGE, 4, I31, 16, ep.BF16, P, P, P),
    (ERANGE, I31 - 1, I31 - 1, 16, ep.BF16, P, P, P),
    (0, 0, 4, 16, ep.BF16, N0, N0, N0),
    (0, 4, 0, 16, ep.BF16, N0, N0, N0),
])
def test_products(rc, M, N, K, out, xq, wq, y):
    assert ep.lib().ep_gemm_int8(xq, P, wq, P, M, N, K, None, out, y, None) == rc
    assert ep.lib().ep_gemm_int8_experts(xq, P, wq, P, P, 4, M, N, K, None, out, y, None) == rc


def test_experts():
    f = ep.lib().ep_gemm_int8_experts
    for E in (0, -1, 1025):
        assert f(P, P, P, P, P, E, 4, 4, 16, None, ep.BF16, P, None) == ERANGE
    assert f(P, P, P, P, None, 4, 4, 4, 16, None, ep.BF16, P, None) == EINVAL
    assert b"offsets" in ep.lib().ep_last_error()


def test_layout():
    f = ep.lib().ep_pad_rows_int8
    assert f(P, 4, 20, P, 31, None) == EINVAL and f(P, 4, 20, P, 16, None) == EINVAL
    assert f(P, 4, 20, ODD, 32, None) == EINVAL and f(None, 4, 20, P, 32, None) == EINVAL
    assert f(P, -4, 20, P, 32, None) == EINVAL and f(P, 4, I31, P, I31, None) == ERANGE
    assert f(P, 2 ** 36, 16, P, 16, None) == ERANGE and f(None, 0, 20, None, 32, None) == 0


def test_sort():
    f, n = ep.lib().ep_sort_tokens, C.c_size_t()
    call = lambda T=4, H=8, ldx=8, ids=P, ib=8, k=2, E=4, rows=P, off=P, pos=P, scr=P, dt=ep.BF16, x=P: \
        f(x, dt, T, H, ldx, ids, ib, k, E, rows, off, pos, scr, None)
    assert call(T=-1) == EINVAL and call(k=-1) == EINVAL and call(H=-1) == EINVAL and call(ldx=7) == EINVAL
    assert call(ib=2) == EINVAL and call(ids=None) == EINVAL and call(off=None) == EINVAL and call(pos=None) == EINVAL
    assert call(x=None) == EINVAL and call(x=ODD) == EINVAL and call(rows=ODD) == EINVAL
    assert call(T=4096, scr=None) == EINVAL                  # more than one block of choices needs scratch
    assert call(E=0) == ERANGE and call(E=1025) == ERANGE and call(T=2 ** 30, k=2) == ERANGE
    assert call(H=2 ** 62, ldx=2 ** 62) == ERANGE and call(dt=9) == EUNSUPPORTED
    s = ep.lib().ep_sort_tokens_scratch
    assert s(4, 2, 4, None) == EINVAL and s(4, 2, 0, C.byref(n)) == ERANGE
    assert s(512, 2, 4, C.byref(n)) == 0 and n.value == 0
    assert s(513, 2, 4, C.byref(n)) == 0 and n.value >= 5 * 4


def test_combine():
    f, g = ep.lib().ep_combine_tokens, ep.lib().ep_combine_tokens_grad
    fw = lambda ys=P, dt=ep.BF16, pos=P, T=4, k=2, H=8, R=8, y=P: f(ys, dt, pos, P, T, k, H, R, y, None)
    bw = lambda ys=P, dt=ep.BF16, pos=P, dy=P, T=4, k=2, H=8, R=8, d=P, dw=P: g(ys, dt, pos, P, dy, T, k, H, R, d, dw, None)
    for call in (fw, bw):
        assert call(T=-1) == EINVAL and call(k=-1) == EINVAL and call(H=-1) == EINVAL and call(R=-1) == EINVAL
        assert call(pos=None) == EINVAL and call(ys=None) == EINVAL and call(ys=ODD) == EINVAL
        assert call(dt=ep.I8) == EUNSUPPORTED and call(R=I31) == ERANGE and call(T=2 ** 30) == ERANGE
        assert call(H=2 ** 61) == ERANGE
    assert fw(y=None) == EINVAL and bw(dy=None) == EINVAL
    assert bw(R=9) == EINVAL                                  # one row per choice
    assert fw(T=0, R=0, ys=None, y=None, pos=None) == 0


def test_compressed_experts():
    f = ep.lib().ep_linear_forward_experts
    hs, off = (C.c_void_p * 2)(), (C.c_int64 * 3)(0, 1, 2)
    for n in (0, -1, 1025):
        assert f(hs, n, ep.BF16, P, off, P, None, P, None) == ERANGE
    assert f(hs, 2, ep.F16, P, off, P, None, P, None) == EUNSUPPORTED
    assert f(hs, 2, ep.BF16, P, off, P, None, P, None) == EINVAL and b"null handle" in ep.lib().ep_last_error()
    assert f(None, 2, ep.BF16, P, off, P, None, P, None) == EINVAL
    assert f(hs, 2, ep.BF16, P, None, P, None, P, None) == EINVAL
    assert ep.lib().ep_linear_forward_int8(None, P, 1, None, P, None) == EINVAL
    many = ep.lib().ep_linear_forward_int8_many
    for n in (-1, 33):
        assert many(hs, n, P, 4, None, hs, None) == ERANGE
    assert many(None, 2, P, 4, None, hs, None) == EINVAL and many(hs, 2, P, 4, None, None, None) == EINVAL
    assert many(hs, 2, P, 4, None, hs, None) == EINVAL and b"null handle" in ep.lib().ep_last_error()
    assert many(None, 0, None, 4, None, None, None) == 0
    with pytest.raises(ValueError, match="at least one"):
        ep.linear_forward_experts([], torch.zeros(1), torch.zeros(1))


def test_binding_refuses_tensors():
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
    f32 = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError, match="GPU"):
        ep.quantize_rows_int8(torch.zeros((2, 8), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="matrix"):
        ep.quantize_rows_int8(torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="GPU"):
        ep.gemm_int8(i8(2, 16), f32(2), i8(3, 16), f32(3))
    with pytest.raises(ValueError, match="out_dtype"):
        ep.gemm_int8(i8(2, 16), f32(2), i8(3, 16), f32(3), out_dtype=torch.int8)
    with pytest.raises(ValueError, match="experts"):
        ep.gemm_int8_experts(i8(2, 16), f32(2), i8(3, 16), f32(3), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        ep.pad_rows_int8(i8(2, 5))
    with pytest.raises(ValueError, match="int32 or int64"):
        ep.sort_tokens(f32(2, 8), f32(2, 1), 4)
    with pytest.raises(ValueError, match="GPU"):
        ep.sort_tokens(f32(2, 8), torch.zeros((2, 1), dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="matrix"):
        ep.combine_tokens(i8(2, 8), torch.zeros((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        ep.combine_tokens(f32(2, 8), torch.zeros((2, 1), dtype=torch.int32))
    with pytest.raises(ValueError, match="int8"):
        ep.CompressedLinear(b"", compute="int4")


def test_fused_int8_rounding_formula():
    """round-half-away(q / k) as trunc(fma(q, fp32(1 / k), 1/2 + fp32(1 / k) / 4)), for every |q| <= 127 k and every
    divisor up to the largest a coordinate needs. fp64 holds the product (39 bits) and the sum exactly, so
    its rounding to fp32 is the fused multiply-add's."""
    for k in range(1, 259):
        q = np.arange(0, min(127 * k, 32767) + 1, dtype=np.int64)
        inv = np.float32(1.0) / np.float32(k)
        half = np.float32(np.float64(np.float32(0.25) * inv) + 0.5)
        t = (q.astype(np.float64) * np.float64(inv) + np.float64(half)).astype(np.float32)
        assert np.array_equal(np.trunc(t).astype(np.int64), (2 * q + k) // (2 * k)), k


def test_routing_refuses_forward_mode():
    """A dual tensor does not require a gradient, so nothing else would tell that its tangent is lost."""
    fw = torch.autograd.forward_ad
    x, ids, pos = torch.randn(4, 8), torch.zeros((4, 1), dtype=torch.int64), torch.zeros((4, 1), dtype=torch.int32)
    with fw.dual_level():
        dual = fw.make_dual(x, torch.ones_like(x))
        weights = fw.make_dual(torch.ones(4, 1), torch.ones(4, 1))
        assert not dual.requires_grad
        for call in (lambda: ep.sort_tokens(dual, ids, 4), lambda: ep.combine_tokens(dual, pos),
                     lambda: ep.combine_tokens(x, pos, weights)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
    with pytest.raises(ValueError, match="forward-mode"):
        torch.func.jvp(lambda v: ep.sort_tokens(v, ids, 4)[0], (x,), (x,))
    # the gradients of the rows and of the sums, which may be dual where their inputs were not
    sort, combine = ep._routing_functions()

    class Saved:
        saved_tensors = (None, pos, None)

    with fw.dual_level():
        for f in (sort, combine):
            with pytest.raises(ValueError, match="forward-mode"):
                Saved.saved_tensors = (pos,) if f is sort else (None, pos, None)
                f.backward(Saved, fw.make_dual(x, x))


@pytest.mark.parametrize("K", [131057, 131071, 131072, I31])
def test_widths_past_the_exact_sums(K):
    L = ep.lib()
    assert L.ep_gemm_int8(P, P, P, P, 4, 4, K, None, ep.BF16, P, None) == ERANGE and b"131056" in L.ep_last_error()
    assert L.ep_gemm_int8_experts(P, P, P, P, P, 2, 4, 4, K, None, ep.BF16, P, None) == ERANGE
