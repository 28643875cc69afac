"""Refusals of the MXFP4 operators on the CPU: sizes in the C ABI, tensors in the binding, before any device work."""
import ctypes as C

import pytest
import torch

import decode_tile_interleaved_rans_amd as ep
import mx_reference as mx

P = C.c_void_p(1 << 20)               # an aligned address that no call here may reach
OFF4 = C.c_void_p((1 << 20) + 4)
ODD = C.c_void_p((1 << 20) + 1)
N0 = None
EINVAL, EUNSUPPORTED, ERANGE = -1, -3, -4


@pytest.mark.parametrize("rc,args", [
    (EINVAL, (P, ep.BF16, -1, 1, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, -1, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, 4, -8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, 3, 8, 8, P, P)),          # not whole matrices
    (EINVAL, (P, ep.BF16, 4, 0, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, 4, 8, 7, P, P)),          # rows overlap
    (EINVAL, (N0, ep.BF16, 4, 4, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, 4, 8, 8, N0, P)),
    (EINVAL, (P, ep.BF16, 4, 4, 8, 8, P, N0)),
    (EINVAL, (ODD, ep.BF16, 4, 4, 8, 8, P, P)),
    (EINVAL, (P, ep.BF16, 4, 4, 8, 8, ODD, P)),
    (EINVAL, (P, ep.BF16, 4, 4, 8, 8, P, ODD)),
    (EUNSUPPORTED, (P, ep.I8, 4, 4, 8, 8, P, P)),
    (EUNSUPPORTED, (P, 77, 4, 4, 8, 8, P, P)),
    (ERANGE, (P, ep.BF16, 4, 4, 2 ** 22 + 1, 2 ** 22 + 1, P, P)),
    (ERANGE, (P, ep.BF16, 2 ** 28, 2 ** 28, 8, 8, P, P)),
    (ERANGE, (P, ep.BF16, 2 ** 40, 1, 8, 8, P, P)),
    (ERANGE, (P, ep.BF16, 2 ** 30, 2 ** 20, 8, 2 ** 40, P, P)),
    (0, (N0, ep.BF16, 0, 0, 8, 8, N0, N0)),
    (0, (N0, ep.BF16, 4, 4, 0, 0, N0, N0)),
])
def test_quantizer(rc, args):
    assert ep.lib().ep_quantize_rows_mxfp4(*args, None) == rc


@pytest.mark.parametrize("rc,args", [
    (EINVAL, (P, P, -1, 1, 128, 8, ep.BF16, P)),
    (EINVAL, (P, P, 4, 4, 100, 8, ep.BF16, P)),
    (EINVAL, (P, P, 4, 4, 128, 129, ep.BF16, P)),
    (EINVAL, (P, P, 4, 4, 128, -1, ep.BF16, P)),
    (EINVAL, (P, P, 4, 3, 128, 8, ep.BF16, P)),
    (EINVAL, (N0, P, 4, 4, 128, 8, ep.BF16, P)),
    (EINVAL, (P, N0, 4, 4, 128, 8, ep.BF16, P)),
    (EINVAL, (P, P, 4, 4, 128, 8, ep.BF16, N0)),
    (EINVAL, (P, P, 4, 4, 128, 8, ep.BF16, ODD)),
    (EINVAL, (ODD, P, 4, 4, 128, 8, ep.BF16, P)),
    (EINVAL, (P, ODD, 4, 4, 128, 8, ep.BF16, P)),
    (EUNSUPPORTED, (P, P, 4, 4, 128, 8, ep.F8E4M3, P)),
    (ERANGE, (P, P, 4, 4, 2 ** 22 + 128, 8, ep.BF16, P)),
    (0, (N0, N0, 0, 0, 128, 8, ep.BF16, N0)),
    (0, (P, P, 4, 4, 128, 0, ep.BF16, N0)),
])
def test_inverse(rc, args):
    assert ep.lib().ep_dequantize_rows_mxfp4(*args, None) == rc


@pytest.mark.parametrize("rc,M,N,K,out,xq,xs,wq,ws,y", [
    (EINVAL, -1, 4, 128, ep.BF16, P, P, P, P, P),
    (EINVAL, 4, 4, 64, ep.BF16, P, P, P, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, OFF4, P, P, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, ODD, P, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, P, OFF4, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, P, P, ODD, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, P, P, P, ODD),
    (EINVAL, 4, 4, 128, ep.BF16, N0, P, P, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, N0, P, P, P),
    (EINVAL, 4, 4, 128, ep.BF16, P, P, P, P, N0),
    (EUNSUPPORTED, 4, 4, 128, ep.I8, P, P, P, P, P),
    (ERANGE, 4, 4, 2 ** 22 + 128, ep.BF16, P, P, P, P, P),
    (ERANGE, 2 ** 27 + 1, 4, 128, ep.BF16, P, P, P, P, P),
    (ERANGE, 4, 2 ** 27 + 1, 128, ep.BF16, P, P, P, P, P),
    (ERANGE, 2 ** 27, 2 ** 27, 128, ep.BF16, P, P, P, P, P),
    (0, 0, 4, 128, ep.BF16, N0, N0, N0, N0, N0),
    (0, 4, 0, 128, ep.BF16, N0, N0, N0, N0, N0),
])
def test_products(rc, M, N, K, out, xq, xs, wq, ws, y):
    assert ep.lib().ep_gemm_mxfp4(xq, xs, wq, ws, M, N, K, None, out, y, None) == rc
    assert ep.lib().ep_gemm_mxfp4_experts(xq, xs, wq, ws, P, 4, M, N, K, None, out, y, None) == rc


def test_experts():
    f = ep.lib().ep_gemm_mxfp4_experts
    for E in (0, -1, 1025):
        assert f(P, P, P, P, P, E, 4, 4, 128, None, ep.BF16, P, None) == ERANGE
    assert f(P, P, P, P, None, 4, 4, 4, 128, None, ep.BF16, P, None) == EINVAL
    assert b"offsets" in ep.lib().ep_last_error()


def test_tensors_on_the_host():
    with pytest.raises(ValueError):
        ep.quantize_rows_mxfp4(torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        ep.quantize_rows_mxfp4(torch.zeros((2, 4, 64)))
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ep.dequantize_rows_mxfp4(u8(4, 64), u8(1, 4, 4))
    with pytest.raises(ValueError):
        ep.gemm_mxfp4(u8(4, 64), u8(1, 4, 4), u8(4, 64), u8(1, 4, 4))


def test_the_reference_itself():
    """The definition's codes are the nearest values of the grid: no other code is nearer, and scales put the
    largest magnitude of a block into [4, 8) units."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn((6, 300), generator=g) * torch.exp(3 * torch.randn((6, 1), generator=g))
    q, s = mx.quantize(x)
    v = mx.values(q, s)
    full = torch.nn.functional.pad(x.double(), (0, 84))
    unit = torch.exp2(s.transpose(0, 1).reshape(6, -1).double() - 127).repeat_interleave(32, 1)
    all_off = ((full.abs() / unit)[..., None].clamp_max(6.0) - mx.GRID).abs().amin(-1)
    assert torch.equal(((full - v).abs() / unit).where((full / unit).abs() <= 6, all_off), all_off)
    top = (full.abs() / unit).reshape(6, -1, 32).amax(-1)
    assert ((top[:, :9] >= 4) & (top[:, :9] < 8)).all()


def test_expert_layer():
    f, n = ep.lib().ep_mlp_forward_experts, C.c_size_t()

    def call(x=P, act=ep.BF16, T=4, H=64, ldx=64, ids=P, ib=8, k=2, E=3, w=P, win=P, si=None, bi=None, wout=P, so=None, bo=None, I=32, N=16,
             scr=P, y=P):
        return f(x, act, T, H, ldx, ids, ib, k, E, w, win, si, bi, wout, so, bo, I, N, scr, y, None)

    assert call(act=ep.F32) == EUNSUPPORTED and call(act=99) == EUNSUPPORTED
    for c in (dict(T=-1), dict(k=-1), dict(H=-1), dict(I=-1), dict(N=-1), dict(ldx=63), dict(ib=2), dict(ids=None), dict(x=None), dict(y=None),
              dict(win=None), dict(wout=None), dict(scr=None), dict(scr=OFF4), dict(x=ODD), dict(y=ODD), dict(win=ODD), dict(wout=ODD),
              dict(ids=OFF4), dict(si=P), dict(so=P), dict(si=P, so=P, win=OFF4), dict(si=P, so=P, wout=OFF4), dict(si=ODD, so=P)):
        assert call(**c) == EINVAL, c
    for c in (dict(T=65), dict(T=64, k=17), dict(E=0), dict(E=1025), dict(H=2 ** 20 + 1, ldx=2 ** 21), dict(I=2 ** 20 + 1), dict(N=2 ** 20 + 1),
              dict(ldx=2 ** 62)):
        assert call(**c) == ERANGE, c
    assert call(T=0, x=None, ids=None, y=None, scr=None) == 0 and call(N=0, y=None) == 0
    s = ep.lib().ep_mlp_forward_experts_scratch
    assert s(4, 2, 3, 32, 16, 0, None) == EINVAL and s(65, 1, 3, 32, 16, 0, C.byref(n)) == ERANGE and s(-1, 1, 3, 32, 16, 0, C.byref(n)) == EINVAL
    assert s(4, 2, 3, 2 ** 20 + 1, 16, 0, C.byref(n)) == ERANGE and s(4, 2, 0, 32, 16, 1, C.byref(n)) == ERANGE
    assert s(4, 2, 3, 130, 16, 1, C.byref(n)) == 0 and n.value >= 8 * 256 * 2
    for T, k, I in ((0, 2, 130), (4, 0, 130), (4, 2, 0)):
        assert s(T, k, 3, I, 16, 0, C.byref(n)) == 0 and n.value == 0


def test_expert_layer_tensors_on_the_host():
    t = torch.zeros
    with pytest.raises(ValueError):
        ep.mlp_forward_experts(t((4, 64), dtype=torch.bfloat16), t((4, 2), dtype=torch.int64), None, t((3, 64, 64), dtype=torch.bfloat16),
                               t((3, 16, 32), dtype=torch.bfloat16))


def test_gradients_are_refused():
    """The quantizer and the products have no gradient: inputs that ask for one are refused, not dropped, before any other check."""
    asks = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, requires_grad=True)
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    gemm = (u8(4, 64), u8(1, 4, 4), u8(6, 64), u8(1, 6, 4))
    experts = (u8(4, 64), u8(1, 4, 4), u8(2, 6, 64), u8(2, 1, 6, 4), torch.zeros(3, dtype=torch.int32))
    calls = [lambda: ep.quantize_rows_mxfp4(asks(4, 64)), lambda: ep.quantize_rows_mxfp4(asks(2, 4, 64)),
             lambda: ep.gemm_mxfp4(*gemm, asks(6, dtype=torch.bfloat16)), lambda: ep.gemm_mxfp4_experts(*experts, asks(2, 6, dtype=torch.bfloat16))]
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):       # without gradients the next check speaks
            call()


def test_tangents_are_refused():
    """The expert layer has no derivative of either mode: its message does not send to the other."""
    import torch.autograd.forward_ad as fwd
    t = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    with fwd.dual_level():
        with pytest.raises(ValueError, match="derivative") as e:
            ep.mlp_forward_experts(fwd.make_dual(t(4, 64), t(4, 64)), torch.zeros((4, 2), dtype=torch.int64), None, t(3, 64, 64), t(3, 16, 32))
        assert "reverse" not in str(e.value)


def test_tangents_of_rows_and_biases_are_refused():
    import torch.autograd.forward_ad as fwd
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    with fwd.dual_level():
        dual = lambda *shape: fwd.make_dual(torch.zeros(shape, dtype=torch.bfloat16), torch.ones(shape, dtype=torch.bfloat16))
        for call in (lambda: ep.quantize_rows_mxfp4(dual(4, 64)), lambda: ep.gemm_mxfp4(u8(4, 64), u8(1, 4, 4), u8(6, 64), u8(1, 6, 4), dual(6))):
            with pytest.raises(ValueError, match="no derivative"):
                call()


def test_relative_error_of_normal_values():
    """What the format costs: products of random normal rows in MXFP4 are 16% off (relative, L2), in INT8 with a scale per row below
    2%. 2 x 65536 values and more make the figure, so that it varies by far less than the 1% between the bounds."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((100, 2048), generator=g), torch.randn((120, 2048), generator=g)
    int8 = lambda t: ((t / t.abs().amax(1, keepdim=True) * 127).round() * t.abs().amax(1, keepdim=True) / 127).double()
    want = x.double() @ w.double().T
    off = lambda a, b: ((a @ b.T - want).norm() / want.norm()).item()
    assert 0.155 < off(mx.values(*mx.quantize(x)), mx.values(*mx.quantize(w))) < 0.165 and off(int8(x), int8(w)) < 0.02
