"""The expert layer for few tokens on the GPU, against its formula in 64 bits."""
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import decode_tile_interleaved_rans_amd as ep
import mx_reference as mx

pytestmark = pytest.mark.gpu


class Layer:
    """A layer's inputs on the CPU, made from a seed, and its definition."""

    def __init__(self, T, k, E, H, I, N, dtype=torch.bfloat16, mxfp4=False, bias=False, seed=0, ids=None):
        g = torch.Generator().manual_seed(seed + 7 * T + H)
        self.k, self.E, self.I, self.dtype = k, E, I, dtype
        self.x = torch.randn((T, H), generator=g).to(dtype)
        self.ids = ids if ids is not None else torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
        self.w = torch.rand((T, self.ids.shape[1]), generator=g)
        win, wout = torch.randn((E, 2 * I, H), generator=g) / max(1, H) ** 0.5, torch.randn((E, N, I), generator=g) / max(1, I) ** 0.5
        self.scales = (None, None)
        if mxfp4:
            (self.win, s1), (self.wout, s2) = mx.quantize(win), mx.quantize(wout)
            self.scales = (s1, s2)
            self.v_in, self.v_out = mx.values(self.win, s1)[..., :H], mx.values(self.wout, s2)[..., :I]
        else:
            self.win, self.wout = win.to(dtype), wout.to(dtype)
            self.v_in, self.v_out = self.win.double(), self.wout.double()
        self.b_in = torch.randn((E, 2 * I), generator=g).to(torch.bfloat16) if bias else None
        self.b_out = torch.randn((E, N), generator=g).to(torch.bfloat16) if bias else None

    def args(self):
        dev = lambda t: t.cuda() if t is not None else None
        return [dev(t) for t in (self.x, self.ids, self.w, self.win, self.wout, *self.scales, self.b_in, self.b_out)]

    def check(self, y):
        """Sums of n products in 32 bits are off by at most n units in the last place, 2^-23, of the sum of the magnitudes. h
        carries the errors of g and u (the slope of silu is at most 1.1), 2^-20 for its own operations (exp, the quotient,
        two products, the share's sum), and half a step of its type; y carries those through the second product."""
        T, half = self.x.shape[0], torch.finfo(self.dtype).eps / 2
        ulp, tiny = 2.0 ** -23, torch.finfo(self.dtype).tiny * half * 2
        x = self.x.double()
        H, I = x.shape[1], self.I
        y0, off = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape, dtype=torch.float64)
        for t in range(T):
            for e in set(self.ids[t].tolist()):
                if not 0 <= e < self.E:
                    continue
                p = self.w[t].double()[self.ids[t] == e].sum() if self.w is not None else (self.ids[t] == e).sum().double()
                a, mag = self.v_in[e] @ x[t], self.v_in[e].abs() @ x[t].abs()
                if self.b_in is not None:
                    a, mag = a + self.b_in[e].double(), mag + self.b_in[e].double().abs()
                d = (H + 1) * ulp * mag
                gate, up, dg, du = a[:I], a[I:], d[:I], d[I:]
                s = gate * torch.sigmoid(gate)
                h = p * s * up
                dh = p.abs() * (1.1 * dg * up.abs() + s.abs() * du + 1.1 * dg * du) + h.abs() * 2.0 ** -20
                dh = dh + (h.abs() + dh) * half + tiny
                y0[t] += self.v_out[e] @ h
                off[t] += self.v_out[e].abs() @ dh + (I + self.ids.shape[1] + 8) * ulp * (self.v_out[e].abs() @ h.abs())
                if self.b_out is not None:
                    y0[t] += p * self.b_out[e].double()
                    off[t] += 2 * self.ids.shape[1] * ulp * (p * self.b_out[e].double()).abs()
        # the sums over the experts, as above, and y's own rounding
        off = off + 2 * self.ids.shape[1] * ulp * y0.abs()
        off = off + (y0.abs() + off) * half + tiny
        got = y.cpu().double()
        worst = ((got - y0).abs() - off).max().item() if y.numel() else 0.0
        assert y.dtype == self.dtype and worst <= 0, worst


CASES = [(1, 1, 1, 128, 16, 16), (1, 4, 8, 256, 128, 256), (2, 2, 4, 100, 33, 70), (7, 2, 8, 333, 150, 129), (16, 4, 16, 512, 96, 320),
         (17, 3, 5, 130, 257, 64), (33, 2, 70, 64, 40, 33), (64, 8, 16, 256, 128, 128), (64, 4, 4, 384, 130, 96), (5, 1, 3, 1, 1, 1),
         (3, 2, 4, 2048, 640, 200), (40, 1, 2, 1025, 64, 15), (64, 16, 200, 32, 16, 24), (9, 2, 1024, 16, 8, 8),
         (64, 8, 128, 256, 256, 512), (48, 4, 48, 300, 700, 130), (16, 8, 128, 64, 128, 64), (16, 8, 128, 64, 1024, 16), (2, 1, 4, 4104, 24, 40)]


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,k,E,H,I,N", CASES)
def test_sizes(T, k, E, H, I, N, dtype, mxfp4):
    l = Layer(T, k, E, H, I, N, dtype, mxfp4, bias=T % 2 == 1)
    args = l.args()
    y = ep.mlp_forward_experts(*args)
    l.check(y)
    assert torch.equal(y, ep.mlp_forward_experts(*args))


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("T,k,E,H,I,N", [(64, 16, 1024, 16, 8, 8), (1, 1024, 1024, 40, 24, 20), (2, 1, 1, 2 ** 20, 8, 8), (2, 1, 1, 8, 2 ** 20, 8),
                                         (2, 1, 1, 8, 8, 2 ** 20), (64, 2, 2, 130, 20, 2 ** 15 + 3)])
def test_limits(T, k, E, H, I, N, mxfp4):
    """The largest numbers of choices and experts, and the longest and widest matrices."""
    l = Layer(T, k, E, H, I, N, mxfp4=mxfp4)
    l.check(ep.mlp_forward_experts(*l.args()))


@pytest.mark.parametrize("mxfp4", [False, True])
def test_choices(mxfp4):
    """Dropped choices, tokens without any, an expert named twice in a token, all tokens on one expert."""
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, 6, (20, 3), generator=g)
    ids[0] = -1
    ids[3] = torch.tensor([2, 2, 2])
    ids[4] = torch.tensor([6, 5, 2 ** 40])
    ids[5] = torch.tensor([-7, 1, 1])
    ids[19, 2] = -1
    for which in (ids, torch.full((64, 2), 1), torch.full((33, 1), 5), torch.full((8, 4), -1)):
        l = Layer(which.shape[0], 3, 6, 200, 70, 90, mxfp4=mxfp4, bias=True, ids=which)
        y = ep.mlp_forward_experts(*l.args())
        l.check(y)
        assert not y[((which < 0) | (which > 5)).all(1)].any()


def test_types_and_strides():
    """int32 expert numbers, no weights, rows of x further apart than H, at odd addresses."""
    l = Layer(12, 2, 5, 150, 40, 60)
    a = l.args()
    want = ep.mlp_forward_experts(*a)
    assert torch.equal(ep.mlp_forward_experts(a[0], a[1].int(), *a[2:]), want)
    room = torch.full((12, 171), float("nan"), dtype=torch.bfloat16, device="cuda")
    room[:, 7:157] = a[0]
    assert torch.equal(ep.mlp_forward_experts(room[:, 7:157], *a[1:]), want)

    def moved(t, by):
        flat = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
        flat[by:] = t.reshape(-1)
        return flat[by:].view(t.shape)

    assert torch.equal(ep.mlp_forward_experts(a[0], a[1], a[2], moved(a[3], 1), moved(a[4], 3)), want)
    l.w = None
    l.check(ep.mlp_forward_experts(a[0], a[1], None, a[3], a[4]))
    q = Layer(12, 2, 5, 150, 40, 60, mxfp4=True).args()
    assert torch.equal(ep.mlp_forward_experts(*q[:3], moved(q[3], 1), moved(q[4], 3), moved(q[5], 1), moved(q[6], 2)),
                       ep.mlp_forward_experts(*q))


@pytest.mark.parametrize("mxfp4", [False, True])
def test_nans_stay_where_they_belong(mxfp4):
    """A token of NaN, an expert nobody chose and a dropped choice's weight change no other token; nor does what the
    scratch held before."""
    ids = torch.tensor([[0, 1], [1, 3], [3, -1], [0, 3], [1, 0]])
    l = Layer(5, 2, 4, 140, 50, 70, mxfp4=mxfp4, ids=ids)
    a = l.args()
    want = ep.mlp_forward_experts(*a)
    a[0][1] = float("nan")
    a[2][2, 1] = float("nan")
    if mxfp4:
        a[5][2] = 255
        a[6][2] = 255
    else:
        a[3][2], a[4][2] = float("nan"), float("inf")
    junk = [torch.full((n, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (10, 10, 10, 5)]
    del junk
    y = ep.mlp_forward_experts(*a)
    assert torch.isnan(y[1]).all()
    keep = [0, 2, 3, 4]
    assert torch.equal(y[keep], want[keep])


def test_empty():
    for T, k, E, H, I, N in ((0, 2, 3, 64, 32, 16), (4, 0, 3, 64, 32, 16), (4, 2, 3, 0, 32, 16), (4, 2, 3, 64, 0, 16), (4, 2, 3, 64, 32, 0)):
        ids = torch.zeros((T, k), dtype=torch.int64)
        for mxfp4 in (False, True):
            l = Layer(T, k, E, H, I, N, bias=False, ids=ids)
            a = l.args()
            if mxfp4:
                a[3:7] = [*ep.quantize_rows_mxfp4(a[3]), *ep.quantize_rows_mxfp4(a[4])]
                a = a[:3] + [a[3], a[5], a[4], a[6]]
            y = ep.mlp_forward_experts(*a)
            assert y.shape == (T, N) and not y.any()
    l = Layer(4, 2, 3, 64, 0, 16, bias=True)
    l.check(ep.mlp_forward_experts(*l.args()))


@pytest.mark.parametrize("mxfp4", [False, True])
def test_against_the_sorted_path(mxfp4):
    """The same layer from sorted tokens and a product per expert: within the two paths' roundings."""
    l = Layer(30, 3, 6, 256, 128, 192, mxfp4=mxfp4, seed=5)
    a = l.args()
    y = ep.mlp_forward_experts(*a).double()
    rows, offsets, pos = ep.sort_tokens(a[0], a[1], 6)
    win, wout = l.v_in.cuda(), l.v_out.cuda()
    o = offsets.tolist()
    ys = torch.zeros((90, 192), dtype=torch.float32, device="cuda")
    for e in range(6):
        gu = rows[o[e]:o[e + 1]].double() @ win[e].T
        ys[o[e]:o[e + 1]] = ((torch.nn.functional.silu(gu[:, :128]) * gu[:, 128:]) @ wout[e].T).float()
    ref = ep.combine_tokens(ys, pos, a[2]).double()
    # h and y are rounded to bf16 here: 2^-8 of each term of the sum and of y; the norms of the terms are bounded by their sum
    assert (y - ref).norm() <= 2 * 2.0 ** -8 * ref.norm() * 3 ** 0.5


def test_other_stream_and_threads():
    l = Layer(16, 2, 8, 512, 256, 512, seed=8)
    a = l.args()
    want = ep.mlp_forward_experts(*a)
    side = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [ep.mlp_forward_experts(*a, stream=side[i % 3]) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)

    def work(i):
        with torch.cuda.stream(side[i]):
            return [ep.mlp_forward_experts(*a) for _ in range(20)]

    with ThreadPoolExecutor(3) as pool:
        done = list(pool.map(work, range(3)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for ys in done for y in ys)


@pytest.mark.parametrize("mxfp4", [False, True])
def test_weights_past_32_bits(mxfp4):
    """The last of the experts lies 2^32 elements (16 bits each, or bytes of codes) behind the first."""
    H, I, N = 32768, 2048, 64
    E = 65 if mxfp4 else 33
    l = Layer(2, 1, 1, H, I, N, mxfp4=mxfp4, ids=torch.zeros((2, 1), dtype=torch.int64))
    a = l.args()
    for i in range(3, 7):
        if a[i] is not None:
            room = torch.zeros((E, *a[i].shape[1:]), dtype=a[i].dtype, device="cuda")
            room[E - 1] = a[i][0]
            a[i] = room
    assert a[3][:E - 1].numel() == 2 ** 32
    a[1] += E - 1
    l.check(ep.mlp_forward_experts(*a))


def test_two_graphs_in_turn():
    """Two graphs of the layer that share a memory pool, replayed in turn, keep to their own inputs."""
    layers = [Layer(64, 4, 16, 256, 1024, 64, mxfp4=True, seed=s) for s in (1, 2)]
    args = [l.args() for l in layers]
    want = [ep.mlp_forward_experts(*a) for a in args]
    torch.cuda.synchronize()
    graphs, out, pool = [], [], torch.cuda.graph_pool_handle()
    for a in args:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], pool=pool):
            out.append(ep.mlp_forward_experts(*a))
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[i], want[i])
        assert torch.equal(ep.mlp_forward_experts(*args[1 - i]), want[1 - i])


@pytest.mark.parametrize("mxfp4", [False, True])
def test_captured_and_replayed(mxfp4):
    """Two captured calls, replayed with other inputs and eager calls between, give the eager results."""
    l = Layer(9, 2, 8, 256, 128, 256, mxfp4=mxfp4, seed=9)
    a = l.args()
    ep.mlp_forward_experts(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ep.mlp_forward_experts(*a)
        z = ep.mlp_forward_experts(y, *a[1:])
    g = torch.Generator().manual_seed(1)
    for i in range(4):
        a[0].copy_(torch.randn((9, 256), generator=g).to(torch.bfloat16))
        a[1].copy_(torch.randint(-1, 8, (9, 2), generator=g))
        a[2].copy_(torch.rand((9, 2), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        first = ep.mlp_forward_experts(*a)
        assert torch.equal(y, first) and torch.equal(z, ep.mlp_forward_experts(first, *a[1:])), i


def test_refusals():
    l = Layer(4, 2, 3, 64, 32, 16, bias=True)
    a = l.args()
    ep.mlp_forward_experts(*a)

    def refused(**change):
        names = ["x", "expert_ids", "weights", "w_in", "w_out", "in_scales", "out_scales", "in_bias", "out_bias"]
        with pytest.raises(ValueError):
            ep.mlp_forward_experts(**{**dict(zip(names, a)), **change})

    x, ids, w, win, wout = a[:5]
    refused(x=x.float())
    refused(x=x.half())
    refused(x=x[0])
    refused(x=x.cpu())
    refused(x=x.clone().requires_grad_())
    refused(weights=w.clone().requires_grad_())
    refused(expert_ids=ids[:3])
    refused(expert_ids=ids.float())
    refused(expert_ids=ids.cpu())
    refused(expert_ids=ids.t().contiguous().t())
    refused(weights=w.double())
    refused(weights=w[:, :1])
    refused(w_in=win[:, :63])
    refused(w_in=win[:2])
    refused(w_in=win.transpose(1, 2))
    refused(w_out=wout[:, :, :31])
    refused(w_out=wout.cpu())
    refused(in_bias=a[7][:, :32])
    refused(out_bias=a[8].float())
    q, s = ep.quantize_rows_mxfp4(win)
    q2, s2 = ep.quantize_rows_mxfp4(wout)
    ep.mlp_forward_experts(x, ids, w, q, q2, s, s2)
    refused(w_in=q, w_out=q2, in_scales=s)
    refused(w_in=q, w_out=q2, in_scales=s, out_scales=s2[:, :, :8])
    refused(w_in=q, w_out=q2)
    big = Layer(65, 1, 3, 64, 32, 16).args()
    with pytest.raises(ValueError, match="sort_tokens"):
        ep.mlp_forward_experts(*big)
    with torch.no_grad():
        ep.mlp_forward_experts(x.clone().requires_grad_(), *a[1:])
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises(ValueError):
        ep.mlp_forward_experts(fwd.make_dual(x, torch.ones_like(x)), *a[1:])


@pytest.mark.parametrize("mxfp4", [False, True])
@pytest.mark.parametrize("T,k,E,H,I,N,dup", [(5, 2, 4, 128, 96, 64, False), (3, 3, 4, 140, 70, 33, True), (64, 2, 8, 128, 130, 96, False),
                                             (40, 8, 128, 64, 256, 64, False)])
@pytest.mark.parametrize("weight,x_scale,out_scale", [(16.0, 48.0, 2.0 ** -8), (2.0 ** -12, 0.045, 2.0 ** 8), (-40.0, 48.0, 2.0 ** -9)])
def test_fp16_weights_far_from_one(T, k, E, H, I, N, dup, weight, x_scale, out_scale, mxfp4):
    """h fits FP16 and the weighted h does not: it would pass 65504, or lose bits below 2^-14. The weights belong to the 32-bit sums, so
    y is off by h's own rounding (half a step, 2^-11 of it or 2^-25) times the weight, and by what Layer.check counts otherwise."""
    ids = torch.full((T, k), 1) if dup else None
    l = Layer(T, k, E, H, I, N, torch.float16, mxfp4, seed=11, ids=ids)
    l.x = (l.x.double() * x_scale).to(torch.float16)
    l.w = torch.full((T, k), weight)
    if mxfp4:
        l.scales = (l.scales[0], (l.scales[1].int() + round(math.log2(out_scale))).to(torch.uint8))
        l.v_out = mx.values(l.wout, l.scales[1])[..., :I]
    else:
        l.wout = (l.wout.double() * out_scale).to(torch.float16)
        l.v_out = l.wout.double()
    ulp, half = 2.0 ** -23, 2.0 ** -11
    y0, off, top = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64), 0.0
    for t in range(T):
        for e in set(l.ids[t].tolist()):
            p = l.w[t].double()[l.ids[t] == e].sum()
            x = l.x[t].double()
            a, d = l.v_in[e] @ x, (H + 1) * ulp * (l.v_in[e].abs() @ x.abs())
            gate, up, dg, du = a[:I], a[I:], d[:I], d[I:]
            s = gate * torch.sigmoid(gate)
            h = s * up
            dh = 1.1 * dg * up.abs() + s.abs() * du + 1.1 * dg * du + h.abs() * 2.0 ** -20
            dh = dh + (h.abs() + dh) * half + 2.0 ** -25
            top = max(top, (h.abs() + dh).max().item())
            y0[t] += p * (l.v_out[e] @ h)
            off[t] += p.abs() * (l.v_out[e].abs() @ dh + (I + k + 8) * ulp * (l.v_out[e].abs() @ h.abs()))
    off = off + 2 * k * ulp * y0.abs()
    off = off + (y0.abs() + off) * half + 2.0 ** -25
    assert top < 65504 and (abs(weight) * top > 65504 or abs(weight) * top < 2.0 ** -14) and (y0.abs() + off).max() < 65504
    got = ep.mlp_forward_experts(*l.args()).cpu().double()
    assert ((got - y0).abs() <= off).all(), ((got - y0).abs() / off).max().item()
