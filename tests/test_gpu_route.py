"""Expert routing on the GPU: tokens sorted by expert, summed back with their weights, and the
gradients, against plain loops and 64-bit sums.

Positions, offsets and sorted rows must be equal exactly. A sum over k choices in fp32 is off by at most
k 2^-24 of the sum of the magnitudes (one fused multiply-add each), then by the output type's rounding
(half of finfo.eps); a dot product over H columns by at most (H + 8) 2^-24 of the sum of its products'
magnitudes, whatever the order."""
import numpy as np
import pytest
import torch

import decode_tile_interleaved_rans_amd as ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def plan(ids, E):
    """(offsets, pos, source) by loops over the choices on the host."""
    T, k = ids.shape
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    pos = np.empty(T * k, np.int64)
    pos[order] = np.arange(T * k)
    pos = np.where(key < E, pos, -1 - pos).astype(np.int32).reshape(T, k)
    off = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(np.int32)
    return off, pos, order // max(k, 1)


def check_sort(x, ids, E):
    rows, off, pos = ep.sort_tokens(x, ids, E)
    woff, wpos, src = plan(ids, E)
    assert off.dtype == torch.int32 and pos.dtype == torch.int32 and rows.dtype == x.dtype
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(pos.cpu().numpy(), wpos)
    n = int(woff[-1])
    bits = lambda t: t.contiguous().view(torch.uint8) if t.element_size() == 1 else t
    assert torch.equal(bits(rows[:n]), bits(x[torch.from_numpy(src[:n]).cuda()]))
    assert not bits(rows[n:]).any()
    return rows, off, pos


def choices(T, k, E, seed, drop=0.1, dtype=torch.int64):
    ids = torch.randint(0, E, (T, k), generator=gen(seed), device="cuda")
    bad = torch.rand((T, k), generator=gen(seed + 1), device="cuda")
    ids = torch.where(bad < drop / 2, -1, torch.where(bad < drop, E, ids))
    return ids.to(dtype)


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 1024), (5, 0, 3), (7, 4, 32), (64, 1, 3), (65, 2, 1), (512, 2, 8),
                                   (513, 2, 8), (128, 8, 1023), (129, 8, 1024), (1024, 1, 5), (1025, 1, 64), (3000, 6, 60),
                                   (20000, 8, 256), (70000, 2, 7), (150001, 1, 1000)])
def test_order(T, k, E):
    x = torch.randn((T, 24), generator=gen(1), device="cuda").to(torch.bfloat16)
    check_sort(x, choices(T, k, E, T + k), E)
    check_sort(x, choices(T, k, E, T + k, drop=0.0, dtype=torch.int32), E)


@pytest.mark.parametrize("H", [1, 3, 8, 100, 1000, 2056, 4099])
@pytest.mark.parametrize("dtype", [*TYPES, torch.int8, torch.float8_e4m3fn, torch.uint8])
def test_rows_of_any_type_and_width(H, dtype):
    for T in (9, 700):
        x = (torch.randn((T, H), generator=gen(H), device="cuda") * 50).to(dtype)
        check_sort(x, choices(T, 3, 10, H), 10)


def test_all_one_expert_all_dropped_and_far_numbers():
    x = torch.randn((900, 16), generator=gen(2), device="cuda")
    for T in (300, 900):
        check_sort(x[:T], torch.full((T, 2), 5, device="cuda"), 6)
        check_sort(x[:T], torch.full((T, 2), -1, device="cuda"), 6)
        far = torch.full((T, 2), 2 ** 32 + 1, device="cuda")       # expert 1 if it were cut to 32 bits
        far[3, 1] = -2 ** 63
        far[4, 0] = 1
        check_sort(x[:T], far, 6)
        check_sort(x[:T], torch.full((T, 2), -2 ** 31, dtype=torch.int32, device="cuda"), 6)


def test_strided_tokens():
    base = torch.randn((800, 300), generator=gen(3), device="cuda").to(torch.bfloat16)
    for x in (base[:, 8:136], base[:, 3:100], base[::2, :64], base[:7, 1:2], base[:1, :]):
        check_sort(x, choices(x.shape[0], 2, 5, 7), 5)


# ------------------------------------------------------------------------------------ sums and gradients
def combine64(ys, pos, w, dy=None):
    """(y, its tolerance base) in 64 bits; with dy also d_ys and d_w."""
    p = pos.long()
    on = (p >= 0)
    at = p.clamp_min(0)
    w64 = torch.ones(p.shape, dtype=torch.float64, device="cuda") if w is None else w.double()
    rows = torch.where(on[..., None], ys.double()[at], 0.0)
    y = (w64[..., None] * rows).sum(1)
    mag = (w64[..., None] * rows).abs().sum(1)
    if dy is None:
        return y, mag
    d_w = (rows * dy.double()[:, None, :]).sum(2)
    d_w_mag = (rows * dy.double()[:, None, :]).abs().sum(2)
    d_ys = torch.zeros_like(ys, dtype=torch.float64)
    d_ys[at[on]] = (w64[..., None] * dy.double()[:, None, :])[on]
    return y, mag, d_ys, d_w, d_w_mag


def close(got, ref, fp32):
    half = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134
    tol = fp32 + half * (ref.abs() + fp32) + tiny
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"largest excess {(err - tol).max().item():.3g}"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 8, 16, 2048), (7, 4, 32, 100), (33, 3, 5, 999), (64, 5, 8, 1024), (300, 2, 8, 4104),
                                     (1000, 9, 12, 64), (2500, 1, 3, 130)])
def test_sum_and_gradients(T, k, E, H, dtype):
    ids = choices(T, k, E, T + H)
    g = gen(T + H + 7)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype).requires_grad_(True)
    rows, off, pos = ep.sort_tokens(x, ids, E)
    ys = torch.randn((T * k, H), generator=g, device="cuda").to(dtype).requires_grad_(True)
    w = torch.rand((T, k), generator=g, device="cuda").requires_grad_(True)
    y = ep.combine_tokens(ys, pos, w)
    d_rows = torch.randn((T * k, H), generator=g, device="cuda").to(dtype)
    dy = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    dx, d_ys, d_w = torch.autograd.grad([rows, y], [x, ys, w], [d_rows, dy])
    ry, mag, rys, rw, rwmag = combine64(ys.detach(), pos, w.detach(), dy)
    close(y.detach(), ry, k * U * mag)
    close(d_ys, rys, U * rys.abs())
    err = (d_w.double() - rw).abs()
    assert (err <= (H + 8) * U * rwmag + 1e-38).all()
    rx, xmag = combine64(d_rows, pos, None)
    close(dx, rx, k * U * xmag)
    assert dx.dtype == dtype and d_ys.dtype == dtype and d_w.dtype == torch.float32
    # one gradient without the others gives the same bits
    y2 = ep.combine_tokens(ys, pos, w.detach())
    assert torch.equal(torch.autograd.grad(y2, ys, dy)[0], d_ys)
    y3 = ep.combine_tokens(ys.detach(), pos, w)
    assert torch.equal(torch.autograd.grad(y3, w, dy)[0], d_w)
    y4 = ep.combine_tokens(ys, pos)
    ones = combine64(ys.detach(), pos, None, dy)
    close(torch.autograd.grad(y4, ys, dy)[0], ones[2], U * ones[2].abs())


def test_gradients_against_differences():
    # y is linear in ys and in w, and rows linear in x: a difference of two calls is the derivative up to
    # the calls' fp32 rounding. Along unit-size steps v: <d, v> against (f(+v) - f(-v)) / 2, both sides off
    # by at most n 2^-24 of the magnitudes, n the length of the longest sum.
    T, k, E, H = 50, 3, 6, 40
    ids = choices(T, k, E, 5)
    g = gen(9)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, ys, w, dy, d_rows = r(T, H), r(T * k, H), r(T, k), r(T, H), r(T * k, H)
    for t in (x, ys, w):
        t.requires_grad_(True)
    rows, _, pos = ep.sort_tokens(x, ids, E)
    y = ep.combine_tokens(ys, pos, w)
    dx, d_ys, d_w = torch.autograd.grad([rows, y], [x, ys, w], [d_rows, dy])
    f_y = lambda ys_, w_: (ep.combine_tokens(ys_, pos, w_).double() * dy.double())
    f_r = lambda x_: (ep.sort_tokens(x_, ids, E)[0].double() * d_rows.double())
    with torch.no_grad():
        for f, at, d in ((lambda v: f_y(ys + v, w), ys, d_ys), (lambda v: f_y(ys, w + v), w, d_w), (lambda v: f_r(x + v), x, dx)):
            v = r(*at.shape)
            up, down = f(v), f(-v)
            diff = (up.sum() - down.sum()) / 2
            want = (d.double() * v.double()).sum()
            bound = (H + 16) * U * 4 * ((up.abs() + down.abs()).sum() + (d.double() * v.double()).abs().sum())
            assert (diff - want).abs() <= bound


def test_dropped_rows_do_not_count():
    # whatever the rows behind the experts' hold, NaN among it, tokens do not see it
    T, k, E, H = 40, 2, 4, 72
    ids = choices(T, k, E, 3, drop=0.4)
    ids[7] = -1                                               # a token with no expert left
    x = torch.randn((T, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    rows, off, pos = ep.sort_tokens(x, ids, E)
    ys = rows.clone()
    ys[int(off[-1]):] = float("nan")
    w = torch.rand((T, k), generator=gen(2), device="cuda")
    w[ids < 0] = float("nan")
    ys.requires_grad_(True)
    w.requires_grad_(True)
    y = ep.combine_tokens(ys, pos, w)
    dy = torch.ones_like(y)
    d_ys, d_w = torch.autograd.grad(y, [ys, w], dy)
    assert torch.isfinite(y).all() and not y[7].any()
    assert not d_ys[int(off[-1]):].any() and not d_w[7].any() and torch.isfinite(d_w).all()


def test_positions_outside_are_left_out():
    ys = torch.randn((10, 32), generator=gen(1), device="cuda")
    pos = torch.tensor([[3, 12], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    y = ep.combine_tokens(ys, pos)
    assert torch.equal(y[0], ys[3]) and not y[1].any()


def test_same_expert_twice():
    x = torch.randn((5, 8), generator=gen(1), device="cuda")
    ids = torch.tensor([[1, 1], [0, 1], [1, 0], [2, 2], [-1, 1]], device="cuda")
    rows, off, pos = check_sort(x, ids, 3)
    assert torch.equal(ep.combine_tokens(rows, pos), torch.stack([2 * x[0], 2 * x[1], 2 * x[2], 2 * x[3], x[4]]))


def test_noncontiguous_gradients():
    T, k, H = 20, 2, 16
    x = torch.randn((T, H), generator=gen(1), device="cuda").requires_grad_(True)
    ids = choices(T, k, 4, 1, drop=0.0)
    rows, _, pos = ep.sort_tokens(x, ids, 4)
    y = ep.combine_tokens(rows, pos)
    (y.sum()).backward()                                      # an expanded gradient of ones
    assert torch.equal(x.grad, torch.full_like(x, float(k)))


def test_captured_and_replayed():
    T, k, E, H = 700, 2, 16, 64
    x = torch.randn((T, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    ids, w = choices(T, k, E, 4), torch.rand((T, k), generator=gen(2), device="cuda")

    def step():
        rows, off, pos = ep.sort_tokens(x, ids, E)
        return rows, off, pos, ep.combine_tokens(rows, pos, w)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                        # two graphs, each with its own scratch
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for i in range(4):
        ids.copy_(choices(T, k, E, 10 + i))
        x.copy_(torch.roll(x, 3, 0))
        for graph, _ in graphs:
            graph.replay()
        want = step()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b), i


def test_training_step_captured_and_replayed():
    # forward and backward in one graph, on leaves of its own; every replay against eager leaves
    T, k, E, H = 600, 2, 8, 128
    ids = choices(T, k, E, 4)
    x, w = torch.randn((T, H), generator=gen(1), device="cuda"), torch.rand((T, k), generator=gen(2), device="cuda")
    dy = torch.randn((T, H), generator=gen(3), device="cuda")

    def step(x, w):
        rows, _, pos = ep.sort_tokens(x, ids, E)
        y = ep.combine_tokens(rows * 2, pos, w)
        return (y, *torch.autograd.grad(y, [x, w], dy))

    gx, gw = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(gx, gw)                                      # warm up; its graph is gone before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [t.detach() for t in step(gx, gw)]
    for i in range(4):
        with torch.no_grad():
            gx.copy_(torch.roll(x, i, 0))
            gw.copy_(torch.roll(w, i, 0))
        ids.copy_(choices(T, k, E, 20 + i))
        graph.replay()
        want = step(gx.detach().clone().requires_grad_(True), gw.detach().clone().requires_grad_(True))
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b.detach()), i


def test_other_stream_with_gradients():
    T, k, E, H = 600, 2, 8, 512
    ids = choices(T, k, E, 4)
    x = torch.randn((T, H), generator=gen(1), device="cuda")
    w = torch.rand((T, k), generator=gen(2), device="cuda")
    dy = torch.randn((T, H), generator=gen(3), device="cuda")

    def grads(stream):
        xa, wa = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
        rows, _, pos = ep.sort_tokens(xa, ids, E, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        y = ep.combine_tokens(rows, pos, wa, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return (y.detach(), *torch.autograd.grad(y, [xa, wa], dy))

    want = grads(None)
    got = grads(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_same_bits_every_time():
    T, k, E, H = 5000, 8, 64, 256
    ids = choices(T, k, E, 4)
    x = torch.randn((T, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    ys = torch.randn((T * k, H), generator=gen(2), device="cuda").to(torch.bfloat16).requires_grad_(True)
    w = torch.rand((T, k), generator=gen(3), device="cuda").requires_grad_(True)
    first = None
    for _ in range(3):
        rows, off, pos = ep.sort_tokens(x, ids, E)
        y = ep.combine_tokens(ys, pos, w)
        out = [rows, off, pos, y.detach(), *torch.autograd.grad(y, [ys, w], torch.ones_like(y))]
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_rows_past_32_bit_offsets():
    # 2.4e9 elements of sorted rows: 64-bit addresses in every kernel
    T, k, E, H = 300000, 2, 16, 4000
    ids = choices(T, k, E, 8, drop=0.0)
    x = (torch.arange(T, device="cuda")[:, None] % 251).to(torch.bfloat16).expand(T, H).contiguous()
    rows, off, pos = ep.sort_tokens(x, ids, E)
    want = torch.empty(T * k, dtype=torch.bfloat16, device="cuda")
    want[pos.long().reshape(-1)] = (torch.arange(T, device="cuda") % 251).to(torch.bfloat16).repeat_interleave(k)
    for c in (0, 1777, H - 1):
        assert torch.equal(rows[:, c], want)
    w = torch.ones((T, k), device="cuda").requires_grad_(True)
    rows.requires_grad_(True)
    y = ep.combine_tokens(rows, pos, w)
    assert torch.equal(y.detach()[:, H - 1], 2 * x[:, 0])      # at most 500: exact in BF16
    d_rows, d_w = torch.autograd.grad(y, [rows, w], x)
    assert torch.equal(d_rows[:, H - 1], want)
    ref = H * x[:, :1].double() ** 2                           # every product exact, sums in fp32
    assert ((d_w.double() - ref).abs() <= (H + 8) * U * ref).all()


def test_rows_can_be_changed_in_place():
    # the sorted rows are the caller's own, with and without a gradient: an in-place step on them is a step of
    # the graph, as on rows taken by an index
    T, k, E, H = 37, 3, 5, 72
    ids, w = choices(T, k, E, 2), torch.rand((T, k), generator=gen(3), device="cuda")
    x = torch.randn((T, H), generator=gen(1), device="cuda")
    dy = torch.randn((T, H), generator=gen(4), device="cuda")
    outs, grads = [], []
    for grad in (False, True):
        leaf = x.clone().requires_grad_(grad)
        rows, off, pos = ep.sort_tokens(leaf, ids, E)
        assert rows.requires_grad == grad and not off.requires_grad and not pos.requires_grad
        rows.mul_(3.0)
        rows += 1.0
        torch.nn.functional.dropout(rows, 0.0, inplace=True)
        outs.append(ep.combine_tokens(rows, pos, w))
        if grad:
            (dx,) = torch.autograd.grad(outs[1], leaf, dy)
    assert torch.equal(outs[0], outs[1].detach())
    taken = ((ids >= 0) & (ids < E)).double() * w.double()
    ref = 3.0 * dy.double() * taken.sum(1, keepdim=True)
    # a row's gradient w dy and its triple, each one rounding, then k sums
    assert ((dx.double() - ref).abs() <= (k + 2) * U * 3.0 * dy.double().abs() * taken.sum(1, keepdim=True)).all()


def test_second_derivative_is_refused():
    x = torch.randn((6, 16), device="cuda").requires_grad_(True)
    ids = choices(6, 2, 3, 1)
    rows, _, pos = ep.sort_tokens(x, ids, 3)
    y = ep.combine_tokens(rows * rows, pos)
    (dx,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_float8_rows_have_no_gradient():
    x = torch.randn((4, 32), device="cuda").to(torch.float8_e4m3fn).requires_grad_(True)
    with pytest.raises(ValueError, match="detach"):
        ep.sort_tokens(x, torch.zeros((4, 1), dtype=torch.int64, device="cuda"), 2)


def test_from_several_threads():
    import threading
    T, k, E, H = 1500, 2, 8, 256
    ids = choices(T, k, E, 4)
    x = torch.randn((T, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    w = torch.rand((T, k), generator=gen(2), device="cuda")
    q, s = ep.quantize_rows_int8(x)

    def work():
        rows, off, pos = ep.sort_tokens(x, ids, E)
        q2, s2 = ep.quantize_rows_int8(rows)
        return rows, off, pos, ep.combine_tokens(rows, pos, w), q2, s2, ep.gemm_int8(q, s, q, s)

    want = work()
    torch.cuda.synchronize()
    errors = []

    def run():
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                for _ in range(5):
                    got = work()
                    torch.cuda.current_stream().synchronize()
                    for a, b in zip(got, want):
                        assert torch.equal(a, b)
        except BaseException as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not errors, errors


def test_threads_end_and_agree():
    # as above, and every worker has to come to its end: one that hangs is a failure, not a silence
    import threading
    T, k, E, H = 900, 3, 16, 136
    ids = choices(T, k, E, 9)
    x = torch.randn((T, H), generator=gen(1), device="cuda")
    w = torch.rand((T, k), generator=gen(2), device="cuda")
    dy = torch.randn((T, H), generator=gen(3), device="cuda")

    def work():
        leaf, wl = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
        rows, off, pos = ep.sort_tokens(leaf, ids, E)
        y = ep.combine_tokens(rows, pos, wl)
        return rows.detach(), off, pos, y.detach(), *torch.autograd.grad(y, [leaf, wl], dy)

    want = work()
    torch.cuda.synchronize()
    errors, ended = [], []

    def run(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got = work()
                    torch.cuda.current_stream().synchronize()
                    for a, b in zip(got, want):
                        assert torch.equal(a, b)
            ended.append(i)
        except BaseException as e:
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,), daemon=True) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not errors, errors
    assert not any(t.is_alive() for t in threads) and sorted(ended) == [0, 1, 2, 3]


# ------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 13, 600])
def test_expert_layer_in_int8(T):
    """Quantize, sort the codes and their scales, multiply per expert, sum back: the INT8 expert layer,
    against the same in 64 bits from the operators' own codes and order."""
    k, E, H, N = 2, 6, 256, 200
    g = gen(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids, w = choices(T, k, E, T), torch.rand((T, k), generator=g, device="cuda")
    wq = torch.randint(-127, 128, (E, N, H), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((E, N), generator=g, device="cuda") * 1e-3
    q, s = ep.quantize_rows_int8(x)
    rq, off, pos = ep.sort_tokens(q, ids, E)
    rs = ep.sort_tokens(s[:, None], ids, E)[0][:, 0].contiguous()
    ys = ep.gemm_int8_experts(rq, rs, wq, ws, off, out_dtype=torch.float32)
    y = ep.combine_tokens(ys, pos, w)
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                v = (wq[e].double() @ q[t].double()) * s[t].double() * ws[e].double() * w[t, j].double()
                want[t] += v
                mag[t] += v.abs()
    assert ((y.double() - want).abs() <= (k + 6) * U * mag + 1e-30).all()
