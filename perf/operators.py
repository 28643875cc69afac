"""Timed cases of the INT8 matrix products and of the expert routing around them.

Five operators: the quantization of activation rows to INT8 ("quantize"), the product of INT8 codes
with a scale per token and per channel ("gemm"), the same product for every expert over the tokens
routed to it ("experts"), tokens sorted by expert and summed back with their weights ("route"), and
the gradients of that pair ("route_grad"). A case is a dict of plain values; prepare() makes what a
program holds before the call, run() is one call, and exact() gives the definition's values in 64
bits. With `own` set, run() makes the calls of the package; otherwise it computes the same outputs
from elementary torch operations.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = 2.0 ** -100            # a row's largest magnitude is raised to this when it is smaller and not zero


# ---------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the activations of one generated token, quantized before each INT8 layer: pure latency
        {"name": "quantize 1x8192 bf16", "op": "quantize", "M": 1, "K": 8192, "dtype": "bf16"},
        # a prefill's activations into the FFN down projection
        {"name": "quantize 4096x10240 bf16", "op": "quantize", "M": 4096, "K": 10240, "dtype": "bf16"},
        # one token through a fused QKV projection: the weight is read once, nothing else counts
        {"name": "gemm 1x11520x3840", "op": "gemm", "M": 1, "N": 11520, "K": 3840, "out": "bf16", "bias": True},
        # a small batch of sequences decoding through a square layer
        {"name": "gemm 16x8192x8192", "op": "gemm", "M": 16, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # ragged: a prompt of odd length, an odd output width (a cut vocabulary), an inner width that
        # is no multiple of 16, fp32 outputs for the logits
        {"name": "gemm 333x5003x3846 fp32", "op": "gemm", "M": 333, "N": 5003, "K": 3846, "out": "fp32", "bias": True},
        # prefill of 4096 tokens through an 8192 x 8192 layer: compute bound
        {"name": "gemm 4096x8192x8192", "op": "gemm", "M": 4096, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # 16 tokens decoding, 4 of 32 experts each: a few rows per expert, every hit expert's weight read
        {"name": "experts 16 of 32x4096x2048", "op": "experts", "T": 16, "k": 4, "E": 32, "N": 4096, "K": 2048, "out": "bf16"},
        # prefill of 4096 tokens, unevenly spread over the experts: compute bound
        {"name": "experts 4096 of 32x2048x4096", "op": "experts", "T": 4096, "k": 4, "E": 32, "N": 2048, "K": 4096, "out": "bf16"},
        # a few tokens decoding: latency of the sort
        {"name": "route 7x2048 4 of 32", "op": "route", "T": 7, "k": 4, "E": 32, "H": 2048, "dtype": "bf16", "drop": 0.0},
        # a long prefill, one choice in 50 dropped (over an expert's capacity): memory bound
        {"name": "route 16384x4096 4 of 64", "op": "route", "T": 16384, "k": 4, "E": 64, "H": 4096, "dtype": "bf16", "drop": 0.02},
        # a small training step of odd length in fp32
        {"name": "route_grad 509x1000 2 of 8 fp32", "op": "route_grad", "T": 509, "k": 2, "E": 8, "H": 1000, "dtype": "fp32", "drop": 0.1},
        # a training step of 4096 tokens, 8 experts each
        {"name": "route_grad 4096x2048 8 of 128", "op": "route_grad", "T": 4096, "k": 8, "E": 128, "H": 2048, "dtype": "bf16", "drop": 0.0},
    ]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithms, odd ones among them."""
    def spread(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(["quantize", "gemm", "gemm", "experts", "route", "route_grad"])
    if op == "quantize":
        M = spread(1, 4096)
        return {"op": op, "M": M, "K": spread(64, 10240, rng.choice([1, 8, 64])), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "gemm":
        M = spread(1, 4096)
        step = rng.choice([1, 16, 64, 256])
        return {"op": op, "M": M, "N": spread(256, 8192, rng.choice([1, 16, 128])), "K": spread(256, 8192, step),
                "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5}
    E = rng.choice([8, 16, 32, 64])
    k = rng.choice([1, 2, 4])
    if op == "experts":
        return {"op": op, "T": spread(1, 4096), "k": k, "E": E, "N": spread(256, 2048, rng.choice([1, 16, 128])),
                "K": spread(256, 4096, 16), "out": rng.choice(["bf16", "fp16"])}
    return {"op": op, "T": spread(1, 4096), "k": k, "E": E, "H": spread(128, 4096, rng.choice([1, 8, 64])),
            "dtype": rng.choice(["bf16", "fp16", "fp32"]), "drop": rng.choice([0.0, 0.05])}


# --------------------------------------------------------------------------------------- the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, M, K, dtype):
    """N(0, 1) rows of differing size with a few channels twenty times larger, as hidden states have."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((M, 1), generator=g, device="cuda"))
    x[:, torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")] *= 20.0
    return x.to(dtype)


def _codes(g, shape):
    return (32.0 * torch.randn(shape, generator=g, device="cuda")).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, shape):
    return 0.01 * torch.exp(0.5 * torch.randn(shape, generator=g, device="cuda"))


def _choices(g, T, k, E, drop):
    """k different experts per token, some experts chosen more often than others; a dropped choice is -1."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    if drop > 0:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < drop, -1, ids)
    return ids, torch.softmax(top, dim=1)


def _plan(ids, E):
    """(order, offsets, pos) of a stable sort of the choices by expert. Dropped choices go last, and
    the position of one is -1 - row."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(E, device=flat.device)[None, :]).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=flat.device)
    pos = torch.where(key < E, pos, -1 - pos).to(torch.int32).reshape(ids.shape)
    return order, offsets, pos


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case)
    if op == "quantize":
        st["x"] = _activations(g, case["M"], case["K"], DTYPES[case["dtype"]])
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["xq"], st["xs"] = _codes(g, (M, K)), _scales(g, (M,))
        st["wq"], st["ws"] = _codes(g, (N, K)), _scales(g, (N,))
        st["b"] = torch.randn((N,), generator=g, device="cuda").to(torch.bfloat16) if case["bias"] else None
    elif op == "experts":
        T, k, E, N, K = (case[c] for c in ("T", "k", "E", "N", "K"))
        ids, _ = _choices(g, T, k, E, 0.0)
        st["offsets"] = _plan(ids, E)[1]
        st["xq"], st["xs"] = _codes(g, (T * k, K)), _scales(g, (T * k,))
        st["wq"], st["ws"] = _codes(g, (E, N, K)), _scales(g, (E, N))
    else:
        T, k, E, H = (case[c] for c in ("T", "k", "E", "H"))
        dtype = DTYPES[case["dtype"]]
        grad = op == "route_grad"
        st["ids"], w = _choices(g, T, k, E, case["drop"])
        st["x"] = torch.randn((T, H), generator=g, device="cuda").to(dtype).requires_grad_(grad)
        st["ys"] = torch.randn((T * k, H), generator=g, device="cuda").to(dtype).requires_grad_(grad)   # the experts' outputs
        st["w"] = w.contiguous().requires_grad_(grad)
        if grad:
            st["d_rows"] = torch.randn((T * k, H), generator=g, device="cuda").to(dtype)   # from the experts' inputs
            st["d_y"] = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    return st


# ---------------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import decode_tile_interleaved_rans_amd as ep
    op = st["op"]
    if op == "quantize":
        q, s = ep.quantize_rows_int8(st["x"])
        return q * s[:, None], s
    if op == "gemm":
        return ep.gemm_int8(st["xq"], st["xs"], st["wq"], st["ws"], st["b"], out_dtype=DTYPES[st["out"]])
    if op == "experts":
        return ep.gemm_int8_experts(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], out_dtype=DTYPES[st["out"]])
    rows, offsets, pos = ep.sort_tokens(st["x"], st["ids"], st["E"])
    y = ep.combine_tokens(st["ys"], pos, st["w"])
    if op == "route":
        return rows, offsets, pos, y
    return torch.autograd.grad([rows, y], [st["x"], st["ys"], st["w"]], [st["d_rows"], st["d_y"]])


def _plain(st):
    op = st["op"]
    if op == "quantize":
        # 64 bits: a quotient next to a rounding border has to fall on its own side
        x = st["x"].double()
        amax = x.abs().amax(1, keepdim=True)
        amax = torch.where(amax > 0, amax.clamp_min(TINY), amax)
        q = torch.where(amax > 0, 127.0 * x / amax, 0.0).round()
        s = (amax / 127.0).float()
        return q.float() * s, s[:, 0]
    if op == "gemm":
        y = (st["xq"].float() @ st["wq"].float().T) * st["xs"][:, None] * st["ws"][None, :]
        if st["b"] is not None:
            y = y + st["b"].float()
        return y.to(DTYPES[st["out"]])
    if op == "experts":
        y = torch.zeros((st["xq"].shape[0], st["N"]), device="cuda")
        offs = st["offsets"].tolist()
        for e in range(st["E"]):
            a, b = offs[e], offs[e + 1]
            if b > a:
                y[a:b] = (st["xq"][a:b].float() @ st["wq"][e].float().T) * st["xs"][a:b, None] * st["ws"][e][None, :]
        return y.to(DTYPES[st["out"]])
    T, k, E = st["T"], st["k"], st["E"]
    order, offsets, pos = _plan(st["ids"], E)
    held = (torch.arange(T * k, device="cuda") < offsets[-1])[:, None]         # rows of a dropped choice stay zero
    at = pos.long().clamp_min(0)
    taken = (pos >= 0).unsqueeze(2)
    if op == "route":
        rows = torch.where(held, st["x"][order // k], 0)
        y = torch.where(taken, st["w"].unsqueeze(2) * st["ys"][at].float(), 0.0).sum(1)
        return rows, offsets, pos, y.to(st["x"].dtype)
    # the formulas of the gradients: dx sums a token's rows, d_ys spreads w dy, d_w is a dot product
    dx = torch.where(taken, st["d_rows"][at].float(), 0.0).sum(1)
    dy = st["d_y"].float()
    d_ys = torch.where(held, st["w"].reshape(-1)[order, None] * dy[order // k], 0.0)
    d_w = torch.where(taken, st["ys"][at].float() * dy[:, None, :], 0.0).sum(2)
    return dx.to(st["x"].dtype), d_ys.to(st["x"].dtype), d_w


# ------------------------------------------------------------------------------------ bytes and work
def work(case):
    """Each input read once, each output written once; the operations of the formulas."""
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "quantize":
        M, K, es = case["M"], case["K"], size[case["dtype"]]
        return {"bytes": M * K * (es + 1) + 4 * M, "flops": 4 * M * K}
    if op == "gemm":
        M, N, K, es = case["M"], case["N"], case["K"], size[case["out"]]
        return {"bytes": M * K + N * K + es * M * N + 4 * (M + N) + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "experts":
        R, E, N, K, es = case["T"] * case["k"], case["E"], case["N"], case["K"], size[case["out"]]
        hit = E * (1.0 - (1.0 - case["k"] / E) ** case["T"])                  # experts that some token chose
        return {"bytes": int(R * K + hit * (N * K + 4 * N) + es * R * N + 4 * R), "flops": 2 * R * N * K}
    T, k, H, es = case["T"], case["k"], case["H"], size[case["dtype"]]
    kept = T * k * (1.0 - case["drop"])
    if op == "route":
        # x read, rows written, ys read, y written, the choices, weights and positions
        return {"bytes": int(es * H * (2 * T + T * k + kept) + T * k * (8 + 4 + 4)), "flops": int(2 * kept * H)}
    # forward as above; backward: d_rows and d_y read, ys read again, dx and d_ys written
    return {"bytes": int(es * H * (2 * T + T * k + kept) + es * H * (2 * T + 2 * kept + T * k) + T * k * (8 + 4 + 4 + 4)),
            "flops": int(6 * kept * H)}


# --------------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].to(torch.float64)
        top = x.abs().max(dim=1).values
        top = torch.where(top == 0, top, torch.clamp(top, min=TINY))
        unit = top / 127.0
        codes = torch.zeros_like(x)
        live = top > 0
        codes[live] = torch.round(x[live] * 127.0 / top[live][:, None])
        return codes * unit[:, None], unit
    if op == "gemm":
        y = torch.mm(st["xq"].to(torch.float64), st["wq"].to(torch.float64).t().contiguous())
        y = y * torch.outer(st["xs"].double(), st["ws"].double())
        return y if st["b"] is None else y + st["b"].double().unsqueeze(0)
    if op == "experts":
        edge = st["offsets"].cpu().tolist()
        y = torch.zeros((st["xq"].shape[0], case["N"]), dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(edge[:-1], edge[1:])):
            if a < b:
                y[a:b] = torch.mm(st["xq"][a:b].to(torch.float64), st["wq"][e].to(torch.float64).t().contiguous())
                y[a:b] *= torch.outer(st["xs"][a:b].double(), st["ws"][e].double())
        return y
    T, k, E, H = (case[c] for c in ("T", "k", "E", "H"))
    # choice by choice on the host: the rows of each expert in the order of their choices
    ids = st["ids"].cpu().tolist()
    rows_of = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t][j] < E:
                rows_of[ids[t][j]].append((t, j))
    edge, source, at = [0], [], [[None] * k for _ in range(T)]
    for e in range(E):
        for t, j in rows_of[e]:
            at[t][j] = len(source)
            source.append(t * k + j)
        edge.append(len(source))
    behind = len(source)                                  # the rows that dropped choices leave unused
    for t in range(T):
        for j in range(k):
            if at[t][j] is None:
                at[t][j] = -1 - behind
                behind += 1
    source = torch.tensor(source, dtype=torch.int64, device="cuda")
    n = source.numel()
    w = st["w"].detach().double().reshape(-1)
    if op == "route":
        rows = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        rows[:n] = st["x"].detach().double()[source // k]
        y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        y.index_add_(0, source // k, st["ys"].detach().double()[:n] * w[source][:, None])
        return (rows, torch.tensor(edge, dtype=torch.int32, device="cuda"),
                torch.tensor(at, dtype=torch.int32, device="cuda").reshape(T, k), y)
    dy = st["d_y"].double()
    dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dx.index_add_(0, source // k, st["d_rows"].double()[:n])
    d_ys = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    d_ys[:n] = dy[source // k] * w[source][:, None]
    d_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    d_w[source] = (dy[source // k] * st["ys"].detach().double()[:n]).sum(1)
    return dx, d_ys, d_w.reshape(T, k)
