"""Timed cases of the microscaled 4-bit floating point (MXFP4) operators and of an expert layer for few tokens.

Four operators: rows quantized to MXFP4 and back to values ("quantize"), the product of two MXFP4 matrices
("gemm"), the same product for every expert over the tokens routed to it ("experts"), and a whole
mixture-of-experts layer, gated MLP experts included, for up to 64 tokens ("mlp"). A case is a dict of plain
values; prepare() makes what a program holds before the call, run() is one call, and exact() gives the
definition's values in 64 bits. With `own` set, run() makes the calls of the package; otherwise it computes
the same outputs from elementary torch operations.

MXFP4: 32 consecutive elements of a row share a scale 2^(b - 127), b a byte; an element is a sign and one of
0, 0.5, 1, 1.5, 2, 3, 4, 6, two to a byte, the even one in the low half. Rows are padded with zeros to whole
128 elements (Kp). Codes are [..., rows, Kp / 2], scales [..., Kp / 128, rows, 4].
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the activations of one generated token, quantized before each layer: pure latency
        {"name": "quantize 1x8192 bf16", "op": "quantize", "M": 1, "K": 8192, "dtype": "bf16"},
        # a prefill's activations into the FFN down projection
        {"name": "quantize 4096x10240 bf16", "op": "quantize", "M": 4096, "K": 10240, "dtype": "bf16"},
        # one token through a fused QKV projection: the weight is read once, nothing else counts
        {"name": "gemm 1x11520x3840", "op": "gemm", "M": 1, "N": 11520, "K": 3840, "out": "bf16", "bias": True},
        # a small batch of sequences decoding through a square layer
        {"name": "gemm 16x8192x8192", "op": "gemm", "M": 16, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # ragged: a prompt of odd length, an odd output width (a cut vocabulary), an inner width that is no
        # multiple of a block, fp32 outputs for the logits
        {"name": "gemm 333x5003x3846 fp32", "op": "gemm", "M": 333, "N": 5003, "K": 3846, "out": "fp32", "bias": True},
        # prefill of 4096 tokens through an 8192 x 8192 layer: compute bound
        {"name": "gemm 4096x8192x8192", "op": "gemm", "M": 4096, "N": 8192, "K": 8192, "out": "bf16", "bias": False},
        # 16 tokens decoding, 4 of 32 experts each: a few rows per expert, every hit expert's weight read
        {"name": "experts 16 of 32x4096x2048", "op": "experts", "T": 16, "k": 4, "E": 32, "N": 4096, "K": 2048, "out": "bf16"},
        # prefill of 4096 tokens, unevenly spread over the experts: compute bound
        {"name": "experts 4096 of 32x2048x4096", "op": "experts", "T": 4096, "k": 4, "E": 32, "N": 2048, "K": 4096, "out": "bf16"},
        # one token through a layer of small BF16 experts: latency of the launches and of four experts' weights
        {"name": "mlp 1x2048x1408 4 of 32 bf16", "op": "mlp", "T": 1, "k": 4, "E": 32, "H": 2048, "I": 1408,
         "dtype": "bf16", "mx": False, "bias": False, "drop": 0.0},
        # 16 sequences decoding through large BF16 experts: nearly every expert's weights are read
        {"name": "mlp 16x4096x2048 4 of 32 bf16", "op": "mlp", "T": 16, "k": 4, "E": 32, "H": 4096, "I": 2048,
         "dtype": "bf16", "mx": False, "bias": False, "drop": 0.0},
        # ragged: odd widths, FP16 activations, biases, and choices dropped by padding tokens
        {"name": "mlp 7x1000x1003 2 of 8 mxfp4", "op": "mlp", "T": 7, "k": 2, "E": 8, "H": 1000, "I": 1003,
         "dtype": "fp16", "mx": True, "bias": True, "drop": 0.1},
        # 64 sequences decoding through many small experts in MXFP4, 8 of 128 each
        {"name": "mlp 64x2048x1408 8 of 128 mxfp4", "op": "mlp", "T": 64, "k": 8, "E": 128, "H": 2048, "I": 1408,
         "dtype": "bf16", "mx": True, "bias": False, "drop": 0.0},
    ]


def draw(rng):
    """One more case of the ranges above: sizes spread over their logarithms, odd ones among them."""
    def spread(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(["quantize", "gemm", "gemm", "experts", "mlp", "mlp"])
    if op == "quantize":
        M = spread(1, 4096)
        return {"op": op, "M": M, "K": spread(64, 10240, rng.choice([1, 8, 64])), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "gemm":
        M = spread(1, 4096)
        return {"op": op, "M": M, "N": spread(256, 8192, rng.choice([1, 16, 128])), "K": spread(256, 8192, rng.choice([1, 32, 128])),
                "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5}
    E = rng.choice([8, 16, 32, 64, 128])
    k = rng.choice([1, 2, 4, 8])
    if op == "experts":
        return {"op": op, "T": spread(1, 4096 // max(1, k // 4)), "k": k, "E": min(E, 64), "N": spread(256, 2048, rng.choice([1, 16, 128])),
                "K": spread(256, 4096, rng.choice([1, 32])), "out": rng.choice(["bf16", "fp16"])}
    most = 32 * 4096 * 2048 // E                                       # of H I: the weights of the largest listed case
    H = spread(256, 4096, rng.choice([1, 8, 64]))
    return {"op": op, "T": spread(1, 64), "k": k, "E": E, "H": H, "I": spread(256, max(256, min(2048, most // H)), rng.choice([1, 8, 64])),
            "dtype": rng.choice(["bf16", "bf16", "fp16"]), "mx": rng.random() < 0.5, "bias": rng.random() < 0.3,
            "drop": rng.choice([0.0, 0.05])}


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


def _round_mx(x):
    """(magnitudes on the grid [..., Kp / 32, 32], exponents [..., Kp / 32, 1]) of rows of 32-bit floats."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, (torch.frexp(top).exponent - 3).clamp_min(-127), -127)      # floor(log2) - 2
    a = torch.ldexp(blocks.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return ((a / step).round() * step).clamp_max(6.0), e, torch.signbit(blocks)


def _quantize(x):
    """Codes [..., rows, Kp / 2] and scales [..., Kp / 128, rows, 4] of rows of 32-bit floats."""
    a, e, minus = _round_mx(x)
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, 7.0)).to(torch.uint8) + 8 * minus.to(torch.uint8)
    pair = code.reshape(*x.shape[:-1], -1, 2)
    scales = (e + 127).to(torch.uint8).reshape(*x.shape[:-1], -1, 4)
    return pair[..., 0] + 16 * pair[..., 1], scales.transpose(-3, -2).contiguous()


def _weight(g, shape):
    """N(0, 1 / K) rows whose sizes differ."""
    w = torch.randn(shape, generator=g, device="cuda")
    w *= torch.exp(0.3 * torch.randn((*shape[:-1], 1), generator=g, device="cuda")) / math.sqrt(shape[-1])
    return w


def _choices(g, T, k, E, drop):
    """k different experts per token, some experts chosen more often than others; a dropped choice is -1."""
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    if drop > 0:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < drop, -1, ids)
    return ids, torch.softmax(top, dim=1)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = dict(case)
    if op == "quantize":
        st["x"] = _activations(g, case["M"], case["K"], DTYPES[case["dtype"]])
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["xq"], st["xs"] = _quantize(_activations(g, M, K, torch.float32))
        st["wq"], st["ws"] = _quantize(_weight(g, (N, K)))
        st["b"] = torch.randn((N,), generator=g, device="cuda").to(torch.bfloat16) if case["bias"] else None
    elif op == "experts":
        T, k, E, N, K = (case[c] for c in ("T", "k", "E", "N", "K"))
        ids, _ = _choices(g, T, k, E, 0.0)
        counts = (ids.reshape(-1)[:, None] == torch.arange(E, device="cuda")[None, :]).sum(0)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["xq"], st["xs"] = _quantize(_activations(g, T * k, K, torch.float32))
        st["wq"], st["ws"] = _quantize(_weight(g, (E, N, K)))
    else:
        T, k, E, H, I = (case[c] for c in ("T", "k", "E", "H", "I"))
        dtype = DTYPES[case["dtype"]]
        st["ids"], w = _choices(g, T, k, E, case["drop"])
        st["w"] = w.contiguous()
        st["x"] = torch.randn((T, H), generator=g, device="cuda").to(dtype)
        for name, shape in (("in", (E, 2 * I, H)), ("out", (E, H, I))):
            m = _weight(g, shape)
            st["w_" + name], st["s_" + name] = _quantize(m) if case["mx"] else (m.to(dtype), None)
            st["b_" + name] = (0.1 * torch.randn(shape[:2], generator=g, device="cuda")).to(torch.bfloat16) if case["bias"] else None
    return st


# ---------------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import decode_tile_interleaved_rans_amd as ep
    op = st["op"]
    if op == "quantize":
        q, s = ep.quantize_rows_mxfp4(st["x"])
        return ep.dequantize_rows_mxfp4(q, s, torch.bfloat16, columns=st["K"])
    if op == "gemm":
        return ep.gemm_mxfp4(st["xq"], st["xs"], st["wq"], st["ws"], st["b"], out_dtype=DTYPES[st["out"]])
    if op == "experts":
        return ep.gemm_mxfp4_experts(st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"], out_dtype=DTYPES[st["out"]])
    return ep.mlp_forward_experts(st["x"], st["ids"], st["w"], st["w_in"], st["w_out"], in_scales=st["s_in"],
                                  out_scales=st["s_out"], in_bias=st["b_in"], out_bias=st["b_out"])


def _values(q, s):
    """The 32-bit values of codes and scales, rows of Kp."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(q & 15).long()], grid[(q >> 4).long()]], -1)
    e = s.transpose(-3, -2).reshape(*q.shape[:-1], -1, 1).int() - 127
    return torch.ldexp(v.reshape(*q.shape[:-1], -1, 32), e).reshape(*q.shape[:-1], -1)


def _plain(st):
    op = st["op"]
    if op == "quantize":
        # every step is exact in 32 bits but the rounding itself: the scales are powers of two
        a, e, minus = _round_mx(st["x"].float())
        v = torch.ldexp(torch.where(minus, -a, a), e).reshape(st["M"], -1)
        return v[:, :st["K"]].to(torch.bfloat16)
    if op == "gemm":
        y = _values(st["xq"], st["xs"]) @ _values(st["wq"], st["ws"]).T
        if st["b"] is not None:
            y = y + st["b"].float()
        return y.to(DTYPES[st["out"]])
    if op == "experts":
        x = _values(st["xq"], st["xs"])
        y = torch.zeros((x.shape[0], st["N"]), device="cuda")
        offs = st["offsets"].tolist()
        for e in range(st["E"]):
            a, b = offs[e], offs[e + 1]
            if b > a:
                y[a:b] = x[a:b] @ _values(st["wq"][e], st["ws"][e]).T
        return y.to(DTYPES[st["out"]])
    # every token through every expert that some token chose, with weight 0 where it did not
    T, E, H, I = (st[c] for c in ("T", "E", "H", "I"))
    ids = st["ids"]
    kept = (ids >= 0) & (ids < E)
    share = torch.zeros((T, E + 1), device="cuda").scatter_add_(1, torch.where(kept, ids, E), st["w"])
    hit = torch.unique(ids[kept])
    n = hit.numel()
    weight = lambda name: _values(st["w_" + name][hit], st["s_" + name][hit]) if st["mx"] else st["w_" + name][hit].float()
    bias = lambda name: st["b_" + name][hit].float() if st["b_" + name] is not None else 0.0
    share = share[:, hit]
    a = (st["x"].float() @ weight("in")[..., :H].reshape(n * 2 * I, H).T).reshape(T, n, 2 * I) + bias("in")
    h = torch.nn.functional.silu(a[..., :I]) * a[..., I:] * share[..., None]
    y = h.reshape(T, n * I) @ weight("out")[..., :I].permute(0, 2, 1).reshape(n * I, H)
    if st["b_out"] is not None:
        y = y + share @ bias("out")
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------------------------ bytes and work
def work(case):
    """Each input read once, each output written once; the operations of the formulas."""
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    mx = 17 / 32                                                          # bytes of an element with its share of a scale
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (size[case["dtype"]] + 2), "flops": 4 * M * K}
    if op == "gemm":
        M, N, K, es = case["M"], case["N"], case["K"], size[case["out"]]
        return {"bytes": int(mx * (M + N) * K) + es * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    hit = E * (1.0 - (1.0 - k / E) ** T)                                  # experts that some token chose
    if op == "experts":
        R, N, K, es = T * k, case["N"], case["K"], size[case["out"]]
        return {"bytes": int(mx * (R * K + hit * N * K) + es * R * N), "flops": 2 * R * N * K}
    H, I = case["H"], case["I"]
    each = mx if case["mx"] else 2
    return {"bytes": int(hit * 3 * H * I * each + 4 * T * H + T * k * 12), "flops": int(6 * T * k * (1 - case["drop"]) * H * I)}


# --------------------------------------------------------------------------- the definition, 64 bits
def _magnitude(c):
    """What the three low bits of a code stand for: subnormal below 2, else one mantissa bit and an exponent."""
    m, e = (c & 1).double(), ((c >> 1) & 3).double()
    return torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e - 1.0))


def _decode(q, s):
    rows, half = q.shape
    v = torch.empty((rows, 2 * half), dtype=torch.float64, device="cuda")
    for part, c in ((0, q % 16), (1, torch.div(q, 16, rounding_mode="floor"))):
        v[:, part::2] = torch.where(c >= 8, -1.0, 1.0) * _magnitude(c)
    scale = torch.exp2(s.double() - 127.0)                                 # [Kp / 128, rows, 4]
    for chunk in range(scale.shape[0]):
        v[:, 128 * chunk:128 * (chunk + 1)] *= scale[chunk].repeat_interleave(32, dim=1)
    return v


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"].double()
        M, K = x.shape
        full = torch.zeros((M, (K + 31) // 32 * 32), dtype=torch.float64, device="cuda")
        full[:, :K] = x
        mag = full.abs().view(M, -1, 32)
        largest = mag.max(dim=2, keepdim=True).values
        unit = torch.exp2(torch.frexp(largest).exponent.double() - 3.0)
        ratio = mag / unit
        code = torch.zeros_like(ratio, dtype=torch.uint8)
        # a magnitude on a border goes to the even code: up to 2, 4 and 6, down to 0, 2, 4 and 6
        for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
            code += ((ratio >= border) if up else (ratio > border)).to(torch.uint8)
        v = _magnitude(code) * unit
        return (torch.sign(full) * v.view(M, -1))[:, :K]
    if op == "gemm":
        y = torch.mm(_decode(st["xq"], st["xs"]), _decode(st["wq"], st["ws"]).t().contiguous())
        return y if st["b"] is None else y + st["b"].double().unsqueeze(0)
    if op == "experts":
        x, edge = _decode(st["xq"], st["xs"]), st["offsets"].cpu().tolist()
        y = torch.zeros((x.shape[0], case["N"]), dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(edge[:-1], edge[1:])):
            if a < b:
                y[a:b] = torch.mm(x[a:b], _decode(st["wq"][e], st["ws"][e]).t().contiguous())
        return y
    T, k, E, H, I = (case[c] for c in ("T", "k", "E", "H", "I"))
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    ids, x = st["ids"].cpu().tolist(), st["x"].double()
    for e in range(E):
        chosen = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == e]
        if not chosen:
            continue
        if case["mx"]:
            up, down = _decode(st["w_in"][e], st["s_in"][e])[:, :H], _decode(st["w_out"][e], st["s_out"][e])[:, :I]
        else:
            up, down = st["w_in"][e].double(), st["w_out"][e].double()
        t = torch.tensor([c[0] for c in chosen], device="cuda")
        j = torch.tensor([c[1] for c in chosen], device="cuda")
        a = torch.mm(x[t], up.t().contiguous())
        if case["bias"]:
            a += st["b_in"][e].double()
        gate, lin = a[:, :I], a[:, I:]
        out = torch.mm(gate / (1.0 + torch.exp(-gate)) * lin, down.t().contiguous())
        if case["bias"]:
            out += st["b_out"][e].double()
        y.index_add_(0, t, st["w"].double()[t, j][:, None] * out)
    return y
