"""MI355X (gfx950) tile-rANS weight codec: Python binding of ``libentropack.so``.

The functions mirror the C ABI in ``include/entropack.h`` and only marshal arguments: the host
encoder, the stream validator and every GPU step run in the compiled library. PyTorch provides
device memory and the current HIP stream. There is no fallback path: if the library is missing,
every call raises.

    stream, bpp = compress(weight, target_bpp=4.0)       # host encoder
    w_hat = decompress(stream, torch.bfloat16)           # GPU decode into a container
    layer = CompressedLinear.from_linear(linear, 4.0)    # fused decode + BF16 MFMA GEMM
"""
from __future__ import annotations

import ctypes as C
import functools
import os

import numpy as np

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libentropack.so")

F32, BF16, F16, F8E4M3, I8, U8 = 0, 1, 2, 3, 4, 5
# Probability precision of the streams CompressedLinear.from_linear codes: with 2^11-slot tables
# (64 KiB in LDS instead of 96 KiB) the fused decode + MFMA forward runs 12 waves per CU instead of
# 8; the stream is about 1% larger and the plain decode runs at the same speed.
LAYER_PROB_BITS = 11
LOSSY, LOSSLESS, LOSSLESS_EXP = 0, 1, 2
# Lossy tile layouts (ep_encode_opts.layout): ROW_LAYOUT keeps each of a tile's 32 rANS states on
# one tile row, so that every block step of a 16-row tile pair yields a 16 x 32 weight block, the B
# operand of one BF16 MFMA, in the decoder's own registers.
BLOCK_ROW_LAYOUT, ROW_LAYOUT = 0, 1
# Tile layout of the streams CompressedLinear.from_linear codes: the row layout, whose forward for
# up to 64 activation rows multiplies the weight straight from the decoder's registers (at 8192 x
# 8192, 4.5 bpp: 80 us for M = 16 against 121 us in layout 0); a plain decode of it (the forward
# above 64 rows) takes about 10% longer.
LAYER_LAYOUT = ROW_LAYOUT
STATUS = {0: "EP_OK", -1: "EP_EINVAL", -2: "EP_ECORRUPT", -3: "EP_EUNSUPPORTED", -4: "EP_ERANGE",
          -5: "EP_EHIP", -6: "EP_ENOMEM", -7: "EP_EDEVICE"}
EXPORTS = ["ep_compress", "ep_free", "ep_stream_info", "ep_upload", "ep_handle_info", "ep_decompress",
           "ep_decompress_many", "ep_decode_symbols", "ep_linear_forward", "ep_gemm_bf16", "ep_handle_check",
           "ep_release", "ep_last_error", "ep_version", "ep_linear_forward_fp8", "ep_quantize_rows_fp8",
           "ep_gemm_fp8", "ep_compress_device", "ep_linear_forward_noalloc", "ep_linear_forward_many",
           "ep_linear_forward_fp8_many", "ep_quantize_rows_int8", "ep_gemm_int8", "ep_gemm_int8_experts",
           "ep_pad_rows_int8", "ep_linear_forward_int8", "ep_linear_forward_int8_many",
           "ep_linear_forward_experts", "ep_sort_tokens_scratch", "ep_sort_tokens",
           "ep_combine_tokens", "ep_combine_tokens_grad", "ep_quantize_rows_mxfp4", "ep_dequantize_rows_mxfp4",
           "ep_gemm_mxfp4", "ep_gemm_mxfp4_experts", "ep_mlp_forward_experts_scratch", "ep_mlp_forward_experts"]


class EPError(RuntimeError):
    def __init__(self, status: int, call: str, msg: str):
        super().__init__(f"{call}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class EncodeOpts(C.Structure):
    _fields_ = [("mode", C.c_int), ("target_bpp", C.c_double), ("prob_bits", C.c_int), ("tile_rows", C.c_int),
                ("n_threads", C.c_int), ("layout", C.c_int)]


class Info(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("mode", C.c_int32), ("src_dtype", C.c_int32),
                ("tile_rows", C.c_int32), ("prob_bits", C.c_int32), ("n_tiles", C.c_uint32),
                ("n_escapes", C.c_uint32), ("step", C.c_float), ("target_bpp", C.c_float),
                ("actual_bpp", C.c_double), ("total_bytes", C.c_uint64), ("payload_bytes", C.c_uint64),
                ("state_bytes", C.c_uint64), ("meta_bytes", C.c_uint64), ("layout", C.c_int32)]

    def as_dict(self) -> dict:
        return {k: getattr(self, k) for k, _ in self._fields_}


_lib = None


def lib() -> C.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m decode_tile_interleaved_rans_amd.build")
        L = C.CDLL(LIB_PATH)
        vp, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
        L.ep_compress.argtypes = [vp, C.c_int, i64, i64, C.POINTER(EncodeOpts), C.POINTER(C.POINTER(C.c_uint8)),
                                  C.POINTER(sz), C.POINTER(C.c_double)]
        L.ep_compress_device.argtypes = [vp, C.c_int, i64, i64, C.POINTER(EncodeOpts), vp,
                                         C.POINTER(C.POINTER(C.c_uint8)), C.POINTER(sz), C.POINTER(C.c_double)]
        L.ep_free.argtypes = [vp]
        L.ep_free.restype = None
        L.ep_stream_info.argtypes = [C.c_char_p, sz, C.POINTER(Info)]
        L.ep_upload.argtypes = [C.c_char_p, sz, vp, C.POINTER(vp)]
        L.ep_handle_info.argtypes = [vp, C.POINTER(Info)]
        L.ep_decompress.argtypes = [vp, C.c_int, vp, vp, vp]
        L.ep_decompress_many.argtypes = [vp, vp, vp, vp, C.c_int, vp]
        L.ep_decode_symbols.argtypes = [vp, vp, vp]
        L.ep_linear_forward.argtypes = [vp, vp, i64, vp, vp, vp]
        L.ep_linear_forward_noalloc.argtypes = [vp, vp, i64, vp, vp, vp]
        L.ep_linear_forward_many.argtypes = [vp, C.c_int, vp, i64, vp, vp, vp]
        L.ep_linear_forward_fp8_many.argtypes = [vp, C.c_int, vp, i64, vp, vp, vp]
        L.ep_gemm_bf16.argtypes = [vp, vp, i64, i64, i64, vp, vp]
        L.ep_linear_forward_fp8.argtypes = [vp, vp, i64, vp, vp, vp]
        L.ep_quantize_rows_fp8.argtypes = [vp, i64, i64, vp, vp, vp]
        L.ep_gemm_fp8.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp]
        L.ep_quantize_rows_int8.argtypes = [vp, C.c_int, i64, i64, i64, vp, vp, vp]
        L.ep_gemm_int8.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, C.c_int, vp, vp]
        L.ep_gemm_int8_experts.argtypes = [vp, vp, vp, vp, vp, C.c_int, i64, i64, i64, vp, C.c_int, vp, vp]
        L.ep_pad_rows_int8.argtypes = [vp, i64, i64, vp, i64, vp]
        L.ep_linear_forward_int8.argtypes = [vp, vp, i64, vp, vp, vp]
        L.ep_linear_forward_int8_many.argtypes = [vp, C.c_int, vp, i64, vp, vp, vp]
        L.ep_linear_forward_experts.argtypes = [vp, C.c_int, C.c_int, vp, vp, vp, vp, vp, vp]
        L.ep_sort_tokens_scratch.argtypes = [i64, C.c_int, C.c_int, C.POINTER(sz)]
        L.ep_sort_tokens.argtypes = [vp, C.c_int, i64, i64, i64, vp, C.c_int, C.c_int, C.c_int, vp, vp, vp, vp, vp]
        L.ep_combine_tokens.argtypes = [vp, C.c_int, vp, vp, i64, C.c_int, i64, i64, vp, vp]
        L.ep_combine_tokens_grad.argtypes = [vp, C.c_int, vp, vp, vp, i64, C.c_int, i64, i64, vp, vp, vp]
        L.ep_quantize_rows_mxfp4.argtypes = [vp, C.c_int, i64, i64, i64, i64, vp, vp, vp]
        L.ep_dequantize_rows_mxfp4.argtypes = [vp, vp, i64, i64, i64, i64, C.c_int, vp, vp]
        L.ep_gemm_mxfp4.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, C.c_int, vp, vp]
        L.ep_gemm_mxfp4_experts.argtypes = [vp, vp, vp, vp, vp, C.c_int, i64, i64, i64, vp, C.c_int, vp, vp]
        L.ep_mlp_forward_experts_scratch.argtypes = [i64, C.c_int, C.c_int, i64, i64, C.c_int, C.POINTER(sz)]
        L.ep_mlp_forward_experts.argtypes = [vp, C.c_int, i64, i64, i64, vp, C.c_int, C.c_int, C.c_int, vp, vp, vp, vp, vp, vp, vp, i64,
                                             i64, vp, vp, vp]
        L.ep_handle_check.argtypes = [vp, vp]
        L.ep_release.argtypes = [vp]
        L.ep_release.restype = None
        L.ep_last_error.restype = C.c_char_p
        L.ep_version.restype = C.c_char_p
        for name in EXPORTS:
            if name not in ("ep_free", "ep_release", "ep_last_error", "ep_version"):
                getattr(L, name).restype = C.c_int
        _lib = L
    return _lib


def _check(rc: int, call: str):
    if rc != 0:
        raise EPError(rc, call, lib().ep_last_error().decode(errors="replace"))


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_DT_OF_TORCH = None


def _dtype_code(t) -> int:
    global _DT_OF_TORCH
    if _DT_OF_TORCH is None:
        torch = _torch()
        _DT_OF_TORCH = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: F8E4M3,
                        torch.int8: I8, torch.uint8: U8}
    if t not in _DT_OF_TORCH:
        raise ValueError(f"unsupported dtype {t}")
    return _DT_OF_TORCH[t]


def _torch_dtype(code: int):
    torch = _torch()
    return {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16, F8E4M3: torch.float8_e4m3fn,
            I8: torch.int8, U8: torch.uint8}[code]


def _stream_ptr(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _run_on(stream):
    """(s, other) for a call that runs on `stream` (default: the current stream). With another
    stream, s first waits for the work queued on the current stream (which produced the inputs);
    the caller allocates its outputs under torch.cuda.stream(s) and, after the call, marks the
    input tensors as used on s (_used_on), so that the caching allocator does not hand their
    memory to other work while s may still read them."""
    torch = _torch()
    cur = torch.cuda.current_stream()
    s = stream if stream is not None else cur
    other = s.cuda_stream != cur.cuda_stream
    if other:
        s.wait_stream(cur)
    return s, other


def _used_on(s, other, *tensors):
    if other:
        for t in tensors:
            if t is not None:
                t.record_stream(s)


# ------------------------------------------------------------------------------------ host side
def compress(w, target_bpp: float = 4.0, *, mode: int = LOSSY, prob_bits: int = 12, tile_rows: int = 16,
             n_threads: int = 0, dtype: int | None = None, layout: int = 0) -> tuple[bytes, float]:
    """Compress a 2-D weight (torch tensor on any device, or numpy array) on the host.
    Returns (stream bytes, actual bits per weight including every byte of metadata).
    layout (lossy only; ep_encode_opts.layout): 0 codes each tile row by row, 1 keeps every rANS
    state on one tile row (ROW_LAYOUT), which the compressed linear forward multiplies straight
    from the decoder's registers; both decode to the same weights."""
    if hasattr(w, "detach"):
        torch = _torch()
        code = _dtype_code(w.dtype)
        t = w.detach().contiguous().cpu()
        view = t.view(torch.int16) if t.element_size() == 2 else (t.view(torch.uint8) if t.element_size() == 1 else t)
        arr = view.numpy()
    else:
        arr = np.ascontiguousarray(w)
        code = dtype if dtype is not None else {np.dtype(np.float32): F32, np.dtype(np.uint8): U8}.get(arr.dtype)
        if code is None:
            raise ValueError("numpy inputs other than float32/uint8 need dtype= (16-bit data as uint16 bits)")
    if arr.ndim != 2:
        raise ValueError("compress takes a 2-D [out_features, in_features] matrix")
    R, Cc = arr.shape
    opts = EncodeOpts(mode, float(target_bpp), prob_bits, tile_rows, n_threads, layout)
    out = C.POINTER(C.c_uint8)()
    n = C.c_size_t()
    bpp = C.c_double()
    _check(lib().ep_compress(arr.ctypes.data_as(C.c_void_p), code, R, Cc, C.byref(opts), C.byref(out), C.byref(n),
                             C.byref(bpp)), "ep_compress")
    data = C.string_at(out, n.value)
    lib().ep_free(out)
    return data, bpp.value


def compress_device(w, target_bpp: float = 4.0, *, prob_bits: int = 12, tile_rows: int = 16,
                    stream=None, layout: int = 0) -> tuple[bytes, float]:
    """Lossy compression on the GPU of a 2-D weight in device memory (torch tensor: float32,
    bfloat16 or float16); the same bytes as compress() on the same values."""
    if w.dim() != 2:
        raise ValueError("compress_device takes a 2-D [out_features, in_features] matrix")
    t = w.detach().contiguous()
    if not t.is_cuda:
        raise ValueError("compress_device takes a tensor in device memory")
    _need(t, "w", t.dtype)
    R, Cc = t.shape
    opts = EncodeOpts(LOSSY, float(target_bpp), prob_bits, tile_rows, 0, layout)
    out = C.POINTER(C.c_uint8)()
    n = C.c_size_t()
    bpp = C.c_double()
    _check(lib().ep_compress_device(C.c_void_p(t.data_ptr()), _dtype_code(t.dtype), R, Cc, C.byref(opts),
                                    _stream_ptr(stream), C.byref(out), C.byref(n), C.byref(bpp)), "ep_compress_device")
    data = C.string_at(out, n.value)
    lib().ep_free(out)
    return data, bpp.value


def lossless_compress(w, *, exponent_coded: bool = False, **kw) -> tuple[bytes, float]:
    """Bit-exact compression. exponent_coded=True (BF16 only) codes the exponent byte with the
    tile rANS and keeps sign and mantissa as uncoded bytes; otherwise every byte plane is coded."""
    return compress(w, 0.0, mode=LOSSLESS_EXP if exponent_coded else LOSSLESS, **kw)


def stream_info(stream: bytes) -> dict:
    info = Info()
    _check(lib().ep_stream_info(stream, len(stream), C.byref(info)), "ep_stream_info")
    return info.as_dict()


def save(path, stream: bytes, bias=None) -> None:
    """Write a stream (and an optional bias vector) to a file. The stream is the whole artifact:
    it is self-describing and versioned, and holds everything the decoder needs ("EntroPack
    PyTorch Guide", sections "Test saved artifacts" and "Diagnose the common failure cases").
    The file is a numpy .npz archive without pickled objects."""
    import numpy as np
    arrays = {"stream": np.frombuffer(stream, np.uint8)}
    if bias is not None:
        if isinstance(bias, np.ndarray):                 # BF16 bit patterns
            arrays["bias_bf16"] = np.asarray(bias, np.uint16)
        else:                                            # a torch tensor of any float dtype
            torch = _torch()
            b = bias.detach().to("cpu", torch.bfloat16).contiguous()
            arrays["bias_bf16"] = b.view(torch.int16).numpy().view(np.uint16)
    with open(path, "wb") as f:
        np.savez(f, **arrays)


def load(path):
    """Read a file written by save(): returns (stream bytes, bias bf16 bits as uint16 or None).
    The stream is validated before it is returned."""
    import numpy as np
    with np.load(path, allow_pickle=False) as z:
        stream = z["stream"].tobytes()
        bias = z["bias_bf16"].copy() if "bias_bf16" in z.files else None
    stream_info(stream)
    return stream, bias


def _need(t, name: str, dtype, shape=None, min_numel: int | None = None):
    """Argument check before a device pointer crosses the C ABI: the kernels trust sizes, so a
    tensor of the wrong shape, dtype, layout or device would be read or written out of bounds."""
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous tensor on the GPU")
    if t.device.index != _torch().cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_torch().cuda.current_device()}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} needs at least {min_numel} elements")


# ------------------------------------------------------------------------------------ device side
class Handle:
    """A validated stream resident on the current GPU."""

    def __init__(self, stream: bytes, hip_stream=None):
        self._h = C.c_void_p()
        _check(lib().ep_upload(stream, len(stream), _stream_ptr(hip_stream), C.byref(self._h)), "ep_upload")
        info = Info()
        _check(lib().ep_handle_info(self._h, C.byref(info)), "ep_handle_info")
        self.info = info.as_dict()
        self.shape = (self.info["rows"], self.info["cols"])

    @property
    def ptr(self):
        return self._h

    def decompress_into(self, out, row_scale=None, stream=None):
        torch = _torch()
        code = _dtype_code(out.dtype) if out.dtype != torch.int16 else None
        if code is None:
            raise ValueError("use decode_symbols_into for int16 outputs")
        if tuple(out.shape) != self.shape or not out.is_contiguous() or not out.is_cuda:
            raise ValueError(f"output must be a contiguous CUDA tensor of shape {self.shape}")
        if row_scale is not None:
            _need(row_scale, "row_scale", torch.float32, min_numel=self.shape[0])
        sp = C.c_void_p(row_scale.data_ptr()) if row_scale is not None else None
        _check(lib().ep_decompress(self._h, code, C.c_void_p(out.data_ptr()), sp, _stream_ptr(stream)),
               "ep_decompress")
        return out

    def decompress(self, dtype=None, stream=None):
        """Decode into a new tensor. FP8 / INT8 return (values, per-row fp32 scale). The outputs
        are allocated on the stream the decode runs on."""
        torch = _torch()
        if dtype is None:
            dtype = _torch_dtype(self.info["src_dtype"]) if self.info["mode"] != LOSSY else torch.bfloat16
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            out = torch.empty(self.shape, dtype=dtype, device="cuda")
            scale = None
            if self.info["mode"] == LOSSY and dtype in (torch.float8_e4m3fn, torch.int8):
                scale = torch.empty(self.shape[0], dtype=torch.float32, device="cuda")
            self.decompress_into(out, scale, s)
        return (out, scale) if scale is not None else out

    def decode_symbols(self, stream=None):
        """Decode the lattice symbols into a new int16 tensor, allocated on the stream the decode
        runs on."""
        torch = _torch()
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            q = torch.empty(self.shape, dtype=torch.int16, device="cuda")
        _check(lib().ep_decode_symbols(self._h, C.c_void_p(q.data_ptr()), C.c_void_p(s.cuda_stream)),
               "ep_decode_symbols")
        return q

    def check(self, stream=None):
        _check(lib().ep_handle_check(self._h, _stream_ptr(stream)), "ep_handle_check")

    def release(self):
        if self._h:
            lib().ep_release(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.release()
        except Exception:
            pass


def upload(stream: bytes, hip_stream=None) -> Handle:
    return Handle(stream, hip_stream)


def decompress(stream: bytes, dtype=None, device: str = "cuda"):
    """Decode a stream on the GPU ("decompress(stream) returns a tensor")."""
    h = Handle(stream)
    try:
        return h.decompress(dtype)
    finally:
        _torch().cuda.current_stream().synchronize()
        h.release()


def decompress_many(handles, outs, scales=None, stream=None):
    """One grouped call over several uploaded matrices."""
    torch = _torch()
    n = len(handles)
    if len(outs) != n or (scales is not None and len(scales) != n):
        raise ValueError("handles, outs and scales must have the same length")
    for i, (h, o) in enumerate(zip(handles, outs)):
        _need(o, f"outs[{i}]", o.dtype, shape=h.shape)
        if scales is not None and scales[i] is not None:
            _need(scales[i], f"scales[{i}]", torch.float32, min_numel=h.shape[0])
    hs = (C.c_void_p * n)(*[h.ptr.value for h in handles])
    cts = (C.c_int * n)(*[_dtype_code(o.dtype) for o in outs])
    os_ = (C.c_void_p * n)(*[o.data_ptr() for o in outs])
    sc = (C.c_void_p * n)(*[(s.data_ptr() if s is not None else None) for s in (scales or [None] * n)])
    _check(lib().ep_decompress_many(hs, cts, os_, sc, n, _stream_ptr(stream)), "ep_decompress_many")


def gemm_bf16(x, w, stream=None):
    """Y = X W^T in BF16 with fp32 accumulation (the library's own MFMA GEMM), on `stream`
    (default: the current stream; another stream first waits for the current one)."""
    torch = _torch()
    M, K = x.shape
    N = w.shape[0]
    _need(x, "x", torch.bfloat16)
    _need(w, "w", torch.bfloat16, shape=(N, K))
    s, other = _run_on(stream)
    with torch.cuda.stream(s):
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(lib().ep_gemm_bf16(C.c_void_p(x.data_ptr()), C.c_void_p(w.data_ptr()), M, N, K, C.c_void_p(y.data_ptr()),
                              C.c_void_p(s.cuda_stream)), "ep_gemm_bf16")
    _used_on(s, other, x, w)
    return y


def quantize_rows_fp8(x, stream=None):
    """Per-row FP8 E4M3 codes of BF16 rows and their fp32 scales (x = codes * scale[row]), on
    `stream` (default: the current stream; another stream first waits for the current one)."""
    torch = _torch()
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    s, other = _run_on(stream)
    with torch.cuda.stream(s):
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        sc = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib().ep_quantize_rows_fp8(C.c_void_p(x.data_ptr()), M, K, C.c_void_p(q.data_ptr()),
                                      C.c_void_p(sc.data_ptr()), C.c_void_p(s.cuda_stream)), "ep_quantize_rows_fp8")
    _used_on(s, other, x)
    return q, sc


def gemm_fp8(xq, xs, wq, ws, bias=None, stream=None):
    """Y = diag(xs) Xq Wq^T diag(ws) (+ bias) from E4M3 codes (uint8 tensors), BF16 output, on
    `stream` (default: the current stream; another stream first waits for the current one)."""
    torch = _torch()
    M, K = xq.shape
    N = wq.shape[0]
    _need(xq, "xq", torch.uint8)
    _need(wq, "wq", torch.uint8, shape=(N, K))
    _need(xs, "xs", torch.float32, shape=(M,))
    _need(ws, "ws", torch.float32, shape=(N,))
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, shape=(N,))
    s, other = _run_on(stream)
    with torch.cuda.stream(s):
        y = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    bp = C.c_void_p(bias.data_ptr()) if bias is not None else None
    _check(lib().ep_gemm_fp8(C.c_void_p(xq.data_ptr()), C.c_void_p(xs.data_ptr()), C.c_void_p(wq.data_ptr()),
                             C.c_void_p(ws.data_ptr()), M, N, K, bp, C.c_void_p(y.data_ptr()), C.c_void_p(s.cuda_stream)),
           "ep_gemm_fp8")
    _used_on(s, other, xq, xs, wq, ws, bias)
    return y


def _need_rows(t, name: str, dtypes):
    """_need for a 2-D matrix whose rows may be further apart than they are long."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    apart = t.stride(0) if rows > 1 and cols > 0 else cols
    if not t.is_cuda or (t.numel() > 0 and ((cols > 1 and t.stride(1) != 1) or apart < cols)):
        raise ValueError(f"{name} must be on the GPU, its elements consecutive within a row and its rows disjoint")
    if t.device.index != _torch().cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_torch().cuda.current_device()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {t.dtype}")
    return rows, cols, apart


def _fits(t, dtype, shape, device: int) -> bool:
    """Whether _need(t, ..., dtype, shape) passes, for `device` the current one: one quick test, so that a
    small call does not spend its time on checks; where it fails, _need says why."""
    return t.is_cuda and t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()


def _on_stream(stream, call, *tensors):
    """call() with `stream` current, ordered as _run_on and _used_on order it. The calls below run on
    the current stream without a stream object or context of their own, which would cost a small
    call more time (9 us) than its kernel takes."""
    s, other = _run_on(stream)
    _used_on(s, other, *tensors)
    with _torch().cuda.stream(s):
        return call()


def _current_raw():
    """The current stream of the current device, as the C ABI takes it."""
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t):
    return None if t is None else t.data_ptr()


_FLOAT_TYPES = None


def _float_types():
    global _FLOAT_TYPES
    if _FLOAT_TYPES is None:
        torch = _torch()
        _FLOAT_TYPES = torch.bfloat16, torch.float16, torch.float32
    return _FLOAT_TYPES


def quantize_rows_int8(x, stream=None):
    """Per-row INT8 codes of BF16, FP16 or FP32 rows [M, K] (rows may be further apart than K) and their
    fp32 scales: scale = max |x| / 127, codes = x / scale rounded to nearest even, exactly. A row with an
    infinity or a NaN gets codes 0 and scale NaN. On `stream` (default: the current stream; another
    stream first waits for the current one)."""
    if stream is not None:
        return _on_stream(stream, lambda: quantize_rows_int8(x), x)
    torch = _torch()
    M, K, ldx = _need_rows(x, "x", _float_types())
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    sc = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib().ep_quantize_rows_int8(_ptr(x), _dtype_code(x.dtype), M, K, ldx, _ptr(q), _ptr(sc), _current_raw()),
           "ep_quantize_rows_int8")
    return q, sc


def pad_rows_int8(codes, stream=None):
    """INT8 codes [..., K] in new memory with K rounded up to a multiple of 16 (of 128 from 1024 to
    130944: whole cache lines), zeros behind: the layout the INT8 products read. They call this for
    codes that lack it; a program with such a weight lays it out once and keeps it (and pads the
    activations' codes to the same width)."""
    if stream is not None:
        return _on_stream(stream, lambda: pad_rows_int8(codes), codes)
    torch = _torch()
    _need(codes, "codes", torch.int8)
    if codes.dim() < 1:
        raise ValueError("codes must have rows")
    K = codes.shape[-1]
    # rows that begin inside a 128-byte line cost the product's loads two lines a piece: 333 x 5003 from
    # rows of 3856 codes 22.8 us, of 3968 17.6
    step = 128 if 1024 <= K <= 130944 else 16
    return _lay_out(codes, (K + step - 1) // step * step)


def _lay_out(codes, ld: int):
    """Contiguous codes [..., K] in new memory, 16-byte aligned, in rows of ld >= K codes."""
    K = codes.shape[-1]
    out = _torch().empty((*codes.shape[:-1], ld), dtype=codes.dtype, device=codes.device)
    _check(lib().ep_pad_rows_int8(_ptr(codes), codes.numel() // K if K else 0, K, _ptr(out), ld, _current_raw()),
           "ep_pad_rows_int8")
    return out


_I8_MAX_K = 131056                   # the widest codes whose sums stay within int32 however they are laid out


def _gemm_int8(xq, xs, wq, ws, offsets, bias, out_dtype):
    torch = _torch()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in _float_types():
        raise ValueError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
    if xq.dim() != 2 or wq.dim() != (2 if offsets is None else 3):
        raise ValueError("xq must be [rows, K] and wq " + ("[N, K]" if offsets is None else "[experts, N, K]"))
    M, K = xq.shape
    lead = tuple(wq.shape[:-1])
    args = [("xq", xq, torch.int8, (M, K)), ("wq", wq, torch.int8, (*lead, K)), ("xs", xs, torch.float32, (M,)),
            ("ws", ws, torch.float32, lead)]
    if bias is not None:
        args.append(("bias", bias, torch.bfloat16, lead))
    if offsets is not None:
        args.append(("offsets", offsets, torch.int32, (lead[0] + 1,)))
    dev = torch.cuda.current_device() if xq.is_cuda else -1
    for name, t, dtype, shape in args:
        if not _fits(t, dtype, shape, dev):
            _need(t, name, dtype, shape=shape)
    # wider codes than the products take are refused below, not copied first
    if K % 16 and K <= _I8_MAX_K:
        xq, wq = pad_rows_int8(xq), pad_rows_int8(wq)
        K = xq.shape[1]
    elif K <= _I8_MAX_K:
        # a weight is read in place whatever the activations' address, and the other way round
        xq = _lay_out(xq, K) if xq.data_ptr() % 16 else xq
        wq = _lay_out(wq, K) if wq.data_ptr() % 16 else wq
    y = torch.empty((M, lead[-1]), dtype=out_dtype, device=xq.device)
    tail = (_ptr(bias), _dtype_code(out_dtype), _ptr(y), _current_raw())
    if offsets is None:
        _check(lib().ep_gemm_int8(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), M, lead[-1], K, *tail), "ep_gemm_int8")
    else:
        _check(lib().ep_gemm_int8_experts(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(offsets), lead[0], M, lead[-1], K,
                                          *tail), "ep_gemm_int8_experts")
    return y


def gemm_int8(xq, xs, wq, ws, bias=None, out_dtype=None, stream=None):
    """Y = diag(xs) Xq Wq^T diag(ws) (+ bias) from INT8 codes xq [M, K] and wq [N, K] with a scale per
    token xs [M] and per channel ws [N] (quantize_rows_int8; a weight's codes and scales come from
    Handle.decompress(torch.int8)); exact int32 sums, output BF16 (default), FP16 or FP32. K a multiple
    of 16 and 16-byte aligned codes are read in place; other widths of both operands, and an operand at
    another address, are laid out first (pad_rows_int8). K is at most 131056. On `stream` (default: the current stream; another stream first waits for the current one)."""
    if stream is not None:
        return _on_stream(stream, lambda: _gemm_int8(xq, xs, wq, ws, None, bias, out_dtype), xq, xs, wq, ws, bias)
    return _gemm_int8(xq, xs, wq, ws, None, bias, out_dtype)


def gemm_int8_experts(xq, xs, wq, ws, offsets, bias=None, out_dtype=None, stream=None):
    """gemm_int8 with a weight per expert, in one launch: rows offsets[e] ... offsets[e + 1] - 1 of xq
    [R, K] meet wq[e] ([experts, N, K], scales ws and bias [experts, N]); rows behind the last expert's
    come out zero. offsets: int32 on the GPU, as sort_tokens gives them (ascending from 0, at most R;
    they are not read on the host)."""
    if stream is not None:
        return _on_stream(stream, lambda: _gemm_int8(xq, xs, wq, ws, offsets, bias, out_dtype),
                          xq, xs, wq, ws, offsets, bias)
    return _gemm_int8(xq, xs, wq, ws, offsets, bias, out_dtype)


# ------------------------------------------------------------------------------------ MXFP4
def quantize_rows_mxfp4(x, stream=None):
    """MXFP4 codes and scales of BF16, FP16 or FP32 rows: x [M, K] (rows may be further apart than K) or, for
    the experts' weights, contiguous [E, M, K]. Blocks of 32 elements of a row share a scale 2^(b - 127), b = max(0,
    floor(log2 max |x|) + 125); codes are x / scale rounded to nearest, ties to even, to 0, 0.5, 1, 1.5, 2, 3, 4
    or 6 with a sign (a block whose largest magnitude is above 6 scale units saturates there). A block with an
    infinity or a NaN gets b = 255 and codes 0, and products with it are NaN.

    Returns (codes, scales), uint8, with Kp the width rounded up to whole 128 elements, zeros behind: codes [..., M,
    Kp / 2], two to a byte, the even element in the low half; scales [..., Kp / 128, M, 4], the bytes b of a row's 128
    elements side by side. Row-major scales s [M, Kp / 32] from elsewhere are
    s.view(M, -1, 4).transpose(0, 1).contiguous(). It has no gradient: an x that asks for one is refused (detach it).
    On `stream` (default: the current stream; another stream first waits for the current one)."""
    if stream is not None:
        return _on_stream(stream, lambda: quantize_rows_mxfp4(x), x)
    torch = _torch()
    _no_gradient("the MXFP4 quantizer has", x)
    dims, dtype, dev = x.dim(), x.dtype, torch.cuda.current_device() if x.is_cuda else None
    if dims == 2:
        M, K = rows, ldx = x.shape
        if not (dtype in _float_types() and x.get_device() == dev and x.is_contiguous()):
            rows, _, ldx = _need_rows(x, "x", _float_types())
    elif dims == 3:
        E, M, K = x.shape
        rows, ldx = E * M, K
        if dtype not in _float_types():
            raise ValueError(f"x must be one of {', '.join(map(str, _float_types()))}, got {dtype}")
        _need(x, "x", dtype)
    else:
        raise ValueError(f"x must be [M, K] or [E, M, K], got shape {tuple(x.shape)}")
    u8, chunks = torch.uint8, (K + 127) // 128
    q = x.new_empty((M, 64 * chunks) if dims == 2 else (E, M, 64 * chunks), dtype=u8)
    s = x.new_empty((chunks, M, 4) if dims == 2 else (E, chunks, M, 4), dtype=u8)
    _check(lib().ep_quantize_rows_mxfp4(x.data_ptr(), _dtype_code(dtype), rows, M, K, ldx, q.data_ptr(), s.data_ptr(),
                                        torch._C._cuda_getCurrentRawStream(dev)), "ep_quantize_rows_mxfp4")
    return q, s


def _mx_shapes(q, s, qname: str, sname: str, dims: int, dev):
    """Checks of MXFP4 codes and scales of `dims` dimensions on the current device `dev` (None: the codes are not
    on a GPU); their padded width. One quick test, as in _fits; where it fails, the reason is looked for."""
    u8, shape = _torch().uint8, q.shape
    half = shape[-1] if len(shape) == dims else 1
    if dims == 2:
        want = (half >> 6, shape[0], 4) if half != 1 else ()
    else:
        want = (shape[0], half >> 6, shape[1], 4) if half != 1 else ()
    if not (half % 64 == 0 and s.shape == want and q.dtype is u8 and s.dtype is u8 and q.get_device() == dev == s.get_device()
            and q.is_contiguous() and s.is_contiguous()):
        if half % 64:
            raise ValueError(f"{qname} must be codes {'[rows, Kp / 2]' if dims == 2 else '[experts, rows, Kp / 2]'}, Kp a multiple of "
                             f"128, got shape {tuple(shape)}")
        _need(q, qname, u8)
        _need(s, sname, u8, shape=want)
    return 2 * half


def dequantize_rows_mxfp4(codes, scales, out_dtype=None, columns=None, stream=None):
    """The values of MXFP4 codes and scales (quantize_rows_mxfp4's, of a matrix or of the experts' matrices) as
    [..., M, columns] in BF16 (default), FP16 or FP32; columns: how many of the Kp padded columns (default: all).
    Exact in BF16 and FP32 for scale bytes up to 252, rounded to nearest even in FP16. On `stream` (default: the
    current stream; another stream first waits for the current one)."""
    if stream is not None:
        return _on_stream(stream, lambda: dequantize_rows_mxfp4(codes, scales, out_dtype, columns), codes, scales)
    torch = _torch()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in _float_types():
        raise ValueError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
    shape, dims = codes.shape, codes.dim()
    if dims not in (2, 3):
        raise ValueError(f"codes must be [M, Kp / 2] or [E, M, Kp / 2], got shape {tuple(shape)}")
    dev = torch.cuda.current_device() if codes.is_cuda else None
    Kp = _mx_shapes(codes, scales, "codes", "scales", dims, dev)
    K = Kp if columns is None else columns
    if not 0 <= K <= Kp:
        raise ValueError(f"columns must be 0 ... {Kp}, got {columns}")
    M = shape[-2]
    y = codes.new_empty((M, K) if dims == 2 else (shape[0], M, K), dtype=out_dtype)
    codes, scales = _mx_aligned(codes, 4), _mx_aligned(scales, 4)
    _check(lib().ep_dequantize_rows_mxfp4(codes.data_ptr(), scales.data_ptr(), M if dims == 2 else M * shape[0], M, Kp, K,
                                          _dtype_code(out_dtype), y.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)),
           "ep_dequantize_rows_mxfp4")
    return y


def _mx_aligned(t, to: int):
    """t, or where its address is no multiple of `to` a copy."""
    return t.clone() if t.data_ptr() % to else t


def _gemm_mxfp4(xq, xs, wq, ws, offsets, bias, out_dtype):
    torch = _torch()
    if bias is not None:
        _no_gradient("the MXFP4 product has", bias)
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in _float_types():
        raise ValueError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
    dev = torch.cuda.current_device() if xq.is_cuda else None
    K = _mx_shapes(xq, xs, "xq", "xs", 2, dev)
    if _mx_shapes(wq, ws, "wq", "ws", 2 if offsets is None else 3, dev) != K:
        raise ValueError(f"xq and wq must have the same width, got {K} and {2 * wq.shape[-1]}")
    M, lead = xq.shape[0], wq.shape[:-1]
    N = lead[-1]
    if bias is not None and not _fits(bias, torch.bfloat16, lead, dev):
        _need(bias, "bias", torch.bfloat16, shape=lead)
    if offsets is not None and not _fits(offsets, torch.int32, (lead[0] + 1,), dev):
        _need(offsets, "offsets", torch.int32, shape=(lead[0] + 1,))
    # codes are read in pieces of 16 bytes, scales in pieces of 4
    xp, wp, xsp, wsp = xq.data_ptr(), wq.data_ptr(), xs.data_ptr(), ws.data_ptr()
    if (xp | wp) & 15 or (xsp | wsp) & 3:
        xq, wq, xs, ws = _mx_aligned(xq, 16), _mx_aligned(wq, 16), _mx_aligned(xs, 4), _mx_aligned(ws, 4)
        xp, wp, xsp, wsp = xq.data_ptr(), wq.data_ptr(), xs.data_ptr(), ws.data_ptr()
    y = xq.new_empty((M, N), dtype=out_dtype)
    tail = (_ptr(bias), _dtype_code(out_dtype), y.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    if offsets is None:
        _check(lib().ep_gemm_mxfp4(xp, xsp, wp, wsp, M, N, K, *tail), "ep_gemm_mxfp4")
    else:
        _check(lib().ep_gemm_mxfp4_experts(xp, xsp, wp, wsp, offsets.data_ptr(), lead[0], M, N, K, *tail), "ep_gemm_mxfp4_experts")
    return y


def gemm_mxfp4(xq, xs, wq, ws, bias=None, out_dtype=None, stream=None):
    """Y = X W^T (+ bias) of two MXFP4 matrices: codes xq [M, Kp / 2] and wq [N, Kp / 2] with scales xs [Kp / 128, M, 4]
    and ws [Kp / 128, N, 4], as quantize_rows_mxfp4 gives them; fp32 sums, bias BF16 [N], output BF16 (default), FP16
    or FP32, rounded once. Codes at an address that is no multiple of 16 are copied first. It has no gradient: a bias that asks for one
    is refused. On `stream` (default: the current stream; another stream first waits for the current one)."""
    if stream is not None:
        return _on_stream(stream, lambda: _gemm_mxfp4(xq, xs, wq, ws, None, bias, out_dtype), xq, xs, wq, ws, bias)
    return _gemm_mxfp4(xq, xs, wq, ws, None, bias, out_dtype)


def gemm_mxfp4_experts(xq, xs, wq, ws, offsets, bias=None, out_dtype=None, stream=None):
    """gemm_mxfp4 with a weight per expert, in one launch: rows offsets[e] ... offsets[e + 1] - 1 of xq [R, Kp / 2]
    (scales xs [Kp / 128, R, 4]) meet wq[e] ([experts, N, Kp / 2], scales ws [experts, Kp / 128, N, 4], bias [experts,
    N]); rows behind the last expert's come out zero. offsets: int32 on the GPU, as sort_tokens gives them
    (ascending from 0, at most R; they are not read on the host)."""
    if stream is not None:
        return _on_stream(stream, lambda: _gemm_mxfp4(xq, xs, wq, ws, offsets, bias, out_dtype),
                          xq, xs, wq, ws, offsets, bias)
    return _gemm_mxfp4(xq, xs, wq, ws, offsets, bias, out_dtype)


# ------------------------------------------------------------------------------------ expert routing
def _no_tangents(*tensors, of="the expert routing has no forward-mode derivative; use reverse mode"):
    """Refuses the dual tensors of forward-mode differentiation: they do not require a gradient, so the
    kernels would drop their tangents without a word."""
    forward_ad = _torch().autograd.forward_ad
    if getattr(forward_ad, "_current_level", 0) < 0:          # no level is open, so there are none; saves 1.5 us
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(of)


def _no_gradient(what: str, *tensors):
    """Refuses tensors that ask for a derivative, of either mode, of a call that has none."""
    torch = _torch()
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{what} no gradient; detach its inputs")
    if getattr(torch.autograd.forward_ad, "_current_level", 0) >= 0:
        _no_tangents(*tensors, of=f"{what} no derivative; detach its inputs")


def _sort_raw(x, ids, n_experts):
    torch = _torch()
    T, k = ids.shape
    _, H, ldx = _need_rows(x, "x", (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8,
                                    torch.float8_e4m3fn))
    need = C.c_size_t()
    _check(lib().ep_sort_tokens_scratch(T, k, n_experts, C.byref(need)), "ep_sort_tokens")
    dev = x.device
    rows = torch.empty((T * k, H), dtype=x.dtype, device=dev)
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    scratch = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
    _check(lib().ep_sort_tokens(_ptr(x), _dtype_code(x.dtype), T, H, ldx, _ptr(ids), ids.element_size(), k, n_experts,
                                _ptr(rows), _ptr(offsets), _ptr(pos), _ptr(scratch), _current_raw()), "ep_sort_tokens")
    return rows, offsets, pos


def _combine_raw(ys, pos, weights):
    T, k = pos.shape
    R, H = ys.shape
    y = _torch().empty((T, H), dtype=ys.dtype, device=ys.device)
    _check(lib().ep_combine_tokens(_ptr(ys), _dtype_code(ys.dtype), _ptr(pos), _ptr(weights), T, k, H, R, _ptr(y),
                                   _current_raw()), "ep_combine_tokens")
    return y


_routing = None


def _routing_functions():
    """The autograd functions of sort_tokens and combine_tokens (torch is imported on first use). Their
    gradients run on the stream the forward ran on, which autograd makes current."""
    global _routing
    if _routing is None:
        torch = _torch()

        def once(backward):
            # refuses a second derivative; its wrapper (4 us) is left out where none can be asked for
            guarded = torch.autograd.function.once_differentiable(backward)
            return lambda ctx, *grads: (guarded if torch.is_grad_enabled() else backward)(ctx, *grads)

        class SortTokens(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, ids, n_experts):
                rows, offsets, pos = _sort_raw(x, ids, n_experts)
                ctx.mark_non_differentiable(offsets, pos)
                ctx.set_materialize_grads(False)             # no zeros are made for offsets and pos
                ctx.save_for_backward(pos)
                return rows, offsets, pos

            @staticmethod
            @once
            def backward(ctx, d_rows, *_):
                if d_rows is None:
                    return None, None, None
                # a token's gradient is the sum of its rows'; dropped choices have no part in it
                _no_tangents(d_rows)
                (pos,) = ctx.saved_tensors
                return _combine_raw(d_rows.contiguous(), pos, None), None, None

        class CombineTokens(torch.autograd.Function):
            @staticmethod
            def forward(ctx, ys, pos, weights):
                want_w = weights is not None and ctx.needs_input_grad[2]
                ctx.save_for_backward(ys if want_w else None, pos, weights)
                ctx.rows = ys.shape[0]
                return _combine_raw(ys, pos, weights)

            @staticmethod
            @once
            def backward(ctx, dy):
                ys, pos, weights = ctx.saved_tensors
                _no_tangents(dy)
                dy = dy.contiguous()
                T, k = pos.shape
                H = dy.shape[1]
                d_ys = torch.empty((ctx.rows, H), dtype=dy.dtype, device=dy.device) if ctx.needs_input_grad[0] else None
                d_w = torch.empty((T, k), dtype=torch.float32, device=dy.device) if ys is not None else None
                _check(lib().ep_combine_tokens_grad(_ptr(ys), _dtype_code(dy.dtype), _ptr(pos), _ptr(weights), _ptr(dy),
                                                    T, k, H, ctx.rows, _ptr(d_ys), _ptr(d_w), _current_raw()),
                       "ep_combine_tokens_grad")
                return d_ys, None, d_w

        _routing = SortTokens, CombineTokens
    return _routing


def sort_tokens(x, expert_ids, n_experts: int, stream=None):
    """Tokens sorted by the experts they chose. x: [T, H] (any element type; rows may be further apart
    than H), expert_ids: [T, k] int32 or int64; a number outside 0 ... n_experts - 1 drops the choice.
    Returns (rows [T k, H], offsets [n_experts + 1] int32, pos [T, k] int32): expert e has rows offsets[e]
    ... offsets[e + 1] - 1, in the order of the choices; choice (t, j) is row pos[t, j], or dropped, with
    pos[t, j] = -1 - row of a zero row behind the last expert's. Differentiable in x (reverse mode; dual
    tensors are refused); the host waits for nothing. On `stream` (default: the current stream; another
    stream first waits for the current one)."""
    torch = _torch()
    if stream is not None:
        return _on_stream(stream, lambda: sort_tokens(x, expert_ids, n_experts), x, expert_ids)
    _no_tangents(x)
    if expert_ids.dim() != 2 or expert_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("expert_ids must be an int32 or int64 tensor of shape [tokens, choices]")
    _need(expert_ids, "expert_ids", expert_ids.dtype)
    if x.dim() != 2 or x.shape[0] != expert_ids.shape[0]:
        raise ValueError(f"x must have shape [{expert_ids.shape[0]}, H], got {tuple(x.shape)}")
    grad = x.requires_grad and torch.is_grad_enabled()
    if grad and x.dtype not in _float_types():
        raise ValueError(f"rows of {x.dtype} have no gradient; detach x")
    if grad:
        return _routing_functions()[0].apply(x, expert_ids, n_experts)
    return _sort_raw(x, expert_ids, n_experts)


def combine_tokens(ys, pos, weights=None, stream=None):
    """The experts' rows summed back per token: y[t] = sum over j of weights[t, j] ys[pos[t, j]] in fp32,
    rounded once to the rows' type; dropped choices are left out, and without weights they are 1. ys:
    [T k, H] BF16, FP16 or FP32 (more rows are allowed where no gradient is wanted), pos: sort_tokens'
    positions [T, k], weights: fp32 [T, k]. Differentiable in ys and weights (reverse mode; dual tensors
    are refused). On `stream` (default: the current stream; another stream first waits for the current
    one)."""
    torch = _torch()
    if stream is not None:
        return _on_stream(stream, lambda: combine_tokens(ys, pos, weights), ys, pos, weights)
    _no_tangents(ys, weights)
    if ys.dim() != 2 or ys.dtype not in _float_types():
        raise ValueError(f"ys must be a bfloat16, float16 or float32 matrix, got {ys.dtype} of shape {tuple(ys.shape)}")
    _need(ys, "ys", ys.dtype)
    if pos.dim() != 2:
        raise ValueError("pos must have shape [tokens, choices]")
    _need(pos, "pos", torch.int32)
    if weights is not None:
        _need(weights, "weights", torch.float32, shape=pos.shape)
    if torch.is_grad_enabled() and (ys.requires_grad or (weights is not None and weights.requires_grad)):
        if ys.shape[0] != pos.numel():
            raise ValueError(f"the gradient takes one row per choice: ys has {ys.shape[0]} rows for {pos.numel()} choices")
        return _routing_functions()[1].apply(ys, pos, weights)
    return _combine_raw(ys, pos, weights)


class CompressedLinear:
    """Linear layer that keeps only the compressed weight and decodes it on every forward
    ("EntroPack PyTorch Guide", section "Replace one linear layer before a whole model").

    compute="bf16" (default): for up to 64 activation rows of a row-layout stream (the layout
    from_linear codes) one kernel decodes every tile pair straight into the B operand of the BF16
    MFMA and the weight is never written; a layout-0 stream is fused that way through LDS for 5 to
    16 rows and by the decode kernel's own products for up to 4. For more rows the weight is decoded
    once per call into scratch slices that stay in the Infinity Cache, and a BF16 MFMA GEMM reads
    them from there (hipBLASLt's from 512 rows, above 64 when in_features <= 4096, from 256 when
    out_features <= 4096; else the library's own).
    compute="fp8": the weight is decoded to FP8 E4M3 with its row scales and the activations are
    quantized per row; the codes meet in the FP8 MFMA, fused in the same cases, else on slices.
    compute="int8": the weight is decoded to INT8 with its row scales and the activations are quantized
    per row (quantize_rows_int8); the codes meet in the INT8 MFMA, fused for up to 64 rows of a
    row-layout stream, else on slices (gemm_int8); the sums are exact either way.

    The forward takes BF16 activations. Other dtypes are refused unless cast=True is passed, so a
    precision change is never silent ("Diagnose compression failures in the correct order")."""

    def __init__(self, stream: bytes, bias=None, compute: str = "bf16"):
        if compute not in ("bf16", "fp8", "int8"):
            raise ValueError("compute must be 'bf16', 'fp8' or 'int8'")
        self.stream = stream
        self.handle = Handle(stream)
        self.out_features, self.in_features = self.handle.shape
        self.bias = bias
        self.compute = compute

    @classmethod
    def from_linear(cls, linear, target_bpp: float = 4.0, compute: str = "bf16", **kw):
        """Compress an nn.Linear's weight (probability precision LAYER_PROB_BITS and tile layout
        LAYER_LAYOUT unless prob_bits= / layout= are given) and keep its bias in BF16 on the GPU."""
        kw.setdefault("prob_bits", LAYER_PROB_BITS)
        kw.setdefault("layout", LAYER_LAYOUT)
        s, _ = compress(linear.weight, target_bpp, **kw)
        bias = None
        if linear.bias is not None:
            bias = linear.bias.detach().to(device="cuda", dtype=_torch().bfloat16).contiguous()
        return cls(s, bias, compute)

    @property
    def actual_bpp(self) -> float:
        return self.handle.info["actual_bpp"]

    def save(self, path) -> None:
        """Write the compressed weight and the bias to a file (see save())."""
        save(path, self.stream, self.bias)

    @classmethod
    def load(cls, path, compute: str = "bf16"):
        """Rebuild a layer from a file written by save(); the bias goes to the current GPU. The
        compute mode is a choice of the forward, not part of the artifact."""
        stream, bias = load(path)
        b = None
        if bias is not None:
            torch = _torch()
            b = torch.from_numpy(bias.view("int16")).view(torch.bfloat16).cuda()
        return cls(stream, b, compute)

    def forward(self, x, stream=None, cast: bool = False):
        """Y = X W^T (+ bias) in BF16 on `stream` (default: the current stream). x must be BF16,
        or cast=True to convert it first. With an explicit stream other than the current one, that
        stream first waits for the work queued on the current stream (which produced x), and the
        conversion and the output allocation run on it."""
        torch = _torch()
        shp = x.shape
        if shp[-1] != self.in_features or not x.is_cuda:
            raise ValueError(f"input must be a GPU tensor with last dimension {self.in_features}, got {tuple(shp)}")
        if x.dtype != torch.bfloat16 and not cast:
            raise ValueError(f"the forward takes bfloat16 activations, got {x.dtype}; pass cast=True to convert")
        if x.device.index != torch.cuda.current_device():
            raise ValueError(f"x is on {x.device}, but the current device is cuda:{torch.cuda.current_device()}")
        if self.bias is not None:
            _need(self.bias, "bias", torch.bfloat16, shape=(self.out_features,))
        s, other = _run_on(stream)
        with torch.cuda.stream(s):
            rows = int(np.prod(shp[:-1], dtype=np.int64))
            x2 = x.reshape(rows, shp[-1]).to(torch.bfloat16).contiguous()
            y = torch.empty((x2.shape[0], self.out_features), dtype=torch.bfloat16, device=x.device)
            bp = C.c_void_p(self.bias.data_ptr()) if self.bias is not None else None
            name = "ep_linear_forward" + ("" if self.compute == "bf16" else "_" + self.compute)
            _check(getattr(lib(), name)(self.handle.ptr, C.c_void_p(x2.data_ptr()), x2.shape[0], bp,
                                        C.c_void_p(y.data_ptr()), C.c_void_p(s.cuda_stream)), name)
        _used_on(s, other, x2, self.bias)   # x (or its converted copy) is read on s after this returns
        return y.reshape(*shp[:-1], self.out_features)

    __call__ = forward


def linear_forward_many(layers, x, stream=None):
    """[layer(x) for layer in layers] for CompressedLinear layers of one compute mode that take the
    same input x (BF16, [..., in_features] on the GPU), each output the same bits as the layer's own
    forward. Up to 64 activation rows of row-layout layers with one prob_bits decode in one fused
    launch (ep_linear_forward_many, ep_linear_forward_fp8_many, ep_linear_forward_int8_many), so that
    small layers share the GPU's rounds of tile pairs; above 64 rows BF16 layers can share one slice
    decode; other cases run the layers one by one."""
    torch = _torch()
    layers = list(layers)
    if not layers:
        return []
    name = "ep_linear_forward" + ("" if layers[0].compute == "bf16" else "_" + layers[0].compute) + "_many"
    if len(layers) > 32 or any(l.compute != layers[0].compute for l in layers):
        return [l(x, stream=stream) for l in layers]
    K = layers[0].in_features
    shp = x.shape
    if any(l.in_features != K for l in layers) or shp[-1] != K or not x.is_cuda:
        raise ValueError("the layers must share in_features, and x must be a GPU tensor of that last dimension")
    if x.dtype != torch.bfloat16:
        raise ValueError(f"the forward takes bfloat16 activations, got {x.dtype}")
    if x.device.index != torch.cuda.current_device():
        raise ValueError(f"x is on {x.device}, but the current device is cuda:{torch.cuda.current_device()}")
    for l in layers:
        if l.bias is not None:
            _need(l.bias, "bias", torch.bfloat16, shape=(l.out_features,))
    s, other = _run_on(stream)
    with torch.cuda.stream(s):
        rows = int(np.prod(shp[:-1], dtype=np.int64))
        x2 = x.reshape(rows, K).contiguous()
        ys = [torch.empty((rows, l.out_features), dtype=torch.bfloat16, device=x.device) for l in layers]
        n = len(layers)
        hs = (C.c_void_p * n)(*[l.handle.ptr.value for l in layers])
        bs = (C.c_void_p * n)(*[(l.bias.data_ptr() if l.bias is not None else None) for l in layers])
        os_ = (C.c_void_p * n)(*[y.data_ptr() for y in ys])
        _check(getattr(lib(), name)(hs, n, C.c_void_p(x2.data_ptr()), rows, bs, os_, C.c_void_p(s.cuda_stream)), name)
    _used_on(s, other, x2, *[l.bias for l in layers])
    return [y.reshape(*shp[:-1], l.out_features) for y, l in zip(ys, layers)]


def linear_forward_experts(layers, x, expert_ids, weights=None, stream=None):
    """A mixture-of-experts layer of compressed experts: y[t] = sum over j of weights[t, j] layer_e(x[t]), e =
    expert_ids[t, j], for CompressedLinear layers of one shape and compute mode; x: BF16 [T, in_features],
    expert_ids: [T, k] int32 or int64 (a number outside 0 ... len(layers) - 1 drops the choice), weights:
    fp32 [T, k] or None (ones). The tokens are sorted by expert (sort_tokens), each expert multiplies its
    rows, the same bits as the layer's own forward of them, and the rows are summed back
    (combine_tokens). Experts without tokens are not decoded, and up to 64 rows each share fused
    launches, so the host reads the experts' row counts once: the call waits for the work queued on its
    stream and cannot be captured into a graph. Differentiable in weights (a router over frozen experts);
    x has to be detached, since a compressed layer has no gradient. On `stream` (default: the current
    stream; another stream first waits for the current one)."""
    torch = _torch()
    layers = list(layers)
    if not layers:
        raise ValueError("linear_forward_experts needs at least one expert")
    if any(l.compute != layers[0].compute or l.handle.shape != layers[0].handle.shape for l in layers):
        raise ValueError("the experts must share their shape and compute mode")
    N, K = layers[0].handle.shape
    if x.dim() != 2 or x.shape[1] != K or x.dtype != torch.bfloat16:
        raise ValueError(f"x must be a bfloat16 tensor of shape [tokens, {K}], got {x.dtype} {tuple(x.shape)}")
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("the compressed experts have no gradient in x; detach it")
    biases = [l.bias for l in layers]
    for b in biases:
        if b is not None:
            _need(b, "bias", torch.bfloat16, shape=(N,))
    if stream is not None:
        return _on_stream(stream, lambda: linear_forward_experts(layers, x, expert_ids, weights), x, expert_ids,
                          weights, *biases)
    n = len(layers)
    rows, offsets, pos = sort_tokens(x, expert_ids, n)
    offs = (C.c_int64 * (n + 1))(*offsets.tolist())
    ys = torch.empty((rows.shape[0], N), dtype=torch.bfloat16, device=x.device)
    hs = (C.c_void_p * n)(*[l.handle.ptr.value for l in layers])
    bs = (C.c_void_p * n)(*[_ptr(b) for b in biases])
    code = {"bf16": BF16, "fp8": F8E4M3, "int8": I8}[layers[0].compute]
    _check(lib().ep_linear_forward_experts(hs, n, code, _ptr(rows), offs, _ptr(offsets), bs, _ptr(ys),
                                           _current_raw()),
           "ep_linear_forward_experts")
    return combine_tokens(ys, pos, weights)


@functools.lru_cache(maxsize=256)
def _mlp_scratch(T: int, k: int, E: int, I: int, N: int, mxfp4: bool) -> int:
    """Bytes of scratch that mlp_forward_experts needs for these sizes."""
    need = C.c_size_t()
    _check(lib().ep_mlp_forward_experts_scratch(T, k, E, I, N, mxfp4, C.byref(need)), "ep_mlp_forward_experts")
    return need.value


def mlp_forward_experts(x, expert_ids, weights, w_in, w_out, in_scales=None, out_scales=None, in_bias=None, out_bias=None,
                        stream=None):
    """A mixture-of-experts layer of gated MLP experts for up to 64 tokens, in two kernels: y[t] = sum over j of weights[t, j]
    (W_out[e] h + out_bias[e]), h = silu(g) u, (g, u) = W_in[e] x[t] + in_bias[e], e = expert_ids[t, j].

    x: BF16 or FP16 [T, H] (rows may be further apart than H), T <= 64; expert_ids: [T, k] int32 or int64, T k <= 1024 (a
    number outside 0 ... experts - 1 drops the choice; the same expert twice in a token counts once, with the sum of the
    weights); weights: fp32 [T, k] or None (ones). w_in: [experts, 2 I, H], rows 0 ... I - 1 of an expert give g, the others u;
    w_out: [experts, N, I]; both of x's type, or, with in_scales and out_scales, MXFP4 codes and scales as
    quantize_rows_mxfp4 gives them (exact in BF16; in FP16 values below 2^-14 lose bits and none may pass 65504). Biases: BF16 [experts, 2 I] and
    [experts, N]. fp32 sums; h is rounded once to x's type (in FP16 a magnitude above 65504 is infinite), and y [T, N] once.

    The weights of the experts that some token chose are read once; the host waits for nothing, so the call can be captured
    into a graph. For more tokens use sort_tokens, a product per expert and combine_tokens. It has no gradient: tensors
    that ask for one are refused. On `stream` (default: the current stream; another stream first waits for the current
    one)."""
    torch = _torch()
    if stream is not None:
        return _on_stream(stream, lambda: mlp_forward_experts(x, expert_ids, weights, w_in, w_out, in_scales, out_scales, in_bias,
                                                              out_bias),
                          x, expert_ids, weights, w_in, w_out, in_scales, out_scales, in_bias, out_bias)
    _no_gradient("the expert layer for few tokens has", x, weights, w_in, w_out, in_bias, out_bias)
    dtype, f32, bf16, u8 = x.dtype, torch.float32, torch.bfloat16, torch.uint8
    if dtype is not bf16 and dtype is not torch.float16:
        raise ValueError(f"x must be bfloat16 or float16, got {dtype}")
    T, H, ldx = _need_rows(x, "x", (dtype,))
    dev, chosen = x.get_device(), expert_ids.shape
    if len(chosen) != 2 or chosen[0] != T or expert_ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"expert_ids must be an int32 or int64 tensor of shape [{T}, choices]")
    k = chosen[1]
    if T > 64 or T * k > 1024:
        raise ValueError(f"at most 64 tokens and 1024 choices, got {T} and {T * k}; for more use sort_tokens, a product per expert and "
                         "combine_tokens")
    if (in_scales is None) != (out_scales is None):
        raise ValueError("in_scales and out_scales go together: both weights are MXFP4, or neither")
    ins, outs = w_in.shape, w_out.shape
    if len(ins) != 3 or len(outs) != 3 or ins[0] != outs[0] or ins[1] % 2:
        raise ValueError(f"w_in must be [experts, 2 I, H] and w_out [experts, N, I], got {tuple(ins)} and {tuple(outs)}")
    E, I, N = ins[0], ins[1] // 2, outs[1]
    ic = (I + 127) // 128
    if in_scales is None:
        args = [("w_in", w_in, dtype, (E, 2 * I, H)), ("w_out", w_out, dtype, (E, N, I))]
    else:
        hc = (H + 127) // 128
        args = [("w_in", w_in, u8, (E, 2 * I, 64 * hc)), ("in_scales", in_scales, u8, (E, hc, 2 * I, 4)),
                ("w_out", w_out, u8, (E, N, 64 * ic)), ("out_scales", out_scales, u8, (E, ic, N, 4))]
    args.append(("expert_ids", expert_ids, expert_ids.dtype, chosen))
    if weights is not None:
        args.append(("weights", weights, f32, chosen))
    if in_bias is not None:
        args.append(("in_bias", in_bias, bf16, (E, 2 * I)))
    if out_bias is not None:
        args.append(("out_bias", out_bias, bf16, (E, N)))
    for name, t, kind, shape in args:
        if not (t.dtype is kind and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
            _need(t, name, kind, shape=shape)
    if in_scales is not None:
        # codes are read in pieces of 16 bytes, scales in pieces of 4
        w_in, w_out = _mx_aligned(w_in, 16), _mx_aligned(w_out, 16)
        in_scales, out_scales = _mx_aligned(in_scales, 4), _mx_aligned(out_scales, 4)
    y, scratch = x.new_empty((T, N)), x.new_empty(_mlp_scratch(T, k, E, I, N, in_scales is not None), dtype=u8)
    _check(lib().ep_mlp_forward_experts(x.data_ptr(), _dtype_code(dtype), T, H, ldx, expert_ids.data_ptr(), expert_ids.element_size(),
                                        k, E, _ptr(weights), w_in.data_ptr(), _ptr(in_scales), _ptr(in_bias), w_out.data_ptr(),
                                        _ptr(out_scales), _ptr(out_bias), I, N, scratch.data_ptr(), y.data_ptr(),
                                        torch._C._cuda_getCurrentRawStream(dev)), "ep_mlp_forward_experts")
    return y
