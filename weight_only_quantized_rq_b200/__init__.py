"""Python binding of librq (include/rq.h): weight-only group-quantized matrix
products for RWKV-7 on B200.

This module only marshals arguments: it passes torch tensors' device pointers
and the current CUDA stream to the C ABI. PyTorch provides device memory and
streams; every step of the computation runs in librq's CUDA kernels. There is
no fallback: if librq.so is missing, every call raises.

Formats (see include/rq.h): ``RQ_W4_SYM_G64`` (symmetric int4, group 64),
``RQ_W8_SYM_G16`` / ``RQ_W8_SYM_G64`` (symmetric int8, group 16 / 64),
``RQ_W6_SYM_G16`` (symmetric 6-bit, group 16), ``RQ_W4_ASYM_SB32``,
``RQ_W5_ASYM_SB32``, ``RQ_W6_ASYM_SB32`` (asymmetric 4-, 5-, 6-bit superblocks
of 8 groups of 32). The strings "w4g64", "w8g16", "w8g64", "w6g16", "w4sb32",
"w5sb32", "w6sb32" are accepted wherever a format is expected.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librq.so")

RQ_OK = 0
RQ_ERR_INVALID_ARG = 1
RQ_ERR_UNSUPPORTED_SHAPE = 2
RQ_ERR_FORMAT_MISMATCH = 3
RQ_ERR_MISALIGNED = 4
RQ_ERR_CUDA = 5
RQ_ERR_DEVICE_TIMEOUT = 6
RQ_ERR_NOT_POSITIVE_DEFINITE = 7

RQ_OUT_F32 = 0
RQ_OUT_BF16 = 1

RQ_ACT_NONE = 0
RQ_ACT_RELU_SQ = 1
ACTS = {None: RQ_ACT_NONE, "none": RQ_ACT_NONE, "relu2": RQ_ACT_RELU_SQ}

RQ_W4_SYM_G64 = 1
RQ_W8_SYM_G16 = 2
RQ_W4_ASYM_SB32 = 3
RQ_W5_ASYM_SB32 = 4
RQ_W6_ASYM_SB32 = 5
RQ_W8_SYM_G64 = 6
RQ_W6_SYM_G16 = 7
FORMAT_IDS = {"w4g64": RQ_W4_SYM_G64, "w8g16": RQ_W8_SYM_G16, "w4sb32": RQ_W4_ASYM_SB32,
              "w5sb32": RQ_W5_ASYM_SB32, "w6sb32": RQ_W6_ASYM_SB32, "w8g64": RQ_W8_SYM_G64,
              "w6g16": RQ_W6_SYM_G16}
SB_FORMATS = (RQ_W4_ASYM_SB32, RQ_W5_ASYM_SB32, RQ_W6_ASYM_SB32)
EXPORTS = ("rq_packed_size", "rq_quantize_pack", "rq_wgemm", "rq_wgemm_batch", "rq_wgemm_out", "rq_wgemm_batch_out",
           "rq_dequant", "rq_grouped_workspace_size", "rq_wgemm_grouped", "rq_lora_workspace_size", "rq_wgemm_lora",
           "rq_route_workspace_size", "rq_route_topk", "rq_route_combine",
           "rq_act_sumsq", "rq_act_finalize", "rq_hessian_accum", "rq_gptq_prepare", "rq_gptq_quantize_pack",
           "rq_status_string", "rq_last_cuda_error", "rq_device_status", "rq_test_hooks", "rq_version")
MAX_BATCH = 160
TC_MIN_M = 3         # activation rows from which int4/int8/4-bit superblock products run on the tensor cores
                     # (5- and 6-bit products run there at every M)
TC_MAX_ITEMS = 96    # products per tensor-core launch (larger batches take several)


def tc_path(fmt, M: int) -> bool:
    """Whether products of this format at M activation rows run on the
    tensor-core kernel (else on the register-path GEMV)."""
    f = fmt_id(fmt)
    if f in (RQ_W5_ASYM_SB32, RQ_W6_ASYM_SB32, RQ_W6_SYM_G16):
        return True
    return M >= TC_MIN_M


class RqSearch(ctypes.Structure):
    _fields_ = [("n_cand", ctypes.c_int), ("t_lo", ctypes.c_float), ("t_hi", ctypes.c_float)]


class RqPacked(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int), ("reserved", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class RqWgemmItem(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w", ctypes.POINTER(RqPacked)), ("y", ctypes.c_void_p)]


class RqGroups(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int), ("R", ctypes.c_int), ("offsets", ctypes.c_void_p), ("in_rows", ctypes.c_void_p),
                ("out_rows", ctypes.c_void_p)]


class RqLora(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("rank", ctypes.c_int), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("ranks", ctypes.c_void_p)]


class RqRouting(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("weights", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("in_rows", ctypes.c_void_p), ("slots", ctypes.c_void_p)]


class RqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {rq_status_string(status)} (status {status})"
        if status == RQ_ERR_CUDA:
            msg += f", cudaError {_lib().rq_last_cuda_error()}"
        super().__init__(msg)


_L = None


def _lib() -> ctypes.CDLL:
    """Load librq.so (built in-tree). Raises if it is absent: there is no
    other implementation to fall back to."""
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"librq.so is not built ({LIB_PATH}); run "
                              "`python -m weight_only_quantized_rq_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I = ctypes.c_void_p, ctypes.c_int
        L.rq_packed_size.argtypes = [I, I, I, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.rq_packed_size.restype = ctypes.c_size_t
        L.rq_quantize_pack.argtypes = [P, I, I, P, ctypes.POINTER(RqSearch), ctypes.POINTER(RqPacked), P]
        L.rq_quantize_pack.restype = I
        L.rq_wgemm.argtypes = [P, I, I, I, ctypes.POINTER(RqPacked), P, P]
        L.rq_wgemm.restype = I
        L.rq_wgemm_batch.argtypes = [ctypes.POINTER(RqWgemmItem), I, I, P]
        L.rq_wgemm_batch.restype = I
        L.rq_wgemm_out.argtypes = [P, I, I, I, ctypes.POINTER(RqPacked), P, I, P]
        L.rq_wgemm_out.restype = I
        L.rq_wgemm_batch_out.argtypes = [ctypes.POINTER(RqWgemmItem), I, I, I, P]
        L.rq_wgemm_batch_out.restype = I
        L.rq_dequant.argtypes = [ctypes.POINTER(RqPacked), P, P]
        L.rq_dequant.restype = I
        L.rq_act_sumsq.argtypes = [P, I, I, P, P]
        L.rq_act_sumsq.restype = I
        L.rq_act_finalize.argtypes = [P, I, ctypes.c_longlong, P, P]
        L.rq_act_finalize.restype = I
        L.rq_hessian_accum.argtypes = [P, I, I, P, P]
        L.rq_hessian_accum.restype = I
        L.rq_gptq_prepare.argtypes = [P, I, ctypes.c_double, P, P, P]
        L.rq_gptq_prepare.restype = I
        L.rq_gptq_quantize_pack.argtypes = [P, I, I, P, P, P, ctypes.POINTER(RqSearch), ctypes.POINTER(RqPacked), P]
        L.rq_gptq_quantize_pack.restype = I
        Z = ctypes.c_size_t
        L.rq_grouped_workspace_size.argtypes = [I, I, I, I, I]
        L.rq_grouped_workspace_size.restype = Z
        L.rq_wgemm_grouped.argtypes = [P, I, I, I, ctypes.POINTER(RqPacked), ctypes.POINTER(RqGroups), P, I, I, I, P, Z, P]
        L.rq_wgemm_grouped.restype = I
        L.rq_lora_workspace_size.argtypes = [I, I, I, I, I]
        L.rq_lora_workspace_size.restype = Z
        L.rq_wgemm_lora.argtypes = [P, I, I, I, ctypes.POINTER(RqPacked), ctypes.POINTER(RqLora), P, P, I, P, Z, P]
        L.rq_wgemm_lora.restype = I
        L.rq_route_workspace_size.argtypes = [I, I, I]
        L.rq_route_workspace_size.restype = Z
        L.rq_route_topk.argtypes = [P, I, I, I, I, I, ctypes.POINTER(RqRouting), P, Z, P]
        L.rq_route_topk.restype = I
        L.rq_route_combine.argtypes = [P, I, P, P, I, I, I, P, I, P]
        L.rq_route_combine.restype = I
        L.rq_status_string.argtypes = [I]
        L.rq_status_string.restype = ctypes.c_char_p
        L.rq_last_cuda_error.argtypes = []
        L.rq_last_cuda_error.restype = I
        L.rq_device_status.argtypes = [P, ctypes.POINTER(I)]
        L.rq_device_status.restype = I
        L.rq_test_hooks.argtypes = [ctypes.c_longlong, I]
        L.rq_test_hooks.restype = I
        L.rq_version.argtypes = []
        L.rq_version.restype = I
        _L = L
    return _L


def lib() -> ctypes.CDLL:
    return _lib()


def fmt_id(fmt) -> int:
    return FORMAT_IDS[fmt] if isinstance(fmt, str) else int(fmt)


def _stream(stream=None) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _check(status: int, where: str) -> None:
    if status != RQ_OK:
        raise RqError(status, where)


# ------------------------------------------------------------------ calls --
def rq_status_string(status: int) -> str:
    return _lib().rq_status_string(int(status)).decode()


def rq_version() -> int:
    return _lib().rq_version()


def rq_packed_size(fmt, K: int, N: int) -> tuple[int, int]:
    """(codes_bytes, scales_bytes); raises for an unsupported shape."""
    cb, sb = ctypes.c_size_t(0), ctypes.c_size_t(0)
    tot = _lib().rq_packed_size(fmt_id(fmt), int(K), int(N), ctypes.byref(cb), ctypes.byref(sb))
    if tot == 0:
        raise RqError(RQ_ERR_UNSUPPORTED_SHAPE, "rq_packed_size")
    return cb.value, sb.value


@dataclass
class Packed:
    """A packed matrix: the descriptor fields plus the two device planes
    (uint8 tensors that own the memory)."""
    fmt: int
    K: int
    N: int
    codes: torch.Tensor
    scales: torch.Tensor | None

    def desc(self) -> RqPacked:
        return RqPacked(self.fmt, self.K, self.N, 0, self.codes.data_ptr(),
                        None if self.scales is None else self.scales.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + (0 if self.scales is None else self.scales.numel())


def alloc_packed(fmt, K: int, N: int, device=None) -> Packed:
    f = fmt_id(fmt)
    cb, sb = rq_packed_size(f, K, N)
    dev = torch.device("cuda") if device is None else torch.device(device)
    codes = torch.empty(cb, dtype=torch.uint8, device=dev)
    scales = torch.empty(sb, dtype=torch.uint8, device=dev) if sb else None
    return Packed(f, int(K), int(N), codes, scales)


def rq_quantize_pack(W: torch.Tensor, fmt, act_sq: torch.Tensor | None = None, n_cand: int = 64,
                     t_lo: float = 0.7, t_hi: float = 1.0, out: Packed | None = None, stream=None) -> Packed:
    """Quantize and pack W (fp32 [N][K], CUDA). Returns the Packed matrix."""
    N, K = W.shape
    if out is None:
        out = alloc_packed(fmt, K, N, W.device)
    sr = RqSearch(int(n_cand), float(t_lo), float(t_hi))
    d = out.desc()
    _check(_lib().rq_quantize_pack(_ptr(W), int(K), int(N), _ptr(act_sq), ctypes.byref(sr), ctypes.byref(d),
                                   _stream(stream)), "rq_quantize_pack")
    return out


def _out_type(dtype) -> int:
    if dtype == torch.float32:
        return RQ_OUT_F32
    if dtype == torch.bfloat16:
        return RQ_OUT_BF16
    raise ValueError("y must be float32 or bfloat16")


def rq_wgemm(x: torch.Tensor, w: Packed, y: torch.Tensor | None = None, stream=None,
             out_dtype=torch.float32) -> torch.Tensor:
    """y = x @ w_hat.T with x bf16 [M][K] and y [M][N] (CUDA tensors), y fp32
    or bf16 (the fp32 result rounded once; by y's dtype, else out_dtype)."""
    M, K = x.shape
    if y is None:
        y = torch.empty(M, w.N, dtype=out_dtype, device=x.device)
    d = w.desc()
    _check(_lib().rq_wgemm_out(_ptr(x), int(M), int(K), int(w.N), ctypes.byref(d), _ptr(y), _out_type(y.dtype),
                               _stream(stream)), "rq_wgemm_out")
    return y


class WgemmBatch:
    """A prepared batch for rq_wgemm_batch: the ctypes item array is built
    once (so repeated calls and CUDA-graph capture pay no marshalling)."""

    def __init__(self, xs, ws, ys):
        if not (len(xs) == len(ws) == len(ys)) or not 1 <= len(xs) <= MAX_BATCH:
            raise ValueError("need 1..160 items with one x, w, y each")
        self.M = int(xs[0].shape[0])
        self._keep = (list(xs), list(ws), list(ys))
        self._descs = [w.desc() for w in ws]
        self._items = (RqWgemmItem * len(xs))()
        self.out = _out_type(ys[0].dtype)
        for i, (x, d, y) in enumerate(zip(xs, self._descs, ys)):
            if int(x.shape[0]) != self.M:
                raise ValueError("every item must have the same M")
            if _out_type(y.dtype) != self.out:
                raise ValueError("every y must have the same dtype")
            self._items[i] = RqWgemmItem(x.data_ptr(), ctypes.pointer(d), y.data_ptr())
        self.count = len(xs)

    def __call__(self, stream=None):
        _check(_lib().rq_wgemm_batch_out(self._items, self.count, self.M, self.out, _stream(stream)),
               "rq_wgemm_batch_out")


def rq_wgemm_batch(xs, ws, ys, stream=None) -> None:
    """Independent products ys[i] = xs[i] @ w_hat_i.T in one launch."""
    WgemmBatch(xs, ws, ys)(stream)


def rq_dequant(w: Packed, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """w_hat as fp32 [N][K] (CUDA)."""
    if out is None:
        out = torch.empty(w.N, w.K, dtype=torch.float32, device=w.codes.device)
    d = w.desc()
    _check(_lib().rq_dequant(ctypes.byref(d), _ptr(out), _stream(stream)), "rq_dequant")
    return out


# ------------------------------------- products that depend on the row --
def _refuse(t, name: str, dtype, shape, device) -> None:
    """Raises the ValueError that says what is wrong with a tensor argument."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _want(t, name: str, dtype, shape, device) -> int:
    """The address of a dense tensor of this dtype and shape on this device;
    anything else is refused."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def _rows(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() == 0:
        raise ValueError(f"{name} must be a tensor with rows")
    return t.shape[0]


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(device: torch.device, stream) -> int:
    """The current stream of `device` if it is the current device and no other
    stream is asked for, else -1 (see _there)."""
    if stream is None and device.type == "cuda" and torch.cuda.current_device() == device.index:
        return _raw_stream(device.index)
    return -1


def _there(device: torch.device, stream):
    """A context in which `device` is current, with `stream` (or the device's
    current stream) as the stream of the call and of its temporary memory."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


class GroupedExperts:
    """E packed expert matrices [N][K] in one Packed of E * N rows, prepared for
    rq_wgemm_grouped calls of at most max_rows rows."""

    def __init__(self, w: Packed, E: int, max_rows: int = 4096):
        E = int(E)
        if E < 1 or w.N % E:
            raise ValueError(f"{w.N} packed rows do not hold {E} equal experts")
        self.w, self.E, self.N, self.K, self.max_rows = w, E, w.N // E, w.K, int(max_rows)
        self.device = w.codes.device
        self._desc = w.desc()
        self._call = _lib().rq_wgemm_grouped
        self._bytes = int(_lib().rq_grouped_workspace_size(w.fmt, self.max_rows, w.K, self.N, E))
        if not self._bytes:
            raise RqError(RQ_ERR_UNSUPPORTED_SHAPE, "rq_grouped_workspace_size")

    def __call__(self, x: torch.Tensor, offsets: torch.Tensor, in_rows: torch.Tensor | None = None,
                 out_rows: torch.Tensor | None = None, y: torch.Tensor | None = None, act=None,
                 out_dtype=torch.float32, stream=None) -> torch.Tensor:
        """y[out_rows[i]] = act(x[in_rows[i]] @ w_hat_e.T) for the rows i in
        [offsets[e], offsets[e + 1]) of every expert e. The number of rows is
        that of in_rows, else of out_rows, else of x. y is [*, N] fp32 or bf16;
        without one a zeroed [rows, N] tensor of out_dtype is made (a pass over
        it that a call with y saves). act: None or "relu2" (max(v, 0)^2). bf16
        results of 16 or more rows per expert on average come from weights in
        fp16, the others from exact products; see include/rq.h."""
        dev, N = self.device, self.N
        T = _rows(x, "x")
        R = T if in_rows is None and out_rows is None else _rows(out_rows if in_rows is None else in_rows, "the row indices")
        px = _want(x, "x", torch.bfloat16, (T, self.K), dev)
        po = _want(offsets, "offsets", torch.int32, (self.E + 1,), dev)
        pi = 0 if in_rows is None else _want(in_rows, "in_rows", torch.int32, (R,), dev)
        pu = 0 if out_rows is None else _want(out_rows, "out_rows", torch.int32, (R,), dev)
        if R > self.max_rows:
            raise ValueError(f"{R} rows, prepared for at most {self.max_rows}")
        if act not in ACTS:
            raise ValueError(f"unknown activation {act!r}")
        st = _here(dev, stream)
        if st < 0:
            with _there(dev, stream):
                return self(x, offsets, in_rows, out_rows, y, act, out_dtype)
        if y is None:
            y = torch.zeros(R, N, dtype=out_dtype, device=dev)
        Ty = _rows(y, "y")
        out = _out_type(y.dtype)
        py = _want(y, "y", y.dtype, (Ty, N), dev)
        if R and Ty:
            if not T:                                   # no row of x: every row of the call is a row of zeros
                T, zeros = 1, torch.zeros(1, self.K, dtype=torch.bfloat16, device=dev)
                px = zeros.data_ptr()
            # temporary memory from PyTorch's caching allocator on the call's stream: calls on other streams and
            # captured graphs get their own
            ws = torch.empty(self._bytes, dtype=torch.uint8, device=dev)
            _check(self._call(px, T, self.K, N, self._desc, RqGroups(self.E, R, po, pi, pu), py, Ty, ACTS[act], out,
                              ws.data_ptr(), self._bytes, st), "rq_wgemm_grouped")
        return y


def rq_wgemm_grouped(x: torch.Tensor, w: Packed, offsets: torch.Tensor, in_rows=None, out_rows=None, y=None, act=None,
                     out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """Packed products grouped by expert: offsets int32 [E + 1], w a Packed of
    E * N rows. See GroupedExperts, which keeps what repeated calls share."""
    R = max(1, _rows(in_rows if in_rows is not None else out_rows if out_rows is not None else x, "x"))
    return GroupedExperts(w, _rows(offsets, "offsets") - 1, R)(x, offsets, in_rows, out_rows, y, act, out_dtype, stream)


class LoraProjection:
    """A packed matrix [N][K] with n slots of low-rank adapters, prepared for
    rq_wgemm_lora calls of at most max_rows rows. A is bf16 [n][r][K], B bf16
    [n][N][r], scales fp32 [n]; ranks int32 [n] (None: every slot uses all r).
    Their contents may be replaced between calls."""

    def __init__(self, w: Packed, A: torch.Tensor, B: torch.Tensor, scales: torch.Tensor, ranks: torch.Tensor | None = None,
                 max_rows: int = 128):
        dev = w.codes.device
        if not isinstance(A, torch.Tensor) or A.dim() != 3:
            raise ValueError("A must be [slots][rank][K]")
        n, r = int(A.shape[0]), int(A.shape[1])
        self._lora = RqLora(n, r, _want(A, "A", torch.bfloat16, (n, r, w.K), dev), _want(B, "B", torch.bfloat16, (n, w.N, r), dev),
                            _want(scales, "scales", torch.float32, (n,), dev),
                            None if ranks is None else _want(ranks, "ranks", torch.int32, (n,), dev))
        self.w, self.max_rows, self.device = w, int(max_rows), dev
        self._keep = (A, B, scales, ranks)
        self._desc = w.desc()
        self._call = _lib().rq_wgemm_lora
        self._bytes = int(_lib().rq_lora_workspace_size(w.fmt, self.max_rows, w.K, w.N, r))
        if not self._bytes:
            raise RqError(RQ_ERR_UNSUPPORTED_SHAPE, "rq_lora_workspace_size")

    def __call__(self, x: torch.Tensor, row_adapter: torch.Tensor, y: torch.Tensor | None = None,
                 out_dtype=torch.float32, stream=None) -> torch.Tensor:
        """y[m] = x[m] @ w_hat.T + scales[a] * (x[m] @ A[a].T) @ B[a].T with
        a = row_adapter[m] (int32 [M]; a row whose a is no slot has none)."""
        dev, N, K = self.device, self.w.N, self.w.K
        M = _rows(x, "x")
        px = _want(x, "x", torch.bfloat16, (M, K), dev)
        pr = _want(row_adapter, "row_adapter", torch.int32, (M,), dev)
        if M > self.max_rows:
            raise ValueError(f"{M} rows, prepared for at most {self.max_rows}")
        st = _here(dev, stream)
        if st < 0:
            with _there(dev, stream):
                return self(x, row_adapter, y, out_dtype)
        if y is None:
            y = torch.empty(M, N, dtype=out_dtype, device=dev)
        out = _out_type(y.dtype)
        py = _want(y, "y", y.dtype, (M, N), dev)
        if M:
            ws = torch.empty(self._bytes, dtype=torch.uint8, device=dev)
            _check(self._call(px, M, K, N, self._desc, self._lora, pr, py, out, ws.data_ptr(), self._bytes, st), "rq_wgemm_lora")
        return y


def rq_wgemm_lora(x: torch.Tensor, w: Packed, A: torch.Tensor, B: torch.Tensor, scales: torch.Tensor,
                  row_adapter: torch.Tensor, ranks=None, y=None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
    """A packed product with a low-rank adapter per row; see LoraProjection,
    which keeps what repeated calls share."""
    return LoraProjection(w, A, B, scales, ranks, max(1, _rows(x, "x")))(x, row_adapter, y, out_dtype, stream)


@dataclass
class Routing:
    """What rq_route_topk gives: ids and weights [T][k], and the chosen pairs
    grouped by expert (offsets [E + 1]; token and slot t k + j of each row)."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    in_rows: torch.Tensor
    slots: torch.Tensor


class TopkRouter:
    """Top-k expert routing of [T][E] logits (fp32 or bf16, CUDA)."""

    def __init__(self, E: int, k: int, renorm: bool = False):
        self.E, self.k, self.renorm = int(E), int(k), bool(renorm)
        self._call, self._size = _lib().rq_route_topk, _lib().rq_route_workspace_size
        if not self._size(1, self.E, self.k):
            raise ValueError("need 1 <= E <= 1024 and 1 <= k <= min(E, 16)")

    def __call__(self, logits: torch.Tensor, stream=None) -> Routing:
        T, k, E, dev = _rows(logits, "logits"), self.k, self.E, logits.device
        kind = _out_type(logits.dtype)
        pl = _want(logits, "logits", logits.dtype, (T, E), dev)
        st = _here(dev, stream)
        if st < 0:
            with _there(dev, stream):
                return self(logits)
        n = T * k
        if T == 0:
            z = torch.empty(0, dtype=torch.int32, device=dev)
            return Routing(z.view(0, k), z.float().view(0, k), torch.zeros(E + 1, dtype=torch.int32, device=dev), z, z)
        size = self._size(T, E, k)
        if not size:
            raise RqError(RQ_ERR_INVALID_ARG, "rq_route_workspace_size")
        # one buffer for the outputs and the workspace, each at a multiple of 16 bytes
        P, Q = (n + 3) & ~3, (E + 4) & ~3
        b = torch.empty(4 * P + Q + size // 4, dtype=torch.int32, device=dev)
        p = b.data_ptr()
        out = RqRouting(p, p + 4 * P, p + 16 * P, p + 8 * P, p + 12 * P)
        _check(self._call(pl, kind, T, E, k, int(self.renorm), out, p + 16 * P + 4 * Q, size, st), "rq_route_topk")
        pair, one = (k, 1), (1,)
        return Routing(b.as_strided((T, k), pair, 0), b.view(torch.float32).as_strided((T, k), pair, P),
                       b.as_strided((E + 1,), one, 4 * P), b.as_strided((n,), one, 2 * P), b.as_strided((n,), one, 3 * P))


def rq_route_topk(logits: torch.Tensor, k: int, renorm: bool = False, stream=None) -> Routing:
    """The k largest of each token's logits with their softmax weights, and the
    chosen pairs grouped by expert; see include/rq.h."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T][E] tensor")
    return TopkRouter(int(logits.shape[1]), k, renorm)(logits, stream)


def rq_route_combine(y: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, out: torch.Tensor | None = None,
                     out_dtype=None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t][j] * y[t k + j] over the j with ids[t][j] >= 0
    (y [T k][N], fp32 or bf16; out of out_dtype, by default y's)."""
    if not isinstance(y, torch.Tensor) or y.dim() != 2 or not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("y must be [T k][N] and ids [T][k]")
    dev = y.device
    (T, k), N = ids.shape, y.shape[1]
    kind = _out_type(y.dtype)
    py = _want(y, "y", y.dtype, (T * k, N), dev)
    pi = _want(ids, "ids", torch.int32, (T, k), dev)
    pw = _want(weights, "weights", torch.float32, (T, k), dev)
    st = _here(dev, stream)
    if st < 0:
        with _there(dev, stream):
            return rq_route_combine(y, ids, weights, out, out_dtype)
    if out is None:
        out = torch.empty(T, N, dtype=y.dtype if out_dtype is None else out_dtype, device=dev)
    po = _want(out, "out", out.dtype, (T, N), dev)
    if T:
        _check(_lib().rq_route_combine(py, kind, pi, pw, T, N, k, po, _out_type(out.dtype), st), "rq_route_combine")
    return out


def rq_act_sumsq(x: torch.Tensor, sum_sq: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Add sum_r x[r][k]^2 (x bf16 [R][K] on the GPU) into the fp64 running
    sums sum_sq[K] (created as zeros when None) and return them."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 [R][K] tensor")
    R, K = int(x.shape[0]), int(x.shape[1])
    if sum_sq is None:
        sum_sq = torch.zeros(K, dtype=torch.float64, device=x.device)
    _check(_lib().rq_act_sumsq(_ptr(x), R, K, _ptr(sum_sq), _stream(stream)), "rq_act_sumsq")
    return sum_sq


def rq_act_finalize(sum_sq: torch.Tensor, rows: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """E[x^2] = fp32(sum_sq / rows), the act_sq that rq_quantize_pack takes."""
    K = int(sum_sq.shape[0])
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=sum_sq.device)
    _check(_lib().rq_act_finalize(_ptr(sum_sq), K, int(rows), _ptr(out), _stream(stream)), "rq_act_finalize")
    return out


def rq_hessian_accum(x: torch.Tensor, H: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """H += x^T x (x bf16 [R][K] on the GPU; H fp64 [K][K], created as zeros
    when None), each element summed in ascending row order. Returns H."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 [R][K] tensor")
    R, K = int(x.shape[0]), int(x.shape[1])
    if H is None:
        H = torch.zeros(K, K, dtype=torch.float64, device=x.device)
    _check(_lib().rq_hessian_accum(_ptr(x), R, K, _ptr(H), _stream(stream)), "rq_hessian_accum")
    return H


def rq_gptq_prepare(H: torch.Tensor, damp: float = 0.01, U: torch.Tensor | None = None,
                    dead: torch.Tensor | None = None, stream=None):
    """The upper Cholesky factor U of the damped inverse Hessian and the dead
    channel flags (H fp64 [K][K] on the GPU). Returns (U, dead)."""
    K = int(H.shape[0])
    if U is None:
        U = torch.empty(K, K, dtype=torch.float64, device=H.device)
    if dead is None:
        dead = torch.empty(K, dtype=torch.uint8, device=H.device)
    _check(_lib().rq_gptq_prepare(_ptr(H), K, float(damp), _ptr(U), _ptr(dead), _stream(stream)), "rq_gptq_prepare")
    return U, dead


def rq_gptq_quantize_pack(W: torch.Tensor, fmt, U: torch.Tensor, dead: torch.Tensor,
                          act_sq: torch.Tensor | None = None, n_cand: int = 64, t_lo: float = 0.7, t_hi: float = 1.0,
                          out: Packed | None = None, stream=None) -> Packed:
    """GPTQ on the preset's grid: quantize W (fp32 [N][K], CUDA) into any
    format with the factor of rq_gptq_prepare. Returns the Packed matrix (same
    planes as rq_quantize_pack)."""
    N, K = W.shape
    if out is None:
        out = alloc_packed(fmt, K, N, W.device)
    sr = RqSearch(int(n_cand), float(t_lo), float(t_hi))
    d = out.desc()
    _check(_lib().rq_gptq_quantize_pack(_ptr(W), int(K), int(N), _ptr(U), _ptr(dead), _ptr(act_sq), ctypes.byref(sr),
                                        ctypes.byref(d), _stream(stream)), "rq_gptq_quantize_pack")
    return out


def rq_device_status(stream=None) -> int:
    """Read and clear the device status word (synchronizes the stream)."""
    word = ctypes.c_int(0)
    st = _lib().rq_device_status(_stream(stream), ctypes.byref(word))
    if st not in (RQ_OK, RQ_ERR_DEVICE_TIMEOUT, RQ_ERR_NOT_POSITIVE_DEFINITE):
        raise RqError(st, "rq_device_status")
    return word.value


def rq_test_hooks(wait_ns: int = 0, flags: int = 0) -> None:
    """Testing hook: the bound of every device wait (0 = the default 2 s)
    and flags (1 = issue no weight copies, so the waits run out)."""
    _check(_lib().rq_test_hooks(int(wait_ns), int(flags)), "rq_test_hooks")


# short aliases
quantize_pack = rq_quantize_pack
wgemm = rq_wgemm
wgemm_batch = rq_wgemm_batch
dequant = rq_dequant
packed_size = rq_packed_size
