"""Python binding of libmuon.so (ctypes).

Argument marshalling only: every step of the computation runs in the CUDA
library. PyTorch supplies device memory (outputs and workspaces are torch
tensors) and the current CUDA stream. If the library is missing, loading it
raises: there is no fallback.
"""

from __future__ import annotations

import ctypes as C
import os
from contextlib import nullcontext
from dataclasses import dataclass, field

HERE = os.path.dirname(os.path.abspath(__file__))
# MUON_BOUNDS_CHECK=1 loads the bounds-checked debug build (built by
# `python -m newton_schulz_10_b200.build --debug`): the same library with
# device-side index checks that report MUON_ERR_INVALID_ARG.
LIB_PATH = os.path.join(HERE, "libmuon_check.so" if os.environ.get("MUON_BOUNDS_CHECK") == "1" else "libmuon.so")
MAX_T = 16

# muon_status
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_WORKSPACE, ERR_CUDA, ERR_NONFINITE, \
    ERR_TIMEOUT, ERR_UNSUPPORTED = range(10)
# muon_dtype
F32, BF16, F16 = 0, 1, 2
F16X2 = 3  # compute type of the stack update: two fp16 planes per operand
# muon_norm
NORM_L1, NORM_L2 = 0, 1

EXPORTS = ("muon_set_wait_timeout_ns", "muon_set_gemm_cta_pair", "muon_status_str", "muon_rows_for_fraction", "muon_ns_params_default",
           "muon_ns_workspace_size", "ns_polar", "gram_ns_polar", "normuon_scale", "muon_select_workspace_size",
           "select_rows", "muon_workspace_size", "muon_step", "muon_step_profiled", "muon_kernel_launch_count",
           "select_rows_noalloc", "muon_step_events", "muon_set_gemm_chain", "muon_momentum",
           "muon_orthogonalize", "muon_apply_update", "grouped_matmul", "grouped_matmul_dx", "grouped_matmul_dw",
           "grouped_workspace_size", "muon_stack_params_default", "muon_stack_workspace_size", "muon_stack_step")


class NsParams(C.Structure):
    _fields_ = [("T", C.c_int32), ("coeffs", (C.c_float * 3) * MAX_T), ("norm_eps", C.c_float),
                ("gram", C.c_int32), ("restart_at", C.c_int32), ("compute", C.c_int32)]


class Matrix(C.Structure):
    _fields_ = [("W", C.c_void_p), ("M", C.c_void_p), ("G", C.c_void_p), ("v", C.c_void_p),
                ("rows", C.c_int64), ("cols", C.c_int64)]


class Params(C.Structure):
    _fields_ = [("mu", C.c_float), ("lr", C.c_float), ("ns", NsParams), ("normuon", C.c_int32),
                ("beta2", C.c_float), ("normuon_eps", C.c_float), ("dion3", C.c_int32),
                ("frac_num", C.c_int32), ("frac_den", C.c_int32), ("select_norm", C.c_int32),
                ("dev_status", C.c_void_p)]


class StepProfile(C.Structure):
    _fields_ = [("ms_total", C.c_float), ("ms_prologue", C.c_float), ("ms_ns", C.c_float),
                ("ms_normuon", C.c_float), ("ms_update", C.c_float), ("kernel_launches", C.c_int64),
                ("gemm_launches", C.c_int64), ("ns_flops", C.c_double), ("ns_flops_dense", C.c_double),
                ("ns_flops_executed", C.c_double), ("bytes_prologue", C.c_double), ("bytes_update", C.c_double)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class Grouped(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("experts", C.c_int32), ("tokens", C.c_int64), ("n", C.c_int64), ("k", C.c_int64),
                ("ldx", C.c_int64), ("ldy", C.c_int64), ("ldw", C.c_int64), ("w_stride", C.c_int64),
                ("offsets", C.c_void_p), ("dev_status", C.c_void_p)]


class StackArray(C.Structure):
    _fields_ = [("W", C.c_void_p), ("M", C.c_void_p), ("G", C.c_void_p), ("copy", C.c_void_p),
                ("w_dtype", C.c_int32), ("g_dtype", C.c_int32), ("copy_dtype", C.c_int32),
                ("count", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("w_stride", C.c_int64), ("w_ld", C.c_int64), ("m_stride", C.c_int64), ("m_ld", C.c_int64),
                ("g_stride", C.c_int64), ("g_ld", C.c_int64), ("copy_stride", C.c_int64), ("copy_ld", C.c_int64)]


class StackParams(C.Structure):
    _fields_ = [("mu", C.c_float), ("lr", C.c_float), ("weight_decay", C.c_float), ("scale", C.c_float),
                ("nesterov", C.c_int32), ("ns", NsParams), ("dev_status", C.c_void_p)]


class MuonError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_str(code)}")


_lib = None


def lib() -> C.CDLL:
    """Load libmuon.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m newton_schulz_10_b200.build`")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_float
        L.muon_set_wait_timeout_ns.argtypes = [C.c_uint64]
        L.muon_set_wait_timeout_ns.restype = None
        L.muon_set_gemm_cta_pair.argtypes = [i32]
        L.muon_set_gemm_cta_pair.restype = None
        L.muon_set_gemm_chain.argtypes = [i32]
        L.muon_set_gemm_chain.restype = None
        L.muon_status_str.argtypes = [i32]
        L.muon_status_str.restype = C.c_char_p
        L.muon_rows_for_fraction.argtypes = [i64, i32, i32]
        L.muon_rows_for_fraction.restype = i64
        L.muon_ns_params_default.argtypes = [C.POINTER(NsParams)]
        L.muon_ns_params_default.restype = None
        L.muon_ns_workspace_size.argtypes = [i64, i64, C.POINTER(NsParams)]
        L.muon_ns_workspace_size.restype = sz
        for name in ("ns_polar", "gram_ns_polar"):
            fn = getattr(L, name)
            fn.argtypes = [vp, i32, vp, i32, i64, i64, C.POINTER(NsParams), vp, sz, vp]
            fn.restype = i32
        L.normuon_scale.argtypes = [vp, i32, i64, i64, vp, vp, f32, f32, vp, vp, vp]
        L.normuon_scale.restype = i32
        L.muon_select_workspace_size.argtypes = [i64]
        L.muon_select_workspace_size.restype = sz
        L.select_rows.argtypes = [vp, i64, i64, i64, i32, vp, vp, sz, vp]
        L.select_rows.restype = i32
        L.select_rows_noalloc.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp]
        L.select_rows_noalloc.restype = i32
        L.muon_workspace_size.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params)]
        L.muon_workspace_size.restype = sz
        L.muon_step.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), vp, sz, vp]
        L.muon_step.restype = i32
        L.muon_step_profiled.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), vp, sz, vp,
                                         C.POINTER(StepProfile)]
        L.muon_step_profiled.restype = i32
        L.muon_step_events.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), vp, sz, vp, C.POINTER(vp)]
        L.muon_step_events.restype = i32
        L.muon_momentum.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), vp]
        L.muon_momentum.restype = i32
        L.muon_orthogonalize.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), C.POINTER(vp), C.POINTER(vp),
                                         C.POINTER(vp), vp, sz, vp]
        L.muon_orthogonalize.restype = i32
        L.muon_apply_update.argtypes = [C.POINTER(Matrix), i32, C.POINTER(Params), C.POINTER(vp), C.POINTER(vp),
                                        C.POINTER(vp), vp]
        L.muon_apply_update.restype = i32
        for name in ("grouped_matmul", "grouped_matmul_dx"):
            fn = getattr(L, name)
            fn.argtypes = [C.POINTER(Grouped), vp, vp, vp, vp]
            fn.restype = i32
        L.grouped_matmul_dw.argtypes = [C.POINTER(Grouped), vp, vp, vp, i32, f32, f32, vp, sz, vp]
        L.grouped_matmul_dw.restype = i32
        L.grouped_workspace_size.argtypes = [i32]
        L.grouped_workspace_size.restype = sz
        L.muon_stack_params_default.argtypes = [C.POINTER(StackParams)]
        L.muon_stack_params_default.restype = None
        L.muon_stack_workspace_size.argtypes = [C.POINTER(StackArray), i32, C.POINTER(StackParams)]
        L.muon_stack_workspace_size.restype = sz
        L.muon_stack_step.argtypes = [C.POINTER(StackArray), i32, C.POINTER(StackParams), vp, sz, vp]
        L.muon_stack_step.restype = i32
        L.muon_kernel_launch_count.argtypes = []
        L.muon_kernel_launch_count.restype = i64
        _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().muon_status_str(code).decode()


def _check(code: int, where: str) -> None:
    if code != OK:
        raise MuonError(code, where)


# ---------------------------------------------------------------------------
# parameters
# ---------------------------------------------------------------------------

WORKLOAD_COEFFS = (3.4445, -4.7750, 2.0315)


def ns_params(T: int = 5, coeffs=None, norm_eps: float = 1e-7, gram: bool = False, restart_at: int = 3,
              compute: int = BF16) -> NsParams:
    p = NsParams()
    lib().muon_ns_params_default(C.byref(p))
    p.T = T
    if coeffs is not None:
        coeffs = list(coeffs)
        if len(coeffs) == 3 and not hasattr(coeffs[0], "__len__"):
            coeffs = [coeffs] * T
        for t, (a, b, c) in enumerate(coeffs[:MAX_T]):
            p.coeffs[t][0], p.coeffs[t][1], p.coeffs[t][2] = a, b, c
    p.norm_eps = norm_eps
    p.gram = int(gram)
    p.restart_at = restart_at
    p.compute = compute
    return p


def step_params(mu=0.95, lr=0.02, ns: NsParams | None = None, normuon=False, beta2=0.95, normuon_eps=1e-8,
                dion3=False, frac=(1, 1), select_norm=NORM_L1, dev_status=None) -> Params:
    p = Params()
    p.mu, p.lr = mu, lr
    p.ns = ns if ns is not None else ns_params()
    p.normuon, p.beta2, p.normuon_eps = int(normuon), beta2, normuon_eps
    p.dion3 = int(dion3)
    p.frac_num, p.frac_den = frac
    p.select_norm = select_norm
    p.dev_status = None if dev_status is None else _ptr(dev_status)
    return p


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}[t.dtype]


def workspace(nbytes: int, device=None):
    """A caller-owned workspace tensor of at least nbytes (256-byte aligned)."""
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def kernel_launch_count() -> int:
    """Kernels this library queued from the calling thread so far."""
    return lib().muon_kernel_launch_count()


def set_gemm_cta_pair(enable: bool) -> None:
    """True (default): CTA-pair tensor-core GEMM; False: single-CTA kernel."""
    lib().muon_set_gemm_cta_pair(int(bool(enable)))


def set_gemm_chain(enable: bool) -> None:
    """True: each Newton-Schulz chain runs as one fused persistent launch;
    False (default): one launch per product."""
    lib().muon_set_gemm_chain(int(bool(enable)))


def set_wait_timeout_ns(ns: int) -> None:
    lib().muon_set_wait_timeout_ns(int(ns))


def rows_for_fraction(n: int, f_num: int, f_den: int) -> int:
    return lib().muon_rows_for_fraction(n, f_num, f_den)


def ns_workspace_size(rows: int, cols: int, p: NsParams) -> int:
    return lib().muon_ns_workspace_size(rows, cols, C.byref(p))


def _polar(name, X, p: NsParams, out_dtype, ws, stream):
    import torch
    assert X.dim() == 2 and X.is_contiguous()
    O = torch.empty(X.shape, dtype=out_dtype or X.dtype, device=X.device)
    if ws is None:
        ws = workspace(ns_workspace_size(X.shape[0], X.shape[1], p), X.device)
    code = getattr(lib(), name)(_ptr(X), _dtype_code(X), _ptr(O), _dtype_code(O), X.shape[0], X.shape[1],
                                C.byref(p), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, name)
    return O, ws


def ns_polar(X, p: NsParams | None = None, out_dtype=None, ws=None, stream=None):
    """O ~= polar(X) by standard (or, with p.gram, Gram) Newton-Schulz.
    Returns (O, workspace); the first 4 workspace bytes hold the device status."""
    return _polar("ns_polar", X, p or ns_params(), out_dtype, ws, stream)


def gram_ns_polar(X, p: NsParams | None = None, out_dtype=None, ws=None, stream=None):
    return _polar("gram_ns_polar", X, p or ns_params(gram=True, compute=F16), out_dtype, ws, stream)


def normuon_scale(O, v, beta2=0.95, eps=1e-8, rows=None, dev_status=None, stream=None):
    """Row scales of Eq. (2) for O (k x m); updates v in place."""
    import torch
    k, m = O.shape
    out = torch.empty(k, dtype=torch.float32, device=O.device)
    code = lib().normuon_scale(_ptr(O), _dtype_code(O), k, m, _ptr(v), _ptr(rows), beta2, eps, _ptr(out),
                               _ptr(dev_status), _stream(stream))
    _check(code, "normuon_scale")
    return out


def select_rows(M, k: int, norm: int = NORM_L1, ws=None, stream=None):
    import torch
    n, m = M.shape
    idx = torch.empty(k, dtype=torch.int32, device=M.device)
    if ws is None:
        ws = workspace(lib().muon_select_workspace_size(n), M.device)
    code = lib().select_rows(_ptr(M), n, m, k, norm, _ptr(idx), _ptr(ws), ws.numel(), _stream(stream))
    _check(code, "select_rows")
    return idx


def select_rows_noalloc(M, k: int, norm: int = NORM_L1, idx=None, dev_status=None, stream=None):
    """select_rows without a workspace (fixed scratch inside the library; at
    most 65536 rows; calls that overlap on the GPU race). idx may be passed
    in to avoid allocating the output here too."""
    import torch
    n, m = M.shape
    if idx is None:
        idx = torch.empty(k, dtype=torch.int32, device=M.device)
    code = lib().select_rows_noalloc(_ptr(M), n, m, k, norm, _ptr(idx), _ptr(dev_status), _stream(stream))
    _check(code, "select_rows_noalloc")
    return idx


def _matrices(mats):
    arr = (Matrix * max(len(mats), 1))()
    for i, m in enumerate(mats):
        W, M, G = m[0], m[1], m[2]
        v = m[3] if len(m) > 3 else None
        shape = next(t for t in (W, M, G) if t is not None).shape
        arr[i] = Matrix(_ptr(W), _ptr(M), _ptr(G), _ptr(v), shape[0], shape[1])
    return arr


def workspace_size(mats, p: Params) -> int:
    return lib().muon_workspace_size(_matrices(mats), len(mats), C.byref(p))


@dataclass
class Step:
    """A prepared optimizer step: the matrix table and a workspace, reused
    across calls (allocation happens once, in __init__)."""
    mats: list
    params: Params
    ws: object = None
    _table: object = field(default=None, repr=False)

    def __post_init__(self):
        self._table = _matrices(self.mats)
        if self.ws is None:
            n = lib().muon_workspace_size(self._table, len(self.mats), C.byref(self.params))
            if n == 0 and len(self.mats) > 0:
                raise MuonError(ERR_INVALID_ARG, "muon_workspace_size")
            device = self.mats[0][0].device if self.mats else "cuda"
            self.ws = workspace(n, device)

    def __call__(self, stream=None) -> None:
        code = lib().muon_step(self._table, len(self.mats), C.byref(self.params), _ptr(self.ws), self.ws.numel(),
                               _stream(stream))
        _check(code, "muon_step")

    def profiled(self, stream=None) -> StepProfile:
        """Run the step with per-phase CUDA events (synchronises)."""
        prof = StepProfile()
        code = lib().muon_step_profiled(self._table, len(self.mats), C.byref(self.params), _ptr(self.ws),
                                        self.ws.numel(), _stream(stream), C.byref(prof))
        _check(code, "muon_step_profiled")
        return prof

    def timed(self, events, stream=None) -> None:
        """Run the step, recording the five torch.cuda.Event objects in
        `events` (enable_timing=True) at its phase boundaries on the stream:
        start, NS chain start, NS chain end, NorMuon end, update end. Does not
        synchronise."""
        import torch
        ts = stream if stream is not None else torch.cuda.current_stream()
        for e in events:
            if not e.cuda_event:  # torch creates the CUDA event at its first record
                e.record(ts)
        handles = (C.c_void_p * 5)(*[e.cuda_event for e in events])
        code = lib().muon_step_events(self._table, len(self.mats), C.byref(self.params), _ptr(self.ws),
                                      self.ws.numel(), _stream(stream), handles)
        _check(code, "muon_step_events")

    def device_status(self) -> int:
        """Deferred device status of the last step (synchronises)."""
        import torch
        if self.params.dev_status:
            raise RuntimeError("status goes to the caller's dev_status")
        return int(self.ws[:4].view(torch.int32).item())


def _ptrs(ts):
    arr = (C.c_void_p * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t)
    return arr


def operand_dtype(p: Params):
    """torch dtype of the orthogonalised rows muon_orthogonalize writes."""
    import torch
    return {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}[p.ns.compute]


def momentum(mats, p: Params, stream=None) -> None:
    """M <- mu M + G (M <- M + G for Dion3) on every (W, M, G[, v]) of mats."""
    _check(lib().muon_momentum(_matrices(mats), len(mats), C.byref(p), _stream(stream)), "muon_momentum")


def orthogonalize(mats, p: Params, O, row_scale, selected=None, ws=None, stream=None):
    """Norms / selection, Newton-Schulz and NorMuon on the momentum of mats;
    writes O[i] (rows x cols, operand dtype), row_scale[i] (rows) and, for
    Dion3, selected[i] (rows, int32). Returns the workspace."""
    table = _matrices(mats)
    if ws is None:
        ws = workspace(lib().muon_workspace_size(table, len(mats), C.byref(p)), mats[0][1].device if mats else None)
    code = lib().muon_orthogonalize(table, len(mats), C.byref(p), _ptrs(O), _ptrs(row_scale),
                                    _ptrs(selected) if selected is not None else None, _ptr(ws), ws.numel(),
                                    _stream(stream))
    _check(code, "muon_orthogonalize")
    return ws


def apply_update(mats, p: Params, O, row_scale, selected=None, stream=None) -> None:
    """W -= lr * row_scale * O per row (Dion3: M *= mu on the selected rows)."""
    code = lib().muon_apply_update(_matrices(mats), len(mats), C.byref(p), _ptrs(O), _ptrs(row_scale),
                                   _ptrs(selected) if selected is not None else None, _stream(stream))
    _check(code, "muon_apply_update")


def muon_step(mats, p: Params | None = None, ws=None, stream=None) -> Step:
    """One optimizer step over mats = [(W, M, G[, v]), ...] (fp32 CUDA
    tensors, updated in place). Returns the Step (reusable)."""
    s = Step(list(mats), p or step_params(), ws)
    s(stream)
    return s


# ---------------------------------------------------------------------------
# products grouped by expert (explicit forward and gradient calls, as in the
# rest of this binding: nothing here is recorded by autograd)
# ---------------------------------------------------------------------------


def _need(ok: bool, code: int, where: str) -> None:
    if not ok:
        raise MuonError(code, where)


def _code_of(t, where: str) -> int:
    import torch
    code = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}.get(t.dtype)
    _need(code is not None, ERR_DTYPE, where)
    return code


def _torch():
    """torch and its 16-bit types, looked up once: the calls below are made for
    a handful of tokens at a time, where every microsecond on the host counts."""
    global _T
    import torch
    _T = (torch, torch.bfloat16, torch.float16, torch.int32, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    torch.cuda.init()  # _cuda_getDevice needs it
    return _T


_T = None


def _call_on(device: int, stream, fn, args, where: str) -> None:
    """fn(*args, stream) with the CUDA device of the tensors current, on the
    given stream or that device's current one."""
    t = _T or _torch()
    raw = t[4](device) if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    if t[5]() == device:
        code = fn(*args, raw)
    else:
        with t[0].cuda.device(device):
            code = fn(*args, raw)
    if code != OK:
        raise MuonError(code, where)


def _on(stream, device):
    """Context in which a call's own allocations come from the memory pool of
    the stream that uses them: the caching allocator hands a freed block out
    again in the order of the stream it was allocated on, so memory of another
    stream may still be in use there, or be handed out while this one runs."""
    if stream is None or device.type != "cuda":  # a tensor elsewhere is refused by the checks
        return nullcontext()
    import torch
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(stream, device))


def _new(like, shape, stream):
    if stream is None:
        return like.new_empty(shape)
    with _on(stream, like.device):
        return like.new_empty(shape)


def _grouped(where, x, y, w, offsets, dev_status):
    """The descriptor and device of a call: x (tokens, k), y (tokens, n), w (experts, n, k)."""
    try:
        (tokens, k), (yt, n), (experts, wn, wk), (entries,) = x.shape, y.shape, w.shape, offsets.shape
    except ValueError:
        raise MuonError(ERR_SHAPE, where) from None
    if wk != k or wn != n or yt != tokens or entries != experts + 1:
        raise MuonError(ERR_SHAPE, where)
    dtype = x.dtype
    device = x.get_device()
    if device < 0:  # before torch's CUDA side is needed
        import torch
        bf16, f16, i32 = torch.bfloat16, torch.float16, torch.int32
    else:
        bf16, f16, i32 = (_T or _torch())[1:4]
    if y.dtype != dtype or (dtype != bf16 and dtype != f16) or offsets.dtype != i32:
        raise MuonError(ERR_DTYPE, where)
    if device < 0 or y.get_device() != device or w.get_device() != device or offsets.get_device() != device:
        raise MuonError(ERR_INVALID_ARG, where)
    (xr, xc), (yr, yc), (we, wr, wc) = x.stride(), y.stride(), w.stride()
    if (k > 1 and (xc != 1 or wc != 1)) or (n > 1 and yc != 1) or (experts > 0 and offsets.stride(0) != 1):
        raise MuonError(ERR_SHAPE, where)
    status = None
    if dev_status is not None:
        if dev_status.dtype != i32 or dev_status.get_device() != device:
            raise MuonError(ERR_INVALID_ARG, where)
        status = dev_status.data_ptr()
    # the stride of a single row is never used: any aligned value will do
    if tokens <= 1:
        xr, yr = (k + 7) & ~7, (n + 7) & ~7
    if n <= 1:
        wr = (k + 7) & ~7
    return Grouped(BF16 if dtype == bf16 else F16, experts, tokens, n, k, xr, yr, wr, we if experts > 1 else 0,
                   offsets.data_ptr(), status), device


def grouped_matmul(x, w, offsets, out=None, dev_status=None, stream=None):
    """y[r] = x[r] @ w[e].T for the rows r of every expert e.

    x (tokens, k) holds the rows sorted by expert, w (experts, n, k) the
    weights (bf16 or fp16, unit column stride, 16-byte rows), offsets
    (experts + 1, int32, on the device) each expert's first row. Rows of `out`
    (tokens, n) that belong to no expert keep their values."""
    if out is None:
        _need(x.dim() == 2 and w.dim() == 3, ERR_SHAPE, "grouped_matmul")
        out = _new(x, (x.shape[0], w.shape[1]), stream)
    if w.dtype != x.dtype:
        raise MuonError(ERR_DTYPE, "grouped_matmul")
    g, device = _grouped("grouped_matmul", x, out, w, offsets, dev_status)
    _call_on(device, stream, (_lib or lib()).grouped_matmul, (C.byref(g), x.data_ptr(), w.data_ptr(), out.data_ptr()),
             "grouped_matmul")
    return out


def grouped_matmul_dx(dy, w, offsets, out=None, dev_status=None, stream=None):
    """dx[r] = dy[r] @ w[e]: the gradient of grouped_matmul for its rows."""
    if out is None:
        _need(dy.dim() == 2 and w.dim() == 3, ERR_SHAPE, "grouped_matmul_dx")
        out = _new(dy, (dy.shape[0], w.shape[2]), stream)
    if w.dtype != dy.dtype:
        raise MuonError(ERR_DTYPE, "grouped_matmul_dx")
    g, device = _grouped("grouped_matmul_dx", out, dy, w, offsets, dev_status)
    _call_on(device, stream, (_lib or lib()).grouped_matmul_dx, (C.byref(g), dy.data_ptr(), w.data_ptr(), out.data_ptr()),
             "grouped_matmul_dx")
    return out


def grouped_workspace_size(experts: int) -> int:
    return lib().grouped_workspace_size(experts)


def _ws_bytes(ws, device: int, where: str) -> int:
    """Bytes of a workspace, which has to be one piece of the device's memory."""
    if ws.get_device() != device or not ws.is_contiguous():
        raise MuonError(ERR_INVALID_ARG, where)
    return ws.numel() * ws.element_size()


def _workspace_on(stream, experts: int, device):
    """A workspace of grouped_matmul_dw from the memory pool of its stream."""
    import torch
    with torch.cuda.device(device):
        n = grouped_workspace_size(experts)
    with _on(stream, device):
        return workspace(n, device)


def grouped_matmul_dw(dy, x, offsets, out=None, alpha: float = 1.0, beta: float = 0.0, ws=None, dev_status=None, stream=None):
    """out[e] = alpha * dy_e.T @ x_e + beta * out[e] over the rows of expert e:
    the gradient of grouped_matmul for its weights (experts, n, k), in fp32 or
    the type of dy and x. beta = 0 does not read `out`; without `out` the
    result is fp32. With beta = the momentum decay and an fp32 momentum as
    `out` this is M <- mu M + G without a gradient in memory."""
    where = "grouped_matmul_dw"
    _need(offsets.dim() == 1 and offsets.shape[0] >= 1, ERR_SHAPE, where)
    experts = offsets.shape[0] - 1
    if out is None:
        import torch
        _need(dy.dim() == 2 and x.dim() == 2, ERR_SHAPE, where)
        _need(beta == 0.0, ERR_INVALID_ARG, where)
        with _on(stream, x.device):
            out = torch.empty((experts, dy.shape[1], -(-x.shape[1] // 8) * 8), dtype=torch.float32, device=x.device)[:, :, :x.shape[1]]
    g, device = _grouped(where, x, dy, out, offsets, dev_status)
    if ws is None:
        ws = _workspace_on(stream, experts, x.device)
    _call_dw(where, g, device, dy, x, out, alpha, beta, ws, stream)
    return out


def _call_dw(where, g, device, dy, x, out, alpha, beta, ws, stream):
    size = _ws_bytes(ws, device, where)
    _call_on(device, stream, (_lib or lib()).grouped_matmul_dw, (C.byref(g), dy.data_ptr(), x.data_ptr(), out.data_ptr(),
                                                       _code_of(out, where), alpha, beta, ws.data_ptr(), size), where)


# ---------------------------------------------------------------------------
# the update of stacks of matrices
# ---------------------------------------------------------------------------


def stack_params(mu: float = 0.95, lr: float = 0.02, weight_decay: float = 0.0, scale: float = 1.0, nesterov: bool = False,
                 ns: NsParams | None = None, dev_status=None) -> StackParams:
    """Parameters of a stack update; ns.compute may be F16X2 (two fp16 planes
    per operand on the tensor cores: O off by about 1e-5 up to n = 256, 4e-5
    at 1024 x 1024, 1e-4 at 4096 x 4096; F32 stays at 6e-6)."""
    p = StackParams()
    lib().muon_stack_params_default(C.byref(p))
    p.mu, p.lr, p.weight_decay, p.scale, p.nesterov = mu, lr, weight_decay, scale, int(nesterov)
    if ns is not None:
        p.ns = ns
    if dev_status is not None:
        import torch
        _need(dev_status.is_cuda and dev_status.dtype == torch.int32 and dev_status.numel() >= 1, ERR_INVALID_ARG, "stack_params")
        p.dev_status = _ptr(dev_status)
        p.status_tensor = dev_status  # lives as long as the parameters that hold its address
    return p


@dataclass
class Stack:
    """count x rows x cols tensors (views with any strides and adjacent
    columns): weights W (fp32, bf16 or fp16), fp32 momentum M, gradient G
    (fp32, bf16, fp16; None when the momentum already holds it) and an
    optional 16-bit copy of the new weights."""
    W: object
    M: object
    G: object = None
    copy: object = None


def _stacks(stacks, where: str):
    import torch
    arr = (StackArray * max(len(stacks), 1))()
    for i, k in enumerate(stacks):
        shape = k.W.shape
        _need(len(shape) == 3, ERR_SHAPE, where)
        given = [t for t in (k.W, k.M, k.G, k.copy) if t is not None]
        _need(k.M is not None and all(t.shape == shape for t in given), ERR_SHAPE, where)
        _need(shape[2] <= 1 or all(t.stride(2) == 1 for t in given), ERR_SHAPE, where)
        _need(k.M.dtype == torch.float32, ERR_DTYPE, where)
        _need(all(t.is_cuda and t.device == stacks[0].W.device for t in given), ERR_INVALID_ARG, where)
        a = arr[i]
        a.W, a.M, a.G, a.copy = _ptr(k.W), _ptr(k.M), _ptr(k.G), _ptr(k.copy)
        a.count, a.rows, a.cols = shape
        a.w_dtype, a.w_stride, a.w_ld = _code_of(k.W, where), k.W.stride(0), k.W.stride(1)
        a.m_stride, a.m_ld = k.M.stride(0), k.M.stride(1)
        if k.G is not None:
            a.g_dtype, a.g_stride, a.g_ld = _code_of(k.G, where), k.G.stride(0), k.G.stride(1)
        if k.copy is not None:
            a.copy_dtype, a.copy_stride, a.copy_ld = _code_of(k.copy, where), k.copy.stride(0), k.copy.stride(1)
    return arr


@dataclass
class StackStep:
    """A prepared update of stacks: the table and a workspace, reused by every
    call. The tensors are updated in place:

        step = StackStep([Stack(W, M, G)], stack_params(...))
        step()                                # M, W from this step's G
        step = StackStep([Stack(W, M)], ...)  # no gradient tensor:
        step.accumulate(0, dy, x, offsets)    # M <- mu M + dy_e^T x_e
        step()                                # W from M

    The workspace belongs to the stream that is current at construction: order
    a call on another stream after it, and keep the object until that call has
    run.
    """
    stacks: list
    params: StackParams
    ws: object = None
    _table: object = field(default=None, repr=False)
    _grouped_ws: list = field(default=None, repr=False)
    _deferred: object = field(default=None, repr=False)  # status word of the accumulate calls

    def __post_init__(self):
        where = "muon_stack_step"
        self._table = _stacks(self.stacks, where)
        self._grouped_ws = [{} for _ in self.stacks]
        if any(k.G is None for k in self.stacks):
            import torch
            self._deferred = torch.zeros(1, dtype=torch.int32, device=self.stacks[0].W.device)
        if self.ws is None:
            import torch
            device = self.stacks[0].W.device if self.stacks else "cuda"
            if self.stacks:
                with torch.cuda.device(device):
                    n = lib().muon_stack_workspace_size(self._table, len(self.stacks), C.byref(self.params))
                _need(n > 0, ERR_INVALID_ARG, "muon_stack_workspace_size")
            else:
                n = 0
            self.ws = workspace(n, device)
        if self.stacks:
            device = self.stacks[0].W.get_device()
            status = getattr(self.params, "status_tensor", None)
            _need(status is None or status.get_device() == device, ERR_INVALID_ARG, where)
            self._ws_bytes = _ws_bytes(self.ws, device, where)

    def __call__(self, stream=None) -> None:
        if not self.stacks:
            return
        _call_on(self.stacks[0].W.get_device(), stream, lib().muon_stack_step,
                 (self._table, len(self.stacks), C.byref(self.params), _ptr(self.ws), self._ws_bytes), "muon_stack_step")

    def accumulate(self, i: int, dy, x, offsets, stream=None) -> None:
        """M <- mu M + dy_e^T x_e for the experts of stack i, whose G is None:
        the momentum step straight from an expert layer's rows. Deferred
        errors (offsets out of order, a wait that ran out) go to the
        parameters' dev_status, else to device_status()."""
        where = "StackStep.accumulate"
        k = self.stacks[i]
        _need(k.G is None, ERR_INVALID_ARG, where)
        if stream is None:
            raw = (_T or _torch())[4](k.M.get_device())
        else:
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        g, device = _grouped(where, x, dy, k.M, offsets, None)
        g.dev_status = self.params.dev_status or self._deferred.data_ptr()
        kept = self._grouped_ws[i]  # one per stream, all kept: a captured graph may hold any of them
        if raw not in kept:
            kept[raw] = _workspace_on(stream, k.M.shape[0], k.M.device)
        _call_dw(where, g, device, dy, x, k.M, 1.0, self.params.mu, kept[raw], stream)

    def device_status(self) -> int:
        """Deferred device status of the last step (synchronises). An error of
        accumulate comes first and is kept until it has been returned here:
        the momentum that it left unspecified outlives the step."""
        import torch
        if self.params.dev_status:
            raise RuntimeError("status goes to the caller's dev_status")
        if self._deferred is not None:
            torch.cuda.synchronize(self._deferred.device)  # accumulate may have run on any stream
            code = int(self._deferred.item())
            if code != OK:
                self._deferred.zero_()
                return code
        if not self.stacks:
            return OK  # no call writes the word
        return int(self.ws.view(-1).view(torch.uint8)[:4].view(torch.int32).item())


def stack_step(stacks, p: StackParams | None = None, ws=None, stream=None) -> StackStep:
    """One update of stacks = [Stack(W, M, G[, copy]), ...]. Returns the
    StackStep (reusable)."""
    stacks = list(stacks)
    p = p or stack_params()
    if stream is not None and ws is None and stacks:
        with _on(stream, stacks[0].W.device):
            s = StackStep(stacks, p)
    else:
        s = StackStep(stacks, p, ws)
    s(stream)
    return s
