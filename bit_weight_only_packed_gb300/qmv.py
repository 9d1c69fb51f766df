"""Thin ctypes binding of the C ABI in include/qmv.h (libqmv.so).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the ABI.  torch is used for device memory and streams.  If the
native library is missing the import of this module raises (there is no
fallback of any kind).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libqmv.so")

QMV_OK = 0
QMV_ERR_INVALID_ARG = -1
QMV_ERR_UNSUPPORTED = -2
QMV_ERR_ALIGNMENT = -3
QMV_ERR_SHAPE = -4
QMV_ERR_CUDA = -5
QMV_ERR_TIMEOUT = -6
QMV_ERR_WORKSPACE = -7
QMV_F32, QMV_F16, QMV_BF16 = 0, 1, 2
QMV_FAST, QMV_EXACT = 0, 1
QMV_PACK_HEADER_BYTES, QMV_PACK_VERSION = 64, 1

# every entry point declared in include/qmv.h, with its ctypes signature
_P, _I, _F, _SZP = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
SIGNATURES = {
    "qmv_create_pack": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _SZP, _SZP]),
    "qmv_pack_weights": (_I, [_P, _P, _P, _P, _P, _P]),
    "qmv_workspace_bytes": (ctypes.c_size_t, [_P, _I, _I, _I, _I]),
    "qmv_gemv": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _I, _I, _P, ctypes.c_size_t, _P]),
    "qmv_fused_rmsnorm_gemv": (_I, [_P, _I, _P, _P, _P, _F, _P, _P, _I, _I, _P, ctypes.c_size_t, _P]),
    "qmv_chunk_gemm": (_I, [_P, _I, _P, _P, _I, _I, _P, ctypes.c_size_t, _P]),
    "qmv_unpack_codes": (_I, [_P, _P, _P]),
    "qmv_pack_info": (_I, [_P, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I),
                           ctypes.POINTER(_I)]),
    "qmv_destroy_pack": (_I, [_P]),
    "qmv_pack_header": (_I, [_P, _P]),
    "qmv_create_pack_from_header": (_I, [ctypes.POINTER(_P), _P, _SZP, _SZP]),
    "qmv_bind_packed": (_I, [_P, _P, _P]),
    "qmv_status_string": (ctypes.c_char_p, [_I]),
    "qmv_last_cuda_error": (_I, []),
    "qmv_device_error": (_I, [ctypes.POINTER(_I), _I]),
    "qmv_set_pdl": (_I, [_I]),
    "qmv_gemv_gather": (_I, [_P, _I, _P, _I, _P, _P, _I, _I, _P]),
    "qmv_argmax_workspace_bytes": (ctypes.c_size_t, []),
    "qmv_gemv_argmax": (_I, [_P, _P, _P, _P, _F, _P, _P, _I, _I, _P, _P, _P, _P]),
    "qmv_chain_workspace_bytes": (ctypes.c_size_t, [_I]),
    "qmv_chain_create": (_I, [ctypes.POINTER(_P), _I, _P, ctypes.c_size_t]),
    "qmv_chain_create_no_alloc": (_I, [ctypes.POINTER(_P), _I]),
    "qmv_chain_add_gemv": (_I, [_P, _P, _P, _P, _I, _I]),
    "qmv_chain_add_fused_rmsnorm_gemv": (_I, [_P, _P, _P, _P, _P, _F, _P, _P, _I, _I]),
    "qmv_chain_run": (_I, [_P, _P]),
    "qmv_chain_info": (_I, [_P, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "qmv_chain_destroy": (_I, [_P]),
    "qmv_w4_create": (_I, [ctypes.POINTER(_P), _I, _I, _I, _I, _I, _SZP]),
    "qmv_w4_pack": (_I, [_P, _P, _P, _P, _P, _P]),
    "qmv_w4_bind": (_I, [_P, _P]),
    "qmv_w4_unpack": (_I, [_P, _P, _P]),
    "qmv_w4_info": (_I, [_P, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I),
                         ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "qmv_w4_destroy": (_I, [_P]),
    "qmv_w4_gemv": (_I, [_P, _I, _P, _I, _I, _P, _I, _I, _P]),
    "qmv_block_norm": (_I, [_I, _I, _P, _I, _I, _P, _I, _P, _P, _I, _F, _F, _P, _F, _F, _P, _I, _P, _I, _I,
                            _P]),
    "qmv_softmax": (_I, [_I, _I, _P, _I, _I, _P, _F, _P, _I, _P]),
    "qmv_verify_draft": (_I, [_I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
}


class QmvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _lib.qmv_status_string(status).decode()
        if status == QMV_ERR_CUDA:
            msg += f" (cudaError {_lib.qmv_last_cuda_error()})"
        super().__init__(f"{fn}: {msg} [{status}]")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqmv.so is not built ({LIB_PATH}); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _check(fn: str, rc: int):
    if rc != QMV_OK:
        raise QmvError(fn, rc)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# Calls on a stream of their own (stream=): torch hands freed memory out again in the
# order of the stream that it was allocated on, so a fresh tensor comes from the memory of
# the stream that writes it (memory of the current stream may still be written there by work
# queued earlier), and tensors that a torch stream reads are recorded on it.  With a raw
# stream handle the caller keeps the inputs alive until the work is done: the handle may no
# longer exist when they are freed.

def _other(stream, device):
    """The stream as torch's, if it is not torch's current one of the device."""
    if stream is None or device.type != "cuda" or _stream(stream) == torch.cuda.current_stream(device).cuda_stream:
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _fresh(shape, dtype, device, stream):
    """A fresh tensor for work on a stream; it may then be used on the current one too."""
    s = _other(stream, device)
    if s is None:
        return torch.empty(shape, dtype=dtype, device=device)
    cur = torch.cuda.current_stream(device)
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(cur)
    return t


def _record(stream, *tensors):
    """The tensors that work on another torch stream uses keep their memory until it is done."""
    if isinstance(stream, torch.cuda.Stream):
        for t in tensors:
            if t is not None and t.is_cuda and _other(stream, t.device) is not None:
                t.record_stream(stream)


def _dptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return t.data_ptr()


_YDT = {QMV_F32: torch.float32, QMV_F16: torch.float16}


def _need(name, t, dtype, n):
    """The tensor behind a pointer argument has the dtype the kernels read or
    write and at least the n elements they touch from its start.  The ABI
    takes bare pointers and cannot check sizes, so this is checked here,
    before any call.  A y_dtype outside QMV_F32/QMV_F16 skips the dtype
    check; the ABI rejects that value itself."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: needs at least {n} elements, has {t.numel()}")


def _need_bytes(name, t, n):
    if t.numel() * t.element_size() < n:
        raise ValueError(f"{name}: needs at least {n} bytes, has {t.numel() * t.element_size()}")


class Pack:
    """A packed weight matrix: the host descriptor plus the device buffers
    (allocated with torch) that hold the packed codes and scales."""

    def __init__(self, N: int, K: int, bits: int, group: int, header: bytes = None):
        h = _P()
        cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
        if header is None:
            _check("qmv_create_pack", _lib.qmv_create_pack(ctypes.byref(h), N, K, bits, group,
                                                            ctypes.byref(cb), ctypes.byref(sb)))
        else:
            if len(header) != QMV_PACK_HEADER_BYTES:
                raise ValueError(f"a pack header is {QMV_PACK_HEADER_BYTES} bytes, got {len(header)}")
            buf = ctypes.create_string_buffer(bytes(header), QMV_PACK_HEADER_BYTES)
            _check("qmv_create_pack_from_header", _lib.qmv_create_pack_from_header(
                ctypes.byref(h), buf, ctypes.byref(cb), ctypes.byref(sb)))
        self.handle = h
        if header is not None:
            n, k, b, g = _I(), _I(), _I(), _I()
            _check("qmv_pack_info", _lib.qmv_pack_info(h, ctypes.byref(n), ctypes.byref(k), ctypes.byref(b),
                                                       ctypes.byref(g)))
            N, K, bits, group = n.value, k.value, b.value, g.value
        self.N, self.K, self.bits, self.group = N, K, bits, group
        self.codes_bytes, self.scales_bytes = cb.value, sb.value
        self.words = None
        self.scales = None

    @classmethod
    def from_header(cls, header: bytes) -> "Pack":
        """The pack described by a saved header (qmv_create_pack_from_header);
        bind its reloaded buffers with bind_packed."""
        return cls(0, 0, 0, 0, header=header)

    def header(self) -> bytes:
        return qmv_pack_header(self)

    def bind_packed(self, words: torch.Tensor, scales: torch.Tensor):
        """words, scales: device buffers holding the packed words and scales of
        this shape (as pack_weights left them, e.g. reloaded from a file)."""
        qmv_bind_packed(self, words, scales)
        self.words, self.scales = words, scales
        return self

    @property
    def packed_bytes(self) -> int:
        return self.codes_bytes + self.scales_bytes

    def pack_weights(self, codes: torch.Tensor, scales: torch.Tensor, stream=None, device=None):
        """codes: device int8 [N, K] signed codes; scales: device fp16 [N, K/group]."""
        dev = codes.device if device is None else torch.device(device)
        self.words = _fresh(self.codes_bytes // 4, torch.int32, dev, stream)
        self.scales = _fresh(self.scales_bytes // 2, torch.float16, dev, stream)
        qmv_pack_weights(self, codes, scales, self.words, self.scales, stream)
        return self

    def close(self):
        if self.handle is not None and self.handle.value:
            _lib.qmv_destroy_pack(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qmv_create_pack(N: int, K: int, bits: int, group: int) -> Pack:
    return Pack(N, K, bits, group)


def qmv_pack_weights(p: Pack, codes, scales, d_codes, d_scales, stream=None):
    G = p.K // p.group
    _need("codes", codes, torch.int8, p.N * p.K)
    _need("scales", scales, torch.float16, p.N * G)
    _need_bytes("d_codes", d_codes, p.codes_bytes)
    _need_bytes("d_scales", d_scales, p.scales_bytes)
    _record(stream, codes, scales, d_codes, d_scales)
    _check("qmv_pack_weights", _lib.qmv_pack_weights(
        p.handle, _dptr(codes), _dptr(scales), _dptr(d_codes), _dptr(d_scales), _stream(stream)))


def _out(y, M, N, y_dtype, like, stream):
    if y is None:
        dt = torch.float16 if y_dtype == QMV_F16 else torch.float32
        y = _fresh((M, N), dt, like.device, stream)
    return y


def qmv_workspace_bytes(p: Pack, M: int, y_dtype=QMV_F32, mode=QMV_FAST, fused=False) -> int:
    """Device scratch bytes a call needs (0 for none)."""
    return int(_lib.qmv_workspace_bytes(p.handle, M, y_dtype, mode, 1 if fused else 0))


def workspace(p: Pack, M: int, y_dtype=QMV_F32, mode=QMV_FAST, fused=False, device=None):
    """A workspace tensor for such calls (None when they need none)."""
    n = qmv_workspace_bytes(p, M, y_dtype, mode, fused)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda") if n else None


def _ws(p, M, y_dtype, mode, fused, ws, like, stream=None):
    """The caller's workspace, checked, or (when none is given) a fresh torch
    allocation of the size the call needs: (pointer, bytes, tensor)."""
    n = qmv_workspace_bytes(p, M, y_dtype, mode, fused)
    if ws is None:
        if n == 0:
            return None, 0, None
        ws = _fresh(n, torch.uint8, like.device, stream)
    _need_bytes("workspace", ws, n)
    return _dptr(ws), ws.numel() * ws.element_size(), ws


def qmv_gemv(p: Pack, x, y=None, y_dtype=QMV_F32, mode=QMV_FAST, stream=None, M=None, workspace=None):
    M = x.shape[0] if (M is None and x.dim() == 2) else (M or 1)
    _need("x", x, torch.float16, M * p.K)
    _need("y", y, _YDT.get(y_dtype), M * p.N)
    y = _out(y, M, p.N, y_dtype, x, stream)
    wp, wb, _keep = _ws(p, M, y_dtype, mode, False, workspace, x, stream)
    _record(stream, p.words, p.scales, x, y, _keep)
    _check("qmv_gemv", _lib.qmv_gemv(p.handle, M, p.N, p.K, p.bits, p.group, _dptr(x), _dptr(y),
                                     y_dtype, mode, wp, wb, _stream(stream)))
    return y


def qmv_chunk_gemm(p: Pack, x, y=None, y_dtype=QMV_F32, mode=QMV_FAST, stream=None, workspace=None):
    M = x.shape[0]
    _need("x", x, torch.float16, M * p.K)
    _need("y", y, _YDT.get(y_dtype), M * p.N)
    y = _out(y, M, p.N, y_dtype, x, stream)
    wp, wb, _keep = _ws(p, M, y_dtype, mode, False, workspace, x, stream)
    _record(stream, p.words, p.scales, x, y, _keep)
    _check("qmv_chunk_gemm", _lib.qmv_chunk_gemm(p.handle, M, _dptr(x), _dptr(y), y_dtype, mode,
                                                 wp, wb, _stream(stream)))
    return y


def qmv_fused_rmsnorm_gemv(p: Pack, x, residual, gamma, eps=1e-6, h_out=None, y=None,
                           y_dtype=QMV_F32, mode=QMV_FAST, stream=None, workspace=None):
    M = x.shape[0] if x.dim() == 2 else 1
    _need("x", x, torch.float16, M * p.K)
    _need("residual", residual, torch.float16, M * p.K)
    _need("gamma", gamma, torch.float16, p.K)
    _need("h_out", h_out, torch.float16, M * p.K)
    _need("y", y, _YDT.get(y_dtype), M * p.N)
    y = _out(y, M, p.N, y_dtype, x, stream)
    wp, wb, _keep = _ws(p, M, y_dtype, mode, True, workspace, x, stream)
    _record(stream, p.words, p.scales, x, residual, gamma, h_out, y, _keep)
    _check("qmv_fused_rmsnorm_gemv", _lib.qmv_fused_rmsnorm_gemv(
        p.handle, M, _dptr(x), _dptr(residual), _dptr(gamma), float(eps), _dptr(h_out), _dptr(y),
        y_dtype, mode, wp, wb, _stream(stream)))
    return y


def qmv_gemv_gather(p: Pack, rows_per_expert: int, expert_ids, x, y=None, y_dtype=QMV_F32,
                    mode=QMV_FAST, stream=None):
    """y [1, n_selected * rows_per_expert]: the selected experts' rows times x."""
    n = expert_ids.numel()
    _need("expert_ids", expert_ids, torch.int32, n)
    _need("x", x, torch.float16, p.K)
    _need("y", y, _YDT.get(y_dtype), n * rows_per_expert)
    y = _out(y, 1, n * rows_per_expert, y_dtype, x, stream)
    _record(stream, p.words, p.scales, expert_ids, x, y)
    _check("qmv_gemv_gather", _lib.qmv_gemv_gather(p.handle, rows_per_expert, _dptr(expert_ids), n,
                                                   _dptr(x), _dptr(y), y_dtype, mode, _stream(stream)))
    return y


def qmv_argmax_workspace(device=None):
    """A zeroed workspace for qmv_gemv_argmax (left zero by every completed call)."""
    return torch.zeros(_lib.qmv_argmax_workspace_bytes(), dtype=torch.uint8, device=device or "cuda")


def qmv_gemv_argmax(p: Pack, x, workspace, residual=None, gamma=None, eps=1e-6, h_out=None, y=None,
                    y_dtype=QMV_F32, mode=QMV_FAST, stream=None, index=None, value=None):
    """(index, value) device tensors of the greedy token; y (logits) is stored
    only if given."""
    _need("x", x, torch.float16, p.K)
    _need("residual", residual, torch.float16, p.K)
    _need("gamma", gamma, torch.float16, p.K)
    _need("h_out", h_out, torch.float16, p.K)
    _need("y", y, _YDT.get(y_dtype), p.N)
    _need("index", index, torch.int32, 1)
    _need("value", value, torch.float32, 1)
    _need_bytes("workspace", workspace, _lib.qmv_argmax_workspace_bytes())
    if index is None:
        index = _fresh(1, torch.int32, x.device, stream)
    if value is None:
        value = _fresh(1, torch.float32, x.device, stream)
    _record(stream, p.words, p.scales, x, workspace, residual, gamma, h_out, y, index, value)
    _check("qmv_gemv_argmax", _lib.qmv_gemv_argmax(
        p.handle, _dptr(x), _dptr(residual), _dptr(gamma), float(eps), _dptr(h_out), _dptr(y), y_dtype,
        mode, _dptr(index), _dptr(value), _dptr(workspace), _stream(stream)))
    return index, value


def qmv_unpack_codes(p: Pack, out=None, stream=None):
    if out is None:
        out = _fresh((p.N, p.K), torch.int8, p.words.device, stream)
    _need("out", out, torch.int8, p.N * p.K)
    _record(stream, p.words, out)
    _check("qmv_unpack_codes", _lib.qmv_unpack_codes(p.handle, _dptr(out), _stream(stream)))
    return out


def qmv_pack_info(p: Pack):
    n, k, b, g = _I(), _I(), _I(), _I()
    _check("qmv_pack_info", _lib.qmv_pack_info(p.handle, ctypes.byref(n), ctypes.byref(k),
                                               ctypes.byref(b), ctypes.byref(g)))
    return n.value, k.value, b.value, g.value


def qmv_pack_header(p: Pack) -> bytes:
    buf = ctypes.create_string_buffer(QMV_PACK_HEADER_BYTES)
    _check("qmv_pack_header", _lib.qmv_pack_header(p.handle, buf))
    return buf.raw


def qmv_create_pack_from_header(header: bytes) -> Pack:
    return Pack.from_header(header)


def qmv_bind_packed(p: Pack, d_codes, d_scales):
    _need_bytes("d_codes", d_codes, p.codes_bytes)
    _need_bytes("d_scales", d_scales, p.scales_bytes)
    _check("qmv_bind_packed", _lib.qmv_bind_packed(p.handle, _dptr(d_codes), _dptr(d_scales)))


def qmv_status_string(status: int) -> str:
    return _lib.qmv_status_string(status).decode()


def qmv_last_cuda_error() -> int:
    return _lib.qmv_last_cuda_error()


def qmv_set_pdl(enable: bool):
    _check("qmv_set_pdl", _lib.qmv_set_pdl(1 if enable else 0))


def qmv_device_error(clear: bool = True) -> int:
    v = _I()
    _check("qmv_device_error", _lib.qmv_device_error(ctypes.byref(v), 1 if clear else 0))
    return v.value


class Chain:
    """A chain of M = 1 matvecs run by one persistent launch (qmv_chain_*).
    The workspace is a torch uint8 device tensor; the tensors of every added
    op are kept referenced for the chain's lifetime."""

    def __init__(self, max_ops: int, device=None, no_alloc: bool = False):
        """no_alloc: use the library's own scratch array (qmv_chain_create_no_alloc)
        instead of a workspace tensor."""
        h = _P()
        if no_alloc:
            self.ws = None
            _check("qmv_chain_create_no_alloc", _lib.qmv_chain_create_no_alloc(ctypes.byref(h), max_ops))
        else:
            n = _lib.qmv_chain_workspace_bytes(max_ops)
            self.ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
            _check("qmv_chain_create", _lib.qmv_chain_create(ctypes.byref(h), max_ops, _dptr(self.ws), n))
        self.handle = h
        self._keep = []

    def add_gemv(self, p: Pack, x, y, y_dtype=QMV_F32, mode=QMV_FAST):
        _need("x", x, torch.float16, p.K)
        _need("y", y, _YDT.get(y_dtype), p.N)
        _check("qmv_chain_add_gemv", _lib.qmv_chain_add_gemv(self.handle, p.handle, _dptr(x), _dptr(y),
                                                             y_dtype, mode))
        self._keep += [p, x, y]
        return self

    def add_fused_rmsnorm_gemv(self, p: Pack, x, residual, gamma, eps, h_out, y, y_dtype=QMV_F32,
                               mode=QMV_FAST):
        _need("x", x, torch.float16, p.K)
        _need("residual", residual, torch.float16, p.K)
        _need("gamma", gamma, torch.float16, p.K)
        _need("h_out", h_out, torch.float16, p.K)
        _need("y", y, _YDT.get(y_dtype), p.N)
        _check("qmv_chain_add_fused_rmsnorm_gemv", _lib.qmv_chain_add_fused_rmsnorm_gemv(
            self.handle, p.handle, _dptr(x), _dptr(residual), _dptr(gamma), float(eps), _dptr(h_out),
            _dptr(y), y_dtype, mode))
        self._keep += [p, x, residual, gamma, h_out, y]
        return self

    def run(self, stream=None):
        _check("qmv_chain_run", _lib.qmv_chain_run(self.handle, _stream(stream)))

    def info(self):
        n, b, sm = _I(), _I(), _I()
        _check("qmv_chain_info", _lib.qmv_chain_info(self.handle, ctypes.byref(n), ctypes.byref(b),
                                                     ctypes.byref(sm)))
        return {"ops": n.value, "barriers": b.value, "smem": sm.value}

    def close(self):
        if self.handle is not None and self.handle.value:
            _lib.qmv_chain_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------- verification-step calls --
# These take row strides, so a tensor may be any 2-D view whose rows are
# contiguous; checks come first and raise ValueError before any call.

_DTYPE = {torch.float32: QMV_F32, torch.float16: QMV_F16, torch.bfloat16: QMV_BF16}
_TORCH = {v: k for k, v in _DTYPE.items()}
_16BIT = (torch.float16, torch.bfloat16)
_FLOAT = (torch.float32, torch.float16, torch.bfloat16)


class _NoHost:
    """In the place of qmv_host.so where it cannot be used: leaves every call to the Python form."""

    @staticmethod
    def leave(*args):
        return None

    w4_gemv = block_norm = softmax = verify_draft = leave


def _load_host():
    """qmv_host.so (csrc/host/qmv_host.cpp): the usual form of these calls in C++.  It holds
    to the headers of the torch and Python that it was built with; without one for those
    that are running, the Python form takes every call, with more host time."""
    path = os.path.join(_HERE, "_lib", "qmv_host.so")
    try:
        from .build import host_abi
        with open(path + ".for") as f:
            built_for = f.read()
        if built_for != host_abi():
            raise ImportError(f"it was built for {built_for}, this is {host_abi()}")
        loader = importlib.machinery.ExtensionFileLoader("qmv_host", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("qmv_host", path, loader=loader))
        loader.exec_module(mod)
    except (OSError, ImportError) as e:
        warnings.warn(f"qmv_host.so is not used ({e}): the verification-step calls take more host time; "
                      "build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        return _NoHost()
    addr = lambda f: ctypes.cast(f, _P).value
    mod.init(addr(_lib.qmv_w4_gemv), addr(_lib.qmv_block_norm), addr(_lib.qmv_softmax), addr(_lib.qmv_verify_draft))
    return mod


_host = _load_host()
# looked up once: these calls are short enough for the host's steps to count
_w4_gemv, _block_norm, _softmax, _verify_draft = (_lib.qmv_w4_gemv, _lib.qmv_block_norm, _lib.qmv_softmax,
                                                  _lib.qmv_verify_draft)
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _done(fn, r):
    """What a call of _host returned: the outputs, or a failing status to raise."""
    if type(r) is int:
        raise QmvError(fn, r)
    return r


def _rows(name, t, dtypes, rows, cols):
    """Row stride of a [rows, cols] tensor ([cols] will do for one row) of one
    of dtypes, after checking that the kernels' reads and writes stay inside it."""
    if t.dtype in dtypes and t.shape == (rows, cols) and t.is_contiguous():
        return cols                     # the usual case, in as few steps as the host can do it
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() == 2:
        r, c = t.shape
        ld, step = t.stride()
    elif t.dim() == 1:
        r, c, ld, step = 1, t.shape[0], t.shape[0], t.stride(0)
    else:
        raise ValueError(f"{name}: expected a [rows, columns] tensor, got {tuple(t.shape)}")
    if r != rows or c != cols:
        raise ValueError(f"{name}: expected [{rows}, {cols}], got {tuple(t.shape)}")
    if c > 1 and step != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows == 1:
        return cols
    if ld < cols or ld > 0x7fffffff:
        raise ValueError(f"{name}: rows overlap or their stride {ld} is too large")
    return ld


def _vec(name, t, dtype, n):
    if t.dtype == dtype and t.numel() == n and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name}: needs {n} elements, has {t.numel()}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _place(stream, first, *others):
    """The stream to launch on, after checking that all tensors lie on the
    current CUDA device."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if dev != _current_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{_current_device()}")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors are on {first.device} and {t.device}")
    if stream is not None:
        _record(stream, first, *others)
    return _raw_stream(dev) if stream is None else _stream(stream)


class W4Pack:
    """4-bit weights with a scale and (optionally) a zero point a group: the host
    descriptor plus the device buffer that holds the packed bytes."""

    def __init__(self, N: int, K: int, group: int = 128, scale_dtype=torch.float16, zeros: bool = True):
        if scale_dtype not in _16BIT:
            raise ValueError(f"scale_dtype: expected torch.float16 or torch.bfloat16, got {scale_dtype}")
        self.handle = None
        h, nb = _P(), ctypes.c_size_t()
        _check("qmv_w4_create", _lib.qmv_w4_create(ctypes.byref(h), N, K, group, _DTYPE[scale_dtype],
                                                   1 if zeros else 0, ctypes.byref(nb)))
        self.handle, self._address = h, h.value
        self.N, self.K, self.group, self.G = N, K, group, -(-K // group)
        self.scale_dtype, self.zeros = scale_dtype, bool(zeros)
        self.packed_bytes = nb.value
        self.packed, self._dev = None, -1       # the packed bytes and their device

    def pack_weights(self, codes, scales, zeros=None, stream=None):
        """codes: device uint8 [N, K], 0..15; scales: device fp16/bf16 [N, K/group];
        zeros: device uint8 [N, K/group] where the pack has zero points."""
        _vec("codes", codes, torch.uint8, self.N * self.K)
        _vec("scales", scales, self.scale_dtype, self.N * self.G)
        if self.zeros != (zeros is not None):
            raise ValueError("zeros: given exactly when the pack has zero points")
        if zeros is not None:
            _vec("zeros", zeros, torch.uint8, self.N * self.G)
        st = _place(stream, codes, scales, zeros)
        packed = _fresh((self.packed_bytes,), torch.uint8, codes.device, stream)
        _check("qmv_w4_pack", _lib.qmv_w4_pack(self.handle, codes.data_ptr(), scales.data_ptr(),
                                               None if zeros is None else zeros.data_ptr(), packed.data_ptr(), st))
        self.packed, self._dev = packed, packed.get_device()
        return self

    def bind_packed(self, packed):
        """packed: a device uint8 buffer with the packed bytes of this shape."""
        _vec("packed", packed, torch.uint8, self.packed_bytes)
        _place(None, packed)
        _check("qmv_w4_bind", _lib.qmv_w4_bind(self.handle, packed.data_ptr()))
        self.packed, self._dev = packed, packed.get_device()
        return self

    def unpack_codes(self, stream=None):
        if self.packed is None:
            raise ValueError("the pack holds no weights yet")
        st = _place(stream, self.packed)
        out = _fresh((self.N, self.K), torch.uint8, self.packed.device, stream)
        _check("qmv_w4_unpack", _lib.qmv_w4_unpack(self.handle, out.data_ptr(), st))
        return out

    def info(self):
        """(N, K, group, scale dtype, has zero points) as the library holds them."""
        v = [_I() for _ in range(5)]
        _check("qmv_w4_info", _lib.qmv_w4_info(self.handle, *map(ctypes.byref, v)))
        n, k, g, d, z = (i.value for i in v)
        return n, k, g, _TORCH[d], bool(z)

    def close(self):
        if self.handle is not None and self.handle.value:
            _lib.qmv_w4_destroy(self.handle)
        self.handle, self._dev = None, -1

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qmv_w4_gemv(p: W4Pack, x, y=None, y_dtype=QMV_F32, stream=None):
    """y [M, N] = x [M, K] . W^T for a W4Pack; x is fp16 or bf16 ([K] counts as M = 1)."""
    if y is None and stream is None:
        r = _host.w4_gemv(p._address, p._dev, p.N, p.K, x, y_dtype)
        if r is not None:
            return _done("qmv_w4_gemv", r)
    N, K = p.N, p.K
    M = x.shape[0] if x.dim() == 2 else 1
    ldx = _rows("x", x, _16BIT, M, K)
    packed = p.packed
    if packed is None:
        raise ValueError("the pack holds no weights yet")
    ydt = _TORCH.get(y_dtype)
    if ydt is None:
        raise ValueError(f"y_dtype: unknown value {y_dtype!r}")
    if y is None:
        st = _place(stream, x, packed)
        ldy, y = N, _fresh((M, N), ydt, x.device, stream)
    else:
        ldy = _rows("y", y, (ydt,), M, N)
        st = _place(stream, x, packed, y)
    rc = _w4_gemv(p.handle, M, x.data_ptr(), ldx, _DTYPE[x.dtype], y.data_ptr(), ldy, y_dtype, st)
    if rc:
        _check("qmv_w4_gemv", rc)
    return y


def qmv_block_norm(y, residual, gamma_pre, gamma_post=None, gate=None, residual_scale=1.0, branch_scale=1.0,
                   gamma_offset=0.0, eps=1e-6, h_out=None, out=None, stream=None):
    """(h, out): h = residual_scale * residual + branch_scale * gate * norm(y), out
    = norm(h); the first norm where gamma_post is given, the gate [D] or [M, D]."""
    if h_out is None and out is None and stream is None:
        r = _host.block_norm(y, residual, gamma_pre, gamma_post, gate, residual_scale, branch_scale, gamma_offset, eps)
        if r is not None:
            return _done("qmv_block_norm", r)
    shape = residual.shape
    if len(shape) == 2:
        M, D = shape
    elif len(shape) == 1:
        M, D = 1, shape[0]
    else:
        raise ValueError(f"residual: expected a [rows, columns] tensor, got {tuple(shape)}")
    dt = residual.dtype
    ldr = _rows("residual", residual, _16BIT, M, D)
    ldy = _rows("y", y, _FLOAT, M, D)
    _vec("gamma_pre", gamma_pre, dt, D)
    ldg = 0
    if gamma_post is not None:
        _vec("gamma_post", gamma_post, dt, D)
    if gate is not None:
        if gate.dim() == 1:
            _vec("gate", gate, dt, D)
        else:
            ldg = _rows("gate", gate, (dt,), M, D)
    ldh = D if h_out is None else _rows("h_out", h_out, (dt,), M, D)
    ldo = D if out is None else _rows("out", out, (dt,), M, D)
    st = _place(stream, y, residual, gamma_pre, gamma_post, gate, h_out, out)
    if h_out is None:
        h_out = _fresh((M, D), dt, y.device, stream)
    if out is None:
        out = _fresh((M, D), dt, y.device, stream)
    rc = _block_norm(M, D, y.data_ptr(), ldy, _DTYPE[y.dtype], residual.data_ptr(), ldr,
                     None if gamma_post is None else gamma_post.data_ptr(),
                     None if gate is None else gate.data_ptr(), ldg, residual_scale, branch_scale,
                     gamma_pre.data_ptr(), gamma_offset, eps, h_out.data_ptr(), ldh, out.data_ptr(), ldo,
                     _DTYPE[dt], st)
    if rc:
        _check("qmv_block_norm", rc)
    return h_out, out


def qmv_softmax(logits, temperature=1.0, out=None, stream=None):
    """fp32 probabilities [rows, V] of logits at a temperature (a number, or a
    device fp32 tensor [rows]); out may be the fp32 logits themselves."""
    if out is None and stream is None:
        r = _host.softmax(logits, temperature)
        if r is not None:
            return _done("qmv_softmax", r)
    shape = logits.shape
    if len(shape) == 2:
        rows, V = shape
    elif len(shape) == 1:
        rows, V = 1, shape[0]
    else:
        raise ValueError(f"logits: expected a [rows, columns] tensor, got {tuple(shape)}")
    ldl = _rows("logits", logits, _FLOAT, rows, V)
    t, t0 = None, 1.0
    if torch.is_tensor(temperature):
        t = temperature
        _vec("temperature", t, torch.float32, rows)
    else:
        t0 = float(temperature)
    ldo = V if out is None else _rows("out", out, (torch.float32,), rows, V)
    st = _place(stream, logits, t, out)
    if out is None:
        out = _fresh((rows, V), torch.float32, logits.device, stream)
    rc = _softmax(rows, V, logits.data_ptr(), ldl, _DTYPE[logits.dtype], None if t is None else t.data_ptr(), t0,
                  out.data_ptr(), ldo, st)
    if rc:
        _check("qmv_softmax", rc)
    return out


def qmv_verify_draft(target, draft_probs, draft, u_accept, u_sample, n_draft=None, tokens=None, n_accepted=None,
                     stream=None):
    """(tokens [B, S+1], n_accepted [B]): target fp32 [B, S+1, V], draft_probs
    fp32 [B, S, V] or None (a drafter that is sure of its tokens), draft int32
    [B, S], u_accept fp32 [B, S], u_sample fp32 [B], n_draft int32 [B] or None.
    draft and u_accept may be None where S is 0."""
    if tokens is None and n_accepted is None and stream is None:
        r = _host.verify_draft(target, draft_probs, draft, u_accept, u_sample, n_draft)
        if r is not None:
            return _done("qmv_verify_draft", r)
    if target.dim() != 3 or target.shape[1] < 1:
        raise ValueError(f"target: expected [B, S+1, V], got {tuple(target.shape)}")
    B, S1, V = target.shape
    S = S1 - 1
    _vec("target", target, torch.float32, B * S1 * V)
    if draft_probs is not None:
        _vec("draft_probs", draft_probs, torch.float32, B * S * V)
    for name, t, dtype in (("draft", draft, torch.int32), ("u_accept", u_accept, torch.float32)):
        if t is not None:
            _vec(name, t, dtype, B * S)
        elif S:
            raise ValueError(f"{name}: needed for {S} drafted tokens")
    _vec("u_sample", u_sample, torch.float32, B)
    if n_draft is not None:
        _vec("n_draft", n_draft, torch.int32, B)
    if tokens is not None:
        _vec("tokens", tokens, torch.int32, B * S1)
    if n_accepted is not None:
        _vec("n_accepted", n_accepted, torch.int32, B)
    st = _place(stream, target, draft_probs, draft, u_accept, u_sample, n_draft, tokens, n_accepted)
    if tokens is None:
        tokens = _fresh((B, S1), torch.int32, target.device, stream)
    if n_accepted is None:
        n_accepted = _fresh((B,), torch.int32, target.device, stream)
    rc = _verify_draft(B, S, V, target.data_ptr(), None if draft_probs is None else draft_probs.data_ptr(),
                       None if draft is None else draft.data_ptr(), None if n_draft is None else n_draft.data_ptr(),
                       None if u_accept is None else u_accept.data_ptr(), u_sample.data_ptr(), tokens.data_ptr(), n_accepted.data_ptr(), st)
    if rc:
        _check("qmv_verify_draft", rc)
    return tokens, n_accepted
