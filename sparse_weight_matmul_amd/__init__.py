"""Python binding of libswm.so, the MI355X sparse-weight matmul library.

Argument marshalling only: every step of the product runs in the library's HIP
kernels.  PyTorch supplies device memory and the current HIP stream; the
binding passes raw pointers, leading dimensions and the stream handle through
the C ABI declared in ``include/swm.h``.  There is no fallback: if the library
is not built or a call fails, an exception is raised.

Layout conventions (as in the C header): W is (M, K) fp16 row-major; X and Y
are token-major, X (N, K) and Y (N, M); Y = X @ (W * mask).T per token.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libswm.so")

STATUS = {
    0: "SWM_OK", 1: "SWM_ERR_INVALID_ARG", 2: "SWM_ERR_SHAPE", 3: "SWM_ERR_ALIGN", 4: "SWM_ERR_OOM",
    5: "SWM_ERR_OVERFLOW", 6: "SWM_ERR_FORMAT", 7: "SWM_ERR_HIP", 8: "SWM_ERR_UNSUPPORTED",
}

# Every symbol include/swm.h declares, with its ctypes signature.
_i64, _u64, _i32, _sz, _vp = ctypes.c_int64, ctypes.c_uint64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p


SWM_CFG_SKIPPING = 1
SWM_CFG_SMFMAC = 2


class TileCfg(ctypes.Structure):
    _fields_ = [("tm", ctypes.c_int32), ("tk", ctypes.c_int32), ("flags", ctypes.c_int32)]


class FormatInfo(ctypes.Structure):
    _fields_ = [("m", _i64), ("k", _i64), ("tm", _i32), ("tk", _i32), ("mt", _i64), ("kt", _i64),
                ("nnz", _u64), ("padded_len", _u64), ("max_tile", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("bytes_header", _u64), ("bytes_tile_ptr", _u64),
                ("bytes_bits", _u64), ("bytes_values", _u64), ("bytes_total", _u64)]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_ if f[0] != "reserved"}


class KvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("table", _vp), ("lengths", _vp),
                ("k_page", _i64), ("k_slot", _i64), ("k_head", _i64),
                ("v_page", _i64), ("v_slot", _i64), ("v_head", _i64),
                ("table_ld", _i64), ("pages", _i64), ("page_size", _i64), ("heads", _i64), ("dim", _i64),
                ("batch", _i64), ("pages_per_seq", _i64)]


_PP = ctypes.POINTER(_vp)
SIGNATURES = {
    "swm_sparse_compress": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, ctypes.POINTER(TileCfg), _vp, _PP]),
    "swm_encode_blob": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, ctypes.POINTER(TileCfg), _vp, _sz,
                               ctypes.POINTER(_sz)]),
    "swm_format_export": (_i32, [_vp, _vp, _sz, ctypes.POINTER(_sz)]),
    "swm_format_import": (_i32, [_vp, _sz, _vp, _PP]),
    "swm_format_validate_blob": (_i32, [_vp, _sz]),
    "swm_format_query": (_i32, [_vp, ctypes.POINTER(FormatInfo)]),
    "swm_size_dry_run": (_i32, [_i64, _i64, _u64, ctypes.POINTER(TileCfg), ctypes.POINTER(FormatInfo)]),
    "swm_format_destroy": (_i32, [_vp]),
    "swm_decompress": (_i32, [_vp, _vp, _i64, _vp]),
    "swm_spmm": (_i32, [_vp, _vp, _i64, _vp, _i64, _i64, _vp]),
    "swm_spmm_workspace_bytes": (_sz, [_vp, _i64]),
    "swm_spmm_ws": (_i32, [_vp, _vp, _i64, _vp, _i64, _i64, _vp, _sz, _vp]),
    "swm_spmm_epilogue_workspace_bytes": (_sz, [_vp, _i64]),
    "swm_spmm_epilogue": (_i32, [_vp, _vp, _i64, _vp, _i64, _i64, _vp, _i32, _vp, _i64, _vp, _sz, _vp]),
    "swm_spmspv": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _vp]),
    "swm_spmspv_noalloc": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, _vp]),
    "swm_spmspv_threshold": (_i32, [_vp, _vp, _i64, _vp, _i64, _i32, ctypes.c_float, _vp]),
    "swm_gate_up_silu": (_i32, [_vp, _vp, _vp, _i64, _vp, _i64, _i32, ctypes.c_float, _vp]),
    "swm_gate_up_silu_workspace_bytes": (_sz, [_vp, _vp, _i64]),
    "swm_gate_up_silu_ws": (_i32, [_vp, _vp, _vp, _i64, _vp, _i64, _i64, ctypes.c_float, _vp, _sz, _vp]),
    "swm_dense_gate_up_silu": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, ctypes.c_float, _vp]),
    "swm_format_enable_skipping": (_i32, [_vp, _vp, ctypes.POINTER(_u64)]),
    "swm_format_enable_smfmac": (_i32, [_vp, _vp, ctypes.POINTER(_u64)]),
    "swm_colruns_encode_blob": (_i32, [_vp, _sz, _vp, _sz, ctypes.POINTER(_sz)]),
    "swm_dense_gemm": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp]),
    "swm_hbm_stream": (_i32, [_vp, _sz, _i32, _i32, _vp, _vp]),
    "swm_paged_attention_workspace_bytes": (_sz, [_vp, _i64, _i32]),
    "swm_paged_attention": (_i32, [_vp, _vp, _i64, _i64, _i64, ctypes.c_float, _vp, _i64, _vp, _i64, _i64, _vp, _i64,
                                   _i64, _vp, _sz, _vp]),
    "swm_kv_evict": (_i32, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                            _vp, _vp]),
    "swm_token_logprobs": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp]),
    "swm_prompt_attention": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _i64,
                                    ctypes.c_float, _i32, _vp, _i64, _i64, _vp]),
    "swm_kv_reserve": (_i32, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "swm_kv_append": (_i32, [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp,
                             _vp]),
    "swm_tree_attention": (_i32, [_vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.c_float, _vp, _i64, _vp,
                                  _i64, _i64, _vp, _sz, _vp]),
    "swm_tree_attention_workspace_bytes": (_sz, [_vp, _i64, _i64]),
    "swm_status_str": (ctypes.c_char_p, [_i32]),
    "swm_last_hip_error": (_i32, []),
    "swm_version": (_i32, []),
}

_lib = None


class SwmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = STATUS.get(code, str(code))
        if code == 7 and _lib is not None:
            msg += f" (hipError {_lib.swm_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def load():
    """Load libswm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run python -m sparse_weight_matmul_amd.build")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(code: int, where: str):
    if code != 0:
        raise SwmError(code, where)


def _cfg(tile, flags=0):
    if tile is None and not flags:
        return None
    tm, tk = tile if tile is not None else (16, 64)
    c = TileCfg(int(tm), int(tk), int(flags))
    return ctypes.byref(c)


def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _host_u16(W):
    a = W.detach().cpu().numpy() if hasattr(W, "detach") else np.asarray(W)
    if a.dtype == np.float16:
        a = a.view(np.uint16)
    if a.dtype != np.uint16 or a.ndim != 2:
        raise TypeError("W must be a 2-D fp16 (or uint16 bit-pattern) array")
    return np.ascontiguousarray(a)


def _host_mask(mask, shape):
    if mask is None:
        return None
    m = mask.detach().cpu().numpy() if hasattr(mask, "detach") else np.asarray(mask)
    if m.shape != shape:
        raise ValueError("mask shape mismatch")
    return np.ascontiguousarray(m.astype(np.uint8))


def _dev2d(t, name, rows=None, cols=None):
    """(pointer, leading dimension) of a 2-D fp16 CUDA tensor with unit column stride."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float16 CUDA tensor")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {rows}")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} has {t.shape[1]} columns, expected {cols}")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"rows of {name} must not overlap")
    return ctypes.c_void_p(t.data_ptr()), max(int(t.stride(0)), int(t.shape[1]), 1)


class Format:
    """A compressed weight resident on the current device (owns its memory)."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        self.info = self.query()

    @property
    def M(self):
        return self.info["m"]

    @property
    def K(self):
        return self.info["k"]

    def query(self) -> dict:
        lib = load()
        inf = FormatInfo()
        _check(lib.swm_format_query(self._h, ctypes.byref(inf)), "swm_format_query")
        return inf.as_dict()

    def export(self) -> bytes:
        lib = load()
        size = ctypes.c_size_t(0)
        _check(lib.swm_format_export(self._h, None, 0, ctypes.byref(size)), "swm_format_export")
        buf = ctypes.create_string_buffer(size.value)
        _check(lib.swm_format_export(self._h, buf, size.value, ctypes.byref(size)), "swm_format_export")
        return buf.raw[:size.value]

    def enable_skipping(self, stream=None) -> int:
        """Attach the column-run encoding used by spmspv for n <= 4; returns its bytes."""
        lib = load()
        nbytes = _u64(0)
        _check(lib.swm_format_enable_skipping(self._h, _stream_ptr(stream), ctypes.byref(nbytes)),
               "swm_format_enable_skipping")
        return int(nbytes.value)

    def enable_smfmac(self, stream=None) -> int:
        """Attach the 2:4 layers of the sparse-matrix-core prefill route; returns their bytes."""
        lib = load()
        nbytes = _u64(0)
        _check(lib.swm_format_enable_smfmac(self._h, _stream_ptr(stream), ctypes.byref(nbytes)),
               "swm_format_enable_smfmac")
        return int(nbytes.value)

    def close(self):
        if self._h:
            load().swm_format_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sparse_compress(W, mask=None, tile=(16, 64), stream=None, skipping=False, smfmac=False) -> Format:
    """Compress a host fp16 W (M, K) with an optional host mask; upload to the
    current device.  skipping=True also builds the column-run encoding that
    lets spmspv skip zero activations (SWM_CFG_SKIPPING); smfmac=True also
    keeps W compacted into 2:4 layers, which spmm and spmm_ws multiply on the
    sparse matrix cores at prefill token counts (SWM_CFG_SMFMAC)."""
    lib = load()
    w = _host_u16(W)
    m = _host_mask(mask, w.shape)
    h = ctypes.c_void_p()
    code = lib.swm_sparse_compress(w.ctypes.data, w.shape[1], None if m is None else m.ctypes.data,
                                   w.shape[1], w.shape[0], w.shape[1],
                                   _cfg(tile, (SWM_CFG_SKIPPING if skipping else 0) | (SWM_CFG_SMFMAC if smfmac else 0)),
                                   _stream_ptr(stream),
                                   ctypes.byref(h))
    _check(code, "swm_sparse_compress")
    return Format(h)


def encode_blob(W, mask=None, tile=(16, 64)) -> bytes:
    """Host-only encoder: the export blob of compress(W, mask) without any GPU."""
    lib = load()
    w = _host_u16(W)
    m = _host_mask(mask, w.shape)
    mp = None if m is None else m.ctypes.data
    size = ctypes.c_size_t(0)
    _check(lib.swm_encode_blob(w.ctypes.data, w.shape[1], mp, w.shape[1], w.shape[0], w.shape[1],
                               _cfg(tile), None, 0, ctypes.byref(size)), "swm_encode_blob")
    buf = ctypes.create_string_buffer(max(size.value, 1))
    _check(lib.swm_encode_blob(w.ctypes.data, w.shape[1], mp, w.shape[1], w.shape[0], w.shape[1],
                               _cfg(tile), buf, size.value, ctypes.byref(size)), "swm_encode_blob")
    return buf.raw[:size.value]


def colruns_encode_blob(tcb_blob: bytes) -> bytes:
    """Host-only: the SWM-CR v2 column-run blob derived from a SWM-TCB v2 blob."""
    lib = load()
    b = ctypes.create_string_buffer(bytes(tcb_blob), max(len(tcb_blob), 1))
    size = ctypes.c_size_t(0)
    _check(lib.swm_colruns_encode_blob(b, len(tcb_blob), None, 0, ctypes.byref(size)), "swm_colruns_encode_blob")
    out = ctypes.create_string_buffer(max(size.value, 1))
    _check(lib.swm_colruns_encode_blob(b, len(tcb_blob), out, size.value, ctypes.byref(size)),
           "swm_colruns_encode_blob")
    return out.raw[:size.value]


def validate_blob(blob: bytes) -> int:
    """Status code of the library's blob validator (0 = valid)."""
    lib = load()
    b = ctypes.create_string_buffer(bytes(blob), max(len(blob), 1))
    return int(lib.swm_format_validate_blob(b, len(blob)))


def format_import(blob: bytes, stream=None) -> Format:
    lib = load()
    b = ctypes.create_string_buffer(bytes(blob), max(len(blob), 1))
    h = ctypes.c_void_p()
    _check(lib.swm_format_import(b, len(blob), _stream_ptr(stream), ctypes.byref(h)), "swm_format_import")
    return Format(h)


def size_dry_run(M: int, K: int, nnz: int, tile=(16, 64)) -> dict:
    lib = load()
    inf = FormatInfo()
    _check(lib.swm_size_dry_run(M, K, nnz, _cfg(tile), ctypes.byref(inf)), "swm_size_dry_run")
    return inf.as_dict()


def size_dry_run_status(M: int, K: int, nnz: int, tile=(16, 64)) -> int:
    lib = load()
    inf = FormatInfo()
    return int(lib.swm_size_dry_run(M, K, nnz, _cfg(tile), ctypes.byref(inf)))


def _out(Y, N, M, like):
    import torch
    if Y is None:
        Y = torch.empty((N, M), dtype=torch.float16, device=like.device)
    return Y


def spmm(fmt: Format, X, Y=None, stream=None):
    """Y (N, M) = X (N, K) @ (W * mask).T on the device."""
    lib = load()
    N = X.shape[0]
    xp, ldx = _dev2d(X, "X", cols=fmt.K)
    Y = _out(Y, N, fmt.M, X)
    yp, ldy = _dev2d(Y, "Y", rows=N, cols=fmt.M)
    _check(lib.swm_spmm(fmt._h, xp, ldx, yp, ldy, N, _stream_ptr(stream)), "swm_spmm")
    return Y


def spmm_workspace_bytes(fmt: Format, N: int) -> int:
    """Device workspace bytes spmm(..., workspace=) uses for N tokens (0: none)."""
    return int(load().swm_spmm_workspace_bytes(fmt._h, int(N)))


def spmm_ws(fmt: Format, X, workspace, Y=None, stream=None):
    """spmm with a caller-owned device workspace (a CUDA uint8 tensor of at
    least spmm_workspace_bytes(fmt, N) bytes, or None): for large N the library
    expands W into it once and runs its dense MFMA kernel.  Same result."""
    lib = load()
    N = X.shape[0]
    xp, ldx = _dev2d(X, "X", cols=fmt.K)
    Y = _out(Y, N, fmt.M, X)
    yp, ldy = _dev2d(Y, "Y", rows=N, cols=fmt.M)
    if workspace is None:
        wp, wb = None, 0
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        wp, wb = ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    _check(lib.swm_spmm_ws(fmt._h, xp, ldx, yp, ldy, N, wp, wb, _stream_ptr(stream)), "swm_spmm_ws")
    return Y


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


def spmm_epilogue_workspace_bytes(fmt: Format, N: int) -> int:
    """Device workspace bytes spmm_epilogue uses for N tokens (0: none)."""
    return int(load().swm_spmm_epilogue_workspace_bytes(fmt._h, int(N)))


def spmm_epilogue(fmt: Format, X, bias=None, act: str = "none", residual=None, workspace=None, Y=None, stream=None):
    """Y (N, M) = act(X @ (W * mask).T + bias) + residual, rounded once: spmm_ws
    with its epilogue in the same launches.  bias: (M,) fp16 or None; act:
    "none", "relu", "silu" or "gelu"; residual: (N, M) fp16 or None, which may
    be Y itself; workspace: a contiguous CUDA tensor of
    spmm_epilogue_workspace_bytes(fmt, N) bytes; None allocates it where the
    call uses one."""
    import torch
    lib = load()
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    N, M, K = X.shape[0], fmt.M, fmt.K
    xp, ldx = _rows(X, "X", N, K)
    device = X.get_device()
    bp = rp = None
    ldr = 0
    if bias is not None:
        if not bias.is_cuda or bias.dtype is not torch.float16 or bias.shape != (M,):
            raise TypeError(f"bias must be a float16 CUDA tensor, ({M},)")
        if bias.get_device() != device:
            raise ValueError(f"bias must be on {X.device}")
        if M > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
        bp = bias.data_ptr()
    if residual is not None:
        rp, ldr = _rows(residual, "residual", N, M)
        if residual.get_device() != device:
            raise ValueError(f"residual must be on {X.device}")
    if Y is None:
        if residual is not None and residual.is_contiguous():
            Y = _empty_like(residual, stream)
        else:
            Y = _empty((N, M), X.dtype, X.device, stream)
    yp, ldy = _rows(Y, "Y", N, M)
    if Y.get_device() != device:
        raise ValueError(f"Y must be on {X.device}")
    wp, wb = None, 0
    if N > 32:  # below, W is streamed
        need = 0 if workspace is not None else int(lib.swm_spmm_epilogue_workspace_bytes(fmt._h, N))
        workspace, wp, wb = _workspace(workspace, need, X.device, stream)
    _check(lib.swm_spmm_epilogue(fmt._h, xp, ldx, yp, ldy, N, bp, ACTIVATIONS[act], rp, ldr, wp, wb,
                                 _raw_stream(stream, device)), "swm_spmm_epilogue")
    return Y


def gate_up_silu(gate: Format, up: Format, X, tau: float = 0.0, H=None, stream=None):
    """Gated FFN hidden activation for 1..32 decode tokens: H (n, M) =
    SiLU(X @ W_g.T) * (X @ W_u.T), entries with |H| < tau stored as +0."""
    lib = load()
    n = X.shape[0]
    xp, ldx = _dev2d(X, "X", cols=gate.K)
    H = _out(H, n, gate.M, X)
    hp, ldh = _dev2d(H, "H", rows=n, cols=gate.M)
    _check(lib.swm_gate_up_silu(gate._h, up._h, xp, ldx, hp, ldh, n, float(tau), _stream_ptr(stream)),
           "swm_gate_up_silu")
    return H


def gate_up_silu_workspace_bytes(gate: Format, up: Format, n: int) -> int:
    """Device workspace bytes gate_up_silu_ws uses for n tokens (0: none)."""
    return int(load().swm_gate_up_silu_workspace_bytes(gate._h, up._h, int(n)))


def gate_up_silu_ws(gate: Format, up: Format, X, workspace, tau: float = 0.0, H=None, stream=None):
    """gate_up_silu for any token count: from 33 tokens the gate and up
    weights are expanded into `workspace` (a contiguous CUDA uint8 tensor of at
    least gate_up_silu_workspace_bytes(gate, up, n) bytes; None below 33
    tokens) and one dense MFMA product forms H with the gated epilogue."""
    lib = load()
    n = X.shape[0]
    xp, ldx = _dev2d(X, "X", cols=gate.K)
    H = _out(H, n, gate.M, X)
    hp, ldh = _dev2d(H, "H", rows=n, cols=gate.M)
    if workspace is None:
        wp, wb = None, 0
    else:
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        wp, wb = ctypes.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size()
    _check(lib.swm_gate_up_silu_ws(gate._h, up._h, xp, ldx, hp, ldh, n, float(tau), wp, wb, _stream_ptr(stream)),
           "swm_gate_up_silu_ws")
    return H


def dense_gate_up_silu(W2, X, tau: float = 0.0, H=None, stream=None):
    """Dense gated FFN step: W2 (2M, K) holds the gate and up weights
    interleaved by row (2m: gate row m, 2m+1: up row m); H (N, M) =
    SiLU(X @ Wg.T) * (X @ Wu.T), |H| < tau stored as +0."""
    lib = load()
    N = X.shape[0]
    if W2.shape[0] % 2:
        raise ValueError("W2 must hold an even number of rows (gate / up interleaved)")
    M, K = W2.shape[0] // 2, W2.shape[1]
    wp, ldw = _dev2d(W2, "W2", cols=K)
    xp, ldx = _dev2d(X, "X", cols=K)
    H = _out(H, N, M, X)
    hp, ldh = _dev2d(H, "H", rows=N, cols=M)
    _check(lib.swm_dense_gate_up_silu(wp, ldw, xp, ldx, hp, ldh, M, K, N, float(tau), _stream_ptr(stream)),
           "swm_dense_gate_up_silu")
    return H


def spmspv(fmt: Format, x, y=None, stream=None):
    """Zero-activation-skipping product for 1..16 tokens; x (n, K), y (n, M).
    Skips on the column-run encoding for n <= 2 when the handle carries it."""
    lib = load()
    n = x.shape[0]
    xp, ldx = _dev2d(x, "x", cols=fmt.K)
    y = _out(y, n, fmt.M, x)
    yp, ldy = _dev2d(y, "y", rows=n, cols=fmt.M)
    _check(lib.swm_spmspv(fmt._h, xp, ldx, yp, ldy, n, _stream_ptr(stream)), "swm_spmspv")
    return y


def spmspv_noalloc(fmt: Format, x, y=None, stream=None):
    """spmspv whose skipping path keeps its partial sums in the library's fixed
    device array (no allocation inside the call); same result, bitwise."""
    lib = load()
    n = x.shape[0]
    xp, ldx = _dev2d(x, "x", cols=fmt.K)
    y = _out(y, n, fmt.M, x)
    yp, ldy = _dev2d(y, "y", rows=n, cols=fmt.M)
    _check(lib.swm_spmspv_noalloc(fmt._h, xp, ldx, yp, ldy, n, _stream_ptr(stream)), "swm_spmspv_noalloc")
    return y


def spmspv_threshold(fmt: Format, x, tau: float, y=None, stream=None):
    """spmspv with activations |x| < tau counted as zero (skipping must be enabled, n <= 4)."""
    lib = load()
    n = x.shape[0]
    xp, ldx = _dev2d(x, "x", cols=fmt.K)
    y = _out(y, n, fmt.M, x)
    yp, ldy = _dev2d(y, "y", rows=n, cols=fmt.M)
    _check(lib.swm_spmspv_threshold(fmt._h, xp, ldx, yp, ldy, n, float(tau), _stream_ptr(stream)),
           "swm_spmspv_threshold")
    return y


def dense_gemm(W, X, Y=None, stream=None):
    """In-house dense baseline: Y (N, M) = X (N, K) @ W.T with dense fp16 W (M, K) on the device."""
    lib = load()
    M, K = W.shape
    N = X.shape[0]
    wp, ldw = _dev2d(W, "W")
    xp, ldx = _dev2d(X, "X", cols=K)
    Y = _out(Y, N, M, X)
    yp, ldy = _dev2d(Y, "Y", rows=N, cols=M)
    _check(lib.swm_dense_gemm(wp, ldw, xp, ldx, yp, ldy, M, K, N, _stream_ptr(stream)), "swm_dense_gemm")
    return Y


def decompress(fmt: Format, W=None, stream=None):
    """Dense fp16 W * mask (M, K) on the device, expanded by the library's kernel."""
    import torch
    lib = load()
    if W is None:
        W = torch.empty((fmt.M, fmt.K), dtype=torch.float16, device="cuda")
    wp, ldw = _dev2d(W, "W", rows=fmt.M, cols=fmt.K)
    _check(lib.swm_decompress(fmt._h, wp, ldw, _stream_ptr(stream)), "swm_decompress")
    return W


def hbm_stream(buf, unroll: int, blocks: int, out=None, stream=None):
    """Calibration read of a whole CUDA tensor `buf` (bytes a multiple of 16)."""
    import torch
    lib = load()
    if out is None:
        out = torch.empty(blocks * 4, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size()
    _check(lib.swm_hbm_stream(ctypes.c_void_p(buf.data_ptr()), nbytes, unroll, blocks,
                              ctypes.c_void_p(out.data_ptr()), _stream_ptr(stream)), "swm_hbm_stream")
    return out


# The serving operators are a few microseconds of work: their wrappers look at
# each tensor's properties once and allocate like a given tensor (the cheapest
# way), so that the calls of a token do not wait for Python.

def _raw_stream(stream, index: int) -> int:
    """Handle of `stream`, or of the current stream of device `index`, which must be the current device."""
    import torch
    current = torch._C._cuda_getDevice()
    if index != current:
        raise ValueError(f"tensors are on cuda:{index}, the current device is cuda:{current}")
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(index)


def _on_stream(make, stream):
    """What make() allocates, as memory of `stream`: a block that the current stream has given back may still be
    in use there, and `stream` need not wait for it.  It is not used again before the current stream, which may
    read it, is done with it either."""
    import torch
    current = torch.cuda.current_stream()
    if stream == current:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(current)
    return t


def _empty(shape, dtype, device, stream):
    """A new tensor of `stream` (None: the current one)."""
    import torch
    if stream is not None:
        return _on_stream(lambda: torch.empty(shape, dtype=dtype, device=device), stream)
    return torch.empty(*shape, dtype=dtype, device=device)  # 0.4 us less than with the tuple


def _empty_like(t, stream):
    """As _empty, with the shape and type of a contiguous tensor."""
    import torch
    if stream is not None:
        return _on_stream(lambda: torch.empty_like(t), stream)
    return torch.empty_like(t)


def _rows(t, name, rows, cols):
    """(pointer, leading dimension) of a (rows, cols) fp16 CUDA tensor with unit column stride."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.float16 or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float16 CUDA tensor")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if ld < cols and rows > 1:  # expanded ones among them: the library steps by a row at least
        raise ValueError(f"rows of {name} must not overlap")
    return t.data_ptr(), max(ld, cols, 1) if rows > 1 else max(cols, 1)


def _workspace(workspace, need, device, stream):
    """(tensor to keep alive, pointer, bytes) of a caller's workspace, or of a new one if there is none."""
    import torch
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _empty((need,), torch.uint8, device, stream)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a CUDA tensor")
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


class PagedCache:
    """A paged key-value cache: pools of key and value rows, the page table
    and the lengths of a batch of sequences.

    k, v: (pages, page_size, heads, dim) fp16 CUDA tensors with unit stride
    along dim, and any other strides that are multiples of 8 (a head-major
    pool is passed as its transpose(1, 2)); dim is a multiple of 8 up to 256.
    table: (batch, pages_per_seq) int32, the page of each run of page_size
    tokens (entries outside the pool name no page); lengths: (batch,) int32.
    The object keeps the tensors and their addresses: their contents may
    change at any time, in place."""

    def __init__(self, k, v, table, lengths):
        import torch
        for name, t in (("k", k), ("v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float16 or t.dim() != 4:
                raise TypeError(f"{name} must be a 4-D float16 CUDA tensor")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError(f"{name} must have unit stride along its last dimension")
        if k.shape != v.shape:
            raise ValueError("k and v must have the same shape")
        for name, t, dim in (("table", table, 2), ("lengths", lengths, 1)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32 or t.dim() != dim:
                raise TypeError(f"{name} must be a {dim}-D int32 CUDA tensor")
        if lengths.shape[0] != table.shape[0]:
            raise ValueError("table and lengths must have one row per sequence")
        if table.shape[1] > 1 and table.stride(1) != 1:
            raise ValueError("table must have unit stride along its last dimension")
        if lengths.shape[0] > 1 and lengths.stride(0) != 1:
            raise ValueError("lengths must be contiguous")
        if not (k.device == v.device == table.device == lengths.device):
            raise ValueError("all tensors of a cache must be on one device")
        self.k, self.v, self.table, self.lengths = k, v, table, lengths
        self.device = k.device
        self.pages, self.page_size, self.heads, self.dim = k.shape
        self.batch, self.pages_per_seq = table.shape
        self.capacity = self.pages_per_seq * self.page_size
        self._slots = torch.Size((self.pages, self.heads, self.page_size))
        # strides of dimensions of one element are arbitrary and never used
        ks = [s if n > 1 else 0 for s, n in zip(k.stride()[:3], k.shape)]
        vs = [s if n > 1 else 0 for s, n in zip(v.stride()[:3], v.shape)]
        self._c = KvCache(k.data_ptr(), v.data_ptr(), table.data_ptr(), lengths.data_ptr(), *ks, *vs,
                          table.stride(0), *k.shape, *table.shape)
        self._p = ctypes.addressof(self._c)
        self._attn_bytes, self._tree_bytes = {}, {}

    def attention_workspace_bytes(self, q_heads: int, weights: bool = False) -> int:
        """Device workspace bytes paged_attention uses (0: none)."""
        key = (int(q_heads), bool(weights))
        if key not in self._attn_bytes:
            self._attn_bytes[key] = int(load().swm_paged_attention_workspace_bytes(self._p, *key))
        return self._attn_bytes[key]

    def tree_workspace_bytes(self, q_heads: int, max_tokens: int) -> int:
        """Device workspace bytes tree_attention uses (0: none)."""
        key = (int(q_heads), int(max_tokens))
        if key not in self._tree_bytes:
            self._tree_bytes[key] = int(load().swm_tree_attention_workspace_bytes(self._p, *key))
        return self._tree_bytes[key]

    def _per_slot(self, t, name, dtype):
        """(pointer, page stride, head stride) of an array with one entry per cached row, (pages, heads, page_size)."""
        import torch
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != self.device or t.dtype is not dtype:
            raise TypeError(f"{name} must be a {dtype} tensor on {self.device}")
        if t.shape != self._slots:
            raise ValueError(f"{name} must be (pages, heads, page_size)")
        page, head, slot = t.stride()
        if self.page_size > 1 and slot != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
        return t.data_ptr(), page, head


def _mask(cache, mask):
    """(pointer, leading dimension) of a mask over the cache's tokens."""
    import torch
    if mask is None:
        return None, 0
    if (not isinstance(mask, torch.Tensor) or not mask.is_cuda or mask.dtype not in (torch.bool, torch.uint8)
            or mask.dim() != 2):
        raise TypeError("mask must be a 2-D bool or uint8 CUDA tensor")
    B = cache.batch
    if mask.shape[0] != B or mask.shape[1] < cache.capacity or mask.device != cache.device:
        raise ValueError(f"mask must be ({B}, >= {cache.capacity}) on {cache.device}")
    if mask.shape[1] > 1 and mask.stride(1) != 1:
        raise ValueError("mask must have unit stride along its last dimension")
    # of one sequence only the first row is read, whatever its stride says
    ld = mask.stride(0) if B > 1 else max(mask.shape[1], 1)
    if B > 1 and ld < cache.capacity:
        raise ValueError("mask rows must not overlap")
    return mask.data_ptr(), ld


def paged_attention(cache: PagedCache, q, scale: Optional[float] = None, mask=None, weights=None, out=None,
                    workspace=None, stream=None):
    """Attention of one new token per sequence over a paged cache: out (B, Hq,
    D) = softmax(scale * q . k) v over each sequence's live tokens (zeros where
    there are none); scale defaults to D ** -0.5.  q: (B, Hq, D) fp16, Hq a
    multiple of the cache's heads.  mask: (B, >= capacity) bool or uint8,
    false drops a token.  weights: (pages, heads, page_size) fp32, grows by
    each row's attention weight summed over the query heads that share it.
    workspace: a CUDA tensor of cache.attention_workspace_bytes(Hq, weights is
    not None) bytes; None allocates it."""
    import torch
    lib = load()
    if not q.is_cuda or q.dtype is not torch.float16 or q.dim() != 3:
        raise TypeError("q must be a 3-D float16 CUDA tensor")
    B, Hq, D = q.shape
    if B != cache.batch or D != cache.dim or q.device != cache.device:
        raise ValueError(f"q must be ({cache.batch}, heads, {cache.dim}) on {cache.device}")
    q_b, q_h, q_d = q.stride()
    if D > 1 and q_d != 1:
        raise ValueError("q must have unit stride along its last dimension")
    if out is None:
        out = _empty_like(q, stream) if q.is_contiguous() else _empty((B, Hq, D), q.dtype, cache.device, stream)
    elif not out.is_cuda or out.dtype != torch.float16 or out.shape != q.shape or out.device != q.device:
        raise TypeError("out must be a float16 CUDA tensor of q's shape")
    elif out.stride(2) != 1:
        raise ValueError("out must have unit stride along its last dimension")
    mp, mask_ld = _mask(cache, mask)
    wp, w_page, w_head = None, 0, 0
    if weights is not None:
        wp, w_page, w_head = cache._per_slot(weights, "weights", torch.float32)
    s = _raw_stream(stream, cache.device.index)
    keep, ws, ws_bytes = _workspace(workspace, cache.attention_workspace_bytes(Hq, weights is not None),
                                    cache.device, stream)
    # a stride along one sequence or one head is never used: pass 0 for it
    _check(lib.swm_paged_attention(cache._p, q.data_ptr(), q_b if B > 1 else 0, q_h if Hq > 1 else 0, Hq,
                                   D ** -0.5 if scale is None else scale, mp, mask_ld, wp, w_page, w_head,
                                   out.data_ptr(), out.stride(0), out.stride(1), ws, ws_bytes, s),
           "swm_paged_attention")
    return out


def kv_evict(cache: PagedCache, weights, positions, budget: int, recent: int = 0, weights_out=None,
             positions_out=None, lengths_out=None, kept=None, stream=None):
    """Cut every sequence of a paged cache back to `budget` tokens per head:
    those within `recent` of the newest position and those with the largest
    accumulated attention weight stay, ties going to the lower slot; the ones
    that stay above the budget move into the slots freed below it.
    weights (fp32) and positions (int32): (pages, heads, page_size), one entry
    per cached row, updated in place unless outputs are given (what is written
    must not be shared by heads or pages, as an expanded tensor is).  Returns the
    new lengths (B,) (the cache's own tensor is left alone: copy them into it)
    and kept (B, heads, budget), the slot each slot's token came from (-1
    where there is none).  No page may belong to two sequences."""
    import torch
    lib = load()
    w = cache._per_slot(weights, "weights", torch.float32)
    p = cache._per_slot(positions, "positions", torch.int32)
    wo = w if weights_out is None else cache._per_slot(weights_out, "weights_out", torch.float32)
    po = p if positions_out is None else cache._per_slot(positions_out, "positions_out", torch.int32)
    budget = int(budget)
    if budget < 0:
        raise ValueError("budget must not be negative")
    if lengths_out is None:
        lengths_out = _empty_like(cache.lengths, stream)
    elif (lengths_out.device != cache.device or lengths_out.dtype != torch.int32
          or lengths_out.shape != (cache.batch,) or not lengths_out.is_contiguous()):
        raise TypeError("lengths_out must be a contiguous int32 CUDA tensor, one entry per sequence")
    shape = (cache.batch, cache.heads, budget)
    if kept is None:
        kept = _empty(shape, torch.int32, cache.device, stream)
    elif (kept.device != cache.device or kept.dtype != torch.int32 or kept.shape != shape
          or not kept.is_contiguous()):
        raise TypeError(f"kept must be a contiguous {shape} int32 CUDA tensor")
    s = _raw_stream(stream, cache.device.index)
    _check(lib.swm_kv_evict(cache._p, *w, *p, budget, int(recent), *wo, *po, lengths_out.data_ptr(),
                            kept.data_ptr(), s), "swm_kv_evict")
    return lengths_out, kept


def token_logprobs(logits, targets=None, top: int = 0, stream=None):
    """(logprobs, entropy, top_ids, top_logprobs) of rows of logits (N, V),
    fp16 or fp32: log p of each row's target token ((N,) int32 or int64; a
    negative one means none and gives 0), the entropy of each row, and its
    `top` <= 64 most likely tokens, equal logits by the lower index.  fp32 and
    int64; logprobs is None without targets, top_ids and top_logprobs are None
    for top = 0."""
    import torch
    lib = load()
    if not logits.is_cuda or logits.dtype not in (torch.float16, torch.float32) or logits.dim() != 2:
        raise TypeError("logits must be a 2-D float16 or float32 CUDA tensor")
    N, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have unit stride along the last dimension")
    device = logits.device
    ld = logits.stride(0) if N > 1 else V
    if ld < V:
        raise ValueError("rows of logits must not overlap")
    s = _raw_stream(stream, device.index)
    tp, wide, logp = None, 0, None
    if targets is not None:
        if targets.dtype not in (torch.int32, torch.int64) or targets.device != device:
            raise TypeError(f"targets must be an int32 or int64 tensor on {device}")
        if targets.shape != (N,) or (N > 1 and targets.stride(0) != 1):
            raise ValueError(f"targets must be contiguous, ({N},)")
        tp, wide = targets.data_ptr(), int(targets.dtype == torch.int64)
        logp = _empty((N,), torch.float32, device, stream)
    entropy = _empty((N,), torch.float32, device, stream) if logp is None else _empty_like(logp, stream)
    top = int(top)
    ids = lps = None
    if top > 0:
        ids = _empty((N, top), torch.int64, device, stream)
        lps = _empty((N, top), torch.float32, device, stream)
    _check(lib.swm_token_logprobs(logits.data_ptr(), int(logits.dtype == torch.float32), N, V, ld, tp, wide,
                                  None if logp is None else logp.data_ptr(), entropy.data_ptr(), top,
                                  None if ids is None else ids.data_ptr(), None if lps is None else lps.data_ptr(),
                                  s), "swm_token_logprobs")
    return logp, entropy, ids, lps


def _heads(t, name, device=None):
    """(pointer, token stride, head stride) of a (tokens, heads, dim) fp16 CUDA tensor with unit stride along dim."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.float16 or t.dim() != 3:
        raise TypeError(f"{name} must be a 3-D float16 CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    T, H, D = t.shape
    token, head, unit = t.stride()
    if unit != 1 and D > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    # a stride along one token or one head is never used
    return t.data_ptr(), token if T > 1 else D, head if H > 1 else 0


def _out_like(q, out, stream):
    """(out, its (pointer, token stride, head stride)) for rows like those of q; a new tensor if there is none."""
    T, Hq, D = q.shape
    if out is None:
        out = _empty((T, Hq, D), q.dtype, q.device, stream)
        return out, (out.data_ptr(), Hq * D, D)
    p = _heads(out, "out", q.device)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    return out, p


def prompt_attention(q, k, v, starts, scale: Optional[float] = None, causal: bool = True, out=None, stream=None):
    """Attention over whole prompts, packed one behind the other: rows
    starts[b] .. starts[b + 1] - 1 of q (T, Hq, D) and of k and v (T, H, D),
    fp16, are sequence b; out (T, Hq, D) = softmax(scale * q . k) v over each
    row's own sequence, up to the row itself if causal.  Hq is a multiple of H,
    D of 8 up to 256; scale defaults to D ** -0.5; any strides that are
    multiples of 8 (views of a stacked product's rows, head-major tensors).
    starts: (B + 1,) int32 on the device.  Rows that belong to no sequence are
    not written.  Unlike paged_attention it adds up no weights: a prompt's rows
    in a cache are ranked by what later tokens give them."""
    import torch
    lib = load()
    qp, device = _heads(q, "q"), q.device
    T, Hq, D = q.shape
    kp, vp = _heads(k, "k", device), _heads(v, "v", device)
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k and v must be ({T}, heads, {D})")
    B = _starts(starts, device)
    out, op = _out_like(q, out, stream)
    s = _raw_stream(stream, device.index)
    _check(lib.swm_prompt_attention(*qp, *kp, *vp, T, Hq, k.shape[1], D, starts.data_ptr(), B,
                                    D ** -0.5 if scale is None else scale, int(bool(causal)), *op, s),
           "swm_prompt_attention")
    return out


def _starts(starts, device) -> int:
    """Sequences that a (B + 1,) int32 tensor of row bounds describes."""
    import torch
    if not isinstance(starts, torch.Tensor) or starts.dtype is not torch.int32 or starts.device != device:
        raise TypeError(f"starts must be an int32 tensor on {device}")
    if starts.dim() != 1 or starts.shape[0] < 1 or not starts.is_contiguous():
        raise ValueError("starts must be contiguous, one entry more than sequences")
    return starts.shape[0] - 1


def tree_attention(cache: PagedCache, q, starts, parents=None, max_tokens: Optional[int] = None,
                   scale: Optional[float] = None, mask=None, out=None, workspace=None, stream=None):
    """Attention of drafted tokens over a paged cache that holds their keys and
    values: rows starts[b] .. starts[b + 1] - 1 of q (T, Hq, D) fp16 are the last
    tokens of sequence b (the cache's lengths count them).  Each sees the tokens
    before the drafted ones, itself, its parent, the parent's parent and so on.
    starts: (B + 1,) int32 on the device.  parents: (T,) int32, a lower index
    among the sequence's drafted tokens, -1 for the sequence itself; None: the
    tokens follow each other.  max_tokens: at least the drafted tokens of any
    sequence, at most 64 (None: the lesser of 64 and T).  mask: (B, >= capacity)
    bool or uint8, false drops a token.  workspace: a CUDA tensor of
    cache.tree_workspace_bytes(Hq, max_tokens) bytes; None allocates it.  Rows
    that belong to no sequence are not written."""
    import torch
    lib = load()
    device = cache.device
    qp = _heads(q, "q", device)
    T, Hq, D = q.shape
    if D != cache.dim:
        raise ValueError(f"q must be (tokens, heads, {cache.dim})")
    if _starts(starts, device) != cache.batch:
        raise ValueError(f"starts must have {cache.batch + 1} entries")
    pp = None
    if parents is not None:
        if not isinstance(parents, torch.Tensor) or parents.dtype is not torch.int32 or parents.device != device:
            raise TypeError(f"parents must be an int32 tensor on {device}")
        if parents.shape != (T,) or not parents.is_contiguous():
            raise ValueError(f"parents must be contiguous, ({T},)")
        pp = parents.data_ptr()
    most = min(64, T) if max_tokens is None else int(max_tokens)
    out, op = _out_like(q, out, stream)
    mp, mask_ld = _mask(cache, mask)
    s = _raw_stream(stream, device.index)
    keep, ws, ws_bytes = _workspace(workspace, cache.tree_workspace_bytes(Hq, most), device, stream)
    _check(lib.swm_tree_attention(cache._p, *qp, Hq, T, starts.data_ptr(), pp, most,
                                  D ** -0.5 if scale is None else scale, mp, mask_ld, *op, ws, ws_bytes, s),
           "swm_tree_attention")
    return out


def _ints(t, name, shape, dtype, device):
    """Address of a contiguous tensor of whole numbers."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {tuple(shape)}")
    return t.data_ptr()


def kv_reserve(cache: PagedCache, counts, free, free_count, tokens: int, starts=None, slots=None, granted=None,
               stream=None):
    """Pages for the tokens that a step adds to each sequence of a paged cache,
    pages back from those that it drops.  Sequence b goes from lengths[b] to
    lengths[b] + counts[b] tokens (negative: dropped from its end); the cache's
    table and lengths change in place, and so do free (int32, one entry per page
    of the pool at least: the free pages) and free_count ((1,) int32, how many).
    Pages come back before any are given out, in order of the sequences; one
    that needs more than are left gets none, and after it only those that need
    none; one that would outgrow the table is left as it is.
    tokens: the sum of the positive counts.  Returns starts (B + 1,) int32, where
    each sequence's added tokens begin among all, slots (tokens,) int64, the
    slot of each of them in the pool (-1: not granted) and granted (B,) int32, by
    how much each length changed.  No two of the tensors may share memory."""
    import torch
    lib = load()
    device, B, tokens = cache.device, cache.batch, int(tokens)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    cp = _ints(counts, "counts", (B,), torch.int32, device)
    if not isinstance(free, torch.Tensor) or free.dim() != 1:
        raise TypeError("free must be a 1-D int32 CUDA tensor")
    fp = _ints(free, "free", free.shape, torch.int32, device)
    np_ = _ints(free_count, "free_count", (1,), torch.int32, device)
    if starts is None:
        starts = _empty((B + 1,), torch.int32, device, stream)
    else:
        _ints(starts, "starts", (B + 1,), torch.int32, device)
    if slots is None:
        slots = _empty((tokens,), torch.int64, device, stream)
    else:
        _ints(slots, "slots", (tokens,), torch.int64, device)
    if granted is None:
        granted = _empty_like(counts, stream)
    else:
        _ints(granted, "granted", (B,), torch.int32, device)
    s = _raw_stream(stream, device.index)
    _check(lib.swm_kv_reserve(cache._p, cp, fp, free.shape[0], np_, tokens, starts.data_ptr(), slots.data_ptr(),
                              granted.data_ptr(), s), "swm_kv_reserve")
    return starts, slots, granted


def kv_append(cache: PagedCache, k, v, slots, weights=None, positions=None, at=None, stream=None):
    """Write key and value rows of new tokens, k and v (T, heads, dim) fp16, into
    their slots of a paged cache: slots (T,) int64 as kv_reserve gives them,
    page * page_size + slot in the page (a slot outside the pool is not
    written; none may appear twice).  weights (fp32) and positions (int32):
    (pages, heads, page_size), as paged_attention and kv_evict use them; the new
    rows' weights become 0 and their positions at[t], at (T,) int32."""
    import torch
    lib = load()
    device = cache.device
    kp, vp = _heads(k, "k", device), _heads(v, "v", device)
    T = k.shape[0]
    if k.shape != (T, cache.heads, cache.dim) or v.shape != k.shape:
        raise ValueError(f"k and v must be (tokens, {cache.heads}, {cache.dim})")
    sp = _ints(slots, "slots", (T,), torch.int64, device)
    w = (None, 0, 0) if weights is None else cache._per_slot(weights, "weights", torch.float32)
    p, ap = (None, 0, 0), None
    if (positions is None) != (at is None):
        raise ValueError("positions and at go together")
    if positions is not None:
        p = cache._per_slot(positions, "positions", torch.int32)
        ap = _ints(at, "at", (T,), torch.int32, device)
    s = _raw_stream(stream, device.index)
    _check(lib.swm_kv_append(cache._p, *kp, *vp, T, sp, *w, *p, ap, s), "swm_kv_append")


def status_str(code: int) -> str:
    return load().swm_status_str(code).decode()


def version() -> int:
    return int(load().swm_version())
