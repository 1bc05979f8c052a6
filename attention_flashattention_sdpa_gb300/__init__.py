"""Python binding of the GB300 fused SDPA library (``include/sdpa.h``).

Argument marshalling only: every step of the attention computation runs in the CUDA
kernels of ``libsdpa_gb300.so``.  PyTorch supplies device memory and the current stream.
The binding keeps the C names: :func:`sdpa_fwd`, :func:`sdpa_bwd`,
:func:`sdpa_workspace_size`, :func:`sdpa_last_error_string`, :func:`sdpa_device_error`; for serving
:func:`sdpa_rope_fwd`, :func:`sdpa_rope_bwd`, :func:`sdpa_cache_write`, :func:`sdpa_cache_read` and
:func:`sdpa_decode`.

Importing this package loads the library and raises ``ImportError`` if it has not been
built (``python -m attention_flashattention_sdpa_gb300._build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional

__all__ = [
    "SdpaError", "Strides", "Problem", "lib", "LIB_PATH", "dtype_code", "make_problem",
    "sdpa_workspace_size", "sdpa_fwd", "sdpa_bwd", "sdpa_last_error_string", "causal_code",
    "sdpa_device_error", "sdpa_version", "sdpa_bwd_noalloc", "NOALLOC_SCRATCH_BYTES", "STATUS",
    "sdpa_dropout_mask_size", "sdpa_dropout_mask",
    "RopeTable", "Rope", "Cache", "CacheRows", "Decode", "sdpa_rope_table", "sdpa_rope_fwd",
    "sdpa_rope_bwd", "sdpa_cache_write", "sdpa_cache_read", "sdpa_decode",
    "sdpa_decode_workspace_size",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsdpa_gb300.so")

STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARG", 2: "SDPA_ERR_UNSUPPORTED",
          3: "SDPA_ERR_LAYOUT", 4: "SDPA_ERR_WORKSPACE", 5: "SDPA_ERR_CUDA",
          6: "SDPA_ERR_TIMEOUT"}

DTYPE_F16, DTYPE_BF16, DTYPE_E4M3, DTYPE_E5M2 = 0, 1, 2, 3


class SdpaError(RuntimeError):
    """A non-OK status from the library; ``status`` holds the code."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("s", ctypes.c_int64),
                ("d", ctypes.c_int64)]


class Problem(ctypes.Structure):
    _fields_ = [
        ("b", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
        ("s_q", ctypes.c_int32), ("s_kv", ctypes.c_int32), ("d", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("attn_scale", ctypes.c_float), ("causal", ctypes.c_int32),
        ("q", Strides), ("k", Strides), ("v", Strides), ("o", Strides),
        ("dout", Strides), ("dq", Strides), ("dk", Strides), ("dv", Strides),
        ("descale_q", ctypes.c_void_p), ("descale_k", ctypes.c_void_p),
        ("descale_v", ctypes.c_void_p),
        ("seq_lens_q", ctypes.c_void_p), ("seq_lens_kv", ctypes.c_void_p),
        ("alibi", ctypes.c_int32), ("alibi_slopes", ctypes.c_void_p),
        ("dropout_p", ctypes.c_float), ("dropout_mask", ctypes.c_void_p),
        ("dropout_mask_t", ctypes.c_void_p),
        ("dout_dtype", ctypes.c_int32), ("descale_do", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("bias_strides", Strides),
        ("dbias", ctypes.c_void_p), ("dbias_strides", Strides),
    ]


class RopeTable(ctypes.Structure):
    _fields_ = [
        ("rot", ctypes.c_int32), ("scaling", ctypes.c_int32), ("base", ctypes.c_double),
        ("factor", ctypes.c_double), ("original_context", ctypes.c_double),
        ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("inv_freq", ctypes.c_void_p),
    ]


class Rope(ctypes.Structure):
    _fields_ = [
        ("b", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_k", ctypes.c_int32), ("s", ctypes.c_int32),
        ("d", ctypes.c_int32), ("rot", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("attn_factor", ctypes.c_float), ("table", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_int64),
        ("q", Strides), ("k", Strides), ("q_out", Strides), ("k_out", Strides),
    ]


class Cache(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("b", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("k_strides", Strides), ("v_strides", Strides), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("page_table_stride", ctypes.c_int64), ("seq_lens_kv", ctypes.c_void_p),
    ]


class CacheRows(ctypes.Structure):
    _fields_ = [
        ("s", ctypes.c_int32), ("dtype", ctypes.c_int32), ("k", Strides), ("v", Strides),
        ("seq_lens_q", ctypes.c_void_p), ("rope", ctypes.c_void_p),
    ]


class Decode(ctypes.Structure):
    _fields_ = [
        ("h_q", ctypes.c_int32), ("s_q", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("attn_scale", ctypes.c_float), ("q", Strides), ("o", Strides),
        ("seq_lens_q", ctypes.c_void_p), ("tree_mask", ctypes.c_void_p),
        ("tree_mask_stride", ctypes.c_int64),
    ]


def _packer(cls=Problem):
    """One struct.Struct that lays out a whole ctypes structure at the offsets ctypes gives it, so
    that it is marshalled by a single pack instead of one ctypes assignment per field."""
    fmt, pos = ["="], 0
    codes = {ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "Q", ctypes.c_int64: "q"}
    for name, typ in cls._fields_:
        off = getattr(cls, name).offset
        fmt.append("x" * (off - pos))
        if typ is Strides:
            fmt.append("qqqq")
        else:
            fmt.append(codes[typ])
        pos = off + ctypes.sizeof(typ)
    fmt.append("x" * (ctypes.sizeof(cls) - pos))
    st = struct.Struct("".join(fmt))
    assert st.size == ctypes.sizeof(cls)
    return st


_PACK = _packer()
_PACK_ROPE, _PACK_CACHE, _PACK_ROWS, _PACK_DECODE = (_packer(c).pack for c in (Rope, Cache, CacheRows, Decode))
_NO_STRIDES = (0, 0, 0, 1)


def causal_code(causal) -> int:
    """False/0: no mask; True/1/"top_left": top-left causal; 2/"bottom_right": bottom-right."""
    if causal in (False, None, 0):
        return 0
    if causal in (True, 1, "top_left"):
        return 1
    if causal in (2, "bottom_right"):
        return 2
    raise ValueError(f"unknown causal mode {causal!r}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m attention_flashattention_sdpa_gb300._build` (nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    P, VP, SZ = ctypes.POINTER(Problem), ctypes.c_void_p, ctypes.c_size_t
    L.sdpa_workspace_size.argtypes = [P, ctypes.c_int, ctypes.POINTER(SZ)]
    L.sdpa_workspace_size.restype = ctypes.c_int
    L.sdpa_fwd.argtypes = [P, VP, VP, VP, VP, VP, VP, SZ, VP]
    L.sdpa_fwd.restype = ctypes.c_int
    L.sdpa_bwd.argtypes = [P, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP, SZ, VP]
    L.sdpa_bwd.restype = ctypes.c_int
    L.sdpa_bwd_noalloc.argtypes = [P, VP, VP, VP, VP, VP, VP, VP, VP, VP, VP]
    L.sdpa_bwd_noalloc.restype = ctypes.c_int
    L.sdpa_dropout_mask_size.argtypes = [P, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
    L.sdpa_dropout_mask_size.restype = ctypes.c_int
    L.sdpa_dropout_mask.argtypes = [P, ctypes.c_uint64, ctypes.c_uint64, VP, VP, VP]
    L.sdpa_dropout_mask.restype = ctypes.c_int
    L.sdpa_last_error_string.argtypes = []
    L.sdpa_last_error_string.restype = ctypes.c_char_p
    L.sdpa_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    L.sdpa_device_error.restype = ctypes.c_int
    L.sdpa_version.argtypes = []
    L.sdpa_version.restype = ctypes.c_int
    L.sdpa_problem_struct_size.argtypes = []
    L.sdpa_problem_struct_size.restype = SZ
    # The serving structs are handed over as packed bytes.
    L.sdpa_rope_table.argtypes = [VP, VP, ctypes.POINTER(ctypes.c_float)]
    L.sdpa_rope_fwd.argtypes = L.sdpa_rope_bwd.argtypes = [VP, VP, VP, VP, VP, VP]
    L.sdpa_cache_write.argtypes = L.sdpa_cache_read.argtypes = [VP, VP, VP, VP, VP]
    L.sdpa_decode_workspace_size.argtypes = [VP, VP, ctypes.POINTER(SZ)]
    L.sdpa_decode.argtypes = [VP, VP, VP, VP, VP, VP, SZ, VP]
    for f in (L.sdpa_rope_table, L.sdpa_rope_fwd, L.sdpa_rope_bwd, L.sdpa_cache_write, L.sdpa_cache_read,
              L.sdpa_decode_workspace_size, L.sdpa_decode):
        f.restype = ctypes.c_int
    L.sdpa_serving_struct_size.argtypes = [ctypes.c_int]
    L.sdpa_serving_struct_size.restype = SZ
    for i, cls in enumerate((RopeTable, Rope, Cache, CacheRows, Decode)):
        if L.sdpa_serving_struct_size(i) != ctypes.sizeof(cls):
            raise ImportError(f"{cls.__name__}: layout mismatch between the library and the binding")
    if L.sdpa_problem_struct_size() != ctypes.sizeof(Problem):
        raise ImportError("sdpa_problem_t layout mismatch between the library and the binding")
    return L


lib = _load()


def sdpa_last_error_string() -> str:
    return lib.sdpa_last_error_string().decode()


def sdpa_version() -> int:
    return lib.sdpa_version()


def _check(status: int):
    if status != 0:
        raise SdpaError(status, sdpa_last_error_string())


_DTYPES = {}


def dtype_code(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16,
                        torch.float8_e4m3fn: DTYPE_E4M3, torch.float8_e5m2: DTYPE_E5M2})
    return _DTYPES[t.dtype]


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _st4(t):
    if t is None:
        return _NO_STRIDES
    if t.dim() != 4:
        raise ValueError("tensors are logical [b, h, s, d] views")
    return t.stride()


def _bst(t):
    """Strides of a [b|1, h|1, s_q, s_kv] bias view; size-1 batch/head dims broadcast."""
    if t is None:
        return (0, 0, 0, 0)
    st = list(t.stride())
    if t.shape[0] == 1:
        st[0] = 0
    if t.shape[1] == 1:
        st[1] = 0
    return st


def _p0(t) -> int:
    return 0 if t is None else t.data_ptr()


def make_problem(q, k, v, o=None, *, attn_scale: Optional[float] = None, causal=False,
                 dout=None, dq=None, dk=None, dv=None, descale_q=None, descale_k=None,
                 descale_v=None, seq_lens_q=None, seq_lens_kv=None, alibi=False,
                 alibi_slopes=None, dropout_p: float = 0.0, dropout_mask=None,
                 dropout_mask_t=None, descale_do=None, bias=None, dbias=None) -> Problem:
    """Fills an sdpa_problem_t from logical [b, h, s, d] torch tensors (no copies).

    ALiBi is on when ``alibi`` is true or ``alibi_slopes`` (fp32 CUDA tensor of h_q slopes)
    is given; without slopes the library uses 2^(-8 (h + 1) / h_q)."""
    b, h_q, s_q, d = q.shape
    h_kv, s_kv = k.shape[1], k.shape[2]
    in_dt = dtype_code(q)
    if o is not None:
        out_dt = dtype_code(o)
    else:
        out_dt = DTYPE_BF16 if in_dt == DTYPE_E4M3 else in_dt
    scale = (1.0 / math.sqrt(d)) if attn_scale is None else float(attn_scale)
    return Problem.from_buffer_copy(_PACK.pack(
        b, h_q, h_kv, s_q, s_kv, d, in_dt, out_dt, scale, causal_code(causal),
        *_st4(q), *_st4(k), *_st4(v), *_st4(o), *_st4(dout), *_st4(dq), *_st4(dk), *_st4(dv),
        _p0(descale_q), _p0(descale_k), _p0(descale_v), _p0(seq_lens_q), _p0(seq_lens_kv),
        1 if (alibi or alibi_slopes is not None) else 0, _p0(alibi_slopes),
        float(dropout_p), _p0(dropout_mask), _p0(dropout_mask_t),
        dtype_code(dout) if dout is not None else in_dt, _p0(descale_do),
        _p0(bias), *_bst(bias), _p0(dbias), *_bst(dbias)))


_RAW_STREAM = None


def _stream(stream, like=None) -> int:
    """The cudaStream_t to launch on: ``stream`` if given, else PyTorch's current stream on the
    device of tensor ``like`` (read through torch's raw accessor when it has one: a few µs
    cheaper per call than building a Stream object)."""
    global _RAW_STREAM
    if stream is not None:
        return int(stream)
    import torch
    if _RAW_STREAM is None:
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", False)
    if _RAW_STREAM and like is not None and like.device.index is not None:
        return _RAW_STREAM(like.device.index)
    return torch.cuda.current_stream().cuda_stream


def sdpa_workspace_size(problem: Problem, is_backward: bool) -> int:
    n = ctypes.c_size_t(0)
    _check(lib.sdpa_workspace_size(ctypes.byref(problem), 1 if is_backward else 0, ctypes.byref(n)))
    return n.value


def sdpa_fwd(q, k, v, o, lse=None, *, attn_scale: Optional[float] = None, causal=False,
             descale_q=None, descale_k=None, descale_v=None, workspace=None, stream=None,
             seq_lens_q=None, seq_lens_kv=None, alibi=False, alibi_slopes=None,
             dropout_p: float = 0.0, dropout_mask=None, bias=None) -> None:
    """O (and LSE when ``lse`` is given: fp32 [b, h_q, s_q] contiguous) from Q, K, V.

    seq_lens_q / seq_lens_kv: optional int32 CUDA tensors of b valid lengths.
    alibi / alibi_slopes: the linear position bias (see :func:`make_problem`).
    dropout_p / dropout_mask: dropout with the row-major keep bits of :func:`sdpa_dropout_mask`."""
    p = make_problem(q, k, v, o, attn_scale=attn_scale, causal=causal, descale_q=descale_q,
                     descale_k=descale_k, descale_v=descale_v, seq_lens_q=seq_lens_q,
                     seq_lens_kv=seq_lens_kv, alibi=alibi, alibi_slopes=alibi_slopes,
                     dropout_p=dropout_p, dropout_mask=dropout_mask, bias=bias)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.sdpa_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                        _ptr(workspace), ws_bytes, _stream(stream, q)))


def sdpa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, *, attn_scale: Optional[float] = None,
             causal=False, stream=None, seq_lens_q=None, seq_lens_kv=None, alibi=False,
             alibi_slopes=None, dropout_p: float = 0.0, dropout_mask_t=None, descale_q=None,
             descale_k=None, descale_v=None, descale_do=None, bias=None, dbias=None) -> None:
    """dQ, dK, dV (overwritten) for the incoming gradient ``dout``; the masking, lengths,
    ALiBi and dropout options must be those of the forward call that produced ``o`` and
    ``lse`` (dropout_mask_t: the transposed keep bits of the same draw).  FP8: E4M3 q, k, v
    and an E5M2 (or E4M3) dout with their fp32 CUDA descales; o, dq, dk, dv in BF16/F16."""
    p = make_problem(q, k, v, o, attn_scale=attn_scale, causal=causal, dout=dout, dq=dq, dk=dk,
                     dv=dv, seq_lens_q=seq_lens_q, seq_lens_kv=seq_lens_kv, alibi=alibi,
                     alibi_slopes=alibi_slopes, dropout_p=dropout_p, dropout_mask_t=dropout_mask_t,
                     descale_q=descale_q, descale_k=descale_k, descale_v=descale_v,
                     descale_do=descale_do, bias=bias, dbias=dbias)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.sdpa_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), ws_bytes, _stream(stream, q)))


def _mask_problem(b: int, h_q: int, s_q: int, s_kv: int, dropout_p: float, causal=False) -> Problem:
    p = Problem()
    p.b, p.h_q, p.s_q, p.s_kv = b, h_q, s_q, s_kv
    p.dropout_p = float(dropout_p)
    p.causal = causal_code(causal)
    return p


def sdpa_dropout_mask_size(b: int, h_q: int, s_q: int, s_kv: int):
    """(bytes of the row-major keep bits, bytes of the transposed ones)."""
    n, n_t = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib.sdpa_dropout_mask_size(ctypes.byref(_mask_problem(b, h_q, s_q, s_kv, 0.0)),
                                      ctypes.byref(n), ctypes.byref(n_t)))
    return n.value, n_t.value


def sdpa_dropout_mask(b: int, h_q: int, s_q: int, s_kv: int, dropout_p: float, seed: int,
                      offset: int, mask=None, mask_t=None, stream=None, causal=False) -> None:
    """Draws the Philox4x32-10 keep bits into ``mask`` (row-major, for sdpa_fwd) and/or
    ``mask_t`` (transposed, for sdpa_bwd): CUDA tensors of sdpa_dropout_mask_size bytes.
    With ``causal`` (no per-batch lengths) tiles above the diagonal are left unwritten."""
    p = _mask_problem(b, h_q, s_q, s_kv, dropout_p, causal)
    _check(lib.sdpa_dropout_mask(ctypes.byref(p), int(seed), int(offset), _ptr(mask), _ptr(mask_t),
                                 _stream(stream, mask if mask is not None else mask_t)))


NOALLOC_SCRATCH_BYTES = 32 << 20  # SDPA_NOALLOC_SCRATCH_BYTES in include/sdpa.h


def sdpa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, *, attn_scale: Optional[float] = None,
                     causal=False, stream=None) -> None:
    """sdpa_bwd without a workspace, for callers that cannot allocate device memory: the
    scratch is a fixed 32 MiB array inside the library, shared by every call (calls must not
    overlap on the GPU; larger problems raise SdpaError with SDPA_ERR_UNSUPPORTED)."""
    p = make_problem(q, k, v, o, attn_scale=attn_scale, causal=causal, dout=dout, dq=dq, dk=dk,
                     dv=dv)
    _check(lib.sdpa_bwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout),
                                _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream, q)))


def sdpa_device_error() -> int:
    """Synchronises the device and returns (and clears) the kernels' error word."""
    f = ctypes.c_uint32(0)
    _check(lib.sdpa_device_error(ctypes.byref(f)))
    return f.value


# ---- serving: rotary positions, a paged cache, attention over it ------------------------------

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def sdpa_rope_table(rot: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                    original_context: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                    inv_freq=None, device="cuda"):
    """(table, attn_factor) for the rotary calls: the turns per position of each of rot/2 pairs as an
    int64 tensor of 64-bit binary fractions on ``device``, and the factor on the rotated values.

    ``scaling``: "none", "linear", "ntk" or "yarn" (by parts), stretching by ``factor`` the
    ``original_context``; or ``inv_freq``: rot/2 frequencies of the caller's own."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}")
    n = max(0, int(rot)) // 2
    freqs = None
    if inv_freq is not None:
        vals = [float(f) for f in inv_freq]
        if len(vals) != n:
            raise ValueError(f"inv_freq needs rot/2 = {n} frequencies, got {len(vals)}")
        freqs = (ctypes.c_double * max(1, n))(*vals)
    cfg = RopeTable(int(rot), ROPE_SCALINGS[scaling], float(base), float(factor), float(original_context),
                    float(beta_fast), float(beta_slow), ctypes.addressof(freqs) if freqs is not None else None)
    out, att = torch.empty(n, dtype=torch.int64), ctypes.c_float(1.0)
    _check(lib.sdpa_rope_table(ctypes.addressof(cfg), out.data_ptr() if n else ctypes.addressof(att), ctypes.byref(att)))
    return out.to(device), att.value


def _code(t, name: str) -> int:
    try:
        return dtype_code(t)
    except KeyError:
        raise ValueError(f"{name}: dtype {t.dtype} is not one the library takes") from None


def _need(ok: bool, message: str):
    if not ok:
        raise ValueError(message)


def _launch(fn, stream, like, *args):
    """Calls ``fn(*args, stream)`` with the device of ``like`` current."""
    import torch
    dev = like.device.index
    if dev == torch.cuda.current_device():
        _check(fn(*args, _stream(stream, like)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream(stream, like)))


def _same_device(like, *tensors):
    dev = like.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors must be on one device ({dev} and {t.device} given)")


def _ints(t, name: str, shape, dtype: str = "torch.int32"):
    """A dense integer tensor of this shape (and nothing where it is None)."""
    if t is not None:
        _need(str(t.dtype) == dtype and tuple(t.shape) == shape and t.is_contiguous(),
              f"{name} must be a contiguous {dtype} tensor of shape {shape}, got {t.dtype} {tuple(t.shape)}")


def _positions(positions, b: int, s: int):
    """(pointer, elements between batches) of positions [b, s], or [s] or [1, s] for every batch."""
    if positions is None:
        return 0, 0
    _need(str(positions.dtype) == "torch.int32" and tuple(positions.shape) in ((b, s), (1, s), (s,))
          and (s == 1 or positions.stride(-1) == 1) and (positions.dim() == 1 or positions.stride(0) >= 0),
          f"positions must be int32 of shape ({b}, {s}), (1, {s}) or ({s},) with a unit last stride")
    shared = positions.dim() == 1 or (positions.shape[0] == 1 and b > 1)
    return positions.data_ptr(), 0 if shared else positions.stride(0)


def _rope(fn, q, k, q_out, k_out, table, positions, interleaved, attn_factor, stream):
    _need(q.dim() == 4, "tensors are logical [b, h, s, d] views")
    b, h_q, s, d = q.shape
    dt, h_k = _code(q, "q"), 0
    _need(q_out.shape == q.shape and q_out.dtype == q.dtype, "q_out must have q's shape and dtype")
    _need((k is None) == (k_out is None), "k and k_out go together")
    if k is not None:
        _need(k.dim() == 4 and k.shape[0] == b and k.shape[2:] == q.shape[2:] and k.dtype == q.dtype,
              "k must be [b, h_k, s, d] with q's b, s, d and dtype")
        _need(k_out.shape == k.shape and k_out.dtype == k.dtype, "k_out must have k's shape and dtype")
        h_k = k.shape[1]
    _need(str(table.dtype) == "torch.int64" and table.dim() == 1 and table.is_contiguous(),
          "table must be the int64 tensor of sdpa_rope_table")
    pos, pos_stride = _positions(positions, b, s)
    _same_device(q, k, q_out, k_out, table, positions)
    p = _PACK_ROPE(b, h_q, h_k, s, d, 2 * table.shape[0], dt, 1 if interleaved else 0, float(attn_factor),
                   table.data_ptr(), pos, pos_stride, *q.stride(), *_st4(k), *q_out.stride(), *_st4(k_out))
    _launch(fn, stream, q, p, q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out))


def sdpa_rope_fwd(q, k, q_out, k_out, table, positions=None, *, interleaved: bool = False,
                  attn_factor: float = 1.0, stream=None) -> None:
    """Rotary positions of Q and K ([b, h, s, d] views, f16/bf16) into q_out and k_out, which may be q
    and k themselves; ``k`` and ``k_out`` may be None.

    table: int64 CUDA tensor of :func:`sdpa_rope_table` (rot = twice its length; the elements of a head
    behind rot are copied).  positions: int32 [b, s] or [s], or None: 0, 1, ... in every batch."""
    _rope(lib.sdpa_rope_fwd, q, k, q_out, k_out, table, positions, interleaved, attn_factor, stream)


def sdpa_rope_bwd(dq_out, dk_out, dq, dk, table, positions=None, *, interleaved: bool = False,
                  attn_factor: float = 1.0, stream=None) -> None:
    """Gradients of :func:`sdpa_rope_fwd`: dq, dk (overwritten) from the gradients of its outputs."""
    _rope(lib.sdpa_rope_bwd, dq_out, dk_out, dq, dk, table, positions, interleaved, attn_factor, stream)


def _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale):
    _need(k_cache.dim() == 4 and k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype,
          "k_cache and v_cache must be [pages, h_kv, page_size, d] views of one shape and dtype")
    pages, h_kv, page_size, d = k_cache.shape
    _need(page_table.dim() == 2 and str(page_table.dtype) == "torch.int32"
          and (page_table.shape[1] == 1 or page_table.stride(1) == 1),
          "page_table must be int32 [b, max_pages] with a unit last stride")
    b, wide = page_table.shape
    _ints(seq_lens_kv, "seq_lens_kv", (b,))
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _ints(t, n, (pages, h_kv, page_size), "torch.float32")
    _same_device(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    return _PACK_CACHE(pages, page_size, h_kv, d, _code(k_cache, "k_cache"), b, wide, k_cache.data_ptr(),
                       v_cache.data_ptr(), *k_cache.stride(), *v_cache.stride(), _p0(k_scale), _p0(v_scale),
                       page_table.data_ptr(), page_table.stride(0), seq_lens_kv.data_ptr())


def _cache_rows(k, v, k_cache, page_table):
    _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype,
          "k and v must be [b, h_kv, s, d] views of one shape and dtype")
    b, h, s, d = k.shape
    _need(b == page_table.shape[0] and h == k_cache.shape[1] and d == k_cache.shape[3],
          "k and v must have the cache's h_kv and d and a row of the page table for each sequence")
    _same_device(k_cache, k, v)
    return b, s


def sdpa_cache_write(k, v, k_cache, v_cache, page_table, seq_lens_kv, *, seq_lens_q=None, k_scale=None,
                     v_scale=None, rope_table=None, positions=None, interleaved: bool = False,
                     attn_factor: float = 1.0, stream=None) -> None:
    """Writes the new rows k, v ([b, h_kv, s, d], f16/bf16) into a paged cache.

    k_cache, v_cache: [pages, h_kv, page_size, d] views (f16, bf16 or float8_e4m3fn; E4M3 needs k_scale and
    v_scale, fp32 [pages, h_kv, page_size]).  page_table: int32 [b, max_pages]; seq_lens_kv: int32 [b] tokens
    of each sequence with these; seq_lens_q: int32 [b] of them new (None: s).  Row i goes to position
    len_kv - len_q + i.  With ``rope_table`` K is rotated first (positions None: each row's position)."""
    c = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    b, s = _cache_rows(k, v, k_cache, page_table)
    _ints(seq_lens_q, "seq_lens_q", (b,))
    _same_device(k_cache, seq_lens_q, rope_table, positions)
    rope, at = None, 0
    if rope_table is not None:
        _need(str(rope_table.dtype) == "torch.int64" and rope_table.dim() == 1 and rope_table.is_contiguous(),
              "rope_table must be the int64 tensor of sdpa_rope_table")
        pos, pos_stride = _positions(positions, b, s)
        rope = ctypes.create_string_buffer(_PACK_ROPE(
            0, 0, 0, 0, 0, 2 * rope_table.shape[0], 0, 1 if interleaved else 0, float(attn_factor),
            rope_table.data_ptr(), pos, pos_stride, *(_NO_STRIDES * 4)))
        at = ctypes.addressof(rope)
    else:
        _need(positions is None, "positions are those of a rope_table")
    r = _PACK_ROWS(s, _code(k, "k"), *k.stride(), *v.stride(), _p0(seq_lens_q), at)
    _launch(lib.sdpa_cache_write, stream, k_cache, c, r, k.data_ptr(), v.data_ptr())


def sdpa_cache_read(k_cache, v_cache, page_table, seq_lens_kv, k, v, *, k_scale=None, v_scale=None,
                    stream=None) -> None:
    """Reads positions 0 .. s-1 of each sequence into dense k, v ([b, h_kv, s, d], f16/bf16); rows at
    and behind its length are zeros.  Arguments as in :func:`sdpa_cache_write`."""
    c = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    _, s = _cache_rows(k, v, k_cache, page_table)
    r = _PACK_ROWS(s, _code(k, "k"), *k.stride(), *v.stride(), 0, 0)
    _launch(lib.sdpa_cache_read, stream, k_cache, c, r, k.data_ptr(), v.data_ptr())


def _decode(q, k_cache, page_table, o, seq_lens_q, attn_scale, causal, tree_mask):
    _need(q.dim() == 4 and o.shape == q.shape and o.dtype == q.dtype, "q and o must be [b, h_q, s_q, d] views of one shape and dtype")
    b, h_q, s_q, d = q.shape
    _need(b == page_table.shape[0] and d == k_cache.shape[3], "q must have the cache's d and a row of the page table for each sequence")
    _ints(seq_lens_q, "seq_lens_q", (b,))
    stride = 0
    if tree_mask is not None:
        words = (s_q + 31) // 32
        _need(str(tree_mask.dtype) in ("torch.int32", "torch.uint32") and tree_mask.dim() == 3
              and tree_mask.shape[0] in (1, b) and tree_mask.shape[1:] == (s_q, words)
              and tree_mask[0].is_contiguous() and tree_mask.stride(0) >= 0,
              f"tree_mask must be int32 ({b} or 1, {s_q}, {words}), dense in its last two dimensions")
        stride = tree_mask.stride(0) if tree_mask.shape[0] == b and b > 1 else 0
    _same_device(k_cache, q, o, seq_lens_q, tree_mask)
    scale = 1.0 / math.sqrt(d) if attn_scale is None else float(attn_scale)
    return _PACK_DECODE(h_q, s_q, _code(q, "q"), causal_code(causal), scale, *q.stride(), *o.stride(),
                        _p0(seq_lens_q), _p0(tree_mask), stride)


def sdpa_decode_workspace_size(q, k_cache, v_cache, page_table, seq_lens_kv, *, k_scale=None, v_scale=None,
                               tree_mask=None) -> int:
    """Workspace bytes of :func:`sdpa_decode` for these sizes (whatever the lengths)."""
    c = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    p = _decode(q, k_cache, page_table, q, None, 1.0, False, tree_mask)
    n = ctypes.c_size_t(0)
    import torch
    with torch.cuda.device(q.device):
        _check(lib.sdpa_decode_workspace_size(c, p, ctypes.byref(n)))
    return n.value


def sdpa_decode(q, k_cache, v_cache, page_table, seq_lens_kv, o, lse=None, *, workspace, seq_lens_q=None,
                k_scale=None, v_scale=None, attn_scale: Optional[float] = None, causal=False, tree_mask=None,
                stream=None) -> None:
    """Attention of the newest tokens q ([b, h_q, s_q, d], already in the cache) over a paged cache: O, and
    LSE when ``lse`` is given (fp32 [b, h_q, s_q] contiguous).

    causal: False, or "bottom_right".  tree_mask: int32 [b or 1, s_q, ceil(s_q/32)], bit j%32 of word j/32 of
    row i set where drafted token i sees drafted token j (itself among them); earlier positions are seen by
    all.  seq_lens_q: rows that take part (None: all).  workspace: sdpa_decode_workspace_size bytes, not
    shared with a call that may run at the same time."""
    c = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    p = _decode(q, k_cache, page_table, o, seq_lens_q, attn_scale, causal, tree_mask)
    if lse is not None:
        _ints(lse, "lse", tuple(q.shape[:3]), "torch.float32")
    _need(workspace is not None and workspace.is_contiguous(), "workspace must be a contiguous tensor")
    _same_device(k_cache, lse, workspace)
    _launch(lib.sdpa_decode, stream, k_cache, c, p, q.data_ptr(), o.data_ptr(), _ptr(lse), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
