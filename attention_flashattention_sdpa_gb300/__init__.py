"""Python binding of the GB300 fused SDPA library (``include/sdpa.h``).

Argument marshalling only: every step of the attention computation runs in the CUDA
kernels of ``libsdpa_gb300.so``.  PyTorch supplies device memory and the current stream.
The binding keeps the C names: :func:`sdpa_fwd`, :func:`sdpa_bwd`,
:func:`sdpa_workspace_size`, :func:`sdpa_last_error_string`, :func:`sdpa_device_error`; for serving
:func:`sdpa_rope_fwd`, :func:`sdpa_rope_bwd`, :func:`sdpa_cache_write`, :func:`sdpa_cache_read` and
:func:`sdpa_decode`; around them :func:`sdpa_cache_fork`, :func:`sdpa_cache_grow`, :func:`sdpa_cache_free`,
:func:`sdpa_cache_compact`, :func:`sdpa_cache_copy`, :func:`sdpa_cache_keep` and :func:`sdpa_verify`.

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
    "RopeTable", "Rope", "Cache", "CacheRows", "Decode", "RopeAxes", "sdpa_rope_table", "sdpa_rope_axes",
    "sdpa_rope_fwd", "sdpa_rope_bwd", "sdpa_cache_write", "sdpa_cache_read", "sdpa_decode",
    "sdpa_decode_workspace_size", "Pages", "Verify", "sdpa_cache_fork", "sdpa_cache_grow", "sdpa_cache_free",
    "sdpa_cache_compact", "sdpa_cache_copy", "sdpa_cache_keep", "sdpa_verify",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsdpa_gb300.so")

STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID_ARG", 2: "SDPA_ERR_UNSUPPORTED",
          3: "SDPA_ERR_LAYOUT", 4: "SDPA_ERR_WORKSPACE", 5: "SDPA_ERR_CUDA",
          6: "SDPA_ERR_TIMEOUT"}

DTYPE_F16, DTYPE_BF16, DTYPE_E4M3, DTYPE_E5M2, DTYPE_F32 = 0, 1, 2, 3, 4


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


class RopeAxes(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("axis", ctypes.c_uint8 * 256), ("axis_stride", ctypes.c_int64)]


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


class Pages(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("b", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("page_table", ctypes.c_void_p), ("page_table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
        ("ref_counts", ctypes.c_void_p), ("page_table_out", ctypes.c_void_p), ("page_table_out_stride", ctypes.c_int64),
        ("ref_counts_out", ctypes.c_void_p),
    ]


class Verify(ctypes.Structure):
    _fields_ = [
        ("b", ctypes.c_int32), ("s", ctypes.c_int32), ("vocab", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("tokens", ctypes.c_void_p), ("parents", ctypes.c_void_p), ("seq_lens_q", ctypes.c_void_p),
        ("uniform", ctypes.c_void_p), ("probs", ctypes.c_void_p), ("probs_b", ctypes.c_int64), ("probs_s", ctypes.c_int64),
        ("draft_probs", ctypes.c_void_p), ("draft_b", ctypes.c_int64), ("draft_s", ctypes.c_int64),
        ("accepted", ctypes.c_void_p), ("path", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p),
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
        elif typ is ctypes.c_uint8 * 256:
            fmt.append("256s")
        else:
            fmt.append(codes[typ])
        pos = off + ctypes.sizeof(typ)
    fmt.append("x" * (ctypes.sizeof(cls) - pos))
    st = struct.Struct("".join(fmt))
    assert st.size == ctypes.sizeof(cls)
    return st


_PACK = _packer()
_PACK_ROPE, _PACK_CACHE, _PACK_ROWS, _PACK_DECODE = (_packer(c).pack for c in (Rope, Cache, CacheRows, Decode))
_PACK_AXES, _PACK_PAGES, _PACK_VERIFY = (_packer(c).pack for c in (RopeAxes, Pages, Verify))
_NO_STRIDES = (0, 0, 0, 1)
_NO_ROPE_STRIDES = 4 * _NO_STRIDES


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
    L.sdpa_rope_axes_fwd.argtypes = L.sdpa_rope_axes_bwd.argtypes = [VP, VP, VP, VP, VP, VP, VP]
    L.sdpa_cache_write_axes.argtypes = [VP, VP, VP, VP, VP, VP]
    L.sdpa_cache_fork.argtypes = [VP, VP, ctypes.c_int32, VP, VP]
    L.sdpa_cache_grow.argtypes = [VP, VP, VP, VP, VP, VP]
    L.sdpa_cache_free.argtypes = [VP, VP, VP]
    L.sdpa_cache_compact.argtypes = L.sdpa_cache_copy.argtypes = [VP, VP, VP, ctypes.c_int32, VP]
    L.sdpa_cache_keep.argtypes = [VP, VP, VP, ctypes.c_int32, VP, VP]
    L.sdpa_verify.argtypes = [VP, VP]
    L.sdpa_cache_write.argtypes = L.sdpa_cache_read.argtypes = [VP, VP, VP, VP, VP]
    L.sdpa_decode_workspace_size.argtypes = [VP, VP, ctypes.POINTER(SZ)]
    L.sdpa_decode.argtypes = [VP, VP, VP, VP, VP, VP, SZ, VP]
    for f in (L.sdpa_rope_table, L.sdpa_rope_fwd, L.sdpa_rope_bwd, L.sdpa_cache_write, L.sdpa_cache_read,
              L.sdpa_decode_workspace_size, L.sdpa_decode, L.sdpa_rope_axes_fwd, L.sdpa_rope_axes_bwd, L.sdpa_cache_write_axes,
              L.sdpa_cache_fork, L.sdpa_cache_grow, L.sdpa_cache_free, L.sdpa_cache_compact, L.sdpa_cache_copy, L.sdpa_cache_keep,
              L.sdpa_verify):
        f.restype = ctypes.c_int
    L.sdpa_serving_struct_size.argtypes = [ctypes.c_int]
    L.sdpa_serving_struct_size.restype = SZ
    for i, cls in enumerate((RopeTable, Rope, Cache, CacheRows, Decode, RopeAxes, Pages, Verify)):
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
    if _RAW_STREAM and like is not None:
        dev = like.get_device()
        if dev >= 0:
            return _RAW_STREAM(dev)
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


def sdpa_rope_axes(sections, *, order: str = "blocks") -> bytes:
    """The axis of each pair of a rotation with several axes, for ``axes=`` of the calls below: ``sections`` gives the number of
    pairs of each axis (1 to 4 axes).  ``order``: "blocks" (the first axis's pairs, then the second's, ...), or "interleaved"
    (dealt out in turns to the axes that still want one).  Any other order is as good: one byte a pair, its axis.

    The frequencies are the table's, pair by pair; for axes with frequencies of their own, ``torch.cat`` of a table of each."""
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 1:
        raise ValueError(f"sections are the pairs of 1 to 4 axes, one at least each, got {sections}")
    if order == "blocks":
        return bytes(a for a, n in enumerate(sections) for _ in range(n))
    if order == "interleaved":
        return bytes(a for turn in range(max(sections)) for a, n in enumerate(sections) if turn < n)
    raise ValueError(f"unknown order {order!r}")


def _bad(message: str):
    raise ValueError(message)


class _Lazy:
    """What the calls below need of torch, looked up once (a call of a few µs is not to import or to
    compare names)."""
    torch = None

    @classmethod
    def load(cls):
        import torch
        cls.int32, cls.int64, cls.float32 = torch.int32, torch.int64, torch.float32
        cls.probs = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
        cls.words = (torch.int32, getattr(torch, "uint32", torch.int32))
        cls.device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        dtype_code(torch.empty(0, dtype=torch.float16))       # (fills the table of types)
        cls.torch = torch        # last: what says that all of it is there, to other threads too
        return cls


def _code(t, name: str) -> int:
    c = _DTYPES.get(t.dtype)
    return _bad(f"{name}: dtype {t.dtype} is not one the library takes") if c is None else c


def _launch(fn, stream, like, dev, *args):
    """Calls ``fn(*args, stream)`` with ``dev``, the device of ``like``, current."""
    if dev == _Lazy.device():
        st = fn(*args, int(stream) if stream is not None else _stream(None, like))
    else:
        with _Lazy.torch.cuda.device(dev):
            st = fn(*args, int(stream) if stream is not None else _stream(None, like))
    if st != 0:
        _check(st)


def _same_device(like, *tensors):
    """Index of the CUDA device that all of them (None aside) are on."""
    dev = like.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on one device ({like.device} and {t.device} given)")
    return dev


def _dense(t, name: str, dtype, shape):
    """A contiguous tensor of this type and shape; its address."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _positions(positions, b: int, s: int):
    """(address, elements between batches) of positions [b, s], or [s] or [1, s] for every batch."""
    if positions is None:
        return 0, 0
    shape, stride = positions.shape, positions.stride()
    if positions.dtype is not _Lazy.int32 or shape not in ((b, s), (1, s), (s,)) or (s > 1 and stride[-1] != 1):
        raise ValueError(f"positions must be int32 of shape ({b}, {s}), (1, {s}) or ({s},) with a unit last stride")
    return positions.data_ptr(), 0 if len(shape) == 1 or (shape[0] == 1 and b > 1) else stride[0]


def _axis_positions(positions, axes, rot: int, b: int, s: int):
    """(address, elements between batches, packed axes) of positions [axes, b, s], or [axes, s] or [axes, 1, s] for every
    batch."""
    if type(axes) is not bytes or len(axes) != rot // 2:
        raise ValueError(f"axes must be bytes, the axis of each of rot/2 = {rot // 2} pairs")
    if positions is None or positions.dtype is not _Lazy.int32:
        raise ValueError("axes need int32 positions")
    shape, stride = positions.shape, positions.stride()
    if len(shape) not in (2, 3) or shape[1:] not in ((b, s), (1, s), (s,)) or (s > 1 and stride[-1] != 1):
        raise ValueError(f"positions must be of shape (axes, {b}, {s}), (axes, 1, {s}) or (axes, {s}) with a unit last stride")
    return (positions.data_ptr(), 0 if len(shape) == 2 or (shape[1] == 1 and b > 1) else stride[1],
            _PACK_AXES(shape[0], axes, stride[0]))


def _table(t, name: str):
    if t.dtype is not _Lazy.int64 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be the int64 tensor of sdpa_rope_table")
    return t.data_ptr(), 2 * t.shape[0]


def _rope(fn, fn_axes, q, k, q_out, k_out, table, positions, interleaved, attn_factor, axes, stream):
    if _Lazy.torch is None:
        _Lazy.load()
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("tensors are logical [b, h, s, d] views")
    b, h_q, s, d = shape
    dtype = q.dtype
    if q_out.shape != shape or q_out.dtype is not dtype:
        raise ValueError("q_out must have q's shape and dtype")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    h_k, k_ptr, k_out_ptr, k_st, k_out_st = 0, None, None, _NO_STRIDES, _NO_STRIDES
    if k is not None:
        ks = k.shape
        if len(ks) != 4 or ks[0] != b or ks[2] != s or ks[3] != d or k.dtype is not dtype:
            raise ValueError("k must be [b, h_k, s, d] with q's b, s, d and dtype")
        if k_out.shape != ks or k_out.dtype is not dtype:
            raise ValueError("k_out must have k's shape and dtype")
        h_k, k_ptr, k_out_ptr, k_st, k_out_st = ks[1], k.data_ptr(), k_out.data_ptr(), k.stride(), k_out.stride()
    dt = _code(q, "q")
    tab, rot = _table(table, "table")
    if axes is None:
        pos, pos_stride = _positions(positions, b, s)
    else:
        pos, pos_stride, several = _axis_positions(positions, axes, rot, b, s)
    dev = _same_device(q, k, q_out, k_out, table, positions)
    p = _PACK_ROPE(b, h_q, h_k, s, d, rot, dt, 1 if interleaved else 0, attn_factor, tab, pos, pos_stride, *q.stride(), *k_st,
                   *q_out.stride(), *k_out_st)
    if axes is None:
        _launch(fn, stream, q, dev, p, q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr)
    else:
        _launch(fn_axes, stream, q, dev, p, several, q.data_ptr(), k_ptr, q_out.data_ptr(), k_out_ptr)


def sdpa_rope_fwd(q, k, q_out, k_out, table, positions=None, *, interleaved: bool = False,
                  attn_factor: float = 1.0, axes: Optional[bytes] = None, stream=None) -> None:
    """Rotary positions of Q and K ([b, h, s, d] views, f16/bf16) into q_out and k_out, which may be q
    and k themselves; ``k`` and ``k_out`` may be None.

    table: int64 CUDA tensor of :func:`sdpa_rope_table` (rot = twice its length; the elements of a head
    behind rot are copied).  positions: int32 [b, s] or [s], or None: 0, 1, ... in every batch.
    axes: None, or the axis of each pair (:func:`sdpa_rope_axes`); positions are then int32 [axes, b, s] or [axes, s], and
    pair i turns by the position on its own axis."""
    _rope(lib.sdpa_rope_fwd, lib.sdpa_rope_axes_fwd, q, k, q_out, k_out, table, positions, interleaved, attn_factor, axes, stream)


def sdpa_rope_bwd(dq_out, dk_out, dq, dk, table, positions=None, *, interleaved: bool = False,
                  attn_factor: float = 1.0, axes: Optional[bytes] = None, stream=None) -> None:
    """Gradients of :func:`sdpa_rope_fwd`: dq, dk (overwritten) from the gradients of its outputs."""
    _rope(lib.sdpa_rope_bwd, lib.sdpa_rope_axes_bwd, dq_out, dk_out, dq, dk, table, positions, interleaved, attn_factor, axes, stream)


def _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale):
    """The packed descriptor of a cache, its shape, and the number of sequences."""
    if _Lazy.torch is None:
        _Lazy.load()
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must be [pages, h_kv, page_size, d] views of one shape and dtype")
    pages, h_kv, page_size, d = shape
    ts, tst = page_table.shape, page_table.stride()
    if len(ts) != 2 or page_table.dtype is not _Lazy.int32 or (ts[1] > 1 and tst[1] != 1):
        raise ValueError("page_table must be int32 [b, max_pages] with a unit last stride")
    lens = _dense(seq_lens_kv, "seq_lens_kv", _Lazy.int32, ts[:1])
    ks = 0 if k_scale is None else _dense(k_scale, "k_scale", _Lazy.float32, shape[:3])
    vs = 0 if v_scale is None else _dense(v_scale, "v_scale", _Lazy.float32, shape[:3])
    return _PACK_CACHE(pages, page_size, h_kv, d, _code(k_cache, "k_cache"), ts[0], ts[1], k_cache.data_ptr(), v_cache.data_ptr(),
                       *k_cache.stride(), *v_cache.stride(), ks, vs, page_table.data_ptr(), tst[0], lens), shape, ts[0]


def _cache_rows(k, v, k_cache, shape, n: int):
    ks = k.shape
    if len(ks) != 4 or v.shape != ks or v.dtype is not k.dtype:
        raise ValueError("k and v must be [b, h_kv, s, d] views of one shape and dtype")
    if ks[0] != n or ks[1] != shape[1] or ks[3] != shape[3]:
        raise ValueError("k and v must have the cache's h_kv and d and a row of the page table for each sequence")
    return ks


def sdpa_cache_write(k, v, k_cache, v_cache, page_table, seq_lens_kv, *, seq_lens_q=None, k_scale=None,
                     v_scale=None, rope_table=None, positions=None, interleaved: bool = False,
                     attn_factor: float = 1.0, axes: Optional[bytes] = None, stream=None) -> None:
    """Writes the new rows k, v ([b, h_kv, s, d], f16/bf16) into a paged cache.

    k_cache, v_cache: [pages, h_kv, page_size, d] views (f16, bf16 or float8_e4m3fn; E4M3 needs k_scale and
    v_scale, fp32 [pages, h_kv, page_size]).  page_table: int32 [b, max_pages]; seq_lens_kv: int32 [b] tokens
    of each sequence with these; seq_lens_q: int32 [b] of them new (None: s).  Row i goes to position
    len_kv - len_q + i.  With ``rope_table`` K is rotated first (positions None: each row's position; with ``axes`` as in
    :func:`sdpa_rope_fwd`)."""
    c, shape, n = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    b, _, s, _ = _cache_rows(k, v, k_cache, shape, n)
    lens_q = 0 if seq_lens_q is None else _dense(seq_lens_q, "seq_lens_q", _Lazy.int32, (b,))
    at = 0
    if rope_table is not None:
        tab, rot = _table(rope_table, "rope_table")
        if axes is None:
            pos, pos_stride = _positions(positions, b, s)
        else:
            pos, pos_stride, several = _axis_positions(positions, axes, rot, b, s)
        rope = Rope.from_buffer_copy(_PACK_ROPE(0, 0, 0, 0, 0, rot, 0, 1 if interleaved else 0, attn_factor, tab, pos, pos_stride,
                                                *_NO_ROPE_STRIDES))
        at = ctypes.addressof(rope)
    elif positions is not None or axes is not None:
        raise ValueError("positions and axes are those of a rope_table")
    dev = _same_device(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale, k, v, seq_lens_q, rope_table, positions)
    r = _PACK_ROWS(s, _code(k, "k"), *k.stride(), *v.stride(), lens_q, at)
    if axes is None:
        _launch(lib.sdpa_cache_write, stream, k_cache, dev, c, r, k.data_ptr(), v.data_ptr())
    else:
        _launch(lib.sdpa_cache_write_axes, stream, k_cache, dev, c, r, several, k.data_ptr(), v.data_ptr())


def sdpa_cache_read(k_cache, v_cache, page_table, seq_lens_kv, k, v, *, k_scale=None, v_scale=None,
                    stream=None) -> None:
    """Reads positions 0 .. s-1 of each sequence into dense k, v ([b, h_kv, s, d], f16/bf16); rows at
    and behind its length are zeros.  Arguments as in :func:`sdpa_cache_write`."""
    c, shape, n = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    ks = _cache_rows(k, v, k_cache, shape, n)
    dev = _same_device(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale, k, v)
    r = _PACK_ROWS(ks[2], _code(k, "k"), *k.stride(), *v.stride(), 0, 0)
    _launch(lib.sdpa_cache_read, stream, k_cache, dev, c, r, k.data_ptr(), v.data_ptr())


def _decode(q, k_cache, shape, n, o, seq_lens_q, attn_scale, causal, tree_mask):
    qs = q.shape
    if len(qs) != 4 or o.shape != qs or o.dtype is not q.dtype:
        raise ValueError("q and o must be [b, h_q, s_q, d] views of one shape and dtype")
    b, h_q, s_q, d = qs
    if b != n or d != shape[3]:
        raise ValueError("q must have the cache's d and a row of the page table for each sequence")
    lens_q = 0 if seq_lens_q is None else _dense(seq_lens_q, "seq_lens_q", _Lazy.int32, (b,))
    tree, tree_stride = 0, 0
    if tree_mask is not None:
        ts, words = tree_mask.shape, (s_q + 31) // 32
        st = tree_mask.stride()
        if tree_mask.dtype not in _Lazy.words or ts not in ((b, s_q, words), (1, s_q, words)) \
                or (words > 1 and st[2] != 1) or (s_q > 1 and st[1] != words):
            raise ValueError(f"tree_mask must be int32 ({b} or 1, {s_q}, {words}), dense in its last two dimensions")
        tree, tree_stride = tree_mask.data_ptr(), st[0] if ts[0] > 1 else 0
    return _PACK_DECODE(h_q, s_q, _code(q, "q"), causal_code(causal), 1.0 / math.sqrt(d) if attn_scale is None else attn_scale,
                        *q.stride(), *o.stride(), lens_q, tree, tree_stride)


def sdpa_decode_workspace_size(q, k_cache, v_cache, page_table, seq_lens_kv, *, k_scale=None, v_scale=None,
                               tree_mask=None) -> int:
    """Workspace bytes of :func:`sdpa_decode` for these sizes (whatever the lengths)."""
    c, shape, n = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    p = _decode(q, k_cache, shape, n, q, None, 1.0, False, tree_mask)
    size = ctypes.c_size_t(0)
    with _Lazy.torch.cuda.device(_same_device(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale, q, tree_mask)):
        _check(lib.sdpa_decode_workspace_size(c, p, ctypes.byref(size)))
    return size.value


def sdpa_decode(q, k_cache, v_cache, page_table, seq_lens_kv, o, lse=None, *, workspace, seq_lens_q=None,
                k_scale=None, v_scale=None, attn_scale: Optional[float] = None, causal=False, tree_mask=None,
                stream=None) -> None:
    """Attention of the newest tokens q ([b, h_q, s_q, d], already in the cache) over a paged cache: O, and
    LSE when ``lse`` is given (fp32 [b, h_q, s_q] contiguous).

    causal: False, or "bottom_right".  tree_mask: int32 [b or 1, s_q, ceil(s_q/32)], bit j%32 of word j/32 of
    row i set where drafted token i sees drafted token j (itself among them); earlier positions are seen by
    all.  seq_lens_q: rows that take part (None: all).  workspace: sdpa_decode_workspace_size bytes, not
    shared with a call that may run at the same time.  The work is split by the page table's columns: with
    ``page_table[:, :n]``, n pages for the longest sequence, short ones take one launch instead of two (a
    workspace for the whole table will do)."""
    c, shape, n = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    p = _decode(q, k_cache, shape, n, o, seq_lens_q, attn_scale, causal, tree_mask)
    lse_ptr = None if lse is None else _dense(lse, "lse", _Lazy.float32, q.shape[:3])
    if workspace is None or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    dev = _same_device(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale, q, o, seq_lens_q, tree_mask, lse, workspace)
    _launch(lib.sdpa_decode, stream, k_cache, dev, c, p, q.data_ptr(), o.data_ptr(), lse_ptr, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())


# ---- pages: who owns which, and pages and rows moved ------------------------------------------

def _page_table(t, name: str, shape=None):
    """(address, shape, elements between rows) of an int32 page table with a unit last stride."""
    ts, st = t.shape, t.stride()
    if len(ts) != 2 or t.dtype is not _Lazy.int32 or (ts[1] > 1 and st[1] != 1) or (shape is not None and ts != shape):
        raise ValueError(f"{name} must be int32 {'[b, max_pages]' if shape is None else tuple(shape)} with a unit last stride")
    return t.data_ptr(), ts, st[0]


def _pages(page_table, seq_lens, ref_counts, table_out, refs_out, page_size, b_out=None):
    """The packed descriptor and the number of rows; outputs that are None are the inputs."""
    if _Lazy.torch is None:
        _Lazy.load()
    int32 = _Lazy.int32
    at, (b, columns), stride = _page_table(page_table, "page_table")
    n = ref_counts.shape
    if len(n) != 1:
        raise ValueError("ref_counts must be int32 [num_pages]")
    refs = _dense(ref_counts, "ref_counts", int32, n)
    out_at, out_stride, refs_at = at, stride, refs
    if table_out is not None:
        out_at, _, out_stride = _page_table(table_out, "page_table_out", (b if b_out is None else b_out, columns))
    if refs_out is not None:
        refs_at = _dense(refs_out, "ref_counts_out", int32, n)
    return _PACK_PAGES(n[0], page_size, b, columns, at, stride, _dense(seq_lens, "seq_lens", int32, (b,)), refs, out_at, out_stride,
                       refs_at), b


def _pairs(src, dst):
    """Addresses and length of a list of pages."""
    n = src.shape
    if len(n) != 1:
        raise ValueError("src and dst must be int32 of one dimension")
    return _dense(src, "src", _Lazy.int32, n), _dense(dst, "dst", _Lazy.int32, n), n[0]


def sdpa_cache_fork(page_table, seq_lens, parents, ref_counts, page_table_out, seq_lens_out, ref_counts_out=None, *,
                    page_size: int, stream=None) -> None:
    """Row i of ``page_table_out`` (int32 [b_out, max_pages]) takes over sequence ``parents[i]`` (int32 [b_out]; outside
    0..b-1: none) of ``page_table`` with its pages, shared, and its length (``seq_lens_out``: int32 [b_out]).  Old rows
    that nobody takes over are freed.

    ref_counts: int32 [num_pages] owners of each page, updated into ref_counts_out (None: in place)."""
    if parents.dim() != 1:
        raise ValueError("parents must be int32 [b_out]")
    n = parents.shape[0]
    p, _ = _pages(page_table, seq_lens, ref_counts, page_table_out, ref_counts_out, page_size, n)
    parents_at = _dense(parents, "parents", _Lazy.int32, (n,))
    lens_at = _dense(seq_lens_out, "seq_lens_out", _Lazy.int32, (n,))
    dev = _same_device(page_table, seq_lens, parents, ref_counts, page_table_out, seq_lens_out, ref_counts_out)
    _launch(lib.sdpa_cache_fork, stream, page_table, dev, p, parents_at, n, lens_at)


def sdpa_cache_grow(page_table, seq_lens, new_lens, ref_counts, src, dst, missing, *, page_size: int, page_table_out=None,
                    ref_counts_out=None, stream=None) -> None:
    """Pages for sequences that grow from ``seq_lens`` to ``new_lens`` (int32 [b]), the lowest free ones (count 0) first.

    A partly filled page that others own too is replaced: (src[i], dst[i]) (int32 [b]; -1: none) is the copy that row i needs
    before it is written, by :func:`sdpa_cache_copy` in every layer's cache.  All or nothing: ``missing`` (int32 [1]) is 0, or
    the number of pages that lacked, and nothing has changed then: what follows goes on with the old lengths and no new rows
    (``rows = torch.where(missing == 0, s, 0)`` as seq_lens_q), or rows of sequences that still share a page would overwrite each
    other.  Outputs that are None: in place."""
    p, b = _pages(page_table, seq_lens, ref_counts, page_table_out, ref_counts_out, page_size)
    new_at = _dense(new_lens, "new_lens", _Lazy.int32, (b,))
    src_at, dst_at, n = _pairs(src, dst)
    if n != b:
        raise ValueError(f"src and dst must have an entry for each of {b} rows")
    missing_at = _dense(missing, "missing", _Lazy.int32, (1,))
    dev = _same_device(page_table, seq_lens, new_lens, ref_counts, src, dst, missing, page_table_out, ref_counts_out)
    _launch(lib.sdpa_cache_grow, stream, page_table, dev, p, new_at, src_at, dst_at, missing_at)


def sdpa_cache_free(page_table, seq_lens, keep_lens, ref_counts, *, page_size: int, page_table_out=None, ref_counts_out=None,
                    stream=None) -> None:
    """Gives back the pages behind ``keep_lens`` (int32 [b]) tokens of each sequence: their entries become -1, their
    pages lose an owner.  Outputs that are None: in place."""
    p, b = _pages(page_table, seq_lens, ref_counts, page_table_out, ref_counts_out, page_size)
    keep_at = _dense(keep_lens, "keep_lens", _Lazy.int32, (b,))
    dev = _same_device(page_table, seq_lens, keep_lens, ref_counts, page_table_out, ref_counts_out)
    _launch(lib.sdpa_cache_free, stream, page_table, dev, p, keep_at)


def sdpa_cache_compact(page_table, seq_lens, ref_counts, src, dst, *, page_size: int, page_table_out=None, ref_counts_out=None,
                       stream=None) -> None:
    """Moves the pages in use together at the front of the cache, at most ``src.numel()`` of them: (src[k], dst[k]) (int32,
    src ascending, -1 behind the last) are the copies to make by :func:`sdpa_cache_copy`.  Outputs that are None: in place."""
    p, _ = _pages(page_table, seq_lens, ref_counts, page_table_out, ref_counts_out, page_size)
    src_at, dst_at, n = _pairs(src, dst)
    dev = _same_device(page_table, seq_lens, ref_counts, src, dst, page_table_out, ref_counts_out)
    _launch(lib.sdpa_cache_compact, stream, page_table, dev, p, src_at, dst_at, n)


def _stored(k_cache, v_cache, k_scale, v_scale):
    """The packed descriptor of a cache without a page table."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must be [pages, h_kv, page_size, d] views of one shape and dtype")
    pages, h_kv, page_size, d = shape
    ks = 0 if k_scale is None else _dense(k_scale, "k_scale", _Lazy.float32, shape[:3])
    vs = 0 if v_scale is None else _dense(v_scale, "v_scale", _Lazy.float32, shape[:3])
    return _PACK_CACHE(pages, page_size, h_kv, d, _code(k_cache, "k_cache"), 0, 0, k_cache.data_ptr(), v_cache.data_ptr(),
                       *k_cache.stride(), *v_cache.stride(), ks, vs, 0, 0, 0)


def sdpa_cache_copy(k_cache, v_cache, src, dst, *, k_scale=None, v_scale=None, stream=None) -> None:
    """Copies pages ``src[i]`` to ``dst[i]`` (int32; pairs with an entry outside the cache are passed over) of K, V and their
    scales.  No page may be the target of two pairs, nor target of one and source of another."""
    if _Lazy.torch is None:
        _Lazy.load()
    c = _stored(k_cache, v_cache, k_scale, v_scale)
    src_at, dst_at, n = _pairs(src, dst)
    dev = _same_device(k_cache, v_cache, src, dst, k_scale, v_scale)
    _launch(lib.sdpa_cache_copy, stream, k_cache, dev, c, src_at, dst_at, n)


def sdpa_cache_keep(k_cache, v_cache, page_table, seq_lens_kv, path, accepted, *, seq_lens_q=None, k_scale=None, v_scale=None,
                    stream=None) -> None:
    """Of the newest s tokens of each sequence (seq_lens_q: int32 [b] of them, None: all s) row ``path[i, j]`` moves to row j for
    j < ``accepted[i]``: int32 [b, s] and [b] of :func:`sdpa_verify`.  The sequences' lengths are then seq_lens_kv -
    seq_lens_q + accepted, which is the caller's to note."""
    c, _, n = _cache(k_cache, v_cache, page_table, seq_lens_kv, k_scale, v_scale)
    if path.dim() != 2:
        raise ValueError("path must be int32 [b, s]")
    s = path.shape[1]
    path_at, accepted_at = _dense(path, "path", _Lazy.int32, (n, s)), _dense(accepted, "accepted", _Lazy.int32, (n,))
    lens_q = 0 if seq_lens_q is None else _dense(seq_lens_q, "seq_lens_q", _Lazy.int32, (n,))
    dev = _same_device(k_cache, v_cache, page_table, seq_lens_kv, path, accepted, seq_lens_q, k_scale, v_scale)
    _launch(lib.sdpa_cache_keep, stream, k_cache, dev, c, path_at, accepted_at, s, lens_q)


def sdpa_verify(tokens, probs, uniform, accepted, path, new_tokens, *, parents=None, draft_probs=None, seq_lens_q=None,
                stream=None) -> None:
    """Drafted tokens verified against the target's probabilities, so that the tokens kept are distributed as the target's own.

    tokens: int32 [b, s], row 0 the newest decided token, the others drafted, row i behind row ``parents[i]`` < i (int32
    [b, s]; None: a chain).  probs: [b, s, vocab] (f16, bf16, f32), the target's distribution behind each row; draft_probs:
    the same of the draft, from which row i of a chain was drawn (None: whatever drafted it).  uniform: fp32 [b, s] in [0, 1).
    seq_lens_q: int32 [b] rows that take part (None: all).

    accepted: int32 [b] rows kept, row 0 among them; path: int32 [b, s], those rows; new_tokens: int32 [b, s], the accepted
    drafts and the token drawn behind them, ``accepted`` in all; -1 behind those.  These lie apart from all inputs.  Rules in
    ``include/sdpa.h``."""
    if _Lazy.torch is None:
        _Lazy.load()
    shape = probs.shape
    if len(shape) != 3 or (shape[2] > 1 and probs.stride(2) != 1) or probs.dtype not in _Lazy.probs:
        raise ValueError("probs must be float16, bfloat16 or float32 [b, s, vocab] with a unit last stride")
    b, s, vocab = shape
    rows, int32 = shape[:2], _Lazy.int32
    draft_at = draft_b = draft_s = 0
    if draft_probs is not None:
        if draft_probs.shape != shape or draft_probs.dtype is not probs.dtype or (vocab > 1 and draft_probs.stride(2) != 1):
            raise ValueError("draft_probs must have probs' shape and dtype, and a unit last stride")
        draft_at, (draft_b, draft_s, _) = draft_probs.data_ptr(), draft_probs.stride()
    p = _PACK_VERIFY(b, s, vocab, _Lazy.probs[probs.dtype], _dense(tokens, "tokens", int32, rows),
                     0 if parents is None else _dense(parents, "parents", int32, rows),
                     0 if seq_lens_q is None else _dense(seq_lens_q, "seq_lens_q", int32, shape[:1]),
                     _dense(uniform, "uniform", _Lazy.float32, rows), probs.data_ptr(), probs.stride(0), probs.stride(1),
                     draft_at, draft_b, draft_s, _dense(accepted, "accepted", int32, shape[:1]), _dense(path, "path", int32, rows),
                     _dense(new_tokens, "new_tokens", int32, rows))
    dev = _same_device(probs, tokens, uniform, accepted, path, new_tokens, parents, draft_probs, seq_lens_q)
    _launch(lib.sdpa_verify, stream, probs, dev, p)
