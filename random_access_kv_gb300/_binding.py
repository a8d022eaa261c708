"""ctypes binding of libfq.so: the C ABI of include/fq.h, include/fractal.h and include/qcache.h under
the same names.

Argument marshalling only: every function takes device buffers as torch CUDA tensors (or raw
integer addresses), passes their addresses and sizes to the C entry point of the same name and
raises ``FQError`` on a non-zero return code. No step of the codec runs here.

The library is loaded from this package directory. If it is missing the import fails loudly
(``FQLibraryMissing``): there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfq.so")
HEADERS = [os.path.join(os.path.dirname(PKG), "include", h) for h in ("fq.h", "fractal.h", "qcache.h")]

FQ_OK, FQ_EINVAL, FQ_ENOMEM, FQ_ECUDA, FQ_EALIGN, FQ_ENODEV = range(6)
FQ_FLAG_RANGE, FQ_FLAG_NONFINITE, FQ_FLAG_TIMEOUT = 1, 2, 4
FA_FLAG_SYMBOL, FA_FLAG_RANGE, FA_FLAG_CORRUPT = 1, 2, 4
QC_FORMATS = {"int8": 0, "e4m3": 1, "e2m1": 2}
QC_FLAG_RANGE, QC_FLAG_NONFINITE, QC_FLAG_TIMEOUT, QC_FLAG_PAGES = 1, 2, 4, 8


class FQLibraryMissing(ImportError):
    pass


class FQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {strerror(code)} ({code})")


_c_void_p, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int

_SIGNATURES = {
    "fq_codebook_load": (_int, [ctypes.POINTER(_c_void_p), _c_void_p, _int, _int, _c_void_p, _int, _int]),
    "fq_encode": (_int, [_c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _i64, _c_void_p]),
    "fq_encode_append": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "fq_decode": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p]),
    "fq_decode_gather": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _i64, _c_void_p, _c_void_p]),
    "fq_decode_gather_f32": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _i64, _c_void_p, _c_void_p]),
    "fq_attend": (_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _i64, _i64, _i64, _i64, _i64, _i64,
                         ctypes.c_float, _c_void_p, _c_void_p]),
    "fq_centroid_sums": (_int, [_c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "fq_selftest_wait": (_int, [_c_void_p, ctypes.c_uint64, _c_void_p]),
    "fq_code_words": (_i64, [_c_void_p, _i64]),
    "fq_record_bits": (_int, [_c_void_p]),
    "fq_shape": (_int, [_c_void_p, ctypes.POINTER(_int), ctypes.POINTER(_int), ctypes.POINTER(_int)]),
    "fq_status": (_int, [_c_void_p, _c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "fq_destroy": (None, [_c_void_p]),
    "fq_strerror": (ctypes.c_char_p, [_int]),
    "fa_ratio_limit": (ctypes.c_double, [_int]),
    "fa_max_segment": (_int, [_int, ctypes.c_double]),
    "fa_create": (_int, [ctypes.POINTER(_c_void_p), _int, ctypes.c_double, _int, _int]),
    "fa_params": (_int, [_c_void_p, ctypes.POINTER(_int), ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_int)]),
    "fa_vertex_table": (_int, [_c_void_p, _c_void_p]),
    "fa_segments": (_i64, [_c_void_p, _i64]),
    "fa_encode": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _i64, _c_void_p, _c_void_p]),
    "fa_decode": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p]),
    "fa_access": (_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p, _c_void_p]),
    "fa_status": (_int, [_c_void_p, _c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "fa_destroy": (None, [_c_void_p]),
    "qc_create": (_int, [ctypes.POINTER(_c_void_p), _int, _int, _int, _int, _int]),
    "qc_page_bytes": (_i64, [_c_void_p]),
    "qc_norm_rope": (_int, [_c_void_p, _int, _i64, _c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _int, _i64, _i64,
                            _c_void_p, ctypes.c_float, _c_void_p, _c_void_p, _i64, _int, _int, _c_void_p, _i64, _i64,
                            _c_void_p, _i64, _i64, _c_void_p]),
    "qc_write": (_int, [_c_void_p, _int, _i64, _c_void_p, _i64, _i64, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _i64,
                        _c_void_p]),
    "qc_read": (_int, [_c_void_p, _int, _i64, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p]),
    "qc_attend": (_int, [_c_void_p, _int, _i64, _int, _int, _c_void_p, _i64, _i64, _i64, _c_void_p, _i64, _c_void_p,
                         _c_void_p, _c_void_p, _c_void_p, _i64, ctypes.c_float, _i64, _c_void_p, _c_void_p, _c_void_p,
                         _i64, _c_void_p]),
    "qc_attend_workspace": (_i64, [_c_void_p, _i64, _int, _int, _i64]),
    "qc_norm_rope_axes": (_int, [_c_void_p, _int, _i64, _c_void_p, _int, _i64, _i64, _c_void_p, _c_void_p, _int, _i64, _i64,
                                 _c_void_p, ctypes.c_float, _c_void_p, _c_void_p, _i64, _c_void_p, _int, _int, _c_void_p, _i64,
                                 _i64, _c_void_p, _i64, _i64, _c_void_p]),
    "qc_plan": (_int, [_c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _i64, _c_void_p, _c_void_p, _i64, _i64, _c_void_p,
                       _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "qc_attend_chunk": (_int, [_c_void_p, _int, _i64, _i64, _int, _c_void_p, _i64, _i64, _c_void_p, _c_void_p, _i64, _c_void_p,
                               _c_void_p, _c_void_p, _c_void_p, _i64, ctypes.c_float, ctypes.c_float, _i64, _i64, _i64, _c_void_p,
                               _c_void_p, _c_void_p, _i64, _c_void_p]),
    "qc_attend_chunk_workspace": (_i64, [_c_void_p, _i64, _i64, _int, _i64, _i64]),
    "qc_verify": (_int, [_c_void_p, _int, _i64, _int, _i64, _c_void_p, _i64, _i64, _c_void_p, _i64, _i64, _c_void_p, _c_void_p,
                         _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "qc_status": (_int, [_c_void_p, _c_void_p, ctypes.POINTER(ctypes.c_uint32)]),
    "qc_destroy": (None, [_c_void_p]),
}

_lib = None


def header_symbols() -> list[str]:
    """Names of the functions declared in the headers under include/."""
    names = set()
    for h in HEADERS:
        with open(h) as f:
            text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
        names.update(re.findall(r"\b((?:fq|fa|qc)_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def lib() -> ctypes.CDLL:
    """The loaded library (loaded on first use)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FQLibraryMissing(f"{LIB_PATH} is not built; run random_access_kv_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().fq_strerror(int(code)).decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr() if t.numel() else None
    if hasattr(t, "ctypes"):            # numpy host array
        return t.ctypes.data
    raise TypeError(f"cannot take the address of {type(t)}")


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != FQ_OK:
        raise FQError(fn, rc)


class Context:
    """Owns an ``fq_ctx*``; frees it with ``fq_destroy`` on ``close()`` or garbage collection."""

    _destroy = "fq_destroy"

    def __init__(self, handle: int):
        self.handle = handle

    @property
    def _as_parameter_(self):
        return ctypes.c_void_p(self.handle)

    def close(self) -> None:
        if self.handle:
            getattr(lib(), self._destroy)(ctypes.c_void_p(self.handle))
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fq_codebook_load(C, Pi, device: int = 0) -> Context:
    """C: float32 [N, k] host array; Pi: float32 [d, d] host array (C-contiguous numpy)."""
    import numpy as np
    C = np.ascontiguousarray(C, dtype=np.float32)
    Pi = np.ascontiguousarray(Pi, dtype=np.float32)
    if C.ndim != 2 or Pi.ndim != 2 or Pi.shape[0] != Pi.shape[1]:
        raise ValueError("C must be [N, k] and Pi [d, d]")
    h = _c_void_p()
    rc = lib().fq_codebook_load(ctypes.byref(h), C.ctypes.data, C.shape[0], C.shape[1],
                                Pi.ctypes.data, Pi.shape[0], int(device))
    _check("fq_codebook_load", rc)
    return Context(h.value)


def fq_encode(ctx: Context, x, M: int, nu, codes, row0: int = 0, stream=None) -> None:
    _check("fq_encode", lib().fq_encode(ctx, _ptr(x), int(M), _ptr(nu), _ptr(codes), int(row0),
                                        _stream(stream)))


def fq_encode_append(ctx: Context, x, n_seq: int, n_new: int, seq_capacity: int, t0: int, nu, codes,
                     stream=None) -> None:
    _check("fq_encode_append", lib().fq_encode_append(ctx, _ptr(x), int(n_seq), int(n_new),
                                                      int(seq_capacity), int(t0), _ptr(nu), _ptr(codes),
                                                      _stream(stream)))


def fq_decode(ctx: Context, nu, codes, M: int, out, stream=None) -> None:
    _check("fq_decode", lib().fq_decode(ctx, _ptr(nu), _ptr(codes), int(M), _ptr(out), _stream(stream)))


def fq_decode_gather(ctx: Context, nu, codes, M: int, idx, n: int, out, stream=None) -> None:
    _check("fq_decode_gather", lib().fq_decode_gather(ctx, _ptr(nu), _ptr(codes), int(M), _ptr(idx), int(n),
                                                      _ptr(out), _stream(stream)))


def fq_decode_gather_f32(ctx: Context, nu, codes, M: int, idx, n: int, out, stream=None) -> None:
    _check("fq_decode_gather_f32", lib().fq_decode_gather_f32(ctx, _ptr(nu), _ptr(codes), int(M), _ptr(idx),
                                                              int(n), _ptr(out), _stream(stream)))


def fq_attend(ctx: Context, nu, codes, M: int, q, n_queries: int, q_per_group: int, T: int, k_row0: int,
              v_row0: int, stride: int, scale: float, out, stream=None) -> None:
    _check("fq_attend", lib().fq_attend(ctx, _ptr(nu), _ptr(codes), int(M), _ptr(q), int(n_queries),
                                        int(q_per_group), int(T), int(k_row0), int(v_row0), int(stride),
                                        float(scale), _ptr(out), _stream(stream)))


def fq_centroid_sums(ctx: Context, x, M: int, nu, codes, sums, counts, stream=None) -> None:
    _check("fq_centroid_sums", lib().fq_centroid_sums(ctx, _ptr(x), int(M), _ptr(nu), _ptr(codes), _ptr(sums),
                                                      _ptr(counts), _stream(stream)))


def fq_selftest_wait(ctx: Context, limit_ns: int, stream=None) -> None:
    _check("fq_selftest_wait", lib().fq_selftest_wait(ctx, int(limit_ns), _stream(stream)))


def fq_code_words(ctx: Context, M: int) -> int:
    w = lib().fq_code_words(ctx, int(M))
    if w < 0:
        raise FQError("fq_code_words", FQ_EINVAL)
    return int(w)


def fq_record_bits(ctx: Context) -> int:
    return int(lib().fq_record_bits(ctx))


def fq_shape(ctx: Context) -> tuple[int, int, int]:
    d, k, N = _int(), _int(), _int()
    _check("fq_shape", lib().fq_shape(ctx, ctypes.byref(d), ctypes.byref(k), ctypes.byref(N)))
    return d.value, k.value, N.value


def fq_status(ctx: Context, stream=None) -> int:
    f = ctypes.c_uint32()
    _check("fq_status", lib().fq_status(ctx, _stream(stream), ctypes.byref(f)))
    return int(f.value)


def fq_destroy(ctx: Context) -> None:
    ctx.close()


def fq_strerror(code: int) -> str:
    return strerror(code)


# Iterated-map archive of symbol streams (include/fractal.h).

class ArchiveContext(Context):
    """Owns an ``fa_ctx*``; frees it with ``fa_destroy``."""

    _destroy = "fa_destroy"


def fa_ratio_limit(N: int) -> float:
    return float(lib().fa_ratio_limit(int(N)))


def fa_max_segment(N: int, r: float) -> int:
    return int(lib().fa_max_segment(int(N), float(r)))


def fa_create(N: int, r: float, L: int, device: int = 0) -> ArchiveContext:
    h = _c_void_p()
    _check("fa_create", lib().fa_create(ctypes.byref(h), int(N), float(r), int(L), int(device)))
    return ArchiveContext(h.value)


def fa_params(ctx: ArchiveContext) -> tuple[int, float, int]:
    N, r, L = _int(), ctypes.c_double(), _int()
    _check("fa_params", lib().fa_params(ctx, ctypes.byref(N), ctypes.byref(r), ctypes.byref(L)))
    return N.value, r.value, L.value


def fa_vertex_table(ctx: ArchiveContext):
    """The context's vertex table as a float64 numpy array [N, 2]."""
    import numpy as np
    N, _, _ = fa_params(ctx)
    V = np.zeros((N, 2), dtype=np.float64)
    _check("fa_vertex_table", lib().fa_vertex_table(ctx, V.ctypes.data))
    return V


def fa_segments(ctx: ArchiveContext, T_cap: int) -> int:
    s = lib().fa_segments(ctx, int(T_cap))
    if s < 0:
        raise FQError("fa_segments", FQ_EINVAL)
    return int(s)


def fa_encode(ctx: ArchiveContext, sym, n_streams: int, n_new: int, T_cap: int, T_old: int, anchors,
              stream=None) -> None:
    _check("fa_encode", lib().fa_encode(ctx, _ptr(sym), int(n_streams), int(n_new), int(T_cap), int(T_old),
                                        _ptr(anchors), _stream(stream)))


def fa_decode(ctx: ArchiveContext, anchors, n_streams: int, T_cap: int, T: int, out, stream=None) -> None:
    _check("fa_decode", lib().fa_decode(ctx, _ptr(anchors), int(n_streams), int(T_cap), int(T), _ptr(out),
                                        _stream(stream)))


def fa_access(ctx: ArchiveContext, anchors, n_streams: int, T_cap: int, T: int, pos, n: int, out,
              stream=None) -> None:
    _check("fa_access", lib().fa_access(ctx, _ptr(anchors), int(n_streams), int(T_cap), int(T), _ptr(pos), int(n),
                                        _ptr(out), _stream(stream)))


def fa_status(ctx: ArchiveContext, stream=None) -> int:
    f = ctypes.c_uint32()
    _check("fa_status", lib().fa_status(ctx, _stream(stream), ctypes.byref(f)))
    return int(f.value)


def fa_destroy(ctx: ArchiveContext) -> None:
    ctx.close()


# Paged cache of quantised keys and values (include/qcache.h).

class CacheContext(Context):
    """Owns a ``qc_ctx*`` and knows its geometry; frees it with ``qc_destroy``."""

    _destroy = "qc_destroy"

    def __init__(self, handle: int, fmt: str, d: int, n_heads: int, page_tokens: int, device: int):
        super().__init__(handle)
        self.fmt, self.d, self.n_heads, self.page_tokens, self.device = fmt, d, n_heads, page_tokens, device


# A decoding step calls these once per layer, so that their checks count: each call states what it wants of its
# tensors in one expression, and only when that fails does `_refuse` look for what to say.

_QC_TYPES, _F32, _I32, _I64, _U8 = {}, None, None, None, None
_raw_stream = None
_NO_STRIDES = (0, 0, 1)


def _qc_init() -> None:
    """Element types and the current stream's getter, once torch is there."""
    global _F32, _I32, _I64, _U8, _raw_stream
    import torch
    _QC_TYPES.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    _F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _refuse(ctx: CacheContext, **what):
    """Says what is wrong with the tensors `what`: name -> (tensor, element type or None, shape, contiguous). A shape's
    None is any size."""
    for name, (t, dtype, shape, flat) in what.items():
        if t is None:
            continue
        if t.device.type != "cuda" or t.device.index != ctx.device:
            raise ValueError(f"{name} is on {t.device}, the context on cuda:{ctx.device}")
        if (t.dtype not in _QC_TYPES) if dtype is None else (t.dtype != dtype):
            raise TypeError(f"{name} is {t.dtype}, not {dtype or 'float16, bfloat16 or float32'}")
        if len(shape) != t.dim() or any(w is not None and w != g for w, g in zip(shape, t.shape)):
            raise ValueError(f"{name} is {tuple(t.shape)}, not {shape}")
        if flat and not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")
        if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name}: the elements of a row are not next to each other")
    raise ValueError("the arguments do not go together")


def qc_create(fmt: str, d: int, n_heads: int, page_tokens: int, device: int = 0) -> CacheContext:
    """fmt: "int8", "e4m3" or "e2m1"."""
    if fmt not in QC_FORMATS:
        raise ValueError(f"fmt is one of {sorted(QC_FORMATS)}, not {fmt!r}")
    h = _c_void_p()
    _check("qc_create", lib().qc_create(ctypes.byref(h), QC_FORMATS[fmt], int(d), int(n_heads), int(page_tokens), int(device)))
    if _raw_stream is None:
        _qc_init()
    ctx = CacheContext(h.value, fmt, int(d), int(n_heads), int(page_tokens), int(device))
    ctx.page_bytes = qc_page_bytes(ctx)
    return ctx


def qc_page_bytes(ctx: CacheContext) -> int:
    b = lib().qc_page_bytes(ctx)
    if b < 0:
        raise FQError("qc_page_bytes", FQ_EINVAL)
    return int(b)


def qc_norm_rope_axes(ctx: CacheContext, q, k, w_q, w_k, eps: float, pos, table, sections, interleaved: bool, q_out, k_out,
                      stream=None) -> None:
    """As qc_norm_rope; sections: how many pairs each axis turns; pos int64 [axes, n]; table float32 [max_pos, 2 sum(sections)]."""
    qc_norm_rope(ctx, q, k, w_q, w_k, eps, pos, table, 2 * sum(sections), interleaved, q_out, k_out, stream, (_int * len(sections))(*sections))


def qc_norm_rope(ctx: CacheContext, q, k, w_q, w_k, eps: float, pos, table, rot: int, interleaved: bool, q_out, k_out,
                 stream=None, _sections=None) -> None:
    """q [n, hq, d] and k [n, hk, d] (either may be None), strided; w_q, w_k float32 [d] or None; pos int64
    [n]; table float32 [max_pos, rot]; q_out, k_out like q and k (themselves, too)."""
    dev, d, sections = ctx.device, ctx.d, _sections
    ok, n, dtype = True, None, None
    if q is not None:
        qs, q0, o0 = q.shape, q.stride(), q_out.stride()
        n, dtype = qs[0], q.dtype
        ok = (len(qs) == 3 and qs[2] == d and q_out.dtype is dtype and q_out.shape == qs and q0[2] == 1 and o0[2] == 1
              and q.get_device() == dev and q_out.get_device() == dev
              and (w_q is None or (w_q.dtype is _F32 and w_q.shape == (d,) and w_q.get_device() == dev and w_q.is_contiguous())))
    if k is not None and ok:
        ks, k0, o1 = k.shape, k.stride(), k_out.stride()
        if q is None:
            n, dtype = ks[0], k.dtype
        ok = (len(ks) == 3 and ks[0] == n and ks[2] == d and k.dtype is dtype and k_out.dtype is dtype and k_out.shape == ks
              and k0[2] == 1 and o1[2] == 1 and k.get_device() == dev and k_out.get_device() == dev
              and (w_k is None or (w_k.dtype is _F32 and w_k.shape == (d,) and w_k.get_device() == dev and w_k.is_contiguous())))
    if n is None:
        raise ValueError("neither q nor k")
    if ok and rot:
        most = table.shape[0]
        ok = (pos.dtype is _I64 and pos.shape == ((n,) if sections is None else (len(sections), n)) and pos.get_device() == dev
              and pos.is_contiguous() and table.dtype is _F32 and table.shape == (most, rot) and table.get_device() == dev
              and table.is_contiguous())
    kind = _QC_TYPES.get(dtype)
    if not ok or kind is None:
        rows = {}
        for name, x, out, w in (("q", q, q_out, w_q), ("k", k, k_out, w_k)):
            if x is not None:
                heads = x.shape[1] if x.dim() > 1 else None
                rows.update({name: (x, None if name == "q" else dtype, (n, heads, d), False), name + "_out": (out, dtype, (n, heads, d), False),
                             "w_" + name: (w, _F32, (d,), True)})
        if rot:
            rows.update(pos=(pos, _I64, (n,) if sections is None else (len(sections), n), True), table=(table, _F32, (None, rot), True))
        _refuse(ctx, **rows)
    if q is None:
        q_in, q_to, hq, wq, q0, o0 = None, None, 0, None, _NO_STRIDES, _NO_STRIDES
    else:
        q_in, q_to, hq, wq = q.data_ptr(), q_out.data_ptr(), qs[1], None if w_q is None else w_q.data_ptr()
    if k is None:
        k_in, k_to, hk, wk, k0, o1 = None, None, 0, None, _NO_STRIDES, _NO_STRIDES
    else:
        k_in, k_to, hk, wk = k.data_ptr(), k_out.data_ptr(), ks[1], None if w_k is None else w_k.data_ptr()
    if rot:
        at, turns = pos.data_ptr(), table.data_ptr()
    else:
        at = turns = None
        most = 0
    at_stream = _raw_stream(dev) if stream is None else _stream(stream)
    if sections is None:
        rc = _lib.qc_norm_rope(ctx.handle, kind, n, q_in, hq, q0[0], q0[1], wq, k_in, hk, k0[0], k0[1], wk, eps, at, turns, most, rot, interleaved,
                               q_to, o0[0], o0[1], k_to, o1[0], o1[1], at_stream)
    else:
        rc = _lib.qc_norm_rope_axes(ctx.handle, kind, n, q_in, hq, q0[0], q0[1], wq, k_in, hk, k0[0], k0[1], wk, eps, at, turns, most, sections,
                                    len(sections), interleaved, q_to, o0[0], o0[1], k_to, o1[0], o1[1], at_stream)
    if rc:
        raise FQError("qc_norm_rope" if sections is None else "qc_norm_rope_axes", rc)


def qc_plan(ctx: CacheContext, lens, news, free_pages, taken, table, starts, slots, pos, taken_out, held=None, held_out=None,
            stream=None) -> None:
    """lens, news int32 [n_seq]; free_pages int32 [n_free]; taken, taken_out int64 [1]; table int32 [n_seq, width], whose
    rows may be part of wider ones; starts int32 [n_seq + 1]; slots, pos int64 [n_tokens]; held, held_out int32 [n_seq] or None."""
    dev, n_seq, n_free, n = ctx.device, lens.shape[0], free_pages.shape[0], slots.shape[0]
    st, width = table.stride(), table.shape[-1]

    def flat(t, dtype, size):
        return t.dtype is dtype and t.shape == (size,) and t.get_device() == dev and t.is_contiguous()

    if not (flat(lens, _I32, n_seq) and flat(news, _I32, n_seq) and flat(free_pages, _I32, n_free) and flat(taken, _I64, 1)
            and flat(taken_out, _I64, 1) and flat(starts, _I32, n_seq + 1) and flat(slots, _I64, n) and flat(pos, _I64, n)
            and table.dtype is _I32 and table.shape == (n_seq, width) and (st[1] == 1 or width == 1) and table.get_device() == dev
            and (st[0] >= width or n_seq <= 1) and (held is None or flat(held, _I32, n_seq)) and (held_out is None or flat(held_out, _I32, n_seq))):
        _refuse(ctx, lens=(lens, _I32, (n_seq,), True), news=(news, _I32, (n_seq,), True), free_pages=(free_pages, _I32, (n_free,), True),
                taken=(taken, _I64, (1,), True), table=(table, _I32, (n_seq, None), False), starts=(starts, _I32, (n_seq + 1,), True),
                slots=(slots, _I64, (n,), True), pos=(pos, _I64, (n,), True), taken_out=(taken_out, _I64, (1,), True),
                held=(held, _I32, (n_seq,), True), held_out=(held_out, _I32, (n_seq,), True))
    rc = _lib.qc_plan(ctx.handle, n_seq, lens.data_ptr(), news.data_ptr(), free_pages.data_ptr(), n_free, taken.data_ptr(),
                      table.data_ptr(), max(st[0], width), width, starts.data_ptr(), n, slots.data_ptr(), pos.data_ptr(),
                      taken_out.data_ptr(), None if held is None else held.data_ptr(), None if held_out is None else held_out.data_ptr(),
                      _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_plan", rc)


def qc_write(ctx: CacheContext, k, v, slots, pages, stream=None) -> None:
    """k, v [n, n_heads, d], strided; slots int64 [n]; pages uint8 [n_pages, qc_page_bytes(ctx)]."""
    dev, shape, dtype = ctx.device, k.shape, k.dtype
    n, n_pages, sk, sv = shape[0], pages.shape[0], k.stride(), v.stride()
    if not (dtype in _QC_TYPES and v.dtype is dtype and shape == (n, ctx.n_heads, ctx.d) and v.shape == shape and sk[2] == 1 and sv[2] == 1
            and k.get_device() == dev and v.get_device() == dev
            and slots.dtype is _I64 and slots.shape == (n,) and slots.get_device() == dev and slots.is_contiguous()
            and pages.dtype is _U8 and pages.shape == (n_pages, ctx.page_bytes) and pages.get_device() == dev and pages.is_contiguous()):
        _refuse(ctx, k=(k, None, (n, ctx.n_heads, ctx.d), False), v=(v, dtype, (n, ctx.n_heads, ctx.d), False),
                slots=(slots, _I64, (n,), True), pages=(pages, _U8, (None, ctx.page_bytes), True))
    rc = _lib.qc_write(ctx.handle, _QC_TYPES[dtype], n, k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0], sv[1], slots.data_ptr(),
                       pages.data_ptr(), n_pages, _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_write", rc)


def qc_read(ctx: CacheContext, pages, slots, k_out, v_out, stream=None) -> None:
    """slots int64 [n]; k_out, v_out [n, n_heads, d], contiguous, or None."""
    dev, n, n_pages = ctx.device, slots.shape[0], pages.shape[0]
    out = k_out if k_out is not None else v_out
    if out is None:
        return
    dtype, shape = out.dtype, (n, ctx.n_heads, ctx.d)
    if not (dtype in _QC_TYPES
            and (k_out is None or (k_out.dtype is dtype and k_out.shape == shape and k_out.get_device() == dev and k_out.is_contiguous()))
            and (v_out is None or (v_out.dtype is dtype and v_out.shape == shape and v_out.get_device() == dev and v_out.is_contiguous()))
            and slots.dtype is _I64 and slots.shape == (n,) and slots.get_device() == dev and slots.is_contiguous()
            and pages.dtype is _U8 and pages.shape == (n_pages, ctx.page_bytes) and pages.get_device() == dev and pages.is_contiguous()):
        _refuse(ctx, slots=(slots, _I64, (n,), True), pages=(pages, _U8, (None, ctx.page_bytes), True),
                k_out=(k_out, None, shape, True), v_out=(v_out, dtype, shape, True))
    rc = _lib.qc_read(ctx.handle, _QC_TYPES[dtype], n, slots.data_ptr(), pages.data_ptr(), n_pages,
                      None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(),
                      _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_read", rc)


def qc_attend(ctx: CacheContext, pages, q, table, lens, nodes, tree, scale: float, max_len: int, out, lse, workspace,
              stream=None) -> None:
    """q [n_seq, n_nodes, n_q_heads, d], strided; table int32 [n_seq, >= places / page_tokens]; lens, nodes int32
    [n_seq] (nodes may be None); tree int32 [n_seq, n_nodes, ceil(n_nodes / 32)] or None; out like q,
    contiguous; lse float32 [n_seq, n_nodes, n_q_heads] or None; workspace from alloc_attend_workspace."""
    dev, d, shape, dtype = ctx.device, ctx.d, q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError(f"q is {tuple(shape)}, not [n_seq, n_nodes, n_q_heads, {d}]")
    n_seq, n_nodes, hq, _ = shape
    n_pages, sq, st, width = pages.shape[0], q.stride(), table.stride(), table.shape[-1]
    if not (shape[3] == d and sq[3] == 1 and q.get_device() == dev and dtype in _QC_TYPES
            and out.dtype is dtype and out.shape == shape and out.get_device() == dev and out.is_contiguous()
            and table.dtype is _I32 and table.shape == (n_seq, width) and (st[1] == 1 or width == 1) and table.get_device() == dev
            and lens.dtype is _I32 and lens.shape == (n_seq,) and lens.get_device() == dev and lens.is_contiguous()
            and (nodes is None
                 or (nodes.dtype is _I32 and nodes.shape == (n_seq,) and nodes.get_device() == dev and nodes.is_contiguous()))
            and (tree is None or (tree.dtype is _I32 and tree.shape == (n_seq, n_nodes, (n_nodes + 31) // 32) and tree.get_device() == dev
                                  and tree.is_contiguous()))
            and (lse is None
                 or (lse.dtype is _F32 and lse.shape == (n_seq, n_nodes, hq) and lse.get_device() == dev and lse.is_contiguous()))
            and pages.dtype is _U8 and pages.shape == (n_pages, ctx.page_bytes) and pages.get_device() == dev and pages.is_contiguous()
            and workspace.dtype is _U8 and workspace.get_device() == dev and workspace.is_contiguous()):
        _refuse(ctx, q=(q, None, (n_seq, n_nodes, hq, d), False), out=(out, dtype, (n_seq, n_nodes, hq, d), True),
                table=(table, _I32, (n_seq, None), False), lens=(lens, _I32, (n_seq,), True), nodes=(nodes, _I32, (n_seq,), True),
                tree=(tree, _I32, (n_seq, n_nodes, (n_nodes + 31) // 32), True), lse=(lse, _F32, (n_seq, n_nodes, hq), True),
                pages=(pages, _U8, (None, ctx.page_bytes), True), workspace=(workspace, _U8, (None,), True))
    if -(-(max_len + n_nodes) // ctx.page_tokens) > width:       # a row's width, which its stride may exceed
        raise FQError("qc_attend", FQ_EINVAL)
    rc = _lib.qc_attend(ctx.handle, _QC_TYPES[dtype], n_seq, n_nodes, hq, q.data_ptr(), sq[0], sq[1], sq[2], table.data_ptr(),
                        st[0] if n_seq > 1 else max(st[0], width), lens.data_ptr(), None if nodes is None else nodes.data_ptr(),
                        None if tree is None else tree.data_ptr(), pages.data_ptr(), n_pages, scale, max_len, out.data_ptr(),
                        None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                        _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_attend", rc)


def qc_attend_workspace(ctx: CacheContext, n_seq: int, n_nodes: int, n_q_heads: int, max_len: int) -> int:
    b = lib().qc_attend_workspace(ctx, int(n_seq), int(n_nodes), int(n_q_heads), int(max_len))
    if b < 0:
        raise FQError("qc_attend_workspace", FQ_EINVAL)
    return int(b)


def qc_attend_chunk(ctx: CacheContext, pages, q, starts, table, lens, prefix, slopes, scale: float, cap: float, window: int,
                    max_len: int, max_new: int, out, lse, workspace, stream=None) -> None:
    """q [n_tokens, n_q_heads, d], strided: the new tokens of all sequences, one sequence after another; starts int32
    [n_seq + 1]; table int32 [n_seq, >= (max_len + max_new) / page_tokens]; lens int32 [n_seq]; prefix int32 [n_seq] or
    None; slopes float32 [n_q_heads] or None; cap, window: 0 for none; out like q, contiguous; lse float32 [n_tokens,
    n_q_heads] or None; workspace from alloc_chunk_workspace. (Single tokens without masks, cap or bias: qc_attend is faster.)"""
    dev, d, shape, dtype = ctx.device, ctx.d, q.shape, q.dtype
    if len(shape) != 3:
        raise ValueError(f"q is {tuple(shape)}, not [n_tokens, n_q_heads, {d}]")
    n, hq, _ = shape
    n_seq, n_pages, sq, st, width = lens.shape[0], pages.shape[0], q.stride(), table.stride(), table.shape[-1]
    if not (shape[2] == d and sq[2] == 1 and q.get_device() == dev and dtype in _QC_TYPES
            and out.dtype is dtype and out.shape == shape and out.get_device() == dev and out.is_contiguous()
            and starts.dtype is _I32 and starts.shape == (n_seq + 1,) and starts.get_device() == dev and starts.is_contiguous()
            and table.dtype is _I32 and table.shape == (n_seq, width) and (st[1] == 1 or width == 1) and table.get_device() == dev
            and lens.dtype is _I32 and lens.shape == (n_seq,) and lens.get_device() == dev and lens.is_contiguous()
            and (prefix is None
                 or (prefix.dtype is _I32 and prefix.shape == (n_seq,) and prefix.get_device() == dev and prefix.is_contiguous()))
            and (slopes is None
                 or (slopes.dtype is _F32 and slopes.shape == (hq,) and slopes.get_device() == dev and slopes.is_contiguous()))
            and (lse is None or (lse.dtype is _F32 and lse.shape == (n, hq) and lse.get_device() == dev and lse.is_contiguous()))
            and pages.dtype is _U8 and pages.shape == (n_pages, ctx.page_bytes) and pages.get_device() == dev and pages.is_contiguous()
            and workspace.dtype is _U8 and workspace.get_device() == dev and workspace.is_contiguous()):
        _refuse(ctx, q=(q, None, (n, hq, d), False), out=(out, dtype, (n, hq, d), True), starts=(starts, _I32, (n_seq + 1,), True),
                table=(table, _I32, (n_seq, None), False), lens=(lens, _I32, (n_seq,), True), prefix=(prefix, _I32, (n_seq,), True),
                slopes=(slopes, _F32, (hq,), True), lse=(lse, _F32, (n, hq), True), pages=(pages, _U8, (None, ctx.page_bytes), True),
                workspace=(workspace, _U8, (None,), True))
    if -(-(max_len + max_new) // ctx.page_tokens) > width:       # a row's width, which its stride may exceed
        raise FQError("qc_attend_chunk", FQ_EINVAL)
    rc = _lib.qc_attend_chunk(ctx.handle, _QC_TYPES[dtype], n_seq, n, hq, q.data_ptr(), sq[0], sq[1], starts.data_ptr(), table.data_ptr(),
                              st[0] if n_seq > 1 else max(st[0], width), lens.data_ptr(), None if prefix is None else prefix.data_ptr(),
                              None if slopes is None else slopes.data_ptr(), pages.data_ptr(), n_pages, scale, cap, window, max_len,
                              max_new, out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_attend_chunk", rc)


def qc_attend_chunk_workspace(ctx: CacheContext, n_seq: int, n_tokens: int, n_q_heads: int, max_len: int, max_new: int) -> int:
    b = lib().qc_attend_chunk_workspace(ctx, int(n_seq), int(n_tokens), int(n_q_heads), int(max_len), int(max_new))
    if b < 0:
        raise FQError("qc_attend_chunk_workspace", FQ_EINVAL)
    return int(b)


def qc_verify(ctx: CacheContext, p, q, tokens, parents, nodes, u, path, out, accepted, stream=None) -> None:
    """p [n_seq, n_nodes + 1, vocab] and q [n_seq, n_nodes, vocab], strided, float32, float16 or bfloat16; tokens, parents int32
    [n_seq, n_nodes] (parents may be None: a chain); nodes int32 [n_seq] or None; u float32 [n_seq, n_nodes + 1]; path
    int32 [n_seq, n_nodes]; out int32 [n_seq, n_nodes + 1]; accepted int32 [n_seq]."""
    dev, shape, dtype = ctx.device, q.shape, q.dtype
    if len(shape) != 3 or p.dim() != 3:
        raise ValueError(f"p is {tuple(p.shape)} and q {tuple(shape)}, not [n_seq, n_nodes + 1, vocab] and [n_seq, n_nodes, vocab]")
    n_seq, t, vocab = shape
    sp, sq = p.stride(), q.stride()

    def flat(x, kind, *size):
        return x.dtype is kind and x.shape == size and x.get_device() == dev and x.is_contiguous()

    if not (dtype in _QC_TYPES and p.dtype is dtype and p.shape == (n_seq, t + 1, vocab) and p.get_device() == dev and q.get_device() == dev
            and (vocab <= 1 or (sp[2] == 1 and sq[2] == 1)) and flat(tokens, _I32, n_seq, t) and (parents is None or flat(parents, _I32, n_seq, t))
            and (nodes is None or flat(nodes, _I32, n_seq)) and flat(u, _F32, n_seq, t + 1) and flat(path, _I32, n_seq, t)
            and flat(out, _I32, n_seq, t + 1) and flat(accepted, _I32, n_seq)):
        _refuse(ctx, p=(p, None, (n_seq, t + 1, vocab), False), q=(q, p.dtype, (n_seq, t, vocab), False), tokens=(tokens, _I32, (n_seq, t), True),
                parents=(parents, _I32, (n_seq, t), True), nodes=(nodes, _I32, (n_seq,), True), u=(u, _F32, (n_seq, t + 1), True),
                path=(path, _I32, (n_seq, t), True), out=(out, _I32, (n_seq, t + 1), True), accepted=(accepted, _I32, (n_seq,), True))
    rc = _lib.qc_verify(ctx.handle, _QC_TYPES[dtype], n_seq, t, vocab, p.data_ptr(), sp[0], sp[1], q.data_ptr(), sq[0], sq[1], tokens.data_ptr(),
                        None if parents is None else parents.data_ptr(), None if nodes is None else nodes.data_ptr(), u.data_ptr(),
                        path.data_ptr(), out.data_ptr(), accepted.data_ptr(), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        raise FQError("qc_verify", rc)


def qc_status(ctx: CacheContext, stream=None) -> int:
    f = ctypes.c_uint32()
    _check("qc_status", lib().qc_status(ctx, _stream(stream), ctypes.byref(f)))
    return int(f.value)


def qc_destroy(ctx: CacheContext) -> None:
    ctx.close()
