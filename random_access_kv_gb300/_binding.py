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
QC_FLAG_RANGE, QC_FLAG_NONFINITE, QC_FLAG_TIMEOUT = 1, 2, 4


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
        self._as_parameter_cached = ctypes.c_void_p(handle)

    @property
    def _as_parameter_(self):
        return self._as_parameter_cached

    def close(self) -> None:
        super().close()
        self._as_parameter_cached = ctypes.c_void_p(0)


_qc_types = {}


def _qc_type(t) -> int:
    """QC_* code of a tensor's element type."""
    if not _qc_types:
        import torch
        _qc_types.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2})
    code = _qc_types.get(t.dtype)
    if code is None:
        raise TypeError(f"rows are float16, bfloat16 or float32, not {t.dtype}")
    return code


def _want(t, what: str, ctx: CacheContext, dtype=None, shape=None) -> None:
    """Refuses what the C call could not see: another device, type or shape, an inner stride, too few rows."""
    if t.device.index != ctx.device or t.device.type != "cuda":
        raise ValueError(f"{what} is on {t.device}, the context on cuda:{ctx.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} is {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what} is {tuple(t.shape)}, not {shape}")


def _want_flat(t, what: str, ctx: CacheContext, dtype, shape=None) -> None:
    _want(t, what, ctx, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{what} is not contiguous")


def _want_heads(t, what: str, ctx: CacheContext, dtype, n: int | None = None, heads: int | None = None) -> None:
    _want(t, what, ctx, dtype)
    s = t.shape
    if len(s) != 3 or s[2] != ctx.d or (n is not None and s[0] != n) or (heads is not None and s[1] != heads):
        raise ValueError(f"{what} is {tuple(s)}, not [{'n' if n is None else n}, {'heads' if heads is None else heads}, {ctx.d}]")
    if t.stride(2) != 1:
        raise ValueError(f"{what}: the elements of a row are not next to each other")


def _want_pages(pages, ctx: CacheContext) -> int:
    import torch
    _want_flat(pages, "pages", ctx, torch.uint8)
    if pages.dim() != 2 or pages.shape[1] != qc_page_bytes(ctx):
        raise ValueError(f"pages is {tuple(pages.shape)}, not [n_pages, {qc_page_bytes(ctx)}]")
    return pages.shape[0]


def qc_create(fmt: str, d: int, n_heads: int, page_tokens: int, device: int = 0) -> CacheContext:
    """fmt: "int8", "e4m3" or "e2m1"."""
    if fmt not in QC_FORMATS:
        raise ValueError(f"fmt is one of {sorted(QC_FORMATS)}, not {fmt!r}")
    h = _c_void_p()
    _check("qc_create", lib().qc_create(ctypes.byref(h), QC_FORMATS[fmt], int(d), int(n_heads), int(page_tokens), int(device)))
    return CacheContext(h.value, fmt, int(d), int(n_heads), int(page_tokens), int(device))


def qc_page_bytes(ctx: CacheContext) -> int:
    b = lib().qc_page_bytes(ctx)
    if b < 0:
        raise FQError("qc_page_bytes", FQ_EINVAL)
    return int(b)


def qc_norm_rope(ctx: CacheContext, q, k, w_q, w_k, eps: float, pos, table, rot: int, interleaved: bool, q_out, k_out,
                 stream=None) -> None:
    """q [n, hq, d] and k [n, hk, d] (either may be None), strided; w_q, w_k float32 [d] or None; pos int64
    [n]; table float32 [max_pos, rot]; q_out, k_out like q and k (themselves, too)."""
    import torch
    args, n, dtype, max_pos = [], None, None, 0
    for x, out, w, name in ((q, q_out, w_q, "q"), (k, k_out, w_k, "k")):
        if x is None:
            args.append((None, 0, 0, 0, None, None, 0, 0))
            continue
        dtype = x.dtype if dtype is None else dtype
        _want_heads(x, name, ctx, dtype, n)
        n = x.shape[0]
        _want_heads(out, name + "_out", ctx, dtype, n, x.shape[1])
        if w is not None:
            _want_flat(w, "w_" + name, ctx, torch.float32, (ctx.d,))
        args.append((_ptr(x), x.shape[1], x.stride(0), x.stride(1), _ptr(w), _ptr(out), out.stride(0), out.stride(1)))
    if n is None:
        raise ValueError("neither q nor k")
    if rot:
        _want_flat(pos, "pos", ctx, torch.int64, (n,))
        _want_flat(table, "table", ctx, torch.float32, (table.shape[0], rot))
        max_pos = table.shape[0]
    a, b = args
    _check("qc_norm_rope", lib().qc_norm_rope(ctx, _qc_type(q if q is not None else k), n, *a[:5], *b[:5], eps,
                                              _ptr(pos) if rot else None, _ptr(table) if rot else None, max_pos, rot,
                                              interleaved, *a[5:], *b[5:], _stream(stream)))


def qc_write(ctx: CacheContext, k, v, slots, pages, stream=None) -> None:
    """k, v [n, n_heads, d], strided; slots int64 [n]; pages uint8 [n_pages, qc_page_bytes(ctx)]."""
    import torch
    n = k.shape[0]
    _want_heads(k, "k", ctx, k.dtype, n, ctx.n_heads)
    _want_heads(v, "v", ctx, k.dtype, n, ctx.n_heads)
    _want_flat(slots, "slots", ctx, torch.int64, (n,))
    n_pages = _want_pages(pages, ctx)
    _check("qc_write", lib().qc_write(ctx, _qc_type(k), n, _ptr(k), k.stride(0), k.stride(1), _ptr(v), v.stride(0),
                                      v.stride(1), _ptr(slots), _ptr(pages), n_pages, _stream(stream)))


def qc_read(ctx: CacheContext, pages, slots, k_out, v_out, stream=None) -> None:
    """slots int64 [n]; k_out, v_out [n, n_heads, d], contiguous, or None."""
    import torch
    n, n_pages = slots.shape[0], _want_pages(pages, ctx)
    _want_flat(slots, "slots", ctx, torch.int64, (n,))
    out = k_out if k_out is not None else v_out
    if out is None:
        return
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            _want_flat(t, name, ctx, out.dtype, (n, ctx.n_heads, ctx.d))
    _check("qc_read", lib().qc_read(ctx, _qc_type(out), n, _ptr(slots), _ptr(pages), n_pages, _ptr(k_out), _ptr(v_out),
                                    _stream(stream)))


def qc_attend(ctx: CacheContext, pages, q, table, lens, nodes, tree, scale: float, max_len: int, out, lse, workspace,
              stream=None) -> None:
    """q [n_seq, n_nodes, n_q_heads, d], strided; table int32 [n_seq, >= places / page_tokens]; lens, nodes int32
    [n_seq] (nodes may be None); tree int32 [n_seq, n_nodes, ceil(n_nodes / 32)] or None; out like q,
    contiguous; lse float32 [n_seq, n_nodes, n_q_heads] or None; workspace from alloc_attend_workspace."""
    import torch
    if q.dim() != 4 or q.shape[3] != ctx.d or q.stride(3) != 1:
        raise ValueError(f"q is {tuple(q.shape)}, not [n_seq, n_nodes, n_q_heads, {ctx.d}] with its rows' elements together")
    n_seq, n_nodes, hq, _ = q.shape
    n_pages = _want_pages(pages, ctx)
    _want(q, "q", ctx)
    _want_flat(out, "out", ctx, q.dtype, (n_seq, n_nodes, hq, ctx.d))
    _want(table, "table", ctx, torch.int32)
    if table.dim() != 2 or table.shape[0] != n_seq or (table.stride(1) != 1 and table.shape[1] > 1):
        raise ValueError(f"table is {tuple(table.shape)}, not [{n_seq}, pages per sequence] with rows of their own")
    if -(-(max_len + n_nodes) // ctx.page_tokens) > table.shape[1]:
        raise FQError("qc_attend", FQ_EINVAL)
    _want_flat(lens, "lens", ctx, torch.int32, (n_seq,))
    if nodes is not None:
        _want_flat(nodes, "nodes", ctx, torch.int32, (n_seq,))
    if tree is not None:
        _want_flat(tree, "tree", ctx, torch.int32, (n_seq, n_nodes, (n_nodes + 31) // 32))
    if lse is not None:
        _want_flat(lse, "lse", ctx, torch.float32, (n_seq, n_nodes, hq))
    _want_flat(workspace, "workspace", ctx, torch.uint8)
    _check("qc_attend", lib().qc_attend(ctx, _qc_type(q), n_seq, n_nodes, hq, _ptr(q), q.stride(0), q.stride(1), q.stride(2),
                                        _ptr(table), table.stride(0), _ptr(lens), _ptr(nodes), _ptr(tree), _ptr(pages),
                                        n_pages, scale, max_len, _ptr(out), _ptr(lse), _ptr(workspace),
                                        workspace.numel(), _stream(stream)))


def qc_attend_workspace(ctx: CacheContext, n_seq: int, n_nodes: int, n_q_heads: int, max_len: int) -> int:
    b = lib().qc_attend_workspace(ctx, int(n_seq), int(n_nodes), int(n_q_heads), int(max_len))
    if b < 0:
        raise FQError("qc_attend_workspace", FQ_EINVAL)
    return int(b)


def qc_status(ctx: CacheContext, stream=None) -> int:
    f = ctypes.c_uint32()
    _check("qc_status", lib().qc_status(ctx, _stream(stream), ctypes.byref(f)))
    return int(f.value)


def qc_destroy(ctx: CacheContext) -> None:
    ctx.close()
