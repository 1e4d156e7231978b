"""Binding of the paged-attention entry points: the full-attention layers that
stand between a hybrid model's GDN layers.

Argument marshalling only, as in the package's other calls: dtypes, devices,
shapes and strides are checked here, then the C ABI of ``include/gdn.h`` runs on
the current torch stream (or the one given).  One cache is k_pages and v_pages
[N][H_kv][page_size][d] (bf16 or float8_e4m3fn) with page_table [R][width],
kv_len [R] and, for its bookkeeping, refs [N], all int32 on the same GPU.
"""
from __future__ import annotations

import ctypes
import math

from . import GdnError, _check, _contig, _dev, _device, _on, _ptr, _stream, _torch, lib

EXPORTS = ("gdn_rope_freqs", "attn_prologue", "attn_paged", "attn_paged_workspace_bytes", "kv_page_workspace_bytes",
           "kv_page_reserve", "kv_page_fork", "kv_page_free", "kv_page_copy", "kv_page_compact")
ROPE_STRETCH = {"none": 0, "linear": 1, "base": 2, "wavelength": 3}

_P, _i32, _i64, _f32, _f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double


class AttnDims(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("B", "T", "R", "H_q", "H_kv", "d", "N", "page_size", "table_width", "max_new",
                                    "window", "cache_type")]


class Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("row_stride", _i64), ("head_stride", _i64)]


class KvCache(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "k_scale", "v_scale", "page_table", "kv_len")]


class Rope(ctypes.Structure):
    _fields_ = [("freqs", _P), ("rot", _i32), ("interleaved", _i32), ("scale", _f32)]


class QkNorm(ctypes.Structure):
    _fields_ = [("q_weight", _P), ("k_weight", _P), ("eps", _f32), ("add", _f32)]


class Pages(ctypes.Structure):
    _fields_ = ([(n, _i32) for n in ("R", "table_width", "N", "page_size")] +
                [(n, _P) for n in ("page_table", "kv_len", "refs", "k", "v")] +
                [("layers", _i32), ("reserved", _i32), ("layer_stride", _i64), ("page_bytes", _i64)])


def declare(L) -> None:
    """Argument types of this module's entry points."""
    D, H, C, G = (ctypes.POINTER(t) for t in (AttnDims, Heads, KvCache, Pages))
    size = ctypes.c_size_t
    for name, args, res in (
            ("gdn_rope_freqs", [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _P], _i32),
            ("attn_prologue", [D, H, H, H, H, C, _P, _P, _P, ctypes.POINTER(Rope), ctypes.POINTER(QkNorm), _P], _i32),
            ("attn_paged", [D, H, C, _P, _P, H, _P, _f32, _P, size, _P], _i32),
            ("attn_paged_workspace_bytes", [D], size),
            ("kv_page_workspace_bytes", [_i32, _i32, _i32], size),
            ("kv_page_reserve", [G, _P, _P, _i32, _P, _P, size, _P], _i32),
            ("kv_page_fork", [G, _P, _P, _i32, _P, _P, size, _P], _i32),
            ("kv_page_free", [G, _P, _i32, _P], _i32),
            ("kv_page_copy", [G, _P, _P, _i32, _P], _i32),
            ("kv_page_compact", [G, _P, _P, _P, size, _P], _i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# ------------------------------------------------------------------ checks

def _cache_type(k_pages, v_pages):
    torch = _torch()
    if k_pages.dtype != v_pages.dtype or k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"k_pages and v_pages must both be bfloat16 or float8_e4m3fn, got {k_pages.dtype}, "
                         f"{v_pages.dtype}")
    return int(k_pages.dtype == torch.float8_e4m3fn)


def _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale):
    """Shape checks of a layer's cache (any device); returns N, H_kv, page_size, d, R, width, cache_type."""
    kind = _cache_type(k_pages, v_pages)
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must both be [N][H_kv][page_size][d]")
    N, H_kv, page, d = shape
    R = kv_len.shape[0] if kv_len.dim() == 1 else -1
    width = 1
    if page_table is not None:
        if page_table.dim() != 2 or page_table.shape[0] != R:
            raise ValueError("page_table must be [R][width] and kv_len [R]")
        width = page_table.shape[1]
    elif R < 0:
        raise ValueError("kv_len must be [R]")
    if kind:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None or tuple(t.shape) != (H_kv,):
                raise ValueError(f"{n} [H_kv] is required for an e4m3 cache")
    return N, H_kv, page, d, R, width, kind


def _packed_layout(row, cu_seqlens):
    if row.dim() != 1 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] != row.shape[0] + 1:
        raise ValueError("row must be [B] and cu_seqlens [B+1]")
    return row.shape[0]


def _heads_layout(t, name, T, H, d):
    """[T][H][d] with contiguous d; returns H."""
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != d or (H is not None and t.shape[1] != H):
        raise ValueError(f"{name} must be [{T}][{'H' if H is None else H}][{d}], got {list(t.shape)}")
    if t.stride(2) != 1 and d > 1:
        raise ValueError(f"{name}: the head's values must be contiguous")
    return t.shape[1]


def _heads(t):
    return Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _ints(t, name):
    return _contig(_dev(t, name, _torch().int32), name)


def _check_cache_tensors(k_pages, v_pages, page_table, kv_len, k_scale, v_scale):
    torch = _torch()
    _contig(_dev(k_pages, "k_pages", k_pages.dtype), "k_pages")
    _contig(_dev(v_pages, "v_pages", v_pages.dtype), "v_pages")
    if page_table is not None:
        _ints(page_table, "page_table")
    _ints(kv_len, "kv_len")
    _contig(_dev(k_scale, "k_scale", torch.float32, allow_none=True), "k_scale")
    _contig(_dev(v_scale, "v_scale", torch.float32, allow_none=True), "v_scale")


# ------------------------------------------------------------------ entry points

def rope_freqs(rot: int, base: float = 10000.0, *, stretch: str = "none", factor: float = 1.0, original: float = 0.0,
               low: float = 1.0, high: float = 32.0, device="cuda"):
    """The rotary frequencies, [rot/2] float64 radians a position on `device` (see ``gdn_rope_freqs`` in
    include/gdn.h).  stretch: "none", "linear", "base" or "wavelength"."""
    if stretch not in ROPE_STRETCH:
        raise ValueError(f"unknown stretch {stretch!r}: one of {sorted(ROPE_STRETCH)}")
    out = (ctypes.c_double * max(1, rot // 2))()
    _check("gdn_rope_freqs", lib().gdn_rope_freqs(rot, base, ROPE_STRETCH[stretch], factor, original, low, high, out))
    return _torch().tensor(list(out)[:rot // 2], dtype=_torch().float64, device=device)


def attn_prologue(q, k, v, q_out, k_pages, v_pages, page_table, kv_len, row, cu_seqlens, freqs, *,
                  interleaved: bool = False, rope_scale: float = 1.0, q_norm=None, k_norm=None,
                  norm_eps: float = 1e-6, norm_add: float = 0.0, positions=None, k_scale=None, v_scale=None,
                  stream=None) -> None:
    """q/k RMS norm, rotary positions and the write of the new tokens' k and v into their pages (see
    ``attn_prologue`` in include/gdn.h).

    q [T][H_q][d], k and v [T][H_kv][d] bf16 by their strides (views of a packed projection are fine), q_out
    like q (or q itself); freqs [rot/2] float64 or None; row [B], cu_seqlens [B+1] int32.  q and q_out may be
    None, and so may k and v (page_table may then be None too)."""
    torch = _torch()
    bf = torch.bfloat16
    if q is None and k is None:
        raise ValueError("nothing to do: q or k and v are required")
    if (q is None) != (q_out is None) or (k is None) != (v is None):
        raise ValueError("q and q_out go together, and so do k and v")
    N, H_kv, page, d, R, width, kind = _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    B = _packed_layout(row, cu_seqlens)
    T = (q if q is not None else k).shape[0]
    H_q = H_kv
    if q is not None:
        H_q = _heads_layout(_dev(q, "q", bf), "q", T, None, d)
        _heads_layout(_dev(q_out, "q_out", bf), "q_out", T, H_q, d)
    if k is not None:
        if page_table is None:
            raise ValueError("page_table is required to store k and v")
        _heads_layout(_dev(k, "k", bf), "k", T, H_kv, d)
        _heads_layout(_dev(v, "v", bf), "v", T, H_kv, d)
    _check_cache_tensors(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    _ints(row, "row")
    _ints(cu_seqlens, "cu_seqlens")
    if positions is not None and tuple(_ints(positions, "positions").shape) != (T,):
        raise ValueError("positions must be [T]")
    rope = norm = None
    if freqs is not None:
        _contig(_dev(freqs, "freqs", torch.float64), "freqs")
        if freqs.dim() != 1 or 2 * freqs.shape[0] > d:
            raise ValueError("freqs must be [rot/2] with rot <= d")
        rope = ctypes.byref(Rope(freqs.data_ptr(), 2 * freqs.shape[0], int(bool(interleaved)), rope_scale))
    for t, n in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if t is not None and tuple(_contig(_dev(t, n, bf), n).shape) != (d,):
            raise ValueError(f"{n} must be [d]")
    if q_norm is not None or k_norm is not None:
        norm = ctypes.byref(QkNorm(q_norm.data_ptr() if q_norm is not None else None,
                                   k_norm.data_ptr() if k_norm is not None else None, norm_eps, norm_add))
    dev = _device(q, k, v, q_out, k_pages, v_pages, page_table, kv_len, row, cu_seqlens, freqs, q_norm, k_norm,
                  positions, k_scale, v_scale)
    dims = AttnDims(B, T, R, H_q, H_kv, d, N, page, width, 0, 0, kind)
    cache = KvCache(k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                    kv_len.data_ptr())
    hq, hk, hv, ho = (None if t is None else ctypes.byref(_heads(t)) for t in (q, k, v, q_out))
    with _on(dev):
        _check("attn_prologue", lib().attn_prologue(
            ctypes.byref(dims), hq, hk, hv, ho, ctypes.byref(cache), row.data_ptr(), cu_seqlens.data_ptr(),
            _ptr(positions), rope, norm, _stream(stream, dev)))


def attn_paged_workspace_bytes(B: int, T: int, max_new: int, H_q: int, H_kv: int, d: int) -> int:
    """The workspace attn_paged needs (see include/gdn.h), in bytes, on the current GPU."""
    n = lib().attn_paged_workspace_bytes(ctypes.byref(AttnDims(B, T, 1, H_q, H_kv, d, 1, 16, 1, max_new, 0, 0)))
    if n == 0:
        raise GdnError("attn_paged_workspace_bytes", 2)
    return n


def attn_paged(q, k_pages, v_pages, page_table, kv_len, row, cu_seqlens, out, workspace, *, max_new: int,
               scale: float | None = None, window: int = 0, lse=None, k_scale=None, v_scale=None,
               stream=None) -> None:
    """Attention of every new token over its row's cached tokens (see ``attn_paged`` in include/gdn.h).

    q and out [T][H_q][d] bf16 by their strides; row [B], cu_seqlens [B+1] int32; workspace a uint8 tensor of
    attn_paged_workspace_bytes; lse [T][H_q] float32 or None; scale defaults to d ** -0.5; no sequence has more
    than max_new new tokens."""
    torch = _torch()
    N, H_kv, page, d, R, width, kind = _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    B = _packed_layout(row, cu_seqlens)
    T = q.shape[0]
    H_q = _heads_layout(_dev(q, "q", torch.bfloat16), "q", T, None, d)
    _heads_layout(_dev(out, "out", torch.bfloat16), "out", T, H_q, d)
    if page_table is None:
        raise ValueError("page_table is required")
    _check_cache_tensors(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    _ints(row, "row")
    _ints(cu_seqlens, "cu_seqlens")
    _contig(_dev(workspace, "workspace", torch.uint8), "workspace")
    if lse is not None and tuple(_contig(_dev(lse, "lse", torch.float32), "lse").shape) != (T, H_q):
        raise ValueError("lse must be [T][H_q]")
    dev = _device(q, out, k_pages, v_pages, page_table, kv_len, row, cu_seqlens, workspace, lse, k_scale, v_scale)
    dims = AttnDims(B, T, R, H_q, H_kv, d, N, page, width, max_new, window, kind)
    cache = KvCache(k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scale), _ptr(v_scale), page_table.data_ptr(),
                    kv_len.data_ptr())
    with _on(dev):
        _check("attn_paged", lib().attn_paged(
            ctypes.byref(dims), ctypes.byref(_heads(q)), ctypes.byref(cache), row.data_ptr(), cu_seqlens.data_ptr(),
            ctypes.byref(_heads(out)), _ptr(lse), 1.0 / math.sqrt(d) if scale is None else scale,
            workspace.data_ptr(), workspace.numel(), _stream(stream, dev)))


def kv_page_workspace_bytes(n: int, R: int, N: int) -> int:
    """The workspace of the bookkeeping calls for lists of up to n rows over R rows and N pages, in bytes."""
    b = lib().kv_page_workspace_bytes(n, R, N)
    if b == 0:
        raise GdnError("kv_page_workspace_bytes", 2)
    return b


def _table_layout(page_table, kv_len, refs):
    """Shape checks of a table with its counts; returns R, width, N."""
    if page_table.dim() != 2 or refs.dim() != 1 or (kv_len is not None and tuple(kv_len.shape) !=
                                                   (page_table.shape[0],)):
        raise ValueError("page_table must be [R][width], kv_len [R] and refs [N]")
    return page_table.shape[0], page_table.shape[1], refs.shape[0]


def _pages_layout(k_pages, v_pages):
    """A layer's pages or several layers' ([layers] in front); returns layers, N, page_size, strides in bytes."""
    if k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype or k_pages.dim() not in (4, 5):
        raise ValueError("k_pages and v_pages must both be [N][H_kv][page_size][d], or [layers] of that")
    layers = k_pages.shape[0] if k_pages.dim() == 5 else 1
    N, H_kv, page, d = k_pages.shape[-4:]
    nbytes = H_kv * page * d * k_pages.element_size()
    return layers, N, page, N * nbytes, nbytes


def _lists(a, b, names):
    _ints(a, names[0])
    if a.dim() != 1:
        raise ValueError(f"{names[0]} must be [n]")
    if b is not None and _ints(b, names[1]).shape != a.shape:
        raise ValueError(f"{names[0]} and {names[1]} must both be [n]")
    return a.shape[0]


def _scratch(result, workspace):
    if tuple(_ints(result, "result").shape) != (2,):
        raise ValueError("result must be [2]")
    return _contig(_dev(workspace, "workspace", _torch().uint8), "workspace")


def kv_page_reserve(page_table, kv_len, refs, rows, add, result, workspace, *, page_size: int, stream=None) -> None:
    """Grow rows by add[i] tokens, with the pages for them (see ``kv_page_reserve`` in include/gdn.h).  result
    [2] int32: rows not served and the first of them or -1."""
    R, width, N = _table_layout(_ints(page_table, "page_table"), _ints(kv_len, "kv_len"), _ints(refs, "refs"))
    n = _lists(rows, add, ("rows", "add"))
    _scratch(result, workspace)
    dev = _device(page_table, kv_len, refs, rows, add, result, workspace)
    g = Pages(R, width, N, page_size, page_table.data_ptr(), kv_len.data_ptr(), refs.data_ptr())
    with _on(dev):
        _check("kv_page_reserve", lib().kv_page_reserve(ctypes.byref(g), rows.data_ptr(), add.data_ptr(), n,
                                                        result.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                                        _stream(stream, dev)))


def kv_page_fork(k_pages, v_pages, page_table, kv_len, refs, src_rows, dst_rows, result, workspace, *,
                 stream=None) -> None:
    """Rows dst become copies of rows src that share whole pages (see ``kv_page_fork`` in include/gdn.h).
    k_pages and v_pages may have a leading layer axis."""
    layers, Np, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    R, width, N = _table_layout(_ints(page_table, "page_table"), _ints(kv_len, "kv_len"), _ints(refs, "refs"))
    if N != Np:
        raise ValueError(f"refs counts {N} pages, the cache has {Np}")
    _contig(_dev(k_pages, "k_pages", k_pages.dtype), "k_pages")
    _contig(_dev(v_pages, "v_pages", v_pages.dtype), "v_pages")
    n = _lists(src_rows, dst_rows, ("src_rows", "dst_rows"))
    _scratch(result, workspace)
    dev = _device(k_pages, v_pages, page_table, kv_len, refs, src_rows, dst_rows, result, workspace)
    g = Pages(R, width, N, page, page_table.data_ptr(), kv_len.data_ptr(), refs.data_ptr(), k_pages.data_ptr(),
              v_pages.data_ptr(), layers, 0, stride, nbytes)
    with _on(dev):
        _check("kv_page_fork", lib().kv_page_fork(ctypes.byref(g), src_rows.data_ptr(), dst_rows.data_ptr(), n,
                                                  result.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                                  _stream(stream, dev)))


def kv_page_free(page_table, kv_len, refs, rows, *, stream=None) -> None:
    """End rows: their pages' counts fall by one, their entries and lengths become 0 (see ``kv_page_free`` in
    include/gdn.h)."""
    R, width, N = _table_layout(_ints(page_table, "page_table"), _ints(kv_len, "kv_len"), _ints(refs, "refs"))
    n = _lists(rows, None, ("rows",))
    dev = _device(page_table, kv_len, refs, rows)
    g = Pages(R, width, N, 16, page_table.data_ptr(), kv_len.data_ptr(), refs.data_ptr())
    with _on(dev):
        _check("kv_page_free", lib().kv_page_free(ctypes.byref(g), rows.data_ptr(), n, _stream(stream, dev)))


def kv_page_copy(k_pages, v_pages, src, dst, *, stream=None) -> None:
    """Page src[i] to page dst[i], in every layer, k and v (see ``kv_page_copy`` in include/gdn.h)."""
    layers, N, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    _contig(_dev(k_pages, "k_pages", k_pages.dtype), "k_pages")
    _contig(_dev(v_pages, "v_pages", v_pages.dtype), "v_pages")
    n = _lists(src, dst, ("src", "dst"))
    dev = _device(k_pages, v_pages, src, dst)
    g = Pages(1, 1, N, page, None, None, None, k_pages.data_ptr(), v_pages.data_ptr(), layers, 0, stride, nbytes)
    with _on(dev):
        _check("kv_page_copy", lib().kv_page_copy(ctypes.byref(g), src.data_ptr(), dst.data_ptr(), n,
                                                  _stream(stream, dev)))


def kv_page_compact(k_pages, v_pages, page_table, refs, remap, result, workspace, *, stream=None) -> None:
    """Move the pages in use to the pool's low numbers (see ``kv_page_compact`` in include/gdn.h).  remap [N]
    int32 gets each page's new number (0: free), result [2] the pages in use and how many moved."""
    layers, Np, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    R, width, N = _table_layout(_ints(page_table, "page_table"), None, _ints(refs, "refs"))
    if N != Np or tuple(_ints(remap, "remap").shape) != (N,):
        raise ValueError(f"refs and remap must be [{Np}] as the cache has pages")
    _contig(_dev(k_pages, "k_pages", k_pages.dtype), "k_pages")
    _contig(_dev(v_pages, "v_pages", v_pages.dtype), "v_pages")
    _scratch(result, workspace)
    dev = _device(k_pages, v_pages, page_table, refs, remap, result, workspace)
    g = Pages(R, width, N, page, page_table.data_ptr(), None, refs.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
              layers, 0, stride, nbytes)
    with _on(dev):
        _check("kv_page_compact", lib().kv_page_compact(ctypes.byref(g), remap.data_ptr(), result.data_ptr(),
                                                        workspace.data_ptr(), workspace.numel(),
                                                        _stream(stream, dev)))
