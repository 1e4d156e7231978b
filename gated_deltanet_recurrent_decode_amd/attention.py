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
import struct

from . import GdnError, _check, lib

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


# The same structures as packed bytes: filling a ctypes structure field by field takes longer than the
# smallest of these calls takes on the GPU.
_DIMS, _HEADS, _CACHE = struct.Struct("12i"), struct.Struct("Pqq"), struct.Struct("6P")
_ROPE, _NORM, _PAGES = struct.Struct("Piif4x"), struct.Struct("PPff"), struct.Struct("4i5P2i2q")
for _packed, _struct in ((_DIMS, AttnDims), (_HEADS, Heads), (_CACHE, KvCache), (_ROPE, Rope), (_NORM, QkNorm),
                         (_PAGES, Pages)):
    assert _packed.size == ctypes.sizeof(_struct), _struct


def declare(L) -> None:
    """Argument types of this module's entry points (structures go as pointers or as packed bytes)."""
    size = ctypes.c_size_t
    for name, args, res in (
            ("gdn_rope_freqs", [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _P], _i32),
            ("attn_prologue", [_P] * 12, _i32),
            ("attn_paged", [_P, _P, _P, _P, _P, _P, _P, _f32, _P, size, _P], _i32),
            ("attn_paged_workspace_bytes", [_P], size),
            ("kv_page_workspace_bytes", [_i32, _i32, _i32], size),
            ("kv_page_reserve", [_P, _P, _P, _i32, _P, _P, size, _P], _i32),
            ("kv_page_fork", [_P, _P, _P, _i32, _P, _P, size, _P], _i32),
            ("kv_page_free", [_P, _P, _i32, _P], _i32),
            ("kv_page_copy", [_P, _P, _P, _i32, _P], _i32),
            ("kv_page_compact", [_P, _P, _P, _P, size, _P], _i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


# ------------------------------------------------------------------ tensors as pointers

_module = None


def _torch():
    global _module
    if _module is None:
        import torch
        _module = torch
    return _module


def _refuse(t, name, dtype, device):
    """Why `t` cannot be used (the checks of the fast paths below, with their messages)."""
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"all tensors must be on one GPU, got {name} on {t.device} and others on cuda:{device}")
    raise ValueError(f"{name}: must be contiguous")


def _gpu(t, name):
    """The index of the GPU that `t` is on; the calls below check that everything else is there too."""
    try:
        device = t.get_device()
    except AttributeError:
        device = -1
    if device < 0:
        _refuse(t, name, None, -1)
    return device


def _at(t, name, dtype, device):
    """A contiguous tensor's address."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, device)


def _at_or_none(t, name, dtype, device):
    return 0 if t is None else _at(t, name, dtype, device)


def _heads(t, name, T, H, d, dtype, device):
    """Packed heads [T][H][d] as the C structure: address, row and head strides."""
    s, step = t.shape, t.stride()
    if s != (T, H, d) or step[2] != 1:
        _heads_layout(t, name, T, H, d)
    if t.dtype is not dtype or t.get_device() != device:
        _refuse(t, name, dtype, device)
    # the stride of an axis of one says nothing, and torch lets it be anything
    return _HEADS.pack(t.data_ptr(), step[0] if T > 1 else 0, step[1] if H > 1 else 0)


def _launch(name, call, device, stream, *args):
    """Call with the stream to launch on, with the tensors' GPU as the current HIP device."""
    torch = _torch()
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)
    else:
        if stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{device}")
        raw = stream.cuda_stream
    now = torch._C._cuda_getDevice()
    if now == device:
        status = call(*args, raw)
    else:
        torch.cuda.set_device(device)
        try:
            status = call(*args, raw)
        finally:
            torch.cuda.set_device(now)
    if status:
        _check(name, status)


# ------------------------------------------------------------------ checks

def _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale):
    """Shape checks of a layer's cache (any device); returns N, H_kv, page_size, d, R, width, cache_type."""
    torch = _torch()
    dtype, shape = k_pages.dtype, k_pages.shape
    if v_pages.dtype is not dtype or dtype not in (torch.bfloat16, torch.float8_e4m3fn):
        raise ValueError(f"k_pages and v_pages must both be bfloat16 or float8_e4m3fn, got {dtype}, {v_pages.dtype}")
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must both be [N][H_kv][page_size][d]")
    N, H_kv, page, d = shape
    rows = kv_len.shape
    if len(rows) != 1:
        raise ValueError("kv_len must be [R]")
    width = 1
    if page_table is not None:
        table = page_table.shape
        if len(table) != 2 or table[0] != rows[0]:
            raise ValueError("page_table must be [R][width] and kv_len [R]")
        width = table[1]
    kind = 0
    if dtype is torch.float8_e4m3fn:
        kind = 1
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None or t.shape != (H_kv,):
                raise ValueError(f"{n} [H_kv] is required for an e4m3 cache")
    return N, H_kv, page, d, rows[0], width, kind


def _cache(k_pages, v_pages, page_table, kv_len, k_scale, v_scale, dev, torch):
    """A layer's cache as the C structure."""
    i32, f32, dtype = torch.int32, torch.float32, k_pages.dtype
    return _CACHE.pack(_at(k_pages, "k_pages", dtype, dev), _at(v_pages, "v_pages", dtype, dev),
                       0 if k_scale is None else _at(k_scale, "k_scale", f32, dev),
                       0 if v_scale is None else _at(v_scale, "v_scale", f32, dev),
                       0 if page_table is None else _at(page_table, "page_table", i32, dev),
                       _at(kv_len, "kv_len", i32, dev))


def _packed_layout(row, cu_seqlens):
    a, b = row.shape, cu_seqlens.shape
    if len(a) != 1 or len(b) != 1 or b[0] != a[0] + 1:
        raise ValueError("row must be [B] and cu_seqlens [B+1]")
    return a[0]


def _packed_heads(t, name):
    """Tokens and heads of a tensor [T][H][d]."""
    s = t.shape
    if len(s) != 3:
        raise ValueError(f"{name} must be [T][H][d], got {list(s)}")
    return s[0], s[1]


def _heads_layout(t, name, T, H, d):
    """Refuses anything but [T][H][d] with contiguous d."""
    s = t.shape
    if len(s) != 3 or s[0] != T or s[2] != d or s[1] != H:
        raise ValueError(f"{name} must be [{T}][{H}][{d}], got {list(s)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name}: the head's values must be contiguous")


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
    bf, i32 = torch.bfloat16, torch.int32
    if q is None and k is None:
        raise ValueError("nothing to do: q or k and v are required")
    if (q is None) != (q_out is None) or (k is None) != (v is None):
        raise ValueError("q and q_out go together, and so do k and v")
    N, H_kv, page, d, R, width, kind = _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    B = _packed_layout(row, cu_seqlens)
    dev = _gpu(row, "row")
    hq = ho = hk = hv = rope = norm = None
    H_q = H_kv
    if q is not None:
        T, H_q = _packed_heads(q, "q")
        hq, ho = _heads(q, "q", T, H_q, d, bf, dev), _heads(q_out, "q_out", T, H_q, d, bf, dev)
    if k is not None:
        if q is None:
            T, _ = _packed_heads(k, "k")
        if page_table is None:
            raise ValueError("page_table is required to store k and v")
        hk, hv = _heads(k, "k", T, H_kv, d, bf, dev), _heads(v, "v", T, H_kv, d, bf, dev)
    if freqs is not None:
        s = freqs.shape
        if len(s) != 1 or 2 * s[0] > d:
            raise ValueError("freqs must be [rot/2] with rot <= d")
        rope = _ROPE.pack(_at(freqs, "freqs", torch.float64, dev), 2 * s[0], int(bool(interleaved)), rope_scale)
    if q_norm is not None or k_norm is not None:
        for t, n in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None and t.shape != (d,):
                raise ValueError(f"{n} must be [d]")
        norm = _NORM.pack(_at_or_none(q_norm, "q_norm", bf, dev), _at_or_none(k_norm, "k_norm", bf, dev), norm_eps,
                          norm_add)
    if positions is not None and positions.shape != (T,):
        raise ValueError("positions must be [T]")
    _launch("attn_prologue", lib().attn_prologue, dev, stream,
            _DIMS.pack(B, T, R, H_q, H_kv, d, N, page, width, 0, 0, kind), hq, hk, hv, ho,
            _cache(k_pages, v_pages, page_table, kv_len, k_scale, v_scale, dev, torch), _at(row, "row", i32, dev),
            _at(cu_seqlens, "cu_seqlens", i32, dev), _at_or_none(positions, "positions", i32, dev), rope, norm)


def attn_paged_workspace_bytes(B: int, T: int, max_new: int, H_q: int, H_kv: int, d: int) -> int:
    """The workspace attn_paged needs (see include/gdn.h), in bytes, on the current GPU."""
    n = lib().attn_paged_workspace_bytes(_DIMS.pack(B, T, 1, H_q, H_kv, d, 1, 16, 1, max_new, 0, 0))
    if n == 0:
        raise GdnError("attn_paged_workspace_bytes", 2)
    return n


def attn_paged(q, k_pages, v_pages, page_table, kv_len, row, cu_seqlens, out, workspace, *, max_new: int,
               scale: float | None = None, window: int = 0, lse=None, k_scale=None, v_scale=None,
               stream=None) -> None:
    """Attention of every new token over its row's cached tokens (see ``attn_paged`` in include/gdn.h).

    q and out [T][H_q][d] bf16 by their strides; row [B], cu_seqlens [B+1] int32; workspace a uint8 tensor of
    attn_paged_workspace_bytes; lse [T][H_q] float32 or None; scale defaults to d ** -0.5; no sequence has more
    than max_new new tokens.  max_new picks the kernel and with it the precision: with max_new * H_q / H_kv above
    16 the softmax's weights are rounded to bf16 for the product with v."""
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    N, H_kv, page, d, R, width, kind = _cache_layout(k_pages, v_pages, page_table, kv_len, k_scale, v_scale)
    B = _packed_layout(row, cu_seqlens)
    T, H_q = _packed_heads(q, "q")
    if page_table is None:
        raise ValueError("page_table is required")
    if lse is not None and lse.shape != (T, H_q):
        raise ValueError("lse must be [T][H_q]")
    dev = _gpu(q, "q")
    _launch("attn_paged", lib().attn_paged, dev, stream,
            _DIMS.pack(B, T, R, H_q, H_kv, d, N, page, width, max_new, window, kind),
            _heads(q, "q", T, H_q, d, bf, dev),
            _cache(k_pages, v_pages, page_table, kv_len, k_scale, v_scale, dev, torch), _at(row, "row", i32, dev),
            _at(cu_seqlens, "cu_seqlens", i32, dev), _heads(out, "out", T, H_q, d, bf, dev),
            _at_or_none(lse, "lse", torch.float32, dev), 1.0 / math.sqrt(d) if scale is None else scale,
            _at(workspace, "workspace", torch.uint8, dev), workspace.numel())


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
    if a.dim() != 1 or (b is not None and b.shape != a.shape):
        raise ValueError(f"{' and '.join(names)} must be [n]")
    return a.shape[0]


def _table(page_table, kv_len, refs, dev):
    torch = _torch()
    i32 = torch.int32
    return (_at(page_table, "page_table", i32, dev), _at_or_none(kv_len, "kv_len", i32, dev),
            _at(refs, "refs", i32, dev))


def _pools(k_pages, v_pages, dev):
    return _at(k_pages, "k_pages", k_pages.dtype, dev), _at(v_pages, "v_pages", v_pages.dtype, dev)


def _scratch(result, workspace, dev):
    torch = _torch()
    if result.shape != (2,):
        raise ValueError("result must be [2]")
    return (_at(result, "result", torch.int32, dev), _at(workspace, "workspace", torch.uint8, dev),
            workspace.numel())


def kv_page_reserve(page_table, kv_len, refs, rows, add, result, workspace, *, page_size: int, stream=None) -> None:
    """Grow rows by add[i] tokens, with the pages for them (see ``kv_page_reserve`` in include/gdn.h).  result
    [2] int32: rows not served and the first of them or -1."""
    i32 = _torch().int32
    R, width, N = _table_layout(page_table, kv_len, refs)
    n = _lists(rows, add, ("rows", "add"))
    dev = _gpu(page_table, "page_table")
    _launch("kv_page_reserve", lib().kv_page_reserve, dev, stream,
            _PAGES.pack(R, width, N, page_size, *_table(page_table, kv_len, refs, dev), 0, 0, 0, 0, 0, 0),
            _at(rows, "rows", i32, dev), _at(add, "add", i32, dev), n, *_scratch(result, workspace, dev))


def kv_page_fork(k_pages, v_pages, page_table, kv_len, refs, src_rows, dst_rows, result, workspace, *,
                 stream=None) -> None:
    """Rows dst become copies of rows src that share whole pages (see ``kv_page_fork`` in include/gdn.h).
    k_pages and v_pages may have a leading layer axis."""
    i32 = _torch().int32
    layers, Np, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    R, width, N = _table_layout(page_table, kv_len, refs)
    if N != Np:
        raise ValueError(f"refs counts {N} pages, the cache has {Np}")
    n = _lists(src_rows, dst_rows, ("src_rows", "dst_rows"))
    dev = _gpu(page_table, "page_table")
    _launch("kv_page_fork", lib().kv_page_fork, dev, stream,
            _PAGES.pack(R, width, N, page, *_table(page_table, kv_len, refs, dev), *_pools(k_pages, v_pages, dev),
                        layers, 0, stride, nbytes),
            _at(src_rows, "src_rows", i32, dev), _at(dst_rows, "dst_rows", i32, dev), n,
            *_scratch(result, workspace, dev))


def kv_page_free(page_table, kv_len, refs, rows, *, stream=None) -> None:
    """End rows: their pages' counts fall by one, their entries and lengths become 0 (see ``kv_page_free`` in
    include/gdn.h)."""
    i32 = _torch().int32
    R, width, N = _table_layout(page_table, kv_len, refs)
    n = _lists(rows, None, ("rows",))
    dev = _gpu(page_table, "page_table")
    _launch("kv_page_free", lib().kv_page_free, dev, stream,
            _PAGES.pack(R, width, N, 16, *_table(page_table, kv_len, refs, dev), 0, 0, 0, 0, 0, 0),
            _at(rows, "rows", i32, dev), n)


def kv_page_copy(k_pages, v_pages, src, dst, *, stream=None) -> None:
    """Page src[i] to page dst[i], in every layer, k and v (see ``kv_page_copy`` in include/gdn.h)."""
    i32 = _torch().int32
    layers, N, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    n = _lists(src, dst, ("src", "dst"))
    dev = _gpu(src, "src")
    _launch("kv_page_copy", lib().kv_page_copy, dev, stream,
            _PAGES.pack(1, 1, N, page, 0, 0, 0, *_pools(k_pages, v_pages, dev), layers, 0, stride, nbytes),
            _at(src, "src", i32, dev), _at(dst, "dst", i32, dev), n)


def kv_page_compact(k_pages, v_pages, page_table, refs, remap, result, workspace, *, stream=None) -> None:
    """Move the pages in use to the pool's low numbers (see ``kv_page_compact`` in include/gdn.h).  remap [N]
    int32 gets each page's new number (0: free), result [2] the pages in use and how many moved."""
    i32 = _torch().int32
    layers, Np, page, stride, nbytes = _pages_layout(k_pages, v_pages)
    R, width, N = _table_layout(page_table, None, refs)
    if N != Np or remap.shape != (N,):
        raise ValueError(f"refs and remap must be [{Np}] as the cache has pages")
    dev = _gpu(page_table, "page_table")
    _launch("kv_page_compact", lib().kv_page_compact, dev, stream,
            _PAGES.pack(R, width, N, page, *_table(page_table, None, refs, dev), *_pools(k_pages, v_pages, dev),
                        layers, 0, stride, nbytes),
            _at(remap, "remap", i32, dev), *_scratch(result, workspace, dev))
