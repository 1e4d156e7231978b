"""CPU: what the paged-attention entry points refuse, at the C ABI (every call
here fails validation or has nothing to do, so nothing is launched) and in the
binding's layout checks (meta tensors)."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from gated_deltanet_recurrent_decode_amd import attention as at

OK, NULL, SHAPE, UNSUPPORTED = 0, 1, 2, 3
FAKE = 0x10000  # never dereferenced


def dims(**kw):
    base = dict(B=2, T=4, R=5, H_q=4, H_kv=2, d=64, N=9, page_size=16, table_width=8, max_new=2, window=0,
                cache_type=0)
    base.update(kw)
    return at.AttnDims(*[base[n] for n, _ in at.AttnDims._fields_])


def heads(p=FAKE, row=256, head=64):
    return at.Heads(p, row, head)


def cache(k=FAKE, v=FAKE, ks=None, vs=None, table=FAKE, n=FAKE):
    return at.KvCache(k, v, ks, vs, table, n)


def paged(d=None, q=None, c=None, row=FAKE, cu=FAKE, out=None, scale=1.0, ws=FAKE, nbytes=1 << 40, no_dims=False):
    d = dims() if d is None else d
    return gdn.lib().attn_paged(None if no_dims else ctypes.byref(d), ctypes.byref(q or heads()),
                                ctypes.byref(c or cache()), row, cu, ctypes.byref(out or heads()), None, scale, ws,
                                nbytes, None)


def test_attn_paged_refusals():
    assert paged(no_dims=True) == NULL
    assert paged(dims(B=0), row=None, ws=None) == OK and paged(dims(T=0), row=None, ws=None) == OK
    for bad in (dict(q=heads(None)), dict(out=heads(None)), dict(row=None), dict(cu=None), dict(ws=None),
                dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(table=None)), dict(c=cache(n=None)),
                dict(d=dims(cache_type=1))):
        assert paged(**bad) == NULL, bad
    for bad in (dict(B=-1), dict(T=-1), dict(R=0), dict(H_q=5), dict(H_kv=0), dict(N=0), dict(table_width=0),
                dict(max_new=-1), dict(window=-1), dict(table_width=1 << 28), dict(T=1 << 30)):
        assert paged(dims(**bad)) == SHAPE, bad
    for bad in (dict(d=96), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(cache_type=2),
                dict(cache_type=-1)):
        assert paged(dims(**bad)) == UNSUPPORTED, bad
    for bad in (dict(q=heads(FAKE + 8)), dict(out=heads(FAKE + 2)), dict(q=heads(row=252)), dict(out=heads(head=60)),
                dict(c=cache(k=FAKE + 8)), dict(c=cache(v=FAKE + 4)), dict(ws=FAKE + 128)):
        assert paged(**bad) == UNSUPPORTED, bad
    assert paged(q=heads(row=-256)) == SHAPE
    assert paged(scale=math.nan) == SHAPE and paged(scale=math.inf) == SHAPE
    need = gdn.attn_paged_workspace_bytes(2, 4, 2, 4, 2, 64)
    assert need > 0 and paged(nbytes=need - 1) == SHAPE
    assert gdn.lib().attn_paged_workspace_bytes(None) == 0
    for bad in (dict(d=96), dict(H_q=5), dict(B=-1)):
        assert gdn.lib().attn_paged_workspace_bytes(ctypes.byref(dims(**bad))) == 0
    with pytest.raises(gdn.GdnError):
        gdn.attn_paged_workspace_bytes(1, 1, 1, 5, 2, 64)


def prologue(d=None, q="h", k="h", v="h", o="h", c=None, row=FAKE, cu=FAKE, rope=None, norm=None):
    ref = lambda x: None if x is None else ctypes.byref(heads() if x == "h" else x)  # noqa: E731
    return gdn.lib().attn_prologue(ctypes.byref(d or dims()), ref(q), ref(k), ref(v), ref(o),
                                   ctypes.byref(c or cache()), row, cu, None,
                                   None if rope is None else ctypes.byref(rope),
                                   None if norm is None else ctypes.byref(norm), None)


def test_attn_prologue_refusals():
    assert prologue(dims(B=0), q=None) == OK
    for bad in (dict(q=None, k=None, v=None, o=None), dict(o=None), dict(q=None), dict(v=None), dict(k=None),
                dict(row=None), dict(cu=None), dict(c=cache(n=None)), dict(c=cache(table=None)), dict(c=cache(k=None)),
                dict(rope=at.Rope(None, 64, 0, 1.0)), dict(d=dims(cache_type=1))):
        assert prologue(**bad) == NULL, bad
    for bad in (dict(rope=at.Rope(FAKE, 66, 0, 1.0)), dict(rope=at.Rope(FAKE, 7, 0, 1.0)),
                dict(rope=at.Rope(FAKE, -2, 0, 1.0)), dict(rope=at.Rope(FAKE, 64, 0, math.inf)),
                dict(norm=at.QkNorm(FAKE, FAKE, -1.0, 0.0)), dict(norm=at.QkNorm(FAKE, FAKE, 1e-6, math.nan)),
                dict(d=dims(H_q=65536, H_kv=65536))):
        assert prologue(**bad) == SHAPE, bad
    for bad in (dict(q=heads(FAKE + 8)), dict(k=heads(row=4)), dict(v=heads(head=4)), dict(o=heads(FAKE + 4)),
                dict(rope=at.Rope(FAKE + 4, 64, 0, 1.0)), dict(norm=at.QkNorm(FAKE + 8, None, 1e-6, 0.0)),
                dict(d=dims(d=32))):
        assert prologue(**bad) == UNSUPPORTED, bad


def test_rope_freqs():
    f = gdn.lib().gdn_rope_freqs
    out = (ctypes.c_double * 64)()
    assert f(64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, None) == NULL
    for bad in ((-2, 1e4, 0, 1.0, 0.0), (3, 1e4, 0, 1.0, 0.0), (64, 0.0, 0, 1.0, 0.0), (64, math.inf, 0, 1.0, 0.0),
                (64, 1e4, 4, 1.0, 0.0), (64, 1e4, 1, 0.0, 0.0), (2, 1e4, 2, 2.0, 0.0), (64, 1e4, 3, 2.0, 0.0)):
        assert f(*bad, 1.0, 32.0, out) == SHAPE, bad
    assert f(64, 1e4, 3, 2.0, 4096.0, 32.0, 32.0, out) == SHAPE
    j = torch.arange(32, dtype=torch.float64)
    plain = 1e4 ** (-2 * j / 64)
    close = lambda a, b: torch.allclose(a, b, rtol=1e-13, atol=0)  # noqa: E731
    assert close(gdn.rope_freqs(64, 1e4, device="cpu"), plain)
    assert close(gdn.rope_freqs(64, 1e4, stretch="linear", factor=4.0, device="cpu"), plain / 4)
    base = gdn.rope_freqs(64, 1e4, stretch="base", factor=4.0, device="cpu")
    assert base[0] == 1 and abs(base[-1] * 4 / plain[-1] - 1) < 1e-12   # the longest wavelength grows by factor
    w = gdn.rope_freqs(64, 1e4, stretch="wavelength", factor=4.0, original=4096.0, low=1.0, high=32.0, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert close(w[turns >= 32], plain[turns >= 32]) and close(w[turns <= 1], plain[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((w < plain) & (w > plain / 4))[mid].all()
    with pytest.raises(ValueError, match="stretch"):
        gdn.rope_freqs(64, stretch="yes", device="cpu")


def pages(**kw):
    base = dict(R=4, table_width=4, N=9, page_size=16, page_table=FAKE, kv_len=FAKE, refs=FAKE, k=FAKE, v=FAKE,
                layers=1, reserved=0, layer_stride=9 * 4096, page_bytes=4096)
    base.update(kw)
    return at.Pages(*[base[n] for n, _ in at.Pages._fields_])


def test_kv_page_refusals():
    L = gdn.lib()
    big = 1 << 40
    table_calls = {
        "reserve": lambda g, n=2, a=FAKE, r=FAKE, w=FAKE, s=big: L.kv_page_reserve(g, a, FAKE, n, r, w, s, None),
        "fork": lambda g, n=2, a=FAKE, r=FAKE, w=FAKE, s=big: L.kv_page_fork(g, a, FAKE, n, r, w, s, None),
    }
    for name, call in table_calls.items():
        assert call(None) == NULL
        assert call(ctypes.byref(pages()), a=None) == NULL
        assert call(ctypes.byref(pages()), r=None) == NULL and call(ctypes.byref(pages()), w=None) == NULL
        assert call(ctypes.byref(pages()), n=-1) == SHAPE and call(ctypes.byref(pages()), n=65536) == SHAPE
        assert call(ctypes.byref(pages()), w=FAKE + 16) == UNSUPPORTED
        need = gdn.kv_page_workspace_bytes(2, 4, 9)
        assert call(ctypes.byref(pages()), s=need - 1) == SHAPE
        for bad, st in ((dict(page_table=None), NULL), (dict(refs=None), NULL), (dict(kv_len=None), NULL),
                        (dict(R=0), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 20) + 1), SHAPE),
                        (dict(table_width=0), SHAPE), (dict(page_size=24), UNSUPPORTED),
                        (dict(table_width=1 << 28), SHAPE)):
            assert call(ctypes.byref(pages(**bad))) == st, (name, bad)
    moves = {
        "fork": lambda g: L.kv_page_fork(g, FAKE, FAKE, 2, FAKE, FAKE, big, None),
        "copy": lambda g: L.kv_page_copy(g, FAKE, FAKE, 2, None),
        "compact": lambda g: L.kv_page_compact(g, FAKE, FAKE, FAKE, big, None),
    }
    for name, call in moves.items():
        for bad, st in ((dict(k=None), NULL), (dict(v=None), NULL), (dict(layers=0), SHAPE),
                        (dict(page_bytes=0), SHAPE),
                        (dict(layers=2, layer_stride=9 * 4096 - 16), SHAPE), (dict(page_bytes=4088), UNSUPPORTED),
                        (dict(k=FAKE + 8), UNSUPPORTED), (dict(layer_stride=9 * 4096 + 8), UNSUPPORTED)):
            assert call(ctypes.byref(pages(**bad))) == st, (name, bad)
    assert L.kv_page_copy(ctypes.byref(pages()), None, FAKE, 2, None) == NULL
    assert L.kv_page_copy(ctypes.byref(pages()), None, None, 0, None) == OK
    assert L.kv_page_copy(ctypes.byref(pages()), FAKE, FAKE, -1, None) == SHAPE
    assert L.kv_page_free(ctypes.byref(pages()), None, 1, None) == NULL
    assert L.kv_page_free(ctypes.byref(pages()), None, 0, None) == OK
    assert L.kv_page_free(None, FAKE, 1, None) == NULL
    assert L.kv_page_compact(ctypes.byref(pages()), None, FAKE, FAKE, big, None) == NULL
    assert gdn.lib().kv_page_workspace_bytes(-1, 1, 1) == 0


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_layouts():
    i32, f32 = torch.int32, torch.float32
    k, v, table, n = meta(9, 2, 16, 64), meta(9, 2, 16, 64), meta(5, 8, dtype=i32), meta(5, dtype=i32)
    assert at._cache_layout(k, v, table, n, None, None) == (9, 2, 16, 64, 5, 8, 0)
    f8 = k.to(torch.float8_e4m3fn)
    s = meta(2, dtype=f32)
    assert at._cache_layout(f8, f8, table, n, s, s)[-1] == 1
    for bad in ((k, meta(9, 2, 16, 128), table, n, None, None), (k, f8, table, n, None, None),
                (k, v, meta(4, 8, dtype=i32), n, None, None), (k, v, table, meta(5, 1, dtype=i32), None, None),
                (f8, f8, table, n, None, s), (f8, f8, table, n, s, meta(3, dtype=f32)),
                (meta(2, 16, 64), meta(2, 16, 64), table, n, None, None),
                (k.to(torch.float16), v.to(torch.float16), table, n, None, None)):
        with pytest.raises(ValueError):
            at._cache_layout(*bad)
    assert at._packed_layout(meta(3, dtype=i32), meta(4, dtype=i32)) == 3
    with pytest.raises(ValueError):
        at._packed_layout(meta(3, dtype=i32), meta(3, dtype=i32))
    at._heads_layout(meta(7, 4, 64), "q", 7, 4, 64)
    assert at._packed_heads(meta(7, 4, 64), "q") == (7, 4)
    with pytest.raises(ValueError):
        at._packed_heads(meta(7, 256), "q")
    for bad in (meta(6, 4, 64), meta(7, 3, 64), meta(7, 4, 32), meta(7, 4, 128)[:, :, ::2]):
        with pytest.raises(ValueError):
            at._heads_layout(bad, "q", 7, 4, 64)
    assert at._pages_layout(meta(3, 9, 2, 16, 64), meta(3, 9, 2, 16, 64)) == (3, 9, 16, 9 * 4096, 4096)
    with pytest.raises(ValueError):
        at._pages_layout(k, meta(8, 2, 16, 64))
    assert at._table_layout(table, n, meta(9, dtype=i32)) == (5, 8, 9)
    with pytest.raises(ValueError):
        at._table_layout(table, meta(4, dtype=i32), meta(9, dtype=i32))


def test_binding_refuses_cpu_tensors_and_missing_parts():
    c = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.attn_paged(q, c, c, i(2, 2), i(2), i(1), i(2), q, torch.zeros(9, dtype=torch.uint8), max_new=1)
    with pytest.raises(ValueError, match="nothing to do"):
        gdn.attn_prologue(None, None, None, None, c, c, i(2, 2), i(2), i(1), i(2), None)
    with pytest.raises(ValueError, match="together"):
        gdn.attn_prologue(q, None, None, None, c, c, i(2, 2), i(2), i(1), i(2), None)
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.kv_page_free(i(2, 2), i(2), i(3), i(1))


def test_the_stride_of_an_axis_of_one_does_not_matter():
    bf = torch.bfloat16
    one = torch.zeros(4, 64, 1, dtype=bf).permute(2, 0, 1)     # one token, its stride 1
    assert one.stride(0) % 8 and at._HEADS.unpack(at._heads(one, "q", 1, 4, 64, bf, -1))[1:] == (0, 64)
    one = torch.zeros(4, 64, dtype=bf).as_strided((4, 1, 64), (64, 3, 1))  # one head
    assert at._HEADS.unpack(at._heads(one, "k", 4, 1, 64, bf, -1))[1:] == (64, 0)
