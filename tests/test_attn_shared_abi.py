"""CPU: what attn_shared refuses, at the C ABI (every call here fails validation or has nothing to do, so nothing is
launched) and in the binding's layout checks."""
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


def shared(d=None, q=None, c=None, row=FAKE, cu=FAKE, groups=FAKE, lens=FAKE, K=1, out=None, scale=1.0, ws=FAKE,
           nbytes=1 << 40, no_dims=False):
    d = dims() if d is None else d
    c = at.KvCache(FAKE, FAKE, None, None, FAKE, FAKE) if c is None else c
    return gdn.lib().attn_shared(None if no_dims else ctypes.byref(d), ctypes.byref(q or heads()), ctypes.byref(c), row,
                                 cu, groups, lens, K, -1, ctypes.byref(out or heads()), None, scale, ws, nbytes, None)


def test_refusals():
    assert shared(no_dims=True) == NULL
    assert shared(dims(B=0), row=None, ws=None) == OK and shared(dims(T=0), row=None, ws=None) == OK
    for bad in (dict(q=heads(None)), dict(out=heads(None)), dict(row=None), dict(cu=None), dict(ws=None),
                dict(groups=None), dict(lens=None), dict(d=dims(cache_type=1)),
                dict(c=at.KvCache(None, FAKE, None, None, FAKE, FAKE))):
        assert shared(**bad) == NULL, bad
    for bad in (dict(B=-1), dict(R=0), dict(H_q=5), dict(max_new=-1), dict(window=-1), dict(T=1 << 30)):
        assert shared(dims(**bad)) == SHAPE, bad
    for bad in (dict(B=1 << 23), dict(T=1 << 26, H_q=16, H_kv=16, max_new=1 << 20), dict(B=1 << 20, H_q=32, H_kv=16)):
        assert shared(dims(**bad)) == SHAPE, bad  # more entries than the join's grid counts
    for bad in (dict(d=96), dict(page_size=8), dict(cache_type=2)):
        assert shared(dims(**bad)) == UNSUPPORTED, bad
    assert shared(K=-1) == SHAPE and shared(K=1025) == SHAPE and shared(scale=math.nan) == SHAPE
    assert shared(q=heads(FAKE + 8)) == UNSUPPORTED and shared(ws=FAKE + 64) == UNSUPPORTED
    need = gdn.attn_shared_workspace_bytes(2, 4, 1, 2, 4, 2, 64)
    assert shared(nbytes=need - 1) == SHAPE
    assert gdn.lib().attn_shared_workspace_bytes(None, 1) == 0
    for bad in (dict(d=96), dict(H_q=5), dict(B=-1)):
        assert gdn.lib().attn_shared_workspace_bytes(ctypes.byref(dims(**bad)), 1) == 0
    with pytest.raises(gdn.GdnError):
        gdn.attn_shared_workspace_bytes(2, 4, 1025, 2, 4, 2, 64)


def test_layout_checks():
    def meta(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")

    bf = torch.bfloat16
    good = dict(q=meta(4, 4, 64, dtype=bf), k_pages=meta(9, 2, 16, 64, dtype=bf), v_pages=meta(9, 2, 16, 64, dtype=bf),
                page_table=meta(5, 8), kv_len=meta(5), row=meta(2), cu_seqlens=meta(3), cu_groups=meta(2),
                shared_len=meta(1), out=meta(4, 4, 64, dtype=bf), workspace=meta(1, dtype=torch.uint8), max_new=2)
    for name, bad, why in (("cu_groups", meta(3), "cu_groups"), ("shared_len", meta(1, 1), "shared_len"),
                           ("page_table", None, "page_table"), ("lse", meta(4), "lse"), ("least", -1, "least"), ("least", 1 << 31, "least"), ("row", meta(3), "row must be")):
        with pytest.raises(ValueError, match=why):
            gdn.attn_shared(**{**good, name: bad})
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.attn_shared(**good)
