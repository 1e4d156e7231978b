"""CPU: what the linear-attention entry points refuse, at the C ABI (every call here fails validation or has
nothing to do, so nothing is launched) and in the binding's layout checks."""
import ctypes
import math

import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from gated_deltanet_recurrent_decode_amd import linear
from gated_deltanet_recurrent_decode_amd.attention import Heads

OK, NULL, SHAPE, UNSUPPORTED = 0, 1, 2, 3
FAKE = 0x10000  # never dereferenced


def dims(**kw):
    base = dict(B=2, T=4, H_k=2, H_v=4, d_k=64, d_v=64, N=9, per_token=1)
    base.update(kw)
    return linear.LinDims(*[base[n] for n, _ in linear.LinDims._fields_])


def heads(p=FAKE, row=512, head=64):
    return Heads(p, row, head)


def call(name, d=None, *, q=None, k=None, v=None, out=None, g=FAKE, state=FAKE, read=FAKE, slots=FAKE, cu=FAKE,
         scale=1.0, ws=FAKE, nbytes=1 << 40, no_dims=False, no_heads=None):
    d = dims() if d is None else d
    ref = [ctypes.byref(x or heads()) for x in (q, k, v, out)]
    if no_heads is not None:
        ref[no_heads] = None
    dp = None if no_dims else ctypes.byref(d)
    if name == "lin_attn_prefill":
        return gdn.lib().lin_attn_prefill(dp, *ref[:3], g, cu, state, read, slots, ref[3], scale, ws, nbytes, None)
    return getattr(gdn.lib(), name)(dp, *ref[:3], g, state, read, slots, ref[3], scale, None)


CALLS = ["lin_attn_step", "lin_attn_step_tokens", "lin_attn_prefill"]


@pytest.mark.parametrize("name", CALLS)
def test_refusals(name):
    assert call(name, no_dims=True) == NULL
    assert call(name, dims(B=0), read=None, g=None, state=None) == OK
    for bad in (dict(q=heads(None)), dict(k=heads(None)), dict(v=heads(None)), dict(out=heads(None)), dict(g=None),
                dict(state=None), dict(read=None), dict(no_heads=0), dict(no_heads=3)):
        assert call(name, **bad) == NULL, bad
    for bad in (dict(B=-1), dict(T=-1), dict(H_k=0), dict(H_v=3), dict(H_v=0), dict(N=0), dict(per_token=2),
                dict(per_token=-1), dict(B=1 << 18), dict(T=1 << 30)):
        assert call(name, dims(**bad)) == SHAPE, bad
    for bad in (dict(d_k=96), dict(d_v=256), dict(d_k=32)):
        assert call(name, dims(**bad)) == UNSUPPORTED, bad
    for bad in (dict(q=heads(FAKE + 8)), dict(k=heads(row=508)), dict(v=heads(head=60)), dict(out=heads(FAKE + 2)),
                dict(state=FAKE + 8), dict(g=FAKE + 2)):
        assert call(name, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=heads(row=-512)), dict(v=heads(head=-64)), dict(k=heads(row=1 << 25)), dict(scale=math.nan),
                dict(scale=math.inf)):
        assert call(name, **bad) == SHAPE, bad


def test_refusals_of_one_call():
    assert call("lin_attn_prefill", dims(T=(1 << 30) - 1, H_k=16, H_v=16)) == SHAPE  # segments of 16 heads
    assert call("lin_attn_step", dims(T=0)) == SHAPE and call("lin_attn_step", dims(B=1 << 10, T=1 << 20)) == SHAPE
    assert call("lin_attn_step_tokens", slots=None) == NULL
    assert call("lin_attn_prefill", cu=None) == NULL and call("lin_attn_prefill", ws=None) == NULL
    assert call("lin_attn_prefill", ws=FAKE + 128) == UNSUPPORTED
    need = gdn.lin_attn_prefill_workspace_bytes(2, 4000, 2, 4, 64, 64)
    assert call("lin_attn_prefill", dims(T=4000), nbytes=need - 1) == SHAPE
    assert gdn.lib().lin_attn_prefill_workspace_bytes(None) == 0
    assert call("lin_attn_prefill", dims(T=(1 << 30) - 1, H_v=1 << 10, H_k=1)) == SHAPE  # threads of a launch
    with pytest.raises(gdn.GdnError):
        gdn.lin_attn_prefill_workspace_bytes(2, 4, 2, 3, 64, 64)


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_layout_checks():
    f32, i32 = torch.float32, torch.int32
    good = dict(q=meta(3, 2, 2, 64), k=meta(3, 2, 2, 64), v=meta(3, 2, 4, 128), g=meta(3, 2, 4, dtype=f32),
                state=meta(9, 4, 64, 128, dtype=f32), read_slot=meta(3, dtype=i32), write_slot=meta(3, dtype=i32),
                out=meta(3, 2, 4, 128))
    for name, bad, why in (("state", meta(9, 4, 64, dtype=f32), "state"), ("q", meta(3, 2, 3, 64), "multiple"),
                           ("q", meta(3, 2, 64), "q must be"), ("g", meta(2, 4, dtype=f32), "g must be"),
                           ("g", meta(3, dtype=f32), "g must be"), ("read_slot", meta(2, dtype=i32), "read_slot"),
                           ("write_slot", meta(4, dtype=i32), "write_slot")):
        with pytest.raises(ValueError, match=why):
            gdn.lin_attn_step(**{**good, name: bad})
    with pytest.raises(ValueError, match="GPU tensor"):
        gdn.lin_attn_step(**good)
    tokens = {n: t for n, t in good.items() if n != "write_slot"}
    with pytest.raises(ValueError, match="token_slots"):
        gdn.lin_attn_step_tokens(**tokens, token_slots=None)
    with pytest.raises(ValueError, match="token_slots"):
        gdn.lin_attn_step_tokens(**tokens, token_slots=meta(3, dtype=i32))
    for x, why in ((meta(3, 2, 2, 32), "must be"), (meta(6, 2, 2, 64)[::2], "fixed stride"),
                   (meta(3, 2, 64, 2).transpose(2, 3), "contiguous"),
                   (meta(3, 4, 2, 64)[:, :2], "fixed stride")):
        with pytest.raises(ValueError, match=why):
            linear._rows(x, "k", 3, 2, 2, 64, torch.bfloat16, 5)
    packed = dict(q=meta(7, 2, 64), k=meta(7, 2, 64), v=meta(7, 4, 64), g=meta(4, dtype=f32),
                  cu_seqlens=meta(3, dtype=i32), state=meta(9, 4, 64, 64, dtype=f32), read_slot=meta(2, dtype=i32),
                  write_slot=None, out=meta(7, 4, 64), workspace=meta(1, dtype=torch.uint8))
    for name, bad, why in (("cu_seqlens", meta(2, dtype=i32), "cu_seqlens"), ("g", meta(6, 4, dtype=f32), "g must be"),
                           ("write_slot", meta(3, dtype=i32), "write_slot"), ("q", meta(7, 3, 64), "multiple"),
                           ("q", meta(7, 128), "q must be")):
        with pytest.raises(ValueError, match=why):
            gdn.lin_attn_prefill(**{**packed, name: bad})
