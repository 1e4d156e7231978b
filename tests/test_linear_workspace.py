"""CPU: a workspace of lin_attn_prefill that is sized for the largest call serves the smaller ones."""
import ctypes

import pytest

import gated_deltanet_recurrent_decode_amd as gdn
from gated_deltanet_recurrent_decode_amd import linear
from gated_deltanet_recurrent_decode_amd.attention import Heads

SHAPE, FAKE = 2, 0x10000  # the address is never dereferenced

HEADS = [(16, 16, 128, 128), (32, 32, 128, 128), (8, 32, 128, 64), (32, 32, 128, 64), (1, 1, 64, 64), (64, 64, 64, 128),
         (128, 128, 128, 128)]


@pytest.mark.parametrize("heads", HEADS)
def test_the_size_never_falls_as_the_call_grows(heads):
    def size(B, T):
        return gdn.lin_attn_prefill_workspace_bytes(B, T, *heads)

    lengths = sorted({1, 2, 127, 128, 129, 2047, 2048, 2049, *range(0, 9000, 7), *range(9000, 70000, 331)})
    for B in (1, 2, 3, 8, 14, 16, 31, 32, 33, 64, 65, 100, 300, 1100, 5000):
        last = 0
        for T in lengths:
            now = size(B, T)
            assert now >= last, (B, T)
            last = now
    counts = sorted({*range(1, 70), *range(70, 1300, 13), 2000, 5000, 8000})
    for T in (0, 1, 77, 129, 300, 2000, 2100, 4096, 4103, 8191, 12800, 30026, 32845, 200000):
        last = 0
        for B in counts:
            now = size(B, T)
            assert now >= last, (B, T)
            last = now


def test_sizes_that_fell():
    for heads, larger, smaller in (((16, 16, 128, 128), (1, 4103), (1, 4096)), ((16, 16, 128, 128), (8, 32845), (8, 32838)),
                                   ((32, 32, 128, 128), (16, 32768), (14, 30026))):
        assert gdn.lin_attn_prefill_workspace_bytes(*larger, *heads) >= gdn.lin_attn_prefill_workspace_bytes(
            *smaller, *heads)


@pytest.mark.parametrize("heads", HEADS)
def test_less_than_the_size_is_refused(heads):
    x = Heads(FAKE, 1 << 15, 128)
    for B, T in ((1, 4096), (3, 129), (40, 3000)):
        need = gdn.lin_attn_prefill_workspace_bytes(B, T, *heads)
        d = linear.LinDims(B, T, *heads, 9, 1)
        r = ctypes.byref(x)
        assert gdn.lib().lin_attn_prefill(ctypes.byref(d), r, r, r, FAKE, FAKE, FAKE, FAKE, FAKE, r, 1.0, FAKE,
                                          need - 1, None) == SHAPE
