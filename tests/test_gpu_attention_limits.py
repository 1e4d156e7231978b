"""GPU: paged attention at the edges of its sizes."""
import pytest
import torch

from tests import attn_helpers as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_recurrent_decode_amd as m
    m.lib()
    return m


def test_overlapping_ranges_of_more_tiles_than_32_bits_count(gdn):
    """Every second range holds all tokens (cu_seqlens 0, T, 0, T, ...): 512 x 2^22 entries in the plan's first round,
    2^31, which a 32-bit sum takes for a negative number.  Nothing outside the workspace is written, and the
    padding row's zeros come out.  All tokens and heads are one place in memory, so that they fit."""
    T, H, d, B = 2 ** 24 - 1, 64, 64, 1024
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(1, 1, d, dtype=A.BF, device="cuda").expand(T, H, d)
    out = torch.full((1, 1, d), 7.0, dtype=A.BF, device="cuda")
    cu = torch.tensor([0, T] * (B // 2) + [0], **i32)
    pages = torch.zeros(2, H, 16, d, dtype=A.BF, device="cuda")
    need = gdn.attn_paged_workspace_bytes(B, T, T, H, H, d)
    big = torch.full((need + 2 * 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    gdn.attn_paged(q, pages, pages, torch.zeros(2, 1, **i32), torch.zeros(2, **i32), torch.zeros(B, **i32), cu,
                   out.expand(T, H, d), big[4096:4096 + need], max_new=T)
    torch.cuda.synchronize()
    assert (big[:4096] == 0x5A).all() and (big[4096 + need:] == 0x5A).all()
    assert (out == 0).all()
