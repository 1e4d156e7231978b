"""GPU: paged attention at the edges of its sizes."""
import pytest
import torch

from tests import attn_helpers as A
from tests import attn_norms as N

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


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [6, 90])
def test_unusable_sequences_of_many_rows_among_single_tokens(gdn, d, kind, B):
    """Sequences longer than max_new (NaN) and padding sequences of any length (zeros), in the kernel of few rows:
    one row more and less than the 128 that a workgroup fills at a time, and many times that."""
    long = [31, 32, 33, 64, 65, 1100]
    lens = [(long[i % 6], 5) if i % 2 else (1, 40 + (97 * i) % 1500) for i in range(B)]
    c = A.Cache(lens, H_q=8, H_kv=2, d=d, page=16, kind=kind, seed=37)
    row = c.row.clone()
    row[1::4] = 0
    q = torch.cat([c.q.cuda(), torch.zeros(3, 8, d, dtype=A.BF, device="cuda")])
    out, lse = torch.full_like(q, 7.0), torch.full((c.T + 3, 8), 7.0, device="cuda")
    a = c.cuda(row=row)
    ws = torch.empty(gdn.attn_paged_workspace_bytes(B, c.T + 3, 1, 8, 2, d), dtype=torch.uint8, device="cuda")
    gdn.attn_paged(q, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"], a["cu_seqlens"], out, ws,
                   max_new=1, lse=lse, k_scale=a["k_scale"], v_scale=a["v_scale"])
    torch.cuda.synchronize()
    want, want_lse, tol, tol_l = N.attention(c, d ** -0.5, 0, "cuda")
    out, lse = out.cpu(), lse.cpu()
    for b in range(B):
        t = slice(int(c.cu[b]), int(c.cu[b + 1]))
        if row[b] == 0:
            assert (out[t] == 0).all() and (lse[t] == -torch.inf).all(), b
        elif b % 2:
            assert out[t].isnan().all() and lse[t].isnan().all(), b
        else:
            N.check_norms(out[t], want[t], tol[t], f"sequence {b}")
            A.check(lse[t], want_lse[t], tol_l[t], f"sequence {b}")
    assert (out[c.T:] == 7).all() and (lse[c.T:] == 7).all()
