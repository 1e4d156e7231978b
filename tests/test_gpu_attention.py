"""GPU: paged attention (attn_paged, through the binding) against 64-bit
references: lengths around every block and page border, head groups, masks,
strides, padding, unusable inputs, streams and captured graphs."""
import math

import pytest
import torch

from tests import attn_helpers as A

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_recurrent_decode_amd as m
    m.lib()
    return m


def run(gdn, c, *, window=0, scale=None, max_new=None, q=None, out=None, lse=True, stream=None, ws=None, **over):
    max_new = max([n for n, _ in c.lens] + [1]) if max_new is None else max_new
    q = c.q.cuda() if q is None else q
    out = torch.full((c.T, c.H_q, c.d), 7.0, dtype=A.BF, device="cuda") if out is None else out
    L = torch.full((c.T, c.H_q), 7.0, device="cuda") if lse else None
    if ws is None:
        ws = torch.full((gdn.attn_paged_workspace_bytes(c.B, c.T, max_new, c.H_q, c.H_kv, c.d),), 0xFF,
                        dtype=torch.uint8, device="cuda")
    a = c.cuda(**over)
    gdn.attn_paged(q, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"], a["cu_seqlens"], out, ws,
                   max_new=max_new, scale=scale, window=window, lse=L, k_scale=a["k_scale"], v_scale=a["v_scale"],
                   stream=stream)
    torch.cuda.synchronize()
    return out, L


def both(gdn, c, window=0, **kw):
    out, lse = run(gdn, c, window=window, **kw)
    o, l, tol, tol_l = A.attention(c, c.d ** -0.5, window)
    A.check(out, o, tol, "out")
    A.check(lse, l, tol_l, "lse")
    return out, lse


BORDERS = [(1, p) for p in (0, 1, 14, 15, 16, 30, 31, 32, 63, 64, 126, 127, 128, 255, 300)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens_at_every_border(gdn, d, kind, page):
    both(gdn, A.Cache(BORDERS, H_q=4, H_kv=2, d=d, page=page, kind=kind, seed=d + page))


@pytest.mark.parametrize("G", [1, 3, 5, 8, 16, 20])
def test_head_groups(gdn, G):
    both(gdn, A.Cache([(1, 70), (2, 40), (5, 0)], H_q=2 * G, H_kv=2, d=128, page=32, seed=G))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 17, 100])
def test_ragged_chunks(gdn, d, kind, window):
    c = A.Cache([(70, 0), (1, 300), (0, 5), (33, 64), (4, 130), (129, 77), (16, 16)], H_q=6, H_kv=2, d=d, page=32,
                kind=kind, seed=window)
    both(gdn, c, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_long_context_is_cut_and_joined(gdn, d, kind):
    # one sequence over every workgroup, and a short one beside it
    both(gdn, A.Cache([(1, 20011), (1, 9)], H_q=4, H_kv=1, d=d, page=64, kind=kind, seed=5))


def test_chunk_behind_a_long_context(gdn):
    both(gdn, A.Cache([(257, 3000)], H_q=4, H_kv=1, d=128, page=64, seed=6))


def test_many_sequences(gdn):
    # more than one round of the scan over sequences, some empty
    lens = [((i * 7) % 3, (i * 37) % 150) for i in range(601)]
    both(gdn, A.Cache(lens, H_q=2, H_kv=1, d=64, page=16, seed=8))


@pytest.mark.parametrize("B", [2, 63, 64, 65, 255, 256, 257, 513])
def test_sequences_around_every_round_of_the_search(gdn, B):
    lens = [((i * 5) % 4 > 0, (i * 29) % 300) for i in range(B - 1)] + [(1, 700)]
    both(gdn, A.Cache([(int(n), p) for n, p in lens], H_q=2, H_kv=2, d=64, page=16, seed=B))


@pytest.mark.parametrize("B", [70, 1023, 1024, 1025])
def test_many_short_chunks(gdn, B):
    # more than one round of the plan over sequences, some of them empty
    lens = [((i * 3) % 7, (i * 37) % 60) for i in range(B - 1)] + [(70, 30)]
    both(gdn, A.Cache(lens, H_q=4, H_kv=1, d=64, page=16, seed=B))


def test_large_scores_and_a_dominant_key(gdn):
    c = A.Cache([(3, 200)], H_q=4, H_kv=2, d=128, page=16, seed=9, q_scale=30.0)
    both(gdn, c)


def test_strided_queries_and_outputs(gdn):
    c = A.Cache([(3, 50), (1, 20)], H_q=6, H_kv=2, d=64, page=16, seed=10)
    wide = torch.full((c.T, 6, 3 * 64), 5.0, dtype=A.BF, device="cuda")
    wide[:, :, 64:128] = c.q.cuda()
    target = torch.full((c.T, 8, 2 * 64), 7.0, dtype=A.BF, device="cuda")
    before = target.clone()
    out, _ = run(gdn, c, q=wide[:, :, 64:128], out=target[:, 1:7, 64:])
    o, _, tol, _ = A.attention(c, 64 ** -0.5)
    A.check(target[:, 1:7, 64:], o, tol, "out")
    target[:, 1:7, 64:] = 7.0
    assert torch.equal(target, before), "written outside the output's heads"
    run(gdn, c, lse=False)


def test_rows_that_see_nothing(gdn):
    # fewer cached tokens than new ones: the first tokens see no position
    c = A.Cache([(6, 0), (2, 4)], H_q=4, H_kv=2, d=64, page=16, seed=11)
    c.kv_len[int(c.row[0])] = 4
    out, lse = both(gdn, c)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    c.kv_len[int(c.row[0])] = 0
    both(gdn, c)


def test_padding_and_unusable_sequences(gdn):
    lens = [(1, 40), (2, 30), (1, 20), (3, 10), (1, 50), (2, 60)]
    c = A.Cache(lens, H_q=4, H_kv=2, d=64, page=16, seed=12)
    want, want_lse, tol, tol_l = A.attention(c, 64 ** -0.5)
    row, table, kv_len = c.row.clone(), c.table.clone(), c.kv_len.clone()
    row[0] = 0                                     # padding
    row[1] = c.R                                   # outside the table
    kv_len[int(row[2])] = c.width * c.page + 1     # longer than the table
    table[int(row[4]), 1] = c.N                    # a page outside the pool
    table[int(row[5]), 0] = 0                      # no page, seen by both tokens
    out, lse = run(gdn, c, row=row, page_table=table, kv_len=kv_len, max_new=2)  # sequence 3 has more tokens
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    for t in (1, 2, 3, 4, 5, 6, 7, 8, 9):
        assert out[t].isnan().all() and lse[t].isnan().all(), t
    # the same without what is unusable
    out, lse = run(gdn, c)
    A.check(out, want, tol, "out")


def test_a_bad_page_behind_the_window_or_later_does_not_show(gdn):
    c = A.Cache([(20, 60)], H_q=2, H_kv=1, d=64, page=16, seed=13)
    table = c.table.clone()
    table[int(c.row[0]), 0] = -5     # positions 0..15
    table[int(c.row[0]), 4] = c.N    # positions 64..79
    out, lse = run(gdn, c, window=20, page_table=table)
    want, _, tol, _ = A.attention(c, 64 ** -0.5, 20)
    # token i stands at 60 + i and sees 41 + i .. 60 + i: the first four miss position 64
    A.check(out[:4], want[:4], tol[:4], "out")
    assert out[4:].isnan().all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("last", [1, 5, 12, 16])
@pytest.mark.parametrize("n", [4, 40])
def test_a_bad_last_page_of_few_cells(gdn, d, kind, last, n):
    """A page outside the pool that holds only the last few keys: the tokens that see it get NaN, no other."""
    c = A.Cache([(n, 96 + last - n)], H_q=8, H_kv=2, d=d, page=16, kind=kind, seed=30)
    table = c.table.clone()
    table[int(c.row[0]), 6] = c.N
    out, lse = run(gdn, c, page_table=table, max_new=40)
    see = min(n, last)
    assert out[n - see:].isnan().all() and lse[n - see:].isnan().all()
    want, want_lse, tol, tol_l = A.attention(c, d ** -0.5)
    A.check(out[:n - see], want[:n - see], tol[:n - see], "out")
    A.check(lse[:n - see], want_lse[:n - see], tol_l[:n - see], "lse")


def test_rows_outside_the_sequences_stay(gdn):
    c = A.Cache([(2, 40), (3, 30)], H_q=4, H_kv=2, d=64, page=16, seed=14)
    cu = c.cu + 4
    q = torch.zeros(c.T + 9, 4, 64, dtype=A.BF, device="cuda")
    q[4:4 + c.T] = c.q.cuda()
    out = torch.full_like(q, 7.0)
    big = A.Cache([(2, 40), (3, 30)], H_q=4, H_kv=2, d=64, page=16, seed=14)
    big.T = c.T + 9
    got, lse = run(gdn, big, q=q, out=out, cu_seqlens=cu)
    want, _, tol, _ = A.attention(c, 64 ** -0.5)
    A.check(got[4:4 + c.T], want, tol, "out")
    assert (got[:4] == 7).all() and (got[4 + c.T:] == 7).all()
    assert (lse[:4] == 7).all() and (lse[4 + c.T:] == 7).all()
    # a sequence whose range leaves the packed tokens
    cu2 = cu.clone()
    cu2[2] = big.T + 1
    got, _ = run(gdn, big, q=q, cu_seqlens=cu2)
    A.check(got[4:6], want[:2], tol[:2], "out")
    assert (got[6:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [6, 150])
def test_a_later_tokens_nan_stays_its_own(gdn, kind, bad, n):
    if kind == "e4m3" and math.isinf(bad):
        pytest.skip("e4m3 has no infinity")
    c = A.Cache([(n, 40)], H_q=4, H_kv=2, d=128, page=16, kind=kind, seed=15)
    r = int(c.row[0])
    for pos, col in ((42, 3), (40 + n - 1, 77)):
        c.v[int(c.table[r, pos // 16]), :, pos % 16, col] = bad
    c.k[int(c.table[r, (40 + n - 2) // 16]), 1, (40 + n - 2) % 16] = math.nan
    for window in (0, 16):
        out, lse = run(gdn, c, window=window)
        want, want_lse, tol, tol_l = A.attention(c, 128 ** -0.5, window)
        # a NaN among the keys makes every output of the tokens that see it NaN
        A.check(out[:, :2], want[:, :2], tol[:, :2], "out")
        A.check(out[:n - 2, 2:], want[:n - 2, 2:], tol[:n - 2, 2:], "out")
        assert out[n - 2:, 2:].isnan().all() and lse[n - 2:, 2:].isnan().all()


def test_the_same_bits_again_in_any_workspace_and_stream(gdn):
    c = A.Cache([(1, 5000), (40, 700), (1, 3)], H_q=8, H_kv=2, d=128, page=32, seed=16)
    first, lse = run(gdn, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, lse2 = run(gdn, c, stream=side)
    assert torch.equal(first.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    # a larger call between them leaves its parts in the workspace
    ws = torch.empty(gdn.attn_paged_workspace_bytes(1, 1, 64, 8, 2, 128), dtype=torch.uint8, device="cuda")
    run(gdn, A.Cache([(1, 30000)], H_q=8, H_kv=2, d=128, page=32, seed=17), ws=ws, max_new=64)
    again, _ = run(gdn, c, ws=ws, max_new=64)
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_the_order_of_the_sequences_does_not_matter(gdn):
    c = A.Cache([(1, 500), (4, 700), (1, 3), (9, 90)], H_q=8, H_kv=2, d=64, page=32, seed=18)
    both(gdn, c)
    order = [2, 0, 3, 1]
    e = A.Cache([c.lens[i] for i in order], H_q=8, H_kv=2, d=64, page=32, seed=18)
    e.k, e.v, e.table, e.kv_len, e.N, e.R, e.width = c.k, c.v, c.table, c.kv_len, c.N, c.R, c.width
    e.row = c.row[order]
    e.q = torch.cat([c.q[int(c.cu[i]):int(c.cu[i + 1])] for i in order])
    both(gdn, e)


def test_a_captured_step_follows_its_lengths(gdn):
    """One graph, replayed while the rows grow, a row turns to padding and pages move."""
    lens = [(1, 30), (1, 140), (1, 900), (1, 0)]
    c = A.Cache(lens, H_q=8, H_kv=2, d=128, page=16, seed=19, width=70)
    a = c.cuda()
    q, out = c.q.cuda(), torch.empty(c.T, 8, 128, dtype=A.BF, device="cuda")
    lse = torch.empty(c.T, 8, device="cuda")
    ws = torch.empty(gdn.attn_paged_workspace_bytes(c.B, c.T, 1, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def call():
        gdn.attn_paged(q, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"], a["cu_seqlens"], out,
                       ws, max_new=1, lse=lse)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(4):
        m = A.Cache([(1, p + 37 * step) for _, p in lens], H_q=8, H_kv=2, d=128, page=16, seed=20 + step, spare=3,
                    width=70)
        pool = min(m.N, c.N) if m.N > c.N else m.N
        if m.N > c.N:  # the captured pool is as large as the first one: keep to its pages
            m = A.Cache([(1, max(0, p - 16 * step)) for _, p in lens], H_q=8, H_kv=2, d=128, page=16,
                        seed=20 + step, spare=3, width=70)
            pool = m.N
        for name, x in (("k_pages", m.k), ("v_pages", m.v)):
            a[name][:pool].copy_(x)
        a["page_table"].copy_(m.table)
        a["kv_len"].copy_(m.kv_len)
        a["row"].copy_(m.row)
        q.copy_(m.q)
        if step == 2:
            a["row"][1] = 0
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse, tol, tol_l = A.attention(m, 128 ** -0.5)
        if step == 2:
            want[1], want_lse[1] = 0, -math.inf
        A.check(out, want, tol, f"replay {step}")
        A.check(lse, want_lse, tol_l, f"replay {step}")
        call()
        eager = out.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("n", [40, 100])
@pytest.mark.parametrize("d", [64, 256])
def test_chunks_that_see_nothing(gdn, d, n):
    # more new tokens than cached ones, in the kernel of long chunks
    c = A.Cache([(n, 0), (70, 0)], H_q=8, H_kv=2, d=d, page=16, seed=22)
    c.kv_len[int(c.row[0])] = n - 33
    out, lse = both(gdn, c, max_new=100)
    assert (out[:33] == 0).all() and (lse[:33] == -math.inf).all()
    c.kv_len[int(c.row[0])] = 0
    both(gdn, c, max_new=100)


@pytest.mark.parametrize("max_new", [0, 3, 99])
def test_more_new_tokens_than_said(gdn, max_new):
    c = A.Cache([(100, 20), (2, 50)], H_q=8, H_kv=2, d=64, page=16, seed=23)
    out, lse = run(gdn, c, max_new=max_new)
    assert out[:100].isnan().all() and lse[:100].isnan().all()
    want, _, tol, _ = A.attention(c, 64 ** -0.5)
    if max_new:
        A.check(out[100:], want[100:], tol[100:], "out")
    else:
        assert out[100:].isnan().all()


def test_unusable_sequences_among_chunks(gdn):
    lens = [(100, 40), (80, 30), (90, 20), (300, 10), (60, 60)]
    c = A.Cache(lens, H_q=4, H_kv=2, d=128, page=16, seed=24)
    want, want_lse, tol, tol_l = A.attention(c, 128 ** -0.5)
    row, table, kv_len = c.row.clone(), c.table.clone(), c.kv_len.clone()
    row[0] = 0
    row[1] = -3
    kv_len[int(row[2])] = -1
    table[int(row[4]), 5] = c.N + 7    # positions 80..95: seen by the tokens from 20 on
    out, lse = run(gdn, c, row=row, page_table=table, kv_len=kv_len)
    assert (out[:100] == 0).all() and (lse[:100] == -math.inf).all()
    assert out[100:270].isnan().all() and lse[100:270].isnan().all()
    A.check(out[270:590], want[270:590], tol[270:590], "out")
    A.check(lse[270:590], want_lse[270:590], tol_l[270:590], "lse")
    assert out[590:].isnan().all() and lse[590:].isnan().all()


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.02])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 90])
def test_other_scales(gdn, scale, kind, n):
    c = A.Cache([(n, 77)], H_q=4, H_kv=2, d=128, page=32, kind=kind, seed=25)
    out, lse = run(gdn, c, scale=scale)
    o, l, tol, tol_l = A.attention(c, scale)
    A.check(out, o, tol, "out")
    A.check(lse, l, tol_l, "lse")


def test_overlapping_sequences_touch_nothing_else(gdn):
    """Ranges that overlap break the precondition; the workspace, sized for ranges that do not, is not overrun."""
    c = A.Cache([(300, 0)] * 3, H_q=8, H_kv=2, d=64, page=16, seed=26)
    cu = torch.tensor([0, 300, 10, 300], dtype=torch.int32)
    c.T, c.q = 300, c.q[:300]
    need = gdn.attn_paged_workspace_bytes(3, 300, 300, 8, 2, 64)
    big = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = run(gdn, c, cu_seqlens=cu, ws=big[:need], max_new=300)
    assert (big[need:] == 0x5A).all()


@pytest.mark.parametrize("n", [3, 60])
def test_pages_past_four_gigabytes(gdn, n):
    """Cells whose byte offsets pass 32 bits: a 5 GiB pool with the sequence at its top."""
    d, H_kv, page = 256, 2, 256
    N = (5 << 30) // (H_kv * page * d * 2)
    c = A.Cache([(n, 700)], H_q=8, H_kv=H_kv, d=d, page=page, seed=21)
    k = torch.zeros(N, H_kv, page, d, dtype=A.BF, device="cuda")
    v = torch.zeros(N, H_kv, page, d, dtype=A.BF, device="cuda")
    up = N - c.N
    k[up:], v[up:] = c.k.cuda(), c.v.cuda()
    table = torch.where(c.table > 0, c.table + up, 0).to(torch.int32).cuda()
    q, out = c.q.cuda(), torch.empty(c.T, 8, d, dtype=A.BF, device="cuda")
    ws = torch.empty(gdn.attn_paged_workspace_bytes(1, c.T, n, 8, H_kv, d), dtype=torch.uint8, device="cuda")
    a = table, c.kv_len.cuda(), c.row.cuda(), c.cu.cuda()
    gdn.attn_paged(q, k, v, *a, out, ws, max_new=n)
    want, _, tol, _ = A.attention(c, d ** -0.5)
    A.check(out, want, tol, "out")
    # the prologue writes there, and pages move there
    x = torch.randn(c.T, H_kv, d, device="cuda").to(A.BF)
    gdn.attn_prologue(None, x, x, None, k, v, *a, None)
    at = (table[int(c.row[0]), 700 // page].item(), 700 % page)
    assert torch.equal(k[at[0], :, at[1]], x[0]) and torch.equal(v[at[0], :, at[1]], x[0])
    i32 = dict(dtype=torch.int32, device="cuda")
    gdn.kv_page_copy(k, v, torch.tensor([at[0]], **i32), torch.tensor([N - c.N - 2], **i32))
    torch.cuda.synchronize()
    assert torch.equal(k[N - c.N - 2].view(torch.int16), k[at[0]].view(torch.int16))
    assert not k[:N - c.N - 2].any()


@pytest.mark.parametrize("n", [5, 300])
def test_a_window_longer_than_any_context(gdn, n):
    """The largest windows see what no window sees, also where the first tokens stand before position 0."""
    c = A.Cache([(n, 0), (1, 40)], H_q=8, H_kv=2, d=64, page=16, seed=27)
    c.kv_len[int(c.row[0])] = n - 3
    want, want_lse = both(gdn, c)
    for window in (c.width * c.page, 2 ** 30, 2 ** 31 - 1):
        out, lse = run(gdn, c, window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), window


def test_two_calls_at_once(gdn):
    """Calls on two streams with a workspace each, of both kernels, do not disturb one another."""
    cases = [A.Cache([(1, 3000)] * 4, H_q=8, H_kv=2, d=128, page=16, seed=28),
             A.Cache([(200, 700)], H_q=8, H_kv=2, d=128, page=16, seed=29)]
    want = [run(gdn, c) for c in cases]
    calls = []
    for c in cases:
        most = max(n for n, _ in c.lens)
        ws = torch.empty(gdn.attn_paged_workspace_bytes(c.B, c.T, most, 8, 2, 128), dtype=torch.uint8, device="cuda")
        calls.append((c.cuda(), c.q.cuda(), torch.zeros(c.T, 8, 128, dtype=A.BF, device="cuda"), ws, most))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(8):
        for (a, q, out, ws, most), s in zip(calls, streams):
            gdn.attn_paged(q, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"], a["cu_seqlens"],
                           out, ws, max_new=most, stream=s)
    torch.cuda.synchronize()
    for (_, _, out, _, _), (o, _) in zip(calls, want):
        assert torch.equal(out, o)
