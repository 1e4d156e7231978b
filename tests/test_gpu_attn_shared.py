"""GPU: attn_shared against attention in 64 bits over each sequence's own row (attn_helpers.py has the reference and
derives the bound: weights rounded to bf16 once, o once)."""
import math

import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from tests import attn_helpers as H

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Forked(H.Cache):
    """groups: (common positions, [(new tokens, own tokens before them)] of its members) each.  Whole common pages
    are the first member's for all, the page that is partly common is a copy (as kv_page_fork leaves them)."""

    def __init__(self, groups, **kw):
        super().__init__([(n, common + own) for common, members in groups for n, own in members], **kw)
        b, self.groups, self.shared = 0, [0], [common for common, _ in groups]
        for common, members in groups:
            for i in range(b + 1, b + len(members)):
                whole, part = common // self.page, common % self.page
                a, r = self.table[int(self.row[b])], self.table[int(self.row[i])]
                r[:whole] = a[:whole]
                if part:
                    for pages in (self.k, self.v):
                        raw = pages.view(torch.uint8)
                        raw[int(r[whole]), :, :part] = raw[int(a[whole]), :, :part]
            b += len(members)
            self.groups.append(b)

    def own(self, which, b, t):
        """(page, offset) of position t of sequence b."""
        return int(self.table[int(self.row[b])][t // self.page]), t % self.page


def run(c, *, window=0, groups=None, shared=None, max_new=None, least=16, **over):
    t = c.cuda(**over)
    K = len(c.groups) - 1 if groups is None else len(groups) - 1
    out = torch.full((c.T, c.H_q, c.d), 7.0, dtype=H.BF, device="cuda")
    lse = torch.full((c.T, c.H_q), 7.0, device="cuda")
    max_new = max(n for n, _ in c.lens) if max_new is None else max_new
    ws = torch.full((gdn.attn_shared_workspace_bytes(c.B, c.T, K, max_new, c.H_q, c.H_kv, c.d),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    gdn.attn_shared(c.q.cuda(), t.pop("k_pages"), t.pop("v_pages"), t.pop("page_table"), t.pop("kv_len"),
                    t.pop("row"), t.pop("cu_seqlens"), i32(c.groups if groups is None else groups),
                    i32(c.shared if shared is None else shared), out, ws, max_new=max_new, window=window,
                    least=least, lse=lse, **t)
    torch.cuda.synchronize()
    return out, lse


def check(c, out, lse, window=0, tokens=slice(None)):
    o, l, tol, tol_l = H.attention(c, c.d ** -0.5, window)
    H.check(out[tokens], o[tokens], tol[tokens], "o")
    H.check(lse[tokens], l[tokens], tol_l[tokens], "lse")


@pytest.mark.parametrize("d,H_q,H_kv", [(64, 4, 2), (128, 8, 1), (256, 4, 2), (128, 5, 1)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(d, H_q, H_kv, kind, page):
    c = Forked([(300, [(1, 5), (1, 0), (1, 130)]), (1000, [(1, 3), (1, 17)]), (40, [(1, 1), (1, 2)]), (200, [(1, 9)])],
               H_q=H_q, H_kv=H_kv, d=d, page=page, kind=kind, seed=d + page)
    check(c, *run(c))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prefix_many_rows(d):
    # several tiles of rows a group, many pieces a tile
    c = Forked([(3001, [(1, i * 7 % 90) for i in range(70)])], H_q=8, H_kv=1, d=d, page=32, seed=1, q_scale=2.0)
    check(c, *run(c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_chunks(d, kind):
    # prompt chunks beside single tokens: own keys of several tiles, causal within
    c = Forked([(700, [(150, 20), (1, 200), (90, 0)]), (333, [(2, 1), (300, 40)])], H_q=4, H_kv=2, d=d, page=64, kind=kind,
               seed=2)
    check(c, *run(c))


@pytest.mark.parametrize("window", [1, 60, 290, 450, 700, 5000])
def test_windows(window):
    # windows that end in the own keys, inside the common ones at another place for each member, before them
    c = Forked([(400, [(1, 10), (30, 100), (1, 300), (5, 0)]), (600, [(1, 2), (70, 3)])], H_q=4, H_kv=2, d=64, page=32,
               seed=3)
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("shared", [[0, 0], [-5, 77], [127, 128], [129, 433], [10 ** 6, 2 ** 31 - 1], [400, 15], [399, 500]])
def test_any_shared_length(shared):
    # shorter than what is common, and longer than what a member has before its new tokens (those agree up to there)
    c = Forked([(400, [(1, 0), (3, 0), (1, 0)]), (500, [(2, 0), (4, 0)])], H_q=4, H_kv=2, d=64, page=16, seed=4)
    check(c, *run(c, shared=shared))


def test_groups_of_none_and_sequences_of_no_group():
    c = Forked([(300, [(1, 4), (1, 5)]), (0, [(2, 200)]), (256, [(1, 8), (1, 9), (1, 7)])], H_q=4, H_kv=1, d=64, page=16,
               seed=5)
    check(c, *run(c, groups=[0, 2, 2, 2, 3, 6], shared=[300, 99, 5, 100, 256]))
    check(c, *run(c, groups=[3, 6], shared=[256]))   # the first three are in no group
    check(c, *run(c, groups=[0, 2], shared=[300]))   # the last four
    check(c, *run(c, groups=[0], shared=[]))         # nobody
    # bounds outside [0, B] count as its ends
    check(c, *run(c, groups=[-4, 2, 3, 99], shared=[300, 7, 256]))


def test_unusable_members():
    c = Forked([(300, [(1, 4), (2, 5), (1, 9), (1, 3), (1, 2)])], H_q=4, H_kv=2, d=64, page=16, seed=6)
    rows = c.row.clone()
    want = H.attention(c, c.d ** -0.5)
    for bad, value in ((0, 0), (0, -1), (3, 0), (3, c.R), (1, 99)):
        row = rows.clone()
        row[bad] = value
        out, lse = run(c, row=row)
        a, e = int(c.cu[bad]), int(c.cu[bad + 1])
        if value == 0:
            assert bool((out[a:e] == 0).all()) and bool((lse[a:e] == -math.inf).all())
        else:
            assert bool(out[a:e].isnan().all()) and bool(lse[a:e].isnan().all())
        keep = torch.ones(c.T, dtype=torch.bool)
        keep[a:e] = False
        H.check(out[keep.cuda()], want[0][keep], want[2][keep], f"o beside row {value} at {bad}")
    # one member with more new tokens than max_new, one whose length is too short for its new tokens
    out, lse = run(c, max_new=1)
    assert bool(out[1:3].isnan().all()) and bool(out[0].isfinite().all()) and bool(out[3:].isfinite().all())
    lens = c.kv_len.clone()
    lens[int(rows[1])] = 1
    out, lse = run(c, kv_len=lens)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all()) and bool(out[2].isfinite().all())
    H.check(out[3:], want[0][3:], want[2][3:], "o")


def test_common_positions_are_read_through_the_first_usable_member():
    c = Forked([(320, [(1, 4), (1, 5), (1, 9)])], H_q=4, H_kv=2, d=64, page=16, seed=7)
    table = c.table.clone()
    for b in (1, 2):  # 20 whole pages in common
        table[int(c.row[b]), :20] = torch.tensor([-7, 10 ** 6] * 10, dtype=torch.int32)
    check(c, *run(c, page_table=table))
    table = c.table.clone()  # a page of the first member outside the pool: all read through it
    table[int(c.row[0]), 3] = c.N
    out, lse = run(c, page_table=table)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    table = c.table.clone()  # a member's own page: that one alone
    table[int(c.row[2]), 20] = 0
    out, lse = run(c, page_table=table)
    assert bool(out[2].isnan().all())
    check(c, out, lse, tokens=slice(0, 2))


def test_infinities_and_nan_in_places_that_are_not_seen():
    c = Forked([(400, [(1, 10), (40, 100), (1, 300)])], H_q=4, H_kv=2, d=64, page=32, seed=8)
    p, o = c.own("v", 0, 100)
    c.v[p, 0, o, 3], c.v[p, 1, o, 5] = math.inf, math.nan
    p, o = c.own("v", 1, 400 + 100 + 20)  # a new token's own value: earlier ones of its chunk do not see it
    c.v[p, 0, o, 9] = -math.inf
    check(c, *run(c))
    window = 330  # position 100 is out of the second member's and the third's windows
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("B", [65, 1500])
def test_many_sequences(B):
    gen = torch.Generator().manual_seed(B)
    own = torch.randint(0, 20, (B,), generator=gen).tolist()
    cut = B // 3
    c = Forked([(150, [(1, x) for x in own[:cut]]), (128, [(1, x) for x in own[cut:cut + 5]]),
                (144, [(1, x) for x in own[cut + 5:]])], H_q=2, H_kv=1, d=64, page=16, seed=9)
    check(c, *run(c))


def test_as_attn_paged_and_the_same_bits_again():
    c = Forked([(2000, [(1, 3), (1, 77), (4, 200)]), (500, [(1, 8), (1, 9)])], H_q=8, H_kv=2, d=128, page=64, seed=10)
    out, lse = run(c)
    t = c.cuda()
    paged, plse = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(gdn.attn_paged_workspace_bytes(c.B, c.T, 4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    gdn.attn_paged(c.q.cuda(), t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"], t["row"], t["cu_seqlens"],
                   paged, ws, max_new=4, lse=plse)
    _, _, tol, tol_l = H.attention(c, c.d ** -0.5)
    H.check(out, paged.double().cpu(), 2 * tol, "o against attn_paged")
    H.check(lse, plse.double().cpu(), 2 * tol_l, "lse against attn_paged")
    for _ in range(2):
        again, _ = run(c)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_captured_and_replayed_with_other_lengths_on_another_stream():
    c = Forked([(640, [(1, 30), (2, 60), (1, 90)])], H_q=4, H_kv=2, d=64, page=32, seed=11)
    t = c.cuda()
    q, groups, shared = c.q.cuda(), i32(c.groups), i32(c.shared)
    out = torch.zeros(c.T, c.H_q, c.d, dtype=H.BF, device="cuda")
    ws = torch.empty(gdn.attn_shared_workspace_bytes(c.B, c.T, 1, 2, 4, 2, 64), dtype=torch.uint8, device="cuda")

    def call():
        gdn.attn_shared(q, t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"], t["row"], t["cu_seqlens"], groups,
                        shared, out, ws, max_new=2, least=16)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    lse = torch.zeros(0)
    H.check(out, H.attention(c, 0.125)[0], H.attention(c, 0.125)[2], "o on another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cutoff, own in ((640, 30), (304, 12), (0, 3)):
        shared[0] = cutoff
        c.kv_len[int(c.row[0])] = 640 + own + 1
        t["kv_len"].copy_(c.kv_len)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        o, _, tol, _ = H.attention(c, 0.125)
        H.check(out, o, tol, f"o of the replay at {cutoff}, {own}")


def test_which_groups_are_read_together():
    # a group that is read together is read through its first member's row: the other rows' entries for the common
    # keys may then name no page at all
    c = Forked([(2048, [(1, i % 40) for i in range(64)]), (48, [(1, 5), (1, 9)])], H_q=4, H_kv=2, d=64, page=64, seed=13)
    table = c.table.clone()
    for i in range(1, 64):
        table[int(c.row[i]), :2048 // 64] = 0
    o, l, tol, tol_l = H.attention(c, c.d ** -0.5)
    for least in (None, 2048, 100):
        out, lse = run(c, least=least, page_table=table.cuda())
        H.check(out, o, tol, f"o from {least} keys on")
        H.check(lse, l, tol_l, f"lse from {least} keys on")
    out, lse = run(c, least=2049, page_table=table.cuda())
    assert bool(out[1:64].isnan().all()) and bool(lse[1:64].isnan().all())
    H.check(out[[0, 64, 65]], o[[0, 64, 65]], tol[[0, 64, 65]], "o of the rows with pages")
    check(c, *run(c, least=None, shared=[100, 48]))  # too little to save


@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_as_attn_paged_where_nothing_can_be_shared(d, kind):
    # short tables, or no groups: single tokens take the path of attn_paged, bit for bit
    c = Forked([(100, [(1, 3), (2, 40), (1, 0)]), (48, [(1, 9), (1, 5)])], H_q=8, H_kv=2, d=d, page=16, kind=kind, seed=15)
    out, lse = run(c, least=None)
    check(c, out, lse)
    t = c.cuda()
    paged, plse = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(gdn.attn_paged_workspace_bytes(c.B, c.T, 2, 8, 2, d), dtype=torch.uint8, device="cuda")
    gdn.attn_paged(c.q.cuda(), t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"], t["row"], t["cu_seqlens"],
                   paged, ws, max_new=2, lse=plse, k_scale=t["k_scale"], v_scale=t["v_scale"])
    nobody = run(c, groups=[0], shared=[])
    for o, l in ((out, lse), nobody):
        assert torch.equal(o.view(torch.int16), paged.view(torch.int16)) and torch.equal(l, plse)


def test_ranges_that_go_back():
    # the third sequence's tokens lie before the first's: its row by itself, and nobody's parts
    c = Forked([(640, [(2, 5), (2, 9), (2, 3), (2, 4)])], H_q=4, H_kv=2, d=64, page=16, seed=14)
    out, lse = run(c, cu_seqlens=torch.tensor([3, 5, 1, 3, 5], dtype=torch.int32))
    c.cu = torch.tensor([1, 1, 1, 3, 3], dtype=torch.int32)
    check(c, out, lse, tokens=slice(1, 3))
    assert bool((out[[0, 5, 6, 7]] == 7).all()) and bool((lse[[0, 5, 6, 7]] == 7).all())


def test_strided_heads():
    c = Forked([(300, [(1, 5), (3, 60)])], H_q=4, H_kv=2, d=64, page=16, seed=12)
    t = c.cuda()
    packed = torch.randn(c.T, 11 * 64, device="cuda").to(H.BF)
    q = packed[:, 128:128 + 256].unflatten(1, (4, 64))
    q.copy_(c.q)
    wide = torch.full((c.T, 8, 64), 7.0, dtype=H.BF, device="cuda")
    ws = torch.empty(gdn.attn_shared_workspace_bytes(c.B, c.T, 1, 3, 4, 2, 64), dtype=torch.uint8, device="cuda")
    gdn.attn_shared(q, t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"], t["row"], t["cu_seqlens"],
                    i32(c.groups), i32(c.shared), wide[:, ::2], ws, max_new=3, least=16)
    torch.cuda.synchronize()
    o, _, tol, _ = H.attention(c, 0.125)
    H.check(wide[:, ::2], o, tol, "o")
    assert bool((wide[:, 1::2] == 7).all())


def test_two_calls_at_once():
    # each on its own stream with its own workspace: the bits of one after the other
    caches = [Forked([(900, [(1, i * 5 % 60) for i in range(20)]), (300, [(1, 8), (1, 2)])], H_q=8, H_kv=2, d=d, page=32,
                     seed=16 + d) for d in (64, 128)]
    alone = [run(c) for c in caches]
    calls = []
    for c in caches:
        t, K = c.cuda(), len(c.groups) - 1
        out = torch.zeros(c.T, c.H_q, c.d, dtype=H.BF, device="cuda")
        ws = torch.empty(gdn.attn_shared_workspace_bytes(c.B, c.T, K, 1, c.H_q, c.H_kv, c.d), dtype=torch.uint8,
                         device="cuda")
        calls.append((c.q.cuda(), t, i32(c.groups), i32(c.shared), out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, t, groups, shared, out, ws, stream in calls:
            gdn.attn_shared(q, t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"], t["row"], t["cu_seqlens"],
                            groups, shared, out, ws, max_new=1, least=16, stream=stream)
    torch.cuda.synchronize()
    for (o, _), call in zip(alone, calls):
        assert torch.equal(o.view(torch.int16), call[4].view(torch.int16))
