"""GPU: the attention prologue (attn_prologue, through the binding) against a
64-bit reference: rotary layouts and widths, norms, cache types, far positions,
strides, padding and unusable tokens."""
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


def inputs(c, seed=0):
    g = torch.Generator().manual_seed(100 + seed)
    x = torch.randn(c.T, (c.H_q + 2 * c.H_kv) * c.d, generator=g).to(A.BF)
    return x


def split(c, x):
    q, k, v = x.split([c.H_q * c.d, c.H_kv * c.d, c.H_kv * c.d], 1)
    return tuple(t.unflatten(1, (-1, c.d)) for t in (q, k, v))


def cells(c, pages):
    """What the new tokens' cells hold, [T][H_kv][d]."""
    got = []
    for b in range(c.B):
        n, r = c.lens[b][0], int(c.row[b])
        for i in range(n):
            p = int(c.kv_len[r]) - n + i
            got.append(pages[int(c.table[r, p // c.page]), :, p % c.page])
    return torch.stack(got) if got else torch.empty(0, c.H_kv, c.d)


def rounded(want, fp32, kind, scale=None):
    """What a stored value may be off by: half a step of its type, and the fp32 work before it."""
    if kind == "bf16":
        return want, A.U_BF * want.abs() + 2 * fp32
    s = scale.double()[None, :, None]
    want, fp32 = (want / s).clamp(-448, 448), fp32 / s
    # below 2^-6 the steps of e4m3 are 2^-9 apart
    return want, torch.maximum(A.U_F8 * want.abs(), torch.tensor(2.0 ** -10)) + 2 * fp32 + 4 * A.U_32 * want.abs()


def run(gdn, c, x, freqs, **kw):
    a = c.cuda()
    xd = x.cuda()
    q, k, v = split(c, xd)
    out = torch.full((c.T, c.H_q, c.d), 7.0, dtype=A.BF, device="cuda")
    gdn.attn_prologue(q, k, v, out, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"],
                      a["cu_seqlens"], None if freqs is None else freqs.cuda(), k_scale=a["k_scale"],
                      v_scale=a["v_scale"], **kw)
    torch.cuda.synchronize()
    return out, a["k_pages"].cpu(), a["v_pages"].cpu()


def others_untouched(c, before, after):
    mine = torch.zeros(before.shape[:3], dtype=torch.bool)
    for b in range(c.B):
        n, r = c.lens[b][0], int(c.row[b])
        for i in range(n):
            p = int(c.kv_len[r]) - n + i
            mine[int(c.table[r, p // c.page]), :, p % c.page] = True
    bits = torch.int16 if before.dtype == A.BF else torch.uint8
    assert torch.equal(before.view(bits)[~mine], after.view(bits)[~mine]), "a cell of no new token changed"


LENS = [(1, 0), (3, 15), (1, 31), (0, 4), (20, 13), (2, 200)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 62), (128, 128), (128, 32), (128, 6), (256, 64), (256, 250), (64, 0)])
def test_layouts(gdn, d, rot, interleaved, kind):
    c = A.Cache(LENS, H_q=6, H_kv=2, d=d, page=16, kind=kind, seed=rot)
    x = inputs(c, rot)
    g = torch.Generator().manual_seed(5)
    wq, wk = (torch.randn(d, generator=g).to(A.BF) for _ in range(2))
    freqs = gdn.rope_freqs(rot, 10000.0, device="cpu")
    with_norm = rot % 4 == 0
    kw = dict(interleaved=interleaved)
    if with_norm:
        kw.update(q_norm=wq.cuda(), k_norm=wk.cuda(), norm_eps=1e-5, norm_add=0.5)
    out, kp, vp = run(gdn, c, x, freqs if rot else None, **kw)
    q, k, v = split(c, x)
    for name, head, got, w in (("q", q, out, wq), ("k", k, cells(c, kp), wk)):
        want, fp32 = A.prologue(c, head, freqs, interleaved=interleaved, weight=w if with_norm else None, eps=1e-5,
                                add=0.5)
        want, tol = rounded(want, fp32, "bf16" if name == "q" else kind, c.k_scale)
        A.check(got.float(), want, tol, name)
    want, tol = rounded(v.double(), 0.0 * v.double(), kind, c.v_scale)
    if kind == "bf16":
        assert torch.equal(cells(c, vp), v)
    A.check(cells(c, vp).float(), want, tol, "v")
    others_untouched(c, c.k, kp)
    others_untouched(c, c.v, vp)


@pytest.mark.parametrize("stretch", ["none", "linear", "base", "wavelength"])
def test_far_positions(gdn, stretch):
    """Positions near a million: an fp32 angle would be off by a tenth of a radian."""
    c = A.Cache([(5, 3)], H_q=4, H_kv=1, d=128, page=16, seed=1)
    freqs = gdn.rope_freqs(128, 1e6, stretch=stretch, factor=8.0, original=32768.0, low=1.0, high=32.0, device="cpu")
    at = torch.tensor([0, 1, 262143, 1000003, 2**30], dtype=torch.int32)
    x = inputs(c)
    out, kp, _ = run(gdn, c, x, freqs, positions=at.cuda(), rope_scale=1.25)
    q, k, _ = split(c, x)
    for head, got in ((q, out), (k, cells(c, kp))):
        want, fp32 = A.prologue(c, head, freqs, scale=1.25, positions=at)
        # at 2^30 the fp64 product itself is off by 2^30 2^-53 a radian at most: nothing
        want, tol = rounded(want, fp32, "bf16")
        A.check(got, want, tol, stretch)


def test_frequencies(gdn):
    f = gdn.rope_freqs(8, 100.0, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64), rtol=1e-15)


def test_queries_alone_in_place_and_keys_alone(gdn):
    c = A.Cache(LENS, H_q=6, H_kv=2, d=64, page=16, seed=3)
    x = inputs(c)
    freqs = gdn.rope_freqs(64, 10000.0, device="cpu")
    full, kp, vp = run(gdn, c, x, freqs)
    a = c.cuda()
    q, k, v = split(c, x.cuda())
    own = q.clone()
    gdn.attn_prologue(own, None, None, own, a["k_pages"], a["v_pages"], None, a["kv_len"], a["row"],
                      a["cu_seqlens"], freqs.cuda())
    gdn.attn_prologue(None, k, v, None, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"],
                      a["cu_seqlens"], freqs.cuda())
    torch.cuda.synchronize()
    assert torch.equal(own.view(torch.int16), full.view(torch.int16))
    assert torch.equal(cells(c, a["k_pages"].cpu()).view(torch.int16), cells(c, kp).view(torch.int16))
    assert torch.equal(cells(c, a["v_pages"].cpu()).view(torch.int16), cells(c, vp).view(torch.int16))


def test_many_tokens_give_the_bits_of_few(gdn):
    # past 1024 tokens a workgroup takes all heads of a token, before that a slice
    c = A.Cache([(1500, 2), (1, 40)], H_q=16, H_kv=4, d=128, page=64, seed=4)
    x = inputs(c)
    freqs = gdn.rope_freqs(128, 10000.0, device="cpu")
    out, kp, _ = run(gdn, c, x, freqs)
    q, k, _ = split(c, x)
    want, fp32 = A.prologue(c, q, freqs)
    want, tol = rounded(want, fp32, "bf16")
    A.check(out, want, tol, "q")
    one = A.Cache([(1, 40)], H_q=16, H_kv=4, d=128, page=64, seed=4)
    o1, _, _ = run(gdn, one, x[1500:], freqs)
    assert torch.equal(o1[0].view(torch.int16), out[1500].view(torch.int16))


def test_saturation_and_nan_in_an_8_bit_cache(gdn):
    c = A.Cache([(2, 3)], H_q=2, H_kv=2, d=64, page=16, kind="e4m3", seed=5)
    x = inputs(c)
    x[0, 2 * 64:2 * 64 + 4] = torch.tensor([1e4, -1e4, math.nan, math.inf], dtype=A.BF)
    x[1, 4 * 64:4 * 64 + 3] = torch.tensor([-math.inf, 3e38, math.nan], dtype=A.BF)
    _, kp, vp = run(gdn, c, x, None)
    k, v = cells(c, kp).float(), cells(c, vp).float()
    assert k[0, 0, 0] == 448 and k[0, 0, 1] == -448 and k[0, 0, 2].isnan() and k[0, 0, 3] == 448
    assert v[1, 0, 0] == -448 and v[1, 0, 1] == 448 and v[1, 0, 2].isnan()


def test_padding_unusable_and_outside_tokens(gdn):
    lens = [(1, 10), (2, 10), (1, 10), (1, 10), (3, 10)]
    c = A.Cache(lens, H_q=4, H_kv=2, d=64, page=16, seed=6)
    x = inputs(c)
    freqs = gdn.rope_freqs(64, 10000.0, device="cpu")
    row, table, kv_len, cu = c.row.clone(), c.table.clone(), c.kv_len.clone(), c.cu.clone()
    row[0] = 0
    row[1] = -1
    table[int(row[2]), 0] = c.N
    kv_len[int(row[3])] = c.width * c.page + 1
    kv_len[int(row[4])] = 2                        # its first token stands before position 0
    q, k, v = split(c, x.cuda())
    a = c.cuda(row=row, page_table=table, kv_len=kv_len)
    out = torch.full((c.T + 2, 4, 64), 7.0, dtype=A.BF, device="cuda")
    q2 = torch.cat([q, q[:2]])
    k2, v2 = torch.cat([k, k[:2]]), torch.cat([v, v[:2]])
    gdn.attn_prologue(q2, k2, v2, out, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"],
                      a["cu_seqlens"], freqs.cuda())
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    assert out[1:6].isnan().all()
    assert out[6:8].isfinite().all() and (out[8:] == 7).all()
    kp = a["k_pages"].cpu()
    changed = (kp.view(torch.int16) != c.k.view(torch.int16)).flatten(1).any(1)
    assert changed.nonzero()[:, 0].tolist() == [int(table[int(row[4]), 0])]
    assert not kp[0].isfinite().any(), "the null page was written"


def test_lengths_far_below_zero(gdn):
    """A length whose distance to the tokens passes 32 bits is a negative position like any other."""
    c = A.Cache([(3, 10), (1, 5)], H_q=4, H_kv=2, d=64, page=16, seed=8)
    kv_len = c.kv_len.clone()
    kv_len[int(c.row[0])] = -2 ** 31
    a = c.cuda(kv_len=kv_len)
    q, k, v = split(c, inputs(c).cuda())
    freqs = gdn.rope_freqs(64, 10000.0)
    for kk, vv, table in ((k, v, a["page_table"]), (None, None, None)):
        out = torch.full((c.T, 4, 64), 7.0, dtype=A.BF, device="cuda")
        gdn.attn_prologue(q, kk, vv, out, a["k_pages"], a["v_pages"], table, a["kv_len"], a["row"], a["cu_seqlens"],
                          freqs)
        torch.cuda.synchronize()
        assert out[:3].isnan().all() and out[3].isfinite().all()


def test_a_captured_prologue_follows_its_lengths(gdn):
    c = A.Cache([(1, 10), (1, 47), (1, 0)], H_q=4, H_kv=2, d=128, page=16, seed=7, width=8)
    freqs = gdn.rope_freqs(64, 10000.0, device="cpu")
    x = inputs(c).cuda()
    q, k, v = split(c, x)
    a = c.cuda()
    out = torch.empty(c.T, 4, 128, dtype=A.BF, device="cuda")
    fd = freqs.cuda()

    def call():
        gdn.attn_prologue(q, k, v, out, a["k_pages"], a["v_pages"], a["page_table"], a["kv_len"], a["row"],
                          a["cu_seqlens"], fd)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        c.kv_len[c.row.long()] = torch.tensor([11 - step, 48 - 3 * step, 1], dtype=torch.int32)
        a["kv_len"].copy_(c.kv_len)
        fresh = inputs(c, step)
        x.copy_(fresh)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, fp32 = A.prologue(c, split(c, fresh)[0], freqs)
        want, tol = rounded(want, fp32, "bf16")
        A.check(out, want, tol, "q")
        want, fp32 = A.prologue(c, split(c, fresh)[1], freqs)
        want, tol = rounded(want, fp32, "bf16")
        A.check(cells(c, a["k_pages"].cpu()), want, tol, "k")
