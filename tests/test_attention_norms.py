"""CPU: the bound per (token, head) of long attention notices a lost or misplaced
block of keys, which the bound per value does not, and lets the kernels'
roundings pass."""
import pytest
import torch

from tests import attn_helpers as A
from tests import attn_norms as N


def rounded(c, scale, lost=None, moved=None):
    """o as the kernels round it, in 64 bits otherwise, with some keys' values left out or exchanged."""
    G, L = c.H_q // c.H_kv, int(c.kv_len[int(c.row[0])])
    o = torch.zeros(c.T, c.H_q, c.d, dtype=torch.float64)
    for h in range(c.H_q):
        k, v = c.gather(0, h // G, "k"), c.gather(0, h // G, "v").clone()
        s = c.q[:, h].double() @ k.T * scale
        s = torch.where(torch.arange(L)[None] <= torch.arange(L - c.T, L)[:, None], s, -torch.inf)
        # a maximum that lags by 2^5.3, so that no weight is exact
        p = torch.exp(s - s.amax(1, keepdim=True)) * 2 ** 5.3
        if lost:
            v[lost[0]:lost[1]] = 0
        if moved:
            v[moved[0]:moved[0] + 32] = v[moved[1]:moved[1] + 32].clone()
        o[:, h] = p.to(torch.bfloat16).double() @ v / p.sum(1, keepdim=True)
    return o.to(torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3])
def test_a_lost_block_shows_and_roundings_do_not(d, kind, n):
    c = A.Cache([(n, 20011)], H_q=4, H_kv=1, d=d, page=64, kind=kind, seed=5)
    scale = d ** -0.5
    want, _, tol, _ = N.attention(c, scale)
    N.check_norms(rounded(c, scale), want, tol, "roundings")
    ratio = (tol / want.norm(dim=-1)).max()
    assert ratio < 0.015, ratio
    for broken in (dict(lost=(5120, 5248)), dict(lost=(19968, 20012 + n)), dict(lost=(0, 32)), dict(moved=(64, 9600))):
        with pytest.raises(AssertionError, match="heads off"):
            N.check_norms(rounded(c, scale, **broken), want, tol, "broken")


@pytest.mark.parametrize("window", [0, 100])
def test_both_references_agree(window):
    c = A.Cache([(5, 40), (1, 300), (0, 9), (3, 0)], H_q=6, H_kv=2, d=64, page=16, kind="e4m3", seed=3)
    c.kv_len[int(c.row[3])] = 2  # its first token sees nothing
    a, b = A.attention(c, 0.125, window), N.attention(c, 0.125, window)
    assert torch.allclose(a[0], b[0], rtol=1e-12, atol=1e-12) and torch.allclose(a[1], b[1], rtol=1e-12, atol=0)


def test_values_that_are_not_finite_have_to_agree():
    want = torch.zeros(2, 1, 4, dtype=torch.float64)
    want[0, 0, 1] = torch.inf
    tol = torch.full((2, 1), 1e-3, dtype=torch.float64)
    N.check_norms(want.float(), want, tol, "same")
    for value in (0.0, -torch.inf, torch.nan):
        got = want.clone()
        got[0, 0, 1] = value
        with pytest.raises(AssertionError, match="not finite"):
            N.check_norms(got, want, tol, "other")
    got = want.clone()
    got[1, 0, 0] = torch.nan
    with pytest.raises(AssertionError, match="not finite"):
        N.check_norms(got, want, tol, "other")


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("window", [0, 300])
def test_the_deal_covers_every_block_once(few, window):
    lens = [(4, 2000), (2, 30), (4, 900)] if few else [(300, 2000), (40, 3), (128, 900)]
    c = A.Cache(lens, H_q=8, H_kv=2, d=128, page=16, seed=1)
    got = {}
    for mine in N.deal(c, window, 64, few):
        assert mine
        for e, a, b, size, _ in mine:
            assert got.get(e, 0) == a < b <= size
            got[e] = b if b < size else -1
    assert set(got.values()) == {-1}
