"""GPU: attn_shared with windows that cut through the common keys, in every kernel; tables wider than their rows."""
import math

import pytest
import torch

from tests import attn_helpers as H
from tests import attn_norms as N
from tests.test_gpu_attn_shared import Forked, check, run

pytestmark = pytest.mark.gpu

# (new tokens, own tokens before them) of the members: single tokens (weights of 15 bits), a few tokens (tiles of 128
# rows), chunks (tiles of 256)
MEMBERS = {"single": [[(1, 10), (1, 100), (1, 300), (1, 0)], [(1, 2), (1, 3)]],
           "few": [[(1, 10), (30, 100), (1, 300), (5, 0)], [(2, 2), (29, 3)]],
           "many": [[(1, 10), (130, 100), (1, 300), (5, 0)], [(1, 2), (170, 3)]]}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", list(MEMBERS))
@pytest.mark.parametrize("window", [1, 60, 333, 450])
def test_windows(d, kind, rows, window):
    a, b = MEMBERS[rows]
    c = Forked([(400, a), (600, b)], H_q=8, H_kv=2, d=d, page=32, kind=kind, seed=61)
    check(c, *run(c, window=window), window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", ["single", "few", "many"])
def test_values_that_are_not_finite_behind_windows(d, rows):
    c = Forked([(400, MEMBERS[rows][0])], H_q=8, H_kv=2, d=d, page=32, seed=62)
    p, o = c.own("v", 0, 100)
    c.v[p, 0, o, 3], c.v[p, 1, o, 5] = math.inf, math.nan
    p, o = c.own("v", 0, 200)
    c.k[p, 0, o, 7], c.k[p, 1, o, 9] = -math.inf, math.nan
    # position 100 is out of some members' windows, 200 and its scores of all
    for window in (150, 311 if rows == "single" else 150):
        out, lse = run(c, window=window)
        o, l, tol, tol_l = H.attention(c, d ** -0.5, window)
        sees = o.isfinite().all(-1).all(-1)  # tokens whose windows end behind both
        assert sees.any()
        H.check(out[sees.cuda()], o[sees], tol[sees], f"o of window {window}")
        H.check(lse[sees.cuda()], l[sees], tol_l[sees], f"lse of window {window}")


@pytest.mark.parametrize("window", [0, 700, 3000])
@pytest.mark.parametrize("d,kind", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_the_plans_own_choice_of_groups(d, kind, window):
    # long enough that the rule takes the first group together, short enough that it leaves the second
    c = Forked([(4096, [(1, i * 11 % 500) for i in range(48)]), (64, [(1, 4), (1, 6)])], H_q=16, H_kv=4, d=d, page=64,
               kind=kind, seed=63)
    out, lse = run(c, least=None, window=window)
    o, l, tol, tol_l = N.attention(c, d ** -0.5, window, "cuda")
    N.check_norms(out, o, tol, "o")
    H.check(lse, l, tol_l, "lse")


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("least", [None, 16])
def test_tables_wider_than_their_rows(d, least):
    # the table's width is what a row may grow to: 65536 positions
    c = Forked([(500, [(1, i * 5 % 40) for i in range(8)])], H_q=16, H_kv=2, d=d, page=16, width=4096, seed=64)
    check(c, *run(c, least=least))
