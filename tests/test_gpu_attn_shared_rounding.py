"""GPU: what attn_shared's outputs lose to rounding where attn_paged's weights keep 15 bits."""
import pytest
import torch

from tests import attn_norms as N
from tests.attn_helpers import BF
from tests.test_gpu_attn_shared import Forked, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,H_q", [(1, 16), (4, 16), (1, 64)])
@pytest.mark.parametrize("least", [16, 1 << 20])
def test_outputs_of_few_rows_are_rounded_once(d, kind, n, H_q, least):
    """Nearly every output is the 64-bit one rounded to bf16, whether the groups are taken together or row by row.

    It is another one only where the 64-bit value lies closer to the middle of two bf16 numbers than the kernel is
    off: a share of 2 e / 2^-8 for an error of e, relative.  Weights kept to 2^-15 and fp32 sums leave an e of about
    10^-5, 0.5%, and up to three times that for the values near 0; weights rounded to bf16 leave 0.001, 25%."""
    c = Forked([(1500, [(n, (613 * i) % 700) for i in range(14)]), (2203, [(n, (97 * i) % 1500) for i in range(10)])],
               H_q=H_q, H_kv=4, d=d, page=64, kind=kind, seed=41, q_scale=2.0)
    out, _ = run(c, least=least)
    o, _, _, _ = N.attention(c, d ** -0.5, 0, "cuda")
    other = (out.cpu() != o.to(BF)).double().mean()
    assert other < 0.02, float(other)


def test_infinities_that_every_row_sees():
    # an infinity in v where every row of a tile sees it: an infinity in its column, no NaN
    c = Forked([(640, [(1, 30), (1, 60), (1, 5)])], H_q=4, H_kv=2, d=64, page=32, seed=42)
    p, o = c.own("v", 0, 100)
    c.v[p, 0, o, 3], c.v[p, 1, o, 5] = float("inf"), -float("inf")
    out, _ = run(c)
    assert bool((out[:, :2, 3] == float("inf")).all()) and bool((out[:, 2:, 5] == -float("inf")).all())
    out[:, :2, 3] = out[:, 2:, 5] = 0
    assert bool(out.isfinite().all())
