"""GPU: large values through lin_attn_prefill, whose states are held at other scales than their own within a call."""
import math

import pytest
import torch

from tests.lin_helpers import BF, Layer
from tests.test_gpu_linear import check_prefill, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("big", [dict(v=1e15, q=1e6), dict(v=1e24), dict(q=1e24), dict(k=1e24), dict(S=1e24),
                                 dict(S=1e15, q=1e6)])
@pytest.mark.parametrize("g", [-0.33, -0.66, -1.3, -4.0])
@pytest.mark.parametrize("d_k,d_v", [(64, 64), (128, 128)])
def test_large_values_stay_finite(big, g, d_k, d_v):
    # log decays that bring the logarithm of a state's scale close to where it is taken anew: after one chunk of 32
    # tokens, after two, after four.  lin_attn_step returns numbers for all of these.
    c = Layer(200, H_k=1, H_v=2, d_k=d_k, d_v=d_v, N=3, seed=31)
    c.g = torch.full_like(c.g, g)
    c.qkv = c.qkv.float()
    for x, name in zip(c.heads(c.qkv), "qkv"):
        x *= big.get(name, 1.0)
    c.qkv = c.qkv.to(BF)
    c.state *= big.get("S", 1.0)
    out, state = prefill(c, [200], [1], [2])
    assert bool(out.isfinite().all()) and bool(state.isfinite().all())
    check_prefill(c, [200], [1], [2], out, state)


def test_growth_of_small_states():
    # logarithms above 0: the state is held at a fraction of its value
    c = Layer(150, H_k=1, H_v=2, N=3, seed=32)
    c.g = torch.full_like(c.g, 0.3)
    c.state *= 1e-15
    c.qkv = (c.qkv.float() * 1e-9).to(BF)
    c.scale = 1e9 * math.exp(-40.0)
    out, state = prefill(c, [150], [1], [2])
    check_prefill(c, [150], [1], [2], out, state)
