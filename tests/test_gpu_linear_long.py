"""GPU: lin_attn_prefill over segments of many chunks, and values that are not finite in every layout of heads."""
import math

import pytest
import torch

from tests.lin_helpers import Layer, close
from tests.test_gpu_linear import prefill

pytestmark = pytest.mark.gpu


def on_gpu(c):
    c.qkv, c.g, c.state = c.qkv.cuda(), c.g.cuda(), c.state.cuda()
    return c


def check(c, lens, read, write, out, state):
    a = 0
    for b, n in enumerate(lens):
        S0 = c.state[read[b]] if read[b] else torch.zeros_like(c.state[0])
        o, tol, states = c.reference(a, a + n, S0)
        close(out[a:a + n], o.cpu(), tol.cpu(), f"out of sequence {b}")
        close(state[write[b]], states[-1][0].cpu(), states[-1][1].cpu(), f"state of sequence {b}")
        a += n


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("H_k,d_v,n", [(64, 64, 5201), (32, 64, 4100), (64, 128, 4500)])
def test_segments_of_many_chunks(H_k, d_v, n, per_token):
    # with 64 heads the chip is full with few segments, which become 9 chunks long and more
    c = on_gpu(Layer(n, H_k=H_k, H_v=64, d_k=64, d_v=d_v, N=3, per_token=per_token, seed=51, spread=0.1))
    out, state = prefill(c, [n], [1], [2], state=c.state.clone())
    check(c, [n], [1], [2], out, state)


def test_hundreds_of_sequences_and_a_long_one():
    # more sequences than rounds of workgroups: segments of 2048 tokens
    lens = [1 + i % 8 for i in range(250)]
    lens[100] = 4500
    B = len(lens)
    c = on_gpu(Layer(sum(lens), H_k=64, H_v=64, d_k=64, d_v=64, N=2 * B + 1, seed=52, spread=0.1))
    read, write = [i + 1 if i % 3 else 0 for i in range(B)], list(range(B + 1, 2 * B + 1))
    out, state = prefill(c, lens, read, write, state=c.state.clone())
    check(c, lens, read, write, out, state)


@pytest.mark.parametrize("H_v,d_k,d_v", [(2, 128, 128), (1, 64, 64), (3, 128, 64), (2, 128, 64), (2, 64, 128)])
@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("at", [37, 199])
def test_values_that_are_not_finite(H_v, d_k, d_v, which, value, at):
    # a token's value that is not finite changes nothing before it, and no other head or column
    c = Layer(300, H_k=1, H_v=H_v, d_k=d_k, d_v=d_v, N=3, seed=53)
    clean, state0 = prefill(c, [300], [1], [2])
    qkv, g, h = c.qkv.clone(), c.g.clone(), H_v - 1
    q, k, v = c.heads(qkv)
    if which == "g":
        g[at, h] = value
    else:
        {"q": q, "k": k, "v": v}[which][at, h if which == "v" else 0, 5] = value
    out, state = prefill(c, [300], [1], [2], qkv=qkv, g=g)
    assert torch.equal(out[:at].view(torch.int16), clean[:at].view(torch.int16)), "a token before it changed"
    odd, odd_state = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(state[2], dtype=torch.bool)
    if which == "q":
        odd[at] = True
    elif which == "k":
        odd[at:], odd_state[:, 5] = True, True
    elif which == "v":
        odd[at:, h, 5], odd_state[h, :, 5] = True, True
    else:
        odd[at:, h], odd_state[h] = True, True
    assert not out[odd].isfinite().any() and not state[2][odd_state].isfinite().any()
    assert torch.equal(out[~odd].view(torch.int16), clean[~odd].view(torch.int16))
    assert torch.equal(state[2][~odd_state], state0[2][~odd_state])
