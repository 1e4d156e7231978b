"""GPU: calls of lin_attn_prefill in a workspace that was sized for a larger one."""
import pytest
import torch

import gated_deltanet_recurrent_decode_amd as gdn
from tests.lin_helpers import Layer
from tests.test_gpu_linear import prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H_k,H_v,d_k,d_v,largest,lens", [
    (16, 16, 128, 128, (1, 4103), [4096]),
    (8, 32, 128, 64, (16, 9000), [300, 2000, 129, 1, 0, 800]),
    (16, 32, 64, 64, (300, 4500), [2300, *[13] * 100]),
])
def test_smaller_calls_in_the_largest_calls_workspace(H_k, H_v, d_k, d_v, largest, lens):
    B, T = len(lens), sum(lens)
    c = Layer(T, H_k=H_k, H_v=H_v, d_k=d_k, d_v=d_v, N=2 * B + 1, seed=21)
    read, write = list(range(1, B + 1)), list(range(B + 1, 2 * B + 1))
    want, want_state = prefill(c, lens, read, write)
    need = gdn.lin_attn_prefill_workspace_bytes(*largest, H_k, H_v, d_k, d_v)
    big = torch.full((need + 2 * 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    out, state = prefill(c, lens, read, write, ws=big[4096:4096 + need])
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(state, want_state)
    assert bool((big[:4096] == 0x5A).all()) and bool((big[4096 + need:] == 0x5A).all())
