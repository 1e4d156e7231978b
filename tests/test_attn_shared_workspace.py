"""CPU: a workspace of attn_shared that is sized for the largest call serves the smaller ones."""
import itertools

import pytest

import gated_deltanet_recurrent_decode_amd as gdn


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H_q,H_kv", [(16, 2), (32, 4), (8, 8), (10, 2), (48, 2), (256, 1)])
def test_the_size_never_falls_as_the_call_grows(d, H_q, H_kv):
    axes = [(1, 2, 63, 300, 2000), (1, 100, 4097, 40000), (0, 1, 5, 1024),
            (1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 25, 26, 32, 33, 64, 128, 129, 200, 256, 1000)]
    sizes = {x: gdn.attn_shared_workspace_bytes(x[0], x[1], x[2], x[3], H_q, H_kv, d) for x in itertools.product(*axes)}
    for x, n in sizes.items():
        for axis, values in enumerate(axes):
            at = values.index(x[axis])
            if at + 1 < len(values):
                more = (*x[:axis], values[at + 1], *x[axis + 1:])
                assert sizes[more] >= n, (x, more)
