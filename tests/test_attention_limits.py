"""CPU: sizes at the edges of what the paged-attention entry points take."""
from tests.test_attention_abi import SHAPE, UNSUPPORTED, dims, heads, prologue


def test_a_prologue_of_more_threads_than_a_launch_counts_is_refused():
    """256 threads a token and 2^32 in a launch: refused as a size, not by the launch."""
    assert prologue(dims(T=1 << 24)) == SHAPE
    # one token less is a size like any other: the next check speaks (q is not aligned)
    assert prologue(dims(T=(1 << 24) - 1), q=heads(0x10008)) == UNSUPPORTED
