"""GPU: kv_page_reserve where rows take hundreds and thousands of pages at once
(prompts admitted), against the rules restated one entry at a time."""
import pytest

from tests.test_gpu_kv_pages import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_recurrent_decode_amd as m
    m.lib()
    return m


def test_prompts_of_hundreds_of_pages(gdn):
    m = Model(R=41, width=520, N=9000, page=16)
    dev = Device(gdn, m)
    rows = [1 + (7 * i) % 40 for i in range(40)]
    add = [500 + (997 * i) % 7500 for i in range(40)]
    add[3] = 0
    dev.reserve(rows[:20], add[:20])
    dev.agree(m.reserve(rows[:20], add[:20]))
    # the pool runs out on the way: the prompts behind that get none, a row whose page has room goes on
    rows2, add2 = rows[20:] + [rows[0], rows[1]], add[20:] + [8, 0]
    dev.reserve(rows2, add2)
    missed = m.reserve(rows2, add2)
    assert 0 < len(missed) < len(rows2)
    dev.agree(missed)
    # ended rows leave holes between the pages that stay
    dev.free(rows[0:20:3])
    m.free(rows[0:20:3])
    dev.agree()
    dev.reserve(rows[0:20:3], add[20:27])
    dev.agree(m.reserve(rows[0:20:3], add[20:27]))


def test_a_prompt_that_does_not_fit_among_others(gdn):
    m = Model(R=9, width=700, N=1500, page=16)
    dev = Device(gdn, m)
    rows, add = [1, 2, 3, 4, 5, 1], [16 * 600, 16 * 300 - 3, 16 * 601, 3, 0, 5]
    for _ in range(2):  # the second time each row goes on from where it is
        dev.reserve(rows, add)
        missed = m.reserve(rows, add)
        assert missed
        dev.agree(missed)
        dev.reserve([2, 3], [3, 40])
        dev.agree(m.reserve([2, 3], [3, 40]))


@pytest.mark.parametrize("tokens", [131072, 16 * 8191 + 1])
def test_one_prompt_of_thousands_of_pages(gdn, tokens):
    m = Model(R=4, width=8193, N=17000, page=16)
    dev = Device(gdn, m)
    dev.reserve([2, 1], [50, 16])
    m.reserve([2, 1], [50, 16])
    dev.reserve([1, 3, 2], [tokens - 16, tokens, 7])
    dev.agree(m.reserve([1, 3, 2], [tokens - 16, tokens, 7]))
