"""The limits that the router's and the adapters' headers state, on the host (no
GPU here): what lies past them is refused by every call, what lies at them is not."""
import ctypes

import pytest

from combine_ep_get_10_b200 import binding as B
from test_lora_cpu import LAYOUT, bwd, fwd, routing
from test_router_cpu import back, desc, loss, topk


@pytest.fixture(scope="module")
def L():
    from combine_ep_get_10_b200 import build

    build.build()
    return B.lib()


def test_more_tokens_than_an_index_holds_are_refused(L):
    """One expert allows the most tokens: T * E < 2^31 alone would let token
    indices a chunk past the last one overflow."""
    most = desc(num_tokens=1 << 30, num_experts=1, num_topk=1)
    assert L.ep_balance_workspace_bytes(ctypes.byref(most), 1) > 0
    for T in ((1 << 30) + 1, 2132973617, (1 << 31) - 1):
        d = ctypes.byref(desc(num_tokens=T, num_experts=1, num_topk=1))
        assert L.ep_balance_workspace_bytes(d, 1) == 0
        assert topk(L, d) == 1 and loss(L, d) == 1 and back(L, d) == 1


def test_more_rows_than_an_index_holds_are_refused(L):
    """A padded buffer may have rows up to the limit whatever the routing's pairs;
    past it a row a few tiles behind the last would overflow."""
    pairs, E = 16, 8
    for rows in ((1 << 31) - 1023, (1 << 31) - 1):
        for mt in (1 << 28, (1 << 31) - 1):
            kw = dict(rows=rows, mode=1, mt=mt, rt=None)
            assert fwd(L, r=routing(T=pairs, E=E), **kw) == 1 and bwd(L, r=routing(T=pairs, E=E), **kw) == 1
        assert L.ep_row_tokens(ctypes.byref(routing()), ctypes.byref(LAYOUT), 1, 1 << 28, rows, 0x7000, None) == 1
    # at the limit the next check speaks: h is missing
    assert fwd(L, rows=(1 << 31) - 1024, mode=1, mt=1 << 28, rt=None, h=None) == 1


def test_the_rule_between_kernels_is_the_one_that_tests_assume():
    import os

    import lora_paths
    from combine_ep_get_10_b200 import build

    with open(os.path.join(build.CSRC, "ep_lora.cu")) as f:
        source = f.read()
    assert lora_paths.RULE in source and "constexpr int kFewRank = 64;" in source
