"""What may be assigned to the binding's objects, and what a call then uses."""
import pytest
import torch

from combine_ep_get_10_b200 import binding as B

BF = torch.bfloat16


def adapters():
    return B.Lora(torch.zeros((4, 8, 64), dtype=BF), torch.zeros((4, 32, 8), dtype=BF), torch.ones(4))


def test_replaced_factors_are_the_ones_that_calls_use():
    lo = adapters()
    for name, t in (("a", torch.ones((4, 8, 64), dtype=BF)), ("b", torch.ones((4, 32, 8), dtype=BF)),
                    ("scales", torch.zeros(4))):
        setattr(lo, name, t)
        assert getattr(lo, name) is t and getattr(lo.desc, name) == t.data_ptr()
    lo.scales = None
    assert lo.desc.scales is None


def test_replaced_factors_are_checked():
    lo = adapters()
    before = (lo.a, lo.b, lo.scales, lo.desc.a, lo.desc.b, lo.desc.scales)
    for name, t, error in (("a", torch.zeros((4, 16, 64), dtype=BF), TypeError), ("a", torch.zeros((4, 8, 64)), TypeError),
                           ("a", None, TypeError), ("b", torch.zeros((5, 32, 8), dtype=BF), TypeError),
                           ("b", torch.zeros((4, 8, 32), dtype=BF).transpose(1, 2), ValueError),
                           ("scales", torch.zeros(5), TypeError)):
        with pytest.raises(error):
            setattr(lo, name, t)
    assert before == (lo.a, lo.b, lo.scales, lo.desc.a, lo.desc.b, lo.desc.scales)


def test_sizes_that_buffers_were_made_for_stay():
    """A call checks its arrays by these and passes on the descriptor's: were
    they to differ, a kernel would write past the arrays."""
    router = B.Router(8, 2)
    stats = B.BalanceStats(router, 4, num_seqs=3, device="cpu")
    for obj, names in ((router, ("num_experts", "num_topk")), (stats, ("num_seqs", "num_experts")),
                       (adapters(), ("E", "rank", "hidden_in", "hidden_out"))):
        for name in names:
            old = getattr(obj, name)
            with pytest.raises(AttributeError):
                setattr(obj, name, old + 1)
            assert getattr(obj, name) == old


def test_a_copy_keeps_its_own_addresses():
    import copy

    lo = adapters()
    other = copy.copy(lo)
    other.a = torch.ones_like(lo.a)
    assert lo.desc.a == lo.a.data_ptr() and other.desc.a == other.a.data_ptr() != lo.desc.a
    stats = B.BalanceStats(B.Router(8, 2), 4, device="cpu")
    other = copy.copy(stats)
    other.losses = torch.zeros_like(stats.losses)
    router = B.Router(8, 2)
    assert stats.at(router, -1)["losses"] == stats.losses.data_ptr()
    assert other.at(router, -1)["losses"] == other.losses.data_ptr() != stats.losses.data_ptr()
