"""The router's entry points refuse bad arguments on the host before anything
is launched (no GPU here), and the binding checks types and shapes."""
import ctypes

import pytest
import torch

from combine_ep_get_10_b200 import binding as B


@pytest.fixture(scope="module")
def L():
    from combine_ep_get_10_b200 import build

    build.build()
    return B.lib()


def desc(**kw):
    f = dict(score=0, logits_dtype=B.EP_FP32, num_tokens=16, num_experts=64, num_topk=4, num_groups=1, topk_groups=1,
             group_top=1, normalize=1, scale=1.0)
    f.update(kw)
    return B.RouterDesc(*(f[n] for n, _ in B.RouterDesc._fields_))


BAD = [(dict(score=2), 1), (dict(score=-1), 1), (dict(logits_dtype=B.EP_FP8_E4M3), 1), (dict(num_tokens=-1), 1),
       (dict(num_experts=0), 1), (dict(num_topk=0), 1), (dict(num_topk=65), 1), (dict(normalize=2), 1),
       (dict(num_groups=0), 1), (dict(num_groups=5), 1), (dict(num_groups=8, topk_groups=0), 1),
       (dict(num_groups=8, topk_groups=9), 1), (dict(group_top=0), 1), (dict(group_top=3), 1),
       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(num_tokens=1 << 26), 1),
       (dict(num_experts=1025), 6), (dict(num_topk=33), 6), (dict(num_experts=60, num_groups=6), 6),
       (dict(num_groups=64), 6)]


def topk(L, d, logits=0x1000, bias=None, mask=None, idx=0x2000, w=0x3000):
    return L.ep_router_topk(d, logits, bias, mask, idx, w, None)


def loss(L, d, logits=0x1000, idx=0x2000, off=None, S=1, losses=0x4000, counts=0x5000, tokens=0x6000, means=None,
         ws=0x100000, n=1 << 30):
    return L.ep_balance_loss(d, logits, idx, None, off, S, losses, counts, tokens, means, ws, n, None)


def back(L, d, logits=0x1000, idx=0x2000, dw=0x3000, off=None, S=1, counts=0x5000, tokens=0x6000, dl=0x7000, out=0x8000):
    return L.ep_router_backward(d, logits, idx, None, dw, off, S, counts, tokens, dl, out, None)


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_descriptions(L, kw, status):
    d = ctypes.byref(desc(**kw))
    assert topk(L, d) == status and loss(L, d) == status and back(L, d) == status
    assert L.ep_balance_workspace_bytes(d, 1) == 0


def test_bad_pointers(L):
    d, h = ctypes.byref(desc()), ctypes.byref(desc(logits_dtype=B.EP_BF16))
    for f in (topk, loss, back):
        assert f(L, None) == 1
        assert f(L, d, logits=None) == 1 and f(L, d, logits=0x1002) == 1 and f(L, h, logits=0x1001) == 1
        assert f(L, d, idx=0x2004) == 1
    assert topk(L, d, idx=None) == 1 and topk(L, d, w=None) == 1 and topk(L, d, w=0x3002) == 1
    assert topk(L, d, bias=0x1002) == 1
    assert loss(L, d, losses=None) == 1 and loss(L, d, counts=None) == 1 and loss(L, d, tokens=None) == 1
    assert loss(L, d, S=0) == 1 and loss(L, d, S=2) == 1 and loss(L, d, off=0x9002, S=2) == 1
    assert loss(L, d, S=(1 << 24) + 1, off=0x9000) == 1
    assert loss(L, d, ws=None) == 4 and loss(L, d, ws=0x100010) == 4
    need = L.ep_balance_workspace_bytes(d, 1)
    assert need % 256 == 0 and need >= (1 + 1) * 64 * 8 and loss(L, d, n=need - 1) == 4
    assert back(L, d, out=None) == 1 and back(L, d, out=0x1000) == 1 and back(L, d, out=0x8002) == 1
    assert back(L, d, idx=None) == 1 and back(L, d, dw=0x3002) == 1
    assert back(L, d, counts=None) == 1 and back(L, d, tokens=None) == 1 and back(L, d, S=0) == 1
    assert back(L, d, S=2) == 1 and back(L, d, dl=0x7002) == 1


def test_workspace_grows_with_tokens_and_sequences(L):
    need = lambda T, S: L.ep_balance_workspace_bytes(ctypes.byref(desc(num_tokens=T)), S)  # noqa: E731
    assert 0 < need(0, 1) <= need(100, 1) < need(10000, 1) < need(10000, 500)
    assert need(100, 0) == 0 and need(100, (1 << 24) + 1) == 0


def test_struct_matches_the_header(L):
    assert ctypes.sizeof(B.RouterDesc) == 40 and B.RouterDesc.scale.offset == 36


def test_binding_checks(L):
    r = B.Router(8, 2)
    idx, w = torch.empty((4, 2), dtype=torch.int64), torch.empty((4, 2))
    with pytest.raises(TypeError):
        B.ep_router_topk(torch.zeros((4, 9)), r, idx, w)  # another number of experts
    with pytest.raises(TypeError):
        B.ep_router_topk(torch.zeros((4, 8), dtype=torch.float16), r, idx, w)
    with pytest.raises(ValueError):
        B.ep_router_topk(torch.zeros((8, 4)).T, r, idx, w)  # strided
    with pytest.raises(ValueError):
        B.ep_router_topk(torch.zeros((4, 8)), r, idx, w)  # not on a GPU
    with pytest.raises(B.EPError):
        B.BalanceStats(B.Router(8, 9), 4, device="cpu")  # more slots than experts
    stats = B.BalanceStats(r, 4, device="cpu")
    assert stats.losses.shape == (1, 2) and stats.counts.shape == (1, 8)
    with pytest.raises(ValueError):
        B.ep_balance_loss(torch.zeros((4, 8)), r, idx, stats)
