"""The low-rank adapter calls refuse bad arguments on the host before anything is
launched (no GPU here), and the binding checks types and shapes."""
import ctypes

import pytest
import torch

from combine_ep_get_10_b200 import binding as B


@pytest.fixture(scope="module")
def L():
    from combine_ep_get_10_b200 import build

    build.build()
    return B.lib()


def routing(T=16, K=1, E=8):
    return B.RoutingDesc(B.EP_ROUTING_TOPK, 0x1000, None, T, K, 0, E, 1)


LAYOUT = B.LayoutDesc(0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None, None, 0x100000, 256)


def lora(**kw):
    f = dict(rank=16, hidden_in=64, hidden_out=128, a=0x2000, b=0x3000, scales=0x4000)
    f.update(kw)
    return B.LoraDesc(*(f[n] for n, _ in B.LoraDesc._fields_))


def fwd(L, r=None, lay=LAYOUT, lo=None, x=0x5000, base=0x6000, mode=0, mt=0, rows=16, rt=0x7000, out=0x8000, h=0x9000):
    r, lo = r or routing(), lo or lora()
    return L.ep_lora(x, base, ctypes.byref(r), ctypes.byref(lay), mode, mt, rows, rt, ctypes.byref(lo), out, h, None)


def bwd(L, r=None, lay=LAYOUT, lo=None, dy=0x5000, x=0x5100, h=0x9000, dxb=0x6000, mode=0, mt=0, rows=16, rt=0x7000,
        dh=0xa000, dx=0xb000, da=0xc000, db=0xd000):
    r, lo = r or routing(), lo or lora()
    return L.ep_lora_backward(dy, x, h, dxb, ctypes.byref(r), ctypes.byref(lay), mode, mt, rows, rt, ctypes.byref(lo),
                              dh, dx, da, db, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_bad_descriptions(L, call):
    for kw in (dict(rank=0), dict(rank=12), dict(rank=-8), dict(hidden_in=0), dict(hidden_in=60), dict(hidden_out=4),
               dict(a=None), dict(b=None), dict(a=0x2008), dict(b=0x3004), dict(scales=0x4002)):
        assert call(L, lo=lora(**kw)) == 1, kw
    for kw in (dict(rank=136), dict(hidden_in=(1 << 20) + 8), dict(hidden_out=(1 << 20) + 8)):
        assert call(L, lo=lora(**kw)) == 6, kw
    assert call(L, r=routing(E=1025)) == 6 and call(L, r=routing(T=(1 << 24) + 1), rows=16) == 6
    assert call(L, r=routing(K=2)) == 1  # a row table needs one adapter a token
    assert call(L, r=B.RoutingDesc(B.EP_ROUTING_EXPERT_CHOICE, None, 0x1000, 16, 0, 4, 8, 1)) == 1
    assert call(L, mode=3) == 1 and call(L, mode=1, mt=0) == 1 and call(L, rows=-1) == 1 and call(L, rows=1 << 31) == 1
    assert call(L, rt=0x7002) == 1
    no_counts = B.LayoutDesc(None, 0x1000, 0x1000, 0x1000, 0x1000, None, None, 0x100000, 256)
    assert call(L, lay=no_counts, mode=1, mt=4) == 1
    no_offsets = B.LayoutDesc(0x1000, None, 0x1000, 0x1000, 0x1000, None, None, 0x100000, 256)
    assert call(L, lay=no_offsets) == 1
    assert call(L, lay=B.LayoutDesc(0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None, None, None, 0)) == 4


def test_bad_pointers(L):
    assert fwd(L, x=None) == 1 and fwd(L, x=0x5008) == 1 and fwd(L, base=0x6008) == 1 and fwd(L, out=None) == 1
    assert fwd(L, out=0x8008) == 1 and fwd(L, h=None) == 1 and fwd(L, h=0x9004) == 1 and fwd(L, out=0x5000) == 1
    assert bwd(L, dy=None) == 1 and bwd(L, dy=0x5008) == 1 and bwd(L, dxb=0x6008) == 1 and bwd(L, dx=0xb008) == 1
    assert bwd(L, dh=None) == 1 and bwd(L, dh=0xa004) == 1 and bwd(L, dh=0x9000) == 1
    assert bwd(L, da=None) == 1 and bwd(L, db=None) == 1 and bwd(L, da=0xc008) == 1 and bwd(L, db=0xd008) == 1
    assert bwd(L, x=None) == 1 and bwd(L, h=None) == 1 and bwd(L, dx=0x5000) == 1 and bwd(L, dx=0x5100) == 1


def test_row_tokens_reject_bad_args(L):
    def rt(r=None, lay=LAYOUT, mode=0, mt=0, rows=16, p=0x7000):
        return L.ep_row_tokens(ctypes.byref(r or routing()), ctypes.byref(lay), mode, mt, rows, p, None)

    assert rt(p=None) == 1 and rt(p=0x7002) == 1 and rt(rows=-1) == 1 and rt(rows=1 << 31) == 1 and rt(mode=1) == 1
    assert rt(r=B.RoutingDesc(B.EP_ROUTING_EXPERT_CHOICE, None, 0x1000, 16, 0, 4, 8, 1)) == 1
    assert rt(lay=B.LayoutDesc(0x1000, 0x1000, 0x1000, 0x1000, None, None, None, 0x100000, 256)) == 1


def test_struct_matches_the_header(L):
    assert ctypes.sizeof(B.LoraDesc) == 40 and B.LoraDesc.a.offset == 16


def test_binding_checks(L):
    bf = torch.bfloat16
    a, b = torch.zeros((4, 8, 64), dtype=bf), torch.zeros((4, 32, 8), dtype=bf)
    with pytest.raises(TypeError):
        B.Lora(a, torch.zeros((4, 32, 16), dtype=bf))  # another rank
    with pytest.raises(TypeError):
        B.Lora(a.float(), b)
    with pytest.raises(TypeError):
        B.Lora(a, b, torch.zeros(3))
    with pytest.raises(ValueError):
        B.Lora(torch.zeros((4, 64, 8), dtype=bf).transpose(1, 2), b)  # strided
    lo = B.Lora(a, b, torch.ones(4))
    r = B.Routing.topk(torch.zeros((5, 1), dtype=torch.int64), 4, 1)
    with pytest.raises(ValueError):  # not on a GPU
        B.ep_lora(torch.zeros((5, 64), dtype=bf), r, None, lo, torch.zeros((5, 32), dtype=bf), torch.zeros((5, 8)))
    with pytest.raises(TypeError):
        B.ep_row_tokens(r, None, torch.zeros(5, dtype=torch.int64))
