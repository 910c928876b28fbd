"""Calls of the low-rank products that their documentation allows or refuses:
layouts that are not the routing's, kernels for many rows at every rank, streams,
graphs replayed with other adapters, large arrays."""
import math

import pytest
import torch

from combine_ep_get_10_b200 import binding as B
from lora_paths import few_rows
from test_gpu_lora import Case, ids

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


@pytest.mark.parametrize("T,part,E,rank", [(5000, 2100, 4, 16), (5000, 2700, 40, 64), (5000, 4900, 3, 128),
                                           (300, 100, 4, 16)])
@pytest.mark.parametrize("mode,mt", [(B.EP_LAYOUT_COMPACT, 0), (B.EP_LAYOUT_PADDED, 2000)])
def test_a_layout_of_more_rows_is_left_alone(T, part, E, rank, mode, mt):
    """With a layout that has more rows than the routing has pairs, nothing is
    computed from scratch that no kernel wrote: outputs keep what they held, the
    factors' gradients are zeros, and the call is flagged."""
    c = Case(ids(T, E, 1, none=0.0), E, rank, 136, 72, 2, tokens=False, mode=mode, max_tokens=mt)
    routing = c.routing.tokens(0, part)
    h = torch.full((c.num_rows, rank), math.nan, device="cuda")
    dh = h.clone()
    out = torch.full((c.num_rows, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((c.num_rows, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    da, db = torch.full_like(c.lora.a, 5.0), torch.full_like(c.lora.b, 5.0)
    B.ep_lora(c.x.cuda(), routing, c.layout, c.lora, out, h, base=c.base.cuda(), **c.kw)
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_OVERFLOW
    B.ep_lora_backward(c.dy.cuda(), c.x.cuda(), h, routing, c.layout, c.lora, dh, dx=dx, da=da, db=db,
                       dx_base=c.dx_base.cuda(), **c.kw)
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_OVERFLOW
    assert bool((out == 5.0).all()) and bool((dx == 5.0).all())
    assert bool(h.isnan().all()) and bool(dh.isnan().all())
    assert not bool(da.any()) and not bool(db.any())
    c.check_forward()  # the layout's own routing is served as before
    assert B.ep_get_device_error(c.layout) == (B.EP_DEVERR_OVERFLOW if mt and c.layout.num_tokens_per_expert.max() > mt
                                               else 0)


def test_a_layout_that_is_not_with_the_rows_is_refused():
    from types import SimpleNamespace

    c = Case(ids(100, 4, 70), 4, 16, 64, 72, 71)
    elsewhere = SimpleNamespace(desc=c.layout.desc, workspace=torch.empty(1, dtype=torch.uint8))
    out = torch.empty((100, 72), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((c.num_rows, 16), device="cuda")
    with pytest.raises(ValueError):
        B.ep_lora(c.x.cuda(), c.routing, elsewhere, c.lora, out, h, row_token=c.row_token)
    with pytest.raises(ValueError):
        B.ep_lora_backward(c.dy.cuda(), None, None, c.routing, elsewhere, c.lora, h, row_token=c.row_token)
    with pytest.raises(ValueError):
        B.ep_row_tokens(c.routing, elsewhere, c.row_token)
    with pytest.raises(ValueError):
        B.ep_row_tokens(c.routing, c.layout, c.row_token.cpu())


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 72])
@pytest.mark.parametrize("T", [30, 2700])
def test_an_infinite_row_gives_what_its_products_give(rank, T):
    """x with an infinity whose products with the first factor are all of one sign
    where they are infinite: h is infinite, and so is what the second factor takes of
    it, whatever ranks the kernel adds to a full step."""
    idx = torch.zeros((T, 1), dtype=torch.int64)
    c = Case(idx, 1, rank, 72, 64, 72, scales=False)
    c.x[3] = 1.0
    c.x[3, 5] = math.inf
    lora = B.Lora(torch.ones_like(c.lora.a), torch.ones_like(c.lora.b))
    out = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((T, rank), device="cuda")
    B.ep_lora(c.x.cuda(), c.routing, c.layout, lora, out, h, row_token=c.row_token)
    rows = (c.row_token == 3).nonzero().squeeze(1)
    assert bool((h[rows] == math.inf).all()) and bool(torch.isfinite(h).all(dim=1).sum() == T - 1)
    assert bool((out[3] == math.inf).all())


def many(T, E, rank, seed, hin, hout, **kw):
    """A case whose forward call takes the two kernels for many rows."""
    idx = ids(T, E, seed, **kw) if isinstance(T, int) else T
    assert not few_rows(idx.numel(), E, rank)
    return Case(idx, E, rank, hin, hout, seed)


def few(T, E, rank, seed, hin, hout, **kw):
    idx = ids(T, E, seed, **kw)
    assert few_rows(idx.numel(), E, rank)
    return Case(idx, E, rank, hin, hout, seed)


@pytest.mark.parametrize("rank,T,E", [(8, 9600, 1), (16, 9600, 1), (24, 9600, 2), (32, 9600, 1), (40, 9600, 1),
                                      (64, 9600, 2), (64, 5200, 300), (16, 5400, 20), (32, 5400, 70)])
def test_stages_wrap_in_the_kernels_for_many_rows(rank, T, E):
    """More steps a CTA than it has stages, in both products of a forward call and
    in both directions."""
    c = many(T, E, rank, 50, 2312, 2056)
    c.check_forward()
    c.check_backward(want=("dx",))


@pytest.mark.parametrize("rank", [16, 32, 64])
def test_uneven_tiles_of_many_rows(rank):
    """Adapters of very different sizes on the kernels for many rows."""
    g = torch.Generator().manual_seed(51)
    sizes = [1, 127, 128, 129, 3, 260, 64, 0, 31, 1700]
    idx = torch.cat([torch.full((n,), e, dtype=torch.int64) for e, n in enumerate(sizes)] + [torch.full((200,), -1)])
    idx = idx[torch.randperm(idx.numel(), generator=g)][:, None]
    for hin, hout in ((72, 2056), (1160, 8)):
        c = many(idx, len(sizes), rank, 52, hin, hout) if rank > 16 else many(idx.clamp(max=8), 9, rank, 52, hin, hout)
        c.check_forward()
        c.check_forward("in place")
        c.check_backward()


@pytest.mark.parametrize("rank", [16, 32, 64, 96])
def test_outputs_of_the_kernels_for_many_rows_stay_in_bounds(rank):
    from test_gpu_canary import Guarded, _check

    hin, hout = 264, 328
    c = many(2700, 5, rank, 53, hin, hout)
    T, n = 2700, c.num_rows
    bf = torch.bfloat16
    out, dx = Guarded((T, hout), bf), Guarded((T, hin), bf)
    h, dh = Guarded((n, rank), torch.float32), Guarded((n, rank), torch.float32)
    da, db = Guarded(c.a.shape, bf), Guarded(c.b.shape, bf)
    B.ep_lora(c.x.cuda(), c.routing, c.layout, c.lora, out.t, h.t, base=c.base.cuda(), row_token=c.row_token)
    B.ep_lora_backward(c.dy.cuda(), c.x.cuda(), h.t, c.routing, c.layout, c.lora, dh.t, dx=dx.t, da=da.t, db=db.t,
                       row_token=c.row_token)
    torch.cuda.synchronize()
    _check(out, dx, h, dh, da, db)


class Step:
    """Layout, row table, both directions, on ids that may change."""

    def __init__(self, c):
        self.c = c
        bf = torch.bfloat16
        self.idx = c.idx.cuda()
        self.routing = B.Routing.topk(self.idx, c.E, 1)
        self.layout = B.Layout(self.routing)
        T = c.idx.shape[0]
        self.x, self.base, self.dy, self.dxb = c.x.cuda(), c.base.cuda(), c.dy.cuda(), c.dx_base.cuda()
        new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.rows = new(T, dtype=torch.int32)
        self.h, self.dh = new(T, c.r), new(T, c.r)
        self.out, self.dx = new(T, c.hout, dtype=bf), new(T, c.hin, dtype=bf)
        self.da, self.db = torch.zeros_like(c.lora.a), torch.zeros_like(c.lora.b)

    def run(self, stream):
        B.ep_get_layout(self.routing, self.layout, stream=stream)
        B.ep_row_tokens(self.routing, self.layout, self.rows, stream=stream)
        B.ep_lora(self.x, self.routing, self.layout, self.c.lora, self.out, self.h, base=self.base, row_token=self.rows,
                  stream=stream)
        B.ep_lora_backward(self.dy, self.x, self.h, self.routing, self.layout, self.c.lora, self.dh, dx=self.dx,
                           da=self.da, db=self.db, dx_base=self.dxb, row_token=self.rows, stream=stream)

    def outputs(self):
        n = int((self.idx >= 0).sum())
        return [t.clone() for t in (self.out, self.dx, self.da, self.db, self.h[:n], self.rows[:n])]


def kinds():
    return [many(2700, 5, 16, 54, 1032, 328), many(3000, 6, 64, 55, 520, 264), few(700, 5, 24, 56, 520, 328),
            many(900, 4, 88, 57, 264, 520)]


def test_a_captured_call_replayed_with_other_adapters():
    for c in kinds():
        step = Step(c)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        step.run(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step.run(side)
        T = c.idx.shape[0]
        for k, other in enumerate((ids(T, c.E, 60, none=0.3), torch.full((T, 1), c.E - 1), torch.full((T, 1), -1),
                                   ids(T, c.E, 61, none=0.0))):
            step.idx.copy_(other)
            for t in (step.out, step.dx, step.da, step.db, step.h, step.dh):
                t.fill_(math.nan)
            graph.replay()
            torch.cuda.synchronize()
            got = step.outputs()
            fresh = Step(c)
            fresh.idx.copy_(other)
            torch.cuda.synchronize()
            fresh.run(torch.cuda.current_stream())
            torch.cuda.synchronize()
            for a, b in zip(got, fresh.outputs()):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
            assert B.ep_get_device_error(step.layout) == 0
        del graph


def test_calls_on_two_streams_at_once():
    """Calls of every kind of kernel beside one another, the one's tensor memory
    and clusters beside the other's."""
    cases = kinds()
    alone = []
    steps = [Step(c) for c in cases]
    for s in steps:
        s.run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append(s.outputs())
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(12):
        for s, q in zip(steps, streams):
            s.run(q)
    torch.cuda.synchronize()
    for s, want in zip(steps, alone):
        for a, b in zip(s.outputs(), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert B.ep_get_device_error(s.layout) == 0


def test_factor_gradients_past_2_31_elements():
    """1024 adapters whose factors hold more than 2^31 values together: the last
    ones', and those of no rows."""
    E, rank, hin, hout = 1024, 128, 16392, 8
    at = torch.tensor([0, 1, 511, 512, 1022, 1023])
    idx = at[torch.arange(100) % 6][:, None]
    g = torch.Generator(device="cuda").manual_seed(62)
    a = torch.zeros((E, rank, hin), dtype=torch.bfloat16, device="cuda")
    assert a.numel() > 2 ** 31
    a[at.cuda()] = (torch.randn((6, rank, hin), generator=g, device="cuda") / 128).to(torch.bfloat16)
    b = torch.randn((E, hout, rank), generator=g, device="cuda").to(torch.bfloat16)
    x = torch.randn((100, hin), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((100, hout), generator=g, device="cuda").to(torch.bfloat16)
    routing = B.Routing.topk(idx.cuda(), E, 1)
    layout = B.ep_get_layout(routing, B.Layout(routing))
    rows = torch.empty(100, dtype=torch.int32, device="cuda")
    B.ep_row_tokens(routing, layout, rows)
    lora = B.Lora(a, b)
    h, dh = torch.empty((100, rank), device="cuda"), torch.empty((100, rank), device="cuda")
    out, dx = torch.empty_like(dy), torch.empty_like(x)
    da, db = torch.full_like(a, 5.0), torch.full_like(b, 5.0)
    B.ep_lora(x, routing, layout, lora, out, h, row_token=rows)
    B.ep_lora_backward(dy, x, h, routing, layout, lora, dh, dx=dx, da=da, db=db, row_token=rows)
    used = torch.zeros(E, dtype=torch.bool, device="cuda")
    used[at.cuda()] = True
    assert not bool(da[~used].any()) and not bool(db[~used].any())
    for e in at.tolist():
        t = (idx[:, 0] == e).nonzero().squeeze(1).cuda()
        hw = x[t].double() @ a[e].double().T
        g_h = dy[t].double() @ b[e].double()
        for got, want, size in ((out[t], hw @ b[e].double().T, hw.abs() @ b[e].double().abs().T),
                                (dx[t], g_h @ a[e].double(), g_h.abs() @ a[e].double().abs()),
                                (da[e], g_h.T @ x[t].double(), g_h.abs().T @ x[t].double().abs()),
                                (db[e], dy[t].double().T @ hw, dy[t].double().abs().T @ hw.abs())):
            # the rounding to bf16, and 2^-18 of the terms' sizes for the sums of fp32
            assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size)
