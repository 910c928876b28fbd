"""Low-rank adapters and their gradients against 64 bits (lora_ref): ranks,
widths, group sizes from none to many tiles, tokens without an adapter, the
compact and padded rows of a dispatch, in place and not, streams, graphs,
guard bytes, bad row tables.

Tolerances.  A product sums n terms a * b of bf16 operands, exact in fp32, in
fp32: the tensor core may cut each addition's aligned terms at 24 bits, so an
error of at most 2^-23 of the sum of the terms' sizes S for each of about n / 16
chained additions, and 2^-24 of S for each of the few sums of parts.  These
inputs have random signs, so partial sums stay below about S / sqrt(n) times
a small factor and the errors do not all point one way; the bound used is
sqrt(n) * 2^-23 * S, n the length of the sum.  An fp32 operand enters as two
bf16 terms and loses 2^-17 of each product: 2^-17 * S more.  A bf16 result is
rounded once: 2^-8 of itself."""
import math

import pytest
import torch

import lora_ref
from combine_ep_get_10_b200 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


def close(got, want, size, n, split, what):
    tol = (math.sqrt(n) * 2.0 ** -23 + (2.0 ** -17 if split else 0.0)) * size + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.cpu().double() - want).abs()
    assert torch.all(err <= tol), "%s: %g times the tolerance" % (what, float((err / tol).max()))


class Case:
    def __init__(self, idx, E, r, hin, hout, seed, *, tokens=True, scales=True, mode=B.EP_LAYOUT_COMPACT, max_tokens=0,
                 num_rows=None):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        T, K = idx.shape
        self.idx, self.E, self.r, self.hin, self.hout, self.tokens = idx, E, r, hin, hout, tokens
        self.kw = dict(mode=mode, max_tokens_per_expert=max_tokens)
        pairs = int(((idx >= 0) & (idx < E)).sum())
        self.num_rows = num_rows if num_rows is not None else (pairs if mode == 0 else E * max_tokens)
        n = T if tokens else self.num_rows
        self.x = torch.randn((n, hin), generator=g).to(bf)
        self.dy = torch.randn((n, hout), generator=g).to(bf)
        self.base = torch.randn((n, hout), generator=g).to(bf)
        self.dx_base = torch.randn((n, hin), generator=g).to(bf)
        self.a = (torch.randn((E, r, hin), generator=g) / math.sqrt(hin)).to(bf)
        self.b = (torch.randn((E, hout, r), generator=g) / math.sqrt(r)).to(bf)
        self.scales = torch.rand(E, generator=g) + 0.25 if scales else None
        self.ref = lora_ref.Ref(idx, self.a, self.b, self.scales, self.num_rows, tokens, mode, max_tokens)
        self.routing = B.Routing.topk(idx.cuda(), E, 1)
        self.layout = B.ep_get_layout(self.routing, B.Layout(self.routing))
        self.lora = B.Lora(self.a.cuda(), self.b.cuda(), None if self.scales is None else self.scales.cuda())
        self.row_token = None
        if tokens:
            self.row_token = torch.full((self.num_rows,), 99, dtype=torch.int32, device="cuda")
            B.ep_row_tokens(self.routing, self.layout, self.row_token, **self.kw)
        self.kw["row_token"] = self.row_token

    def forward(self, base="separate", stream=None):
        out = torch.full((self.x.shape[0], self.hout), 5.0, dtype=torch.bfloat16, device="cuda")
        if base == "in place":
            out.copy_(self.base)
        h = torch.zeros((self.num_rows, self.r), device="cuda")
        at = {"separate": self.base.cuda(), "in place": out, "none": None}[base]
        torch.cuda.synchronize()
        B.ep_lora(self.x.cuda(), self.routing, self.layout, self.lora, out, h, base=at, stream=stream, **self.kw)
        torch.cuda.synchronize()
        return out, h

    def check_forward(self, base="separate"):
        out, h = self.forward(base)
        before = torch.full((self.x.shape[0], self.hout), 5.0, dtype=torch.bfloat16)
        if base == "in place":
            before = self.base
        want, hw, size, hsize = self.ref.forward(self.x, None if base == "none" else self.base, before)
        close(h, hw, hsize, self.hin, False, "h")
        close(out, want, size, self.hin + self.r, True, "out")

    def backward(self, h, dx_base="separate", want=("dx", "da")):
        dx = torch.full((self.x.shape[0], self.hin), 5.0, dtype=torch.bfloat16, device="cuda")
        if dx_base == "in place":
            dx.copy_(self.dx_base)
        at = {"separate": self.dx_base.cuda(), "in place": dx, "none": None}[dx_base]
        da = torch.full(self.a.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        db = torch.full(self.b.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        dh = torch.zeros((self.num_rows, self.r), device="cuda")
        both = "da" in want
        B.ep_lora_backward(self.dy.cuda(), self.x.cuda() if both else None, h if both else None, self.routing,
                           self.layout, self.lora, dh, dx=dx if "dx" in want else None, da=da if both else None,
                           db=db if both else None, dx_base=at, **self.kw)
        torch.cuda.synchronize()
        return dx, da, db

    def check_backward(self, dx_base="separate", want=("dx", "da")):
        _, h, _, _ = self.ref.forward(self.x, None, torch.zeros((self.x.shape[0], self.hout)))
        h = h.float()
        dx, da, db = self.backward(h.cuda(), dx_base, want)
        before = torch.full((self.x.shape[0], self.hin), 5.0, dtype=torch.bfloat16)
        if dx_base == "in place":
            before = self.dx_base
        (rdx, rda, rdb), (sdx, sda, sdb) = self.ref.backward(self.dy, self.x, h,
                                                             None if dx_base == "none" else self.dx_base, before)
        most = max(1, max(r.numel() for _, r, _ in self.ref.groups))
        if "dx" in want:
            close(dx, rdx, sdx, self.hout + self.r, True, "dx")
        else:
            assert bool((dx == (5.0 if dx_base != "in place" else dx)).all())
        if "da" in want:
            close(da, rda, sda, self.hout + most, True, "da")
            close(db, rdb, sdb, most, True, "db")


def ids(T, E, seed, none=0.1, K=1):
    g = torch.Generator().manual_seed(seed)
    if K == 1:
        idx = torch.randint(0, E, (T, 1), generator=g)
    else:
        idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) if T else torch.empty((0, K),
                                                                                                     dtype=torch.int64)
    idx[torch.rand((T, K), generator=g) < none] = -1
    return idx


SHAPES = [(1, 1, 8, 8, 8), (1, 4, 16, 64, 72), (5, 3, 24, 136, 40), (64, 1, 32, 256, 256), (65, 2, 40, 264, 520),
          (200, 7, 64, 512, 264), (130, 40, 16, 1032, 128), (333, 5, 128, 320, 776), (700, 3, 72, 128, 64),
          (97, 1000, 8, 96, 96), (300, 1024, 16, 64, 48)]


@pytest.mark.parametrize("T,E,r,hin,hout", SHAPES)
def test_forward_over_shapes(T, E, r, hin, hout):
    c = Case(ids(T, E, 1), E, r, hin, hout, 2)
    for base in ("separate", "in place", "none"):
        c.check_forward(base)


@pytest.mark.parametrize("T,E,r,hin,hout", SHAPES)
def test_backward_over_shapes(T, E, r, hin, hout):
    c = Case(ids(T, E, 3), E, r, hin, hout, 4, scales=T % 2 == 0)
    for base in ("separate", "in place", "none"):
        c.check_backward(base)
    c.check_backward(want=("dx",))
    c.check_backward(want=("da",))
    c.check_backward(want=())


@pytest.mark.parametrize("rank", list(range(8, 129, 8)))
def test_every_rank(rank):
    c = Case(ids(150, 4, rank), 4, rank, 200, 152, 5)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("mode,mt", [(B.EP_LAYOUT_COMPACT, 0), (B.EP_LAYOUT_PADDED, 40), (B.EP_LAYOUT_PADDED, 9)])
@pytest.mark.parametrize("E,K", [(16, 4), (3, 2)])
def test_dispatched_rows(mode, mt, E, K):
    """x, base and out are the rows of a dispatch; rows of no pair keep what
    they held, a padded buffer that is full drops the rest."""
    c = Case(ids(60, E, 6, none=0.2, K=K), E, 32, 136, 264, 7, tokens=False, mode=mode, max_tokens=mt)
    for base in ("separate", "in place", "none"):
        c.check_forward(base)
        c.check_backward(base)
    assert B.ep_get_device_error(c.layout) == (B.EP_DEVERR_OVERFLOW if mt and c.layout.num_tokens_per_expert.max() > mt
                                               else 0)


def test_padded_rows_with_a_row_table():
    c = Case(ids(90, 6, 8), 6, 16, 128, 136, 9, mode=B.EP_LAYOUT_PADDED, max_tokens=30)
    c.check_forward()
    c.check_backward()
    assert B.ep_get_device_error(c.layout) == 0


def test_skewed_groups_and_groups_without_rows():
    idx = torch.zeros((500, 1), dtype=torch.int64)
    idx[:3] = 5
    idx[3:7] = -1
    idx[450:] = 63
    c = Case(idx, 64, 32, 256, 512, 10)
    c.check_forward()
    c.check_backward()


def test_no_rows_at_all():
    for T in (0, 70):
        c = Case(torch.full((T, 1), -1, dtype=torch.int64), 3, 16, 64, 72, 11)
        assert c.num_rows == 0
        c.check_forward()
        c.check_forward("none")
        c.check_backward()


def test_row_buffer_too_small_is_flagged():
    idx = ids(100, 4, 12, none=0.0)
    full = Case(idx, 4, 16, 128, 128, 13)
    for rows in (0, 37):
        c = Case(idx, 4, 16, 128, 128, 13, tokens=False, num_rows=rows)
        B.ep_get_device_error(c.layout)
        c.check_forward()
        assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_OVERFLOW
        c.check_backward()
        assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_OVERFLOW
    assert B.ep_get_device_error(full.layout) == 0


def test_bad_row_tokens_are_skipped_and_flagged():
    c = Case(ids(100, 4, 14, none=0.0), 4, 16, 128, 128, 15)
    out, h = c.forward()
    good = c.row_token.clone()
    bad = [3, 64, 99]
    tokens = good[bad].tolist()
    c.row_token[bad] = torch.tensor([-1, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out2, h2 = c.forward()
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_BAD_INDEX
    keep = torch.ones(100, dtype=torch.bool)
    keep[tokens] = False
    assert torch.equal(out2.cpu()[keep], out.cpu()[keep])
    assert bool((out2.cpu()[tokens] == 5.0).all())  # no row, and not a token without an adapter
    rows = torch.ones(100, dtype=torch.bool)
    rows[bad] = False
    assert torch.equal(h2.cpu()[rows], h.cpu()[rows]) and not bool(h2.cpu()[bad].any())
    h2[bad] = math.nan  # a row that is skipped does not count in da, db
    dx, da, db = c.backward(h2)
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_BAD_INDEX
    assert not bool(da.isnan().any()) and not bool(db.isnan().any())


def test_infinities_stay_in_their_rows():
    c = Case(ids(80, 2, 16, none=0.0), 2, 16, 72, 64, 17)
    clean, _ = c.forward()
    c.x[7, 3], c.x[9, 5] = math.inf, math.nan
    out, _ = c.forward()
    rows = torch.ones(80, dtype=torch.bool)
    rows[[7, 9]] = False
    assert torch.equal(out.cpu()[rows], clean.cpu()[rows])
    want = (c.base[7].double() + c.ref.s[c.idx[7, 0]] *
            ((c.x[7].double() @ c.ref.a[c.idx[7, 0]].T) @ c.ref.b[c.idx[7, 0]].T))
    got = out.cpu()[7].double()
    # an infinite h gives infinities or NaN where 64 bits do
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    assert bool(out.cpu()[9].isnan().all())


def test_row_tokens_equal_the_dispatch():
    for mode, mt in ((B.EP_LAYOUT_COMPACT, 0), (B.EP_LAYOUT_PADDED, 11)):
        idx = ids(77, 9, 18, none=0.2, K=3)
        routing = B.Routing.topk(idx.cuda(), 9, 3)
        layout = B.ep_get_layout(routing, B.Layout(routing))
        rows = int((idx >= 0).sum()) if mode == 0 else 9 * mt
        src = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        recv = torch.empty((rows, 64), dtype=torch.bfloat16, device="cuda")
        B.ep_dispatch(torch.zeros((77, 64), dtype=torch.bfloat16, device="cuda"), routing, layout, recv, mode=mode,
                      max_tokens_per_expert=mt, recv_src=src)
        flags = B.ep_get_device_error(layout)
        got = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
        B.ep_row_tokens(routing, layout, got, mode=mode, max_tokens_per_expert=mt)
        assert torch.equal(got, src)
        assert B.ep_get_device_error(layout) == flags


def test_same_bytes_every_time_on_a_side_stream_and_in_a_graph():
    c = Case(ids(600, 6, 19), 6, 32, 1024, 520, 20)
    out, h = c.forward()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out2, h2 = c.forward(stream=side)
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16)) and torch.equal(h, h2)
    x, base, dy, dxb = c.x.cuda(), c.base.cuda(), c.dy.cuda(), c.dx_base.cuda()
    dx, da, db = torch.empty_like(x), torch.empty_like(c.lora.a), torch.empty_like(c.lora.b)
    dh, o3, h3 = torch.empty_like(h), torch.empty_like(out), torch.empty_like(h)

    def step(stream):
        B.ep_get_layout(c.routing, c.layout, stream=stream)
        B.ep_row_tokens(c.routing, c.layout, c.row_token, stream=stream)
        B.ep_lora(x, c.routing, c.layout, c.lora, o3, h3, base=base, row_token=c.row_token, stream=stream)
        B.ep_lora_backward(dy, x, h3, c.routing, c.layout, c.lora, dh, dx=dx, da=da, db=db, dx_base=dxb,
                           row_token=c.row_token, stream=stream)

    torch.cuda.synchronize()
    step(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in (o3, h3, dx, da, db)]
    assert torch.equal(eager[0].view(torch.int16), out.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for _ in range(3):
        for t in (o3, h3, dx, da, db, dh):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o3, h3, dx, da, db), eager):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    """<gradient, direction> equals the central difference of sum(dy * out) in
    64 bits: the objective is linear in x, in a and in b, so the difference is
    exact and what is left is the gradient's own rounding."""
    c = Case(ids(120, 3, 21), 3, 24, 136, 120, 22)
    _, h, _, _ = c.ref.forward(c.x, None, torch.zeros((120, c.hout)))
    dx, da, db = c.backward(h.float().cuda(), "none")
    g = torch.Generator().manual_seed(23)
    zero = torch.zeros((120, c.hout))

    def value(x, a, b):
        r = lora_ref.Ref(c.idx, c.a, c.b, c.scales, c.num_rows, True)
        r.a, r.b = a, b
        return float((c.dy.double() * r.forward(x, None, zero)[0]).sum())

    x, a, b = c.x.double(), c.a.double(), c.b.double()
    for name, grad, f in (("dx", dx, lambda u, s: value(x + s * u, a, b)), ("da", da, lambda u, s: value(x, a + s * u, b)),
                          ("db", db, lambda u, s: value(x, a, b + s * u))):
        u = torch.randn(grad.shape, generator=g, dtype=torch.float64)
        slope = (f(u, 1.0) - f(u, -1.0)) / 2
        got = (grad.cpu().double() * u)
        # every element is off by at most 2^-8 of itself (bf16) and 2^-12 of the largest one
        tol = 2.0 ** -8 * float(got.abs().sum()) + 2.0 ** -12 * float(grad.abs().max()) * float(u.abs().sum())
        assert abs(float(got.sum()) - slope) <= tol, name


def test_outputs_stay_in_bounds():
    from test_gpu_canary import Guarded, _check

    c = Case(ids(83, 5, 24), 5, 24, 136, 264, 25)
    T, bf = 83, torch.bfloat16
    out, dx = Guarded((T, 264), bf), Guarded((T, 136), bf)
    h, dh = Guarded((c.num_rows, 24), torch.float32), Guarded((c.num_rows, 24), torch.float32)
    da, db = Guarded(c.a.shape, bf), Guarded(c.b.shape, bf)
    rt = Guarded((c.num_rows,), torch.int32)
    B.ep_row_tokens(c.routing, c.layout, rt.t)
    B.ep_lora(c.x.cuda(), c.routing, c.layout, c.lora, out.t, h.t, base=c.base.cuda(), row_token=rt.t)
    B.ep_lora_backward(c.dy.cuda(), c.x.cuda(), h.t, c.routing, c.layout, c.lora, dh.t, dx=dx.t, da=da.t, db=db.t,
                       row_token=rt.t)
    torch.cuda.synchronize()
    _check(out, dx, h, dh, da, db, rt)


def test_large_row_offsets():
    """Rows past 2^31 elements: x and out hold T * H > 2^31 values, the routed
    tokens lie at both ends."""
    T, hin, hout, E = 310000, 7168, 8, 2
    idx = torch.full((T, 1), -1, dtype=torch.int64)
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1])
    idx[at, 0] = torch.tensor([0, 1, 0, 1, 0])
    g = torch.Generator().manual_seed(26)
    few = torch.randn((5, hin), generator=g).to(torch.bfloat16)
    x = torch.empty((T, hin), dtype=torch.bfloat16, device="cuda")
    x[at.cuda()] = few.cuda()
    a = (torch.randn((E, 16, hin), generator=g) / 80).to(torch.bfloat16)
    b = torch.randn((E, hout, 16), generator=g).to(torch.bfloat16)
    routing = B.Routing.topk(idx.cuda(), E, 1)
    layout = B.ep_get_layout(routing, B.Layout(routing))
    row_token = torch.empty(5, dtype=torch.int32, device="cuda")
    B.ep_row_tokens(routing, layout, row_token)
    out, h = torch.empty((T, hout), dtype=torch.bfloat16, device="cuda"), torch.empty((5, 16), device="cuda")
    lora = B.Lora(a.cuda(), b.cuda())
    B.ep_lora(x, routing, layout, lora, out, h, row_token=row_token)
    ref = lora_ref.Ref(idx[at], a, b, None, 5, True)
    want, _, size, _ = ref.forward(few, None, torch.zeros((5, hout)))
    close(out[at.cuda()], want, size, hin + 16, True, "out")
    dy = torch.zeros((T, hout), dtype=torch.bfloat16, device="cuda")
    dyf = torch.randn((5, hout), generator=g).to(torch.bfloat16)
    dy[at.cuda()] = dyf.cuda()
    dx = x  # in place, on what x held: the shared projection's gradient
    dh = torch.empty((5, 16), device="cuda")
    B.ep_lora_backward(dy, None, None, routing, layout, lora, dh, dx=dx, dx_base=dx, row_token=row_token)
    (rdx, _, _), (sdx, _, _) = ref.backward(dyf, few, torch.zeros((5, 16)), few, torch.zeros((5, hin)))
    close(dx[at.cuda()], rdx, sdx, hout + 16, True, "dx")


@pytest.mark.parametrize("rank", [16, 24, 64, 72, 128])
def test_long_runs_of_stages(rank):
    """More steps a CTA than it has stages, for each of the three products:
    many adapters (no tile's columns or hidden width is split), then long groups."""
    c = Case(ids(340, 300, 27), 300, rank, 1160, 1096, 28)
    c.check_forward()
    c.check_backward(want=("dx",))
    c = Case(ids(1500, 2, 29), 2, rank, 136, 264, 30)
    c.check_forward()
    c.check_backward()


def test_shares_of_uneven_tiles():
    """Adapters of very different sizes, where the column steps of a tile are
    shared out by its rows: every share is worked on."""
    g = torch.Generator().manual_seed(31)
    for E, sizes in ((9, (1, 127, 128, 129, 3, 260, 64, 0, 31)), (40, None)):
        if sizes is None:
            sizes = torch.randint(0, 90, (E,), generator=g).tolist()
        idx = torch.cat([torch.full((n,), e, dtype=torch.int64) for e, n in enumerate(sizes)])
        idx = idx[torch.randperm(idx.numel(), generator=g)][:, None]
        for hout in (2056, 8):
            c = Case(idx, E, 16, 72, hout, 32)
            c.check_forward()
            c.check_backward(want=("dx",))


@pytest.mark.parametrize("rank", [8, 40, 64, 96])
def test_bad_row_tokens_at_every_rank(rank):
    """Entries of no token in several stages and tiles: their rows are zeros in
    h, their tokens keep what they held, no gradient sees them."""
    c = Case(ids(400, 2, 33, none=0.0), 2, rank, 264, 136, 34)
    out, h = c.forward()
    dx, da, db = c.backward(h)
    bad = torch.tensor([0, 5, 63, 64, 130, 199, 200, 399])
    tokens = c.row_token.cpu()[bad].long()
    c.row_token[bad.cuda()] = torch.tensor([-1, 400, -5, 2 ** 31 - 1, -2 ** 31, 400, 401, -1], dtype=torch.int32,
                                           device="cuda")
    out2, h2 = c.forward()
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_BAD_INDEX
    keep = torch.ones(400, dtype=torch.bool)
    keep[tokens] = False
    assert torch.equal(out2.cpu()[keep], out.cpu()[keep]) and bool((out2.cpu()[tokens] == 5.0).all())
    assert not bool(h2.cpu()[bad].any())
    c.x[tokens] = math.nan
    c.dy[tokens] = math.inf
    h2[bad.cuda()] = math.nan
    dx2, da2, db2 = c.backward(h2)
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_BAD_INDEX
    assert torch.equal(dx2.cpu()[keep], dx.cpu()[keep])
    assert bool(torch.isfinite(da2).all()) and bool(torch.isfinite(db2).all())


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 88, 128])
@pytest.mark.parametrize("T,E", [(1, 7), (16, 1), (90, 9), (130, 70)])
def test_few_rows_an_adapter(rank, T, E):
    """Sixteen rows an adapter and less, one more than that for some: widths that
    end inside a block of 32, base in place, missing and separate, rows that no
    pair names, entries of no token."""
    for hin, hout in ((8, 40), (1000, 72), (4104, 1048)):
        c = Case(ids(T, E, rank, none=0.15), E, rank, hin, hout, 35)
        for base in ("separate", "in place", "none"):
            c.check_forward(base)
    c = Case(ids(T, E, rank, none=0.3), E, rank, 264, 136, 36, tokens=False, mode=B.EP_LAYOUT_PADDED, max_tokens=5)
    c.check_forward()
    assert (B.ep_get_device_error(c.layout) != 0) == bool(c.layout.num_tokens_per_expert.max() > 5)
    if T > 20:
        c = Case(ids(T, E, rank, none=0.0), E, rank, 264, 136, 37)
        out, h = c.forward()
        bad = torch.tensor([1, 8, T - 1])
        tokens = c.row_token.cpu()[bad].long()
        c.row_token[bad.cuda()] = torch.tensor([-1, T, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        out2, h2 = c.forward()
        assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_BAD_INDEX
        keep = torch.ones(T, dtype=torch.bool)
        keep[tokens] = False
        assert torch.equal(out2.cpu()[keep], out.cpu()[keep]) and bool((out2.cpu()[tokens] == 5.0).all())
        assert not bool(h2.cpu()[bad].any())


@pytest.mark.parametrize("rank", [8, 32, 56, 128])
def test_gradients_of_long_groups_in_parts(rank):
    """One adapter, or a few of very different sizes, whose rows several CTAs
    share: every part counts, empty ones too, and the sums are the same bytes
    every time."""
    for idx in (torch.zeros((1900, 1), dtype=torch.int64), ids(1700, 1, 38, none=0.2),
                torch.cat([torch.zeros(2400), torch.ones(3), torch.full((200,), 2.0), torch.full((70,), -1.0)])
                .long()[torch.randperm(2673, generator=torch.Generator().manual_seed(39))][:, None]):
        c = Case(idx, int(idx.max()) + 1, rank, 136, 328, 40)
        c.check_backward()
        _, h, _, _ = c.ref.forward(c.x, None, torch.zeros((c.x.shape[0], c.hout)))
        first, again = (c.backward(h.float().cuda()) for _ in range(2))
        for a, b in zip(first, again):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_both_sides_of_the_choice_of_kernels():
    """Forward calls just within and just past the limits in rows at which the
    kernel for few rows gives way to those for many."""
    for rank, E, T in ((16, 1, 2048), (16, 1, 2049), (32, 3, 2048), (32, 3, 2049), (64, 2, 128), (64, 2, 129),
                       (8, 9, 2304), (8, 9, 2305), (40, 20, 320), (40, 20, 321), (72, 20, 40)):
        c = Case(ids(T, E, T, none=0.05), E, rank, 136, 200, 41)
        c.check_forward()
        c.check_forward("in place")


def test_a_part_of_a_routing_with_the_whole_layout_is_flagged_or_refused():
    c = Case(ids(700, 4, 42, none=0.0), 4, 16, 128, 128, 43, tokens=False)
    part = c.routing.tokens(0, 100)
    out, h = torch.zeros((c.num_rows, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((c.num_rows, 16), device="cuda")
    B.ep_lora(c.x.cuda(), c.routing, c.layout, c.lora, out, h)
    assert B.ep_get_device_error(c.layout) == 0
    B.ep_lora(c.x.cuda(), part, c.layout, c.lora, out, h)
    assert B.ep_get_device_error(c.layout) == B.EP_DEVERR_OVERFLOW
    with pytest.raises(ValueError):
        B.ep_lora(c.x.cuda(), part, B.layout_tokens(c.layout, c.routing, 0, 100), c.lora, out, h)
