"""How exact the low-rank products are: fp32 operands enter the tensor core with
all of their bits, and sums do not lose bits with their length."""
import math

import pytest
import torch

from combine_ep_get_10_b200 import binding as B
from lora_paths import few_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


def rows_of(ids, E):
    routing = B.Routing.topk(ids[:, None].contiguous().cuda(), E, 1)
    layout = B.ep_get_layout(routing, B.Layout(routing))
    rows = torch.empty(int((ids >= 0).sum()), dtype=torch.int32, device="cuda")
    B.ep_row_tokens(routing, layout, rows)
    return routing, layout, rows


def bf(t):
    return t.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("T", [40, 2100])
def test_products_with_h_and_dh_keep_every_bit(rank, T):
    """h of (1 + 2^-9 + 2^-20, 2^-9), the second one taken from the first, beside a
    base of -1 leaves 2^-20, exactly; two bf16 terms of h (1 and 2^-9) would leave
    0.  Every token on its own scale; the same for dx."""
    hin, hout, E = 136, 72, 2
    ids = torch.arange(T) % E
    routing, layout, rows = rows_of(ids, E)
    scale = 2.0 ** (torch.arange(T) % 5).float() * (1 - 2 * (torch.arange(T) % 2)).float()
    even = (torch.arange(rank) % 2 == 0).float()

    def factors(inner, outer):
        down, up = torch.zeros(rank, inner), torch.zeros(outer, rank)
        down[:, 0], down[:, 1], down[:, 2] = even, 2.0 ** -10 * even, 1.0
        pair = 2 * (torch.arange(outer) % (rank // 2))
        up[torch.arange(outer), pair], up[torch.arange(outer), pair + 1] = 1.0, -1.0
        x = torch.zeros(T, inner)
        x[:, 0], x[:, 1], x[:, 2] = scale, scale * 2.0 ** -10, scale * 2.0 ** -9
        return x, down, up, (scale * 2.0 ** -20)[:, None].expand(T, outer)

    x, a, b, want = factors(hin, hout)
    lora = B.Lora(bf(a.expand(E, -1, -1).contiguous()), bf(b.expand(E, -1, -1).contiguous()))
    h = torch.empty((T, rank), device="cuda")
    out = bf((-scale[:, None]).expand(T, hout))
    B.ep_lora(bf(x), routing, layout, lora, out, h, base=out, row_token=rows)
    assert torch.equal(h.cpu()[:, 0].abs().unique(), (2.0 ** torch.arange(5).float()) * (1 + 2.0 ** -9 + 2.0 ** -20))
    assert torch.equal(out.float().cpu(), want)
    dy, b, a, want = factors(hout, hin)
    lora = B.Lora(bf(a.T.expand(E, -1, -1).contiguous()), bf(b.T.expand(E, -1, -1).contiguous()))
    dx = bf((-scale[:, None]).expand(T, hin))
    B.ep_lora_backward(bf(dy), None, None, routing, layout, lora, h, dx=dx, dx_base=dx, row_token=rows)
    assert torch.equal(dx.float().cpu(), want)


@pytest.mark.parametrize("rank", [8, 32, 40, 128])
def test_factor_gradients_keep_every_bit(rank):
    """Three rows an adapter of which the second and third take most of the first
    away: da = (1 + 2^-9 + 2^-20) - 1 - 2^-9, db the same with 2^-23."""
    E, hin, hout = 5, 136, 72
    T = 3 * E
    ids = torch.arange(T) % E
    routing, layout, rows = rows_of(ids, E)
    third = torch.arange(T) // E
    b = torch.zeros(E, hout, rank)
    b[:, 0], b[:, 1], b[:, 2] = 1.0, 2.0 ** -10, 1.0
    dy = torch.zeros(T, hout)
    dy[:, 0] = torch.tensor([1.0, -1.0, 0.0])[third]
    dy[:, 1] = torch.tensor([2.0 ** -10, 0.0, 0.0])[third]
    dy[:, 2] = torch.tensor([2.0 ** -9, 0.0, -2.0 ** -9])[third]
    dy[:, 3] = torch.tensor([1.0, -1.0, -1.0])[third]
    by_token = torch.tensor([1 + 2.0 ** -9 + 2.0 ** -23, 1.0, 2.0 ** -9])[third]
    h = by_token[rows.cpu().long()][:, None].expand(T, rank).contiguous().cuda()
    dh = torch.empty_like(h)
    lora = B.Lora(torch.zeros((E, rank, hin), dtype=torch.bfloat16, device="cuda"), bf(b))
    da, db = torch.empty_like(lora.a), torch.empty_like(lora.b)
    B.ep_lora_backward(bf(dy), torch.ones((T, hin), dtype=torch.bfloat16, device="cuda"), h, routing, layout, lora, dh,
                       da=da, db=db, row_token=rows)
    assert bool((da.float() == 2.0 ** -20).all())
    assert bool((db[:, 3].float() == 2.0 ** -23).all())


@pytest.mark.parametrize("rank,T,E,hin", [(16, 64, 8, 7168), (64, 2000, 128, 7168), (16, 2100, 1, 16384),
                                          (32, 6000, 80, 7168), (64, 7000, 300, 4096), (128, 3000, 200, 8192)])
def test_long_sums_stay_as_exact_as_short_ones(rank, T, E, hin):
    """h of both kinds of kernels against 64 bits, in the 2-norm.  A chain of 16
    products on the tensor core is off by at most 2^-23 of the sum so far at each
    step, 2^-24 on average: 16 * 2^-24 of the chain's own size.  Chains are
    added in fp32: 2^-24 for each of n / 256 additions (one kernel's chains, n / 16
    / 8 of 16 terms each, are half as long), of random sign.  One chain of n / 16
    would be off by n / 64 * 2^-24 and more, all towards zero."""
    g = torch.Generator(device="cuda").manual_seed(rank)
    ids = torch.randint(0, E, (T,), generator=torch.Generator().manual_seed(T))
    routing, layout, rows = rows_of(ids, E)
    x = torch.randn((T, hin), generator=g, device="cuda").to(torch.bfloat16)
    a = (torch.randn((E, rank, hin), generator=g, device="cuda") / math.sqrt(hin)).to(torch.bfloat16)
    lora = B.Lora(a, torch.zeros((E, 8, rank), dtype=torch.bfloat16, device="cuda"))
    h = torch.empty((T, rank), device="cuda")
    out = torch.empty((T, 8), dtype=torch.bfloat16, device="cuda")
    B.ep_lora(x, routing, layout, lora, out, h, row_token=rows)
    at = rows.long()
    want = torch.empty((T, rank), dtype=torch.float64, device="cuda")
    ad = ids.cuda()[at]
    for e in range(E):
        sel = (ad == e).nonzero().squeeze(1)
        want[sel] = x[at[sel]].double() @ a[e].double().T
    err = float((h.double() - want).norm() / want.norm())
    tol = (16 + math.sqrt(hin / 128)) * 2.0 ** -24
    assert err <= tol, "%s: %.3g, tolerance %.3g" % ("few" if few_rows(T, E, rank) else "many", err, tol)


@pytest.mark.parametrize("rank", [16, 32, 64, 128])
@pytest.mark.parametrize("E", [1, 64])
def test_sums_over_many_rows_stay_exact(rank, E):
    """db of 16384 equal rows and one that takes them all away again (values of 8
    and 24 bits, so that every addition has bits to cut): what is left is the sums'
    error.  A chain of 16 products (256 rows) is off by at most
    16 * 2^-23 of its own sum, the additions of the chains by 2^-24 of the sum so
    far each: n * h * (32 + 64) * 2^-24 at most, with the row that takes away n * h
    as much in one addition.  One chain of 1024 would be off by some 500 n h 2^-24."""
    n = 16384
    ids = torch.zeros(n + 1, dtype=torch.int64)
    routing, layout, rows = rows_of(ids, E)
    h1 = 1 + torch.rand(rank, generator=torch.Generator().manual_seed(rank))
    h = h1.expand(n + 1, rank).contiguous().cuda()
    d = 1 + 127 / 128
    dy = torch.full((n + 1, 72), d, dtype=torch.bfloat16, device="cuda")
    dy[n] = -d * n
    lora = B.Lora(torch.zeros((E, rank, 72), dtype=torch.bfloat16, device="cuda"),
                  torch.zeros((E, 72, rank), dtype=torch.bfloat16, device="cuda"))
    da, db = torch.empty_like(lora.a), torch.empty_like(lora.b)
    B.ep_lora_backward(dy, torch.zeros((n + 1, 72), dtype=torch.bfloat16, device="cuda"), h, routing, layout, lora,
                       torch.empty_like(h), da=da, db=db, row_token=rows)
    off = float((db[0].float().abs() / (n * d * h1.cuda())).max())
    assert off <= (32 + 64 + 2) * 2.0 ** -24, off * 2 ** 24
    assert not bool(da.any())
