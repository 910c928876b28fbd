"""The router, the balance losses and the gradient of the logits against the
64-bit definitions (router_ref), over sizes, types, groups, biases, masks and
rows with nothing open; in streams and captured graphs.

Tolerances (u = 2^-24, fp32's half ulp).  A weight is a ratio of exponentials
or sigmoids: expf is within 2 ulp = 4u, its argument l - max is rounded by u of
its size (|l - max| <= 40 in these inputs: 40u), a sum of up to E = 1024
terms in 32 lanes of 32 adds 37u, and the rest (quotient, scale, 1 + e) a few u:
below 128u = 7.7e-6 of the value.  A gradient is a sum of products of such
factors with differences g - mean, whose error is relative to the size of g
and mean, not of the difference: below 4 * 128u of the row's largest term,
2^-8 of the value more for bf16."""
import math

import pytest
import torch

import router_ref as ref
from combine_ep_get_10_b200 import binding as B

pytestmark = pytest.mark.gpu

RTOL = 128 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


def make(T, E, dtype, seed, closed=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) * spread + 0.5 * torch.randn((1, E), generator=g)
    l[torch.rand((T, E), generator=g) < closed] = -math.inf
    return l.to(dtype), g


def route(logits, K, sigmoid=False, bias=None, mask=None, groups=1, topk_groups=1, group_top=1, normalize=True,
          scale=1.0, stream=None):
    T, E = logits.shape
    router = B.Router(E, K, score=B.EP_SCORE_SIGMOID if sigmoid else B.EP_SCORE_SOFTMAX, num_groups=groups,
                      topk_groups=topk_groups, group_top=group_top, normalize=normalize, scale=scale)
    idx = torch.full((T, K), 77, dtype=torch.int64, device="cuda")
    w = torch.full((T, K), 77.0, device="cuda")
    B.ep_router_topk(logits.cuda(), router, idx, w, bias=None if bias is None else bias.cuda(),
                     token_mask=None if mask is None else mask.cuda(), stream=stream)
    return idx.cpu(), w.cpu()


def check_route(logits, K, **kw):
    idx, w = route(logits, K, **kw)
    ridx, rw = ref.topk(logits, K, **kw)
    assert torch.equal(idx, ridx), (idx[(idx != ridx).any(dim=1)][:3], ridx[(idx != ridx).any(dim=1)][:3])
    # 2^-126: where a weight itself is below the normal range
    assert torch.all((w.double() - rw).abs() <= RTOL * rw.abs() + 2.0 ** -126), (w.double() - rw).abs().max()
    return idx, w


SIZES = [(1, 1, 1), (1, 8, 2), (7, 8, 8), (33, 60, 6), (130, 160, 6), (65, 256, 8), (9, 333, 3), (5, 1000, 32),
         (3, 1024, 32), (257, 32, 1), (6, 97, 31)]


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_topk_over_sizes(T, E, K, sigmoid, dtype):
    logits, g = make(T, E, dtype, 1)
    check_route(logits, K, sigmoid=sigmoid, normalize=True)
    check_route(logits, K, sigmoid=sigmoid, normalize=False, scale=2.5)
    check_route(logits, K, sigmoid=sigmoid, bias=0.3 * torch.randn(E, generator=g), scale=0.5)


@pytest.mark.parametrize("E,G,KG,K", [(8, 2, 1, 3), (64, 8, 3, 8), (160, 8, 3, 6), (256, 8, 4, 8), (256, 32, 5, 20),
                                      (1024, 4, 2, 32), (36, 4, 4, 7), (12, 4, 2, 6), (32, 32, 7, 7), (8, 8, 3, 2)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_topk_with_groups(E, G, KG, K, top, sigmoid):
    for seed, dtype, closed in [(2, torch.float32, 0.0), (3, torch.bfloat16, 0.0), (4, torch.float32, 0.5)]:
        logits, g = make(70, E, dtype, seed, closed)
        kw = dict(sigmoid=sigmoid, groups=G, topk_groups=KG, group_top=top)
        check_route(logits, K, **kw)
        check_route(logits, K, bias=0.2 * torch.randn(E, generator=g), normalize=False, **kw)


def test_topk_masks_closed_rows_and_strange_values():
    logits, g = make(40, 48, torch.float32, 5, closed=0.6)
    logits[3] = -math.inf  # nothing open
    logits[4, 1:] = -math.inf  # one expert open
    logits[5] = math.nan
    logits[6, 7] = math.nan  # one closed by NaN
    logits[7] = torch.finfo(torch.float32).min  # masked by the type's lowest value, all alike
    logits[8, 5:] = torch.finfo(torch.float32).min
    logits[9, 3] = math.inf
    logits[10] = -200.0 + logits[10].nan_to_num(0.0, neginf=0.0)  # sigmoids that underflow
    mask = (torch.rand(40, generator=g) < 0.7).to(torch.uint8)
    mask[3:11] = 1
    bias = 0.1 * torch.randn(48, generator=g)
    bias[2], bias[11] = -math.inf, math.nan  # closed for the choice
    for sigmoid in (False, True):
        for kw in (dict(), dict(bias=bias), dict(groups=4, topk_groups=2, group_top=2), dict(mask=mask),
                   dict(mask=mask, bias=bias, groups=8, topk_groups=3)):
            check_route(logits, 6, sigmoid=sigmoid, **kw)
    # normalize off: row 10's sigmoids are below fp32's range and come out as 0 or denormal
    check_route(logits, 6, sigmoid=True, normalize=False)


def test_equal_values_go_to_the_lowest_id():
    zeros = torch.zeros((9, 64))
    coarse = torch.randint(-2, 3, (50, 64), generator=torch.Generator().manual_seed(6)).float()
    coarse[coarse == 0] = -0.0
    coarse[:, ::3] = coarse[:, ::3].abs()  # +0 and -0 are equal
    for logits in (zeros, coarse, coarse.to(torch.bfloat16)):
        for sigmoid in (False, True):
            for kw in (dict(), dict(bias=torch.zeros(64)), dict(groups=8, topk_groups=3, group_top=2),
                       dict(groups=8, topk_groups=3, bias=torch.full((64,), -0.25))):
                check_route(logits, 8, sigmoid=sigmoid, **kw)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_values_closer_than_fp32_tells_apart(sigmoid):
    """Pairs of experts whose score + bias differ by parts of an fp32 ulp: the
    order is that of 64 bits."""
    g = torch.Generator().manual_seed(7)
    T, E = 64, 32
    logits = torch.randn((T, E), generator=g)
    s = ref.scores(logits.double(), sigmoid)
    # bias that makes the experts nearly equal for token 0, rounded to fp32
    bias = (0.9 - s[0]).float()
    logits[1:] = logits[0] + 1e-6 * torch.randn((T - 1, E), generator=g)
    check_route(logits, 8, sigmoid=sigmoid, bias=bias)
    check_route(logits, 4, sigmoid=sigmoid, bias=bias, groups=8, topk_groups=3, group_top=2)


def test_unaligned_logits():
    """Rows that do not start on 16 bytes (a buffer offset by one element)."""
    for dtype in (torch.float32, torch.bfloat16):
        logits, _ = make(20, 256, dtype, 8)
        raw = torch.empty(20 * 256 + 1, dtype=dtype, device="cuda")
        view = raw[1:].view(20, 256)
        view.copy_(logits)
        idx = torch.empty((20, 8), dtype=torch.int64, device="cuda")
        w = torch.empty((20, 8), device="cuda")
        B.ep_router_topk(view, B.Router(256, 8), idx, w)
        ridx, rw = ref.topk(logits, 8)
        assert torch.equal(idx.cpu(), ridx)
        d = torch.empty(20 * 256 + 1, dtype=dtype, device="cuda")[1:].view(20, 256)
        dw = torch.randn((20, 8), generator=torch.Generator().manual_seed(1))
        B.ep_router_backward(view, B.Router(256, 8), idx, d, d_topk_weights=dw.cuda())
        rd = ref.backward(logits, ridx, 8, d_w=dw)
        assert torch.all((d.cpu().double() - rd).abs() <= 4 * RTOL * dw.abs().max() + 2.0 ** -8 * rd.abs())


def test_no_tokens():
    for sigmoid in (False, True):
        idx, w = route(torch.empty((0, 16)), 4, sigmoid=sigmoid)
        assert idx.shape == (0, 4) and w.shape == (0, 4)
    router = B.Router(16, 4)
    logits = torch.empty((0, 16), device="cuda")
    idx = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    stats = B.BalanceStats(router, 0, num_seqs=3)
    for t in (stats.losses, stats.counts, stats.seq_tokens, stats.mean_scores):
        t.fill_(9)
    B.ep_balance_loss(logits, router, idx, stats, seq_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert not any(bool(t.any()) for t in (stats.losses, stats.counts, stats.seq_tokens, stats.mean_scores))
    B.ep_router_backward(logits, router, idx, torch.empty_like(logits), stats=stats,
                         d_losses=torch.ones((3, 2), device="cuda"),
                         seq_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))


def check_balance(logits, K, sigmoid, normalize, mask=None, offsets=None, scale=1.5, seed=0, idx=None):
    T, E = logits.shape
    g = torch.Generator().manual_seed(seed)
    if idx is None:
        idx = ref.topk(logits, K, sigmoid=sigmoid, mask=mask)[0]
    S = 1 if offsets is None else len(offsets) - 1
    d_w = torch.randn((T, K), generator=g)
    d_l = torch.rand((S, 2), generator=g) + 0.1
    router = B.Router(E, K, score=B.EP_SCORE_SIGMOID if sigmoid else B.EP_SCORE_SOFTMAX, normalize=normalize,
                      scale=scale)
    stats = B.BalanceStats(router, T, num_seqs=S)
    dev = dict(token_mask=None if mask is None else mask.cuda(), seq_offsets=None if offsets is None else
               torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    B.ep_balance_loss(logits.cuda(), router, idx.cuda(), stats, **dev)
    losses, counts, tokens, means = ref.balance(logits, idx, K, sigmoid, mask, offsets)
    assert torch.equal(stats.counts.cpu().long(), counts)
    assert torch.equal(stats.seq_tokens.cpu().long(), tokens)
    assert torch.all((stats.mean_scores.cpu().double() - means).abs() <= 2 * RTOL * means + 1e-37)
    # the z loss squares m + log(sum): u of the larger of the two and logf's 1 ulp on either
    top = ref.clean(logits).amax(dim=1)
    top = float(top[~torch.isneginf(top)].abs().max()) if bool((~torch.isneginf(top)).any()) else 0.0
    got = stats.losses.cpu().double()
    assert torch.all((got[:, 0] - losses[:, 0]).abs() <= 3 * RTOL * losses[:, 0].abs() + 1e-37)
    assert torch.all((got[:, 1] - losses[:, 1]).abs() <= RTOL * (losses[:, 1] + (top + 8) ** 2))
    for dw, dl in ((d_w, d_l), (d_w, None), (None, d_l), (None, None)):
        d = torch.full_like(logits, 7.0).cuda()
        B.ep_router_backward(logits.cuda(), router, idx.cuda(), d, d_topk_weights=None if dw is None else dw.cuda(),
                             stats=stats, d_losses=None if dl is None else dl.cuda(), token_mask=dev["token_mask"],
                             seq_offsets=dev["seq_offsets"])
        rd = ref.backward(logits, idx, K, sigmoid, normalize, scale, dw, dl, mask, offsets)
        size = torch.zeros(T, 1, dtype=torch.float64)
        if dw is not None:
            size += scale * dw.abs().amax(dim=1, keepdim=True).double() * K
        if dl is not None:
            for s, (a, b) in enumerate(ref.spans(T, offsets)):
                n = max(1, int(tokens[s]))
                size[a:b] += float(dl[s, 0]) * E / (K * n * n) * float(counts[s].max())
                size[a:b] += float(dl[s, 1]) * 2 * (top + 8) / n
        bound = 4 * RTOL * size + (2.0 ** -8 * rd.abs() if logits.dtype == torch.bfloat16 else 0) + 1e-37
        got = d.cpu().double()
        assert torch.all((got - rd).abs() <= bound), ((got - rd).abs() / bound).max()
        if dw is None and dl is None:
            assert not bool(d.any())


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (64, 8, 2), (65, 60, 6), (200, 160, 6), (129, 256, 8),
                                   (70, 1000, 20), (66, 1024, 32), (33, 32, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_balance_and_gradient_over_sizes(T, E, K, sigmoid, dtype):
    logits, _ = make(T, E, dtype, 11)
    check_balance(logits, K, sigmoid, normalize=(T % 2 == 1))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_balance_sequences_masks_and_closed_rows(sigmoid, normalize):
    T, E, K = 300, 40, 4
    logits, g = make(T, E, torch.float32, 12, closed=0.3)
    logits[10] = -math.inf
    logits[11, :-1] = -math.inf
    logits[200:203] = math.nan
    logits[20] = logits[20] - 150.0  # sigmoids that underflow
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8)
    mask[220:230] = 0
    many = [0] + sorted(torch.randint(0, T + 1, (69,), generator=g).tolist()) + [T]
    for offsets in (None, [0, T], [0, 0, 1, 65, 65, 200, 220, 230, T], [5, 100, 290], [0] * 40 + [T], [T, T], many):
        check_balance(logits, K, sigmoid, normalize, mask=mask, offsets=offsets)


def test_ids_that_are_missing_bad_or_repeated():
    T, E, K = 80, 24, 5
    logits, g = make(T, E, torch.float32, 13, closed=0.2)
    idx = torch.randint(-1, E, (T, K), generator=g)  # repeats, -1 and ids of closed logits among them
    idx[0] = torch.tensor([3, 3, 3, 3, 3])
    idx[1] = torch.tensor([E, -2, 1 << 40, -(1 << 40), 4])
    idx[2] = -1
    for sigmoid in (False, True):
        for normalize in (False, True):
            check_balance(logits, K, sigmoid, normalize, idx=idx)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(sigmoid, normalize):
    """The kernel's gradient along a direction equals the central difference of
    the 64-bit objective along it, to the gradient's own tolerance."""
    T, E, K = 12, 16, 3
    logits, g = make(T, E, torch.float32, 14)
    idx = ref.topk(logits, K, sigmoid=sigmoid)[0]
    offsets = [0, 5, T]
    d_w, d_l = torch.randn((T, K), generator=g), torch.rand((2, 2), generator=g)
    router = B.Router(E, K, score=B.EP_SCORE_SIGMOID if sigmoid else B.EP_SCORE_SOFTMAX, normalize=normalize, scale=2.0)
    stats = B.BalanceStats(router, T, num_seqs=2)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    B.ep_balance_loss(logits.cuda(), router, idx.cuda(), stats, seq_offsets=off)
    d = torch.empty_like(logits, device="cuda")
    B.ep_router_backward(logits.cuda(), router, idx.cuda(), d, d_topk_weights=d_w.cuda(), stats=stats,
                         d_losses=d_l.cuda(), seq_offsets=off)
    f = lambda x: ref.objective(x, logits, idx, K, sigmoid, normalize, 2.0, d_w, d_l, None, offsets)  # noqa: E731
    for _ in range(4):
        u = torch.randn((T, E), generator=g, dtype=torch.float64)
        h = 1e-4
        slope = float(f(logits.double() + h * u) - f(logits.double() - h * u)) / (2 * h)
        got = float((d.cpu().double() * u).sum())
        # h^2 of the third derivative (|u|^3 of order 1 each, coefficients below 10) and the gradient's rounding
        assert abs(got - slope) <= 1e-5 * float(u.abs().sum())


def test_same_bytes_every_time_and_on_a_side_stream():
    logits, g = make(3000, 256, torch.bfloat16, 15)
    router = B.Router(256, 8, normalize=False)
    l = logits.cuda()
    off = torch.tensor([0, 700, 701, 2900, 3000], dtype=torch.int32, device="cuda")
    d_l = torch.rand((4, 2), generator=g).cuda()
    d_w = torch.randn((3000, 8), generator=g).cuda()
    torch.cuda.synchronize()

    def step(stream=None):
        idx = torch.empty((3000, 8), dtype=torch.int64, device="cuda")
        w = torch.empty((3000, 8), device="cuda")
        stats = B.BalanceStats(router, 3000, num_seqs=4)
        d = torch.empty_like(l)
        B.ep_router_topk(l, router, idx, w, stream=stream)
        B.ep_balance_loss(l, router, idx, stats, seq_offsets=off, stream=stream)
        B.ep_router_backward(l, router, idx, d, d_topk_weights=d_w, stats=stats, d_losses=d_l, seq_offsets=off,
                             stream=stream)
        return [idx, w, stats.losses, stats.counts, stats.mean_scores, d]

    first = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = step(side)
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_training_step_in_a_cuda_graph():
    T, E, K = 500, 64, 6
    router = B.Router(E, K, score=B.EP_SCORE_SIGMOID, num_groups=4, topk_groups=2, group_top=2, scale=2.5)
    l = torch.empty((T, E), device="cuda")
    bias = torch.zeros(E, device="cuda")
    idx = torch.empty((T, K), dtype=torch.int64, device="cuda")
    w, d = torch.empty((T, K), device="cuda"), torch.empty((T, E), device="cuda")
    d_l, d_w = torch.tensor([[1e-2, 1e-3]], device="cuda"), torch.randn((T, K), device="cuda")
    stats = B.BalanceStats(router, T)

    def step(stream):
        B.ep_router_topk(l, router, idx, w, bias=bias, stream=stream)
        B.ep_balance_loss(l, router, idx, stats, stream=stream)
        B.ep_router_backward(l, router, idx, d, d_topk_weights=d_w, stats=stats, d_losses=d_l, stream=stream)

    s = torch.cuda.Stream()
    l.copy_(make(T, E, torch.float32, 16)[0])
    torch.cuda.synchronize()
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s)
    for seed in (17, 18):
        logits = make(T, E, torch.float32, seed)[0]
        l.copy_(logits)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, w, stats.losses, stats.counts, d)]
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for a, b in zip(got, (idx, w, stats.losses, stats.counts, d)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        ridx, _ = ref.topk(logits, K, sigmoid=True, bias=torch.zeros(E), groups=4, topk_groups=2, group_top=2, scale=2.5)
        assert torch.equal(got[0].cpu(), ridx)


def test_outputs_stay_in_bounds():
    """Guard bytes around every output of odd-sized calls stay as they were."""
    from test_gpu_canary import Guarded, _check

    T, E, K, S = 67, 45, 5, 3
    for dtype in (torch.float32, torch.bfloat16):
        logits, g = make(T, E, dtype, 19)
        router = B.Router(E, K)
        idx, w, d = Guarded((T, K), torch.int64), Guarded((T, K), torch.float32), Guarded((T, E), dtype)
        stats = B.BalanceStats(router, T, num_seqs=S)
        need = stats.workspace.numel()
        guards = dict(losses=Guarded((S, 2), torch.float32), counts=Guarded((S, E), torch.int32),
                      seq_tokens=Guarded((S,), torch.int32), mean_scores=Guarded((S, E), torch.float32),
                      workspace=Guarded((need,), torch.uint8))
        for k, v in guards.items():
            setattr(stats, k, v.t)
        off = torch.tensor([0, 3, 3, T], dtype=torch.int32, device="cuda")
        B.ep_router_topk(logits.cuda(), router, idx.t, w.t)
        B.ep_balance_loss(logits.cuda(), router, idx.t, stats, seq_offsets=off)
        B.ep_router_backward(logits.cuda(), router, idx.t, d.t, d_topk_weights=torch.ones((T, K), device="cuda"),
                             stats=stats, d_losses=torch.ones((S, 2), device="cuda"), seq_offsets=off)
        torch.cuda.synchronize()
        _check(idx, w, d, *guards.values())


def test_offsets_that_are_not_sorted_stay_in_bounds():
    """Offsets that decrease or leave [0, T] name no sequence that is defined,
    but nothing outside the outputs is touched and the ordinary call after it
    is right."""
    T, E, K = 150, 16, 2
    logits, _ = make(T, E, torch.float32, 20)
    router = B.Router(E, K)
    stats = B.BalanceStats(router, T, num_seqs=4)
    idx = ref.topk(logits, K)[0].cuda()
    d = torch.empty((T, E), device="cuda")
    for off in ([0, 100, 50, 120, T], [-5, 1000, -7, 3, 2 ** 31 - 1], [T, 0, T, 0, T]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        B.ep_balance_loss(logits.cuda(), router, idx, stats, seq_offsets=o)
        B.ep_router_backward(logits.cuda(), router, idx, d, stats=stats, d_losses=torch.ones((4, 2), device="cuda"),
                             seq_offsets=o)
    torch.cuda.synchronize()
    check_balance(logits, K, False, True, offsets=[0, 10, 20, 30, T])


def test_a_workspace_holds_nothing_between_calls():
    """The workspace needs no initialisation, and one workspace serves calls of
    other sizes and numbers of sequences in turn."""
    E, K = 48, 3
    router = B.Router(E, K)
    big = B.BalanceStats(router, 4000, num_seqs=40).workspace
    g = torch.Generator().manual_seed(21)
    for fill in (0xff, 0x00, 0x7f):
        big.fill_(fill)
        for T, S in ((4000, 1), (3000, 40), (10, 3), (4000, 2), (600, 40)):
            logits, _ = make(T, E, torch.float32, T + S)
            cuts = sorted(torch.randint(0, T + 1, (S - 1,), generator=g).tolist())
            off = [0] + cuts + [T]
            stats = B.BalanceStats(router, T, num_seqs=S)
            stats.workspace = big
            idx = logits.topk(K, dim=1).indices.cuda()
            B.ep_balance_loss(logits.cuda(), router, idx, stats, seq_offsets=torch.tensor(off, dtype=torch.int32).cuda())
            for s in range(S):
                want = torch.bincount(idx[off[s]:off[s + 1]].reshape(-1).cpu(), minlength=E)
                assert torch.equal(stats.counts[s].cpu().long(), want)
                p = torch.softmax(logits[off[s]:off[s + 1]].double(), dim=1)
                mean = p.sum(dim=0) / max(1, off[s + 1] - off[s])
                assert torch.all((stats.mean_scores[s].cpu().double() - mean).abs() <= 2 * RTOL * mean)


def test_groups_closer_than_fp32_tells_apart():
    """Groups whose values differ by parts of an fp32 ulp, in every size of
    group: the order is that of 64 bits, ties to the lower group."""
    g = torch.Generator().manual_seed(22)
    for E, G in ((64, 8), (256, 8), (48, 16), (1024, 4), (8, 8)):
        base = torch.randn((1, E // G), generator=g)
        logits = base.repeat(1, G).repeat(40, 1) + 2e-7 * torch.randn((40, E), generator=g)
        logits[0] = base.repeat(1, G)  # all groups alike
        bias = 1e-8 * torch.randn(E, generator=g)
        for sigmoid in (False, True):
            for top in (1, 2):
                check_route(logits, 2, sigmoid=sigmoid, groups=G, topk_groups=max(1, G // 2), group_top=top)
                check_route(logits, 2, sigmoid=sigmoid, groups=G, topk_groups=max(1, G // 2), group_top=top, bias=bias)


def test_statistics_buffers_are_checked_when_set():
    r = B.Router(8, 2)
    stats = B.BalanceStats(r, 64, num_seqs=2)
    with pytest.raises(TypeError):
        stats.losses = torch.empty((3, 2), device="cuda")
    with pytest.raises(TypeError):
        stats.counts = torch.empty((2, 8), device="cuda")
    with pytest.raises(ValueError):
        stats.mean_scores = torch.empty((8, 2), device="cuda").T
    with pytest.raises(TypeError):
        stats.workspace = stats.workspace[:-256]
    stats.seq_tokens = torch.empty(2, dtype=torch.int32)  # another device
    logits, idx = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        B.ep_balance_loss(logits, r, idx, stats, seq_offsets=torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):  # of another number of experts
        B.ep_balance_loss(torch.zeros((4, 9), device="cuda"), B.Router(9, 2), idx, B.BalanceStats(r, 64))


def test_many_sequences():
    """More sequences than tokens: most are empty, each is right."""
    T, E, K, S = 3000, 24, 3, 5000
    logits, g = make(T, E, torch.float32, 23)
    off = [0] + sorted(torch.randint(0, T + 1, (S - 1,), generator=g).tolist()) + [T]
    off[10:20] = [off[9]] * 10
    idx = logits.topk(K, dim=1).indices
    router = B.Router(E, K)
    stats = B.BalanceStats(router, T, num_seqs=S)
    o = torch.tensor(off, dtype=torch.int32)
    B.ep_balance_loss(logits.cuda(), router, idx.cuda(), stats, seq_offsets=o.cuda())
    n = (o[1:] - o[:-1]).long()
    assert torch.equal(stats.seq_tokens.cpu().long(), n)
    seq = torch.repeat_interleave(torch.arange(S), n)
    counts = torch.zeros((S, E), dtype=torch.int64).index_add_(0, seq, torch.nn.functional.one_hot(idx, E).sum(dim=1))
    assert torch.equal(stats.counts.cpu().long(), counts)
    p = torch.softmax(logits.double(), dim=1)
    mean = torch.zeros((S, E), dtype=torch.float64).index_add_(0, seq, p) / n.clamp(min=1)[:, None]
    assert torch.all((stats.mean_scores.cpu().double() - mean).abs() <= 2 * RTOL * mean)
    want = (counts * mean).sum(dim=1) * E / (K * n.clamp(min=1))
    assert torch.all((stats.losses[:, 0].cpu().double() - want).abs() <= 3 * RTOL * want)
    d = torch.empty_like(logits, device="cuda")
    dl = torch.rand((S, 2), generator=g)
    B.ep_router_backward(logits.cuda(), router, idx.cuda(), d, stats=stats, d_losses=dl.cuda(), seq_offsets=o.cuda())
    x = logits.double().requires_grad_(True)
    q = torch.softmax(x, dim=1)
    m = torch.zeros((S, E), dtype=torch.float64).index_add(0, seq, q) / n.clamp(min=1)[:, None]
    z = torch.zeros(S, dtype=torch.float64).index_add(0, seq, torch.logsumexp(x, dim=1) ** 2) / n.clamp(min=1)
    total = (dl[:, 0].double() * (counts * m).sum(dim=1) * E / (K * n.clamp(min=1)) + dl[:, 1].double() * z).sum()
    rd, = torch.autograd.grad(total, x)
    # a term is at most gb * counts, or 2 |lse| of the z loss (|lse| <= 16), over the sequence's tokens
    size = (dl[seq, 0].double() * E / (K * n[seq] ** 2) * counts[seq].amax(dim=1) + dl[seq, 1].double() * 32 / n[seq])
    assert torch.all((d.cpu().double() - rd).abs() <= 4 * RTOL * size[:, None])
