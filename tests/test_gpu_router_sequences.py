"""Balance losses of very many sequences: right for every mix of lengths, and in
time that grows with them, not with their square.  Tolerances: as in
test_gpu_router."""
import pytest
import torch

from combine_ep_get_10_b200 import binding as B
from test_gpu_router import RTOL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


def cut(lengths, first):
    ends = torch.tensor([first] + list(lengths)).cumsum(0)
    return ends.to(torch.int32).cuda()


def lengths(kind, S, g):
    n = torch.randint(0, 4, (S,), generator=g)
    if kind == "some long":  # several chunks each, at the ends and in between, neighbours too
        n[[0, 1, S // 3, S // 2, S - 1]] = torch.tensor([700, 2500, 1, 9000, 4000])
    elif kind == "about a chunk":
        n = torch.randint(0, 300, (S,), generator=g)
    elif kind == "one":
        n[:] = 0
        n[S // 2] = 20000
    return n.tolist()


@pytest.mark.parametrize("kind,S,E", [("short", 4000, 24), ("some long", 3000, 24), ("about a chunk", 150, 40),
                                      ("about a chunk", 700, 8), ("one", 1000, 16), ("some long", 37, 256),
                                      ("about a chunk", 20, 383), ("about a chunk", 20, 384), ("about a chunk", 20, 385),
                                      ("about a chunk", 20, 707), ("about a chunk", 20, 719), ("about a chunk", 20, 722),
                                      ("about a chunk", 20, 723), ("short", 30, 1024)])
@pytest.mark.parametrize("first,behind", [(0, 0), (333, 70)])
def test_many_sequences_of_all_lengths(kind, S, E, first, behind):
    g = torch.Generator().manual_seed(S + E)
    K, n = 3, lengths(kind, S, g)
    off = cut(n, first)
    T = int(off[-1]) + behind
    logits = (1.5 * torch.randn((T, E), generator=g)).cuda()
    mask = (torch.rand(T, generator=g) < 0.9).to(torch.uint8).cuda()
    router = B.Router(E, K)
    idx = logits.topk(K, dim=1).indices.contiguous()
    stats = B.BalanceStats(router, T, num_seqs=S)
    stats.losses.fill_(float("nan"))
    stats.mean_scores.fill_(float("nan"))
    stats.counts.fill_(77)
    stats.seq_tokens.fill_(77)
    B.ep_balance_loss(logits, router, idx, stats, token_mask=mask, seq_offsets=off)

    # by sequence, S for a token of none
    token = torch.arange(T, device="cuda")
    seq = torch.searchsorted(off.long(), token, right=True) - 1
    seq[(token < first) | (token >= off[-1])] = S
    live = mask.double()
    add = lambda v: torch.zeros((S + 1,) + v.shape[1:], dtype=torch.float64, device="cuda").index_add_(0, seq, v)  # noqa: E731
    q = torch.softmax(logits.double(), dim=1)
    lse = torch.logsumexp(logits.double(), dim=1)
    tokens = add(live)
    nz = tokens.clamp(min=1.0)
    hit = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx, 1.0)
    counts, mean, z = add(hit * live[:, None]), add(q * live[:, None]) / nz[:, None], add(lse * lse * live) / nz
    balance = E / (K * nz) * (counts * mean).sum(dim=1)
    assert torch.equal(stats.seq_tokens.double(), tokens[:S])
    assert torch.equal(stats.counts.double(), counts[:S])
    assert torch.all((stats.mean_scores - mean[:S]).abs() <= 2 * RTOL * mean[:S])
    assert torch.all((stats.losses[:, 0] - balance[:S]).abs() <= 3 * RTOL * balance[:S])
    assert torch.all((stats.losses[:, 1] - z[:S]).abs() <= RTOL * (z[:S] + (lse.abs().max() + 8) ** 2))

    dl = torch.rand((S, 2), generator=g).cuda() + 0.1
    d = torch.full_like(logits, 7.0)
    B.ep_router_backward(logits, router, idx, d, stats=stats, d_losses=dl, token_mask=mask, seq_offsets=off)
    of = torch.cat([dl.double(), torch.zeros((1, 2), dtype=torch.float64, device="cuda")])[seq]
    gain = (of[:, 0] * live * E / (K * nz[seq] ** 2))[:, None] * counts[seq]
    dz = of[:, 1] * live * 2 * lse / nz[seq]
    want = q * (gain - (gain * q).sum(dim=1, keepdim=True) + dz[:, None])
    size = gain.amax(dim=1) + dz.abs()
    assert torch.all((d - want).abs() <= 4 * RTOL * size[:, None] + 1e-37)
    again = B.BalanceStats(router, T, num_seqs=S)
    B.ep_balance_loss(logits, router, idx, again, token_mask=mask, seq_offsets=off)
    for name in ("losses", "counts", "seq_tokens", "mean_scores"):
        assert torch.equal(getattr(again, name), getattr(stats, name))


def test_time_grows_with_the_sequences_not_with_their_square():
    """Four times the sequences (and tokens) take about four times as long, where
    a look at all sequences for each of them would take sixteen times."""
    def us(S):
        T, E, K = 2 * S, 8, 2
        logits = torch.randn((T, E), device="cuda")
        router = B.Router(E, K)
        idx = logits.topk(K, dim=1).indices.contiguous()
        stats = B.BalanceStats(router, T, num_seqs=S)
        off = torch.arange(0, T + 1, 2, dtype=torch.int32, device="cuda")
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            B.ep_balance_loss(logits, router, idx, stats, seq_offsets=off)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3)
        return best

    few, many = us(16384), us(65536)
    assert many < 8 * few, (few, many)


def test_arrays_past_2_32_bytes():
    """Logits and gradients of more than 2^32 bytes, in which the last rows are as
    right as the first."""
    T, E, K = 2 ** 21 - 1, 1024, 2
    logits = torch.empty((T, E), device="cuda")
    for t in range(0, T, 1 << 18):
        part = logits[t:t + (1 << 18)]
        part.copy_(torch.randn((1 << 18, E), generator=torch.Generator(device="cuda").manual_seed(t), device="cuda")
                   [:part.shape[0]])
    router = B.Router(E, K)
    idx, w = torch.empty((T, K), dtype=torch.int64, device="cuda"), torch.empty((T, K), device="cuda")
    B.ep_router_topk(logits, router, idx, w)
    stats = B.BalanceStats(router, T, num_seqs=2)
    off = torch.tensor([0, T - 1000, T], dtype=torch.int32, device="cuda")
    B.ep_balance_loss(logits, router, idx, stats, seq_offsets=off)
    d = torch.empty_like(logits)
    dl = torch.tensor([[1.0, 0.0], [0.5, 0.25]], device="cuda")
    dw = torch.ones((T, K), device="cuda")
    dw[:, 1] = -1.0
    B.ep_router_backward(logits, router, idx, d, d_topk_weights=dw, stats=stats, d_losses=dl, seq_offsets=off)
    for t0, t1, s, n in ((0, 200, 0, T - 1000), (T - 1200, T - 1000, 0, T - 1000), (T - 1000, T, 1, 1000)):
        l = logits[t0:t1].double()
        top = l.topk(K, dim=1)
        assert torch.equal(idx[t0:t1], top.indices)
        want = torch.softmax(top.values, dim=1)
        assert torch.all((w[t0:t1] - want).abs() <= RTOL * want)
        q = torch.softmax(l, dim=1)
        gain = dl[s, 0].double() * E / (K * n * n) * stats.counts[s].double()
        grad = q * (gain - (gain * q).sum(dim=1, keepdim=True)) + \
            (dl[s, 1] * 2 * torch.logsumexp(l, dim=1) / n)[:, None] * q
        part = want * (dw[t0:t1] - (want * dw[t0:t1]).sum(dim=1, keepdim=True))
        grad.scatter_add_(1, top.indices, part)
        size = gain.max() + float(dl[s, 1]) * 2 * 16 / n + 2.0
        assert torch.all((d[t0:t1] - grad).abs() <= 4 * RTOL * size)
    last = torch.bincount(idx[T - 1000:].reshape(-1), minlength=E)
    assert torch.equal(stats.counts[1].long(), last) and int(stats.counts[0].sum()) == (T - 1000) * K
