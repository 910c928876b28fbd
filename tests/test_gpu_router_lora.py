"""The router, the layout, a dispatch, low-rank experts on the dispatched rows
and the combine, and the way back to the router's logits, as one step: eager,
and captured once and replayed on other inputs.

Each link is compared with 64 bits on the values that it was given: ids
exactly, weights and the logits' gradient with the bounds of test_gpu_router,
rows and factors' gradients with those of test_gpu_lora, the combine within
1e-6 + 1e-5 of its value (fp32 sums of K = 4 products)."""
import math

import pytest
import torch

import lora_ref
import router_ref
from combine_ep_get_10_b200 import binding as B
from test_gpu_lora import close

pytestmark = pytest.mark.gpu

T, E, K, H, R, S = 300, 16, 4, 264, 24, 3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from combine_ep_get_10_b200 import build

    build.build()
    B.lib()


class Step:
    """The buffers of a step and one pass over them."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.router = B.Router(E, K, score=B.EP_SCORE_SIGMOID, num_groups=4, topk_groups=2, group_top=2, scale=1.5)
        self.bias = (0.1 * torch.randn(E, generator=g)).cuda()
        self.logits, self.x, self.d_out = new(T, E), new(T, H, dtype=bf), new(T, H, dtype=bf)
        self.offsets = torch.tensor([0, 100, 100, T], dtype=torch.int32, device="cuda")
        self.d_losses = (torch.rand((S, 2), generator=g) + 0.1).cuda()
        self.a = (torch.randn((E, R, H), generator=g) / math.sqrt(H)).to(bf)
        self.b = (torch.randn((E, H, R), generator=g) / math.sqrt(R)).to(bf)
        self.scales = torch.rand(E, generator=g) + 0.5
        self.lora = B.Lora(self.a.cuda(), self.b.cuda(), self.scales.cuda())
        self.idx, self.w = new(T, K, dtype=torch.int64), new(T, K)
        self.routing = B.Routing.topk(self.idx, E, 1)
        self.layout = B.Layout(self.routing)
        n = T * K  # every token has K experts: no expert is closed
        self.rows, self.y, self.src, self.row_w = new(n, H, dtype=bf), new(n, H, dtype=bf), new(n, dtype=torch.int32), new(n)
        self.h, self.dh, self.out = new(n, R), new(n, R), new(T, H)
        self.dy, self.dx, self.d_w = new(n, H, dtype=bf), new(n, H, dtype=bf), new(T, K)
        self.da, self.db = new(E, R, H, dtype=bf), new(E, H, R, dtype=bf)
        self.stats, self.d_logits = B.BalanceStats(self.router, T, num_seqs=S), new(T, E)
        self.fill(seed)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed + 1000)
        self.logits.copy_(torch.randn((T, E), generator=g) + 0.5 * torch.randn((1, E), generator=g))
        self.x.copy_(torch.randn((T, H), generator=g))
        self.d_out.copy_(torch.randn((T, H), generator=g))

    def run(self, stream=None):
        s, r, lay = stream, self.routing, self.layout
        B.ep_router_topk(self.logits, self.router, self.idx, self.w, bias=self.bias, stream=s)
        B.ep_get_layout(r, lay, stream=s)
        B.ep_dispatch(self.x, r, lay, self.rows, topk_weights=self.w, recv_src=self.src, recv_weights=self.row_w, stream=s)
        B.ep_lora(self.rows, r, lay, self.lora, self.y, self.h, base=self.rows, stream=s)
        B.ep_combine(self.y, r, lay, self.w, self.out, stream=s)
        # back: the combine's gradients are the rows of d_out times their weights, and dot products with y
        d_rows = self.d_out[self.src.long()].float()
        self.dy.copy_(d_rows * self.row_w[:, None])
        row = (lay.expert_offsets[self.idx] + lay.slot.view(T, K)).long()
        self.d_w.copy_((self.y.float() * d_rows).sum(dim=1)[row])
        B.ep_lora_backward(self.dy, self.rows, self.h, r, lay, self.lora, self.dh, dx=self.dx, da=self.da, db=self.db,
                           dx_base=self.dy, stream=s)
        B.ep_balance_loss(self.logits, self.router, self.idx, self.stats, seq_offsets=self.offsets, stream=s)
        B.ep_router_backward(self.logits, self.router, self.idx, self.d_logits, d_topk_weights=self.d_w, stats=self.stats,
                             d_losses=self.d_losses, seq_offsets=self.offsets, stream=s)

    def outputs(self):
        return [self.idx, self.w, self.rows, self.y, self.h, self.out, self.dx, self.da, self.db, self.stats.losses,
                self.stats.counts, self.d_logits]

    def check(self):
        torch.cuda.synchronize()
        logits, idx = self.logits.cpu(), self.idx.cpu()
        want, w = router_ref.topk(logits, K, sigmoid=True, bias=self.bias.cpu(), groups=4, topk_groups=2, group_top=2,
                                  scale=1.5)
        assert torch.equal(idx, want)
        assert torch.all((self.w.cpu().double() - w).abs() <= 128 * 2.0 ** -24 * w)
        ref = lora_ref.Ref(idx, self.a, self.b, self.scales, T * K, False)
        rows = torch.zeros((T * K, H), dtype=torch.bfloat16)
        at = torch.empty((T, K), dtype=torch.int64)
        seen = [0] * T
        for r, e, t in lora_ref.rows_of(idx, E):
            rows[r] = self.x[t].cpu()
            at[t, int((idx[t] == e).nonzero()[0])] = r
            seen[t] += 1
        assert seen == [K] * T and torch.equal(self.rows.cpu(), rows)
        y, h, size, hsize = ref.forward(rows, rows, rows)
        close(self.h, h, hsize, H, False, "h")
        close(self.y, y, size, H + R, True, "y")
        got_y = self.y.cpu().double()
        out = (self.w.cpu().double()[:, :, None] * got_y[at]).sum(dim=1)
        assert torch.all((self.out.cpu().double() - out).abs() <= 1e-6 + 1e-5 * out.abs())
        (dx, da, db), (sdx, sda, sdb) = ref.backward(self.dy.cpu(), rows, self.h.cpu(), self.dy.cpu(), rows)
        most = max(r.numel() for _, r, _ in ref.groups)
        close(self.dx, dx, sdx, H + R, True, "dx")
        close(self.da, da, sda, H + most, True, "da")
        close(self.db, db, sdb, most, True, "db")
        losses, counts, tokens, _ = router_ref.balance(logits, idx, K, True, None, self.offsets.tolist())
        assert torch.equal(self.stats.counts.cpu().long(), counts) and torch.equal(self.stats.seq_tokens.cpu().long(), tokens)
        # the z loss squares m + log(sum): u of the larger of the two (|m| <= 8 here)
        assert torch.all((self.stats.losses.cpu().double() - losses).abs() <= 128 * 2.0 ** -24 * (3 * losses + 16.0 ** 2))
        d_w, d_l = self.d_w.cpu(), self.d_losses.cpu()
        d = router_ref.backward(logits, idx, K, True, True, 1.5, d_w, d_l, None, self.offsets.tolist())
        scale = torch.zeros((T, 1), dtype=torch.float64) + 1.5 * K * d_w.abs().amax(dim=1, keepdim=True).double()
        for i, (a, b) in enumerate(router_ref.spans(T, self.offsets.tolist())):
            n = max(1, int(tokens[i]))
            scale[a:b] += float(d_l[i, 0]) * E / (K * n * n) * float(counts[i].max()) + float(d_l[i, 1]) * 2 * 16 / n
        assert torch.all((self.d_logits.cpu().double() - d).abs() <= 4 * 128 * 2.0 ** -24 * scale)


def test_step():
    step = Step(1)
    step.run()
    step.check()


def test_captured_step_on_other_inputs():
    step = Step(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.run()
    for seed in (3, 4):
        step.fill(seed)
        graph.replay()
        step.check()
        got = [t.clone() for t in step.outputs()]
        step.run()
        torch.cuda.synchronize()
        for a, b in zip(got, step.outputs()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_steps_on_two_streams_at_once():
    """Two steps with buffers of their own, submitted in turn without waiting."""
    steps = [Step(5), Step(6)]
    alone = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in s.outputs()])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, q in zip(steps, streams):
            with torch.cuda.stream(q):
                s.run()
    torch.cuda.synchronize()
    for s, first in zip(steps, alone):
        for a, b in zip(s.outputs(), first):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
