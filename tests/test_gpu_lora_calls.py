"""Calls of the low-rank products that their documentation allows or refuses:
layouts that are not the routing's, kernels for many rows at every rank, streams,
graphs replayed with other adapters, large arrays."""
import math

import pytest
import torch

from combine_ep_get_10_b200 import binding as B
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
