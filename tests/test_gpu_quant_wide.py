"""Quantised dispatch at hidden sizes whose row buffers are about as large as the
shared memory that a kernel has without asking for more."""
import numpy as np
import pytest

from combine_ep_get_10_b200 import workloads as W
from test_gpu_quant import _gpu, _run, _rng  # noqa: F401 (the module's fixture)
import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16256, 16288, 16304, 16320, 16336, 16352, 16368, 16384])
@pytest.mark.parametrize("dt", [W.INT8_PER_TOKEN, W.FP8_E4M3_PER_TOKEN])
def test_rows_about_48_kb(H, dt):
    rng = _rng(H)
    T, E, K = 5, 8, 8
    x = oracle.f32_to_bf16(rng.standard_normal((T, H)).astype(np.float32))
    idx = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int64)
    ref, _, codes, scales, flags, _, _ = _run(x, idx, E, 1, dt)
    assert flags == 0
    want = np.ascontiguousarray(ref["recv"]).view(np.uint8).reshape(codes.shape)
    assert np.array_equal(codes, want)
    assert np.array_equal(scales, np.ascontiguousarray(ref["recv_scales"]).view(np.uint8).reshape(scales.shape))
