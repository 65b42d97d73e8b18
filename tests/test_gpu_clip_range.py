"""Clipping at the ends of fp32's range: norms that fp32 does not hold."""
import math

import pytest
import torch

import sparse_gemm_nm_b200 as nm
from test_gpu_clip import BF, DEV, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [[4], [1, 2, 1], [3, 40001]])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("apart", [True, False])
def test_a_norm_above_the_largest_float_scales_nothing(sizes, dtype, apart):
    """Finite gradients whose norm fp32 does not hold: it is handed back as Inf, and they stay as they are."""
    ts = [torch.full((n,), 2e38, device=DEV, dtype=dtype) for n in sizes]
    keep = [t.clone() for t in ts]
    out = [torch.zeros_like(t) for t in ts] if apart else None
    assert math.isinf(float(nm.clip_grads(ts, 1.0, out=out)))
    assert all(torch.equal(t, k) for t, k in zip(out or ts, keep))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_largest_norm_is_scaled(dtype):
    """A norm just below the largest float."""
    big = torch.full((1,), torch.finfo(dtype).max, device=DEV, dtype=dtype)
    assert float(nm.clip_grads([big], 2.0)) == torch.finfo(dtype).max
    assert abs(float(big) - 2.0) <= 2.0 ** -8 * 2.0
