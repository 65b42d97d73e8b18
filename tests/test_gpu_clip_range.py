"""Clipping at the ends of fp32's range, against 64 bits: norms that fp32 does not hold, and factors that it holds in fewer
bits or not at all.  Tolerances as in test_gpu_clip.py.
"""
import math

import pytest
import torch

import sparse_gemm_nm_b200 as nm
from test_gpu_clip import BF, DEV, F32, NORM, norm_of

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


@pytest.mark.parametrize("norm,max_norm", [(4e37, 1e-3), (4e37, 0.3), (4e37, 3.0), (1e37, 1e-8), (1e30, 1e-37), (1e-3, 1e-42),
                                           (4e37, 0.0)])
@pytest.mark.parametrize("sizes", [[1], [3, 8, 1000], [16385, 40003]])
@pytest.mark.parametrize("odd", [False, True])
def test_factors_below_the_smallest_normal_float(norm, max_norm, sizes, odd):
    """Where max_norm / norm is below 2^-126 fp32 has it in fewer bits or as zero; the products may be ordinary numbers.

    A product below 2^-126 itself is rounded to a multiple of 2^-149, in bf16 of 2^-133: half of that, absolutely.
    """
    g = torch.Generator(device=DEV).manual_seed(3)
    ts = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + 1, generator=g, device=DEV) / sum(sizes) ** 0.5 * norm
        ts.append(t.to(BF if i % 2 else F32)[1:] if odd else t.to(BF if i % 2 else F32)[1:].clone())
    want = norm_of(ts)
    factor = max_norm / want
    out = [torch.full_like(t, 9) for t in ts]
    got = nm.clip_grads(ts, max_norm, out=out)
    assert abs(float(got) - want) <= NORM * want
    for t, o in zip(ts, out):
        ref = t.double() * factor
        half, least = (2.0 ** -8, 2.0 ** -134) if t.dtype == BF else (2.0 ** -24, 2.0 ** -150)
        # fp32 first, then bf16: both roundings of a small product
        bound = (half + NORM + 2.0 ** -23) * ref.abs() + (least + 2.0 ** -150) * (1 + 2.0 ** -7)
        assert ((o.double() - ref).abs() <= bound).all()
    same = nm.clip_grads(ts, max_norm)  # in place: the same bits
    assert torch.equal(same, got) and all(torch.equal(a, b) for a, b in zip(ts, out))
