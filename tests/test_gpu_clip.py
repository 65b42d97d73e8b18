"""The norm over many gradients and their scaling, against 64 bits.

The squares of 32 elements are added in fp32 (32 2^-24 relative, a quarter of it on average), everything else in 64 bits: the
norm is within 16 2^-24 + its own rounding 2^-24.  The factor carries the same error, the product a rounding of its own.
"""
import math

import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NORM = 18 * 2.0 ** -24


def grads(sizes, g, scale=1.0):
    out = []
    for i, n in enumerate(sizes):
        out.append((torch.randn(n, generator=g, device=DEV) * scale).to(BF if i % 2 else F32))
    return out


def norm_of(ts):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in ts))


@pytest.mark.parametrize("sizes", [[1], [7, 0, 1, 16384], [16385, 33, 100003], [5] * 64, [3, 40000] * 40,
                                   [11] * 700 + [50001], [2 ** 21 + 1, 8]])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0, math.inf])
def test_clip(sizes, max_norm):
    g = torch.Generator(device=DEV).manual_seed(len(sizes))
    ts = grads(sizes, g)
    ref = [t.double() for t in ts]
    want = norm_of(ts)
    keep = [t.clone() for t in ts]
    out = [torch.full_like(t, 9) for t in ts]
    norm = nm.clip_grads(ts, max_norm, out=out)
    assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    assert abs(float(norm) - want) <= NORM * want
    factor = max_norm / want if want > max_norm else 1.0
    for t, r in zip(out, ref):
        half = 2.0 ** -8 if t.dtype == BF else 2.0 ** -24
        if factor == 1.0:
            assert torch.equal(t.double(), r)
        else:
            assert ((t.double() - factor * r).abs() <= (half + NORM + 2.0 ** -23) * (factor * r).abs() + 1e-45).all()
    same = nm.clip_grads(ts, max_norm)  # in place: the same bits
    assert torch.equal(same, norm) and all(torch.equal(a, b) for a, b in zip(ts, out))


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e15, 3e18, 1e25])
def test_norms_whose_squares_leave_fp32(scale):
    g = torch.Generator(device=DEV).manual_seed(4)
    ts = grads([5000, 70001, 64], g, scale)
    want = norm_of(ts)
    assert abs(float(nm.clip_grads(ts, want / 3)) - want) <= NORM * want
    assert abs(norm_of(ts) - want / 3) <= 2.0 ** -8 * want


def test_tensors_off_16_bytes_and_zeros():
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randn(20001, generator=g, device=DEV).to(BF)[1:]
    b = torch.randn(999, generator=g, device=DEV)[3:]
    z = torch.zeros(100000, device=DEV, dtype=BF)
    for ts in ([a, b, z], [z]):
        want = norm_of(ts)
        out = [torch.empty_like(t) for t in ts]
        norm = nm.clip_grads(ts, 1.0, out=out)
        assert abs(float(norm) - want) <= NORM * want
        for t, o in zip(ts, out):
            f = min(1.0, 1.0 / want) if want else 1.0
            half = 2.0 ** -8 if t.dtype == BF else 2.0 ** -24
            assert ((o.double() - f * t.double()).abs() <= (half + NORM + 2.0 ** -23) * (f * t.double()).abs()).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_no_number_scales_nothing(bad):
    g = torch.Generator(device=DEV).manual_seed(6)
    ts = grads([3000, 500], g)
    ts[1][77] = bad
    keep = [t.clone() for t in ts]
    norm = nm.clip_grads(ts, 0.1)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ts, keep))


def test_norm_alone_captured_and_streams():
    g = torch.Generator(device=DEV).manual_seed(7)
    ts = grads([100, 4000, 30001], g)
    want = norm_of(ts)
    norm = torch.empty((), device=DEV)
    nm.nm_clip_grads(ts, None, [t.numel() for t in ts], [nm._out_type(t.dtype) for t in ts], 0.0, norm)
    assert abs(float(norm) - want) <= NORM * want
    out = [torch.empty_like(t) for t in ts]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nm.clip_grads(ts, 2.0, out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, norm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = nm.clip_grads(ts, 2.0, out=out)
    for _ in range(2):
        for t in ts:
            t.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert abs(float(n) - norm_of(ts)) <= NORM * norm_of(ts)
        assert abs(norm_of(out) - 2.0) <= 2.0 ** -8 * 2
