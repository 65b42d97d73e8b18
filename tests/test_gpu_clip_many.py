"""Clipping of more gradients than a launch takes."""
import pytest
import torch

import sparse_gemm_nm_b200 as nm
from test_gpu_clip import NORM

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n", [640, 641, 2000, 30000])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_many(n, max_norm):
    """n gradients of 1 to 5 elements, 32 bytes apart; what lies between them stays."""
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn((n, 8), generator=g, device=DEV)
    y, norm = torch.full_like(x, 9), torch.empty((), device=DEV)
    sizes = [1 + i % 5 for i in range(n)]
    mine = torch.arange(8, device=DEV)[None, :] < torch.tensor(sizes, device=DEV)[:, None]
    at, to = ([t.data_ptr() + 32 * i for i in range(n)] for t in (x, y))
    nm.nm_clip_grads(at, to, sizes, [nm.NM_OUT_F32] * n, max_norm, norm)
    ref = x.double() * mine
    want = float(ref.norm())
    assert abs(float(norm) - want) <= NORM * want
    ref *= min(1.0, max_norm / want)
    assert ((y.double() - ref).abs() <= (NORM + 3 * 2.0 ** -24) * ref.abs())[mine].all() and (y[~mine] == 9).all()
    keep = x.clone()
    nm.nm_clip_grads(at, at, sizes, [nm.NM_OUT_F32] * n, max_norm, norm)  # in place: the same bits
    assert torch.equal(x[mine], y[mine]) and torch.equal(x[~mine], keep[~mine])


def test_the_norm_alone_takes_no_second_pass():
    """One pass over the gradients, where clipping has two and writes them."""
    x = torch.ones(1 << 28, device=DEV)
    norm = torch.empty((), device=DEV)

    def best(outs):
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            nm.nm_clip_grads([x], outs, [x.numel()], [nm.NM_OUT_F32], 1.0, norm)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    alone = best(None)
    assert float(norm) == 2.0 ** 14
    y = torch.empty_like(x)
    assert alone < best([y]) and (y == 2.0 ** -14).all()
