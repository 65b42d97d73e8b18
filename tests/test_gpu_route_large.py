"""The router of more tokens than four CTAs an SM place at a time: each takes several chunks of 512 tokens."""
import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def logits(E, T, g):
    return torch.randn((E, (T + 7) // 8 * 8), generator=g, device=DEV, dtype=BF)[:, :T]


@pytest.mark.parametrize("E,T,k", [(48, 303105, 3), (5, 700003, 2), (1024, 310001, 2), (1, 400000, 1), (64, 1000001, 8)])
def test_columns(E, T, k):
    g = torch.Generator(device=DEV).manual_seed(E + T)
    l = logits(E, T, g)
    l[:, torch.rand(T, generator=g, device=DEV) < 0.1] = -torch.inf  # padding
    expert, gate, slot, source, offsets = nm.experts_route(l, k)
    top, want = l.sort(dim=0, descending=True, stable=True)
    want = torch.where(top[:k] > -torch.inf, want[:k], -1)
    assert torch.equal(expert.long(), want)
    flat = want.flatten()
    order = torch.where(flat < 0, E, flat) * T + torch.arange(T, device=DEV).repeat(k)
    want_source = order.argsort()
    used = int((flat >= 0).sum())
    assert torch.equal(source[:used].long(), want_source[:used]) and (source[used:] == -1).all()
    want_slot = torch.full_like(flat, -1)
    want_slot[want_source[:used]] = torch.arange(used, device=DEV)
    assert torch.equal(slot.flatten().long(), want_slot)
    count = torch.bincount(flat[flat >= 0], minlength=E)
    assert torch.equal(offsets[1:].long(), count.cumsum(0)) and int(offsets[0]) == 0


def test_time_grows_with_the_tokens():
    """Eight times the tokens take eight times as long, and not 54 times (every CTA's pass over all counts)."""
    def best(T):
        l = logits(2, T, torch.Generator(device=DEV).manual_seed(1))
        nm.experts_route(l, 1)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            nm.experts_route(l, 1)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert best(1 << 26) < 20 * best(1 << 23)
