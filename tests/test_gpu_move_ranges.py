"""The gradient of the combine with more ranges of columns than a grid's second axis holds (65535 of 16384 columns)."""
import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def test_combine_gradient_of_a_billion_columns():
    """One row: every output is one product of two bf16 numbers, which fp32 holds exactly.  About 18 GB."""
    T = 129
    k = 65535 * 16384 // T + 100
    S = k * T
    assert S > 65535 * 16384 and S < 2 ** 31 - 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    dY = torch.randn((1, 136), generator=g, device=DEV).to(BF)[:, :T]
    Yg = torch.empty((1, (S + 7) // 8 * 8), dtype=BF, device=DEV)
    Yg.view(torch.int16).random_(0x3F80, 0x4080, generator=g)  # 1 to 4
    Yg = Yg[:, :S]
    source = torch.arange(S, dtype=torch.int32, device=DEV)  # column j T + t holds token t at its j-th expert
    dyg, dgate = nm.experts_combine_grad(dY, Yg, source.view(k, T), source)
    step = 128 * T * 8000
    for a in range(0, S, step):
        b = min(a + step, S)
        dy = dY[0].float().repeat((b - a) // T)
        assert torch.equal(dyg[0, a:b].float(), dy)
        assert torch.equal(dgate.view(-1)[a:b], dy * Yg[0, a:b].float())
