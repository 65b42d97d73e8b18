"""Forms of the moves that the sizes of test_gpu_route.py do not take, with its checks: four rows of long ones as a word
(gather), several groups of rows in a CTA's tile or one after the other, and columns in more ranges than a grid's axis has.
"""
import math

import pytest
import torch

import sparse_gemm_nm_b200 as nm
from test_gpu_route import BF, DEV, F32, padded, test_combine as check_combine
from test_gpu_route import test_combine_gradient as check_combine_gradient, test_gather as check_gather

pytestmark = pytest.mark.gpu

SIZES = [  # rows, T, k, experts
    (1801, 8189, 2, 8),   # words of four rows, three turns of every CTA
    (9001, 301, 1, 8),    # three groups of four rows side by side; two in turn for the gradient
    (20003, 300, 2, 16),  # eight; five or six
    (3001, 2300, 1, 8),   # gradient: two groups in turn, four CTAs to an SM
    (100, 70001, 1, 8),   # ... words of one row
    (100, 110001, 1, 4),  # ... from global memory
]


@pytest.mark.parametrize("rows,T,k,E", SIZES)
def test_gather(rows, T, k, E):
    check_gather(rows, T, k, E)


@pytest.mark.parametrize("rows,T,k,E", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_combine(rows, T, k, E, dtype):
    check_combine(rows, T, k, E, dtype, True)


@pytest.mark.parametrize("rows,T,k,E", SIZES)
@pytest.mark.parametrize("gated", [True, False])
def test_combine_gradient(rows, T, k, E, gated):
    check_combine_gradient(rows, T, k, E, gated)


def test_few_columns_of_many_tokens():
    """Columns that name some of the tokens only: the gradient takes groups of two rows in turn."""
    g = torch.Generator(device=DEV).manual_seed(1)
    rows, T, S = 3001, 20001, 300
    source = torch.randperm(T, generator=g, device=DEV)[:S].int()
    slot = torch.full((1, T), -1, dtype=torch.int32, device=DEV)
    slot[0, source.long()] = torch.arange(S, dtype=torch.int32, device=DEV)
    gate = torch.rand((1, T), generator=g, device=DEV)
    dY = padded(torch.randn((rows, T), generator=g, device=DEV), BF)
    Yg = padded(torch.randn((rows, S), generator=g, device=DEV), BF)
    assert torch.equal(nm.experts_gather(dY, source), dY[:, source.long()])
    y = nm.experts_combine(Yg, slot, gate, out_dtype=F32)
    want = torch.zeros((rows, T), dtype=torch.float64, device=DEV)
    want[:, source.long()] = Yg.double() * gate[0, source.long()].double()
    assert ((y.double() - want).abs() <= 2.0 ** -24 * want.abs()).all()
    dyg, dgate = nm.experts_combine_grad(dY, Yg, slot, source, gate)
    ref = dY[:, source.long()].double() * gate[0, source.long()].double()
    assert ((dyg.double() - ref).abs() <= 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -7)).all()
    prod = dY[:, source.long()].double() * Yg.double()
    got = dgate[0, source.long()].double()
    assert ((got - prod.sum(0)).abs() <= (rows + 1) * 2.0 ** -24 * prod.abs().sum(0)).all()
    assert (dgate[slot < 0] == 0).all()
