"""Products grouped by expert with few columns an expert: equal shares of the reduction, joined.  Every case takes that form
(three launches).  The cases cut tiles across two, three and many pairs, leave pairs with a partial sum at both ends of their
share or with whole tiles between them, and have fewer shares than pairs.

Tolerance: as in test_gpu_experts.py, and the join adds the partial sums of a tile in fp32: 2^-24 of the sum of magnitudes
each.  A share has at least four stages (128 columns of W' forward, 64 rows backward), so a tile has stages / 4 + 2 at most.
"""
import pytest
import torch

import sparse_gemm_nm_b200 as nm
from test_gpu_experts import BF, DEV, F32, experts, offsets_of, rows

pytestmark = pytest.mark.gpu

# E, R, K, counts, first column, columns behind the last expert
FORWARD = [
    (1, 64, 2304, [1], 0, 0),
    (1, 16, 11024, [1], 0, 0),
    (2, 300, 6000, [5, 30], 0, 0),
    (3, 700, 8192, [64, 1, 20], 3, 2),
    (8, 512, 2816, [200, 0, 3, 1, 0, 20, 7, 9], 7, 9),
    (25, 1000, 2192, [(i * 7) % 5 for i in range(25)], 1, 0),
    (40, 264, 2320, [(i * 5) % 4 for i in range(40)], 0, 3),
    (40, 1000, 2192, [1 + i % 2 for i in range(40)], 2, 1),
    (1, 4096, 4096, [32], 0, 0),
    (3, 512, 4096, [0, 0, 0], 4, 5),
]
BACKWARD = [
    (1, 1409, 64, [4], 0, 0),
    (1, 11007, 16, [1], 0, 0),
    (2, 3001, 304, [5, 30], 0, 0),
    (3, 4095, 720, [64, 1, 20], 3, 2),
    (8, 1990, 512, [200, 0, 3, 1, 0, 20, 7, 9], 7, 9),
    (25, 2101, 1008, [(i * 7) % 5 for i in range(25)], 1, 0),
    (40, 1700, 272, [(i * 5) % 4 for i in range(40)], 0, 3),
    (40, 1609, 1008, [1 + i % 2 for i in range(40)], 2, 1),
    (1, 4096, 4096, [32], 0, 0),
    (3, 4096, 512, [0, 0, 0], 4, 5),
]


def close(y, ref, mag, n, stages, what):
    half = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
    bound = (2 * (n / 16 + 2) * 2.0 ** -23 + (stages / 4 + 2) * 2.0 ** -24) * mag + half * ref.abs() * (1 + 2.0 ** -6) + 1e-38
    bad = (y.double() - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, first {bad.nonzero()[:3].tolist()}"


def launches(call):
    before = nm.nm_launch_count()
    out = call()
    assert nm.nm_launch_count() - before == 3, "not in equal shares"
    return out


@pytest.mark.parametrize("E,R,K,counts,start,behind", FORWARD)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(E, R, K, counts, start, behind, dtype):
    g = torch.Generator(device=DEV).manual_seed(E * 1000 + R + K)
    values, meta, dense = experts(E, R, K, g)
    at, off = offsets_of(counts, start)
    S = at[-1] + behind
    X = rows(K, S, g, pad=8)
    y = torch.full((R, (S + 7) // 8 * 8), 7.0, device=DEV, dtype=dtype)
    launches(lambda: nm.nm_experts_spmm(values, meta, 2, 4, E, R, K, X, X.stride(0), S, off, y, y.stride(0),
                                        nm.NM_OUT_F32 if dtype == F32 else nm.NM_OUT_BF16))
    nm.nm_device_status()
    assert (y[:, :start] == 7).all() and (y[:, at[-1]:] == 7).all()
    for e in range(E):
        x = X[:, at[e]:at[e + 1]].double()
        close(y[:, at[e]:at[e + 1]], dense[e] @ x, dense[e].abs() @ x.abs(), K // 2, K / 128, f"expert {e}")


@pytest.mark.parametrize("E,R,K,counts,start,behind", BACKWARD)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_input_gradient(E, R, K, counts, start, behind, dtype):
    g = torch.Generator(device=DEV).manual_seed(E * 1000 + R + K + 1)
    values, meta, dense = experts(E, R, K, g)
    at, off = offsets_of(counts, start)
    S = at[-1] + behind
    dY = rows(R, S, g, pad=16)
    dx = torch.full((K, (S + 7) // 8 * 8), 7.0, device=DEV, dtype=dtype)
    launches(lambda: nm.nm_experts_spmm_t(values, meta, 2, 4, E, R, K, dY, dY.stride(0), S, off, dx, dx.stride(0),
                                          nm.NM_OUT_F32 if dtype == F32 else nm.NM_OUT_BF16))
    nm.nm_device_status()
    assert (dx[:, :start] == 7).all() and (dx[:, at[-1]:] == 7).all()
    for e in range(E):
        d = dY[:, at[e]:at[e + 1]].double()
        close(dx[:, at[e]:at[e + 1]], dense[e].T @ d, dense[e].T.abs() @ d.abs(), R, R / 64, f"expert {e}")


SQUARE = (3, 4096, 4096)  # both products take the form for up to 96 columns


def both(values, meta, X, dY, off, stream=None):
    K = X.shape[0]
    return (launches(lambda: nm.experts_spmm(values, meta, 2, 4, K, X, off, stream=stream)),
            launches(lambda: nm.experts_spmm_t(values, meta, 2, 4, K, dY, off, stream=stream)))


def test_columns_and_experts_are_apart():
    """A NaN or Inf in one expert's weights or columns, or in columns of no expert, stays there."""
    g = torch.Generator(device=DEV).manual_seed(5)
    E, R, K = SQUARE
    values, meta, _ = experts(E, R, K, g)
    at, off = offsets_of([11, 30, 13], 2)
    X, dY = rows(K, at[-1] + 3, g), rows(R, at[-1] + 3, g)
    good = both(values, meta, X, dY, off)
    for t in (X, dY):
        t[:, :2], t[:, at[-1]:] = float("inf"), float("nan")
    values[1, R // 2, 3] = float("nan")
    values[1, R - 1, 5] = float("inf")
    X[7, at[1] + 1] = float("inf")
    dY[9, at[2] - 1] = float("nan")
    bad = both(values, meta, X, dY, off)
    for e in (0, 2):
        for a, b in zip(good, bad):
            assert torch.equal(a[:, at[e]:at[e + 1]], b[:, at[e]:at[e + 1]])
    assert all(b[:, at[1]:at[2]].isnan().any() for b in bad)


def test_captured_and_replayed_with_other_counts():
    g = torch.Generator(device=DEV).manual_seed(6)
    E, R, K = SQUARE
    values, meta, _ = experts(E, R, K, g)
    S = 40
    X, dY = rows(K, S, g), rows(R, S, g)
    off = torch.tensor([0, 9, 9, 40], dtype=torch.int32, device=DEV)
    both(values, meta, X, dY, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(values, meta, X, dY, off)
    for at in ([0, 9, 9, 40], [0, 0, 0, 40], [0, 1, 2, 40], [0, 40, 40, 40]):
        off.copy_(torch.tensor(at, dtype=torch.int32))
        X.normal_()
        dY.normal_()
        graph.replay()
        for a, b in zip(out, both(values, meta, X, dY, off)):
            assert torch.equal(a, b)


def test_streams_and_repeats():
    """Calls on two streams at once, each repeated: equal bits."""
    g = torch.Generator(device=DEV).manual_seed(7)
    E, R, K = SQUARE
    values, meta, _ = experts(E, R, K, g)
    off = torch.tensor([0, 20, 21, 90], dtype=torch.int32, device=DEV)
    X, dY = rows(K, 90, g), rows(R, 90, g)
    want = both(values, meta, X, dY, off)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [both(values, meta, X, dY, off, s) for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))
    nm.nm_device_status()
