"""Products grouped by expert against the formulas in 64 bits.

Tolerance of a result y = sum of n products p_i: the tensor cores add 16 products at a time to an fp32 sum, which may lose up
to one unit of the sum's last place each time, so (n / 16 + 2) 2^-23 sum|p_i|, twice over for truncation; then half a step
of the output's type, 2^-8 |y| for bf16.
"""
import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rows(r, c, g, dtype=BF, std=1.0, pad=0):
    """r x c with padded 16-byte rows."""
    per = 8 if dtype == BF else 4
    ld = (c + per - 1) // per * per + pad
    return (torch.randn((r, max(ld, per)), generator=g, device=DEV) * std).to(dtype)[:, :c]


def experts(E, R, K, g):
    """(values E x R x K/2, meta, dense E x R x K in 64 bits)."""
    W = (torch.randn((E, R, K), generator=g, device=DEV) * 0.05).to(BF)
    parts = [nm.prune_compress(W[e], 2, 4) for e in range(E)]
    values = torch.stack([p[0] for p in parts])
    meta = torch.stack([p[1] for p in parts])
    dense = torch.stack([nm.decompress(v, w, K, 2, 4) for v, w in parts])
    return values, meta, dense.double()


def offsets_of(counts, start=0):
    at = [start]
    for c in counts:
        at.append(at[-1] + c)
    return at, torch.tensor(at, dtype=torch.int32, device=DEV)


def close(y, ref, mag, n, what):
    half = 2.0 ** -8 if y.dtype == BF else 2.0 ** -24
    bound = 2 * (n / 16 + 2) * 2.0 ** -23 * mag + half * ref.abs() * (1 + 2.0 ** -6) + 1e-38
    bad = (y.double() - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, first {bad.nonzero()[:3].tolist()}"


CASES = [
    # E, R, K, counts, first column, columns behind the last expert
    (1, 64, 128, [1], 0, 0),
    (1, 1, 16, [1], 0, 0),
    (2, 256, 256, [256, 256], 0, 0),
    (3, 200, 144, [5, 0, 9], 3, 11),
    (4, 129, 400, [0, 0, 17, 0], 0, 2),
    (8, 512, 1040, [3, 1, 7, 0, 2, 8, 15, 1], 0, 0),
    (5, 300, 272, [100, 33, 64, 1, 250], 7, 30),
    (2, 768, 2064, [513, 260], 1, 0),
    (3, 96, 1536, [225, 448, 31], 5, 9),
    (2, 40, 16, [1025, 3], 0, 6),
    (40, 24, 64, [i % 5 for i in range(40)], 2, 1),
    (300, 8, 32, [(i * 7) % 3 for i in range(300)], 0, 0),
    (1, 1030, 128, [2000], 0, 0),
    (6, 16, 4096, [700, 0, 129, 128, 127, 4], 6, 0),
    (2, 300, 6000, [5, 40], 0, 0),
    (1, 70, 11008, [1], 0, 7),
    (9, 1300, 1024, [30, 0, 128, 127, 1, 64, 65, 2, 90], 5, 3),
    (1, 4096, 912, [61], 3, 0),
    (2, 5000, 160, [7, 20], 1, 4),
    (3, 700, 8192, [70, 1, 25], 0, 3),
    (3, 6000, 704, [90, 1, 5], 9, 0),
    (2, 333, 256, [257, 250], 7, 0),
    # several strips of column tiles
    (3, 300, 272, [3400, 100, 2900], 3, 5),
    (2, 600, 1040, [6500, 2110], 0, 0),
]


@pytest.mark.parametrize("E,R,K,counts,start,behind", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(E, R, K, counts, start, behind, dtype):
    g = torch.Generator(device=DEV).manual_seed(E * 1000 + R + K)
    values, meta, dense = experts(E, R, K, g)
    at, off = offsets_of(counts, start)
    S = at[-1] + behind
    X = rows(K, S, g, pad=8)
    y = torch.full((R, (S + 7) // 8 * 8), 7.0, device=DEV, dtype=dtype)
    nm.nm_experts_spmm(values, meta, 2, 4, E, R, K, X, X.stride(0), S, off, y, y.stride(0),
                       nm.NM_OUT_F32 if dtype == F32 else nm.NM_OUT_BF16)
    nm.nm_device_status()
    assert (y[:, :start] == 7).all() and (y[:, at[-1]:] == 7).all()
    for e in range(E):
        x = X[:, at[e]:at[e + 1]].double()
        close(y[:, at[e]:at[e + 1]], dense[e] @ x, dense[e].abs() @ x.abs(), K // 2, f"expert {e}")


@pytest.mark.parametrize("E,R,K,counts,start,behind", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_input_gradient(E, R, K, counts, start, behind, dtype):
    g = torch.Generator(device=DEV).manual_seed(E * 1000 + R + K + 1)
    values, meta, dense = experts(E, R, K, g)
    at, off = offsets_of(counts, start)
    S = at[-1] + behind
    dY = rows(R, S, g, pad=16)
    dx = torch.full((K, (S + 7) // 8 * 8), 7.0, device=DEV, dtype=dtype)
    nm.nm_experts_spmm_t(values, meta, 2, 4, E, R, K, dY, dY.stride(0), S, off, dx, dx.stride(0),
                         nm.NM_OUT_F32 if dtype == F32 else nm.NM_OUT_BF16)
    nm.nm_device_status()
    assert (dx[:, :start] == 7).all() and (dx[:, at[-1]:] == 7).all()
    for e in range(E):
        d = dY[:, at[e]:at[e + 1]].double()
        close(dx[:, at[e]:at[e + 1]], dense[e].T @ d, dense[e].T.abs() @ d.abs(), R, f"expert {e}")


@pytest.mark.parametrize("E,R,K,counts,start,behind", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_survivor_gradient(E, R, K, counts, start, behind, dtype):
    g = torch.Generator(device=DEV).manual_seed(E * 1000 + R + K + 2)
    values, meta, _ = experts(E, R, K, g)
    kept = torch.stack([nm.decompress(torch.ones_like(values[e]), meta[e], K, 2, 4) for e in range(E)]) != 0
    at, off = offsets_of(counts, start)
    S = at[-1] + behind
    X, dY = rows(K, S, g), rows(R, S, g, pad=8)
    X[:, :start], dY[:, at[-1]:] = float("nan"), float("inf")  # columns of no expert
    dv = nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off, out_dtype=dtype)
    nm.nm_device_status()
    for e in range(E):
        d, x = dY[:, at[e]:at[e + 1]].double(), X[:, at[e]:at[e + 1]].double()
        ref = (d @ x.T)[kept[e]].view(R, K // 2)
        mag = (d.abs() @ x.abs().T)[kept[e]].view(R, K // 2)
        close(dv[e], ref, mag, counts[e], f"expert {e}")
        if counts[e] == 0:
            assert (dv[e] == 0).all()


def test_columns_and_experts_are_apart():
    """A NaN or Inf in one expert's weights or columns stays with it, in all three products."""
    g = torch.Generator(device=DEV).manual_seed(5)
    E, R, K, counts = 4, 70, 96, [21, 30, 13, 27]
    values, meta, dense = experts(E, R, K, g)
    at, off = offsets_of(counts, 2)
    X, dY = rows(K, at[-1], g), rows(R, at[-1], g)
    good = [nm.experts_spmm(values, meta, 2, 4, K, X, off), nm.experts_spmm_t(values, meta, 2, 4, K, dY, off),
            nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off)]
    for e in (1, 3):
        values[e, R // 2, 3] = float("nan")
        values[e, R - 1, 5] = float("inf")
        X[7, at[e] + 1] = float("inf")
        dY[9, at[e + 1] - 1] = float("nan")
    bad = [nm.experts_spmm(values, meta, 2, 4, K, X, off), nm.experts_spmm_t(values, meta, 2, 4, K, dY, off),
           nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off)]
    for e in (0, 2):
        for a, b in zip(good[:2], bad[:2]):
            assert torch.equal(a[:, at[e]:at[e + 1]], b[:, at[e]:at[e + 1]])
        assert torch.equal(good[2][e], bad[2][e])
    assert bad[0][:, at[1]:at[2]].isnan().any() and bad[2][1].isnan().any()


def test_offsets_outside_the_matrix_are_clamped():
    g = torch.Generator(device=DEV).manual_seed(6)
    values, meta, dense = experts(2, 64, 64, g)
    X, dY = rows(64, 24, g), rows(64, 24, g)
    wild = torch.tensor([-9, 10, 2 ** 30], dtype=torch.int32, device=DEV)
    tame = torch.tensor([0, 10, 24], dtype=torch.int32, device=DEV)
    for a, b in ((nm.experts_spmm(values, meta, 2, 4, 64, X, o), nm.experts_spmm_t(values, meta, 2, 4, 64, dY, o))
                 for o in (wild, tame)):
        assert torch.equal(a, nm.experts_spmm(values, meta, 2, 4, 64, X, tame))
        assert torch.equal(b, nm.experts_spmm_t(values, meta, 2, 4, 64, dY, tame))
    assert torch.equal(nm.experts_sddmm(meta, 2, 4, 64, 64, dY, X, wild), nm.experts_sddmm(meta, 2, 4, 64, 64, dY, X, tame))


def test_captured_and_replayed_with_other_counts():
    """The counts are read when the kernels run: a captured step serves any of them."""
    g = torch.Generator(device=DEV).manual_seed(7)
    E, R, K, S = 3, 130, 160, 90
    values, meta, _ = experts(E, R, K, g)
    X, dY = rows(K, S, g), rows(R, S, g)
    off = torch.tensor([0, 20, 50, 90], dtype=torch.int32, device=DEV)

    def step():
        return (nm.experts_spmm(values, meta, 2, 4, K, X, off), nm.experts_spmm_t(values, meta, 2, 4, K, dY, off),
                nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for at in ([0, 20, 50, 90], [0, 0, 90, 90], [0, 31, 33, 90]):
        off.copy_(torch.tensor(at, dtype=torch.int32))
        X.normal_()
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_streams_and_repeats():
    """Calls on two streams at once, each repeated: equal bits."""
    g = torch.Generator(device=DEV).manual_seed(8)
    E, R, K, S = 4, 512, 512, 700
    values, meta, _ = experts(E, R, K, g)
    off = torch.tensor([0, 333, 334, 600, 700], dtype=torch.int32, device=DEV)
    X, dY = rows(K, S, g), rows(R, S, g)
    want = nm.experts_spmm(values, meta, 2, 4, K, X, off), nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for s in streams:
            got.append((nm.experts_spmm(values, meta, 2, 4, K, X, off, stream=s),
                        nm.experts_sddmm(meta, 2, 4, R, K, dY, X, off, stream=s)))
    torch.cuda.synchronize()
    for y, dv in got:
        assert torch.equal(y, want[0]) and torch.equal(dv, want[1])


def test_nothing_to_do():
    values, meta = torch.empty((0, 8, 8), dtype=BF, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    off = torch.zeros(1, dtype=torch.int32, device=DEV)
    X = torch.randn((16, 8), device=DEV).to(BF)
    assert nm.experts_spmm(values, meta, 2, 4, 16, X, off).shape == (8, 8)
    g = torch.Generator(device=DEV).manual_seed(9)
    values, meta, _ = experts(2, 8, 16, g)
    none = torch.empty((16, 0), dtype=BF, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert nm.experts_spmm(values, meta, 2, 4, 16, none, off).shape == (8, 0)
    assert (nm.experts_sddmm(meta, 2, 4, 8, 16, none[:8], none, off) == 0).all()
    X = torch.randn((16, 24), device=DEV).to(BF)
    assert (nm.experts_sddmm(meta, 2, 4, 8, 16, X[:8], X, off) == 0).all()
