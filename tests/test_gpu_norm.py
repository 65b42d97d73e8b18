"""Layer norm over the features of each token, forward and backward, against the 64-bit definition.

Tolerances are error bounds of the float32 arithmetic: a sum whose longest
chain has n additions is off by at most n u / (1 - n u) of the sum of
magnitudes (u = 2^-24), and the result is rounded once to its type (at most
2^-8 of its magnitude for bf16).  A thread adds at most K / 32 rows and T / 256
strips, plus fewer than 40 joins.
"""
import pytest
import torch

import sparse_gemm_nm_b200 as nm
import train_reference as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# (K, T): one token, one feature, ragged strips, every strip width and cluster size, slabs above a quarter of an SM,
# and a K too large for a cluster's shared memory, where the strip is read again in every pass
SHAPES = [(1, 1), (5, 1), (1, 9), (24, 17), (768, 197), (257, 64), (4096, 40), (5120, 16), (4097, 72), (8200, 33),
          (33000, 9), (9, 5000), (500, 20000), (40000, 50), (113000, 3)]


def rows(A, dtype):
    """A (float64, CPU) on the device as dtype, rows padded to 16 bytes; padding holds NaN, which nothing may read."""
    per = 4 if dtype == F32 else 8
    r, c = A.shape
    buf = torch.full((r, -(-c // per) * per), float("nan"), dtype=dtype, device=DEV)
    buf[:, :c] = A.to(dtype).to(DEV)
    return buf[:, :c]


def f64(t):
    return t.detach().to("cpu", torch.float64)


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def half_step(dtype):
    return ref.UBF16 if dtype == BF else ref.U32


def case(K, T, xt, offset=0.0):
    x = rows(rand(K, T, seed=K + T) * 1.5 + offset, xt)
    gamma = (1 + 0.1 * rand(K, seed=3)).float().to(DEV)
    beta = (0.1 * rand(K, seed=4)).float().to(DEV)
    return x, gamma, beta


def check_forward(x, gamma, beta, eps, y, mean, rstd):
    K = x.shape[0]
    X, g, b = f64(x), f64(gamma) if gamma is not None else None, f64(beta) if beta is not None else None
    ry, rm, rr = ref.layer_norm(X, g, b, eps)
    c = ref.chain(K // 32 + 40)
    e_mean = c * X.abs().mean(0) + ref.U32 * rm.abs()
    # squares about a mean that is off by e_mean, added with relative error c; then a square root and a division
    e_rstd = rr * (c + 4 * ref.U32 + (e_mean * rr) ** 2)
    assert (f64(mean) - rm).abs().le(e_mean + 1e-30).all()
    assert (f64(rstd) - rr).abs().le(e_rstd).all()
    gm = (g if g is not None else torch.ones(K, dtype=torch.float64)).abs()[:, None]
    bm = b.abs()[:, None] if b is not None else 0.0
    h = ((X - rm) * rr).abs()
    e = gm * (h * (e_rstd / rr + 4 * ref.U32) + e_mean * rr * (1 + 1e-3)) + 2 * ref.U32 * (ry.abs() + bm)
    bound = e + half_step(y.dtype) * (ry.abs() + e) + 1e-30
    bad = (f64(y) - ry).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} values off by up to {float(((f64(y) - ry).abs() / bound).max()):.2f} bounds"


def check_backward(dy, x, mean, rstd, gamma, dx, dgamma, dbeta):
    K, T = x.shape
    X, dY, m, r = f64(x), f64(dy), f64(mean), f64(rstd)
    g = f64(gamma) if gamma is not None else torch.ones(K, dtype=torch.float64)
    h, gy = (X - m) * r, g[:, None] * dY
    c = ref.chain(K // 32 + 40)
    c1, c2 = gy.sum(0) / K, (gy * h).sum(0) / K
    want = r * (gy - c1 - h * c2)
    e1, e2 = (c + 3 * ref.U32) * gy.abs().mean(0), (c + 8 * ref.U32) * (gy * h).abs().mean(0)
    e = r * (6 * ref.U32 * (gy.abs() + c1.abs() + (h * c2).abs()) + e1 + h.abs() * e2) * (1 + 1e-3)
    bound = e + half_step(dx.dtype) * (want.abs() + e) + 1e-30
    assert (f64(dx) - want).abs().le(bound).all()
    ct = ref.chain(T // 256 + 60)
    assert (f64(dgamma) - (dY * h).sum(1)).abs().le((ct + 4 * ref.U32) * (dY * h).abs().sum(1) + 1e-30).all()
    assert (f64(dbeta) - dY.sum(1)).abs().le(ct * dY.abs().sum(1) + 1e-30).all()


@pytest.mark.parametrize("K,T", SHAPES)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_forward(K, T, xt, yt):
    x, gamma, beta = case(K, T, xt)
    for g, b in ((gamma, beta), (None, beta), (gamma, None), (None, None)):
        y, mean, rstd = nm.layer_norm(x, g, b, eps=1e-5, out_dtype=yt)
        assert y.dtype == yt and y.shape == (K, T)
        check_forward(x, g, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("K,T", SHAPES)
@pytest.mark.parametrize("xt,dt", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("affine", [True, False])
def test_backward(K, T, xt, dt, affine):
    x, gamma, beta = case(K, T, xt)
    gamma = gamma if affine else None
    dy = rows(rand(K, T, seed=9), dt)
    _, mean, rstd = nm.layer_norm(x, gamma, beta)
    dx, dgamma, dbeta = nm.layer_norm_grad(dy, x, mean, rstd, gamma)
    assert dx.dtype == xt and dx.shape == (K, T)
    check_backward(dy, x, mean, rstd, gamma, dx, dgamma, dbeta)


def test_backward_against_autograd_of_the_definition():
    x, gamma, beta = case(300, 70, F32)
    dy = rows(rand(300, 70, seed=10), F32)
    _, mean, rstd = nm.layer_norm(x, gamma, beta)
    got = nm.layer_norm_grad(dy, x, mean, rstd, gamma)
    want = ref.layer_norm_grad(f64(dy), f64(x), f64(gamma), f64(beta))
    for a, b in zip(got, want):
        # mean and rstd carry float32 roundings here (relative 2^-24 times a sum of 300): far below 1e-5
        assert (f64(a) - b).norm() <= 1e-5 * b.norm()


@pytest.mark.parametrize("offset", [100.0, -3000.0])
def test_a_large_common_offset_does_not_cancel(offset):
    x, gamma, beta = case(1000, 50, F32, offset)
    y, mean, rstd = nm.layer_norm(x, gamma, beta, out_dtype=F32)
    check_forward(x, gamma, beta, 1e-5, y, mean, rstd)


def test_equal_features_give_beta():
    x = torch.full((512, 24), 0.75, dtype=BF, device=DEV)  # the mean of equal bf16 values is exact
    beta = rand(512, seed=1).float().to(DEV)
    y, mean, rstd = nm.layer_norm(x, None, beta, out_dtype=F32)
    assert torch.equal(y, beta[:, None].expand(512, 24)) and torch.equal(mean, torch.full((24,), 0.75, device=DEV))


@pytest.mark.parametrize("K,T", [(768, 100), (113000, 9), (40, 3)])
def test_a_bad_token_stays_alone(K, T):
    """NaN and Inf of one token reach no other token's output."""
    x, gamma, beta = case(K, T, BF)
    y0, m0, r0 = nm.layer_norm(x, gamma, beta)
    dy = rows(rand(K, T, seed=2), BF)
    dx0 = nm.layer_norm_grad(dy, x, m0, r0, gamma)[0]
    x2 = rows(f64(x), BF)
    x2[K // 2, 1] = float("nan")
    x2[0, 2] = float("inf")
    y, m, r = nm.layer_norm(x2, gamma, beta)
    dx = nm.layer_norm_grad(dy, x2, m, r, gamma)[0]
    assert y[:, 1].isnan().all() and y[:, 2].isnan().any()
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[:, keep], y0[:, keep]) and torch.equal(dx[:, keep], dx0[:, keep])


def test_padding_is_left_alone_and_strides_are_free():
    K, T, ld = 130, 21, 64
    X = torch.full((K, ld), float("nan"), dtype=BF, device=DEV)
    X[:, :T] = rand(K, T, seed=1).to(BF).to(DEV)
    Y = torch.full((K, 40), 5.0, dtype=BF, device=DEV)
    stats = torch.full((2, T + 1), 5.0, device=DEV)
    nm.nm_layer_norm(X, ld, nm.NM_OUT_BF16, K, T, None, None, 1e-5, Y, 40, nm.NM_OUT_BF16, stats[0], stats[1])
    check_forward(X[:, :T], None, None, 1e-5, Y[:, :T], stats[0, :T], stats[1, :T])
    assert (Y[:, T:] == 5).all() and (stats[:, T] == 5).all()
    dY = torch.full((K, 24), float("nan"), dtype=F32, device=DEV)
    dY[:, :T] = rand(K, T, seed=2).float().to(DEV)
    dX = torch.full((K, 48), 5.0, dtype=BF, device=DEV)
    sums = torch.full((2, K + 1), 5.0, device=DEV)
    nm.nm_layer_norm_grad(dY, 24, nm.NM_OUT_F32, X, ld, nm.NM_OUT_BF16, K, T, None, stats[0], stats[1], dX, 48,
                          sums[0], sums[1])
    check_backward(dY[:, :T], X[:, :T], stats[0, :T], stats[1, :T], None, dX[:, :T], sums[0, :K], sums[1, :K])
    assert (dX[:, T:] == 5).all() and (sums[:, K] == 5).all()


def test_optional_outputs():
    x, gamma, beta = case(64, 16, BF)
    y, mean, rstd = nm.layer_norm(x, gamma, beta)
    Y = torch.empty((64, 16), dtype=BF, device=DEV)
    nm.nm_layer_norm(x, 16, 0, 64, 16, gamma, beta, 1e-5, Y, 16, 0)
    assert torch.equal(Y, y)
    dy = rows(rand(64, 16, seed=1), BF)
    dx, dgamma, dbeta = nm.layer_norm_grad(dy, x, mean, rstd, gamma)
    for want in (None, "dgamma", "dbeta"):
        dX, v = torch.empty((64, 16), dtype=BF, device=DEV), torch.full((64,), 5.0, device=DEV)
        nm.nm_layer_norm_grad(dy, 16, 0, x, 16, 0, 64, 16, gamma, mean, rstd, dX, 16, v if want == "dgamma" else None,
                              v if want == "dbeta" else None)
        assert torch.equal(dX, dx)
        assert torch.equal(v, dgamma if want == "dgamma" else dbeta if want == "dbeta" else torch.full_like(v, 5.0))


def test_no_tokens():
    x = torch.zeros((8, 0), dtype=BF, device=DEV)
    before = nm.nm_launch_count()
    y, mean, rstd = nm.layer_norm(x)
    assert y.shape == (8, 0) and nm.nm_launch_count() == before
    dx, dgamma, dbeta = nm.layer_norm_grad(x, x, mean, rstd)
    assert dx.shape == (8, 0) and not dgamma.any() and not dbeta.any()


def test_offsets_past_32_bits():
    K, T, ld = 4, 20, 1 << 30  # row 3 starts 3 * 2^30 elements in
    X = torch.empty((K * ld,), dtype=BF, device=DEV).view(K, ld)[:, :T]
    X.copy_(rand(K, T, seed=1))
    y, mean, rstd = nm.layer_norm(X, out_dtype=F32)
    check_forward(X, None, None, 1e-5, y, mean, rstd)
    dy = rows(rand(K, T, seed=2), BF)
    check_backward(dy, X, mean, rstd, None, *nm.layer_norm_grad(dy, X, mean, rstd))
    del X
    torch.cuda.empty_cache()


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    x, gamma, beta = case(768, 1000, BF)
    dy = rows(rand(768, 1000, seed=1), BF)
    first = nm.layer_norm(x, gamma, beta)
    grads = nm.layer_norm_grad(dy, x, first[1], first[2], gamma)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in side * 3:  # two streams at once
        y = nm.layer_norm(x, gamma, beta, stream=s)
        runs.append(y + nm.layer_norm_grad(dy, x, y[1], y[2], gamma, stream=s))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = nm.layer_norm(x, gamma, beta)
            outs.append(y + nm.layer_norm_grad(dy, x, y[1], y[2], gamma))
        graphs.append(g)
    for s, g in zip(side * 2, graphs * 2):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for got in runs + outs:
        assert all(torch.equal(a, b) for a, b in zip(got, first + grads))


def test_refusals():
    x = torch.zeros((16, 8), dtype=BF, device=DEV)
    v16, v8 = torch.zeros(16, device=DEV), torch.zeros(8, device=DEV)
    with pytest.raises(ValueError, match="gamma"):
        nm.layer_norm(x, v8)
    with pytest.raises(ValueError, match="beta"):
        nm.layer_norm(x, v16, v16.to(BF))
    with pytest.raises(ValueError, match="adjacent"):
        nm.layer_norm(x.t())
    with pytest.raises(ValueError, match="X must be"):
        nm.layer_norm(x.half())
    with pytest.raises(ValueError, match="output type"):
        nm.layer_norm(x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="shape"):
        nm.layer_norm_grad(torch.zeros((16, 16), dtype=BF, device=DEV), x, v8, v8)
    with pytest.raises(ValueError, match="CUDA"):
        nm.layer_norm(x.cpu())
    for bad in (torch.zeros((16, 9), dtype=BF, device=DEV), torch.zeros((16, 17), dtype=BF, device=DEV)[:, 1:9]):
        with pytest.raises(nm.NmError) as e:
            nm.layer_norm(bad)
        assert e.value.status == nm.NM_ERR_MISALIGNED
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(nm.NmError) as e:
            nm.layer_norm(x, eps=eps)
        assert e.value.status == nm.NM_ERR_INVALID_ARG
    with pytest.raises(nm.NmError):
        nm.layer_norm(torch.zeros((0, 8), dtype=BF, device=DEV))
