"""Cross entropy of a pruned output head and its gradients against the 64-bit definition.

Tolerances.  A logit is a float32 sum of K products of bf16 numbers (exact in
float32), in any order and truncated at worst: off by at most K 2^-23 times
the sum of magnitudes.  lse moves by at most the largest logit error, plus the
roundings of the exponentials (a few 2^-22 and 2^-23 of their arguments) and
of their sum.  G is rounded to bf16 once (2^-8) and carries the errors of
exp(z - lse); dX and dV add R or T such terms and are rounded once.  On top, the
acceptance rule of the library's GEMMs for whole results: a relative Frobenius
error of at most 5e-3.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_nm_b200 as nm
import train_reference as ref
import workloads as wl
from gpu_helpers import DEV, FROB_TOL, to_dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def padded(bits):
    """bf16 bits on the device, rows padded to 16 bytes with NaN, which nothing may use."""
    r, c = bits.shape
    buf = np.full((r, -(-c // 8) * 8), 0x7FC0, np.uint16)
    buf[:, :c] = bits
    return to_dev(buf)[:, :c]


def f64(t):
    return t.detach().to("cpu", torch.float64)


class Case:
    def __init__(self, R, K, T, n=2, m=4, permuted=False, seed=0, scale=0.05):
        self.R, self.K, self.T, self.n, self.m = R, K, T, n, m
        vals, meta = oracle.compress(wl.normal_bf16((R, K), scale, seed + 1), n, m)
        X = wl.normal_bf16((K, T), 1.0, seed + 2)
        self.values, self.meta = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV)
        self.X = padded(X)
        self.perm = wl.permutation(K, seed + 3) if permuted else None
        self.idx = None if self.perm is None else torch.from_numpy(self.perm).to(DEV)
        rng = np.random.Generator(np.random.PCG64(seed + 4))
        target = rng.integers(0, R, T).astype(np.int32)
        target[rng.random(T) < 0.15] = -100
        special = [0, R - 1, R, -1, 2 ** 31 - 1, min(R - 1, 255), min(R - 1, 256)]
        target[:len(special)] = special[:T]
        self.target = torch.from_numpy(target)
        self.dloss = torch.from_numpy(rng.standard_normal(T).astype(np.float32))
        w = wl.bf16_to_f32(oracle.decompress(vals, meta, K, n, m)).astype(np.float64)
        x = wl.bf16_to_f32(X).astype(np.float64)
        self.w, self.x = torch.from_numpy(w), torch.from_numpy(x if self.perm is None else x[self.perm])
        self.cols = torch.from_numpy(oracle.positions(meta, R, K, n, m).astype(np.int64))
        self.cols += (torch.arange(self.cols.shape[1]) // n * m)[None, :]

    def args(self):
        return self.values, self.meta, self.n, self.m, self.K, self.X, self.target.to(DEV)

    def logit_error(self):
        return self.K * 2.0 ** -23 * (self.w.abs() @ self.x.abs())

    def check_loss(self, loss, lse):
        z = self.w @ self.x
        want_loss, want_lse = ref.cross_entropy(z, self.target.long())
        ez = self.logit_error().max(0).values
        spread = z.max(0).values - z.min(0).values + 1
        e = ez + 2.0 ** -20 + (self.R / 200 + 60) * 2.0 ** -24 + spread * 2.0 ** -22 + 2.0 ** -22 * want_lse.abs()
        assert (f64(lse) - want_lse).abs().le(e).all()
        e_loss = 2 * e + 2.0 ** -23 * (want_loss.abs() + z.abs().max(0).values)
        has = (self.target >= 0) & (self.target < self.R)
        assert (f64(loss) - want_loss).abs().le(e_loss).all()
        assert (f64(loss)[~has] == 0).all()

    def check_grad(self, lse, dX, dV):
        z, dl = self.w @ self.x, self.dloss.double()
        G, dXp, dW = ref.cross_entropy_grad(self.w, self.x, self.target.long(), dl)
        has = (self.target >= 0) & (self.target < self.R)
        p = torch.softmax(z, 0) * has * dl.abs()
        # exp(z - lse) of a logit and an lse that are off: relative, doubled for the second order
        rel = 2 * (2 * self.logit_error().max(0).values + 2.0 ** -19 + (z.abs().max(0).values + 1) * 2.0 ** -20)
        eG = G.abs() * ref.UBF16 + p * rel * (1 + ref.UBF16)
        if dX is not None:
            w, aG = self.w.abs(), G.abs() + eG
            e = w.T @ eG + self.R * 2.0 ** -23 * (w.T @ aG)
            bound = e + ref.UBF16 * (dXp.abs() + e) + 1e-30
            want = dXp if self.perm is None else torch.empty_like(dXp).index_copy_(0, torch.from_numpy(self.perm).long(), dXp)
            back = bound if self.perm is None else torch.empty_like(bound).index_copy_(0, torch.from_numpy(self.perm).long(), bound)
            assert (f64(dX) - want).abs().le(back).all()
            assert (f64(dX) - want).norm() <= FROB_TOL * want.norm() + 1e-30
        if dV is not None:
            x, aG = self.x.abs(), G.abs() + eG
            e = (eG @ x.T + self.T * 2.0 ** -23 * (aG @ x.T)).gather(1, self.cols)
            want = dW.gather(1, self.cols)
            assert (f64(dV) - want).abs().le(e + ref.UBF16 * (want.abs() + e) + 1e-30).all()
            assert (f64(dV) - want).norm() <= FROB_TOL * want.norm() + 1e-30

    def run(self, **kw):
        loss, lse = nm.spmm_xent(*self.args(), idx=self.idx)
        return (loss, lse) + nm.spmm_xent_grad(*self.args(), lse, self.dloss.to(DEV), idx=self.idx, **kw)


# (R, K, T): one class; one token; the skinny, one-SM and SM-pair GEMMs behind it; ragged rows, columns and tokens;
# several pieces of the vocabulary (7168 rows each at T = 2300) whose last is ragged
SHAPES = [(1, 16, 1), (2, 64, 9), (1000, 768, 256), (300, 128, 37), (513, 264, 197), (2050, 1280, 200), (700, 2048, 24),
          (8500, 128, 2300)]


@pytest.mark.parametrize("R,K,T", SHAPES)
@pytest.mark.parametrize("permuted", [False, True])
def test_loss_and_gradients(R, K, T, permuted):
    c = Case(R, K, T, permuted=permuted, seed=R + T)
    loss, lse, dX, dV = c.run()
    torch.cuda.synchronize()
    nm.nm_device_status()
    c.check_loss(loss, lse)
    c.check_grad(lse, dX, dV)


@pytest.mark.parametrize("n,m", [(1, 2), (1, 4), (1, 8), (2, 8), (3, 4), (5, 16)])
@pytest.mark.parametrize("R,K,T", [(520, 256, 200), (70, 48, 20), (300, 384, 33)])
def test_other_patterns(n, m, R, K, T):
    c = Case(R, K, T, n, m, permuted=True, seed=m + T)
    loss, lse, dX, dV = c.run()
    nm.nm_device_status()
    c.check_loss(loss, lse)
    c.check_grad(lse, dX, dV)


# 32-deep tiles enough for every SM, where a token count inside the first or third 16 is padded before the skinny GEMM
@pytest.mark.parametrize("T,permuted", [(1, False), (13, True), (16, False), (33, True), (47, False)])
def test_loss_of_few_tokens_over_a_large_vocabulary(T, permuted):
    c = Case(20000, 2048, T, permuted=permuted, seed=21)
    loss, lse = nm.spmm_xent(*c.args(), idx=c.idx)
    nm.nm_device_status()
    c.check_loss(loss, lse)


@pytest.mark.parametrize("K,T", [(256, 256), (256, 20), (40, 70)])
def test_large_logits_neither_overflow_nor_vanish(K, T):
    """Logits of several hundred: exp of them overflows unless the column's largest is taken off first."""
    c = Case(600, K, T, seed=5, scale=20.0)
    loss, lse, dX, dV = c.run()
    assert lse.isfinite().all() and (lse > 100).any()
    c.check_loss(loss, lse)
    c.check_grad(lse, dX, dV)


def test_one_gradient_alone():
    c = Case(520, 256, 200, seed=6)
    loss, lse, dX, dV = c.run()
    x_only, v_only = c.run(need_dv=False), c.run(need_dx=False)
    assert x_only[3] is None and v_only[2] is None
    assert torch.equal(x_only[2], dX) and torch.equal(v_only[3], dV)


@pytest.mark.parametrize("T", [256, 20])
def test_no_token_has_a_loss(T):
    c = Case(300, 128, T, seed=7)
    c.target.fill_(-100)
    loss, lse, dX, dV = c.run()
    assert not loss.any() and not dX.any() and not dV.any()
    c.check_loss(loss, lse)


@pytest.mark.parametrize("token", [7, 20, 33])
def test_a_bad_token_stays_alone(token):
    c = Case(600, 256, 200, seed=8)
    loss, lse, dX, _ = c.run()
    c.X[3, token] = float("nan")
    loss2, lse2, dX2, _ = c.run()
    keep = [t for t in range(200) if t != token]
    assert lse2[token].isnan()
    if 0 <= c.target[token] < 600:
        assert loss2[token].isnan() and dX2[:, token].isnan().any()
    else:  # a token without a loss has neither, whatever its features are
        assert loss2[token] == 0 and not dX2[:, token].any()
    assert torch.equal(loss2[keep], loss[keep]) and torch.equal(dX2[:, keep], dX[:, keep])


def test_no_tokens():
    c = Case(40, 64, 8, seed=9)
    X, none = c.X[:, :0], torch.zeros(0, device=DEV)
    loss, lse = nm.spmm_xent(c.values, c.meta, 2, 4, 64, X, none.int())
    dX, dV = nm.spmm_xent_grad(c.values, c.meta, 2, 4, 64, X, none.int(), none, none)
    assert loss.shape == lse.shape == (0,) and dX.shape == (64, 0) and not dV.any()


def test_outputs_beyond_the_tokens_are_left_alone():
    c = Case(600, 256, 197, seed=10)
    loss, lse, dX, dV = c.run()
    out = torch.full((2, 200), 5.0, device=DEV)
    t = c.target.to(DEV)
    nm.nm_spmm_xent(c.values, c.meta, 2, 4, 600, 256, None, c.X, c.X.stride(0), 197, t, out[0], out[1])
    assert torch.equal(out[0, :197], loss) and torch.equal(out[1, :197], lse) and (out[:, 197:] == 5).all()
    wide = torch.full((256, 216), 5.0, dtype=BF, device=DEV)
    dv = torch.full((601, 128), 5.0, dtype=BF, device=DEV)
    nm.nm_spmm_xent_grad(c.values, c.meta, 2, 4, 600, 256, None, c.X, c.X.stride(0), 197, t, lse, c.dloss.to(DEV), wide,
                         216, dv)
    assert torch.equal(wide[:, :197], dX) and (wide[:, 197:] == 5).all()
    assert torch.equal(dv[:600], dV) and (dv[600] == 5).all()


def test_index_map_entries_outside_drop_their_rows():
    c = Case(300, 128, 40, permuted=True, seed=11)
    gone = [3, 77]
    row = c.perm[gone].copy()
    c.perm[gone] = [-1, 128]
    c.idx = torch.from_numpy(c.perm).to(DEV)
    c.x[gone] = 0.0
    loss, lse = nm.spmm_xent(*c.args(), idx=c.idx)
    c.check_loss(loss, lse)
    dX = torch.full((128, 40), 5.0, dtype=BF, device=DEV)
    nm.nm_spmm_xent_grad(c.values, c.meta, 2, 4, 300, 128, c.idx, c.X, c.X.stride(0), 40, c.target.to(DEV), lse,
                         c.dloss.to(DEV), dX, 40)
    assert (dX[row.tolist()] == 5).all()  # rows that no entry names are not written
    dXp = ref.cross_entropy_grad(c.w, c.x, c.target.long(), c.dloss.double())[1]
    keep = [k for k in range(128) if k not in gone]
    got = f64(dX)[c.perm[keep].astype(np.int64)]
    assert (got - dXp[keep]).norm() <= FROB_TOL * dXp[keep].norm()


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    c = Case(2050, 256, 300, permuted=True, seed=12)
    first = c.run()
    torch.cuda.synchronize()
    args, dl = c.args(), c.dloss.to(DEV)
    torch.cuda.synchronize()

    def once(stream=None):
        loss, lse = nm.spmm_xent(*args, idx=c.idx, stream=stream)
        return (loss, lse) + nm.spmm_xent_grad(*args, lse, dl, idx=c.idx, stream=stream)

    side = [torch.cuda.Stream() for _ in range(2)]
    runs = [once(s) for s in side * 3]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once())
        graphs.append(g)
    for s, g in zip(side * 2, graphs * 2):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    nm.nm_device_status()
    for got in runs + outs:
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_refusals():
    c = Case(32, 64, 8, seed=13)
    t, v8 = c.target.to(DEV), torch.zeros(8, device=DEV)
    ok = (c.values, c.meta, 2, 4, 64, c.X)
    for kw, match in (((*ok, t.long()), "target"), ((*ok, t[:7]), "target"), ((c.values[:, :16], *ok[1:], t), "values"),
                      ((c.values, c.meta[:4], *ok[2:], t), "meta"), ((*ok[:5], c.X[:60], t), "rows"),
                      ((*ok[:5], c.X.float(), t), "X must be"), ((*ok[:5], c.X.cpu(), t), "CUDA")):
        with pytest.raises(ValueError, match=match):
            nm.spmm_xent(*kw)
    with pytest.raises(ValueError, match="idx"):
        nm.spmm_xent(*ok, t, idx=torch.arange(64, device=DEV))
    with pytest.raises(ValueError, match="lse"):
        nm.spmm_xent_grad(*ok, t, v8[:4], v8)
    with pytest.raises(ValueError, match="dloss"):
        nm.spmm_xent_grad(*ok, t, v8, v8.double())
    with pytest.raises(nm.NmError) as e:
        nm.spmm_xent_grad(*ok, t, v8, v8, need_dx=False, need_dv=False)
    assert e.value.status == nm.NM_ERR_INVALID_ARG
    with pytest.raises(nm.NmError) as e:
        nm.spmm_xent(c.values, c.meta, 2, 5, 64, c.X, t)
    assert e.value.status == nm.NM_ERR_INVALID_ARG


# one SM pair's tile of dX over thousands of rows, taken in several ranges; with several pieces, the last too small for all
@pytest.mark.parametrize("R,K,T", [(9000, 136, 14), (5000, 256, 200), (4500, 128, 300)])
def test_gradients_of_a_large_vocabulary_and_few_features(R, K, T):
    c = Case(R, K, T, seed=23)
    loss, lse, dX, dV = c.run()
    nm.nm_device_status()
    c.check_loss(loss, lse)
    c.check_grad(lse, dX, dV)


# The SM-pair epilogue; the one-SM, skinny (whole and split) and dense GEMMs, whose logits the pair kernel reads
@pytest.mark.parametrize("R,K,T", [(600, 128, 256), (300, 1280, 200), (600, 256, 100), (700, 2048, 24), (500, 136, 80)])
@pytest.mark.parametrize("above", [20.0, 60.0, 200.0])
def test_loss_of_a_confident_token_is_small_and_not_negative(R, K, T, above):
    """Target logits far above the rest, where the loss is far below the logits' own roundings.

    The target has the largest logit, so the loss is log(1 + sum of exp(z - z_target)): no term of the size of the logits
    is left in it.  An error e in every logit changes a term by a factor of exp(2 e); the exponentials add 2^-19 (their
    arguments are below 128 where a term counts); every addition to a sum between 1 and 2 rounds by 2^-24, and a sum takes
    at most 32 + 8 + 8 + 32 of them on its way (fewer in the SM-pair epilogue).
    """
    c = Case(R, K, T, seed=31, scale=0.3)
    rng = np.random.Generator(np.random.PCG64(32))
    target = rng.integers(0, R, T)
    w = c.w[torch.from_numpy(target)]
    x = (above * rng.uniform(0.9, 1.1, T))[:, None] * (w / (w * w).sum(1, keepdim=True)).numpy() + 0.02 * rng.standard_normal((T, K))
    X = wl.bf16_bits(x.T.astype(np.float32))
    c.X, c.x = padded(X), torch.from_numpy(wl.bf16_to_f32(X).astype(np.float64))
    c.target = torch.from_numpy(target.astype(np.int32))
    loss, lse = nm.spmm_xent(*c.args())
    z = c.w @ c.x
    top = z.gather(0, c.target.long()[None, :])[0]
    rest = (z - top).exp().scatter_(0, c.target.long()[None, :], 0.0)
    assert (rest < 1).all()  # the target leads everywhere
    want = torch.log1p(rest.sum(0))
    e = 2 * c.logit_error().max(0).values
    got = f64(loss)
    assert (got >= 0).all(), f"{int((got < 0).sum())} negative losses, down to {float(got.min()):.2e}"
    assert (got - want).abs().le(want * (2 * e + 2.0 ** -19) + 80 * 2.0 ** -24).all()
    c.check_loss(loss, lse)


@pytest.mark.parametrize("K,T", [(768, 192), (768, 248), (768, 255), (768, 256), (776, 256), (768, 100), (768, 16)])
def test_gradients_of_few_tokens_carry_two_terms_on_every_gemm(K, T):
    """Up to 256 tokens dX and dV are the 64-bit gradients but for their own rounding, on whichever GEMM the shape takes.

    A value off by a relative d before it is rounded lands on the other side of a rounding boundary with a probability of
    at most d x / ulp(x), and is then off by ulp(x) <= 2^-7 x from the rounded exact value: a relative Frobenius distance of
    sqrt(d 2^-7).  G's second term loses 2^-17; d = 2^-13 leaves 16 times that for the float32 logits and sums: 2^-10.  One
    term alone (errors of 1.5e-3) would give 2.4e-3.
    """
    c = Case(1000, K, T, permuted=True, seed=41)
    loss, lse, dX, dV = c.run()
    c.check_grad(lse, dX, dV)
    G, dXp, dW = ref.cross_entropy_grad(c.w, c.x, c.target.long(), c.dloss.double())
    want = torch.empty_like(dXp).index_copy_(0, torch.from_numpy(c.perm).long(), dXp), dW.gather(1, c.cols)
    for got, exact in zip((dX, dV), want):
        assert (f64(got) - f64(exact.to(BF))).norm() <= 2.0 ** -10 * exact.norm()


# Each source of G: both SM-pair epilogues, and the pass over the logits of the one-SM, skinny and dense GEMMs
@pytest.mark.parametrize("K,T", [(256, 200), (256, 264), (256, 100), (256, 24), (40, 300)])
def test_a_token_with_no_weight_in_the_loss_has_no_gradient(K, T):
    """dloss = 0 masks a token as a target outside does: its column of dX is 0 although its logits are not finite."""
    c = Case(600, K, T, seed=51)
    c.target.copy_(torch.arange(T) % 600)
    masked = [0, 3, 17, T - 1]
    c.dloss[masked] = 0.0
    dX, dV = c.run()[2:]
    assert not dX[:, masked].any()
    c.X[5, masked[:2]] = float("nan")
    c.X[5, masked[2:]] = float("inf")
    dX2 = c.run()[2]
    assert torch.equal(dX2, dX)


def test_pieces_of_a_large_vocabulary_of_few_tokens():
    """Several pieces whose G has two terms, the last one ragged: one token of eight features, half a million rows."""
    c = Case(530_001, 16, 1, seed=61)
    c.target.fill_(300_000)
    loss, lse, dX, dV = c.run()
    nm.nm_device_status()
    c.check_loss(loss, lse)
    c.check_grad(lse, dX, dV)


def test_two_terms_repeat_bit_for_bit_on_streams_and_in_graphs():
    cases = [Case(1500, 256, T, permuted=True, seed=62 + T) for T in (200, 256, 37)]
    data = [(c.args(), c.dloss.to(DEV), c.idx) for c in cases]

    def once(stream=None):
        out = []
        for args, dl, idx in data:
            loss, lse = nm.spmm_xent(*args, idx=idx, stream=stream)
            out += [loss, lse, *nm.spmm_xent_grad(*args, lse, dl, idx=idx, stream=stream)]
        return out

    first = once()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    runs = [once(s) for s in side * 2]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(once())
        graphs.append(g)
    for s, g in zip(side * 2, graphs * 3):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    nm.nm_device_status()
    for got in runs + outs:
        assert all(torch.equal(a, b) for a, b in zip(got, first))
