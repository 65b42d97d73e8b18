"""Low-rank adapters of many requests beside the pruned projection, and their gradients, against the 64-bit definition.

Tolerances, with u = 2^-24 and 2^-23 for an addition that truncates: S = A x
adds at most 128 products before it leaves the tensor core's accumulator and
K / 128 + 16 parts after that.  As an operand S loses 2^-16 in two bf16 terms
(bf16 results) or 2^-24 in three (fp32 results) and is multiplied by the scale
once; rank (or T) products of each term add up.  The projection is a float32
sum of K products.  The result is rounded once to its type.
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
TRUNC = 2.0 ** -23


def padded(bits):
    r, c = bits.shape
    buf = np.full((r, -(-c // 8) * 8), 0x7FC0, np.uint16)  # NaN, which nothing may use
    buf[:, :c] = bits
    return to_dev(buf)[:, :c]


def f64(t):
    return t.detach().to("cpu", torch.float64)


def host(bits):
    return torch.from_numpy(wl.bf16_to_f32(bits).astype(np.float64))


class Case:
    def __init__(self, R, K, T, adapters, rank, kind="mixed", permuted=False, scaled=True, n=2, m=4, seed=0):
        self.R, self.K, self.T, self.n, self.m, self.N, self.rank = R, K, T, n, m, adapters, rank
        vals, meta = oracle.compress(wl.normal_bf16((R, K), 0.05, seed + 1), n, m)
        X, dY = wl.normal_bf16((K, T), 1.0, seed + 2), wl.normal_bf16((R, T), 1.0, seed + 3)
        A = wl.normal_bf16((adapters, rank, K), K ** -0.5, seed + 4)
        B = wl.normal_bf16((adapters, R, rank), 0.5 * rank ** -0.5, seed + 5)
        rng = np.random.Generator(np.random.PCG64(seed + 6))
        if kind == "mixed":
            a = rng.integers(-1, adapters + 1, T)
        elif kind == "runs":
            a = np.sort(rng.integers(0, adapters, T))
        elif kind == "none":
            a = np.where(rng.random(T) < 0.5, -1, 2 ** 31 - 1)
        else:  # one adapter, the last
            a = np.full(T, adapters - 1)
        self.ids = torch.from_numpy(a.astype(np.int64))
        self.adapter = self.ids.to(torch.int32).to(DEV)
        self.scale = torch.from_numpy(rng.uniform(-2, 2, adapters).astype(np.float32)).to(DEV) if scaled else None
        self.values, self.meta = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV)
        self.X, self.dY, self.A, self.B = padded(X), padded(dY), to_dev(A), to_dev(B)
        self.perm = torch.from_numpy(wl.permutation(K, seed + 7).astype(np.int64)) if permuted else None
        self.idx = None if self.perm is None else self.perm.to(torch.int32).to(DEV)
        self.w = host(oracle.decompress(vals, meta, K, n, m))
        self.x, self.dy, self.a, self.b = host(X), host(dY), host(A), host(B)
        self.s = f64(self.scale) if scaled else None

    def forward(self, dtype=BF, **kw):
        return nm.spmm_lora(self.values, self.meta, self.n, self.m, self.K, self.X, self.A, self.B, self.adapter,
                            self.scale, idx=self.idx, out_dtype=dtype, **kw)

    def backward(self, dtype=BF, **kw):
        return nm.spmm_lora_t(self.values, self.meta, self.n, self.m, self.K, self.dY, self.A, self.B, self.adapter,
                              self.scale, idx=self.idx, out_dtype=dtype, **kw)

    def grads(self, dtype=BF, **kw):
        return nm.lora_grad(self.dY, self.X, self.A, self.B, self.adapter, self.scale, out_dtype=dtype, **kw)

    def _per(self, M):
        """|scale_a| |M_a| stacked to rows x (adapters * rank), for products with _low()."""
        s = torch.ones(self.N, dtype=torch.float64) if self.s is None else self.s.abs()
        return (M.abs() * s[:, None, None]).permute(1, 0, 2).reshape(M.shape[1], -1)

    def _low(self, M, z, dtype):
        """Magnitudes of S = M_a z at its tokens (adapters * rank x T) and what may be off in them as operands."""
        serves = (self.ids[None] == torch.arange(self.N)[:, None]).double()[:, None]
        D = z.shape[0]
        mag = ((M.abs().reshape(-1, D) @ z.abs()).view(self.N, self.rank, -1) * serves).reshape(self.N * self.rank, -1)
        val = ((M.reshape(-1, D) @ z).view(self.N, self.rank, -1) * serves).reshape(self.N * self.rank, -1).abs()
        off = (128 * TRUNC + (D / 128 + 16) * ref.U32) * mag
        return val, off + (val + off) * ((2.0 ** -16 if dtype == BF else 2.0 ** -24) + 2 * ref.U32)

    def check(self, got, want, off):
        half = ref.UBF16 if got.dtype == BF else ref.U32
        bound = off + half * (want.abs() + off) + 1e-30
        bad = (f64(got) - want).abs() > bound
        assert not bad.any(), f"{int(bad.sum())} values off by up to {float(((f64(got) - want).abs() / bound).max()):.2f} bounds"
        assert (f64(got) - want).norm() <= (FROB_TOL if got.dtype == BF else 2e-5) * want.norm() + 1e-30

    def check_forward(self, y):
        xp = self.x if self.perm is None else self.x[self.perm]
        want = ref.lora(self.w, xp, self.a, self.b, self.ids, self.s, self.x)
        val, off = self._low(self.a, self.x, y.dtype)
        B = self._per(self.b)
        low = B @ off + (4 * self.rank + 8) * TRUNC * (B @ (val + off))
        base = self.K * TRUNC * (self.w.abs() @ xp.abs())
        self.check(y, want, low + base + 2 * ref.U32 * want.abs())

    def check_backward(self, dx):
        want = ref.lora_grad(self.dy, self.w, self.x, self.a, self.b, self.ids, self.s, self.perm)[0]
        val, off = self._low(self.b.transpose(1, 2), self.dy, dx.dtype)
        A = self._per(self.a.transpose(1, 2))
        low = A @ off + (4 * self.rank + 8) * TRUNC * (A @ (val + off))
        base = self.R * TRUNC * (self.w.T.abs() @ self.dy.abs())
        if self.perm is not None:
            base = torch.empty_like(base).index_copy_(0, self.perm, base)
        self.check(dx, want, low + base + 2 * ref.U32 * want.abs())

    def check_grads(self, dA, dB):
        _, wA, wB = ref.lora_grad(self.dy, self.w, self.x, self.a, self.b, self.ids, self.s, self.perm)
        s = torch.ones(self.N, dtype=torch.float64) if self.s is None else self.s.abs()
        c = 192 * TRUNC + (self.T / 64 + 16) * ref.U32
        for got, want, M, z, other in ((dB, wB, self.a, self.x, self.dy),
                                       (dA, wA, self.b.transpose(1, 2), self.dy, self.x)):
            val, off = self._low(M, z, got.dtype)
            e = (off + c * (val + off)) @ other.abs().T  # adapters * rank x rows
            e = e.view(self.N, self.rank, -1) * s[:, None, None]
            e = e.transpose(1, 2) if got is dB else e
            self.check(got, want, e + 2 * ref.U32 * want.abs())


# (R, K, T, adapters, rank): one token; the skinny (split and whole), one-SM and SM-pair GEMMs; odd ranks and rows that
# start off 16 bytes; ragged row, token and reduction tiles; more adapters than a tile has tokens; the largest rank
SHAPES = [(6, 24, 1, 1, 1), (300, 264, 37, 3, 5), (130, 136, 200, 16, 16), (513, 512, 256, 4, 64), (256, 1024, 16, 16, 16),
          (1000, 384, 64, 70, 8), (70, 100, 65, 5, 33), (520, 256, 1000, 8, 12), (200, 2560, 130, 2, 128),
          (4096, 128, 8, 3, 20)]


@pytest.mark.parametrize("R,K,T,N,rank", SHAPES)
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(R, K, T, N, rank, kind, dtype):
    c = Case(R, K, T, N, rank, kind, permuted=kind == "runs", scaled=kind == "mixed", seed=R + T)
    y = c.forward(dtype)
    torch.cuda.synchronize()
    nm.nm_device_status()
    assert y.dtype == dtype and y.shape == (R, T)
    c.check_forward(y)


@pytest.mark.parametrize("R,K,T,N,rank", SHAPES)
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_input_gradient(R, K, T, N, rank, kind, dtype):
    c = Case(R, K, T, N, rank, kind, permuted=kind == "mixed", scaled=kind == "mixed", seed=R + T + 1)
    dx = c.backward(dtype)
    torch.cuda.synchronize()
    nm.nm_device_status()
    assert dx.dtype == dtype and dx.shape == (K, T)
    c.check_backward(dx)


@pytest.mark.parametrize("R,K,T,N,rank", SHAPES)
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_adapter_gradients(R, K, T, N, rank, kind, dtype):
    c = Case(R, K, T, N, rank, kind, scaled=kind == "runs", seed=R + T + 2)
    dA, dB = c.grads(dtype)
    assert dA.shape == (N, rank, K) and dB.shape == (N, R, rank) and dA.dtype == dB.dtype == dtype
    c.check_grads(dA, dB)


@pytest.mark.parametrize("n,m", [(1, 2), (1, 8), (3, 4)])
@pytest.mark.parametrize("T", [16, 100, 256])
def test_other_patterns(n, m, T):
    c = Case(260, 384, T, 4, 16, n=n, m=m, permuted=True, seed=m + T)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("T", [16, 100, 256])
def test_no_token_has_an_adapter(T):
    """The projection alone: what the plain calls give, up to the order of their sums."""
    c = Case(256, 512, T, 3, 8, "none", permuted=True, seed=T)
    y, dx, (dA, dB) = c.forward(), c.backward(), c.grads()
    c.check_forward(y)
    c.check_backward(dx)
    assert not dA.any() and not dB.any()
    c.N, c.A, c.B, c.scale = 0, c.A[:0], c.B[:0], None
    assert torch.equal(c.forward(F32), nm.spmm(c.values, c.meta, 2, 4, 512, c.X, idx=c.idx, out_dtype=F32))
    assert torch.equal(c.backward(), dx)
    assert c.grads()[0].shape == (0, 8, 512)


def test_one_adapter_has_every_token():
    c = Case(520, 640, 700, 5, 16, "one", seed=3)
    c.check_forward(c.forward())
    dA, dB = c.grads(F32)
    c.check_grads(dA, dB)
    assert not dA[:4].any() and not dB[:4].any()


@pytest.mark.parametrize("T", [16, 100, 256])
def test_requests_do_not_reach_each_other(T):
    """A NaN in one token, or in one adapter's weights, stays in its token, its adapter's tokens and its gradients."""
    c = Case(256, 512, T, 3, 16, "mixed", seed=4)
    c.adapter[:6] = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32)
    y, dx, dA, dB = c.forward(), c.backward(), *c.grads()
    c.X[5, 1] = float("nan")
    c.dY[7, 1] = float("nan")  # token 1 belongs to adapter 1
    y2, dx2, dA2, dB2 = c.forward(), c.backward(), *c.grads()
    keep = torch.arange(T, device=DEV) != 1
    assert y2[:, 1].isnan().any() and dx2[:, 1].isnan().any()
    assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(dx2[:, keep], dx[:, keep])
    assert dA2[1].isnan().any() and torch.equal(dA2[[0, 2]], dA[[0, 2]]) and torch.equal(dB2[[0, 2]], dB[[0, 2]])
    c = Case(256, 512, T, 3, 16, "mixed", seed=4)
    c.adapter[:6] = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32)
    c.A[1, 3, 9] = float("inf")
    c.B[1, 4, 5] = float("nan")
    y2, dx2, dA2, dB2 = c.forward(), c.backward(), *c.grads()
    keep = c.adapter != 1
    assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(dx2[:, keep], dx[:, keep])
    assert y2[4, ~keep].isnan().all() and torch.equal(dA2[[0, 2]], dA[[0, 2]]) and torch.equal(dB2[[0, 2]], dB[[0, 2]])


def test_index_map_entries_outside_leave_the_adapters_part():
    c = Case(130, 256, 40, 2, 8, "runs", permuted=True, seed=5)
    row = c.perm[[3, 77]].clone()
    c.idx[3], c.idx[77] = -1, 256
    dx = c.backward(F32)
    full = torch.zeros((256, 40), dtype=torch.float64)
    keep = torch.ones(256, dtype=torch.bool)
    keep[[3, 77]] = False
    full[c.perm[keep]] = (c.w.T @ c.dy)[keep]
    low = ref.lora_grad(c.dy, torch.zeros_like(c.w), c.x, c.a, c.b, c.ids, c.s)[0]
    assert (f64(dx) - full - low).norm() <= 2e-5 * (full + low).norm()
    assert (f64(dx)[row] - low[row]).norm() <= 2e-5 * low[row].norm()
    xp = c.x[c.perm]
    xp[[3, 77]] = 0
    assert (f64(c.forward(F32)) - ref.lora(c.w, xp, c.a, c.b, c.ids, c.s, c.x)).norm() <= 2e-5 * (c.w @ xp).norm()


def test_unaligned_adapters_and_padding():
    """A and B that start off 16 bytes, and outputs beyond the tokens left alone."""
    c = Case(130, 256, 37, 2, 16, "mixed", seed=6)
    y, dx, dA, dB = c.forward(), c.backward(), *c.grads()
    off = [torch.empty(M.numel() + 1, dtype=BF, device=DEV)[1:].view(M.shape) for M in (c.A, c.B)]
    off[0].copy_(c.A)
    off[1].copy_(c.B)
    c.A, c.B = off
    for a, b in zip((c.forward(), c.backward(), *c.grads()), (y, dx, dA, dB)):
        assert torch.equal(a, b)
    Y = torch.full((130, 56), 5.0, dtype=BF, device=DEV)
    nm.nm_spmm_lora(c.values, c.meta, 2, 4, 130, 256, None, c.X, c.X.stride(0), 37, c.A, c.B, 16, 2, c.scale, c.adapter, Y,
                    56)
    assert torch.equal(Y[:, :37], y) and (Y[:, 37:] == 5).all()
    dX = torch.full((256, 48), 5.0, device=DEV)
    nm.nm_spmm_lora_t(c.values, c.meta, 2, 4, 130, 256, None, c.dY, c.dY.stride(0), 37, c.A, c.B, 16, 2, c.scale,
                      c.adapter, dX, 48, nm.NM_OUT_F32)
    c.check_backward(dX[:, :37])
    assert (dX[:, 37:] == 5).all()


def test_one_gradient_alone():
    c = Case(130, 256, 100, 2, 16, seed=7)
    dA, dB = c.grads()
    for one in (0, 1):
        out = torch.full_like((dA, dB)[one], 5.0)
        args = [None, None]
        args[one] = out
        nm.nm_lora_grad(130, 256, c.dY, c.dY.stride(0), c.X, c.X.stride(0), 100, c.A, c.B, 16, 2, c.scale, c.adapter,
                        *args)
        assert torch.equal(out, (dA, dB)[one])


def test_empty_sizes():
    c = Case(64, 128, 16, 2, 8, seed=8)
    none, no_ids = c.X[:, :0], c.adapter[:0]
    args = (c.values, c.meta, 2, 4, 128)
    assert nm.spmm_lora(*args, none, c.A, c.B, no_ids).shape == (64, 0)
    assert nm.spmm_lora_t(*args, c.dY[:, :0], c.A, c.B, no_ids).shape == (128, 0)
    dA, dB = nm.lora_grad(c.dY[:, :0], none, c.A, c.B, no_ids)
    assert not dA.any() and not dB.any()
    # no rows of W': an empty output, a zero input gradient, adapters' gradients that are zero or empty
    B0, dY0 = c.B[:, :0], c.dY[:0]
    assert nm.spmm_lora(c.values[:0], c.meta[:0], 2, 4, 128, c.X, c.A, B0, c.adapter).shape == (0, 16)
    assert not nm.spmm_lora_t(c.values[:0], c.meta[:0], 2, 4, 128, dY0, c.A, B0, c.adapter).any()
    dA, dB = nm.lora_grad(dY0, c.X, c.A, B0, c.adapter)
    assert not dA.any() and dB.shape == (2, 0, 8)


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    cases = [Case(520, 512, 300, 4, 16, "mixed", permuted=True, seed=9), Case(256, 1024, 16, 8, 16, "mixed", seed=10)]

    def once(stream=None):
        out = []
        for c in cases:
            out += [c.forward(stream=stream), c.backward(stream=stream), *c.grads(F32, stream=stream)]
        return out

    first = once()
    torch.cuda.synchronize()
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
    c = Case(64, 128, 16, 2, 8, seed=11)
    ok = (c.values, c.meta, 2, 4, 128, c.X, c.A, c.B, c.adapter)

    def swap(i, v):
        return ok[:i] + (v,) + ok[i + 1:]

    for args, match in ((swap(6, c.A[:, :4]), "A must be"), (swap(6, c.A.float()), "A must be"), (swap(7, c.B[:1]), "A must"),
                        (swap(8, c.adapter.long()), "adapter"), (swap(8, c.adapter[:15]), "adapter"),
                        (swap(5, c.X[:100]), "rows"), (swap(7, c.B.cpu()), "CUDA")):
        with pytest.raises(ValueError, match=match):
            nm.spmm_lora(*args)
    with pytest.raises(ValueError, match="scale"):
        nm.spmm_lora(*ok, torch.ones(3, device=DEV))
    with pytest.raises(ValueError, match="output type"):
        nm.spmm_lora(*ok, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="dY has"):
        nm.spmm_lora_t(*swap(5, c.dY[:60]))
    with pytest.raises(ValueError, match="tokens"):
        nm.lora_grad(c.dY[:, :8], c.X, c.A, c.B, c.adapter)
    big_a, big_b = torch.zeros((1, 129, 128), dtype=BF, device=DEV), torch.zeros((1, 64, 129), dtype=BF, device=DEV)
    with pytest.raises(nm.NmError) as e:
        nm.spmm_lora(*ok[:6], big_a, big_b, c.adapter)
    assert e.value.status == nm.NM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("rank,dtype", [(20, F32), (40, BF), (100, F32)])
def test_adapter_gradients_of_many_tokens(rank, kind, dtype):
    """A dozen token tiles and more to every CTA of a cluster: several groups of products, ring slots taken again."""
    c = Case(200, 96, 7003, 2, rank, kind, scaled=True, seed=rank)
    c.check_grads(*c.grads(dtype))


@pytest.mark.parametrize("T,permuted", [(1, False), (5, True), (37, False)])
def test_few_tokens_of_a_large_projection(T, permuted):
    """Stages enough for every SM: X goes through rows of 16 or 48 tokens before the skinny GEMM."""
    c = Case(13824, 2816, T, 3, 8, "mixed", permuted=permuted, scaled=True, seed=61)
    for dtype in (BF, F32):
        y = c.forward(dtype)
        torch.cuda.synchronize()
        nm.nm_device_status()
        c.check_forward(y)


@pytest.mark.parametrize("rank,dtype", [(8, BF), (48, F32), (100, BF)])
def test_tiles_of_many_adapters_share_a_ring(rank, dtype):
    """A CTA of the shrink takes dozens of adapters one after the other, each through the ring that held the sums of the last."""
    c = Case(130, 1000, 4500, 40, rank, "mixed", seed=rank)
    c.check_grads(*c.grads(dtype))
    first = c.grads(dtype)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(c.grads(dtype), first))


# More than eight 128-deep stages: the adapters inside the 256 x 256 form of the SM-pair GEMM.  Token counts before, at and
# behind a column tile; up to the eight blocks of 64 rank rows that fit; several tiles to an SM pair; many rows to few tokens
# (column tiles go fastest)
LONG = [(520, 1152, 200, 3, 20), (520, 1152, 256, 8, 64), (300, 2048, 264, 16, 32), (1600, 1152, 264, 4, 16),
        (2600, 1152, 2056, 5, 16), (8000, 1280, 640, 2, 64)]


@pytest.mark.parametrize("R,K,T,N,rank", LONG)
@pytest.mark.parametrize("kind", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_of_a_long_reduction(R, K, T, N, rank, kind, dtype):
    c = Case(R, K, T, N, rank, kind, permuted=kind == "runs", scaled=kind == "mixed", seed=R + T)
    y = c.forward(dtype)
    torch.cuda.synchronize()
    nm.nm_device_status()
    c.check_forward(y)


@pytest.mark.parametrize("T", [200, 264])
def test_requests_do_not_reach_each_other_in_a_long_reduction(T):
    def case():
        c = Case(300, 1152, T, 3, 40, "mixed", seed=44)
        c.adapter[:6] = torch.tensor([0, 1, 2, 0, 1, 2], dtype=torch.int32)
        return c

    c = case()
    y = c.forward()
    c.X[5, 1] = float("nan")  # token 1 belongs to adapter 1
    keep = torch.arange(T, device=DEV) != 1
    y2 = c.forward()
    assert y2[:, 1].isnan().any() and torch.equal(y2[:, keep], y[:, keep])
    c = case()
    c.A[1, 3, 9] = float("inf")
    c.B[1, 4, 5] = float("nan")
    keep = c.adapter != 1
    y2 = c.forward()
    assert torch.equal(y2[:, keep], y[:, keep]) and y2[4, ~keep].isnan().all()
