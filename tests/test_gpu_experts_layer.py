"""A layer of pruned experts as it is used: router, gather, two grouped products with an activation between them, combine;
then all gradients, and their clipping.  Against autograd of the same layer in 64 bits.

Tolerance: between the 64-bit layer and this one lie at most eight roundings to bf16 on the way to any gradient (the gathered
output of each product, the activation, the combine, and the same backwards), each 2^-9 of a value's size on average and 2^-8
at most: 8 x 2^-8 = 3e-2 of the norm.
"""
import threading

import pytest
import torch

import sparse_gemm_nm_b200 as nm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


class Layer:
    def __init__(self, E, D, H, k, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.E, self.D, self.H, self.k = E, D, H, k
        self.up, self.up_meta, self.up_dense = self.weights(E, H, D, g)
        self.down, self.down_meta, self.down_dense = self.weights(E, D, H, g)
        self.g = g

    @staticmethod
    def weights(E, R, K, g):
        W = (torch.randn((E, R, K), generator=g, device=DEV) * (2 / K) ** 0.5).to(BF)
        parts = [nm.prune_compress(W[e], 2, 4) for e in range(E)]
        v, m = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        return v, m, torch.stack([nm.decompress(v[e], m[e], K, 2, 4) for e in range(E)])

    def inputs(self, T):
        def rows(r):
            return torch.randn((r, (T + 7) // 8 * 8), generator=self.g, device=DEV).to(BF)[:, :T]
        logits = rows(self.E)
        if T > 2:
            logits[:, 1] = -torch.inf  # a token of padding
            logits[1:, 2] = -torch.inf  # one that may use a single expert
        return rows(self.D), logits, rows(self.D)

    def step(self, X, logits, dY, renorm=True, stream=None):
        """(Y, dX, dlogits, dup, ddown)."""
        E, D, H, s = self.E, self.D, self.H, dict(stream=stream)
        expert, gate, slot, source, off = nm.experts_route(logits, self.k, renorm=renorm, **s)
        xg = nm.experts_gather(X, source, **s)
        h = nm.experts_spmm(self.up, self.up_meta, 2, 4, D, xg, off, **s)
        with torch.cuda.stream(stream):
            a = h.relu_()  # in place: rows stay on 16 bytes
        yg = nm.experts_spmm(self.down, self.down_meta, 2, 4, H, a, off, **s)
        Y = nm.experts_combine(yg, slot, gate, **s)
        dyg, dgate = nm.experts_combine_grad(dY, yg, slot, source, gate, **s)
        da = nm.experts_spmm_t(self.down, self.down_meta, 2, 4, H, dyg, off, **s)
        ddown = nm.experts_sddmm(self.down_meta, 2, 4, D, H, dyg, a, off, **s)
        with torch.cuda.stream(stream):
            dh = da.mul_(a > 0)
        dxg = nm.experts_spmm_t(self.up, self.up_meta, 2, 4, D, dh, off, **s)
        dup = nm.experts_sddmm(self.up_meta, 2, 4, H, D, dh, xg, off, **s)
        dX = nm.experts_combine(dxg, slot, **s)
        dlogits = nm.experts_route_grad(logits, expert, gate, dgate, renorm=renorm, **s)
        return Y, dX, dlogits, dup, ddown

    def exact(self, X, logits, dY, renorm=True):
        E, k, T = self.E, self.k, X.shape[1]
        x, l = X.double().requires_grad_(), logits.double().requires_grad_()
        up, down = self.up_dense.double().requires_grad_(), self.down_dense.double().requires_grad_()
        live = (l > -torch.inf).any(0)
        safe = torch.where(live, l, 0.0)
        top = safe.topk(k, dim=0)
        chosen = torch.zeros_like(safe, dtype=torch.bool).scatter_(0, top.indices, True) & live & (l > -torch.inf)
        p = torch.softmax(torch.where(chosen, safe, -1e300) if renorm else torch.where(l > -torch.inf, safe, -1e300), 0) * chosen
        y = sum(p[e] * (down[e] @ torch.relu(up[e] @ x)) for e in range(E))
        dx, dl, du, dd = torch.autograd.grad(y, (x, l, up, down), dY.double())
        keep = [torch.stack([nm.decompress(torch.ones_like(v[e]), m[e], K, 2, 4) for e in range(E)]) != 0
                for v, m, K in ((self.up, self.up_meta, self.D), (self.down, self.down_meta, self.H))]
        return y.detach(), dx, dl, du[keep[0]].view(self.up.shape), dd[keep[1]].view(self.down.shape)


def near(got, want, name):
    assert (got.double() - want).norm() <= 3e-2 * want.norm() + 1e-30, name
    assert got.isfinite().all(), name


@pytest.mark.parametrize("E,D,H,k,T", [(8, 256, 512, 2, 600), (4, 144, 320, 1, 5), (16, 128, 64, 4, 333), (6, 512, 400, 3, 1),
                                       (3, 64, 1024, 2, 4100)])
@pytest.mark.parametrize("renorm", [True, False])
def test_layer_and_its_gradients(E, D, H, k, T, renorm):
    layer = Layer(E, D, H, k, E + T)
    X, logits, dY = layer.inputs(T)
    got, want = layer.step(X, logits, dY, renorm), layer.exact(X, logits, dY, renorm)
    nm.nm_device_status()
    for g, w, name in zip(got, want, ("Y", "dX", "dlogits", "dup", "ddown")):
        near(g, w, name)
    grads = [got[3], got[4], torch.randn(D, device=DEV)]
    want_norm = sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5
    norm = nm.clip_grads(grads, want_norm / 2)
    assert abs(float(norm) - want_norm) <= 1e-6 * want_norm
    assert abs(sum(float((t.double() ** 2).sum()) for t in grads) ** 0.5 - want_norm / 2) <= 4e-3 * want_norm


def test_one_token_at_a_time_equals_the_batch():
    """Serving: a decoding step of single tokens gives each what the batch gives it, to the sums' order."""
    layer = Layer(8, 512, 768, 2, 3)
    X, logits, dY = layer.inputs(12)
    Y = layer.step(X, logits, dY)[0]
    for t in range(12):
        one = [torch.zeros((m.shape[0], 8), dtype=BF, device=DEV)[:, :1].copy_(m[:, t:t + 1]) for m in (X, dY)]
        y = layer.step(one[0], logits[:, t:t + 1].contiguous(), one[1])[0]
        assert (y[:, 0].double() - Y[:, t].double()).abs().max() <= 2.0 ** -6 * Y[:, t].double().abs().max() + 1e-30


def test_captured_step_on_new_tokens():
    layer = Layer(8, 256, 320, 2, 4)
    X, logits, dY = layer.inputs(200)
    layer.step(X, logits, dY)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(X, logits, dY)
    for _ in range(3):
        for t in (X, logits, dY):
            t.normal_()
        graph.replay()
        for a, b in zip(out, layer.step(X, logits, dY)):
            assert torch.equal(a, b)


def test_two_graphs_and_eager_calls_in_turn():
    """Two captured steps and eager ones share the staging pool and nothing else."""
    layer = Layer(4, 128, 256, 2, 5)
    sets = [layer.inputs(T) for T in (70, 301)]
    want = [layer.step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.step(*s)
        graphs.append((g, out))
    for _ in range(4):
        for (g, out), w, s in zip(graphs, want, sets):
            g.replay()
            for a, b, c in zip(out, w, layer.step(*s)):
                assert torch.equal(a, b) and torch.equal(c, b)


def test_streams_and_threads():
    """The same steps from three threads on streams of their own."""
    layer = Layer(8, 256, 384, 2, 6)
    sets = [layer.inputs(T) for T in (64, 500, 9)]
    want = [layer.step(*s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(10):
            got = layer.step(*sets[i], stream=s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    nm.nm_device_status()
