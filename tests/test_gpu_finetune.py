"""One fine-tuning step through the operators together, as a user strings them:

    layer norm -> pruned projection with adapters -> cross entropy of a pruned head, and every gradient back.

Each forward result is compared with the 64-bit formula at the inputs the kernel got, and every gradient with 64-bit
autograd of the whole chain, evaluated at the activations the kernels produced (their bf16 roundings are constants
there), so that what is left is the rounding of the gradients on their way back.

Tolerances.  Going back, a gradient is rounded to bf16 at G, at the head's dX, at the adapters' dX and at the layer
norm's dX: four times at most 2^-8 of every element.  The maps between are linear with independent random entries
(layer norm's backward only takes two directions out), which on average keep the size of an error relative to the
value's; so 4 * 2^-8 = 1.6e-2 bounds the relative Frobenius error, and the 32-bit sums in between are far below.
"""
import subprocess
import sys
import threading

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
GRAD_TOL = 4 * ref.UBF16


def f64(t):
    return t.detach().to("cpu", torch.float64)


def padded(shape, scale, seed):
    """bf16 on the device, rows padded to 16 bytes."""
    bits = wl.normal_bf16(shape, scale, seed)
    buf = np.zeros((shape[0], -(-shape[1] // 8) * 8), np.uint16)
    buf[:, :shape[1]] = bits
    return to_dev(buf)[:, :shape[1]]


def pruned(R, K, scale, seed):
    """(values, meta, W' in float64, index map, W' Pi's columns in X's order) of a permuted 2:4 matrix."""
    vals, meta = oracle.compress(wl.normal_bf16((R, K), scale, seed), 2, 4)
    w = torch.from_numpy(wl.bf16_to_f32(oracle.decompress(vals, meta, K, 2, 4)).astype(np.float64))
    perm = torch.from_numpy(wl.permutation(K, seed + 1))
    cols = torch.from_numpy(oracle.positions(meta, R, K, 2, 4).astype(np.int64))
    cols += (torch.arange(cols.shape[1]) // 2 * 4)[None, :]
    return to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV), w, perm.to(DEV), perm.long(), cols


class Step:
    def __init__(self, K, R, V, T, N=3, rank=8, seed=0):
        self.K, self.R, self.V, self.T, self.N = K, R, V, T, N
        rng = np.random.Generator(np.random.PCG64(seed))
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
        self.X = padded((K, T), 1.5, seed + 1)
        self.gamma, self.beta = 1 + 0.2 * f(K), 0.2 * f(K)
        self.proj, self.head = pruned(R, K, K ** -0.5, seed + 2), pruned(V, R, R ** -0.5, seed + 4)
        self.A, self.B = (0.1 * f(N, rank, K)).to(BF), (0.3 * f(N, R, rank)).to(BF)
        self.scale = 1 + 0.5 * f(N).abs()
        self.adapter = torch.from_numpy(rng.integers(-1, N, T).astype(np.int32))
        target = rng.integers(0, V, T).astype(np.int32)
        target[1::7] = -100
        self.target = torch.from_numpy(target)
        self.dloss = f(T)
        self.dev = {k: getattr(self, k).to(DEV) for k in
                    ("gamma", "beta", "A", "B", "scale", "adapter", "target", "dloss")}

    def run(self, stream=None):
        d, (pv, pm, _, pi, *_), (hv, hm, _, hi, *_) = self.dev, self.proj, self.head
        Y, mean, rstd = nm.layer_norm(self.X, d["gamma"], d["beta"], stream=stream)
        low = (d["A"], d["B"], d["adapter"], d["scale"])
        H = nm.spmm_lora(pv, pm, 2, 4, self.K, Y, *low, idx=pi, stream=stream)
        loss, lse = nm.spmm_xent(hv, hm, 2, 4, self.R, H, d["target"], idx=hi, stream=stream)
        dH, dhead = nm.spmm_xent_grad(hv, hm, 2, 4, self.R, H, d["target"], lse, d["dloss"], idx=hi, stream=stream)
        dA, dB = nm.lora_grad(dH, Y, *low, out_dtype=F32, stream=stream)
        dY = nm.spmm_lora_t(pv, pm, 2, 4, self.K, dH, *low, idx=pi, stream=stream)
        dX, dgamma, dbeta = nm.layer_norm_grad(dY, self.X, mean, rstd, d["gamma"], stream=stream)
        return dict(Y=Y, H=H, loss=loss, dhead=dhead, dA=dA, dB=dB, dX=dX, dgamma=dgamma, dbeta=dbeta)

    def loss64(self, leaves, got=None):
        """Sum of dloss * loss in 64 bits; with the kernels' results, Y and H take their values, not their gradients."""
        pin = (lambda v, t: v) if got is None else (lambda v, t: v + (f64(t) - v).detach())
        Y = pin(ref.layer_norm(leaves["dX"], leaves["dgamma"], leaves["dbeta"])[0], got and got["Y"])
        w, perm = self.proj[2], self.proj[4]
        H = ref.lora(w, Y[perm], leaves["dA"], leaves["dB"], self.adapter, self.scale.double(), Y)
        self.wants = (Y, H)
        H = pin(H, got and got["H"])
        loss, _ = ref.cross_entropy(leaves["dhead"] @ H[self.head[4]], self.target.long())
        self.wants += (loss,)
        return (loss * self.dloss.double()).sum()

    def leaves(self):
        v = dict(dX=f64(self.X), dgamma=self.gamma.double(), dbeta=self.beta.double(), dA=f64(self.A), dB=f64(self.B),
                 dhead=self.head[2].clone())
        return {k: t.requires_grad_() for k, t in v.items()}


def rel(got, want):
    return (f64(got) - want).norm().item() / max(want.norm().item(), 1e-30)


# (K, R, V, T): one token; a few; a ragged batch; the SM-pair GEMMs; nothing a multiple of anything
SHAPES = [(256, 384, 1000, 1), (256, 384, 1000, 13), (384, 256, 777, 37), (256, 512, 1000, 256), (136, 204, 77, 45)]


@pytest.mark.parametrize("K,R,V,T", SHAPES)
def test_a_step_against_the_whole_derivative(K, R, V, T):
    c = Step(K, R, V, T, seed=T)
    got = c.run()
    nm.nm_device_status()
    leaves = c.leaves()
    names = list(leaves)
    want = dict(zip(names, torch.autograd.grad(c.loss64(leaves, got), [leaves[n] for n in names])))
    Y, H, loss = (w.detach() for w in c.wants)
    assert rel(got["H"], H) <= FROB_TOL
    assert rel(got["Y"], ref.layer_norm(f64(c.X), c.gamma.double(), c.beta.double())[0]) <= ref.UBF16
    assert (f64(got["loss"]) - loss).abs().max() <= 1e-4 * (1 + loss.abs().max())  # 32-bit logits of a few units
    want["dhead"] = want["dhead"].gather(1, c.head[5])
    for n in names:
        assert rel(got[n], want[n]) <= GRAD_TOL, n


@pytest.mark.parametrize("K,R,V,T", SHAPES[2:4])
def test_gradients_against_differences_of_the_loss(K, R, V, T):
    """Along a direction D the loss rises by <gradient, D>: central differences of the 64-bit loss.

    The kernels' activations are rounded to bf16 and the differenced loss's are not: Y and H, 2^-8 each, on top of the
    four roundings of the gradients; the direction is the gradient itself, where an error counts in full."""
    c = Step(K, R, V, T, seed=90 + T)
    got = c.run()
    leaves = {k: v.detach() for k, v in c.leaves().items()}
    for n in ("dX", "dgamma", "dbeta", "dA", "dB"):
        D = f64(got[n])
        D = D / D.norm()
        h = 1e-4
        up, down = (c.loss64({**leaves, n: leaves[n] + s * h * D}).item() for s in (1, -1))
        rise, along = (up - down) / (2 * h), (f64(got[n]) * D).sum().item()
        assert abs(rise - along) <= (GRAD_TOL + 2 * ref.UBF16) * abs(along), n


@pytest.mark.parametrize("T", [13, 256])
def test_a_step_repeats_on_streams_in_graphs_and_from_threads(T):
    c = Step(256, 384, 1000, T, seed=7)
    first = c.run()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in side * 2:
        runs.append(c.run(stream=s.cuda_stream))  # a stream other than torch's current one, by its handle
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            runs.append(c.run())
        graphs.append(g)
    eager = []

    def work(i):
        with torch.cuda.stream(side[i]):
            for _ in range(3):
                graphs[i].replay()
                eager.append(c.run())
            side[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    nm.nm_device_status()
    assert len(eager) == 6
    for got in runs + eager:
        for n, v in got.items():
            assert torch.equal(v, first[n]), n


FIRST_CALL_UNDER_CAPTURE = """
import torch, sparse_gemm_nm_b200 as nm
torch.manual_seed(0)
W = torch.randn(256, 128, device="cuda").bfloat16()
X = torch.randn(128, 24, device="cuda").bfloat16()
A, B = torch.randn(1, 8, 128, device="cuda").bfloat16(), torch.randn(1, 256, 8, device="cuda").bfloat16()
adapter = torch.zeros(24, dtype=torch.int32, device="cuda")
target = torch.arange(24, dtype=torch.int32, device="cuda")
values, meta = nm.prune_compress(W, 2, 4)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def step():
    Y, mean, rstd = nm.layer_norm(X)
    H = nm.spmm_lora(values, meta, 2, 4, 128, Y, A, B, adapter)
    loss, lse = nm.spmm_xent(values, meta, 2, 4, 128, Y, target)
    grads = nm.spmm_xent_grad(values, meta, 2, 4, 128, Y, target, lse, torch.ones_like(loss))
    return (H, loss) + grads + nm.lora_grad(H, Y, A, B, adapter) + nm.layer_norm_grad(grads[0], X, mean, rstd)
with torch.cuda.graph(g):
    captured = step()
g.replay()
torch.cuda.synchronize()
eager = step()
g.replay()
torch.cuda.synchronize()
nm.nm_device_status()
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
print("same")
"""


def test_a_process_may_capture_its_first_step():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_UNDER_CAPTURE], capture_output=True, text=True, timeout=300,
                       cwd=wl.__file__.rsplit("/", 2)[0])
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


@pytest.mark.parametrize("T", [1, 13, 16, 37, 48])
def test_the_loss_waits_for_the_launch_before_it(T):
    """Each call reads what the one before it in the stream writes last, with nothing in between; several K ranges and
    pieces of the vocabulary in the loss, its input copied to wider rows (T = 1, 13, 37) and not."""
    K, V = 2048, 20000
    vals, meta = oracle.compress(wl.normal_bf16((V, K), 0.02, 31), 2, 4)
    head = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV), 2, 4, K
    xs = [padded((K, T), 1.0, 32 + i) for i in range(4)]
    target = torch.arange(T, dtype=torch.int32, device=DEV)
    calm = []
    for x in xs:
        Y = nm.layer_norm(x)[0]
        torch.cuda.synchronize()
        calm.append(nm.spmm_xent(*head, Y, target))
        torch.cuda.synchronize()
    out = padded((K, T), 1.0, 40)  # every layer norm writes here, and every loss reads it
    ld = out.stride(0)
    hurried = []
    for x in xs * 3:
        nm.nm_layer_norm(x, x.stride(0), nm.NM_OUT_BF16, K, T, None, None, 1e-5, out, ld, nm.NM_OUT_BF16, None, None)
        hurried.append(nm.spmm_xent(*head, out, target))
    torch.cuda.synchronize()
    nm.nm_device_status()
    for i, got in enumerate(hurried):
        assert all(torch.equal(a, b) for a, b in zip(got, calm[i % 4]))


@pytest.mark.parametrize("R,K,T", [(130, 256, 200), (70, 72, 37), (300, 128, 24)])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_weights_that_start_on_any_element(R, K, T, off):
    """Views of a larger buffer as the 2:4 values: every call gives what aligned values give, up to the order of sums."""
    g = torch.Generator().manual_seed(R + off)
    vals, meta = oracle.compress(wl.normal_bf16((R, K), 0.05, 71), 2, 4)
    aligned, meta = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV)
    buf = torch.zeros(aligned.numel() + off, dtype=torch.bfloat16, device=DEV)
    values = buf[off:].view(aligned.shape)
    values.copy_(aligned)
    X, dY = (torch.zeros((r, -(-T // 8) * 8), dtype=torch.bfloat16, device=DEV)[:, :T] for r in (K, R))
    X.copy_(torch.randn((K, T), generator=g))
    dY.copy_(torch.randn((R, T), generator=g))
    A, B = (torch.randn(s, generator=g).to(DEV, torch.bfloat16) for s in ((2, 4, K), (2, R, 4)))
    ids = torch.randint(0, 2, (T,), generator=g, dtype=torch.int32).to(DEV)
    target = torch.randint(0, R, (T,), generator=g, dtype=torch.int32).to(DEV)
    dloss = torch.rand(T, generator=g).to(DEV)

    def calls(v):
        loss, lse = nm.spmm_xent(v, meta, 2, 4, K, X, target)
        return (loss, lse, *nm.spmm_xent_grad(v, meta, 2, 4, K, X, target, lse, dloss),
                nm.spmm_lora(v, meta, 2, 4, K, X, A, B, ids), nm.spmm_lora_t(v, meta, 2, 4, K, dY, A, B, ids),
                nm.spmm_t(v, meta, 2, 4, K, dY), nm.decompress(v, meta, K, 2, 4))

    for got, want in zip(calls(values), calls(aligned)):
        # float32 sums in another order; each side rounds its result to bf16 once, and G before it
        assert (got.double() - want.double()).norm() <= GRAD_TOL * want.double().norm()
    nm.nm_device_status()
