"""The operators around a projection from several host threads, each on a stream of its own, many calls deep.

Every call has to give bit for bit what it gave alone, and every stream has to come to its end: the launches of the
streams share the SMs, so that waits inside the kernels take their slow paths.  Ragged strips and tiles, clusters of
every size, one and several pieces of a vocabulary, adapters in both GEMMs.
"""
import random
import threading
import time

import pytest
import torch

import sparse_gemm_nm_b200 as nm
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rows(g, r, c, dtype=BF):
    per = 4 if dtype == F32 else 8
    return torch.randn((r, -(-c // per) * per), generator=g, device=DEV).to(dtype)[:, :c]


def norm(g, K, T, dtype):
    x, dy = rows(g, K, T, dtype), rows(g, K, T)
    gamma = torch.randn(K, generator=g, device=DEV)

    def call():
        y, mean, rstd = nm.layer_norm(x, gamma, gamma, out_dtype=BF)
        return (y, mean, rstd, *nm.layer_norm_grad(dy, x, mean, rstd, gamma))
    return call


def weights(g, R, K):
    return nm.prune_compress((torch.randn((R, K), generator=g, device=DEV) * 0.05).to(BF), 2, 4)


def adapters(g, R, K, T, n, rank):
    values, meta = weights(g, R, K)
    X, dY = rows(g, K, T), rows(g, R, T)
    A, B = (torch.randn(s, generator=g, device=DEV).to(BF) for s in ((n, rank, K), (n, R, rank)))
    ids = torch.randint(-1, n, (T,), generator=g, device=DEV, dtype=torch.int32)
    idx = torch.randperm(K, generator=g, device=DEV).int()

    def call():
        return (nm.spmm_lora(values, meta, 2, 4, K, X, A, B, ids, idx=idx),
                nm.spmm_lora_t(values, meta, 2, 4, K, dY, A, B, ids, idx=idx), *nm.lora_grad(dY, X, A, B, ids, out_dtype=F32))
    return call


def entropy(g, R, K, T):
    values, meta = weights(g, R, K)
    X = rows(g, K, T)
    target = torch.randint(0, R, (T,), generator=g, device=DEV, dtype=torch.int32)
    dloss = torch.rand(T, generator=g, device=DEV)

    def call():
        loss, lse = nm.spmm_xent(values, meta, 2, 4, K, X, target)
        return (loss, lse, *nm.spmm_xent_grad(values, meta, 2, 4, K, X, target, lse, dloss))
    return call


def projection(g, R, K, T):
    """The library's other calls on one shape: forward, permuted, one-call, hybrid, both gradients, and the other formats."""
    W = (torch.randn((R, K), generator=g, device=DEV) * 0.05).to(BF)
    values, meta = nm.prune_compress(W, 2, 4)
    v18, m18 = nm.prune_compress(W, 1, 8)
    X, dY = rows(g, K, T), rows(g, R, T)
    idx = torch.randperm(K, generator=g, device=DEV).int()
    tiles = torch.randint(0, 2, (-(-R // 128), -(-K // 128)), generator=g, device=DEV, dtype=torch.uint8)
    W8 = torch.randint(-9, 10, (R, K), generator=g, device=DEV, dtype=torch.int8)
    X8 = torch.randint(-9, 10, (K, -(-T // 16) * 16), generator=g, device=DEV, dtype=torch.int8)
    v8, m8 = nm.prune_compress_i8(W8)
    vf, mf = nm.prune_compress_tf32(W.float())
    Xf = rows(g, K, T, F32)

    def call():
        return (nm.spmm(values, meta, 2, 4, K, X), nm.spmm(values, meta, 2, 4, K, X, idx=idx, out_dtype=F32),
                nm.spmm(v18, m18, 1, 8, K, X), nm.prune_spmm(W, 2, 4, X), nm.hybrid_spmm(W, values, meta, tiles, X),
                nm.spmm_t(values, meta, 2, 4, K, dY), nm.sddmm(meta, 2, 4, R, K, dY, X), nm.spmm_i8(v8, m8, K, X8),
                nm.spmm_tf32(vf, mf, K, Xf), nm.decompress(values, meta, K, 2, 4))
    return call


def run_together(calls, seconds=10):
    alone = []
    for call in calls:
        alone.append(call())
        torch.cuda.synchronize()
    wrong, ended = [], [0] * 3
    start = time.monotonic()

    def work(k):
        pick, stream = random.Random(k), torch.cuda.Stream()
        with torch.cuda.stream(stream):
            while time.monotonic() - start < seconds:
                got = [(i, calls[i]()) for i in (pick.randrange(len(calls)) for _ in range(pick.randint(3, 15)))]
                done = torch.cuda.Event()
                done.record()
                until = time.monotonic() + 20
                while not done.query():  # no synchronisation, which a stuck stream would not come back from
                    if time.monotonic() > until:
                        wrong.append(f"thread {k}: its stream does not come to an end")
                        return
                    time.sleep(0.0005)
                for i, out in got:
                    if not all(torch.equal(a, b) for a, b in zip(out, alone[i])):
                        wrong.append(f"thread {k}: call {i} differs")
                        return
                ended[k] += len(got)

    threads = [threading.Thread(target=work, args=(k,), daemon=True) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong, wrong
    assert all(ended)
    nm.nm_device_status()


def test_threads_on_streams_of_their_own():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    calls = [norm(g, 1893, 97, F32), norm(g, 23, 3528, F32), norm(g, 10, 15, F32), norm(g, 768, 5001, BF),
             norm(g, 5120, 13, BF), adapters(g, 309, 5888, 1006, 3, 49), adapters(g, 267, 512, 2308, 13, 8),
             adapters(g, 330, 1152, 4096, 6, 12), adapters(g, 2602, 5096, 53, 3, 1), adapters(g, 24, 72, 6, 2, 8),
             adapters(g, 2000, 1024, 16, 8, 16), entropy(g, 9492, 88, 4099), entropy(g, 3, 152, 8192), entropy(g, 94, 240, 1),
             entropy(g, 183, 2280, 618), entropy(g, 803, 128, 3), entropy(g, 3000, 768, 200), entropy(g, 2000, 512, 1000)]
    run_together(calls)


def test_threads_on_streams_of_their_own_through_the_other_calls():
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    run_together([projection(g, 1000, 512, 264), projection(g, 300, 1152, 1000), projection(g, 520, 256, 24),
                  projection(g, 260, 144, 200), norm(g, 768, 1001, BF), entropy(g, 9492, 88, 4099)])
