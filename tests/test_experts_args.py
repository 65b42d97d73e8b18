"""What the calls of a layer of experts and the clipping refuse on the host, before any launch."""
import ctypes

import pytest
import torch

import sparse_gemm_nm_b200 as nm

I, U, A16, OK = nm.NM_ERR_INVALID_ARG, nm.NM_ERR_UNSUPPORTED, nm.NM_ERR_MISALIGNED, nm.NM_OK


@pytest.fixture(scope="module")
def L():
    return nm.lib()


def test_products(L):
    def fwd(fn="nm_experts_spmm", n=2, m=4, E=2, R=8, K=32, X=16, ldx=8, S=8, off=16, Y=16, ldy=8, yt=0, values=16, meta=16):
        return getattr(L, fn)(values, meta, n, m, E, R, K, X, ldx, S, off, Y, ldy, yt, None)

    def grad(n=2, m=4, E=2, R=8, K=32, dY=16, lddy=8, X=16, ldx=8, S=8, off=16, dV=16, dt=0, meta=16):
        return L.nm_experts_sddmm(meta, n, m, E, R, K, dY, lddy, X, ldx, S, off, dV, dt, None)

    for fn in ("nm_experts_spmm", "nm_experts_spmm_t"):
        for bad in (dict(E=-1), dict(R=-1), dict(K=-1), dict(K=0), dict(S=-1), dict(n=4), dict(m=5), dict(K=30), dict(yt=2),
                    dict(off=None), dict(values=None), dict(meta=None), dict(X=None), dict(Y=None), dict(ldx=7), dict(ldy=7)):
            assert fwd(fn, **bad) == I, (fn, bad)
        for bad in (dict(n=1), dict(n=1, m=2), dict(K=24), dict(E=1025), dict(R=1 << 31), dict(S=1 << 31), dict(K=1 << 31)):
            assert fwd(fn, **bad) == U, (fn, bad)
        for bad in (dict(X=8), dict(Y=2), dict(ldx=12), dict(ldy=9), dict(off=18), dict(values=18), dict(meta=20), dict(yt=1, ldy=9)):
            assert fwd(fn, **bad) == A16, (fn, bad)
        assert fwd(fn, E=0) == fwd(fn, S=0) == OK
    assert fwd(R=0) == OK and fwd("nm_experts_spmm_t", R=0) == I
    for bad in (dict(E=-1), dict(R=-1), dict(K=0), dict(K=30), dict(S=-1), dict(n=4), dict(dt=2), dict(off=None), dict(dV=None),
                dict(meta=None), dict(X=None), dict(dY=None), dict(ldx=7), dict(lddy=7)):
        assert grad(**bad) == I, bad
    for bad in (dict(n=1), dict(K=24), dict(E=1025), dict(E=1024, R=1 << 26, K=1 << 20)):
        assert grad(**bad) == U, bad
    for bad in (dict(dV=24), dict(meta=18), dict(off=17), dict(X=8), dict(dY=8), dict(ldx=12), dict(lddy=12)):
        assert grad(**bad) == A16, bad
    assert grad(E=0) == grad(R=0) == OK


def test_router(L):
    def fwd(l=16, ld=8, t=0, E=4, T=8, k=2, expert=16, gate=16, slot=16, source=16, off=16):
        return L.nm_experts_route(l, ld, t, E, T, k, 1, expert, gate, slot, source, off, None)

    def grad(l=16, ld=8, t=0, E=4, T=8, k=2, expert=16, gate=16, dgate=16, dl=16, ldd=8):
        return L.nm_experts_route_grad(l, ld, t, E, T, k, 0, expert, gate, dgate, dl, ldd, None)

    for f in (fwd, grad):
        for bad in (dict(E=0), dict(E=-1), dict(T=-1), dict(k=0), dict(k=5), dict(t=3), dict(l=None), dict(ld=7),
                    dict(expert=None), dict(gate=None)):
            assert f(**bad) == I, bad
        for bad in (dict(E=1025), dict(E=40, k=17), dict(T=1 << 30)):
            assert f(**bad) == U, bad
        for bad in (dict(l=17), dict(t=1, l=18), dict(expert=18), dict(gate=17)):
            assert f(**bad) == A16, bad
    for bad in (dict(slot=None), dict(source=None), dict(off=None)):
        assert fwd(**bad) == I, bad
    for bad in (dict(slot=18), dict(source=18), dict(off=18)):
        assert fwd(**bad) == A16, bad
    assert grad(dgate=None) == grad(dl=None) == grad(ldd=7) == I
    assert grad(dgate=18) == grad(dl=17) == A16
    assert grad(T=0) == OK


def test_moves(L):
    def gather(X=16, ldx=8, K=4, T=8, source=16, S=16, Xg=16, ldg=16):
        return L.nm_experts_gather(X, ldx, K, T, source, S, Xg, ldg, None)

    def combine(Yg=16, ldg=16, S=16, R=4, T=8, k=2, slot=16, gate=16, Y=16, ldy=8, yt=0):
        return L.nm_experts_combine(Yg, ldg, S, R, T, k, slot, gate, Y, ldy, yt, None)

    def grad(dY=16, lddy=8, R=4, T=8, k=2, Yg=16, ldg=16, S=16, slot=16, source=16, gate=16, dYg=16, lddg=16, dgate=16):
        return L.nm_experts_combine_grad(dY, lddy, R, T, k, Yg, ldg, S, slot, source, gate, dYg, lddg, dgate, None)

    for bad in (dict(K=-1), dict(T=-1), dict(S=-1), dict(T=0), dict(source=None), dict(X=None), dict(Xg=None), dict(ldx=7),
                dict(ldg=15)):
        assert gather(**bad) == I, bad
    assert gather(X=8) == gather(ldg=20) == gather(source=18) == A16
    assert gather(K=0) == gather(S=0) == OK and gather(T=1 << 31) == U
    for bad in (dict(R=-1), dict(T=-1), dict(S=-1), dict(k=0), dict(slot=None), dict(Yg=None), dict(Y=None), dict(ldy=7),
                dict(ldg=15), dict(yt=2)):
        assert combine(**bad) == I, bad
    assert combine(Yg=8) == combine(ldy=12) == combine(slot=18) == combine(gate=18) == A16
    assert combine(R=0) == combine(T=0) == OK and combine(T=1 << 30) == U
    for bad in (dict(R=-1), dict(T=-1), dict(S=-1), dict(k=0), dict(slot=None), dict(source=None), dict(dgate=None),
                dict(dY=None), dict(Yg=None), dict(dYg=None), dict(lddy=7), dict(ldg=15), dict(lddg=15), dict(T=0)):
        assert grad(**bad) == I, bad
    for bad in (dict(dY=8), dict(Yg=8), dict(dYg=8), dict(lddy=12), dict(slot=18), dict(source=18), dict(gate=18), dict(dgate=18)):
        assert grad(**bad) == A16, bad
    assert grad(T=0, S=0) == OK


def test_clipping(L):
    def clip(grads=(16, 32), outs=(16, 32), sizes=(3, 4), types=(0, 1), max_norm=1.0, norm=16, count=None):
        n = len(grads)
        P = ctypes.c_void_p * n
        return L.nm_clip_grads(P(*grads), None if outs is None else P(*outs), (ctypes.c_int64 * n)(*sizes),
                               (ctypes.c_int * n)(*types), n if count is None else count, max_norm, norm, None)

    for bad in (dict(count=-1), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(types=(0, 2)),
                dict(sizes=(-1, 4)), dict(grads=(None, 32)), dict(outs=(16, None))):
        assert clip(**bad) == I, bad
    for bad in (dict(norm=18), dict(grads=(17, 32)), dict(grads=(16, 34)), dict(outs=(16, 33))):
        assert clip(**bad) == A16, bad
    assert L.nm_clip_grads(None, None, None, None, 2, 1.0, 16, None) == I


def test_clipping_refuses_outputs_that_overlap(L):
    def clip(grads, outs, sizes, types):
        n = len(grads)
        P = ctypes.c_void_p * n
        return L.nm_clip_grads(P(*grads), P(*outs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*types), n, 1.0, 16, None)

    f32, bf = nm.NM_OUT_F32, nm.NM_OUT_BF16
    for bad in (((64, 64), (64, 64), (4, 4), (f32, f32)),  # one gradient twice
                ((64, 128), (256, 256), (4, 4), (f32, f32)),  # into one place
                ((64, 76), (64, 76), (4, 4), (f32, f32)),  # the second starts in the first
                ((76, 64), (76, 64), (4, 4), (f32, f32)),
                ((64, 128), (128, 64), (1, 1), (bf, bf)),  # exchanged
                ((64, 128), (70, 256), (4, 4), (bf, bf)),  # an output inside its own gradient
                ((0x100000, 0x2000), (0x100000, 0x110000 - 2), (0x10000 // 4, 8), (f32, bf))):
        assert clip(*bad) == I and b"overlap" in L.nm_last_error(), bad
    if not torch.cuda.is_available():  # side by side, or of no elements: no refusal before the device is asked for
        for good in (((80, 64), (80, 64), (4, 4), (f32, f32)), ((64, 64), (128, 256), (4, 4), (f32, f32)),
                     ((64, 64), (64, 64), (4, 0), (f32, f32)), ((64, 72), (128, 136), (4, 4), (bf, bf))):
            assert clip(*good) not in (I, A16, U, OK), good


def test_wrappers_refuse():
    bf, i32 = torch.bfloat16, torch.int32
    X, off = torch.zeros((16, 8), dtype=bf), torch.zeros(3, dtype=i32)
    values, meta = torch.zeros((2, 8, 8), dtype=bf), torch.zeros(2 * nm.nm_meta_words(8, 16, 2, 4), dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        nm.experts_spmm(values, meta, 2, 4, 16, X, off)
    with pytest.raises(ValueError, match="CUDA"):
        nm.experts_route(X, 2)
    with pytest.raises(ValueError, match="CUDA"):
        nm.clip_grads([X], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        nm.clip_grads([], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        nm.clip_grads([X.T], 1.0)
    with pytest.raises(ValueError, match="sizes"):
        nm.clip_grads([X], 1.0, out=[X[:8]])
    for v, m, o, what in ((values[0], meta, off, "three dimensions"), (values[:, :, :4], meta, off, "contiguous"),
                          (values, meta[:-1], off, "meta"), (values, meta, off[:2], "offsets"), (values, meta, off.long(), "offsets")):
        with pytest.raises(ValueError, match=what):
            nm._experts(v, m, 2, 4, 16, o)
    with pytest.raises(nm.NmError):
        nm._experts(values, meta, 2, 4, 15, off)
    with pytest.raises(ValueError, match="gate"):
        nm._pairs(2, 8, (torch.zeros((2, 7)), "gate", torch.float32))
