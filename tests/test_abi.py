"""The C-ABI library loads on a CPU-only machine and exports what include/nm.h declares.

No call here reaches a device: only the size helpers and argument checks that
the library answers on the host before any CUDA call.
"""
import ctypes
import os
import re

import pytest

import sparse_gemm_nm_b200 as nm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def declared_functions():
    src = open(os.path.join(ROOT, "include", "nm.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = re.findall(r"^\s*NM_API\s+[^(]*?\b(nm_[a-z0-9_]+)\s*\(", src, flags=re.M)
    return sorted(set(names))


@pytest.fixture(scope="module")
def lib():
    from sparse_gemm_nm_b200 import build
    build.build()
    return nm.lib()


def test_header_declares_the_five_calls():
    names = declared_functions()
    for call in ["nm_prune_compress", "nm_decompress", "nm_spmm", "nm_spmm_permuted", "nm_hybrid_spmm"]:
        assert call in names


def test_every_declared_symbol_is_exported(lib):
    for name in declared_functions():
        assert hasattr(lib, name), name
        assert name in nm.SIGNATURES, f"binding lacks a signature for {name}"


def test_size_helpers_match_oracle(lib):
    import oracle
    for R, K, n, m in [(4096, 11008, 2, 4), (13824, 5120, 2, 4), (6, 24, 2, 4), (3072, 768, 1, 8),
                       (256, 24, 1, 4), (33, 96, 3, 4), (5, 48, 5, 8)]:
        assert nm.nm_meta_words(R, K, n, m) == oracle.meta_words(R, K, n, m)
        assert nm.nm_value_cols(K, n, m) == oracle.value_cols(K, n, m)


def test_size_helpers(lib):
    assert nm.nm_index_bits(4) == 2 and nm.nm_index_bits(8) == 3 and nm.nm_index_bits(2) == 1
    assert nm.nm_index_bits(3) == 0
    assert nm.nm_value_cols(4096, 2, 4) == 2048
    assert nm.nm_meta_words(4096, 4096, 2, 4) == 4096 * 4096 // 32   # tiled 2:4
    assert nm.nm_meta_words(16, 24, 2, 4) == 64                      # one padded block
    assert nm.nm_meta_words(17, 128, 2, 4) == 128
    assert nm.nm_meta_words(3, 768, 1, 8) == 30                      # row-wise, 10 words a row
    assert nm.nm_meta_words(4, 10, 2, 4) == -1     # K % M != 0
    assert nm.nm_value_cols(16, 4, 4) == -1        # N must be below M


def test_host_argument_checks(lib):
    L = lib
    # bad pattern, K % M, negative sizes and null pointers are refused before any launch
    assert L.nm_prune_compress(None, 4, 16, 16, 5, 4, None, None, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_prune_compress(None, 4, 18, 18, 2, 4, None, None, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_prune_compress(None, 4, 16, 8, 2, 4, None, None, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_prune_compress(None, -1, 16, 16, 2, 4, None, None, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_prune_compress(None, 4, 16, 16, 2, 4, None, None, None) == nm.NM_ERR_INVALID_ARG
    assert b"null" in L.nm_last_error()
    assert L.nm_decompress(None, None, 4, 16, 1, 3, None, 16, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_spmm(None, None, 2, 4, 8, 30, None, 8, 8, None, 8, 0, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_spmm(None, None, 2, 4, 8, 32, None, 8, 8, None, 4, 0, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_spmm(None, None, 2, 4, 8, 32, None, 8, 8, None, 8, 7, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_spmm_permuted(None, None, 2, 4, 8, 32, None, None, 8, 8, None, 8, 0, None) == nm.NM_ERR_INVALID_ARG
    # empty outputs are a no-op that never touches the device
    assert L.nm_spmm(None, None, 2, 4, 0, 32, None, 8, 8, None, 8, 0, None) == nm.NM_OK
    assert L.nm_spmm(None, None, 2, 4, 8, 32, None, 8, 0, None, 8, 0, None) == nm.NM_OK
    assert L.nm_prune_compress(None, 0, 16, 16, 2, 4, None, None, None) == nm.NM_OK


def test_status_strings(lib):
    for s in range(7):
        assert nm.lib().nm_status_string(s)
    assert nm.nm_version() >= 100


def test_product_package_does_not_touch_the_oracle():
    """The product path never imports, links or loads the oracle."""
    pkg = os.path.join(ROOT, "sparse_gemm_nm_b200")
    for dirpath, _, files in os.walk(pkg):
        for f in files:
            if f.endswith((".py", ".cu", ".cuh", ".h", ".cpp")):
                text = open(os.path.join(dirpath, f)).read()
                assert "oracle" not in text.replace("oracle as the", ""), f


def test_host_argument_checks_of_the_format_calls(lib):
    """The TF32, INT8 and diagonal calls refuse bad shapes, leading dimensions and nulls before any launch."""
    L = lib
    I = nm.NM_ERR_INVALID_ARG
    assert L.nm_prune_compress_tf32(None, 4, 5, 6, None, None, None) == I          # odd K (1:2)
    assert L.nm_prune_compress_tf32(None, 4, 8, 6, None, None, None) == I          # ldw < K
    assert L.nm_prune_compress_tf32(None, 4, 8, 8, None, None, None) == I          # null pointers
    assert L.nm_prune_compress_tf32(None, 0, 8, 8, None, None, None) == nm.NM_OK   # empty
    assert L.nm_decompress_tf32(None, None, 4, 7, None, 8, None) == I
    assert L.nm_spmm_tf32(None, None, 4, 8, None, 8, 8, None, 8, 7, None) == I     # bad output dtype
    assert L.nm_spmm_tf32(None, None, 4, 8, None, 8, 8, None, 4, 0, None) == I     # ldy < T
    assert L.nm_spmm_tf32(None, None, 4, 8, None, 8, 8, None, 8, 0, None) == I     # Y null
    assert L.nm_spmm_tf32(None, None, 0, 8, None, 8, 8, None, 8, 0, None) == nm.NM_OK
    assert L.nm_diag_prune_compress(None, 4, 8, 8, 9, None, None, None) == I       # D > K
    assert L.nm_diag_prune_compress(None, 4, 8, 6, 2, None, None, None) == I       # ldw < K
    assert L.nm_diag_expand(None, None, 9, 4, 8, None, 8, None) == I               # D > K
    assert L.nm_diag_spmm(None, None, 9, 4, 8, None, None, 8, 8, None, 8, 0, None) == I
    assert L.nm_diag_spmm(None, None, 2, 4, 8, None, None, 8, 8, None, 4, 0, None) == I  # ldy < T
    assert L.nm_prune_compress_i8(None, 4, 16, 8, None, None, None) == I           # ldw < K
    assert L.nm_spmm_i8(None, None, 4, 16, None, 16, 16, None, 8, None) == I       # ldy < T


def test_host_argument_checks_of_layer_norm(lib):
    """Refused before any launch: sizes, types, eps, nulls, strides and alignment."""
    L, I = lib, nm.NM_ERR_INVALID_ARG

    def fwd(X=16, ldx=8, xt=0, K=4, T=8, eps=1e-5, Y=16, ldy=8, yt=0):
        return L.nm_layer_norm(X, ldx, xt, K, T, None, None, eps, Y, ldy, yt, None, None, None)

    def bwd(dY=16, lddy=8, dt=0, X=16, ldx=8, xt=0, K=4, T=8, mean=16, rstd=16, dX=16, lddx=8):
        return L.nm_layer_norm_grad(dY, lddy, dt, X, ldx, xt, K, T, None, mean, rstd, dX, lddx, None, None, None)

    for bad in (dict(K=-1), dict(T=-1), dict(K=0), dict(xt=2), dict(yt=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(X=None), dict(Y=None), dict(ldx=7), dict(ldy=7)):
        assert fwd(**bad) == I, bad
    for bad in (dict(X=8), dict(Y=2), dict(ldx=12), dict(ldy=9), dict(xt=1, ldx=9)):
        assert fwd(**bad) == nm.NM_ERR_MISALIGNED, bad
    assert fwd(K=1 << 31) == fwd(T=1 << 31) == nm.NM_ERR_UNSUPPORTED
    assert fwd(T=0) == nm.NM_OK
    for bad in (dict(K=-1), dict(T=-1), dict(K=0), dict(xt=2), dict(dt=9), dict(X=None), dict(dY=None),
                dict(dX=None), dict(mean=None), dict(rstd=None), dict(lddy=7), dict(ldx=7), dict(lddx=7)):
        assert bwd(**bad) == I, bad
    for bad in (dict(dY=8), dict(X=8), dict(dX=8), dict(lddy=12), dict(lddx=12)):
        assert bwd(**bad) == nm.NM_ERR_MISALIGNED, bad
    assert bwd(T=0) == nm.NM_OK


def test_host_argument_checks_of_cross_entropy(lib):
    """Refused before any launch: pattern, sizes, nulls, strides and alignment."""
    L, I = lib, nm.NM_ERR_INVALID_ARG

    def loss(n=2, m=4, R=8, K=32, X=16, ldx=8, T=8, target=16, out=16, lse=16, values=16):
        return L.nm_spmm_xent(values, 16, n, m, R, K, None, X, ldx, T, target, out, lse, None)

    def grad(n=2, m=4, R=8, K=32, X=16, ldx=8, T=8, target=16, lse=16, dloss=16, dX=16, lddx=8, dV=16):
        return L.nm_spmm_xent_grad(16, 16, n, m, R, K, None, X, ldx, T, target, lse, dloss, dX, lddx, dV, None)

    for bad in (dict(n=4), dict(m=5), dict(K=30), dict(R=0), dict(K=0), dict(R=-1), dict(T=-1), dict(X=None),
                dict(target=None), dict(out=None), dict(lse=None), dict(values=None), dict(ldx=7)):
        assert loss(**bad) == I, bad
    assert loss(X=8) == loss(ldx=12) == nm.NM_ERR_MISALIGNED
    assert loss(T=1 << 31) == loss(R=1 << 31) == nm.NM_ERR_UNSUPPORTED
    assert loss(T=0) == nm.NM_OK
    for bad in (dict(n=4), dict(K=30), dict(R=0), dict(T=-1), dict(X=None), dict(target=None), dict(lse=None),
                dict(dloss=None), dict(dX=None, dV=None), dict(lddx=7), dict(ldx=7)):
        assert grad(**bad) == I, bad
    assert grad(dX=8) == grad(lddx=12) == grad(dV=17) == nm.NM_ERR_MISALIGNED
    assert grad(T=0, dV=None) == nm.NM_OK


def test_host_argument_checks_of_the_adapters(lib):
    """Refused before any launch: pattern, sizes, rank, number of adapters, nulls, strides and alignment."""
    L, I, A16, U = lib, nm.NM_ERR_INVALID_ARG, nm.NM_ERR_MISALIGNED, nm.NM_ERR_UNSUPPORTED

    def fwd(fn="nm_spmm_lora", n=2, m=4, R=8, K=32, X=16, ldx=8, T=8, A=16, B=16, rank=4, num=2, adapter=16, Y=16, ldy=8,
            yt=0, values=16):
        return getattr(L, fn)(values, 16, n, m, R, K, None, X, ldx, T, A, B, rank, num, None, adapter, Y, ldy, yt, None)

    def grad(R=8, K=32, dY=16, lddy=8, X=16, ldx=8, T=8, A=16, B=16, rank=4, num=2, adapter=16, dA=16, dB=16, dt=0):
        return L.nm_lora_grad(R, K, dY, lddy, X, ldx, T, A, B, rank, num, None, adapter, dA, dB, dt, None)

    for fn in ("nm_spmm_lora", "nm_spmm_lora_t"):
        for bad in (dict(n=4), dict(K=30), dict(R=-1), dict(T=-1), dict(rank=0), dict(num=-1), dict(yt=3), dict(Y=None),
                    dict(ldy=7)):
            assert fwd(fn, **bad) == I, (fn, bad)
        assert fwd(fn, rank=129) == fwd(fn, num=32768) == U
        assert fwd(fn, Y=8) == fwd(fn, ldy=12) == A16
        assert fwd(fn, T=0) == nm.NM_OK
    for bad in (dict(R=-1), dict(K=-1), dict(T=-1), dict(rank=0), dict(num=-1), dict(dt=2), dict(dA=None, dB=None),
                dict(A=None), dict(B=None), dict(adapter=None), dict(dY=None), dict(X=None), dict(ldx=7), dict(lddy=7)):
        assert grad(**bad) == I, bad
    assert grad(rank=129) == grad(num=32768) == grad(T=1 << 31) == U
    assert grad(dA=17) == grad(dt=1, dB=18) == grad(X=8) == grad(lddy=12) == grad(A=17) == A16
    assert grad(num=0) == nm.NM_OK


def test_host_checks_of_element_alignment(lib):
    """Vectors and words that start off 4 bytes, and values off 2, are refused: the kernels' loads of them would fault."""
    A = nm.NM_ERR_MISALIGNED
    for i in range(4):  # gamma, beta, mean, rstd
        p = [16] * 4
        p[i] = 18
        assert lib.nm_layer_norm(16, 8, 0, 4, 8, p[0], p[1], 1e-5, 16, 8, 0, p[2], p[3], None) == A
    for i in range(5):  # gamma, mean, rstd, dgamma, dbeta
        p = [16] * 5
        p[i] = 18
        for T in (8, 0):
            assert lib.nm_layer_norm_grad(16, 8, 0, 16, 8, 0, 4, T, p[0], p[1], p[2], 16, 8, p[3], p[4], None) == A
    for i in range(6):  # values, meta, idx, target, loss, lse
        p = [16] * 6
        p[i] = 17 if i == 0 else 18
        assert lib.nm_spmm_xent(p[0], p[1], 2, 4, 8, 32, p[2], 16, 8, 8, p[3], p[4], p[5], None) == A
        # values, meta, idx, target, lse, dloss
        assert lib.nm_spmm_xent_grad(p[0], p[1], 2, 4, 8, 32, p[2], 16, 8, 8, p[3], p[4], p[5], 16, 8, 16, None) == A
    for fn in (lib.nm_spmm_lora, lib.nm_spmm_lora_t):
        for i in range(5):  # values, meta, idx, scale, adapter
            p = [16] * 5
            p[i] = 17 if i == 0 else 18
            assert fn(p[0], p[1], 2, 4, 8, 32, p[2], 16, 8, 8, 16, 16, 4, 2, p[3], p[4], 16, 8, 0, None) == A
    for p in ((18, 16), (16, 18)):  # scale, adapter
        assert lib.nm_lora_grad(8, 32, 16, 8, 16, 8, 8, 16, 16, 4, 2, *p, 16, 16, 0, None) == A


def test_compress_refuses_outputs_that_its_stores_cannot_take(lib):
    """2:4 stores pairs of values and of metadata words; a pointer off their size would fault."""
    assert lib.nm_prune_compress(16, 4, 8, 8, 2, 4, 18, 16, None) == nm.NM_ERR_MISALIGNED
    assert lib.nm_prune_compress(16, 4, 8, 8, 2, 4, 16, 20, None) == nm.NM_ERR_MISALIGNED
