"""Columns behind the last token belong to the caller: the dense SM-pair GEMMs leave them as they were.

The outputs are the leading columns of a wider matrix whose other columns hold
a sentinel; the last token ends inside a 16-byte unit.
"""
import numpy as np
import pytest
import torch

import oracle
import sparse_gemm_nm_b200 as nm
import workloads as wl
from gpu_helpers import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 37, 197, 258])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_input_gradient_stops_at_the_last_token(T, dtype):
    R, K, ld = 130, 264, 280
    vals, meta = oracle.compress(wl.normal_bf16((R, K), 0.1, 1), 2, 4)
    dY = to_dev(wl.normal_bf16((R, ld), 1.0, 2))
    values, meta = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV)
    dX = torch.full((K, ld), 5.0, dtype=dtype, device=DEV)
    yt = nm.NM_OUT_F32 if dtype == torch.float32 else nm.NM_OUT_BF16
    nm.nm_spmm_t(values, meta, 2, 4, R, K, None, dY, ld, T, dX, ld, yt)
    full = nm.spmm_t(values, meta, 2, 4, K, dY, out_dtype=dtype)
    assert torch.equal(dX[:, :T], full[:, :T]) and (dX[:, T:] == 5).all()


@pytest.mark.parametrize("T", [3, 101])
def test_int8_and_tf32_outputs_stop_at_the_last_token(T):
    R, K, ld = 70, 64, 112
    v8, m8 = nm.prune_compress_i8(torch.from_numpy(wl.integer_i8((R, K), -9, 9, 3)).to(DEV))
    X8 = torch.from_numpy(wl.integer_i8((K, ld), -9, 9, 4)).to(DEV)
    Y8 = torch.full((R, ld), 5, dtype=torch.int32, device=DEV)
    nm.nm_spmm_i8(v8, m8, R, K, X8, ld, T, Y8, ld)
    assert torch.equal(Y8[:, :T], nm.spmm_i8(v8, m8, K, X8)[:, :T]) and (Y8[:, T:] == 5).all()
    vf, mf = nm.prune_compress_tf32(torch.from_numpy(wl.normal_f32((R, K), 1.0, 5)).to(DEV))
    Xf = torch.from_numpy(wl.normal_f32((K, ld), 1.0, 6)).to(DEV)
    Yf = torch.full((R, ld), 5.0, device=DEV)
    nm.nm_spmm_tf32(vf, mf, R, K, Xf, ld, T, Yf, ld)
    assert torch.equal(Yf[:, :T], nm.spmm_tf32(vf, mf, K, Xf)[:, :T]) and (Yf[:, T:] == 5).all()


@pytest.mark.parametrize("T", [193, 194, 227, 256, 513, 1001, 1030])
def test_int8_and_tf32_outputs_of_many_tokens_stop_at_the_last_token(T):
    """The sparse SM-pair GEMM (192 tokens and more): each tail of a 16-byte unit, in its own chunk of columns or not."""
    R, K, ld = 300, 512, -(-T // 16) * 16 + 16
    v8, m8 = nm.prune_compress_i8(torch.from_numpy(wl.integer_i8((R, K), -9, 9, 3)).to(DEV))
    X8 = torch.from_numpy(wl.integer_i8((K, ld), -9, 9, 4)).to(DEV)
    Y8 = torch.full((R, ld), 5, dtype=torch.int32, device=DEV)
    nm.nm_spmm_i8(v8, m8, R, K, X8, ld, T, Y8, ld)
    assert torch.equal(Y8[:, :T], nm.spmm_i8(v8, m8, K, X8)[:, :T]) and (Y8[:, T:] == 5).all()
    vf, mf = nm.prune_compress_tf32(torch.from_numpy(wl.normal_f32((R, K), 1.0, 5)).to(DEV))
    Xf = torch.from_numpy(wl.normal_f32((K, ld), 1.0, 6)).to(DEV)
    for dtype, yt in ((torch.float32, nm.NM_OUT_F32), (torch.bfloat16, nm.NM_OUT_BF16)):
        Yf = torch.full((R, ld), 5.0, dtype=dtype, device=DEV)
        nm.nm_spmm_tf32(vf, mf, R, K, Xf, ld, T, Yf, ld, yt)
        assert torch.equal(Yf[:, :T], nm.spmm_tf32(vf, mf, K, Xf, out_dtype=dtype)[:, :T]) and (Yf[:, T:] == 5).all()


@pytest.mark.parametrize("T", [7, 9, 63, 65, 71, 129, 255, 260, 513, 1031])
def test_every_tail_of_a_row_in_the_dense_gemms(T):
    """Rows of the input gradient, INT8, TF32 and diagonal products that end anywhere in a chunk of columns."""
    R, K, ld = 300, 264, -(-T // 16) * 16 + 16
    vals, meta = oracle.compress(wl.normal_bf16((R, K), 0.1, 11), 2, 4)
    dY = to_dev(wl.normal_bf16((R, ld), 1.0, 12))
    values, meta = to_dev(vals), torch.from_numpy(meta.view(np.int32)).to(DEV)
    for dtype, yt in ((torch.bfloat16, nm.NM_OUT_BF16), (torch.float32, nm.NM_OUT_F32)):
        dX = torch.full((K, ld), 5.0, dtype=dtype, device=DEV)
        nm.nm_spmm_t(values, meta, 2, 4, R, K, None, dY, ld, T, dX, ld, yt)
        full = nm.spmm_t(values, meta, 2, 4, K, dY, out_dtype=dtype)
        assert torch.equal(dX[:, :T], full[:, :T]) and (dX[:, T:] == 5).all()
    W = to_dev(wl.normal_bf16((K, R), 1.0, 13))  # K rows of R columns
    off, dv = nm.diag_prune_compress(W, 17)
    for dtype, yt in ((torch.bfloat16, nm.NM_OUT_BF16), (torch.float32, nm.NM_OUT_F32)):
        Y = torch.full((K, ld), 5.0, dtype=dtype, device=DEV)
        nm.nm_diag_spmm(dv, off, 17, K, R, None, dY, ld, T, Y, ld, yt)
        full = torch.full((K, ld), 5.0, dtype=dtype, device=DEV)
        nm.nm_diag_spmm(dv, off, 17, K, R, None, dY, ld, ld, full, ld, yt)
        assert torch.equal(Y[:, :T], full[:, :T]) and (Y[:, T:] == 5).all()
    v8, m8 = nm.prune_compress_i8(torch.from_numpy(wl.integer_i8((R, 80), -9, 9, 3)).to(DEV))  # K % 32 != 0: the dense GEMM
    X8 = torch.from_numpy(wl.integer_i8((80, ld), -9, 9, 4)).to(DEV)
    Y8 = torch.full((R, ld), 5, dtype=torch.int32, device=DEV)
    nm.nm_spmm_i8(v8, m8, R, 80, X8, ld, T, Y8, ld)
    assert torch.equal(Y8[:, :T], nm.spmm_i8(v8, m8, 80, X8)[:, :T]) and (Y8[:, T:] == 5).all()
