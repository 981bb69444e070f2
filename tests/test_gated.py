"""Gated feed-forward block without a GPU: the oracle's gradients against
differences, and the argument checks that come before any device work."""
import ctypes

import numpy as np
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm
from oracle import ffn

A, B, C, D = 4096, 1 << 20, 1 << 24, 1 << 28   # aligned addresses that are never followed


def test_oracle_hand_worked_block():
    X = np.array([[1.0, 2.0]])
    W = np.array([[1.0, 0.0], [0.0, -1.0], [2.0, 0.0], [0.0, 0.5]])   # two gate rows, two up rows
    p = ffn.gated_pre(X, W, scale=[1, 1, 2, 1], bias=[0, 0, 0, 3])
    np.testing.assert_array_equal(p, [[1, -2, 4, 4]])
    np.testing.assert_array_equal(ffn.gated(p, "none"), [[4, -8]])
    np.testing.assert_array_equal(ffn.gated(p, "relu"), [[4, 0]])
    np.testing.assert_allclose(ffn.gated(p, "silu"), [[4 * 0.7310585786300049, -8 * 0.11920292202211755]], rtol=1e-15)
    np.testing.assert_allclose(ffn.gated(p, "gelu"), [[4 * 0.8413447460685429, -8 * 0.022750131948179195]], rtol=1e-14)
    np.testing.assert_array_equal(ffn.gated_dp(p, [[1.0, 10.0]], "relu"), [[4, 0, 1, 0]])


@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu"])
def test_oracle_gradients_agree_with_differences(act):
    rng = np.random.default_rng(1)
    X, W, b, dY = (rng.standard_normal(s) for s in ((5, 8), (12, 8), (12,), (5, 6)))
    W = ffn.mask(W, 2, 4)
    loss = lambda X, W, b: float((ffn.gated(ffn.gated_pre(X, W, bias=b), act) * dY).sum())  # noqa: E731
    dp = ffn.gated_dp(ffn.gated_pre(X, W, bias=b), dY, act)
    grads = (dp @ W, dp.T @ X, dp.sum(0))
    for i, g in enumerate(grads):
        for _ in range(4):
            args = [X, W, b]
            d = rng.standard_normal(args[i].shape)
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (g * d).sum()) < 1e-6


@pytest.mark.parametrize("args,status", [
    ((None, 4, 8, nm.NM_INT8, 2, 4), nm.NM_ERR_INVALID),
    ((16, 0, 8, nm.NM_INT8, 2, 4), nm.NM_ERR_INVALID),
    ((16, -4, 8, nm.NM_INT8, 2, 4), nm.NM_ERR_INVALID),
    ((16, -(1 << 62), 8, nm.NM_INT8, 2, 4), nm.NM_ERR_INVALID),
    ((16, 1 << 62, 8, nm.NM_INT8, 2, 4), nm.NM_ERR_UNSUPPORTED),
    ((16, (1 << 23) + 1, 8, nm.NM_INT8, 2, 4), nm.NM_ERR_UNSUPPORTED),   # 2 n_ff above 2^24
    ((16, 4, 10, nm.NM_INT8, 2, 4), nm.NM_ERR_INVALID),
    ((16, 4, 8, nm.NM_FP32, 2, 4), nm.NM_ERR_INVALID),
    ((16, 4, 8, nm.NM_INT8, 3, 4), nm.NM_ERR_UNSUPPORTED),
    ((17, 4, 8, nm.NM_FP16, 2, 4), nm.NM_ERR_INVALID),
])
def test_compress_gated_refusals(args, status):
    out = ctypes.c_void_p(7)
    assert nm.lib().nm_compress_gated(*args, None, ctypes.byref(out)) == status
    assert out.value is None and nm.nm_last_error() != ""


def test_null_handles():
    L = nm.lib()
    n = ctypes.c_size_t()
    assert L.nm_compress_gated(A, 4, 8, nm.NM_INT8, 2, 4, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_gated(None, A, 1, B, None, None, None) == nm.NM_ERR_INVALID
    assert L.nm_gated_backward_workspace(None, 1, ctypes.byref(n)) == nm.NM_ERR_INVALID
    assert L.nm_gated_backward(None, A, B, C, 1, 2, D, None, None, A, 0, None) == nm.NM_ERR_INVALID


def test_binding_refuses_before_the_library():
    with pytest.raises(ValueError):
        nm.nm_compress_gated(torch.zeros(5, 64, dtype=torch.int8), 2, 4)      # odd number of rows
    with pytest.raises(ValueError):
        nm.nm_compress_gated(torch.zeros(4, 64), 2, 4)                         # fp32
    with pytest.raises(ValueError):
        nm.nm_compress_gated(torch.zeros(4, 64, dtype=torch.int8), 2, 4)      # on the host
