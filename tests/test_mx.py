"""Microscaled 4-bit floating point without a GPU: the oracle's pins, and the
argument checks of the C ABI that come before any device work."""
import ctypes

import numpy as np
import pytest

import structured_sparse_gemm_compress_b200 as nm
from oracle import ffn

A, B, C = 4096, 1 << 20, 1 << 24   # aligned addresses that are never followed


def quantise(T=4, k=64, ldx=64, dt=nm.NM_BF16, X=A, Q=B, S=C):
    return nm.lib().nm_mx_quantize(X, T, k, ldx, dt, Q, S, None)


def test_oracle_hand_worked_block():
    # largest magnitude 7: e = 2 - 2 = 0, so the values round on the grid itself
    x = np.zeros((1, 32))
    x[0, :14] = [7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, -0.25, -5.5, 0.2501, -0.0, 4.99]
    codes, byte = ffn.mx_quantize(x)
    assert byte[0, 0] == 127
    #                              7  .25 .75 1.25 1.75 2.5 3.5 5 6.5 -.25 -5.5 .2501 -0 4.99
    assert list(codes[0, :14]) == [7, 0, 2, 2, 4, 4, 6, 6, 7, 8, 15, 1, 8, 6]
    assert list(codes[0, 14:]) == [0] * 18
    v = ffn.mx_values(codes, byte)
    assert list(v[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4]


def test_oracle_scale_limits():
    x = np.zeros((4, 32))
    x[1, 3] = 2.0 ** -126                       # e would be -128: held at -127
    x[2, 5] = np.float64(np.finfo(np.float32).max)
    x[3, 7] = np.inf
    codes, byte = ffn.mx_quantize(x)
    assert list(byte[:, 0]) == [0, 0, 252, 255]
    assert codes[1, 3] == 4 and ffn.mx_values(codes, byte)[1, 3] == 2.0 ** -126
    assert codes[2, 5] == 7 and not codes[3].any()
    assert np.isnan(ffn.mx_values(codes, byte)[3]).all()


def test_oracle_nearest_by_enumeration():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 64)) * 2.0 ** rng.integers(-20, 20, (5, 1))
    codes, byte = ffn.mx_quantize(x)
    got = np.abs(ffn.mx_values(codes, byte) - x)
    s = 2.0 ** (np.repeat(byte, 32, axis=1).astype(float) - 127)
    grid = np.concatenate([-ffn.LEVELS, ffn.LEVELS])
    best = np.abs(grid[None, None, :] * s[:, :, None] - x[:, :, None]).min(axis=2)
    np.testing.assert_array_equal(got, best)


def test_oracle_mask_is_the_top_n_rule():
    W = np.array([[1.0, -1.0, 1.0, 0.5, 2.0, 0.0, -3.0, 0.0]])
    np.testing.assert_array_equal(ffn.mask(W, 2, 4), [[1, -1, 0, 0, 2, 0, -3, 0]])
    np.testing.assert_array_equal(ffn.mask(W, 2, 8), [[0, 0, 0, 0, 2, 0, -3, 0]])


def test_oracle_slopes_agree_with_differences():
    v = np.linspace(-6, 6, 241)[:, None] + 0.0125
    for name in ("none", "gelu", "silu", "relu"):
        d = (ffn.act(v + 1e-5, name) - ffn.act(v - 1e-5, name)) / 2e-5
        np.testing.assert_allclose(ffn.act_slope(v, name), d, atol=1e-8)


def test_scale_bytes():
    assert nm.nm_mx_scale_bytes(0, 32) == 0
    assert nm.nm_mx_scale_bytes(1, 32) == 1024
    assert nm.nm_mx_scale_bytes(129, 288) == 4096
    assert nm.nm_mx_scale_bytes((1 << 31) - 1, 1 << 24) == (1 << 24) * (1 << 16) * 1024
    for bad in ((-1, 32), (4, 0), (4, 31), (4, -32)):
        with pytest.raises(nm.NMError) as e:
            nm.nm_mx_scale_bytes(*bad)
        assert e.value.status == nm.NM_ERR_INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(dt=nm.NM_INT8), nm.NM_ERR_INVALID),
    (dict(dt=9), nm.NM_ERR_INVALID),
    (dict(T=-1), nm.NM_ERR_INVALID),
    (dict(k=0, ldx=64), nm.NM_ERR_INVALID),
    (dict(k=48), nm.NM_ERR_INVALID),                   # not whole blocks of 32
    (dict(ldx=32), nm.NM_ERR_INVALID),                 # below k
    (dict(ldx=65), nm.NM_ERR_INVALID),                 # rows not on 16 bytes
    (dict(dt=nm.NM_FP32, ldx=66), nm.NM_ERR_INVALID),
    (dict(X=None), nm.NM_ERR_INVALID),
    (dict(Q=None), nm.NM_ERR_INVALID),
    (dict(S=None), nm.NM_ERR_INVALID),
    (dict(X=A + 2), nm.NM_ERR_INVALID),                # misaligned
    (dict(Q=B + 8), nm.NM_ERR_INVALID),
    (dict(S=C + 4), nm.NM_ERR_INVALID),
    (dict(Q=A + 64), nm.NM_ERR_INVALID),               # overlaps X
    (dict(S=A), nm.NM_ERR_INVALID),
    (dict(S=B), nm.NM_ERR_INVALID),                    # overlaps Q
    (dict(T=1 << 31), nm.NM_ERR_UNSUPPORTED),
    (dict(k=(1 << 24) + 32, ldx=(1 << 24) + 32), nm.NM_ERR_UNSUPPORTED),
])
def test_quantise_refusals(kw, status):
    assert quantise(**kw) == status
    assert nm.nm_last_error() != ""


def test_empty_calls_are_no_ops():
    L = nm.lib()
    assert quantise(T=0, X=None, Q=None, S=None) == nm.NM_OK
    assert L.nm_mx_dequantize(None, None, 0, 64, nm.NM_FP16, None, None) == nm.NM_OK


@pytest.mark.parametrize("args,status", [
    ((None, B, 4, 64, nm.NM_BF16, C), nm.NM_ERR_INVALID),
    ((A, None, 4, 64, nm.NM_BF16, C), nm.NM_ERR_INVALID),
    ((A, B, 4, 64, nm.NM_BF16, None), nm.NM_ERR_INVALID),
    ((A, B, 4, 64, nm.NM_INT8, C), nm.NM_ERR_INVALID),
    ((A, B, 4, 40, nm.NM_BF16, C), nm.NM_ERR_INVALID),
    ((A + 1, B, 4, 64, nm.NM_BF16, C), nm.NM_ERR_INVALID),
    ((A, B, 4, 64, nm.NM_BF16, A), nm.NM_ERR_INVALID),
    ((A, B, -4, 64, nm.NM_BF16, C), nm.NM_ERR_INVALID),
])
def test_dequantise_refusals(args, status):
    assert nm.lib().nm_mx_dequantize(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((None, 4, 64, nm.NM_BF16, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 0, 64, nm.NM_BF16, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 4, 48, nm.NM_BF16, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 4, 64, nm.NM_INT8, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 4, 64, nm.NM_MXFP4, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 4, 64, nm.NM_BF16, 3, 4, 0), nm.NM_ERR_UNSUPPORTED),
    ((A, 4, 64, nm.NM_BF16, 5, 4, 0), nm.NM_ERR_INVALID),
    ((A + 8, 4, 64, nm.NM_BF16, 2, 4, 0), nm.NM_ERR_INVALID),
    ((A, 5, 64, nm.NM_BF16, 2, 4, 1), nm.NM_ERR_INVALID),          # gated with an odd number of rows
    ((A, (1 << 24) + 1, 64, nm.NM_BF16, 2, 4, 0), nm.NM_ERR_UNSUPPORTED),
])
def test_compress_mx_refusals(args, status):
    out = ctypes.c_void_p(7)
    assert nm.lib().nm_compress_mx(*args, None, ctypes.byref(out)) == status
    assert out.value is None and nm.nm_last_error() != ""


def test_null_handles():
    L = nm.lib()
    assert L.nm_spmm_mx(None, A, B, 1, C, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_mx_gated(None, A, B, 1, C, None, None) == nm.NM_ERR_INVALID
    assert L.nm_compress_mx(A, 4, 64, nm.NM_BF16, 2, 4, 0, None, None) == nm.NM_ERR_INVALID


def test_binding_refuses_before_the_library():
    import torch
    with pytest.raises(ValueError):
        nm.nm_mx_quantize(torch.zeros(4, 64, dtype=torch.int8))
    with pytest.raises(ValueError):
        nm.nm_mx_quantize(torch.zeros(4, 128)[:, ::2])
    with pytest.raises(ValueError):
        nm.nm_compress_mx(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError):
        nm.nm_mx_dequantize(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8),
                            dtype=torch.int8)


def test_missing_compiled_binding_is_an_error(monkeypatch):
    import sys

    import torch
    monkeypatch.setattr(nm, "_module", None)
    monkeypatch.setitem(sys.modules, nm.__name__ + "._binding", None)
    monkeypatch.delattr(nm, "_binding", raising=False)
    with pytest.raises(RuntimeError, match="binding is missing"):
        nm.nm_mx_quantize(torch.zeros(4, 64))


def test_binding_checks_tensors_and_arity():
    import torch
    native = nm._native()
    with pytest.raises(TypeError):
        native.mx_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="must be a tensor"):
        nm.nm_mx_quantize([1.0, 2.0])
    with pytest.raises(ValueError, match="CUDA device"):
        nm.nm_mx_quantize(torch.zeros(4, 64))
