"""Sums and roundings of the gated block's gradients, on the GPU against 64 bits.

The header's bound: with h half a unit of the handle's type and A = |dp| |Wm| summed
over n = 2 n_ff terms (dW: |dp| |X| over n = T), a gradient r is within
    (h + min(n, 2^14) 2^-26 + 2^-17 + n 2^-38) A + h |r|
of the exact one.  h A is the rounding of dp.  A run of at most 2^14 products takes
n / 16 tensor-core steps, each off by a unit in the last place of a partial sum that A
bounds (2^-23, truncated) and as much again for the alignment within the step: n / 8
2^-23 = n 2^-26; the fp32 additions of the runs and of at most 74 parts of a cut sum
round to nearest, n 2^-14 2^-24 and 74 x 2^-24 < 2^-17.  Where the inputs make dp exact
in the handle's type, the first h is left out here.
"""
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm

pytestmark = pytest.mark.gpu

DTS = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _no_forced_plan(monkeypatch):
    for k in ("NMSPMM_FORCE_GRAD_BN", "NMSPMM_GRAD_SPLIT"):
        monkeypatch.delenv(k, raising=False)


def sum_error(n):
    return min(n, 2 ** 14) * 2.0 ** -26 + 2.0 ** -17 + n * 2.0 ** -38


def product(a, b):
    """a @ b in 64 bits, the summed axis in pieces."""
    out = torch.zeros((a.shape[0], b.shape[1]), dtype=torch.float64, device="cuda")
    for i in range(0, a.shape[1], 1 << 17):
        out += a[:, i:i + (1 << 17)].double() @ b[i:i + (1 << 17)].double()
    return out


def close(got, left, right, n, dp_error=0.0):
    """left @ right against got; dp_error: what each element of left may be off by."""
    half = torch.finfo(got.dtype).eps / 2
    ref, A = product(left, right), product(left.abs(), right.abs())
    tol = sum_error(n) * A
    if isinstance(dp_error, torch.Tensor):
        tol = tol + product(dp_error, right.abs()) * (1 + sum_error(n))
    tol = tol + half * (ref.abs() + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def backward(h, X, P, dY, act):
    """The gradients, with everything around them and in the workspace poisoned."""
    T, k, F = X.shape[0], X.shape[1], dY.shape[1]
    bufs = [torch.full((n + 64,), 77.0, dtype=t, device="cuda")
            for n, t in ((T * k, X.dtype), (2 * F * k, X.dtype), (2 * F, torch.float32))]
    ws = torch.full((nm.nm_gated_backward_workspace(h, T),), 0xFF, dtype=torch.uint8, device="cuda")
    dX, dW, db = nm.nm_gated_backward(h, X, P, dY, act=act, dX=bufs[0][:-64].view(T, k), dW=bufs[1][:-64].view(2 * F, k),
                                      dbias=bufs[2][:-64], workspace=ws)
    torch.cuda.synchronize()
    assert nm.nm_device_status(h) == nm.NM_OK
    assert all(bool((b[-64:] == 77).all()) for b in bufs)
    return dX, dW, db


def positive(shape, g, dt):
    return (0.125 + 0.125 * torch.rand(shape, generator=g, device="cuda")).to(dt)


def one_sign(dt, T, k, F, seed=0):
    """A block whose sums have terms of one sign and whose dp, half of P with its halves
    changed over, is exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X, P, W = positive((T, k), g, dt), positive((T, 2 * F), g, dt), positive((2 * F, k), g, dt)
    dY = torch.full((T, F), 0.5, dtype=dt, device="cuda")
    return nm.nm_compress_gated(W, 4, 4), X, P, dY, W, torch.cat((P[:, F:], P[:, :F]), dim=1) * 0.5


@pytest.mark.parametrize("split", ["0", "1"])          # whole sums; sums cut over idle pairs
@pytest.mark.parametrize("bn", [128, 256])
def test_long_sums_of_one_sign(monkeypatch, bn, split):
    monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", str(bn))
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", split)
    for T, k, F in ((1 << 20, 64, 16), (48, 64, 1 << 19)):
        h, X, P, dY, W, dp = one_sign(torch.float16, T, k, F)
        dX, dW, _ = backward(h, X, P, dY, "none")
        close(dX, dp, W, 2 * F)
        close(dW, dp.t(), X, T)


@pytest.mark.parametrize("split", ["0", "1"])
@pytest.mark.parametrize("T", [(1 << 14) - 1, 1 << 14, (1 << 14) + 1, (1 << 15) + 65])
@pytest.mark.parametrize("dt", list(DTS))
def test_sums_around_a_run(monkeypatch, dt, T, split):
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", split)
    h, X, P, dY, W, dp = one_sign(DTS[dt], T, 72, 40, seed=T)
    dX, dW, _ = backward(h, X, P, dY, "none")
    close(dX, dp, W, 80)
    close(dW, dp.t(), X, T)
    # and many tiles on every pair, the accumulators in turn
    h, X, P, dY, W, dp = one_sign(DTS[dt], 2600, 520, T // 2, seed=T)
    dX, dW, _ = backward(h, X, P, dY, "none")
    close(dX, dp, W, T // 2 * 2)
    close(dW, dp.t(), X, 2600)


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("T,k,F", [(1379, 768, 2051), (2000, 1024, 1024)])
def test_dp_is_rounded_once_and_nothing_else(dt, T, k, F):
    """Without an activation dp = (dY u, dY g) is exact in fp32, so its rounding to the handle's
    type is known: against products of that dp only the sums and the result's rounding are left."""
    g = torch.Generator(device="cuda").manual_seed(F)
    X, P, dY, W = (torch.randn(s, generator=g, device="cuda").to(DTS[dt])
                   for s in ((T, k), (T, 2 * F), (T, F), (2 * F, k)))
    h = nm.nm_compress_gated(W, 2, 4)
    Wm = nm.nm_decompress(h)
    dX, dW, _ = backward(h, X, P, dY, "none")
    dp = (torch.cat((P[:, F:], P[:, :F]), dim=1).float() * dY.float().repeat(1, 2)).to(DTS[dt])
    close(dX, dp, Wm, 2 * F)
    close(dW, dp.t(), X, T)
