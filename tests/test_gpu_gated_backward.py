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

FP16: dp is stored times a power of two where its largest magnitude m is outside [2^-4,
2^15).  Within, an element below fp16's normal range is off by 2^-25 <= 2^-21 m; scaled
to m in [2^14, 2^15) by 2^-39 m: h |dp| + 2^-21 m covers both.
"""
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm
from test_gpu_gated import check_backward, dp_reference

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


# ------------------------------------------------------------------ fp16: dp beyond fp16's range

def fp16_case(T, k, F, scales, act, seed=0, spike=None):
    """X, P, dY, W of normal values times `scales`; spike: one entry of dY times that."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X, P, dY, W = ((torch.randn(s, generator=g, device="cuda") * c).half()
                   for s, c in zip(((T, k), (T, 2 * F), (T, F), (2 * F, k)), scales))
    if spike:
        dY[T // 2, F // 3] *= spike
    return X, P, dY, W


def check_range(T, k, F, scales, act="none", N=2, M=4, seed=0, spike=None):
    X, P, dY, W = fp16_case(T, k, F, scales, act, seed, spike)
    h = nm.nm_compress_gated(W, N, M)
    dX, dW, db = backward(h, X, P, dY, act)
    dp, e = dp_reference(P, dY, act)
    dp, e = torch.from_numpy(dp).cuda(), torch.from_numpy(e).cuda()
    # the header's error of an element of dp, and what the activation adds
    e = e + 2.0 ** -11 * (dp.abs() + e) + 2.0 ** -21 * float(dp.abs().max())
    assert torch.isfinite(dX).all() and torch.isfinite(dW).all()
    close(dX, dp, nm.nm_decompress(h), 2 * F, e)
    close(dW, dp.t(), X, T, e.t())
    return dp, dX, dW


@pytest.mark.parametrize("T,k,F", [(1, 64, 24), (65, 128, 64), (200, 264, 1030), (3000, 64, 40), (333, 520, 129)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
@pytest.mark.parametrize("scales", [(2.0 ** -9, 300.0, 300.0, 2.0 ** -9),     # |dp| up to a million and more
                                    (100.0, 2.0 ** -10, 2.0 ** -14, 3.0),    # |dp| around 2^-24, dX and dW not
                                    (1.0, 1.0, 2.0 ** -12, 1.0)])            # gradients of a mean: below fp16's normal range
def test_dp_beyond_the_range_of_fp16(T, k, F, act, scales):
    check_range(T, k, F, scales, act, seed=T)


@pytest.mark.parametrize("F", [40, 41])
def test_one_large_dp_among_ordinary_ones(F):
    dp, _, _ = check_range(100, 64, F, (2.0 ** -6, 30.0, 1.0, 2.0 ** -8), spike=2.0 ** 13, seed=3)
    assert float(dp.abs().max()) > 65504


@pytest.mark.parametrize("F", [1, 8])
def test_powers_of_two_come_out_exactly(F):
    """A single dp of 2^s: both sides of every border of the range, to the bit."""
    for s in range(-29, 30):
        w = min(max(-s, -14), 15)
        X = torch.full((1, 8), 2.0 ** w, device="cuda").half()
        W = torch.zeros((2 * F, 8), device="cuda").half()
        W[0] = 2.0 ** w
        P, dY = torch.zeros((1, 2 * F), device="cuda").half(), torch.zeros((1, F), device="cuda").half()
        P[0, F], dY[0, 0] = 2.0 ** (s // 2), 2.0 ** (s - s // 2)
        dX, dW, db = backward(nm.nm_compress_gated(W, 4, 4), X, P, dY, "none")
        assert bool((dX == 2.0 ** (s + w)).all()) and bool((dW[0] == 2.0 ** (s + w)).all()), s
        assert not dW[1:].any() and float(db[0]) == 2.0 ** s


def test_nothing_and_infinities_in_dp():
    T, k, F = 90, 64, 48
    X, P, dY, W = fp16_case(T, k, F, (1.0, 1.0, 2.0 ** -13, 1.0), "none")
    h = nm.nm_compress_gated(W, 2, 4)
    dX, dW, db = backward(h, X, P, torch.zeros_like(dY), "none")
    assert not dX.any() and not dW.any() and not db.any()
    # an infinity spoils its token and its two channels, and the others keep their range
    P[7, 5] = P[7, F + 5] = 1.0
    dY[7, 5] = 0.0
    clean = backward(h, X, P, dY, "none")
    dY[7, 5] = float("inf")
    dX, dW, _ = backward(h, X, P, dY, "none")
    rows, cols = [t for t in range(T) if t != 7], [f for f in range(2 * F) if f % F != 5]
    assert torch.equal(dX[rows], clean[0][rows]) and torch.equal(dW[cols], clean[1][cols])
    assert not torch.isfinite(dX[7]).any() and not torch.isfinite(dW[[5, F + 5]]).any()


def test_range_is_decided_in_the_captured_call():
    T, k, F = 150, 128, 80
    sets = [fp16_case(T, k, F, s, "silu", seed=i) for i, s in enumerate((
        (1.0, 1.0, 1.0, 1.0), (2.0 ** -9, 300.0, 300.0, 1.0), (1.0, 1.0, 2.0 ** -14, 1.0)))]
    W = sets[0][3] * 2.0 ** -6
    h = nm.nm_compress_gated(W, 2, 4)
    want = [nm.nm_gated_backward(h, *s[:3], bias_grad=True) for s in sets]
    held = [t.clone() for t in sets[0][:3]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nm.nm_gated_backward(h, *held, bias_grad=True)
    for i in (0, 1, 2, 1, 0):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        graph.replay()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("split", ["0", "1"])
@pytest.mark.parametrize("down", [2.0 ** -14, 2.0 ** -10])
def test_long_sums_of_a_scaled_dp(monkeypatch, down, split):
    """Runs, parts and the scaling together: dp below fp16's normal range, exact once it is scaled."""
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", split)
    for T, k, F in ((1 << 18, 64, 16), (48, 64, 1 << 17)):
        h, X, P, dY, W, dp = one_sign(torch.float16, T, k, F, seed=1)
        dX, dW, db = backward(h, X, P, dY * (2 * down), "none")
        dp = dp.double() * (2 * down)
        close(dX, dp, W, 2 * F)
        close(dW, dp.t(), X, T)
        ref = dp.sum(0)
        assert bool(((db.double() - ref).abs() <= (T / 8 + 24) * 2.0 ** -24 * ref).all())


# ------------------------------------------------------------------ sums cut over idle pairs

@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("T,k,F", [(1500, 64, 1500), (3000, 128, 700), (3000, 64, 1500), (1500, 72, 1501)])
def test_both_products_cut(monkeypatch, T, k, F, dt, bn):
    """Parts of both products' tiles in one call: slots and joined tiles of the second come after
    the first's.  The same results every time, and from calls for one product alone."""
    monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", str(bn))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = nm.nm_gated_backward_plan_for_shape(F, k, T, sms)
    assert plan["splits_dx"] > 1 and plan["splits_dw"] > 1 and plan["complete"] == 1
    h, X, P, dY, (dX, dW, db) = check_backward(dt, T, k, F, seed=T)
    for _ in range(5):
        x, w, b = nm.nm_gated_backward(h, X.cuda(), P.cuda(), dY.cuda(), bias_grad=True)
        assert torch.equal(x, dX) and torch.equal(w, dW) and torch.equal(b, db)
    if dt == "fp16":        # and the parts of a scaled dp
        check_range(T, k, F, (2.0 ** -9, 300.0, 300.0, 2.0 ** -9), "silu", seed=T)
