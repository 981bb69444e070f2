"""Gated feed-forward block on the GPU against the 64-bit oracle.

Forward, per element: INT8 accumulators are exact (rounded once to fp32, 2^-24
relative); 16-bit products are exact in fp32 and the tensor core adds them 16 (or
32) at a time into an fp32 sum, each addition off by at most a unit in the last
place of a partial sum that A = sum |x||w| bounds, and as much again for the
alignment within one step: e_acc = (k / 8 + 4) 2^-23 A.  The output stage adds its
roundings, the activations' errors and the output type's half unit as in
test_gpu_mx.

Gradients: dp is formed in fp32 (relative errors of act and act' below), rounded
to the handle's type for the products (half = finfo.eps / 2 relative), the sums
err like the forward ones, and the result is rounded once:
    |dX - ref| <= e_dp |Wm| + (n / 8 + 4) 2^-23 |dp| |Wm| + half |ref|, n = 2 n_ff
and likewise dW with n = T.  dbias sums fp32 values with at most T / 8 + 24
additions in a row: e_dp32 summed + (T / 8 + 24) 2^-24 sum |dp|.
act': SiLU s (1 + x (1 - s)) with s off by (5e-7 + 1.3e-7 |x|) relative gives
(1.5e-6 + 3e-7 |x|)(1 + |x|) s; GELU Phi + x phi with Phi off by 1.5e-7 / 2 and the
power of two by (5e-7 + 0.7e-7 x^2) relative gives 2e-7 + (1e-6 + 1e-7 x^2)
(Phi + |x| phi).
"""
import math

import numpy as np
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm
from oracle import ffn
from test_gpu_mx import act_error, f64, rounded

pytestmark = pytest.mark.gpu

DTS = {"int8": torch.int8, "fp16": torch.float16, "bf16": torch.bfloat16}
ODT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
ACTS = ["none", "gelu", "silu", "relu"]


@pytest.fixture(autouse=True)
def _no_forced_plan(monkeypatch):
    for k in ("NMSPMM_FORCE_BN", "NMSPMM_FORCE_SPLITK", "NMSPMM_FORCE_XS", "NMSPMM_FORCE_GRID",
              "NMSPMM_FORCE_PAIR", "NMSPMM_SPLIT_GLOBAL", "NMSPMM_FORCE_GRAD_BN", "NMSPMM_GRAD_SPLIT"):
        monkeypatch.delenv(k, raising=False)


def problem(dt, T, k, F, N, M, seed=0):
    g = torch.Generator().manual_seed(seed)
    if dt == "int8":
        X = torch.randint(-128, 128, (T, k), generator=g).to(torch.int8)
        W = torch.randint(-127, 128, (2 * F, k), generator=g).to(torch.int8)
        s = (0.5 + torch.rand(2 * F, generator=g)) / (5400 * math.sqrt(k * N / M))
    else:
        X = torch.randn((T, k), generator=g).to(DTS[dt])
        W = (torch.randn((2 * F, k), generator=g) / math.sqrt(k)).to(DTS[dt])
        s = None
    b = 0.5 * torch.randn(2 * F, generator=g)
    return X, W, s, b


def forward_reference(dt, X, Wm, s, b, act, odt):
    x, w = f64(X), f64(Wm)
    p, A, k = x @ w.T, np.abs(x) @ np.abs(w).T, x.shape[1]
    e = 2.0 ** -24 * np.abs(p) if dt == "int8" else (k / 8 + 4) * 2.0 ** -23 * A
    if s is not None:
        s = f64(s)
        p, e = p * s, e * np.abs(s)
        e = e + 2.0 ** -24 * np.abs(p)
    if b is not None:
        p = p + f64(b)
        e = e + 2.0 ** -24 * (np.abs(p) + e)
    F = p.shape[1] // 2
    a, ea = act_error(p[:, :F], e[:, :F], act)
    u, eu = p[:, F:], e[:, F:]
    y = a * u
    ey = np.abs(u) * ea + np.abs(a) * eu + ea * eu + 2.0 ** -24 * np.abs(y)
    return y, rounded(y, ey, odt) if odt is not None else ey, p, e


def check_forward(dt, T, k, F, N=2, M=4, act="silu", out="float32", bias=True, save=False, seed=0):
    X, W, s, b = problem(dt, T, k, F, N, M, seed)
    if not bias:
        b = None
    h = nm.nm_compress_gated(W.cuda(), N, M)
    odt = ODT[out] if out in ODT else (torch.float32 if dt == "int8" else DTS[dt])
    ybuf = torch.full((T * F + 64,), 77.0, dtype=odt, device="cuda")
    pbuf = torch.full((T * 2 * F + 64,), 77.0, dtype=DTS[dt], device="cuda") if save else None
    Y = ybuf[:T * F].view(T, F)
    P = pbuf[:T * 2 * F].view(T, 2 * F) if save else None
    nm.nm_spmm_gated(h, X.cuda(), Y=Y, P=P, scale=None if s is None else s.cuda(),
                     bias=None if b is None else b.cuda(), act=act, out=out)
    torch.cuda.synchronize()
    assert nm.nm_device_status(h) == nm.NM_OK
    Wm = torch.from_numpy(ffn.mask(f64(W), N, M))
    y, tol, p, e = forward_reference(dt, X, Wm, s, b, act, odt)
    err = np.abs(f64(Y) - y)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    assert bool((ybuf[T * F:] == 77).all())
    if save:
        assert (np.abs(f64(P) - p) <= rounded(p, e, DTS[dt])).all()
        assert bool((pbuf[T * 2 * F:] == 77).all())
    return h, Y


@pytest.mark.parametrize("N,M", [(1, 4), (2, 4), (2, 8), (4, 8), (4, 4), (8, 8)])
@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("F", [1, 17, 80])
def test_compress_gated_formats(dt, N, M, F):
    """Decompressed and canonical formats are in W's own row order, as nm_compress gives them."""
    _, W, _, _ = problem(dt, 1, 272, F, N, M, seed=F)
    h, ref = nm.nm_compress_gated(W.cuda(), N, M), nm.nm_compress(W.cuda(), N, M)
    assert torch.equal(nm.nm_decompress(h), nm.nm_decompress(ref))
    for a, b in zip(nm.nm_export(h), nm.nm_export(ref)):
        assert torch.equal(a, b)
    W2 = W.flip(0).contiguous().cuda()
    nm.nm_recompress(h, W2)
    assert torch.equal(nm.nm_decompress(h), nm.nm_decompress(nm.nm_compress(W2, N, M)))
    assert nm.nm_query(h)["n_out"] == 2 * F


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("T,k,F", [(1, 64, 1), (1, 768, 100), (2, 96, 15), (31, 128, 16), (33, 272, 17), (128, 512, 64),
                                   (129, 1024, 65), (197, 768, 333), (300, 400, 128)])
def test_forward_sizes(dt, T, k, F):
    check_forward(dt, T, k, F, save=dt != "int8", seed=T + F)


@pytest.mark.parametrize("N,M", [(1, 4), (2, 8), (4, 8), (4, 4)])
@pytest.mark.parametrize("dt", list(DTS))
def test_forward_patterns(dt, N, M):
    check_forward(dt, 140, 320, 90, N, M, act="gelu", bias=False, save=dt != "int8")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["float32", "float16", "bfloat16", "default"])
@pytest.mark.parametrize("dt", list(DTS))
def test_forward_output_stage(dt, out, act):
    check_forward(dt, 70, 256, 40, act=act, out=out)


@pytest.mark.parametrize("dt,image", [("int8", (2, 4)), ("int8", (4, 8)), ("bf16", (2, 4)), ("fp16", (4, 4))])
@pytest.mark.parametrize("pair,bn", [(0, 32), (0, 64), (0, 128), (0, 192), (1, 128), (1, 192)])
@pytest.mark.parametrize("F", [147, 152])       # p stored element by element, in whole runs
def test_forced_tiles(monkeypatch, dt, image, pair, bn, F):
    monkeypatch.setenv("NMSPMM_FORCE_PAIR", str(pair))
    monkeypatch.setenv("NMSPMM_FORCE_BN", str(bn))
    h, _ = check_forward(dt, 461, 320, F, *image, save=dt != "int8", out="float16")
    plan = nm.nm_plan_query(h, 461)
    if not (bn == 192 and pair == 0 and image != (2, 4)):   # two stages only: the planner keeps to 128
        assert (plan["pair"], plan["bn"]) == (pair, bn)


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("splits", [2, 3, 5, 8])
@pytest.mark.parametrize("bn", [32, 128])
def test_cluster_split(monkeypatch, dt, splits, bn):
    monkeypatch.setenv("NMSPMM_FORCE_SPLITK", str(splits))
    monkeypatch.setenv("NMSPMM_FORCE_BN", str(bn))
    h, _ = check_forward(dt, 37, 8 * (256 if dt == "int8" else 128), 75, save=dt != "int8", act="gelu")
    plan = nm.nm_plan_query(h, 37)
    assert plan["cluster"] == 1 and plan["splits"] > 1


def test_planner_splits_a_long_k_on_chip():
    h, _ = check_forward("int8", 16, 4096, 96)
    assert nm.nm_plan_query(h, 16)["cluster"] == 1


def test_planner_takes_the_pair_where_its_output_stage_pays():
    # half as many 256-channel x 128-token tiles as pairs: with p saved only (the
    # plan of the other calls is the one nm_plan_query reports)
    h, _ = check_forward("bf16", 300, 768, 2048, out="default", save=True)
    assert nm.nm_plan_query(h, 300)["pair"] == 0
    h, _ = check_forward("fp16", 790, 768, 2048, out="default")
    assert nm.nm_plan_query(h, 790)["pair"] == 1
    h, _ = check_forward("bf16", 301, 2048, 2056, N=4, M=8, out="default")   # an odd number of 128-row tiles
    assert nm.nm_plan_query(h, 301)["pair"] == 1
    h, _ = check_forward("bf16", 9600, 768, 64, out="default", save=True)    # one tile: half a pair
    assert nm.nm_plan_query(h, 9600)["pair"] == 0


def test_int8_output_codes():
    """Without an activation the arithmetic is fixed: the codes are exact."""
    X, W, s, b = problem("int8", 75, 256, 41, 2, 4)
    h = nm.nm_compress_gated(W.cuda(), 2, 4)
    Y = nm.nm_spmm_gated(h, X.cuda(), scale=s.cuda(), bias=b.cuda(), act="none", out="int8", out_scale=7.0)
    acc = (f64(X) @ ffn.mask(f64(W), 2, 4).T).astype(np.float32)
    p = (acc * s.numpy()).astype(np.float32) + b.numpy()
    v = (p[:, :41] * p[:, 41:]).astype(np.float32) * np.float32(7.0)
    np.testing.assert_array_equal(Y.cpu().numpy(), np.clip(np.rint(v), -128, 127).astype(np.int8))


@pytest.mark.parametrize("act", ACTS)
def test_activation_of_every_fp16_value(act):
    # p is the fp16 value itself and the up half is 1, so y is act(p) alone
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.float16)
    v = v[torch.isfinite(v)]
    X = torch.zeros((v.numel(), 64), dtype=torch.float16)
    X[:, 0], X[:, 4] = v, 1.0
    W = torch.zeros((2, 64), dtype=torch.float16)
    W[0, 0] = W[1, 4] = 1.0
    h = nm.nm_compress_gated(W.cuda(), 4, 4)
    y = f64(nm.nm_spmm_gated(h, X.cuda(), act=act, out="float32"))[:, 0]
    g, tol = act_error(f64(v), 0.0, act)
    assert (np.abs(y - g) <= tol + 1e-30).all()


def test_extreme_gates():
    """Gates far out: the activations neither overflow nor lose their limits."""
    W = torch.zeros((2, 64), dtype=torch.float16)
    W[0, 0] = W[1, 1] = 1.0
    g = torch.tensor([-60000.0, -200.0, -100.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 100.0, 200.0, 60000.0])
    X = torch.zeros((12, 64), dtype=torch.float16)
    X[:, 0] = g.to(torch.float16)
    X[:, 1] = 1.0
    h = nm.nm_compress_gated(W.cuda(), 4, 4)
    for act in ACTS:
        Y = f64(nm.nm_spmm_gated(h, X.cuda(), act=act, out="float32"))[:, 0]
        ref, e = act_error(f64(X)[:, 0], np.zeros(12), act)
        assert (np.abs(Y - ref) <= e + 2.0 ** -24 * np.abs(ref) + 1e-36).all(), act


# ------------------------------------------------------------------ gradients

def slope_error(x, act):
    d = ffn.act_slope(x, act)
    if act == "silu":
        s = 1 / (1 + np.exp(-np.clip(x, -700, 700)))
        return d, (1.5e-6 + 3e-7 * np.abs(x)) * (1 + np.abs(x)) * s + 1e-30
    if act == "gelu":
        phi = np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        cdf = np.abs(d - x * phi)
        return d, 2e-7 + (1e-6 + 1e-7 * x * x) * (cdf + np.abs(x) * phi)
    return d, np.zeros_like(d)


def dp_reference(P, dY, act):
    p, dy = f64(P), f64(dY)
    F = p.shape[1] // 2
    g, u = p[:, :F], p[:, F:]
    a, ea = act_error(g, np.zeros_like(g), act)
    d, ed = slope_error(g, act)
    dp = np.concatenate([dy * u * d, dy * a], axis=1)
    e = np.concatenate([np.abs(dy * u) * ed, np.abs(dy) * ea], axis=1) + 3 * 2.0 ** -24 * np.abs(dp)
    return dp, e


def check_backward(dt, T, k, F, N=2, M=4, act="silu", seed=0, exact_p=False):
    X, W, _, _ = problem(dt, T, k, F, N, M, seed)
    g = torch.Generator().manual_seed(seed + 9)
    P = torch.randn((T, 2 * F), generator=g).to(DTS[dt])
    dY = torch.randn((T, F), generator=g).to(DTS[dt])
    h = nm.nm_compress_gated(W.cuda(), N, M)
    guard = 64
    outs = {}
    for name, n, t in (("dX", T * k, DTS[dt]), ("dW", 2 * F * k, DTS[dt]), ("dbias", 2 * F, torch.float32)):
        outs[name] = torch.full((n + guard,), 77.0, dtype=t, device="cuda")
    ws = torch.full((nm.nm_gated_backward_workspace(h, T),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    dX, dW, db = nm.nm_gated_backward(h, X.cuda(), P.cuda(), dY.cuda(), act=act, dX=outs["dX"][:T * k].view(T, k),
                                      dW=outs["dW"][:2 * F * k].view(2 * F, k), dbias=outs["dbias"][:2 * F],
                                      workspace=ws)
    torch.cuda.synchronize()
    assert nm.nm_device_status(h) == nm.NM_OK
    for o in outs.values():
        assert bool((o[-guard:] == 77).all())
    dp, e32 = dp_reference(P, dY, act)
    w, x = ffn.mask(f64(W), N, M), f64(X)
    half = torch.finfo(DTS[dt]).eps / 2
    e16 = e32 + half * (np.abs(dp) + e32) + (2.0 ** -25 if dt == "fp16" else 0.0)

    def close(got, left, eleft, right, n):
        ref = left @ right
        tol = eleft @ np.abs(right) + (n / 8 + 4) * 2.0 ** -23 * ((np.abs(left) + eleft) @ np.abs(right))
        tol = rounded(ref, tol, DTS[dt])
        err = np.abs(f64(got) - ref)
        assert (err <= tol).all(), float((err / tol).max())

    close(dX, dp, e16, w, 2 * F)
    close(dW, dp.T, e16.T, x, T)
    ref = dp.sum(0)
    tol = e32.sum(0) + (T / 8 + 24) * 2.0 ** -24 * np.abs(dp).sum(0)
    assert (np.abs(f64(db) - ref) <= tol).all()
    return h, X, P, dY, (dX, dW, db)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("T,k,F", [(1, 8, 1), (1, 64, 24), (3, 16, 7), (63, 64, 8), (64, 72, 33), (65, 128, 64),
                                   (127, 136, 65), (129, 256, 128), (200, 264, 129), (257, 512, 255), (320, 320, 264),
                                   (1031, 96, 40)])
def test_backward_sizes(dt, T, k, F):
    check_backward(dt, T, k, F, seed=T + F)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("N,M", [(1, 4), (2, 8), (4, 8), (4, 4)])
def test_backward_activations_and_patterns(dt, act, N, M):
    check_backward(dt, 150, 192, 72, N, M, act=act, seed=3)


@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("T,k,F", [(2500, 768, 700), (300, 1024, 2600), (130, 200, 96)])
def test_backward_many_tiles(monkeypatch, T, k, F, bn):
    """More tiles than CTA pairs, each product in turn the one with the longer sums; both tile widths."""
    monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", str(bn))
    check_backward("bf16", T, k, F, act="gelu", seed=1)


@pytest.mark.parametrize("bn", [128, 256])
@pytest.mark.parametrize("T,k,F", [(200, 264, 1030), (3000, 64, 40), (1500, 136, 700), (1, 512, 2048)])
def test_backward_split_sums(monkeypatch, T, k, F, bn):
    """Few tiles with long sums: parts of a tile's sum on several pairs, the same result every time."""
    monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", str(bn))
    h, X, P, dY, (dX, dW, db) = check_backward("bf16", T, k, F, seed=T)
    for _ in range(10):
        x, w, b = nm.nm_gated_backward(h, X.cuda(), P.cuda(), dY.cuda(), bias_grad=True)
        assert torch.equal(x, dX) and torch.equal(w, dW) and torch.equal(b, db)
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", "0")
    check_backward("bf16", T, k, F, seed=T)


def test_backward_parts_and_repeats():
    h, X, P, dY, (dX, dW, db) = check_backward("bf16", 333, 264, 100, seed=5)
    L, T = nm.lib(), 333
    ws = torch.empty(nm.nm_gated_backward_workspace(h, T), dtype=torch.uint8, device="cuda")
    Xc, Pc, dYc = X.cuda(), P.cuda(), dY.cuda()
    for which in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1), (1, 1, 1)):
        got = [torch.full_like(t, 3.0) for t in (dX, dW, db)]
        ptr = [t.data_ptr() if on else None for t, on in zip(got, which)]
        assert L.nm_gated_backward(h.raw, Xc.data_ptr() if which[1] else None, Pc.data_ptr(), dYc.data_ptr(), T, 2, *ptr,
                                   ws.data_ptr(), ws.numel(), None) == nm.NM_OK
        torch.cuda.synchronize()
        for t, want, on in zip(got, (dX, dW, db), which):
            assert torch.equal(t, want) if on else bool((t == 3.0).all())


def test_backward_agrees_with_differences():
    """Inputs chosen so that p is exact in fp16; the directional derivatives of the
    64-bit loss against the GPU's gradients, within the gradients' own bound."""
    T, k, F = 24, 32, 12
    g = torch.Generator().manual_seed(2)
    X = (torch.randint(-4, 5, (T, k), generator=g) / 4).half()
    W = (torch.randint(-4, 5, (2 * F, k), generator=g) / 8).half()
    b = (torch.randint(-8, 9, (2 * F,), generator=g) / 16).float()
    dY = torch.randn((T, F), generator=g).half()
    h = nm.nm_compress_gated(W.cuda(), 2, 4)
    P = torch.empty((T, 2 * F), dtype=torch.float16, device="cuda")
    for act in ("silu", "gelu", "none"):
        nm.nm_spmm_gated(h, X.cuda(), P=P, bias=b.cuda(), act=act)
        x, w, bb, dy = f64(X), ffn.mask(f64(W), 2, 4), f64(b), f64(dY)
        np.testing.assert_array_equal(f64(P), ffn.gated_pre(x, w, bias=bb))
        grads = nm.nm_gated_backward(h, X.cuda(), P, dY.cuda(), act=act, bias_grad=True)
        dp, e = dp_reference(P, dY, act)
        e16 = e + 2.0 ** -11 * np.abs(dp) + 2.0 ** -25
        loss = lambda x, w, bb: float((ffn.gated(ffn.gated_pre(x, w, bias=bb), act) * dy).sum())  # noqa: E731
        rng = np.random.default_rng(7)
        tols = (e16 @ np.abs(w) + 1e-5 * (np.abs(dp) @ np.abs(w)), e16.T @ np.abs(x) + 1e-5 * (np.abs(dp).T @ np.abs(x)),
                e.sum(0) + 1e-5 * np.abs(dp).sum(0))
        for i in range(3):
            args = [x, w, bb]
            d = rng.standard_normal(args[i].shape)
            hi, lo = list(args), list(args)
            hi[i], lo[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
            got = f64(grads[i])
            tol = (tols[i] * np.abs(d)).sum() + (2.0 ** -11 * np.abs(got * d)).sum() + 1e-6
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (got * d).sum()) <= tol


def test_empty_batch():
    W = torch.randn((48, 64), device="cuda").bfloat16()
    h = nm.nm_compress_gated(W, 2, 4)
    e = lambda n: torch.empty((0, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert nm.nm_spmm_gated(h, e(64), P=e(48)).shape == (0, 24)
    dX, dW, db = nm.nm_gated_backward(h, e(64), e(48), e(24), bias_grad=True)
    assert dX.shape == (0, 64) and not dW.any() and not db.any()


def test_training_step_captured():
    """Forward, backward, weight update and re-pack in one captured step, replayed on new batches."""
    T, k, F = 150, 128, 80
    X, W, _, b = problem("bf16", T, k, F, 2, 4, seed=4)
    W, b = W.cuda(), b.cuda()
    x, dy = X.cuda().clone(), torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    h = nm.nm_compress_gated(W, 2, 4)
    P = torch.empty((T, 2 * F), dtype=torch.bfloat16, device="cuda")

    def step(h, w):
        Y = nm.nm_spmm_gated(h, x, P=P, bias=b)
        dX, dW, db = nm.nm_gated_backward(h, x, P, dy, bias_grad=True)
        w.add_(dW, alpha=-0.125)
        nm.nm_recompress(h, w)
        return Y, dX, dW, db

    w0 = W.clone()
    dy.normal_()
    step(nm.nm_compress_gated(w0, 2, 4), w0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(h, W)
    nm.nm_recompress(h, W)
    h2, w2 = nm.nm_compress_gated(W, 2, 4), W.clone()
    for seed in (5, 6):
        x.copy_(problem("bf16", T, k, F, 2, 4, seed=seed)[0])
        dy.normal_()
        graph.replay()
        got = [t.clone() for t in out]
        want = step(h2, w2)
        for a, c in zip(got, want):
            assert torch.equal(a, c)
        assert torch.equal(W, w2)


def test_two_streams_share_a_handle():
    W = torch.randn((512, 256), device="cuda").bfloat16()
    h = nm.nm_compress_gated(W, 2, 4)
    xs = [torch.randn((t, 256), device="cuda").bfloat16() for t in (100, 1500)]
    want = [nm.nm_spmm_gated(h, x) for x in xs]
    ps = [torch.randn((x.shape[0], 512), device="cuda").bfloat16() for x in xs]
    grads = [nm.nm_gated_backward(h, x, p, y) for x, p, y in zip(xs, ps, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        ys = [nm.nm_spmm_gated(h, x, stream=s) for x, s in zip(xs, streams)]
        gs = [nm.nm_gated_backward(h, x, p, y, stream=s) for x, p, y, s in zip(xs, ps, ys, streams)]
        torch.cuda.synchronize()
        for a, c in zip(ys, want):
            assert torch.equal(a, c)
        for a, c in zip(gs, grads):
            assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


def test_far_rows_match_a_small_call(monkeypatch):
    """Element offsets past 2^31 in p and dp."""
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", "0")     # the same order of sums in both calls
    T, k, F, tail = 140_011, 64, 8192, 130
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((T, k), generator=g, device="cuda").bfloat16()
    W = torch.randn((2 * F, k), generator=g, device="cuda").bfloat16()
    h = nm.nm_compress_gated(W, 2, 4)
    P = torch.empty((T, 2 * F), dtype=torch.bfloat16, device="cuda")
    Y = nm.nm_spmm_gated(h, X, P=P)
    p = torch.empty((tail, 2 * F), dtype=torch.bfloat16, device="cuda")
    y = nm.nm_spmm_gated(h, X[-tail:].contiguous(), P=p)
    # the two calls' plans differ (token tiles, cluster splits), so their sums may, by the
    # bound of the header on either side; then a step of bf16 (2^-7) apart, and for
    # y = silu(g) u what those differences make of it (|silu'| < 1.1, |silu(g)| <= |g|)
    e = 2 * (k / 8 + 4) * 2.0 ** -23 * (X[-tail:].float().abs() @ W.float().abs().t())
    gate, up = p[:, :F].float().abs(), p[:, F:].float().abs()
    assert bool(((P[-tail:].float() - p.float()).abs() <= e + 2.0 ** -7 * (p.float().abs() + e)).all())
    ey = 1.1 * e[:, :F] * (1.01 * up + e[:, F:]) + (1.01 * gate + e[:, :F]) * e[:, F:]
    assert bool(((Y[-tail:].float() - y.float()).abs() <= ey + 2.0 ** -7 * (y.float().abs() + ey)).all())
    dX, dW, db = nm.nm_gated_backward(h, X, P, Y, bias_grad=True)
    small = nm.nm_gated_backward(h, X[-tail:].contiguous(), P[-tail:].contiguous(), Y[-tail:].contiguous())
    assert torch.equal(dX[-tail:], small[0])
    # dW and dbias are sums over T: halves of the batch add up to the whole
    half = 70_016
    parts = [nm.nm_gated_backward(h, X[r].contiguous(), P[r].contiguous(), Y[r].contiguous(), bias_grad=True)
             for r in (slice(0, half), slice(half, T))]
    for i, whole in ((1, dW), (2, db)):
        a, b = parts[0][i].double(), parts[1][i].double()
        assert float((a + b - whole.double()).norm() / whole.double().norm()) < (1e-2 if i == 1 else 1e-5)


def test_host_threads_share_a_handle():
    import threading
    W = torch.randn((512, 256), device="cuda").bfloat16()
    h = nm.nm_compress_gated(W, 2, 4)
    xs = [torch.randn((t, 256), device="cuda").bfloat16() for t in (20, 300, 1500)]

    def block(x):
        p = torch.empty((x.shape[0], 512), dtype=torch.bfloat16, device="cuda")
        y = nm.nm_spmm_gated(h, x, P=p)
        return (y, p) + nm.nm_gated_backward(h, x, p, y, bias_grad=True)

    want = [block(x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = block(xs[i])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_refusals_on_a_handle(monkeypatch):
    W8 = torch.randint(-127, 128, (64, 64), dtype=torch.int8).cuda()
    h8, plain = nm.nm_compress_gated(W8, 2, 4), nm.nm_compress(W8, 2, 4)
    Wb = torch.randn((64, 64), device="cuda").bfloat16()
    hb = nm.nm_compress_gated(Wb, 2, 4)
    X8, Xb = torch.zeros((8, 64), dtype=torch.int8, device="cuda"), torch.zeros((8, 64), device="cuda").bfloat16()

    def status(f, *a, **kw):
        with pytest.raises(nm.NMError) as e:
            f(*a, **kw)
        return e.value.status

    assert status(nm.nm_spmm_gated, plain, X8, Y=torch.empty((8, 32), device="cuda")) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm, h8, X8) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_ex, hb, Xb) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_gated, hb, Xb, out="int8") == nm.NM_ERR_UNSUPPORTED
    assert status(nm.nm_spmm_gated, h8, X8, out="int32") == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_gated, h8, X8, out="int8", out_scale=-1.0) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_gated, h8, X8, P=torch.empty((8, 64), dtype=torch.int8, device="cuda")) \
        == nm.NM_ERR_UNSUPPORTED
    assert status(nm.nm_gated_backward_workspace, h8, 8) == nm.NM_ERR_UNSUPPORTED
    assert status(nm.nm_gated_backward_workspace, plain, 8) == nm.NM_ERR_INVALID
    assert status(nm.nm_gated_backward_workspace, hb, -1) == nm.NM_ERR_INVALID
    monkeypatch.setenv("NMSPMM_FORCE_SPLITK", "2")
    monkeypatch.setenv("NMSPMM_SPLIT_GLOBAL", "1")
    Wl = torch.randn((64, 512), device="cuda").bfloat16()
    hl = nm.nm_compress_gated(Wl, 2, 4)
    assert status(nm.nm_spmm_gated, hl, torch.zeros((8, 512), device="cuda").bfloat16()) == nm.NM_ERR_UNSUPPORTED

    L = nm.lib()
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    o = buf.data_ptr()
    x, p, dy, dx, dw, ws, n = o, o + 8192, o + 16384, o + 32768, o + 65536, o + 131072, 1 << 19
    back = lambda *a: L.nm_gated_backward(hb.raw, *a, None)  # noqa: E731
    need = nm.nm_gated_backward_workspace(hb, 8)
    assert back(x, p, dy, 8, 2, None, None, None, ws, n) == nm.NM_ERR_INVALID        # nothing to compute
    assert back(x, p, dy, 8, 7, dx, dw, None, ws, n) == nm.NM_ERR_INVALID            # unknown activation
    assert back(x, p, dy, -1, 2, dx, dw, None, ws, n) == nm.NM_ERR_INVALID
    assert back(x, p, dy, (1 << 26) + 1, 2, dx, dw, None, ws, n) == nm.NM_ERR_UNSUPPORTED
    assert back(x, p, dy, 8, 2, dx, dw, None, ws, need - 1) == nm.NM_ERR_INVALID     # workspace too small
    assert back(x, p, dy, 8, 2, dx, dw, None, None, n) == nm.NM_ERR_INVALID
    assert back(None, p, dy, 8, 2, dx, dw, None, ws, n) == nm.NM_ERR_INVALID
    assert back(x, None, dy, 8, 2, dx, dw, None, ws, n) == nm.NM_ERR_INVALID
    assert back(x, p, None, 8, 2, dx, dw, None, ws, n) == nm.NM_ERR_INVALID
    assert back(x + 8, p, dy, 8, 2, dx, dw, None, ws, n) == nm.NM_ERR_INVALID        # misaligned
    assert back(x, p, dy, 8, 2, p, dw, None, ws, n) == nm.NM_ERR_INVALID             # dX over P
    assert back(x, p, dy, 8, 2, dx, dx, None, ws, n) == nm.NM_ERR_INVALID            # dW over dX
    assert back(x, p, dy, 8, 2, dx, dw, None, o, n) == nm.NM_ERR_INVALID             # workspace over everything
    fw = lambda *a: L.nm_spmm_gated(hb.raw, *a, None, None)  # noqa: E731
    assert fw(x, -1, dx, None) == nm.NM_ERR_INVALID
    assert fw(x, 1 << 31, dx, None) == nm.NM_ERR_UNSUPPORTED
    assert fw(x, (1 << 31) - 255, dx, None) == nm.NM_ERR_UNSUPPORTED                 # the last tile's end
    assert fw(None, 8, dx, None) == nm.NM_ERR_INVALID
    assert fw(x, 8, x, None) == nm.NM_ERR_INVALID                                    # Y over X
    assert fw(x, 8, dx, dx) == nm.NM_ERR_INVALID                                     # P over Y
    assert fw(x, 8, dx, p + 8) == nm.NM_ERR_INVALID
    Wk = torch.randn((8, 12), device="cuda").bfloat16()
    hk = nm.nm_compress_gated(Wk, 2, 4)                                              # k off a 16-byte row
    assert L.nm_spmm_gated(hk.raw, x, 8, dx, None, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_gated_backward(hk.raw, x, p, dy, 8, 2, dx, dw, None, ws, n, None) == nm.NM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        nm.nm_spmm_gated(hb, Xb, act="tanh")
    with pytest.raises(ValueError):
        nm.nm_spmm_gated(hb, Xb, bias=torch.zeros(32, device="cuda"))
    with pytest.raises(ValueError):
        nm.nm_gated_backward(hb, Xb, Xb, Xb)
