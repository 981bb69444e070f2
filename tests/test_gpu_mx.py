"""Microscaled 4-bit floating point on the GPU: quantisation and the values back
bit for bit against the oracle, the products within a derived bound.

Bound of a product, per element, against 64 bits.  Every product of two 4-bit
values and its scale is exact in fp32; the tensor core adds the 32-blocks of a
row in some order into an fp32 sum, so each of the k / 32 additions (and the few
that combine them) is off by at most one unit in the last place of a partial
sum, which the sum of magnitudes A = sum |x||w| bounds:
    e_acc = (k / 32 + 4) 2^-23 A.
The output stage rounds once per step (half a unit, 2^-24 relative): scale s and
bias b give |s| e_acc + 2^-24 (|s| A + |p|) in all for p; GELU and SiLU change a
value by at most 1.13 and 1.1 times as much and add their own error (GELU 4e-7
|p| + 2e-6 |g|, SiLU (6e-7 + 1.3e-7 max(0, -p)) |g|); a gated product y = a u is off by
|u| e_a + |a| e_u + e_a e_u + 2^-24 |y|; the output type adds half a unit,
finfo.eps / 2 relative (fp16 also half its smallest subnormal).
"""
import numpy as np
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm
from oracle import ffn

pytestmark = pytest.mark.gpu

DTS = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def act_error(p, e, name):
    g = ffn.act(p, name)
    if name == "gelu":
        return g, 1.13 * e + 4e-7 * np.abs(p) + 2e-6 * np.abs(g)
    if name == "silu":
        return g, 1.1 * e + (6e-7 + 1.3e-7 * np.maximum(0, -p)) * np.abs(g) + 1e-36
    return g, e


def rounded(y, e, dt):
    half = torch.finfo(dt).eps / 2
    return e + half * (np.abs(y) + e) + (2.0 ** -25 if dt == torch.float16 else 0.0)


def pre_activation(X, W, scale, bias, per_sum=32):
    """p and its error bound in 64 bits."""
    p, A, k = X @ W.T, np.abs(X) @ np.abs(W).T, X.shape[1]
    e = (k / per_sum + 4) * 2.0 ** -23 * A
    if scale is not None:
        p, A, e = p * scale, A * np.abs(scale), e * np.abs(scale)
        e = e + 2.0 ** -24 * A
    if bias is not None:
        p = p + bias
        e = e + 2.0 ** -24 * (np.abs(p) + e)
    return p, e


def product_reference(X, W, scale, bias, act, gated, dt):
    p, e = pre_activation(X, W, scale, bias)
    if not gated:
        y, e = act_error(p, e, act)
        return y, rounded(y, e, dt)
    f = p.shape[1] // 2
    a, ea = act_error(p[:, :f], e[:, :f], act)
    u, eu = p[:, f:], e[:, f:]
    y = a * u
    e = np.abs(u) * ea + np.abs(a) * eu + ea * eu + 2.0 ** -24 * np.abs(y)
    return y, rounded(y, e, dt)


def make(rows, k, dt, seed, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k), generator=g, dtype=torch.float64)
    if spread:
        x *= 2.0 ** torch.randint(-spread, spread + 1, (rows, k // 32, 1), generator=g).expand(-1, -1, 32).reshape(
            rows, k)
    return x.to(dt)


def check_quantised(x, Q, S):
    codes, byte = ffn.mx_quantize(f64(x))
    np.testing.assert_array_equal(Q.cpu().numpy(), ffn.mx_pack_codes(codes))
    np.testing.assert_array_equal(S.cpu().numpy(), ffn.mx_pack_scales(byte))
    return ffn.mx_values(codes, byte)


@pytest.mark.parametrize("T,k", [(1, 32), (1, 64), (3, 96), (31, 128), (127, 160), (128, 256), (129, 288), (257, 544),
                                 (5, 2080)])
@pytest.mark.parametrize("dt", list(DTS))
def test_quantise_bit_exact(dt, T, k):
    x = make(T, k, DTS[dt], seed=T + k, spread=6)
    x[T // 2, :32] = 0
    Q = torch.full((T, k // 2), 0xAB, dtype=torch.uint8, device="cuda")
    S = torch.full((nm.nm_mx_scale_bytes(T, k),), 0xCD, dtype=torch.uint8, device="cuda")
    assert nm.nm_mx_quantize(x.cuda(), Q=Q, S=S)[0] is Q
    v = check_quantised(x, Q, S)
    for out in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(f64(nm.nm_mx_dequantize(Q, S, dtype=out)), v)
    np.testing.assert_array_equal(nm.nm_mx_dequantize(Q, S, dtype=torch.float16).cpu().numpy(),
                                  v.astype(np.float16))


@pytest.mark.parametrize("dt", list(DTS))
def test_quantise_edges(dt):
    """Ties, subnormals, the largest values, infinities, NaN, signed zeros."""
    t = DTS[dt]
    fi = torch.finfo(t)
    x = torch.zeros((9, 64), dtype=t)
    x[0, :13] = torch.tensor([7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -2.5, -5.0, -0.0]).to(t)
    x[1, :4] = torch.tensor([fi.max, -fi.max, fi.max / 2, fi.tiny]).to(t)
    x[2, 0] = fi.smallest_normal
    x[2, 1] = fi.smallest_normal / 2            # subnormals
    x[3, 5] = fi.smallest_normal / 4
    x[3, 6] = -fi.smallest_normal / 8
    x[4, 1] = float("inf")
    x[4, 40] = 3.0                              # the other block of the row is untouched
    x[5, 33] = float("nan")
    x[5, 0] = 1.0
    x[6, 2] = -float("inf")
    x[7, :32] = 6.0
    x[8, :32] = torch.linspace(-8, 8, 32).to(t)
    Q, S = nm.nm_mx_quantize(x.cuda())
    v = check_quantised(x, Q, S)
    np.testing.assert_array_equal(f64(nm.nm_mx_dequantize(Q, S, dtype=torch.float32)), v)


def test_quantise_row_stride_and_offset():
    big = make(200, 512, torch.bfloat16, seed=1).cuda()
    x = big[3:150, 64:64 + 288]                 # rows 1024 bytes apart, starting 128 bytes in
    Q, S = nm.nm_mx_quantize(x)
    check_quantised(x, Q, S)
    with pytest.raises(nm.NMError) as e:
        nm.nm_mx_quantize(big[:, 4:36])         # starts off a 16-byte boundary
    assert e.value.status == nm.NM_ERR_INVALID


def test_dequantise_every_code_and_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    byte = np.arange(256, dtype=np.uint8)[:, None]
    Q = torch.from_numpy(ffn.mx_pack_codes(codes)).cuda()
    S = torch.from_numpy(ffn.mx_pack_scales(byte)).cuda()
    v = ffn.mx_values(codes, byte)
    big = np.abs(v[253:255]) > np.finfo(np.float32).max     # beyond fp32: infinite in all three types
    v[253:255][big] = np.copysign(np.inf, v[253:255][big])
    got = nm.nm_mx_dequantize(Q, S, dtype=torch.float32)
    np.testing.assert_array_equal(f64(got), v)
    np.testing.assert_array_equal(f64(nm.nm_mx_dequantize(Q, S)), f64(got.to(torch.bfloat16)))
    np.testing.assert_array_equal(f64(nm.nm_mx_dequantize(Q, S, dtype=torch.float16)), f64(got.to(torch.float16)))


def test_far_rows_match_a_small_call():
    """Element offsets past 2^31 in the activation, its codes' values and the output."""
    T, k, n, tail = 4_300_033, 512, 512, 161
    x = torch.empty((T, k), dtype=torch.bfloat16, device="cuda")
    x[-tail:].normal_()
    x[:-tail] = x[-tail]
    start = (T - tail) // 128 * 128             # the small call's rows start on a scale tile
    small = x[start:].clone()
    Q, S = nm.nm_mx_quantize(x)
    q, s = nm.nm_mx_quantize(small)
    assert torch.equal(Q[start:], q) and torch.equal(S.view(-1, 2048)[start // 128:].reshape(-1), s)
    nm.nm_mx_dequantize(Q, S, X=x)
    assert torch.equal(x[start:], nm.nm_mx_dequantize(q, s))
    W = make(n, k, torch.bfloat16, 3).cuda()
    h = nm.nm_compress_mx(W)
    Y = nm.nm_spmm_mx(h, Q, S, Y=x)             # the values are not needed any more
    assert torch.equal(Y[start:], nm.nm_spmm_mx(h, q, s))
    assert torch.equal(Y[0], Y[1_000_000])      # equal rows in, equal rows out
    hg = nm.nm_compress_mx(W, gated=True)
    Yg = nm.nm_spmm_mx_gated(hg, Q, S, out="float32")
    assert torch.equal(Yg[start:], nm.nm_spmm_mx_gated(hg, q, s, out="float32"))


def test_host_threads_share_a_handle():
    import threading
    W = make(512, 512, torch.bfloat16, 5).cuda()
    h = nm.nm_compress_mx(W)
    xs = [make(t, 512, torch.bfloat16, 6 + t).cuda() for t in (33, 700, 1300)]
    want = [nm.nm_spmm_mx(h, *nm.nm_mx_quantize(x)) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                y = nm.nm_spmm_mx(h, *nm.nm_mx_quantize(xs[i]))
                s.synchronize()
                if not torch.equal(y, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("N,M", [(1, 4), (2, 4), (2, 8), (4, 8), (4, 4), (8, 8)])
@pytest.mark.parametrize("dt", list(DTS))
def test_compress_mx_values(dt, N, M):
    W = make(37, 96, DTS[dt], seed=N * 8 + M, spread=3)
    W[0, :8] = 1.0                              # ties: the lower positions stay
    W[1] = 0
    h = nm.nm_compress_mx(W.cuda(), N, M)
    ref = lambda w: ffn.mx_values(*ffn.mx_quantize(ffn.mask(f64(w), N, M)))  # noqa: E731
    np.testing.assert_array_equal(f64(nm.nm_decompress(h)), ref(W))
    W2 = make(37, 96, DTS[dt], seed=99)
    nm.nm_recompress(h, W2.cuda())
    np.testing.assert_array_equal(f64(nm.nm_decompress(h)), ref(W2))
    assert nm.nm_query(h) == {"n_out": 37, "k": 96, "N": N, "M": M, "dtype": nm.NM_MXFP4}


@pytest.mark.parametrize("F", [1, 15, 16, 17, 40])
def test_compress_mx_gated_keeps_row_order(F):
    W = make(2 * F, 64, torch.bfloat16, seed=F)
    h = nm.nm_compress_mx(W.cuda(), 2, 4, gated=True)
    np.testing.assert_array_equal(f64(nm.nm_decompress(h)), ffn.mx_values(*ffn.mx_quantize(ffn.mask(f64(W), 2, 4))))


def run_product(T, k, n, dt="bf16", out="float32", act="none", scale=False, bias=False, gated=False, NM=(4, 4), seed=0):
    X, W = make(T, k, DTS[dt], seed + 1, spread=2), make(n, k, DTS[dt], seed + 2, spread=2)
    g = torch.Generator().manual_seed(seed + 3)
    s = torch.rand(n, generator=g) * 0.05 if scale else None
    b = torch.randn(n, generator=g) if bias else None
    h = nm.nm_compress_mx(W.cuda(), *NM, gated=gated)
    Q, S = nm.nm_mx_quantize(X.cuda())
    odt = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16, "default": DTS[dt]}[out]
    cols = n // 2 if gated else n
    buf = torch.full((T + 2, cols), 77.0, dtype=odt, device="cuda")
    call = nm.nm_spmm_mx_gated if gated else nm.nm_spmm_mx
    al = (T * cols * buf.element_size()) % 16
    Y = buf.view(-1)[:T * cols].view(T, cols)
    call(h, Q, S, Y=Y, scale=None if s is None else s.cuda(), bias=None if b is None else b.cuda(), act=act, out=out)
    torch.cuda.synchronize()
    assert nm.nm_device_status(h) == nm.NM_OK and al >= 0
    assert bool((buf.view(-1)[T * cols:] == 77).all())          # nothing behind the last row
    ref, tol = product_reference(ffn.mx_values(*ffn.mx_quantize(f64(X))),
                                 ffn.mx_values(*ffn.mx_quantize(ffn.mask(f64(W), *NM))),
                                 None if s is None else f64(s), None if b is None else f64(b), act, gated, odt)
    err = np.abs(f64(Y) - ref)
    assert (err <= tol).all(), (T, k, n, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("T,k,n", [
    (1, 32, 1), (1, 64, 8), (2, 96, 7), (31, 128, 33), (127, 160, 64), (128, 256, 65), (129, 288, 127), (255, 64, 129),
    (256, 512, 191), (257, 544, 193), (300, 768, 200), (5, 2080, 385), (513, 96, 1001), (1, 1056, 640),
])
def test_product_sizes(T, k, n):
    run_product(T, k, n, seed=T + n)


@pytest.mark.parametrize("bn", [64, 128, 192])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [512, 514, 1030])
def test_every_tile_width(monkeypatch, n, out, gated, bn):
    """Tiles that start anywhere in a scale tile; several tiles per CTA pair in the last case."""
    monkeypatch.setenv("NMSPMM_FORCE_MX_BN", str(bn))
    run_product(300, 288, n, out=out, act="gelu", bias=True, gated=gated, seed=n)


@pytest.mark.parametrize("out", ["float32", "float16", "bfloat16", "default"])
@pytest.mark.parametrize("scale,bias,act", [(False, False, "none"), (True, False, "gelu"), (False, True, "none"),
                                            (True, True, "gelu")])
@pytest.mark.parametrize("n", [200, 203])       # tensor stores, plain stores
def test_product_output_stage(out, scale, bias, act, n):
    run_product(140, 320, n, dt="fp16", out=out, act=act, scale=scale, bias=bias, NM=(2, 4), seed=5)


@pytest.mark.parametrize("T,k,F", [(1, 32, 1), (3, 64, 15), (130, 96, 16), (129, 288, 17), (200, 256, 96), (257, 320, 97),
                                   (64, 800, 500)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu", "relu"])
def test_gated_product(T, k, F, act):
    run_product(T, k, 2 * F, act=act, gated=True, bias=True, scale=F % 2 == 0, out="float32", seed=F)


@pytest.mark.parametrize("out", ["float16", "bfloat16", "default"])
@pytest.mark.parametrize("F", [64, 72, 75])
def test_gated_product_types(out, F):
    run_product(135, 160, 2 * F, dt="fp32", act="silu", gated=True, out=out, NM=(4, 8), seed=F)


def test_not_a_number_stays_in_its_row():
    X = make(140, 96, torch.bfloat16, 1)
    W = make(70, 96, torch.bfloat16, 2).cuda()
    h = nm.nm_compress_mx(W)
    clean = nm.nm_spmm_mx(h, *nm.nm_mx_quantize(X.cuda()))
    X[17, 40] = float("inf")
    X[139, 3] = float("nan")
    Y = nm.nm_spmm_mx(h, *nm.nm_mx_quantize(X.cuda()))
    keep = [t for t in range(140) if t not in (17, 139)]
    assert torch.equal(Y[keep], clean[keep])
    assert bool(Y[17].isnan().all()) and bool(Y[139].isnan().all())


def test_large_product_sampled():
    T, k, n = 6304, 1024, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((T, k), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((n, k), generator=g, device="cuda").to(torch.bfloat16)
    h = nm.nm_compress_mx(W)
    Q, S = nm.nm_mx_quantize(X)
    Y = nm.nm_spmm_mx(h, Q, S, out="float32")
    x, w = nm.nm_mx_dequantize(Q, S, dtype=torch.float32).double(), nm.nm_decompress(h).double()
    err = (Y.double() - x @ w.t()).abs()
    assert bool((err <= (k / 32 + 4) * 2.0 ** -23 * (x.abs() @ w.abs().t()) + 2.0 ** -24 * Y.abs()).all())


def test_repeated_calls_agree_and_empty_calls_do_nothing():
    W = make(300, 256, torch.bfloat16, 3).cuda()
    h = nm.nm_compress_mx(W)
    Q, S = nm.nm_mx_quantize(make(900, 256, torch.bfloat16, 4).cuda())
    Y = nm.nm_spmm_mx(h, Q, S)
    for _ in range(20):
        assert torch.equal(nm.nm_spmm_mx(h, Q, S), Y)
    Q0, S0 = nm.nm_mx_quantize(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert nm.nm_spmm_mx(h, Q0, S0).shape == (0, 300)
    assert nm.nm_mx_dequantize(Q0, S0).shape == (0, 256)


def test_two_streams_share_a_handle():
    W = make(512, 512, torch.bfloat16, 5).cuda()
    h = nm.nm_compress_mx(W)
    xs = [make(t, 512, torch.bfloat16, 6 + t).cuda() for t in (700, 1300)]
    want = [nm.nm_spmm_mx(h, *nm.nm_mx_quantize(x)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for x, s in zip(xs, streams):
            Q, S = nm.nm_mx_quantize(x, stream=s)
            got.append(nm.nm_spmm_mx(h, Q, S, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured_feed_forward_block():
    """quantise, gated product, quantise, product, captured once and replayed on new inputs."""
    k, F, T = 256, 320, 197
    Wgu, Wd = make(2 * F, k, torch.bfloat16, 1).cuda(), make(k, F, torch.bfloat16, 2).cuda()
    hg, hd = nm.nm_compress_mx(Wgu, 2, 4, gated=True), nm.nm_compress_mx(Wd)
    X = torch.zeros((T, k), dtype=torch.bfloat16, device="cuda")

    def block():
        Y = nm.nm_spmm_mx_gated(hg, *nm.nm_mx_quantize(X))
        return nm.nm_spmm_mx(hd, *nm.nm_mx_quantize(Y), out="float32")

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for seed in (3, 4):
        X.copy_(make(T, k, torch.bfloat16, seed))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, block())
        # the second product against 64 bits, from the gated values as the first product gave them
        Y = nm.nm_spmm_mx_gated(hg, *nm.nm_mx_quantize(X))
        y = ffn.mx_values(*ffn.mx_quantize(f64(Y)))
        ref, tol = product_reference(y, f64(nm.nm_decompress(hd)), None, None, "none", False, torch.float32)
        assert (np.abs(f64(got) - ref) <= tol).all()


def test_refusals_on_a_handle():
    W = make(64, 64, torch.bfloat16, 1).cuda()
    h, hg = nm.nm_compress_mx(W), nm.nm_compress_mx(W, gated=True)
    plain = nm.nm_compress(W, 2, 4)
    X = make(8, 64, torch.bfloat16, 2).cuda()
    Q, S = nm.nm_mx_quantize(X)

    def status(f, *a, **kw):
        with pytest.raises(nm.NMError) as e:
            f(*a, **kw)
        return e.value.status

    assert status(nm.nm_spmm_mx, hg, Q, S) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_mx_gated, h, Q, S) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_mx, plain, Q, S) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_mx, h, Q, S, act="silu") == nm.NM_ERR_UNSUPPORTED
    assert status(nm.nm_spmm_mx, h, Q, S, out="int8") == nm.NM_ERR_UNSUPPORTED
    assert status(nm.nm_spmm, h, X) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_ex, h, X) == nm.NM_ERR_INVALID
    assert status(nm.nm_export_sizes, h) == nm.NM_ERR_INVALID
    assert status(nm.nm_plan_query, h, 8) == nm.NM_ERR_INVALID
    assert status(nm.nm_spmm_ex, plain, X, act="silu") == nm.NM_ERR_UNSUPPORTED
    L = nm.lib()
    y = torch.empty(8 * 64 * 4, dtype=torch.uint8, device="cuda")
    q, s, o = Q.data_ptr(), S.data_ptr(), y.data_ptr()
    assert L.nm_spmm_mx(h.raw, q, s, -1, o, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_mx(h.raw, None, s, 8, o, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_mx(h.raw, q, s, 8, o + 8, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_mx(h.raw, q, s, 8, q, None, None) == nm.NM_ERR_INVALID
    assert L.nm_spmm_mx(h.raw, q, s, 1 << 31, o, None, None) == nm.NM_ERR_UNSUPPORTED
    ep = nm.NMEpilogue(0, 7, None, None, 1.0)
    import ctypes
    assert L.nm_spmm_mx(h.raw, q, s, 8, o, ctypes.byref(ep), None) == nm.NM_ERR_INVALID
    for bad in (dict(Q=Q[:, :16]), dict(S=S[:512])):
        with pytest.raises(ValueError):
            nm.nm_spmm_mx(h, **{"Q": Q, "S": S, **bad})
    with pytest.raises(ValueError):
        nm.nm_spmm_mx(h, Q, S, scale=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        nm.nm_recompress(h, W.float())
