"""Inputs that the kernel just before wrote.

The library's kernels are launched with programmatic stream serialization, so one may
be resident while the kernel that writes its scale, bias or weight image still runs.
None of them may therefore read global memory through the non-coherent path, whose
data has to be read-only for the reading kernel's lifetime (CPU: the sources), and
each sees the values of the call before it (GPU)."""
import os
import re

import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm

CSRC = os.path.join(os.path.dirname(os.path.abspath(nm.__file__)), "csrc")
# what kernels launched by launch_pdl are made of
PDL_SOURCES = ("nm_spmm_kernels.cuh", "nm_spmm.cu", "nm_gated.cu", "nm_grad.cu", "nm_mx.cu", "nm_unpack.cuh", "nm_act.cuh",
               "nm_stage.cuh", "nm_device.cuh")


def code(name):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", PDL_SOURCES)
def test_no_non_coherent_loads(name):
    assert not re.search(r"__ldg\s*\(|\.nc\b", code(name))


def test_packed_image_is_read_through_coherent_loads():
    # plain loads through a const __restrict__ pointer may become non-coherent ones
    body = code("nm_unpack.cuh").split("unpack_unit", 1)[1]
    assert "__restrict__ bpack" in body
    assert not re.search(r"(?<!ld_coherent\()\*?reinterpret_cast<const[^>]*>\(chunk", body)


def products(monkeypatch):
    """name -> (vector length, product taking a bias vector)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((40, 1024), generator=g, device="cuda").half()
    W = torch.randn((256, 1024), generator=g, device="cuda").half()
    hx, hg = nm.nm_compress(W, 2, 4), nm.nm_compress_gated(W, 2, 4)
    hm, hmg = nm.nm_compress_mx(W), nm.nm_compress_mx(W, gated=True)
    ht, Xt = nm.nm_compress_tile(W, 2, 8), X.t().contiguous()
    QS = nm.nm_mx_quantize(X)

    def forced(call, **env):
        def run(b):
            for k, v in env.items():
                monkeypatch.setenv(k, v)
            y = call(b)
            for k in env:
                monkeypatch.delenv(k)
            return y
        return run

    ex = lambda b: nm.nm_spmm_ex(hx, X, bias=b, act="gelu", out="float32")  # noqa: E731
    gated = lambda b: nm.nm_spmm_gated(hg, X, bias=b, out="float32")        # noqa: E731
    one, pair, split = {"NMSPMM_FORCE_PAIR": "0", "NMSPMM_FORCE_BN": "32", "NMSPMM_CSPLIT": "0"}, {
        "NMSPMM_FORCE_PAIR": "1"}, {"NMSPMM_FORCE_SPLITK": "4", "NMSPMM_FORCE_BN": "32"}
    return {
        "ex": forced(ex, **one), "ex pair": forced(ex, **pair), "ex split": forced(ex, **split),
        "gated": forced(gated, **one), "gated pair": forced(gated, **pair), "gated split": forced(gated, **split),
        "gather": lambda b: nm.nm_spmm_gather_ex(ht, Xt, bias=b, out="float32"),
        "mx": lambda b: nm.nm_spmm_mx(hm, *QS, bias=b, out="float32"),
        "mx gated": lambda b: nm.nm_spmm_mx_gated(hmg, *QS, bias=b, out="float32"),
    }


@pytest.mark.gpu
def test_bias_written_by_the_kernel_before(monkeypatch):
    calls = products(monkeypatch)
    codes = [nm.nm_mx_quantize(torch.randn((1, 256), device="cuda")) for _ in range(2)]
    values = [nm.nm_mx_dequantize(*c, dtype=torch.float32).view(-1) for c in codes]
    b = torch.empty((1, 256), device="cuda")
    for name, call in calls.items():
        want = []
        for v in values:
            want.append(call(v))
            torch.cuda.synchronize()
        got = []
        for i in range(60):
            nm.nm_mx_dequantize(*codes[i & 1], dtype=torch.float32, X=b)
            got.append(call(b.view(-1)))
        torch.cuda.synchronize()
        for i, y in enumerate(got):
            assert torch.equal(y, want[i & 1]), (name, i)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("N,M", [(2, 4), (4, 8)])
def test_weight_packed_by_the_kernel_before(dt, N, M):
    """dX reads the packed weight that nm_recompress has just written."""
    g = torch.Generator(device="cuda").manual_seed(2)
    W = [torch.randn((192, 256), generator=g, device="cuda").to(dt) for _ in range(2)]
    X, P, dY = (torch.randn(s, generator=g, device="cuda").to(dt) for s in ((50, 256), (50, 192), (50, 96)))
    want = [nm.nm_gated_backward(nm.nm_compress_gated(w, N, M), X, P, dY)[0] for w in W]
    h = nm.nm_compress_gated(W[0], N, M)
    got = []
    for i in range(40):
        nm.nm_recompress(h, W[i & 1])
        got.append(nm.nm_gated_backward(h, X, P, dY)[0])
    torch.cuda.synchronize()
    for i, d in enumerate(got):
        assert torch.equal(d, want[i & 1]), i
