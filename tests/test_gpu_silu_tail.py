"""SiLU where its reciprocal leaves fp32's normal range, against the header's bound.

The gates are fp32 biases, so every value is reached exactly.  1 / (1 + exp(-v)) falls
below 2^-126 at v = -87.3365 and the hardware's reciprocal flushes it there: what is
lost is |v| 2^-126 = 1.027e-36 at most, the absolute term of the bound."""
import os
import re

import numpy as np
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm
from oracle import ffn

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nmspmm.h")


def header_terms():
    text = re.sub(r"\n \*", " ", open(HEADER).read())
    m = re.search(r"SiLU is within\s+\(([0-9.e-]+) \+ ([0-9.e-]+) max\(0, -v\)\) \|SiLU\(v\)\| \+\s+([0-9.e-]+) of", text)
    return [float(x) for x in m.groups()]


def test_absolute_term_covers_the_flushed_reciprocal():
    v = np.linspace(-87.5, -87.0, 5001)
    flushed = np.abs(v * 2.0 ** -126)
    assert header_terms()[2] >= flushed[1 + np.exp(-v) >= 2.0 ** 126].max()


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
def test_silu_tail(mx):
    rel, slope, least = header_terms()
    v = torch.cat((torch.linspace(-90, -86, 4001), torch.linspace(-87.37, -87.33, 4001), torch.linspace(-1, 1, 70)))
    F = v.numel()
    bias = torch.cat((v, torch.ones(F))).cuda()
    W = torch.zeros((2 * F, 32), dtype=torch.bfloat16, device="cuda")
    X = torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda")
    if mx:
        h = nm.nm_compress_mx(W, gated=True)
        y = nm.nm_spmm_mx_gated(h, *nm.nm_mx_quantize(X), bias=bias, act="silu", out="float32")
    else:
        h = nm.nm_compress_gated(W, 4, 4)
        y = nm.nm_spmm_gated(h, X, bias=bias, act="silu", out="float32")
    y, g = y.double().cpu().numpy(), ffn.act(v.double().numpy(), "silu")
    tol = (rel + slope * np.maximum(0, -v.double().numpy())) * np.abs(g) + least
    err = np.abs(y - g)
    assert (err <= tol).all(), float((err / tol).max())
