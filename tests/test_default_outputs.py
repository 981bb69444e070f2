"""The default output type of every kind of handle, by the header's rules (CPU)."""
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm


def handle(dt, gated=False, src=None):
    return nm.NMHandle(0, 256, 768, 2, 4, dt, gated=gated, src=src)


@pytest.mark.parametrize("h,plain,scaled", [
    (handle(nm.NM_INT8), "int32", "float32"),
    (handle(nm.NM_INT8, gated=True), "float32", "float32"),      # no raw accumulators behind a gate
    (handle(nm.NM_FP16, gated=True), "float16", "float16"),
    (handle(nm.NM_BF16), "bfloat16", "bfloat16"),
    (handle(nm.NM_MXFP4, src=torch.float32), "float32", "float32"),
    (handle(nm.NM_MXFP4, src=torch.float16, gated=True), "float16", "float16"),
    (handle(nm.NM_MXFP4, src=torch.bfloat16), "bfloat16", "bfloat16"),
])
def test_default_output_of_every_handle(h, plain, scaled):
    assert nm.resolve_out(h, "default", None, None, "none") == plain
    assert nm.resolve_out(h, "default", object(), None, "none") == scaled
    assert str(nm.out_dtype(h, False)) == "torch." + plain
    assert str(nm.out_dtype(h, True)) == "torch." + scaled
