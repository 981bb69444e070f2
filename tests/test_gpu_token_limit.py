"""Token counts whose last tile ends beyond 2^31 are refused before anything is launched (the
kernels count tokens in 32 bits, to the end of the last tile)."""
import pytest
import torch

import structured_sparse_gemm_compress_b200 as nm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [(1 << 31) - 255, (1 << 31) - 1, 1 << 31, 1 << 40])
def test_products_refuse(T):
    L = nm.lib()
    W = torch.randint(-127, 128, (128, 64), dtype=torch.int8, device="cuda")
    X, Y = torch.zeros(1 << 16, dtype=torch.int8, device="cuda"), torch.zeros(1 << 16, dtype=torch.int8, device="cuda")
    x, y = X.data_ptr(), Y.data_ptr()
    h, ht, hg = nm.nm_compress(W, 2, 4), nm.nm_compress_tile(W, 2, 4), nm.nm_compress_gated(W, 2, 4)
    assert L.nm_spmm(h.raw, x, T, y, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_spmm_ex(h.raw, x, T, y, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_spmm_noalloc(h.raw, x, T, y, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_spmm_gather(ht.raw, x, T + 1024 & ~15, T, y, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_spmm_gather_ex(ht.raw, x, T + 1024 & ~15, T, y, None, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_spmm_gated(hg.raw, x, T, y, None, None, None) == nm.NM_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert not Y.any()
