"""How the backward pass shares out its two products over CTA pairs, on the CPU through
nm_gated_backward_plan_for_shape."""
import ctypes
import random

import pytest

import structured_sparse_gemm_compress_b200 as nm


@pytest.fixture(autouse=True)
def _no_forced_plan(monkeypatch):
    for k in ("NMSPMM_FORCE_GRAD_BN", "NMSPMM_GRAD_SPLIT"):
        monkeypatch.delenv(k, raising=False)


@pytest.mark.parametrize("bn", [None, "128", "256"])
@pytest.mark.parametrize("seed", range(4))
def test_every_stage_is_one_pairs(monkeypatch, seed, bn):
    if bn:
        monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", bn)
    rng = random.Random(seed)
    size = lambda hi: int(round(2 ** rng.uniform(0, hi)))  # noqa: E731
    cut = 0
    for _ in range(400):
        F, k, T, sms = size(13), 8 * size(8), size(15), rng.choice((2, 20, 132, 148, 160))
        dx, dw = rng.choice(((1, 1), (1, 1), (1, 0), (0, 1)))
        p = nm.nm_gated_backward_plan_for_shape(F, k, T, sms, dx=dx, dw=dw)
        assert p["complete"] == 1, (F, k, T, sms, p)
        assert p["bn"] in (128, 256) and 1 <= p["grid"] <= sms // 2
        assert (p["splits_dx"] > 0) == bool(dx) and (p["splits_dw"] > 0) == bool(dw)
        cut += p["splits_dx"] > 1 or p["splits_dw"] > 1
        # no pair has more than its share and a unit of each product (and what cutting is worth)
        kb = 2 * -(-F // 64), -(-T // 64)
        tiles = (dx * -(-T // 256) * -(-k // p["bn"]), dw * 2 * -(-F // 256) * -(-k // p["bn"]))
        longest = max(kb[0] if dx else 0, kb[1] if dw else 0)
        units = tiles[0] * max(1, p["splits_dx"]) + tiles[1] * max(1, p["splits_dw"])
        share = (tiles[0] * kb[0] + tiles[1] * kb[1] + 6 * units) / p["grid"]
        assert p["stages"] <= share + 2 * (longest + 6)
    assert cut >= 10        # the draws reach the cut sums


@pytest.mark.parametrize("T,k,F,splits", [
    (200, 264, 1030, (5, 1)), (1, 512, 2048, (8, 1)), (3000, 64, 40, (1, 6)),              # one product cut
    (1500, 64, 1500, (6, 3)), (3000, 128, 700, (3, 6)), (3000, 64, 1500, (3, 3)),            # both
    (1500, 136, 700, (1, 1)), (6304, 1024, 4096, (1, 1)), (1379, 768, 2051, (1, 1)),         # neither
])
@pytest.mark.parametrize("bn", ["128", "256"])
def test_cut_sums_on_a_b200(monkeypatch, bn, T, k, F, splits):
    monkeypatch.setenv("NMSPMM_FORCE_GRAD_BN", bn)
    p = nm.nm_gated_backward_plan_for_shape(F, k, T, 148)
    assert (p["splits_dx"], p["splits_dw"]) == splits
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", "0")
    p = nm.nm_gated_backward_plan_for_shape(F, k, T, 148)
    assert (p["splits_dx"], p["splits_dw"]) == (1, 1)


def test_runs_of_an_accumulator(monkeypatch):
    """2^14 summed elements at most."""
    monkeypatch.setenv("NMSPMM_GRAD_SPLIT", "0")
    for T, runs in ((1, 1), (1 << 14, 1), ((1 << 14) + 1, 2), (1 << 20, 64)):
        assert nm.nm_gated_backward_plan_for_shape(64, 64, T, 148)["runs_dw"] == runs
    for F, runs in ((1, 1), (1 << 13, 1), ((1 << 13) + 1, 2), (1 << 19, 64)):
        assert nm.nm_gated_backward_plan_for_shape(F, 64, 64, 148)["runs_dx"] == runs


def test_refusals():
    info = nm.NMGradPlanInfo()
    call = lambda *a: nm.lib().nm_gated_backward_plan_for_shape(*a, ctypes.byref(info))  # noqa: E731
    assert nm.lib().nm_gated_backward_plan_for_shape(8, 8, 8, 1, 1, 148, None) == nm.NM_ERR_INVALID
    for bad in ((0, 8, 8, 1, 1, 148), (8, 0, 8, 1, 1, 148), (8, 8, 0, 1, 1, 148), (8, 8, 8, 0, 0, 148), (8, 8, 8, 1, 1, 1)):
        assert call(*bad) == nm.NM_ERR_INVALID
    for large in (((1 << 23) + 1, 8, 8, 1, 1, 148), (8, (1 << 24) + 1, 8, 1, 1, 148), (8, 8, (1 << 26) + 1, 1, 1, 148)):
        assert call(*large) == nm.NM_ERR_UNSUPPORTED
    with pytest.raises(nm.NMError):
        nm.nm_gated_backward_plan_for_shape(0, 8, 8, 148)
