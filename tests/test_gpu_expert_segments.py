"""Segments that no dispatch leaves: the products refuse what they cannot count."""
import numpy as np
import pytest
import torch

from _experts import Activations, dev, weights
from _harness import SENTINEL, filled, moe

pytestmark = pytest.mark.gpu


def _call(m, swiglu, a, wq, ws, seg, counts, n, k):
    status = m.new_status()
    args = (dev(a.codes), dev(a.scales), dev(np.asarray(counts, np.int32)), dev(wq), dev(ws))
    kw = dict(seg_indptr=dev(np.asarray(seg, np.int64)), scale_layout="row")
    if swiglu:
        outs = [filled((a.rows, n // 2), torch.uint8), filled((a.rows, n // 16), torch.uint8)]
        m.moe_expert_gemm_swiglu("normal", *args, *outs, status, 100.0, **kw)
    else:
        outs = [filled((a.rows, n), torch.bfloat16)]
        m.moe_expert_gemm("normal", *args, *outs, status, **kw)
    torch.cuda.synchronize()
    return int(status.item()), outs


@pytest.mark.parametrize("swiglu", [False, True])
def test_segments_that_all_overlap_are_refused(swiglu):
    """64 experts that each claim all 1280 rows: 640 row tiles where experts without a common row have at most 10 + 64. With
    more rows and experts the tiles of the output would not fit 31 bits. Nothing is written."""
    m = moe()
    rng = np.random.default_rng(1)
    E, R, n, k = 64, 1280, 64, 64
    a = Activations(rng, "normal", [R], 0, 1, k, "row")
    wq, ws, _, _ = weights(rng, E * (1 + swiglu), n, k)
    code, outs = _call(m, swiglu, a, wq.reshape(E, -1, k // 2), ws.reshape(E, -1), np.zeros(E + 1), [R] * E, n, k)
    assert code == m.MOE_ERR_INVALID_ARG
    assert all((o.view(torch.uint8) == SENTINEL).all() for o in outs)


def test_the_most_row_tiles_that_separate_experts_can_have():
    """One row beyond a whole tile for each expert: 2 tiles an expert, not refused."""
    m = moe()
    rng = np.random.default_rng(2)
    E, n, k = 40, 32, 64
    counts = [129] * E
    a = Activations(rng, "normal", counts, 0, 1, k, "row")
    wq, ws, wv, _ = weights(rng, E, n, k)
    code, (out,) = _call(m, False, a, wq, ws, a.seg, counts, n, k)
    assert code == 0
    got = out.double().cpu().numpy()
    for e in range(E):
        rows = slice(129 * e, 129 * (e + 1))
        want, mag = a.values[rows] @ wv[e].T, np.abs(a.values[rows]) @ np.abs(wv[e]).T
        # exact in fp32 but for its last bits (64 products of few bits), then one bf16 rounding
        assert (np.abs(got[rows] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * mag).all()
