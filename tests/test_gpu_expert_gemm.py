"""The products over a dispatched layout's experts against 64-bit references."""
import numpy as np
import pytest
import torch

from _experts import ACC, BF16_STEP, E2M1, E4M3, Activations, dev, silu, silu_slope, tile_index, values, weights
from _harness import SENTINEL, filled, moe

pytestmark = pytest.mark.gpu

CASES = [  # mode, counts, M, align, n, k, scales
    ("masked", [1], 1, 1, 16, 64, "row"),
    ("masked", [1], 16, 1, 64, 64, "swizzled"),
    ("masked", [3, 0, 16, 1], 16, 1, 144, 192, "row"),
    ("masked", [3, 0, 16, 1], 16, 1, 144, 192, "swizzled"),
    ("masked", [0, 0, 0], 8, 1, 64, 128, "swizzled"),
    ("masked", [128, 127, 129, 1], 130, 1, 272, 320, "swizzled"),
    ("masked", [128, 5, 128, 64], 128, 1, 256, 1088, "swizzled"),
    ("masked", [300, 0, 257], 384, 1, 384, 256, "swizzled"),
    ("masked", [300, 0, 257], 301, 1, 528, 576, "row"),
    ("normal", [5], 0, 1, 32, 64, "row"),
    ("normal", [1, 1, 1, 0, 1], 0, 1, 128, 448, "swizzled"),
    ("normal", [130, 0, 5, 300, 77], 0, 1, 240, 320, "row"),
    ("normal", [130, 0, 5, 300, 77], 0, 1, 320, 192, "swizzled"),
    ("normal", [130, 0, 5, 300, 77], 0, 16, 256, 704, "swizzled"),
    ("normal", [130, 0, 5, 300, 77], 0, 128, 640, 1024, "swizzled"),
    ("normal", [256, 512, 128], 0, 128, 512, 2112, "row"),
    ("normal", [2] * 150 + [0] * 40 + [9] * 10, 0, 8, 80, 128, "swizzled"),
    ("normal", [1, 0, 2] * 341 + [3], 0, 1, 16, 64, "row"),             # 1024 experts, the most there can be
    ("masked", [257, 130], 260, 1, 272, 4160, "row"),                   # many slots, scales not whole 16-byte pieces
    ("masked", [257, 130], 260, 1, 272, 4096, "row"),                   # the same with whole ones
]
IDS = ["-".join(map(str, (c[0], len(c[1]), max(c[1]), c[4], c[5], c[6], c[3]))) for c in CASES]


def _product(case, alpha=True, seed=0, spare=0, stream=None):
    mode, counts, M, align, n, k, scales = case
    m = moe()
    rng = np.random.default_rng(seed + n + k)
    a = Activations(rng, mode, counts, M, align, k, scales, spare)
    wq, ws, wv, inv = weights(rng, len(counts), n, k)
    al = (inv / np.float32(a.g)).astype(np.float32) if alpha else np.ones(len(counts), np.float32)
    out = filled((a.rows, n), torch.bfloat16)
    status = m.new_status()
    args = [dev(a.codes), dev(a.scales), dev(np.array(counts, np.int32)), dev(wq), dev(ws)]
    torch.cuda.synchronize()
    m.moe_expert_gemm(mode, *args, out, status, alpha=dev(al) if alpha else None, seg_indptr=dev(a.seg),
                      max_tokens_per_expert=M, scale_layout=scales, stream=stream)
    torch.cuda.synchronize()
    m.check_status(status)
    return a, wv, al, out


def _check_product(counts, a, wv, al, out):
    got = out.float().cpu().numpy().astype(np.float64)
    for e, c in enumerate(counts):
        rows = slice(a.base[e], a.base[e] + c)
        want = a.values[rows] @ wv[e].T * al[e]
        mag = np.abs(a.values[rows]) @ np.abs(wv[e]).T * al[e]
        bad = np.abs(got[rows] - want) > BF16_STEP * np.abs(want) + ACC * mag
        assert not bad.any(), (e, int(bad.sum()), np.argwhere(bad)[:4].tolist())
    rest = np.ones(a.rows, bool)
    rest[a.used] = False
    raw = out.view(torch.uint8).cpu().numpy()
    assert (raw[rest] == SENTINEL).all(), "rows that no expert has were written"


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_product(case):
    a, wv, al, out = _product(case)
    _check_product(case[1], a, wv, al, out)


def test_product_without_alpha_and_with_spare_rows():
    case = ("normal", [70, 3], 0, 1, 96, 128, "swizzled")
    a, wv, al, out = _product(case, alpha=False, spare=200)
    _check_product(case[1], a, wv, al, out)


def test_product_on_another_stream():
    case = ("masked", [40, 9], 64, 1, 256, 512, "swizzled")
    s = torch.cuda.Stream()
    a, wv, al, out = _product(case, stream=s)
    _check_product(case[1], a, wv, al, out)


def test_products_on_two_streams_at_once():
    """Calls that share nothing may overlap: each result is that of the call alone."""
    m = moe()
    jobs = []
    for i, case in enumerate([("masked", [200, 3, 140], 256, 1, 512, 1024, "swizzled"),
                              ("normal", [90, 300], 0, 1, 768, 512, "row")]):
        mode, counts, M, align, n, k, scales = case
        rng = np.random.default_rng(i)
        a = Activations(rng, mode, counts, M, align, k, scales)
        wq, ws, wv, inv = weights(rng, len(counts), n, k)
        args = (dev(a.codes), dev(a.scales), dev(np.array(counts, np.int32)), dev(wq), dev(ws))
        outs = [filled((a.rows, n), torch.bfloat16) for _ in range(6)]
        jobs.append((mode, args, outs, dict(seg_indptr=dev(a.seg), max_tokens_per_expert=M, scale_layout=scales),
                     torch.cuda.Stream(), a, wv, counts))
    status = m.new_status()
    torch.cuda.synchronize()
    for r in range(6):
        for mode, args, outs, kw, stream, *_ in jobs:
            m.moe_expert_gemm(mode, *args, outs[r], status, stream=stream, **kw)
    torch.cuda.synchronize()
    m.check_status(status)
    for *_, outs, kw, stream, a, wv, counts in jobs:
        _check_product(counts, a, wv, np.ones(len(counts)), outs[0])
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


def test_counts_beyond_the_layout_are_cut_and_reported():
    m = moe()
    rng = np.random.default_rng(3)
    M, n, k = 32, 128, 128
    a = Activations(rng, "masked", [32, 32], M, 1, k, "row")
    wq, ws, wv, inv = weights(rng, 2, n, k)
    for counts, code in (([40, 32], m.MOE_ERR_CAPACITY), ([-1, 32], m.MOE_ERR_INVALID_ARG)):
        out, status = filled((64, n), torch.bfloat16), m.new_status()
        m.moe_expert_gemm("masked", dev(a.codes), dev(a.scales), dev(np.array(counts, np.int32)), dev(wq), dev(ws),
                          out, status, max_tokens_per_expert=M, scale_layout="row")
        torch.cuda.synchronize()
        assert int(status.item()) == code
        kept = [min(max(c, 0), M) for c in counts]
        a.used = np.concatenate([np.arange(e * M, e * M + c) for e, c in enumerate(kept)])
        _check_product(kept, a, wv, np.ones(2), out)
    # normal: the last segment runs past the buffer
    seg = np.array([0, 32, 64], np.int64)
    out, status = filled((64, n), torch.bfloat16), m.new_status()
    m.moe_expert_gemm("normal", dev(a.codes), dev(a.scales), dev(np.array([32, 50], np.int32)), dev(wq), dev(ws), out,
                      status, seg_indptr=dev(seg), scale_layout="row")
    torch.cuda.synchronize()
    assert int(status.item()) == m.MOE_ERR_CAPACITY
    a.used = np.arange(64)
    _check_product([32, 32], a, wv, np.ones(2), out)


SWIGLU = [  # mode, counts, M, align, inter, k, scales
    ("masked", [1], 1, 1, 64, 64, "row"),
    ("masked", [3, 0, 16, 1], 16, 1, 192, 192, "row"),
    ("masked", [3, 0, 16, 1], 16, 1, 192, 192, "swizzled"),
    ("masked", [128, 127, 129, 1], 130, 1, 128, 320, "swizzled"),
    ("masked", [128, 5, 128], 128, 1, 320, 1088, "swizzled"),
    ("normal", [130, 0, 5, 300, 77], 0, 1, 192, 320, "row"),
    ("normal", [130, 0, 5, 300, 77], 0, 1, 64, 192, "swizzled"),
    ("normal", [130, 0, 5, 300, 77], 0, 128, 704, 576, "swizzled"),
    ("normal", [2] * 150 + [0] * 40 + [9] * 10, 0, 8, 64, 128, "swizzled"),
]


@pytest.mark.parametrize("case", SWIGLU, ids=["-".join(map(str, (c[0], len(c[1]), max(c[1]), c[4], c[5], c[6], c[3])))
                                              for c in SWIGLU])
def test_swiglu(case):
    """Every block scale and code lies between those of the smallest and the largest h that the sums' error allows."""
    mode, counts, M, align, n, k, scales = case
    m = moe()
    rng = np.random.default_rng(n + k)
    a = Activations(rng, mode, counts, M, align, k, scales)
    E, C = len(counts), n // 16
    wq, ws, wv, inv = weights(rng, 2 * E, n, k)
    al = (inv[0::2] / np.float32(a.g)).astype(np.float32)
    H_SCALE = 168.0
    tiles = m.nvfp4_scale_bytes(a.rows, n, scales)
    codes, sf = filled((a.rows, n // 2), torch.uint8), filled((tiles,), torch.uint8)
    status = m.new_status()
    m.moe_expert_gemm_swiglu(mode, dev(a.codes), dev(a.scales), dev(np.array(counts, np.int32)),
                             dev(wq.reshape(E, 2 * n, k // 2)), dev(ws), codes, sf, status, H_SCALE, alpha=dev(al),
                             seg_indptr=dev(a.seg), max_tokens_per_expert=M, scale_layout=scales)
    torch.cuda.synchronize()
    m.check_status(status)
    codes, sf = codes.cpu().numpy(), sf.cpu().numpy()
    at = tile_index(a.rows, C) if scales == "swizzled" else np.arange(a.rows * C).reshape(a.rows, C)
    got = sf[at]
    e4m3 = E4M3[:127]
    mids4 = (e4m3[1:] + e4m3[:-1]) / 2
    mids2 = (E2M1[1:8] + E2M1[:7]) / 2
    for e, c in enumerate(counts):
        rows = slice(a.base[e], a.base[e] + c)
        x = a.values[rows]
        G, U = (x @ wv[2 * e + j].T * al[e] for j in (0, 1))
        eG, eU = (ACC * (np.abs(x) @ np.abs(wv[2 * e + j]).T) * al[e] for j in (0, 1))
        h = U * silu(G)
        # first order in both errors, their product, and 16 binary32 roundings of exp, divide and products
        eh = silu_slope() * eG * (np.abs(U) + eU) + np.abs(silu(G)) * eU + 2.0 ** -20 * np.abs(h)
        mag = np.abs(h).reshape(-1, C, 16)
        err = eh.reshape(-1, C, 16)
        lo = np.maximum(mag - err, 0).max(2) / 6 * H_SCALE * (1 - 2.0 ** -20)
        hi = (mag + err).max(2) / 6 * H_SCALE * (1 + 2.0 ** -20)
        s = got[rows]
        assert ((s >= np.searchsorted(mids4, lo, "left")) & (s <= np.searchsorted(mids4, hi, "right"))).all(), e
        v = E4M3[s][:, :, None]
        with np.errstate(divide="ignore", invalid="ignore"):
            y = np.where(v > 0, h.reshape(-1, C, 16) * H_SCALE / v, 0)
            ey = np.where(v > 0, err * H_SCALE / v, 0) + 2.0 ** -20 * np.abs(y)
        q = np.empty((c, n), np.int64)
        q[:, 0::2], q[:, 1::2] = codes[rows] & 15, codes[rows] >> 4
        q = q.reshape(-1, C, 16)
        low = np.searchsorted(mids2, np.maximum(np.abs(y) - ey, 0), "left")
        high = np.searchsorted(mids2, np.abs(y) + ey, "right")
        assert ((q & 7) >= low).all() and ((q & 7) <= high).all(), e
        sure = np.abs(y) > ey
        assert (((q >> 3) == (y < 0)) | ~sure | (v == 0)).all(), e
    rest = np.ones(a.rows, bool)
    rest[a.used] = False
    assert (codes[rest] == SENTINEL).all() and (got[rest] == SENTINEL).all(), "rows that no expert has were written"


def test_offsets_past_32_bits():
    """The last expert's weights and rows lie beyond 4 GiB of their buffers."""
    m = moe()
    rng = np.random.default_rng(5)
    E, M, n, k = 70, 8192, 4096, 4096     # out: 4.7 GB
    a = Activations(rng, "normal", [3], 0, 1, k, "row")
    wq, ws, wv, inv = weights(rng, 1, n, k)
    codes = torch.zeros((E, M, k // 2), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((E * M, k // 16), dtype=torch.uint8, device="cuda")
    codes[-1, :3], sf[-M:-M + 3] = dev(a.codes), dev(a.scales)
    W = torch.zeros((E, n, k // 2), dtype=torch.uint8, device="cuda")
    S = torch.zeros((E, m.nvfp4_scale_bytes(n, k, "swizzled")), dtype=torch.uint8, device="cuda")
    W[-1], S[-1] = dev(wq[0]), dev(ws[0])
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    count[-1] = 3
    out = torch.zeros((E, M, n), dtype=torch.bfloat16, device="cuda")
    status = m.new_status()
    m.moe_expert_gemm("masked", codes, sf, count, W, S, out, status, max_tokens_per_expert=M, scale_layout="row")
    m.check_status(status)
    want = a.values @ wv[0].T
    mag = np.abs(a.values) @ np.abs(wv[0]).T
    got = out[-1, :3].double().cpu().numpy()
    assert (np.abs(got - want) <= BF16_STEP * np.abs(want) + ACC * mag).all()
    assert not out[-1, 3:].any() and not out[:-1].any()
