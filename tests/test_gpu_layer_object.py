"""MoELayer beyond its few tokens, stage by stage, and weights without factors."""
import numpy as np
import pytest
import torch

from _experts import ACC, BF16_STEP, silu, tile_index, values
from _harness import moe

pytestmark = pytest.mark.gpu


def _rows(codes, tiles, rows):
    """The values of whole matrices in the tiled scale layout."""
    C = codes.shape[1] // 8
    return values(codes[:rows], tiles[tile_index(rows, C)])


def _case(E, I, H, K, T, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=gen) * H ** -0.5).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=gen) * I ** -0.5).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
    ids[7] = -1
    ids[11, 1] = -1
    return w13, w2, x, ids, torch.rand(T, K, device="cuda", generator=gen)


@pytest.mark.parametrize("E,I,H,K,T", [(6, 256, 512, 3, 200), (5, 192, 320, 2, 130)])
def test_the_chain_stage_by_stage(E, I, H, K, T):
    """Each stage against 64 bits on the quantised operands that it was given: no row may be another's, and no tolerance hides
    NVFP4's own rounding."""
    m = moe()
    w13, w2, x, ids, w = _case(E, I, H, K, T, 5)
    q = m.quantize_experts(w13, w2)
    g_in, g_h = 2688.0 / 6.0, 2688.0 / 12.0
    layer = m.MoELayer(q, K, T, input_scale=g_in, inter_scale=g_h, few_tokens=0)
    out = layer(x, ids, w).double().cpu().numpy()
    layer.check()
    cpu = {n: getattr(layer, n).cpu().numpy() for n in ("seg_indptr", "masked_m", "src2dst", "x_codes", "x_scales", "h_codes",
                                                        "h_scales")}
    rows = T * K + E * 127
    pairs = np.flatnonzero(ids.flatten().cpu().numpy() >= 0)
    at = cpu["src2dst"][pairs]
    exp = ids.flatten().cpu().numpy()[pairs]
    assert len(set(at.tolist())) == len(pairs)
    assert np.array_equal(np.bincount(exp, minlength=E), cpu["masked_m"])
    # rows: each pair's token, quantised
    want = m.quantize_nvfp4(x, torch.tensor([g_in], device="cuda"), scale_layout="row")
    assert np.array_equal(cpu["x_codes"][at], want.codes.cpu().numpy()[pairs // K])
    assert np.array_equal(cpu["x_scales"][tile_index(rows, H // 16)][at], want.scales.cpu().numpy()[pairs // K])
    xv = _rows(cpu["x_codes"], cpu["x_scales"], rows)
    hv = _rows(cpu["h_codes"], cpu["h_scales"], rows)
    y = layer.expert_out.double().cpu().numpy()
    for e in range(E):
        r = at[exp == e]
        assert (r >= cpu["seg_indptr"][e]).all() and (r < cpu["seg_indptr"][e] + cpu["masked_m"][e]).all()
        c13, s13 = q.w13[e].cpu().numpy(), q.w13_scales.view(E, 2, -1)[e].cpu().numpy()
        wv = [_rows(c13[j * I:(j + 1) * I], s13[j], I) for j in (0, 1)]
        a13 = float(q.alpha13[e]) / g_in
        G, U = (xv[r] @ v.T * a13 for v in wv)
        eG, eU = (ACC * (np.abs(xv[r]) @ np.abs(v).T) * a13 for v in wv)
        h = U * silu(G)
        eh = 1.1 * eG * (np.abs(U) + eU) + np.abs(silu(G)) * eU + 2.0 ** -19 * np.abs(h)
        # half of e2m1's widest step is a sixth of the block's largest, by a scale that is off by 2^-4
        most = np.repeat(np.abs(h).reshape(len(r), -1, 16).max(2), 16, axis=1)
        assert (np.abs(hv[r] / g_h - h) <= 0.18 * most + 2 * np.repeat(eh.reshape(len(r), -1, 16).max(2), 16, axis=1)).all(), e
        w2v = _rows(q.w2[e].cpu().numpy(), q.w2_scales.view(E, -1)[e].cpu().numpy(), H)
        a2 = float(q.alpha2[e]) / g_h
        want = hv[r] @ w2v.T * a2
        bad = np.abs(y[r] - want) > BF16_STEP * np.abs(want) + ACC * (np.abs(hv[r]) @ np.abs(w2v).T) * a2
        assert not bad.any(), e
    wn = w.double().cpu().numpy().flatten()
    want, mag = np.zeros((T, H)), np.zeros((T, H))
    np.add.at(want, pairs // K, y[at] * wn[pairs, None])
    np.add.at(mag, pairs // K, np.abs(y[at]) * wn[pairs, None])
    assert (np.abs(out - want) <= BF16_STEP * np.abs(want) + 2.0 ** -20 * mag).all()
    assert not out[7].any()


def test_weights_without_factors():
    """ExpertWeights without alphas stand for what their codes and scales say, for few tokens and for many."""
    m = moe()
    E, I, H, K, T = 4, 128, 256, 2, 90
    w13, w2, x, ids, w = _case(E, I, H, K, T, 6)
    one = torch.ones(E, device="cuda")
    q13 = m.quantize_nvfp4((w13 * 64).view(2 * E, I, H), one.repeat(2))
    q2 = m.quantize_nvfp4(w2 * 64, one)
    parts = (q13.codes.view(E, 2 * I, H // 2), q2.codes, q13.scales, q2.scales)
    scales = dict(input_scale=2688.0 / 6.0, inter_scale=2688.0 / 65536.0)
    with_ones = m.MoELayer(m.ExpertWeights(*parts, one, one), K, T, **scales)
    without = m.MoELayer(m.ExpertWeights(*parts), K, T, **scales)
    for n in (T, 3):
        want = with_ones(x[:n], ids[:n], w[:n])
        got = without(x[:n], ids[:n], w[:n])
        with_ones.check()
        without.check()
        assert want.float().norm() > 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))
