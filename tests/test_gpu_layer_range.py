"""The few-token layer with NVFP4 weights on rows whose values spread over many binary orders: neither the blocks of 16 nor an
outlier's neighbours lose their values to the largest one of their row."""
import numpy as np
import pytest
import torch

from _experts import ACC, BF16_STEP, E2M1, E4M3, dev, interleave, silu, weights
from _harness import filled, moe
from _terms import Differences
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _bf16(v):
    return torch.from_numpy(f32_to_bf16_bits(np.asarray(v, np.float32)).view(np.int16).copy()).cuda().view(torch.bfloat16)


def _run(x, ids, w, w13, s13, a13, w2, s2, a2, stream=None):
    m = moe()
    T, H = x.shape
    E, I, K = w13.shape[0], w13.shape[1] // 2, ids.shape[1]
    out, status = filled((T, H), torch.bfloat16), m.new_status()
    args = [dev(v) for v in (ids, w, w13, w2)]
    more = [dev(v) for v in (s13, s2, a13, a2)]
    ws = m.new_layer_workspace(T, K, H, I, E)
    torch.cuda.synchronize()
    m.moe_layer_few_tokens(x, *args, out, ws, status, *more, stream=stream)
    torch.cuda.synchronize()
    m.check_status(status)
    return out.double().cpu().numpy()


def _want(x, ids, w, v13, v2):
    """Output and allowance: fp32 sums, and 2^-12 of a block's largest for each value of x and of h."""
    T, H = x.shape
    most = lambda v: np.repeat(np.abs(v).reshape(-1, 16).max(1), 16)  # noqa: E731
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, f in zip(ids[t], w[t].astype(np.float64)):
            I = v2[e].shape[1]
            g, u = np.split(v13[e] @ x[t], [I])
            eg, eu = np.split(np.abs(v13[e]) @ (ACC * np.abs(x[t]) + 2.0 ** -12 * most(x[t])), [I])
            h = u * silu(g)
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -19 * np.abs(h)
            y[t] += f * (v2[e] @ h)
            err[t] += f * (np.abs(v2[e]) @ (eh + ACC * np.abs(h) + 2.0 ** -12 * most(h)))
    return y, err


def _check(got, want, err):
    """Each value within its allowance, and all together within twice what rounding to bf16 takes (0.0017 of the norm; the terms
    add less: up to 2^-5 of the values of the 15 neighbours of an outlier, 2^-16 of the others)."""
    bad = np.abs(got - want) > BF16_STEP * np.abs(want) + err
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel < 2.0 ** -8, rel


SHAPES = [(1, 512, 256, 8, 4), (5, 1088, 192, 4, 3), (33, 320, 320, 3, 2), (64, 256, 128, 2, 2), (20, 2112, 704, 40, 4)]


@pytest.mark.parametrize("shape", SHAPES, ids=["-".join(map(str, s)) for s in SHAPES])
@pytest.mark.parametrize("order", [10, 14, 20, 24, 28, 45, 100])
def test_an_outlier_of_x_that_no_weight_looks_at(shape, order):
    """An element of 2^order in every second row, whose column of W13 is 0: the other values count as if it were not there."""
    T, H, I, E, K = shape
    rng = np.random.default_rng(order + T)
    x = bf16_bits_to_f32(f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32)))
    col = 5 * H // 7
    x[0::2, col] = 2.0 ** order
    q13, s13, v13, i13 = weights(rng, 2 * E, I, H)
    q2, s2, v2, i2 = weights(rng, E, H, I)
    q13[:, :, col // 2] &= 0xf0 if col % 2 == 0 else 0x0f
    for v in v13:
        v[:, col] = 0
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    w = rng.random((T, K), dtype=np.float32)
    got = _run(_bf16(x), ids, w, q13.reshape(E, 2 * I, H // 2), s13.reshape(E, -1), i13[0::2], q2, s2, i2)
    want = _want(x.astype(np.float64), ids, w,
                 [np.concatenate(v13[2 * e:2 * e + 2]) * np.float64(i13[2 * e]) for e in range(E)],
                 [v2[e] * np.float64(i2[e]) for e in range(E)])
    _check(got, *want)


def _flat(rng, R, K, sf):
    """Weights of random codes with one scale byte a row: codes, tiles, values."""
    q = rng.integers(0, 256, (R, K // 2)).astype(np.uint8)
    v = np.empty((R, K))
    v[:, 0::2], v[:, 1::2] = E2M1[q & 15], E2M1[q >> 4]
    return q, interleave(np.repeat(sf[:, None], K // 16, axis=1).astype(np.uint8)), v * E4M3[sf][:, None]


@pytest.mark.parametrize("T,H,I", [(1, 512, 256), (6, 256, 512), (40, 192, 704)])
@pytest.mark.parametrize("order", [13, 20, 28])
def test_an_outlier_of_h_that_no_weight_looks_at(T, H, I, order):
    """One row of W13, gate and up, has scales of 2^(order/2) times the others', and its column of W2 is 0."""
    rng = np.random.default_rng(order + T)
    E, K = 3, 2
    big = I // 3
    sf = np.full(2 * I, 0x08)                                              # 2^-6
    sf[[big, I + big]] += 8 * np.array([order // 2, order - order // 2])   # e4m3: eight codes a binary order
    parts = [[_flat(rng, I, H, sf[j * I:(j + 1) * I]) for j in (0, 1)] for _ in range(E)]
    a13 = np.full(E, 64 / (2.6 * H ** 0.5), np.float32)                    # gates of about N(0, 1)
    w2 = [_flat(rng, H, I, np.full(H, 0x38)) for _ in range(E)]
    for q, _, v in w2:
        q[:, big // 2] &= 0xf0 if big % 2 == 0 else 0x0f
        v[:, big] = 0
    a2 = np.full(E, I ** -0.5, np.float32)
    x = bf16_bits_to_f32(f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32)))
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    w = rng.random((T, K), dtype=np.float32)
    got = _run(_bf16(x), ids, w, np.stack([np.concatenate([p[0][0], p[1][0]]) for p in parts]),
               np.stack([np.concatenate([p[0][1], p[1][1]]) for p in parts]), a13, np.stack([q for q, _, _ in w2]),
               np.stack([s for _, s, _ in w2]), a2)
    want = _want(x.astype(np.float64), ids, w,
                 [np.concatenate([p[0][2], p[1][2]]) * np.float64(a13[e]) for e, p in enumerate(parts)],
                 [v * np.float64(a2[e]) for e, (_, _, v) in enumerate(w2)])
    _check(got, *want)


@pytest.mark.parametrize("top", [0, 60, 120])
@pytest.mark.parametrize("step", [3, 7, 15])
def test_blocks_of_all_sizes(top, step):
    """Block b of x is 2^(top - step b) times N(0, 1) (down to 2^-100, then it starts again), every element seen by itself: up
    rows pick one each, W2 picks one h each. So h has all these sizes as well."""
    T, n = 3, 256
    rng = np.random.default_rng(top + step)
    scale = 2.0 ** (top - step * np.arange(n // 16) % (top + 100)).astype(np.float64)
    x = np.zeros((T, n + 64), np.float32)
    x[:, :n] = bf16_bits_to_f32(f32_to_bf16_bits((rng.standard_normal((T, n)) * np.repeat(scale, 16)).astype(np.float32)))
    x[:, n] = 1.0                                                          # the gate's element: gates of 6
    H, I = n + 64, n
    up, gate, down = np.zeros((I, H), int), np.zeros((I, H), int), np.zeros((H, I), int)
    up[np.arange(I), np.arange(I)] = 1
    gate[:, n] = 1
    down[np.arange(I), np.arange(I)] = 1
    six = (gate[:, 0::2] != 0) * 5                                         # code 7 instead of code 2
    w13 = np.concatenate([Differences.codes(gate) + six, Differences.codes(up)])[None].astype(np.uint8)
    s13 = np.concatenate([Differences.scales(gate), Differences.scales(up)])[None]
    one = np.ones(1, np.float32)
    got = _run(_bf16(x), np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32), w13, s13, one, Differences.codes(down)[None],
               Differences.scales(down)[None], one)
    want = x[:, :n].astype(np.float64) * silu(6.0)
    most = np.repeat(np.abs(want).reshape(T, -1, 16).max(2), 16, axis=1)
    # 2^-12 of the block's largest for x and for h, silu's 2^-20 among the rest, one bf16 rounding
    bad = np.abs(got[:, :n] - want) > 2.0 ** -8 * np.abs(want) + 2.05 * 2.0 ** -12 * most
    assert not bad.any(), np.argwhere(bad)[:4].tolist()
    assert not got[:, n:].any()


def test_differences_of_neighbours():
    """What five terms leave, seen in differences of nearly equal x and h: four terms would leave eight times as much."""
    d = Differences()
    w13 = np.concatenate([d.codes(d.gate), d.codes(d.up)])[None]
    s13 = np.concatenate([d.scales(d.gate), d.scales(d.up)])[None]
    one = np.ones(1, np.float32)
    T = len(d.x)
    out = _run(_bf16(d.x), np.zeros((T, 1), np.int32), np.ones((T, 1), np.float32), w13, s13, one, d.codes(d.down)[None],
               d.scales(d.down)[None], one)
    assert d.holds(out), d.errors(out)


def test_wide_rows_leave_the_others_alone():
    """Rows of many windows in the groups of ordinary ones change no bit of these, and give the same bits every time."""
    rng = np.random.default_rng(3)
    T, H, I, E, K = 24, 576, 320, 3, 2
    x = bf16_bits_to_f32(f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32)))
    q13, s13, _, i13 = weights(rng, 2 * E, I, H)
    q2, s2, _, i2 = weights(rng, E, H, I)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    w = rng.random((T, K), dtype=np.float32)
    args = (ids, w, q13.reshape(E, 2 * I, H // 2), s13.reshape(E, -1), i13[0::2], q2, s2, i2)
    plain = _run(_bf16(x), *args)
    wide = x.copy()
    wide[5::6] *= np.repeat(2.0 ** -(9.0 * np.arange(H // 16) % 113), 16).astype(np.float32)
    first = _run(_bf16(wide), *args)
    keep = np.arange(T) % 6 != 5
    assert np.array_equal(first[keep], plain[keep])
    for _ in range(2):
        assert np.array_equal(_run(_bf16(wide), *args, stream=torch.cuda.Stream()), first)
