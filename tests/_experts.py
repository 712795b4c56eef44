"""References in 64 bits and inputs for the tests of the expert operators."""
import numpy as np
import torch

import oracle
from workloads import bf16_bits_to_f32, random_bf16

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
E4M3 = np.array([oracle.e4m3_to_float(c) for c in range(256)])   # 0x7f, 0xff: NaN
BF16_STEP = 2.0 ** -8          # a bf16 rounding is off by at most 2^-9 of the value; twice that for ties of two sides
# fp32 accumulation: at most 2^-23 of the sum of magnitudes for each partial sum that is rounded (a
# matrix instruction may cut instead of round); sums here have at most 512 of them, in whatever order
ACC = 512 * 2.0 ** -23


def interleave(sf):
    """The 128 x 4 tile bytes of scales [R, C]."""
    return oracle.nvfp4_sf_interleave(np.ascontiguousarray(sf))


def tile_index(R, C):
    """Byte of scale (r, c) in the tiles of an [R, C] matrix, from the definition."""
    r, c = np.arange(R)[:, None], np.arange(C)[None, :]
    return ((r // 128) * (C // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def values(codes, sf):
    """float64 values of codes [R, K/2] and scales [R, K/16]."""
    v = np.empty((codes.shape[0], codes.shape[1] * 2))
    v[:, 0::2], v[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    return v * np.repeat(E4M3[sf], 16, axis=1)


def quantise_rows(x_bits, g):
    """codes and scales of bf16 rows [R, K], in the quantiser's binary32 steps (the formats are the oracle's)."""
    R, K = x_bits.shape
    x = bf16_bits_to_f32(x_bits).reshape(R, K // 16, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        t = (np.abs(x).max(-1) * np.float32(1 / 6)) * g
        sf = oracle.e4m3_from_float_array(t).reshape(R, K // 16)
        v = E4M3[sf].astype(np.float32)
        r = np.where(v > 0, g / v, np.float32(0))
        q = oracle.e2m1_from_float_array(x * r[..., None]).reshape(R, K)
    q = np.where(np.repeat(v > 0, 16, axis=1), q, 0).astype(np.uint8)
    return q[:, 0::2] | (q[:, 1::2] << 4), sf


def quantised(rng, R, K, std=1.0):
    """NVFP4 rows of N(0, std^2): codes, scales [R, K/16] and their global scale."""
    x = random_bf16(rng, (R, K), std)
    amax = np.abs(bf16_bits_to_f32(x)).max() if x.size else 1.0
    g = float(np.float32(2688.0) / np.float32(amax))
    codes, sf = np.zeros((R, K // 2), np.uint8), np.zeros((R, K // 16), np.uint8)
    for r in range(R):
        codes[r], sf[r] = oracle.quant_nvfp4_row(x[r], g)
    return codes, sf, g


def weights(rng, matrices, R, K):
    """[matrices] NVFP4 matrices [R, K]: codes, tile bytes per matrix, values in 64 bits, 1/g."""
    codes, tiles, vals, inv = [], [], [], []
    for _ in range(matrices):
        q, sf, g = quantised(rng, R, K, K ** -0.5)
        codes.append(q)
        tiles.append(interleave(sf))
        vals.append(values(q, sf))
        inv.append(1 / g)
    return np.stack(codes), np.stack(tiles), vals, np.array(inv, np.float32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def layout(mode, counts, M, align, spare=0):
    """First row of each expert, seg_indptr and the number of rows."""
    counts = np.asarray(counts)
    if mode == "masked":
        base = np.arange(len(counts)) * M
        return base, np.zeros(len(counts) + 1, np.int64), len(counts) * M
    seg = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)]).astype(np.int64)
    return seg[:-1], seg, int(seg[-1]) + spare


def rows_of(base, counts):
    return np.concatenate([np.arange(b, b + c) for b, c in zip(base, counts)] + [np.zeros(0, np.int64)]).astype(np.int64)


class Activations:
    """Quantised rows in a layout; every row that no expert has holds NaN scales and codes 0xff."""

    def __init__(self, rng, mode, counts, M, align, K, scales, spare=0):
        self.base, self.seg, self.rows = layout(mode, counts, M, align, spare)
        self.used = rows_of(self.base, counts)
        q, sf, self.g = quantised(rng, len(self.used), K)
        self.codes = np.full((self.rows, K // 2), 0xff, np.uint8)
        full = np.full((-(-self.rows // 128) * 128, K // 16), 0xff, np.uint8)
        self.codes[self.used], full[self.used] = q, sf
        self.values = np.zeros((self.rows, K))
        self.values[self.used] = values(q, sf)
        self.scales = interleave(full) if scales == "swizzled" else full[:self.rows].copy()


def silu(v):
    return v / (1 + np.exp(-v))


def silu_slope():
    """A bound of |d silu / dv|."""
    return 1.1
