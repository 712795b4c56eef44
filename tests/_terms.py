"""The few-token layer's sums of NVFP4 blocks, restated: what the terms of a block leave, and a layer whose output is made
of that."""
import numpy as np

import oracle
from _experts import E2M1, E4M3, interleave, silu
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

ORDERS, SPREAD = 13, 11   # binary orders of a further pass, and of the first


def split(x, terms=5):
    """The sums of NVFP4 blocks for each 16 values of the rows x [R, K] (binary32): `terms` a pass, with the row's largest at
    [2^8, 2^9) in the first and 2^13 times what is left in each further one, of which there is one for each 13 binary orders
    after the first 11 between the row's largest and the least largest of eight neighbours that is not zero."""
    x = np.asarray(x, np.float64)
    R = len(x)
    exponent = lambda v: np.frexp(v)[1] - 1  # noqa: E731
    top = np.abs(x).max(1)
    eights = np.abs(x).reshape(R, -1, 8).max(2)
    least = np.where(eights > 0, eights, np.inf).min(1)
    row = exponent(np.where(top > 0, top, 256.0))
    below = row - exponent(np.where(np.isfinite(least), least, top))
    passes = 1 + np.maximum(below - SPREAD + ORDERS - 1, 0) // ORDERS
    left = np.ldexp(x, (8 - row)[:, None]).reshape(R, -1, 16)
    total = np.zeros_like(left)
    for p in range(passes.max()):
        live = (p < passes)[:, None, None]
        for i in range(terms):
            m = np.abs(left).max(2)
            sf = oracle.e4m3_from_float_array((m * 8.0 ** i / 6).astype(np.float32).ravel()).reshape(m.shape)
            s = E4M3[sf] / 8.0 ** i
            y = np.where(s[..., None] > 0, left / np.where(s > 0, s, 1)[..., None], 0).astype(np.float32)
            q = oracle.e2m1_from_float_array(np.ascontiguousarray(y.ravel())).reshape(y.shape)
            part = E2M1[q] * s[..., None]
            total += np.where(live, np.ldexp(part, -ORDERS * p), 0)
            left = left - part
        left = np.ldexp(left, ORDERS)
    return np.ldexp(total.reshape(R, -1), (row - 8)[:, None])


GATE = 8.0


class Differences:
    """One expert, gates of 8, and outputs that are differences of two nearly equal x (the first 248 rows) or h (rows 256 to
    503), so that what the terms leave is large against the bf16 of the output. Weights are exact: 0, 1 and -1."""
    H, I, PAIRS = 512, 768, 248

    def __init__(self, T=8, seed=0):
        rng = np.random.default_rng(seed)
        x = np.zeros((T, self.H), np.float32)
        v = bf16_bits_to_f32(f32_to_bf16_bits((rng.uniform(0.25, 1, (T, self.PAIRS)) * rng.choice([-1, 1], (T, self.PAIRS)))
                                              .astype(np.float32)))
        x[:, 0:2 * self.PAIRS:2] = v
        x[:, 1:2 * self.PAIRS:2] = bf16_bits_to_f32((f32_to_bf16_bits(v) + 1).astype(np.uint16))   # the next bf16 value
        x[:, -1] = GATE
        self.x = x
        P, H, I = self.PAIRS, self.H, self.I
        up, gate, down = np.zeros((I, H), int), np.zeros((I, H), int), np.zeros((H, I), int)
        gate[:, -1] = 1
        m = np.arange(P)
        up[m, 2 * m + 1], up[m, 2 * m] = 1, -1
        up[256 + np.arange(2 * P), np.arange(2 * P)] = 1
        down[m, m] = 1
        down[256 + m, 256 + 2 * m + 1], down[256 + m, 256 + 2 * m] = 1, -1
        self.up, self.gate, self.down = up, gate, down

    @staticmethod
    def codes(w):
        """Weights of 0, 1 and -1 as codes [R, K/2] (1 is code 2)."""
        q = np.where(w == 0, 0, np.where(w > 0, 2, 10)).astype(np.uint8)
        return q[:, 0::2] | (q[:, 1::2] << 4)

    @staticmethod
    def scales(w):
        return interleave(np.full((w.shape[0], w.shape[1] // 16), 0x38, np.uint8))

    def output(self, terms):
        """The layer's output with sums of `terms` blocks, in 64 bits but for its bf16."""
        x = split(self.x, terms)
        h = (x @ self.up.T) * silu(x @ self.gate.T)
        y = split(h.astype(np.float32), terms) @ self.down.T
        return bf16_bits_to_f32(f32_to_bf16_bits(y.astype(np.float32))).astype(np.float64)

    def errors(self, out):
        """Root mean square of the differences' errors, in units of the largest magnitude of their x's block, and the largest:
        for the differences of x and of h."""
        P = self.PAIRS
        x = self.x.astype(np.float64)
        want = x[:, 1:2 * P:2] - x[:, 0:2 * P:2]
        most = np.repeat(np.abs(x[:, :2 * P]).reshape(len(x), -1, 16).max(2), 8, axis=1)
        e = [(out[:, at:at + P] / silu(GATE) - want) / most for at in (0, 256)]
        return [float(np.sqrt((v ** 2).mean())) for v in e], [float(np.abs(v).max()) for v in e]

    # A term leaves typically a twelfth of the block's largest: five 2^-17.9, four 2^-14.3. A difference has two of these, the
    # differences of h also two of h's own; the output's bf16 adds at most 2^-17. So the root mean squares are about 2^-16.9 and
    # 2^-16.6 with five terms, and 2^-13.8 or more with four: the limits lie between.
    RMS = (2.0 ** -16, 2.0 ** -15.5)
    # at worst 2^-12 of the block's largest for each of two, and of two of h
    MOST = (2.0 ** -11 + 2.0 ** -17, 2.0 ** -10 + 2.0 ** -17)

    def holds(self, out):
        rms, most = self.errors(out)
        return all(r <= lim for r, lim in zip(rms, self.RMS)) and all(r <= lim for r, lim in zip(most, self.MOST))
