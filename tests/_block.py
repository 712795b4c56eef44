"""Inputs and bounds for the tests of a MoE block's bf16 operators. References are in 64 bits."""
import numpy as np
import torch

from _experts import layout, rows_of

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # a rounding, relative to the value


def acc(terms):
    """Error of an fp32 sum of `terms` products relative to the sum of their magnitudes: 2^-24 for each partial sum that is
    rounded, and for what a matrix instruction cuts as it lines up 16 products, in whatever order."""
    return (terms + 32) * 2.0 ** -24


class Rows:
    """A layout's rows: counts, first rows, the arguments that say so, and buffers whose unused rows are NaN."""

    def __init__(self, mode, counts, M=0, align=1, spare=0, seed=0):
        self.mode, self.counts, self.M = mode, np.asarray(counts), M
        self.base, seg, self.rows = layout(mode, counts, M, align, spare)
        used = rows_of(self.base, self.counts)
        self.used = torch.from_numpy(used).cuda()
        self.expert = torch.from_numpy(np.repeat(np.arange(len(counts)), self.counts)).cuda()
        self.count = torch.from_numpy(self.counts.astype(np.int32)).cuda()
        self.where = dict(seg_indptr=torch.from_numpy(seg).cuda() if mode == "normal" else None, max_tokens_per_expert=M)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @property
    def E(self):
        return len(self.counts)

    def values(self, width, std=1.0):
        """bf16 rows of N(0, std^2), NaN where no expert's row lies."""
        x = torch.full((self.rows, width), float("nan"), dtype=torch.bfloat16, device="cuda")
        x[self.used] = (torch.randn(len(self.used), width, device="cuda", generator=self.gen) * std).bfloat16()
        return x

    def weights(self, *shape):
        return (torch.randn(self.E, *shape, device="cuda", generator=self.gen) * shape[-1] ** -0.5).bfloat16()

    def each(self):
        """(expert, its rows as a slice) of all experts, without rows too."""
        return [(e, slice(int(b), int(b) + int(c))) for e, (b, c) in enumerate(zip(self.base, self.counts))]

    def per_expert(self, x, f):
        """f(rows of x in 64 bits, e) of every expert, in the layout's rows; zeros elsewhere."""
        out = None
        for e, at in self.each():
            y = f(x[at].double(), e)
            if out is None:
                out = torch.zeros(self.rows, y.shape[1], dtype=torch.float64, device="cuda")
            out[at] = y
        return out

    def ok(self):
        torch.cuda.synchronize()
        assert int(self.status) == 0


def untouched(out, rows, fill):
    """Whether the rows of `out` that no expert has still hold the byte `fill`."""
    free = torch.ones(rows.rows, dtype=torch.bool, device="cuda")
    free[rows.used] = False
    return bool((out.view(rows.rows, -1)[free].view(torch.uint8) == fill).all())


def close(got, want, bound):
    """Every value within its bound, and finite; names the worst."""
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    if bad.any():
        i = int(torch.where(bad, d / bound.clamp(min=1e-300), torch.zeros_like(d)).nan_to_num(1e300).argmax())
        at = np.unravel_index(i, tuple(got.shape))
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} values off, worst at {tuple(int(v) for v in at)}: got "
                             f"{float(got.flatten()[i])}, want {float(want.flatten()[i])} within {float(bound.flatten()[i])}")


def along(grad, bound, loss, seed, step=1e-5):
    """`grad`, whose values are within `bound` of the gradient, against differences of loss(change) in 64 bits. Directions have
    the gradient's own signs: the derivative is then as large as what the roundings of its terms could add up to is small,
    2^-8 of it, and the same bound refuses a gradient that is 5 % too large or too small, or lacks a part as large. The
    differences themselves are good to 1e-6 of it."""
    gen = torch.Generator(device=grad.device).manual_seed(seed)
    g = grad.double().nan_to_num(0)
    for _ in range(4):
        d = g.sign() * torch.randn(g.shape, device=g.device, generator=gen, dtype=torch.float64).abs()
        want = (loss(step * d) - loss(-step * d)) / (2 * step)
        got = float((g * d).sum())
        most = float((bound * d.abs()).sum()) + 1e-6 * abs(want)
        assert got > 0 and abs(got - want) <= most, (got, want, most)
        assert abs(1.05 * got - want) > most and abs(0.95 * got - want) > most, (got, want, most)
