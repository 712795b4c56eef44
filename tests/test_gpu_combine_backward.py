"""The combine's gradient against 64 bits, against differences, and beside the combine itself."""
import numpy as np
import pytest
import torch

from _block import HALF, acc, along, close
from _harness import filled, moe

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, H, E, K, masked=False, align=1, invalid=0.2, M=0, seed=0):
        m = moe()
        self.T, self.H, self.E, self.K, self.mode = T, H, E, K, "masked" if masked else "normal"
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
        self.ids[torch.rand(T, K, device="cuda", generator=gen) < invalid] = -1
        self.w = torch.rand(T, K, device="cuda", generator=gen) - 0.3
        self.status = m.new_status()
        self.M = M or (T if masked else 0)
        self.seg = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        self.s2d = torch.empty(T * K, dtype=torch.int32, device="cuda")
        reorder = torch.empty(T * K + E * (align - 1), dtype=torch.int32, device="cuda")
        mm = torch.empty(E, dtype=torch.int32, device="cuda")
        m.moe_route_meta_ex(self.ids, E, self.seg, self.s2d, reorder, mm, self.status, m.new_workspace(T, K, E),
                            expert_alignment=align)
        self.rows = E * self.M if masked else T * K + E * (align - 1)
        d = self.s2d.long().view(T, K)
        if masked:
            e = self.ids.long().clamp(min=0)
            rank = d - self.seg[e]
            self.row = torch.where((self.ids >= 0) & (rank < self.M), e * self.M + rank, -1)
        else:
            self.row = torch.where(self.ids >= 0, d, -1)
        self.grad = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
        self.eo = torch.full((self.rows, H), float("nan"), device="cuda", dtype=torch.bfloat16)
        used = self.row[self.row >= 0]
        self.eo[used] = torch.randn(len(used), H, device="cuda", generator=gen).bfloat16()
        self.args = dict(max_tokens_per_expert=self.M, expert_out_rows=0 if masked else self.rows)

    def run(self, eo, rows, w, stream=None):
        moe().moe_combine_backward(self.mode, self.grad, eo, self.ids, self.w, self.E, self.s2d, self.seg, rows, w,
                                   self.status, stream=stream, **self.args)

    def check(self, rows, w):
        torch.cuda.synchronize()
        t, k = torch.nonzero(self.row >= 0, as_tuple=True)
        at = self.row[t, k]
        g = self.grad[t].double()
        if rows is not None:
            want = g * self.w[t, k].double()[:, None]
            close(rows[at], want, (HALF[torch.bfloat16] + 2.0 ** -23) * want.abs())
            free = torch.ones(self.rows, dtype=torch.bool, device="cuda")
            free[at] = False
            assert bool((rows[free].view(torch.uint8) == 0xa5).all())
        if w is not None:
            want, mag = torch.zeros_like(self.w, dtype=torch.float64), torch.zeros_like(self.w, dtype=torch.float64)
            want[t, k], mag[t, k] = (g * self.eo[at].double()).sum(-1), (g * self.eo[at].double()).abs().sum(-1)
            # a lane adds 16 products of each of its slices, then nine steps join lanes and warps
            close(w, want, 1.01 * acc(16 * (self.H // 512 + 1)) * mag)


@pytest.mark.parametrize("what", ["both", "rows", "weights"])
@pytest.mark.parametrize("T,H,E,K,kw", [
    (1, 8, 1, 1, dict(invalid=0.0)), (1, 4096, 16, 8, dict(invalid=0.0)), (37, 264, 8, 3, dict()),
    (64, 1032, 32, 9, dict(align=16)), (20, 512, 24, 16, dict(align=128)), (130, 2120, 8, 2, dict(masked=True)),
    (50, 7168, 16, 16, dict(masked=True, invalid=0.5)), (9, 520, 4, 4, dict(invalid=1.0)), (300, 128, 6, 6, dict(masked=True, invalid=0.0))])
def test_gradient(T, H, E, K, kw, what):
    c = Case(T, H, E, K, **kw)
    rows = filled((c.rows, H), torch.bfloat16) if what != "weights" else None
    w = filled((T, K), torch.float32) if what != "rows" else None
    c.run(c.eo if what != "rows" else None, rows, w)
    c.check(rows, w)
    assert int(c.status) == 0


def test_rows_in_place():
    c = Case(40, 1032, 8, 3, align=4)
    want, w0 = filled((c.rows, c.H), torch.bfloat16), torch.zeros(40, 3, device="cuda")
    c.run(c.eo, want, w0)
    eo, w1 = c.eo.clone(), torch.zeros_like(w0)
    c.run(eo, eo, w1)
    torch.cuda.synchronize()
    at = c.row[c.row >= 0]
    assert torch.equal(eo[at], want[at]) and torch.equal(w0, w1)


def test_gradient_against_differences():
    """Of the combine in 64 bits, whose value the library's combine is shown to have."""
    m = moe()
    c = Case(12, 64, 5, 3, invalid=0.3, seed=3)
    eo = c.eo.double().nan_to_num(0)
    t, k = torch.nonzero(c.row >= 0, as_tuple=True)

    def combine(eo, w):
        out = torch.zeros(c.T, c.H, dtype=torch.float64, device="cuda")
        return out.index_add_(0, t, eo[c.row[t, k]] * w[t, k][:, None])

    out = torch.zeros(c.T, c.H, dtype=torch.bfloat16, device="cuda")
    m.moe_combine_ex("normal", c.eo, c.ids, c.w, c.E, c.s2d, c.seg, out, c.status, expert_out_rows=c.rows)
    wd = c.w.double()
    close(out, combine(eo, wd), HALF[torch.bfloat16] * combine(eo, wd).abs() + acc(3) * combine(eo.abs(), wd.abs()))
    rows, gw = torch.zeros(c.rows, c.H, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.T, c.K, device="cuda")
    c.run(c.eo, rows, gw)
    gen, g = torch.Generator(device="cuda").manual_seed(4), c.grad.double()
    for _ in range(4):
        d = torch.randn(eo.shape, device="cuda", generator=gen, dtype=torch.float64)
        want = float(((combine(eo + d, wd) - combine(eo - d, wd)) / 2 * g).sum())
        terms = rows.double() * d
        assert abs(float(terms.sum()) - want) <= 1.01 * HALF[torch.bfloat16] * float(terms.abs().sum())
        d = torch.randn(wd.shape, device="cuda", generator=gen, dtype=torch.float64)
        want = float(((combine(eo, wd + d) - combine(eo, wd - d)) / 2 * g).sum())
        assert abs(float((gw.double() * d).sum()) - want) <= 1e-5 * float((gw.double() * d).abs().sum()) + 1e-5


def test_reported_slots():
    """What the combine reports and skips is reported and skipped alike."""
    m = moe()
    c = Case(10, 128, 4, 2, masked=True, invalid=0.0, M=3, seed=5)      # more pairs than slots: the rest has no row
    rows, w = filled((c.rows, c.H), torch.bfloat16), filled((10, 2), torch.float32)
    c.run(c.eo, rows, w)
    c.check(rows, w)
    c.status.zero_()
    c.ids[3, 1] = 99
    c.row[3, 1] = -1
    rows, w = filled((c.rows, c.H), torch.bfloat16), filled((10, 2), torch.float32)
    c.run(c.eo, rows, w)
    c.check(rows, w)
    assert int(c.status) == m.MOE_ERR_BAD_EXPERT_ID
    n = Case(10, 128, 4, 2, invalid=0.0, seed=6)
    n.s2d[5] = n.rows + 7
    n.row[2, 1] = -1
    rows, w = filled((n.rows, n.H), torch.bfloat16), filled((10, 2), torch.float32)
    n.run(n.eo, rows, w)
    n.check(rows, w)
    assert int(n.status) == m.MOE_ERR_INVALID_ARG


def test_tokens_that_are_not_finite_stay_alone():
    c = Case(20, 520, 6, 3, invalid=0.0, seed=7)
    outs = []
    for bad in (False, True):
        if bad:
            c.grad[4, ::2] = float("nan")
            c.eo[c.row[9, 1], ::5] = float("inf")
        rows, w = torch.zeros(c.rows, c.H, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, 3, device="cuda")
        c.run(c.eo, rows, w)
        rows[c.row[4]] = 0
        w[4] = 0
        w[9, 1] = 0
        outs.append((rows, w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_streams_graphs_and_repetition():
    c = Case(200, 2056, 16, 6, seed=8)

    def fresh():
        return torch.zeros(c.rows, c.H, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.T, c.K, device="cuda")

    want = fresh()
    c.run(c.eo, *want)
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [fresh() for _ in streams]
    torch.cuda.synchronize()
    for s, g in zip(streams, got):
        c.run(c.eo, *g, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    got = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(c.eo, *got)
    got[1].fill_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    m = moe()
    M, H, T, E = 600000, 4096, 3, 2
    ids = torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda")
    meta = m.route_meta(ids, E)
    eo = torch.zeros(E * M, H, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(9)
    at = torch.tensor([0, M, M + 1], device="cuda")
    eo[at] = torch.randn(3, H, device="cuda", generator=gen).bfloat16()
    grad = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    want = (grad.double() * eo[at].double()).sum(-1, keepdim=True)
    mag = (grad.double() * eo[at].double()).abs().sum(-1, keepdim=True)
    w, st = torch.zeros(T, 1, device="cuda"), m.new_status()
    m.moe_combine_backward("masked", grad, eo, ids, torch.full((T, 1), 0.5, device="cuda"), E, meta.src2dst,
                           meta.seg_indptr, eo, w, st, max_tokens_per_expert=M)
    torch.cuda.synchronize()
    assert int(st) == 0
    close(w, want, acc(16 * 9) * mag)
    assert torch.equal(eo[at], (grad.float() * 0.5).bfloat16())
    assert np.isclose(float(eo.view(-1).count_nonzero()), float((grad * 0.5).count_nonzero()))


def test_gradient_along_itself():
    c = Case(12, 64, 5, 3, invalid=0.3, seed=3)
    t, k = torch.nonzero(c.row >= 0, as_tuple=True)
    eo, g, wd = c.eo.double().nan_to_num(0), c.grad.double(), c.w.double()

    def loss(de, dw):
        return float(((eo + de)[c.row[t, k]] * (wd + dw)[t, k][:, None] * g[t]).sum())

    rows, gw = torch.zeros(c.rows, c.H, dtype=torch.bfloat16, device="cuda"), torch.zeros(c.T, c.K, device="cuda")
    c.run(c.eo, rows, gw)
    torch.cuda.synchronize()
    along(rows, 1.01 * HALF[torch.bfloat16] * rows.double().abs(), lambda d: loss(d, 0), 5)
    terms = torch.zeros_like(wd)
    terms[t, k] = (eo[c.row[t, k]].abs() * g[t].abs()).sum(-1)
    along(gw, 2 * acc(64) * terms, lambda d: loss(0, d), 6)
