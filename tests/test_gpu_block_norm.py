"""The root-mean-square norm, its FP8 rows and its gradient, against 64 bits."""
import pytest
import torch

from _block import HALF, acc, along, close
from _harness import bytes_of, filled, moe

pytestmark = pytest.mark.gpu

EPS = 1e-6
B = HALF[torch.bfloat16]
# r: a thread adds 32 squares at most, ten steps join threads: 42 roundings, half of them in the root, and four more
R = 2.0 ** -19
SIZES = [(1, 8), (3, 128), (7, 256), (5, 264), (33, 512), (2, 1024), (9, 1032), (4, 2176), (130, 4096), (3, 7168), (2, 8192),
         (2, 8200), (1, 16384), (2, 32768), (700, 136)]


def _inputs(T, H, residual=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    big = 1 + 20 * (torch.rand(H, device="cuda", generator=gen) < 0.02)
    x = (torch.randn(T, H, device="cuda", generator=gen) * big).bfloat16()
    res = (torch.randn(T, H, device="cuda", generator=gen) * 3 * big).bfloat16() if residual else None
    return x, res, (1 + 0.2 * torch.randn(H, device="cuda", generator=gen)).bfloat16(), gen


def _norm64(x, res, w, eps=EPS):
    s = x if res is None else (x.float() + res.float()).bfloat16()
    r = (s.double().square().mean(-1) + eps).rsqrt()
    return s, r, s.double() * r[:, None] * w.double()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SIZES)
def test_bf16(T, H, residual):
    x, res, w, _ = _inputs(T, H, residual)
    y = moe().rmsnorm(x, w, EPS, residual=res, keep=True)
    s, r, want = _norm64(x, res, w)
    assert y.codes is None and y.scales is None
    assert torch.equal(y.sum, s) and (y.sum is x) == (res is None)
    close(y.rstd, r, R * r)
    close(y.out, want, (B + 2 * R) * want.abs())


@pytest.mark.parametrize("quant", ["fp8g128", "fp8g128_ue8m0"])
@pytest.mark.parametrize("T,H", [(T, H) for T, H in SIZES if H % 128 == 0])
def test_fp8(T, H, quant):
    x, res, w, _ = _inputs(T, H, seed=1)
    x[0, :128], res[0, :128] = 0, 0                    # a group of zeros: the least scale
    y = moe().rmsnorm(x, w, EPS, residual=res, quant=quant, bf16=True)
    s, _, want = _norm64(x, res, w)
    assert torch.equal(y.sum, s) and y.rstd is None
    close(y.out, want, (B + 2 * R) * want.abs())
    groups = want.view(T, -1, 128)
    scale = groups.abs().amax(-1).clamp(min=1e-10) / 448
    if quant == "fp8g128":
        assert y.scales.dtype == torch.float32
        close(y.scales, scale, 4 * R * scale)
        got = y.scales.double()
    else:
        got = torch.ldexp(torch.ones_like(scale), y.scales.int() - 127)
        assert bool(((got >= scale * (1 - 4 * R)) & (got <= 2 * scale * (1 + 4 * R))).all())
    values = y.codes.view(torch.float8_e4m3fn).double().view(T, -1, 128) * got[..., None]
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its normal numbers
    close(values, groups, (2.0 ** -4 + 4 * R) * groups.abs() + 2.0 ** -10 * got[..., None])
    only = moe().rmsnorm(x, w, EPS, residual=res, quant=quant)
    assert only.out is None and torch.equal(only.codes, y.codes) and torch.equal(only.scales, y.scales)


def test_fp8_rows_are_the_dispatchs():
    """Where a row's values are exact in bf16, codes and scales are the dispatch's, bit for bit: a row of +-2^j has
    mean square m, and eps is chosen so that 1 / sqrt(m + eps) is a power of two."""
    m = moe()
    T, H = 6, 512
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.where(torch.rand(T, H, device="cuda", generator=gen) < 0.5, -1.0, 1.0)
    x = (x * torch.tensor([0.5, 1.0], device="cuda")[torch.arange(H, device="cuda") % 2]).bfloat16()   # m = 0.625
    w = (0.01 + torch.rand(H, device="cuda", generator=gen)).bfloat16()
    ids = torch.arange(T, dtype=torch.int32, device="cuda")[:, None].contiguous()
    for quant in ("fp8g128", "fp8g128_ue8m0"):
        y = m.rmsnorm(x, w, 0.375, quant=quant, bf16=True, keep=True)
        assert bool((y.rstd == 1).all())
        meta = m.route_meta(ids, T)
        st = m.new_status()
        codes = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
        scales = torch.zeros_like(y.scales)
        m.moe_dispatch_ex("normal", quant, "row", y.out, ids, T, meta.src2dst, meta.seg_indptr, codes, scales, st)
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(codes, y.codes) and torch.equal(scales, y.scales)


def test_fp8_rows_through_the_dispatch():
    """Codes and scale rows pass through the dispatch as bytes."""
    m = moe()
    T, H, E, K = 50, 1024, 6, 2
    x, res, w, gen = _inputs(T, H, seed=3)
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
    y = m.rmsnorm(x, w, EPS, residual=res, quant="fp8g128")
    meta = m.route_meta(ids, E)
    st = m.new_status()
    codes = torch.zeros(T * K, H, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(T * K, H // 128, device="cuda")
    for rows, out in ((y.codes, codes), (y.scales.view(torch.uint8), scales.view(torch.uint8))):
        m.moe_dispatch_ex("normal", "fp8_passthrough", "row", rows, ids, E, meta.src2dst, meta.seg_indptr, out, None, st)
    torch.cuda.synchronize()
    assert int(st) == 0
    at = meta.src2dst.long()
    token = torch.arange(T * K, device="cuda") // K
    assert torch.equal(codes[at], y.codes[token]) and torch.equal(scales[at], y.scales[token])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SIZES + [(0, 136), (1300, 1024), (1000, 264)])
def test_gradient(T, H, residual):
    m = moe()
    x, res, w, gen = _inputs(T, H, residual, 4)
    y = m.rmsnorm(x, w, EPS, residual=res, keep=True)
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    gs = torch.randn(T, H, device="cuda", generator=gen).bfloat16() if residual else None
    dx, dw = m.rmsnorm_backward(g, y.sum, w, y.rstd, grad_residual=gs)
    leaf = y.sum.double().requires_grad_()
    wd = w.double().requires_grad_()
    r = (leaf.square().mean(-1) + EPS).rsqrt()
    (leaf * r[:, None] * wd).backward(g.double())
    want = leaf.grad + (gs.double() if residual else 0)
    hat, gw = (leaf * r[:, None]).detach().abs(), (g.double() * w.double()).abs()
    parts = r.detach()[:, None] * (gw + hat * (gw * hat).mean(-1, keepdim=True))
    # r to R, the mean by 43 roundings of its terms, four more of the two terms before they cancel
    close(dx, want, B * want.abs() + 6 * R * parts + 2.0 ** -23 * (want.abs() + parts))
    close(dw, wd.grad, (2 * R + acc(T)) * (g.double().abs() * hat).sum(0) + 2.0 ** -126)


def test_gradient_against_differences():
    m = moe()
    T, H = 5, 64
    x, res, w, gen = _inputs(T, H, seed=5)
    y = m.rmsnorm(x, w, EPS, residual=res, keep=True)
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    dx, dw = m.rmsnorm_backward(g, y.sum, w, y.rstd)

    def loss(s, w):
        return float((s * (s.square().mean(-1, keepdim=True) + EPS).rsqrt() * w * g.double()).sum())

    s, wd, step = y.sum.double(), w.double(), 1e-6
    for _ in range(5):
        d = torch.randn(T, H, device="cuda", generator=gen, dtype=torch.float64)
        want = (loss(s + step * d, wd) - loss(s - step * d, wd)) / (2 * step)
        assert abs(float((dx.double() * d).sum()) - want) <= B * float((dx.double() * d).abs().sum()) + 1e-6
        d = d[0]
        want = (loss(s, wd + step * d) - loss(s, wd - step * d)) / (2 * step)
        assert abs(float((dw.double() * d).sum()) - want) <= 1e-6 * float((dw.double() * d).abs().sum()) + 1e-6


def test_in_place_and_guards():
    m = moe()
    T, H = 37, 1160
    x, res, w, gen = _inputs(T, H, seed=6)
    want = m.rmsnorm(x, w, EPS, residual=res, keep=True)
    for which in ("x", "residual"):
        a, b = x.clone(), res.clone()
        out, rstd = filled((T, H), torch.bfloat16), filled((T,), torch.float32)
        m.moe_rmsnorm(a, w, EPS, out, b, sum=a if which == "x" else b, rstd=rstd)
        torch.cuda.synchronize()
        assert torch.equal(a if which == "x" else b, want.sum) and torch.equal(out, want.out) and torch.equal(rstd, want.rstd)
        assert torch.equal(b if which == "x" else a, res if which == "x" else x)
    g, gs = (torch.randn(T, H, device="cuda", generator=gen).bfloat16() for _ in range(2))
    dx, dw = m.rmsnorm_backward(g, want.sum, w, want.rstd, gs)
    n = m.moe_rmsnorm_backward_workspace_size(T, H)
    for which in (g.clone(), gs.clone()):
        first = torch.equal(which, g)
        got_w, ws = filled((H,), torch.float32), filled((n,), torch.uint8)
        m.moe_rmsnorm_backward(which if first else g, want.sum, w, want.rstd, which, got_w, ws, gs if first else which)
        torch.cuda.synchronize()
        assert torch.equal(which, dx) and torch.equal(got_w, dw)


def test_rows_that_are_not_finite_stay_alone():
    m = moe()
    for H in (256, 2048):
        x, res, w, gen = _inputs(9, H, seed=7)
        want = m.rmsnorm(x, w, EPS, residual=res, quant="fp8g128", bf16=True, keep=True)
        x[3, 5], x[6, 7] = float("nan"), float("inf")
        got = m.rmsnorm(x, w, EPS, residual=res, quant="fp8g128", bf16=True, keep=True)
        keep = [0, 1, 2, 4, 5, 7, 8]
        for a, b in zip(got, want):
            assert torch.equal(a[keep], b[keep])
        assert bool(got.out[3].isnan().all())


def test_zero_rows_and_empty_batches():
    m = moe()
    H = 384
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    z = torch.zeros(4, H, device="cuda", dtype=torch.bfloat16)
    y = m.rmsnorm(z, w, 1e-6, residual=z, quant="fp8g128", bf16=True, keep=True)
    assert not y.out.any() and not (y.codes & 0x7f).any() and bool(y.rstd.isfinite().all())
    dx, dw = m.rmsnorm_backward(torch.ones_like(z), y.sum, w, y.rstd)
    assert bool(dx.isfinite().all()) and not dw.any()
    y = m.rmsnorm(z[:0], w, quant="fp8g128", keep=True)
    assert y.codes.shape == (0, H) and y.scales.shape == (0, 3)


def test_streams_graphs_and_repetition():
    m = moe()
    T, H = 500, 2048
    x, res, w, gen = _inputs(T, H, seed=8)
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()

    def both(stream=None):
        y = m.rmsnorm(x, w, EPS, residual=res, quant="fp8g128", bf16=True, keep=True, stream=stream)
        return (*y, *m.rmsnorm_backward(g, y.sum, w, y.rstd, g, stream=stream))

    want = both()
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [both(s) for _ in range(2) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.view(torch.uint8).fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all((bytes_of(a) == bytes_of(b)).all() for a, b in zip(got, want))


def test_offsets_past_32_bits():
    m = moe()
    T, H = 70000, 32768
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(9)
    x[-2:] = torch.randn(2, H, device="cuda", generator=gen)
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    y = m.rmsnorm(x, w, EPS, quant="fp8g128", bf16=True, keep=True)
    last = m.rmsnorm(x[-2:].contiguous(), w, EPS, quant="fp8g128", bf16=True, keep=True)
    for a, b in zip(y, last):
        assert torch.equal(a[-2:], b)
    dx, _ = m.rmsnorm_backward(y.out, x, w, y.rstd)
    want, _ = m.rmsnorm_backward(last.out, x[-2:].contiguous(), w, last.rstd)
    assert torch.equal(dx[-2:], want)


# Gradients of so many values have their rows on the way in shared memory, two or four of them.
AHEAD = [(2049, 8192), (4111, 4104), (8200, 2056), (16400, 1032), (2347, 7168)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", AHEAD)
def test_gradient_of_many_rows(T, H, residual):
    test_gradient(T, H, residual)


@pytest.mark.parametrize("T,H", AHEAD[:3])
def test_gradient_of_many_rows_in_place(T, H):
    m = moe()
    x, res, w, gen = _inputs(T, H, seed=8)
    y = m.rmsnorm(x, w, EPS, residual=res, keep=True)
    g, gs = (torch.randn(T, H, device="cuda", generator=gen).bfloat16() for _ in range(2))
    dx, dw = m.rmsnorm_backward(g, y.sum, w, y.rstd, gs)
    n = m.moe_rmsnorm_backward_workspace_size(T, H)
    for first in (True, False):
        which = (g if first else gs).clone()
        got_w, ws = filled((H,), torch.float32), filled((n,), torch.uint8)
        m.moe_rmsnorm_backward(which if first else g, y.sum, w, y.rstd, which, got_w, ws, gs if first else which)
        torch.cuda.synchronize()
        assert torch.equal(which, dx) and torch.equal(got_w, dw)


@pytest.mark.parametrize("T,H", [(900, 12288), (700, 16384), (611, 10240)])
def test_long_rows(T, H):
    test_bf16(T, H, True)
    test_fp8(T, H, "fp8g128")


def test_gradient_along_itself():
    m = moe()
    T, H = 5, 64
    x, res, w, gen = _inputs(T, H, seed=5)
    y = m.rmsnorm(x, w, EPS, residual=res, keep=True)
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    dx, dw = m.rmsnorm_backward(g, y.sum, w, y.rstd)
    s, wd, gd = y.sum.double(), w.double(), g.double()

    def loss(ds, dw):
        v = s + ds
        return float((v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * (wd + dw) * gd).sum())

    # as in test_gradient
    r = (s.square().mean(-1, keepdim=True) + EPS).rsqrt()
    hat, gw = (s * r).abs(), (gd * wd).abs()
    parts = r * (gw + hat * (gw * hat).mean(-1, keepdim=True))
    along(dx, 1.01 * B * dx.double().abs() + 7 * R * parts, lambda c: loss(c, 0), 20)
    along(dw, 2 * (2 * R + acc(T)) * (gd.abs() * hat).sum(0), lambda c: loss(0, c), 21)


@pytest.mark.parametrize("mode", ["normal", "masked"])
@pytest.mark.parametrize("quant", ["fp8g128", "fp8g128_ue8m0"])
@pytest.mark.parametrize("H", [2048, 2176, 7168])
def test_padded_scale_rows_through_the_dispatch(H, quant, mode):
    m = moe()
    T, E, K = 33, 6, 2
    x, res, w, gen = _inputs(T, H, seed=11)
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
    y = m.rmsnorm(x, w, EPS, residual=res, quant=quant)
    scale_bytes = y.scales.view(torch.uint8).view(T, -1)
    n = scale_bytes.shape[1]
    padded = torch.zeros(T, (n + 31) // 32 * 32, dtype=torch.uint8, device="cuda")
    padded[:, :n] = scale_bytes
    meta, st = m.route_meta(ids, E), m.new_status()
    rows, M = (T * K, 0) if mode == "normal" else (E * T, T)
    outs = []
    for src in (y.codes, padded):
        out = torch.zeros(rows, src.shape[1], dtype=torch.uint8, device="cuda")
        m.moe_dispatch_ex(mode, "fp8_passthrough", "row", src, ids, E, meta.src2dst, meta.seg_indptr, out, None, st,
                          max_tokens_per_expert=M)
        outs.append(out)
    torch.cuda.synchronize()
    assert int(st) == 0
    at, token, e = meta.src2dst.long(), torch.arange(T * K, device="cuda") // K, ids.flatten().long()
    if mode == "masked":
        at = e * T + at - meta.seg_indptr[e]
    assert torch.equal(outs[0][at], y.codes[token]) and torch.equal(outs[1][at, :n], scale_bytes[token])
