"""The bf16 products over a layout's experts and their gradients, against 64 bits."""
import numpy as np
import pytest
import torch

from _block import HALF, Rows, acc, along, close, untouched
from _harness import filled, moe

pytestmark = pytest.mark.gpu

LAYOUTS = [
    ("normal", [1], dict()),
    ("normal", [5, 0, 130, 1, 64, 255], dict()),
    ("normal", [256, 257, 0, 512, 31, 33], dict(spare=3)),
    ("normal", [3, 0, 0, 140, 17], dict(align=128, spare=1)),
    ("normal", [700, 2], dict(align=16)),
    ("normal", [0, 0, 0], dict(spare=5)),
    ("masked", [1, 0, 7, 8, 2, 3, 0, 1], dict(M=8)),
    ("masked", [300, 0, 299, 17], dict(M=300)),
    ("masked", [1] * 5, dict(M=1)),
]
SHAPES = [(8, 8), (64, 128), (136, 72), (264, 200), (520, 1544), (256, 64), (128, 8), (1032, 320)]
CASES = [(i, s) for i in range(len(LAYOUTS)) for s in (SHAPES if i in (1, 2) else SHAPES[2 + i % 3:5 + i % 3:2])]


def _rows(i, seed=0):
    mode, counts, kw = LAYOUTS[i]
    return Rows(mode, counts, seed=seed, **kw)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("i,shape", CASES)
def test_product(i, shape, transposed):
    n, k = shape
    r = _rows(i)
    a = r.values(k)
    w = r.weights(*((k, n) if transposed else (n, k)))
    out = filled((r.rows, n), torch.bfloat16)
    moe().moe_expert_gemm_bf16(r.mode, a, r.count, w, out, r.status, transposed=transposed, **r.where)
    r.ok()
    m = [v.double() if transposed else v.double().T for v in w]
    want = r.per_expert(a, lambda x, e: x @ m[e])
    mag = r.per_expert(a, lambda x, e: x.abs() @ m[e].abs())
    close(out[r.used], want[r.used], (HALF[torch.bfloat16] * want.abs() + 1.01 * acc(k) * mag)[r.used])
    assert untouched(out, r, 0xa5)


def _swiglu64(G, U):
    p = torch.sigmoid(G)
    return U * G * p, U * p * (1 + G * (1 - p)), G * p       # h, dh/dG, dh/dU


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("i,shape", CASES)
def test_swiglu(i, shape, keep):
    I, k = shape
    r = _rows(i, 1)
    a, w = r.values(k, 2.0), r.weights(2 * I, k)
    h, gu = filled((r.rows, I), torch.bfloat16), filled((r.rows, 2 * I), torch.bfloat16) if keep else None
    moe().moe_expert_gemm_swiglu_bf16(r.mode, a, r.count, w, h, r.status, gate_up=gu, **r.where)
    r.ok()
    y = r.per_expert(a, lambda x, e: x @ w[e].double().T)[r.used]
    err = 1.01 * acc(k) * r.per_expert(a, lambda x, e: x.abs() @ w[e].double().abs().T)[r.used]
    G, U = y[:, :I], y[:, I:]
    want, dG, dU = _swiglu64(G, U)
    # |d silu| <= 1.1 everywhere: the sums' errors reach h by both factors, their product too
    bound = 1.1 * err[:, :I] * (U.abs() + err[:, I:]) + dU.abs() * err[:, I:] + (HALF[torch.bfloat16] + 2.0 ** -19) * want.abs()
    close(h[r.used], want, bound)
    assert untouched(h, r, 0xa5)
    if keep:
        close(gu[r.used], y, HALF[torch.bfloat16] * y.abs() + err)
        assert untouched(gu, r, 0xa5)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("i,shape", CASES)
def test_dswiglu(i, shape, inplace):
    I, k = shape
    r = _rows(i, 2)
    g, gu, w2 = r.values(k), r.values(2 * I, 3.0), r.weights(k, I)
    saved = gu.clone()
    out = gu if inplace else filled((r.rows, 2 * I), torch.bfloat16)
    moe().moe_expert_gemm_dswiglu_bf16(r.mode, g, r.count, w2, gu, out, r.status, **r.where)
    r.ok()
    dh = r.per_expert(g, lambda x, e: x @ w2[e].double())[r.used]
    err = 1.01 * acc(k) * r.per_expert(g, lambda x, e: x.abs() @ w2[e].double().abs())[r.used]
    G, U = saved[r.used, :I].double(), saved[r.used, I:].double()
    _, dG, dU = _swiglu64(G, U)
    p, q = torch.sigmoid(G), torch.sigmoid(-G)
    # the factors' own errors, of the terms of 1 + G q before they cancel: four roundings and p, q to 2^-20
    parts = U.abs() * p * (1 + G.abs() * q)
    bG = (dG.abs() + 2.0 ** -18 * parts) * err + dh.abs() * 2.0 ** -18 * parts + HALF[torch.bfloat16] * (dh * dG).abs()
    bU = dU.abs() * err + (HALF[torch.bfloat16] + 2.0 ** -18) * (dh * dU).abs()
    close(out[r.used, :I], dh * dG, bG + 2.0 ** -130)
    close(out[r.used, I:], dh * dU, bU + 2.0 ** -130)
    if not inplace:
        assert untouched(out, r, 0xa5)
        assert torch.equal(gu.view(torch.int16), saved.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("i,shape", CASES)
def test_weight_gradient(i, shape, dtype, accumulate):
    m, n = shape
    r = _rows(i, 3)
    a, b = r.values(m), r.values(n)
    out = filled((r.E, m, n), dtype)
    base = torch.zeros(r.E, m, n, dtype=torch.float64, device="cuda")
    if accumulate:
        out.copy_(torch.randn(r.E, m, n, device="cuda", generator=r.gen))
        base = out.double()
    moe().moe_expert_wgrad_bf16(r.mode, a, b, r.count, out, r.status, accumulate=accumulate, **r.where)
    r.ok()
    for e, at in r.each():
        x, y = a[at].double(), b[at].double()
        want, err = base[e] + x.T @ y, 1.01 * acc(int(r.counts[e])) * (x.abs().T @ y.abs())
        close(out[e], want, HALF[dtype] * want.abs() + 2.0 ** -24 * (want.abs() + base[e].abs()) + err)
        if not r.counts[e]:
            assert torch.equal(out[e].double(), base[e])


def test_gradients_against_differences():
    """The gradients of a small chain, gate and up to the down product, against differences of the loss in 64 bits."""
    m = moe()
    r = Rows("normal", [3, 0, 6, 2], align=4, seed=5)
    H, I = 24, 16
    x, w13, w2, g = r.values(H), r.weights(2 * I, H), r.weights(H, I), r.values(H)
    h, gu = torch.zeros(r.rows, I, device="cuda").bfloat16(), torch.zeros(r.rows, 2 * I, device="cuda").bfloat16()
    m.moe_expert_gemm_swiglu_bf16("normal", x, r.count, w13, h, r.status, gate_up=gu, **r.where)
    d, dx = torch.zeros_like(gu), torch.zeros_like(x)
    m.moe_expert_gemm_dswiglu_bf16("normal", g, r.count, w2, gu, d, r.status, **r.where)
    m.moe_expert_gemm_bf16("normal", d, r.count, w13, dx, r.status, transposed=True, **r.where)
    d13, d2 = torch.zeros_like(w13, dtype=torch.float32), torch.zeros_like(w2, dtype=torch.float32)
    m.moe_expert_wgrad_bf16("normal", d, x, r.count, d13, r.status, **r.where)
    m.moe_expert_wgrad_bf16("normal", g, h, r.count, d2, r.status, **r.where)
    r.ok()

    def loss(x, w13, w2):
        total = 0.0
        for e, at in r.each():
            y = x[at] @ w13[e].T
            total = total + ((y[:, I:] * torch.nn.functional.silu(y[:, :I])) @ w2[e].T * g[at].double()).sum()
        return float(total)

    v = [x.double().nan_to_num(0), w13.double(), w2.double()]
    gen = torch.Generator(device="cuda").manual_seed(6)
    for i, grad in enumerate((dx, d13, d2)):
        for _ in range(4):
            direction = torch.randn(v[i].shape, device="cuda", generator=gen, dtype=torch.float64)
            if i == 0:
                mask = torch.zeros(r.rows, 1, dtype=torch.float64, device="cuda")
                mask[r.used] = 1
                direction *= mask
            step = 1e-5
            up, down = ([t + s * step * direction if j == i else t for j, t in enumerate(v)] for s in (1, -1))
            want = (loss(*up) - loss(*down)) / (2 * step)
            got = float((grad.double().nan_to_num(0) * direction).sum())
            # four roundings to bf16 on the way (h, gate_up, its gradient, the result), 2^-8 each of terms that a
            # direction adds up in random signs
            scale = float((grad.double().nan_to_num(0).abs() * direction.abs()).sum())
            assert abs(got - want) <= 4 * 2.0 ** -8 * scale, (i, got, want)


@pytest.mark.parametrize("op", ["product", "transposed", "swiglu", "dswiglu", "weights"])
def test_rows_that_are_not_finite_stay_alone(op):
    """Infinities and NaNs in one expert's row leave the other rows' and experts' results as they are, bit for bit."""
    m = moe()
    r = Rows("normal", [40, 33, 0, 5], seed=7)
    n, k = 72, 136
    a, w, gu = r.values(k), r.weights(2 * n, k), r.values(2 * n)
    poisoned = a.clone()
    bad = int(r.base[1]) + 4
    poisoned[bad, ::3] = float("nan")
    poisoned[bad, 1::3] = float("inf")
    outs = []
    for x in (a, poisoned):
        if op == "weights":
            out = torch.zeros(r.E, k, 2 * n, device="cuda")
            m.moe_expert_wgrad_bf16("normal", x, gu, r.count, out, r.status, **r.where)
            out[1] = 0
        elif op == "swiglu":
            out = torch.zeros(r.rows, n, device="cuda", dtype=torch.bfloat16)
            m.moe_expert_gemm_swiglu_bf16("normal", x, r.count, w, out, r.status, **r.where)
            out[bad] = 0
        elif op == "dswiglu":
            out = torch.zeros(r.rows, 2 * n, device="cuda", dtype=torch.bfloat16)
            m.moe_expert_gemm_dswiglu_bf16("normal", x, r.count, w[:, :n].transpose(1, 2).contiguous(), gu, out, r.status,
                                           **r.where)
            out[bad] = 0
        else:
            out = torch.zeros(r.rows, 2 * n, device="cuda", dtype=torch.bfloat16)
            t = op == "transposed"
            m.moe_expert_gemm_bf16("normal", x, r.count, w.transpose(1, 2).contiguous() if t else w, out, r.status,
                                   transposed=t, **r.where)
            out[bad] = 0
        outs.append(out)
    r.ok()
    assert bool(outs[0].isfinite().all()) and torch.equal(*outs)


def test_reported_counts():
    """Counts beyond the layout are cut off and reported, negative ones skipped, overlapping segments refused."""
    m = moe()
    n, k = 64, 128
    gen = torch.Generator(device="cuda").manual_seed(8)
    a = torch.randn(64, k, device="cuda", generator=gen).bfloat16()
    w = torch.randn(2, n, k, device="cuda", generator=gen).bfloat16()

    def run(mode, count, seg=None, M=0):
        out, st = filled((64, n), torch.bfloat16), torch.zeros(1, dtype=torch.int32, device="cuda")
        m.moe_expert_gemm_bf16(mode, a, torch.tensor(count, dtype=torch.int32, device="cuda"), w, out, st,
                               seg_indptr=None if seg is None else torch.tensor(seg, device="cuda"),
                               max_tokens_per_expert=M)
        grad, st2 = torch.zeros(2, k, k, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        m.moe_expert_wgrad_bf16(mode, a, a, torch.tensor(count, dtype=torch.int32, device="cuda"), grad, st2,
                                seg_indptr=None if seg is None else torch.tensor(seg, device="cuda"),
                                max_tokens_per_expert=M)
        torch.cuda.synchronize()
        written = (out.view(torch.int16) != -23131).any(1)  # 0xa5a5
        return int(st), int(st2), written, grad

    s, s2, written, grad = run("masked", [40, 3], M=32)
    assert s == s2 == m.MOE_ERR_CAPACITY and int(written.sum()) == 35 and bool(written[:35].all())
    ref = a[:32].double().T @ a[:32].double()
    close(grad[0], ref, 2 * acc(32) * (a[:32].double().abs().T @ a[:32].double().abs()) + 2.0 ** -23 * ref.abs())
    s, s2, written, _ = run("normal", [10, 60], seg=[0, 10, 70])
    assert s == s2 == m.MOE_ERR_CAPACITY and bool(written.all())
    s, s2, written, grad = run("normal", [-5, 6], seg=[0, 10, 16])
    assert s == s2 == m.MOE_ERR_INVALID_ARG and int(written.sum()) == 6 and bool(written[10:16].all()) and not grad[0].any()
    s, s2, written, grad = run("normal", [1 << 30, 4], seg=[1 << 40, 0, 4])
    assert s == s2 == m.MOE_ERR_CAPACITY and int(written.sum()) == 4 and not grad[0].any()


def test_segments_that_overlap():
    m = moe()
    E, rows, n, k = 64, 300, 8, 8
    a = torch.ones(rows, k, device="cuda").bfloat16()
    w = torch.ones(E, n, k, device="cuda").bfloat16()
    out, st = filled((rows, n), torch.bfloat16), torch.zeros(1, dtype=torch.int32, device="cuda")
    count = torch.full((E,), rows, dtype=torch.int32, device="cuda")
    seg = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    m.moe_expert_gemm_bf16("normal", a, count, w, out, st, seg_indptr=seg)
    torch.cuda.synchronize()
    assert int(st) == m.MOE_ERR_INVALID_ARG and bool((out.view(torch.uint8) == 0xa5).all())
    grad = torch.zeros(E, k, n, device="cuda")
    st.zero_()
    m.moe_expert_wgrad_bf16("normal", a, a, count, grad, st, seg_indptr=seg)
    torch.cuda.synchronize()
    assert int(st) == 0 and bool((grad == rows).all())


@pytest.mark.parametrize("op", ["product", "weights"])
def test_many_experts(op):
    m = moe()
    rng = np.random.default_rng(9)
    r = Rows("normal", rng.integers(0, 5, 1024), seed=9)
    n, k = 40, 72
    a = r.values(k)
    if op == "weights":
        b, out = r.values(n), torch.zeros(r.E, k, n, device="cuda")
        m.moe_expert_wgrad_bf16("normal", a, b, r.count, out, r.status, **r.where)
        r.ok()
        want = torch.zeros(r.E, k, n, dtype=torch.float64, device="cuda")
        mag = want.clone()
        x, y = a[r.used].double(), b[r.used].double()
        want.index_add_(0, r.expert, x[:, :, None] * y[:, None, :])
        mag.index_add_(0, r.expert, (x[:, :, None] * y[:, None, :]).abs())
        close(out, want, 1.01 * acc(4) * mag + HALF[torch.float32] * want.abs())
        return
    w, out = r.weights(n, k), filled((r.rows, n), torch.bfloat16)
    m.moe_expert_gemm_bf16("normal", a, r.count, w, out, r.status, **r.where)
    r.ok()
    x, v = a[r.used].double(), w.double()[r.expert]
    want, mag = (x[:, None] * v).sum(-1), (x[:, None] * v).abs().sum(-1)
    close(out[r.used], want, HALF[torch.bfloat16] * want.abs() + 1.01 * acc(k) * mag)


def test_offsets_past_32_bits():
    """Rows and weights whose elements lie beyond 2^31, and beyond 2^32 bytes."""
    m = moe()
    n, k, M = 64, 4096, 270000
    count = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    a = torch.zeros(2 * M, k, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(10)
    for e, c in ((0, 3), (1, 5)):
        a[e * M:e * M + c] = torch.randn(c, k, device="cuda", generator=gen)
    w = (torch.randn(2, n, k, device="cuda", generator=gen) / 64).bfloat16()
    out, st = torch.zeros(2 * M, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_expert_gemm_bf16("masked", a, count, w, out, st, max_tokens_per_expert=M)
    g = torch.zeros(2, k, n, device="cuda")
    m.moe_expert_wgrad_bf16("masked", a, out, count, g, st, max_tokens_per_expert=M)
    back = torch.zeros(2 * M, k, dtype=torch.bfloat16, device="cuda")
    m.moe_expert_gemm_bf16("masked", out, count, w, back, st, transposed=True, max_tokens_per_expert=M)
    torch.cuda.synchronize()
    assert int(st) == 0
    for e, c in ((0, 3), (1, 5)):
        at = slice(e * M, e * M + c)
        x, v = a[at].double(), w[e].double()
        close(out[at], x @ v.T, HALF[torch.bfloat16] * (x @ v.T).abs() + acc(k) * (x.abs() @ v.abs().T))
        y = out[at].double()
        close(g[e], x.T @ y, 2.0 ** -23 * (x.T @ y).abs() + acc(c) * (x.abs().T @ y.abs()))
        close(back[at], y @ v, HALF[torch.bfloat16] * (y @ v).abs() + acc(n) * (y.abs() @ v.abs()))


def _both(m, r, a, w, b, out, grad, stream=None):
    m.moe_expert_gemm_bf16(r.mode, a, r.count, w, out, r.status, stream=stream, **r.where)
    m.moe_expert_wgrad_bf16(r.mode, a, b, r.count, grad, r.status, stream=stream, **r.where)


def test_streams_graphs_and_repetition():
    """The same bits on repetition, on another stream, on two streams at once and from a graph."""
    m = moe()
    r = Rows("normal", [300, 5, 0, 129], align=16, seed=11)
    n, k = 520, 1032
    a, w, b = r.values(k), r.weights(n, k), r.values(n)

    def fresh():
        return torch.zeros(r.rows, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(r.E, k, n, device="cuda")

    want = fresh()
    _both(m, r, a, w, b, *want)
    for _ in range(3):
        got = fresh()
        _both(m, r, a, w, b, *got)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fresh() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, got):
            _both(m, r, a, w, b, *g, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))
    got = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _both(m, r, a, w, b, *got)
    for _ in range(2):
        for t in got:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0][r.used], want[0][r.used]) and torch.equal(got[1], want[1])
    r.ok()


def test_dswiglu_of_far_gates():
    """Gates and ups up to bf16's ends: no infinity or NaN where the gradient has none, and p's own precision."""
    m = moe()
    gates = torch.tensor([0.0, 1e-30, 0.5, 3.0, 20.0, 80.0, 88.0, 95.0, 103.0, 110.0, 300.0, 1e5, 1e20, 3e38], device="cuda")
    gates = torch.cat([gates, -gates]).bfloat16()
    ups = torch.tensor([0.0, 1.0, -3.0, 1e-20, 1e10, 1e25, 3e38], device="cuda").bfloat16()
    I, R = gates.numel() + 4, 7 * 3
    gu = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[:, :gates.numel()] = gates
    gu[:, I:] = ups.repeat_interleave(3)[:, None]
    dh = torch.tensor([1.0, 1e-15, -2e10], device="cuda").bfloat16().repeat(7)
    g = torch.zeros(R, 8, dtype=torch.bfloat16, device="cuda")
    g[:, 0] = dh
    w2 = torch.zeros(1, 8, I, dtype=torch.bfloat16, device="cuda")
    w2[:, 0] = 1
    out, st = torch.zeros_like(gu), torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_expert_gemm_dswiglu_bf16("normal", g, torch.tensor([R], dtype=torch.int32, device="cuda"), w2, gu, out, st,
                                   seg_indptr=torch.tensor([0, R], device="cuda"))
    torch.cuda.synchronize()
    G, U, D = gu[:, :I].double(), gu[:, I:].double(), dh.double()[:, None]
    p, q = torch.sigmoid(G), torch.sigmoid(-G)
    tiny = 2.0 ** -149                  # exp(-|G|) may be off by a subnormal step, and p or q with it
    for got, want, slope, parts in ((out[:, :I], D * U * p * (1 + G * q), U * (1 + G.abs()), U.abs() * p * (1 + G.abs() * q)),
                                    (out[:, I:], D * G * p, G, (G * p).abs())):
        # each product of factors may be rounded to a subnormal too, before dh multiplies it
        bound = (HALF[torch.bfloat16] + 2.0 ** -18) * want.abs() + D.abs() * (2.0 ** -18 * parts + 2 * tiny * (slope.abs() + 2))
        most = torch.finfo(torch.bfloat16).max
        fits = want.abs() + bound < most
        assert not got.isnan().any()
        close(got[fits], want[fits], bound[fits] + 2.0 ** -133)
        over = want.abs() - bound > most    # where the bound itself is that large a value says nothing
        assert bool(over.any()) and bool((got[over].double().abs() >= 0.98 * most).all())


def test_threads_with_sizes_of_their_own():
    """Host threads whose calls differ in experts, sizes and streams, the kernels' first calls among them."""
    import threading
    m = moe()
    jobs = []
    for i, (E, n, k) in enumerate([(1, 64, 64), (1024, 8, 16), (16, 520, 136), (200, 40, 72)]):
        r = Rows("normal", [3] * E, seed=20 + i)
        a, b, w = r.values(k), r.values(n), r.weights(n, k)
        jobs.append((r, a, w, b, torch.zeros(r.rows, n, device="cuda").bfloat16(), torch.zeros(E, k, n, device="cuda")))
    want = []
    for r, a, w, b, out, grad in jobs:
        x, v = a[r.used].double(), w.double()[r.expert]
        y = b[r.used].double().view(r.E, 3, -1)
        x3 = x.view(r.E, 3, -1)
        want.append((torch.einsum("rk,rnk->rn", x, v), torch.einsum("rk,rnk->rn", x.abs(), v.abs()),
                     torch.einsum("erk,ern->ekn", x3, y), torch.einsum("erk,ern->ekn", x3.abs(), y.abs())))
    torch.cuda.synchronize()
    wrong = []

    def work(job):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                _both(m, *job, stream=s)
            s.synchronize()
        except Exception as e:          # noqa: BLE001 - reported by the test
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for (r, a, w, b, out, grad), (y, ymag, g, gmag) in zip(jobs, want):
        r.ok()
        close(out, y, HALF[torch.bfloat16] * y.abs() + 1.01 * acc(w.shape[2]) * ymag)
        close(grad, g, HALF[torch.float32] * g.abs() + 1.01 * acc(3) * gmag)


def test_tensors_of_another_device_are_refused(monkeypatch):
    m = moe()
    r = Rows("normal", [3], seed=30)
    a, w, out = r.values(64), r.weights(64, 64), torch.zeros(3, 64, device="cuda").bfloat16()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        m.moe_expert_gemm_bf16("normal", a, r.count, w, out, r.status, **r.where)


# With a long k an expert's rows may lie in tiles of up to 288, whose accumulators meet: such tiles before and behind each
# other, small ones, and experts of several, in some rounds of a pair's tiles.
WIDE = len(LAYOUTS)
LAYOUTS += [("normal", [270, 288, 257, 40, 0, 530, 289, 576, 17, 283, 860, 256] * 2, dict(spare=2)),
            ("masked", [288, 1, 287, 0, 260, 200, 288, 33] * 4, dict(M=288))]


@pytest.mark.parametrize("op", ["nk", "kn", "swiglu", "dswiglu"])
@pytest.mark.parametrize("shape", [(2056, 2056), (520, 4104), (1032, 7176)])
@pytest.mark.parametrize("i", [WIDE, WIDE + 1])
def test_more_than_256_rows(i, shape, op):
    if op == "swiglu":
        test_swiglu(i, shape, True)
    elif op == "dswiglu":
        test_dswiglu(i, shape, True)
    else:
        test_product(i, shape, op == "kn")


def test_more_than_256_rows_repeated():
    r = Rows("normal", [264] * 60 + [31, 288, 290, 0, 281] * 8, seed=9)
    n, k = 1536, 2048
    a, w = r.values(k), r.weights(n, k)
    outs = [filled((r.rows, n), torch.bfloat16) for _ in range(3)]
    for out in outs:
        moe().moe_expert_gemm_bf16(r.mode, a, r.count, w, out, r.status, **r.where)
    r.ok()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_added_subnormal_gradients(dtype):
    r = Rows("normal", [3, 0, 40])
    a, b = torch.zeros(r.rows, 264, dtype=torch.bfloat16, device="cuda"), r.values(136)
    out = torch.full((3, 264, 136), 2.0 ** -130, dtype=dtype, device="cuda")
    moe().moe_expert_wgrad_bf16(r.mode, a, b, r.count, out, r.status, accumulate=True, **r.where)
    r.ok()
    assert bool((out == 2.0 ** -130).all())


@pytest.mark.parametrize("E", [128, 200, 1024])
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, True)])
def test_weight_gradient_of_many_experts(E, dtype, accumulate):
    """The ring has another number of slots where there are many experts."""
    r = Rows("normal", [(7 * e) % 150 for e in range(E)], seed=4)
    a, b = r.values(72), r.values(136)
    out = torch.randn(E, 72, 136, device="cuda", generator=r.gen).to(dtype)
    old = out.double() if accumulate else torch.zeros_like(out, dtype=torch.float64)
    moe().moe_expert_wgrad_bf16(r.mode, a, b, r.count, out, r.status, accumulate=accumulate, **r.where)
    r.ok()
    for e, at in r.each():
        x, y = a[at].double(), b[at].double()
        want = old[e] + x.T @ y
        bound = 1.01 * acc(150) * (x.abs().T @ y.abs()) + (HALF[dtype] + HALF[torch.float32]) * want.abs() + 2.0 ** -23 * old[e].abs()
        close(out[e], want, bound)


@pytest.mark.parametrize("m", [8, 16, 24, 40, 136, 264, 272, 520])
@pytest.mark.parametrize("n", [64, 72, 136, 200, 264, 392])
def test_added_bf16_gradients_of_rows_that_part_a_warp(m, n):
    """Row counts that end inside a warp's 32 rows of the result, with one to four pieces of its columns: lanes with and
    without a row add, and load the next piece together. Added twice, on repetition the same bits."""
    r = Rows("normal", [70, 0, 1, 33, 16, 0, 130], seed=m + n)
    a, b = r.values(m), r.values(n)
    first = torch.randn(r.E, m, n, device="cuda", generator=r.gen).bfloat16()
    outs = []
    for _ in range(2):
        out = first.clone()
        moe().moe_expert_wgrad_bf16(r.mode, a, b, r.count, out, r.status, accumulate=True, **r.where)
        outs.append(out)
    r.ok()
    assert torch.equal(*outs)
    for e, at in r.each():
        x, y = a[at].double(), b[at].double()
        want, old = first[e].double() + x.T @ y, first[e].double().abs()
        bound = 1.01 * acc(int(r.counts[e])) * (x.abs().T @ y.abs()) + (HALF[torch.bfloat16] + 2.0 ** -23) * want.abs()
        close(outs[0][e], want, bound + 2.0 ** -23 * old)


@pytest.mark.parametrize("op", ["product", "transposed", "swiglu", "dswiglu"])
def test_segments_that_overlap_too_far(op):
    """Refused by every product, nothing written, and the next call is as ever; the ring has its size from no tile then."""
    m = moe()
    E, rows, n, k = 64, 300, 72, 136
    gen = torch.Generator(device="cuda").manual_seed(40)
    a = torch.randn(rows, k, device="cuda", generator=gen).bfloat16()
    w = torch.randn(E, *((k, n) if op in ("transposed", "dswiglu") else (2 * n if op == "swiglu" else n, k)), device="cuda",
                    generator=gen).bfloat16()
    gu = torch.randn(rows, 2 * n, device="cuda", generator=gen).bfloat16()
    outs = []
    for count, seg in (([rows] * E, [0] * (E + 1)), ([rows] + [0] * (E - 1), [0] + [rows] * E)):
        out, st = filled((rows, 2 * n if op == "dswiglu" else n), torch.bfloat16), m.new_status()
        c, where = torch.tensor(count, dtype=torch.int32, device="cuda"), dict(seg_indptr=torch.tensor(seg, device="cuda"))
        for _ in range(3):
            if op == "swiglu":
                m.moe_expert_gemm_swiglu_bf16("normal", a, c, w, out, st, **where)
            elif op == "dswiglu":
                m.moe_expert_gemm_dswiglu_bf16("normal", a, c, w, gu, out, st, **where)
            else:
                m.moe_expert_gemm_bf16("normal", a, c, w, out, st, transposed=op == "transposed", **where)
        torch.cuda.synchronize()
        outs.append((int(st), out))
    assert outs[0][0] == m.MOE_ERR_INVALID_ARG and bool((outs[0][1].view(torch.uint8) == 0xa5).all())
    assert outs[1][0] == 0 and bool(outs[1][1].isfinite().all()) and not bool((outs[1][1].view(torch.uint8) == 0xa5).all())


# Beyond some 490 experts their counts leave shared memory for five slots of the largest tiles, not six.
FIVE = len(LAYOUTS)
LAYOUTS += [("normal", [(257 + e // 8 % 32) if e % 8 == 3 else e % 2 for e in range(E)], dict(spare=1)) for E in (520, 1024)]


@pytest.mark.parametrize("op", ["nk", "kn", "swiglu", "dswiglu"])
@pytest.mark.parametrize("i", [FIVE, FIVE + 1])
def test_more_than_256_rows_of_many_experts(i, op):
    test_more_than_256_rows(i, (392, 2056), op)


def test_each_gradient_along_itself():
    """Each operator's gradient by itself, of values that it is given exactly, so that its own rounding is all it is off by."""
    m = moe()
    r = Rows("normal", [3, 0, 6, 2], align=4, seed=5)
    H, I, B = 24, 16, HALF[torch.bfloat16]
    x, w13, w2, g, gu = r.values(H), r.weights(2 * I, H), r.weights(H, I), r.values(H), r.values(2 * I, 2.0)
    experts = [(e, at) for e, at in r.each() if r.counts[e]]
    d, dx = torch.zeros_like(gu), torch.zeros_like(x)
    m.moe_expert_gemm_dswiglu_bf16("normal", g, r.count, w2, gu, d, r.status, **r.where)
    m.moe_expert_gemm_bf16("normal", gu, r.count, w13, dx, r.status, transposed=True, **r.where)
    d13 = torch.zeros_like(w13, dtype=torch.float32)
    m.moe_expert_wgrad_bf16("normal", gu, x, r.count, d13, r.status, **r.where)
    r.ok()
    x64, w64, g64, gu64 = (t.double().nan_to_num(0) for t in (x, w13, g, gu))

    def through_swiglu(change):
        y = gu64 + change
        h = y[:, I:] * torch.nn.functional.silu(y[:, :I])
        return sum(float((h[at] @ w2[e].double().T * g64[at]).sum()) for e, at in experts)

    def product(dx, dw):
        return sum(float(((x64[at] + dx[at]) @ (w64[e] + dw[e]).T * gu64[at]).sum()) for e, at in experts)

    # as in test_dswiglu, the sums' and the factors' own errors before they cancel
    dh, mag = (r.per_expert(a, lambda v, e, w=w: v @ w[e]) for a, w in ((g, w2.double()), (g.abs(), w2.double().abs())))
    G, U = gu64[:, :I], gu64[:, I:]
    p, q = torch.sigmoid(G), torch.sigmoid(-G)
    parts, err = U.abs() * p * (1 + G.abs() * q), 1.01 * acc(H) * mag
    own = torch.cat(((parts + 1) * err + 2.0 ** -18 * dh.abs() * parts, (G * p).abs() * err + 2.0 ** -18 * (dh * G * p).abs()), 1)
    along(d, 1.01 * B * d.double().abs() + 2 * own, through_swiglu, 6)
    terms = r.per_expert(gu.abs(), lambda v, e: v @ w64[e].abs())
    along(dx, 1.01 * B * dx.double().nan_to_num(0).abs() + 2 * acc(2 * I) * terms, lambda c: product(c, 0 * w64), 7)
    terms = torch.zeros_like(w64)
    for e, at in experts:
        terms[e] = gu64[at].abs().T @ x64[at].abs()
    along(d13, 2.0 ** -23 * d13.double().abs() + 2 * acc(6) * terms, lambda c: product(0 * x64, c), 8)
