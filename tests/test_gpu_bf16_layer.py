"""A whole MoE block in bf16, there and back: norm, layer, and the gradients of everything, against autograd in 64 bits."""
import pytest
import torch

from _harness import moe

pytestmark = pytest.mark.gpu


def _case(E, H, I, K, T, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=gen) * H ** -0.5).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=gen) * I ** -0.5).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
    if T > 3:
        ids[2] = -1
        ids[3, -1] = -1
    return w13, w2, x, ids, torch.rand(T, K, device="cuda", generator=gen), gen


def _layer64(x, ids, w, w13, w2):
    I = w2.shape[2]
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(w13.shape[0]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        y = x[t] @ w13[e].T
        out = out.index_add(0, t, (y[:, I:] * torch.nn.functional.silu(y[:, :I])) @ w2[e].T * w[t, k][:, None])
    return out


def _off(got, want):
    n = want.norm()
    return float((got.double() - want).norm() / n) if n > 0 else float(got.double().norm())


# In norm, a rounding to bf16 is 2^-8 / sqrt(3) off at most, and a value passes through at most six of them between an
# input and a gradient: less than 2^-8 * sqrt(6 / 3) if they were independent; all adding up, 6 * 2^-8 / sqrt(3).
OFF = 6 * 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("E,H,I,K,T", [(4, 64, 24, 2, 1), (6, 528, 136, 3, 90), (16, 1024, 256, 4, 700)])
def test_block_there_and_back(E, H, I, K, T):
    m = moe()
    w13, w2, x, ids, w, gen = _case(E, H, I, K, T)
    res = (2 * torch.randn(T, H, device="cuda", generator=gen)).bfloat16()
    nw = (1 + 0.1 * torch.randn(H, device="cuda", generator=gen)).bfloat16()
    layer = m.BF16MoELayer(w13, w2, K, T, train=True)
    y = m.rmsnorm(x, nw, 1e-6, residual=res, keep=True)
    out = layer(y.out, ids, w).clone()
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    # the block's output is sum + layer(norm(sum)): its gradient flows into the sum by both ways
    grads = layer.backward(g)
    dx, dnw = m.rmsnorm_backward(grads.x, y.sum, nw, y.rstd, grad_residual=g)
    layer.check()
    leaves = [t.double().requires_grad_() for t in (y.sum, nw, w, w13, w2)]
    s, n64, w64, a13, a2 = leaves
    want = _layer64(s * (s.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * n64, ids, w64, a13, a2)
    (s + want).backward(g.double())
    assert _off(out, want.detach()) <= OFF
    for got, leaf in zip((dx, dnw, grads.topk_weights, grads.w13, grads.w2), leaves):
        assert _off(got, leaf.grad) <= OFF
    assert not (grads.topk_weights[ids < 0]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_accumulated_gradients(dtype):
    """Two micro-batches, the second added to the first; an expert without rows keeps what it has."""
    m = moe()
    w13, w2, x, ids, w, gen = _case(5, 128, 64, 2, 40, 1)
    ids[ids == 4] = -1
    layer = m.BF16MoELayer(w13, w2, 2, 40, train=True, grad_dtype=dtype)
    g = torch.randn(40, 128, device="cuda", generator=gen).bfloat16()
    parts = []
    for i, at in enumerate((slice(0, 25), slice(25, 40))):
        layer(x[at], ids[at], w[at])
        parts.append(tuple(t.float().clone() for t in layer.backward(g[at])[2:]))
    layer(x[:25], ids[:25], w[:25])
    layer.backward(g[:25])
    layer(x[25:], ids[25:], w[25:])
    both = layer.backward(g[25:], accumulate=True)
    layer.check()
    # each part rounded, and their sum
    step = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    for got, a, b in zip(both[2:], *parts):
        assert got.dtype is dtype
        assert bool(((got.float() - (a + b)).abs() <= 2 * step * (a.abs() + b.abs() + (a + b).abs())).all())
        assert not got[4].any()


def test_serving():
    """Few tokens and many, against 64 bits; the same layer with any number of them."""
    m = moe()
    E, H, I, K, T = 8, 512, 256, 3, 300
    w13, w2, x, ids, w, _ = _case(E, H, I, K, T, 2)
    layer = m.BF16MoELayer(w13, w2, K, T)
    assert layer.few == 4 * E // K
    want = _layer64(x.double(), ids, w.double(), w13.double(), w2.double())
    for n in (T, 1, 5, layer.few, layer.few + 1, 0, T):
        got = layer(x[:n], ids[:n], w[:n])
        layer.check()
        assert got.shape == (n, H)
        assert _off(got, want[:n]) <= OFF
        if n > 2:
            assert not got[2].any()
    with pytest.raises(RuntimeError, match="train=True"):
        layer.backward(x)


def test_no_tokens():
    """A step without tokens: no output, and weights' gradients of zero."""
    m = moe()
    w13, w2, x, ids, w, _ = _case(4, 64, 32, 2, 10, 6)
    layer = m.BF16MoELayer(w13, w2, 2, 10, train=True)
    layer(x, ids, w)
    layer.backward(x)
    assert layer.grad_w2.any()
    assert layer(x[:0], ids[:0], w[:0]).shape == (0, 64)
    kept = layer.grad_w13.clone()
    grads = layer.backward(x[:0], accumulate=True)
    assert torch.equal(grads.w13, kept)
    layer(x[:0], ids[:0], w[:0])
    grads = layer.backward(x[:0])
    layer.check()
    assert grads.x.shape == (0, 64) and not grads.w13.any() and not grads.w2.any()


def test_an_expert_twice_in_a_token():
    m = moe()
    w13, w2, x, ids, w, gen = _case(4, 64, 32, 3, 20, 3)
    ids[:, 1] = ids[:, 0]
    layer = m.BF16MoELayer(w13, w2, 3, 20, train=True)
    out = layer(x, ids, w).clone()
    g = torch.randn(20, 64, device="cuda", generator=gen).bfloat16()
    grads = layer.backward(g)
    layer.check()
    leaves = [t.double().requires_grad_() for t in (x, w, w13, w2)]
    want = _layer64(leaves[0], ids, *leaves[1:])
    want.backward(g.double())
    assert _off(out, want.detach()) <= OFF
    for got, leaf in zip(grads, leaves):
        assert _off(got, leaf.grad) <= OFF


def test_step_in_a_graph():
    """A whole training step captured and replayed on other values, beside eager steps."""
    m = moe()
    E, H, I, K, T = 6, 256, 128, 2, 100
    w13, w2, x, ids, w, gen = _case(E, H, I, K, T, 4)
    layer = m.BF16MoELayer(w13, w2, K, T, train=True)
    g = torch.randn(T, H, device="cuda", generator=gen).bfloat16()

    def step():
        out = layer(x, ids, w)
        return (out, *layer.backward(g))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    w13b, w2b, xb, idsb, wb, _ = _case(E, H, I, K, T, 5)
    for a, b in zip((w13, w2, x, ids, w), (w13b, w2b, xb, idsb, wb)):
        a.copy_(b)
    want = [t.clone() for t in step()]
    for t in outs:
        t.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    layer.check()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    m = moe()
    w13, w2, x, ids, w, _ = _case(4, 64, 32, 2, 10)
    for bad in ((w13[:, :63].contiguous(), w2), (w13, w2[1:].contiguous()), (w13.float(), w2), (w13, w2.half())):
        with pytest.raises(ValueError):
            m.BF16MoELayer(*bad, 2, 10)
    with pytest.raises(ValueError, match="grad_dtype"):
        m.BF16MoELayer(w13, w2, 2, 10, train=True, grad_dtype=torch.float16)
    odd13, odd2 = (torch.zeros(2, 16, 24, device="cuda").bfloat16(), torch.zeros(2, 24, 8, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="multiple"):
        m.BF16MoELayer(odd13, odd2, 1, 10)
    layer = m.BF16MoELayer(w13, w2, 2, 10, train=True)
    with pytest.raises(ValueError, match="11 tokens"):
        layer(torch.zeros(11, 64, device="cuda").bfloat16(), None, None)
    with pytest.raises(ValueError):
        layer(x, ids[:, :1].contiguous(), w)
    with pytest.raises(RuntimeError, match="forward pass"):
        layer.backward(x)
    layer(x, ids, w)
    with pytest.raises(ValueError, match="grad_out"):
        layer.backward(x[:5])
    layer.backward(x)
    with pytest.raises(RuntimeError, match="forward pass"):
        layer.backward(x)                 # its rows are gone
    layer.check()
