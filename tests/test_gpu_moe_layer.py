"""The few-token layer and the whole layer object against 64-bit references."""
import numpy as np
import pytest
import torch

from _experts import ACC, BF16_STEP, dev, quantised, silu, silu_slope, values, weights
from _harness import filled, moe
from workloads import bf16_bits_to_f32, random_bf16

pytestmark = pytest.mark.gpu

CASES = [  # T, H, I, E, K, weights, invalid rate, duplicates
    (1, 64, 64, 1, 1, "nvfp4", 0, False),
    (1, 16, 16, 1, 1, "bf16", 0, False),
    (1, 320, 192, 8, 4, "nvfp4", 0, False),
    (2, 256, 128, 4, 2, "nvfp4", 0.5, False),
    (3, 304, 80, 6, 3, "bf16", 0.2, False),
    (5, 576, 320, 16, 8, "nvfp4", 0.1, False),
    (7, 272, 336, 5, 4, "bf16", 0.1, True),
    (8, 1088, 128, 3, 3, "nvfp4", 0, False),
    (17, 448, 192, 40, 8, "nvfp4", 0.1, False),
    (33, 512, 256, 4, 4, "bf16", 0, False),
    (64, 192, 448, 2, 2, "nvfp4", 0.05, False),
    (64, 256, 64, 300, 16, "bf16", 0.3, False),
    (64, 128, 128, 3, 16, "nvfp4", 0, True),
    (64, 64, 64, 1024, 16, "nvfp4", 0.02, False),       # the most experts and slots
    (1, 2112, 192, 2, 2, "nvfp4", 0, False),            # a row shared out over a cluster of eight
    (2, 1040, 144, 3, 2, "bf16", 0, False),
    (40, 8256, 64, 5, 1, "nvfp4", 0, False),            # several rounds of the ring, groups of 12 pairs
    (64, 4112, 48, 1, 1, "bf16", 0, False),             # an expert with 64 tokens
]


class Layer:
    def __init__(self, T, H, I, E, K, kind, invalid, dup, seed=0):
        rng = np.random.default_rng(T * 7 + H + I + seed)
        self.x = random_bf16(rng, (T, H))
        ids = rng.integers(0, E, (T, K)) if dup else np.argsort(rng.random((T, E)), axis=1)[:, :K]
        if dup:
            ids[:, 0] = ids[:, -1]
        ids = np.where(rng.random((T, K)) < invalid, -1, ids)
        if invalid and T > 1:
            ids[T // 2] = -1                                     # a token that no expert gets
        self.ids = np.ascontiguousarray(ids, dtype=np.int32)
        self.w = rng.random((T, K), dtype=np.float32)
        self.kw = {}
        if kind == "nvfp4":
            q13, s13, v13, _ = weights(rng, 2 * E, I, H)
            q2, s2, v2, _ = weights(rng, E, H, I)
            a13, a2 = (rng.uniform(0.5, 2.0, E).astype(np.float32) / 2.0 ** 10 for _ in range(2))
            self.w13, self.w2 = dev(q13.reshape(E, 2 * I, H // 2)), dev(q2)
            self.v13 = [np.concatenate(v13[2 * e:2 * e + 2]) * a13[e] for e in range(E)]
            self.v2 = [v2[e] * a2[e] for e in range(E)]
            self.kw = dict(w13_scales=dev(s13), w2_scales=dev(s2), alpha13=dev(a13), alpha2=dev(a2))
        else:
            b13, b2 = random_bf16(rng, (E, 2 * I, H), H ** -0.5), random_bf16(rng, (E, H, I), I ** -0.5)
            self.w13, self.w2 = (torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16) for b in (b13, b2))
            self.v13, self.v2 = (bf16_bits_to_f32(b).astype(np.float64) for b in (b13, b2))

    def want(self):
        """The output and the error that fp32 sums and a 16-bit h allow, in 64 bits."""
        x = bf16_bits_to_f32(self.x).astype(np.float64)
        T, H = x.shape
        y, err = np.zeros((T, H)), np.zeros((T, H))
        for t in range(T):
            for e, w in zip(self.ids[t], self.w[t].astype(np.float64)):
                if not 0 <= e < len(self.v2):
                    continue
                I = self.v2[e].shape[1]
                g, u = np.split(self.v13[e] @ x[t], [I])
                eg, eu = np.split(ACC * (np.abs(self.v13[e]) @ np.abs(x[t])), [I])
                h = u * silu(g)
                eh = silu_slope() * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + 2.0 ** -16 * np.abs(h)
                y[t] += w * (self.v2[e] @ h)
                err[t] += w * (np.abs(self.v2[e]) @ (eh + ACC * np.abs(h)))
        return y, err

    def run(self, stream=None, ids=None):
        m = moe()
        T, H = self.x.shape
        E, I, K = self.w13.shape[0], self.w13.shape[1] // 2, self.ids.shape[1]
        out = filled((T, H), torch.bfloat16)
        ws = filled((m.moe_layer_workspace_size(T, K, H, I, E) + 256,), torch.uint8)
        ws = ws[-ws.data_ptr() % 256:]
        self.status = m.new_status()
        x = torch.from_numpy(self.x.view(np.int16)).cuda().view(torch.bfloat16)
        ids, w = dev(self.ids if ids is None else ids), dev(self.w)
        torch.cuda.synchronize()
        m.moe_layer_few_tokens(x, ids, w, self.w13, self.w2, out, ws, self.status, stream=stream, **self.kw)
        torch.cuda.synchronize()
        return out


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_few_tokens(case):
    layer = Layer(*case)
    got = layer.run().double().cpu().numpy()
    assert int(layer.status.item()) == 0
    want, err = layer.want()
    bad = np.abs(got - want) > BF16_STEP * np.abs(want) + err
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    empty = (layer.ids < 0).all(1)
    assert not got[empty].any()


def test_same_bits_every_time():
    layer = Layer(24, 576, 320, 12, 6, "nvfp4", 0.1, False)
    first = layer.run().view(torch.int16)
    for _ in range(3):
        assert torch.equal(layer.run(torch.cuda.Stream()).view(torch.int16), first)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
def test_a_token_that_is_not_finite_leaves_the_others_alone(kind):
    layer = Layer(9, 320, 192, 4, 2, kind, 0, False)
    want = layer.run().view(torch.int16)
    layer.x = layer.x.copy()
    layer.x[3, 5], layer.x[3, 100], layer.x[3, 319] = 0x7fc0, 0x7f80, 0xff80      # NaN, infinity, -infinity
    layer.x[7] = 0x7fff
    got = layer.run().view(torch.int16)
    assert int(layer.status.item()) == 0
    finite = [t for t in range(9) if t not in (3, 7)]
    assert torch.equal(got[finite], want[finite])


def test_gates_far_from_zero():
    """silu of gates from -3e38 to 3e38, by one-element dot products: x W13 = (gate, 1), W2 picks h."""
    m = moe()
    gates = torch.tensor([-3e38, -1e30, -200, -104, -89, -80.5, -50, -3, -1e-3, 0, 1e-3, 3, 50, 80.5, 89, 104, 1e30, 3e38])
    H = I = 32
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16)
    n = len(gates)
    w13[0, :n, 0] = gates.bfloat16()
    w13[0, I:, 0] = 1
    w2 = torch.eye(H)[None].bfloat16()
    x = torch.zeros(1, H, dtype=torch.bfloat16)
    x[0, 0] = 1
    out, status = torch.empty(1, H, dtype=torch.bfloat16, device="cuda"), m.new_status()
    m.moe_layer_few_tokens(x.cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"),
                           w13.cuda(), w2.cuda(), out, m.new_layer_workspace(1, 1, H, I, 1), status)
    m.check_status(status)
    g = w13[0, :n, 0].double()
    want = g / (1 + torch.exp(-g))
    got = out[0, :n].double().cpu()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 1e-31).all(), got.tolist()


def test_layers_on_two_streams_at_once():
    layers = [Layer(9, 576, 320, 12, 6, "nvfp4", 0.1, False), Layer(30, 272, 336, 5, 4, "bf16", 0.1, True, seed=1)]
    alone = [layer.run().view(torch.int16).clone() for layer in layers]
    m = moe()
    runs, status = [], m.new_status()
    for layer in layers:
        T, H = layer.x.shape
        E, I, K = layer.w13.shape[0], layer.w13.shape[1] // 2, layer.ids.shape[1]
        x = torch.from_numpy(layer.x.view(np.int16)).cuda().view(torch.bfloat16)
        runs.append((x, dev(layer.ids), dev(layer.w), layer, m.new_layer_workspace(T, K, H, I, E), torch.cuda.Stream(),
                     [torch.empty_like(x) for _ in range(8)]))
    torch.cuda.synchronize()
    for r in range(8):
        for x, ids, w, layer, ws, stream, outs in runs:
            m.moe_layer_few_tokens(x, ids, w, layer.w13, layer.w2, outs[r], ws, status, stream=stream, **layer.kw)
    torch.cuda.synchronize()
    m.check_status(status)
    for (*_, outs), want in zip(runs, alone):
        for o in outs:
            assert torch.equal(o.view(torch.int16), want)


def test_bad_ids_are_skipped_and_reported():
    m = moe()
    layer = Layer(6, 256, 128, 4, 3, "bf16", 0, False)
    ids = layer.ids.copy()
    ids[1, 1], ids[3, 0], ids[4] = 4, -2, 1 << 30
    got = layer.run(ids=ids).double().cpu().numpy()
    assert int(layer.status.item()) == m.MOE_ERR_BAD_EXPERT_ID
    layer.ids = np.where((ids < 0) | (ids >= 4), -1, ids).astype(np.int32)
    want, err = layer.want()
    assert (np.abs(got - want) <= BF16_STEP * np.abs(want) + err).all() and not got[4].any()


def test_no_tokens():
    m = moe()
    e = torch.zeros((2, 64, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    m.moe_layer_few_tokens(x, torch.zeros((0, 2), dtype=torch.int32, device="cuda"),
                           torch.zeros((0, 2), device="cuda"), e, e[:, :, :32].contiguous(), x, None, m.new_status())


def test_weights_past_32_bits():
    """The last expert of more than 2^32 weights."""
    m = moe()
    E, I, H = 40, 4096, 20480
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    w13[-1], w2[-1] = torch.randn(2 * I, H, device="cuda") * H ** -0.5, torch.randn(H, I, device="cuda") * I ** -0.5
    x = torch.randn(1, H, device="cuda").bfloat16()
    ids, w = torch.tensor([[E - 1]], dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    out, status = torch.empty_like(x), m.new_status()
    m.moe_layer_few_tokens(x, ids, w, w13, w2, out, m.new_layer_workspace(1, 1, H, I, E), status)
    m.check_status(status)
    g, u = (w13[-1].double() @ x[0].double()).split(I)
    want = w2[-1].double() @ (u * torch.nn.functional.silu(g))
    # the elementwise bound of the other cases, with every sum's magnitude at its typical value: K * 0.8^2 * sigma^2
    assert ((out[0].double() - want).abs() <= BF16_STEP * want.abs() + 64 * ACC).all()


def _experts(E, I, H, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w13 = (torch.randn(E, 2 * I, H, device="cuda", generator=gen) * H ** -0.5).bfloat16()
    w2 = (torch.randn(E, H, I, device="cuda", generator=gen) * I ** -0.5).bfloat16()
    return w13, w2


def test_layer_object_chooses_by_tokens_and_agrees_with_bf16():
    """Few and many tokens of one quantised layer against the unquantised layer in 64 bits. A value quantised to
    NVFP4 is off by about a tenth (rms), and independent factors of a sum add in squares: three quantised
    factors (gate, up and down weights) give 0.17, with the tokens' rows (twice) and h six of them 0.25."""
    m = moe()
    E, I, H, K, T = 6, 256, 512, 3, 200
    w13, w2 = _experts(E, I, H, 1)
    layer = m.MoELayer(m.quantize_experts(w13, w2), K, T, input_scale=2688.0 / 6.0, inter_scale=2688.0 / 12.0,
                       few_tokens=64)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :K].int().contiguous()
    ids[7] = -1
    w = torch.rand(T, K, device="cuda", generator=gen).softmax(1)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        g, u = (x[t].double() @ w13[e].double().T).chunk(2, 1)
        want.index_add_(0, t, (u * torch.nn.functional.silu(g)) @ w2[e].double().T * w[t, k].double()[:, None])
    for n in (T, 1, 64, 65, T):
        got = layer(x[:n], ids[:n], w[:n])
        layer.check()
        assert got.shape == (n, H)
        rel = ((got.double() - want[:n]).norm() / want[:n].norm()).item()
        assert rel < (0.35 if n > 64 else 0.25), (n, rel)
        if n > 7:
            assert not got[7].any()


def test_layer_object_in_a_graph():
    m = moe()
    E, I, H, K = 4, 128, 256, 2
    w13, w2 = _experts(E, I, H, 3)
    layer = m.MoELayer(m.quantize_experts(w13, w2), K, 96, input_scale=400.0, inter_scale=200.0)
    assert layer.few == 4 * E // K
    for T in (5, 96):
        x = torch.randn(T, H, device="cuda").bfloat16()
        ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda")
        w = torch.rand(T, K, device="cuda")
        eager = layer(x, ids, w).clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x, ids, w)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        layer.check()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))


def test_layer_object_refuses():
    m = moe()
    w13, w2 = _experts(2, 64, 128, 4)
    with pytest.raises(m.MoEError, match="UNSUPPORTED"):
        m.MoELayer(m.ExpertWeights(w13, w2), 2, 65)
    with pytest.raises(ValueError, match="input_scale"):
        m.MoELayer(m.quantize_experts(w13, w2), 2, 65)
    layer = m.MoELayer(m.ExpertWeights(w13, w2), 2, 4)
    with pytest.raises(ValueError, match="5 tokens"):
        layer(torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda"), None, None)


@pytest.mark.parametrize("T", [2, 64])          # both ways
def test_layer_object_refuses_other_shapes(T):
    m = moe()
    w = m.quantize_experts(*(torch.randn(4, *s, device="cuda").bfloat16() for s in ((128, 128), (128, 64))))
    layer = m.MoELayer(w, 2, 64, input_scale=100.0, inter_scale=100.0)
    x = torch.zeros(T, 128, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(T, 2, device="cuda", dtype=torch.int32)
    g = torch.zeros(T, 2, device="cuda")
    layer(x, ids, g)
    for bad in ((x[:, :64].contiguous(), ids, g), (x, ids[:, :1].contiguous(), g), (x, ids, g[:-1]),
                (x, ids[:-1], g), (torch.cat([x, x], 1), ids, g), (x, ids, torch.cat([g, g], 1))):
        with pytest.raises(ValueError):
            layer(*bad)
    torch.cuda.synchronize()
    layer.check()


def test_example_runs():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_layer_nvfp4.py"), "--tokens", "1,70", "--experts",
                        "8", "--hidden", "512", "--inter", "256", "--topk", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.count("tokens:") == 2
