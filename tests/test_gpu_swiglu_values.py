"""silu(gate) * up value by value, over the whole range of gates."""
import numpy as np
import pytest
import torch

from _experts import dev, interleave
from _harness import moe

pytestmark = pytest.mark.gpu


def test_h_of_1024_gates():
    """The fp32 values of h that the few-token layer leaves at the start of its workspace, pair by pair, with NVFP4 weights.
    Expert p has the factor alpha[p] and sees x = (1.5, 0, ..): gate 1.5 alpha[p] and up 2688 times that, both rounded once.
    Relative error: 2^-22 of 2^t, 2^-23 of the reciprocal, seven roundings of 2^-24: below 2^-20. From gate -87 on 2^t is the
    square of one of half the exponent (2^-21) and, from -87.3 on, subnormal (half a step of 2^-149, times gate and up). h has
    subnormal values of its own."""
    m = moe()
    T, K, H, I, E = 64, 16, 64, 64, 1024
    gates = np.concatenate([-np.linspace(80, 104, 400), np.linspace(-80, 100, 400), np.logspace(-30, 10, 112),
                            -np.logspace(-30, 4, 112)])
    assert len(gates) == E
    alpha = (gates / 1.5).astype(np.float32)
    codes = np.zeros((E, 2 * I, H // 2), np.uint8)
    codes[:, :I, 0], codes[:, I:, 0] = 2, 7                                # 1 and 6
    sf = [interleave(np.full((I, H // 16), c, np.uint8)) for c in (0x38, 0x7e)]  # 1 and 448
    s13 = np.tile(np.stack(sf).reshape(-1), (E, 1))
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.5
    ids = torch.arange(E, dtype=torch.int32, device="cuda").view(T, K)
    w2, s2 = (torch.zeros(E, n, dtype=torch.uint8, device="cuda") for n in (H * I // 2, 128 * I // 16))
    ws, status = m.new_layer_workspace(T, K, H, I, E), m.new_status()
    m.moe_layer_few_tokens(x, ids, torch.ones(T, K, device="cuda"), dev(codes), w2.view(E, H, I // 2), torch.empty_like(x), ws, status,
                           dev(s13), s2, dev(alpha))
    m.check_status(status)
    h = ws[:T * K * I * 4].view(torch.float32).view(E, I).double().cpu().numpy()
    assert (h == h[:, :1]).all()
    g = (np.float32(1.5) * alpha).astype(np.float64)
    u = (np.float32(1.5 * 2688) * alpha).astype(np.float64)
    want = u * g * np.where(g < 0, np.exp(-np.abs(g)), 1) / (1 + np.exp(-np.abs(g)))
    rel = np.where(g < -87, 2.0 ** -19, 2.0 ** -20)
    bad = np.abs(h[:, 0] - want) > rel * np.abs(want) + 2.0 ** -150 * (np.abs(g * u) + 1)
    assert not bad.any(), [(g[i], h[i, 0], want[i]) for i in np.flatnonzero(bad)[:5]]


def test_far_gates_with_large_ups():
    """Gates between -80 and -88 leave values that a large up makes large again: x W13 = (gate, 1e36), W2 picks h."""
    m = moe()
    gates = torch.tensor([-79, -80, -80.5, -81, -83, -85, -87, -87.5, -88, -88.5, -104, -120, -3e38])
    H = I = 32
    n = len(gates)
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.bfloat16)
    w13[0, :n, 0] = gates.bfloat16()
    w13[0, I:, 0] = 1e36
    x = torch.zeros(1, H, dtype=torch.bfloat16)
    x[0, 0] = 1
    out, status = torch.empty(1, H, dtype=torch.bfloat16, device="cuda"), m.new_status()
    m.moe_layer_few_tokens(x.cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"),
                           w13.cuda(), torch.eye(H)[None].bfloat16().cuda(), out, m.new_layer_workspace(1, 1, H, I, 1),
                           status)
    m.check_status(status)
    g, u = w13[0, :n, 0].double(), w13[0, I, 0].double()
    want = u * g * torch.exp(g) / (1 + torch.exp(g))
    got = out[0, :n].double().cpu()
    # one bf16 rounding (and the 16 bits that h has here), or the step of a subnormal 2^t
    bad = (got - want).abs() > 2.0 ** -8 * want.abs() + 2.0 ** -150 * (g * u).abs()
    assert not bad.any(), list(zip(got.tolist(), want.tolist()))
