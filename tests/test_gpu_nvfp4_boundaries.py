"""Block scales on the boundary between two e4m3 values: one quantiser in the dispatch, the weights' quantisation and the
requantised SwiGLU outputs."""
import numpy as np
import pytest
import torch

import oracle
from _experts import E4M3
from _harness import moe
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _on_boundaries():
    """Pairs (largest magnitude of a block, global scale) whose scale is another one when a product with the rounded 1/6
    stands for the division by 6."""
    a = (1 + np.arange(128) / 128).astype(np.float32)[:, None, None]
    mid = ((E4M3[1:127] + E4M3[:126]) / 2)[40:120, None]
    g = (6 * mid / a).astype(np.float32)
    g = (g.view(np.int32) + np.arange(-3, 4, dtype=np.int32)).view(np.float32)
    a = np.broadcast_to(a, g.shape)
    ways = [(a / np.float32(6)) * g, (a * np.float32(1 / 6)) * g]
    code = [oracle.e4m3_from_float_array(t.ravel()).reshape(t.shape) for t in ways]
    at = code[0] != code[1]
    return a[at], g[at], code[0][at]


def test_scales_on_boundaries_are_those_of_the_dispatch():
    m = moe()
    a, g, code = _on_boundaries()
    n = len(a)
    assert n > 1000
    bits = np.zeros((n, 1, 64), np.uint16)
    bits[:, 0, ::16] = f32_to_bf16_bits(a)[:, None]
    bits[:, 0, 1::16] = f32_to_bf16_bits(-a / 2)[:, None]
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    q = m.quantize_nvfp4(x, torch.from_numpy(g).cuda(), scale_layout="row")
    codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(scales.reshape(n, 4), np.repeat(code[:, None], 4, axis=1))
    for i in range(n):
        want_q, want_s = oracle.quant_nvfp4_row(bits[i, 0], float(g[i]))
        assert np.array_equal(codes[i, 0], want_q) and np.array_equal(scales[i].ravel(), want_s), (a[i], g[i])
    for i in range(0, n, n // 20):        # and the dispatch itself
        seg = torch.tensor([0, 1], device="cuda")
        zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        rows, sf = torch.zeros(1, 32, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, dtype=torch.uint8, device="cuda")
        status = m.new_status()
        m.moe_dispatch_ex("normal", "nvfp4b16", "row", x[i], zero, 1, zero.flatten(), seg, rows, sf, status, out_rows=1,
                          input_global_scale=float(g[i]))
        m.check_status(status)
        assert torch.equal(rows, q.codes[i]) and torch.equal(sf.flatten(), q.scales[i].flatten())


@pytest.mark.parametrize("g", [1.0, 2688.0, 448.0, 2.0 ** 100, 2.0 ** 120, 2.0 ** -100, 3e38, 1.5692307949066162])
def test_every_largest_magnitude(g):
    """Blocks of every finite bf16 magnitude (subnormal ones among them), bit for bit those of the dispatch's definition."""
    m = moe()
    bits = np.zeros((0x7f80, 16), np.uint16)
    bits[:, 3] = np.arange(0x7f80) | 0x8000
    bits[:, 7] = np.arange(0x7f80) // 2
    x = torch.from_numpy(bits.reshape(-1, 64).view(np.int16)).cuda().view(torch.bfloat16)
    q = m.quantize_nvfp4(x, torch.tensor([g], device="cuda"), scale_layout="row")
    want_q, want_s = oracle.quant_nvfp4_row(bits.ravel(), float(np.float32(g)))
    assert np.array_equal(q.scales.cpu().numpy().ravel(), want_s)
    assert np.array_equal(q.codes.cpu().numpy().ravel(), want_q)
