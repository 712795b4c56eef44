"""NVFP4 quantisation and read-back against the definition on the CPU, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from _experts import E4M3, interleave, quantise_rows, values
from _harness import filled, moe
from workloads import bf16_bits_to_f32, f32_to_bf16_bits, random_bf16

pytestmark = pytest.mark.gpu


def _run(x, g, layout):
    """x [G, R, H] bf16 bits, g [G]: codes and scales as numpy, and the read-back as bf16 bits."""
    m = moe()
    G, R, H = x.shape
    xd = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    gd = torch.from_numpy(np.asarray(g, np.float32)).cuda()
    codes = filled((G, R, H // 2), torch.uint8)
    scales = filled((G, m.nvfp4_scale_bytes(R, H, layout)), torch.uint8)
    out = filled((G, R, H), torch.bfloat16)
    m.moe_quantize_nvfp4(xd, gd, codes, scales, layout)
    m.moe_dequantize_nvfp4(codes, scales, gd, out, layout)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy(), out.view(torch.int16).cpu().numpy().view(np.uint16)


def _check(x, g, layout):
    codes, scales, back = _run(x, g, layout)
    G, R, H = x.shape
    for j in range(G):
        want_q, want_s = quantise_rows(x[j], g[j])
        assert np.array_equal(codes[j], want_q)
        flat = interleave(want_s) if layout == "swizzled" else want_s.reshape(-1)
        assert np.array_equal(scales[j], flat)
        with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
            want = values(want_q, want_s).astype(np.float32) / np.float32(g[j])   # the product is exact in binary32
        finite = np.isfinite(want)
        assert np.array_equal(back[j][finite], f32_to_bf16_bits(want)[finite])


@pytest.mark.parametrize("layout", ["row", "swizzled"])
@pytest.mark.parametrize("G,R,H", [(1, 1, 64), (1, 1, 7168), (2, 5, 192), (3, 127, 64), (1, 128, 256), (2, 129, 448),
                                   (1, 300, 1088), (5, 33, 320), (40, 2, 128)])
def test_quantise_and_back(G, R, H, layout):
    rng = np.random.default_rng(G * 1000 + R + H)
    x = random_bf16(rng, (G, R, H), 2.0)
    g = 2688.0 / np.maximum(np.abs(bf16_bits_to_f32(x)).reshape(G, -1).max(1), 1e-6)
    _check(x, g.astype(np.float32), layout)


@pytest.mark.parametrize("H", [16, 48, 80])
def test_hidden_sizes_of_the_row_layout(H):
    rng = np.random.default_rng(H)
    _check(random_bf16(rng, (2, 7, H)), np.array([300.0, 7.0], np.float32), "row")


@pytest.mark.parametrize("layout", ["row", "swizzled"])
def test_edge_values(layout):
    """Zero and -0 rows, subnormals, huge elements; global scales that zero or saturate every block scale."""
    rng = np.random.default_rng(7)
    x = random_bf16(rng, (6, 9, 128))
    x[:, 0] = 0
    x[:, 1] = 0x8000
    x[:, 2] = rng.integers(1, 128, 128)                       # subnormal
    x[:, 3, ::16] = f32_to_bf16_bits(np.full(8, 3e38, np.float32))
    x[:, 4] = f32_to_bf16_bits(np.array([5.0, 2.5, 0.25, 0.75, 1.25, 1.75, 3.5, 6.0] * 16, np.float32))  # ties
    _check(x, np.array([1.0, 0.0, 1e-30, 1e30, 448.0, 2.0 ** -100], np.float32), layout)


def test_every_scale_is_read_back():
    """A block whose maximum is 6 * value(sf) / g gets that scale, for every positive e4m3 value."""
    sf = np.array([c for c in range(1, 127)])
    v = (6 * E4M3[sf]).astype(np.float32)
    x = np.zeros((1, len(sf), 64), np.uint16)
    x[0, :, 0] = f32_to_bf16_bits(v)
    codes, scales, back = _run(x, [1.0], "row")
    assert np.array_equal(scales.reshape(len(sf), 4)[:, 0], sf)
    assert np.array_equal(back[0, :, 0], x[0, :, 0])


def test_unaligned_buffers():
    """bf16 rows at 16 bytes, codes at 8, row-major scales at any byte."""
    m = moe()
    x = torch.randn(1, 70, 192, device="cuda").bfloat16()
    g = torch.tensor([300.0], device="cuda")
    want = m.quantize_nvfp4(x, g, scale_layout="row")
    shifted = torch.empty(x.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(x.shape)
    shifted.copy_(x)
    n = want.scales.numel()
    codes, scales = filled((want.codes.numel() + 8,), torch.uint8), filled((n + 1,), torch.uint8)
    m.moe_quantize_nvfp4(shifted, g, codes[8:], scales[1:], "row")
    assert torch.equal(codes[8:], want.codes.flatten()) and torch.equal(scales[1:], want.scales.flatten())
    assert (codes[:8] == 0xa5).all() and int(scales[0]) == 0xa5
    out = filled((x.numel() + 8,), torch.bfloat16)
    m.moe_dequantize_nvfp4(codes[8:], scales[1:], g, out[8:].view(x.shape), "row")
    assert torch.equal(out[8:].view(torch.int16), m.dequantize_nvfp4(want, g).view(torch.int16).flatten())


def test_empty_calls_write_nothing():
    m = moe()
    g = torch.ones(1, device="cuda")
    for shape in ((0, 4, 64), (1, 0, 64)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        codes, scales = filled((64,), torch.uint8), filled((64,), torch.uint8)
        m.moe_quantize_nvfp4(x, g, codes, scales)
        m.moe_dequantize_nvfp4(codes, scales, g, x)
        assert (codes == 0xa5).all() and (scales == 0xa5).all()


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^31 elements."""
    m = moe()
    R, H = 300_001, 7168
    x = torch.zeros((1, R, H), dtype=torch.bfloat16, device="cuda")
    x[0, -2:] = torch.randn(2, H, device="cuda")
    g = torch.tensor([100.0], device="cuda")
    q = m.quantize_nvfp4(x, g)
    tail = m.quantize_nvfp4(x[:, -2:].contiguous(), g, scale_layout="row")
    assert torch.equal(q.codes[0, -2:], tail.codes[0]) and not q.codes[0, :-2].any()
    at = torch.tensor([((R - 2 + i) // 128 * (H // 64) + c // 4) * 512 + (R - 2 + i) % 32 * 16
                       + (R - 2 + i) % 128 // 32 * 4 + c % 4 for i in range(2) for c in range(H // 16)], device="cuda")
    assert torch.equal(q.scales[0][at], tail.scales.flatten())
    back = m.dequantize_nvfp4(q, g)
    assert torch.equal(back[0, -2:], m.dequantize_nvfp4(tail, g)[0]) and not back[0, :-2].any()


def test_agrees_with_the_dispatch_quantiser():
    """The dispatch divides by 6 where the quantiser multiplies by 1/6: a block's scale may go to the other neighbour of a
    boundary, and to nothing else; blocks with the same scale have the same codes."""
    rng = np.random.default_rng(11)
    x = random_bf16(rng, (1, 64, 1024))
    g = 2688.0 / 4.0                     # many scales on boundaries
    codes, scales, _ = _run(x, [g], "row")
    same = total = 0
    for r in range(64):
        q, sf = oracle.quant_nvfp4_row(x[0, r], g)
        s = scales[0].reshape(64, 64)[r]
        assert (np.abs(sf.astype(int) - s.astype(int)) <= 1).all()
        eq = sf == s
        assert (codes[0, r].reshape(64, 8)[eq] == q.reshape(64, 8)[eq]).all()
        t = np.abs(bf16_bits_to_f32(x[0, r])).reshape(64, 16).max(1).astype(np.float64) / 6 * g
        mid = (E4M3[sf] + E4M3[s]) / 2
        assert (np.abs(t - mid)[~eq] <= 2.0 ** -22 * t[~eq]).all()
        same, total = same + int(eq.sum()), total + 64
    assert same >= 0.9 * total


def test_one_matrix():
    m = moe()
    x, g = torch.randn(5, 128, device="cuda").bfloat16(), torch.tensor([200.0], device="cuda")
    one, group = m.quantize_nvfp4(x, g), m.quantize_nvfp4(x[None], g)
    assert one.codes.shape == (5, 64) and torch.equal(one.codes, group.codes[0]) and torch.equal(one.scales, group.scales[0])
    assert torch.equal(m.dequantize_nvfp4(one, g), m.dequantize_nvfp4(group, g)[0])


@pytest.mark.parametrize("raw", [False, True])
def test_results_belong_to_the_stream_that_writes_them(raw):
    """Memory that the current stream still works on is not handed to a call on another one."""
    m = moe()
    g = torch.ones(1, device="cuda")
    x = torch.ones(256, 4096, device="cuda", dtype=torch.bfloat16)
    want = m.quantize_nvfp4(x, g)
    back = m.dequantize_nvfp4(want, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(10 ** 7)
    held = [torch.zeros_like(want.codes), torch.zeros_like(want.scales), torch.zeros_like(back)]
    at = [t.data_ptr() for t in held]
    for t in held:
        t.fill_(7)
    del held, t                          # free again for the current stream, and not yet written by it
    q = m.quantize_nvfp4(x, g, stream=side.cuda_stream if raw else side)
    y = m.dequantize_nvfp4(q, g, stream=side.cuda_stream if raw else side)
    assert not {q.codes.data_ptr(), q.scales.data_ptr(), y.data_ptr()} & set(at)
    torch.cuda.synchronize()
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales) and torch.equal(y, back)
