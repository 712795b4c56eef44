"""What the few-token layer's sums of NVFP4 blocks leave of a block, by their restatement on the CPU."""
import numpy as np
import pytest

from _terms import Differences, split


@pytest.mark.parametrize("below", [0, 5, 11, 13, 14, 20, 27, 28, 40, 90])
def test_five_terms_leave_at_most_2_to_the_minus_12_of_a_block(below):
    """Whatever the row's largest value is: here 2^below times the blocks', or up to twice that."""
    rng = np.random.default_rng(below)
    x = np.zeros((400, 65 * 16), np.float32)
    x[:, 3] = 2.0 ** below
    b = rng.standard_normal((400, 64, 16))
    b *= (2.0 ** -rng.random((400, 64)) / np.abs(b).max(2))[..., None]
    x[:, 16:] = b.reshape(400, -1)
    left = np.abs(split(x) - x)[:, 16:].reshape(400, 64, 16)
    most = np.abs(x[:, 16:]).reshape(400, 64, 16).max(2)
    assert (left.max(2) <= 2.0 ** -12 * most).all()
    assert np.sqrt((left ** 2).mean() / (most ** 2).mean()) <= 2.0 ** -14.5


@pytest.mark.parametrize("below", [11, 14, 17, 20, 30, 60])
def test_the_neighbours_of_an_outlier_keep_their_values(below):
    """In the block of an outlier 2^below times its neighbours: 2^-18 of the outlier is left by a pass, 2^-36 by two, and so
    on, and rows of more than 11 orders have another pass: less than 2^-5 of the neighbours is left."""
    rng = np.random.default_rng(below)
    x = rng.standard_normal((400, 64)).astype(np.float32)
    x[:, 21] = 2.0 ** below
    left = (split(x) - x)[:, 16:32]
    left[:, 5] = 0
    assert np.sqrt((left ** 2).mean()) <= 2.0 ** -5


def test_the_differences_tell_five_terms_from_four():
    d = Differences()
    assert d.holds(d.output(5)), d.errors(d.output(5))
    assert not d.holds(d.output(4)), d.errors(d.output(4))
    rms, _ = d.errors(d.output(4))
    assert all(r > 2 * lim for r, lim in zip(rms, d.RMS))


def test_a_lost_fifth_term_of_h_alone_is_told():
    d = Differences()
    x = split(d.x, 5)
    from _experts import silu
    from workloads import bf16_bits_to_f32, f32_to_bf16_bits
    h = ((x @ d.up.T) * silu(x @ d.gate.T)).astype(np.float32)
    out = bf16_bits_to_f32(f32_to_bf16_bits((split(h, 4) @ d.down.T).astype(np.float32))).astype(np.float64)
    assert not d.holds(out), d.errors(out)
