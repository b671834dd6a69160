"""Rotary positions at frequencies of any size: angles in exact integers."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import tiled_online_softmax_02_gb300 as attn


def two_pi(bits):
    """2 pi as a fraction, by pi = 16 atan(1 / 5) - 4 atan(1 / 239) in integers."""
    one = 1 << (bits + 16)

    def atan(n):
        term = total = one // n
        k = 1
        while term:
            term //= n * n
            k += 2
            total += -(term // k) if k % 4 == 3 else term // k
        return total
    return Fraction(2 * (16 * atan(5) - 4 * atan(239)), one)


TURN = two_pi(400)


def angle(pos, freq):
    """pos * freq modulo a turn, in [0, 2 pi), rounded once."""
    w = pos * Fraction(float(freq))
    return float(w - TURN * (w // TURN))


def test_exact_angles():
    assert abs(float(TURN) - 2 * math.pi) < 1e-15 and abs(TURN - two_pi(500)) < Fraction(1, 1 << 398)
    assert abs(angle(3, 0.731) - 3 * 0.731) < 1e-14 and abs(angle(-1, 1.0) - (2 * math.pi - 1)) < 1e-14
    assert abs(math.sin(angle(123456, 1.0)) - math.sin(123456.0)) < 1e-9


FREQS = [1e-9, 1.0, 126.9, 127.99, 128.0, 255.0, 257.3, 1000.0, 1e6, 123456789.123, 2.0 ** 40 + 1, 3e15, 2.0 ** 53 - 1, 1e18, 4e18]


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("freq", FREQS)
def test_angles_at_far_positions(freq, sign):
    """Angles to 2^-24 turns, sine and cosine to 2^-22 of 1 beside that, products and sums of fp32: 2^-20 in all."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.Generator(np.random.PCG64(5))
    pos = np.concatenate([[0, 1, -1, 2, 77777, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1], rng.integers(-2 ** 31, 2 ** 31, 200)])
    q = torch.zeros((len(pos), 1, 2), device="cuda")
    q[..., 0] = 1.0
    got, _ = attn.attn_rope(q, None, torch.tensor([sign * freq], dtype=torch.float64, device="cuda"),
                            positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    w = np.array([angle(int(p), sign * freq) for p in pos])
    want = np.stack([np.cos(w), np.sin(w)], -1)
    assert np.abs(got[:, 0].double().cpu().numpy() - want).max() <= 2.0 ** -20
