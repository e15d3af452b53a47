"""The e4m3 oracle pinned to the format's definition, exact rationals and
torch's own narrowing."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8


def test_decode_closed_forms():
    d = fp8.decode(np.arange(256))
    assert d[0] == 0 and d[1] == 2.0 ** -9 and d[7] == 7 * 2.0 ** -9 and d[8] == 2.0 ** -6
    assert d[0x38] == 1.0 and d[0x3F] == 1.875 and d[0x7E] == 448.0 and np.isnan(d[0x7F]) and np.isnan(d[0xFF])
    assert np.signbit(d[0x80]) and d[0xFE] == -448.0
    assert np.all(np.diff(d[:127]) > 0)


def test_decode_and_encode_agree_with_torch():
    codes = np.arange(256).astype(np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode(codes), t, equal_nan=True)
    assert np.array_equal(fp8.encode(t[~np.isnan(t)]), codes[~np.isnan(t)])
    g = np.random.default_rng(3)
    v = np.concatenate([g.standard_normal(20000) * 2.0 ** g.integers(-12, 9, 20000), [448.0, 463.9, -448.0]])
    v = np.clip(v, -448, 448).astype(np.float32)
    assert np.array_equal(fp8.encode(v), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_encode_is_nearest_with_even_ties():
    grid = [Fraction(float(x)) for x in fp8.decode(np.arange(127))]
    mid = [(a + b) / 2 for a, b in zip(grid, grid[1:])]
    for j, m in enumerate(mid):
        assert fp8.encode(float(m)) == (j if j % 2 == 0 else j + 1)
        assert fp8.encode(np.nextafter(float(m), 0)) == j
        assert fp8.encode(np.nextafter(float(m), 1e9)) == j + 1
        assert fp8.encode(-float(m)) == (j if j % 2 == 0 else j + 1) + 128


def test_steps():
    s, i = fp8.step(np.array([448.0, 1.0, 0.0, 1e-37, np.inf, np.nan, 3.4e38], np.float32))
    assert s[0] == 1 and i[0] == 1 and s[1] == np.float32(1) / np.float32(448)
    assert s[2] == 2.0 ** -126 and s[3] == 2.0 ** -126 and i[2] == 2.0 ** 126
    assert np.isnan(s[4]) and np.isnan(s[5]) and np.isfinite(s[6])


@pytest.mark.parametrize("n,k", [(1, 128), (129, 256), (300, 384)])
def test_blocks_reach_the_largest_code_and_stay_within_half_a_step(n, k):
    g = np.random.default_rng(n)
    w = (g.standard_normal((n, k)) * np.exp(g.standard_normal((n, 1)))).astype(np.float32)
    q, s = fp8.quantize(w)
    back = fp8.decode(q) * np.repeat(s.T, 128, 1)
    blocks = np.abs(fp8.decode(q)).reshape(n, k // 128, 128)
    assert np.all(blocks.max(2) == 448)
    # half a step of a 4-bit significand, 2^-9 steps at the lowest binade; i and v i rounded
    assert np.all(np.abs(back - w) <= (2.0 ** -4 + 2.0 ** -22) * np.abs(w) + np.repeat(s.T, 128, 1) * 2.0 ** -10)
    codes, scale = fp8.quantize_weight(w)
    assert scale.shape == (-(-n // 128), k // 128)
    for a in range(scale.shape[0]):
        for b in range(k // 128):
            assert scale[a, b] == fp8.step(np.abs(w[128 * a:128 * a + 128, 128 * b:128 * b + 128]).max())[0]
            assert np.abs(fp8.decode(codes[128 * a:128 * a + 128, 128 * b:128 * b + 128])).max() == 448


def test_norm_and_swiglu_closed_forms():
    v, h = fp8.rms_norm(np.array([[3.0, -4.0]]), [1.0, 2.0], 0.0, np.array([[0.0, 8.0]]))
    assert np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(v, np.array([[3.0, 8.0]]) / np.sqrt(12.5), rtol=1e-15)
    assert np.allclose(fp8.swiglu(np.array([[0.0, 1.0, -1000.0, 5.0, 7.0, 2.0]])), [[0.0, 7.0 / (1 + np.exp(-1.0)), 0.0]])


def test_product_by_hand():
    x = np.full((1, 256), 0x38, np.uint8)      # 1
    w = np.full((130, 256), 0x40, np.uint8)    # 2
    scale = np.array([[1.0, 2.0], [4.0, 8.0]])
    y, size, top = fp8.product(x, np.array([[0.5], [0.25]]), w, scale)
    assert np.all(y[0, :128] == 256 * (0.5 + 0.5)) and np.all(y[0, 128:] == 256 * (2 + 2)) and np.array_equal(y, size)
    assert np.array_equal(top, y / 8)
    x[0, 3], w[0, 3], x[0, 5] = 0x7E, 0xFE, 0  # 448 and -448: 2^16 in binades
    y, size, top = fp8.product(x, np.array([[1.0], [1.0]]), w, np.ones((2, 2)))
    assert y[0, 0] == 2 * 254 - 448.0 ** 2 and size[0, 0] == 2 * 254 + 448.0 ** 2 and top[0, 0] == 2.0 ** 16 + 31 * 2
