"""The 64-bit definition of the microscaled 4-bit format that the GPU tests
compare with, pinned by hand-worked values, and the host-only helpers."""
import numpy as np
import pytest

from tests import mx_ref as ref


def one(values):
    x = np.zeros((1, 32))
    x[0, :len(values)] = values
    codes, scales = ref.quantize(x)
    return ref.dequantize(codes, scales)[0, :len(values)], int(scales[0, 0]), codes[0]


def test_scale_puts_the_largest_between_four_and_eight():
    for top, byte in ((4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (0.99, 124), (2.0 ** -130, 0), (0.0, 0),
                      (2.0 ** 127, 252)):
        assert one([top, -top / 2])[1] == byte, top


def test_rounding_by_hand():
    v, byte, codes = one([6, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1, -0.2])
    assert byte == 127
    assert v.tolist() == [6, 0, 0.5, 1, 1, 2, 2, 4, 4, -6, 0]
    assert codes[:6].tolist() == [0x07, 0x21, 0x42, 0x64, 0xF6, 0x08]
    assert one([7.9, 1.0])[0].tolist() == [6, 1]  # above 6


def test_bad_blocks():
    for v in (np.inf, -np.inf, np.nan):
        x = np.ones((1, 64))
        x[0, 40] = v
        codes, scales = ref.quantize(x)
        assert scales.tolist() == [[125, 255]] and (codes[0, 16:] == 0).all()
        back = ref.dequantize(codes, scales)
        assert (back[0, :32] == 1).all() and np.isnan(back[0, 32:]).all()


def test_ffn_tolerance_covers_a_turned_code():
    rng = np.random.default_rng(1)
    x, g, u, d = (rng.standard_normal(s) for s in ((3, 64), (64, 64), (64, 64), (96, 64)))
    y, tol = ref.ffn(x, g, u, d)
    assert y.shape == tol.shape == (3, 96) and (tol > 0).all() and (tol < 1e-2 * np.abs(y).max()).any()


def test_expert_layout():
    import quantized_moe_expert_sigmoid_amd as m
    n, offs = m.moe_mx_expert_layout(6144, 2048)
    codes, scales = 6144 * 2048 // 2, 6144 * 2048 // 32
    assert offs == [0, codes, 2 * codes, 3 * codes, 3 * codes + scales, 3 * codes + 2 * scales]
    assert n == 3 * (codes + scales) == 20_054_016
    assert m.moe_mx_expert_layout(64, 64)[1] == [0, 2048, 4096, 6144, 6400, 6656]
    with pytest.raises(m.MoeError):
        m.moe_mx_expert_layout(64, 32)
