"""The tolerance of the 4-bit FFN's tests, pinned from both sides: it holds what
a code or a block's scale that turns within the sums' error does to the result,
only the terms for that hold it, and elsewhere it is no wider than the sums."""
import numpy as np
import pytest

from tests import mx_ref as ref

ROWS, H, I, OUT = 5, 128, 128, 96


def matrices(seed):
    rng = np.random.default_rng(seed)
    return [ref.dequantize(*ref.quantize(rng.standard_normal(s) * s[1] ** -0.5)) for s in ((ROWS, H), (I, H), (I, H), (OUT, I))]


def sums_only(x, gate, up, down):
    """The tolerance without turned codes and scales."""
    a = ref.silu(x @ gate.T) * (x @ up.T)
    return (I / 64 + 16) * 2.0 ** -23 * (np.abs(ref.dequantize(*ref.quantize(a))) @ np.abs(down).T)


def check_turn(x, gate, up, down, row, block, other):
    """`other`: the block's values with the code or scale turned. Its result is inside the tolerance in the row where that
    happens, and outside without the turned terms wherever down's values are not zero; most of the other rows have the
    sums' errors alone."""
    y, tol = ref.ffn(x, gate, up, down)
    q = ref.dequantize(*ref.quantize(ref.silu(x @ gate.T) * (x @ up.T)))
    turned = q.copy()
    turned[row, block] = other
    change = np.abs(turned @ down.T - y)
    moved = change[row] > 0
    assert moved.mean() > 0.7 and (change[row] <= tol[row]).all()
    plain = sums_only(x, gate, up, down)
    assert (change[row] > 100 * plain[row])[moved].mean() > 0.95
    rest = np.arange(ROWS) != row
    assert (tol[rest] <= 1.0001 * plain[rest]).mean() > 0.5


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("mid", range(7))
def test_a_turned_code(seed, mid):
    """up's row is scaled so that one value lies on the midpoint of two codes; the other of the two is taken."""
    x, gate, up, down = matrices(seed)
    row, block, scale = 2, slice(32, 64), 2.0 ** -2
    a = (ref.silu(x @ gate.T) * (x @ up.T))
    # the block's largest value becomes 7 scales, another one the midpoint
    top, at = 32 + np.argsort(-np.abs(a[row, block]))[[0, 3]]
    up[block] *= 0.1 * scale / np.abs(a[row, block]).max()
    a = (ref.silu(x @ gate.T) * (x @ up.T))
    up[top] *= 7 * scale / np.abs(a[row, top])
    value = (ref.GRID[mid] + ref.GRID[mid + 1]) / 2 * scale
    up[at] *= value / np.abs(a[row, at])
    a = (ref.silu(x @ gate.T) * (x @ up.T))
    assert abs(abs(a[row, at]) - value) < 1e-12 and ref.quantize(a)[1][row, 1] == 125
    q = ref.dequantize(*ref.quantize(a))[row, block]
    ends = np.sign(a[row, at]) * ref.GRID[[mid, mid + 1]] * scale
    assert q[at - 32] in ends
    other = q.copy()
    other[at - 32] = ends.sum() - q[at - 32]
    check_turn(x, gate, up, down, row, block, other)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("side", [-1, 1])
def test_a_turned_scale(seed, side):
    """A block's largest value lies just below or above a power of two; the block is quantised with the other scale."""
    x, gate, up, down = matrices(seed)
    row, block = 2, slice(64, 96)
    a = ref.silu(x @ gate.T) * (x @ up.T)
    up[block] *= 2.0 * (1 + side * 2.0 ** -40) / np.abs(a[row, block]).max()
    a = ref.silu(x @ gate.T) * (x @ up.T)
    byte = int(ref.quantize(a)[1][row, 2])
    assert byte == (125 if side < 0 else 126)
    other = 2.0 ** (byte - side - 127)  # scales are twice as far or half as far apart
    v = a[row, block] / other
    mags = ref.GRID[np.abs(np.minimum(np.abs(v), 6)[:, None] - ref.GRID).argmin(axis=1)]
    check_turn(x, gate, up, down, row, block, np.sign(v) * mags * other)


def test_elsewhere_it_is_the_sums():
    """Random values: half of all tolerances are below 2^-14 of the results' usual size, so a value that is off by more
    than a few of the sums' roundings shows."""
    for seed in range(3):
        y, tol = ref.ffn(*matrices(10 + seed))
        assert (tol > 0).all() and np.median(tol) < 2.0 ** -14 * np.median(np.abs(y))
