"""silu(g) u of the 4-bit FFN where exp(-g) passes the range of 32 bits and
silu(g) does not."""
import numpy as np
import pytest

from tests import mx_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

N = 64  # rows of gate and up, values of the result


def codes_of(values):
    """Codes and scales of a matrix whose rows 4 bits hold."""
    codes, scales = ref.quantize(values)
    assert np.array_equal(ref.dequantize(codes, scales), values)
    return codes, scales


def gate_rows(g):
    """Rows of 64 whose sums are g, multiples of 1/4 in [-96, -80]."""
    m = np.zeros((N, 64))
    m[:, 0], m[:, 1] = -64, -16
    for i, left in enumerate(-g - 80):
        at = 32
        while left > 0:
            m[i, at] = -max(v for v in (0.25, 0.5, 0.75, 1, 1.5, 2, 3) if v <= left)
            left += m[i, at]
            at += 1
    m[:, 63] = np.where(m[:, 63] == 0, 3, m[:, 63])  # the second block's scale is 1/2 in every row
    m[:, 62] = np.where(m[:, 63] == 3, -3, m[:, 62])
    assert np.array_equal(m.sum(axis=1), g)
    return m


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import quantized_moe_expert_sigmoid_amd as m
    m.lib()
    return m


def run(moe, T, E, gate, up):
    """The FFN of T tokens of ones, each of one expert; all experts are the same, down hands a through."""
    ctx = moe.MoeCtx(0)
    try:
        blocks = moe.MxExpertBlocks(E, 64, N)
        for e in range(E):
            views = blocks.views(e)
            for i, m in enumerate((gate, up, np.eye(64))):
                for view, part in zip((views[i], views[3 + i]), codes_of(m)):
                    view.copy_(torch.from_numpy(part))
        x = torch.ones((T, 64), device="cuda")
        idx = torch.arange(T, dtype=torch.int32, device="cuda")[:, None] % E
        out = torch.full_like(x, 9.0)
        moe.moe_expert_ffn_mx(ctx, blocks.table, False, x, idx, torch.ones((T, 1), device="cuda"), N, out)
        ctx.check()
        return out.double().cpu().numpy()
    finally:
        ctx.close()


def quantized(a, margin):
    """a in 4 bits; no value within `margin` of a place where its code turns."""
    codes, scales = ref.quantize(a[None])
    v = np.abs(a) / np.repeat(ref.scale_of(scales), 32)
    mid = (ref.GRID[1:] + ref.GRID[:-1]) / 2
    assert (np.abs(v[:, None] / mid - 1) > margin).all()
    return ref.dequantize(codes, scales)[0]


CALLS = [(1, 1), (2, 16), (5, 2), (200, 3)]


@pytest.mark.parametrize("T,E", CALLS)
def test_far_below_zero(moe, T, E):
    """Gates of -80 to -95.75: exp(-g) passes fp32's range at -88.7, silu(g) leaves that of its normal numbers at -91.8.
    up = 2^p brings silu(g) u between 2^-8 and 2^-6; 4 bits of it are compared exactly (no value lies within 2^-12 of a
    place where its code turns, and a subnormal silu is within 2^-16 of its value here)."""
    g = -80 - 0.25 * np.arange(N)
    p = -8 - np.floor(np.log2(-ref.silu(g)))
    up = np.zeros((N, 64))
    up[:, 5] = 2.0 ** p
    want = quantized(ref.silu(g) * 2.0 ** p, 2.0 ** -12)
    assert (want != 0).all()
    got = run(moe, T, E, gate_rows(g), up)
    assert np.array_equal(got, np.tile(want, (T, 1))), np.argwhere(got != want)[:4].tolist()


@pytest.mark.parametrize("T,E", CALLS)
def test_gates_of_any_size(moe, T, E):
    """Gates from 2^-20 to 6 x 2^122 of both signs: above zero silu(g) is g, far below it nothing, and no NaN."""
    rng = np.random.default_rng(3)
    k = np.concatenate([np.arange(-20, 12), np.linspace(12, 122, 32).round()])
    g = rng.choice([1, 2, 4, 6], N) * 2.0 ** k * np.where(rng.random(N) < 0.5, -1, 1)
    gate, up = np.zeros((N, 64)), np.zeros((N, 64))
    gate[np.arange(N), rng.integers(0, 64, N)] = g
    up[:, 33] = 2.0 ** -k
    assert (g[k > 7] < 0).sum() > 10 and (g[k > 7] > 0).sum() > 10
    want = quantized(ref.silu(g) * 2.0 ** -k, 2.0 ** -12)
    got = run(moe, T, E, gate, up)
    assert np.array_equal(got, np.tile(want, (T, 1))), np.argwhere(got != want)[:4].tolist()
