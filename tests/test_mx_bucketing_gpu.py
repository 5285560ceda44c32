"""The 4-bit FFN's bucketing at and around the most entries that one workgroup
takes (32768, 128 KB of LDS), and what timing counts on both sides of it."""
import numpy as np
import pytest

from tests.test_mx_gpu import BF16, Experts, check_ffn

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import quantized_moe_expert_sigmoid_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ctx(moe):
    c = moe.MoeCtx(0)
    yield c
    c.close()


@pytest.fixture(scope="module")
def experts(moe, ctx):
    return Experts(moe, ctx, 5, 20, 64, 64)


def call(moe, ctx, experts, x, idx, w):
    out = torch.full_like(x, 9.0)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table[:19], False, x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(),
                          64, out)
    return out


def random_call(rng, T, k):
    x = torch.from_numpy(rng.standard_normal((T, 64))).to(BF16).cuda()
    idx = np.argsort(rng.random((T, 19)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < 0.1] = -1
    return x, idx, np.where(idx < 0, 0, rng.random((T, k))).astype(np.float32)


SIZES = [(2049, 8), (3001, 7), (6553, 5), (4096, 8), (2048, 16), (32768, 1), (32769, 1), (4681, 7)]


@pytest.mark.parametrize("T,k", SIZES)
def test_many_entries(moe, ctx, experts, T, k):
    """A token's result is what it is in a call of few tokens, bit for bit: tokens are independent, and a tile's lines too
    (calls of 64 tokens and of thousands take the same stages of 256 k here, two blocks long). Some tokens also against the
    definition."""
    rng = np.random.default_rng(T)
    x, idx, w = random_call(rng, T, k)
    out = call(moe, ctx, experts, x, idx, w)
    ctx.check()
    for t in {0, 64, T // 2, T - 64}:
        part = slice(t, t + 64)
        few = call(moe, ctx, experts, x[part], idx[part], w[part])
        assert torch.equal(out[part], few), t
    ctx.check()
    some = rng.permutation(T)[:300]
    at = torch.from_numpy(some).cuda()
    check_ffn(out[at], x[at], idx[some], w[some], experts, 19, False)


@pytest.mark.parametrize("T,k", [(4096, 8), (4681, 7)])
def test_many_entries_with_bad_ids(moe, ctx, experts, T, k):
    """Ids out of range and repeated ones, in the last token and in others: reported, and without effect."""
    rng = np.random.default_rng(k)
    x, idx, w = random_call(rng, T, k)
    w = rng.random((T, k)).astype(np.float32)
    good = idx.copy()
    for t in (0, 1023, 1024, T - 1):
        idx[t, :4] = (2, 2, 19, -7)
        good[t, :4] = (2, -1, -1, -1)
        idx[t, 4:], good[t, 4:] = -1, -1
    out = call(moe, ctx, experts, x, idx, w)
    with pytest.raises(moe.MoeError):
        ctx.check()
    want = call(moe, ctx, experts, x, good, w)
    ctx.check()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,launches", [(50, 1), (4096, 1), (4097, 2)])
def test_timing_counts_the_quantiser(moe, experts, T, launches):
    """Up to 32768 entries bucketing and quantiser are one launch; beyond it both are counted under the same stage, the
    quantiser as a launch of its own."""
    c = moe.MoeCtx(0)
    try:
        x, idx, w = random_call(np.random.default_rng(1), T, 8)
        plain = call(moe, c, experts, x, idx, w)
        c.enable_timing(True)
        timed = call(moe, c, experts, x, idx, w)
        times = c.read_timing()
        c.enable_timing(False)
        assert torch.equal(plain, timed)
        assert times["bucket"][1] == launches and times["bucket"][0] > 0, times
        for stage in ("gateup", "down", "combine"):
            assert times[stage][1] == 1 and times[stage][0] > 0, times
    finally:
        c.close()
