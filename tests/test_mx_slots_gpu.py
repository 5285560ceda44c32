"""The experts' FFN in 4 bits holds the slots' results in 32 bits whatever the
type and however many tokens share a call: only the sum is rounded."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.test_mx_gpu import BF16, FP16, FP32, TYPES, Experts

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


def routing(rng, T, k, E):
    idx = np.argsort(rng.random((T, E)) + 0.3 * np.arange(E) / E, axis=1)[:, :k].astype(np.int32)
    return torch.from_numpy(idx).cuda(), torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()


CALLS = [(1, 2, 8, 128, 64, True), (2, 2, 20, 512, 192, True), (3, 8, 9, 192, 128, False), (4, 8, 64, 512, 512, True),
         (33, 4, 6, 256, 128, True), (200, 3, 5, 192, 320, False), (700, 2, 3, 512, 512, True), (2100, 16, 20, 64, 64, True)]


@pytest.mark.parametrize("T,k,E,H,I,shared", CALLS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_16_bit_results_are_32_bit_ones_rounded(moe, ctx, dtype, T, k, E, H, I, shared):
    """The same hidden states, held in 16 bits and in 32: the same blocks, products and sums, so the results of the one
    are those of the other rounded once. Twice the same call: the same bits."""
    rng = np.random.default_rng(T + H)
    experts = Experts(moe, ctx, T + k, E + int(shared), H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).cuda()
    idx, w = routing(rng, T, k, E)
    out = []
    for v in (x, x, x.float()):
        out.append(torch.full_like(v, 9.0))
        moe.moe_expert_ffn_mx(ctx, experts.blocks.table, shared, v, idx, w, I, out[-1])
    ctx.check()
    assert out[2].abs().max() > 0.1
    assert torch.equal(out[0], out[1])
    assert torch.equal(out[0], out[2].to(dtype))


@pytest.mark.parametrize("T", [2, 3, 4, 70, 600])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_token_alone_is_the_token_in_a_batch(moe, ctx, dtype, T):
    """Sums that 32 bits hold exactly do not depend on the kernels that make them. gate, up and down have one scale, tokens
    small whole numbers: sums of gate and up are multiples of 2^-8 below 2^6; blocks of silu(g) u lie within a few powers
    of two (asserted), so down's sums of 128 products are multiples of some 2^n and below 2^(n + 24)."""
    E, k, H, I = 40, 3, 128, 128
    rng = np.random.default_rng(T)
    blocks = moe.MxExpertBlocks(E + 1, H, I)
    for e in range(E + 1):
        for i, v in enumerate(blocks.views(e)):
            if i < 3:
                v.copy_(torch.from_numpy(rng.integers(0, 256, tuple(v.shape), dtype=np.uint8)))
            else:
                v.fill_(120)
    x = torch.from_numpy(rng.choice([0.0, 1, 2, 3, 4, 6], (T, H)) * rng.choice([-1.0, 1.0], (T, H)))
    x[:, ::32] = 4  # every block has the scale one
    x = x.to(dtype).cuda()
    idx, w = routing(rng, T, k, E)
    for e in range(E + 1):
        gate, up = (ref.dequantize(v.cpu().numpy(), s.cpu().numpy()) for v, s in zip(blocks.views(e)[:2], blocks.views(e)[3:5]))
        xv = x.double().cpu().numpy()
        g = xv @ gate.T
        scales = ref.quantize(ref.silu(g) * (xv @ up.T))[1].astype(int)
        # a code is a multiple of 2^-1 up to 6, its products with down's up to 36 and multiples of 2^-2: 128 of them within
        # 2^(13 + 2) steps of one scale, and nine powers of two of scales are left
        assert (scales.max(axis=1) - scales.min(axis=1)).max() <= 9
    batch = torch.empty_like(x)
    moe.moe_expert_ffn_mx(ctx, blocks.table, True, x, idx, w, I, batch)
    for t in range(0, T, max(1, T // 20)):
        alone = torch.empty_like(x[:1])
        moe.moe_expert_ffn_mx(ctx, blocks.table, True, x[t:t + 1], idx[t:t + 1], w[t:t + 1], I, alone)
        assert torch.equal(alone[0], batch[t]), t
    ctx.check()
    assert batch.isfinite().all() and (batch != 0).float().mean() > 0.9


@pytest.mark.parametrize("T,k,E,H,I", [(1, 4, 8, 256, 128), (8, 4, 8, 256, 128), (150, 3, 6, 512, 192)])
def test_norm_of_the_error(moe, ctx, T, k, E, H, I):
    """bf16 results are off by the rounding of the sum: at most 2^-8 of each value where no code turned. The fp32 call of
    the same tokens says where the sums are; every value within 2^-8 of it, and the norm of all within 2^-8 / sqrt(3)
    times 1.05 (a rounding error is uniform within half a step, and a half step is at most 2^-8 of the value)."""
    rng = np.random.default_rng(k)
    experts = Experts(moe, ctx, 3, E + 1, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    idx, w = routing(rng, T, k, E)
    got, want = torch.empty_like(x), torch.empty((T, H), device="cuda")
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, x, idx, w, I, got)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, x.float(), idx, w, I, want)
    d = got.double() - want.double()
    assert (d.abs() <= 2.0 ** -8 * want.double().abs() + 2.0 ** -130).all()
    assert d.norm() <= 1.05 * 2.0 ** -8 / 3 ** 0.5 * want.double().norm()
