"""MoeLayer's weights set from another stream than the context's, nothing
synchronised: fp32 copies outlive the quantiser that reads them."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bits", [8, 4, 2, "mx"])
@pytest.mark.parametrize("on_gpu", [False, True])
def test_weights_set_while_the_context_is_busy(bits, on_gpu):
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.layer import MoeLayer
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    H, I, E, k, T = 256, 128, 6, 2, 9
    rng = np.random.default_rng(1)
    mats = [[rng.standard_normal(s).astype(np.float32) * s[1] ** -0.5 for s in ((I, H), (I, H), (H, I))]
            for _ in range(E + 1)]
    router = [rng.standard_normal(s).astype(np.float32) for s in ((E, H), (E,))]
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    busy = torch.randn((4096, 4096), device="cuda")

    def fill(layer, of):
        for e in range(E):
            layer.set_expert_fp32(e, *(of(m) for m in mats[e]))
        layer.set_shared_fp32(*(of(m) for m in mats[E]))
        layer.set_router(*(of(m) for m in router))

    def wait_a_while():  # about 100 ms on the current stream
        y = busy
        for _ in range(40):
            y = torch.mm(y, busy).mul_(2.0 ** -6)
        return y

    plain = moe.MoeCtx(0)
    want = MoeLayer(plain, H, I, E, k, bits=bits)
    fill(want, lambda m: m)
    result = want.forward(x)["out"].clone()
    torch.cuda.synchronize()

    ctx, caller = moe.MoeCtx(0, torch.cuda.Stream()), torch.cuda.Stream()
    got = MoeLayer(ctx, H, I, E, k, bits=bits)
    torch.cuda.synchronize()
    with torch.cuda.stream(ctx.stream):
        wait_a_while()
    with torch.cuda.stream(caller):
        if on_gpu:  # still in the making when they are handed over, gone right after
            zero = wait_a_while()[0, 0] * 0
            fill(got, lambda m: torch.from_numpy(m).cuda().double() + zero)
        else:
            fill(got, lambda m: m)
        junk = [torch.full((I, H), float("nan"), device="cuda") for _ in range(8)]
    ctx.stream.synchronize()
    out = got.forward(x)["out"]
    torch.cuda.synchronize()
    for c in (plain, ctx):
        c.check()
    for a, b in ((got.experts, want.experts), (got.shared, want.shared)):
        for e in range(a.n if a is not None else 0):
            for p, q in zip(a.views(e), b.views(e)):
                assert torch.equal(p, q), e
    assert torch.equal(out, result) and out.isfinite().all()
    del junk
    for c in (plain, ctx):
        c.close()
