"""The 4-bit operators as they are used together: the layer with bits="mx",
and the experts' FFN step by step through the grouped product."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.test_mx_gpu import BF16, FP32, Experts, check_ffn

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


@pytest.mark.parametrize("T,shared,top_p", [(1, True, 0.0), (5, False, 0.0), (60, True, 0.7)])
def test_layer(moe, ctx, T, shared, top_p):
    from quantized_moe_expert_sigmoid_amd.layer import MoeLayer
    H, I, E, k = 192, 128, 8, 3
    rng = np.random.default_rng(T)
    layer = MoeLayer(ctx, H, I, E, k, bits="mx", has_shared=shared, top_p=top_p)
    mats = [[rng.standard_normal(s).astype(np.float32) * s[1] ** -0.5 for s in ((I, H), (I, H), (H, I))]
            for _ in range(E + int(shared))]
    for e in range(E):
        layer.set_expert_fp32(e, *mats[e])
    if shared:
        layer.set_shared_fp32(*mats[E])
    else:
        with pytest.raises(AttributeError):
            layer.set_shared_fp32(*mats[0])
    with pytest.raises(IndexError):
        layer.set_expert_fp32(E, *mats[0])
    layer.set_router(rng.standard_normal((E, H)).astype(np.float32) * 0.1, rng.standard_normal(E).astype(np.float32) * 0.1)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda()
    b = layer.forward(x)
    ctx.check()
    experts = Experts.__new__(Experts)
    experts.values = [[ref.dequantize(*ref.quantize(m.astype(np.float64))) for m in three] for three in mats]
    idx, w = b["idx"].cpu().numpy(), b["w"].cpu().numpy()
    assert idx.shape == (T, k) and (top_p > 0 or (idx >= 0).all())
    check_ffn(b["out"], x, idx, w, experts, E, shared)
    # the router is the one of the other widths
    topk_idx, topk_w = torch.empty_like(b["idx"]), torch.empty_like(b["w"])
    moe.moe_router_topk(ctx, x, layer.w_router, layer.bias, k, topk_idx, topk_w, top_p=top_p)
    assert torch.equal(topk_idx, b["idx"]) and torch.equal(topk_w, b["w"])


def test_steps_make_the_ffn(moe, ctx):
    """Quantiser, bucketing, grouped products and combine, one after another, against the one call."""
    T, k, E, H, I = 45, 3, 7, 256, 192
    rng = np.random.default_rng(11)
    experts = Experts(moe, ctx, 4, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).float().cuda()
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm = i32(E), i32(E + 1), i32(T * k)
    moe.moe_bucket_tokens(ctx, idx, E, counts, offsets, perm)
    xq = moe.moe_mx_quantize(ctx, x, u8(T, H // 2), u8(T, H // 32))
    stack = [torch.stack([experts.blocks.views(e)[i] for e in range(E)]) for i in range(6)]
    g, u = torch.empty((T * k, I), device="cuda"), torch.empty((T * k, I), device="cuda")
    for out, i in ((g, 0), (u, 1)):
        moe.moe_mx_grouped_matmul(ctx, *xq, stack[i], stack[3 + i], offsets, out, in_rows=perm // k)
    aq = moe.moe_mx_quantize(ctx, g / (1 + torch.exp(-g)) * u, u8(T * k, I // 2), u8(T * k, I // 32))
    y = torch.zeros((T, k + 1, H), device="cuda")
    place = perm // k * (k + 1) + perm % k
    moe.moe_mx_grouped_matmul(ctx, *aq, stack[2], stack[5], offsets, y.view(-1, H), out_rows=place.int())
    out = moe.moe_combine(ctx, y, w, False, torch.empty((T, H), device="cuda"))
    whole = moe.moe_expert_ffn_mx(ctx, experts.blocks.table, False, x, idx, w, I, torch.empty_like(x))
    ctx.check()
    for got in (out, whole):
        check_ffn(got, x, idx.cpu().numpy(), w.cpu().numpy(), experts, E, False)


@pytest.mark.parametrize("T", [1, 2, 40])
def test_ffn_graph(moe, T):
    """A captured call replayed on other tokens and routing, eager work between."""
    E, k, H, I = 16, 2, 192, 128
    stream = torch.cuda.Stream()
    c = moe.MoeCtx(0, stream)
    rng = np.random.default_rng(T)
    try:
        with torch.cuda.stream(stream):
            experts = Experts(moe, c, 6, E + 1, H, I)
            x, out = torch.zeros((T, H), dtype=BF16, device="cuda"), torch.zeros((T, H), dtype=BF16, device="cuda")
            idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
            w = torch.zeros((T, k), device="cuda")
            call = lambda o: moe.moe_expert_ffn_mx(c, experts.blocks.table, True, x, idx, w, I, o)  # noqa: E731
            idx.copy_(torch.arange(k, dtype=torch.int32).expand(T, k))
            call(out)
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call(out)
            for _ in range(4):
                x.copy_(torch.from_numpy(rng.standard_normal((T, H))))
                idx.copy_(torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)))
                w.copy_(torch.from_numpy(rng.random((T, k)).astype(np.float32)))
                out.zero_()
                g.replay()
                eager = torch.empty_like(out)
                call(eager)
                stream.synchronize()
                assert torch.equal(out, eager)
                check_ffn(out, x, idx.cpu().numpy(), w.cpu().numpy(), experts, E, True)
            c.check()
    finally:
        c.close()


def test_two_contexts_on_two_streams(moe):
    """Calls of two contexts that overlap do not meet in a workspace."""
    E, k, H, I, T = 6, 2, 512, 256, 150
    rng = np.random.default_rng(2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ctxs = [moe.MoeCtx(0, s) for s in streams]
    try:
        experts = Experts(moe, ctxs[0], 6, E, H, I)
        data = []
        for _ in range(2):
            x = torch.from_numpy(rng.standard_normal((T, H))).to(FP32).cuda()
            idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
            w = rng.random((T, k)).astype(np.float32)
            data.append((x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), torch.empty_like(x)))
        torch.cuda.synchronize()
        for _ in range(5):
            for c, (x, idx, w, out) in zip(ctxs, data):
                moe.moe_expert_ffn_mx(c, experts.blocks.table, False, x, idx, w, I, out)
        torch.cuda.synchronize()
        for c, (x, idx, w, out) in zip(ctxs, data):
            c.check()
            check_ffn(out, x, idx.cpu().numpy(), w.cpu().numpy(), experts, E, False)
    finally:
        for c in ctxs:
            c.close()


@pytest.mark.parametrize("T", [1, 3, 50])
def test_ffn_timing(moe, T):
    """With per-kernel timing on results are the same, and every launch is counted."""
    E, k, H, I = 24, 2, 128, 192
    c = moe.MoeCtx(0)
    try:
        experts = Experts(moe, c, 3, E + 1, H, I)
        rng = np.random.default_rng(T)
        x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
        idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda()
        w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
        plain, timed = torch.empty_like(x), torch.empty_like(x)
        moe.moe_expert_ffn_mx(c, experts.blocks.table, True, x, idx, w, I, plain)
        c.enable_timing(True)
        for _ in range(3):
            moe.moe_expert_ffn_mx(c, experts.blocks.table, True, x, idx, w, I, timed)
        times = c.read_timing()
        c.enable_timing(False)
        assert torch.equal(plain, timed)
        for stage in ("gateup", "down") + (("bucket", "combine") if T > 3 else ()):
            assert times[stage][1] == 3 and times[stage][0] > 0, times
    finally:
        c.close()


def test_experts_gigabytes_apart(moe):
    """The table's pointers may lie anywhere: one expert's block far from the others'."""
    E, k, H, I, T = 3, 2, 256, 128, 20
    c = moe.MoeCtx(0)
    try:
        experts = Experts(moe, c, 4, E, H, I)
        far = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
        table = experts.blocks.table.clone()
        old = table[1].cpu()
        start = int(old.min())
        at = (far.data_ptr() + far.numel() - 2 * experts.blocks.block_bytes) // 256 * 256
        views = experts.blocks.views(1)
        offsets = [int(v) - start for v in old]
        base = at - far.data_ptr()
        for v, o in zip(views, offsets):
            far[base + o:base + o + v.numel()].copy_(v.reshape(-1))
        table[1] = torch.tensor([at + o for o in offsets])
        rng = np.random.default_rng(1)
        x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
        idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        w = rng.random((T, k)).astype(np.float32)
        for n in (1, T):
            out = torch.empty_like(x[:n])
            moe.moe_expert_ffn_mx(c, table, False, x[:n], torch.from_numpy(idx[:n]).cuda(), torch.from_numpy(w[:n]).cuda(), I,
                                  out)
            check_ffn(out, x[:n], idx[:n], w[:n], experts, E, False)
        c.check()
    finally:
        c.close()
