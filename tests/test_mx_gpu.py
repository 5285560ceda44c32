"""Microscaled 4-bit floating point (quantiser and back, product, product
grouped by expert, the experts' FFN) against the definition in 64 bits on the
CPU, through the public entry points. Tolerances: see mx_ref.py."""
import numpy as np
import pytest

from tests import mx_ref as ref
from tests.gpu_util import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, FP16, FP32]


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


def quantize(moe, ctx, x):
    rows, K = x.shape
    codes = torch.full((rows, K // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_mx_quantize(ctx, x, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


def check_quantized(got, x):
    codes, scales = ref.quantize(x.double().cpu().numpy())
    assert np.array_equal(got[1], scales), np.argwhere(got[1] != scales)[:4]
    assert np.array_equal(got[0], codes), np.argwhere(got[0] != codes)[:4]


# --- quantiser ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 64), (3, 96), (7, 2080), (257, 160), (5, 6144), (1, 65536), (2049, 32)])
def test_quantize(moe, ctx, dtype, rows, K):
    g = torch.Generator().manual_seed(rows * 7 + K)
    x = torch.randn((rows, K), generator=g) * torch.exp2(torch.randint(-12, 12, (rows, K // 32), generator=g)
                                                         ).repeat_interleave(32, 1)
    x = x.to(dtype).cuda()
    check_quantized(quantize(moe, ctx, x), x)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantize_every_pattern(moe, ctx, dtype):
    """Every 16-bit pattern as a block's largest value beside smaller ones, and every pattern beside a largest one."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = torch.zeros((65536, 32), dtype=dtype)
    x[:, 5] = bits
    for j, f in enumerate((1.0, 0.75, -0.5, 0.4375, 0.3125, -0.21875, 0.15625, 0.0625, 0.03125, -0.09375)):
        x[:, 10 + j] = (bits.float() * f).to(dtype)
    x = x.cuda()
    check_quantized(quantize(moe, ctx, x), x)
    y = torch.zeros((2048, 32), dtype=dtype)
    y[:] = bits.view(2048, 32)
    y[:, 0] = torch.where(y[:, 0].isfinite(), y[:, 0], torch.tensor(1.0, dtype=dtype))
    check_quantized(quantize(moe, ctx, y.cuda()), y)


def test_quantize_ends(moe, ctx):
    """Ties, zeros of both signs, the smallest and largest numbers, infinities and NaN, in fp32."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    near = torch.cat([mids, torch.nextafter(mids, torch.tensor(0.0)), torch.nextafter(mids, torch.tensor(9.0))])
    block = torch.cat([near, -near[:7], torch.tensor([7.9999995])])
    assert block.numel() == 32
    rows = [block * 2.0 ** e for e in (-127, -126, -125, -60, -3, 0, 1, 60, 124, 125)]
    rows.append(torch.zeros(32))
    rows.append(-torch.zeros(32))
    rows.append(torch.full((32,), 2.0 ** -149))
    rows.append(torch.arange(32) * 2.0 ** -149)
    rows.append(torch.full((32,), 2.0 ** -126))
    rows.append(torch.full((32,), torch.finfo(FP32).max))
    for v in (float("inf"), -float("inf"), float("nan")):
        for at in (0, 9, 31):
            r = torch.randn(32, generator=torch.Generator().manual_seed(at))
            r[at] = v
            rows.append(r)
    rows.append(torch.tensor([float("nan"), float("inf")] * 16))
    x = torch.stack(rows).cuda()
    got = quantize(moe, ctx, x)
    check_quantized(got, x)
    # a bad block leaves its neighbours alone
    y = torch.randn((2, 96), generator=torch.Generator().manual_seed(1))
    y[0, 40] = float("nan")
    check_quantized(quantize(moe, ctx, y.cuda()), y)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strided(moe, ctx, dtype):
    x = torch.randn((37, 224), generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    for view in (x[:, :96], x[:, 32:192], x[::3, 64:], x[4:5, 8:40]):
        check_quantized(quantize(moe, ctx, view), view)
    assert quantize(moe, ctx, x[:0])[0].shape == (0, 112)


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantize_every_code_and_scale(moe, ctx, dtype):
    codes = torch.arange(256, dtype=torch.uint8)[None, :].repeat(256, 1)  # a row: every byte, 16 blocks
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    out = torch.full((256, 512), 7.0, dtype=dtype, device="cuda")
    moe.moe_mx_dequantize(ctx, codes.cuda(), scales.cuda(), out)
    want = torch.from_numpy(ref.dequantize(codes.numpy(), scales.numpy())).float().to(dtype)  # exact in fp32, rounded once
    got = out.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    assert torch.equal(got[ok], want[ok])
    assert torch.equal(torch.signbit(got[ok]), torch.signbit(want[ok]))


def test_round_trip_of_values(moe, ctx):
    """What 4 bits hold comes back as it was, but for blocks whose largest code is below 4 (their scale was not the smallest)."""
    rng = np.random.default_rng(5)
    codes, scales = ref.random_matrix(rng, 64, 256)
    codes[:, ::16] |= 0x70  # a 6 in every block
    out = torch.empty((64, 256), device="cuda")
    moe.moe_mx_dequantize(ctx, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), out)
    c, s = quantize(moe, ctx, out)
    assert np.array_equal(c, codes) and np.array_equal(s, scales)


# --- product -----------------------------------------------------------------

def dev(pair):
    return [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in pair]


def product(moe, ctx, x, w, dtype):
    out = torch.full((x[0].shape[0] + 1, w[0].shape[0]), 12345.0, dtype=dtype, device="cuda")
    moe.moe_mx_matmul(ctx, *dev(x), *dev(w), out[:-1])
    torch.cuda.synchronize()
    assert (out[-1] == out.new_tensor(12345.0)).all()  # nothing behind the last row
    return out[:-1]


SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (15, 33, 128), (16, 64, 160), (17, 100, 256), (31, 5, 288), (33, 257, 512),
         (64, 130, 544), (65, 256, 1024), (100, 300, 1536), (129, 513, 416), (257, 255, 768), (300, 1000, 2048),
         (1, 4097, 6144), (3, 640, 16384), (40, 96, 6176), (513, 770, 288), (24, 129, 2560), (60, 200, 4096), (20, 2000, 512),
         (31, 700, 1504), (257, 300, 4096)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(moe, ctx, M, N, K):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    x, w = ref.random_matrix(rng, M, K), ref.random_matrix(rng, N, K, lo=110, hi=122)
    for dtype in TYPES:
        ref.check_product(product(moe, ctx, x, w, dtype), ref.dequantize(*x), ref.dequantize(*w), (M, N, K, dtype))


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (20, 40, 352), (200, 300, 800)])
def test_product_bad_blocks(moe, ctx, M, N, K):
    """A block of NaN spoils its row's results and no others; scales of all sizes."""
    rng = np.random.default_rng(M)
    x, w = ref.random_matrix(rng, M, K, lo=100, hi=150), ref.random_matrix(rng, N, K, lo=90, hi=140)
    x[1][M // 2, K // 32 - 1] = 255
    w[1][N - 1, 0] = 255
    w[1][N // 3, K // 64] = 255
    got = product(moe, ctx, x, w, FP32)
    ref.check_product(got, ref.dequantize(*x), ref.dequantize(*w))
    assert int(got.isnan().sum()) > 0
    if M > 1:
        assert not got[0].isnan().all()


def test_product_small_and_large_scales(moe, ctx):
    rng = np.random.default_rng(8)
    for lo, hi, wlo, whi in ((0, 2, 125, 129), (250, 254, 1, 4), (60, 70, 60, 66)):
        x, w = ref.random_matrix(rng, 40, 192, lo=lo, hi=hi), ref.random_matrix(rng, 50, 192, lo=wlo, hi=whi)
        ref.check_product(product(moe, ctx, x, w, FP32), ref.dequantize(*x), ref.dequantize(*w), (lo, wlo))


@pytest.mark.parametrize("M,N,K", [(5, 64, 512), (40, 200, 512), (200, 300, 1024), (300, 300, 128)])
def test_product_unaligned_scales(moe, ctx, M, N, K):
    """Scales at any address (a matrix of a stack, for instance)."""
    rng = np.random.default_rng(K)
    x, w = ref.random_matrix(rng, M, K), ref.random_matrix(rng, N, K)
    for ax, aw in ((1, 0), (0, 3), (4, 8)):
        sx = torch.empty(ax + x[1].size, dtype=torch.uint8, device="cuda")[ax:].view(M, -1)
        sw = torch.empty(aw + w[1].size, dtype=torch.uint8, device="cuda")[aw:].view(N, -1)
        sx.copy_(torch.from_numpy(x[1]))
        sw.copy_(torch.from_numpy(w[1]))
        out = torch.empty((M, N), device="cuda")
        moe.moe_mx_matmul(ctx, torch.from_numpy(x[0]).cuda(), sx, torch.from_numpy(w[0]).cuda(), sw, out)
        ref.check_product(out, ref.dequantize(*x), ref.dequantize(*w), (M, ax, aw))


def test_product_nothing(moe, ctx):
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    out = torch.full((0, 8), 1.0, device="cuda")
    moe.moe_mx_matmul(ctx, e(0, 32), e(0, 2), e(8, 32), e(8, 2), out)
    moe.moe_mx_matmul(ctx, e(4, 32), e(4, 2), e(0, 32), e(0, 2), torch.empty((4, 0), device="cuda"))


# --- grouped -----------------------------------------------------------------

def grouped(moe, ctx, x, w, counts, dtype, in_rows=None, out_rows=None, rows=None, first=0):
    offsets = first + np.concatenate([[0], np.cumsum(counts)])
    L = int(offsets[-1]) + 3 if in_rows is None and out_rows is None else len(out_rows if in_rows is None else in_rows)
    R = rows or L
    out = torch.full((R, w[0].shape[1]), 12345.0, dtype=dtype, device="cuda")
    i32 = lambda v: None if v is None else torch.from_numpy(np.asarray(v, dtype=np.int32)).cuda()  # noqa: E731
    moe.moe_mx_grouped_matmul(ctx, *dev(x), *dev(w), i32(offsets), out, in_rows=i32(in_rows), out_rows=i32(out_rows))
    torch.cuda.synchronize()
    xv, wv = ref.dequantize(*x), ref.dequantize(*w)
    left = np.ones(R, dtype=bool)
    for e in range(len(counts)):
        lines = np.arange(offsets[e], offsets[e + 1])
        if len(lines) == 0:
            continue
        src = lines if in_rows is None else np.asarray(in_rows)[lines]
        dst = lines if out_rows is None else np.asarray(out_rows)[lines]
        ref.check_product(out[torch.from_numpy(dst).cuda()], xv[src], wv[e], (e, len(lines)))
        left[dst] = False
    assert (out[torch.from_numpy(left).cuda()] == out.new_tensor(12345.0)).all()


COUNTS = [[1], [0, 5, 0, 0, 17, 1], [0, 0], [16, 16, 0, 32], [3] * 70, [200, 0, 1, 64, 65, 130, 2, 0], [0] * 200 + [7] + [0] * 55,
          [1] * 256, [700, 3]]


@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("N,K", [(96, 128), (130, 352), (200, 1536), (257, 512)])
def test_grouped(moe, ctx, i, N, K):
    counts = COUNTS[i]
    rng = np.random.default_rng(i)
    L = int(sum(counts))
    w = ref.random_matrix(rng, len(counts), N, K, lo=112, hi=122)
    for dtype, gather, scatter in ((FP32, False, False), (BF16, True, False), (FP16, True, True), (BF16, False, True)):
        X = 11 if gather else L + 3
        x = ref.random_matrix(rng, X, K)
        in_rows = rng.integers(0, X, L) if gather else None
        out_rows = rng.permutation(L + 5)[:L] if scatter else None
        grouped(moe, ctx, x, w, counts, dtype, in_rows, out_rows, L + 5 if scatter or gather else L + 3)


def test_grouped_from_line_three(moe, ctx):
    """Lines before the first expert's and behind the last one's are left as they were."""
    rng = np.random.default_rng(2)
    x, w = ref.random_matrix(rng, 40, 64), ref.random_matrix(rng, 3, 48, 64)
    grouped(moe, ctx, x, w, [5, 0, 20], BF16, first=3)


def test_grouped_bad_rows(moe, ctx):
    """Rows and offsets out of range: reported, nothing out of range read or written, other lines right."""
    rng = np.random.default_rng(4)
    x, w = ref.random_matrix(rng, 8, 96), ref.random_matrix(rng, 2, 32, 96)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    xd, wd = dev(x), dev(w)
    want = ref.dequantize(*x)
    out = torch.full((8, 32), 5.0, device="cuda")
    moe.moe_mx_grouped_matmul(ctx, *xd, *wd, i32([0, 4, 6]), out, in_rows=i32([0, 8, 2, -1, 7, 5]),
                              out_rows=i32([1, 2, 3, 4, 2 ** 30, 6]))
    with pytest.raises(moe.MoeError):
        ctx.check()
    ctx.check()
    got = out.cpu()
    for line, r in ((0, 1), (2, 3)):
        ref.check_product(out[r:r + 1], want[[0, 0, 2][line]][None], ref.dequantize(w[0][0], w[1][0]))
    ref.check_product(out[6:7], want[5][None], ref.dequantize(w[0][1], w[1][1]))
    assert (got[[0, 2, 4, 5, 7]] == 5.0).all()
    for offsets in ([0, 5, 3], [-7, 2, 4], [0, 3, 2 ** 30], [2 ** 30, 2 ** 30 + 1, 2 ** 30 + 2]):
        moe.moe_mx_grouped_matmul(ctx, *xd, *wd, i32(offsets), torch.empty((8, 32), device="cuda"))
        with pytest.raises(moe.MoeError):
            ctx.check()


def test_graph_replay(moe, ctx):
    """A captured call replayed on other offsets, rows and values, with eager work between."""
    rng = np.random.default_rng(6)
    E, N, K, L = 6, 160, 256, 50
    w = ref.random_matrix(rng, E, N, K)
    stream = torch.cuda.Stream()
    c = moe.MoeCtx(0, stream)
    try:
        with torch.cuda.stream(stream):
            x = dev(ref.random_matrix(rng, 20, K))
            wd = dev(w)
            offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
            in_rows = torch.zeros(L, dtype=torch.int32, device="cuda")
            out = torch.zeros((L, N), device="cuda")
            moe.moe_mx_grouped_matmul(c, *x, *wd, offsets, out, in_rows=in_rows)
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                moe.moe_mx_grouped_matmul(c, *x, *wd, offsets, out, in_rows=in_rows)
            for _ in range(4):
                counts = rng.multinomial(rng.integers(1, L + 1), np.ones(E) / E)
                rows = rng.integers(0, 20, L)
                xn = ref.random_matrix(rng, 20, K)
                for t, v in zip((*x, offsets, in_rows), (*xn, np.concatenate([[0], np.cumsum(counts)]), rows)):
                    t.copy_(torch.from_numpy(v.astype(np.int32) if v.dtype == np.int64 else v))
                out.zero_()
                g.replay()
                eager = torch.zeros_like(out)
                moe.moe_mx_grouped_matmul(c, *x, *wd, offsets, eager, in_rows=in_rows)
                stream.synchronize()
                assert torch.equal(out, eager)
                n = int(counts.sum())
                e = np.repeat(np.arange(E), counts)
                xv, wv = ref.dequantize(*xn), ref.dequantize(*w)
                for l in (0, n - 1):
                    ref.check_product(out[l:l + 1], xv[rows[l]][None], wv[e[l]])
                assert (out[n:] == 0).all()
    finally:
        c.close()


# --- the experts' FFN ----------------------------------------------------------

class Experts:
    def __init__(self, moe, ctx, seed, n, H, I):
        rng = np.random.default_rng(seed)
        self.blocks = moe.MxExpertBlocks(n, H, I)
        self.values = []
        for e in range(n):
            m = [rng.standard_normal(s) * s[1] ** -0.5 for s in ((I, H), (I, H), (H, I))]
            self.blocks.pack_from_fp32(ctx, e, *[torch.from_numpy(v).float().cuda() for v in m])
        torch.cuda.synchronize()
        for e in range(n):
            v = [t.cpu().numpy() for t in self.blocks.views(e)]
            self.values.append([ref.dequantize(v[i], v[3 + i]) for i in range(3)])


def check_ffn(out, x, idx, w, experts, E, shared):
    """Slots' tolerances are added up with their weights; a bf16 call rounds each slot's result, all round the sum."""
    u = ref.U[out.dtype]
    xv = ref.dequantize(*ref.quantize(x.double().cpu().numpy()))
    T = x.shape[0]
    want, tol, mass = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    pairs = [(e, *np.nonzero(idx == e)) for e in range(E)]
    if shared:
        pairs.append((E, np.arange(T), None))
    for e, t, j in pairs:
        if len(t) == 0:
            continue
        y, ty = ref.ffn(xv[t], *experts.values[e])
        f = np.ones((len(t), 1)) if j is None else w[t, j].astype(np.float64)[:, None]
        np.add.at(want, t, f * y)
        np.add.at(tol, t, np.abs(f) * (ty + (u * np.abs(y) if out.dtype == BF16 else 0)))
        np.add.at(mass, t, np.abs(f * y))
    tol = (tol + 20 * 2.0 ** -24 * mass) * 1.01 + u * np.abs(want) * 1.01 + 2.0 ** -24 * (out.dtype == FP16)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float((np.abs(got - want) / tol).max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,E,H,I,shared", [(1, 2, 8, 128, 64, True), (1, 8, 64, 320, 192, False), (2, 1, 1, 64, 64, True),
                                              (3, 4, 16, 192, 448, True), (33, 2, 5, 256, 128, True),
                                              (70, 3, 9, 448, 320, False), (300, 2, 4, 128, 576, True),
                                              (6, 2, 7, 512, 1024, True), (130, 2, 3, 1536, 512, True),
                                              (700, 2, 3, 512, 512, False), (900, 1, 2, 192, 320, True),
                                              (1, 4, 6, 512, 1536, True), (1, 1, 3, 8192, 64, False),
                                              (1, 16, 20, 64, 8192, True), (2, 2, 16, 1024, 512, True),
                                              (3, 1, 12, 192, 1088, False), (2, 3, 24, 8128, 128, True)])
def test_ffn(moe, ctx, dtype, T, k, E, H, I, shared):
    rng = np.random.default_rng(T + k + E)
    experts = Experts(moe, ctx, T, E + int(shared), H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).cuda()
    idx = np.argsort(rng.random((T, E)) + 0.3 * np.arange(E), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    if T > 2:
        idx[1, -1], w[1, -1] = -1, 0  # a dropped slot
        w[2, 0] = 0
    out = torch.full_like(x, 9.0)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, shared, x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), I,
                          out)
    ctx.check()
    check_ffn(out, x, idx, w, experts, E, shared)


@pytest.mark.parametrize("T,E", [(1, 6), (5, 6), (2, 40)])
def test_ffn_bad_ids(moe, ctx, T, E):
    """An id out of range and a repeated one add nothing and are reported."""
    k, H, I = 4, 128, 128
    experts = Experts(moe, ctx, 1, E + 1, H, I)
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((T, H))).float().cuda()
    w = rng.random((T, k)).astype(np.float32)
    for bad in ([3, E, -5, 0], [2, 2, 1, 2], [-1, -1, -1, -1], [5, -1, 5, -1], [2 ** 31 - 1, -2 ** 31, 1, 1]):
        idx = np.tile(np.array([0, 1, 2, 3], dtype=np.int32), (T, 1))
        idx[T - 1] = bad
        out = torch.empty_like(x)
        moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, x, torch.from_numpy(idx).cuda(),
                              torch.from_numpy(w).cuda(), I, out)
        if bad[0] != -1:
            with pytest.raises(moe.MoeError):
                ctx.check()
        ctx.check()
        used = idx.copy()
        for j in range(k):
            if not 0 <= bad[j] < E or bad[j] in bad[:j]:
                used[T - 1, j] = -1
        check_ffn(out, x, used, w, experts, E, True)


def test_ffn_of_nan(moe, ctx):
    """A token that holds NaN gets NaN; the others are as without it."""
    E, k, H, I, T = 4, 2, 128, 64, 40
    experts = Experts(moe, ctx, 9, E, H, I)
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda()
    clean, out = torch.empty_like(x), torch.empty_like(x)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, False, x, idx, w, I, clean)
    x[7, 70] = float("nan")
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, False, x, idx, w, I, out)
    ctx.check()
    assert out[7].isnan().all()
    keep = torch.arange(T, device="cuda") != 7
    assert torch.equal(out[keep], clean[keep])


# --- refusals ------------------------------------------------------------------

def test_refusals(moe, ctx):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    f = lambda *s, t=FP32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bad = (TypeError, ValueError, moe.MoeError)
    calls = [
        lambda: moe.moe_mx_quantize(ctx, f(4, 48), u8(4, 24), u8(4, 1)),  # no whole blocks
        lambda: moe.moe_mx_quantize(ctx, f(4, 64, t=torch.float64), u8(4, 32), u8(4, 2)),
        lambda: moe.moe_mx_quantize(ctx, f(64, 4).t(), u8(4, 32), u8(4, 2)),  # columns strided
        lambda: moe.moe_mx_quantize(ctx, f(4, 66)[:, :64], u8(4, 32), u8(4, 2)),  # row stride no multiple of 4
        lambda: moe.moe_mx_quantize(ctx, f(4, 68)[:, 1:65], u8(4, 32), u8(4, 2)),  # address not aligned
        lambda: moe.moe_mx_quantize(ctx, f(4, 64).cpu(), u8(4, 32), u8(4, 2)),
        lambda: moe.moe_mx_quantize(ctx, f(4, 64), u8(4, 32), u8(4, 1)),
        lambda: moe.moe_mx_quantize(ctx, f(1, 65568), u8(1, 32784), u8(1, 2049)),  # K too large
        lambda: moe.moe_mx_quantize(ctx, f(64), u8(32), u8(2)),
        lambda: moe.moe_mx_dequantize(ctx, u8(4, 32), u8(4, 2), f(4, 32)),
        lambda: moe.moe_mx_dequantize(ctx, u8(4, 24), u8(4, 1), f(4, 48)),
        lambda: moe.moe_mx_dequantize(ctx, u8(4, 32), u8(4, 2), torch.zeros((4, 64), dtype=torch.int32, device="cuda")),
        lambda: moe.moe_mx_matmul(ctx, u8(4, 32), u8(4, 2), u8(8, 48), u8(8, 3), f(4, 8)),  # K differ
        lambda: moe.moe_mx_matmul(ctx, u8(4, 32), u8(4, 2), u8(8, 32), u8(8, 2), f(8, 4).t()),
        lambda: moe.moe_mx_matmul(ctx, u8(4, 32), u8(4, 1), u8(8, 32), u8(8, 2), f(4, 8)),
        lambda: moe.moe_mx_matmul(ctx, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), f(4, 8)),
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), i32(2), f(4, 8)),
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), i32(3), f(4, 8),
                                          in_rows=i32(4), out_rows=i32(3)),
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), i32(3), f(4, 8),
                                          in_rows=i32(6)),  # out has too few rows
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(4, 32), u8(4, 2), u8(2, 8, 32), u8(2, 8, 2), i32(3), f(9, 8),
                                          out_rows=i32(6)),  # x has too few rows
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(0, 32), u8(0, 2), u8(2, 8, 32), u8(2, 8, 2), i32(3), f(4, 8),
                                          in_rows=i32(4)),  # lines of no row
        lambda: moe.moe_mx_grouped_matmul(ctx, u8(4, 32), u8(4, 2), u8(1025, 1, 32), u8(1025, 1, 2), i32(1026), f(4, 1)),
        lambda: moe.moe_mx_expert_layout(96, 64),
        lambda: moe.MxExpertBlocks(1, 64, 32),
    ]
    table = torch.zeros((3, 6), dtype=torch.int64, device="cuda")
    ffn = lambda x, idx, w, I, out, t=table, sh=True: moe.moe_expert_ffn_mx(ctx, t, sh, x, idx, w, I, out)  # noqa: E731
    same = f(2, 64)
    calls += [
        lambda: ffn(f(2, 96), i32(2, 2), f(2, 2), 64, f(2, 96)),
        lambda: ffn(f(2, 64), i32(2, 2), f(2, 2), 96, f(2, 64)),
        lambda: ffn(f(2, 64), i32(2, 3), f(2, 3), 64, f(2, 64)),  # k above E
        lambda: ffn(f(2, 64), i32(2, 2), f(2, 2), 64, f(2, 64, t=BF16)),
        lambda: ffn(f(2, 64), i32(2, 2), f(1, 2), 64, f(2, 64)),
        lambda: ffn(f(2, 64), i32(3, 2), f(3, 2), 64, f(2, 64)),
        lambda: ffn(f(2, 64), i32(2, 2), f(2, 2), 64, f(2, 64), t=table[:1]),
        lambda: ffn(f(2, 64, t=torch.float64), i32(2, 2), f(2, 2), 64, f(2, 64, t=torch.float64)),
        lambda: ffn(same, i32(2, 2), f(2, 2), 64, same),
        lambda: ffn(f(2, 8256), i32(2, 2), f(2, 2), 64, f(2, 8256)),
    ]
    for i, call in enumerate(calls):
        log("refusal", i)
        with pytest.raises(bad):
            call()
    assert ffn(f(0, 64), i32(0, 2), f(0, 2), 64, f(0, 64)).shape == (0, 64)
    ctx.check()


@pytest.mark.parametrize("T,k,E", [(4097, 8, 9), (2050, 16, 300), (1000, 5, 1024), (64, 7, 7)])
def test_ffn_bucketing(moe, ctx, T, k, E):
    """Many entries (one workgroup's and more than that), odd numbers of slots, dropped ones among them."""
    H, I = 64, 64
    rng = np.random.default_rng(k)
    experts = Experts(moe, ctx, 5, E, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < 0.1] = -1
    w = np.where(idx < 0, 0, rng.random((T, k))).astype(np.float32)
    out = torch.empty_like(x)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, False, x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), I,
                          out)
    ctx.check()
    check_ffn(out, x, idx, w, experts, E, False)


# --- more tiles than workgroups ---------------------------------------------------

@pytest.mark.parametrize("M,N,K,at", [(2100, 9000, 64, 0), (2100, 9000, 96, 1), (3, 50000, 128, 0), (20, 100000, 512, 0),
                                      (700, 20000, 512, 0), (1000, 9100, 1056, 0)])
def test_product_of_many_tiles(moe, ctx, M, N, K, at):
    """Workgroups take several tiles each, of few stages and of more."""
    rng = np.random.default_rng(M + K)
    x, w = ref.random_matrix(rng, M, K), ref.random_matrix(rng, N, K, lo=112, hi=122)
    sw = torch.empty(at + w[1].size, dtype=torch.uint8, device="cuda")[at:].view(N, -1)
    sw.copy_(torch.from_numpy(w[1]))
    out = torch.full((M + 1, N), 12345.0, device="cuda")
    moe.moe_mx_matmul(ctx, *dev(x), torch.from_numpy(w[0]).cuda(), sw, out[:-1])
    ref.check_product(out[:-1], ref.dequantize(*x), ref.dequantize(*w), (M, N, K))
    assert (out[-1] == 12345.0).all()


@pytest.mark.parametrize("E,N,K,most", [(300, 1100, 96, 9), (300, 600, 512, 40), (64, 2100, 64, 300), (40, 2100, 512, 900)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_grouped_of_many_tiles(moe, ctx, E, N, K, most, dtype):
    """Tiles without lines before, between and behind those that a workgroup computes; lines gathered and scattered."""
    rng = np.random.default_rng(E + most)
    counts = np.where(rng.random(E) < 0.4, 0, rng.integers(0, most, E))
    counts[:E // 8] = 0
    counts[-E // 8:] = 0
    L = int(counts.sum())
    x, w = ref.random_matrix(rng, 37, K), ref.random_matrix(rng, E, N, K, lo=112, hi=122)
    grouped(moe, ctx, x, w, counts, dtype, rng.integers(0, 37, L), rng.permutation(L + 9)[:L], L + 9)


@pytest.mark.parametrize("T,k,E,H,I", [(40, 8, 100, 64, 2048), (40, 8, 50, 512, 1024), (700, 4, 20, 192, 1600),
                                       (900, 4, 12, 512, 2560)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ffn_of_many_tiles(moe, ctx, T, k, E, H, I, dtype):
    rng = np.random.default_rng(T + E)
    experts = Experts(moe, ctx, E, E + 1, H, I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).cuda()
    idx = np.argsort(rng.random((T, E)) + 0.02 * np.arange(E), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    out = torch.full_like(x, 9.0)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), I, out)
    ctx.check()
    check_ffn(out, x, idx, w, experts, E, True)


# --- offsets beyond 32 bits ---------------------------------------------------------

def test_quantize_far(moe, ctx):
    """More than 2^31 values and 2^32 bytes, there and back, and a row stride that passes 2^32 bytes within a few rows."""
    rows, K = (1 << 21) + 5, 1056
    x = torch.empty((rows, K), device="cuda").normal_()
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    moe.moe_mx_quantize(ctx, x, codes, scales)
    out = torch.empty((rows, K), dtype=BF16, device="cuda")
    moe.moe_mx_dequantize(ctx, codes, scales, out)
    for r in (0, (1 << 29) // K, (1 << 30) // K, (1 << 31) // K, rows - 3):
        part = slice(r, r + 3)
        check_quantized((codes[part].cpu().numpy(), scales[part].cpu().numpy()), x[part])
        want = ref.dequantize(codes[part].cpu().numpy(), scales[part].cpu().numpy())
        assert np.array_equal(out[part].double().cpu().numpy(), want)  # 4 bits' values are bf16's too
    del x, out
    y = torch.empty((50, 1 << 26), dtype=BF16, device="cuda")[:, 64:160]
    y.copy_(torch.randn((50, 96), generator=torch.Generator().manual_seed(2)))
    check_quantized(quantize(moe, ctx, y), y)


def test_grouped_far(moe, ctx):
    """Rows of x, weights and out beyond 2^32 bytes."""
    E, N, K, X, R = 600, 2048, 8192, 1_100_000, 600_000
    rand = lambda lo, hi, *s: torch.randint(lo, hi, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    w, sw = rand(0, 256, E, N, K // 2), rand(112, 122, E, N, K // 32)
    x, sx = rand(0, 256, X, K // 2), rand(118, 130, X, K // 32)
    assert min(w.numel(), x.numel(), R * N * 4) > 1 << 32
    i32 = lambda v: torch.from_numpy(np.asarray(v, dtype=np.int32)).cuda()  # noqa: E731
    rng = np.random.default_rng(0)
    for lines in ((0, 0, 1), (1, 20, 7), (60, 0, 300)):
        counts = np.zeros(E, dtype=np.int64)
        counts[[0, E - 2, E - 1]] = lines
        L = int(counts.sum())
        in_rows, out_rows = X - 1 - rng.permutation(1000)[:L], R - 1 - rng.permutation(1000)[:L]
        in_rows[0], out_rows[-1] = X - 1, R - 1
        out_rows[:-1] = R - 2 - rng.permutation(1000)[:L - 1]
        out = torch.full((R, N), 12345.0, device="cuda")
        moe.moe_mx_grouped_matmul(ctx, x, sx, w, sw, i32(np.concatenate([[0], np.cumsum(counts)])), out, in_rows=i32(in_rows),
                                  out_rows=i32(out_rows))
        ctx.check()
        first = 0
        for e in np.flatnonzero(counts):
            l = slice(first, first + int(counts[e]))
            src, dst = torch.from_numpy(in_rows[l]).cuda(), torch.from_numpy(out_rows[l]).cuda()
            ref.check_product(out[dst], ref.dequantize(x[src].cpu().numpy(), sx[src].cpu().numpy()),
                              ref.dequantize(w[e].cpu().numpy(), sw[e].cpu().numpy()), (lines, e))
            out[dst] = 12345.0
            first = l.stop
        assert (out == 12345.0).all()


# --- ends of the ranges, NaN where nothing may come from it ------------------------------

@pytest.mark.parametrize("M,N", [(2, 70), (70, 130), (300, 257)])
def test_product_of_longest_rows(moe, ctx, M, N):
    rng = np.random.default_rng(M)
    x, w = ref.random_matrix(rng, M, 65536), ref.random_matrix(rng, N, 65536, lo=112, hi=122)
    ref.check_product(product(moe, ctx, x, w, FP32), ref.dequantize(*x), ref.dequantize(*w), (M, N))


@pytest.mark.parametrize("T", [1, 2, 3, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ffn_of_bad_token_and_unused_bad_expert(moe, ctx, T, bad):
    """A token that holds NaN or an infinity gets NaN, others what they get without it; an expert of NaN that has
    weight 0 adds nothing."""
    E, k, H, I = 40, 3, 192, 128
    experts = Experts(moe, ctx, 11, E + 1, H, I)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(BF16).cuda()
    idx = np.argsort(rng.random((T, E - 1)), axis=1)[:, :k].astype(np.int32)
    idx[:, 1] = E - 1
    w = rng.random((T, k)).astype(np.float32)
    w[:, 1] = 0
    for v in experts.blocks.views(E - 1)[3:]:
        v.fill_(255)
    args = (torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), I)
    out = torch.empty_like(x)
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, x, *args, out)
    ctx.check()
    check_ffn(out, x, np.where(idx == E - 1, -1, idx), w, experts, E, True)
    spoiled, y = torch.empty_like(x), x.clone()
    y[T - 1, H - 1] = bad
    moe.moe_expert_ffn_mx(ctx, experts.blocks.table, True, y, *args, spoiled)
    assert spoiled[T - 1].isnan().all()
    assert torch.equal(spoiled[:T - 1], out[:T - 1])
