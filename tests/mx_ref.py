"""Microscaled 4-bit floating point in 64 bits on the CPU: the definition that
the GPU's results are compared with."""
import numpy as np
import torch

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative


def quantize(x):
    """codes [rows][K / 2] and scale bytes [rows][K / 32] of x (float64 numpy [rows][K])."""
    b = x.reshape(x.shape[0], -1, 32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(b).max(axis=2)
        bad = ~np.isfinite(b).all(axis=2)
        e = np.where(top > 0, np.frexp(np.where(bad, 1.0, top))[1] - 1, -999) - 2
        byte = np.where(bad, 255, np.maximum(e, -127) + 127).astype(np.uint8)
        v = np.where(bad[..., None], 0.0, b) / np.where(bad, 1.0, 2.0 ** (np.maximum(e, -127)))[..., None]
    a = np.minimum(np.abs(v), 6.0)
    # the nearest of the grid; of two as near the even code
    d = np.abs(a[..., None] - GRID)
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(bad[..., None], 0, code | (np.signbit(v).astype(np.int64) << 3)).reshape(x.shape)
    return (code[:, 0::2] | code[:, 1::2] << 4).astype(np.uint8), byte


def scale_of(byte):
    return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def dequantize(codes, scales):
    """Values (float64) of codes [..., K / 2] and scales [..., K / 32]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    return v * np.repeat(scale_of(scales), 32, axis=-1)


def random_matrix(rng, *shape, lo=118, hi=130):
    """Codes and scales of a matrix [..., K]: any code, scale bytes lo .. hi."""
    K = shape[-1]
    return (rng.integers(0, 256, (*shape[:-1], K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*shape[:-1], K // 32), dtype=np.uint8))


def check_product(got, x, w, what=""):
    """got (tensor [M][N]) against x w^T of float64 matrices.

    Products of codes are exact and a matrix instruction adds 64 or 128 of them to an
    fp32 sum; however it rounds inside, no sum is off by more than 2^-23 of the sum of
    absolute terms, and there are at most K / 64 + 16 of them (partial sums of up to 16
    waves are added at the end). The result is rounded once more. All elements together
    (2-norm): roundings are independent, and below a sixth of the worst case's square
    root for each: u + 2^-23 sqrt(K / 64 + 16) of the root of the sum of squared terms."""
    u = U[got.dtype]
    want, mass = x @ w.T, np.abs(x) @ np.abs(w).T
    n = x.shape[1] / 64 + 16
    g = got.double().cpu().numpy()
    top = 65504.0 * (1 + 2.0 ** -12) if got.dtype == torch.float16 else np.inf
    fits = np.abs(want) < top * (1 - 2.0 ** -11)
    assert np.array_equal(np.isnan(g), np.isnan(want)), what
    ok = fits & ~np.isnan(want)
    tol = n * 2.0 ** -23 * mass + u * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -24 * (got.dtype == torch.float16)
    bad = np.abs(g - want)[ok] > tol[ok]
    assert not bad.any(), (what, int(bad.sum()), np.argwhere((np.abs(g - want) > tol) & ok)[:4].tolist())
    if ok.sum() > 1000:
        norm = np.sqrt((want[ok] ** 2).sum())
        wide = np.sqrt(((x ** 2) @ (w ** 2).T)[ok].sum())
        assert np.sqrt(((g - want)[ok] ** 2).sum()) <= u * norm + 2.0 ** -23 * np.sqrt(n) * wide, what


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def ffn(x, gate, up, down):
    """One expert's FFN of rows x (float64, already 4-bit values): (y, tolerance).

    gate, up, down: float64 values. The GPU's a = silu(g) u is off by what its fp32
    sums are off (2^-23 of the sums' absolute terms for each of K / 64 + 16 roundings),
    times silu's slope (below 1.1) or the other factor, and 2^-20 of its own size for
    exp, division and product. Where that may turn a code (or, for the whole block, its
    scale), the result may move by the step between codes times down's element; and
    down's own sums round as above."""
    H, I = x.shape[1], gate.shape[0]
    g, u = x @ gate.T, x @ up.T
    n = H / 64 + 16
    dg, du = (n * 2.0 ** -23 * (np.abs(x) @ np.abs(m).T) for m in (gate, up))
    a = silu(g) * u
    da = 1.1 * dg * np.abs(u) + (np.abs(g) + dg) * du + 2.0 ** -20 * np.abs(a) + 2.0 ** -126
    codes, scales = quantize(a)
    q = dequantize(codes, scales)
    rows = x.shape[0]
    s = np.repeat(scale_of(scales), 32, axis=1)
    v, dv = np.abs(a) / s, da / s
    mid = (GRID[1:] + GRID[:-1]) / 2
    turn = (np.abs(v[..., None] - mid) <= dv[..., None]).any(-1)
    step = np.where(turn, 2.0 * s, 0.0)  # the widest step between codes
    top = np.abs(a).reshape(rows, -1, 32).max(axis=2)
    dtop = da.reshape(rows, -1, 32).max(axis=2)
    below, above = np.frexp(top - dtop)[1], np.frexp(top + dtop)[1]
    step = np.maximum(step, np.repeat((below != above) * 4.0 * scale_of(scales), 32, axis=1))
    tol = step @ np.abs(down).T + (I / 64 + 16) * 2.0 ** -23 * (np.abs(q) @ np.abs(down).T)
    return q @ down.T, tol
