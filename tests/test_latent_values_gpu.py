"""Expanded form: values that leave the elements' range.

A cached latent of one row is large, the heads' keys do not use it and their
values do, so that the row's keys and scores are finite and three of its values
are +-infinity or NaN once rounded to elements. Queries that do not see the row
have no part of it; those that see it get these values and no others."""
import copy

import numpy as np
import pytest

from tests.gpu_util import log
from tests.test_latent_gpu import HALF, TINY, WIDE, Problem, ctx, moe  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# (large latent, weight): finite elements whose product is beyond the type
BIG = {"fp16": (60000.0, 2.0), "bf16": (3e38, 2.0)}


def problem(seed, q, n, dims, dtype, rows):
    """rows: {sequence: positions of its broken rows}."""
    p = Problem(seed, q, n, **dims, dtype=dtype, page=16)
    big, w = BIG[dtype]
    p.w_kv[:, :, 5] = 0
    p.w_kv[:, p.dn + 3, 5] = w
    p.w_kv[:, p.dn + p.dv - 1, 5] = -w
    flat = p.cache.view(-1, p.dc + p.dr)
    flat[:, 5] = 0
    for b, at in rows.items():
        flat[p.slots(b)[at], 5] = big
    return p


def check(p, rows, moe, ctx, heads):  # noqa: F811
    """Columns 3 and dv - 1 are +inf and -inf for queries that see a broken row; all else is as without them."""
    log(f"{p.dims} {p.dtype} q {p.q_len} n {p.n} rows {rows}")
    got = p.run(moe, ctx, "expanded").double().cpu().numpy()[:, heads]
    ctx.check()
    plain = copy.copy(p)
    plain.H, plain.q, plain.w_kv, plain.cache = len(heads), p.q[:, heads], p.w_kv[heads], p.cache.clone()
    flat = plain.cache.view(-1, p.dc + p.dr)
    for b, at in rows.items():
        flat[p.slots(b)[at], 5] = 0
    ref, tol = plain.reference("expanded")
    hit = np.zeros(p.T, dtype=bool)
    for b, at in rows.items():
        hit[p.start[b]:p.start[b + 1]] = p.seen(b)[:, at].any(1)
    assert hit.any() and not hit.all()
    assert (got[hit][..., 3] == np.inf).all() and (got[hit][..., p.dv - 1] == -np.inf).all()
    rest = np.ones(got.shape, dtype=bool)
    rest[hit, :, 3] = rest[hit, :, p.dv - 1] = False
    assert np.isfinite(got[rest]).all()
    over = (np.abs(np.where(rest, got, 0) - ref) > tol) & rest
    assert not over.any(), np.argwhere(over)[:4]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dims", [TINY, dict(WIDE, H=2), dict(HALF, H=2)], ids=["tiny", "wide", "half"])
def test_infinite_values_reach_who_sees_them(moe, ctx, dims, dtype):  # noqa: F811
    for rows in ({0: [100]}, {0: [139], 2: [0]}, {0: [71, 72, 90, 131]}, {1: [5]}):
        p = problem(111, [70, 3, 1], [140, 8, 65], dims, dtype, rows)
        check(p, rows, moe, ctx, list(range(p.H)))


@pytest.mark.parametrize("dims", [dict(TINY, H=128), dict(WIDE, H=128), dict(HALF, H=128)],
                         ids=["tiny", "wide", "half"])
def test_infinite_values_in_prompts_of_many_rows(moe, ctx, dims):  # noqa: F811
    rows = {0: [257], 1: [199, 230, 462], 2: [1]}
    check(problem(112, [300, 263, 2], [300, 463, 2], dims, "fp16", rows), rows, moe, ctx, [0, 77])


def test_a_nan_among_the_values(moe, ctx):  # noqa: F811
    """A weight that is NaN makes one value of every row NaN; the other values are as they were."""
    p = Problem(113, [40], [90], **TINY, dtype="fp16")
    p.w_kv[:, p.dn + 9, 0] = float("nan")
    out = p.run(moe, ctx, "expanded").double().cpu().numpy()
    ctx.check()
    assert np.isnan(out[..., 9]).all()
    clean = copy.copy(p)
    clean.w_kv = p.w_kv.clone()
    clean.w_kv[:, p.dn + 9] = 0
    ref, tol = clean.reference("expanded")
    rest = np.arange(p.dv) != 9
    assert (np.abs(out - ref)[..., rest] <= tol[..., rest]).all()
