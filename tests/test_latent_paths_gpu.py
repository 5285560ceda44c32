"""Latent attention through the kernels and ways of sharing the work out that
only larger or uneven calls take, against the definition in 64 bits (the
tolerances are test_latent_gpu.py's). Calls of many heads are compared at some
of their heads, of different XCDs."""
import copy

import numpy as np
import pytest

from tests.gpu_util import log
from tests.latent_plan import plan
from tests.test_latent_gpu import HALF, SMALL, TINY, U, WIDE, Problem, ctx, moe, random_tree  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check(p, moe, ctx, form, heads=None, **kw):  # noqa: F811
    heads = list(range(p.H)) if heads is None else heads
    log(f"{form} {p.dims} {p.dtype} q {p.q_len[:8]} n {p.n[:8]} tree {p.tree is not None}")
    out = p.run(moe, ctx, form, **kw)
    ctx.check()
    part = copy.copy(p)
    part.H, part.q, part.w_kv = len(heads), p.q[:, heads], p.w_kv[heads]
    ref, tol = part.reference(form)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    got = got[:, heads]
    over = np.abs(got - ref) > tol
    assert not over.any(), (np.argwhere(over)[:4], np.abs(got - ref)[over][:4], tol[over][:4])
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    log(f"  relative error {rel / U[p.dtype]:.2f} u")
    assert rel <= 3 * U[p.dtype]


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# --- prompts: row tiles of 256 tokens, from ceil(T / 256) heads > CUs on -----------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dims", [dict(d, H=128, dr=dr) for d in (TINY, WIDE, HALF) for dr in (32, 64)],
                         ids=lambda d: "-".join(str(v) for v in d.values()))
def test_prompts_of_many_rows(moe, ctx, dims, dtype):  # noqa: F811
    """Whole and ragged row tiles, tiles that hold the rows before the call and the call's own, short sequences."""
    q, n = [300, 1, 0, 257, 33], [300, 70, 40, 700, 32]
    assert -(-sum(q) // 256) * dims["H"] > cus()
    check(Problem(101, q, n, **dims, dtype=dtype, page=16), moe, ctx, "expanded", heads=[0, 9, 58, 127])


def test_prompts_of_half_the_heads(moe, ctx):  # noqa: F811
    q, n = [1090, 190], [1090, 450]
    assert -(-sum(q) // 256) * 64 > cus()
    check(Problem(102, q, n, **HALF, page=64), moe, ctx, "expanded", heads=[0, 13, 63])


# --- row tiles of 64 rows ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dims", [HALF, dict(WIDE, H=33), dict(HALF, H=50, dr=32), dict(SMALL, H=64),
                                  dict(SMALL, H=40, dr=64), dict(TINY, H=48), dict(TINY, H=64, dr=64)],
                         ids=lambda d: "-".join(str(v) for v in d.values()))
def test_single_tokens_of_33_to_64_heads(moe, ctx, dims, dtype):  # noqa: F811
    n = [1, 31, 32, 33, 301, 1500, 64]
    assert plan([1] * 7, n, dims["H"], dims["dc"], cus())["rows"] == 64
    check(Problem(103, [1] * 7, n, **dims, dtype=dtype), moe, ctx, "absorbed", heads=[0, 5, 31, 32, dims["H"] - 1])


# --- even runs, each row tile charged with its start -----------------------------------

@pytest.mark.parametrize("dims, scale, max_q", [(WIDE, 1, None), (HALF, 2, None), (dict(WIDE, H=16), 2, 1),
                                                (dict(HALF, H=32), 2, 2), (dict(SMALL, H=64), 2, None),
                                                (dict(TINY, H=128), 2, None), (dict(SMALL, H=16), 5, 1)],
                         ids=["wide", "half", "wide-32", "half-64", "small", "tiny", "small-32"])
def test_even_runs_with_a_charge(moe, ctx, dims, scale, max_q):  # noqa: F811
    """More row tiles than workgroups, and much to do: runs that end in the charge, within a row tile and at its
    end; row tiles of one and of many workgroups; sequences without rows and without tokens between them."""
    q = [200 * scale, 3, 0, 60 * scale, 1, 5, 2, 1]
    n = [200 * scale + 500, 3, 77, 60 * scale + 1900, 9000, 5, 0, 33]
    if scale == 5:
        q[0], n[0] = 1000, 1200
    how = plan(q, n, dims["H"], dims["dc"], cus(), max_q)
    log(how)
    assert how["piece"] == 0 and how["over"] == 12 and how["parts"] >= 3 and how["row_tiles"] >= how["n_wg"]
    p = Problem(104, q, n, **dims, page=16)
    check(p, moe, ctx, "absorbed", heads=[0, dims["H"] // 2 + 1, dims["H"] - 1],
          **({} if max_q is None else {"max_q": max_q}))


def test_even_runs_of_trees(moe, ctx):  # noqa: F811
    rng = np.random.default_rng(7)
    q, n = [64, 40, 64, 1, 50, 64], [900, 2000, 64, 5000, 333, 700]
    how = plan(q, n, 128, 512, cus())
    assert how["piece"] == 0 and how["over"] == 12 and how["parts"] >= 3
    check(Problem(105, q, n, **WIDE, tree=random_tree(rng, q)), moe, ctx, "absorbed", heads=[0, 77, 127])


# --- the join of many partial results in a call of many row tiles -------------------------

@pytest.mark.parametrize("dims", [dict(WIDE, H=32), HALF, WIDE, SMALL, dict(SMALL, H=64), dict(SMALL, H=100),
                                  dict(TINY, H=48), dict(TINY, H=128)],
                         ids=lambda d: "-".join(str(v) for v in d.values()))
def test_one_long_sequence_among_short_ones(moe, ctx, dims):  # noqa: F811
    n = [40, 1, 20000] + [10 + 3 * i for i in range(33)]
    how = plan([1] * 36, n, dims["H"], dims["dc"], cus())
    log(how)
    # more than 16 row tiles by the call's rows, more than 16 partial results
    assert -(-36 * dims["H"] // how["rows"]) > 16 and how["parts"] > 16
    check(Problem(106, [1] * 36, n, **dims, page=16), moe, ctx, "absorbed", heads=[0, dims["H"] // 2, dims["H"] - 1])


# --- trees in the other type ---------------------------------------------------------------

@pytest.mark.parametrize("dims", [TINY, dict(HALF, H=9), HALF, dict(WIDE, H=16), SMALL],
                         ids=["tiny", "half-9", "half", "wide-16", "small"])
def test_trees_in_fp16(moe, ctx, dims):  # noqa: F811
    rng = np.random.default_rng(8)
    q, n = [3, 64, 1, 17, 0, 40], [100, 64, 1, 17 + 47, 12, 40 + 130]
    check(Problem(107, q, n, **dims, dtype="fp16", tree=random_tree(rng, q)), moe, ctx, "absorbed",
          heads=[0, dims["H"] // 2, dims["H"] - 1])


# --- workspaces of more than 2^32 bytes -------------------------------------------------------

def test_expanded_rows_beyond_32_bits(moe, ctx):  # noqa: F811
    """2^16 rows of 128 heads, 256 elements each: the last heads' rows lie past 2^32 bytes."""
    p = Problem(108, [3, 2], [68000, 50], **WIDE, page=64)
    assert sum(p.n) * p.H * (p.dn + p.dv) * 2 > 2 ** 32
    check(p, moe, ctx, "expanded", heads=[0, 126, 127])


def test_absorbed_queries_beyond_32_bits(moe, ctx):  # noqa: F811
    """131073 tokens of 128 heads ahead of the tokens that are looked at; their own sequence has no rows."""
    p = Problem(109, [5, 1], [60, 33], **dict(TINY, H=128))
    d, many = p.gpu(), 2 ** 17 + 1
    assert many * p.H * p.dc * 2 > 2 ** 32
    q = torch.zeros((many + p.T, p.H, p.dn + p.dr), dtype=d["q"].dtype, device="cuda")
    q[many:] = d["q"]
    d["q"] = q
    d["out"] = torch.full((many + p.T, p.H, p.dv), 7.0, dtype=q.dtype, device="cuda")
    d["q_start"] = torch.tensor([0, many, many + 5, many + 6], dtype=torch.int32, device="cuda")
    d["kv_len"] = torch.tensor([0, 60, 33], dtype=torch.int32, device="cuda")
    d["table"] = torch.cat([d["table"][:1], d["table"]]).contiguous()
    out = p.run(moe, ctx, "absorbed", d, max_q=many)
    ctx.check()
    assert not out[:many].any()
    heads = [0, 127]
    part = copy.copy(p)
    part.H, part.q, part.w_kv = 2, p.q[:, heads], p.w_kv[heads]
    ref, tol = part.reference("absorbed")
    got = out[many:].double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got[:, heads] - ref) <= tol).all()
