"""Latent attention (the cache's writer, the absorbed form for single tokens
and drafted trees, the expanded form for prompts) against the definition in
64 bits on the CPU, through the public entry points.

Tolerances. u is the elements' unit roundoff (bf16 2^-8, fp16 2^-11). Both
forms round four things on the way to an output: what the scores are made of
(the absorbed query, or the expanded keys: a relative u on every product of a
score), the softmax weights (u), what the last product takes (u) and the
output (u).
 - Element by element, in the worst case: a score is off by at most ds = u
   scale sum |products|, so a weight by a factor within e^(2 ds), and the
   result by at most (e^(2 max ds) (1 + u)^2 - 1) times the sum of absolute
   terms, plus u of the result; fp32 sums of up to 2^17 terms add less than
   2^-10 of that and are covered by the factor 1.05.
 - Over all elements (2-norm): the four roundings are independent with a rms
   below u / sqrt(3) of what they round, the scores' rms is at most 1.5 in
   these inputs, so the expected relative error is u sqrt((1.5^2 + 3) / 3) <
   1.4 u; 3 u is accepted.
"""
import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
WIDE = dict(H=128, dc=512, dr=64, dn=128, dv=128)
HALF = dict(H=64, dc=512, dr=64, dn=192, dv=256)
SMALL = dict(H=16, dc=256, dr=32, dn=64, dv=64)
TINY = dict(H=5, dc=128, dr=32, dn=64, dv=64)


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


def tdtype(name):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


class Problem:
    """Inputs on the GPU and, in 64 bits, on the CPU."""

    def __init__(self, seed, q, n, H, dc, dr, dn, dv, dtype="bf16", page=16, tree=None, scale=None, spare=2,
                 q_std=1.0, poison=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.q_len, self.n = list(q), list(n)
        self.dims = dict(H=H, dc=dc, dr=dr, dn=dn, dv=dv)
        self.dtype, self.page = dtype, page
        self.H, self.dc, self.dr, self.dn, self.dv = H, dc, dr, dn, dv
        t = tdtype(dtype)
        B, T = len(q), int(sum(q))
        self.B, self.T = B, T
        pages = [-(-x // page) for x in n]
        n_pages = sum(pages) + spare
        ids = rng.permutation(n_pages)
        self.table = np.full((B, max(pages + [1])), 2 ** 30, dtype=np.int32)  # entries behind a sequence: never read
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = ids[at:at + pages[b]]
            at += pages[b]
        self.cache = torch.randn((n_pages, page, dc + dr), generator=g).to(t)
        self.q = (torch.randn((T, H, dn + dr), generator=g) * q_std).to(t)
        self.w_kv = (torch.randn((H, dn + dv, dc), generator=g) * dc ** -0.5).to(t)
        self.start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.tree = tree
        self.scale = float((dn + dr) ** -0.5 if scale is None else scale)
        if poison is not None:
            self.poison(poison)

    def slots(self, b):
        j = np.arange(self.n[b])
        return torch.from_numpy(self.table[b, j // self.page].astype(np.int64) * self.page + j % self.page)

    def poison(self, value):
        """Every cache row that no sequence holds becomes `value`."""
        flat = self.cache.view(-1, self.dc + self.dr)
        used = torch.zeros(flat.shape[0], dtype=torch.bool)
        for b in range(self.B):
            used[self.slots(b)] = True
        flat[~used] = value

    def seen(self, b):
        nq, n = self.q_len[b], self.n[b]
        before = n - nq
        j = np.arange(n)
        s = np.zeros((nq, n), dtype=bool)
        for i in range(nq):
            if self.tree is None:
                s[i] = j <= before + i
            else:
                word = int(self.tree[self.start[b] + i]) & (2 ** 64 - 1)
                for jj in range(n):
                    r = jj - before
                    s[i, jj] = r < 0 or (r < 64 and bool((word >> r) & 1))
        return s

    def reference(self, form):
        """(out [T][H][dv], element-wise worst-case bound), from the definition in 64 bits."""
        u = U[self.dtype]
        out = np.zeros((self.T, self.H, self.dv))
        tol = np.zeros_like(out)
        flat = self.cache.view(-1, self.dc + self.dr)
        w = self.w_kv.double().numpy()
        wk, wv = w[:, :self.dn], w[:, self.dn:]
        for b in range(self.B):
            lo, hi = self.start[b], self.start[b + 1]
            if hi == lo:
                continue
            rows = flat[self.slots(b)].double().numpy()
            seen = self.seen(b)
            rows = np.where(seen.any(0)[:, None], rows, 0.0)  # rows that no query sees have no part
            c, k = rows[:, :self.dc], rows[:, self.dc:]
            q = self.q[lo:hi].double().numpy()
            for h in range(self.H):
                qn, qr = q[:, h, :self.dn], q[:, h, self.dn:]
                key, val = c @ wk[h].T, c @ wv[h].T
                z = (qn @ key.T + qr @ k.T) * self.scale
                if form == "absorbed":
                    ds = u * self.scale * (np.abs(qn @ wk[h]) @ np.abs(c).T)
                    mag = lambda p: (p @ np.abs(c)) @ np.abs(wv[h]).T  # noqa: E731
                else:
                    ds = u * self.scale * (np.abs(qn) @ np.abs(key).T)
                    mag = lambda p: p @ np.abs(val)  # noqa: E731
                z = np.where(seen, z, -np.inf)
                top = z.max(axis=1, initial=-np.inf, keepdims=True) if z.shape[1] else np.full((hi - lo, 1), -np.inf)
                p = np.exp(z - np.where(np.isfinite(top), top, 0.0))
                l = p.sum(axis=1, keepdims=True)
                p = np.divide(p, l, out=np.zeros_like(p), where=l > 0)
                out[lo:hi, h] = p @ val
                worst = np.where(seen, ds, 0.0).max(axis=1, initial=0.0, keepdims=True)
                tol[lo:hi, h] = (np.exp(2 * worst) * (1 + u) ** 2 - 1) * mag(p) * 1.05
        return out, tol + 1.05 * u * np.abs(out) + 1e-7

    def gpu(self):
        d = dict(table=torch.from_numpy(self.table).cuda(), q_start=torch.from_numpy(self.start).cuda(),
                 kv_len=torch.tensor(self.n, dtype=torch.int32).cuda(), cache=self.cache.cuda(), q=self.q.cuda(),
                 w_kv=self.w_kv.cuda())
        d["w_kt"] = d["w_kv"][:, :self.dn].transpose(1, 2).contiguous()
        d["tree"] = None if self.tree is None else torch.from_numpy(
            np.array(self.tree, dtype=np.uint64).view(np.int64)).cuda()
        d["out"] = torch.full((self.T, self.H, self.dv), 7.0, dtype=tdtype(self.dtype), device="cuda")
        return d

    def cfg(self, moe):
        return moe.LatentCfg(self.H, self.dc, self.dr, self.dn, self.dv, tdtype(self.dtype), self.page, self.scale)

    def run(self, moe, ctx, form, d=None, **kw):
        d = self.gpu() if d is None else d
        qn, qr = d["q"][..., :self.dn], d["q"][..., self.dn:]
        if form == "absorbed":
            moe.moe_latent_attend(ctx, self.cfg(moe), qn, qr, d["w_kt"], d["w_kv"], d["cache"], d["table"],
                                  d["q_start"], d["kv_len"], kw.get("max_q", max(self.q_len + [0])), d["out"],
                                  tree=d["tree"])
        else:
            moe.moe_latent_prompt(ctx, self.cfg(moe), qn, qr, d["w_kv"], d["cache"], d["table"], d["q_start"],
                                  d["kv_len"], kw.get("n_kv", sum(self.n)), d["out"])
        return d["out"]

    def check(self, moe, ctx, form, norm=3.0, **kw):
        log(f"{form} {self.dims} {self.dtype} page {self.page} q {self.q_len[:8]} n {self.n[:8]} "
            f"tree {self.tree is not None}")
        out = self.run(moe, ctx, form, **kw)
        ctx.check()
        got = out.double().cpu().numpy()
        ref, tol = self.reference(form)
        assert np.isfinite(got).all()
        over = np.abs(got - ref) > tol
        assert not over.any(), (np.argwhere(over)[:4], np.abs(got - ref)[over][:4], tol[over][:4])
        if norm and np.linalg.norm(ref) > 0:
            rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
            log(f"  relative error {rel / U[self.dtype]:.2f} u")
            assert rel <= norm * U[self.dtype], rel
        return out


def random_tree(rng, q):
    words = []
    for n in q:
        own = []
        for i in range(n):
            parent = int(rng.integers(0, i)) if i else -1
            own.append((own[parent] if parent >= 0 else 0) | (1 << i))
        words += own
    return words


# --- both forms, lengths ------------------------------------------------------

EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257]


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dims", [TINY, SMALL, dict(HALF, H=3), dict(WIDE, H=7)], ids=["tiny", "small", "half", "wide"])
def test_single_tokens_at_edge_lengths(moe, ctx, form, dtype, dims):
    Problem(11, [1] * len(EDGES), EDGES, **dims, dtype=dtype).check(moe, ctx, form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("page", [1, 16, 64, 128])
def test_pieces_of_prompts(moe, ctx, form, page):
    q = [33, 1, 64, 65, 0, 130, 7]
    n = [33, 40, 200, 65, 50, 131, 300]
    Problem(12, q, n, **SMALL, page=page, poison=float("nan")).check(moe, ctx, form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("dims", [dict(d, H=H) for d, H in ((TINY, 1), (SMALL, 33), (HALF, 64), (WIDE, 128),
                                                            (dict(TINY, dr=64), 31), (dict(SMALL, dr=64), 65),
                                                            (dict(WIDE, dr=32), 2), (dict(WIDE, dn=64, dv=64), 96),
                                                            (dict(TINY, dn=192, dv=256), 4))],
                         ids=lambda d: "-".join(str(v) for v in d.values()))
def test_head_layouts(moe, ctx, form, dims):
    Problem(13, [1, 3, 2], [70, 150, 2], **dims).check(moe, ctx, form)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_long_prompt(moe, ctx, form):
    Problem(14, [301, 515], [301, 1030], **dict(WIDE, H=2)).check(moe, ctx, form)
    Problem(15, [300], [777], **dict(HALF, H=2), dtype="fp16").check(moe, ctx, form)


def test_long_context_is_split_and_joined(moe, ctx):
    Problem(16, [1, 1, 2], [9001, 3, 20000], **dict(WIDE, H=4), page=64).check(moe, ctx, "absorbed")
    Problem(17, [1], [30011], **dict(HALF, H=2), page=64, dtype="fp16").check(moe, ctx, "absorbed")


def test_many_sequences(moe, ctx):
    rng = np.random.default_rng(3)
    n = [int(x) for x in rng.integers(0, 90, size=1024)]
    q = [min(1, x) for x in n]
    Problem(18, q, n, **dict(TINY, H=2)).check(moe, ctx, "absorbed")
    q = [int(min(x, rng.integers(0, 4))) for x in n]
    Problem(19, q, n, **dict(TINY, H=2)).check(moe, ctx, "expanded")


# --- trees ---------------------------------------------------------------------

@pytest.mark.parametrize("dims", [TINY, dict(HALF, H=9), dict(WIDE, H=16)], ids=["tiny", "half", "wide"])
def test_trees(moe, ctx, dims):
    rng = np.random.default_rng(5)
    q = [3, 64, 1, 17, 0, 40]
    n = [100, 64, 1, 17 + 47, 12, 40 + 130]
    Problem(21, q, n, **dims, tree=random_tree(rng, q)).check(moe, ctx, "absorbed")


def test_tree_words_are_free(moe, ctx):
    """Any bits: none (nothing seen where there is no prefix), later rows, bits behind the tree's end."""
    q, n = [5, 4, 3], [5, 44, 3]
    words = [0, 0b10110, 0, 1, 2 ** 64 - 1, 0, 0b1111, 0b1000, 2 ** 63, 0b1, 0, 0b100]
    out = Problem(22, q, n, **SMALL, tree=words).check(moe, ctx, "absorbed")
    assert bool((out[0] == 0).all()) and bool((out[10] == 0).all())  # nothing seen
    assert bool((out[5] != 0).any())  # the prefix is seen


def test_a_chain_is_the_causal_form(moe, ctx):
    q, n = [6, 3], [60, 90]
    chain = [(1 << (i + 1)) - 1 for x in q for i in range(x)]
    a = Problem(23, q, n, **SMALL)
    b = Problem(23, q, n, **SMALL, tree=chain)
    assert torch.equal(a.run(moe, ctx, "absorbed"), b.run(moe, ctx, "absorbed"))


# --- what is not seen -----------------------------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_rows_hold_anything(moe, ctx, bad):
    """Rows behind a sequence's end, rows of other branches and later rows of the call."""
    base = Problem(31, [4, 2], [70, 18], **SMALL, tree=[0b0001, 0b0011, 0b0101, 0b1001, 0b01, 0b10])
    ref, tol = base.reference("absorbed")
    p = Problem(31, [4, 2], [70, 18], **SMALL, tree=[0b0001, 0b0011, 0b0101, 0b1001, 0b01, 0b10], poison=bad)
    flat = p.cache.view(-1, p.dc + p.dr)
    flat[p.slots(0)[67]] = bad  # own row 1 of sequence 0: seen by its token 1 only
    got = p.run(moe, ctx, "absorbed").double().cpu().numpy()
    ctx.check()
    rest = [0, 2, 3, 4, 5]
    assert np.isfinite(got[rest]).all() and (np.abs(got - ref)[rest] <= tol[rest]).all()
    assert not np.isfinite(got[1]).any()
    for form in ("absorbed", "expanded"):
        base = Problem(32, [70], [140], **SMALL)
        ref, tol = base.reference(form)
        p = Problem(32, [70], [140], **SMALL, poison=bad)
        p.cache.view(-1, p.dc + p.dr)[p.slots(0)[100]] = bad  # own row 30
        got = p.run(moe, ctx, form).double().cpu().numpy()
        ctx.check()
        assert np.isfinite(got[:30]).all() and (np.abs(got - ref)[:30] <= tol[:30]).all()
        assert not np.isfinite(got[30:]).any()


def test_infinite_value_is_told_apart(moe, ctx):
    """An infinite value of a seen row, behind a finite score, gives that infinity and not NaN."""
    for form in ("absorbed", "expanded"):
        p = Problem(33, [1, 2], [40, 41], **SMALL)
        p.q[:] = 0  # scores 0 (and 0 x inf would be NaN: the keys of the row stay finite below)
        p.w_kv[:, :p.dn] = 0
        p.w_kv[:, p.dn:] = 0
        p.w_kv[:, p.dn:, 3] = 1.0
        row = p.cache.view(-1, p.dc + p.dr)[p.slots(1)[40]]
        row[:] = 1.0
        big = torch.finfo(tdtype(p.dtype)).max
        row[3] = big
        ref, tol = p.reference(form)
        got = p.run(moe, ctx, form).double().cpu().numpy()
        ctx.check()
        assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


# --- scores ----------------------------------------------------------------------

@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_large_and_zero_scores(moe, ctx, form):
    # scores of some hundreds: softmax is nearly one row; the worst-case bound holds, the 2-norm one is not meant
    Problem(41, [2, 1], [90, 300], **SMALL, dtype="fp16", q_std=8.0, scale=1.0).check(moe, ctx, form, norm=None)
    Problem(42, [2, 1], [90, 300], **SMALL, dtype="fp16", scale=0.0).check(moe, ctx, form)
    Problem(43, [2, 1], [90, 300], **SMALL, dtype="fp16", scale=-0.2).check(moe, ctx, form)


def test_rising_scores_rescale_the_sums(moe, ctx):
    """Scores that rise along the cache, so that the running maximum moves in every tile."""
    for form in ("absorbed", "expanded"):
        p = Problem(44, [1, 40], [1000, 700], **SMALL, dtype="fp16")
        for b in range(2):
            s = p.slots(b)
            flat = p.cache.view(-1, p.dc + p.dr)
            flat[s, p.dc:] = 0
            flat[s, p.dc] = (torch.arange(len(s)) * 0.05).to(flat.dtype)
        p.q[..., p.dn:] = 0
        p.q[..., p.dn] = 8.0
        p.check(moe, ctx, form, norm=None)


# --- empty and uncovered ------------------------------------------------------------

@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_rows_without_anything_to_see(moe, ctx, form):
    """Sequences of no rows, more tokens than rows, no tokens."""
    out = Problem(51, [2, 5, 0, 1], [0, 3, 7, 20], **TINY).check(moe, ctx, form)
    assert bool((out[:2] == 0).all()) and bool((out[2:4] == 0).all()) and bool((out[4:7] != 0).any())


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_tokens_of_no_sequence_are_left(moe, ctx, form):
    p = Problem(52, [3, 2], [30, 20], **TINY)
    d = p.gpu()
    d["q_start"] = torch.tensor([1, 3, 4], dtype=torch.int32, device="cuda")
    out = p.run(moe, ctx, form, d)
    ctx.check()
    assert bool((out[0] == 7).all()) and bool((out[4] == 7).all()) and bool((out[1:4] != 7).any())


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_no_tokens_no_sequences(moe, ctx, form):
    p = Problem(53, [0, 0], [5, 0], **TINY)
    p.run(moe, ctx, form)
    p = Problem(54, [], [], **TINY)
    p.run(moe, ctx, form)
    ctx.check()


# --- memory ---------------------------------------------------------------------------

@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_offsets_beyond_32_bits(moe, ctx, form):
    """Pages whose elements lie past 2^32 of the cache."""
    p = Problem(61, [2, 1], [100, 70], **dict(WIDE, H=2), page=64)
    d = p.gpu()
    row = p.dc + p.dr
    n_pages = (2 ** 32 + 2 ** 22) // (64 * row)
    cache = torch.empty((n_pages, 64, row), dtype=torch.bfloat16, device="cuda")
    used = sorted({int(x) for b in range(2) for x in p.table[b, :-(-p.n[b] // 64)]})
    table = p.table.copy()
    for i, old in enumerate(used):
        cache[n_pages - 1 - 2 * i] = d["cache"][old]
        table[p.table == old] = n_pages - 1 - 2 * i
    d["table"] = torch.from_numpy(table).cuda()
    small = p.run(moe, ctx, form).clone()
    d["cache"] = cache
    assert torch.equal(p.run(moe, ctx, form, d), small)
    ctx.check()


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_strides_of_the_queries(moe, ctx, form):
    p = Problem(62, [3, 1], [50, 20], **SMALL)
    d = p.gpu()
    plain = p.run(moe, ctx, form, d).clone()
    cfg = p.cfg(moe)
    # heads before tokens, and rotary parts of their own
    qn = torch.empty((p.H, p.T, p.dn + 8), dtype=d["q"].dtype, device="cuda")[..., :p.dn].transpose(0, 1)
    qn.copy_(d["q"][..., :p.dn])
    qr = d["q"][..., p.dn:].contiguous()
    out = torch.empty_like(plain)
    if form == "absorbed":
        moe.moe_latent_attend(ctx, cfg, qn, qr, d["w_kt"], d["w_kv"], d["cache"], d["table"], d["q_start"],
                              d["kv_len"], 3, out)
    else:
        moe.moe_latent_prompt(ctx, cfg, qn, qr, d["w_kv"], d["cache"], d["table"], d["q_start"], d["kv_len"], 70, out)
    assert torch.equal(out, plain)


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
def test_same_bits_again_and_under_larger_hints(moe, ctx, form):
    p = Problem(63, [3, 1, 20], [500, 2000, 90], **dict(HALF, H=8))
    d = p.gpu()
    a = p.run(moe, ctx, form, d).clone()
    for _ in range(3):
        assert torch.equal(p.run(moe, ctx, form, d), a)
    p.check(moe, ctx, form, max_q=24, n_kv=5000)
    p.check(moe, ctx, form, max_q=1)


def test_another_stream(moe):
    s = torch.cuda.Stream()
    c = moe.MoeCtx(0, stream=s)
    try:
        p = Problem(64, [3, 1], [50, 20], **SMALL)
        d = p.gpu()
        torch.cuda.synchronize()
        for form in ("absorbed", "expanded"):
            p.run(moe, c, form, d)
            s.synchronize()
            ref, tol = p.reference(form)
            assert (np.abs(d["out"].double().cpu().numpy() - ref) <= tol).all()
    finally:
        c.close()


def test_graph_replays_on_other_lengths(moe):
    """A captured step follows the lengths, tables, masks and queries that its arrays hold at replay."""
    cap = torch.cuda.Stream()
    c = moe.MoeCtx(0, stream=cap)
    try:
        probs = [Problem(65 + i, [3, 2], n, **SMALL, tree=random_tree(np.random.default_rng(i), [3, 2]))
                 for i, n in enumerate(([400, 90], [5, 2], [90, 333]))]
        wide = max(p.table.shape[1] for p in probs)
        pages = max(p.cache.shape[0] for p in probs)
        d = probs[0].gpu()
        d["table"] = torch.zeros((2, wide), dtype=torch.int32, device="cuda")
        d["cache"] = torch.zeros((pages, 16, 288), dtype=torch.bfloat16, device="cuda")

        def load(p):
            e = p.gpu()
            d["table"].zero_()
            d["table"][:, :p.table.shape[1]] = e["table"]
            d["cache"][:p.cache.shape[0]] = e["cache"]
            for k in ("q", "kv_len", "tree", "w_kv", "w_kt", "q_start"):
                d[k].copy_(e[k])
            torch.cuda.synchronize()

        load(probs[0])
        probs[0].run(moe, c, "absorbed", d)  # the scratch grows before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=cap):
            probs[0].run(moe, c, "absorbed", d)
        for p in probs + probs[:1]:
            load(p)
            d["out"].fill_(9)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            replayed = d["out"].clone()
            p.run(moe, c, "absorbed", d)
            torch.cuda.synchronize()
            assert torch.equal(replayed, d["out"])
            ref, tol = p.reference("absorbed")
            assert (np.abs(replayed.double().cpu().numpy() - ref) <= tol).all()
        c.check()
    finally:
        c.close()


# --- reported on the device -----------------------------------------------------------

@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("what", ["page", "negative page", "start", "negative length", "length", "end"])
def test_bad_bounds_are_reported(moe, ctx, form, what):
    p = Problem(71, [2, 1], [40, 20], **TINY)
    d = p.gpu()
    if what == "page":
        d["table"][0, 0] = d["cache"].shape[0]
    elif what == "negative page":
        d["table"][1, 1] = -1
    elif what == "start":
        d["q_start"][1] = -5
    elif what == "negative length":
        d["kv_len"][1] = -1
    elif what == "length":
        d["table"].clamp_(max=d["cache"].shape[0] - 1)
        d["kv_len"][1] = d["table"].shape[1] * p.page + 1
    else:
        d["q_start"][2] = 50
    p.run(moe, ctx, form, d, n_kv=200)
    with pytest.raises(moe.MoeError) as ex:
        ctx.check()
    assert ex.value.status == moe.MOE_EINVAL and "latent" in str(ex.value)
    ctx.check()  # cleared


@pytest.mark.parametrize("form", ["absorbed", "expanded"])
@pytest.mark.parametrize("back", [0, 90])
def test_starts_that_go_back_are_reported(moe, ctx, form, back):
    """Sequences that share queries ask for more row tiles than T tokens have."""
    p = Problem(74, [130] + [0] * 7, [150] + [20] * 7, **TINY)
    d = p.gpu()
    d["kv_len"].fill_(20)
    d["q_start"][2:] = torch.tensor([back, 130, back, 130, back, 130, 130], dtype=torch.int32)
    p.run(moe, ctx, form, d, n_kv=200)
    with pytest.raises(moe.MoeError):
        ctx.check()
    p.check(moe, ctx, form)


def test_too_small_a_workspace_is_reported(moe, ctx):
    p = Problem(72, [1, 2, 1], [40, 20, 30], **TINY)
    ref, tol = p.reference("expanded")
    out = p.run(moe, ctx, "expanded", n_kv=65)
    with pytest.raises(moe.MoeError):
        ctx.check()
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref)[:3] <= tol[:3]).all() and (got[3] == 7).all()


def test_a_tree_longer_than_its_word_is_reported(moe, ctx):
    p = Problem(73, [66], [80], **TINY, tree=[1] * 66)
    d = p.gpu()
    p.run(moe, ctx, "absorbed", d, max_q=64)
    with pytest.raises(moe.MoeError):
        ctx.check()


# --- refused on the host ------------------------------------------------------------------

def test_refusals(moe, ctx):
    p = Problem(81, [2], [20], **TINY)
    d = p.gpu()

    def cfg(**kw):
        v = dict(n_heads=5, d_latent=128, d_rope=32, d_nope=64, d_v=64, dtype=torch.bfloat16, page_size=16)
        v.update(kw)
        return moe.LatentCfg(**v)

    def both(c, err, **kw):
        e = dict(d, **kw)
        qn = kw.get("qn", e["q"][..., :64])
        qr = kw.get("qr", e["q"][..., 64:])
        for f in ("a", "e"):
            with pytest.raises(err):
                if f == "a":
                    moe.moe_latent_attend(ctx, c, qn, qr, e["w_kt"], e["w_kv"], e["cache"], e["table"], e["q_start"],
                                          e["kv_len"], 2, e["out"])
                else:
                    moe.moe_latent_prompt(ctx, c, qn, qr, e["w_kv"], e["cache"], e["table"], e["q_start"],
                                          e["kv_len"], 20, e["out"])

    both(cfg(), TypeError, w_kv=d["w_kv"].float())
    both(cfg(), TypeError, cache=d["cache"].cpu())
    both(cfg(), ValueError, out=d["out"][:1])
    both(cfg(), ValueError, w_kv=d["w_kv"][:, :100])
    both(cfg(), ValueError, qn=d["q"][..., 0:128:2])
    both(cfg(), TypeError, kv_len=d["kv_len"].long())
    odd = torch.zeros((2, 5, 100), dtype=torch.bfloat16, device="cuda")
    both(cfg(), moe.MoeError, qn=odd[..., :64])                       # strides no multiple of 8
    both(cfg(), moe.MoeError, qn=torch.zeros((2 * 5 * 64 + 8,), dtype=torch.bfloat16,
                                             device="cuda")[1:641].view(2, 5, 64))  # not 16-byte aligned
    both(cfg(scale=float("nan")), moe.MoeError)
    both(cfg(scale=float("inf")), moe.MoeError)
    for bad in (dict(d_latent=192), dict(d_rope=48), dict(d_nope=64, d_v=128), dict(n_heads=0), dict(n_heads=129),
                dict(page_size=24)):
        c = cfg(**bad)
        q = torch.zeros((2, c.n_heads, c.d_nope + c.d_rope), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(moe.MoeError) as ex:
            moe.moe_latent_prompt(ctx, c, q[..., :c.d_nope], q[..., c.d_nope:],
                                  torch.zeros((c.n_heads, c.d_nope + c.d_v, c.d_latent), dtype=torch.bfloat16,
                                              device="cuda"),
                                  torch.zeros((3, c.page_size, c.d_latent + c.d_rope), dtype=torch.bfloat16,
                                              device="cuda"),
                                  d["table"], d["q_start"], d["kv_len"], 20,
                                  torch.zeros((2, c.n_heads, c.d_v), dtype=torch.bfloat16, device="cuda"))
        assert ex.value.status == moe.MOE_EINVAL
    with pytest.raises(TypeError):
        cfg(dtype=torch.float32)
    args = (d["q"][..., :64], d["q"][..., 64:], d["w_kt"], d["w_kv"], d["cache"], d["table"], d["q_start"],
            d["kv_len"])
    with pytest.raises(moe.MoeError):
        moe.moe_latent_attend(ctx, cfg(), *args, 3, d["out"])         # max_q above T
    with pytest.raises(ValueError):
        moe.moe_latent_attend(ctx, cfg(), *args, 2, d["out"], tree=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_latent_prompt(ctx, cfg(), args[0], args[1], *args[3:], -1, d["out"])
    torch.cuda.synchronize()
    assert bool((d["out"] == 7).all())  # nothing was enqueued
    ctx.check()


# --- the cache's writer -----------------------------------------------------------------------

def append_reference(kv, turn, pos, norm_w, eps, dc):
    kv = kv.double().numpy()
    c = kv[:, :dc]
    if norm_w is not None:
        c = c / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps) * norm_w.double().numpy()
    return c, rotate_reference(kv[:, dc:], turn, pos)


def rotate_reference(x, turn, pos):
    t = turn.double().numpy()[pos]
    z = x[..., 0::2] + 1j * x[..., 1::2]
    w = t[..., 0] + 1j * t[..., 1]
    z = z * w.reshape(w.shape[:1] + (1,) * (z.ndim - 2) + w.shape[1:])
    return np.stack([z.real, z.imag], axis=-1).reshape(x.shape)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dims", [TINY, SMALL, HALF, dict(WIDE, dr=32)], ids=["tiny", "small", "half", "wide"])
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("norm", [True, False])
def test_append(moe, ctx, dtype, dims, T, norm):
    """fp32 arithmetic rounded once: within u of the exact value, and 2^-21 for the fp32 steps (at most six roundings
    of 2^-24 each, the mean's sum of at most 512 squares in a tree adding 2^-20 of it at most, halved by the root)."""
    H, dc, dr, dn = dims["H"], dims["dc"], dims["dr"], dims["dn"]
    g = torch.Generator().manual_seed(90 + T)
    rng = np.random.default_rng(90 + T)
    t, page, n_pages = tdtype(dtype), 16, 9
    wide = torch.randn((T, dc + dr + 16), generator=g).to(t).cuda()
    kv = wide[:, :dc + dr]
    turn = torch.randn((300, dr // 2, 2), generator=g)
    pos = rng.integers(0, 300, size=T)
    pos[0] = 299
    slot = rng.permutation(page * n_pages)[:T]
    if T > 1:
        slot[5] = -1
    w = (1 + 0.2 * torch.randn((dc,), generator=g)) if norm else None
    q = torch.randn((T, H, dn + dr), generator=g).to(t)
    cache = torch.full((n_pages, page, dc + dr), 3.0, dtype=t, device="cuda")
    qr = torch.zeros((T, H, dr), dtype=t, device="cuda")
    cfg = moe.LatentCfg(H, dc, dr, dn, dims["dv"], t, page)
    log("append", dims, dtype, T, norm)
    moe.moe_latent_append(ctx, cfg, kv, turn.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(),
                          torch.from_numpy(slot.astype(np.int64)).cuda(), cache,
                          norm_w=None if w is None else w.cuda(), eps=1e-5, q_rope=q.cuda()[..., dn:], q_rope_out=qr)
    ctx.check()
    c, k = append_reference(kv.cpu(), turn, pos, w, 1e-5, dc)
    got = cache.double().cpu().numpy().reshape(-1, dc + dr)
    u = U[dtype] + 2.0 ** -19
    kept = slot >= 0
    assert (np.abs(got[slot[kept], :dc] - c[kept]) <= u * np.abs(c[kept]) + 1e-7).all()
    # a turned pair is a sum of two products: the fp32 steps are relative to their sizes
    size = np.abs(kv.double().cpu().numpy()[:, dc:]).max() * np.abs(turn.double().numpy()).max() * 2
    assert (np.abs(got[slot[kept], dc:] - k[kept]) <= u * np.abs(k[kept]) + 2.0 ** -22 * size).all()
    rest = np.setdiff1d(np.arange(page * n_pages), slot[kept])
    assert (got[rest] == 3.0).all()
    r = rotate_reference(q.double().numpy()[..., dn:], turn, pos)
    size = np.abs(q.double().numpy()).max() * np.abs(turn.double().numpy()).max() * 2
    assert (np.abs(qr.double().cpu().numpy() - r) <= u * np.abs(r) + 2.0 ** -22 * size).all()


def test_append_without_queries_and_of_nothing(moe, ctx):
    cfg = moe.LatentCfg(2, 128, 32, 64, 64, torch.bfloat16, 16)
    cache = torch.zeros((2, 16, 160), dtype=torch.bfloat16, device="cuda")
    turn = torch.zeros((4, 16, 2), device="cuda")
    turn[..., 0] = 1.0
    kv = torch.randn((3, 160), device="cuda").bfloat16()
    pos = torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda")
    slot = torch.tensor([31, 0, 7], device="cuda")
    moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot, cache)
    ctx.check()
    assert torch.equal(cache.view(-1, 160)[slot], kv)  # no norm, no angle: the row itself
    moe.moe_latent_append(ctx, cfg, kv[:0], turn, pos[:0], slot[:0], cache)
    ctx.check()


@pytest.mark.parametrize("what", ["slot", "slot below -1", "pos", "negative pos"])
def test_append_reports_bad_places(moe, ctx, what):
    cfg = moe.LatentCfg(2, 128, 32, 64, 64, torch.bfloat16, 16)
    cache = torch.full((2, 16, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    turn = torch.ones((4, 16, 2), device="cuda")
    kv = torch.randn((2, 160), device="cuda").bfloat16()
    pos = torch.tensor([0, {"pos": 4, "negative pos": -1}.get(what, 1)], dtype=torch.int32, device="cuda")
    slot = torch.tensor([3, {"slot": 32, "slot below -1": -2}.get(what, 5)], device="cuda")
    q = torch.randn((2, 2, 32), device="cuda").bfloat16()
    moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot, cache, q_rope=q, q_rope_out=torch.empty_like(q))
    with pytest.raises(moe.MoeError) as ex:
        ctx.check()
    assert ex.value.status == moe.MOE_EINVAL
    flat = cache.view(-1, 160)
    assert bool((flat[3] != 3.0).any()) and int((flat != 3.0).any(dim=1).sum()) == 1


def test_append_refusals(moe, ctx):
    cfg = moe.LatentCfg(2, 128, 32, 64, 64, torch.bfloat16, 16)
    cache = torch.full((2, 16, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    turn = torch.ones((4, 16, 2), device="cuda")
    kv = torch.randn((2, 160), device="cuda").bfloat16()
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    slot = torch.tensor([3, 4], device="cuda")
    q = torch.randn((2, 2, 32), device="cuda").bfloat16()
    with pytest.raises(TypeError):
        moe.moe_latent_append(ctx, cfg, kv.float(), turn, pos, slot, cache)
    with pytest.raises(TypeError):
        moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot.int(), cache)
    with pytest.raises(ValueError):
        moe.moe_latent_append(ctx, cfg, kv[:, :128], turn, pos, slot, cache)
    with pytest.raises(ValueError):
        moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot, cache, q_rope=q)
    with pytest.raises(ValueError):
        moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot, cache, q_rope_out=q)
    with pytest.raises(moe.MoeError):
        moe.moe_latent_append(ctx, cfg, kv, turn, pos, slot, cache, norm_w=torch.ones(128, device="cuda"), eps=-1.0)
    odd = torch.zeros((2, 164), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_latent_append(ctx, cfg, odd[:, :160], turn, pos, slot, cache)
    torch.cuda.synchronize()
    assert bool((cache == 3.0).all())
