"""Measured cases of the operators on microscaled 4-bit floating point.

A row is cut into blocks of 32 values that share one power of two; each value
is a 4-bit float (0, 0.5, 1, 1.5, 2, 3, 4 or 6, with a sign). Experts kept
this way need: the quantiser of weights and hidden states and the way back, the
product of two such matrices (projections, the shared expert), the product
grouped by expert with ragged sizes, and the experts' whole FFN.

`own` chooses between the plain form (elementary torch operations in 32 bits,
rounded once at the end) and the framework's kernels. Cases are dicts of plain
values:

    op      "round", "product", "grouped" or "ffn"
    dtype   of what is quantised and of the results
    round:    rows, K           rows to 4 bits and back
    product:  M, N, K           M rows by N rows of weights, both in 4 bits
    grouped:  T, k, E, N, K     each token's row by the weights of its k experts;
                                scatter: results in the tokens' order, not the experts'
    ffn:      T, k, E, H, I     hidden states in, hidden states out
    skew    how uneven the routing is (0: every expert as likely)
"""
import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32
# hidden 6144, 256 experts of intermediate 2048 and one shared, 8 a token
GLM = {"H": 6144, "I": 2048, "E": 256, "k": 8}


def listed():
    return [
        # the hidden state of one token, before its layer: pure latency
        {"name": "round_token", "op": "round", "dtype": "fp32", "rows": 1, "K": 6144},
        # a prompt's hidden states
        {"name": "round_prompt", "op": "round", "dtype": "bf16", "rows": 2047, "K": 6144},
        # the gate matrices of 16 experts, as they are read in
        {"name": "round_weights", "op": "round", "dtype": "fp32", "rows": 32768, "K": 6144},
        # one token through the attention's query projection (128 heads of 128 + 64)
        {"name": "product_token", "op": "product", "dtype": "bf16", "M": 1, "N": 24576, "K": 6144},
        # drafted tokens through the down projection of a shared expert, narrow and ragged
        {"name": "product_draft", "op": "product", "dtype": "fp16", "M": 33, "N": 6144, "K": 2048},
        # a prompt through the query projection
        {"name": "product_prompt", "op": "product", "dtype": "bf16", "M": 2048, "N": 24576, "K": 6144},
        # one token through gate and up of its experts
        {"name": "grouped_token", "op": "grouped", "dtype": "fp32", "T": 1, "k": 8, "E": 64, "N": 4096, "K": 6144,
         "skew": 0.0, "scatter": False},
        # 32 sequences of one token and two drafts each through down of their experts
        {"name": "grouped_verify", "op": "grouped", "dtype": "bf16", "T": 96, "k": 8, "E": 256, "N": 6144, "K": 2048,
         "skew": 1.0, "scatter": True},
        # a prompt through gate and up
        {"name": "grouped_prompt", "op": "grouped", "dtype": "bf16", "T": 2047, "k": 8, "E": 256, "N": 4096,
         "K": 6144, "skew": 0.5, "scatter": False},
        # the layer's experts: one token, a batch of 64 with uneven routing, a prompt
        {"name": "ffn_token", "op": "ffn", "dtype": "bf16", "T": 1, **GLM, "shared": True, "skew": 0.0},
        {"name": "ffn_batch", "op": "ffn", "dtype": "fp16", "T": 64, **GLM, "shared": True, "skew": 1.5},
        {"name": "ffn_prompt", "op": "ffn", "dtype": "bf16", "T": 2048, **GLM, "shared": True, "skew": 0.5},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["round", "product", "product", "grouped", "grouped", "ffn"])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"] if op != "ffn" else ["bf16", "fp16"])}
    if op == "round":
        case["K"] = 32 * log(1, 512)
        case["rows"] = log(1, min(200000, 200_000_000 // case["K"]))
        return case
    if op == "product":
        case["K"] = 32 * log(2, 512)
        case["M"] = log(1, 4096)
        case["N"] = log(32, min(24576, 300_000_000_000 // (case["K"] * case["M"])))
        return case
    case["E"] = log(1, 256)
    case["k"] = rng.randint(1, min(16, case["E"]))
    case["skew"] = rng.choice([0.0, 0.5, 1.0, 1.5])
    if op == "grouped":
        case["K"] = 32 * log(2, 256)
        case["N"] = log(32, min(8192, 6_000_000_000 // (case["E"] * case["K"])))
        case["T"] = log(1, min(2048, 16384 // case["k"], 400_000_000_000 // (case["k"] * case["N"] * case["K"])))
        case["scatter"] = rng.choice([True, False])
    else:
        case["H"] = 64 * log(2, 128)
        case["I"] = 64 * log(1, max(1, min(128, 9_000_000_000 // (3 * case["E"] * case["H"] * 64))))
        case["shared"] = rng.choice([True, False])
        top = 600_000_000_000 // (3 * (case["k"] + 1) * case["H"] * case["I"])
        case["T"] = log(1, min(2048, 16384 // case["k"], max(1, top)))
    return case


@functools.lru_cache(maxsize=64)
def _pattern(T, k, E, skew):
    """k distinct experts a token; the same experts' loads for every seed."""
    rng = np.random.default_rng([T, k, E, int(10 * skew)])
    z = -skew * np.log(np.arange(1, E + 1))[None, :] + rng.gumbel(size=(T, E))
    return np.argsort(-z, axis=1)[:, :k].astype(np.int32)


def _lines(case):
    """Experts' loads, largest first."""
    return np.sort(np.bincount(_pattern(case["T"], case["k"], case["E"], case["skew"]).ravel(),
                               minlength=case["E"]))[::-1]


def work(case):
    held = 0.5 + 1 / BLOCK
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "round":
        return {"bytes": case["rows"] * case["K"] * 2 * size, "flops": case["rows"] * case["K"] * 4}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * held + M * N * size, "flops": 2 * M * N * K}
    active, lines = int((_lines(case) > 0).sum()), case["T"] * case["k"]
    if case["op"] == "grouped":
        N, K = case["N"], case["K"]
        return {"bytes": (case["T"] + active * N) * K * held + lines * N * size, "flops": 2 * lines * N * K}
    H, I, shared = case["H"], case["I"], int(case["shared"])
    return {"bytes": (active + shared) * 3 * H * I * held + case["T"] * (2 * H * size + 8 * case["k"]),
            "flops": 6 * (lines + shared * case["T"]) * H * I}


# ---------------------------------------------------------------------------
# The format in torch
# ---------------------------------------------------------------------------

def _split(x):
    """Rows in 32 bits: 4-bit values [..., K / 32, 32] and the blocks' exponents [..., K / 32, 1]."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(top).exponent - 3  # the largest value lies in [4, 8) then
    e = torch.where(top == 0, -127, e.clamp(-127, 127))
    v = torch.ldexp(b, -e)
    a = v.abs().clamp_max(6.0)
    # halves up to 2, whole numbers up to 4, even ones above; ties to the even mantissa
    q = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(q, v), e


def _pack(x):
    """Rows in 32 bits: codes [..., K / 2] (the first of a pair in the low half) and scales [..., K / 32]."""
    q, e = _split(x)
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(q).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


@functools.lru_cache(maxsize=2)
def _tables(dtype):
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device="cuda")
    v = torch.cat([v, -v])
    byte = torch.arange(256, device="cuda")
    scale = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan], dtype=dtype, device="cuda")
    return torch.stack([v[byte & 15], v[byte >> 4]], dim=-1), scale


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    pairs, scale = _tables(torch.float32)
    return (pairs[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK)) * scale[scales.int()][..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)
    rng = np.random.default_rng([seed, 41])
    dtype = DTYPES[case["dtype"]]

    def hidden(rows, K):
        """Hidden states: near one, a few channels much larger."""
        x = torch.randn((rows, K), generator=gen, device="cuda")
        loud = torch.rand((K,), generator=gen, device="cuda") < 0.01
        return x * torch.where(loud, 10.0, 1.0)

    def weights(n, N, K):
        """n matrices of N rows in 4 bits, at the scale that keeps products near one."""
        codes = torch.empty((n, N, K // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((n, N, K // BLOCK), dtype=torch.uint8, device="cuda")
        step = max(1, 100_000_000 // (N * K))
        for i in range(0, n, step):
            m = min(step, n - i)
            codes[i:i + m], scales[i:i + m] = _pack(torch.randn((m, N, K), generator=gen, device="cuda") * K ** -0.5)
        return codes, scales

    s = {"case": case}
    if case["op"] == "round":
        rows, K = case["rows"], case["K"]
        s["x"] = (hidden(rows, K) if case["dtype"] != "fp32" else hidden(rows, K) * K ** -0.5).to(dtype)
        s["codes"] = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((rows, K // BLOCK), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["x"])
        return s
    if case["op"] == "product":
        s["x"] = _pack(hidden(case["M"], case["K"]))
        w = weights(1, case["N"], case["K"])
        s["w"] = w[0][0], w[1][0]
        s["out"] = torch.empty((case["M"], case["N"]), dtype=dtype, device="cuda")
        return s
    # routing: a fixed pattern of loads, the experts' names and the tokens' order by the seed
    T, k, E = case["T"], case["k"], case["E"]
    idx = rng.permutation(E).astype(np.int32)[_pattern(T, k, E, case["skew"])][rng.permutation(T)]
    idx = rng.permuted(idx, axis=1)
    s["most"] = int(_lines(case)[0])
    s["idx"] = torch.from_numpy(np.ascontiguousarray(idx)).cuda()
    if case["op"] == "grouped":
        # lines sorted by expert, as the bucketing leaves them
        entry = np.argsort(idx.ravel(), kind="stable").astype(np.int32)
        count = np.bincount(idx.ravel(), minlength=E)
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(count)]).astype(np.int32)).cuda()
        s["token"] = torch.from_numpy((entry // k).astype(np.int32)).cuda()
        s["entry"] = torch.from_numpy(entry).cuda() if case["scatter"] else None
        s["x"] = _pack(hidden(T, case["K"]))
        s["w"] = weights(E, case["N"], case["K"])
        s["out"] = torch.empty((T * k, case["N"]), dtype=dtype, device="cuda")
        return s
    H, I, n = case["H"], case["I"], E + int(case["shared"])
    s["x"] = hidden(T, H).to(dtype)
    p = rng.random((T, k)) + 0.05
    s["p"] = torch.from_numpy((p / p.sum(1, keepdims=True)).astype(np.float32)).cuda()
    s["gate"], s["up"], s["down"] = weights(n, I, H), weights(n, I, H), weights(n, H, I)
    # an expert's six addresses a row, the shared expert's last
    parts = [s[name][i] for i in (0, 1) for name in ("gate", "up", "down")]
    s["table"] = torch.tensor([[p.data_ptr() + e * p[0].numel() for p in parts] for e in range(n)], device="cuda")
    s["out"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------

def _plain_round(s):
    q, e = _split(s["x"].float())
    return torch.ldexp(q, e).flatten(-2).to(s["x"].dtype)


def _plain_product(s):
    return torch.matmul(_values(*s["x"]), _values(*s["w"]).t()).to(s["out"].dtype)


def _places(idx, E, most):
    """Per (token, slot) entry its expert and its place among the expert's lines; E * most places in all."""
    flat = idx.flatten().long()
    order = torch.argsort(flat, stable=True)
    first = torch.searchsorted(flat[order], torch.arange(E, device="cuda"))
    rank = torch.empty_like(order)
    rank[order] = torch.arange(len(flat), device="cuda") - first[flat[order]]
    return flat * most + rank


def _by_expert(rows, w, idx, most):
    """rows [T * k][K], each by the weights of its expert."""
    T, k = idx.shape
    E = w[0].shape[0]
    if T * k < E:  # few lines: each line's own matrix
        return torch.matmul(_values(w[0][idx.flatten().long()], w[1][idx.flatten().long()]), rows[..., None])[..., 0]
    place = _places(idx, E, most)
    padded = torch.zeros((E * most, rows.shape[-1]), device="cuda")
    padded[place] = rows
    both = torch.matmul(padded.unflatten(0, (E, most)), _values(*w).transpose(1, 2))
    return both.flatten(0, 1)[place]


def _plain_grouped(s):
    x = _values(*s["x"]).repeat_interleave(s["case"]["k"], dim=0)
    out = _by_expert(x, s["w"], s["idx"], s["most"])
    if s["entry"] is None:
        out = out[torch.argsort(s["idx"].flatten(), stable=True)]
    return out.to(s["out"].dtype)


def _again(x):
    q, e = _split(x)
    return torch.ldexp(q, e).flatten(-2)


def _plain_ffn(s):
    k, E = s["case"]["k"], s["case"]["E"]
    x = _again(s["x"].float())
    lines = x.repeat_interleave(k, dim=0)
    routed = lambda rows, name: _by_expert(rows, (s[name][0][:E], s[name][1][:E]), s["idx"], s["most"])  # noqa: E731
    swiglu = lambda g, u: g / (1 + torch.exp(-g)) * u  # noqa: E731
    y = routed(_again(swiglu(routed(lines, "gate"), routed(lines, "up"))), "down")
    out = (y.unflatten(0, (-1, k)) * s["p"][..., None]).sum(1)
    if s["case"]["shared"]:
        last = lambda rows, name: torch.matmul(rows, _values(s[name][0][E], s[name][1][E]).t())  # noqa: E731
        out = out + last(_again(swiglu(last(x, "gate"), last(x, "up"))), "down")
    return out.to(s["out"].dtype)


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=1)
def _context():
    import quantized_moe_expert_sigmoid_amd as moe
    return moe, moe.MoeCtx(torch.cuda.current_device())


def _own(s):
    moe, ctx = _context()
    c = s["case"]
    if c["op"] == "round":
        moe.moe_mx_quantize(ctx, s["x"], s["codes"], s["scales"])
        return moe.moe_mx_dequantize(ctx, s["codes"], s["scales"], s["out"])
    if c["op"] == "product":
        return moe.moe_mx_matmul(ctx, *s["x"], *s["w"], s["out"])
    if c["op"] == "grouped":
        return moe.moe_mx_grouped_matmul(ctx, *s["x"], *s["w"], s["offsets"], s["out"], in_rows=s["token"],
                                         out_rows=s["entry"])
    return moe.moe_expert_ffn_mx(ctx, s["table"], c["shared"], s["x"], s["idx"], s["p"], c["I"], s["out"])


def run(state):
    if own:
        return _own(state)
    return {"round": _plain_round, "product": _plain_product, "grouped": _plain_grouped,
            "ffn": _plain_ffn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _nearest(x):
    """Each block of 32 by its own power of two to the nearest 4-bit value, by comparison with the midpoints."""
    b = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().max(-1, keepdim=True).values
    scale = 2.0 ** (torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 2).clamp(-127, 127)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = (b / scale).abs()
    at = torch.bucketize(a, mid)  # a midpoint goes down ...
    up = (a == mid[at.clamp_max(6)]) & (at % 2 == 1)  # ... but up where the one above is even
    return (torch.sign(b) * grid[at + up] * scale).reshape(x.shape)


def _double(codes, scales):
    pairs, scale = _tables(torch.float64)
    v = torch.stack([pairs[(codes & 15).long(), 0], pairs[(codes >> 4).long(), 0]], dim=-1).flatten(-2)
    return v * scale[scales.long()].repeat_interleave(BLOCK, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "round":
        parts = [_nearest(x) for x in s["x"].split(max(1, 20_000_000 // case["K"]))]
        return torch.cat(parts)
    if case["op"] == "product":
        x = _double(*s["x"])
        return torch.cat([x @ _double(c, e).t() for c, e in zip(s["w"][0].split(4096), s["w"][1].split(4096))], dim=1)
    T, k, E = case["T"], case["k"], case["E"]
    idx = s["idx"].long()
    if case["op"] == "grouped":
        x, out, lo = _double(*s["x"]), torch.empty(s["out"].shape, dtype=torch.float64, device="cuda"), 0
        for e in range(E):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            if len(t):
                at = t * k + j if case["scatter"] else slice(lo, lo + len(t))
                out[at] = x[t] @ _double(s["w"][0][e], s["w"][1][e]).t()
                lo += len(t)
        return out
    x = _nearest(s["x"])
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(E + int(case["shared"])):
        t, j = torch.nonzero(idx == e, as_tuple=True) if e < E else (torch.arange(T, device="cuda"), None)
        if len(t):
            g, u, d = (_double(s[name][0][e], s[name][1][e]) for name in ("gate", "up", "down"))
            g, u = x[t] @ g.t(), x[t] @ u.t()
            y = _nearest(g * torch.sigmoid(g) * u) @ d.t()
            out.index_add_(0, t, y if j is None else y * s["p"][t, j].double()[:, None])
    return out
