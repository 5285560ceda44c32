"""Measured cases of the latent-attention operators.

A decoder layer whose attention keeps one latent vector a token (SURVEY of the
source pages: 32,768 floats of keys and values against 576) needs four things
beside the expert layer: the cache's writer, attention of single tokens over
the paged cache (absorbed form), the same for a tree of drafted tokens, and
attention of prompts (expanded form).

`own` chooses between the plain form (elementary torch operations in 32 bits,
rounded once at the end) and the framework's kernels. Cases are dicts of plain
values:

    op      "append", "attend", "tree" or "prompt"
    heads, dc, dr, dn, dv, dtype, page      the layer and its cache
    B, q_lo, q_hi, kv_lo, kv_hi             sequences; their new tokens and
                                            earlier cached tokens are spread
                                            evenly between the two bounds
"""
import functools
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# heads 128 with key and value parts of 128 each are the pages' 32,768 floats a token, latent 512 + rotary 64 their 576
WIDE = {"heads": 128, "dc": 512, "dr": 64, "dn": 128, "dv": 128, "dtype": "bf16", "page": 64}
# half the heads, each twice as wide
HALF = {"heads": 64, "dc": 512, "dr": 64, "dn": 192, "dv": 256, "dtype": "bf16", "page": 64}
# a small layer: few heads, small pages
SMALL = {"heads": 16, "dc": 256, "dr": 32, "dn": 64, "dv": 64, "dtype": "fp16", "page": 16}


def listed():
    return [
        # one generated token enters the cache: pure latency
        {"name": "append_token", "op": "append", **WIDE, "B": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 700, "kv_hi": 700},
        # prompts of several requests enter it at once
        {"name": "append_prompts", "op": "append", **HALF, "dtype": "fp16", "B": 7, "q_lo": 150, "q_hi": 1450,
         "kv_lo": 0, "kv_hi": 0},
        # one user, early in a conversation
        {"name": "attend_short", "op": "attend", **HALF, "B": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 300, "kv_hi": 300},
        # one user, a very long context
        {"name": "attend_long", "op": "attend", **WIDE, "B": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 131071,
         "kv_hi": 131071},
        # a serving batch, ragged
        {"name": "attend_batch", "op": "attend", **WIDE, "B": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 1000,
         "kv_hi": 7999},
        # a small layer's batch, from empty caches on
        {"name": "attend_small", "op": "attend", **SMALL, "B": 33, "q_lo": 1, "q_hi": 1, "kv_lo": 0, "kv_hi": 3001},
        # verification: 32 sequences of one token and two drafts each
        {"name": "tree_verify", "op": "tree", **HALF, "B": 32, "q_lo": 3, "q_hi": 3, "kv_lo": 500, "kv_hi": 4500},
        # one user with a wide draft
        {"name": "tree_one", "op": "tree", **WIDE, "B": 1, "q_lo": 25, "q_hi": 25, "kv_lo": 2111, "kv_hi": 2111},
        # a batch of full trees: as many products as bytes allow
        {"name": "tree_full", "op": "tree", **WIDE, "B": 8, "q_lo": 40, "q_hi": 64, "kv_lo": 900, "kv_hi": 8000},
        # a short prompt
        {"name": "prompt_short", "op": "prompt", **HALF, "B": 1, "q_lo": 509, "q_hi": 509, "kv_lo": 0, "kv_hi": 0},
        # pieces of prompts, some behind an already cached part
        {"name": "prompt_pieces", "op": "prompt", **WIDE, "dtype": "fp16", "B": 5, "q_lo": 1, "q_hi": 1023,
         "kv_lo": 0, "kv_hi": 4100},
        # one long prompt
        {"name": "prompt_long", "op": "prompt", **WIDE, "B": 1, "q_lo": 4096, "q_hi": 4096, "kv_lo": 0, "kv_hi": 0},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend", "tree", "prompt"])
    case = {"op": op, **rng.choice([WIDE, HALF, SMALL])}
    case["heads"] = rng.choice([h for h in (5, 8, 16, 20, 32, 48, 64, 96, 128) if h <= case["heads"]])
    case["dtype"] = rng.choice(["bf16", "fp16"])
    case["page"] = rng.choice([1, 16, 32, 64, 128])
    if op == "append":
        B = log(1, 64)
        q = log(1, 5600 // B)
        lo, top = 0, 100
    elif op == "attend":
        B, q = log(1, 64), 1
        lo, top = log(1, 200), 131071 // B
    elif op == "tree":
        B, q = log(1, 32), rng.randint(2, 64)
        lo, top = log(1, 200), 28000 // max(B, q // 8)
    else:
        B = log(1, 8)
        q = log(1, 4096 // B)
        lo, top = 0, max(1, min(4096, 4096 * 2048 // (B * q)) // B)
    kv = [min(lo, top), log(1, max(1, top))]
    case.update({"B": B, "q_lo": max(1, q // 2) if op != "attend" else 1, "q_hi": q, "kv_lo": min(kv),
                 "kv_hi": max(kv)})
    return case


def _lengths(case):
    """New tokens and whole lengths of the sequences (the same multiset of pairs for every seed)."""
    B = case["B"]
    at = np.arange(B) / max(B - 1, 1)
    q = np.rint(case["q_lo"] + at * (case["q_hi"] - case["q_lo"])).astype(np.int64)
    kv = np.rint(case["kv_lo"] + at[::-1] * (case["kv_hi"] - case["kv_lo"])).astype(np.int64)
    return q, kv + q


def work(case):
    q, n = _lengths(case)
    H, dc, dr, dn, dv = (case[k] for k in ("heads", "dc", "dr", "dn", "dv"))
    T, S = int(q.sum()), int(n.sum())
    if case["op"] == "append":
        return {"bytes": 2 * T * (2 * (dc + dr) + 2 * H * dr) + 4 * T * dr + 4 * dc,
                "flops": T * (4 * dc + 3 * dr * (H + 1))}
    moved = 2 * (S * (dc + dr) + H * (dn + dv) * dc + T * H * (dn + dr + dv))
    if case["op"] == "prompt":
        pairs = int((q * (n - q) + q * (q + 1) // 2).sum())
        return {"bytes": moved, "flops": 2 * H * (pairs * (dn + dr + dv) + S * dc * (dn + dv))}
    return {"bytes": moved, "flops": 2 * H * (int((q * n).sum()) * (2 * dc + dr) + T * dc * (dn + dv))}


def _tree_masks(rng, q):
    """One 64-bit word a node: itself and its ancestors in a random tree whose first node is the last sure token."""
    words = []
    for n in q:
        own_words = []
        for i in range(int(n)):
            parent = int(rng.integers(0, i)) if i else -1
            own_words.append((own_words[parent] if parent >= 0 else 0) | (1 << i))
        words += own_words
    return np.array(words, dtype=np.uint64).view(np.int64)


def prepare(case, seed):
    rng = np.random.default_rng([seed, 77])
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    dtype = DTYPES[case["dtype"]]
    H, dc, dr, dn, dv, page = (case[k] for k in ("heads", "dc", "dr", "dn", "dv", "page"))
    q, n = _lengths(case)
    order = rng.permutation(case["B"])
    q, n = q[order], n[order]
    T = int(q.sum())

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    # the cache: every sequence's pages anywhere in it, a few pages of other requests between them
    pages = -(-n // page)
    n_pages = int(pages.sum()) + 3
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.zeros((case["B"], int(pages.max())), dtype=np.int32)
    first = np.concatenate([[0], np.cumsum(pages)])
    for b in range(case["B"]):
        table[b, :pages[b]] = ids[first[b]:first[b + 1]]
    start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    seq = np.repeat(np.arange(case["B"]), q)
    pos = np.arange(T) - start[seq] + (n - q)[seq]
    s = {"case": case, "T": T, "max_q": int(q.max()), "max_kv": int(n.max()), "n_kv": int(n.sum()),
         "q_start": torch.from_numpy(start).cuda(), "kv_len": torch.from_numpy(n.astype(np.int32)).cuda(),
         "table": torch.from_numpy(table).cuda(), "cache": normal(n_pages, page, dc + dr),
         "q": normal(T, H, dn + dr)}
    if case["op"] == "append":
        # outputs of the layer's down projection, their places, and the table of rotations
        s["kv"] = normal(T, dc + dr, std=0.7)
        s["norm_w"] = 1.0 + 0.1 * torch.randn((dc,), generator=gen, device="cuda")
        angle = (np.arange(int(n.max()))[:, None] * 10000.0 ** (-np.arange(dr // 2) * 2.0 / dr)[None, :])
        turn = np.stack([np.cos(angle), np.sin(angle)], axis=-1).astype(np.float32)
        s["turn"] = torch.from_numpy(turn).cuda()
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        slot = table[seq, pos // page].astype(np.int64) * page + pos % page
        slot[rng.random(T) < 0.01] = -1  # tokens that are not kept
        s["slots"] = torch.from_numpy(slot).cuda()
        s["q_rope"] = torch.empty((T, H, dr), dtype=dtype, device="cuda")
        return s
    # expansion weights at the scale that keeps keys and values near one; the key rows transposed for the absorbed form
    s["w_kv"] = normal(H, dn + dv, dc, std=dc ** -0.5)
    s["w_kt"] = s["w_kv"][:, :dn].transpose(1, 2).contiguous()
    s["out"] = torch.empty((T, H, dv), dtype=dtype, device="cuda")
    s["scale"] = (dn + dr) ** -0.5
    s["tree"] = torch.from_numpy(_tree_masks(rng, q)).cuda() if case["op"] == "tree" else None
    return s


# ---------------------------------------------------------------------------
# Plain form
# ---------------------------------------------------------------------------

def _rotate(x, turn):
    """Pairs (2i, 2i + 1) of the last axis turned by the angles whose (cos, sin) are turn[..., i, :]."""
    a, b = x[..., 0::2], x[..., 1::2]
    c, d = turn[..., 0], turn[..., 1]
    return torch.stack([a * c - b * d, a * d + b * c], dim=-1).flatten(-2)


def _plain_append(s):
    case = s["case"]
    dc, dn, dtype = case["dc"], case["dn"], s["cache"].dtype
    kv, turn = s["kv"].float(), s["turn"][s["pos"].long()]
    c = kv[:, :dc]
    c = c * torch.rsqrt((c * c).mean(dim=-1, keepdim=True) + EPS) * s["norm_w"]
    row = torch.cat([c, _rotate(kv[:, dc:], turn)], dim=-1).to(dtype)
    kept = s["slots"] >= 0
    s["cache"].view(-1, row.shape[-1])[s["slots"][kept]] = row[kept]
    s["q_rope"].copy_(_rotate(s["q"][..., dn:].float(), turn[:, None]).to(dtype))
    return {"cache": s["cache"], "q_rope": s["q_rope"]}


def _places(s):
    """Per token: its sequence and its index in it; per sequence: new tokens and length."""
    start, n = s["q_start"].long(), s["kv_len"].long()
    tok = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(start, tok, right=True) - 1
    return seq, tok - start[seq], start[1:] - start[:-1], n


def _rows(s):
    """The sequences' cached rows, padded to the longest: [B][max_kv][dc + dr] in 32 bits."""
    page = s["case"]["page"]
    j = torch.arange(s["max_kv"], device="cuda")
    return s["cache"][s["table"].long()[:, j // page], j % page].float()


def _visible(s, seq, i, q, n):
    """[B][max_q][max_kv]: which cached positions a query sees."""
    B = s["case"]["B"]
    j = torch.arange(s["max_kv"], device="cuda")
    rank = torch.arange(s["max_q"], device="cuda")
    after = j[None, None, :] - (n - q)[:, None, None]  # index among the sequence's new tokens, negative before them
    if s["tree"] is None:
        seen = after <= rank[None, :, None]
    else:
        words = torch.zeros((B, s["max_q"]), dtype=torch.int64, device="cuda")
        words[seq, i] = s["tree"]
        seen = (after < 0) | (((words[:, :, None] >> after.clamp(0, 63)) & 1) == 1)
    return seen & (j[None, None, :] < n[:, None, None]) & (rank[None, :, None] < q[:, None, None])


def _softmax(z, seen):
    z = torch.where(seen, z, -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(dim=-1, keepdim=True).clamp_min(1e-30)


def _plain_absorbed(s):
    case = s["case"]
    H, dc, dn = case["heads"], case["dc"], case["dn"]
    seq, i, q, n = _places(s)
    rows = _rows(s)
    query = s["q"].float()
    inner = torch.matmul(query[..., :dn].transpose(0, 1), s["w_kv"][:, :dn].float()).transpose(0, 1)
    padded = torch.zeros((case["B"], s["max_q"], H, rows.shape[-1]), device="cuda")
    padded[seq, i] = torch.cat([inner, query[..., dn:]], dim=-1)
    z = torch.matmul(padded.flatten(1, 2), rows.transpose(1, 2)).view(case["B"], s["max_q"], H, -1) * s["scale"]
    p = _softmax(z, _visible(s, seq, i, q, n)[:, :, None, :])
    inner = torch.matmul(p.flatten(1, 2), rows[..., :dc]).view(case["B"], s["max_q"], H, dc)[seq, i]
    out = torch.matmul(inner.transpose(0, 1), s["w_kv"][:, dn:].float().transpose(1, 2)).transpose(0, 1)
    return out.to(s["out"].dtype).contiguous()


def _plain_expanded(s):
    case = s["case"]
    B, H, dc, dn = case["B"], case["heads"], case["dc"], case["dn"]
    seq, i, q, n = _places(s)
    rows = _rows(s)
    both = torch.matmul(rows[..., :dc].reshape(-1, dc), s["w_kv"].float().flatten(0, 1).t())
    both = both.view(B, -1, H, dn + case["dv"]).transpose(1, 2)
    padded = torch.zeros((B, s["max_q"], H, dn + case["dr"]), device="cuda")
    padded[seq, i] = s["q"].float()
    padded = padded.transpose(1, 2)
    z = torch.matmul(padded[..., :dn], both[..., :dn].transpose(2, 3))
    z += torch.matmul(padded[..., dn:], rows[:, None, :, dc:].transpose(2, 3))
    z *= s["scale"]
    p = _softmax(z, _visible(s, seq, i, q, n)[:, None])
    out = torch.matmul(p, both[..., dn:]).transpose(1, 2)[seq, i]
    return out.to(s["out"].dtype).contiguous()


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=1)
def _context():
    import quantized_moe_expert_sigmoid_amd as moe
    return moe, moe.MoeCtx(torch.cuda.current_device())


@functools.lru_cache(maxsize=256)
def _config(heads, dc, dr, dn, dv, dtype, page, scale):
    moe, _ = _context()
    return moe.LatentCfg(heads, dc, dr, dn, dv, DTYPES[dtype], page, scale)


def _own(s):
    moe, ctx = _context()
    c = s["case"]
    cfg = _config(c["heads"], c["dc"], c["dr"], c["dn"], c["dv"], c["dtype"], c["page"], s.get("scale", 1.0))
    q, dn = s["q"], c["dn"]
    if c["op"] == "append":
        moe.moe_latent_append(ctx, cfg, s["kv"], s["turn"], s["pos"], s["slots"], s["cache"], norm_w=s["norm_w"],
                              eps=EPS, q_rope=q[..., dn:], q_rope_out=s["q_rope"])
        return {"cache": s["cache"], "q_rope": s["q_rope"]}
    if c["op"] == "prompt":
        return moe.moe_latent_prompt(ctx, cfg, q[..., :dn], q[..., dn:], s["w_kv"], s["cache"], s["table"],
                                     s["q_start"], s["kv_len"], s["n_kv"], s["out"])
    return moe.moe_latent_attend(ctx, cfg, q[..., :dn], q[..., dn:], s["w_kt"], s["w_kv"], s["cache"], s["table"],
                                 s["q_start"], s["kv_len"], s["max_q"], s["out"], tree=s["tree"])


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "append":
        return _plain_append(state)
    return _plain_expanded(state) if state["case"]["op"] == "prompt" else _plain_absorbed(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    dc, dr, dn = case["dc"], case["dr"], case["dn"]
    page = case["page"]
    if case["op"] == "append":
        kv, q = s["kv"].double(), s["q"].double()[..., dn:]
        c = kv[:, :dc] / torch.sqrt(kv[:, :dc].square().sum(1, keepdim=True) / dc + EPS) * s["norm_w"].double()
        t = torch.view_as_complex(s["turn"].double())[s["pos"].long()]
        k = torch.view_as_real(torch.view_as_complex(kv[:, dc:].reshape(-1, dr // 2, 2)) * t).flatten(1)
        qr = torch.view_as_real(torch.view_as_complex(q.reshape(*q.shape[:2], dr // 2, 2)) * t[:, None]).flatten(2)
        cache = s["cache"].double()
        flat = cache.view(-1, dc + dr)
        for t0 in torch.nonzero(s["slots"] >= 0).flatten().split(4096):
            flat[s["slots"][t0]] = torch.cat([c, k], 1)[t0]
        return {"cache": cache, "q_rope": qr}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    start, n = s["q_start"].tolist(), s["kv_len"].tolist()
    for b in range(case["B"]):
        lo, hi = start[b], start[b + 1]
        j = torch.arange(n[b], device="cuda")
        rows = s["cache"][s["table"][b, j // page].long(), j % page].double()
        first = n[b] - (hi - lo)
        seen = torch.ones((hi - lo, n[b]), dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen[:, first:] = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device="cuda").tril()
        else:
            bits = torch.arange(hi - lo, device="cuda")
            seen[:, first:] = ((s["tree"][lo:hi, None] >> bits) & 1).bool()
        step = max(1, min(case["heads"], int(2e9 / (8 * n[b] * (dn + case["dv"] + 2 * (hi - lo))))))
        for h in range(0, case["heads"], step):
            w = s["w_kv"][h:h + step].double()
            key = torch.matmul(rows[None, :, :dc], w[:, :dn].transpose(1, 2))
            val = torch.matmul(rows[None, :, :dc], w[:, dn:].transpose(1, 2))
            q = s["q"][lo:hi, h:h + step].double().transpose(0, 1)
            z = torch.matmul(q[..., :dn], key.transpose(1, 2)) + torch.matmul(q[..., dn:], rows[None, :, dc:].transpose(1, 2))
            p = torch.softmax((z * s["scale"]).masked_fill(~seen, -math.inf), dim=-1)
            out[lo:hi, h:h + step] = torch.matmul(p, val).transpose(0, 1)
    return out
