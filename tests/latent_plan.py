"""The rules by which the absorbed form shares its work out, in Python, for tests
that have to reach a certain way of it (csrc/latent_gemm.hip, make_plan;
csrc/latent_attend.hip, pick)."""


def up(x, y):
    return -(-x // y)


def plan(q, n, H, dc, n_cu, max_q=None, tokens=32, charge=12):
    """q new tokens and n cached rows a sequence. Returns rows: rows of a row tile; n_wg: workgroups; piece: cache
    tiles of a piece (0: even runs); over: units a row tile is charged with; row_tiles; parts: the most partial
    results of one row tile."""
    max_q = max(list(q) + [1]) if max_q is None else max(max_q, 1)
    wm = 1 if max_q * H <= 32 else 2 if max_q * H <= 64 else 4
    rows, blocks = 32 * wm, dc // 32 // (4 // wm)
    n_wg = n_cu // 8 * 8 * (2 if dc < 512 and blocks <= 4 else 1)
    rt = [up(a * H, rows) for a in q]
    ct = [max(1, up(b, tokens)) for b in n]
    total, n_rows, most = sum(r * k for r, k in zip(rt, ct)), sum(rt), max([k for r, k in zip(rt, ct) if r] + [1])
    piece, even = 0, up(total, n_wg)
    if 0 < n_rows < n_wg:
        for size in range(even, min(even + min(charge, 15), up(total, n_wg - n_rows)) + 1):
            pieces = sum(r * up(k, size) for r, k in zip(rt, ct))
            if pieces <= n_wg:
                piece = max(size, most) if most - size <= pieces * rows // 4096 else size
                break
    over = charge if not piece and total >= 4 * n_wg else 0
    if piece:
        parts = max([up(k, piece) for r, k in zip(rt, ct) if r] + [1])
    else:
        per, at, parts = max(up(sum(r * (k + over) for r, k in zip(rt, ct)), n_wg), 1), 0, 1
        for r, k in zip(rt, ct):
            for _ in range(r):
                parts = max(parts, (at + over + k - 1) // per - (at + over) // per + 1)
                at += k + over
    return dict(rows=rows, n_wg=n_wg, piece=piece, over=over, row_tiles=n_rows, parts=parts)
