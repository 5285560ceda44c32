"""One latent-attention layer with its paged cache, over the C ABI.

Every call appends the new tokens (moe_latent_append) and attends to the
sequences' cached rows: moe_latent_attend for single tokens and drafted trees,
moe_latent_prompt for prompts. Everything runs on the context's stream. A call
starts after the work that the caller's current stream holds, and that stream
waits for the call, so that tensors made and used on it need no further
ordering. The sequences' pages and lengths are kept on the host and sent with
each call.
"""
from __future__ import annotations

import itertools

import torch

from . import MOE_ENOMEM, LatentCfg, MoeCtx, MoeError, moe_latent_append, moe_latent_attend, moe_latent_prompt

MAX_EXPANDED = 1 << 24  # cached rows that moe_latent_prompt takes


class LatentAttention:
    """n_pages pages of page_size rows serve all sequences; a row holds a
    token's normed latent and rotated key. Positions run from 0 to
    max_positions - 1."""

    def __init__(self, ctx: MoeCtx, n_heads: int, d_latent: int = 512, d_rope: int = 64, d_nope: int = 128,
                 d_v: int = 128, n_pages: int = 256, page_size: int = 64, max_positions: int = 8192,
                 rope_base: float = 10000.0, eps: float = 1e-6, dtype: torch.dtype = torch.bfloat16,
                 device: str = "cuda"):
        self.ctx, self.eps, self.device = ctx, eps, device
        self.cfg = LatentCfg(n_heads, d_latent, d_rope, d_nope, d_v, dtype, page_size)
        with torch.cuda.stream(ctx.stream):
            self.cache = torch.zeros((n_pages, page_size, d_latent + d_rope), dtype=dtype, device=device)
        angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * rope_base ** (
            -torch.arange(d_rope // 2, dtype=torch.float64) * 2 / d_rope)
        with torch.cuda.stream(ctx.stream):
            self.turn = torch.stack([angle.cos(), angle.sin()], dim=-1).float().to(device)
        self.w_kv = self.w_kt = self.norm_w = None
        self._free = list(range(n_pages - 1, -1, -1))
        self._pages: dict[int, list[int]] = {}
        self._len: dict[int, int] = {}
        self._next = 0

    # -- weights -----------------------------------------------------------
    def set_weights(self, w_kv, norm_w=None):
        """w_kv [H][d_nope + d_v][d_latent] (a head's key rows, then its value
        rows), norm_w [d_latent] or None (latents enter the cache as they are).
        The layer keeps copies: what is given may be overwritten or freed after
        the call."""
        c, stream, caller = self.cfg, self.ctx.stream, torch.cuda.current_stream(self.cache.device)
        w_kv, norm_w = torch.as_tensor(w_kv).detach(), None if norm_w is None else torch.as_tensor(norm_w).detach()
        shape = (c.n_heads, c.d_nope + c.d_v, c.d_latent)
        if w_kv.shape != shape:
            raise ValueError(f"w_kv shape {tuple(w_kv.shape)} != {shape}")
        if norm_w is not None and norm_w.shape != (c.d_latent,):
            raise ValueError(f"norm_w shape {tuple(norm_w.shape)} != {(c.d_latent,)}")
        stream.wait_stream(caller)  # the weights may still be on their way there
        with torch.cuda.stream(stream):
            self.w_kv = torch.empty(shape, dtype=c.dtype, device=self.device).copy_(w_kv)
            # the absorbed form's layout of the key rows
            self.w_kt = self.w_kv[:, :c.d_nope].transpose(1, 2).contiguous()
            self.norm_w = None
            if norm_w is not None:
                self.norm_w = torch.empty(c.d_latent, dtype=torch.float32, device=self.device).copy_(norm_w)
        caller.wait_stream(stream)

    # -- sequences ----------------------------------------------------------
    def new_sequence(self) -> int:
        s = self._next
        self._next += 1
        self._pages[s], self._len[s] = [], 0
        return s

    def drop_sequence(self, seq: int):
        self._free += self._pages.pop(seq)
        del self._len[seq]

    def length(self, seq: int) -> int:
        return self._len[seq]

    def _row(self, seq: int, j: int) -> int:
        p = self.cfg.page_size
        return self._pages[seq][j // p] * p + j % p

    def _room(self, need: int):
        if need > len(self._free):
            raise RuntimeError(f"latent cache: {need} pages are needed, {len(self._free)} are free")

    def _resize(self, seq: int, n: int):
        pages, p = self._pages[seq], self.cfg.page_size
        need = -(-n // p)
        self._room(need - len(pages))
        while len(pages) < need:
            pages.append(self._free.pop())
        while len(pages) > need:
            self._free.append(pages.pop())
        self._len[seq] = n

    def keep(self, seq: int, n_own: int, nodes):
        """After a call that gave `seq` n_own new tokens: keep those numbered
        `nodes` (ascending, a path of the tree), in that order, and drop the others."""
        nodes = list(nodes)
        before = self._len[seq] - n_own
        if n_own < 0 or before < 0:
            raise ValueError(f"n_own {n_own} of a sequence of {self._len[seq]} tokens")
        if any(not 0 <= v < n_own for v in nodes) or any(a >= b for a, b in zip(nodes, nodes[1:])):
            raise ValueError(f"nodes must ascend within 0..{n_own - 1}")
        flat = self.cache.view(-1, self.cache.shape[-1])
        if nodes:
            with torch.cuda.stream(self.ctx.stream):
                src = torch.tensor([self._row(seq, before + v) for v in nodes], device=self.device)
                dst = torch.tensor([self._row(seq, before + i) for i in range(len(nodes))], device=self.device)
                flat[dst] = flat[src]
        self._resize(seq, before + len(nodes))

    # -- forward --------------------------------------------------------------
    def forward(self, seqs, counts, q: torch.Tensor, kv: torch.Tensor, tree=None, depth=None) -> torch.Tensor:
        """Append counts[i] tokens to sequence seqs[i] and attend. q
        [T][H][d_nope + d_rope] and kv [T][d_latent + d_rope]: the tokens'
        projections before norm and rotation, sequence after sequence. tree: the
        tokens' visibility words (ints, bit j: own token j of the sequence) for
        drafts that branch, with depth: each token's distance in positions from
        its sequence's first new one. Returns [T][H][d_v]. A call that raises leaves
        the sequences as they were."""
        c = self.cfg
        T = sum(counts)
        if (q.shape[0] != T or kv.shape[0] != T or len(seqs) != len(counts) or len(set(seqs)) != len(seqs) or
                any(n < 0 for n in counts)):
            raise ValueError("one q and kv row a token, each sequence once")
        if (tree is None) != (depth is None):
            raise ValueError("tree and depth go together")
        if tree is not None and (len(tree) != T or len(depth) != T or max(counts, default=0) > 64 or
                                 any(int(d) < 0 for d in depth)):
            raise ValueError("a word and a depth (from 0) a token, 64 tokens a sequence at most")
        if tree is not None and any(not 0 <= int(w) < 1 << 64 for w in tree):
            raise ValueError("a token's word has 64 bits")
        if self.w_kv is None:
            raise RuntimeError("set_weights comes first")
        before = [self._len[s] for s in seqs]
        p = self.cfg.page_size
        self._room(sum(max(-(-(b + n) // p) - len(self._pages[s]), 0) for s, n, b in zip(seqs, counts, before)))
        ends = [b + (n if depth is None else 1 + max(map(int, depth[t:t + n]), default=-1))
                for n, b, t in zip(counts, before, itertools.accumulate(counts, initial=0))]
        if max(ends, default=0) > self.turn.shape[0]:
            raise ValueError(f"position {max(ends) - 1} is behind max_positions {self.turn.shape[0]}")
        try:
            return self._enqueue(seqs, counts, q, kv, tree, depth, before)
        except BaseException:
            # given back in the order that leaves the free pages as they were
            for s, b in reversed(list(zip(seqs, before))):
                self._resize(s, b)
            raise

    def _enqueue(self, seqs, counts, q, kv, tree, depth, before) -> torch.Tensor:
        """forward after its own checks: the pages of the new tokens, then the calls."""
        c = self.cfg
        T = sum(counts)
        start, pos, slot = [0], [], []
        for s, n, b in zip(seqs, counts, before):
            self._resize(s, b + n)
            first = start[-1]
            pos += [b + (i if depth is None else int(depth[first + i])) for i in range(n)]
            slot += [self._row(s, b + i) for i in range(n)]
            start.append(first + n)
        wide = max([len(self._pages[s]) for s in seqs] + [1])
        table = [self._pages[s] + [0] * (wide - len(self._pages[s])) for s in seqs]

        def send(values, dtype):
            return torch.tensor(values, dtype=dtype).to(self.device)

        stream, caller = self.ctx.stream, torch.cuda.current_stream(self.cache.device)
        out = torch.empty((T, c.n_heads, c.d_v), dtype=c.dtype, device=self.device)  # the caller's memory, its stream's
        if stream != caller:
            stream.wait_stream(caller)  # q and kv may still be in the making
        words = None
        try:
            with torch.cuda.stream(stream):
                if tree is not None:
                    words = send([int(w) - (1 << 64) if int(w) >> 63 else int(w) for w in tree], torch.int64)
                table, start_d = send(table, torch.int32).view(len(seqs), wide), send(start, torch.int32)
                kv_len = send([self._len[s] for s in seqs], torch.int32)
                q_rope = torch.empty((T, c.n_heads, c.d_rope), dtype=c.dtype, device=self.device)
                moe_latent_append(self.ctx, c, kv, self.turn, send(pos, torch.int32), send(slot, torch.int64),
                                  self.cache, norm_w=self.norm_w, eps=self.eps, q_rope=q[..., c.d_nope:],
                                  q_rope_out=q_rope)
                lengths = [self._len[s] for s in seqs]
                expanded = tree is None and self.expands(counts, lengths)
                if expanded:
                    try:
                        moe_latent_prompt(self.ctx, c, q[..., :c.d_nope], q_rope, self.w_kv, self.cache, table,
                                          start_d, kv_len, sum(lengths), out)
                    except MoeError as e:
                        if e.status != MOE_ENOMEM:
                            raise
                        expanded = False  # no room for the expanded rows: the other form needs none
                if not expanded:
                    moe_latent_attend(self.ctx, c, q[..., :c.d_nope], q_rope, self.w_kt, self.w_kv, self.cache, table,
                                      start_d, kv_len, max(counts, default=0), out, tree=words)
        finally:
            if stream != caller:
                caller.wait_stream(stream)  # which may now read out, and overwrite or free q and kv
        return out

    def expands(self, counts, lengths) -> bool:
        """Whether the expanded form can run and takes fewer products: it pays d_latent
        (d_nope + d_v) a cached row to save 2 d_latent - d_nope - d_v a query and
        row. Measured (128 heads, 2000 rows before the call; us expanded,
        absorbed): 64 tokens 133, 85; 128 tokens 139, 123 (absorbed takes 0.84 of
        the products); 256 tokens 153, 190 (1.33)."""
        c = self.cfg
        if sum(lengths) > MAX_EXPANDED:
            return False
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(counts, lengths))
        wide = c.d_latent * (c.d_nope + c.d_v)
        absorbed = pairs * (2 * c.d_latent + c.d_rope) + sum(counts) * wide
        return pairs * (c.d_nope + c.d_rope + c.d_v) + sum(lengths) * wide < absorbed
