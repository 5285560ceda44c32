"""How the absorbed form deals its work to the workgroups (csrc/latent_plan.h,
compiled for the host): every cache tile of every row tile exactly once, every
joined row tile from the right partial results, and the right places in
sequences of more than 2^31 units."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.latent_plan import plan, up

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "latent_plan.h"
extern "C" void shares(int n_wg, int B, const int64_t *start, const int *rows, const int *k, int64_t all, int64_t per,
                       int piece, int over, int *wg, int64_t *shared) {
  for (int w = 0; w < n_wg; ++w) {
    WgDesc d{};
    TileDesc t{};
    const int64_t v = w * per;
    if (v < all) {
      const int b = latent_last_at_or_below(start, B, v);
      d.b = b;
      latent_share(w, v, all, per, piece, over, b, start[b], rows[b], k[b], &d, &t);
    }
    const int o[4] = {d.b, d.mt, d.at, d.n};
    for (int i = 0; i < 4; ++i) wg[4 * w + i] = o[i];
    const int64_t s[6] = {t.b, t.mt, t.w0, t.n, t.step, t.u0};
    for (int i = 0; i < 6; ++i) shared[6 * w + i] = s[i];
  }
}
extern "C" int64_t div_up(int64_t x, int64_t y) { return latent_div_up(x, y); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "shim.cpp").write_text(SHIM)
    so = str(at / "shim.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I",
                    os.path.join(ROOT, "quantized_moe_expert_sigmoid_amd", "csrc"), str(at / "shim.cpp"), "-o", so],
                   check=True)
    lib = ctypes.CDLL(so)
    lib.div_up.restype = ctypes.c_int64
    lib.div_up.argtypes = [ctypes.c_int64, ctypes.c_int64]
    return lib


def shares(host, n_wg, rows, k, piece, over):
    """(per, workgroups' (b, mt, at, n), shared row tiles' (b, mt, w0, n, step, u0))."""
    B = len(rows)
    units = [r * (up(c, piece) if piece else c + over) for r, c in zip(rows, k)]
    start, at = [], 0
    for u in units:
        start.append(at)
        at += u
    per = 1 if piece else max(up(at, n_wg), 1)
    wg, shared = (ctypes.c_int * (4 * n_wg))(), (ctypes.c_int64 * (6 * n_wg))()
    host.shares(n_wg, B, (ctypes.c_int64 * B)(*start), (ctypes.c_int * B)(*rows), (ctypes.c_int * B)(*k),
                ctypes.c_int64(at), ctypes.c_int64(per), piece, over, wg, shared)
    return per, start, at, [tuple(wg[4 * w:4 * w + 4]) for w in range(n_wg)], \
        [t for t in (tuple(shared[6 * w:6 * w + 6]) for w in range(n_wg)) if t[3]]


def check(host, n_wg, rows, k, piece, over):
    per, _, _, wg, shared = shares(host, n_wg, rows, k, piece, over)
    done, parts = {}, {}  # whole row tiles; (slot) -> row tile and its cache tiles
    for w, (b, mt, at, left) in enumerate(wg):
        first = True
        while left > 0:  # as the kernel walks
            if rows[b]:
                units = min(left, k[b] + over - at)
                lo, hi = max(at - over, 0), max(at + units - over, 0)
                if hi > lo:
                    if hi - lo == k[b]:
                        assert (b, mt) not in done
                        done[b, mt] = k[b]
                    else:
                        slot = 2 * w + (0 if first else 1)
                        assert slot not in parts
                        parts[slot] = (b, mt, lo, hi)
                left -= units
            first, at, mt = False, 0, mt + 1
            if mt >= rows[b]:
                mt, b = 0, b + 1
    for b, mt, w0, n, step, u0 in shared:
        got = []
        for i in range(n):
            w = w0 + i * step
            got.append(parts.pop(2 * w + (0 if w * per >= u0 else 1)))
        assert all(g[:2] == (b, mt) for g in got) and (b, mt) not in done
        ranges = sorted(g[2:] for g in got)
        assert ranges[0][0] == 0 and ranges[-1][1] == k[b]
        assert all(x[1] == y[0] for x, y in zip(ranges, ranges[1:]))
        done[b, mt] = k[b]
    assert not parts
    assert len(done) == sum(rows)


def test_every_tile_once(host):
    rng = random.Random(5)
    for _ in range(400):
        B = rng.choice([1, 2, 3, 7, 40, 200])
        q = [rng.choice([0, 1, 1, 2, 5, rng.randint(0, 64), rng.randint(0, 300 // B + 1)]) for _ in range(B)]
        n = [x + rng.choice([0, 0, rng.randint(0, 40), rng.randint(0, 3000 // B + 1), rng.randint(0, 20000 // B)])
             for x in q]
        H, dc, n_cu = rng.choice([1, 5, 16, 33, 64, 128]), rng.choice([128, 256, 512]), rng.choice([8, 64, 256])
        how = plan(q, n, H, dc, n_cu)
        rows, k = [up(x * H, how["rows"]) for x in q], [max(1, up(x, 32)) for x in n]
        if sum(rows) == 0:
            continue
        check(host, how["n_wg"], rows, k, how["piece"], how["over"])


@pytest.mark.parametrize("over", [0, 12])
def test_even_runs_of_any_sizes(host, over):
    rng = random.Random(6)
    for _ in range(300):
        B, n_wg = rng.randint(1, 30), rng.choice([8, 16, 64])
        rows = [rng.choice([0, 1, rng.randint(0, 9)]) for _ in range(B)]
        k = [rng.choice([1, 2, rng.randint(1, 12), rng.randint(1, 400)]) for _ in range(B)]
        if sum(rows):
            check(host, n_wg, rows, k, 0, over)


@pytest.mark.parametrize("rows, k", [([2 ** 20], [2 ** 13]), ([5, 2 ** 18, 3], [700, 2 ** 14, 9]),
                                     ([2 ** 16 + 3, 2 ** 20], [2 ** 15 + 1, 2 ** 12 + 7]), ([2 ** 22], [2 ** 16])])
@pytest.mark.parametrize("over", [0, 12])
def test_places_beyond_31_bits(host, rows, k, over):
    """Each workgroup's row tile and place, and the joined row tiles, from the numbering itself."""
    n_wg = 256
    per, start, total, wg, shared = shares(host, n_wg, rows, k, 0, over)
    assert total > 2 ** 31 and per < 2 ** 31
    named = {}
    for w, (b, mt, at, n) in enumerate(wg):
        v = w * per
        want = max(i for i in range(len(rows)) if start[i] <= v)
        assert (b, (mt, at)) == (want, divmod(v - start[want], k[want] + over)) and n == min(per, total - v)
        assert mt < rows[b]
        u0 = v - at
        if at > over and (u0 + over) // per == w - 1:
            named[b, mt] = (w - 1, (u0 + over + k[b] - 1) // per - (w - 1) + 1, 1, u0)
    assert {t[:2]: t[2:] for t in shared} == named


def test_div_up(host):
    for x, y in [(0, 1), (1, 1), (7, 2), (2 ** 31 - 1, 1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 256), (2 ** 40 + 1, 256),
                 (2 ** 31 - 300, 256), (2 ** 31 - 256, 256), (2 ** 31 - 257, 256), (5, 2 ** 40)]:
        assert host.div_up(x, y) == up(x, y)
