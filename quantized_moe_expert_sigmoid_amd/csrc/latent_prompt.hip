// Latent attention, expanded form: keys and values of every head computed from
// the cache, then causal attention.
//
// As in the absorbed form a lane keeps one query row: S^T = K Q^T, P^T, O^T +=
// V^T P^T with v_mfma_f32_32x32x16 (see latent_attend.hip for the layouts). A
// workgroup takes 256 (or 128) tokens of one head, 32 a wave, two waves a SIMD, so
// that one wave's exponentials run under the other's products; its tiles of keys and
// values come into LDS by asynchronous loads, one being read, the others in
// flight.
//
// Statistics, scores and sums are fp32; the expanded keys and values and P^T are
// rounded to the element type, since the products read elements and 32 bits would
// double the workspace's bytes (0.0028 relative in bf16, 0.0017 of it the output's
// own rounding).
//
// Measured: 4096 tokens of 128 heads, keys of 128 + 64, values of 128: rows 7 us,
// expansion 163 us (latent_gemm.hip), attention 745 to 760 us by machine, 687 GFLOP
// at 915 TFLOP/s; of 64 heads, keys of 192 + 64, values of 256: expansion 143 us,
// attention 607 us, 550 GFLOP at 905 TFLOP/s, with 25 registers of a lane spilled.
// The library's product of 8192 x 8192 x 8192 reaches 1350. The products bound it,
// at the clock (1.7 to 2.1 GHz) that they leave.
#include "latent.h"

#include <algorithm>

namespace {

// The plan: off[b] = first expanded row of sequence b (B + 1 entries), the
// row tiles. Sequences that do not fit n_kv rows are
// reported and left out (off = -1).
struct PromptTile {
  int b, i0;
};
struct PromptWs {
  int32_t *off;      // [B + 1]
  int32_t *n_tiles;
  PromptTile *tile;
  uint16_t *c;       // [n_kv][dc] latents
  uint16_t *kr;      // [n_kv][dr] rotary keys
  uint16_t *x;       // [H][n_kv][dn + dv] keys and values
  int64_t n_kv;
  int tile_rows;     // query tokens of a row tile
  int max_tiles;     // row tiles of T tokens at most; starts that go back (reported) could ask for more
};

// The sequences' cache rows one after another (a wave a row, 16 bytes a lane, the
// rotary part by the first lanes again). Every workgroup sums the lengths by
// itself; the first one also writes the plan: row tiles by falling number of
// tokens they see, so that the workgroups that take them end together.
__global__ __launch_bounds__(256) void prompt_rows_kernel(LatentArgs a, PromptWs ws) {
  constexpr int kPer = 4;  // sequences a thread
  constexpr int kSort = 256;
  __shared__ int off_s[1024], tmp[8], sees[kSort];
  __shared__ PromptTile tile_s[kSort];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool first = blockIdx.x == 0;
  int len[kPer], nt[kPer], nq[kPer], sum = 0, tsum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    const LatentSeq s = b < a.B ? latent_seq(a, b) : LatentSeq{};
    len[i] = s.len;
    nq[i] = s.nq;
    nt[i] = (s.nq + ws.tile_rows - 1) / ws.tile_rows;
    sum = (int)min((int64_t)sum + len[i], (int64_t)1 << 30);  // a total that saturates is above n_kv anyway
    tsum += nt[i];
  }
  int at = sum, tat = tsum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(at, o, 64), y = __shfl_up(tat, o, 64);
    at = lane >= o ? (int)min((int64_t)at + x, (int64_t)1 << 30) : at;
    tat += lane >= o ? y : 0;
  }
  if (lane == 63) {
    tmp[wave] = at;
    tmp[4 + wave] = tat;
  }
  __syncthreads();
  int64_t before = 0;
  int tbefore = 0, n_tiles = 0;
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? tmp[w] : 0;
    tbefore += w < wave ? tmp[4 + w] : 0;
    n_tiles += tmp[4 + w];
  }
  const bool sorted = n_tiles <= min(kSort, ws.max_tiles);
  int64_t o = before + at - sum;
  int t = tbefore + tat - tsum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    const bool fits = o + len[i] <= ws.n_kv;
    off_s[b] = fits ? (int)o : -1;
    if (first && b < a.B) {
      if (!fits) atomicOr(a.err, (uint32_t)ERRF_LATENT);
      ws.off[b] = fits ? (int)o : -1;
      if (!sorted)
        for (int k = 0; k < nt[i] && t + k < ws.max_tiles; ++k) ws.tile[t + k] = PromptTile{b, k * ws.tile_rows};
      else
        for (int k = 0; k < nt[i]; ++k) {
          tile_s[t + k] = PromptTile{b, k * ws.tile_rows};
          sees[t + k] = max(0, min(len[i], len[i] - nq[i] + min(nq[i], (k + 1) * ws.tile_rows)));
        }
      // the last sequence that fits ends the expanded rows
      if (fits && b + 1 == a.B) ws.off[a.B] = (int)(o + len[i]);
      if (!fits && o <= ws.n_kv) ws.off[a.B] = (int)o;
    }
    o += len[i];
    t += nt[i];
  }
  if (first && tid == 0) *ws.n_tiles = min(n_tiles, ws.max_tiles);
  __syncthreads();
  if (first && sorted && tid < n_tiles) {
    const int mine = sees[tid];
    int rank = 0;
    for (int x = 0; x < n_tiles; ++x) rank += sees[x] > mine || (sees[x] == mine && x < tid);
    ws.tile[rank] = tile_s[tid];
  }
  // rows, spread over all workgroups
  for (int b = 0; b < a.B; ++b) {
    const int off = off_s[b], n = (b + 1 < 1024 && off_s[b + 1] >= 0 && b + 1 < a.B) ? off_s[b + 1] - off : -1;
    if (off < 0) continue;
    const int rows = n >= 0 ? n : latent_seq(a, b).len;
    const uint16_t *cache = static_cast<const uint16_t *>(a.cache) + 8 * lane;
    // workgroup and wave take rows off + j = id (mod all), so that short sequences use different ones
    const int all = gridDim.x * 4, id = blockIdx.x * 4 + wave;
    for (int j = (id - off % all + all) % all; j < rows; j += all) {
      const uint16_t *row = cache + latent_row(a, b, j) * (a.dc + a.dr);
      if (8 * lane < a.dc)
        *reinterpret_cast<u32x4 *>(ws.c + (int64_t)(off + j) * a.dc + 8 * lane) = *reinterpret_cast<const u32x4 *>(row);
      if (8 * lane < a.dr)
        *reinterpret_cast<u32x4 *>(ws.kr + (int64_t)(off + j) * a.dr + 8 * lane) =
            *reinterpret_cast<const u32x4 *>(row + a.dc);
    }
  }
}

__device__ __forceinline__ int swz(int token) { return ((token >> 1 & 1) << 2) | (token >> 2 & 3); }

template <int DN, int DR, int DV, int W>
struct Prompt {
  static constexpr int kTB = DV > 128 || W == 4 ? 1 : 2, kNT = 32 * kTB;  // 32 or 64 tokens a tile
  static constexpr int kPN = DN / 64, kPK = kPN + 1, kPV = DV / 64;  // panels of 64 columns: keys (rotary part last), values
  static constexpr int kPanelB = kNT * 128, kTileB = (kPK + kPV) * kPanelB;
  static constexpr int kBufs = 3;
  static constexpr int kLoads = (kPK + kPV) * kNT / 8 / W;  // of a wave and tile
  static constexpr int kStep = W * 8 / kNT;                // waves that share a block of 8 tokens
  static constexpr int kKS = (DN + DR) / 16, kNB = DV / 32;
  static_assert(kBufs * kTileB <= 160 << 10 && (kPK + kPV) % kStep == 0, "");
};

template <typename E, int DN, int DR, int DV, int W>
__global__ __launch_bounds__(64 * W, W / 4) void latent_prompt_kernel(LatentArgs a, PromptWs ws, float c2,
                                                                      uint32_t flip) {
  using C = Prompt<DN, DR, DV, W>;
  constexpr int kRows = 32 * W;
  constexpr int kNT = C::kNT, kTB = C::kTB, kNB = C::kNB, DX = DN + DV, kAhead = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kBufs * C::kTileB];
  // an XCD (ids go round the 8 of them) takes whole heads, so that workgroups that share keys share an L2; the tiles
  // that see the most go first, of all its heads (head by head left 23% of the CUs' time at the end idle)
  const int nt = uniform(*ws.n_tiles), per_xcd = (a.H + 7) / 8, id = blockIdx.x >> 3;
  const int h = (blockIdx.x & 7) + 8 * (id % per_xcd);
  if (id / per_xcd >= nt || h >= a.H) return;
  const PromptTile pt = ws.tile[id / per_xcd];
  const int b = uniform(pt.b), i0 = uniform(pt.i0), off0 = uniform(ws.off[b]);
  if (off0 < 0) return;
  const LatentSeq r = latent_seq(a, b);
  const LatentSeq s{uniform(r.t0), uniform(r.nq), uniform(r.len), uniform(r.before)};
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int qi = i0 + wave * 32 + l32;
  const bool live = qi < s.nq;
  const int t = s.t0 + min(qi, s.nq - 1);
  const int last = min(s.nq, i0 + kRows) - 1;                          // the workgroup's last query
  const int n = (max(0, min(s.len, s.before + last + 1)) + kNT - 1) / kNT;  // tiles it sees
  // nothing from position w_end on is seen by the wave
  const int w_end = min(s.len, s.before + min(s.nq, i0 + wave * 32 + 32));
  const bool any = i0 + wave * 32 < s.nq;

  u16x8 q[C::kKS];
  {
    const uint16_t *q1 = static_cast<const uint16_t *>(a.q_nope) + t * a.nope_t + h * a.nope_h + 8 * hl;
    const uint16_t *q2 = static_cast<const uint16_t *>(a.q_rope) + t * a.rope_t + h * a.rope_h + 8 * hl;
#pragma unroll
    for (int k = 0; k < C::kKS; ++k) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(16 * k < DN ? q1 + 16 * k : q2 + (16 * k - DN));
      v ^= flip;
      q[k] = __builtin_bit_cast(u16x8, v);
    }
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int ld_row = lane >> 3, rb = wave & (kNT / 8 - 1);  // the wave's block of 8 tokens
  const int ld_unit = (lane & 7) ^ swz((8 * rb + ld_row) & 15);
  const uint8_t *xh = reinterpret_cast<const uint8_t *>(ws.x) + ((int64_t)h * ws.n_kv + off0) * (DX * 2);
  const uint8_t *kr = reinterpret_cast<const uint8_t *>(ws.kr) + (int64_t)off0 * (DR * 2);
  // tile i: prepared, then loaded panel by panel; positions behind the last row repeat it, behind the last tile
  // nothing is loaded (but counted)
  const uint8_t *x_src = nullptr, *k_src = nullptr;
  uint32_t to = 0;
  int on = 0;
  auto prepare = [&](int i) {
    const int j0 = uniform(min(i * kNT + 8 * rb, max(s.len - 1, 0) & ~7));
    const int row = min(ld_row, s.len - 1 - j0);
    x_src = uniform(xh + (int64_t)j0 * (DX * 2)) + (row * (DX * 2) + ld_unit * 16);
    k_src = uniform(kr + (int64_t)j0 * (DR * 2)) + (row * (DR * 2) + (DR == 64 ? ld_unit : ld_unit & 3) * 16);
    to = uniform(lds0 + (i % C::kBufs) * C::kTileB + rb * 1024);
    on = uniform(i < n ? -1 : 0);
  };
  // panels: keys, rotary keys, values; with tiles of 32 tokens two waves share a block of 8 and take every other one
  constexpr int kStep = C::kStep;
  const int odd_wave = kStep == 1 ? 0 : uniform(wave >> 2);
  auto load = [&](auto i) {
    constexpr int g = i * kStep;
    if constexpr (kStep == 1) {
      if constexpr (g == C::kPN)
        lds_load16<0>(k_src, to + g * C::kPanelB, on);
      else
        lds_load16<(g < C::kPN ? g : g - 1) * 128>(x_src, to + g * C::kPanelB, on);
    } else {
      const int gg = g + odd_wave;
      const uint8_t *p = gg == C::kPN ? k_src : x_src + (gg < C::kPN ? gg : gg - 1) * 128;
      lds_load16<0>(p, uniform(to + gg * C::kPanelB), on);
    }
  };
  int k_off[4], v_off[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) k_off[i] = l32 * 128 + (((2 * i + hl) ^ swz(l32 & 15)) << 4);
  const int vt = 4 * hl + ((lane & 15) >> 2);
#pragma unroll
  for (int h8 = 0; h8 < 2; ++h8)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      v_off[h8][p] = (vt + 8 * h8) * 128 +
                     (((4 * p + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swz(vt + 8 * h8)) << 4) + (lane & 1) * 8;

  f32x16 acc[kNB];
#pragma unroll
  for (int i = 0; i < kNB; ++i) acc[i] = f32x16{};
  float m = -__builtin_inff(), l = 0.0f;
  int cleared = s.len;  // first position of a tile whose values were partly cleared
  if (n > 0)
#pragma unroll
    for (int i = 0; i < C::kBufs - 1; ++i) {
      prepare(i);
      static_for<0, C::kLoads>(load);
    }
  for (int it = 0; it < n; ++it) {
    WAIT_VM((C::kBufs - 2) * C::kLoads);
    asm volatile("s_barrier" ::: "memory");
    prepare(it + C::kBufs - 1);
    const int j0 = it * kNT;
    const bool masked = j0 + kNT > s.before + i0 + 1;  // the same in every wave: some row of the workgroup does not see all
    if (!masked && !any) {
      static_for<0, C::kLoads>(load);
      continue;
    }
    uint8_t *kv = lds + (it % C::kBufs) * C::kTileB, *vv = kv + C::kPK * C::kPanelB;
    // Operands are read kAhead products before they are used, the next tile's loads go in between, and the order is
    // held (see latent_attend.hip).
    constexpr int kZ = C::kKS * kTB, kV = 2 * kTB * kNB;  // products
    constexpr int kEvery = kZ >= 2 * C::kLoads ? 2 : 1;
    static_assert(kZ / kEvery >= C::kLoads, "every load has its place");
    auto k_read = [&](int i) {
      const int k = i / kTB, tb = i % kTB;
      return *reinterpret_cast<const u16x8 *>(kv + k_off[k & 3] + (k >> 2) * C::kPanelB + tb * 32 * 128);
    };
    auto v_read = [&](int i) {
      const int ks = i / kNB, nb = i % kNB;
      const uint8_t *src = vv + (nb >> 1) * C::kPanelB + ks * 16 * 128;
      const u16x4 lo = lds_read_tr(src + v_off[0][nb & 1]), hi = lds_read_tr(src + v_off[1][nb & 1]);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    f32x16 z[kTB];
#pragma unroll
    for (int tb = 0; tb < kTB; ++tb) z[tb] = f32x16{};
    u16x8 ring[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ring[i] = k_read(i);
    __builtin_amdgcn_sched_barrier(0);
    static_for<0, kZ>([&](auto i) {
      z[i % kTB] = E::mfma(ring[i % kAhead], q[i / kTB], z[i % kTB]);
      if (i + kAhead < kZ)
        ring[i % kAhead] = k_read(i + kAhead);
      else if (i + kAhead - kZ < kV)
        ring[i % kAhead] = v_read(i + kAhead - kZ);
      if constexpr (i % kEvery == kEvery - 1 && i / kEvery < C::kLoads) load(std::integral_constant<int, i / kEvery>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    if (masked) {
      // tokens the lane's row sees, as bits
      const uint64_t vis64 = [&] {
        const int c = min(max(min(s.before + qi + 1, s.len) - j0, 0), 64);
        return c == 64 ? ~0ull : (1ull << c) - 1;
      }() >> (4 * hl);
      // A value that is NaN or infinite would reach the rows that do not see it as 0 x NaN or 0 x inf. Its score does not
      // tell: keys and values are products of their own, and a value may leave the elements' range where the score stays
      // finite. So the values themselves are looked at, 8 to 32 of them a lane; in the rare tile that has such elements
      // they are cleared here, and added at the end for the rows that see them.
      const int row = lane & (kNT - 1);
      auto unit = [&](int c) {
        return reinterpret_cast<u32x4 *>(vv + (c >> 3) * C::kPanelB + row * 128 + (((c & 7) ^ swz(row & 15)) << 4));
      };
      // the sign bits of elements whose exponent bits are all set: one more at their low end carries into it
      auto flags = [](uint32_t x) { return ((x & E::kExp * 0x10001u) + (E::kExp & -E::kExp) * 0x10001u) & 0x80008000u; };
      auto any_flag = [&](u32x4 x) { return (flags(x[0]) | flags(x[1]) | flags(x[2]) | flags(x[3])) != 0; };
      constexpr int kShare = W * 64 / kNT;  // units looked at at a time
      static_assert(DV / 8 % kShare == 0, "");
      const int c0 = wave * (64 / kNT) + lane / kNT;
      bool broken = false;
#pragma unroll
      for (int c = 0; c < DV / 8; c += kShare) broken |= any_flag(*unit(c + c0));
      if (__syncthreads_or(broken)) {
        cleared = min(cleared, j0);
        broken = false;
#pragma unroll 1
        for (int c = 0; c < DV / 8; ++c) broken |= any_flag(*unit(c));
        const uint64_t bad = __ballot(broken);  // of 32 tokens: twice
        __syncthreads();
#pragma unroll 1
        for (int c = c0; c < DV / 8; c += kShare) {
          u32x4 x = *unit(c);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] &= ~((flags(x[e]) >> 15) * 0xffffu);
          *unit(c) = x;
        }
        // a row that sees one behind a score of -inf: 0 x inf
#pragma unroll
        for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 32 * tb + 8 * (i >> 2) + (i & 3);
            l = ((vis64 & (bad >> (4 * hl))) >> j & 1) & (z[tb][i] == -__builtin_inff()) ? __builtin_nanf("") : l;
          }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAhead && i < kV; ++i) ring[(kZ + i) % kAhead] = v_read(i);  // once more
      }
#pragma unroll
      for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          z[tb][i] = (vis64 >> (32 * tb + 8 * (i >> 2) + (i & 3))) & 1 ? z[tb][i] : -__builtin_inff();
    }
    if (j0 >= w_end) continue;  // nothing of this tile is seen by the wave
    float top = z[0][0];
#pragma unroll
    for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, z[tb][i]);
    top = max_halves(top) * c2;
    // the reference follows the maximum when that has grown by 2^8 (see latent_attend.hip)
    if (__any(top > m + 8.0f)) {
      const float mn = fmaxf(m, top);
      const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < kNB; ++i) acc[i] *= f;
    }
    const float base = m == -__builtin_inff() ? 0.0f : -m;
    // the weights of 16 tokens at a time, each group's between the products of the group before
    auto weight = [&](int i) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z[i / 16][i % 16], c2, base));
      l += e;
      return e;
    };
    f32x8 e;
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = weight(i);
    u16x8 p = E::from_f32x8(e);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int ks = i / kNB, nb = i % kNB;
      if (ks && nb == 0) p = E::from_f32x8(e);
      acc[nb] = E::mfma(ring[(kZ + i) % kAhead], p, acc[nb]);
      if (i + kAhead < kV) ring[(kZ + i) % kAhead] = v_read(i + kAhead);
      if (ks + 1 < 2 * kTB)
#pragma unroll
        for (int j = nb * 8 / kNB; j < (nb + 1) * 8 / kNB; ++j) e[j] = weight(8 * (ks + 1) + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  l += __shfl_xor(l, 32, 64);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t *o = static_cast<uint16_t *>(a.out) + ((int64_t)t * a.H + h) * DV + 8 * hl;
#pragma unroll
  for (int i = 0; i < kNB; ++i) {
    f32x16 r = acc[i] * inv;
    // what was cleared, for the rows that see it: any weight times NaN or an infinity is that again
#pragma unroll 1
    for (int j = cleared; j < w_end; ++j) {
      const uint8_t *v = xh + (int64_t)j * (DX * 2) + (DN + 32 * i) * 2 + 8 * hl;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const u16x4 x = *reinterpret_cast<const u16x4 *>(v + 16 * g);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          r[4 * g + e] += (j <= s.before + qi) & ((x[e] & E::kExp) == E::kExp) ? E::to_f32(x[e]) : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const u32x4 v = rows8<E>(f32x4{r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]},
                               f32x4{r[4 * j + 4], r[4 * j + 5], r[4 * j + 6], r[4 * j + 7]});
      if (live) *reinterpret_cast<u32x4 *>(o + 32 * i + 8 * j) = v;
    }
  }
}

template <typename E, int DN, int DR, int DV, int W>
moe_status launch(moe_ctx *ctx, const LatentArgs &a, int64_t n_kv) {
  constexpr int kRows = 32 * W;
  const int64_t tiles = a.T / kRows + a.B;  // at most: every sequence adds one tile that is not full
  MoeLayout lay;
  const size_t o_off = lay.take(4 * (size_t)(a.B + 1)), o_nt = lay.take(4), o_tile = lay.take(sizeof(PromptTile) * tiles),
               o_c = lay.take(2 * (size_t)n_kv * a.dc), o_kr = lay.take(2 * (size_t)n_kv * DR),
               o_x = lay.take(2 * (size_t)n_kv * a.H * (DN + DV));
  void *scr = nullptr;
  moe_status st = moe_scratch(ctx, lay.size, &scr);
  if (st) return st;
  char *p = static_cast<char *>(scr);
  const PromptWs ws{reinterpret_cast<int32_t *>(p + o_off),  reinterpret_cast<int32_t *>(p + o_nt),
                    reinterpret_cast<PromptTile *>(p + o_tile), reinterpret_cast<uint16_t *>(p + o_c),
                    reinterpret_cast<uint16_t *>(p + o_kr),  reinterpret_cast<uint16_t *>(p + o_x),
                    n_kv,
                    kRows,
                    (int)tiles};
  const unsigned row_blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n_kv + 3) / 4, 1024));
  hipLaunchKernelGGL(prompt_rows_kernel, dim3(row_blocks), dim3(256), 0, ctx->stream, a, ws);
  MOE_CHECK_LAUNCH("prompt_rows_kernel");
  if (n_kv > 0) {
    const ExpandGemm expand{ws.c, static_cast<const uint16_t *>(a.w_kv), ws.x, ws.off + a.B, (int)n_kv, a.H, DN + DV,
                            a.dc};
    if ((st = launch_expand_gemm(ctx, E::kDtype, expand))) return st;
  }
  const float c2 = latent_c2(a.scale);
  hipLaunchKernelGGL((latent_prompt_kernel<E, DN, DR, DV, W>), dim3((unsigned)(tiles * ((a.H + 7) / 8) * 8)), dim3(64 * W), 0,
                     ctx->stream, a, ws, c2, a.scale < 0 ? 0x80008000u : 0u);
  MOE_CHECK_LAUNCH("latent_prompt_kernel");
  return MOE_OK;
}

template <typename E, int DR>
moe_status pick(moe_ctx *ctx, const LatentArgs &a, int64_t n_kv) {
  // row tiles of 256 tokens read keys and values half as often; of 128 where those would leave CUs without work
  if ((a.T + 255) / 256 * (int64_t)a.H > ctx->n_cu)
    return a.dn == 64    ? launch<E, 64, DR, 64, 8>(ctx, a, n_kv)
           : a.dn == 128 ? launch<E, 128, DR, 128, 8>(ctx, a, n_kv)
                         : launch<E, 192, DR, 256, 8>(ctx, a, n_kv);
  return a.dn == 64    ? launch<E, 64, DR, 64, 4>(ctx, a, n_kv)
         : a.dn == 128 ? launch<E, 128, DR, 128, 4>(ctx, a, n_kv)
                       : launch<E, 192, DR, 256, 4>(ctx, a, n_kv);
}

}  // namespace

moe_status launch_latent_prompt(moe_ctx *ctx, int dtype, const LatentArgs &a, int64_t n_kv) {
  if (dtype == MOE_BF16) return a.dr == 64 ? pick<Bf16, 64>(ctx, a, n_kv) : pick<Bf16, 32>(ctx, a, n_kv);
  return a.dr == 64 ? pick<Fp16, 64>(ctx, a, n_kv) : pick<Fp16, 32>(ctx, a, n_kv);
}
