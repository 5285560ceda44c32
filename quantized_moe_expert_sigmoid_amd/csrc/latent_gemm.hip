// Products of the heads' expansion weights: absorbed queries, the last product
// of the absorbed form, expanded keys and values.
//
// C^T (n x m) = B A^T with v_mfma_f32_32x32x16, so that a lane ends with four
// consecutive n of one row m and stores 8 bytes at a time.
#include "latent.h"

namespace {

// --- the absorbed form's plan, by one workgroup of 256 ---------------------------
template <typename T>
__device__ T scan_excl(T v, T *tmp, T &total) {  // exclusive sums over the workgroup's threads
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  T s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const T x = __shfl_up(s, o, 64);
    s += lane >= o ? x : T(0);
  }
  if (lane == 63) tmp[wave] = s;
  __syncthreads();
  T before = 0;
  total = 0;
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? tmp[w] : T(0);
    total += tmp[w];
  }
  __syncthreads();
  return before + s - v;
}

// Two ways to share the units out (see latent_attend.hip): pieces of row tiles, a
// piece a workgroup, where there are fewer row tiles than workgroups and the
// largest piece is not much above even work; even runs otherwise.
__device__ void make_plan(const LatentPlan &p, uint8_t *lds) {
  constexpr int kPer = 4;  // sequences a thread
  int64_t *start = reinterpret_cast<int64_t *>(lds), *tmp = start + 1024;  // of a sequence's units, or pieces
  int *t0s = reinterpret_cast<int *>(tmp + 8), *nqs = t0s + 1024, *lens = nqs + 1024;
  const int tid = threadIdx.x;
  auto tiles_of = [&](int len) { return max(1, (len + p.tokens - 1) / p.tokens); };
  const int row_shift = __ffs(p.rows) - 1;
  auto rows_of = [&](int nq) { return (nq * p.a.H + p.rows - 1) >> row_shift; };
  int64_t u = 0;
  int rt = 0, most = 1;  // row tiles (above the workgroups' number only that they are matters), the longest one's cache tiles
  int rr[kPer], kk[kPer];  // row tiles, cache tiles
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    rr[i] = 0;
    kk[i] = 1;
    if (b < p.a.B) {
      const LatentSeq s = latent_seq(p.a, b);
      t0s[b] = s.t0;
      nqs[b] = s.nq;
      lens[b] = s.len;
      rr[i] = rows_of(s.nq);
      kk[i] = tiles_of(s.len);
      if (rr[i]) most = max(most, kk[i]);
    }
    u += (int64_t)rr[i] * kk[i];
    rt += min(rr[i], 1 << 20);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    u += __shfl_xor(u, o, 64);
    rt += __shfl_xor(rt, o, 64);
    most = max(most, __shfl_xor(most, o, 64));
  }
  int *tmp32 = reinterpret_cast<int *>(tmp + 4);
  if ((tid & 63) == 0) {
    tmp[tid >> 6] = u;
    tmp32[tid >> 6] = rt;
    tmp32[4 + (tid >> 6)] = most;
  }
  __syncthreads();
  int64_t total = 0;
  int n_rows = 0;
  for (int w = 0; w < 4; ++w) {
    total += tmp[w];
    n_rows += tmp32[w];
    most = max(most, tmp32[4 + w]);
  }
  __syncthreads();
  const int64_t even = latent_div_up(total, p.n_wg);

  // the smallest pieces that are no more than the workgroups: 16 sizes at a time, 16 threads a size
  int piece = 0;
  if (n_rows > 0 && n_rows < p.n_wg) {
    const int64_t size = even + (tid >> 4), top = min(even + min(p.over, 15), latent_div_up(total, p.n_wg - n_rows));
    int c = 0;
    if (size <= top)
      for (int b = tid & 15; b < p.a.B; b += 16)
        c += (int)min((int64_t)rows_of(nqs[b]) * (int64_t)(((uint32_t)tiles_of(lens[b]) + (uint32_t)size - 1) / (uint32_t)size),
                      (int64_t)1 << 20);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) c += __shfl_xor(c, o, 64);
    const uint64_t fit = __ballot(size <= top && c <= p.n_wg);
    const int lane = fit ? __ffsll((unsigned long long)fit) - 1 : 0, pieces = __shfl(c, lane, 64);
    if ((tid & 63) == 0) tmp32[tid >> 6] = fit ? ((tid >> 6) * 4 + lane / 16) << 16 | pieces : 16 << 16;
    __syncthreads();
    const int best = min(min(tmp32[0], tmp32[1]), min(tmp32[2], tmp32[3]));
    __syncthreads();
    if (best < 16 << 16) {
      piece = (int)even + (best >> 16);
      // Whole row tiles where those are no more than a few cache tiles longer: the join of 256 pieces of 128 rows costs
      // 12 to 17 us, a cache tile 1.9 us (128 heads, 128 tokens of one sequence: the four kernels take 56 us so and 71
      // us in pieces with nothing before them, 68 and 78 us with 200 tokens, 78 and 83 us with 400; but one token over
      // 101 rows, whose pieces are 4, 35 us and 31 us).
      if (most - piece <= (best & 0xffff) * p.rows / 4096) piece = max(piece, most);
    }
  }
  // even runs: where a workgroup has few cache tiles it is better off with fewer of them than with even work
  const int over = !piece && total >= 4 * (int64_t)p.n_wg ? p.over : 0;
  int64_t mine = 0, all;
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += (int64_t)rr[i] * (piece ? (kk[i] + piece - 1) / piece : kk[i] + over);
  int64_t at0 = scan_excl<int64_t>(mine, tmp, all);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    start[tid * kPer + i] = at0;
    at0 += (int64_t)rr[i] * (piece ? (kk[i] + piece - 1) / piece : kk[i] + over);
  }
  __syncthreads();
  const int64_t per = piece ? 1 : max(latent_div_up(all, p.n_wg), (int64_t)1);
  // a share is a 32-bit number of units; more, hours of work, is reported and left out
  const bool fits = per < (int64_t)1 << 31;
  if (!fits && tid == 0) atomicOr(p.a.err, (uint32_t)ERRF_LATENT);
  int shared0 = 0;
  for (int w0 = 0; w0 < p.n_wg; w0 += 256) {
    const int w = w0 + tid;
    const int64_t v = w * per;
    WgDesc d{};
    TileDesc t{};
    if (w < p.n_wg && v < all && fits) {
      // the last sequence that starts at or before v is the one that has it: those without units share their
      // successor's start
      const int b = latent_last_at_or_below(start, p.a.B, v);
      d = WgDesc{b, 0, 0, 0, t0s[b], nqs[b], lens[b], over};
      latent_share(w, v, all, per, piece, over, b, start[b], rows_of(nqs[b]), tiles_of(lens[b]), &d, &t);
    }
    if (w < p.n_wg) p.wg[w] = d;
    int n;
    const int at = scan_excl<int>(t.n > 0, tmp32, n);
    if (t.n > 0) p.shared[shared0 + at] = t;
    shared0 += n;
  }
  if (tid == 0) *p.head = PlanHead{per, shared0};
}

// --- more rows: tiles of 64 or 128 rows x 64 or 128 columns through LDS --------
// Steps of 64 k: a row's 128 bytes of a step lie in LDS as 8 units of 16, unit c
// at c ^ swz(row) (16 rows' equal units then spread over the 64 banks). One stage
// is read while the others are loaded; two workgroups a CU, of 128 x 128 with two
// stages, of the smaller tiles with three (128 heads, 64 tokens: 13.6 and 8.8 us
// for the absorbed queries and the last product with tiles of 64 x 128, 14.3 and
// 11.4 us with 128 x 128; 512 tokens: 34.6 and 24.1 us with 128 x 128, 40.3 and
// 32.2 us with 128 x 64, which are for 64 columns only).
constexpr int kBK = 64;

__device__ __forceinline__ int swz(int row) { return ((row >> 1 & 1) << 2) | (row >> 2 & 3); }

template <typename E, int BM, int BN>
__global__ __launch_bounds__(256, 2) void head_gemm_tile_kernel(HeadGemm g, LatentPlan plan) {
  constexpr int kStage = (BM + BN) * 128, kStages = 3 * kStage <= 80 << 10 ? 3 : 2;
  constexpr int kNB = BN / 64, kMB = BM / 64;        // blocks of 32 columns and of 32 rows of a wave
  constexpr int kA = BM / 32, kLoads = kA + BN / 32;  // loads of a wave and stage: 8 rows x 128 bytes each
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStage];
  if (plan.n_wg && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) make_plan(plan, lds);
    return;
  }
  const int n_tiles = g.N / BN;
  const int m0 = blockIdx.x / n_tiles * BM, n0 = blockIdx.x % n_tiles * BN, h = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * (BN / 2), l32 = lane & 31, hl = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const uint16_t *src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = ((i < kA ? i : i - kA) * 4 + wave) * 8 + (lane >> 3);
    src[i] = (i < kA ? g.A + (int64_t)min(m0 + r, g.M - 1) * g.a_m + h * g.a_h
                     : g.B + h * g.b_h + (int64_t)(n0 + r) * g.K) +
             ((lane & 7) ^ swz(r & 15)) * 8;
  }
  auto load = [&](int s) {  // behind the last step nothing is loaded (but counted)
    const uint32_t to = uniform(lds0 + s % kStages * kStage + wave * 1024);
    const int on = uniform(s * kBK < g.K ? -1 : 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      lds_load16<0>(src[i] + s * kBK, to + (i < kA ? i * 4096 : BM * 128 + (i - kA) * 4096), on);
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(s);
  f32x16 acc[kNB][kMB];
#pragma unroll
  for (int i = 0; i < kNB; ++i)
#pragma unroll
    for (int j = 0; j < kMB; ++j) acc[i][j] = f32x16{};
  int off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) off[k] = l32 * 128 + (((2 * k + hl) ^ swz(l32 & 15)) << 4);
  for (int s = 0; s * kBK < g.K; ++s) {
    WAIT_VM((kStages - 2) * kLoads);
    asm volatile("s_barrier" ::: "memory");
    load(s + kStages - 1);
    const uint8_t *as = lds + s % kStages * kStage + wm * 128, *bs = lds + s % kStages * kStage + (BM + wn) * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u16x8 af[kMB], bf[kNB];
#pragma unroll
      for (int j = 0; j < kMB; ++j) af[j] = *reinterpret_cast<const u16x8 *>(as + j * 4096 + off[k]);
#pragma unroll
      for (int i = 0; i < kNB; ++i) bf[i] = *reinterpret_cast<const u16x8 *>(bs + i * 4096 + off[k]);
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int j = 0; j < kMB; ++j) acc[i][j] = E::mfma(bf[i], af[j], acc[i][j]);
    }
  }
  const int M = g.hi ? min(g.M, *g.hi) : g.M, lo = g.lo ? *g.lo : 0;
#pragma unroll
  for (int j = 0; j < kMB; ++j) {
    const int m = m0 + wm + 32 * j + l32;
    uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 + wn + 8 * hl;
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const f32x16 &r = acc[i][j];
        const u32x4 v = rows8<E>(f32x4{r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]},
                                 f32x4{r[4 * q + 4], r[4 * q + 5], r[4 * q + 6], r[4 * q + 7]});
        if (m >= lo && m < M) *reinterpret_cast<u32x4 *>(c + 32 * i + 8 * q) = v;
      }
  }
}

// --- few rows: the weights' bytes are the bound ---------------------------------
// A workgroup takes 32 rows x 32 columns, each wave a quarter of k: both operands
// come from memory straight in the products' layout (16 bytes a lane, a column's
// k in order), all of a wave's loads in flight at once; the quarters are summed
// through LDS. 128 heads, 8 tokens (17 MB of weights each): 7.0 and 5.6 us. Twice
// and four times the rows so were no faster than tiles: 16.0 and 16.7 us for 64
// tokens, against 13.6 and 8.8.
constexpr int kPlanLds = 8 * 1024 + 64 + 3 * 4096;

template <typename E>
__global__ __launch_bounds__(256) void head_gemm_stream_kernel(HeadGemm g, LatentPlan plan) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kPlanLds > 16384 ? kPlanLds : 16384];
  if (plan.n_wg && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0 && blockIdx.z == 0) make_plan(plan, lds);
    return;
  }
  const int m0 = blockIdx.z * 32, n0 = blockIdx.x * 32, h = blockIdx.y;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int m = m0 + l32, steps = g.K / 64, k0 = wave * steps * 16;
  const uint16_t *a = g.A + (int64_t)min(m, g.M - 1) * g.a_m + h * g.a_h + k0 + 8 * hl;
  const uint16_t *b = g.B + h * g.b_h + (int64_t)(n0 + l32) * g.K + k0 + 8 * hl;
  constexpr int kMax = 8;  // K up to 512
  u16x8 af[kMax], bf[kMax];
#pragma unroll
  for (int i = 0; i < kMax; ++i)
    if (i < steps) {
      bf[i] = *reinterpret_cast<const u16x8 *>(b + 16 * i);
      af[i] = *reinterpret_cast<const u16x8 *>(a + 16 * i);
    }
  const int M = g.hi ? min(g.M, *g.hi) : g.M, lo = g.lo ? *g.lo : 0;
  f32x16 acc = {};
#pragma unroll
  for (int i = 0; i < kMax; ++i)
    if (i < steps) acc = E::mfma(bf[i], af[i], acc);
  f32x4 *box = reinterpret_cast<f32x4 *>(lds);  // [wave][4 rows of c][lane]
#pragma unroll
  for (int q = 0; q < 4; ++q)
    box[(wave * 4 + q) * 64 + lane] = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  if (wave >= 2) return;
  f32x4 sum[2];  // wave w: columns 16 w .. 16 w + 15
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    sum[q] = box[(2 * wave + q) * 64 + lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) sum[q] += box[(w * 4 + 2 * wave + q) * 64 + lane];
  }
  const u32x4 v = rows8<E>(sum[0], sum[1]);
  if (m >= lo && m < M)
    *reinterpret_cast<u32x4 *>(g.C + m * g.c_m + h * g.c_h + n0 + 16 * wave + 8 * hl) = v;
}

// --- expanded keys and values: tiles of 256 rows x 256 columns ----------------------
// The heads' weights are one matrix of H N columns. Steps of 64 k as above, two
// stages; 8 waves of 64 rows x 128 columns, two a SIMD. K is short (2 to 8 steps),
// so a workgroup goes on from tile to tile: the next tile's first step is loaded
// under the last step's products, and a tile's stores drain under the next one's
// products (with a tile a workgroup, which loads, multiplies and stores in turn,
// 4096 rows of 128 heads of 256 columns took 181 us; 163 us so,
// 137 GFLOP and 268 MB written).
template <typename E>
__global__ __launch_bounds__(512, 1) void expand_gemm_kernel(ExpandGemm g) {
  constexpr int kStage = 512 * 128, kLoads = 8, kStores = 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
  const int M = min(g.M, uniform(*g.hi)), cols = g.H * g.N;
  // an XCD (ids go round the 8 of them) takes whole column tiles, row tile by row tile
  const int xcd = blockIdx.x & 7, m_tiles = (M + 255) / 256, n_tiles = (cols + 255) / 256;
  const int count = (n_tiles - xcd + 7) / 8 * m_tiles, stride = gridDim.x >> 3;
  int t = blockIdx.x >> 3;
  if (t >= count) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int wm = (wave & 3) * 64, wn = (wave >> 2) * 128;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  auto m_of = [&](int tile) { return tile % m_tiles * 256; };
  auto n_of = [&](int tile) { return (xcd + 8 * (tile / m_tiles)) * 256; };
  // loads: 8 rows x 128 bytes a wave and instruction; waves 0-3 rows, 4-7 columns (weights)
  const uint16_t *src[kLoads];
  auto aim = [&](int tile) {
    const int first = wave < 4 ? m_of(tile) : n_of(tile), last = (wave < 4 ? M : cols) - 1;
    const uint16_t *base = wave < 4 ? g.A : g.B;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = ((wave & 3) * kLoads + i) * 8 + (lane >> 3), unit = (lane & 7) ^ swz(r & 15);
      src[i] = base + (int64_t)min(first + r, last) * g.K + unit * 8;
    }
  };
  auto load = [&](int i, int s, int on) {
    lds_load16<0>(src[i] + s * kBK, uniform(lds0 + (s & 1) * kStage + (wave * kLoads + i) * 1024), uniform(on));
  };
  int off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) off[k] = l32 * 128 + (((2 * k + hl) ^ swz(l32 & 15)) << 4);
  const int steps = g.K / kBK;  // even: a tile's first step goes to the stage that its predecessor's last one does not use
  aim(t);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) load(i, 0, -1);
  bool stores = false;  // the tile before has left exactly kStores stores behind this one's first loads
  for (; t < count; t += stride) {
    const int m0 = m_of(t), n0 = n_of(t);
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    for (int s = 0; s < steps; ++s) {
      if (s == 0 && stores)
        WAIT_VM(kStores);
      else
        WAIT_VM(0);
      asm volatile("s_barrier" ::: "memory");
      const uint8_t *as = lds + (s & 1) * kStage + wm * 128, *bs = lds + (s & 1) * kStage + (256 + wn) * 128;
      u16x8 af[2][2], bf[2][4];
      auto read = [&](int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j) af[k & 1][j] = *reinterpret_cast<const u16x8 *>(as + j * 4096 + off[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) bf[k & 1][i] = *reinterpret_cast<const u16x8 *>(bs + i * 4096 + off[k]);
      };
      read(0);
      const bool end = s + 1 == steps;
      const int on = !end || t + stride < count ? -1 : 0, next = end ? 0 : s + 1;
      if (end && on) aim(t + stride);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < 3) read(k + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = E::mfma(bf[k & 1][i], af[k & 1][j], acc[i][j]);
          if (4 * k + i < kLoads) load(4 * k + i, next, on);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    // The results go out through the stage that the last step used, a wave's 32 rows x 128 columns at a time in 8 KB
    // of its own (unit c of a row at c ^ row % 16), so that a store writes four rows' 256 bytes in a row: stored as
    // they lie in the registers, 32 bytes of 32 rows at a time, they cost 50 us of the 169.
    stores = m0 + 256 <= M && n0 + 256 <= cols;
    asm volatile("s_barrier" ::: "memory");  // the last step's readers are done
    uint8_t *box = lds + kStage + wave * 8192;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const f32x16 &r = acc[i][j];
          const u32x4 v = rows8<E>(f32x4{r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]},
                                   f32x4{r[4 * q + 4], r[4 * q + 5], r[4 * q + 6], r[4 * q + 7]});
          *reinterpret_cast<u32x4 *>(box + l32 * 256 + (((4 * i + q + hl) ^ (l32 & 15)) << 4)) = v;
        }
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = 4 * p + (lane >> 4), unit = lane & 15;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(box + row * 256 + ((unit ^ (row & 15)) << 4));
        const int m = m0 + wm + 32 * j + row, n = n0 + wn + unit * 8, h = n / g.N;
        uint16_t *c = g.C + ((int64_t)h * g.M + m) * g.N + (n - h * g.N);
        if (stores || (m < M && n < cols)) *reinterpret_cast<u32x4 *>(c) = v;
      }
    }
  }
}

template <typename E>
void launch(moe_ctx *ctx, const HeadGemm &g, int H, const LatentPlan &p) {
  const unsigned extra = p.n_wg ? 1 : 0;  // a column of workgroups whose first makes the plan
  if (g.M <= 32)
    hipLaunchKernelGGL(head_gemm_stream_kernel<E>, dim3(g.N / 32 + extra, H, (g.M + 31) / 32), dim3(256), 0,
                       ctx->stream, g, p);
  else if (g.M <= 64 && g.N % 128 == 0)
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 64, 128>), dim3(g.N / 128 + extra, H), dim3(256), 0, ctx->stream, g, p);
  else if (g.N % 128 == 0)
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 128, 128>), dim3((g.M + 127) / 128 * (g.N / 128) + extra, H), dim3(256),
                       0, ctx->stream, g, p);
  else
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 128, 64>), dim3((g.M + 127) / 128 * (g.N / 64) + extra, H), dim3(256),
                       0, ctx->stream, g, p);
}

}  // namespace

moe_status launch_head_gemm(moe_ctx *ctx, int dtype, const HeadGemm &g, int H, const LatentPlan &plan) {
  if (dtype == MOE_BF16)
    launch<Bf16>(ctx, g, H, plan);
  else
    launch<Fp16>(ctx, g, H, plan);
  MOE_CHECK_LAUNCH("head_gemm kernel");
  return MOE_OK;
}

moe_status launch_expand_gemm(moe_ctx *ctx, int dtype, const ExpandGemm &g) {
  const dim3 grid(ctx->n_cu / 8 * 8);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(expand_gemm_kernel<Bf16>, grid, dim3(512), 0, ctx->stream, g);
  else
    hipLaunchKernelGGL(expand_gemm_kernel<Fp16>, grid, dim3(512), 0, ctx->stream, g);
  MOE_CHECK_LAUNCH("expand_gemm_kernel");
  return MOE_OK;
}
