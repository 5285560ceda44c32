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

__device__ int last_at_or_below(const int64_t *cum, int n, int64_t v) {  // cum ascending, cum[0] <= v: the last such i
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ void make_plan(const LatentPlan &p, uint8_t *lds) {
  constexpr int kPer = 4;  // sequences a thread
  int64_t *units = reinterpret_cast<int64_t *>(lds), *tmp = units + 1024;
  const int tid = threadIdx.x;
  int64_t u = 0, uu[kPer], rt = 0, rr[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    uu[i] = rr[i] = 0;
    if (b < p.a.B) {
      const LatentSeq s = latent_seq(p.a, b);
      rr[i] = ((int64_t)s.nq * p.a.H + p.rows - 1) / p.rows;
      uu[i] = rr[i] * max(1, (s.len + p.tokens - 1) / p.tokens);
    }
    u += uu[i];
    rt += rr[i];
  }
  int64_t total, n_rows, u0 = scan_excl<int64_t>(u, tmp, total);
  const int64_t r0 = scan_excl<int64_t>(rt, tmp, n_rows);
  // where a workgroup has few cache tiles it is better off with fewer of them than with even work
  const int over = total >= 8 * (int64_t)p.n_wg ? p.over : 0;
  u0 += over * r0;
  total += over * n_rows;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    units[tid * kPer + i] = u0;
    u0 += uu[i] + over * rr[i];
  }
  __syncthreads();
  const int64_t per = max((total + p.n_wg - 1) / p.n_wg, (int64_t)1);
  int shared0 = 0;
  for (int w0 = 0; w0 < p.n_wg; w0 += 256) {
    const int w = w0 + tid;
    const int64_t v = w * per;
    WgDesc d{0, 0, 0, 0};
    TileDesc t{};
    if (w < p.n_wg && v < total) {
      // the last sequence that starts at or before v is the one that has it: those without units share their
      // successor's start
      const int b = last_at_or_below(units, 1024, v);
      const LatentSeq s = latent_seq(p.a, b);
      const int k = max(1, (s.len + p.tokens - 1) / p.tokens);
      const int64_t r = v - units[b];
      d = WgDesc{b, (int)(r / (k + over)), (int)(r % (k + over)), (int)min(per, total - v)};
      // shared with the workgroups before, and the first boundary in this row tile
      const int64_t u0 = v - d.at;
      const int first = (int)((u0 + over) / per);
      if (d.at > over && first == w - 1) t = TileDesc{b, d.mt, first, (int)((u0 + over + k - 1) / per), u0};
    }
    if (w < p.n_wg) p.wg[w] = d;
    int64_t n;
    const int64_t at = scan_excl<int64_t>(t.w1 > 0, tmp, n);
    if (t.w1 > 0) p.shared[shared0 + at] = t;
    shared0 += (int)n;
  }
  if (tid == 0) *p.head = PlanHead{per, over, shared0};
}

// --- many rows: tiles of 128 rows x 64 or 128 columns through LDS --------------
// Steps of 64 k: a row's 128 bytes of a step lie in LDS as 8 units of 16, unit c
// at c ^ swz(row) (16 rows' equal units then spread over the 64 banks). Two
// stages: one is read while the other is loaded.
constexpr int kBM = 128, kBK = 64;

__device__ __forceinline__ int swz(int row) { return ((row >> 1 & 1) << 2) | (row >> 2 & 3); }

template <typename E, int BN>
__global__ __launch_bounds__(256, 2) void head_gemm_tile_kernel(HeadGemm g, LatentPlan plan) {
  constexpr int kStage = (kBM + BN) * 128, kNB = BN / 64;  // blocks of 32 n of a wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
  if (plan.n_wg && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) make_plan(plan, lds);
    return;
  }
  const int M = g.hi ? min(g.M, uniform(*g.hi)) : g.M, lo = g.lo ? uniform(*g.lo) : 0;
  const int n_tiles = g.N / BN;
  const int m0 = blockIdx.x / n_tiles * kBM, n0 = blockIdx.x % n_tiles * BN, h = blockIdx.y;
  if (m0 >= M || m0 + kBM <= lo) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * (BN / 2), l32 = lane & 31, hl = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // loads: 8 rows x 128 bytes a wave and instruction; lane's row in the block and its unit
  const int r8 = lane >> 3;
  const uint16_t *a_src[kBM / 32];
  const uint16_t *b_src[BN / 32];
#pragma unroll
  for (int i = 0; i < kBM / 32; ++i) {
    const int r = (i * 4 + wave) * 8 + r8, m = min(m0 + r, M - 1);
    a_src[i] = g.A + (int64_t)m * g.a_m + h * g.a_h + ((lane & 7) ^ swz(r & 15)) * 8;
  }
#pragma unroll
  for (int i = 0; i < BN / 32; ++i) {
    const int r = (i * 4 + wave) * 8 + r8;
    b_src[i] = g.B + h * g.b_h + (int64_t)(n0 + r) * g.K + ((lane & 7) ^ swz(r & 15)) * 8;
  }
  auto load = [&](int stage, int k0) {
    const uint32_t to = uniform(lds0 + stage * kStage + wave * 1024);
#pragma unroll
    for (int i = 0; i < kBM / 32; ++i) lds_load16<0>(a_src[i] + k0, to + i * 4096);
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) lds_load16<0>(b_src[i] + k0, to + kBM * 128 + i * 4096);
  };
  f32x16 acc[kNB][2];
#pragma unroll
  for (int i = 0; i < kNB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  int off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) off[k] = l32 * 128 + (((2 * k + hl) ^ swz(l32 & 15)) << 4);
  load(0, 0);
  for (int k0 = 0, st = 0; k0 < g.K; k0 += kBK, st ^= 1) {
    WAIT_VM(0);
    asm volatile("s_barrier" ::: "memory");
    if (k0 + kBK < g.K) load(st ^ 1, k0 + kBK);
    const uint8_t *as = lds + st * kStage + wm * 128, *bs = lds + st * kStage + (kBM + wn) * 128;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u16x8 af[2], bf[kNB];
#pragma unroll
      for (int j = 0; j < 2; ++j) af[j] = *reinterpret_cast<const u16x8 *>(as + j * 4096 + off[k]);
#pragma unroll
      for (int i = 0; i < kNB; ++i) bf[i] = *reinterpret_cast<const u16x8 *>(bs + i * 4096 + off[k]);
#pragma unroll
      for (int i = 0; i < kNB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = E::mfma(bf[i], af[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
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
// A wave takes 32 rows x 32 columns and reads both operands from memory straight
// in the products' layout (16 bytes a lane, a column's k in order), 128 k of
// loads in flight before the products of the previous 128.
template <typename E>
__global__ __launch_bounds__(256) void head_gemm_stream_kernel(HeadGemm g, LatentPlan plan) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[8 * 1024 + 64];
  if (plan.n_wg && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0 && blockIdx.z == 0) make_plan(plan, lds);
    return;
  }
  const int M = g.hi ? min(g.M, uniform(*g.hi)) : g.M, lo = g.lo ? uniform(*g.lo) : 0;
  const int m0 = blockIdx.z * 32;
  const int lane = threadIdx.x & 63, n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 32, h = blockIdx.y;
  if (m0 >= M || m0 + 32 <= lo || n0 >= g.N) return;
  const int l32 = lane & 31, hl = lane >> 5;
  const int m = m0 + l32;
  const int ma = min(m, M - 1);
  const uint16_t *a = g.A + (int64_t)ma * g.a_m + h * g.a_h + 8 * hl;
  const uint16_t *b = g.B + h * g.b_h + (int64_t)(n0 + l32) * g.K + 8 * hl;
  constexpr int kC = 4;  // products (16 k) of a batch of loads
  f32x16 acc = {};
  u16x8 af[2][kC], bf[2][kC];
  auto load = [&](int s, int k0) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      bf[s][i] = *reinterpret_cast<const u16x8 *>(b + k0 + 16 * i);
      af[s][i] = *reinterpret_cast<const u16x8 *>(a + k0 + 16 * i);
    }
  };
  load(0, 0);
  for (int k0 = 0; k0 < g.K; k0 += 2 * 16 * kC) {
    const bool two = k0 + 16 * kC < g.K;
    if (two) load(1, k0 + 16 * kC);
#pragma unroll
    for (int i = 0; i < kC; ++i) acc = E::mfma(bf[0][i], af[0][i], acc);
    if (k0 + 2 * 16 * kC < g.K) load(0, k0 + 2 * 16 * kC);
    if (two)
#pragma unroll
      for (int i = 0; i < kC; ++i) acc = E::mfma(bf[1][i], af[1][i], acc);
  }
  uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 + 8 * hl;
#pragma unroll
  for (int q = 0; q < 4; q += 2) {
    const u32x4 v = rows8<E>(f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]},
                             f32x4{acc[4 * q + 4], acc[4 * q + 5], acc[4 * q + 6], acc[4 * q + 7]});
    if (m >= lo && m < M) *reinterpret_cast<u32x4 *>(c + 8 * q) = v;
  }
}

// --- expanded keys and values: tiles of 256 rows x 256 columns ----------------------
// The heads' weights are one matrix of H N columns. Steps of 32 k: a row's 64
// bytes of a step are 4 units of 16 in LDS, unit c at c ^ (row / 4) % 4 (16 rows'
// equal units then lie in different banks). Four stages, one read while three are
// in flight; 8 waves of 64 rows x 128 columns, two a SIMD.
template <typename E>
__global__ __launch_bounds__(512, 1) void expand_gemm_kernel(ExpandGemm g) {
  constexpr int kStage = 512 * 64, kStages = 4, kLoads = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages * kStage];
  const int M = min(g.M, uniform(*g.hi)), cols = g.H * g.N;
  // an XCD (ids go round the 8 of them) takes whole column tiles, row tile by row tile
  const int m_tiles = (g.M + 255) / 256, local = blockIdx.x >> 3;
  const int m0 = local % m_tiles * 256, n0 = ((blockIdx.x & 7) + 8 * (local / m_tiles)) * 256;
  if (m0 >= M || n0 >= cols) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int wm = (wave & 3) * 64, wn = (wave >> 2) * 128;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // loads: 16 rows x 64 bytes a wave and instruction; waves 0-3 rows, 4-7 columns (weights)
  const uint16_t *src[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = ((wave & 3) * kLoads + i) * 16 + (lane >> 2), unit = (lane & 3) ^ (r >> 2 & 3);
    src[i] = (wave < 4 ? g.A + (int64_t)min(m0 + r, M - 1) * g.K : g.B + (int64_t)min(n0 + r, cols - 1) * g.K) + unit * 8;
  }
  auto load = [&](int i, int s) {
    lds_load16<0>(src[i] + s * 32, uniform(lds0 + (s % kStages) * kStage + (wave * kLoads + i) * 1024),
                  uniform(s * 32 < g.K ? -1 : 0));
  };
  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  int off[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) off[k] = l32 * 64 + (((2 * k + hl) ^ (l32 >> 2 & 3)) << 4);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(i, s);
  const int steps = g.K / 32;
  for (int s = 0; s < steps; ++s) {
    WAIT_VM((kStages - 2) * kLoads);
    asm volatile("s_barrier" ::: "memory");
    const uint8_t *as = lds + (s % kStages) * kStage + wm * 64, *bs = lds + (s % kStages) * kStage + (256 + wn) * 64;
    u16x8 af[2][2], bf[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int j = 0; j < 2; ++j) af[k][j] = *reinterpret_cast<const u16x8 *>(as + j * 2048 + off[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) bf[k][i] = *reinterpret_cast<const u16x8 *>(bs + i * 2048 + off[k]);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = E::mfma(bf[k][i], af[k][j], acc[i][j]);
        if (i & 1) load(2 * k + (i >> 1), s + kStages - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + wn + 32 * i;
    if (n >= cols) break;
    const int h = n / g.N;
    uint16_t *c = g.C + ((int64_t)h * g.M) * g.N + (n - h * g.N) + 8 * hl;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int m = m0 + wm + 32 * j + l32;
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        const f32x16 &r = acc[i][j];
        const u32x4 v = rows8<E>(f32x4{r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]},
                                 f32x4{r[4 * q + 4], r[4 * q + 5], r[4 * q + 6], r[4 * q + 7]});
        if (m < M) *reinterpret_cast<u32x4 *>(c + (int64_t)m * g.N + 8 * q) = v;
      }
    }
  }
}

template <typename E>
void launch(moe_ctx *ctx, const HeadGemm &g, int H, const LatentPlan &p) {
  const unsigned extra = p.n_wg ? 1 : 0;  // a column of workgroups whose first makes the plan
  if (g.M <= 64)
    hipLaunchKernelGGL(head_gemm_stream_kernel<E>, dim3((g.N + 127) / 128 + extra, H, (g.M + 31) / 32), dim3(256), 0,
                       ctx->stream, g, p);
  else if (g.N % 128 == 0)
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 128>), dim3((g.M + kBM - 1) / kBM * (g.N / 128) + extra, H), dim3(256),
                       0, ctx->stream, g, p);
  else
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 64>), dim3((g.M + kBM - 1) / kBM * (g.N / 64) + extra, H), dim3(256),
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
  const unsigned m_tiles = (g.M + 255) / 256, n_tiles = (g.H * g.N + 255) / 256;
  const dim3 grid(m_tiles * ((n_tiles + 7) / 8) * 8);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(expand_gemm_kernel<Bf16>, grid, dim3(512), 0, ctx->stream, g);
  else
    hipLaunchKernelGGL(expand_gemm_kernel<Fp16>, grid, dim3(512), 0, ctx->stream, g);
  MOE_CHECK_LAUNCH("expand_gemm_kernel");
  return MOE_OK;
}
