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
  int64_t *units = reinterpret_cast<int64_t *>(lds), *tiles = units + 1024, *tmp = tiles + 1024;
  const int tid = threadIdx.x;
  int64_t u = 0, t = 0, uu[kPer], tt[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    uu[i] = tt[i] = 0;
    if (b < p.a.B) {
      const LatentSeq s = latent_seq(p.a, b);
      tt[i] = ((int64_t)s.nq * p.a.H + p.rows - 1) / p.rows;
      uu[i] = tt[i] * (max(1, (s.len + p.tokens - 1) / p.tokens) + p.over);
    }
    u += uu[i];
    t += tt[i];
  }
  int64_t total, n_tiles;
  int64_t u0 = scan_excl<int64_t>(u, tmp, total), t0 = scan_excl<int64_t>(t, tmp, n_tiles);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    units[tid * kPer + i] = u0;
    tiles[tid * kPer + i] = t0;
    u0 += uu[i];
    t0 += tt[i];
  }
  __syncthreads();
  const int64_t per = max((total + p.n_wg - 1) / p.n_wg, (int64_t)p.over + 1);
  if (tid == 0) *p.head = PlanHead{per, (int)n_tiles};
  for (int w = tid; w < p.n_wg; w += 256) {
    const int64_t v = w * per;
    WgDesc d{0, 0, 0, 0};
    if (v < total) {
      // the last sequence that starts at or before v is the one that has it: those without units share their
      // successor's start
      const int b = last_at_or_below(units, 1024, v);
      const LatentSeq s = latent_seq(p.a, b);
      const int k = max(1, (s.len + p.tokens - 1) / p.tokens) + p.over;
      const int64_t r = v - units[b];
      d = WgDesc{b, (int)(r / k), (int)(r % k), (int)min(per, total - v)};
    }
    p.wg[w] = d;
  }
  for (int i = tid; i < n_tiles; i += 256) {
    const int b = last_at_or_below(tiles, 1024, i), mt = (int)(i - tiles[b]);
    const LatentSeq s = latent_seq(p.a, b);
    const int k = max(1, (s.len + p.tokens - 1) / p.tokens);
    const int64_t v = units[b] + (int64_t)mt * (k + p.over);
    p.tile[i] = TileDesc{b, mt, (int)((v + p.over) / per), (int)((v + p.over + k - 1) / per), v};
  }
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
    a_src[i] = g.A + (g.rows ? g.rows[m] : (int64_t)m) * g.a_m + h * g.a_h + ((lane & 7) ^ swz(r & 15)) * 8;
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
    if (m < lo || m >= M) continue;
    uint16_t *c = g.C + m * g.c_m + h * g.c_h + (n0 + wn) / 16 * g.c_n + 4 * hl;
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u16x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = E::from_f32(acc[i][j][4 * q + e]);
        *reinterpret_cast<u16x4 *>(c + (2 * i + (q >> 1)) * g.c_n + 8 * (q & 1)) = v;
      }
  }
}

// --- few rows: the weights' bytes are the bound ---------------------------------
// A wave takes 32 rows x 32 columns and reads both operands from memory straight
// in the products' layout (16 bytes a lane, a column's k in order), 128 k of
// loads in flight before the products of the previous 128.
template <typename E>
__global__ __launch_bounds__(256) void head_gemm_stream_kernel(HeadGemm g, LatentPlan plan) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * 8 * 1024 + 64];
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
  const uint16_t *a = g.A + (g.rows ? g.rows[ma] : (int64_t)ma) * g.a_m + h * g.a_h + 8 * hl;
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
  if (m < lo || m >= M) return;
  uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 / 16 * g.c_n + 4 * hl;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u16x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = E::from_f32(acc[4 * q + e]);
    *reinterpret_cast<u16x4 *>(c + (q >> 1) * g.c_n + 8 * (q & 1)) = v;
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
