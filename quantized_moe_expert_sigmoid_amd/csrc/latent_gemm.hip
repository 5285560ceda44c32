// Products of the heads' expansion weights: absorbed queries, the last product
// of the absorbed form, expanded keys and values.
//
// C^T (n x m) = B A^T with v_mfma_f32_32x32x16, so that a lane ends with four
// consecutive n of one row m and stores 8 bytes at a time.
#include "latent.h"

namespace {

// --- many rows: tiles of 128 rows x 64 or 128 columns through LDS --------------
// Steps of 64 k: a row's 128 bytes of a step lie in LDS as 8 units of 16, unit c
// at c ^ swz(row) (16 rows' equal units then spread over the 64 banks). Two
// stages: one is read while the other is loaded.
constexpr int kBM = 128, kBK = 64;

__device__ __forceinline__ int swz(int row) { return ((row >> 1 & 1) << 2) | (row >> 2 & 3); }

template <typename E, int BN>
__global__ __launch_bounds__(256, 2) void head_gemm_tile_kernel(HeadGemm g) {
  constexpr int kStage = (kBM + BN) * 128, kNB = BN / 64;  // blocks of 32 n of a wave
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
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
    for (int i = 0; i < kBM / 32; ++i) lds_load16_v(a_src[i] + k0, to + i * 4096);
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) lds_load16_v(b_src[i] + k0, to + kBM * 128 + i * 4096);
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
    uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 + wn + 4 * hl;
#pragma unroll
    for (int i = 0; i < kNB; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        u16x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = E::from_f32(acc[i][j][4 * q + e]);
        *reinterpret_cast<u16x4 *>(c + 32 * i + 8 * q) = v;
      }
  }
}

// --- few rows: the weights' bytes are the bound ---------------------------------
// A wave takes 32 rows x 32 columns and reads both operands from memory straight
// in the products' layout (16 bytes a lane, a column's k in order), 128 k of
// loads in flight before the products of the previous 128.
template <typename E>
__global__ __launch_bounds__(256) void head_gemm_stream_kernel(HeadGemm g) {
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
  uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 + 4 * hl;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u16x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = E::from_f32(acc[4 * q + e]);
    *reinterpret_cast<u16x4 *>(c + 8 * q) = v;
  }
}

template <typename E>
void launch(moe_ctx *ctx, const HeadGemm &g, int H) {
  if (g.M <= 64)
    hipLaunchKernelGGL(head_gemm_stream_kernel<E>, dim3((g.N + 127) / 128, H, (g.M + 31) / 32), dim3(256), 0,
                       ctx->stream, g);
  else if (g.N % 128 == 0)
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 128>), dim3((g.M + kBM - 1) / kBM * (g.N / 128), H), dim3(256), 0,
                       ctx->stream, g);
  else
    hipLaunchKernelGGL((head_gemm_tile_kernel<E, 64>), dim3((g.M + kBM - 1) / kBM * (g.N / 64), H), dim3(256), 0,
                       ctx->stream, g);
}

}  // namespace

moe_status launch_head_gemm(moe_ctx *ctx, int dtype, const HeadGemm &g, int H) {
  if (dtype == MOE_BF16)
    launch<Bf16>(ctx, g, H);
  else
    launch<Fp16>(ctx, g, H);
  MOE_CHECK_LAUNCH("head_gemm kernel");
  return MOE_OK;
}
