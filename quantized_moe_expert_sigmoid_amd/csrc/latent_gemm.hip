// Products of the heads' expansion weights: absorbed queries, the last product
// of the absorbed form, expanded keys and values.
#include "latent.h"

namespace {

constexpr int kGT = 64;
constexpr int kGPad = 8;

template <typename E>
__global__ __launch_bounds__(256) void head_gemm_kernel(HeadGemm g) {
  __shared__ uint16_t as[kGT][kGT + kGPad], bs[kGT][kGT + kGPad];
  const int M = g.hi ? min(g.M, *g.hi) : g.M, lo = g.lo ? *g.lo : 0;
  const int m0 = blockIdx.x * kGT, n0 = blockIdx.y * kGT, h = blockIdx.z;
  if (m0 >= M || m0 + kGT <= lo) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wn = (wave >> 1) * 32, wm = (wave & 1) * 32, l32 = lane & 31, hl = lane >> 5;
  f32x16 acc = {};
  for (int k0 = 0; k0 < g.K; k0 += kGT) {
    __syncthreads();
    for (int i = threadIdx.x; i < kGT * 8; i += 256) {
      const int r = i >> 3, c = (i & 7) * 8;
      const int m = min(m0 + r, M - 1);
      *reinterpret_cast<u16x8 *>(&as[r][c]) =
          *reinterpret_cast<const u16x8 *>(g.A + (g.rows ? g.rows[m] : m) * g.a_m + h * g.a_h + k0 + c);
      *reinterpret_cast<u16x8 *>(&bs[r][c]) =
          *reinterpret_cast<const u16x8 *>(g.B + h * g.b_h + (int64_t)(n0 + r) * g.K + k0 + c);
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kGT; kk += 16)
      acc = E::mfma(*reinterpret_cast<const u16x8 *>(&bs[wn + l32][kk + 8 * hl]),
                      *reinterpret_cast<const u16x8 *>(&as[wm + l32][kk + 8 * hl]), acc);
  }
  const int m = m0 + wm + l32;
  if (m < lo || m >= M) return;
  uint16_t *c = g.C + m * g.c_m + h * g.c_h + n0 + wn + 4 * hl;
#pragma unroll
  for (int i = 0; i < 16; ++i) c[8 * (i >> 2) + (i & 3)] = E::from_f32(acc[i]);
}

}  // namespace

moe_status launch_head_gemm(moe_ctx *ctx, int dtype, const HeadGemm &g, int H) {
  const dim3 grid((g.M + kGT - 1) / kGT, g.N / kGT, H);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(head_gemm_kernel<Bf16>, grid, dim3(256), 0, ctx->stream, g);
  else
    hipLaunchKernelGGL(head_gemm_kernel<Fp16>, grid, dim3(256), 0, ctx->stream, g);
  MOE_CHECK_LAUNCH("head_gemm_kernel");
  return MOE_OK;
}
