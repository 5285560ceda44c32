// Products on microscaled 4-bit floating point for few lines an expert: the
// weights' bytes are the bound.
//
// C^T (n x m) = W X^T with v_mfma_scale_f32_16x16x128_f8f6f4. A workgroup takes
// 16 rows of weights and a unit of up to 16 lines; its 8 waves share out k in
// runs of 128 and sum through LDS. Both operands come from memory straight in
// the products' layout: lane l has 16 bytes, block l / 16 of four, of row l % 16.
#include "mx.h"

namespace {

constexpr int kWaves = 8, kTile = 16;

struct Weights {
  const uint8_t *w, *s;
};

// The four blocks 4 step .. of row r of codes c and scales s, one a lane; behind the row's end zeros.
__device__ __forceinline__ void load_block(const uint8_t *c, const uint8_t *s, int64_t r, int blocks, int step,
                                           i32x4 &code, int &scale) {
  const int b = 4 * step + ((threadIdx.x & 63) >> 4);
  code = i32x4{};
  scale = 127;
  if (b < blocks) {
    code = *reinterpret_cast<const i32x4 *>(c + (r * blocks + b) * 16);
    scale = s[r * blocks + b];
  }
}

// One 16 x 16 tile of W X^T over the whole k: in wave 0's lanes afterwards, as a product leaves it. box: 4 KB a tile.
template <int NM>
__device__ __forceinline__ void tile_product(const Weights (&m)[NM], int64_t n, const MxProduct &p, int64_t row,
                                             f32x4 *box, f32x4 (&sum)[NM]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, blocks = p.K / kMxBlock;
  const int steps = (blocks + 3) / 4, per = (steps + kWaves - 1) / kWaves;
#pragma unroll
  for (int i = 0; i < NM; ++i) sum[i] = f32x4{};
  for (int s = wave * per; s < min(steps, (wave + 1) * per); ++s) {
    i32x4 x, w;
    int sx, sw;
    load_block(p.x, p.sx, row, blocks, s, x, sx);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      load_block(m[i].w, m[i].s, n, blocks, s, w, sw);
      sum[i] = mx_mfma16(w, sw, x, sx, sum[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NM; ++i) box[(wave * NM + i) * 64 + lane] = sum[i];
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 0; i < NM; ++i)
    for (int w = 1; w < kWaves; ++w) sum[i] += box[(w * NM + i) * 64 + lane];
}

template <int DTYPE, bool DOWN>
__global__ __launch_bounds__(kWaves * 64) void mx_stream_kernel(MxProduct p) {
  typedef MxOut<DTYPE> O;
  __shared__ f32x4 box[kWaves * 64];
  const int n_tiles = (p.N + 15) / 16, lane = threadIdx.x & 63;
  const MxUnit u = mx_unit<kTile>(p, blockIdx.x / n_tiles);
  if (u.n == 0) return;
  const int n0 = blockIdx.x % n_tiles * 16;
  Weights m[1] = {{p.w + u.e * p.w_e, p.sw + u.e * p.sw_e}};
  if constexpr (DOWN) m[0] = Weights{p.table[u.e].down, p.table[u.e].s_down};
  const int64_t line = u.first + min(lane & 15, u.n - 1), row = mx_in_row(p, line);
  f32x4 sum[1];
  tile_product<1>(m, min(n0 + (lane & 15), p.N - 1), p, max(row, (int64_t)0), box, sum);
  if (threadIdx.x >= 64 || (lane & 15) >= u.n || row < 0) return;
  const int64_t r = mx_out_row(p, line);
  if (r < 0) return;
  const int n = n0 + 4 * (lane >> 4);
  typename O::T *out = static_cast<typename O::T *>(p.out) + r * p.N + n;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.N) out[i] = O::one(sum[0][i]);
}

// The same for gate and up, 32 of their rows a workgroup (a block of the result): silu(g) u and its codes.
__global__ __launch_bounds__(kWaves * 64) void mx_stream_gateup_kernel(MxProduct p, uint8_t *scales) {
  __shared__ f32x4 box[2 * kWaves * 64];
  const int n_tiles = p.N / 32, lane = threadIdx.x & 63;
  const MxUnit u = mx_unit<kTile>(p, blockIdx.x / n_tiles);
  if (u.n == 0) return;
  const int n0 = blockIdx.x % n_tiles * 32;
  const moe_mx_expert_w &t = p.table[u.e];
  const Weights m[2] = {{t.gate, t.s_gate}, {t.up, t.s_up}};
  const int64_t line = u.first + min(lane & 15, u.n - 1), row = mx_in_row(p, line);
  f32x4 a[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 sum[2];
    tile_product<2>(m, n0 + 16 * h + (lane & 15), p, max(row, (int64_t)0), box, sum);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) a[h][i] = moe_silu_f32(sum[0][i]) * sum[1][i];
  }
  if (threadIdx.x >= 64) return;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(a[i >> 2][i & 3]) & 0x7fffffffu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  if ((lane & 15) >= u.n || row < 0) return;
  const uint32_t byte = mx_scale_byte(top);
  const float s = mx_scale_value(byte);
  uint8_t *c = static_cast<uint8_t *>(p.out) + (line * p.N + n0) / 2 + 2 * (lane >> 4);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w = 0;
    if (byte != 255) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[h][0], a[h][1], s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[h][2], a[h][3], s, 1);
    }
    *reinterpret_cast<uint16_t *>(c + 8 * h) = (uint16_t)w;
  }
  if (lane < 16) scales[(line * p.N + n0) / 32] = (uint8_t)byte;
}

// Units there are at most.
int64_t units(const MxProduct &p) {
  const int64_t routed = p.offsets ? (p.L < p.E ? p.L : p.L / kTile + p.E) : (p.L + kTile - 1) / kTile;
  return routed + (p.shared + kTile - 1) / kTile;
}

template <int DTYPE>
void product(moe_ctx *ctx, const MxProduct &p) {
  const dim3 grid((unsigned)(units(p) * ((p.N + 15) / 16)));
  hipLaunchKernelGGL((mx_stream_kernel<DTYPE, false>), grid, dim3(kWaves * 64), 0, ctx->stream, p);
}

}  // namespace

moe_status launch_mx_product(moe_ctx *ctx, int dtype, const MxProduct &p) {
  switch (dtype) {
    case MOE_FP32: product<MOE_FP32>(ctx, p); break;
    case MOE_BF16: product<MOE_BF16>(ctx, p); break;
    default: product<MOE_FP16>(ctx, p); break;
  }
  MOE_CHECK_LAUNCH("mx product kernel");
  return MOE_OK;
}

moe_status launch_mx_gateup(moe_ctx *ctx, const MxProduct &p, uint8_t *scales) {
  moe_launch(ctx, MOE_STAGE_GATEUP, mx_stream_gateup_kernel, dim3((unsigned)(units(p) * (p.N / 32))),
             dim3(kWaves * 64), p, scales);
  MOE_CHECK_LAUNCH("mx gate/up kernel");
  return MOE_OK;
}

moe_status launch_mx_down(moe_ctx *ctx, int dtype, const MxProduct &p) {
  const dim3 grid((unsigned)(units(p) * ((p.N + 15) / 16)));
  if (dtype == MOE_BF16)
    moe_launch(ctx, MOE_STAGE_DOWN, mx_stream_kernel<MOE_BF16, true>, grid, dim3(kWaves * 64), p);
  else
    moe_launch(ctx, MOE_STAGE_DOWN, mx_stream_kernel<MOE_FP32, true>, grid, dim3(kWaves * 64), p);
  MOE_CHECK_LAUNCH("mx down kernel");
  return MOE_OK;
}
