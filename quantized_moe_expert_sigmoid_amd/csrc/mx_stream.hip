// Products on microscaled 4-bit floating point for few lines an expert: the
// weights' bytes are the bound.
//
// C^T (n x m) = W X^T with v_mfma_scale_f32_16x16x128_f8f6f4. A wave takes 16
// rows of weights (gate/up: 32 of each, a block of the result), up to 16 lines
// and a share of k; both operands come from memory straight in the products'
// layout: lane l has 16 bytes, block l / 16 of four, of row l % 16. The loads of
// several steps are in flight at once; a workgroup's 8 waves are KW shares of k,
// summed through LDS, times 8 / KW tiles of rows.
#include <type_traits>

#include "mx.h"

namespace {

constexpr int kWaves = 8, kTile = 16;

enum { kPlain, kDown, kGateUp };

struct Rows {
  const uint8_t *c, *s;  // a lane's row: codes from its first block of the wave's first step on, scales
};

// Steps of 128 k of NT tiles of weights' rows, U of them in flight. WORDS: rows of scales are whole words, four blocks a
// word, all four read and the lane's one moved down; otherwise single bytes.
template <int NT, int U, bool WORDS>
__device__ __forceinline__ void run_steps(const Rows &x, const Rows (&w)[NT], int s0, int s1, int blocks,
                                          f32x4 (&acc)[NT]) {
  const int q = (threadIdx.x & 63) >> 4;
  auto batch = [&](int s, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;  // U steps, all blocks there
    i32x4 xc[U], wc[U][NT];
    int xs[U], ws[U][NT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int b = 4 * (kWhole ? s + i : min(s + i, s1 - 1)) + q;
      const int at = kWhole ? b : min(b, blocks - 1), word = WORDS ? at - q : at;
#pragma unroll
      for (int t = 0; t < NT; ++t) wc[i][t] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(w[t].c + at * 16));
      xc[i] = *reinterpret_cast<const i32x4 *>(x.c + at * 16);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        ws[i][t] = WORDS ? *reinterpret_cast<const int *>(w[t].s + word) : w[t].s[at];
      xs[i] = WORDS ? *reinterpret_cast<const int *>(x.s + word) : x.s[at];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!kWhole) {  // blocks behind the row, steps behind the share: nothing times one
        const bool there = s + i < s1 && 4 * (s + i) + q < blocks;
        if (!there) xc[i] = i32x4{};
        xs[i] = there ? xs[i] : WORDS ? 0x7f7f7f7f : 127;
#pragma unroll
        for (int t = 0; t < NT; ++t) ws[i][t] = there ? ws[i][t] : WORDS ? 0x7f7f7f7f : 127;
      }
      const int sx = WORDS ? xs[i] >> 8 * q : xs[i];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = mx_mfma16(wc[i][t], WORDS ? ws[i][t] >> 8 * q : ws[i][t], xc[i], sx, acc[t]);
    }
  };
  int s = s0;
  for (; s + U <= s1 && 4 * (s + U) <= blocks; s += U) batch(s, std::true_type{});
  for (; s < s1; s += U) batch(s, std::false_type{});
}

template <int MODE, int KW, bool WORDS, int DTYPE>
__global__ __launch_bounds__(kWaves * 64, 4) void mx_stream_kernel(MxProduct p, uint8_t *a_scales) {
  typedef MxOut<DTYPE> O;
  constexpr int NT = MODE == kGateUp ? 4 : 1, U = MODE == kGateUp ? 3 : 6, kCols = MODE == kGateUp ? 32 : 16;
  __shared__ f32x4 box[KW > 1 ? kWaves * NT * 64 : 1];
  const int lane = threadIdx.x & 63, wave = mx_uniform((int)(threadIdx.x >> 6)), kw = wave % KW;
  const MxUnit u = mx_unit<kTile>(p, blockIdx.y);
  if (u.n == 0) return;
  const int n0 = ((int)blockIdx.x * (kWaves / KW) + wave / KW) * kCols;
  const int64_t line = u.first + min(lane & 15, u.n - 1), row = mx_in_row(p, line);
  const int blocks = p.K / kMxBlock, steps = (blocks + 3) / 4, per = (steps + KW - 1) / KW;

  f32x4 sum[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) sum[t] = f32x4{};
  if (n0 < p.N) {
    const int64_t xr = max(row, (int64_t)0) * blocks;
    const Rows x{p.x + xr * 16, p.sx + xr};
    Rows w[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t r = (int64_t)min(n0 + (t & 1) * 16 + (lane & 15), p.N - 1) * blocks;
      if constexpr (MODE == kPlain)
        w[t] = Rows{p.w + u.e * p.w_e + r * 16, p.sw + u.e * p.sw_e + r};
      else if constexpr (MODE == kDown)
        w[t] = Rows{p.table[u.e].down + r * 16, p.table[u.e].s_down + r};
      else if (t < 2)
        w[t] = Rows{p.table[u.e].gate + r * 16, p.table[u.e].s_gate + r};
      else
        w[t] = Rows{p.table[u.e].up + r * 16, p.table[u.e].s_up + r};
    }
    run_steps<NT, U, WORDS>(x, w, kw * per, min(steps, (kw + 1) * per), blocks, sum);
  }
  if constexpr (KW > 1) {
#pragma unroll
    for (int t = 0; t < NT; ++t) box[(wave * NT + t) * 64 + lane] = sum[t];
    __syncthreads();
    if (kw) return;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 1; i < KW; ++i) sum[t] += box[((wave + i) * NT + t) * 64 + lane];
  }
  if (n0 >= p.N) return;

  if constexpr (MODE == kGateUp) {
    // lane l has rows 16 t + 4 (l / 16) .. of line l % 16: a block of 32 is four lanes'
    f32x4 a[2];
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[t][i] = moe_silu_f32(sum[t][i]) * sum[2 + t][i];
        top = max(top, __float_as_uint(a[t][i]) & 0x7fffffffu);
      }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if ((lane & 15) >= u.n || row < 0) return;
    const uint32_t byte = mx_scale_byte(top);
    const float s = mx_scale_value(byte);
    uint8_t *c = static_cast<uint8_t *>(p.out) + (line * p.N + n0) / 2 + 2 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t v = 0;
      if (byte != 255) {
        v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[t][0], a[t][1], s, 0);
        v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[t][2], a[t][3], s, 1);
      }
      *reinterpret_cast<uint16_t *>(c + 8 * t) = (uint16_t)v;
    }
    if (lane < 16) a_scales[(line * p.N + n0) / kMxBlock] = (uint8_t)byte;
  } else {
    if ((lane & 15) >= u.n || row < 0) return;
    const int64_t r = mx_out_row(p, line);
    if (r < 0) return;
    const int n = n0 + 4 * (lane >> 4);
    typename O::T *out = static_cast<typename O::T *>(p.out) + r * p.N + n;
    if (p.N % 4 == 0) {
      if (n < p.N) *reinterpret_cast<typename O::V *>(out) = O::of(sum[0]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) out[i] = O::one(sum[0][i]);
    }
  }
}

// Units there are at most.
int64_t units(const MxProduct &p) {
  const int64_t routed = p.offsets ? (p.L < p.E ? p.L : p.L / kTile + p.E) : (p.L + kTile - 1) / kTile;
  return routed + (p.shared + kTile - 1) / kTile;
}

template <int MODE, int KW, bool WORDS, int DTYPE>
void run(moe_ctx *ctx, const MxProduct &p, int64_t n_units, int tiles, uint8_t *a_scales) {
  const int n_wg = (tiles * KW + kWaves - 1) / kWaves;
  const dim3 grid(n_wg, (unsigned)n_units), block(kWaves * 64);
  auto kernel = mx_stream_kernel<MODE, KW, WORDS, DTYPE>;
  if (MODE == kPlain)
    hipLaunchKernelGGL(kernel, grid, block, 0, ctx->stream, p, a_scales);
  else
    moe_launch(ctx, MODE == kDown ? MOE_STAGE_DOWN : MOE_STAGE_GATEUP, kernel, grid, block, p, a_scales);
}

template <int MODE, bool WORDS, int DTYPE>
void pick(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  const int cols = MODE == kGateUp ? 32 : 16, tiles = (p.N + cols - 1) / cols, steps = (p.K + 127) / 128;
  const int64_t n = units(p);
  // as few shares of k as make 16 waves a CU
  int kw = 1;
  while (kw < 8 && n * tiles * kw < 16 * ctx->n_cu && steps >= 4 * kw) kw *= 2;
  switch (kw) {
    case 1: run<MODE, 1, WORDS, DTYPE>(ctx, p, n, tiles, a_scales); break;
    case 2: run<MODE, 2, WORDS, DTYPE>(ctx, p, n, tiles, a_scales); break;
    case 4: run<MODE, 4, WORDS, DTYPE>(ctx, p, n, tiles, a_scales); break;
    default: run<MODE, 8, WORDS, DTYPE>(ctx, p, n, tiles, a_scales); break;
  }
}

template <int MODE, int DTYPE>
void launch(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  if (p.K % 128 == 0)
    pick<MODE, true, DTYPE>(ctx, p, a_scales);
  else
    pick<MODE, false, DTYPE>(ctx, p, a_scales);
}

}  // namespace

moe_status launch_mx_product(moe_ctx *ctx, int dtype, const MxProduct &p) {
  switch (dtype) {
    case MOE_FP32: launch<kPlain, MOE_FP32>(ctx, p, nullptr); break;
    case MOE_BF16: launch<kPlain, MOE_BF16>(ctx, p, nullptr); break;
    default: launch<kPlain, MOE_FP16>(ctx, p, nullptr); break;
  }
  MOE_CHECK_LAUNCH("mx product kernel");
  return MOE_OK;
}

moe_status launch_mx_gateup(moe_ctx *ctx, const MxProduct &p, uint8_t *scales) {
  launch<kGateUp, MOE_FP32>(ctx, p, scales);
  MOE_CHECK_LAUNCH("mx gate/up kernel");
  return MOE_OK;
}

moe_status launch_mx_down(moe_ctx *ctx, int dtype, const MxProduct &p) {
  if (dtype == MOE_BF16)
    launch<kDown, MOE_BF16>(ctx, p, nullptr);
  else
    launch<kDown, MOE_FP32>(ctx, p, nullptr);
  MOE_CHECK_LAUNCH("mx down kernel");
  return MOE_OK;
}
