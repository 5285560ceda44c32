// Products on microscaled 4-bit floating point that are too small for the tile
// kernels to fill the chip: few lines, few rows of weights.
//
// C^T (n x m) = W X^T with v_mfma_scale_f32_16x16x128_f8f6f4. A workgroup takes 16
// rows of weights and up to 16 NM lines; its 8 waves share out k and sum through
// LDS. Both operands come from memory straight in the products' layout: lane l
// has 16 bytes, block l / 16 of four, of row l % 16. All of a wave's loads of U
// steps are in flight at once, so a share of k takes one or two round trips to
// memory where a tile takes one for every two stages.
// One line, 24576 rows of 6144 (80 MB): 15.4 us, 5.2 TB/s; what tiles take instead
// stands at mx_tiles (mx_tile.hip).
#include <type_traits>

#include "mx.h"

namespace {

constexpr int kWaves = 8;

struct Rows {
  const uint8_t *c, *s;  // a lane's row: its codes and its scales
};

// Steps of 128 k, U of them in flight. WORDS: rows of scales are whole words, four blocks a word, all four read and the
// lane's one moved down; otherwise single bytes.
template <int NM, int U, bool WORDS>
__device__ __forceinline__ void run_steps(const Rows (&x)[NM], const Rows &w, int s0, int s1, int blocks,
                                          f32x4 (&acc)[NM]) {
  const int q = (threadIdx.x & 63) >> 4;
  auto batch = [&](int s, auto whole) {
    constexpr bool kWhole = decltype(whole)::value;  // U steps, all blocks there
    i32x4 xc[U][NM], wc[U];
    int xs[U][NM], ws[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!kWhole && s + i >= s1) continue;  // all lanes alike
      const int b = 4 * (s + i) + q, at = kWhole ? b : min(b, blocks - 1), word = WORDS ? at - q : at;
      wc[i] = *reinterpret_cast<const i32x4 *>(w.c + at * 16);
      ws[i] = WORDS ? *reinterpret_cast<const int *>(w.s + word) : w.s[at];
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        xc[i][j] = *reinterpret_cast<const i32x4 *>(x[j].c + at * 16);
        xs[i][j] = WORDS ? *reinterpret_cast<const int *>(x[j].s + word) : x[j].s[at];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (!kWhole && s + i >= s1) continue;
      const bool there = kWhole || 4 * (s + i) + q < blocks;  // behind a row's end nothing times one
      const int sw = there ? (WORDS ? ws[i] >> 8 * q : ws[i]) : 127;
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        const int sx = there ? (WORDS ? xs[i][j] >> 8 * q : xs[i][j]) : 127;
        acc[j] = mx_mfma16(wc[i], sw, there ? xc[i][j] : i32x4{}, sx, acc[j]);
      }
    }
  };
  int s = s0;
  for (; s + U <= s1 && 4 * (s + U) <= blocks; s += U) batch(s, std::true_type{});
  for (; s < s1; s += U) batch(s, std::false_type{});
}

template <int NM, int U, bool WORDS, int DTYPE>
__global__ __launch_bounds__(kWaves * 64, 4) void mx_stream_kernel(MxProduct p) {
  typedef MxOut<DTYPE> O;
  __shared__ f32x4 box[kWaves * NM * 64];
  const int lane = threadIdx.x & 63, wave = mx_uniform((int)(threadIdx.x >> 6));
  MxUnits<16 * NM> lines;
  lines.load(p);
  const MxUnit u = lines.find(p, blockIdx.y);
  if (u.n == 0) return;
  const int n0 = (int)blockIdx.x * 16;
  const int blocks = p.K / kMxBlock, steps = (blocks + 3) / 4, per = (steps + kWaves - 1) / kWaves;
  Rows x[NM];
#pragma unroll
  for (int j = 0; j < NM; ++j) {
    const int64_t r = max(mx_in_row(p, u.first + min(16 * j + (lane & 15), u.n - 1)), (int64_t)0) * blocks;
    x[j] = Rows{p.x + r * 16, p.sx + r};
  }
  const int64_t r = (int64_t)min(n0 + (lane & 15), p.N - 1) * blocks;
  const Rows w{p.w + u.e * p.w_e + r * 16, p.sw + u.e * p.sw_e + r};
  f32x4 sum[NM];
#pragma unroll
  for (int j = 0; j < NM; ++j) sum[j] = f32x4{};
  run_steps<NM, U, WORDS>(x, w, wave * per, min(steps, (wave + 1) * per), blocks, sum);
#pragma unroll
  for (int j = 0; j < NM; ++j) box[(wave * NM + j) * 64 + lane] = sum[j];
  __syncthreads();
  if (wave >= NM) return;
  // wave j: lines 16 j ..
  f32x4 c = box[wave * 64 + lane];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) c += box[(i * NM + wave) * 64 + lane];
  const int m = 16 * wave + (lane & 15), n = n0 + 4 * (lane >> 4);
  if (m >= u.n || (p.in_rows && mx_in_row(p, u.first + m) < 0)) return;
  const int64_t to = mx_out_row(p, u.first + m);
  if (to < 0) return;
  typename O::T *out = static_cast<typename O::T *>(p.out) + to * p.N + n;
  if (p.N % 4 == 0) {
    if (n < p.N) *reinterpret_cast<typename O::V *>(out) = O::of(c);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < p.N) out[i] = O::one(c[i]);
  }
}

template <int NM, int U, bool WORDS, int DTYPE>
void run(moe_ctx *ctx, const MxProduct &p) {
  const int64_t units = p.offsets ? (p.L < p.E ? p.L : p.L / (16 * NM) + p.E) : (p.L + 16 * NM - 1) / (16 * NM);
  hipLaunchKernelGGL((mx_stream_kernel<NM, U, WORDS, DTYPE>), dim3((p.N + 15) / 16, (unsigned)units), dim3(kWaves * 64), 0,
                     ctx->stream, p);
}

template <bool WORDS, int DTYPE>
void pick(moe_ctx *ctx, const MxProduct &p) {
  const int64_t lines = p.offsets ? p.L / p.E : p.L;
  if (lines <= 16)
    run<1, 6, WORDS, DTYPE>(ctx, p);
  else if (lines <= 32)
    run<2, 6, WORDS, DTYPE>(ctx, p);
  else
    run<4, 3, WORDS, DTYPE>(ctx, p);
}

template <int DTYPE>
void launch(moe_ctx *ctx, const MxProduct &p) {
  if (p.K % (4 * kMxBlock) == 0 && (((uintptr_t)p.sx | (uintptr_t)p.sw) & 3) == 0)
    pick<true, DTYPE>(ctx, p);
  else
    pick<false, DTYPE>(ctx, p);
}

}  // namespace

moe_status launch_mx_product(moe_ctx *ctx, int dtype, const MxProduct &p) {
  switch (dtype) {
    case MOE_FP32: launch<MOE_FP32>(ctx, p); break;
    case MOE_BF16: launch<MOE_BF16>(ctx, p); break;
    default: launch<MOE_FP16>(ctx, p); break;
  }
  MOE_CHECK_LAUNCH("mx product kernel");
  return MOE_OK;
}
