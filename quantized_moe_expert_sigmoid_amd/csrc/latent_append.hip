// Writer of the latent cache: norm of the latents, rotation of the keys' and
// the queries' rotary parts. One pass over the data; a wave takes one token's
// row (a 16-byte unit a lane) or 64 units of the queries' rotary parts. Sums and
// rotations are fp32, rounded once to the element type. The bytes are the bound:
// 5800 tokens of 64 heads read and write 106 MB in 23 us, 4.6 TB/s (a large copy:
// 4.9); one token is a launch of 2.8 us.
#include "latent.h"

namespace {

constexpr int kWaves = 4;

// One 16-byte unit: pairs (2i, 2i + 1), i = 0..3, turned by (cos, sin) = turn[2i], turn[2i + 1].
template <typename E>
__device__ __forceinline__ u16x8 rotate8(u16x8 v, const float *turn) {
  const float4 t0 = *reinterpret_cast<const float4 *>(turn), t1 = *reinterpret_cast<const float4 *>(turn + 4);
  const float cs[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
  u16x8 o;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float x = E::to_f32(v[i]), y = E::to_f32(v[i + 1]);
    o[i] = E::from_f32(__builtin_fmaf(x, cs[i], -(y * cs[i + 1])));
    o[i + 1] = E::from_f32(__builtin_fmaf(x, cs[i + 1], y * cs[i]));
  }
  return o;
}

template <typename E>
__global__ __launch_bounds__(kWaves * MOE_WAVE) void latent_append_kernel(LatentAppendArgs a) {
  const int lane = threadIdx.x & (MOE_WAVE - 1);
  const int64_t item = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (item < a.T) {
    const int t = (int)item;
    const int64_t slot = a.slot[t];
    const int pos = a.pos[t];
    const bool bad = slot < -1 || slot >= a.n_rows || pos < 0 || pos >= a.n_pos;
    if (bad && lane == 0) atomicOr(a.err, (uint32_t)ERRF_LATENT);
    if (bad || slot < 0) return;
    const uint16_t *src = static_cast<const uint16_t *>(a.kv) + t * a.kv_t;
    uint16_t *dst = static_cast<uint16_t *>(a.cache) + slot * (a.dc + a.dr);
    const int c = lane * 8;
    const bool has = c < a.dc;
    float f[8], sq = 0.0f;
    if (has) {
      const u16x8 v = *reinterpret_cast<const u16x8 *>(src + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = E::to_f32(v[i]);
        sq = __builtin_fmaf(f[i], f[i], sq);
      }
    }
    if (a.norm_w) {
      const float inv = 1.0f / __builtin_sqrtf(wave_sum_f32(sq) / (float)a.dc + a.eps);
      if (has) {
        const float4 w0 = *reinterpret_cast<const float4 *>(a.norm_w + c);
        const float4 w1 = *reinterpret_cast<const float4 *>(a.norm_w + c + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
      }
    }
    if (has) {
      u16x8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = E::from_f32(f[i]);
      *reinterpret_cast<u16x8 *>(dst + c) = o;
    }
    if (c < a.dr)
      *reinterpret_cast<u16x8 *>(dst + a.dc + c) = rotate8<E>(*reinterpret_cast<const u16x8 *>(src + a.dc + c),
                                                              a.turn + (int64_t)pos * a.dr + c);
    return;
  }
  if (!a.q_rope) return;
  const int per_row = a.dr / 8;
  const int64_t unit = (item - a.T) * MOE_WAVE + lane;
  const int64_t row = unit / per_row;
  if (row >= (int64_t)a.T * a.H) return;
  const int u = (int)(unit - row * per_row) * 8;
  const int t = (int)(row / a.H), h = (int)(row - (int64_t)t * a.H);
  const int pos = a.pos[t];
  if (pos < 0 || pos >= a.n_pos) {
    atomicOr(a.err, (uint32_t)ERRF_LATENT);
    return;
  }
  const uint16_t *src = static_cast<const uint16_t *>(a.q_rope) + t * a.rope_t + h * a.rope_h + u;
  *reinterpret_cast<u16x8 *>(static_cast<uint16_t *>(a.q_rope_out) + row * a.dr + u) =
      rotate8<E>(*reinterpret_cast<const u16x8 *>(src), a.turn + (int64_t)pos * a.dr + u);
}

}  // namespace

moe_status launch_latent_append(moe_ctx *ctx, int dtype, const LatentAppendArgs &a) {
  const int64_t units = a.q_rope ? (int64_t)a.T * a.H * (a.dr / 8) : 0;
  const int64_t items = a.T + (units + MOE_WAVE - 1) / MOE_WAVE;
  const dim3 grid((unsigned)((items + kWaves - 1) / kWaves)), block(kWaves * MOE_WAVE);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(latent_append_kernel<Bf16>, grid, block, 0, ctx->stream, a);
  else
    hipLaunchKernelGGL(latent_append_kernel<Fp16>, grid, block, 0, ctx->stream, a);
  MOE_CHECK_LAUNCH("latent_append_kernel");
  return MOE_OK;
}
