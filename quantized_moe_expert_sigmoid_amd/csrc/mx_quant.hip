// Rows to microscaled 4-bit floating point and back.
//
// A block of 32 values gets the scale 2^(floor(log2 max|x|) - 2), so that its
// largest value comes to lie in [4, 8); x / scale is rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even mantissa, above 5 to 6). The
// division is by a power of two, so nothing is rounded but the code itself,
// which v_cvt_scalef32_pk_fp4_f32 does two at a time.
//
// Bound by the bytes. A thread has 8 values of a block (16 bytes of a 16-bit
// type, 32 of fp32), four neighbouring lanes share a block's maximum by DPP, and
// a thread stores its 8 codes as one word.
#include "mx.h"

namespace {

// n threads' worth of values, `segs` threads a row (a multiple of four), rows x_t elements apart.
template <int DTYPE>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void *x, int64_t n, int segs, int64_t x_t,
                                                          uint32_t *codes, uint8_t *scales) {
  typedef typename MxOut<DTYPE>::T T;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;  // whole quads: n is a multiple of four
  const int64_t row = i / segs;
  float v[8];
  mx_load8<DTYPE>(static_cast<const T *>(x) + row * x_t + (i - row * segs) * 8, v);
  uint32_t byte;
  codes[i] = mx_codes8(v, byte);
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

template <int DTYPE>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint32_t *codes, const uint8_t *scales, int64_t n,
                                                            void *out) {
  typedef MxOut<DTYPE> O;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint32_t w = codes[i], byte = scales[i >> 2];
  // the product with the scale is exact (or the number nearest to it); 255: NaN
  const float s = byte == 255 ? __builtin_nanf("") : mx_scale_value(byte);
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1),
             c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  typename O::V *o = reinterpret_cast<typename O::V *>(static_cast<typename O::T *>(out) + i * 8);
  o[0] = O::of(f32x4{a[0] * s, a[1] * s, b[0] * s, b[1] * s});
  o[1] = O::of(f32x4{c[0] * s, c[1] * s, d[0] * s, d[1] * s});
}

template <int DTYPE>
moe_status quantize(moe_ctx *ctx, const void *x, int64_t rows, int K, int64_t x_t, uint8_t *codes, uint8_t *scales) {
  const int64_t n = rows * (K / 8);
  hipLaunchKernelGGL(mx_quantize_kernel<DTYPE>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, ctx->stream, x, n,
                     K / 8, x_t, reinterpret_cast<uint32_t *>(codes), scales);
  MOE_CHECK_LAUNCH("mx_quantize_kernel");
  return MOE_OK;
}

template <int DTYPE>
moe_status dequantize(moe_ctx *ctx, const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, void *out) {
  const int64_t n = rows * (K / 8);
  hipLaunchKernelGGL(mx_dequantize_kernel<DTYPE>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, ctx->stream,
                     reinterpret_cast<const uint32_t *>(codes), scales, n, out);
  MOE_CHECK_LAUNCH("mx_dequantize_kernel");
  return MOE_OK;
}

// out[t] = y_shared[t] + sum_j w[t][j] y[t][j], fused multiply-adds in fp32 in slot order, rounded once. Slots of zero
// weight and slots whose id is no expert, or one that an earlier slot of the token has, are left out unread. y: the
// T * k slots in order, then the shared expert's T rows. A workgroup's threads have one token, so that ids and weights
// are scalars; every slot's values are loaded before the first is used.
template <int Y, int DTYPE>
__global__ __launch_bounds__(256) void mx_combine_kernel(const typename MxOut<Y>::T *y, const int32_t *idx,
                                                         const float *w, int T, int k, int E, int H, int has_shared,
                                                         typename MxOut<DTYPE>::T *out) {
  typedef typename MxOut<Y>::V V;
  constexpr int kMaxK = 16;
  const int per = (H / 4 + 255) / 256;
  const int64_t t = blockIdx.x / per;
  const int h = (int)(blockIdx.x % per * 256 + threadIdx.x) * 4;
  if (h >= H) return;
  bool used[kMaxK];
  int id[kMaxK];
  float f[kMaxK];
  V v[kMaxK], sh = {};
  if (has_shared) sh = *reinterpret_cast<const V *>(y + (T * (int64_t)k + t) * H + h);
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    id[j] = idx[t * k + min(j, k - 1)];
    f[j] = w[t * k + min(j, k - 1)];
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    used[j] = j < k && f[j] != 0.0f && id[j] >= 0 && id[j] < E;
#pragma unroll
    for (int i = 0; i < j; ++i) used[j] &= id[i] != id[j];
    if (used[j]) v[j] = *reinterpret_cast<const V *>(y + (t * k + j) * H + h);
  }
  f32x4 acc = {(float)sh[0], (float)sh[1], (float)sh[2], (float)sh[3]};
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)
    if (used[j]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = __builtin_fmaf(f[j], (float)v[j][c], acc[c]);
    }
  *reinterpret_cast<typename MxOut<DTYPE>::V *>(out + t * H + h) = MxOut<DTYPE>::of(acc);
}

template <int Y, int DTYPE>
void combine(moe_ctx *ctx, const void *y, const int32_t *idx, const float *w, int T, int k, int E, int H,
             int has_shared, void *out) {
  typedef typename MxOut<Y>::T TY;
  typedef typename MxOut<DTYPE>::T TO;
  moe_launch(ctx, MOE_STAGE_COMBINE, mx_combine_kernel<Y, DTYPE>,
             dim3((unsigned)(T * ((H / 4 + 255) / 256))), dim3(256), static_cast<const TY *>(y), idx, w, T, k,
             E, H, has_shared, static_cast<TO *>(out));
}

}  // namespace

moe_status launch_mx_quantize(moe_ctx *ctx, int dtype, const void *x, int64_t rows, int K, int64_t x_t,
                              uint8_t *codes, uint8_t *scales) {
  switch (dtype) {
    case MOE_FP32: return quantize<MOE_FP32>(ctx, x, rows, K, x_t, codes, scales);
    case MOE_BF16: return quantize<MOE_BF16>(ctx, x, rows, K, x_t, codes, scales);
    default: return quantize<MOE_FP16>(ctx, x, rows, K, x_t, codes, scales);
  }
}

moe_status launch_mx_dequantize(moe_ctx *ctx, int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int K, void *out) {
  switch (dtype) {
    case MOE_FP32: return dequantize<MOE_FP32>(ctx, codes, scales, rows, K, out);
    case MOE_BF16: return dequantize<MOE_BF16>(ctx, codes, scales, rows, K, out);
    default: return dequantize<MOE_FP16>(ctx, codes, scales, rows, K, out);
  }
}

moe_status launch_mx_combine(moe_ctx *ctx, int y_dtype, int dtype, const void *y, const int32_t *idx, const float *w,
                             int T, int k, int E, int H, int has_shared, void *out) {
  if (y_dtype == MOE_BF16)
    combine<MOE_BF16, MOE_BF16>(ctx, y, idx, w, T, k, E, H, has_shared, out);
  else if (dtype == MOE_FP16)
    combine<MOE_FP32, MOE_FP16>(ctx, y, idx, w, T, k, E, H, has_shared, out);
  else
    combine<MOE_FP32, MOE_FP32>(ctx, y, idx, w, T, k, E, H, has_shared, out);
  MOE_CHECK_LAUNCH("mx_combine_kernel");
  return MOE_OK;
}
