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
// 2047 rows of 6144 bf16: 7.5 us, and 7.1 us back; 32768 rows of 6144 fp32 (912 MB):
// 194 us (4.7 TB/s) and 181 us back (5.0), a copy's rate here being 5.1.
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

// Lines by expert and the tokens' rows in 4 bits, in one launch: workgroup 0 buckets the (token, slot) entries (an id of -1
// gets none; one that is no expert, or that an earlier slot of the token has, gets none and is reported), the others
// quantise. Entries of an expert are in no particular order: a line's result does not depend on its place. 64 tokens of 8
// experts: 6 us, 2048: 17 to 21 (two launches: 13 us more with 64 tokens).
constexpr int kPrepEntries = 32768;  // 128 KB of LDS

template <int DTYPE>
__global__ __launch_bounds__(1024) void mx_prep_kernel(const void *x, int64_t n, uint32_t *codes, uint8_t *scales,
                                                       const int32_t *idx, int entries, int k, int E, int32_t *offsets,
                                                       int32_t *perm, uint32_t *err) {
  extern __shared__ uint16_t ids[];  // [entries], then the entries in their order (stored one by one they took 10 us)
  uint16_t *order = ids + entries;
  __shared__ int count[1024], sums[16];
  const int tid = threadIdx.x;
  if (blockIdx.x) {
    const int64_t i = (int64_t)(blockIdx.x - 1) * 1024 + tid;
    if (i >= n) return;
    float v[8];
    mx_load8<DTYPE>(static_cast<const typename MxOut<DTYPE>::T *>(x) + i * 8, v);
    uint32_t byte;
    codes[i] = mx_codes8(v, byte);
    if ((tid & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    return;
  }
  const int lane = tid & 63, wave = tid >> 6;
  count[tid] = 0;
  __syncthreads();
  for (int t = tid; t * k < entries; t += 1024) {  // a thread has a token's ids at once
    int id[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) id[j] = j < k ? idx[t * k + j] : -1;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      bool ok = id[j] >= 0 && id[j] < E;
#pragma unroll
      for (int i = 0; i < j; ++i) ok &= id[i] != id[j];
      bad |= !ok && id[j] != -1;
      if (j < k) ids[t * k + j] = ok ? (uint16_t)id[j] : (uint16_t)0xffff;
      if (ok) atomicAdd(&count[id[j]], 1);
    }
    if (bad) atomicOr(err, (uint32_t)ERRF_BAD_INDEX);
  }
  __syncthreads();
  const int c = count[tid], sum = mx_scan(c);
  if (lane == 63) sums[wave] = sum;
  __syncthreads();
  int at = sum - c;
  for (int w = 0; w < wave; ++w) at += sums[w];
  if (tid < E) offsets[tid] = at;
  if (tid == E - 1) offsets[E] = at + c;
  count[tid] = at;
  __syncthreads();
  for (int i = tid; i < entries; i += 1024)
    if (ids[i] != 0xffff) order[atomicAdd(&count[ids[i]], 1)] = (uint16_t)i;
  __syncthreads();
  int all = 0;
  for (int w = 0; w < 16; ++w) all += sums[w];
  for (int i = tid; i < all; i += 1024) perm[i] = order[i];
}

template <int DTYPE>
moe_status prep(moe_ctx *ctx, const void *x, int T, int H, uint8_t *codes, uint8_t *scales, const int32_t *idx, int k, int E,
                int32_t *offsets, int32_t *perm) {
  const int64_t n = (int64_t)T * (H / 8);
  moe_launch_lds(ctx, MOE_STAGE_BUCKET, mx_prep_kernel<DTYPE>, dim3((unsigned)((n + 1023) / 1024 + 1)), dim3(1024),
                 (size_t)T * k * 4, x, n, reinterpret_cast<uint32_t *>(codes), scales, idx, T * k, k, E, offsets, perm,
                 ctx->dev_small);
  MOE_CHECK_LAUNCH("mx_prep_kernel");
  return MOE_OK;
}

// out[t] = y_shared[t] + sum_j w[t][j] y[t][j], fused multiply-adds in fp32 in slot order, rounded once. Slots of zero
// weight and slots whose id is no expert, or one that an earlier slot of the token has, are left out unread. y: the
// T * k slots in order, then the shared expert's T rows. A workgroup's threads have one token, so that ids and weights
// are scalars; every slot's values are loaded before the first is used. 2048 tokens of 8 slots and the shared
// expert's, hidden 6144, bf16 out (478 MB): 89 us, 5.4 TB/s; 64 tokens 5.8 us. (Slots in bf16: 45 us, and 5% less for the
// whole call, but a token's result then depends on how many share its call, and is off by 0.0024 of its norm, not 0.0017.)
template <int DTYPE>
__global__ __launch_bounds__(256) void mx_combine_kernel(const float *y, const int32_t *idx, const float *w, int T, int k,
                                                         int E, int H, int has_shared, typename MxOut<DTYPE>::T *out) {
  constexpr int kMaxK = 16;
  struct V8 {
    f32x4 a, b;
  };
  const int per = (H / 8 + 255) / 256;
  const int64_t t = blockIdx.x / per;
  const int h = (int)(blockIdx.x % per * 256 + threadIdx.x) * 8;
  if (h >= H) return;
  bool used[kMaxK];
  int id[kMaxK];
  float f[kMaxK];
  V8 v[kMaxK], sh = {};
  if (has_shared) sh = *reinterpret_cast<const V8 *>(y + (T * (int64_t)k + t) * H + h);
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
    if (used[j]) v[j] = *reinterpret_cast<const V8 *>(y + (t * k + j) * H + h);
  }
  f32x4 a = sh.a, b = sh.b;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)
    if (used[j]) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        a[c] = __builtin_fmaf(f[j], v[j].a[c], a[c]);
        b[c] = __builtin_fmaf(f[j], v[j].b[c], b[c]);
      }
    }
  typename MxOut<DTYPE>::V *o = reinterpret_cast<typename MxOut<DTYPE>::V *>(out + t * H + h);
  o[0] = MxOut<DTYPE>::of(a);
  o[1] = MxOut<DTYPE>::of(b);
}

template <int DTYPE>
void combine(moe_ctx *ctx, const float *y, const int32_t *idx, const float *w, int T, int k, int E, int H, int has_shared,
             void *out) {
  moe_launch(ctx, MOE_STAGE_COMBINE, mx_combine_kernel<DTYPE>, dim3((unsigned)(T * ((H / 8 + 255) / 256))), dim3(256), y,
             idx, w, T, k, E, H, has_shared, static_cast<typename MxOut<DTYPE>::T *>(out));
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

moe_status launch_mx_prep(moe_ctx *ctx, int dtype, const void *x, int T, int H, uint8_t *codes, uint8_t *scales,
                          const int32_t *idx, int k, int E, int32_t *counts, int32_t *offsets, int32_t *perm) {
  if ((int64_t)T * k > kPrepEntries) {  // more than one workgroup buckets well
    {
      MoeTimer tm_(ctx, MOE_STAGE_BUCKET);
      moe_status st = launch_mx_quantize(ctx, dtype, x, T, H, H, codes, scales);
      if (st) return st;
    }
    return launch_bucket_public(ctx, idx, T, k, E, counts, offsets, perm);
  }
  switch (dtype) {
    case MOE_FP32: return prep<MOE_FP32>(ctx, x, T, H, codes, scales, idx, k, E, offsets, perm);
    case MOE_BF16: return prep<MOE_BF16>(ctx, x, T, H, codes, scales, idx, k, E, offsets, perm);
    default: return prep<MOE_FP16>(ctx, x, T, H, codes, scales, idx, k, E, offsets, perm);
  }
}

moe_status launch_mx_combine(moe_ctx *ctx, int dtype, const float *y, const int32_t *idx, const float *w, int T, int k, int E,
                             int H, int has_shared, void *out) {
  switch (dtype) {
    case MOE_FP32: combine<MOE_FP32>(ctx, y, idx, w, T, k, E, H, has_shared, out); break;
    case MOE_BF16: combine<MOE_BF16>(ctx, y, idx, w, T, k, E, H, has_shared, out); break;
    default: combine<MOE_FP16>(ctx, y, idx, w, T, k, E, H, has_shared, out);
  }
  MOE_CHECK_LAUNCH("mx_combine_kernel");
  return MOE_OK;
}
