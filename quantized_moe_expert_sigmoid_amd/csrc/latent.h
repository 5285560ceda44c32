// Shared by the latent-attention kernels (latent*.hip, latent.cpp).
#pragma once

#include "moe_internal.h"

// One call's arrays as the kernels see them (device pointers, strides in elements).
struct LatentArgs {
  int T, B, H, dc, dr, dn, dv;
  int page_shift;  // log2 of the page size
  int max_pages;
  int64_t n_pages;
  float scale;
  const void *q_nope, *q_rope, *cache;
  int64_t nope_t, nope_h, rope_t, rope_h;
  const int32_t *page_table, *q_start, *kv_len;
  const uint64_t *tree;
  const void *w_kt, *w_kv;
  void *out;
  uint32_t *err;
};

struct LatentAppendArgs {
  int T, H, dc, dr, n_pos;
  int64_t n_rows;  // of the cache
  const void *kv;
  int64_t kv_t;
  const float *norm_w;
  float eps;
  const float *turn;
  const int32_t *pos;
  const int64_t *slot;
  void *cache;
  const void *q_rope;
  int64_t rope_t, rope_h;
  void *q_rope_out;
  uint32_t *err;
};

moe_status launch_latent_append(moe_ctx *ctx, int dtype, const LatentAppendArgs &a);
moe_status launch_latent_attend(moe_ctx *ctx, int dtype, const LatentArgs &a, int max_q);
moe_status launch_latent_prompt(moe_ctx *ctx, int dtype, const LatentArgs &a, int64_t n_kv);

#if defined(__HIPCC__)

// bf16 and fp16 elements: conversions round to nearest even, NaN stays NaN.
struct Bf16 {
  uint16_t u;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t from_f32(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
  }
};
struct Fp16 {
  uint16_t u;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t from_f32(float f) {
    return __builtin_bit_cast(uint16_t, (_Float16)f);
  }
};

// A sequence's bounds, made safe: tokens [t0, t0 + nq) of the call, len cached
// rows, the first `before` of them older than the call (negative when the
// sequence has fewer rows than tokens).
struct LatentSeq {
  int t0, nq, len, before;
};
__device__ __forceinline__ LatentSeq latent_seq(const LatentArgs &a, int b) {
  const int lo = a.q_start[b], hi = a.q_start[b + 1], n = a.kv_len[b];
  const int64_t cap = (int64_t)a.max_pages << a.page_shift;
  LatentSeq s;
  const bool ok = lo >= 0 && lo <= hi && hi <= a.T && n >= 0 && n <= cap && !(a.tree && hi - lo > 64);
  if (!ok) atomicOr(a.err, (uint32_t)ERRF_LATENT);
  s.t0 = min(max(lo, 0), a.T);
  s.nq = max(min(hi, a.T) - s.t0, 0);
  s.len = n < 0 ? 0 : (int)min((int64_t)n, cap);
  s.before = s.len - s.nq;
  return s;
}
// Cache row of position j (< len) of sequence b; a page id out of range is
// reported and row 0 taken.
__device__ __forceinline__ int64_t latent_row(const LatentArgs &a, int b, int j) {
  const int p = a.page_table[(int64_t)b * a.max_pages + (j >> a.page_shift)];
  if (p < 0 || p >= a.n_pages) {
    atomicOr(a.err, (uint32_t)ERRF_LATENT);
    return 0;
  }
  return ((int64_t)p << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}

#endif  // __HIPCC__
