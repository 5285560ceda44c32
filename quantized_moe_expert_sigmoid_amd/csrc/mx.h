// Shared by the kernels on microscaled 4-bit floating point (mx*.hip, mx.cpp).
//
// A row of K values is K / 32 blocks; a block has one scale byte s, worth
// 2^(s - 127) (255: not a number), and 32 codes of 4 bits, two a byte, the
// first in the low half: sign, then 0, 0.5, 1, 1.5, 2, 3, 4 or 6. So a block's
// codes are 16 bytes, what one lane gives to a matrix instruction.
#pragma once

#include <type_traits>

#include "moe_internal.h"

constexpr int kMxBlock = 32;

// A product's arrays as the kernels see them (device pointers).
struct MxProduct {
  const uint8_t *x, *sx;  // codes and scales of X rows of K values
  int64_t X;
  // weights, N rows of K values an expert: expert e's at w + e * w_e ..., or where table says
  const uint8_t *w, *sw;
  int64_t w_e, sw_e;
  const moe_mx_expert_w *table;
  int N, K;
  // lines: line l is row in_rows[l] / k of x (NULL: l) and goes to row out_rows[l] of out (NULL: l)
  const int32_t *offsets;  // [E + 1], expert e's lines are offsets[e] ..; NULL: one expert has all L of them
  int E;
  int64_t L;
  const int32_t *in_rows, *out_rows;
  int k;
  int64_t shared;  // lines L .. L + shared - 1 are expert E's and rows 0 .. of x where `tokens`, else rows L ..
  bool tokens;     // x has a row a token
  void *out;
  int64_t R;  // rows of out
  uint32_t *err;
};

moe_status launch_mx_quantize(moe_ctx *ctx, int dtype, const void *x, int64_t rows, int K, int64_t x_t,
                              uint8_t *codes, uint8_t *scales);
moe_status launch_mx_dequantize(moe_ctx *ctx, int dtype, const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int K, void *out);
// Tokens' rows in 4 bits and, by expert, their entries t * k + j.
moe_status launch_mx_prep(moe_ctx *ctx, int dtype, const void *x, int T, int H, uint8_t *codes, uint8_t *scales,
                          const int32_t *idx, int k, int E, int32_t *counts, int32_t *offsets, int32_t *perm);
// Whether a product goes to the tile kernels.
bool mx_tiles(const moe_ctx *ctx, const MxProduct &p);
// out = x w^T line by line
moe_status launch_mx_product(moe_ctx *ctx, int dtype, const MxProduct &p);
moe_status launch_mx_tile_product(moe_ctx *ctx, int dtype, const MxProduct &p);
// The experts' FFN of T tokens on hidden states x of x_dtype, each slot by itself: gate and up into lines (codes a and
// scales sa, slot by slot, then the shared expert's), then down with the combine into out.
struct MxOne {
  const void *x;
  int dtype;
  const moe_mx_expert_w *table;
  const int32_t *idx;
  const float *w;
  int T, H, I, E, k, shared;
  uint8_t *a, *sa;
  void *out;
  uint32_t *err;
};
moe_status launch_mx_one(moe_ctx *ctx, const MxOne &p);
// silu(x gate^T) * (x up^T) line by line (the table's gate and up), in 4 bits: out's row l is line l
moe_status launch_mx_gateup(moe_ctx *ctx, const MxProduct &p, uint8_t *scales);
// the table's down, fp32 results
moe_status launch_mx_down(moe_ctx *ctx, const MxProduct &p);
moe_status launch_mx_combine(moe_ctx *ctx, int dtype, const float *y, const int32_t *idx, const float *w, int T, int k, int E,
                             int H, int has_shared, void *out);

#if defined(__HIPCC__)

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// Results' types: four fp32 values rounded once (to nearest even) and stored together.
template <int DTYPE>
struct MxOut;
template <>
struct MxOut<MOE_FP32> {
  typedef float T;
  typedef f32x4 V;
  static __device__ __forceinline__ V of(f32x4 v) { return v; }
  static __device__ __forceinline__ T one(float v) { return v; }
  static __device__ __forceinline__ float back(T v) { return v; }
};
template <>
struct MxOut<MOE_BF16> {
  typedef __bf16 T;
  typedef bf16x4 V;
  static __device__ __forceinline__ V of(f32x4 v) { return __builtin_convertvector(v, bf16x4); }
  static __device__ __forceinline__ T one(float v) { return (__bf16)v; }
  static __device__ __forceinline__ float back(T v) { return (float)v; }
};
template <>
struct MxOut<MOE_FP16> {
  typedef _Float16 T;
  typedef f16x4 V;
  static __device__ __forceinline__ V of(f32x4 v) { return __builtin_convertvector(v, f16x4); }
  static __device__ __forceinline__ T one(float v) { return (_Float16)v; }
  static __device__ __forceinline__ float back(T v) { return (float)v; }
};

// The scale byte of a block whose largest |x| has these bits: the largest value
// comes to lie in [4, 8); values above 6 become 6. Zero and the smallest
// numbers get the smallest scale, an infinity or NaN anywhere the byte 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  const uint32_t e = top >> 23;
  return e == 255 ? 255u : e < 2 ? 0u : e - 2;
}
// 2^(s - 127), s < 255
__device__ __forceinline__ float mx_scale_value(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x400000u); }

template <int DTYPE>
__device__ __forceinline__ void mx_load8(const void *p, float (&v)[8]) {
  if constexpr (DTYPE == MOE_FP32) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const typename MxOut<DTYPE>::V a = reinterpret_cast<const typename MxOut<DTYPE>::V *>(p)[0],
                                   b = reinterpret_cast<const typename MxOut<DTYPE>::V *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)a[i], v[4 + i] = (float)b[i];
  }
}

// Maximum over the four lanes of a quad, in all of them.
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));  // lanes 1, 0, 3, 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));  // lanes 2, 3, 0, 1
}

// Codes of a thread's 8 values of a block and, in all four lanes, the block's scale byte.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t &byte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);  // orders NaN above infinity
  byte = mx_scale_byte(mx_quad_max(top));
  if (byte == 255) return 0;
  const float s = mx_scale_value(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

// silu(g) = g / (1 + 2^(-g log2 e)) with the hardware's exponential and reciprocal, each within a unit in the last place;
// the product with log2 e in two parts, since its rounding, times g, is an error of the exponential. Below -64 both 1 and
// the exponential are taken 2^-64 times as large, and so in the end the quotient: exp(-g) passes fp32's range at -88.7,
// silu(g) falls below its normal numbers at -91.8 and below half the smallest number at -108.7. Where |hi| is 192 or more
// the exponential is 0 or infinite and has no second part (0 or infinity times one is NaN). Within 2^-21 of the value where
// that is a normal number, else within 2^-148 (every number was tried); -infinity: NaN, as by the formula. (Exact division
// and a polynomial: 60 instructions a value, 2 us of a tile's end.)
__device__ __forceinline__ float mx_silu(float g) {
  constexpr float kLog2e = 1.4426950408889634f, kRest = (float)(1.4426950408889634074 - (double)kLog2e);
  const float hi = -g * kLog2e, lo = __builtin_fmaf(-g, kRest, __builtin_fmaf(-g, kLog2e, -hi));
  const bool far = g < -64.0f;
  const float one = far ? 0x1p-64f : 1.0f;
  const float e = __builtin_amdgcn_exp2f(far ? hi - 64.0f : hi);  // hi - 64 is exact: smaller than hi, a multiple of its last place
  // e (1 + lo ln 2)
  const float d = one + (__builtin_fabsf(hi) < 192.0f ? __builtin_fmaf(e, lo * 0.6931471805599453f, e) : e);
  return g * __builtin_amdgcn_rcpf(d) * one;
}

// c += a b^T with v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds block l / 16 (of four) of row l % 16 of a and of b and
// in the low bytes of sa and sb these blocks' scales; of c it holds column l % 16 (b's row), rows 4 (l / 16) + i.
__device__ __forceinline__ f32x4 mx_mfma16(i32x4 a, int sa, i32x4 b, int sb, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1),
                                                          __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), c,
                                                          4, 4, 0, sa, 0, sb);
}

// f(integral_constant<int, A>) .. f(integral_constant<int, B - 1>)
template <int A, int B, typename F>
__device__ __forceinline__ void mx_static_for(F &&f) {
  if constexpr (A < B) {
    f(std::integral_constant<int, A>{});
    mx_static_for<A + 1, B>(f);
  }
}

// c += a b^T: lane l holds 32 k of row l % 32 of a and of b, block l / 32 of two, and byte S of sa and sb is its scale; of
// c it holds column l % 32 (b's row), rows 8 (i / 4) + 4 (l / 32) + i % 4.
template <int S>
__device__ __forceinline__ f32x16 mx_mfma32(i32x4 a, int sa, i32x4 b, int sb, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1),
                                                         __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), c,
                                                         4, 4, S, sa, S, sb);
}

static __device__ __attribute__((aligned(16))) const uint8_t mx_zeros[16] = {};

// 16 bytes a lane from global memory straight into LDS, in order of lanes from byte `to` on; on, high: -1, or 0 for a load
// that moves nothing but is counted all the same, for the lower and the upper 32 lanes. In assembly so that the compiler does not wait for it; the kernel waits
// by count (vmcnt). All lanes must be active.
__device__ __forceinline__ void mx_lds_load16(const void *p, uint32_t to, int on, int high) {
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %3\n\t"
               "global_load_lds_dwordx4 %0, off\n\ts_mov_b64 exec, -1" ::"v"(p), "s"(to), "s"(on), "s"(high)
               : "memory");
}
// -1 where a < b, else 0, in a scalar register: computed from a comparison, the compiler has been seen to hand the
// assembly above a vector register.
__device__ __forceinline__ int mx_below(int a, int b) {
  int r;
  asm("s_cmp_lt_i32 %1, %2\n\ts_cselect_b32 %0, -1, 0" : "=s"(r) : "s"(a), "s"(b) : "scc");
  return r;
}
// The same for a byte a lane, each into a word.
__device__ __forceinline__ void mx_lds_load1(const void *p, uint32_t to, int on) {
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\t"
               "global_load_lds_ubyte %0, off\n\ts_mov_b64 exec, -1" ::"v"(p), "s"(to), "s"(on)
               : "memory");
}
// s_waitcnt vmcnt(n) alone
#define WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))

// A unit of work: up to `tile` lines of one expert.
struct MxUnit {
  int e;           // expert; E for the shared one
  int64_t first;   // its first line
  int n;           // lines; 0: no such unit
};
__device__ __forceinline__ int mx_uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t mx_uniform(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)mx_uniform((int)(v >> 32)) << 32 | (uint32_t)mx_uniform((int)v));
}

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int mx_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from 1, 2, 4, 8 lanes before, within 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 of the 16 before, lane 31
  return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
}

// The lines in tiles: units are the shared expert's tiles first, then each
// expert's, in order. Every wave finds its unit by itself, in one round trip
// to memory: a lane counts the tiles of E / 64 experts in a row (at most 16), a
// scan over the wave's lanes and a ballot name the lane. Offsets that do not
// ascend within 0 .. L are reported and cut to that range.
template <int TILE>
struct MxUnits {
  int v[17];  // offsets of this lane's experts, the next lane's first one last
  int tiles, sum, per;

  __device__ __forceinline__ bool used(int i) const { return i <= 4 || (i + 3) / 4 * 4 - 4 < per; }  // all lanes alike
  __device__ __forceinline__ void load(const MxProduct &p) {
    if (!p.offsets) return;
    const int lane = (int)(threadIdx.x & 63), top = (int)p.L;
    per = (p.E + 63) / 64;
    const int e0 = lane * per;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (used(4 * c + 1)) {
        if (c == 0) v[0] = p.offsets[min(e0, p.E)];
#pragma unroll
        for (int i = 1; i <= 4; ++i) v[4 * c + i] = p.offsets[min(e0 + min(4 * c + i, per), p.E)];
      }
    bool ok = v[0] >= 0 && v[0] <= top;
    v[0] = min(max(v[0], 0), top);
    tiles = 0;
#pragma unroll
    for (int i = 1; i <= 16; ++i)
      if (used(i)) {
        ok &= v[i] >= v[i - 1] && v[i] <= top;
        v[i] = max(v[i - 1], min(v[i], top));
        tiles += (v[i] - v[i - 1] + TILE - 1) / TILE;
      }
    if (!ok) atomicOr(p.err, (uint32_t)ERRF_MX);
    sum = mx_scan(tiles);
  }
  __device__ __forceinline__ MxUnit find(const MxProduct &p, int64_t u) const {
    const int64_t s = (p.shared + TILE - 1) / TILE;
    if (u < s) return MxUnit{p.E, p.L + u * TILE, (int)min((int64_t)TILE, p.shared - u * TILE)};
    u -= s;
    if (!p.offsets) {
      const int64_t left = p.L - u * TILE;
      return MxUnit{0, u * TILE, (int)max((int64_t)0, min((int64_t)TILE, left))};
    }
    const uint64_t past = __ballot((int64_t)sum > u);
    if (!past) return MxUnit{0, 0, 0};
    const int who = __ffsll((unsigned long long)past) - 1;
    int left = (int)u - __builtin_amdgcn_readlane(sum - tiles, who), lo = __builtin_amdgcn_readlane(v[0], who);
    MxUnit r{0, 0, 0};
#pragma unroll
    for (int i = 1; i <= 16; ++i)
      if (used(i) && r.n == 0) {
        const int hi = __builtin_amdgcn_readlane(v[i], who), n = (hi - lo + TILE - 1) / TILE;
        if (left < n) r = MxUnit{who * per + i - 1, lo + left * TILE, min(TILE, hi - lo - left * TILE)};
        left -= n;
        lo = hi;
      }
    return r;
  }
};

// Row of x of a line, and where its result goes; -1: out of range, which is reported.
__device__ __forceinline__ int64_t mx_in_row(const MxProduct &p, int64_t line) {
  int64_t r = line;
  if (p.tokens && line >= p.L)
    r = line - p.L;
  else if (p.in_rows)
    r = p.in_rows[line] / p.k;
  if (r >= 0 && r < p.X) return r;
  atomicOr(p.err, (uint32_t)ERRF_MX);
  return -1;
}
__device__ __forceinline__ int64_t mx_out_row(const MxProduct &p, int64_t line) {
  const int64_t r = line < p.L && p.out_rows ? p.out_rows[line] : line;
  if (r >= 0 && r < p.R) return r;
  atomicOr(p.err, (uint32_t)ERRF_MX);
  return -1;
}

#endif  // __HIPCC__
