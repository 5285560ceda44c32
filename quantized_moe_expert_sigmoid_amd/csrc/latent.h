// Shared by the latent-attention kernels (latent*.hip, latent.cpp).
#pragma once

#include <type_traits>

#include "latent_plan.h"
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

// How the absorbed form's work is shared out (latent_plan.h), written by one
// workgroup of the kernel that absorbs the queries.
struct PlanHead {
  int64_t per;   // units of a workgroup
  int n_shared;  // TileDescs
};
struct LatentPlan {
  LatentArgs a;
  PlanHead *head;
  WgDesc *wg;
  TileDesc *shared;
  int rows, tokens, over;  // rows of a row tile, tokens of a cache tile, units charged for a row tile's start and end
  int n_wg;                // 0: no plan
};

// C[m][h][n] = sum_k A[m][h][k] B[h][n][k]; element (m, h, 0) of A at m a_m + h
// a_h, of C at m c_m + h c_h; B's heads b_h apart. K is a multiple of 64, N of
// 64.
struct HeadGemm {
  const uint16_t *A, *B;
  uint16_t *C;
  const int32_t *lo, *hi;  // nullable, on the device: only rows lo <= m < hi
  int M, N, K;
  int64_t a_m, a_h, b_h, c_m, c_h;
};
moe_status launch_head_gemm(moe_ctx *ctx, int dtype, const HeadGemm &g, int H, const LatentPlan &plan);

// All heads' keys and values of the rows m < *hi (<= M): C[h][m][n] = sum_k
// A[m][k] B[h][n][k], N a multiple of 64, K of 128.
struct ExpandGemm {
  const uint16_t *A, *B;
  uint16_t *C;
  const int32_t *hi;
  int M, H, N, K;
};
moe_status launch_expand_gemm(moe_ctx *ctx, int dtype, const ExpandGemm &g);

// The exponentials are powers of two of c2 z. A negative scale turns the
// queries' signs instead, and zero is taken as 1e-30 (masked scores, -inf, must
// not meet inf x 0).
static inline float latent_c2(float scale) {
  const float c = (scale < 0 ? -scale : scale) * 1.44269504088896340736f;
  return c > 1e-30f ? c : 1e-30f;
}

#if defined(__HIPCC__)

// f(integral_constant<int, A>) .. f(integral_constant<int, B - 1>)
template <int A, int B, typename F>
__device__ __forceinline__ void static_for(F &&f) {
  if constexpr (A < B) {
    f(std::integral_constant<int, A>{});
    static_for<A + 1, B>(f);
  }
}

// s_waitcnt vmcnt(n) alone
#define WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))

typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// bf16 and fp16 elements: conversions round to nearest even, NaN stays NaN.
// mfma: c += a b with v_mfma_f32_32x32x16: lane l holds 8 consecutive k of
// row (a) or column (b) l % 32, k = 8 (l / 32) ..; of c it holds column l % 32,
// rows 8 (i / 4) + 4 (l / 32) + i % 4 for i = 0..15.
struct Bf16 {
  static constexpr int kDtype = MOE_BF16;
  static constexpr uint32_t kExp = 0x7f80;  // exponent bits
  static __device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t from_f32(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
  static __device__ __forceinline__ u16x8 from_f32x8(f32x8 f) {
    return __builtin_bit_cast(u16x8, __builtin_convertvector(f, bf16x8));
  }
  static __device__ __forceinline__ f32x16 mfma(u16x8 a, u16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};
struct Fp16 {
  static constexpr int kDtype = MOE_FP16;
  static constexpr uint32_t kExp = 0x7c00;
  static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t from_f32(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
  static __device__ __forceinline__ u16x8 from_f32x8(f32x8 f) {
    return __builtin_bit_cast(u16x8, __builtin_convertvector(f, f16x8));
  }
  static __device__ __forceinline__ f32x16 mfma(u16x8 a, u16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
};

// Accumulators kept in the accumulation registers (AGPRs) whatever else a
// kernel holds. With ordinary variables the compiler moves such an array to
// vector registers wherever vector instructions touch it (256 of them at once,
// which spills); here every access names the class. The compiler does not see
// matrix instructions inside assembly, so the waits it would add stand here: two
// wait states from a vector write to a product that reads it, and settle()
// before the accumulators are read back.
template <typename E, bool PINNED>
struct AccTile {  // few of them: ordinary variables
  f32x16 c;
  __device__ __forceinline__ void mfma(u16x8 a, u16x8 b, bool) { c = E::mfma(a, b, c); }
  __device__ __forceinline__ void scale(float f) { c *= f; }
  __device__ __forceinline__ f32x4 get4(int j) const { return f32x4{c[4 * j], c[4 * j + 1], c[4 * j + 2], c[4 * j + 3]}; }
};
template <typename E, int N>
__device__ __forceinline__ void settle(AccTile<E, false> (&)[N]) {}
template <typename E, int N>
__device__ __forceinline__ void clear(AccTile<E, false> (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) t[i].c = f32x16{};
}

#if defined(__HIP_DEVICE_COMPILE__)  // the host pass does not know the register class
template <typename E>
struct AccTile<E, true> {
  f32x16 c;
  // c += a b; fresh: an operand may have been written by the vector instruction just before
  __device__ __forceinline__ void mfma(u16x8 a, u16x8 b, bool fresh) {
    if (fresh) asm("s_nop 1" : "+v"(a), "+v"(b));
    if constexpr (E::kDtype == MOE_BF16)
      asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    else
      asm("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float x = c[e], t;
      asm("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1"
          : "+a"(x), "=&v"(t)
          : "v"(f));
      c[e] = x;
    }
  }
  __device__ __forceinline__ float get(int e) const {
    float x;
    asm("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(c[e]));
    return x;
  }
  __device__ __forceinline__ f32x4 get4(int j) const { return f32x4{get(4 * j), get(4 * j + 1), get(4 * j + 2), get(4 * j + 3)}; }
};
template <typename E, int N>
__device__ __forceinline__ void settle(AccTile<E, true> (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+a"(t[i].c));
  asm volatile("s_nop 15\n\ts_nop 15");  // a 32x32x16 product's result is readable after at most 18 states
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+a"(t[i].c));
}
template <typename E, int N>
__device__ __forceinline__ void clear(AccTile<E, true> (&t)[N]) {
  const u16x8 z = {};
#pragma unroll
  for (int i = 0; i < N; ++i)  // volatile: a product each, not one value copied about
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %1, 0" : "=a"(t[i].c) : "v"(z));
  settle(t);
}
#else
template <typename E>
struct AccTile<E, true> {
  __device__ void mfma(u16x8 a, u16x8 b, bool fresh);
  __device__ void scale(float f);
  __device__ float get(int e) const;
  __device__ f32x4 get4(int j) const;
};
template <typename E, int N>
__device__ void settle(AccTile<E, true> (&t)[N]);
template <typename E, int N>
__device__ void clear(AccTile<E, true> (&t)[N]);
#endif

// Results of a 32 x 32 product, four consecutive rows a lane, as elements: the
// 16 rows 16 j .. of a lane's column, of which lane l stores 8, rows 16 j + 8 (l /
// 32) .., in one 16-byte store.
template <typename E>
__device__ __forceinline__ u32x4 rows8(f32x4 a, f32x4 b) {  // rows 16 j + 4 half .., rows 16 j + 8 + 4 half ..
  const f32x8 f = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  const u32x4 p = __builtin_bit_cast(u32x4, E::from_f32x8(f));
  const auto x = __builtin_amdgcn_permlane32_swap(p[0], p[2], false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(p[1], p[3], false, false);
  return u32x4{x[0], y[0], x[1], y[1]};
}

// Maximum of lanes l and l + 32, in both.
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Transposed 8-byte LDS read (ds_read_b64_tr_b16): within 16 lanes, lane 4 e +
// i's address is that of 4 elements of row e, columns 4 i ..; lane c receives
// column c of rows 0..3.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u16x4 lds_read_tr(const uint8_t *p) {
  return __builtin_bit_cast(u16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4 *)(p)));
}
// 16 bytes a lane from global memory straight into LDS, 1 KB a wave: lane i's
// go to LDS byte to + 16 i. Written in assembly because the compiler, which
// does not follow which LDS bytes such a load writes, would wait for all of
// them before any LDS read; there is no result register, and the caller waits
// for the loads by count (vmcnt) before the barrier behind which they are read.
// OFF is added to p and not to the place; on: -1, or 0 for a load that moves
// nothing but is counted all the same. All lanes must be active.
template <int OFF>
__device__ __forceinline__ void lds_load16(const void *p, uint32_t to, int on = -1) {
  // an instruction's offset counts on both sides
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\t"
               "global_load_lds_dwordx4 %0, off offset:%3\n\ts_mov_b64 exec, -1" ::"v"(p),
               "s"(to - OFF), "s"(on), "n"(OFF)
               : "memory");
}

// A sequence's bounds, made safe: tokens [t0, t0 + nq) of the call, len cached
// rows, the first `before` of them older than the call (negative when the
// sequence has fewer rows than tokens).
struct LatentSeq {
  int t0, nq, len, before;
};
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
  const uint64_t v = (uint64_t)p;
  return (const uint8_t *)((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}
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
// Cache row of position j (< len, rows fit 31 bits) of sequence b; a page id out of range is
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
