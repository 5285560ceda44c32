// C entry points of the operators on microscaled 4-bit floating point: every
// argument is checked here, before anything is enqueued.
#include "mx.h"

#define REQUIRE(cond, ...)                                 \
  do {                                                     \
    if (!(cond)) return moe_fail(MOE_EINVAL, __VA_ARGS__); \
  } while (0)

static moe_status bind(const char *fn, moe_ctx *ctx) {
  REQUIRE(ctx, "%s: ctx is NULL", fn);
  MOE_HIP(hipSetDevice(ctx->device));
  return MOE_OK;
}

static bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16 || dtype == MOE_FP32; }
static bool k_ok(int K) { return K > 0 && K % kMxBlock == 0 && K <= (1 << 16); }
static bool dim_ok(int v) { return v > 0 && v % 64 == 0 && v <= 8192; }

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxValues = (int64_t)1 << 34;  // of one quantiser's call

extern "C" moe_status moe_mx_quantize(moe_ctx *ctx, int dtype, const void *x, int64_t rows, int K, int64_t x_t,
                                      uint8_t *codes, uint8_t *scales) {
  const char *fn = "moe_mx_quantize";
  moe_status st = bind(fn, ctx);
  if (st) return st;
  REQUIRE(dtype_ok(dtype), "%s: dtype %d is not MOE_BF16, MOE_FP16 or MOE_FP32", fn, dtype);
  REQUIRE(k_ok(K), "%s: K %d must be a positive multiple of 32, at most 65536", fn, K);
  REQUIRE(rows >= 0 && rows <= kMaxRows && rows * K <= kMaxValues, "%s: rows %lld of %d", fn, (long long)rows, K);
  const int unit = dtype == MOE_FP32 ? 4 : 8;
  REQUIRE(x_t >= K && x_t % unit == 0, "%s: x_t %lld must be a multiple of %d, at least K %d", fn, (long long)x_t, unit,
          K);
  if (rows == 0) return MOE_OK;
  REQUIRE(x && codes && scales, "%s: NULL pointer", fn);
  REQUIRE(moe_aligned16(x) && moe_aligned16(codes), "%s: x and codes must be 16-byte aligned", fn);
  return launch_mx_quantize(ctx, dtype, x, rows, K, x_t, codes, scales);
}

extern "C" moe_status moe_mx_dequantize(moe_ctx *ctx, int dtype, const uint8_t *codes, const uint8_t *scales,
                                        int64_t rows, int K, void *out) {
  const char *fn = "moe_mx_dequantize";
  moe_status st = bind(fn, ctx);
  if (st) return st;
  REQUIRE(dtype_ok(dtype), "%s: dtype %d is not MOE_BF16, MOE_FP16 or MOE_FP32", fn, dtype);
  REQUIRE(k_ok(K), "%s: K %d must be a positive multiple of 32, at most 65536", fn, K);
  REQUIRE(rows >= 0 && rows <= kMaxRows && rows * K <= kMaxValues, "%s: rows %lld of %d", fn, (long long)rows, K);
  if (rows == 0) return MOE_OK;
  REQUIRE(codes && scales && out, "%s: NULL pointer", fn);
  REQUIRE(moe_aligned16(codes) && moe_aligned16(out), "%s: codes and out must be 16-byte aligned", fn);
  return launch_mx_dequantize(ctx, dtype, codes, scales, rows, K, out);
}

// Checks shared by the two products.
static moe_status product_check(const char *fn, moe_ctx *ctx, int dtype, const MxProduct &p) {
  moe_status st = bind(fn, ctx);
  if (st) return st;
  REQUIRE(dtype_ok(dtype), "%s: dtype %d is not MOE_BF16, MOE_FP16 or MOE_FP32", fn, dtype);
  REQUIRE(k_ok(p.K), "%s: K %d must be a positive multiple of 32, at most 65536", fn, p.K);
  REQUIRE(p.N >= 0 && p.N <= (1 << 20), "%s: N %d", fn, p.N);
  REQUIRE(p.L >= 0 && p.L <= (1 << 22) && p.X >= 0 && p.X <= kMaxRows && p.R >= 0 && p.R <= kMaxRows,
          "%s: %lld lines, %lld rows of x, %lld of out", fn, (long long)p.L, (long long)p.X, (long long)p.R);
  if (p.L == 0 || p.N == 0) return MOE_OK;
  REQUIRE(p.x && p.sx && p.w && p.sw && p.out, "%s: NULL pointer", fn);
  REQUIRE(moe_aligned16(p.x) && moe_aligned16(p.w) && moe_aligned16(p.out),
          "%s: the codes of x and w, and out, must be 16-byte aligned", fn);
  return MOE_OK;
}

// The product by the kernels that its lines call for.
static moe_status product_run(moe_ctx *ctx, int dtype, MxProduct &p) {
  p.err = ctx->dev_small;
  return mx_tiles(ctx, p) ? launch_mx_tile_product(ctx, dtype, p) : launch_mx_product(ctx, dtype, p);
}

extern "C" moe_status moe_mx_matmul(moe_ctx *ctx, int dtype, const uint8_t *x, const uint8_t *sx, int64_t M,
                                    const uint8_t *w, const uint8_t *sw, int N, int K, void *out) {
  MxProduct p{};
  p.x = x, p.sx = sx, p.X = M, p.w = w, p.sw = sw, p.N = N, p.K = K, p.E = 1, p.L = M, p.k = 1, p.out = out, p.R = M;
  moe_status st = product_check("moe_mx_matmul", ctx, dtype, p);
  if (st || M == 0 || N == 0) return st;
  return product_run(ctx, dtype, p);
}

extern "C" moe_status moe_mx_grouped_matmul(moe_ctx *ctx, int dtype, const uint8_t *x, const uint8_t *sx, int64_t X,
                                            const uint8_t *w, const uint8_t *sw, int E, int N, int K,
                                            const int32_t *offsets, int64_t L, const int32_t *in_rows,
                                            const int32_t *out_rows, void *out, int64_t R) {
  const char *fn = "moe_mx_grouped_matmul";
  MxProduct p{};
  p.x = x, p.sx = sx, p.X = X, p.w = w, p.sw = sw, p.N = N, p.K = K, p.E = E, p.L = L, p.k = 1, p.out = out, p.R = R;
  p.offsets = offsets, p.in_rows = in_rows, p.out_rows = out_rows;
  moe_status st = product_check(fn, ctx, dtype, p);
  if (st) return st;
  REQUIRE(E >= 1 && E <= 1024, "%s: E %d", fn, E);
  REQUIRE(in_rows || X >= L, "%s: without in_rows x needs %lld rows, it has %lld", fn, (long long)L, (long long)X);
  REQUIRE(out_rows || R >= L, "%s: without out_rows out needs %lld rows, it has %lld", fn, (long long)L, (long long)R);
  if (L == 0 || N == 0) return MOE_OK;
  REQUIRE(offsets, "%s: offsets is NULL", fn);
  REQUIRE(X > 0 && R > 0, "%s: %lld lines, but x has %lld rows and out %lld", fn, (long long)L, (long long)X,
          (long long)R);
  p.w_e = (int64_t)N * (K / 2);
  p.sw_e = (int64_t)N * (K / kMxBlock);
  return product_run(ctx, dtype, p);
}

extern "C" size_t moe_mx_expert_layout(int H, int I, size_t *offsets_host) {
  if (H <= 0 || I <= 0 || H % 64 || I % 64) return 0;
  const size_t codes = (size_t)H * I / 2, scales = (size_t)H * I / kMxBlock;
  const size_t part[6] = {codes, codes, codes, scales, scales, scales};
  MoeLayout l;
  for (int i = 0; i < 6; ++i) {
    const size_t o = l.take(part[i]);
    if (offsets_host) offsets_host[i] = o;
  }
  return l.size;
}

extern "C" moe_status moe_expert_ffn_mx(moe_ctx *ctx, int dtype, const moe_mx_expert_w *experts, int has_shared,
                                        const void *x, const int32_t *topk_idx, const float *topk_w, int T, int H,
                                        int I, int E, int k, void *out) {
  const char *fn = "moe_expert_ffn_mx";
  moe_status st = bind(fn, ctx);
  if (st) return st;
  REQUIRE(dtype_ok(dtype), "%s: dtype %d is not MOE_BF16, MOE_FP16 or MOE_FP32", fn, dtype);
  REQUIRE(T >= 0, "%s: T %d", fn, T);
  REQUIRE(dim_ok(H) && dim_ok(I), "%s: H %d and I %d must be positive multiples of 64, <= 8192", fn, H, I);
  REQUIRE(E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E, "%s: E %d k %d", fn, E, k);
  REQUIRE((int64_t)T * (k + 1) <= (1 << 22), "%s: T*(k+1) too large", fn);
  if (T == 0) return MOE_OK;
  REQUIRE(experts && x && topk_idx && topk_w && out, "%s: NULL pointer", fn);
  REQUIRE(moe_aligned16(x) && moe_aligned16(out), "%s: x and out must be 16-byte aligned", fn);
  REQUIRE(x != out, "%s: out must not be x", fn);
  const int64_t routed = (int64_t)T * k, lines = routed + (has_shared ? T : 0);
  void *scr = nullptr;
  MoeLayout l;
  const size_t o_a = l.take((size_t)lines * I / 2), o_sa = l.take((size_t)lines * I / kMxBlock);
  // slot by slot: no bucketing, no launches for the quantiser and the combine; tokens that share experts read them twice
  if (T == 1 || (T <= 3 && E >= 4 * T * k)) {
    if ((st = moe_scratch(ctx, l.size, &scr))) return st;
    uint8_t *b = static_cast<uint8_t *>(scr);
    return launch_mx_one(ctx, MxOne{x, dtype, experts, topk_idx, topk_w, T, H, I, E, k, has_shared ? 1 : 0, b + o_a, b + o_sa,
                                    out, ctx->dev_small});
  }
  const size_t o_y = l.take((size_t)lines * H * 4), o_x = l.take((size_t)T * H / 2),
               o_sx = l.take((size_t)T * H / kMxBlock), o_counts = l.take(4 * E), o_offsets = l.take(4 * (E + 1)),
               o_perm = l.take(4 * routed);
  if ((st = moe_scratch(ctx, l.size, &scr))) return st;
  uint8_t *b = static_cast<uint8_t *>(scr);
  int32_t *offsets = reinterpret_cast<int32_t *>(b + o_offsets), *perm = reinterpret_cast<int32_t *>(b + o_perm);
  if ((st = launch_mx_prep(ctx, dtype, x, T, H, b + o_x, b + o_sx, topk_idx, k, E, reinterpret_cast<int32_t *>(b + o_counts),
                           offsets, perm)))
    return st;
  MxProduct p{};
  p.x = b + o_x, p.sx = b + o_sx, p.X = T, p.table = experts, p.N = I, p.K = H, p.E = E, p.L = routed, p.k = k;
  p.offsets = offsets, p.in_rows = perm, p.shared = has_shared ? T : 0, p.tokens = true;
  p.out = b + o_a, p.R = lines, p.err = ctx->dev_small;
  if ((st = launch_mx_gateup(ctx, p, b + o_sa))) return st;
  p.x = b + o_a, p.sx = b + o_sa, p.X = lines, p.N = H, p.K = I, p.tokens = false;
  p.out_rows = p.in_rows, p.in_rows = nullptr, p.out = b + o_y;
  if ((st = launch_mx_down(ctx, p))) return st;
  return launch_mx_combine(ctx, dtype, reinterpret_cast<float *>(b + o_y), topk_idx, topk_w, T, k, E, H, has_shared, out);
}
