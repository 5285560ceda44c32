// C entry points of the latent attention: every argument is checked here,
// before anything is enqueued.
#include "latent.h"

#define REQUIRE(cond, ...)                                 \
  do {                                                     \
    if (!(cond)) return moe_fail(MOE_EINVAL, __VA_ARGS__); \
  } while (0)

static bool pow2_upto(int v, int top) { return v >= 1 && v <= top && (v & (v - 1)) == 0; }

static moe_status cfg_check(const char *fn, moe_ctx *ctx, const moe_latent_cfg *c) {
  REQUIRE(ctx, "%s: ctx is NULL", fn);
  REQUIRE(c, "%s: cfg is NULL", fn);
  MOE_HIP(hipSetDevice(ctx->device));
  REQUIRE(c->dtype == MOE_BF16 || c->dtype == MOE_FP16, "%s: dtype %d is not MOE_BF16 or MOE_FP16", fn, c->dtype);
  REQUIRE(c->n_heads >= 1 && c->n_heads <= 128, "%s: n_heads %d", fn, c->n_heads);
  REQUIRE(c->d_latent == 128 || c->d_latent == 256 || c->d_latent == 512, "%s: d_latent %d not in {128,256,512}", fn,
          c->d_latent);
  REQUIRE(c->d_rope == 32 || c->d_rope == 64, "%s: d_rope %d not in {32,64}", fn, c->d_rope);
  REQUIRE(pow2_upto(c->page_size, 65536), "%s: page_size %d is not a power of two up to 65536", fn, c->page_size);
  return MOE_OK;
}

static int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

extern "C" moe_status moe_latent_append(moe_ctx *ctx, const moe_latent_cfg *cfg, int T, const void *kv, int64_t kv_t,
                                        const float *norm_w, float eps, const float *turn, int n_pos,
                                        const int32_t *pos, const int64_t *slot, void *cache, int64_t n_pages,
                                        const void *q_rope, int64_t rope_t, int64_t rope_h, void *q_rope_out) {
  const char *fn = "moe_latent_append";
  moe_status st = cfg_check(fn, ctx, cfg);
  if (st) return st;
  REQUIRE(T >= 0 && T <= (1 << 20), "%s: T %d", fn, T);
  REQUIRE(eps >= 0.0f, "%s: eps must not be negative or NaN", fn);
  REQUIRE(n_pos >= 0 && n_pages >= 0 && n_pages <= (int64_t)1 << 31, "%s: n_pos %d, n_pages %lld", fn, n_pos,
          (long long)n_pages);
  const int row = cfg->d_latent + cfg->d_rope;
  REQUIRE(kv_t >= row && kv_t % 8 == 0, "%s: kv_t %lld must be a multiple of 8, at least %d", fn, (long long)kv_t, row);
  REQUIRE(!q_rope || (rope_t % 8 == 0 && rope_h % 8 == 0), "%s: rope_t and rope_h must be multiples of 8", fn);
  REQUIRE(!q_rope == !q_rope_out, "%s: q_rope and q_rope_out go together", fn);
  if (T == 0) return MOE_OK;
  REQUIRE(kv && turn && pos && slot && cache, "%s: NULL pointer", fn);
  REQUIRE(moe_aligned16(kv) && moe_aligned16(cache) && moe_aligned16(turn) && moe_aligned16(norm_w) &&
              moe_aligned16(q_rope) && moe_aligned16(q_rope_out),
          "%s: pointers must be 16-byte aligned", fn);
  LatentAppendArgs a{T,     cfg->n_heads, cfg->d_latent, cfg->d_rope, n_pos, n_pages * cfg->page_size,
                     kv,    kv_t,         norm_w,        eps,         turn,  pos,
                     slot,  cache,        q_rope,        rope_t,      rope_h, q_rope_out,
                     ctx->dev_small};
  return launch_latent_append(ctx, cfg->dtype, a);
}

// Checks shared by the two attention forms; *work is false when there is nothing to compute.
static moe_status call_args(const char *fn, moe_ctx *ctx, const moe_latent_cfg *c, const moe_latent_call *call,
                            const void *w_kv, LatentArgs *a, bool *work) {
  *work = false;
  moe_status st = cfg_check(fn, ctx, c);
  if (st) return st;
  REQUIRE(call, "%s: call is NULL", fn);
  REQUIRE((c->d_nope == 64 && c->d_v == 64) || (c->d_nope == 128 && c->d_v == 128) ||
              (c->d_nope == 192 && c->d_v == 256),
          "%s: (d_nope, d_v) (%d, %d) not in {(64,64), (128,128), (192,256)}", fn, c->d_nope, c->d_v);
  REQUIRE(c->scale - c->scale == 0.0f, "%s: scale must be finite", fn);
  REQUIRE(call->T >= 0 && call->T <= (1 << 20), "%s: T %d", fn, call->T);
  REQUIRE(call->B >= 0 && call->B <= 1024, "%s: B %d", fn, call->B);
  REQUIRE(call->nope_t % 8 == 0 && call->nope_h % 8 == 0 && call->rope_t % 8 == 0 && call->rope_h % 8 == 0,
          "%s: query strides must be multiples of 8", fn);
  REQUIRE(call->max_pages >= 0 && call->n_pages >= 0 && call->n_pages <= (int64_t)1 << 31,
          "%s: max_pages %d, n_pages %lld", fn, call->max_pages, (long long)call->n_pages);
  REQUIRE(call->n_pages * c->page_size <= (int64_t)1 << 31, "%s: %lld pages of %d rows: above 2^31 rows", fn,
          (long long)call->n_pages, c->page_size);
  REQUIRE((int64_t)call->max_pages * c->page_size <= (int64_t)1 << 30, "%s: max_pages %d of %d rows: above 2^30 rows",
          fn, call->max_pages, c->page_size);
  if (call->T == 0 || call->B == 0) return MOE_OK;
  REQUIRE(call->q_nope && call->q_rope && call->q_start && call->kv_len && call->out && w_kv, "%s: NULL pointer", fn);
  REQUIRE(call->max_pages == 0 || (call->cache && call->page_table && call->n_pages > 0),
          "%s: the cache and its page table are needed when max_pages > 0", fn);
  REQUIRE(moe_aligned16(call->q_nope) && moe_aligned16(call->q_rope) && moe_aligned16(call->cache) &&
              moe_aligned16(call->out) && moe_aligned16(w_kv),
          "%s: pointers must be 16-byte aligned", fn);
  *a = LatentArgs{call->T,      call->B,          c->n_heads,    c->d_latent,  c->d_rope,
                  c->d_nope,    c->d_v,           log2_of(c->page_size), call->max_pages, call->n_pages,
                  c->scale,     call->q_nope,     call->q_rope,  call->cache,  call->nope_t,
                  call->nope_h, call->rope_t,     call->rope_h,  call->page_table, call->q_start,
                  call->kv_len, nullptr,          nullptr,       w_kv,         call->out,
                  ctx->dev_small};
  *work = true;
  return MOE_OK;
}

extern "C" moe_status moe_latent_attend(moe_ctx *ctx, const moe_latent_cfg *cfg, const moe_latent_call *call,
                                        const void *w_kt, const void *w_kv, const uint64_t *tree, int max_q) {
  const char *fn = "moe_latent_attend";
  LatentArgs a;
  bool work;
  moe_status st = call_args(fn, ctx, cfg, call, w_kv, &a, &work);
  if (st) return st;
  REQUIRE(max_q >= 0 && max_q <= call->T, "%s: max_q %d of T %d", fn, max_q, call->T);
  REQUIRE(!tree || max_q <= 64, "%s: a tree has at most 64 tokens, max_q is %d", fn, max_q);
  if (!work) return MOE_OK;
  REQUIRE(w_kt && moe_aligned16(w_kt), "%s: w_kt is NULL or not 16-byte aligned", fn);
  a.w_kt = w_kt;
  a.tree = tree;
  return launch_latent_attend(ctx, cfg->dtype, a, max_q);
}

extern "C" moe_status moe_latent_prompt(moe_ctx *ctx, const moe_latent_cfg *cfg, const moe_latent_call *call,
                                        const void *w_kv, int64_t n_kv) {
  const char *fn = "moe_latent_prompt";
  LatentArgs a;
  bool work;
  moe_status st = call_args(fn, ctx, cfg, call, w_kv, &a, &work);
  if (st) return st;
  REQUIRE(n_kv >= 0 && n_kv <= (int64_t)1 << 24, "%s: n_kv %lld", fn, (long long)n_kv);
  if (!work) return MOE_OK;
  return launch_latent_prompt(ctx, cfg->dtype, a, n_kv);
}
