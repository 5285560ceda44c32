// Latent attention, expanded form: keys and values of every head computed from
// the cache, then causal attention.
#include "latent.h"

namespace {

// The prompts' plan: off[b] = first expanded row of sequence b (B + 1 entries),
// the expanded rows' cache rows. Sequences that do not fit n_kv rows are
// reported and left out (off = -1).
__global__ __launch_bounds__(1024) void prompt_plan_kernel(LatentArgs a, int64_t n_kv, int32_t *off) {
  __shared__ int scan[1024];
  const int b = threadIdx.x;
  int len = b < a.B ? latent_seq(a, b).len : 0;
  // saturating sum: a total that does not fit is above n_kv anyway
  scan[b] = len;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = b >= o ? scan[b - o] : 0;
    __syncthreads();
    scan[b] = (int)min((int64_t)scan[b] + v, (int64_t)1 << 30);
    __syncthreads();
  }
  if (b < a.B) {
    const bool fits = scan[b] <= n_kv;
    if (!fits) atomicOr(a.err, (uint32_t)ERRF_LATENT);
    off[b] = fits ? scan[b] - len : -1;
  }
  if (b == 0) {
    int total = 0;
    for (int i = 0; i < a.B; ++i)
      if (scan[i] <= n_kv) total = scan[i];
    off[a.B] = total;
  }
}

__global__ __launch_bounds__(256) void prompt_rows_kernel(LatentArgs a, const int32_t *off, int64_t *rows) {
  const int b = blockIdx.y;
  if (off[b] < 0) return;
  const LatentSeq s = latent_seq(a, b);
  for (int j = blockIdx.x * 256 + threadIdx.x; j < s.len; j += gridDim.x * 256) rows[off[b] + j] = latent_row(a, b, j);
}

// One query row: query i of sequence b, head h.
template <typename E>
__global__ __launch_bounds__(256) void attend_row_kernel(LatentArgs a, const uint16_t *q1, int64_t q1_t, int64_t q1_h,
                                                         int dk, int dv, const uint16_t *kx, const uint16_t *vx,
                                                         int64_t x_row, int64_t x_h, const int32_t *off, uint16_t *o,
                                                         int64_t o_t, int64_t o_h) {
  __shared__ float q[640], p[256], red[4];
  __shared__ int64_t row[256];
  const int tid = threadIdx.x, t = blockIdx.x, h = blockIdx.y;
  int b = -1;
  LatentSeq s{};
  for (int i = 0; i < a.B; ++i) {
    const LatentSeq c = latent_seq(a, i);
    if (t >= c.t0 && t < c.t0 + c.nq) {
      b = i;
      s = c;
    }
  }
  if (b < 0 || (off && off[b] < 0)) return;
  const uint16_t *q2 = static_cast<const uint16_t *>(a.q_rope) + t * a.rope_t + h * a.rope_h;
  for (int i = tid; i < dk + a.dr; i += 256) q[i] = E::to_f32(i < dk ? q1[t * q1_t + h * q1_h + i] : q2[i - dk]);
  float m = -__builtin_inff(), l = 0.0f, acc0 = 0.0f, acc1 = 0.0f;
  const int i = t - s.t0;
  const uint16_t *cache = static_cast<const uint16_t *>(a.cache);
  for (int j0 = 0; j0 < s.len; j0 += 256) {
    __syncthreads();
    const int j = j0 + tid;
    bool vis = j < s.len;
    if (vis && j >= s.before) {
      const int r = j - s.before;
      vis = a.tree ? r < 64 && ((a.tree[t] >> r) & 1) : r <= i;
    }
    float z = -__builtin_inff();
    row[tid] = -1;
    if (vis) {
      const int64_t cr = latent_row(a, b, j);
      const uint16_t *k2 = cache + cr * (a.dc + a.dr) + a.dc;
      const uint16_t *k1 = kx ? kx + (off[b] + j) * x_row + h * x_h : cache + cr * (a.dc + a.dr);
      row[tid] = kx ? off[b] + j : cr;
      z = 0.0f;
      for (int d = 0; d < dk; ++d) z = __builtin_fmaf(q[d], E::to_f32(k1[d]), z);
      for (int d = 0; d < a.dr; ++d) z = __builtin_fmaf(q[dk + d], E::to_f32(k2[d]), z);
      z *= a.scale;
    }
    const float wm = wave_max_f32(z);
    if ((tid & 63) == 0) red[tid >> 6] = wm;
    __syncthreads();
    const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = mn == -__builtin_inff() ? 0.0f : mn;
    const float w = vis ? expf(z - base) : 0.0f, f = expf(m - base);
    const float ws = wave_sum_f32(w);
    p[tid] = w;
    __syncthreads();
    if ((tid & 63) == 0) red[tid >> 6] = ws;
    __syncthreads();
    l = l * f + (red[0] + red[1] + red[2] + red[3]);
    m = mn;
    acc0 *= f;
    acc1 *= f;
    for (int n = 0; n < 256; ++n) {
      if (row[n] < 0) continue;
      const uint16_t *v = vx ? vx + row[n] * x_row + h * x_h : cache + row[n] * (a.dc + a.dr);
      if (tid < dv) acc0 = __builtin_fmaf(p[n], E::to_f32(v[tid]), acc0);
      if (tid + 256 < dv) acc1 = __builtin_fmaf(p[n], E::to_f32(v[tid + 256]), acc1);
    }
  }
  uint16_t *out = o + t * o_t + h * o_h;
  const bool none = m == -__builtin_inff();
  if (tid < dv) out[tid] = E::from_f32(none ? 0.0f : acc0 / l);
  if (tid + 256 < dv) out[tid + 256] = E::from_f32(none ? 0.0f : acc1 / l);
}

template <typename E>
moe_status prompt(moe_ctx *ctx, const LatentArgs &a, int64_t n_kv) {
  MoeLayout lay;
  const int dx = a.dn + a.dv;
  const size_t o_off = lay.take(4 * (size_t)(a.B + 1)), o_rows = lay.take(8 * (size_t)n_kv),
               o_x = lay.take(2 * (size_t)n_kv * a.H * dx);
  void *scr = nullptr;
  moe_status st = moe_scratch(ctx, lay.size, &scr);
  if (st) return st;
  int32_t *off = reinterpret_cast<int32_t *>((char *)scr + o_off);
  int64_t *rows = reinterpret_cast<int64_t *>((char *)scr + o_rows);
  uint16_t *x = reinterpret_cast<uint16_t *>((char *)scr + o_x);
  hipLaunchKernelGGL(prompt_plan_kernel, dim3(1), dim3(1024), 0, ctx->stream, a, n_kv, off);
  MOE_CHECK_LAUNCH("prompt_plan_kernel");
  const int64_t hx = (int64_t)a.H * dx;
  if (n_kv > 0) {
    hipLaunchKernelGGL(prompt_rows_kernel, dim3(16, a.B), dim3(256), 0, ctx->stream, a, off, rows);
    MOE_CHECK_LAUNCH("prompt_rows_kernel");
    if ((st = launch_head_gemm(ctx, E::kDtype,
                           HeadGemm{(const uint16_t *)a.cache, (const uint16_t *)a.w_kv, x, rows, nullptr, off + a.B, (int)n_kv,
                                    dx, a.dc, a.dc + a.dr, 0, (int64_t)dx * a.dc, hx, dx},
                           a.H)))
      return st;
  }
  hipLaunchKernelGGL(attend_row_kernel<E>, dim3(a.T, a.H), dim3(256), 0, ctx->stream, a, (const uint16_t *)a.q_nope,
                     a.nope_t, a.nope_h, a.dn, a.dv, x, x + a.dn, hx, (int64_t)dx, off, (uint16_t *)a.out,
                     (int64_t)a.H * a.dv, (int64_t)a.dv);
  MOE_CHECK_LAUNCH("attend_row_kernel");
  return MOE_OK;
}

}  // namespace

moe_status launch_latent_prompt(moe_ctx *ctx, int dtype, const LatentArgs &a, int64_t n_kv) {
  return dtype == MOE_BF16 ? prompt<Bf16>(ctx, a, n_kv) : prompt<Fp16>(ctx, a, n_kv);
}
