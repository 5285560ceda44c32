// Latent attention, expanded form: keys and values of every head computed from
// the cache, then causal attention.
//
// As in the absorbed form a lane keeps one query row: S^T = K Q^T, P^T, O^T +=
// V^T P^T with v_mfma_f32_32x32x16 (see latent_attend.hip for the layouts). A
// workgroup takes 256 tokens of one head, 32 a wave, two waves a SIMD, so that
// one wave's exponentials run under the other's products; its tiles of keys and
// values come into LDS by asynchronous loads, one being read, the others in
// flight.
#include "latent.h"

namespace {

constexpr int kRows = 256;  // query tokens of a workgroup

// The plan: off[b] = first expanded row of sequence b (B + 1 entries), the
// row tiles, the expanded rows' cache rows. Sequences that do not fit n_kv rows are
// reported and left out (off = -1).
struct PromptTile {
  int b, i0;
};
struct PromptWs {
  int32_t *off;      // [B + 1]
  int32_t *n_tiles;
  PromptTile *tile;
  int64_t *rows;     // [n_kv] cache row of an expanded row
  uint16_t *kr;      // [n_kv][dr] rotary keys
  uint16_t *x;       // [H][n_kv][dn + dv] keys and values
  int64_t n_kv;
};

__global__ __launch_bounds__(1024) void prompt_plan_kernel(LatentArgs a, PromptWs ws) {
  __shared__ int scan[1024], tiles[1024];
  const int b = threadIdx.x;
  const LatentSeq s = b < a.B ? latent_seq(a, b) : LatentSeq{};
  const int nt = (s.nq + kRows - 1) / kRows;
  scan[b] = s.len;
  tiles[b] = nt;
  __syncthreads();
  for (int o = 1; o < 1024; o <<= 1) {
    const int v = b >= o ? scan[b - o] : 0, t = b >= o ? tiles[b - o] : 0;
    __syncthreads();
    scan[b] = (int)min((int64_t)scan[b] + v, (int64_t)1 << 30);  // a total that saturates is above n_kv anyway
    tiles[b] += t;
    __syncthreads();
  }
  if (b < a.B) {
    const bool fits = scan[b] <= ws.n_kv;
    if (!fits) atomicOr(a.err, (uint32_t)ERRF_LATENT);
    ws.off[b] = fits ? scan[b] - s.len : -1;
    for (int i = 0; i < nt; ++i) ws.tile[tiles[b] - nt + i] = PromptTile{b, i * kRows};
    // the last sequence that fits ends the expanded rows
    if (fits && (b + 1 == a.B || scan[b + 1] > ws.n_kv)) ws.off[a.B] = scan[b];
    if (!fits && b == 0) ws.off[a.B] = 0;
  }
  if (b == 1023) *ws.n_tiles = tiles[b];
}

// Cache rows and rotary keys of the expanded rows.
__global__ __launch_bounds__(256) void prompt_rows_kernel(LatentArgs a, PromptWs ws) {
  const int b = blockIdx.y, off = ws.off[b];
  if (off < 0) return;
  const LatentSeq s = latent_seq(a, b);
  const int units = a.dr / 8;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < s.len * units; i += gridDim.x * 256) {
    const int j = i / units, u = i - j * units;
    const int64_t row = latent_row(a, b, j);
    if (u == 0) ws.rows[off + j] = row;
    reinterpret_cast<u32x4 *>(ws.kr)[(int64_t)(off + j) * units + u] = *reinterpret_cast<const u32x4 *>(
        static_cast<const uint16_t *>(a.cache) + row * (a.dc + a.dr) + a.dc + 8 * u);
  }
}

__device__ __forceinline__ int swz(int token) { return ((token >> 1 & 1) << 2) | (token >> 2 & 3); }

template <int DN, int DR, int DV>
struct Prompt {
  static constexpr int kTB = DV > 128 ? 1 : 2, kNT = 32 * kTB;  // 32 or 64 tokens a tile
  static constexpr int kPN = DN / 64, kPK = kPN + 1, kPV = DV / 64;  // panels of 64 columns: keys (rotary part last), values
  static constexpr int kPanelB = kNT * 128, kTileB = (kPK + kPV) * kPanelB;
  static constexpr int kBufs = 3;
  static constexpr int kLoads = (kPK + kPV) * kNT / 64;  // of a wave and tile
  static constexpr int kKS = (DN + DR) / 16, kNB = DV / 32;
  static_assert(kBufs * kTileB <= 160 << 10 && (kPK + kPV) * kNT % 64 == 0, "");
};

template <typename E, int DN, int DR, int DV>
__global__ __launch_bounds__(512, 1) void latent_prompt_kernel(LatentArgs a, PromptWs ws, float c2, uint32_t flip) {
  using C = Prompt<DN, DR, DV>;
  constexpr int kNT = C::kNT, kTB = C::kTB, kNB = C::kNB, DX = DN + DV;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kBufs * C::kTileB];
  // an XCD (ids go round the 8 of them) takes whole heads, so that workgroups that share keys share an L2; late
  // tiles, which see the most, go first
  const int nt = uniform(*ws.n_tiles), id = blockIdx.x >> 3;
  const int h = (blockIdx.x & 7) + 8 * (id / max(nt, 1));
  if (nt == 0 || h >= a.H) return;
  const PromptTile pt = ws.tile[nt - 1 - id % nt];
  const int b = uniform(pt.b), i0 = uniform(pt.i0), off0 = uniform(ws.off[b]);
  if (off0 < 0) return;
  const LatentSeq r = latent_seq(a, b);
  const LatentSeq s{uniform(r.t0), uniform(r.nq), uniform(r.len), uniform(r.before)};
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int qi = i0 + wave * 32 + l32;
  const bool live = qi < s.nq;
  const int t = s.t0 + min(qi, s.nq - 1);
  const int last = min(s.nq, i0 + kRows) - 1;                          // the workgroup's last query
  const int n = (max(0, min(s.len, s.before + last + 1)) + kNT - 1) / kNT;  // tiles it sees
  // what the wave sees: all rows up to w_all, none from w_end on
  const int w_all = s.before + i0 + wave * 32 + 1;
  const int w_end = min(s.len, s.before + min(s.nq, i0 + wave * 32 + 32));
  const bool any = i0 + wave * 32 < s.nq;

  u16x8 q[C::kKS];
  {
    const uint16_t *q1 = static_cast<const uint16_t *>(a.q_nope) + t * a.nope_t + h * a.nope_h + 8 * hl;
    const uint16_t *q2 = static_cast<const uint16_t *>(a.q_rope) + t * a.rope_t + h * a.rope_h + 8 * hl;
#pragma unroll
    for (int k = 0; k < C::kKS; ++k) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(16 * k < DN ? q1 + 16 * k : q2 + (16 * k - DN));
      v ^= flip;
      q[k] = __builtin_bit_cast(u16x8, v);
    }
  }

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  const int ld_row = lane >> 3, rb = wave & (kNT / 8 - 1);  // the wave's block of 8 tokens
  const int ld_unit = (lane & 7) ^ swz((8 * rb + ld_row) & 15);
  const uint8_t *xh = reinterpret_cast<const uint8_t *>(ws.x) + ((int64_t)h * ws.n_kv + off0) * (DX * 2);
  const uint8_t *kr = reinterpret_cast<const uint8_t *>(ws.kr) + (int64_t)off0 * (DR * 2);
  auto load = [&](int i) {  // positions behind the last row repeat it
    const int j0 = min(i * kNT + 8 * rb, (s.len - 1) & ~7);
    const int row = min(ld_row, s.len - 1 - j0);
    const uint32_t to = uniform(lds0 + (i % C::kBufs) * C::kTileB + rb * 1024);
    const uint8_t *x0 = uniform(xh + (int64_t)j0 * (DX * 2)), *k0 = uniform(kr + (int64_t)j0 * (DR * 2));
    const uint32_t xo = row * (DX * 2) + ld_unit * 16, ko = row * (DR * 2) + (DR == 64 ? ld_unit : ld_unit & 3) * 16;
    // panels: keys, rotary keys, values; with tiles of 32 tokens two waves share a block of 8
    constexpr int kStep = 64 / kNT;
#pragma unroll
    for (int g = 0; g < C::kPK + C::kPV; g += kStep) {
      const int gg = kStep == 1 ? g : g + uniform(wave >> 2);
      if (gg == C::kPN)
        lds_load16_s(k0, ko, to + gg * C::kPanelB);
      else
        lds_load16_s(uniform(x0 + (gg < C::kPN ? gg : gg - 1) * 128), xo, to + gg * C::kPanelB);
    }
  };
  int k_off[4], v_off[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) k_off[i] = l32 * 128 + (((2 * i + hl) ^ swz(l32 & 15)) << 4);
  const int vt = 4 * hl + ((lane & 15) >> 2);
#pragma unroll
  for (int h8 = 0; h8 < 2; ++h8)
#pragma unroll
    for (int p = 0; p < 2; ++p)
      v_off[h8][p] = (vt + 8 * h8) * 128 +
                     (((4 * p + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swz(vt + 8 * h8)) << 4) + (lane & 1) * 8;

  f32x16 acc[kNB];
#pragma unroll
  for (int i = 0; i < kNB; ++i) acc[i] = f32x16{};
  float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
  for (int i = 0; i < C::kBufs - 1; ++i)
    if (i < n) load(i);
  for (int it = 0; it < n; ++it) {
    if (it + 1 < n)
      WAIT_VM(C::kLoads);
    else
      WAIT_VM(0);
    asm volatile("s_barrier" ::: "memory");
    if (it + 2 < n) load(it + 2);
    const int j0 = it * kNT;
    const bool masked = j0 + kNT > s.before + i0 + 1;  // the same in every wave: some row of the workgroup does not see all
    if (!masked && !any) continue;
    uint8_t *kv = lds + (it % C::kBufs) * C::kTileB, *vv = kv + C::kPK * C::kPanelB;
    f32x16 z[kTB];
#pragma unroll
    for (int tb = 0; tb < kTB; ++tb) z[tb] = f32x16{};
#pragma unroll
    for (int k = 0; k < C::kKS; ++k)
#pragma unroll
      for (int tb = 0; tb < kTB; ++tb)
        z[tb] = E::mfma(*reinterpret_cast<const u16x8 *>(kv + k_off[k & 3] + (k >> 2) * C::kPanelB + tb * 32 * 128), q[k],
                        z[tb]);
    if (masked) {
      // tokens the lane's row sees, as bits
      const uint64_t vis64 = [&] {
        const int c = min(max(min(s.before + qi + 1, s.len) - j0, 0), 64);
        return c == 64 ? ~0ull : (1ull << c) - 1;
      }() >> (4 * hl);
      bool odd = false;
#pragma unroll
      for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool v = (vis64 >> (32 * tb + 8 * (i >> 2) + (i & 3))) & 1;
          odd |= !v & !(__builtin_fabsf(z[tb][i]) < __builtin_inff());
          z[tb][i] = v ? z[tb][i] : -__builtin_inff();
        }
      // An unseen row that holds NaN or infinities would reach the sums as 0 x NaN: see latent_attend.hip.
      if (__syncthreads_or(odd)) {
        bool broken = false;
        const int row = lane & (kNT - 1);
#pragma unroll 1
        for (int c = 0; c < DV / 8; ++c) {
          const u16x8 v = *reinterpret_cast<const u16x8 *>(vv + (c >> 3) * C::kPanelB + row * 128 +
                                                           (((c & 7) ^ swz(row & 15)) << 4));
#pragma unroll
          for (int e = 0; e < 8; ++e) broken |= (v[e] & E::kExp) == E::kExp;
        }
        const uint64_t bad = __ballot(broken);
        __syncthreads();
        if (broken)
#pragma unroll 1
          for (int c = wave; c < DV / 8; c += 8)
            *reinterpret_cast<u32x4 *>(vv + (c >> 3) * C::kPanelB + row * 128 + (((c & 7) ^ swz(row & 15)) << 4)) =
                u32x4{0, 0, 0, 0};
#pragma unroll
        for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            z[tb][i] = (bad >> (32 * tb + 8 * (i >> 2) + 4 * hl + (i & 3))) & 1 ? -__builtin_inff() : z[tb][i];
        if (bad & (kNT == 64 ? ~0ull : 0xffffffffull) & (vis64 << (4 * hl))) l = __builtin_nanf("");
        __syncthreads();
      }
    }
    if (j0 >= w_end) continue;  // nothing of this tile is seen by the wave
    float top = z[0][0];
#pragma unroll
    for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, z[tb][i]);
    top = max_halves(top) * c2;
    // the reference follows the maximum when that has grown by 2^8 (see latent_attend.hip)
    if (__any(top > m + 8.0f)) {
      const float mn = fmaxf(m, top);
      const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < kNB; ++i) acc[i] *= f;
    }
    const float base = m == -__builtin_inff() ? 0.0f : -m;
    u16x8 p[2 * kTB];
#pragma unroll
    for (int tb = 0; tb < kTB; ++tb)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        f32x8 e;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][8 * half + i], c2, base));
          l += e[i];
        }
        p[2 * tb + half] = E::from_f32x8(e);
      }
#pragma unroll
    for (int ks = 0; ks < 2 * kTB; ++ks)
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        const uint8_t *src = vv + (nb >> 1) * C::kPanelB + ks * 16 * 128;
        const u16x4 lo = lds_read_tr(src + v_off[0][nb & 1]), hi = lds_read_tr(src + v_off[1][nb & 1]);
        acc[nb] = E::mfma(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), p[ks], acc[nb]);
      }
  }
  (void)w_all;
  l += __shfl_xor(l, 32, 64);
  if (!live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t *o = static_cast<uint16_t *>(a.out) + ((int64_t)t * a.H + h) * DV + 4 * hl;
#pragma unroll
  for (int i = 0; i < kNB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u16x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = E::from_f32(acc[i][4 * j + e] * inv);
      *reinterpret_cast<u16x4 *>(o + 32 * i + 8 * j) = v;
    }
}

template <typename E, int DN, int DR, int DV>
moe_status launch(moe_ctx *ctx, const LatentArgs &a, int64_t n_kv) {
  const int64_t tiles = a.T / kRows + a.B;  // at most: every sequence adds one tile that is not full
  MoeLayout lay;
  const size_t o_off = lay.take(4 * (size_t)(a.B + 1)), o_nt = lay.take(4), o_tile = lay.take(sizeof(PromptTile) * tiles),
               o_rows = lay.take(8 * (size_t)n_kv), o_kr = lay.take(2 * (size_t)n_kv * DR),
               o_x = lay.take(2 * (size_t)n_kv * a.H * (DN + DV));
  void *scr = nullptr;
  moe_status st = moe_scratch(ctx, lay.size, &scr);
  if (st) return st;
  char *p = static_cast<char *>(scr);
  const PromptWs ws{reinterpret_cast<int32_t *>(p + o_off),  reinterpret_cast<int32_t *>(p + o_nt),
                    reinterpret_cast<PromptTile *>(p + o_tile), reinterpret_cast<int64_t *>(p + o_rows),
                    reinterpret_cast<uint16_t *>(p + o_kr),  reinterpret_cast<uint16_t *>(p + o_x),
                    n_kv};
  hipLaunchKernelGGL(prompt_plan_kernel, dim3(1), dim3(1024), 0, ctx->stream, a, ws);
  MOE_CHECK_LAUNCH("prompt_plan_kernel");
  if (n_kv > 0) {
    hipLaunchKernelGGL(prompt_rows_kernel, dim3(16, a.B), dim3(256), 0, ctx->stream, a, ws);
    MOE_CHECK_LAUNCH("prompt_rows_kernel");
    const HeadGemm expand{static_cast<const uint16_t *>(a.cache), static_cast<const uint16_t *>(a.w_kv), ws.x, ws.rows,
                          nullptr, ws.off + a.B, (int)n_kv, DN + DV, a.dc, a.dc + DR, 0, (int64_t)(DN + DV) * a.dc,
                          DN + DV, n_kv * (DN + DV), 16};
    if ((st = launch_head_gemm(ctx, E::kDtype, expand, a.H, LatentPlan{}))) return st;
  }
  const float c2 = latent_c2(a.scale);
  hipLaunchKernelGGL((latent_prompt_kernel<E, DN, DR, DV>), dim3((unsigned)(tiles * ((a.H + 7) / 8) * 8)), dim3(512), 0,
                     ctx->stream, a, ws, c2, a.scale < 0 ? 0x80008000u : 0u);
  MOE_CHECK_LAUNCH("latent_prompt_kernel");
  return MOE_OK;
}

template <typename E, int DR>
moe_status pick(moe_ctx *ctx, const LatentArgs &a, int64_t n_kv) {
  return a.dn == 64    ? launch<E, 64, DR, 64>(ctx, a, n_kv)
         : a.dn == 128 ? launch<E, 128, DR, 128>(ctx, a, n_kv)
                       : launch<E, 192, DR, 256>(ctx, a, n_kv);
}

}  // namespace

moe_status launch_latent_prompt(moe_ctx *ctx, int dtype, const LatentArgs &a, int64_t n_kv) {
  if (dtype == MOE_BF16) return a.dr == 64 ? pick<Bf16, 64>(ctx, a, n_kv) : pick<Bf16, 32>(ctx, a, n_kv);
  return a.dr == 64 ? pick<Fp16, 64>(ctx, a, n_kv) : pick<Fp16, 32>(ctx, a, n_kv);
}
