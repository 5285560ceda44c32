// Products on microscaled 4-bit floating point in tiles through LDS, for many
// lines an expert.
//
// C^T (n x m) = W X^T with v_mfma_scale_f32_32x32x64_f8f6f4. A workgroup takes BM
// lines of one expert and BN rows of weights; steps of 128 k, 64 bytes a row and
// one word of four scale bytes, come by asynchronous loads. A row's four units of
// 16 bytes lie at unit ^ (row / 4 % 4), so that the 16 rows of a read meet
// different banks. Half l / 32 of a wave takes units 2 (l / 32) and the next, so
// that a lane's two scale bytes of a step are neighbours and the instruction picks
// one of them.
//
// A wave has the operands of the next product step in registers before the
// present one begins, and a stage's place is loaded again while its last products
// run: STAGES - 1 stages are in flight.
#include "mx.h"

namespace {

__device__ __attribute__((aligned(16))) const uint8_t mx_zeros[16] = {};

// 16 or 4 bytes a lane from global memory straight into LDS, in order of lanes from byte `to` on; on: -1, or 0 for a load
// that moves nothing but is counted all the same. In assembly so that the compiler does not wait for it; the kernel waits
// by count (vmcnt). All lanes must be active.
__device__ __forceinline__ void lds_load16(const void *p, uint32_t to, int on) {
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\t"
               "global_load_lds_dwordx4 %0, off\n\ts_mov_b64 exec, -1" ::"v"(p), "s"(to), "s"(on)
               : "memory");
}
__device__ __forceinline__ void lds_load4(const void *p, uint32_t to, int on) {
  asm volatile("s_mov_b32 m0, %1\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\t"
               "global_load_lds_dword %0, off\n\ts_mov_b64 exec, -1" ::"v"(p), "s"(to), "s"(on)
               : "memory");
}
// s_waitcnt vmcnt(n) alone
#define WAIT_VM(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | (7 << 4) | (15 << 8))

// c += a b^T: lane l holds 32 k of row l % 32 of a and of b, block l / 32 of two, and byte S of sa and sb is its scale; of
// c it holds column l % 32 (b's row), rows 8 (i / 4) + 4 (l / 32) + i % 4.
template <int S>
__device__ __forceinline__ f32x16 mfma32(i32x4 a, int sa, i32x4 b, int sb, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1),
                                                         __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), c,
                                                         4, 4, S, sa, S, sb);
}

enum { kPlain, kDown, kGateUp };

// How workgroups map to tiles: blocks of G units x GN column tiles go round the 8 XCDs; within one, units run fastest.
struct TileMap {
  int n_tiles, units, g, gn;
};
TileMap tile_map(int64_t units, int n_tiles) {
  TileMap m;
  m.n_tiles = n_tiles, m.units = (int)units;
  m.g = units < 4 ? (int)units : 4;
  m.gn = 32 / m.g < n_tiles ? 32 / m.g : n_tiles;
  return m;
}
unsigned tile_grid(const TileMap &m) {
  const int64_t blocks = (int64_t)((m.units + m.g - 1) / m.g) * ((m.n_tiles + m.gn - 1) / m.gn);
  return (unsigned)((blocks + 7) / 8 * 8 * m.g * m.gn);
}

template <int BM, int BN, int WM, int WN, int STAGES, int OCC, int MODE, int DTYPE>
__global__ __launch_bounds__(WM *WN * 64, OCC) void mx_tile_kernel(MxProduct p, TileMap map, uint8_t *a_scales) {
  typedef MxOut<DTYPE> O;
  constexpr int kWaves = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr int kRows = BM + BN, kStage = kRows * 64, kScales = kRows * 4;
  constexpr int kLoads = kRows / 16 / kWaves, kLoadsS = (kRows / 64 + kWaves - 1) / kWaves, kPer = kLoads + kLoadsS;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;  // of the result
  static_assert(BM % 64 == 0 && BN % 64 == 0 && kRows % (16 * kWaves) == 0);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * (kStage + kScales)];

  const int xcd = blockIdx.x & 7, j0 = blockIdx.x >> 3, per_block = map.g * map.gn;
  const int block = j0 / per_block * 8 + xcd, rest = j0 % per_block, across = (map.n_tiles + map.gn - 1) / map.gn;
  const int unit = block / across * map.g + rest % map.g, nt = block % across * map.gn + rest / map.g;
  if (unit >= map.units || nt >= map.n_tiles) return;
  const MxUnit u = mx_unit<BM>(p, unit);
  if (u.n == 0) return;
  const int n0 = nt * kCols;
  const int lane = threadIdx.x & 63, wave = mx_uniform((int)(threadIdx.x >> 6)), l32 = lane & 31, hl = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  const uint8_t *w[2], *sw[2];
  if constexpr (MODE == kPlain) {
    w[0] = w[1] = p.w + u.e * p.w_e;
    sw[0] = sw[1] = p.sw + u.e * p.sw_e;
  } else if constexpr (MODE == kDown) {
    w[0] = w[1] = p.table[u.e].down;
    sw[0] = sw[1] = p.sw ? p.sw + u.e * p.sw_e : p.table[u.e].s_down;
  } else {
    w[0] = p.table[u.e].gate, w[1] = p.table[u.e].up;
    sw[0] = p.sw ? p.sw + u.e * p.sw_e : p.table[u.e].s_gate;
    sw[1] = p.sw ? p.sw2 + u.e * p.sw_e : p.table[u.e].s_up;
  }
  const int blocks = p.K / kMxBlock, steps = (blocks + 3) / 4, full = blocks / 4;
  // sources: row r of the tile, the lines first, then the weights' rows (gate's, then up's)
  auto row_of = [&](int r, int &which) -> int64_t {
    if (r < BM) return max(mx_in_row(p, u.first + min(r, u.n - 1)), (int64_t)0);
    const int n = r - BM;
    which = MODE == kGateUp && n >= kCols;
    return min(n0 + n - which * kCols, p.N - 1);
  };
  const int mine = (lane & 3) ^ (lane >> 4 & 3);  // the unit of its row that a lane loads
  const uint8_t *src[kLoads], *src_s[kLoadsS];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = (i * kWaves + wave) * 16 + (lane >> 2);
    int which = 0;
    const int64_t row = row_of(r, which);
    src[i] = (r < BM ? p.x : w[which]) + (row * blocks + mine) * 16;
  }
#pragma unroll
  for (int i = 0; i < kLoadsS; ++i) {
    const int r = min((i * kWaves + wave) * 64, kRows - 64) + lane;
    int which = 0;
    const int64_t row = row_of(r, which);
    src_s[i] = r < BM ? p.sx + row * p.sx_t : sw[which] + row * p.sw_t;
  }
  auto load = [&](int s) {
    const uint32_t to = lds0 + s % STAGES * kStage + wave * 1024, to_s = lds0 + STAGES * kStage + s % STAGES * kScales;
    const int on = mx_uniform(s < steps ? -1 : 0);
    const bool there = s < full || 4 * s + mine < blocks;  // behind a row's end zeros
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      lds_load16(there ? src[i] + s * 64 : mx_zeros, mx_uniform((int)(to + i * kWaves * 1024)), on);
#pragma unroll
    for (int i = 0; i < kLoadsS; ++i) {
      const int r = (i * kWaves + wave) * 64;
      lds_load4(src_s[i] + s * 4, mx_uniform((int)(to_s + min(r, kRows - 64) * 4)), mx_uniform(r < kRows ? on : 0));
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) load(s);

  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

  // a lane's places: rows l32 of 32, unit 2 hl + k
  int row_x[FM], row_w[FN], off[2];
#pragma unroll
  for (int j = 0; j < FM; ++j) row_x[j] = (wm * FM + j) * 32;
#pragma unroll
  for (int i = 0; i < FN; ++i)
    row_w[i] = BM + (MODE == kGateUp ? (i < FN / 2 ? wn * FN / 2 + i : (BN / 64) + wn * FN / 2 + i - FN / 2) : wn * FN + i) * 32;
#pragma unroll
  for (int k = 0; k < 2; ++k) off[k] = l32 * 64 + (((2 * hl + k) ^ (l32 >> 2 & 3)) << 4);

  i32x4 xf[2][FM], wf[2][FN];
  int xs[2][FM], ws[2][FN];
  auto read = [&](int s, int k) {  // operands of product step k of stage s
    const uint8_t *b = lds + s % STAGES * kStage + off[k];
#pragma unroll
    for (int i = 0; i < FN; ++i) wf[k][i] = *reinterpret_cast<const i32x4 *>(b + row_w[i] * 64);
#pragma unroll
    for (int j = 0; j < FM; ++j) xf[k][j] = *reinterpret_cast<const i32x4 *>(b + row_x[j] * 64);
  };
  auto read_scales = [&](int s) {
    const uint8_t *b = lds + STAGES * kStage + s % STAGES * kScales + l32 * 4 + 2 * hl;
#pragma unroll
    for (int i = 0; i < FN; ++i) ws[s & 1][i] = *reinterpret_cast<const uint16_t *>(b + row_w[i] * 4);
#pragma unroll
    for (int j = 0; j < FM; ++j) xs[s & 1][j] = *reinterpret_cast<const uint16_t *>(b + row_x[j] * 4);
  };
  WAIT_VM((STAGES - 1) * kPer);
  asm volatile("s_barrier" ::: "memory");
  read(0, 0);
  read_scales(0);
  auto stage = [&](int s, auto odd) {
    constexpr int P = decltype(odd)::value;
    read(s, 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = mfma32<0>(wf[0][i], ws[P][i], xf[0][j], xs[P][j], acc[i][j]);
    // this stage is read, the next one is there, for every wave
    __builtin_amdgcn_sched_barrier(0);
    WAIT_VM((STAGES - 2) * kPer);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    read(s + 1, 0);
    read_scales(s + 1);
    load(s + STAGES);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = mfma32<1>(wf[1][i], ws[P][i], xf[1][j], xs[P][j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int s = 0; s < steps; s += 2) {
    stage(s, std::integral_constant<int, 0>{});
    if (s + 1 < steps) stage(s + 1, std::integral_constant<int, 1>{});
  }
  WAIT_VM(0);

  if constexpr (MODE == kGateUp) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int m = row_x[j] + l32;
      const int64_t line = u.first + min(m, u.n - 1);
#pragma unroll
      for (int i = 0; i < FN / 2; ++i) {
        const int n = n0 + row_w[i] - BM;
        float a[16];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          a[e] = moe_silu_f32(acc[i][j][e]) * acc[i + FN / 2][j][e];
          top = max(top, __float_as_uint(a[e]) & 0x7fffffffu);
        }
        // the other half of the wave has the block's other 16 values
        const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
        const uint32_t byte = mx_scale_byte(max((uint32_t)both[0], (uint32_t)both[1]));
        const float s = mx_scale_value(byte);
        uint32_t h[2];  // 16 bits: codes of rows 8 g + 4 hl .., g = 0, 1 and g = 2, 3
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t v = 0;
          v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[8 * g], a[8 * g + 1], s, 0);
          v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[8 * g + 2], a[8 * g + 3], s, 1);
          v = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[8 * g + 4], a[8 * g + 5], s, 2);
          h[g] = byte == 255 ? 0u : __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v, a[8 * g + 6], a[8 * g + 7], s, 3);
        }
        // lower half: the first two words of the block's codes, upper half: the other two
        const auto x = __builtin_amdgcn_permlane32_swap(h[0], h[1], false, false);
        const uint32_t lo = x[0], hi = x[1];
        const uint2 c = {(lo & 0xffffu) | hi << 16, lo >> 16 | (hi & 0xffff0000u)};
        if (m < u.n && n < p.N) {
          *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + (line * p.N + n) / 2 + 8 * hl) = c;
          if (hl == 0) a_scales[(line * p.N + n) / kMxBlock] = (uint8_t)byte;
        }
      }
    }
  } else {
    const bool vec = p.N % 4 == 0;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int m = row_x[j] + l32;
      int64_t r = -1;
      if (m < u.n) {
        r = mx_out_row(p, u.first + m);
        if (MODE == kPlain && p.in_rows && mx_in_row(p, u.first + m) < 0) r = -1;
      }
      if (r < 0) continue;
      typename O::T *out = static_cast<typename O::T *>(p.out) + r * p.N;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int n = n0 + row_w[i] - BM + 8 * g + 4 * hl;
          const f32x16 &c = acc[i][j];
          const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          if (vec) {
            if (n < p.N) *reinterpret_cast<typename O::V *>(out + n) = O::of(v);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.N) out[n + e] = O::one(v[e]);
          }
        }
    }
  }
}

// blockIdx.y: the expert.
__global__ __launch_bounds__(256) void mx_pad_scales_kernel(const uint8_t *s, const moe_mx_expert_w *table, int part,
                                                            int64_t rows, int blocks, int per, uint32_t *out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * per) return;
  const uint8_t *from = table ? (&table[blockIdx.y].gate)[part] : s + blockIdx.y * rows * blocks;
  const int64_t row = i / per;
  const int b = (int)(i - row * per) * 4;
  uint32_t v = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (b + e < blocks) v |= (uint32_t)from[row * blocks + b + e] << (8 * e);
  out[blockIdx.y * rows * per + i] = v;
}

template <int BM, int BN, int WM, int WN, int STAGES, int OCC, int MODE, int DTYPE>
void run(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  const int64_t units = (p.offsets ? (p.L < p.E ? p.L : p.L / BM + p.E) : (p.L + BM - 1) / BM) + (p.shared + BM - 1) / BM;
  const int cols = MODE == kGateUp ? BN / 2 : BN;
  const TileMap m = tile_map(units, (p.N + cols - 1) / cols);
  auto kernel = mx_tile_kernel<BM, BN, WM, WN, STAGES, OCC, MODE, DTYPE>;
  if (MODE == kPlain)
    hipLaunchKernelGGL(kernel, dim3(tile_grid(m)), dim3(WM * WN * 64), 0, ctx->stream, p, m, a_scales);
  else
    moe_launch(ctx, MODE == kDown ? MOE_STAGE_DOWN : MOE_STAGE_GATEUP, kernel, dim3(tile_grid(m)), dim3(WM * WN * 64), p,
               m, a_scales);
}

template <int MODE, int DTYPE>
void pick(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  const int64_t lines = p.offsets ? p.L / p.E : p.L;
  if (lines > 128)
    run<256, 256, 2, 4, 4, 2, MODE, DTYPE>(ctx, p, a_scales);
  else
    run<64, 256, 1, 4, 3, 2, MODE, DTYPE>(ctx, p, a_scales);
}

}  // namespace

moe_status launch_mx_pad_scales(moe_ctx *ctx, const uint8_t *s, const moe_mx_expert_w *table, int part, int64_t rows,
                                int experts, int K, uint8_t *out) {
  const int blocks = K / kMxBlock, per = (blocks + 3) / 4;
  hipLaunchKernelGGL(mx_pad_scales_kernel, dim3((unsigned)((rows * per + 255) / 256), experts), dim3(256), 0,
                     ctx->stream, s, table, part, rows, blocks, per, reinterpret_cast<uint32_t *>(out));
  MOE_CHECK_LAUNCH("mx_pad_scales_kernel");
  return MOE_OK;
}

bool mx_tiles(int64_t lines, int E) { return lines > 16 * (int64_t)E; }

moe_status launch_mx_tile_product(moe_ctx *ctx, int dtype, const MxProduct &p) {
  switch (dtype) {
    case MOE_FP32: pick<kPlain, MOE_FP32>(ctx, p, nullptr); break;
    case MOE_BF16: pick<kPlain, MOE_BF16>(ctx, p, nullptr); break;
    default: pick<kPlain, MOE_FP16>(ctx, p, nullptr); break;
  }
  MOE_CHECK_LAUNCH("mx tile kernel");
  return MOE_OK;
}
moe_status launch_mx_tile_gateup(moe_ctx *ctx, const MxProduct &p, uint8_t *scales) {
  pick<kGateUp, MOE_FP32>(ctx, p, scales);
  MOE_CHECK_LAUNCH("mx gate/up tile kernel");
  return MOE_OK;
}
moe_status launch_mx_tile_down(moe_ctx *ctx, int dtype, const MxProduct &p) {
  if (dtype == MOE_BF16)
    pick<kDown, MOE_BF16>(ctx, p, nullptr);
  else
    pick<kDown, MOE_FP32>(ctx, p, nullptr);
  MOE_CHECK_LAUNCH("mx down tile kernel");
  return MOE_OK;
}
