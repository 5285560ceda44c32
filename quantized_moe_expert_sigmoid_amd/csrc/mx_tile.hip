// Products on microscaled 4-bit floating point in tiles through LDS, for many
// lines an expert.
//
// C^T (n x m) = W X^T with v_mfma_scale_f32_32x32x64_f8f6f4. A workgroup takes BM
// lines of one expert and BN rows of weights; stages of KU blocks of 32 k (4 or 8),
// 16 KU bytes a row, come by asynchronous loads. A row's units of 16 bytes lie at
// unit ^ swz(row), so that the 16 rows of a read meet different banks. Half l / 32 of
// a wave takes units KU / 2 (l / 32) and the next ones, so that a lane's scales of a
// stage are neighbours.
//
// Scales come 16 bytes a row for every 16 / KU stages where rows of scales are
// multiples of 16 bytes (a stage's own 8 bytes of each row were a third of all
// requests: 2047 tokens grouped over 256 experts 1074 us so and 925 us with 16); a
// lane reads the word it needs and the instruction picks a byte. Other rows' scales
// come a byte a lane, each into a word of its own.
//
// A wave has the operands of the next product step in registers before the
// present one begins, and a stage's place is loaded again while its last products
// run: STAGES - 1 stages are in flight.
//
// 2048 lines, 24576 rows of 6144: 187 us, 3.3 PFLOP/s (without the products 146,
// without the loads 138: neither hides the other whole). The 1.2 GB that are
// loaded, 0.25 of them from memory, come at 32 KB a us and CU where nothing else is
// done.
// 2047 tokens of 8 of 256 experts of 4096 rows of 6144: 769 us, without the products
// 758: 4.2 GB read (3.4 GB are distinct) at 5.4 TB/s, a plain read's rate being 7.1.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx.h"

namespace {

enum { kPlain, kDown, kGateUp };

// How workgroups map to tiles: blocks of g units x gn column tiles go round the 8 XCDs; within one, units run fastest.
// With a unit an expert nothing is shared but a few lines, and single tiles go round, so that all XCDs have as many (one
// token of 9 experts: one XCD had 72 workgroups and another 40).
struct TileMap {
  int n_tiles, units, g, gn;
  int total;  // places, a multiple of 8: those of the last blocks that no tile has are passed over
};
TileMap tile_map(int64_t units, int n_tiles, bool apart) {
  TileMap m;
  m.n_tiles = n_tiles, m.units = (int)units;
  m.g = apart ? 1 : units < 4 ? (int)units : 4;
  m.gn = apart ? 1 : 32 / m.g < n_tiles ? 32 / m.g : n_tiles;
  const int64_t blocks = (int64_t)((m.units + m.g - 1) / m.g) * ((m.n_tiles + m.gn - 1) / m.gn);
  m.total = (int)((blocks + 7) / 8 * 8 * m.g * m.gn);
  return m;
}
template <int BM, int BN, int WM, int WN, int KU, int STAGES, int OCC, bool WIDE, int MODE, int DTYPE>
__global__ __launch_bounds__(WM *WN * 64, OCC) void mx_tile_kernel(MxProduct p, TileMap map, uint8_t *a_scales) {
  typedef MxOut<DTYPE> O;
  constexpr int kWaves = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr int kRows = BM + BN, kRowB = KU * 16, kStage = kRows * kRowB, kAt = STAGES * kStage;
  // scales: stages of a load, loads kept, bytes of one
  constexpr int kChunk = WIDE ? 16 / KU : 1, kChunks = (STAGES + kChunk - 2) / kChunk + 1;
  constexpr int kScales = kRows * (WIDE ? 16 : 4 * KU);
  constexpr int kRowsL = 64 / KU, kRowsS = WIDE ? 64 : 64 / KU;  // rows of a load instruction, of codes and of scales
  constexpr int kLoads = kRows / kRowsL / kWaves, kLoadsS = (kRows / kRowsS + kWaves - 1) / kWaves, kPer = kLoads + kLoadsS;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;  // of the result
  static_assert(kRows % (kRowsL * kWaves) == 0 && kWaves * kRowsL % 16 == 0 && (KU == 4 || KU == 8));
  static_assert(MODE != kGateUp || FN % 2 == 0 || (FN == 1 && WN % 2 == 0));
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kAt + kChunks * kScales];

  const int blocks = p.K / kMxBlock, steps = (blocks + KU - 1) / KU;
  MxUnits<BM> lines;
  lines.load(p);
  const int lane = threadIdx.x & 63, wave = mx_uniform((int)(threadIdx.x >> 6)), l32 = lane & 31, hl = lane >> 5;
  const int wm = wave % WM, wn = wave / WM;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;
  // of a row's KU units unit c lies at c ^ swz(row): 256 bytes hold 16 / KU rows
  auto swz = [](int row) { return KU == 4 ? row >> 2 & 3 : (row >> 1 & 1) << 2 | (row >> 2 & 3); };

  const int mine = (lane % KU) ^ swz((wave * kRowsL + lane / KU) & 15);  // the unit of its row that a lane loads
  const uint8_t *src[kLoads], *src_s[kLoadsS];
  // the workgroup's next tile that has lines, and where its rows come from: the lines first, then the weights' rows
  // (gate's, then up's). What a load instruction of codes has is known here, where all waves' rows of it are of one kind;
  // deciding lane by lane cost 4 us of a workgroup's start.
  int at = blockIdx.x, n0 = 0;
  MxUnit u{0, 0, 0};
  auto next = [&]() -> bool {
    const int per_block = map.g * map.gn, across = (map.n_tiles + map.gn - 1) / map.gn;
    for (u.n = 0; at < map.total && u.n == 0; at += gridDim.x) {
      const int j = at >> 3, block = j / per_block * 8 + (at & 7), rest = j % per_block;
      const int unit = block / across * map.g + rest % map.g, nt = block % across * map.gn + rest / map.g;
      if (unit >= map.units || nt >= map.n_tiles) continue;
      u = lines.find(p, unit);
      n0 = nt * kCols;
    }
    if (u.n == 0) return false;
    const uint8_t *w[2], *sw[2];
    if constexpr (MODE == kPlain) {
      w[0] = w[1] = p.w + u.e * p.w_e;
      sw[0] = sw[1] = p.sw + u.e * p.sw_e;
    } else if constexpr (MODE == kDown) {
      w[0] = w[1] = p.table[u.e].down;
      sw[0] = sw[1] = p.table[u.e].s_down;
    } else {
      w[0] = p.table[u.e].gate, w[1] = p.table[u.e].up;
      sw[0] = p.table[u.e].s_gate, sw[1] = p.table[u.e].s_up;
    }
    auto x_row = [&](int r) { return max(mx_in_row(p, u.first + min(r, u.n - 1)), (int64_t)0) * blocks; };
    auto w_row = [&](int n) { return (int64_t)min(n0 + n, p.N - 1) * blocks; };
    mx_static_for<0, kLoads>([&](auto ic) {
      constexpr int first = decltype(ic)::value * kWaves * kRowsL, n = first - BM;
      static_assert(BM % (kWaves * kRowsL) == 0 && kCols % (kWaves * kRowsL) == 0);
      const int r = wave * kRowsL + lane / KU;
      if constexpr (n < 0)
        src[ic] = p.x + (x_row(first + r) + mine) * 16;
      else
        src[ic] = w[n >= kCols] + (w_row(n % kCols + r) + mine) * 16;
    });
    mx_static_for<0, kLoadsS>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const int r = min((i * kWaves + wave) * kRowsS, kRows - kRowsS) + (WIDE ? lane : lane / KU), n = r - BM;
      const int64_t row = n < 0 ? x_row(r) : w_row(MODE == kGateUp && n >= kCols ? n - kCols : n);
      const uint8_t *s = n < 0 ? p.sx : MODE == kGateUp && n >= kCols ? sw[1] : sw[0];
      src_s[i] = s + row + (WIDE ? 0 : lane % KU);
    });
    // here before the first loads of stages: the compiler, which does not count those, would wait for them too
    mx_static_for<0, kLoads>([&](auto ic) {
      const uint8_t *&a = src[ic];
      asm volatile("" : "+v"(a));
    });
    mx_static_for<0, kLoadsS>([&](auto ic) {
      const uint8_t *&a = src_s[ic];
      asm volatile("" : "+v"(a));
    });
    return true;
  };
  // piece i of stage s: rows of codes, then of scales. Sources go on by a stage each time they are used; those of the
  // last stage, if it is not whole, are zeros where a row ends.
  auto load = [&](int s, int i) {
    const int on = mx_below(mx_uniform(s), mx_uniform(steps));
    if (i < kLoads) {
      mx_lds_load16(src[i], mx_uniform((int)(lds0 + s % STAGES * kStage + (i * kWaves + wave) * 1024)), on, on);
      src[i] += kRowB;
    } else {
      const int j = i - kLoads, r = (j * kWaves + wave) * kRowsS;
      const int to = mx_uniform((int)(lds0 + kAt + s / kChunk % kChunks * kScales + min(r, kRows - kRowsS) * (kScales / kRows)));
      const int on_s = on & mx_below(r, kRows) & mx_below(s % kChunk, 1);
      if constexpr (WIDE)
        mx_lds_load16(src_s[j], to, on_s, on_s);
      else
        mx_lds_load1(src_s[j], to, on_s);
      src_s[j] += KU;
    }
  };
  auto last = [&](int s) {  // before the first piece of stage s
    if (WIDE || s != blocks / KU || blocks % KU == 0) return;
    if (KU * s + mine >= blocks)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) src[i] = mx_zeros;
    if (KU * s + lane % KU >= blocks)
#pragma unroll
      for (int i = 0; i < kLoadsS; ++i) src_s[i] = mx_zeros;
  };
  // A stage's pieces are spread over the products of kPhases product steps, from the one on in which its place is free.
  constexpr int kSteps = KU / 2, kPhases = STAGES == 2 ? 2 : kSteps;
  constexpr auto first_of = [](int phase) { return phase >= kPhases ? kPer : phase * kPer / kPhases; };
  auto begin = [&] {
    mx_static_for<0, STAGES>([&](auto sc) {
      constexpr int s = decltype(sc)::value;
      last(s);
      mx_static_for<0, s < STAGES - 1 ? kPer : first_of(1)>([&](auto ic) { load(s, decltype(ic)::value); });
    });
  };
  if (!next()) return;
  begin();

  // a lane's places: rows l32 of 32, units KU / 2 hl + k
  int row_x[FM], row_w[FN], off[KU / 2];
#pragma unroll
  for (int j = 0; j < FM; ++j) row_x[j] = (wm * FM + j) * 32;
#pragma unroll
  for (int i = 0; i < FN; ++i)
    row_w[i] = BM + 32 * (MODE != kGateUp || FN == 1 ? wn * FN + i
                          : i < FN / 2               ? wn * FN / 2 + i
                                                     : BN / 64 + wn * FN / 2 + i - FN / 2);
#pragma unroll
  for (int k = 0; k < KU / 2; ++k) off[k] = l32 * kRowB + (((KU / 2 * hl + k) ^ swz(l32 & 15)) << 4);

  i32x4 xf[2][FM], wf[2][FN];
  // a stage's scales: a word of bytes, or a word for each product step
  typedef int Words __attribute__((ext_vector_type(KU / 2)));
  typedef typename std::conditional<!WIDE, Words, typename std::conditional<KU == 8, int, uint16_t>::type>::type Scale;
  Scale xs[2][FM], ws[2][FN];
  auto read = [&](int s, int k, int i) {  // operand i of product step k of stage s
    const uint8_t *b = lds + s % STAGES * kStage + off[k];
    if (i < FN)
      wf[k & 1][i] = *reinterpret_cast<const i32x4 *>(b + row_w[i] * kRowB);
    else
      xf[k & 1][i - FN] = *reinterpret_cast<const i32x4 *>(b + row_x[i - FN] * kRowB);
  };
  auto read_scales = [&](int s, int to) {
    constexpr int kRowS = kScales / kRows;
    const uint8_t *b = lds + kAt + s / kChunk % kChunks * kScales + l32 * kRowS;
    b += WIDE ? s % kChunk * KU + KU / 2 * hl : 2 * KU * hl;
#pragma unroll
    for (int i = 0; i < FN; ++i) ws[to][i] = *reinterpret_cast<const Scale *>(b + row_w[i] * kRowS);
#pragma unroll
    for (int j = 0; j < FM; ++j) xs[to][j] = *reinterpret_cast<const Scale *>(b + row_x[j] * kRowS);
  };
  f32x16 acc[FN][FM];
  auto stage = [&](int s, auto parity) {
    constexpr int P = decltype(parity)::value;
    mx_static_for<0, kSteps>([&](auto kc) {
      constexpr int k = decltype(kc)::value, kPhase = (k + 1) % kSteps;
      const int s_load = s + STAGES - (kPhase ? 1 : 0);
      if constexpr (kPhase == 0) {  // this stage is read, the next one is there, for every wave
        WAIT_VM((STAGES - 2) * kPer);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        last(s_load);
      }
      __builtin_amdgcn_sched_barrier(0);
      // Between the products: the next step's operands, in the first half of them, and the loads.
      constexpr int F = FN * FM, kHalf = F > 1 ? F / 2 : 1, R = FN + FM;
      constexpr int kBegin = first_of(kPhase), kNum = first_of(kPhase + 1) - kBegin;
      mx_static_for<0, F>([&](auto tc) {
        constexpr int t = decltype(tc)::value, i = t / FM, j = t % FM;
        if constexpr (WIDE)
          acc[i][j] = mx_mfma32<k>(wf[k & 1][i], ws[P][i], xf[k & 1][j], xs[P][j], acc[i][j]);
        else
          acc[i][j] = mx_mfma32<0>(wf[k & 1][i], ws[P][i][k], xf[k & 1][j], xs[P][j][k], acc[i][j]);
        if constexpr (t < kHalf) {
#pragma unroll
          for (int r = t * R / kHalf; r < (t + 1) * R / kHalf; ++r) read(kPhase ? s : s + 1, kPhase, r);
          if constexpr (kPhase == 0 && t == kHalf - 1) read_scales(s + 1, 1 - P);
        }
#pragma unroll
        for (int l = kBegin + t * kNum / F; l < kBegin + (t + 1) * kNum / F; ++l) load(s_load, l);
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };
  // Tile after tile, a chip's worth of workgroups: the next tile's lines are looked up and its first stages asked for
  // before this one's results are stored, unless those pass through LDS (workgroup a tile: 96 tokens of 8 of 256 experts,
  // 6144 rows of 2048, 236 us, so 220; 2048 tokens' FFN 1352 and 1323; one product of 2048 x 24576 x 6144 the same).
  constexpr bool kHandOver = MODE == kGateUp && FN == 1;
  for (;;) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
    WAIT_VM((STAGES - 2) * kPer + first_of(1));
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int i = 0; i < FN + FM; ++i) read(0, 0, i);
    read_scales(0, 0);
    for (int s = 0; s < steps; s += 2) {
      stage(s, std::integral_constant<int, 0>{});
      if (s + 1 < steps) stage(s + 1, std::integral_constant<int, 1>{});
    }
    WAIT_VM(0);
    const MxUnit done = u;
    const int done_n0 = n0;
    int64_t to[FM];  // rows of out, -1: none
    if constexpr (MODE != kGateUp) {
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int m = row_x[j] + l32;
        to[j] = -1;
        if (m < done.n) {
          to[j] = mx_out_row(p, done.first + m);
          if (MODE == kPlain && p.in_rows && mx_in_row(p, done.first + m) < 0) to[j] = -1;
        }
        asm volatile("" : "+v"(to[j]));
      }
    }
    bool more = false;
    if (kHandOver || at < map.total)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every wave has read its last stage
    if constexpr (!kHandOver) {
      more = next();
      if (more) begin();
    }

    if constexpr (MODE == kGateUp) {
      // gate and up of the same rows meet in one wave: they are there, or up's wave hands its own over through LDS
      constexpr int kPairs = FN > 1 ? FN / 2 : 1;
      f32x16 up[kPairs][FM];
      bool mine_too = true;
      if constexpr (FN > 1) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) up[i][j] = acc[i + FN / 2][j];
      } else {
        f32x4 *box = reinterpret_cast<f32x4 *>(lds) + (wn % (WN / 2) * WM + wm) * FM * 4 * 64 + lane;
        mine_too = wn < WN / 2;
        if (!mine_too) {
#pragma unroll
          for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              box[(4 * j + g) * 64] = f32x4{acc[0][j][4 * g], acc[0][j][4 * g + 1], acc[0][j][4 * g + 2], acc[0][j][4 * g + 3]};
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) up[0][j][e] = box[(4 * j + e / 4) * 64][e % 4];
      }
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if (!mine_too) break;
        const int m = row_x[j] + l32;
        const int64_t line = done.first + min(m, done.n - 1);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const int n = done_n0 + row_w[i] - BM;
          float a[16];
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            a[e] = mx_silu(acc[i][j][e]) * up[i][j][e];
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
          if (m < done.n && n < p.N) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + (line * p.N + n) / 2 + 8 * hl) = c;
            if (hl == 0) a_scales[(line * p.N + n) / kMxBlock] = (uint8_t)byte;
          }
        }
      }
    } else {
      // 16 bytes a store: four fp32 values; of 16-bit ones two groups of four, of which the halves of a wave (one line's, both
      // here or neither) trade one each. Rows that do not end on 16 bytes: one value a store.
      const bool vec = p.N % (DTYPE == MOE_FP32 ? 4 : 8) == 0;
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if (to[j] < 0) continue;
        typename O::T *out = static_cast<typename O::T *>(p.out) + to[j] * p.N;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const f32x16 &c = acc[i][j];
          const int n = done_n0 + row_w[i] - BM;
          if (vec && DTYPE != MOE_FP32) {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
              typedef MxOut<DTYPE == MOE_FP32 ? MOE_BF16 : DTYPE> H;
              const f32x4 lo = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
              const f32x4 hi = {c[4 * g + 4], c[4 * g + 5], c[4 * g + 6], c[4 * g + 7]};
              const uint2 a = __builtin_bit_cast(uint2, H::of(lo)), b = __builtin_bit_cast(uint2, H::of(hi));
              const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false);
              const auto y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
              const uint4 v = {x[0], y[0], x[1], y[1]};
              if (n + 8 * (g + hl) < p.N) *reinterpret_cast<uint4 *>(out + n + 8 * (g + hl)) = v;
            }
            continue;
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int at = n + 8 * g + 4 * hl;
            const f32x4 v = {c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
            if (vec) {
              if (at < p.N) *reinterpret_cast<typename O::V *>(out + at) = O::of(v);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (at + e < p.N) out[at + e] = O::one(v[e]);
            }
          }
        }
      }
    }
    if constexpr (kHandOver) {
      if (at < map.total) __syncthreads();  // what was handed over is read
      more = next();
      if (more) begin();
    }
    if (!more) break;
  }
}

template <int PER_CU, int BM, int BN, int WM, int WN, int KU, int STAGES, int OCC, bool WIDE, int MODE, int DTYPE>
void run(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  const int64_t units = (p.offsets ? (p.L < p.E ? p.L : p.L / BM + p.E) : (p.L + BM - 1) / BM) + (p.shared + BM - 1) / BM;
  const int cols = MODE == kGateUp ? BN / 2 : BN;
  const TileMap m = tile_map(units, (p.N + cols - 1) / cols, p.offsets && p.L <= (int64_t)p.E * BM);
  auto kernel = mx_tile_kernel<BM, BN, WM, WN, KU, STAGES, OCC, WIDE, MODE, DTYPE>;
  const int most = ctx->n_cu / 8 * 8 * PER_CU;
  const dim3 grid(m.total < most ? m.total : most), block(WM * WN * 64);
  if (MODE == kPlain)
    hipLaunchKernelGGL(kernel, grid, block, 0, ctx->stream, p, m, a_scales);
  else
    moe_launch(ctx, MODE == kDown ? MOE_STAGE_DOWN : MOE_STAGE_GATEUP, kernel, grid, block, p, m, a_scales);
}

// The tiles there are, lines x rows of weights (gate/up: half as many of each). For a step of 256 k a workgroup takes
// `full` us where every CU has its `per_cu` workgroups, less with fewer, and `alone` us where a CU has one (measured
// with 24576, 8192, 6144 and 4096 rows of 2048 to 8192 k; the estimates below are within 40% where the weights' bytes
// are not the bound and put the tiles in the measured order but for differences of 20%). Few lines an expert want few
// lines a tile (256 experts, 16384 lines of 6144 by 4096: 32 x 128 1074 us, 64 x 128 844, 128 x 128 862, 128 x 256 809,
// 256 x 256 1043), a full chip large ones (4096 lines of 6144 by 24576: 817, 549, 419, 407, 376 us), little work many.
// 128 x 128 is for what is between them: 6423 lines of 6144 by 2642 in these five tiles 188, 136, 113, 166 and 166 us, 2805
// lines of 6656 by 3206 116, 92, 79, 92 and 95, 5088 lines of 8 experts of 7168 by 2124 159, 122, 99, 139 and 174.
struct Tile {
  int bm, bn, per_cu;
  double full, alone;
};
constexpr Tile kTiles[] = {{32, 64, 4, 0.84, 0.27}, {32, 128, 2, 0.68, 0.36}, {64, 128, 2, 0.95, 0.51}, {128, 128, 2, 1.45, 0.9},
                           {128, 256, 1, 1.41, 1.2}, {256, 256, 1, 2.6, 2.2}};

double tile_time(const moe_ctx *ctx, const MxProduct &p, const Tile &t, int cols) {
  // experts with lines have their share of them and half a tile more, but at least one tile
  const double active = p.offsets ? (double)(p.L < p.E ? p.L : p.E) : 1;
  double units = p.offsets ? active * std::max(1.0, (double)p.L / (active * t.bm) + 0.5) : (double)((p.L + t.bm - 1) / t.bm);
  units += (double)((p.shared + t.bm - 1) / t.bm);
  const double wg = units * ((p.N + cols - 1) / cols), slots = (double)t.per_cu * ctx->n_cu;
  const double rounds = std::floor(wg / slots), rest = std::ceil((wg - rounds * slots) / ctx->n_cu);
  return (p.K + 255) / 256 * (rounds * t.full + (rest == 0 ? 0.0 : std::max(t.alone, rest * t.full / t.per_cu))) + 5;
}

int pick(const moe_ctx *ctx, const MxProduct &p, int mode, double *time) {
  int best = 0;
  double least = 1e30;
  for (int i = 0; i < (int)(sizeof kTiles / sizeof *kTiles); ++i) {
    const double v = tile_time(ctx, p, kTiles[i], kTiles[i].bn / (mode == kGateUp ? 2 : 1));
    if (v < least) least = v, best = i;
  }
  if (time) *time = least;
  return best;
}

// Stages: as many as the LDS holds for `per_cu` workgroups a CU (scales as words: fewer).
template <bool WIDE, int MODE, int DTYPE>
void launch_tile(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  switch (pick(ctx, p, MODE, nullptr)) {
    case 0: run<4, 32, 64, 1, 2, 8, 3, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
    case 1: run<2, 32, 128, 1, 4, 8, 3, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
    case 2: run<2, 64, 128, 2, 2, 8, WIDE ? 3 : 2, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
    case 3: run<2, 128, 128, 2, 2, WIDE ? 8 : 4, WIDE ? 2 : 3, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
    case 4: run<1, 128, 256, 2, 4, 8, WIDE ? 3 : 2, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
    default: run<1, 256, 256, 2, 4, 4, 4, 2, WIDE, MODE, DTYPE>(ctx, p, a_scales); break;
  }
}
template <int MODE, int DTYPE>
void launch(moe_ctx *ctx, const MxProduct &p, uint8_t *a_scales) {
  if (p.K % (16 * kMxBlock) == 0 && moe_aligned16(p.sx) && moe_aligned16(p.sw))  // sw: NULL with a table, whose own are aligned
    launch_tile<true, MODE, DTYPE>(ctx, p, a_scales);
  else
    launch_tile<false, MODE, DTYPE>(ctx, p, a_scales);
}

}  // namespace

// Up to 64 lines an expert can go to the kernels without tiles (mx_stream.hip), whose time the requests of all
// workgroups' rows make: with 16 NM lines and s steps of 1024 k each wave, 1 + NM (less: the lines there are) times
// s + 8, 0.1225 us for every 256 workgroups. 4096 rows of 6144: 1, 16, 32 and 64 lines 4.9, 5.9, 7.6 and 11.1 us there,
// 13.2 us in tiles of 32 x 128; 6144 rows of 2048: 5.0, 6.5, 8.3 and 12.1, 7.6 us in tiles. Where bytes are the bound,
// tiles read them at 5 TB/s, the others for one line alone (24576 rows of 6144: 17 us, tiles 20.5; 8 lines 22.9 and
// 20.9) and at about 3.5 for more or for several experts (4 tokens of 8 experts, 4096 rows of 6144: 104 and 73 us).
bool mx_tiles(const moe_ctx *ctx, const MxProduct &p) {
  const double active = p.offsets ? (double)(p.L < p.E ? p.L : p.E) : 1, lines = (double)p.L / active;
  if (lines > 64) return true;
  const double nm = lines <= 16 ? lines / 16 : lines <= 32 ? 2 : 4, wg = active * ((p.N + 15) / 16) / ctx->n_cu;
  const double stream = 2.5 + (wg < 1 ? 1 : wg) * (1 + nm) * 0.1225 * ((p.K + 1023) / 1024 + 8);
  const double bytes = active * p.N * (double)p.K * 17 / 32 * 1e-6;  // over TB/s: us
  double tile;
  pick(ctx, p, kPlain, &tile);
  return std::max(stream, bytes / (p.L == 1 ? 5 : 3.5) + 2.5) > std::max(tile, bytes / 5 + 3.5);
}

moe_status launch_mx_tile_product(moe_ctx *ctx, int dtype, const MxProduct &p) {
  switch (dtype) {
    case MOE_FP32: launch<kPlain, MOE_FP32>(ctx, p, nullptr); break;
    case MOE_BF16: launch<kPlain, MOE_BF16>(ctx, p, nullptr); break;
    default: launch<kPlain, MOE_FP16>(ctx, p, nullptr); break;
  }
  MOE_CHECK_LAUNCH("mx tile kernel");
  return MOE_OK;
}
moe_status launch_mx_gateup(moe_ctx *ctx, const MxProduct &p, uint8_t *scales) {
  launch<kGateUp, MOE_FP32>(ctx, p, scales);
  MOE_CHECK_LAUNCH("mx gate/up tile kernel");
  return MOE_OK;
}
moe_status launch_mx_down(moe_ctx *ctx, const MxProduct &p) {
  launch<kDown, MOE_FP32>(ctx, p, nullptr);
  MOE_CHECK_LAUNCH("mx down tile kernel");
  return MOE_OK;
}
