// The experts' FFN of one to three tokens: every slot by itself, no bucketing, the
// hidden state quantised where it is used, the combine in down's workgroups.
//
// Bound by the weights' bytes and by three latencies in a row (ids, addresses,
// weights). A wave streams 32 rows of weights by asynchronous loads into LDS of its
// own, 4 KB a stage of 256 k, and waits for no other wave; the products are
// v_mfma_scale_f32_32x32x64_f8f6f4 with the line's codes, which lie in LDS, in all
// 32 columns. 8 of 256 experts of 6144 x 2048 and a shared one, one token (181 MB):
// gate/up 28 us (4.3 TB/s) and down 14 (4.2), 44 us as a call; bucketing, tiles of
// 32 x 64 and a combine of its own took 58. Six or eight stages a wave: 58 to 61;
// the waves' walks along k each beginning elsewhere: the same.
#include "mx.h"

namespace {

constexpr int KU = 8, kStage = 32 * 16 * KU, kMaxK = 8192;

// LDS bytes: scales of a wave's stages, a line's codes and scales in whole stages.
constexpr int scales_bytes(bool wide, int stages) { return wide ? (stages / 2 + 1) * 512 : stages * 32 * KU * 4; }
constexpr int line_codes(int blocks) { return (blocks + KU - 1) / KU * KU * 16; }
constexpr int line_scales(bool wide, int blocks) { return (blocks + KU - 1) / KU * KU * (wide ? 1 : 4); }
constexpr int line_bytes(bool wide, int blocks) { return line_codes(blocks) + (line_scales(wide, blocks) + 15) / 16 * 16; }

// A wave's 32 rows of K values, rows blocks * 16 bytes apart, and their scales. WIDE: rows of scales are multiples of 16
// bytes and come 16 bytes for every two stages; else a byte a lane, each into a word.
template <bool WIDE, int STAGES>
struct Stream {
  static constexpr int kLoadsS = WIDE ? 1 : 4, kPer = 4 + kLoadsS, kChunk = WIDE ? 2 : 1;
  static constexpr int kChunks = WIDE ? STAGES / 2 + 1 : STAGES, kScales = WIDE ? 512 : 32 * KU * 4;
  const uint8_t *src[4], *src_s[kLoadsS];
  const uint8_t *lds;
  uint32_t at;
  int blocks, steps;

  static __device__ __forceinline__ int swz(int row) { return (row >> 1 & 1) << 2 | (row >> 2 & 3); }
  static __device__ __forceinline__ int mine(int i, int lane) { return (lane & 7) ^ swz((i * 8 + (lane >> 3)) & 15); }

  __device__ __forceinline__ void begin(const uint8_t *w, const uint8_t *s, int row, int n_blocks, uint8_t *box) {
    const int lane = threadIdx.x & 63;
    lds = box;
    at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)box;
    blocks = n_blocks, steps = (blocks + KU - 1) / KU;
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = w + ((int64_t)(row + i * 8 + (lane >> 3)) * blocks + mine(i, lane)) * 16;
#pragma unroll
    for (int i = 0; i < kLoadsS; ++i)
      src_s[i] = s + (int64_t)(row + (WIDE ? lane & 31 : i * 8 + (lane >> 3))) * blocks + (WIDE ? 0 : lane & 7);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) load(i);
  }
  __device__ __forceinline__ void load(int s) {
    const int lane = threadIdx.x & 63, on = mx_below(mx_uniform(s), mx_uniform(steps));
    if (s == blocks / KU && blocks % KU) {  // the last stage: zeros where a row ends
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (KU * s + mine(i, lane) >= blocks) src[i] = mx_zeros;
#pragma unroll
      for (int i = 0; i < kLoadsS; ++i)
        if (!WIDE && KU * s + (lane & 7) >= blocks) src_s[i] = mx_zeros;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mx_lds_load16(src[i], mx_uniform((int)(at + s % STAGES * kStage + i * 1024)), on, on);
      src[i] += 16 * KU;
    }
    const int to = mx_uniform((int)(at + STAGES * kStage + s / kChunk % kChunks * kScales)), on_s = on & mx_below(s & (kChunk - 1), 1);
#pragma unroll
    for (int i = 0; i < kLoadsS; ++i) {
      if constexpr (WIDE)
        mx_lds_load16(src_s[i], to, on_s, 0);
      else
        mx_lds_load1(src_s[i], to + i * 256, on_s);
      src_s[i] += KU;
    }
  }
  // Products with a line (codes, scales as bytes or words): lane l has rows 8 (i / 4) + 4 (l / 32) + i % 4 of the 32.
  __device__ __forceinline__ f32x16 run(const uint8_t *line, const uint8_t *line_s) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, hl = lane >> 5;
    f32x16 acc = {};
    for (int s = 0; s < steps; ++s) {
      WAIT_VM((STAGES - 1) * kPer);
      asm volatile("" ::: "memory");
      const uint8_t *b = lds + s % STAGES * kStage + l32 * 128;
      const uint8_t *c = lds + STAGES * kStage + s / kChunk % kChunks * kScales;
      i32x4 wf[4], xf[4], ws, xs;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        wf[k] = *reinterpret_cast<const i32x4 *>(b + (((4 * hl + k) ^ swz(l32 & 15)) << 4));
        xf[k] = *reinterpret_cast<const i32x4 *>(line + (KU * s + 4 * hl + k) * 16);
      }
      if constexpr (WIDE) {
        ws[0] = *reinterpret_cast<const int *>(c + l32 * 16 + s % 2 * 8 + 4 * hl);
        xs[0] = *reinterpret_cast<const int *>(line_s + KU * s + 4 * hl);
      } else {
        ws = *reinterpret_cast<const i32x4 *>(c + (l32 * KU + 4 * hl) * 4);
        xs = *reinterpret_cast<const i32x4 *>(line_s + (KU * s + 4 * hl) * 4);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the stage's place is loaded again
      load(s + STAGES);
      mx_static_for<0, 4>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        if constexpr (WIDE)
          acc = mx_mfma32<k>(wf[k], ws[0], xf[k], xs[0], acc);
        else
          acc = mx_mfma32<0>(wf[k], ws[k], xf[k], xs[k], acc);
      });
    }
    WAIT_VM(0);
    return acc;
  }
};

// Whether a slot's expert is one, and no earlier slot of the token has it; others but -1 are reported.
__device__ __forceinline__ bool slot_ok(const MxOne &p, int t, int j) {
  const int id = p.idx[t * p.k + j];
  bool ok = id >= 0 && id < p.E;
  for (int i = 0; i < j; ++i) ok &= p.idx[t * p.k + i] != id;
  if (!ok && id != -1) atomicOr(p.err, (uint32_t)ERRF_BAD_INDEX);
  return ok;
}

template <bool WIDE>
__device__ __forceinline__ void put_scale(uint8_t *line_s, int block, uint32_t byte) {
  if constexpr (WIDE)
    line_s[block] = (uint8_t)byte;
  else
    reinterpret_cast<uint32_t *>(line_s)[block] = byte;
}

// silu(gate x) (up x) of one line, 32 rows of each: a wave gate's, the other up's. Every workgroup quantises the token itself while
// its first weights are on their way, so that no launch goes before this one.
template <bool WIDE, int STAGES>
__global__ __launch_bounds__(128) void mx_one_gateup_kernel(MxOne p) {
  constexpr int kWave = STAGES * kStage + scales_bytes(WIDE, STAGES);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kWave + line_bytes(WIDE, kMaxK / 32)];
  __shared__ float both[2][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = mx_uniform(tid >> 6), n0 = blockIdx.x * 32;
  const int line = blockIdx.y, routed = p.T * p.k, blocks = p.H / kMxBlock, steps = (blocks + KU - 1) / KU;
  const int t = line < routed ? line / p.k : line - routed;
  uint8_t *codes = lds + 2 * kWave, *line_s = codes + line_codes(blocks);
  // the token's values, on their way while the expert is looked up
  constexpr int kC = kMaxK / 8 / 128;
  float v[kC][8];
  auto values = [&](auto type) {
    typedef typename MxOut<decltype(type)::value>::T T;
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (i * 128 + tid < blocks * 4)
        mx_load8<decltype(type)::value>(static_cast<const T *>(p.x) + (int64_t)t * p.H + (i * 128 + tid) * 8, v[i]);
  };
  if (p.dtype == MOE_FP32)
    values(std::integral_constant<int, MOE_FP32>{});
  else if (p.dtype == MOE_BF16)
    values(std::integral_constant<int, MOE_BF16>{});
  else
    values(std::integral_constant<int, MOE_FP16>{});
  int e = p.E;
  if (line < routed) {
    if (!slot_ok(p, t, line - t * p.k) || p.w[line] == 0.0f) return;
    e = mx_uniform(p.idx[line]);
  }
  const moe_mx_expert_w &m = p.table[e];
  const uint8_t *w = wave ? m.up : m.gate, *s = wave ? m.s_up : m.s_gate;
  // the values are here before the first stages are asked for: the compiler, which does not count those, would wait for
  // them too
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(v[i][j]));
  Stream<WIDE, STAGES> stream;
  stream.begin(w, s, n0, blocks, lds + wave * kWave);
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = i * 128 + tid;
    if (c < steps * KU * 4) {  // whole quads; zeros behind the row's end
      uint32_t byte = 0, code = 0;
      if (c < blocks * 4) code = mx_codes8(v[i], byte);
      reinterpret_cast<uint32_t *>(codes)[c] = code;
      if ((c & 3) == 0) put_scale<WIDE>(line_s, c >> 2, byte);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const f32x16 acc = stream.run(codes, line_s);
  if ((lane & 31) == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) both[wave][8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)] = acc[i];
  }
  __syncthreads();
  if (tid >= 4) return;
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = mx_silu(both[0][8 * tid + i]) * both[1][8 * tid + i];
  uint32_t byte;
  const uint32_t code = mx_codes8(a, byte);
  const int64_t at = ((int64_t)line * p.I + n0) / kMxBlock;
  reinterpret_cast<uint32_t *>(p.a)[at * 4 + tid] = code;
  if (tid == 0) p.sa[at] = (uint8_t)byte;
}

// 32 rows of a token's result: a wave a slot (down's rows of its expert), then the weighted sum, the shared expert's part
// first and the slots in order, as moe_combine adds them.
template <bool WIDE, int STAGES, int DTYPE>
__global__ __launch_bounds__(1024) void mx_one_down_kernel(MxOne p) {
  typedef MxOut<DTYPE> O;
  extern __shared__ __attribute__((aligned(1024))) uint8_t dyn[];
  constexpr int kWave = STAGES * kStage + scales_bytes(WIDE, STAGES);
  const int lane = threadIdx.x & 63, wave = mx_uniform((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
  const int n0 = blockIdx.x * 32, t = blockIdx.y, blocks = p.I / kMxBlock, steps = (blocks + KU - 1) / KU, slots = p.k + p.shared;
  const int per = kWave + line_bytes(WIDE, blocks);
  uint8_t *box = dyn + wave * per, *codes = box + kWave, *line_s = codes + line_codes(blocks);
  float *sums = reinterpret_cast<float *>(dyn + waves * per);  // [slots][32], then the slots' weights, 0: not used
  float *weight = sums + slots * 32;
  for (int j = wave; j < slots; j += waves) {
    int e = p.E;
    float f = 1.0f;
    if (j < p.k) {
      f = slot_ok(p, t, j) ? p.w[t * p.k + j] : 0.0f;
      e = p.idx[t * p.k + j];
    }
    if (lane == 0) weight[j] = f;
    if (mx_uniform(f == 0.0f ? 1 : 0)) continue;
    const int64_t line = j < p.k ? (int64_t)t * p.k + j : (int64_t)p.T * p.k + t;
    // the line's codes, 16 bytes a lane and load, and scales
    i32x4 c[kMaxK / 32 / 64];
    uint32_t b[kMaxK / 32 / 64];
#pragma unroll
    for (int i = 0; i < kMaxK / 32 / 64; ++i) {
      const int u = i * 64 + lane;
      c[i] = i32x4{}, b[i] = 0;
      if (u < blocks) {
        c[i] = reinterpret_cast<const i32x4 *>(p.a)[line * blocks + u];
        b[i] = p.sa[line * blocks + u];
      }
    }
    const moe_mx_expert_w &m = p.table[mx_uniform(e)];
    const uint8_t *w = m.down, *s = m.s_down;
#pragma unroll
    for (int i = 0; i < kMaxK / 32 / 64; ++i) asm volatile("" : "+v"(c[i]), "+v"(b[i]));
    Stream<WIDE, STAGES> stream;
    stream.begin(w, s, n0, blocks, box);
#pragma unroll
    for (int i = 0; i < kMaxK / 32 / 64; ++i) {
      const int u = i * 64 + lane;
      if (u < steps * KU) {
        reinterpret_cast<i32x4 *>(codes)[u] = c[i];
        put_scale<WIDE>(line_s, u, b[i]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const f32x16 acc = stream.run(codes, line_s);
    if ((lane & 31) == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sums[j * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3)] = acc[i];
    }
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  float out = p.shared ? sums[p.k * 32 + lane] : 0.0f;
  for (int j = 0; j < p.k; ++j)
    if (weight[j] != 0.0f) out = __builtin_fmaf(weight[j], sums[j * 32 + lane], out);
  static_cast<typename O::T *>(p.out)[(int64_t)t * p.H + n0 + lane] = O::one(out);
}

template <bool WIDE>
void gateup(moe_ctx *ctx, const MxOne &p) {
  moe_launch(ctx, MOE_STAGE_GATEUP, mx_one_gateup_kernel<WIDE, 3>, dim3(p.I / 32, p.T * (p.k + p.shared)), dim3(128), p);
}

template <bool WIDE, int STAGES, int DTYPE>
void down(moe_ctx *ctx, const MxOne &p, int waves, size_t lds) {
  moe_launch_lds(ctx, MOE_STAGE_DOWN, mx_one_down_kernel<WIDE, STAGES, DTYPE>, dim3(p.H / 32, p.T), dim3(waves * 64), lds, p);
}

template <bool WIDE, int DTYPE>
void pick_down(moe_ctx *ctx, const MxOne &p) {
  // a wave a slot if the LDS holds them (three stages each if it holds those), else as many as it does, in turn
  const int slots = p.k + p.shared, most = 160 * 1024 - slots * 33 * 4;
  const int line = line_bytes(WIDE, p.I / kMxBlock);
  const int per3 = 3 * kStage + scales_bytes(WIDE, 3) + line, per2 = 2 * kStage + scales_bytes(WIDE, 2) + line;
  const int want = slots < 16 ? slots : 16;
  const bool three = want * per3 <= most;
  const int per = three ? per3 : per2, waves = want * per <= most ? want : most / per;
  const size_t lds = (size_t)waves * per + slots * 33 * 4;
  if (three)
    down<WIDE, 3, DTYPE>(ctx, p, waves, lds);
  else
    down<WIDE, 2, DTYPE>(ctx, p, waves, lds);
}

template <int DTYPE>
void launch_down(moe_ctx *ctx, const MxOne &p) {
  if (p.I % 512 == 0)
    pick_down<true, DTYPE>(ctx, p);
  else
    pick_down<false, DTYPE>(ctx, p);
}

}  // namespace

moe_status launch_mx_one(moe_ctx *ctx, const MxOne &p) {
  if (p.H % 512 == 0)
    gateup<true>(ctx, p);
  else
    gateup<false>(ctx, p);
  MOE_CHECK_LAUNCH("mx_one_gateup_kernel");
  switch (p.dtype) {
    case MOE_FP32: launch_down<MOE_FP32>(ctx, p); break;
    case MOE_BF16: launch_down<MOE_BF16>(ctx, p); break;
    default: launch_down<MOE_FP16>(ctx, p); break;
  }
  MOE_CHECK_LAUNCH("mx_one_down_kernel");
  return MOE_OK;
}
