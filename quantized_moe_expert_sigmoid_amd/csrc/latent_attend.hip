// Latent attention, absorbed form: attention of every head over the cache's
// rows as they are.
//
// Rows of queries (token i of a sequence, head h) are independent but share
// every key and value, so a workgroup takes 32 WM rows of one sequence and a
// run of its cache tiles of 32 tokens:
//   S^T (tokens x rows) = K Q^T,  P^T = softmax,  O^T (latent x rows) += V^T P^T
// with v_mfma_f32_32x32x16. A wave keeps 32 rows and 1 / WN of the latents of
// O^T: a lane holds one row (l % 32) in S^T, P^T and O^T alike, so the running
// maximum and sum are a lane's own registers and P^T feeds the second product
// without leaving the lane (the tokens' order in the sum is free: both operands
// take k slot (half, j) as token 4 half + j or, from j = 4 on, 8 + 4 half + j -
// 4). The WN waves of a row group compute the same S^T: the repeated products
// are cheaper than an exchange where the cache's bytes are the bound.
//
// Statistics, scores and sums are fp32. Rounded to the element type are the
// absorbed queries, P and the sums of latents, since the products that take them
// read elements; each costs half a unit in the last place of its operand, and the
// three together 0.003 relative in bf16 where the output's own rounding is 0.0017.
//
// Measured (this kernel alone, 128 heads, latents of 512): 64 sequences of one
// token over 1000 to 8000 rows 96 us, 835 TFLOP/s and 3.5 TB/s; 8 of 40 to 64
// tokens 500 us, 950 TFLOP/s. The products bound it: a cache tile of a row tile is
// 2176 cycles of them and takes 3700, of which the first product's two chains of
// 36 take 1450 for 1152, and the exponentials that nothing hides 450. Row tiles of
// 64 rather than 128 rows, two workgroups a CU, hide more but read twice the LDS
// and the cache for the same products: the four kernels took 188 us against 146
// for the former, 886 against 610 for the latter.
#include "latent.h"

#include <algorithm>
#include <type_traits>

namespace {

constexpr int kNT = 32;  // tokens of a cache tile

// A unit of work is one cache tile for one row tile. Where there are fewer row
// tiles than workgroups, each row tile's cache tiles are cut into equal pieces,
// as many as the workgroups allow, and a workgroup takes one piece: it then
// starts and ends one run only, which costs about as much as kOver cache tiles
// (queries and first tiles to wait for, a partial result of 2 KB a row to write).
// Where that leaves some with kOver tiles more than even work, and where there
// are more row tiles, units are numbered sequence by sequence, row tile by row
// tile, cache tile by cache tile, each row tile with kOver units ahead of its
// cache tiles, and workgroup w takes units [w per, (w + 1) per). Either way the
// lengths are read on the device and all workgroups have about the same work. A
// row tile whose cache tiles several workgroups share is joined from their
// partial results by the merge kernel.
constexpr int kOver = 12;

struct AttendWs {
  const PlanHead *head;
  const WgDesc *wg;
  const TileDesc *shared;
  float *part;        // [2 n_wg][WM][dc / 32][4][64] x 4: O^T in the order of the lanes' registers
  float2 *ml;         // [2 n_wg][32 WM]: running maximum and sum
  const uint16_t *q;  // [T][H][dc] absorbed queries
  uint16_t *u;        // [T][H][dc] sums of latents
};

__device__ __forceinline__ int row_tiles(const LatentArgs &a, const LatentSeq &s, int mt) {
  return (s.nq * a.H + mt - 1) / mt;
}
__device__ __forceinline__ int kv_tiles(const LatentSeq &s) { return max(1, (s.len + kNT - 1) / kNT); }

// --- attention -----------------------------------------------------------------
// A cache tile lies in LDS as panels of 64 columns: [panel][token][8 units of 16
// bytes], a token's unit c at place c ^ swz(token). swz spreads 16 consecutive
// tokens' equal units, and 4 tokens' runs of 4 units, over all 64 banks, which
// is what the two products read at a time.
__device__ __forceinline__ int swz(int token) { return ((token >> 1 & 1) << 2) | (token >> 2 & 3); }

template <int DC, int DR, int WM, int WN>
struct Attend {
  static constexpr int kWaves = WM * WN, kMT = 32 * WM, kDK = DC + DR;
  static constexpr int kPanels = (kDK + 63) / 64, kPanelB = kNT * 128, kTileB = kPanels * kPanelB;
  static constexpr int kKS = kDK / 16;           // steps of the first product
  static constexpr int kNB = DC / 32 / WN;       // blocks of 32 latents of a wave
  // Every third step's query operand stays in LDS where O^T takes 256 registers a lane (32 rows of 512 latents): all
  // steps' operands would take 144 of the other 256.
  static constexpr int kQL = kNB >= 16 ? kKS / 3 : 0;
  static constexpr bool in_lds(int k) { return kQL && k % 3 == 2; }
  static_assert(!kQL || kQL == kKS / 3, "");
  static constexpr int kBufs = kQL || DC < 512 ? 3 : 4;  // tile buffers: one being read, the others in flight
  static constexpr int kQB = kWaves * kQL * 1024;
  static constexpr int kLds = kBufs * kTileB + kQB;
  // small rows of few registers: two workgroups a CU, so that one computes while the other starts or ends a run (at
  // the price of 13 to 18 spilled registers with row tiles of 64 rows for latents of 256, mostly outside the loop)
  static constexpr int kPerCu = DC < 512 && kNB <= 4 ? 2 : 1;
  static_assert(kWaves == 4 && kPerCu * kLds <= 160 << 10, "4 waves load a tile's 32 tokens, 8 each");
};

template <typename E, int DC, int DR, int WM, int WN>
__global__ __launch_bounds__(256, (Attend<DC, DR, WM, WN>::kPerCu)) void latent_attend_kernel(
    LatentArgs a, AttendWs ws, float c2, uint32_t flip) {
  using C = Attend<DC, DR, WM, WN>;
  constexpr int kNB = C::kNB, kBufs = C::kBufs, kPanels = C::kPanels, kAhead = C::kPerCu == 2 ? 4 : 6, kChains = 2;
  constexpr int kLoadStep = (C::kKS - 4) / kPanels;  // a panel's load every so many products
  static_assert(kLoadStep >= 1, "every load has its place");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, l32 = lane & 31, hl = lane >> 5;
  // neighbours in the unit order share cache rows: keep them on one XCD (ids go round the 8 XCDs)
  const int w = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const WgDesc d = ws.wg[w];
  const int over = uniform(d.over);
  LatentSeq s{uniform(d.t0), uniform(d.nq), uniform(d.len), uniform(d.len) - uniform(d.nq)};
  int b = uniform(d.b), mt = uniform(d.mt), at = uniform(d.at), left = uniform(d.n);
  bool first = true;
  const uint8_t *cache = static_cast<const uint8_t *>(a.cache);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

  // lane constants of the three LDS access patterns
  const int ld_row = lane >> 3;  // loads: token in the wave's block of 8
  const int ld_unit = (lane & 7) ^ swz((8 * wave + ld_row) & 15);
  // a last panel of 32 columns: its upper units repeat the lower ones
  const int ld_last = C::kDK % 64 ? (ld_unit & 3) - ld_unit : 0;
  int k_off[4], v_off[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) k_off[i] = l32 * 128 + (((2 * i + hl) ^ swz(l32 & 15)) << 4);
  const int vt = 4 * hl + ((lane & 15) >> 2);  // token (mod 16) of the transposed reads; the second read is 8 on
#pragma unroll
  for (int h8 = 0; h8 < 2; ++h8)
#pragma unroll
    for (int p = 0; p < 2; ++p)  // the wave's first block of latents is an odd one where it has one alone
      v_off[h8][p] = (vt + 8 * h8) * 128 +
                     (((4 * (p ^ (kNB == 1 ? wn & 1 : 0)) + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swz(vt + 8 * h8)) << 4) + (lane & 1) * 8;

  while (left > 0) {
    const int nt = row_tiles(a, s, C::kMT), kts = kv_tiles(s);
    const int units = min(left, kts + over - at);                        // of this row tile
    const int kt = max(at - over, 0), n = max(at + units - over, 0) - kt;  // first cache tile, cache tiles
    if (nt > 0 && n > 0) {
      // the wave's rows; lanes behind the last row repeat it and store nothing
      const int row = mt * C::kMT + wm * 32 + l32;
      const bool live = row < s.nq * a.H;
      const int row_c = min(row, s.nq * a.H - 1), qi = row_c / a.H, t = s.t0 + qi;
      const uint64_t word = a.tree ? a.tree[t] : 0;
      // the tokens of the tile from position j0 that the lane's row sees, as bits
      auto seen = [&](int j0) {
        const int old = min(max(s.before - j0, 0), 32), own = j0 - s.before;
        uint32_t v = (uint32_t)((1ull << old) - 1);
        if (a.tree)
          v |= own >= 0 ? (uint32_t)(word >> min(own, 63)) & (own < 64 ? ~0u : 0u)
                        : (uint32_t)(word << min(-own, 63)) & (own > -64 ? ~0u : 0u);
        else
          v = (uint32_t)((1ull << min(max(s.before + qi + 1 - j0, 0), 32)) - 1);
        return v & (uint32_t)((1ull << min(max(s.len - j0, 0), 32)) - 1);
      };

      // The wave's 8 tokens of tile i of this run, into its buffer: prepared, then loaded panel by panel. Positions
      // behind the sequence's last row repeat that row; behind the run's last tile nothing is loaded (but counted).
      // The pages come from a lane each: of 64 tiles where a page holds a tile's 8 tokens, of 8 tiles' 8 tokens
      // where it does not, so that a tile's pages cost no memory access of its own.
      const bool small = a.page_shift < 3;
      int pages = 0;
      auto read_pages = [&](int i) {
        const int j = small ? (kt + i + (lane >> 3)) * kNT + 8 * wave + (lane & 7) : (kt + i + lane) * kNT + 8 * wave;
        pages = a.page_table[(int64_t)b * a.max_pages + (min(j, s.len - 1) >> a.page_shift)];
        if (pages < 0 || pages >= a.n_pages) {
          atomicOr(a.err, (uint32_t)ERRF_LATENT);
          pages = 0;
        }
      };
      const uint8_t *src = nullptr;
      uint32_t to = 0, place = lds0 + wave * 1024;
      int on = 0, j_next = 0, page_next = 0;
      auto prepare = [&](int i, auto part) {  // in four parts, for between the products
        if constexpr (part == 0) {
          if ((i & (small ? 7 : 63)) == 0) read_pages(i);
          // a tile that lies behind the last row altogether repeats that row
          const int j0 = min((kt + i) * kNT + 8 * wave, s.len - 1), r = min(ld_row, s.len - 1 - j0);
          j_next = j0 + r;
          page_next = __shfl(pages, small ? (i & 7) * 8 + r : i & 63, 64);
        } else if constexpr (part == 1) {
          to = place;
          place = place - lds0 >= (uint32_t)((kBufs - 1) * C::kTileB) ? place - (kBufs - 1) * C::kTileB : place + C::kTileB;
          on = (i - n) >> 31;
        } else if constexpr (part == 2) {
          const uint32_t row = ((uint32_t)page_next << a.page_shift) + (j_next & ((1 << a.page_shift) - 1));
          src = cache + (uint64_t)row * (C::kDK * 2) + ld_unit * 16;
        }
      };
      auto load = [&](auto g) {
        if constexpr (C::kDK % 64 && g == kPanels - 1)
          lds_load16<g * 128>(src + ld_last * 16, uniform(to + g * C::kPanelB), uniform(on));
        else
          lds_load16<g * 128>(src, uniform(to + g * C::kPanelB), uniform(on));
      };

      // The first tiles' loads are asked for ahead of the queries and fly while those are read. Not so with row tiles of
      // 64 rows for latents of 512 and 256 and of 128 for 256: the compiler reuses registers between the two and waits
      // for the tiles before it asks for a query.
      if (s.len > 0)
#pragma unroll
        for (int i = 0; i < kBufs - 1; ++i) {
          static_for<0, 3>([&](auto part) { prepare(i, part); });
          static_for<0, kPanels>(load);
        }
      u16x8 q[C::kKS - C::kQL];
      u16x8 *q_lds = reinterpret_cast<u16x8 *>(lds + kBufs * C::kTileB + wave * (C::kQL * 1024)) + lane;
      {
        const int h = row_c - qi * a.H;
        const uint16_t *q1 = ws.q + ((int64_t)s.t0 * a.H + row_c) * DC + 8 * hl;
        const uint16_t *q2 = static_cast<const uint16_t *>(a.q_rope) + t * a.rope_t + h * a.rope_h + 8 * hl;
#pragma unroll
        for (int k = 0; k < C::kKS; ++k) {
          const u32x4 v = *reinterpret_cast<const u32x4 *>(16 * k < DC ? q1 + 16 * k : q2 + (16 * k - DC)) ^ flip;
          if (C::in_lds(k))
            q_lds[k / 3 * 64] = __builtin_bit_cast(u16x8, v);
          else
            q[C::kQL ? k - k / 3 : k] = __builtin_bit_cast(u16x8, v);
        }
      }

      AccTile<E, (kNB > 4)> acc[kNB];
      clear(acc);
      float m = -__builtin_inff(), l = 0.0f;
      if (s.len > 0)
        for (int it = 0; it < n; ++it) {
          WAIT_VM((kBufs - 2) * kPanels);  // only later tiles' loads are outstanding: the wave's part of this one is there
          asm volatile("s_barrier" ::: "memory");  // the other waves' parts are; the oldest buffer's readers are done
          uint8_t *kv = lds + (it % kBufs) * C::kTileB;
          auto v_read = [&](int i) {  // block i % kNB of latents, tokens 16 (i / kNB) ..
            const uint8_t *src = kv + ((wn * kNB + i % kNB) >> 1) * C::kPanelB + i / kNB * (16 * 128);
            const u16x4 lo = lds_read_tr(src + v_off[0][i % kNB & 1]), hi = lds_read_tr(src + v_off[1][i % kNB & 1]);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          };
          u16x8 ring[kAhead];
          // Operands are read kAhead products before they are used, and the order is held: left to itself the
          // compiler reads each one just before its product and waits for it.
          f32x16 zs[kChains];
#pragma unroll
          for (int i = 0; i < kChains; ++i) zs[i] = f32x16{};
          {
            auto k_read = [&](int k) {
              return *reinterpret_cast<const u16x8 *>(kv + k_off[k & 3] + (k >> 2) * C::kPanelB);
            };
            u16x8 qf[2];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ring[k] = k_read(k);
            if (C::kQL) {
              qf[0] = q_lds[0];
              qf[1] = q_lds[64];
            }
            __builtin_amdgcn_sched_barrier(0);
            // The next tile's loads go in between: a wave that issued its 9 in a row would stand still until the
            // memory path has taken them, 16 cycles each for 4 waves. The last steps read the second product's first
            // operands.
            static_for<0, C::kKS>([&](auto k) {
              const u16x8 qk = C::in_lds(k) ? qf[k / 3 & 1] : q[C::kQL ? k - k / 3 : k];
              zs[k % kChains] = E::mfma(ring[k % kAhead], qk, zs[k % kChains]);
              if (k + kAhead < C::kKS)
                ring[k % kAhead] = k_read(k + kAhead);
              else if (k + kAhead - C::kKS < 2 * kNB)
                ring[k % kAhead] = v_read(k + kAhead - C::kKS);
              if (C::in_lds(k) && k / 3 + 2 < C::kQL) qf[k / 3 & 1] = q_lds[(k / 3 + 2) * 64];
              if constexpr (k < 3)
                prepare(it + kBufs - 1, k);
              else if constexpr ((k - 4) % kLoadStep == 0 && (k - 4) / kLoadStep < kPanels)
                load(std::integral_constant<int, (k - 4) / kLoadStep>{});
              __builtin_amdgcn_sched_barrier(0);
            });
          }
          f32x16 z = zs[0];
#pragma unroll
          for (int i = 1; i < kChains; ++i) z += zs[i];
          const int j0 = (kt + it) * kNT;
          if (j0 + kNT > s.before) {  // the tile holds tokens that not every row sees
            const uint32_t vis = seen(j0) >> (4 * hl);
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const bool v = (vis >> (8 * (i >> 2) + (i & 3))) & 1;
              odd |= !v & !(__builtin_fabsf(z[i]) < __builtin_inff());
              z[i] = v ? z[i] : -__builtin_inff();
            }
            // An unseen row that holds NaN or infinities gives such a score, and would reach the sums as 0 x NaN or
            // 0 x inf: then the tile's rows are looked through, the broken ones cleared for every wave, and the rows
            // that do see one get a NaN sum.
            if (__syncthreads_or(odd)) {
              bool broken = false;
#pragma unroll 1
              for (int c = hl; c < DC / 8; c += 2) {
                const u16x8 v = *reinterpret_cast<const u16x8 *>(kv + (c >> 3) * C::kPanelB + l32 * 128 +
                                                                 (((c & 7) ^ swz(l32 & 15)) << 4));
#pragma unroll
                for (int e = 0; e < 8; ++e) broken |= (v[e] & E::kExp) == E::kExp;
              }
              const uint64_t halves = __ballot(broken);
              const uint32_t bad = (uint32_t)halves | (uint32_t)(halves >> 32);
              __syncthreads();
              if ((bad >> l32) & 1)
#pragma unroll 1
                for (int c = 2 * wave + hl; c < DC / 8; c += 8)
                  *reinterpret_cast<u32x4 *>(kv + (c >> 3) * C::kPanelB + l32 * 128 +
                                             (((c & 7) ^ swz(l32 & 15)) << 4)) = u32x4{0, 0, 0, 0};
#pragma unroll
              for (int i = 0; i < 16; ++i)
                z[i] = (bad >> (8 * (i >> 2) + 4 * hl + (i & 3))) & 1 ? -__builtin_inff() : z[i];
              if (bad & (vis << (4 * hl))) l = __builtin_nanf("");
              __syncthreads();
#pragma unroll
              for (int i = 0; i < kAhead && i < 2 * kNB; ++i) ring[(C::kKS + i) % kAhead] = v_read(i);  // once more
            }
          }
          float top = z[0];
#pragma unroll
          for (int i = 1; i < 16; ++i) top = fmaxf(top, z[i]);
          top = max_halves(top) * c2;
          // The reference of the exponentials follows the maximum only when that has grown by 2^8: until then
          // weights up to 2^8 are as exact as weights up to 1, and the sums need no rescaling.
          if (__any(top > m + 8.0f)) {
            const float mn = fmaxf(m, top);
            const float f = m == mn ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int i = 0; i < kNB; ++i) acc[i].scale(f);
          }
          const float base = m == -__builtin_inff() ? 0.0f : -m;
          // the second half's exponentials go between the first half's products
          auto weight = [&](int i) {
            const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z[i], c2, base));
            l += e;
            return e;
          };
          f32x8 e;
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = weight(i);
          u16x8 p = E::from_f32x8(e);
#pragma unroll
          for (int i = 0; i < 2 * kNB; ++i) {
            if (i == kNB) p = E::from_f32x8(e);
            acc[i % kNB].mfma(ring[(C::kKS + i) % kAhead], p, i % kNB == 0);
            if (i + kAhead < 2 * kNB) ring[(C::kKS + i) % kAhead] = v_read(i + kAhead);
            if (i < kNB)
#pragma unroll
              for (int j = i * 8 / kNB; j < (i + 1) * 8 / kNB; ++j) e[j] = weight(8 + j);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      l += __shfl_xor(l, 32, 64);
      settle(acc);
      if (n == kts) {  // the whole row tile: finished here
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t *o = ws.u + ((int64_t)s.t0 * a.H + row) * DC + wn * (kNB * 32) + 8 * hl;
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const u32x4 v = rows8<E>(acc[i].get4(j) * inv, acc[i].get4(j + 1) * inv);
            if (live) *reinterpret_cast<u32x4 *>(o + 32 * i + 8 * j) = v;
          }
      } else {
        const int slot = 2 * w + (first ? 0 : 1);
        float *o = ws.part + (((int64_t)slot * WM + wm) * WN + wn) * (kNB * 1024);
#pragma unroll
        for (int i = 0; i < kNB; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4 *>(o + ((i * 4 + j) * 64 + lane) * 4) = acc[i].get4(j);
        if (hl == 0 && wn == 0) ws.ml[(int64_t)slot * C::kMT + wm * 32 + l32] = make_float2(m, l);
      }
      __syncthreads();  // the tiles are no longer read
    }
    first = false;
    left -= nt > 0 ? units : 0;
    at = 0;
    if (nt == 0 || ++mt == nt) {
      mt = 0;
      ++b;
      if (left > 0) {
        const LatentSeq r = latent_seq(a, b);
        s = LatentSeq{uniform(r.t0), uniform(r.nq), uniform(r.len), uniform(r.before)};
      }
    }
  }
}

// Join of the row tiles that several workgroups share: a workgroup takes 8 J
// latents (J runs of 1 KB of each partial result) of 32 rows. J = 8, up to kFew
// partial results: a wave takes two of the runs. Otherwise a wave takes every
// fourth partial result, and the waves are joined through LDS. J = 1 is for few
// row tiles of many partial results, J = 8 for many row tiles (one token over
// 131072 rows: 22 us with 1, 66 us with 8; 64 tokens over 1000-8000 rows: 26 and
// 16 us). The lengths are on the device, so the host chooses by the call's row tiles
// alone: one sequence of 131072 rows among 16 and among 31 of 500 gets J = 8 and
// takes 33 and 74 us. The bytes are the bound: 67 MB of partial results of 256
// workgroups, read in 16 us, 4.2 TB/s; with none it is a launch, 4.6 us.
constexpr int kFew = 16;

template <typename E, int WM, int J>
__global__ __launch_bounds__(256) void latent_merge_kernel(LatentArgs a, AttendWs ws) {
  __shared__ float box[4][J][64][4];
  __shared__ float2 box_ml[4][64];
  const int ti = blockIdx.x / WM, wm = blockIdx.x % WM;
  if (ti >= ws.head->n_shared) return;
  const TileDesc d = ws.shared[ti];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), l32 = lane & 31, hl = lane >> 5;
  const int64_t per = ws.head->per, whole = (int64_t)a.dc * 32;  // floats of a partial result's 32 rows
  const int j0 = blockIdx.y * J, n = d.n;
  auto slot = [&](int i) {
    const int w = d.w0 + min(i, n - 1) * d.step;
    return (int64_t)(2 * w + (w * per >= d.u0 ? 0 : 1)) * WM + wm;
  };
  auto pow2 = [](float x, float top) { return x == top ? 1.0f : __builtin_amdgcn_exp2f(x - top); };
  auto store = [&](int j, f32x4 sum, float l) {
    const LatentSeq s = latent_seq(a, d.b);
    const int row = d.mt * 32 * WM + wm * 32 + l32;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    u16x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = E::from_f32(sum[e] * inv);
    if (row < s.nq * a.H)
      *reinterpret_cast<u16x4 *>(ws.u + ((int64_t)s.t0 * a.H + row) * a.dc + 8 * (j0 + j) + 4 * hl) = v;
  };
  if (J == 8 && n <= kFew) {
    float2 ml[kFew];
    float m = -__builtin_inff(), l = 0.0f;
#pragma unroll
    for (int i = 0; i < kFew; ++i)
      if (i < n) ml[i] = ws.ml[slot(i) * 32 + l32];
    f32x4 v[2][4], sum[2] = {};
#pragma unroll
    for (int i = 0; i < kFew; ++i)
      if (i < n) m = fmaxf(m, ml[i].x);
#pragma unroll
    for (int i0 = 0; i0 < kFew; i0 += 4) {
      if (i0 >= n) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          v[j][i] = *reinterpret_cast<const f32x4 *>(ws.part + slot(i0 + i) * whole + ((j0 + 2 * wave + j) * 64 + lane) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < n) {
          const float f = pow2(ml[i0 + i].x, m);
          l += ml[i0 + i].y * f;
#pragma unroll
          for (int j = 0; j < 2; ++j) sum[j] += v[j][i] * f;
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) store(2 * wave + j, sum[j], l);
    return;
  }
  float m = -__builtin_inff(), l = 0.0f;
  f32x4 acc[J] = {};
  constexpr int kB = J == 1 ? 8 : 1;  // partial results read at a time
  for (int i = wave; i < n; i += 4 * kB) {
    float2 ml[kB];
    f32x4 v[kB][J];
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      ml[k] = ws.ml[slot(i + 4 * k) * 32 + l32];
      const float *o = ws.part + slot(i + 4 * k) * whole + (j0 * 64 + lane) * 4;
#pragma unroll
      for (int j = 0; j < J; ++j) v[k][j] = *reinterpret_cast<const f32x4 *>(o + j * 256);
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kB; ++k) mn = i + 4 * k < n ? fmaxf(mn, ml[k].x) : mn;
    const float f = pow2(m, mn);
    l *= f;
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] *= f;
#pragma unroll
    for (int k = 0; k < kB; ++k)
      if (i + 4 * k < n) {
        const float g = pow2(ml[k].x, mn);
        l += ml[k].y * g;
#pragma unroll
        for (int j = 0; j < J; ++j) acc[j] += v[k][j] * g;
      }
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) *reinterpret_cast<f32x4 *>(box[wave][j][lane]) = acc[j];
  box_ml[wave][lane] = make_float2(m, l);
  __syncthreads();
  if (J == 1 && wave) return;
#pragma unroll
  for (int w = 0; w < 4; ++w) m = fmaxf(m, box_ml[w][lane].x);
  l = 0.0f;
  constexpr int kJ = J == 1 ? 1 : J / 4;  // runs a wave finishes
  f32x4 sum[kJ] = {};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 ml = box_ml[w][lane];
    const float f = pow2(ml.x, m);
    l += ml.y * f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) sum[j] += *reinterpret_cast<const f32x4 *>(box[w][kJ * wave + j][lane]) * f;
  }
#pragma unroll
  for (int j = 0; j < kJ; ++j) store(kJ * wave + j, sum[j], l);
}

template <typename E, int DC, int DR, int WM, int WN>
moe_status launch(moe_ctx *ctx, const LatentArgs &a) {
  using C = Attend<DC, DR, WM, WN>;
  const int n_wg = ctx->n_cu / 8 * 8 * C::kPerCu;  // whole multiples of the 8 XCDs
  MoeLayout lay;
  const size_t o_head = lay.take(sizeof(PlanHead)), o_wg = lay.take(sizeof(WgDesc) * n_wg),
               o_shared = lay.take(sizeof(TileDesc) * n_wg),
               o_part = lay.take(sizeof(float) * 2 * n_wg * C::kMT * DC),
               o_ml = lay.take(sizeof(float2) * 2 * n_wg * C::kMT),
               o_q = lay.take(2 * (size_t)a.T * a.H * DC), o_u = lay.take(2 * (size_t)a.T * a.H * DC);
  void *scr = nullptr;
  moe_status st = moe_scratch(ctx, lay.size, &scr);
  if (st) return st;
  char *p = static_cast<char *>(scr);
  PlanHead *head = reinterpret_cast<PlanHead *>(p + o_head);
  WgDesc *wg = reinterpret_cast<WgDesc *>(p + o_wg);
  TileDesc *shared = reinterpret_cast<TileDesc *>(p + o_shared);
  uint16_t *q = reinterpret_cast<uint16_t *>(p + o_q), *u = reinterpret_cast<uint16_t *>(p + o_u);
  const AttendWs ws{head, wg, shared, reinterpret_cast<float *>(p + o_part), reinterpret_cast<float2 *>(p + o_ml), q, u};
  const int64_t hc = (int64_t)a.H * DC;
  const HeadGemm absorb{static_cast<const uint16_t *>(a.q_nope), static_cast<const uint16_t *>(a.w_kt), q, nullptr,
                        nullptr, a.T, DC, a.dn, a.nope_t, a.nope_h, (int64_t)DC * a.dn, hc, DC};
  const LatentPlan plan{a, head, wg, shared, C::kMT, kNT, kOver, n_wg};
  if ((st = launch_head_gemm(ctx, E::kDtype, absorb, a.H, plan))) return st;
  const float c2 = latent_c2(a.scale);
  hipLaunchKernelGGL((latent_attend_kernel<E, DC, DR, WM, WN>), dim3(n_wg), dim3(256), 0, ctx->stream, a, ws,
                     c2, a.scale < 0 ? 0x80008000u : 0u);
  MOE_CHECK_LAUNCH("latent_attend_kernel");
  const int64_t tiles = ((int64_t)a.T * a.H + C::kMT - 1) / C::kMT;
  if (tiles <= 16)
    hipLaunchKernelGGL((latent_merge_kernel<E, WM, 1>), dim3((unsigned)std::min<int64_t>(n_wg, tiles + a.B) * WM, DC / 8),
                       dim3(256), 0, ctx->stream, a, ws);
  else
    hipLaunchKernelGGL((latent_merge_kernel<E, WM, 8>), dim3((unsigned)std::min<int64_t>(n_wg, tiles + a.B) * WM, DC / 64),
                       dim3(256), 0, ctx->stream, a, ws);
  MOE_CHECK_LAUNCH("latent_merge_kernel");
  const HeadGemm up{u, static_cast<const uint16_t *>(a.w_kv) + (int64_t)a.dn * DC, static_cast<uint16_t *>(a.out),
                    a.q_start, a.q_start + a.B, a.T, a.dv, DC, hc, DC, (int64_t)(a.dn + a.dv) * DC,
                    (int64_t)a.H * a.dv, a.dv};
  return launch_head_gemm(ctx, E::kDtype, up, a.H, LatentPlan{});
}

template <typename E, int DC, int DR>
moe_status pick(moe_ctx *ctx, const LatentArgs &a, int max_q) {
  const int rows = std::max(1, max_q) * a.H;
  if (rows <= 32) return launch<E, DC, DR, 1, 4>(ctx, a);
  if (rows <= 64) return launch<E, DC, DR, 2, 2>(ctx, a);
  return launch<E, DC, DR, 4, 1>(ctx, a);
}

template <typename E>
moe_status attend(moe_ctx *ctx, const LatentArgs &a, int max_q) {
  if (a.dr == 64)
    return a.dc == 512   ? pick<E, 512, 64>(ctx, a, max_q)
           : a.dc == 256 ? pick<E, 256, 64>(ctx, a, max_q)
                         : pick<E, 128, 64>(ctx, a, max_q);
  return a.dc == 512   ? pick<E, 512, 32>(ctx, a, max_q)
         : a.dc == 256 ? pick<E, 256, 32>(ctx, a, max_q)
                       : pick<E, 128, 32>(ctx, a, max_q);
}

}  // namespace

moe_status launch_latent_attend(moe_ctx *ctx, int dtype, const LatentArgs &a, int max_q) {
  return dtype == MOE_BF16 ? attend<Bf16>(ctx, a, max_q) : attend<Fp16>(ctx, a, max_q);
}
