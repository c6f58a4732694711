// Attention over the 8-bit cache for many rows a head, on the fifth-generation tensor cores.
//
// Up to 128 rows (new tokens x query heads of one key/value head) share what is read. A CTA goes over the
// cache 128 tokens at a time:
//   scores [128 rows x 128 tokens] = q [shared memory] k^T [shared memory]
//   outputs [128 rows x D] += weights [tensor memory] v [shared memory]
// Tiles of tokens go in turn to two streams, each with scores, outputs, maxima and sums of its own for the same
// rows: while the tensor cores work for one stream, the softmax of the other runs, a thread a row. At an
// item's end the two streams are joined, half of the D values by each.
//
// Codes become float16 as in sv_attn8.cu, exact, on their way from the bytes that bulk copies bring to operands
// in the 128-byte swizzle. A block's exponents go into the softmax: t = score 2^e(keys) scale + e(values) in
// base 2, weights 2^(t - M) in float16 for outputs of codes, and 2^-e(values) of them for the sum.
//
// One persistent CTA an SM, its warps specialised: eight for the softmax, four unpack codes (and queries), one
// issues products, one copies, one walks through the items. The work is cut and joined as in sv_attn.cu, in
// units of 128 tokens.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <type_traits>
#include <utility>

#include "spec_kv.h"
#include "sv_attn.cuh"
#include "sv_kv.h"
#include "sv_ptx.cuh"
#include "sv_tc.cuh"
#include "sv_tc_attn.cuh"

namespace sv {
namespace {

constexpr int kWarpUnpack = 8, kWarpMma = 16, kWarpCopy = 17, kWarpItems = 18;
constexpr int kThreads = 640, kSoftmaxThreads = 256;
constexpr int kR = 128, kUnit = 128;  // rows of a tile, tokens of a unit

// Work as it is cut.
struct Work8 {
  static constexpr int kRows = kR, kUnit = sv::kUnit, kDearest = 4, kOver = 12, kLeast = 2;
  static __device__ __forceinline__ int weight(int) { return 4; }
};

template <int D>
struct Shape8 {
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;       // bytes of 128 rows of 64 float16 values
  static constexpr int kTile = kSlabs * kSlab;  // queries, keys or values of a unit as operands
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kRaw = 8 * 16 * D + 128;  // codes of a unit's keys or values; heads of the blocks
  static constexpr int kRaws = D == 128 ? 5 : 8;
  static constexpr int kSmem = 1024 + (1 + kStages) * kTile + kRaws * kRaw;
  static constexpr long long kPart = kR * (D + 2);
};

// An item, or the part of it that the run has: units unit .. end - 1 of it.
struct Item8 {
  Walk w;
  int unit, end, rows;
  int all_see;  // tokens that every row sees
  int whole;    // all of the item
  int last;     // the run ends with it
};

struct Shared8 {
  uint64_t raw_full[8], raw_empty[8];    // bytes of the cache
  uint64_t full[6], empty[6];            // operands
  uint64_t q_full[4], q_free;            // queries of an item; spent
  uint64_t s_full[2], p_full[2];         // scores; weights
  uint64_t o_done[2], o_free;            // outputs of an item; read
  uint64_t item_full[4], item_free[4];
  uint64_t end;
  Item8 items[4];
  uint32_t tmem;
  int last;
  Run run;
  Walk first;
  longlong2 scan[kThreads / 32];
  uint2 absent[16];                      // per unit modulo 16: blocks without a page, blocks past the length
  alignas(16) float4 heads[8][8];        // per unit modulo 8 and block: 2^e of keys, e of values, 2^-e, marks
  alignas(16) long long off[16][8];      // per unit modulo 16: where its blocks lie
  float qc[4][kR];                       // per row: score of a product of the operands
  float top[2][2][kR], sum[2][2][kR], bad[2][2][kR];  // of two items, of two streams
};

// Two float16 values of the bytes that `sel` picks
template <uint32_t sel>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(0xE480E480u));
  return r;
}

// Loads and stores at a register's address plus a constant
template <int off>
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at), "n"(off));
  return v;
}
template <int off>
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0+%1], {%2, %3, %4, %5};" ::"r"(at), "n"(off), "r"(a), "r"(b), "r"(c), "r"(d));
}
// f(0), ..., f(N - 1) with constants as arguments
template <int... I, class F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N>
using Upto = std::make_integer_sequence<int, N>;

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn8_tc_kernel(const __grid_constant__ AttnParams P) {
  using C = Shape8<D>;
  using B = Kv8Block<D>;
  extern __shared__ unsigned char dsm[];
  __shared__ __align__(16) Shared8 S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* sq = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);
  unsigned char* ring = sq + C::kTile;
  unsigned char* raws = ring + C::kStages * C::kTile;

  if (tid == 0) {
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], 4);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&S.full[i], 4);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_done[i], 1);
    }
    mbar_init(&S.q_free, 1);
    mbar_init(&S.o_free, 8);
    mbar_init(&S.end, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.q_full[i], 8);
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_free[i], 18);
      S.items[i] = Item8{};
      S.items[i].last = 1;  // what a role reads that gave up waiting
    }
    fence_mbar_init();
  }
  if (!find_run<kThreads, Work8>(P, S.scan, &S.run, &S.first)) return;
  if (warp == kWarpMma) tmem_alloc(&S.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  constexpr uint32_t kColO = 256;  // scores of the streams at columns 0 and 128, outputs from here

  // Every wait has a limit. A role that met it leaves; what comes out is not used.
  int tries = kWaitTries;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar), p = parity & 1u;
    int left = tries;
    while (!mbar_try(at, p))
      if (--left <= 0) {
        tries = 0;
        break;
      }
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    if (!__all_sync(0xFFFFFFFFu, tries > 0)) tries = 0;
  };
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp < kWarpUnpack) {
    // ---- scores to weights: a thread a row, units of one stream
    more_registers<152>();
    const int g = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t cols = tmem + lanes + 128 * g, outs = tmem + lanes + kColO;
    int phase = 0;
    uint32_t done0 = 0, done1 = 0;  // items that used a stream's outputs
    uint32_t unit0 = 0;  // units of the run before the item
    for (int k = 0;; ++k) {
      wait_warp(&S.item_full[k & 3], k >> 2);
      if (tries <= 0) break;
      const Item8& it = S.items[k & 3];
      const int units = it.end - it.unit, first_unit = it.unit, all_see = it.all_see, rows = it.rows;
      const int tok = (it.w.rt * kR + min(row, rows - 1)) / P.group;
      const int sees = min(max(it.w.len - it.w.n + tok + 1, 0), it.w.len);
      wait_warp(&S.q_full[k & 3], k >> 2);
      const float qc = row < rows ? S.qc[k & 3][row] : 0.f;
      float m = -FLT_MAX, poison = 0.f;  // NaN once the row sees a marked value
      float2 l2 = make_float2(0.f, 0.f);
      for (int u = g; u < units && tries > 0; u += 2, ++phase) {
        wait_warp(&S.s_full[g], phase);
        if (tries <= 0) break;
        tc_fence_after();
        const float4* heads = S.heads[(unit0 + u) & 7];
        const int lim = sees - kUnit * (first_unit + u);
        const bool masked = kUnit * (first_unit + u + 1) > all_see;  // some row does not see some of these
        // The row's factor of block b: held, so that a sum of 0 stays 0; what is past that decides the
        // softmax by itself
        auto factor = [&](float keys) { return fminf(fmaxf(qc * keys, -1.2676506e30f), 1.2676506e30f); };
        // Once for the maximum, half of the columns at a time, and once for the weights: both halves at
        // once, or read once, leave the compiler short of registers.
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        uint32_t marks = 0;
        auto maxima = [&](int half, auto masked) {
          uint32_t r[64];
          tmem_ld64(cols + 64 * half, r);
          float4 h[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) h[b] = heads[4 * half + b];
          tmem_wait_ld(r);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            marks |= __float_as_uint(h[b].w);
            const float f = factor(h[b].x);
            const float2 f2 = make_float2(f, f), e2 = make_float2(h[b].y, h[b].y);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const int at = 16 * b + 2 * n;
              float2 z = fma2(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), f2, e2);
              if constexpr (masked) {
                if (64 * half + at >= lim) z.x = -INFINITY;
                if (64 * half + at + 1 >= lim) z.y = -INFINITY;
              }
              x[n & 3] = max3(x[n & 3], z.x, z.y);
            }
          }
        };
        if (masked) {
          maxima(0, std::true_type());
          maxima(1, std::true_type());
        } else {
          maxima(0, std::false_type());
          maxima(1, std::false_type());
        }
        if (marks) {
          for (int b = 0; b < 8; ++b) {
            const uint32_t w = __float_as_uint(heads[b].w);
            const int here = lim - 16 * b;
            const uint32_t seen = here >= 16 ? 0xFFFFu : here > 0 ? (1u << here) - 1u : 0u;
            if (w & seen) l2.x = NAN;
            if ((w >> 16) & seen) poison = NAN;
          }
        }
        const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        const bool move = top - m > kSlack;
        if (u < 2) {
          if (move) m = top - kLift;
        } else if (__any_sync(0xFFFFFFFFu, move)) {
          // the products before these scores are done: nobody else is at the outputs
          const float now = move ? top - kLift : m, down = ex2_fast(m - now);
          m = now;
          l2.x *= down;
          l2.y *= down;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            float o[32];
            uint32_t w[32];
            tmem_ld32(outs + D * g + d, o);
#pragma unroll
            for (int n = 0; n < 32; ++n) w[n] = __float_as_uint(o[n] * down);
            tmem_st32(outs + D * g + d, w);
          }
        }
        // Far from 0 the score that was rounded for the maximum is not the one that a fused operation has here.
        const bool far = row < rows && fabsf(m) > 1048576.f && m > -FLT_MAX;
        auto weights = [&](int half, auto masked, auto rounded) {
          uint32_t r[64], w[32];
          tmem_ld64(cols + 64 * half, r);
          float4 h[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) h[b] = heads[4 * half + b];
          tmem_wait_ld(r);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float f = factor(h[b].x), e = rounded && far ? h[b].y : h[b].y - m;
            const float2 f2 = make_float2(f, f), e2 = make_float2(e, e);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const int at = 16 * b + 2 * n;
              float2 z = fma2(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), f2, e2);
              if constexpr (masked) {
                if (64 * half + at >= lim) z.x = -INFINITY;
                if (64 * half + at + 1 >= lim) z.y = -INFINITY;
              }
              if constexpr (rounded) z = add2(z, far ? make_float2(-m, -m) : make_float2(0.f, 0.f));
              z.x = ex2_fast(z.x);
              z.y = ex2_fast(z.y);
              sum = add2(sum, z);
              w[8 * b + n] = pack_f16x2(z.x, z.y);
            }
            l2 = fma2(sum, make_float2(h[b].z, h[b].z), l2);
          }
          tmem_st32(cols + 32 * half, w);
        };
        if (__any_sync(0xFFFFFFFFu, far)) {
          weights(0, std::true_type(), std::true_type());
          weights(1, std::true_type(), std::true_type());
        } else if (masked) {
          weights(0, std::true_type(), std::false_type());
          weights(1, std::true_type(), std::false_type());
        } else {
          weights(0, std::false_type(), std::false_type());
          weights(1, std::false_type(), std::false_type());
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&S.p_full[g]);
      }
      if (tries <= 0) break;
      unit0 += units;

      // ---- join the streams: each has half of the values of both
      S.top[k & 1][g][row] = m;
      S.sum[k & 1][g][row] = l2.x + l2.y;
      S.bad[k & 1][g][row] = poison;
      named_sync(1, kSoftmaxThreads);
      const float m0 = S.top[k & 1][0][row], m1 = S.top[k & 1][1][row], M = fmaxf(m0, m1);
      const float f0 = ex2_fast(m0 - M), f1 = ex2_fast(m1 - M);
      const float L = S.sum[k & 1][0][row] * f0 + S.sum[k & 1][1][row] * f1;
      const bool whole = it.whole;
      const float all = (whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f) + S.bad[k & 1][0][row] + S.bad[k & 1][1][row];
      const float2 a0 = make_float2(f0 * all, f0 * all), a1 = make_float2(f1 * all, f1 * all);
      const Walk& w = it.w;
      const long long at = out_row(P, w, kR, min(row, rows - 1));
      float* part = P.part + (2 * static_cast<long long>(blockIdx.x) + (w.base < S.run.u0 ? 0 : 1)) * C::kPart;
      if (units > 0) wait_warp(&S.o_done[0], done0++);
      if (units > 1) wait_warp(&S.o_done[1], done1++);
      if (tries <= 0) break;
      tc_fence_after();
#pragma unroll 1
      for (int d = D / 2 * g; d < D / 2 * (g + 1); d += 32) {
        float2 o[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n] = make_float2(0.f, 0.f);
        if (units > 0) {
          float x[32];
          tmem_ld32(outs + d, x);
#pragma unroll
          for (int n = 0; n < 16; ++n) o[n] = fma2(make_float2(x[2 * n], x[2 * n + 1]), a0, o[n]);
        }
        if (units > 1) {
          float x[32];
          tmem_ld32(outs + D + d, x);
#pragma unroll
          for (int n = 0; n < 16; ++n) o[n] = fma2(make_float2(x[2 * n], x[2 * n + 1]), a1, o[n]);
        }
        if (row >= rows) continue;
        if (whole) {
          uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + at * D + d);
#pragma unroll
          for (int n = 0; n < 4; ++n)
            to[n] = make_uint4(pack_bf16(o[4 * n].x, o[4 * n].y), pack_bf16(o[4 * n + 1].x, o[4 * n + 1].y),
                               pack_bf16(o[4 * n + 2].x, o[4 * n + 2].y), pack_bf16(o[4 * n + 3].x, o[4 * n + 3].y));
        } else {
          float4* to = reinterpret_cast<float4*>(part + row * D + d);
#pragma unroll
          for (int n = 0; n < 8; ++n) to[n] = make_float4(o[2 * n].x, o[2 * n].y, o[2 * n + 1].x, o[2 * n + 1].y);
        }
      }
      tc_fence_before();
      if (units > 0) arrive_warp(&S.o_free);
      if (g == 0 && row < rows) {
        if (whole) {
          store_lse(P, at, M, L);
        } else {
          part[kR * D + row] = M;
          part[kR * D + kR + row] = L;
        }
      }
      if (!whole)
        join_pieces<kSoftmaxThreads, kR, D, 4>(P, w, S.run, rows, tid, &S.last,
                                               [] { named_sync(2, kSoftmaxThreads); });
      const int last = it.last;
      arrive_warp(&S.item_free[k & 3]);
      if (last) break;
    }
  } else if (warp < kWarpMma) {
    // ---- codes (and queries) to operands
    fewer_registers<64>();
    const int wid = warp & 3, which = (warp - kWarpUnpack) >> 2;  // keys, values
    // Where this thread's 16-byte chunks of codes lie, and what they become: D / 16 of keys (16 values of a token)
    // or of values (8 of a pair of tokens), of the blocks 2 wid and 2 wid + 1. Eight lanes in a row keep the banks
    // apart, of the bytes that they read and of the operands that they write. D = 128: what the places are
    // exchanged with depends on a chunk's number by a bit.
    constexpr int N = D / 16;
    const uint32_t a_raw = smem_u32(raws), a_ring = smem_u32(ring);
    uint32_t from, to;
    if (which == 0) {
      const int row = D == 128 ? 2 * (lane >> 4) + ((lane >> 2) & 1) : lane >> 2;  // of 4 or 8 at a time
      const int j = D == 128 ? (lane & 3) + 4 * (((lane >> 2) ^ (lane >> 3)) & 1) : lane & 3;
      from = a_raw + (32 * wid + row) * D + 16 * B::key_place(row, j);
      to = a_ring + (j >> 2) * C::kSlab + (32 * wid + row) * 128 + (((2 * (j & 3)) ^ row) << 4);
    } else {
      constexpr int PV = D / 8;  // chunks of a pair
      const int pair = lane / PV, x = lane % PV;
      from = a_raw + (16 * wid + pair) * 2 * D + 16 * B::val_place(pair, x);
      to = a_ring + (x >> 3) * C::kSlab + (16 * wid + pair) * 256 + (((x & 7) ^ (2 * pair)) << 4);
    }
    uint32_t pos0 = 0, unit0 = 0, used = 0;
    for (int k = 0;; ++k) {
      wait_warp(&S.item_full[k & 3], k >> 2);
      if (tries <= 0) break;
      const Item8& it = S.items[k & 3];
      const int units = it.end - it.unit, rows = it.rows, last = it.last, row0 = it.w.rt * kR, r0 = it.w.r0;
      const int head0 = it.w.h * P.group;
      arrive_warp(&S.item_free[k & 3]);
      if (units > 0) {
        constexpr int QV = D / 8, PASS = 128 / QV, NQ = kR / PASS / 2;  // vectors of a row, rows at a time
        const int j = lane % QV, rr = kR / 2 * which + (32 * wid + lane) / QV;  // half of the rows
        uint4 x[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int row = row0 + PASS * n + rr, i = row / P.group;
          x[n] = make_uint4(0u, 0u, 0u, 0u);
          if (PASS * n + rr < rows)
            x[n] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) + (r0 + i) * P.qs +
                                                        static_cast<long long>(head0 + row - i * P.group) * D) + j);
        }
        if (used > 0) wait_warp(&S.q_free, used - 1);
        if (tries <= 0) break;
        ++used;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          if (kR / 2 * which + PASS * n >= rows) break;
          const int r = PASS * n + rr;
          unsigned most = largest_finite(x[n]);
#pragma unroll
          for (int d = QV / 2; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d, QV));
          float undo;
          const float up = query_scale(most, P.c, &undo);
          if (j == 0) S.qc[k & 3][r] = undo;
          uint32_t f[4];
          query_f16(x[n], up, f);
          *reinterpret_cast<uint4*>(sq + (j >> 3) * C::kSlab + r * 128 + (((j & 7) ^ (r & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_async_shared();
      }
      arrive_warp(&S.q_full[k & 3]);

      for (int u = 0; u < units; ++u) {
        // keys of an item's first two units come first, then values and keys in turn
        const uint32_t pos = pos0 + (which == 0 ? max(2 * u - 1, 0) : min(2 * u + 2, 2 * units - 1));
        const uint32_t raw = pos % C::kRaws, st = pos % C::kStages;
        const uint32_t src = from + raw * C::kRaw, dst = to + st * C::kTile;
        wait_warp(&S.raw_full[raw], pos / C::kRaws);
        if (tries <= 0) break;
        const uint2 gone = S.absent[(unit0 + u) & 15];
        const uint32_t none = ((gone.x | gone.y) >> (2 * wid)) & 3u;
        uint4 c[N];
        if (which == 0) {
          each(Upto<N>(), [&](auto n_) { c[n_] = ld_shared_v4<n_ * 512>(src); });
          if (lane < 2) {
            uint2 h = *reinterpret_cast<const uint2*>(raws + raw * C::kRaw + 8 * 16 * D + 16 * (2 * wid + lane));
            if ((none >> lane) & 1u)  // without a page: marked keys
              h = make_uint2(0u, (gone.x >> (2 * wid + lane)) & 1u ? 0xFFFFu : 0u);
            const int ek = static_cast<signed char>(h.x & 0xFFu), ev = static_cast<signed char>((h.x >> 8) & 0xFFu);
            S.heads[(unit0 + u) & 7][2 * wid + lane] =
                make_float4(__int_as_float((ek + 127) << 23), static_cast<float>(ev), __int_as_float((127 - ev) << 23),
                            __uint_as_float(h.y));
          }
        } else {
          each(Upto<N>(), [&](auto n_) {
            constexpr int n = n_;
            c[n] = ld_shared_v4<n * 512>(D == 128 && (n & 1) ? src ^ 64u : src);
          });
        }
        if (none) {
          each(Upto<N>(), [&](auto n_) {
            constexpr int n = n_;
            if ((none >> (n >= N / 2)) & 1u) c[n] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          });
        }
        if (pos >= C::kStages) wait_warp(&S.empty[st], pos / C::kStages - 1);
        if (tries <= 0) break;
        each(Upto<N>(), [&](auto n_) {
          constexpr int n = n_;
          const uint32_t at = D == 128 && (n & 1) ? dst ^ 64u : dst;
          constexpr int off = n * (D == 128 ? 512 : 1024);
          if (which == 0) {
            st_shared_v4<off>(at, code_pair<0x4140>(c[n].x), code_pair<0x4342>(c[n].x), code_pair<0x4140>(c[n].y),
                              code_pair<0x4342>(c[n].y));
            st_shared_v4<off>(at ^ 16u, code_pair<0x4140>(c[n].z), code_pair<0x4342>(c[n].z), code_pair<0x4140>(c[n].w),
                              code_pair<0x4342>(c[n].w));
          } else {
            st_shared_v4<off>(at, code_pair<0x4240>(c[n].x), code_pair<0x4240>(c[n].y), code_pair<0x4240>(c[n].z),
                              code_pair<0x4240>(c[n].w));
            st_shared_v4<off + 128>(at ^ 16u, code_pair<0x4341>(c[n].x), code_pair<0x4341>(c[n].y),
                                    code_pair<0x4341>(c[n].z), code_pair<0x4341>(c[n].w));
          }
        });
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.raw_empty[raw]);
          mbar_arrive(&S.full[st]);
        }
      }
      pos0 += 2 * units;
      if (tries <= 0) break;
      unit0 += units;
      if (last) break;
    }
  } else {
    fewer_registers<48>();
    if (warp == kWarpMma) {
      // ---- products: one elected thread does it all (see sv_prompt.cu)
      constexpr uint32_t kScores = (1u << 4) | (16u << 17) | (8u << 24);  // float16 operands, float32 sums
      constexpr uint32_t kOutputs = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17) | (8u << 24);
      if (elect_one()) {
        const uint32_t a_q = operand_lo(smem_u32(sq), 16), a_key = operand_lo(smem_u32(ring), 16);
        const uint32_t a_val = operand_lo(smem_u32(ring), C::kSlab);
        uint32_t pos = 0, items = 0, weights[2] = {0, 0};
        for (int k = 0;; ++k) {
          wait(&S.item_full[k & 3], k >> 2);
          const int units = S.items[k & 3].end - S.items[k & 3].unit, last = S.items[k & 3].last;
          mbar_arrive(&S.item_free[k & 3]);
          if (tries <= 0) break;
          if (units > 0) wait(&S.q_full[k & 3], k >> 2);
          auto step = [&](int u, auto g_) {  // scores of unit u, outputs of the one before
            constexpr int g = decltype(g_)::value;
            if (u < units) {
              const uint32_t st = pos % C::kStages;
              wait(&S.full[st], pos / C::kStages);
              if (tries <= 0) return;
              tc_fence_after();
              const uint32_t key = a_key + st * (C::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * C::kSlab + 32 * (kk & 3)) >> 4;
                mma_ss(tmem + 128 * g, a_q + off, key + off, kScores, kk > 0);
              }
              tc_commit(&S.s_full[g]);
              tc_commit(&S.empty[st]);
              if (u == units - 1) tc_commit(&S.q_free);
              ++pos;
            }
            if (u > 0) {
              constexpr int e = g ^ 1;
              const uint32_t st = pos % C::kStages;
              wait(&S.full[st], pos / C::kStages);
              if (u == 1 && items > 0) wait(&S.o_free, items - 1);
              wait(&S.p_full[e], weights[e]++);
              if (tries <= 0) return;
              tc_fence_after();
              const uint32_t val = a_val + st * (C::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ts(tmem + kColO + D * e, tmem + 128 * e + 8 * kk, val + ((2048 * kk) >> 4), kOutputs,
                       u > 2 || kk > 0);
              tc_commit(&S.empty[st]);
              if (u >= units - 1) tc_commit(&S.o_done[e]);
              ++pos;
            }
          };
          for (int u = 0; u <= units && tries > 0 && units > 0; u += 2) {
            step(u, std::integral_constant<int, 0>());
            if (u + 1 <= units && tries > 0) step(u + 1, std::integral_constant<int, 1>());
          }
          items += units > 0;
          if (last || tries <= 0) break;
        }
        // all products are done before the memory goes
        tc_commit(&S.end);
        if (!mbar_wait_bounded(&S.end, 0, kWaitCycles)) tries = 0;
      }
      __syncwarp();
    } else if (warp == kWarpCopy) {
      // ---- copies. Where the blocks lie is looked up four units at a time, a lane a block, and a round
      // before it is needed.
      const int bpp_log = 31 - __clz(P.ps >> 4);  // blocks of a page: a power of two
      const int mine = lane >> 3, block = lane & 7;
      uint32_t pos = 0, unit0 = 0;
      for (int k = 0;; ++k) {
        wait_warp(&S.item_full[k & 3], k >> 2);
        if (tries <= 0) break;
        const Item8& it = S.items[k & 3];
        const int units = it.end - it.unit, unit = it.unit, len = it.w.len, h = it.w.h, last = it.last;
        const int32_t* table = P.table + static_cast<long long>(it.w.b) * P.max_blocks;
        arrive_warp(&S.item_free[k & 3]);
        auto look_up = [&](int u) {  // -2: past the length or the item
          const int blk = 8 * (unit + u + mine) + block;
          return u + mine < units && 16 * blk < len ? max(table[blk >> bpp_log], -1) : -2;
        };
        auto copy = [&](int u, bool values) {
          const uint32_t st = pos % C::kRaws;
          if (pos >= C::kRaws) wait_warp(&S.raw_empty[st], pos / C::kRaws - 1);
          if (tries <= 0) return;
          const long long off = S.off[(unit0 + u) & 15][block];
          const bool there = lane < 8 && off >= 0;
          const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, there));
          if (lane == 0) {
            if (n)
              mbar_arrive_expect_tx(&S.raw_full[st], n * (values ? 16 * D : 16 * D + 16));
            else
              mbar_arrive(&S.raw_full[st]);
          }
          __syncwarp();
          if (there) {
            unsigned char* to = raws + st * C::kRaw;
            bulk_g2s(to + block * 16 * D, P.cache + off + (values ? B::kValCodes : B::kKeyCodes), 16 * D, &S.raw_full[st]);
            if (!values) bulk_g2s(to + 8 * 16 * D + 16 * block, P.cache + off + B::kHead, 16, &S.raw_full[st]);
          }
          ++pos;
        };
        int page = look_up(0);
        for (int u = 0; u <= units && tries > 0; ++u) {
          if (u < units) {
            if ((u & 3) == 0) {
              const bool there = page >= 0 && page < P.num_pages, lost = page >= -1 && !there;
              const int blk = 8 * (unit + u + mine) + block;
              const uint32_t all_lost = __ballot_sync(0xFFFFFFFFu, lost), none = __ballot_sync(0xFFFFFFFFu, page == -2);
              S.off[(unit0 + u + mine) & 15][block] =
                  there ? ((((static_cast<long long>(page) * P.hkv) + h) << bpp_log) + (blk & ((1 << bpp_log) - 1))) *
                              B::kBytes
                        : -1;
              if (block == 0)
                S.absent[(unit0 + u + mine) & 15] =
                    make_uint2((all_lost >> (8 * mine)) & 0xFFu, (none >> (8 * mine)) & 0xFFu);
              page = look_up(u + 4);
              __syncwarp();
            }
            copy(u, false);
          }
          if (u > 0 && tries > 0) copy(u - 1, true);
        }
        if (tries <= 0) break;
        unit0 += units;
        if (last) break;
      }
      // no copy is in flight when the CTA ends, whoever gave up
      for (uint32_t p = pos > C::kRaws ? pos - C::kRaws : 0; p < pos; ++p)
        if (!mbar_wait_bounded(&S.raw_full[p % C::kRaws], (p / C::kRaws) & 1, kWaitCycles)) tries = 0;
    } else if (warp == kWarpItems && lane == 0) {
      // ---- items, ahead of all others
      Walk w = S.first;
      int unit = static_cast<int>(S.run.u0 - w.base);
      for (int k = 0;; ++k) {
        if (k >= 4) wait(&S.item_free[k & 3], (k >> 2) - 1);
        if (tries <= 0) break;
        const int end = static_cast<int>(min(static_cast<long long>(w.nu), S.run.u1 - w.base));
        Item8& it = S.items[k & 3];
        it.w = w;
        it.rows = min(kR, w.n * P.group - w.rt * kR);
        const int i0 = w.rt * kR / P.group, i1 = (w.rt * kR + it.rows - 1) / P.group;
        it.all_see = w.len - w.n + i0 + 1;
        // units that no row of the tile sees are left out
        const int seen = min(max(w.len - w.n + i1 + 1, 0), w.len);
        it.unit = unit;
        it.end = max(unit, min(end, (seen + kUnit - 1) / kUnit));
        it.whole = w.base >= S.run.u0 && end == w.nu;
        const bool last = w.base + end >= S.run.u1;
        it.last = last;
        mbar_arrive(&S.item_full[k & 3]);
        if (last) break;
        next_item<Work8>(P, w);
        unit = 0;
      }
    }
  }
  if (tries <= 0) atomicOr(P.err, 1u);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_dim8_tc(const AttnParams& P, int sms, cudaStream_t stream) {
  using C = Shape8<D>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn8_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn8_tc_kernel<D><<<sms, kThreads, C::kSmem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention8_tc(const AttnParams& P, int D, int sms, cudaStream_t stream) {
  return D == 64 ? launch_dim8_tc<64>(P, sms, stream) : launch_dim8_tc<128>(P, sms, stream);
}

}  // namespace sv
