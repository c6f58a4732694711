// Attention over the 8-bit cache for many rows a head, on the fifth-generation tensor cores.
//
// Up to 128 rows (new tokens x query heads of one key/value head) share what is read, or 256 as two tiles. A
// CTA goes over the cache 128 tokens at a time:
//   scores [128 rows x 128 tokens] = q [shared memory] k^T [shared memory]
//   outputs [128 rows x D] += weights [tensor memory] v [shared memory]
// There are two streams, each with scores, outputs, maxima and sums of its own: while the tensor cores work for
// one, the softmax of the other runs, a thread a row. Up to 128 rows, tiles of tokens go to them in turn, and at
// an item's end the two are joined, half of the D values by each. With more rows (PAIR) each has a tile of rows
// of its own, so that codes are unpacked once for both.
//
// Codes come as they are, by bulk copies into a ring, and become float16 on their way through registers to
// operands in the 128-byte swizzle. With the conversion, for nothing, goes a power of two that brings a unit's
// blocks to one exponent, for keys and for values, which joins the factor of the scores and the exponent of the
// weights as in sv_attn8.cu. That is exact where the exponents are within 2^14 (2^4 for values) of one another; a
// unit where they are not has its codes as they are, and each block its own factors in the softmax. With each block's own factors always, its threads ran out of registers and took a half more
// time; values as bfloat16, which need none, cost twice the instructions where codes are converted.
//
// One persistent CTA an SM, its warps specialised: eight for the softmax, four unpack keys and values
// (and bring queries), one issues products, one copies, one walks through the items. The work is cut and
// joined as in sv_attn.cu, in units of 128 tokens.
//
// What bounds it: 1500 new of 16384 tokens twice, 32 + 8 heads of 128, take 660 us, 1165 TFLOP/s, 0.60 of the
// measured bf16 rate, with the tensor cores busy for 0.51 of their cycles and 0.47 of the issue slots used:
// softmax and conversion wait for each other's bytes in the shared memory, which the products' operands keep
// busy. With few rows the conversion bounds it, whatever the rows (64 sequences of up to 8192 tokens, 48 rows a
// head: 154 us, 0.35 of the copy rate). Plain loads into registers a
// tile ahead took 1079 us; more threads to unpack and operands in bfloat16 were slower than these, too.
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

constexpr int kWarpUnpack = 8, kWarpMma = 12, kWarpCopy = 13, kWarpItems = 14;
constexpr int kThreads = 512, kSoftmaxThreads = 256;
constexpr int kR = 128, kUnit = 128;  // rows of a tile, tokens of a unit

// Some token is marked; the exponents of a unit are too far apart, or those of values too far below others before it
constexpr uint32_t kMarked = 1 << 16, kUneven = 1 << 17;
// ... by more than this: a code times 2^-14 is exact in float16; weights times 2^e of a unit's largest values
// are held to 2^-36 of the row's largest, which is 2^-32 of it by each block's own e.
constexpr int kEvenKeys = 14, kEvenValues = 4;
constexpr float kLift8 = 11.f;  // weights are held times 2^11, and moved when they pass 2^15

// Work as it is cut. PAIR: two tiles of rows share a unit of tokens.
template <bool PAIR>
struct Work8 {
  static constexpr int kRows = PAIR ? 2 * kR : kR, kUnit = sv::kUnit, kDearest = 4, kOver = 12, kLeast = 2;
  static __device__ __forceinline__ int weight(int) { return 4; }
};

template <int D, bool PAIR>
struct Shape8 {
  static constexpr int kRows = PAIR ? 2 * kR : kR;
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;       // bytes of 128 rows of 64 float16 values
  static constexpr int kTile = kSlabs * kSlab;  // queries, keys or values of a unit as operands
  static constexpr int kStages = D == 64 ? 6 : 3;
  static constexpr int kRaw = 8 * 16 * D + 128;  // codes of a unit's keys or values; heads of the blocks
  static constexpr int kRaws = D == 64 ? 8 : PAIR ? 3 : 5;
  static constexpr int kQueries = PAIR ? 2 : 1;  // tiles of queries
  static constexpr int kSmem = 1024 + (kQueries + kStages) * kTile + kRaws * kRaw;
  static constexpr long long kPart = kRows * (D + 2);
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
  uint64_t o_done[2], o_free;            // outputs of an item; read (without PAIR)
  uint64_t item_full[4], item_free[4];
  uint64_t meet, end;
  Item8 items[4];
  uint32_t tmem;
  int last;
  Run run;
  Walk first;
  longlong2 scan[kThreads / 32];
  uint2 absent[16];                      // per unit modulo 16: blocks without a page, blocks past the length
  alignas(16) long long off[16][8];      // ... and where its blocks lie
  // per unit modulo 8: what its operands were multiplied with, and the same of each block by itself
  uint32_t unit[8];                      // e of keys and of values plus 64, kMarked, kUneven, 14 bits of its number
  alignas(16) float4 heads[8][8];        // 2^e of keys, e of values, marks
  float qc[4][2 * kR];                   // per row: score of a product of the operands
  float top[2][2][kR], sum[2][2][kR], bad[2][2][kR];  // of two items, of two streams
};

// Two codes, of the bytes that `sel` picks, times a power of two in float16 (twice in `by`; less: -1152 times
// that): a byte under 0x64 is 1024 + code + 128, and all of it is exact.
template <uint32_t sel>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t by, uint32_t less) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(by), "r"(less));
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

// A row's factor of the scores for keys times this: held, so that a sum of 0 stays 0 and what is not seen stays
// so. Operands are below 2^16 and 2^7: at the lower limit, a scale of 0 among what comes there, no score counts;
// at the upper one nothing but their signs does.
__device__ __forceinline__ float score_factor(float qc, float keys, float c) {
  return copysignf(fminf(fmaxf(fabsf(qc * keys), 7.8886091e-31f), 1.2676506e30f), c);
}

// A unit whose codes are operands as they are: each block with its own factors, and weights that may be none (see
// times_two_to), so that the sum takes exponentials of its own. 32 columns at a time, twice. Functions of their
// own: inlined, they make the kernel slower that hardly ever comes here (1500 of 16384 tokens twice: 712 -> 725 us).
struct Uneven8 {
  uint32_t cols;  // of the scores
  const float4* heads;
  int lim;        // tokens that the row sees
  float qc, c;
  __device__ __forceinline__ void scores(int b, const float* x, float2* z) const {  // of block b
    const float4 hb = heads[b];
    const float f = score_factor(qc, hb.x, c);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      z[n] = make_float2(__fmaf_rn(x[2 * n], f, hb.y), __fmaf_rn(x[2 * n + 1], f, hb.y));
      if (16 * b + 2 * n >= lim) z[n].x = -INFINITY;
      if (16 * b + 2 * n + 1 >= lim) z[n].y = -INFINITY;
    }
  }
  __device__ __noinline__ float maximum() const {
    float t = -INFINITY;
#pragma unroll 1
    for (int part = 0; part < 4; ++part) {
      float x[32];
      tmem_ld32(cols + 32 * part, x);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float2 z[8];
        scores(2 * part + b, x + 16 * b, z);
#pragma unroll
        for (int n = 0; n < 8; ++n) t = max3(t, z[n].x, z[n].y);
      }
    }
    return t;
  }
  // Weights, over the scores; returns their part of the softmax's sum
  __device__ __noinline__ float2 weights(float m) const {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int part = 0; part < 4; ++part) {
      float x[32];
      uint32_t w[16];
      tmem_ld32(cols + 32 * part, x);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float2 z[8];
        scores(2 * part + b, x + 16 * b, z);
        const float e = heads[2 * part + b].y;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          sum = add2(sum, make_float2(ex2_fast(z[n].x - e - m), ex2_fast(z[n].y - e - m)));
          w[8 * b + n] = pack_f16(ex2_fast(__fadd_rn(z[n].x, -m)), ex2_fast(__fadd_rn(z[n].y, -m)));
        }
      }
      tmem_st16(cols + 16 * part, w);  // over scores that have been read
    }
    return sum;
  }
};

template <int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) attn8_tc_kernel(const __grid_constant__ AttnParams P) {
  using C = Shape8<D, PAIR>;
  using W = Work8<PAIR>;
  using B = Kv8Block<D>;
  extern __shared__ unsigned char dsm[];
  __shared__ __align__(16) Shared8 S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* sq = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);
  unsigned char* ring = sq + C::kQueries * C::kTile;
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
    mbar_init(&S.meet, kWarpUnpack);
    mbar_init(&S.end, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.q_full[i], 4);
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_free[i], 14);
      S.items[i] = Item8{};
      S.items[i].last = 1;  // what a role reads that gave up waiting
    }
    for (int i = 0; i < 8; ++i) S.unit[i] = ~0u;  // no unit that comes to this place
    fence_mbar_init();
  }
  if (!find_run<kThreads, W>(P, S.scan, &S.run, &S.first)) return;
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
    more_registers<184>();
    const int g = warp >> 2, row = tid & 127, item_row = PAIR ? tid : row;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t cols = tmem + lanes + 128 * g, outs = tmem + lanes + kColO;
    const float fill = P.c < 0.f ? INFINITY : -INFINITY;
    int phase = 0;
    uint32_t done0 = 0, done1 = 0;  // items that used a stream's outputs
    uint32_t unit0 = 0;  // units of the run before the item
    uint32_t meets = 0;
    auto meet = [&] {  // all softmax warps, those apart that gave up
      arrive_warp(&S.meet);
      wait_warp(&S.meet, meets++);
    };
    for (int k = 0;; ++k) {
      wait_warp(&S.item_full[k & 3], k >> 2);
      if (tries <= 0) break;
      const Item8& it = S.items[k & 3];
      const int units = it.end - it.unit, first_unit = it.unit, all_see = it.all_see, rows = it.rows;
      const int tok = (it.w.rt * C::kRows + min(item_row, rows - 1)) / P.group;
      const int sees = min(max(it.w.len - it.w.n + tok + 1, 0), it.w.len);
      wait_warp(&S.q_full[k & 3], k >> 2);
      const float qc = item_row < rows ? S.qc[k & 3][item_row] : 0.f;
      float m = -FLT_MAX, poison = 0.f;  // NaN once the row sees a marked value
      float2 l2 = make_float2(0.f, 0.f);
      const bool idle = PAIR && kR * g >= rows;  // no rows of this stream's
      for (int u = PAIR ? 0 : g; u < units && tries > 0 && !idle; u += PAIR ? 1 : 2, ++phase) {
        // One word says all about the unit: it is read ahead of the wait, since any access to the shared memory is
        // long on its way while the tensor cores read their operands.
        const volatile uint32_t* about_at = &S.unit[(unit0 + u) & 7];
        uint32_t about = *about_at;
        wait_warp(&S.s_full[g], phase);
        if (tries <= 0) break;
        tc_fence_after();
        if (((about >> 18) ^ (unit0 + u)) & 0x3FFFu) about = *about_at;  // it was too early
        const float4* heads = S.heads[(unit0 + u) & 7];
        const int unit_e = static_cast<int>((about >> 8) & 0xFFu) - 64;  // of the values
        const float keys = __int_as_float(((about & 0xFFu) + 63) << 23);
        const int lim = sees - kUnit * (first_unit + u);
        const bool masked = kUnit * (first_unit + u + 1) > all_see;  // some row does not see some of these
        // The row's maximum t has come: moves m, with the sums and outputs
        auto move_to = [&](float t) {
          const bool move = t - m > kSlack;
          if (u < (PAIR ? 1 : 2)) {
            if (move) m = t - kLift8;
          } else if (__any_sync(0xFFFFFFFFu, move)) {
            // the products before these scores are done: nobody else is at the outputs
            const float now = move ? t - kLift8 : m, down = ex2_fast(m - now);
            l2.x = times_two_to(l2.x, m - now);
            l2.y = times_two_to(l2.y, m - now);
            m = now;
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
        };
        if (about & kMarked) {
          for (int b = 0; b < 8; ++b) {
            const uint32_t w = __float_as_uint(heads[b].z);
            const int here = lim - 16 * b;
            const uint32_t seen = here >= 16 ? 0xFFFFu : here > 0 ? (1u << here) - 1u : 0u;
            if (w & seen) l2.x = NAN;
            if ((w >> 16) & seen) poison = NAN;
          }
        }
        if (!(about & kUneven)) {
          uint32_t r[128];
          tmem_ld64(cols, r);
          tmem_ld64(cols + 64, r + 64);
          const float f = score_factor(qc, keys, P.c), e = static_cast<float>(unit_e);
          tmem_wait_ld(r);
          tmem_wait_ld(r + 64);
          if (masked) {
#pragma unroll
            for (int n = 0; n < 128; ++n)
              if (n >= lim) r[n] = __float_as_uint(fill);
          }
          float t;
          if (P.c < 0.f) {
            float x[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
            for (int n = 0; n < 128; n += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = min3(x[e], __uint_as_float(r[n + 2 * e]), __uint_as_float(r[n + 2 * e + 1]));
            t = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
          } else {
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 128; n += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = max3(x[e], __uint_as_float(r[n + 2 * e]), __uint_as_float(r[n + 2 * e + 1]));
            t = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
          }
          move_to(__fmaf_rn(t, f, e));
          const float2 f2 = make_float2(f, f), b2 = make_float2(e - m, e - m);
          // Far from 0 the score that was rounded for the maximum is not the one that a fused operation has here
          const bool far = item_row < rows && fabsf(m) > 1048576.f && m > -FLT_MAX;
          float2 sum = make_float2(0.f, 0.f);
          auto weights = [&](auto rounded) {
#pragma unroll
            for (int part = 0; part < 4; ++part) {
              uint32_t w[16];
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                const float2 z = make_float2(__uint_as_float(r[32 * part + 2 * n]), __uint_as_float(r[32 * part + 2 * n + 1]));
                float2 p = fma2(z, f2, b2);
                if constexpr (rounded) {
                  if (far) p = make_float2(__fadd_rn(__fmaf_rn(z.x, f, e), -m), __fadd_rn(__fmaf_rn(z.y, f, e), -m));
                }
                p.x = ex2_fast(p.x);
                p.y = ex2_fast(p.y);
                sum = add2(sum, p);
                w[n] = pack_f16(p.x, p.y);
              }
              tmem_st16(cols + 16 * part, w);
            }
          };
          if (__any_sync(0xFFFFFFFFu, far))
            weights(std::true_type());
          else
            weights(std::false_type());
          const float undo = __int_as_float((127 - unit_e) << 23);
          l2 = fma2(sum, make_float2(undo, undo), l2);
        } else {
          const Uneven8 slow{cols, heads, lim, qc, P.c};
          move_to(slow.maximum());
          l2 = add2(l2, slow.weights(m));
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&S.p_full[g]);
      }
      if (tries <= 0) break;
      unit0 += units;

      const bool whole = it.whole;
      const Walk& w = it.w;
      const long long at = out_row(P, w, C::kRows, min(item_row, rows - 1));
      float* part = P.part + (2 * static_cast<long long>(blockIdx.x) + (w.base < S.run.u0 ? 0 : 1)) * C::kPart;
      float M = m, L = l2.x + l2.y, all = poison, f0 = 1.f, f1 = 0.f;
      int from = 0, to = D;  // of the outputs
      if (!PAIR) {
        // ---- join the streams: each has half of the values of both
        S.top[k & 1][g][row] = m;
        S.sum[k & 1][g][row] = L;
        S.bad[k & 1][g][row] = poison;
        meet();
        const float m0 = S.top[k & 1][0][row], m1 = S.top[k & 1][1][row];
        M = fmaxf(m0, m1);
        f0 = ex2_fast(m0 - M);
        f1 = ex2_fast(m1 - M);
        L = times_two_to(S.sum[k & 1][0][row], m0 - M) + times_two_to(S.sum[k & 1][1][row], m1 - M);
        all = S.bad[k & 1][0][row] + S.bad[k & 1][1][row];
        from = D / 2 * g;
        to = from + D / 2;
        if (units > 0) wait_warp(&S.o_done[0], done0++);
        if (units > 1) wait_warp(&S.o_done[1], done1++);
      } else if (units > 0 && !idle) {
        wait_warp(&S.o_done[g], done0++);
      }
      if (tries <= 0) break;
      tc_fence_after();
      all += whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
      const float2 a0 = make_float2(f0 * all, f0 * all), a1 = make_float2(f1 * all, f1 * all);
      if (!idle) {
#pragma unroll 1
        for (int d = from; d < to; d += 32) {
          float2 o[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) o[n] = make_float2(0.f, 0.f);
          if (units > 0) {
            float x[32];
            tmem_ld32(outs + (PAIR ? D * g : 0) + d, x);
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] = fma2(make_float2(x[2 * n], x[2 * n + 1]), a0, o[n]);
          }
          if (!PAIR && units > 1) {
            float x[32];
            tmem_ld32(outs + D + d, x);
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n] = fma2(make_float2(x[2 * n], x[2 * n + 1]), a1, o[n]);
          }
          if (item_row >= rows) continue;
          if (whole) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + at * D + d);
#pragma unroll
            for (int n = 0; n < 4; ++n)
              out[n] = make_uint4(pack_bf16(o[4 * n].x, o[4 * n].y), pack_bf16(o[4 * n + 1].x, o[4 * n + 1].y),
                                  pack_bf16(o[4 * n + 2].x, o[4 * n + 2].y), pack_bf16(o[4 * n + 3].x, o[4 * n + 3].y));
          } else {
            float4* out = reinterpret_cast<float4*>(part + item_row * D + d);
#pragma unroll
            for (int n = 0; n < 8; ++n) out[n] = make_float4(o[2 * n].x, o[2 * n].y, o[2 * n + 1].x, o[2 * n + 1].y);
          }
        }
      }
      tc_fence_before();
      // With PAIR a stream's outputs are read by its own warps alone, and the next item's first products into them
      // wait for weights that these warps give afterwards. (Warps without rows would count here ahead of the
      // others, item after item, and a phase that is two ahead is waited for in vain.)
      if (!PAIR && units > 0) arrive_warp(&S.o_free);
      if ((PAIR || g == 0) && item_row < rows) {
        if (whole) {
          store_lse(P, at, M, L);
        } else {
          part[C::kRows * D + item_row] = M;
          part[C::kRows * D + C::kRows + item_row] = L;
        }
      }
      if (!whole)
        join_pieces<kSoftmaxThreads, C::kRows, D, 4, true>(P, w, S.run, rows, tid, &S.last, meet);
      const int last = it.last;
      arrive_warp(&S.item_free[k & 3]);
      if (last) break;
    }
  } else if (warp < kWarpMma) {
    // ---- codes (and queries) to operands
    fewer_registers<80>();
    const int wid = warp & 3;
    // Where this thread's 16-byte chunks of codes lie, and what they become: D / 16 of keys (16 values of a token)
    // and of values (8 of a pair of tokens), of the blocks 2 wid and 2 wid + 1. Eight lanes in a row keep the banks
    // apart of the operands that they write. D = 128: what the places are exchanged with depends on a chunk's
    // number by a bit.
    constexpr int N = D / 16;
    const uint32_t a_ring = smem_u32(ring);
    uint32_t key_from, key_to, value_from, value_to;  // in a stage of bytes; in a tile of operands
    {
      const int row = D == 128 ? 2 * (lane >> 4) + ((lane >> 2) & 1) : lane >> 2;  // of 4 or 8 at a time
      const int j = D == 128 ? (lane & 3) + 4 * (((lane >> 2) ^ (lane >> 3)) & 1) : lane & 3;
      key_from = smem_u32(raws) + (32 * wid + row) * D + 16 * B::key_place(row, j);
      key_to = a_ring + (j >> 2) * C::kSlab + (32 * wid + row) * 128 + (((2 * (j & 3)) ^ row) << 4);
      constexpr int PV = D / 8;  // chunks of a pair
      const int pair = lane / PV, x = lane % PV;
      value_from = smem_u32(raws) + (16 * wid + pair) * 2 * D + 16 * B::val_place(pair, x);
      value_to = a_ring + (x >> 3) * C::kSlab + (16 * wid + pair) * 256 + (((x & 7) ^ (2 * pair)) << 4);
    }
    uint32_t pos0 = 0, unit0 = 0, used = 0;
    for (int k = 0;; ++k) {
      wait_warp(&S.item_full[k & 3], k >> 2);
      if (tries <= 0) break;
      const Item8& it = S.items[k & 3];
      const int units = it.end - it.unit, rows = it.rows, last = it.last, row0 = it.w.rt * C::kRows, r0 = it.w.r0;
      const int head0 = it.w.h * P.group;
      arrive_warp(&S.item_free[k & 3]);
      if (units > 0) {
        constexpr int QV = D / 8, PASS = 128 / QV, NQ = kR / PASS / 2;  // vectors of a row, rows at a time
        const int j = lane % QV;
        bool waited = used == 0;
        ++used;
#pragma unroll 1
        for (int n0 = 0; n0 < 2 * C::kRows / kR; ++n0) {  // half a tile at a time
          const int rr = kR / 2 * n0 + (32 * wid + lane) / QV;
          uint4 x[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            const int row = row0 + PASS * n + rr, i = row / P.group;
            x[n] = make_uint4(0u, 0u, 0u, 0u);
            if (PASS * n + rr < rows)
              x[n] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) + (r0 + i) * P.qs +
                                                          static_cast<long long>(head0 + row - i * P.group) * D) + j);
          }
          if (!waited) wait_warp(&S.q_free, used - 2);
          waited = true;
          if (tries <= 0) break;
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if (kR / 2 * n0 + PASS * n >= rows) break;
            const int r = PASS * n + rr;
            unsigned most = largest_finite(x[n]);
#pragma unroll
            for (int d = QV / 2; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d, QV));
            float undo;
            const float up = query_scale(most, P.c, &undo);
            if (j == 0) S.qc[k & 3][r] = undo;
            uint32_t f[4];
            query_f16(x[n], up, f);
            *reinterpret_cast<uint4*>(sq + (r >> 7) * C::kTile + (j >> 3) * C::kSlab + (r & 127) * 128 +
                                      (((j & 7) ^ (r & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
          }
        }
        if (tries <= 0) break;
        fence_async_shared();
      }
      arrive_warp(&S.q_full[k & 3]);

      const int places = 2 * units;
      // Which tile comes at a place: of unit *u, keys or values
      auto tile_at = [&](int p, int* u) {
        if (PAIR) {
          *u = p >> 1;
          return (p & 1) != 0;
        }
        const bool values = p == places - 1 || (p >= 2 && !(p & 1));  // keys are a unit ahead
        *u = p == places - 1 ? units - 1 : values ? (p - 2) >> 1 : (p + 1) >> 1;
        return values;
      };
      // What codes of values are multiplied with, of the last unit whose heads were read and of the one before
      uint32_t now_by0 = 0, now_by1 = 0, old_by0 = 0, old_by1 = 0;
      int heads_at = -1, loud = -128;  // the largest exponent of values of the item's units
      for (int p = 0; p < places; ++p) {
        int u;
        const bool values = tile_at(p, &u);
        const uint32_t pos = pos0 + p, st = pos % C::kStages, raw = pos % C::kRaws;
        const uint32_t dst = (values ? value_to : key_to) + st * C::kTile;
        const uint32_t src = (values ? value_from : key_from) + raw * C::kRaw;
        wait_warp(&S.raw_full[raw], pos / C::kRaws);
        if (tries <= 0) break;
        const uint2 gone = S.absent[(unit0 + u) & 15];
        uint4 c[N];
        each(Upto<N>(), [&](auto n_) {
          constexpr int n = n_;
          c[n] = ld_shared_v4<n * 512>(D == 128 && (n & 1) && values ? src ^ 64u : src);
        });
        uint32_t by0 = u == heads_at ? now_by0 : old_by0, by1 = u == heads_at ? now_by1 : old_by1;
        if (!values) {
          // Heads: what the unit's codes are multiplied with, so that they have one exponent, if that is exact
          uint2 head = *reinterpret_cast<const uint2*>(raws + raw * C::kRaw + 8 * 16 * D + 16 * (lane & 7));
          const bool lost = (gone.x >> (lane & 7)) & 1u, there = !lost && !((gone.y >> (lane & 7)) & 1u);
          if (!there) head = make_uint2(0u, lost ? 0xFFFFu : 0u);  // without a page: marked keys
          const int ek = min(max(static_cast<int>(static_cast<signed char>(head.x & 0xFFu)), kKv8Low), kKv8High);
          const int ev = min(max(static_cast<int>(static_cast<signed char>((head.x >> 8) & 0xFFu)), kKv8Low), kKv8High);
          const int most_k = __reduce_max_sync(0xFFFFFFFFu, there ? ek : kKv8Low);
          const int most_v = __reduce_max_sync(0xFFFFFFFFu, there ? ev : kKv8Low);
          loud = max(loud, most_v);
          const bool uneven = __any_sync(0xFFFFFFFFu, there && (most_k - ek > kEvenKeys || most_v - ev > kEvenValues)) ||
                              most_v < loud - static_cast<int>(kQuiet);
          const uint32_t marked = __any_sync(0xFFFFFFFFu, head.y != 0) ? kMarked : 0u;
          // 2^(e - the largest) twice, in float16
          const uint32_t by_k = uneven || !there ? 0x3C003C00u : static_cast<uint32_t>(15 + ek - most_k) * 0x04000400u;
          const uint32_t by_v = uneven || !there ? 0x3C003C00u : static_cast<uint32_t>(15 + ev - most_v) * 0x04000400u;
          by0 = __shfl_sync(0xFFFFFFFFu, by_k, 2 * wid);
          by1 = __shfl_sync(0xFFFFFFFFu, by_k, 2 * wid + 1);
          old_by0 = now_by0;
          old_by1 = now_by1;
          now_by0 = __shfl_sync(0xFFFFFFFFu, by_v, 2 * wid);
          now_by1 = __shfl_sync(0xFFFFFFFFu, by_v, 2 * wid + 1);
          heads_at = u;
          auto two = [](int e) { return __int_as_float((e + 127) << 23); };
          if (wid == 0 && lane < 8)
            S.heads[(unit0 + u) & 7][lane] = make_float4(two(ek), static_cast<float>(ev), __uint_as_float(head.y), 0.f);
          if (wid == 0 && lane == 8)
            *const_cast<volatile uint32_t*>(&S.unit[(unit0 + u) & 7]) =
                static_cast<uint32_t>(most_k + 64) | static_cast<uint32_t>(most_v + 64) << 8 | marked |
                (uneven ? kUneven : 0u) | (unit0 + u) << 18;
        }
        const uint32_t none = ((gone.x | gone.y) >> (2 * wid)) & 3u;
        if (none) {
          each(Upto<N>(), [&](auto n_) {
            constexpr int n = n_;
            if ((none >> (n / (N / 2))) & 1u) c[n] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
          });
        }
        const uint32_t less0 = mul_f16x2(by0, 0xE480E480u), less1 = mul_f16x2(by1, 0xE480E480u);  // times -1152
        if (pos >= C::kStages) wait_warp(&S.empty[st], pos / C::kStages - 1);
        if (tries <= 0) break;
        if (!values) {
          each(Upto<N>(), [&](auto n_) {
            constexpr int n = n_;
            const uint32_t to = D == 128 && (n & 1) ? dst ^ 64u : dst;
            constexpr int off = n * (D == 128 ? 512 : 1024);
            const uint32_t by = n < N / 2 ? by0 : by1, less = n < N / 2 ? less0 : less1;
            st_shared_v4<off>(to, code_pair<0x4140>(c[n].x, by, less), code_pair<0x4342>(c[n].x, by, less),
                              code_pair<0x4140>(c[n].y, by, less), code_pair<0x4342>(c[n].y, by, less));
            st_shared_v4<off>(to ^ 16u, code_pair<0x4140>(c[n].z, by, less), code_pair<0x4342>(c[n].z, by, less),
                              code_pair<0x4140>(c[n].w, by, less), code_pair<0x4342>(c[n].w, by, less));
          });
        } else {
          each(Upto<N>(), [&](auto n_) {
            constexpr int n = n_;
            const uint32_t to = D == 128 && (n & 1) ? dst ^ 64u : dst;
            constexpr int off = n * (D == 128 ? 512 : 1024);
            const uint32_t by = n < N / 2 ? by0 : by1, less = n < N / 2 ? less0 : less1;
            st_shared_v4<off>(to, code_pair<0x4240>(c[n].x, by, less), code_pair<0x4240>(c[n].y, by, less),
                              code_pair<0x4240>(c[n].z, by, less), code_pair<0x4240>(c[n].w, by, less));
            st_shared_v4<off + 128>(to ^ 16u, code_pair<0x4341>(c[n].x, by, less), code_pair<0x4341>(c[n].y, by, less),
                                    code_pair<0x4341>(c[n].z, by, less), code_pair<0x4341>(c[n].w, by, less));
          });
        }
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
    fewer_registers<64>();
    if (warp == kWarpMma) {
      // ---- products: one elected thread does it all (see sv_prompt.cu)
      constexpr uint32_t kScores = (1u << 4) | (16u << 17) | (8u << 24);  // float16 operands, float32 sums
      constexpr uint32_t kOutputs = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17) | (8u << 24);
      if (elect_one()) {
        const uint32_t a_q = operand_lo(smem_u32(sq), 16), a_key = operand_lo(smem_u32(ring), 16);
        const uint32_t a_val = operand_lo(smem_u32(ring), C::kSlab);
        uint32_t pos = 0, items = 0, weights[2] = {0, 0};  // items: with units
        for (int k = 0;; ++k) {
          wait(&S.item_full[k & 3], k >> 2);
          const int units = S.items[k & 3].end - S.items[k & 3].unit, last = S.items[k & 3].last;
          const int streams = PAIR && S.items[k & 3].rows <= kR ? 1 : 2;
          mbar_arrive(&S.item_free[k & 3]);
          if (tries <= 0) break;
          if (units > 0) wait(&S.q_full[k & 3], k >> 2);
          auto full = [&](uint32_t p) {
            wait(&S.full[p % C::kStages], p / C::kStages);
            tc_fence_after();
          };
          auto scores = [&](auto g_, uint32_t p) {  // of stream g, keys at place p
            constexpr int g = g_;
            const uint32_t q = a_q + (PAIR ? g * (C::kTile >> 4) : 0), key = a_key + p % C::kStages * (C::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::kSlab + 32 * (kk & 3)) >> 4;
              mma_ss(tmem + 128 * g, q + off, key + off, kScores, kk > 0);
            }
            tc_commit(&S.s_full[g]);
          };
          auto outputs = [&](auto g_, uint32_t p, bool first) {
            constexpr int g = g_;
            wait(&S.p_full[g], weights[g]++);
            if (tries <= 0) return;
            tc_fence_after();
            const uint32_t val = a_val + p % C::kStages * (C::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + kColO + D * g, tmem + 128 * g + 8 * kk, val + ((2048 * kk) >> 4), kOutputs, !first || kk > 0);
          };
          const std::integral_constant<int, 0> s0;
          const std::integral_constant<int, 1> s1;
          if constexpr (PAIR) {
            // scores of the next unit behind the outputs of this one, stream by stream
            if (units > 0) {
              full(pos);
              if (tries <= 0) break;
              scores(s0, pos);
              if (streams > 1) scores(s1, pos);
              tc_commit(&S.empty[pos % C::kStages]);
              if (units == 1) tc_commit(&S.q_free);
            }
            for (int u = 0; u < units; ++u) {
              const uint32_t values = pos + 2 * u + 1, keys = values + 1;
              const bool more = u + 1 < units;
              full(values);
              outputs(s0, values, u == 0);
              if (tries <= 0) break;
              if (more) full(keys); else tc_commit(&S.o_done[0]);
              if (tries <= 0) break;
              if (more) scores(s0, keys);
              if (streams > 1) {
                outputs(s1, values, u == 0);
                if (tries <= 0) break;
                tc_commit(&S.empty[values % C::kStages]);
                if (more) scores(s1, keys); else tc_commit(&S.o_done[1]);
              } else {
                tc_commit(&S.empty[values % C::kStages]);
              }
              if (more) tc_commit(&S.empty[keys % C::kStages]);
              if (u + 2 == units) tc_commit(&S.q_free);
            }
            pos += 2 * units;
          } else {
            auto step = [&](int u, auto g_, auto e_) {  // scores of unit u, outputs of the one before
              if (u < units) {
                full(pos);
                if (tries <= 0) return;
                scores(g_, pos);
                tc_commit(&S.empty[pos++ % C::kStages]);
                if (u == units - 1) tc_commit(&S.q_free);
              }
              if (u > 0) {
                full(pos);
                if (u == 1 && items > 0) wait(&S.o_free, items - 1);
                outputs(e_, pos, u <= 2);
                if (tries <= 0) return;
                tc_commit(&S.empty[pos++ % C::kStages]);
                if (u >= units - 1) tc_commit(&S.o_done[e_]);
              }
            };
            for (int u = 0; u <= units && tries > 0 && units > 0; u += 2) {
              step(u, s0, s1);
              if (u + 1 <= units && tries > 0) step(u + 1, s1, s0);
            }
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
        auto inside = [&](int u) { return u + mine < units && 16 * (8 * (unit + u + mine) + block) < len; };
        auto look_up = [&](int u) {  // nothing is done with it before the next round
          int page = 0;
          if (inside(u)) page = __ldg(table + ((8 * (unit + u + mine) + block) >> bpp_log));
          return page;
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
        const int lag = PAIR ? 0 : 1;  // units that values are behind keys
        for (int u = 0; u < units + lag && tries > 0; ++u) {
          if (u < units) {
            if ((u & 3) == 0) {
              const bool in = inside(u), there = in && page >= 0 && page < P.num_pages;
              const int blk = 8 * (unit + u + mine) + block;
              const uint32_t lost = __ballot_sync(0xFFFFFFFFu, in && !there), none = __ballot_sync(0xFFFFFFFFu, !in);
              S.off[(unit0 + u + mine) & 15][block] =
                  there ? ((((static_cast<long long>(page) * P.hkv) + h) << bpp_log) + (blk & ((1 << bpp_log) - 1))) *
                              B::kBytes
                        : -1;
              if (block == 0)
                S.absent[(unit0 + u + mine) & 15] = make_uint2((lost >> (8 * mine)) & 0xFFu, (none >> (8 * mine)) & 0xFFu);
              page = look_up(u + 4);
              __syncwarp();
            }
            copy(u, false);
          }
          if (u >= lag && tries > 0) copy(u - lag, true);
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
        it.rows = min(C::kRows, w.n * P.group - w.rt * C::kRows);
        const int i0 = w.rt * C::kRows / P.group, i1 = (w.rt * C::kRows + it.rows - 1) / P.group;
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
        next_item<W>(P, w);
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

template <int D, bool PAIR>
cudaError_t launch_dim8_tc(const AttnParams& P, int sms, cudaStream_t stream) {
  using C = Shape8<D, PAIR>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn8_tc_kernel<D, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn8_tc_kernel<D, PAIR><<<sms, kThreads, C::kSmem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention8_tc(const AttnParams& params, int D, long long rows, int sms, cudaStream_t stream) {
  AttnParams P = params;
  if (P.c == 0.f) P.c = 0.f;  // without a sign, which would be that of the scores
  // Measured in us with pairs / without. 8 sequences of 16384 tokens, 8 heads of 128: 160 rows 141 / 194, 256 rows
  // 161 / 196; 6000 rows of two 660 / 980; 2 heads of 64: 160 rows 54 / 60, 12000 rows 295 / 462. Against it:
  // 256 rows of two sequences of 32768 tokens 137 / 121, whose pieces of twice the rows take longer to join.
  const bool pair = rows > kR;
  if (D == 64) return pair ? launch_dim8_tc<64, true>(P, sms, stream) : launch_dim8_tc<64, false>(P, sms, stream);
  return pair ? launch_dim8_tc<128, true>(P, sms, stream) : launch_dim8_tc<128, false>(P, sms, stream);
}

}  // namespace sv
