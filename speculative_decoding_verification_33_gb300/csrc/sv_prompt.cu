// Causal attention over whole prompts, packed (spec_prompt_attention), on the fifth-generation tensor cores.
//
// A CTA takes two tiles of up to 128 rows (tokens x query heads of one key/value head, so that grouped heads
// share what is loaded) and goes over the keys and values that they see, 128 tokens at a time:
//   scores [128 rows x 128 tokens] = q [shared memory] k^T [shared memory]
//   outputs [128 rows x D] += weights [tensor memory] v [shared memory]
// with scores and outputs of both tiles in tensor memory. While the tensor cores work for one tile, the
// softmax of the other runs: a thread a row, one pass with the running maximum and sum; the weights go back
// over the scores as bfloat16, since the operands of a product have one type and the values are that. A row's
// maximum is moved only when a score exceeds it by 2^8, and only then are outputs read back and scaled, by the
// row's own threads: the products before have ended by then, since the next scores were issued behind them.
//
// One persistent CTA an SM, its warps specialised: eight take scores to weights, four take outputs to memory,
// one issues products, one copies (TMA), one looks after values that no row may see, one fetches items. Values that
// are not finite cost their items some microseconds, wherever they are and however many. Items
// come from a counter, in the order of their cost where that can be had, so that the last ones are short, and
// two at a time: with four, CTAs held items that others had time for (24 prompts of up to 1000 tokens, 28 + 4
// heads: 55 -> 52 us; 12 + 12 heads of 64: 119 -> 101).
//
// What bounds it, on long prompts: the tensor cores, at 0.68 of their cycles and 0.81 of the measured bf16 rate
// (8191 tokens, 32 + 8 heads of 128: 351 us, 1566 TFLOP/s by what rows see; 16384 tokens: 1320, 1666), held up by the
// softmax's way from scores to weights, a latency: 0.38 of the issue slots are used. On short prompts: the
// changes from item to item, about 5 us for each of 128 rows twice, most of it waits for memory. Tiles of 64
// tokens with scores twice in tensor memory (long prompts 370 -> 516 us: such products read their queries
// twice as often), the next item's first scores behind this one's last products (registers spilled: 350 ->
// 390), and, for heads of 64, weights in columns of their own (no change) were built and not kept.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "sv_attn.cuh"
#include "sv_kv.h"
#include "sv_ptx.cuh"
#include "sv_tc.cuh"
#include "sv_tc_attn.cuh"

namespace sv {
namespace {

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// ------------------------------------------------------------------------------------------
// the kernel
// ------------------------------------------------------------------------------------------
constexpr int kWarpOut = 8, kWarpMma = 12, kWarpCopy = 13, kWarpValues = 14;  // and items
constexpr int kPromptThreads = 512;
constexpr int kSeqs = 1024, kLevels = 1024;  // sequences and tiles of one that items are ordered for

template <int D>
struct PromptShape {
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;       // bytes of 128 rows of 64 values
  static constexpr int kTile = kSlabs * kSlab;  // of queries, keys or values
  static constexpr int kStages = 8 / kSlabs;    // of keys and values in turn: an even number
  static constexpr int kSmem = 1024 + (2 + kStages) * kTile;
};

// Two tiles of rows, a and b: tokens from `tok` of the sequence that starts at row r0; those of tile b follow.
struct PromptItem {
  int r0, n, head;  // sequence: first row, length; key/value head
  int tok, last;    // first and last token of the item
  int tiles[2];     // of keys, that a tile sees; 0: it has no rows
  int half[2];      // its rows see the first half alone of the last of these
  int near;         // the first tile of keys with tokens behind `tok`
  int end;          // no item: the last one
};

struct PromptShared {
  uint64_t full[8], empty[8];                // keys and values
  uint64_t q_full[2], q_free[2];             // queries of a tile
  uint64_t s_full[2], p_full[2];             // scores; weights
  uint64_t o_done[2], o_free[2];             // outputs of an item; read
  uint64_t stat[2][2];                       // sums and maxima of a tile; tiles in turn use two
  uint64_t item_full[2], item_free[2];
  uint64_t fit[4];                           // values at an odd place of the ring are fit for products
  uint64_t noted[2];                         // an item's values that are not finite
  uint64_t end;
  PromptItem items[2];
  float sum[2][2][128], top[2][2][128];
  int bad[2];                                // some value behind the item's first token is not finite:
  int first[2][3][128];                      // the first such token of each dimension: NaN, infinity, -infinity
  uint32_t tmem;
  int levels, total;
  int count[kLevels + 1], more[kLevels + 1], start[kLevels + 1], order[kSeqs];
};

// Values that are not finite, of tokens that some of an item's rows do not see (a weight of 0 would not keep
// them out of a product): cleared for the products, and the first token of each kind in each dimension is
// noted, for the rows that see it. `tile`: 128 tokens, of which from .. to - 1 are looked at; the first is token
// t0, with its key at k. Where a key is not finite either, its weights are NaN or 0 and the values count as
// NaN. A warp, eight lanes a token.
template <int D>
__device__ __forceinline__ void note_values(unsigned char* tile, int t0, int from, int to, const __nv_bfloat16* k,
                                            long long stride, int (*first)[128]) {
  const int lane = threadIdx.x & 31;
  auto finite = [](uint32_t x) { return (x & 0x7F80u) != 0x7F80u; };
  auto half = [](const uint4& w, int i) { return ((&w.x)[i >> 1] >> (16 * (i & 1))) & 0xFFFFu; };
#pragma unroll 1
  for (int r0 = from; r0 < to; r0 += 4) {
    const int r = r0 + (lane >> 3);
    bool fine = true;  // its key
#pragma unroll 1
    for (int s = 0; s < D / 64; ++s) {
      if (r >= to) continue;
      const uint4 w = *reinterpret_cast<const uint4*>(k + r * stride + 64 * s + 8 * (lane & 7));
#pragma unroll
      for (int i = 0; i < 8; ++i) fine = fine && finite(half(w, i));
    }
    fine = ((__ballot_sync(0xFFFFFFFFu, fine) >> (lane & 24)) & 0xFFu) == 0xFFu;
#pragma unroll 1
    for (int s = 0; s < D / 64; ++s) {
      if (r >= to) continue;
      uint4* at = reinterpret_cast<uint4*>(tile + s * 128 * 128 + 128 * r + 16 * (lane & 7));
      const int d = 64 * s + 8 * ((lane & 7) ^ (r & 7));  // the 128-byte swizzle
      uint4 w = *at;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = half(w, i);
        if (finite(x)) continue;
        atomicMin(&first[x & 0x7Fu || !fine ? 0 : x >> 15 ? 2 : 1][d + i], t0 + r);
        (&w.x)[i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
      }
      *at = w;
    }
  }
}
// ... and added to what the products gave the row of this token: a weight of finite scores is more than 0, so that
// the result is the same infinity, or NaN.
template <int D>
__device__ __forceinline__ void add_noted(__nv_bfloat16* out, int token, const int (*first)[128]) {
#pragma unroll 1
  for (int d = 0; d < D; ++d) {
    const bool nan = token >= first[0][d], up = token >= first[1][d], down = token >= first[2][d];
    if (!nan && !up && !down) continue;
    float x = __bfloat162float(out[d]);
    if (up) x += INFINITY;
    if (down) x -= INFINITY;
    out[d] = __float2bfloat16_rn(nan ? NAN : x);
  }
}

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const __grid_constant__ PromptParams P) {
  using C = PromptShape<D>;
  extern __shared__ unsigned char dsm[];
  __shared__ __align__(16) PromptShared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* sq = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);
  unsigned char* ring = sq + 2 * C::kTile;
  const int per = 128 / P.group;  // tokens of a tile

  auto sequence = [&](int b, int& first, int& n) {
    first = min(max(P.cu[b], 0), P.T);
    n = min(max(P.cu[b + 1], first), P.T) - first;
  };
  auto tiles_of = [&](int b) {
    int first, n;
    sequence(b, first, n);
    return (n + 2 * per - 1) / (2 * per);
  };

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1 + (i & 1));  // values: read by the warp that looks after them, too
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_free[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 4);
      mbar_init(&S.o_done[i], 1);
      mbar_init(&S.o_free[i], 4);
      mbar_init(&S.stat[i][0], 4);
      mbar_init(&S.stat[i][1], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.noted[i], 1);
      mbar_init(&S.item_full[i], 1);
      mbar_init(&S.item_free[i], 15);
      S.items[i] = PromptItem{};
      S.items[i].end = 1;  // what a role reads that gave up waiting
    }
    for (int i = 0; i < C::kStages / 2; ++i) mbar_init(&S.fit[i], 1);
    mbar_init(&S.end, 1);
    fence_mbar_init();
    S.levels = 0;
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == kWarpMma) tmem_alloc(&S.tmem, 512);
  for (int i = tid; i <= kLevels; i += kPromptThreads) S.count[i] = 0;
  __syncthreads();

  // ---- Items by cost: the tiles with most keys of all sequences first. Level t has the tile t of each
  // sequence that has more than t of them; with the sequences in the order of their tiles, these are the
  // first more[t], and start[t] is what levels above hold.
  if (P.B <= kSeqs) {
    for (int b = tid; b < P.B; b += kPromptThreads) {
      const int t = tiles_of(b);
      if (t > 0) atomicMax(&S.levels, t);
      if (t > 0 && t <= kLevels) atomicAdd(&S.count[t], 1);
    }
    __syncthreads();
    const int levels = S.levels;
    if (levels <= kLevels && warp == 0) {
      int seqs = 0, items = 0;  // with more tiles than the levels that are left
      if (lane == 0) S.more[levels] = 0;
      for (int t0 = levels - 1; t0 >= 0; t0 -= 32) {
        const int t = t0 - lane;
        int m = t >= 0 ? S.count[t + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int x = __shfl_up_sync(0xFFFFFFFFu, m, d);
          if (lane >= d) m += x;
        }
        m = t >= 0 ? m + seqs : 0;
        int i = m;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int x = __shfl_up_sync(0xFFFFFFFFu, i, d);
          if (lane >= d) i += x;
        }
        if (t >= 0) {
          S.more[t] = m;
          S.start[t] = items + i - m;
        }
        seqs = __shfl_sync(0xFFFFFFFFu, m, min(31, t0));
        items += __shfl_sync(0xFFFFFFFFu, i, 31);
      }
      if (lane == 0) S.total = items;
      __syncwarp();
      for (int t = lane; t <= levels; t += 32) S.count[t] = S.more[t];  // where the next of t tiles goes
      __syncwarp();
      for (int b0 = 0; b0 < P.B; b0 += 32) {
        const int b = b0 + lane, t = b < P.B ? tiles_of(b) : 0;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, t);
        const int at = S.count[t] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (t > 0) {
          S.order[at] = b;
          if ((same >> lane) == 1u) S.count[t] = at + 1;  // the last of them
        }
        __syncwarp();
      }
    }
  }
  const bool ordered = P.B <= kSeqs && S.levels <= kLevels;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  constexpr uint32_t kColO = 256;  // scores of the tiles at columns 0 and 128, outputs from here

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
  // The k-th item, or false at the end. `done` hands its place back.
  auto item = [&](int k, PromptItem& it) {
    wait_warp(&S.item_full[k & 1], k >> 1);
    it = S.items[k & 1];
    arrive_warp(&S.item_free[k & 1]);
    return tries > 0 && !it.end;
  };

  if (warp < kWarpOut) {
    // ---- scores to weights: a thread a row
    more_registers<184>();
    const int g = warp >> 2, row = tid & 127, i = row / P.group;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t cols = tmem + lanes + 128 * g, outs = tmem + lanes + kColO + D * g;
    const float c = P.c, fill = c < 0.f ? INFINITY : -INFINITY;
    int phase = 0, use = 0;
    PromptItem it;
    for (int k = 0; item(k, it); ++k) {
      const int first = it.tok + g * per, sees = min(first + i, it.last) + 1;
      const int tiles = g ? it.tiles[1] : it.tiles[0], half = g ? it.half[1] : it.half[0];
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int j = 0; j < tiles && tries > 0; ++j, ++phase) {
        wait_warp(&S.s_full[g], phase);
        tc_fence_after();
        uint32_t r[128];
        tmem_ld64(cols, r);
        tmem_ld64(cols + 64, r + 64);
        tmem_wait_ld(r);
        tmem_wait_ld(r + 64);
        if (128 * j + 127 > first) {  // some row does not see some of these
          const int lim = sees - 128 * j;
#pragma unroll
          for (int n = 0; n < 128; ++n)
            if (n >= lim) r[n] = __float_as_uint(fill);
        }
        float t;
        if (c < 0.f) {
          float x[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
          for (int n = 0; n < 128; n += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = min3(x[e], __uint_as_float(r[n + 2 * e]), __uint_as_float(r[n + 2 * e + 1]));
          t = fminf(fminf(x[0], x[1]), fminf(x[2], x[3])) * c;
        } else {
          float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int n = 0; n < 128; n += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = max3(x[e], __uint_as_float(r[n + 2 * e]), __uint_as_float(r[n + 2 * e + 1]));
          t = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * c;
        }
        if (j == 0) {
          m = t;
        } else {
          const bool move = t > m + 8.f;
          if (__any_sync(0xFFFFFFFFu, move)) {
            // the products before these scores are done: nobody else is at the outputs
            const float down = move ? ex2_fast(m - t) : 1.f;
            if (move) m = t;
            l2.x *= down;
            l2.y *= down;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              float o[32];
              uint32_t w[32];
              tmem_ld32(outs + d, o);
#pragma unroll
              for (int n = 0; n < 32; ++n) w[n] = __float_as_uint(o[n] * down);
              tmem_st32(outs + d, w);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : -m;
        const float2 c2 = make_float2(c, c), b2 = make_float2(base, base);
        const bool far = fabsf(base) > 1048576.f;
        auto weights = [&](auto rounded) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              float2 p = make_float2(__uint_as_float(r[64 * h + 2 * n]), __uint_as_float(r[64 * h + 2 * n + 1]));
              if constexpr (rounded)
                p = far ? make_float2(__fadd_rn(__fmul_rn(p.x, c), base), __fadd_rn(__fmul_rn(p.y, c), base))
                        : fma2(p, c2, b2);
              else
                p = fma2(p, c2, b2);
              p.x = ex2_fast(p.x);
              p.y = ex2_fast(p.y);
              l2 = add2(l2, p);
              w[n] = pack_bf16(p.x, p.y);
            }
            tmem_st32(cols + 32 * h, w);
            if (half && j + 1 == tiles) break;
          }
        };
        // Far from 0 the score that was rounded for the maximum is not the one that a fused operation has here
        if (__any_sync(0xFFFFFFFFu, far))
          weights(std::true_type());
        else
          weights(std::false_type());
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&S.p_full[g]);
      }
      if (tiles) {
        S.sum[use & 1][g][row] = l2.x + l2.y;
        S.top[use & 1][g][row] = m;
        arrive_warp(&S.stat[use & 1][g]);
        ++use;
      }
    }
  } else if (warp < kWarpMma) {
    // ---- outputs to memory: a thread a row
    fewer_registers<72>();
    const int row = tid & 127, i = row / P.group;
    const uint32_t outs = tmem + (static_cast<uint32_t>(warp & 3) << 21) + kColO;
    const bool wide = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;  // whole sectors
    int use[2] = {0, 0};
    auto row_of = [&](const PromptItem& it, int tok) {
      return static_cast<long long>(it.r0 + tok) * P.hq + it.head * P.group + row - i * P.group;
    };
    for (int k = 0;; ++k) {
      wait_warp(&S.item_full[k & 1], k >> 1);
      const PromptItem it = S.items[k & 1];
      if (tries <= 0 || it.end) break;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!it.tiles[g]) continue;
        const int u = use[g]++;
        wait_warp(&S.stat[u & 1][g], u >> 1);
        wait_warp(&S.o_done[g], u);
        if (tries <= 0) break;
        tc_fence_after();
        const float l = S.sum[u & 1][g][row], m = S.top[u & 1][g][row];
        const float inv = 1.f / l;
        const int tok = it.tok + g * per + i;
        const bool there = i < per && tok <= it.last;
        const long long at = row_of(it, tok);
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(P.out) + at * D;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          float o[32];
          tmem_ld32(outs + D * g + d, o);
          if (d + 32 == D) {
            tc_fence_before();
            arrive_warp(&S.o_free[g]);
          }
          uint32_t w[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) w[n] = pack_bf16(o[2 * n] * inv, o[2 * n + 1] * inv);
          if (there) {
            if (wide) {
#pragma unroll
              for (int n = 0; n < 16; n += 8)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + d + 2 * n), "r"(w[n]),
                             "r"(w[n + 1]), "r"(w[n + 2]), "r"(w[n + 3]), "r"(w[n + 4]), "r"(w[n + 5]), "r"(w[n + 6]),
                             "r"(w[n + 7])
                             : "memory");
            } else {
#pragma unroll
              for (int n = 0; n < 16; n += 4)
                *reinterpret_cast<uint4*>(to + d + 2 * n) = make_uint4(w[n], w[n + 1], w[n + 2], w[n + 3]);
            }
          }
        }
        if (there && P.lse) P.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
      }
      wait_warp(&S.noted[k & 1], k >> 1);
      if (tries <= 0) break;
      if (S.bad[k & 1] && i < per)
        for (int g = 0; g < 2; ++g) {
          const int tok = it.tok + g * per + i;
          if (tok <= it.last)
            add_noted<D>(static_cast<__nv_bfloat16*>(P.out) + row_of(it, tok) * D, tok, S.first[k & 1]);
        }
      arrive_warp(&S.item_free[k & 1]);  // and the places of that number elsewhere
    }
  } else {
    fewer_registers<72>();
    if (warp == kWarpMma) {
      // ---- products: one elected thread does it all. It is held up until nearly all products that it has
      // issued are done, so that what it does between them leaves the tensor cores idle: waits that are over
      // by then come first.
      constexpr uint32_t kScores = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
      constexpr uint32_t kOutputs = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                    (static_cast<uint32_t>(D / 8) << 17) | (8u << 24);
      if (elect_one()) {
        const uint32_t a_q = operand_lo(smem_u32(sq), 16), a_ring = operand_lo(smem_u32(ring), 16);
        const uint32_t a_val = operand_lo(smem_u32(ring), C::kSlab);
        uint32_t pos = 0, use[2] = {0, 0}, weights[2] = {0, 0};
        auto scores = [&](int g, uint32_t p, bool last) {  // of the keys at place p of the ring
          const uint32_t q = a_q + g * (C::kTile >> 4), k = a_ring + (p % C::kStages) * (C::kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kSlab + 32 * (kk & 3)) >> 4;
            mma_ss(tmem + 128 * g, q + off, k + off, kScores, kk > 0);
          }
          tc_commit(&S.s_full[g]);
          if (last) tc_commit(&S.q_free[g]);
        };
        auto wait_full = [&](uint32_t p) { wait(&S.full[p % C::kStages], p / C::kStages); };
        for (int k = 0;; ++k) {
          wait(&S.item_full[k & 1], k >> 1);
          const int tiles[2] = {S.items[k & 1].tiles[0], S.items[k & 1].tiles[1]}, end = S.items[k & 1].end;
          const int half[2] = {S.items[k & 1].half[0], S.items[k & 1].half[1]};
          mbar_arrive(&S.item_free[k & 1]);
          if (end || tries <= 0) break;
          const int most = max(tiles[0], tiles[1]);
          wait_full(pos);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (!tiles[g]) continue;
            wait(&S.q_full[g], use[g]);
            if (tries <= 0) break;
            tc_fence_after();
            scores(g, pos, tiles[g] == 1);
          }
          if (tries <= 0) break;
          tc_commit(&S.empty[pos % C::kStages]);
          for (int j = 0; j < most; ++j) {
            const uint32_t values = pos + 2 * j + 1, keys = values + 1;
            // Values come by way of the warp that looks after them, always: a barrier that is not waited for in
            // each of its phases can be one behind, and seem to be done
            if (j + 1 < most) wait_full(keys);
            wait(&S.fit[values % C::kStages / 2], values / C::kStages);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (j >= tiles[g]) continue;
              if (j == 0 && use[g] > 0) wait(&S.o_free[g], use[g] - 1);
              wait(&S.p_full[g], weights[g]++);
              if (tries <= 0) break;
              tc_fence_after();
              const uint32_t v = a_val + (values % C::kStages) * (C::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                if (kk < 4 || j + 1 < tiles[g] || !half[g])
                  mma_ts(tmem + kColO + D * g, tmem + 128 * g + 8 * kk, v + ((2048 * kk) >> 4), kOutputs, j > 0 || kk > 0);
              if (j + 1 < tiles[g])
                scores(g, keys, j + 2 == tiles[g]);
              else
                tc_commit(&S.o_done[g]);
            }
            if (tries <= 0) break;
            tc_commit(&S.empty[values % C::kStages]);
            if (j + 1 < most) tc_commit(&S.empty[keys % C::kStages]);
          }
          if (tries <= 0) break;
          pos += 2 * most;
          use[0] += tiles[0] > 0;
          use[1] += tiles[1] > 0;
        }
        // all products are done before the memory goes
        tc_commit(&S.end);
        if (!mbar_wait_bounded(&S.end, 0, kWaitCycles)) tries = 0;
      }
      __syncwarp();
    } else if (warp == kWarpCopy) {
      // ---- copies
      int pos = 0, use[2] = {0, 0};
      PromptItem it;
      for (int k = 0; item(k, it); ++k) {
        const int most = max(it.tiles[0], it.tiles[1]);
        auto put = [&](const CUtensorMap* map, int z) {
          const int stage = pos % C::kStages;
          if (pos >= C::kStages) wait_warp(&S.empty[stage], pos / C::kStages - 1);
          if (tries <= 0) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&S.full[stage], C::kTile);
            for (int s = 0; s < C::kSlabs; ++s)
              tma_load_3d(ring + stage * C::kTile + s * C::kSlab, map, 64 * s, it.head, z, &S.full[stage]);
          }
          __syncwarp();
          ++pos;
        };
        auto queries = [&](int g) {
          if (!it.tiles[g]) return;
          if (use[g] > 0) wait_warp(&S.q_free[g], use[g] - 1);
          if (tries <= 0) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&S.q_full[g], C::kSlabs * 128 * per * P.group);
            for (int s = 0; s < C::kSlabs; ++s)
              tma_load_3d(sq + g * C::kTile + s * C::kSlab, &mq, 64 * s, it.head * P.group, it.r0 + it.tok + g * per,
                          &S.q_full[g]);
          }
          __syncwarp();
          ++use[g];
        };
        put(&mk, it.r0);
        queries(0);
        queries(1);
        put(&mv, it.r0);
        for (int j = 1; j < most && tries > 0; ++j) {
          put(&mk, it.r0 + 128 * j);
          put(&mv, it.r0 + 128 * j);
        }
      }
      // no copy is in flight when the CTA ends, whoever gave up
      for (int p = max(0, pos - C::kStages); p < pos; ++p)
        if (!mbar_wait_bounded(&S.full[p % C::kStages], (p / C::kStages) & 1, kWaitCycles)) tries = 0;
      for (int g = 0; g < 2; ++g)
        if (use[g] > 0 && !mbar_wait_bounded(&S.q_full[g], (use[g] - 1) & 1, kWaitCycles)) tries = 0;
    } else if (warp == kWarpValues) {
      // ---- values next to the rows' own tokens. Those behind the item's last token, which no row sees, are
      // cleared; of those behind its first one, what is not finite is cleared and noted.
      int pos = 1;
      PromptItem it;
      for (int k = 0; item(k, it); ++k) {
        const int most = max(it.tiles[0], it.tiles[1]);
        bool noted = false;
        for (int j = 0; j < most; ++j, pos += 2) {
          const int stage = pos % C::kStages;
          wait_warp(&S.full[stage], pos / C::kStages);
          if (tries <= 0) break;
          if (j >= it.near) {
            const int from = max(it.tok + 1 - 128 * j, 0), to = min(it.last + 1 - 128 * j, 128);
            bool bad = false;
            unsigned char* tile = ring + stage * C::kTile + 16 * (lane & 7);
#pragma unroll 1
            for (int r0 = (from & ~15) + (lane >> 3); r0 < 128; r0 += 16) {  // 16 rows at a time, all read at once
              uint4 w[4][C::kSlabs];
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int s = 0; s < C::kSlabs; ++s)
                  w[u][s] = *reinterpret_cast<const uint4*>(tile + s * C::kSlab + 128 * (r0 + 4 * u));
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int r = r0 + 4 * u;
                const uint32_t f = 0x7FFF7FFFu;
                uint32_t x = 0;
#pragma unroll
                for (int s = 0; s < C::kSlabs; ++s) {
                  x = __vmaxu2(x, __vmaxu2(__vmaxu2(w[u][s].x & f, w[u][s].y & f), __vmaxu2(w[u][s].z & f, w[u][s].w & f)));
                  if (r >= to) *reinterpret_cast<uint4*>(tile + s * C::kSlab + 128 * r) = make_uint4(0u, 0u, 0u, 0u);
                }
                if (r >= from && r < to && ((x & 0xFFFFu) >= 0x7F80u || (x >> 16) >= 0x7F80u)) bad = true;
              }
            }
            if (__any_sync(0xFFFFFFFFu, bad)) {
              if (!noted)
                for (int i = lane; i < 3 * 128; i += 32) S.first[k & 1][i / 128][i % 128] = INT_MAX;
              noted = true;
              __syncwarp();
              const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(P.k) + (it.r0 + 128LL * j) * P.ks +
                                          static_cast<long long>(it.head) * D;
              note_values<D>(ring + stage * C::kTile, 128 * j, from, to, keys, P.ks, S.first[k & 1]);
            }
            fence_async_shared();
          }
          arrive_warp(&S.fit[stage / 2]);
          if (j == most - 1) {
            if (lane == 0) S.bad[k & 1] = noted;
            arrive_warp(&S.noted[k & 1]);
          }
          arrive_warp(&S.empty[stage]);
        }
        if (tries <= 0) break;
      }
    } else {
      // ---- items: the first one is this CTA's number, the others come from the counter
      int b = 0, before = 0;  // without an order: sequences from b on, tiles of those before
      for (int k = 0;; ++k) {
        if (k >= 2) wait_warp(&S.item_free[k & 1], (k >> 1) - 1);
        if (tries <= 0) break;
        int i = blockIdx.x;
        if (k > 0) {
          if (lane == 0) i = gridDim.x + atomicAdd(&P.queue[0], 1u);
          i = __shfl_sync(0xFFFFFFFFu, i, 0);
        }
        const int u = i / P.hkv;
        int t = -1, seq = 0;  // tile of a sequence
        if (ordered) {
          if (u < S.total) {
            int hi = S.levels - 1;  // the lowest level that starts at u or before; starts grow as levels fall
            t = 0;
            while (t < hi) {
              const int mid = (t + hi) >> 1;
              if (S.start[mid] <= u) hi = mid; else t = mid + 1;
            }
            seq = S.order[u - S.start[t]];
          }
        } else {
          for (; b < P.B; b += 32) {
            const int mine = b + lane < P.B ? tiles_of(b + lane) : 0;
            int all = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const int x = __shfl_up_sync(0xFFFFFFFFu, all, d);
              if (lane >= d) all += x;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + all > u);
            if (past) {
              const int at = __ffs(past) - 1;
              seq = b + at;
              t = before + __shfl_sync(0xFFFFFFFFu, all, at) - 1 - u;  // its last tile first
              break;
            }
            before += __shfl_sync(0xFFFFFFFFu, all, 31);
          }
        }
        if (lane == 0) {
          PromptItem it{};
          it.end = t < 0;
          if (t >= 0) {
            sequence(seq, it.r0, it.n);
            it.head = i - u * P.hkv;
            it.tok = 2 * per * t;
            it.last = min(it.tok + 2 * per, it.n) - 1;
            const int last0 = min(it.tok + per - 1, it.last);
            it.tiles[0] = last0 / 128 + 1;
            it.tiles[1] = last0 < it.last ? it.last / 128 + 1 : 0;
            it.near = (it.tok + 1) / 128;
            it.half[0] = last0 % 128 < 64;
            it.half[1] = it.last % 128 < 64;
          }
          S.items[k & 1] = it;
          mbar_arrive(&S.item_full[k & 1]);
        }
        __syncwarp();
        if (t < 0) break;
      }
      // the last CTA to come here leaves the counter at zero
      if (lane == 0 && atomicAdd(&P.queue[1], 1u) == gridDim.x - 1) {
        P.queue[0] = 0;
        P.queue[1] = 0;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
  if (tries <= 0) atomicOr(P.err, 1u);
}

// A tensor [T][H][D] of bfloat16, read in boxes of 64 values, `heads` heads and `tokens` tokens.
bool make_map3(CUtensorMap* m, const void* p, int T, int H, int D, long long stride, int heads, int tokens) {
  using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::once_flag once;
  static EncodeFn encode = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<EncodeFn>(f);
  });
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_prompt_dim(const PromptParams& P, int sms, cudaStream_t stream) {
  using C = PromptShape<D>;
  const int per = 128 / P.group;
  CUtensorMap mq, mk, mv;
  if (!make_map3(&mq, P.q, P.T, P.hq, D, P.qs, P.group, per) || !make_map3(&mk, P.k, P.T, P.hkv, D, P.ks, 1, 128) ||
      !make_map3(&mv, P.v, P.T, P.hkv, D, P.vs, 1, 128))
    return cudaErrorInvalidValue;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  // no more items than full tiles and one more of each sequence
  const long long items = (P.T / (2LL * per) + std::min(P.B, P.T)) * P.hkv;
  const unsigned ctas = static_cast<unsigned>(std::min<long long>(sms, std::max(1LL, items)));
  prompt_kernel<D><<<ctas, kPromptThreads, C::kSmem, stream>>>(mq, mk, mv, P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& params, int D, int sms, cudaStream_t stream) {
  PromptParams P = params;
  // A scale of 0 is taken as the least one, so that what is not seen stays so: a product, whatever it is, counts
  // as less than 2^-20
  if (P.c == 0.f) P.c = FLT_TRUE_MIN;
  return D == 64 ? launch_prompt_dim<64>(P, sms, stream) : launch_prompt_dim<128>(P, sms, stream);
}

}  // namespace sv
