// The attention kernel of register operands (mma.sync), for the formats of the cache: a format says how
// a block's bytes become operands. sv_attn.cu (4 bits) holds the reasons of its structure.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "sv_attn.cuh"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

// F: the cache's format (Kv4 in sv_attn.cu, Kv8 in sv_attn8.cu).
template <class F, int NT>
struct AttnShape {
  static constexpr int D = F::D;
  static constexpr int kPairs = 4;  // with two CTAs an SM, 128 registers a thread
  static constexpr int kThreads = 64 * kPairs;
  static constexpr int kPerSm = 2;
  static constexpr int kRows = 8 * NT;
  static constexpr int kOwn = F::template kOwn<NT>;  // blocks of a unit for each warp of a pair
  static constexpr int kUnit = 32 * kOwn;  // tokens
  // Work as it is cut
  static constexpr int kDearest = kOwn * F::cost(NT);
  static constexpr int kOver = F::kOver;
  static constexpr int kLeast = F::template kLeast<NT>;
  static __device__ __forceinline__ int weight(int rows) {
    const int tiles = NT == 1 ? 1 : max((rows + 7) >> 3, NT - 1 > 2 ? 2 : NT - 1);
    return kOwn * F::cost(tiles);
  }
  static constexpr int kBlock = F::kBlock;
  static constexpr int kStage = 2 * kOwn * kBlock;
  static constexpr int kStages = F::template kStages<NT>;
  static constexpr int kRing = kPairs * kStages * kStage;
  static constexpr int kQ = NT * (D / 16) * 32 * 8;
  static constexpr int kP = kPairs * 2 * kOwn * NT * 32 * 8;
  static constexpr int kOutStride = D + 4;  // floats of a row of a joining buffer
  static constexpr int kOut = kPairs * 8 * kOutStride * 4;
  // the first joining buffer lies over the queries and weights, which are spent by then
  static constexpr int kShared = kQ + kP > kOut ? kQ + kP : kOut;
  static constexpr int kStat = (kPairs + 2 * kPairs + 2 * kPairs + 2) * kRows * 4;
  static constexpr int kSmem = kRing + kShared + kOut + kStat + kPairs * kStages * 12;
  static constexpr int kPart = kRows * (D + 2);  // floats of one piece's results
  static_assert(2 * (kSmem + 4096 + 1024) <= 228 * 1024, "two CTAs an SM");
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where a pair's producer looks up next.
struct Producer {
  Walk w;
  long long u;
};

template <int N>
using Int = std::integral_constant<int, N>;

template <class F, int NT>
__global__ void __launch_bounds__(AttnShape<F, NT>::kThreads, AttnShape<F, NT>::kPerSm)
    attn_kernel(AttnParams P) {
  using S = AttnShape<F, NT>;
  constexpr int D = F::D;
  constexpr int NP = S::kPairs, NS = S::kStages, R = S::kRows, KS = D / 16, MH = D / 32;
  constexpr int OWN = S::kOwn, NB = 2 * OWN, UNIT = S::kUnit;
  constexpr int QV = D / 8;  // 16-byte vectors of a query row
  constexpr int QPER = (R * QV + S::kThreads - 1) / S::kThreads;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  uint2* sq = reinterpret_cast<uint2*>(smem + S::kRing);            // query operands [NT][KS][lane]
  uint2* sp = reinterpret_cast<uint2*>(smem + S::kRing + S::kQ);    // weights [pair][block][NT][lane]
  float* so[2] = {reinterpret_cast<float*>(smem + S::kRing),        // joining buffers
                  reinterpret_cast<float*>(smem + S::kRing + S::kShared)};
  float* swm = so[1] + S::kOut / 4;               // [pair][R] running maxima
  float* swl = swm + NP * R;                      // [warp][R] sums
  float* sx = swl + 2 * NP * R;                   // [warp][R] maxima of a unit
  int* svis = reinterpret_cast<int*>(sx + 2 * NP * R);  // [R] tokens that a row sees
  float* sqc = reinterpret_cast<float*>(svis + R);      // [R] score of a product of the operands
  uint64_t* bars = reinterpret_cast<uint64_t*>(sqc + R);
  uint32_t* slost = reinterpret_cast<uint32_t*>(bars + NP * NS);  // per stage: blocks not there
  __shared__ longlong2 s_scan[2 * NP];
  __shared__ Run s_run;
  __shared__ Walk s_walk[2];
  __shared__ Producer s_prod[NP];
  __shared__ long long s_queue[NP][32][NB];  // where the blocks of a pair's next units lie
  __shared__ int s_last;
  __shared__ int s_low[NP][2];  // per warp: kQuiet below the largest exponent of values that it has come to in the item

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = warp >> 1, h = warp & 1;
  const int g = lane >> 2, c = lane & 3;
  if (tid < NP * NS) {
    mbar_init(&bars[tid], 1);
    fence_mbar_init();
  }

  if (!find_run<S::kThreads, S>(P, s_scan, &s_run, &s_walk[0])) return;
  if (tid < NP) {
    s_prod[tid].w = s_walk[0];
    s_prod[tid].u = s_run.u0 + tid;
  }
  __syncthreads();

  // ---- the pair's producer, its first warp: copies of its units into the ring. Where the blocks of
  // the next 32 units lie is looked up 32 at a time, a lane a unit, so that a copy waits for no
  // page number.
  unsigned char* my_ring = ring + pair * NS * S::kStage;
  uint64_t* my_bar = bars + pair * NS;
  uint32_t* my_lost = slost + pair * NS;
  long long (*my_queue)[NB] = s_queue[pair];
  int queued = 0;  // units of the queue that are copied
  int issued = 0;  // by this thread
  // Tries that a wait has. Once one has run out, the thread waits no longer and issues no copies.
  int tries = kWaitTries;
  auto look_up = [&]() {
    const int bpp_log = 31 - __clz(P.ps >> 4);  // blocks of a page: a power of two
    const long long u1 = s_run.u1, u = s_prod[pair].u + NP * lane;
    Walk w = s_prod[pair].w;
    long long off[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) off[i] = -1;
    if (u < u1) {
      while (u >= w.base + w.nu) next_item<S>(P, w);
      const int blk = NB * static_cast<int>(u - w.base);
      const int32_t* row = P.table + static_cast<long long>(w.b) * P.max_blocks;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        if (16 * (blk + i) >= w.len) break;
        const int page = row[(blk + i) >> bpp_log];
        if (static_cast<unsigned>(page) < static_cast<unsigned>(P.num_pages))
          off[i] = (((static_cast<long long>(page) * P.hkv + w.h) << bpp_log) +
                    ((blk + i) & ((1 << bpp_log) - 1))) * S::kBlock;
      }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) my_queue[lane][i] = off[i];
    __syncwarp();
    if (lane == 31) {
      s_prod[pair].u = u + NP;
      if (u < u1) s_prod[pair].w = w;
    }
    queued = 0;
    __syncwarp();
  };
  auto issue = [&](int stage) {  // copy the next unit into the stage
    if (queued == 32) look_up();
    if (lane == 0 && tries > 0) {
      ++issued;
      long long off[NB];
      uint32_t lost = 0;
      int n = 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        off[i] = my_queue[queued][i];
        n += off[i] >= 0;
        lost |= (off[i] < 0 ? 1u : 0u) << i;
      }
      my_lost[stage] = lost;
      if (n == 0) {
        mbar_arrive(&my_bar[stage]);
      } else {
        mbar_arrive_expect_tx(&my_bar[stage], n * S::kBlock);
        unsigned char* to = my_ring + stage * S::kStage;
        auto together = [&] { bulk_g2s(to, P.cache + off[0], S::kStage, &my_bar[stage]); };
        auto apart = [&] {
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (off[i] >= 0) bulk_g2s(to + i * S::kBlock, P.cache + off[i], S::kBlock, &my_bar[stage]);
        };
        // one run of bytes, or not; a condition for both sizes costs those of two blocks 2 % (the
        // compiler's schedule of what follows changes)
        if constexpr (NB == 2) {
          if (!lost && off[NB - 1] == off[0] + (NB - 1) * S::kBlock) together(); else apart();
        } else {
          if (!lost && off[1] - off[0] == S::kBlock && off[2] - off[1] == S::kBlock &&
              off[3] - off[2] == S::kBlock) together(); else apart();
        }
      }
    }
    ++queued;
  };
  if (h == 0) {
    look_up();
    for (int i = 0; i < NS; ++i) issue(i);
  }

  // ---- queries
  uint4 raw[QPER];
  auto load_q = [&](const Walk& w) {
    const int rows = min(R, w.n * P.group - w.rt * R);
#pragma unroll
    for (int n = 0; n < QPER; ++n) {
      const int i = tid + n * S::kThreads, r = i / QV;
      raw[n] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int row = w.rt * R + r, tok = row / P.group, hh = w.h * P.group + row % P.group;
        raw[n] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) +
                                                      (w.r0 + tok) * P.qs +
                                                      static_cast<long long>(hh) * D) + i % QV);
      }
    }
  };
  auto store_q = [&](const Walk& w) {
    const int rows = min(R, w.n * P.group - w.rt * R);
#pragma unroll
    for (int n = 0; n < QPER; ++n) {
      const int i = tid + n * S::kThreads, r = i / QV, j = i % QV;
      if (i >= R * QV) break;  // whole warps
      unsigned most = largest_finite(raw[n]);
#pragma unroll
      for (int d = QV / 2; d > 0; d >>= 1)
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d, QV));
      float undo;
      const float up = query_scale(most, P.c, &undo);
      if (j == 0) {
        svis[r] = w.len - w.n + (w.rt * R + min(r, rows - 1)) / P.group + 1;
        sqc[r] = undo;
      }
      uint32_t f[4];
      query_f16(raw[n], up, f);
      // values 8j .. 8j + 7: thread 8j / (D/4) of the row, steps s and s + 1 of the inner dimension
      const int s = 8 * j % (D / 4) / 4;
      uint2* to = sq + ((r >> 3) * KS + s) * 32 + (r & 7) * 4 + 8 * j / (D / 4);
      to[0] = make_uint2(f[0], f[1]);
      to[32] = make_uint2(f[2], f[3]);
    }
  };
  load_q(s_walk[0]);

  // ---- items of the run
  int unit = static_cast<int>(s_run.u0 - s_walk[0].base) + pair;  // next unit of this pair in the item
  int stage = 0, spent = -1;  // stage of that unit; stage of the last one, to be filled again
  uint32_t phase = 0;         // per stage: parity of the next copy
  uint2* my_p = sp + pair * NB * NT * 32;
  for (int item = 0;; item ^= 1) {
    const Walk& w = s_walk[item];
    const int end = static_cast<int>(min(static_cast<long long>(w.nu), s_run.u1 - w.base));
    const int len = w.len;
    const int rows = min(R, w.n * P.group - w.rt * R);  // rows of this tile
    const int tiles = (rows + 7) >> 3;
    store_q(w);
    if (tid < 2 * NP) s_low[0][tid] = kKv8Low;
    if (tid == 0) {
      Walk nw = w;
      next_item<S>(P, nw);
      s_walk[item ^ 1] = nw;
    }
    __syncthreads();
    const int all_see = svis[0];  // tokens that every row of the tile sees

    float O[NT][MH][4], m[NT][2], l[NT][2];
    int low = 0;  // exponents of values from here to kQuiet above need nothing but their weights
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < MH; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[t][j][k] = 0.f;
      m[t][0] = m[t][1] = -FLT_MAX;
      l[t][0] = l[t][1] = 0.f;
    }

    // The pair's units of this item, for TN tiles of rows: no branch on the tile inside
    auto run = [&](auto tn) {
      constexpr int TN = decltype(tn)::value;
      for (; unit < end; unit += NP) {
        const unsigned char* sb = my_ring + stage * S::kStage;
        const int t0 = unit * UNIT;
        {
          const uint32_t bar = smem_u32(&my_bar[stage]), parity = (phase >> stage) & 1u;
          for (int left = tries; !mbar_try(bar, parity);)
            if (--left <= 0) {  // a copy that never came: its rows are not used
              tries = 0;
              break;
            }
          __syncwarp();
        }
        phase ^= 1u << stage;
        const uint32_t lost = my_lost[stage];
        typename F::Head head[OWN];  // of this warp's blocks
        uint32_t marks = 0;
#pragma unroll
        for (int o = 0; o < OWN; ++o) head[o].load(sb + (h * OWN + o) * S::kBlock, (lost >> (h * OWN + o)) & 1u);
        bool masked = t0 + UNIT > all_see || lost;
        if constexpr (F::kHeads) {
          low = s_low[pair][h];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint2 w = F::head(sb + b * S::kBlock);
            marks |= w.y;
            masked = masked || static_cast<unsigned>(F::lift(w) - low) > kQuiet;
          }
        }
        masked = masked || marks;

        // scores of this warp's blocks and the tile's rows
        float s[OWN][TN][4];
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
          typename F::Keys kc;
          kc.load(sb + (h * OWN + o) * S::kBlock, g, c);
#pragma unroll
          for (int t = 0; t < TN; ++t) s[o][t][0] = s[o][t][1] = s[o][t][2] = s[o][t][3] = 0.f;
#pragma unroll
          for (int i = 0; i < KS / F::kSteps; ++i) {
            uint32_t kf[F::kSteps][4];
            kc.operands(i, kf);
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int n = 0; n < F::kSteps; ++n) {
                const uint2 q = sq[(t * KS + F::kSteps * i + n) * 32 + lane];
                mma16816(s[o][t], kf[n][0], kf[n][1], kf[n][2], kf[n][3], q.x, q.y);
              }
          }
        }
        // in base 2, rounded before the maximum is taken, so that the largest weight is exact
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const float2 qc = *reinterpret_cast<const float2*>(sqc + 8 * t + 2 * c);
#pragma unroll
          for (int o = 0; o < OWN; ++o) {
            if constexpr (F::kHeads) {
              const float2 f = head[o].key_scale(qc);
              const float e = head[o].lift;
#pragma unroll
              for (int k = 0; k < 4; ++k) s[o][t][k] = __fmaf_rn(s[o][t][k], k & 1 ? f.y : f.x, e);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) s[o][t][k] = __fmul_rn(s[o][t][k], k & 1 ? qc.y : qc.x);
            }
          }
        }
        // Tokens of a block whose weights may be none, into the sums
        auto add_quiet = [&](int o) {
          if constexpr (F::kHeads) {
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int k = 0; k < 4; ++k) l[t][k & 1] += ex2_fast(s[o][t][k] - head[o].lift - m[t][k & 1]);
            head[o].undo = 0.f;
          }
        };
        bool later = false;
        static_assert(!F::kHeads || OWN == 1, "one block of its own for each warp");
        if (masked) {
          if constexpr (F::kHeads) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              if (!((lost >> b) & 1u)) low = max(low, F::lift(F::head(sb + b * S::kBlock)) - static_cast<int>(kQuiet));
            __syncwarp();
            if (lane == 0) s_low[pair][h] = low;
          }
#pragma unroll
          for (int o = 0; o < OWN; ++o) {
            const int tb = t0 + 16 * (h * OWN + o) + g;
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (tb + 8 * (k >> 1) >= svis[8 * t + 2 * c + (k & 1)])
                  s[o][t][k] = -INFINITY;
                else if ((lost >> (h * OWN + o)) & 1u)
                  s[o][t][k] = NAN;
                else if constexpr (F::kHeads)
                  if ((head[o].marks >> (g + 8 * (k >> 1))) & 1u) s[o][t][k] = NAN;
              }
            if constexpr (F::kHeads) {
              if (head[o].e < low) {  // far above the maximum they would be infinite: they come when it has moved
#pragma unroll
                for (int t = 0; t < TN; ++t)
#pragma unroll
                  for (int k = 0; k < 4; ++k) later = later || s[o][t][k] - m[t][k & 1] > kSlack;
                if (!later) add_quiet(o);
              }
            }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
          for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              top = fmaxf(top, fmaxf(s[o][t][e], s[o][t][e + 2]) - m[t][e]);
        const bool move = named_sync_or(1 + pair, 64, top > kSlack);
        // both warps are past the last unit
        if (h == 0 && spent >= 0) issue(spent);
        if (move) {  // a new maximum of some row, for both warps
          float* x = sx + 2 * pair * R;
#pragma unroll
          for (int t = 0; t < TN; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = fmaxf(s[0][t][e], s[0][t][e + 2]);
              if (OWN == 2) y = fmaxf(y, fmaxf(s[OWN - 1][t][e], s[OWN - 1][t][e + 2]));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
              if (g == 0) x[h * R + 8 * t + 2 * c + e] = y;
            }
          }
          named_sync(1 + pair, 64);
#pragma unroll
          for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = 8 * t + 2 * c + e;
              const float y = fmaxf(m[t][e], fmaxf(x[r], x[R + r]) - kLift);
              const float half = F::kHeads ? ex2_fast(0.5f * (m[t][e] - y)) : 0.f;
              const float down = F::kHeads ? half * half : ex2_fast(m[t][e] - y);
              l[t][e] = F::kHeads ? l[t][e] * half * half : l[t][e] * down;
              m[t][e] = y;
#pragma unroll
              for (int j = 0; j < MH; ++j) {
                O[t][j][e] *= down;
                O[t][j][e + 2] *= down;
              }
            }
          if constexpr (F::kHeads)
            if (later) add_quiet(0);
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = ex2_fast(s[o][t][k] - m[t][k & 1]);
              if constexpr (F::kHeads)
                l[t][k & 1] = fmaf(x[k], head[o].undo, l[t][k & 1]);
              else
                l[t][k & 1] += x[k];
            }
            my_p[((h * OWN + o) * NT + t) * 32 + lane] =
                make_uint2(transpose8x8(pack_f16(x[0], x[1])), transpose8x8(pack_f16(x[2], x[3])));
          }
        typename F::Values vc[NB];  // read ahead of the barrier
#pragma unroll
        for (int b = 0; b < NB; ++b) vc[b].load(sb + b * S::kBlock, g, c, h);
        named_sync(1 + pair, 64);

        // this warp's half of the outputs, over all blocks
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (masked && ((lost >> b) & 1u)) continue;  // nothing to add, or its rows are NaN already
          uint32_t nan_at = 0, vf[MH][4];
          if constexpr (F::kHeads) {
            if (masked) nan_at = F::marks(sb + b * S::kBlock) >> 16;
          } else {
            if (masked) nan_at = vc[b].mask(c, t0 + 16 * b, len, all_see);
          }
          vc[b].operands(vf);
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            const uint2 p = my_p[(b * NT + t) * 32 + lane];
#pragma unroll
            for (int j = 0; j < MH; ++j)
              mma16816(O[t][j], vf[j][0], vf[j][1], vf[j][2], vf[j][3], p.x, p.y);
          }
          if (masked && __any_sync(0xFFFFFFFFu, nan_at != 0)) {
            nan_at |= __shfl_xor_sync(0xFFFFFFFFu, nan_at, 1);
            nan_at |= __shfl_xor_sync(0xFFFFFFFFu, nan_at, 2);
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int seen = svis[8 * t + 2 * c + e] - t0 - 16 * b;
                const uint32_t sees = seen >= 16 ? 0xFFFFu : seen > 0 ? (1u << seen) - 1u : 0u;
                if (nan_at & sees) {
#pragma unroll
                  for (int j = 0; j < MH; ++j) O[t][j][e] = O[t][j][e + 2] = NAN;
                }
              }
          }
        }
        spent = stage;
        stage = stage + 1 == NS ? 0 : stage + 1;
      }
    };
    if constexpr (NT == 1) {
      run(Int<1>());
    } else if constexpr (NT == 2) {
      if (tiles == 1) run(Int<1>()); else run(Int<2>());
    } else if constexpr (NT == 3) {
      if (tiles <= 2) run(Int<2>()); else run(Int<3>());
    } else {
      if (tiles <= 2) run(Int<2>()); else if (tiles == 3) run(Int<3>()); else run(Int<4>());
    }

    // ---- join the pairs
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        if (g == 0) {
          swl[warp * R + 8 * t + 2 * c + e] = x;
          if (h == 0) swm[pair * R + 8 * t + 2 * c + e] = m[t][e];
        }
      }
    unit -= w.nu;  // in the next item
    const bool whole = w.base >= s_run.u0 && end == w.nu;
    const int my_slot = 2 * blockIdx.x + (w.base < s_run.u0 ? 0 : 1);
    float* my_part = P.part + static_cast<long long>(my_slot) * S::kPart;
    __syncthreads();
    const bool more = w.base + w.nu < s_run.u1;
    if (more) load_q(s_walk[item ^ 1]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t >= tiles) break;
      float* buf = so[t & 1];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < NP; ++i) M = fmaxf(M, swm[i * R + 8 * t + 2 * c + e]);
        const float f = ex2_fast(m[t][e] - M);
        // row 2c + e lies at place c + 4e: rows of neighbouring threads 4 banks apart
        float* to = buf + (pair * 8 + c + 4 * e) * S::kOutStride + F::first_value(g, h);
#pragma unroll
        for (int j = 0; j < MH; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(O[t][j][e] * f, O[t][j][e + 2] * f, O[t][j + 1][e] * f,
                          O[t][j + 1][e + 2] * f);
      }
      __syncthreads();
      for (int i = tid; i < 8 * D / 4; i += S::kThreads) {
        const int place = i / (D / 4), d = 4 * (i % (D / 4)), r = 8 * t + 2 * (place & 3) + (place >> 2);
        if (r >= rows) continue;
        float M = -FLT_MAX, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NP; ++k) M = fmaxf(M, swm[k * R + r]);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float l2 = swl[2 * k * R + r] + swl[(2 * k + 1) * R + r], dm = swm[k * R + r] - M;
          if constexpr (F::kHeads) L += times_two_to(l2, dm); else L += l2 * ex2_fast(dm);
          const float4 x = *reinterpret_cast<const float4*>(buf + (k * 8 + place) * S::kOutStride + d);
          o.x += x.x;
          o.y += x.y;
          o.z += x.z;
          o.w += x.w;
        }
        if (whole) {
          finish(P, w, R, r, d, D, o, M, L);
        } else {
          *reinterpret_cast<float4*>(my_part + r * D + d) = o;
          if (d == 0) {
            my_part[R * D + r] = M;
            my_part[R * D + R + r] = L;
          }
        }
      }
    }
    if (!whole)
      join_pieces<S::kThreads, R, D, 8, F::kHeads>(P, w, s_run, rows, tid, &s_last, [] { __syncthreads(); });
    if (!more) break;
    __syncthreads();  // the joining buffers and statistics are free
  }
  if (tries <= 0) {
    // no copy into this CTA's memory outlives it
    for (int i = max(0, issued - NS); i < issued; ++i)
      mbar_wait_bounded(&my_bar[i % NS], (i / NS) & 1, kWaitCycles);
    atomicOr(P.err, 1u);
  }
}

template <class F, int NT>
cudaError_t launch_tiles(const AttnParams& P, int sms, cudaStream_t stream) {
  using S = AttnShape<F, NT>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn_kernel<F, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn_kernel<F, NT><<<sms * S::kPerSm, S::kThreads, S::kSmem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sv
