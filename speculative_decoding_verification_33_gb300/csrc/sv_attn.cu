// Causal attention of each sequence's new tokens over the 4-bit paged cache (spec_kv4_attention).
//
// Everything that a sequence's rows (new tokens x query heads of one key/value head) need of the
// cache is read once for all of them: a block of 16 tokens is 18 D bytes, its products with R
// rows 64 D R operations. The unit of work is two or four blocks for one tile of R = 8 NT rows. All
// units of the call, sequence after sequence, are cut into equal runs, one per persistent CTA, so
// that the load is even whatever the lengths are; a head that is cut has its pieces joined by the
// last CTA that finishes one of them, in their order, so results do not depend on timing.
//
// Transposed products: scores^T = K q^T with 16 tokens as the rows of the matrix instruction
// (m16n8k16) and 8 query rows as its columns, outputs^T = V^T p^T with 16 values as rows. So few
// query rows waste nothing, and codes go from the cache's bytes to operands in registers: a
// byte of key codes is a pair of one token's values, a byte of value codes one value of two
// tokens, which is what the instruction takes in one register either way. e2m1 * e4m3 has at
// most 6 significant bits, exact in float16. The order of the inner dimension is free as long as
// both operands share it: thread c of a token takes values c D/4 .. c D/4 + D/4 - 1, in one load.
//
// A pair of warps takes a unit: each computes the scores and weights of half its tokens, passes
// the weights through shared memory, and sums half of the D outputs over all of the unit's tokens.
// Nothing is computed twice, and a warp holds half the accumulators that a warp alone would, so
// that 16 warps fit on an SM, where 8 left half of the issue slots to waits (64 sequences of up to
// 8192 tokens, 24 rows a head, before the work was cut by cost: 111 us, a warp alone 147 us).
//
// Each pair streams its units through a ring in shared memory with bulk copies that it issues
// itself; no barrier spans the pairs until a head ends, and then the SM's other CTA streams on.
//
// What bounds it with more than 8 rows is latency: a block of 16 tokens (D = 128) takes 64 conversions,
// 64 products with scales and 16 matrix instructions a tile of 8 rows, besides the softmax, and 16 warps
// an SM, in pairs that wait for one another twice a unit, have too little of it that is independent. With
// 20 rows 55 % of the issue slots, 42 % of the tensor pipe's cycles and 0.41 of the copy rate are used;
// most stalls are fixed latencies and the pairs' barriers. With 4 rows the bytes are near: 0.78. 524301
// tokens of 8 heads take 114 us with 4 rows (5.3 TB/s, 0.78 of the measured copy rate), 169 with 16,
// 216 with 20 (0.41); 64 sequences of up to 8192 tokens with 4 to 24 rows 88 us (0.35); one request
// of 4097 tokens 11 us, most of it the way from the lengths to the pages, the bytes and the join.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "spec_kv.h"
#include "sv_attn.cuh"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

template <int D, int NT>
struct AttnShape {
  static constexpr int kPairs = 4;  // with two CTAs an SM, 128 registers a thread
  static constexpr int kThreads = 64 * kPairs;
  static constexpr int kPerSm = 2;
  static constexpr int kRows = 8 * NT;
  // Blocks of a unit for each warp of a pair. With one tile of rows there are registers for two: half
  // the barriers, 122 us (now 114) instead of 135 for 524301 tokens of 8 heads and 4 rows, 58 instead of 61 for
  // 64 sequences of up to 8192. With two tiles that takes 160 instead of 168 us and 75 instead of
  // 72.5, and for 256 sequences of up to 1024 tokens 78 instead of 68.
  static constexpr int kOwn = NT == 1 ? 2 : 1;
  static constexpr int kUnit = 32 * kOwn;  // tokens
  // Work as it is cut: 524301 tokens of 8 heads take 135, 168, 215 and 287 us with 1 to 4 tiles and
  // one block a warp. With an item's start and end for nothing, 64 sequences of up to 8192 tokens, 24
  // rows a head, take 113 us and 256 of up to 1024 tokens 135 us; for 96, 89 and 86 us.
  static constexpr int kDearest = kOwn * (NT == 1 ? 5 : NT == 2 ? 6 : NT == 3 ? 8 : 10);
  static constexpr int kOver = 96;
  // Every pair of a CTA gets three units or so at least: with one, more pieces are to be joined, and
  // one request of 4000 tokens, 24 rows a head, takes 21.9 us instead of 17.6
  static constexpr int kLeast = 3 * kPairs / kOwn;
  static __device__ __forceinline__ int weight(int rows) {
    const int tiles = NT == 1 ? 1 : max((rows + 7) >> 3, NT - 1 > 2 ? 2 : NT - 1);
    return kOwn * (tiles <= 1 ? 5 : tiles == 2 ? 6 : tiles == 3 ? 8 : 10);
  }
  static constexpr int kBlock = KvBlock<D>::kBytes;
  static constexpr int kStage = 2 * kOwn * kBlock;
  static constexpr int kStages = (kOwn == 1 ? 3 : 2) * (128 / D);
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

// A thread's key codes of the tokens g and g + 8 of a block, and their scales (two of 16 values
// each for D = 128) as float16 pairs.
template <int D>
struct KeyCodes {
  uint32_t a[D / 32], b[D / 32], sa[2], sb[2];
  __device__ __forceinline__ void load(const unsigned char* blk, int g, int c) {
    if (D == 128) {
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(blk + g * 64 + c * 16);
      *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(blk + g * 64 + 512 + c * 16);
      const unsigned char* s = blk + KvBlock<D>::kKeyScales + g * 8 + 2 * c;
      const uint32_t x = e4m3x2(*reinterpret_cast<const uint16_t*>(s));
      const uint32_t y = e4m3x2(*reinterpret_cast<const uint16_t*>(s + 64));
      sa[0] = __byte_perm(x, x, 0x1010);
      sa[1] = __byte_perm(x, x, 0x3232);
      sb[0] = __byte_perm(y, y, 0x1010);
      sb[1] = __byte_perm(y, y, 0x3232);
    } else {
      *reinterpret_cast<uint2*>(a) = *reinterpret_cast<const uint2*>(blk + g * 32 + c * 8);
      *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(blk + g * 32 + 256 + c * 8);
      const uint32_t x = blk[KvBlock<D>::kKeyScales + g * 4 + c];
      const uint32_t y = blk[KvBlock<D>::kKeyScales + 32 + g * 4 + c];
      sa[0] = sa[1] = e4m3x2(x | (x << 8));
      sb[0] = sb[1] = e4m3x2(y | (y << 8));
    }
  }
  // Word i: 8 values of each token, the operands of two steps of the inner dimension
  __device__ __forceinline__ void operands(int i, uint32_t (&f)[2][4]) const {
    uint32_t x[4], y[4];
    e2m1x8(a[i], x);
    e2m1x8(b[i], y);
    const uint32_t fa = sa[D == 128 ? i / 2 : 0], fb = sb[D == 128 ? i / 2 : 0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[h][0] = mul_f16x2(x[2 * h], fa);
      f[h][1] = mul_f16x2(y[2 * h], fb);
      f[h][2] = mul_f16x2(x[2 * h + 1], fa);
      f[h][3] = mul_f16x2(y[2 * h + 1], fb);
    }
  }
};

// Half h of a thread's values of a block: D / 16 values of the token pairs c and c + 4.
template <int D>
struct ValueCodes {
  static constexpr int N = D / 64;  // words of codes of one token pair
  uint32_t a[N], b[N], sa, sb;
  __device__ __forceinline__ void load(const unsigned char* blk, int g, int c, int h) {
    const unsigned char* codes = blk + KvBlock<D>::kValCodes + c * D +
                                 KvBlock<D>::kChunk * KvBlock<D>::place(c, g) + 4 * N * h;
    const unsigned char* scales = blk + KvBlock<D>::kValScales + c * (D / 8) +
                                  2 * (D == 128 ? g : g >> 1);
    if (D == 128) {
      *reinterpret_cast<uint2*>(a) = *reinterpret_cast<const uint2*>(codes);
      *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(codes + 4 * D);
    } else {
      a[0] = *reinterpret_cast<const uint32_t*>(codes);
      b[0] = *reinterpret_cast<const uint32_t*>(codes + 4 * D);
    }
    sa = *reinterpret_cast<const uint16_t*>(scales);
    sb = *reinterpret_cast<const uint16_t*>(scales + D / 2);
  }
  // A token that some row does not see must not reach it as 0 * NaN: its scale is taken as 0 where
  // the cache holds nothing (past the length) or a NaN. Bit i of what is returned says that token
  // i, which some rows see, has a NaN scale among this thread's values.
  __device__ __forceinline__ uint32_t mask(int c, int t0, int len, int all_see) {
    uint32_t nan_at = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 2 * c + (k & 1) + 8 * (k >> 1), sh = 8 * (k & 1);
      uint32_t& s = k < 2 ? sa : sb;
      const bool bad = ((s >> sh) & 0x7Fu) == 0x7Fu;
      if (t0 + i >= len || (bad && t0 + i >= all_see)) s &= ~(0xFFu << sh);
      if (bad && t0 + i < len && t0 + i >= all_see) nan_at |= 1u << i;
    }
    return nan_at;
  }
  __device__ __forceinline__ void operands(uint32_t (&f)[D / 32][4]) const {
    const uint32_t fa = e4m3x2(sa), fb = e4m3x2(sb);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t x[4], y[4];
      e2m1x8(a[i], x);
      e2m1x8(b[i], y);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        f[2 * i + n][0] = mul_f16x2(x[2 * n], fa);
        f[2 * i + n][1] = mul_f16x2(x[2 * n + 1], fa);
        f[2 * i + n][2] = mul_f16x2(y[2 * n], fb);
        f[2 * i + n][3] = mul_f16x2(y[2 * n + 1], fb);
      }
    }
  }
};

// Where a pair's producer looks up next.
struct Producer {
  Walk w;
  long long u;
};

template <int N>
using Int = std::integral_constant<int, N>;

template <int D, int NT>
__global__ void __launch_bounds__(AttnShape<D, NT>::kThreads, AttnShape<D, NT>::kPerSm)
    attn_kernel(AttnParams P) {
  using S = AttnShape<D, NT>;
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
    if (tid == 0) {
      Walk nw = w;
      next_item<S>(P, nw);
      s_walk[item ^ 1] = nw;
    }
    __syncthreads();
    const int all_see = svis[0];  // tokens that every row of the tile sees

    float O[NT][MH][4], m[NT][2], l[NT][2];
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
        const bool masked = t0 + UNIT > all_see || lost;

        // scores of this warp's blocks and the tile's rows
        float s[OWN][TN][4];
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
          KeyCodes<D> kc;
          kc.load(sb + (h * OWN + o) * S::kBlock, g, c);
#pragma unroll
          for (int t = 0; t < TN; ++t) s[o][t][0] = s[o][t][1] = s[o][t][2] = s[o][t][3] = 0.f;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t kf[2][4];
            kc.operands(i, kf);
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const uint2 q = sq[(t * KS + 2 * i + n) * 32 + lane];
                mma16816(s[o][t], kf[n][0], kf[n][1], kf[n][2], kf[n][3], q.x, q.y);
              }
          }
        }
        // in base 2, rounded before the maximum is taken, so that the largest weight is exact
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const float2 qc = *reinterpret_cast<const float2*>(sqc + 8 * t + 2 * c);
#pragma unroll
          for (int o = 0; o < OWN; ++o)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[o][t][k] = __fmul_rn(s[o][t][k], k & 1 ? qc.y : qc.x);
        }
        if (masked) {
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
              const float down = ex2_fast(m[t][e] - y);
              m[t][e] = y;
              l[t][e] *= down;
#pragma unroll
              for (int j = 0; j < MH; ++j) {
                O[t][j][e] *= down;
                O[t][j][e + 2] *= down;
              }
            }
        }
#pragma unroll
        for (int o = 0; o < OWN; ++o)
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = ex2_fast(s[o][t][k] - m[t][k & 1]);
              l[t][k & 1] += x[k];
            }
            my_p[((h * OWN + o) * NT + t) * 32 + lane] =
                make_uint2(transpose8x8(pack_f16(x[0], x[1])), transpose8x8(pack_f16(x[2], x[3])));
          }
        ValueCodes<D> vc[NB];  // read ahead of the barrier
#pragma unroll
        for (int b = 0; b < NB; ++b) vc[b].load(sb + b * S::kBlock, g, c, h);
        named_sync(1 + pair, 64);

        // this warp's half of the outputs, over all blocks
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (masked && ((lost >> b) & 1u)) continue;  // nothing to add, or its rows are NaN already
          uint32_t nan_at = 0, vf[MH][4];
          if (masked) nan_at = vc[b].mask(c, t0 + 16 * b, len, all_see);
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
        float* to = buf + (pair * 8 + c + 4 * e) * S::kOutStride + (D / 8) * g + (D / 16) * h;
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
          L += (swl[2 * k * R + r] + swl[(2 * k + 1) * R + r]) * ex2_fast(swm[k * R + r] - M);
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
      join_pieces<S::kThreads, R, D, 8>(P, w, s_run, rows, tid, &s_last, [] { __syncthreads(); });
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

template <int D, int NT>
cudaError_t launch_tiles(const AttnParams& P, int sms, cudaStream_t stream) {
  using S = AttnShape<D, NT>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn_kernel<D, NT><<<sms * S::kPerSm, S::kThreads, S::kSmem, stream>>>(P);
  return cudaGetLastError();
}

// Rows of a tile, at most. For D = 128 the kernel of sv_attn_tc.cu takes what has more: with 28 rows
// a head it takes 231 us for 524301 tokens of 8 heads, 106 us for 64 sequences of up to 8192 tokens
// and 23.5 us for 8 of 2000, this one 296, 109 and 28.3; with 24 rows it takes 219, 103 and 22.5 us,
// this one 215, 89 and 20.2. It has no form for D = 64.
template <int D>
constexpr int kMaxRows = D == 128 ? 24 : 32;

template <int D>
cudaError_t launch_dim(const AttnParams& P, long long all, int sms, cudaStream_t stream) {
  // rows of a tile: a sequence's rows in as few tiles as hold them, evenly
  const long long tiles = (all + kMaxRows<D> - 1) / kMaxRows<D>;
  switch (((all + tiles - 1) / tiles + 7) / 8) {
    case 1: return launch_tiles<D, 1>(P, sms, stream);
    case 2: return launch_tiles<D, 2>(P, sms, stream);
    case 3: return launch_tiles<D, 3>(P, sms, stream);
  }
  if constexpr (kMaxRows<D> > 24) return launch_tiles<D, 4>(P, sms, stream);
  return cudaErrorInvalidValue;  // not reached
}

}  // namespace

size_t attention_workspace_bytes(int sms) {
  // two pieces a CTA, two CTAs an SM
  return kAttnHeader + static_cast<size_t>(sms) * 4 * kTcMaxRows * (128 + 2) * sizeof(float);
}

cudaError_t launch_attention(const AttnParams& P, int D, int max_new, int sms,
                             cudaStream_t stream) {
  const long long all = std::max(1LL, static_cast<long long>(max_new) * P.group);
  if (D == 64) return launch_dim<64>(P, all, sms, stream);
  return all <= kMaxRows<128> ? launch_dim<128>(P, all, sms, stream) : launch_attention_tc(P, sms, stream);
}

}  // namespace sv
