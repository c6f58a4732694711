// Shared by the attention kernels over the paged caches (4 bits: sv_attn.cu, sv_attn_tc.cu; 8 bits: sv_attn8.cu,
// sv_attn8_tc.cu): how the work is cut between CTAs and joined, and conversions. Prompts (sv_prompt.cu) take the
// waits from here.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {

constexpr long long kWaitCycles = 4000000000LL;  // about 2 s: a copy that never came
constexpr float kLift = 7.f;    // weights are held times 2^7: float16 has more room above 1 than below
constexpr float kSlack = 15.f;  // and may grow to 2^15 before the running maximum is moved

// Work is cut by what it is estimated to cost, in the cost of small parts of a unit. A kernel says
// (class W) how many rows a tile and tokens a unit have, what a unit costs for a tile of so many
// rows, and what an item's start and end cost together; that is counted behind its last unit.
//
// Where a run of units lies: item (sequence b, head h, row tile rt) with its nu units.
struct Walk {
  long long base;  // the item's first unit
  long long cost;  // of all that comes before
  int b, h, rt;
  int rts, nu, len, n, r0;
  int wt;          // cost of a unit
  int past;        // cu_new[b + 1]
  int len1, past1;  // lengths of sequence b + 1: loaded with sequence b, used after it
};

template <class W>
__device__ __forceinline__ void set_seq(const AttnParams& P, int b, int first, int past, int len,
                                        Walk& w) {
  const int c0 = min(max(first, 0), P.T), c1 = min(max(past, c0), P.T);
  w.b = b;
  w.r0 = c0;
  w.n = c1 - c0;
  w.past = past;
  w.len = min(max(len, 0), P.max_blocks * P.ps);
  w.rts = (w.n * P.group + W::kRows - 1) / W::kRows;
  w.nu = max(1, (w.len + W::kUnit - 1) / W::kUnit);
  w.wt = W::weight(min(W::kRows, w.n * P.group));
}
template <class W>
__device__ __forceinline__ void load_seq(const AttnParams& P, int b, Walk& w) {
  set_seq<W>(P, b, P.cu[b], P.cu[b + 1], P.lens[b], w);
}
__device__ __forceinline__ void load_ahead(const AttnParams& P, Walk& w) {
  w.len1 = P.lens[min(w.b + 1, P.B - 1)];
  w.past1 = P.cu[min(w.b + 2, P.B)];
}
template <class W>
__device__ __forceinline__ long long item_cost(const Walk& w) {
  return static_cast<long long>(w.nu) * w.wt + W::kOver;
}
template <class W>
__device__ __forceinline__ void next_item(const AttnParams& P, Walk& w) {
  w.base += w.nu;
  w.cost += item_cost<W>(w);
  if (++w.rt < w.rts) return;
  w.rt = 0;
  if (++w.h < P.hkv) return;
  w.h = 0;
  do {
    const int b = w.b + 1;
    if (b >= P.B) {
      w.b = P.B;
      w.nu = 1 << 30;  // nothing follows
      return;
    }
    set_seq<W>(P, b, w.past, w.past1, w.len1, w);
    load_ahead(P, w);
  } while (w.n == 0);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The four bytes of `w` as four registers of two e2m1 values each, in float16
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One try of a wait: the hardware holds the thread for some microseconds if the phase is not done.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr int kWaitTries = 1 << 19;  // a second or more

// Over the 8-bit cache weights carry 2^e of their values' block, so that the maximum M that they are held to, of
// score + e, says nothing of how large the softmax's sum is beside them: that is the sum of 2^(score - M), from
// 2^-121 up to 2^75. So sums are scaled in two steps, for a factor of less than 2^-126 may take one of 2^60 to
// where it still counts; and tokens whose e lies so far below the largest one there that their weights may be none
// come into them by score - M itself. (Otherwise what is lost of a weight is below 2^(-126 - e) in the sum. M lies
// 2^7 below score + e of some token, whose part of the sum is 2^(7 - e): 2^43 times as much or more.)
constexpr unsigned kQuiet = 90;  // exponents of values, all from -60 on
__device__ __forceinline__ float times_two_to(float x, float d) {
  const float half = ex2_fast(0.5f * d);
  return x * half * half;
}

// Weights and values (o: 4 dimensions from d of row r of the item's tile, sum L at maximum M, in
// base 2) into the output and its log-sum.
__device__ __forceinline__ long long out_row(const AttnParams& P, const Walk& w, int tile_rows,
                                             int r) {
  const int row = w.rt * tile_rows + r;
  return static_cast<long long>(w.r0 + row / P.group) * P.hq + w.h * P.group + row % P.group;
}
__device__ __forceinline__ void store_lse(const AttnParams& P, long long at, float M, float L) {
  if (P.lse) P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}
__device__ __forceinline__ void finish(const AttnParams& P, const Walk& w, int tile_rows, int r,
                                       int d, int D, float4 o, float M, float L) {
  const float inv = L == 0.f ? 0.f : P.vs / L;
  const long long at = out_row(P, w, tile_rows, r);
  const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + at * D + d) = make_uint2(
      *reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
  if (d == 0) store_lse(P, at, M, L);
}

// This CTA's run of the call's units: first unit, past the last, the cost of all, CTAs that share it.
struct Run {
  long long u0, u1, all, ctas;
};

// The CTA that has the unit which starts at this cost: the last one whose share starts there or before.
__device__ __forceinline__ int cta_of(const Run& run, long long cost) {
  return static_cast<int>(divide((cost + 1) * run.ctas + run.all - 1, run.all)) - 1;
}

// Finds the run and the item that holds its first unit; false if there is none for this CTA. Every
// thread calls it. A CTA's share costs as much as kLeast of the dearest units at least, so that an
// item's pieces lie with neighbours. Ends with a barrier.
template <int THREADS, class W>
__device__ __forceinline__ bool find_run(const AttnParams& P, longlong2* scan, Run* run, Walk* first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Walk w;
  const int per = (P.B + THREADS - 1) / THREADS;
  const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
  longlong2 mine = make_longlong2(0, 0);  // cost, units
  for (int b = b0; b < b1; ++b) {
    load_seq<W>(P, b, w);
    const long long items = static_cast<long long>(w.rts) * P.hkv;
    mine.x += items * item_cost<W>(w);
    mine.y += items * w.nu;
  }
  longlong2 x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long cost = __shfl_up_sync(0xFFFFFFFFu, x.x, d);
    const long long units = __shfl_up_sync(0xFFFFFFFFu, x.y, d);
    if (lane >= d) {
      x.x += cost;
      x.y += units;
    }
  }
  if (lane == 31) scan[warp] = x;
  if (tid == 0) run->u0 = run->u1 = 0;
  __syncthreads();
  longlong2 before = make_longlong2(x.x - mine.x, x.y - mine.y), all = make_longlong2(0, 0);
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const longlong2 n = scan[i];
    if (i < warp) {
      before.x += n.x;
      before.y += n.y;
    }
    all.x += n.x;
    all.y += n.y;
  }
  constexpr int kShare = W::kLeast * W::kDearest;
  const long long ctas = min(static_cast<long long>(gridDim.x), divide(all.x + kShare - 1, kShare));
  if (blockIdx.x >= ctas) return false;
  const long long c0 = divide(all.x * blockIdx.x, ctas), c1 = divide(all.x * (blockIdx.x + 1), ctas);
  const bool has0 = c0 >= before.x && c0 < before.x + mine.x;
  const bool has1 = c1 >= before.x && c1 < before.x + mine.x;
  if (has0 || has1) {
    for (int b = b0; b < b1; ++b) {
      load_seq<W>(P, b, w);
      const long long one = item_cost<W>(w), items = static_cast<long long>(w.rts) * P.hkv;
      // the first unit that starts at c or later: past the item's last if c lies behind that
      auto unit_at = [&](long long c, long long item) {
        const long long i = divide(c - before.x - item * one + w.wt - 1, w.wt);
        return before.y + item * w.nu + min(i, static_cast<long long>(w.nu));
      };
      if (c0 >= before.x && c0 < before.x + items * one) {
        const long long item = divide(c0 - before.x, one);
        run->u0 = unit_at(c0, item);
        run->all = all.x;
        run->ctas = ctas;
        Walk at = w;
        at.h = static_cast<int>(divide(item, w.rts));
        at.rt = static_cast<int>(item - static_cast<long long>(at.h) * w.rts);
        at.base = before.y + item * w.nu;
        at.cost = before.x + item * one;
        load_ahead(P, at);
        if (run->u0 == at.base + at.nu) next_item<W>(P, at);
        *first = at;
      }
      if (c1 >= before.x && c1 < before.x + items * one) run->u1 = unit_at(c1, divide(c1 - before.x, one));
      before.x += items * one;
      before.y += items * w.nu;
    }
  }
  if (tid == 0 && blockIdx.x + 1 == ctas) run->u1 = all.y;
  __syncthreads();
  return run->u0 < run->u1;
}

// A CTA has two pieces of items at most, one that ends an item or goes on with it and one that
// starts one, at P.part in this order (R x D outputs, maxima, sums). A piece is written: counts
// it, and in the last CTA to arrive at the item joins its pieces, in their order. THREADS threads
// call it, tid of them this one, with `sync` a barrier among them. HEADS: of the 8-bit cache.
template <int THREADS, int R, int D, int BATCH, bool HEADS, class Sync>
__device__ __forceinline__ void join_pieces(const AttnParams& P, const Walk& w, const Run& run,
                                            int rows, int tid, int* s_last, Sync sync) {
  constexpr long long kPart = R * (D + 2);
  // pieces of this item lie with CTAs first .. last
  const int first = cta_of(run, w.cost);
  const int last = cta_of(run, w.cost + static_cast<long long>(w.nu - 1) * w.wt);
  __threadfence();
  sync();
  if (tid == 0) *s_last = atomicAdd(&P.arrived[first], 1u) == static_cast<unsigned>(last - first);
  sync();
  if (!*s_last) return;
  __threadfence();
  auto part_of = [&](int k) {
    return P.part + static_cast<long long>(2 * k + (k == first ? 1 : 0)) * kPart;
  };
  for (int i = tid; i < rows * (D / 4); i += THREADS) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    float M = -FLT_MAX, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // a few pieces at a time, so that their loads are in flight together
    for (int k0 = first; k0 <= last; k0 += BATCH) {
      float m[BATCH], l[BATCH], top = M;
      float4 x[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        m[i] = -FLT_MAX;
        l[i] = 0.f;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + i <= last) {
          const float* part = part_of(k0 + i);
          m[i] = __ldcg(part + R * D + r);
          l[i] = __ldcg(part + R * D + R + r);
          x[i] = __ldcg(reinterpret_cast<const float4*>(part + r * D + d));
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) top = fmaxf(top, m[i]);
      const float half = ex2_fast((HEADS ? 0.5f : 1.f) * (M - top)), down = HEADS ? half * half : half;
      L = HEADS ? L * half * half : L * down;
      M = top;
      o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float half = ex2_fast((HEADS ? 0.5f : 1.f) * (m[i] - M)), f = HEADS ? half * half : half;
        L += HEADS ? l[i] * half * half : l[i] * f;
        o.x += x[i].x * f;
        o.y += x[i].y * f;
        o.z += x[i].z * f;
        o.w += x[i].w * f;
      }
    }
    finish(P, w, R, r, d, D, o, M, L);
  }
  if (tid == 0) P.arrived[first] = 0;  // ready for the next call
}

// Queries as float16: each row times a power of two that brings its largest finite magnitude
// (`most`, bf16 bits) to 2^14 .. 2^15, so that a value down to 2^-28 of that one is exact; *undo is
// what takes a product back, times c.
__device__ __forceinline__ float query_scale(unsigned most, float c, float* undo) {
  const int k = min(14 - (static_cast<int>(most >> 7) - 127), 100);
  *undo = c * __int_as_float((127 - k) << 23);
  return __int_as_float((k + 127) << 23);
}
__device__ __forceinline__ unsigned largest_finite(uint4 raw) {
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
  unsigned most = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned v = (x[k >> 1] >> (16 * (k & 1))) & 0x7FFFu;
    if (v < 0x7F80u) most = max(most, v);
  }
  return most;
}
__device__ __forceinline__ void query_f16(uint4 raw, float up, uint32_t (&f)[4]) {
  const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int m = 0; m < 4; ++m)
    f[m] = pack_f16(__uint_as_float(x[m] << 16) * up, __uint_as_float(x[m] & 0xFFFF0000u) * up);
}

}  // namespace sv
