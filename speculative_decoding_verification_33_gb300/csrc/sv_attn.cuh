// Shared by the attention kernels over the 4-bit cache (sv_attn.cu, sv_attn_tc.cu): how the work is
// cut between CTAs and joined, and conversions.
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

// Where a run of units lies: item (sequence b, head h, row tile rt) with its nu units.
struct Walk {
  long long base;  // the item's first unit
  int b, h, rt;
  int rts, nu, len, n, r0;
  int past;        // cu_new[b + 1]
  int len1, past1;  // lengths of sequence b + 1: loaded with sequence b, used after it
};

template <int R, int UNIT>
__device__ __forceinline__ void set_seq(const AttnParams& P, int b, int first, int past, int len,
                                        Walk& w) {
  const int c0 = min(max(first, 0), P.T), c1 = min(max(past, c0), P.T);
  w.b = b;
  w.r0 = c0;
  w.n = c1 - c0;
  w.past = past;
  w.len = min(max(len, 0), P.max_blocks * P.ps);
  w.rts = (w.n * P.group + R - 1) / R;
  w.nu = max(1, (w.len + UNIT - 1) / UNIT);
}
template <int R, int UNIT>
__device__ __forceinline__ void load_seq(const AttnParams& P, int b, Walk& w) {
  set_seq<R, UNIT>(P, b, P.cu[b], P.cu[b + 1], P.lens[b], w);
}
__device__ __forceinline__ void load_ahead(const AttnParams& P, Walk& w) {
  w.len1 = P.lens[min(w.b + 1, P.B - 1)];
  w.past1 = P.cu[min(w.b + 2, P.B)];
}
__device__ __forceinline__ long long seq_units(const AttnParams& P, const Walk& w) {
  return static_cast<long long>(w.rts) * P.hkv * w.nu;
}
template <int R, int UNIT>
__device__ __forceinline__ void next_item(const AttnParams& P, Walk& w) {
  w.base += w.nu;
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
    set_seq<R, UNIT>(P, b, w.past, w.past1, w.len1, w);
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

// This CTA's run of the call's units. run: first unit, past the last, all units, CTAs that have any.
struct Run {
  long long u0, u1, U, ctas;
};

// Finds the run and the item that holds its first unit; false if there is none for this CTA. Every
// thread calls it; `least` units a CTA at least. Ends with a barrier.
template <int THREADS, int R, int UNIT>
__device__ __forceinline__ bool find_run(const AttnParams& P, int least, long long* scan, Run* run,
                                         Walk* first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Walk w;
  const int per = (P.B + THREADS - 1) / THREADS;
  const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    load_seq<R, UNIT>(P, b, w);
    mine += seq_units(P, w);
  }
  long long x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  long long before = 0, U = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    const long long n = scan[i];
    if (i < warp) before += n;
    U += n;
  }
  before += x - mine;
  const long long ctas = min(static_cast<long long>(gridDim.x), divide(U + least - 1, least));
  if (blockIdx.x >= ctas) return false;
  const long long u0 = divide(U * blockIdx.x, ctas);
  if (u0 >= before && u0 < before + mine) {
    for (int b = b0; b < b1; ++b) {
      load_seq<R, UNIT>(P, b, w);
      const long long n = seq_units(P, w);
      if (u0 < before + n) {
        const long long item = divide(u0 - before, w.nu);
        w.h = static_cast<int>(divide(item, w.rts));
        w.rt = static_cast<int>(item - static_cast<long long>(w.h) * w.rts);
        w.base = before + item * w.nu;
        load_ahead(P, w);
        *first = w;
        run->u0 = u0;
        run->u1 = divide(U * (blockIdx.x + 1), ctas);
        run->U = U;
        run->ctas = ctas;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  return true;
}

// A piece of an item is written (R x D outputs, maxima, sums at P.part + slot * part_floats): counts
// it, and in the last CTA to arrive at the item joins its pieces, in their order. THREADS threads
// call it, tid of them this one, with `sync` a barrier among them.
template <int THREADS, int R, int D, int BATCH, class Sync>
__device__ __forceinline__ void join_pieces(const AttnParams& P, const Walk& w, const Run& run,
                                            int rows, int tid, int* s_last, Sync sync) {
  constexpr long long kPart = R * (D + 2);
  // pieces of this item lie with CTAs first .. last
  const int first = static_cast<int>(divide((w.base + 1) * run.ctas + run.U - 1, run.U)) - 1;
  const int last = static_cast<int>(divide((w.base + w.nu) * run.ctas + run.U - 1, run.U)) - 1;
  __threadfence();
  sync();
  if (tid == 0) *s_last = atomicAdd(&P.arrived[first], 1u) == static_cast<unsigned>(last - first);
  sync();
  if (!*s_last) return;
  __threadfence();
  const int slot0 = 2 * first + (divide(run.U * first, run.ctas) >= w.base ? 0 : 1);
  auto part_of = [&](int k) {
    return P.part + static_cast<long long>(k == first ? slot0 : 2 * k) * kPart;
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
      const float down = ex2_fast(M - top);
      M = top;
      L *= down;
      o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float f = ex2_fast(m[i] - M);
        L += l[i] * f;
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
