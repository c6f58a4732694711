// Causal attention over whole prompts, packed (spec_prompt_attention).
//
// The row kernel: a warp takes one row of one query head and goes once over the tokens that the row sees,
// 32 at a time, a lane a token for the scores and D / 32 values of the output, with the running maximum and
// sum of the softmax.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

// Row `row` of the call, of query head `head`, whose sequence starts at r0; a warp calls it. q: the row as
// float32 in shared memory, this warp's own.
template <int D>
__device__ void prompt_row(const PromptParams& P, int r0, int row, int head, float* q) {
  constexpr int V = D / 32;  // values of a lane
  const int lane = threadIdx.x & 31, hk = head / P.group;
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(P.q) + row * P.qs + static_cast<long long>(head) * D;
  __syncwarp();
  for (int i = lane; i < D; i += 32) q[i] = __bfloat162float(qp[i]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int t0 = r0; t0 <= row; t0 += 32) {
    float z = -INFINITY;
    if (t0 + lane <= row) {
      const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.k) + (t0 + lane) * P.ks +
                                                      static_cast<long long>(hk) * D);
      float sum = 0.f;
      for (int i = 0; i < D / 8; ++i) {
        const uint4 w = __ldg(k + i);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum = fmaf(__uint_as_float(x[j] << 16), q[8 * i + 2 * j], sum);
          sum = fmaf(__uint_as_float(x[j] & 0xFFFF0000u), q[8 * i + 2 * j + 1], sum);
        }
      }
      z = sum * P.c;
    }
    float top = z;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.f : m1;
    const float down = exp2f(m - base);  // 0 where m is -inf
    const float p = exp2f(z - base);     // a NaN stays one
    m = m1;
    float add = p;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
    l = l * down + add;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= down;
    const int n = min(32, row - t0 + 1);
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(0xFFFFFFFFu, p, j);
      const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(P.v) + (t0 + j) * P.vs +
                               static_cast<long long>(hk) * D + V * lane;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(pj, __bfloat162float(v[i]), o[i]);
    }
  }
  const long long at = static_cast<long long>(row) * P.hq + head;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(P.out) + at * D + V * lane;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = __float2bfloat16_rn(o[i] / l);
  if (lane == 0 && P.lse) P.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
}

// The first row of the sequence of row `row`, or -1 where it has none.
__device__ int sequence_of(const PromptParams& P, int row) {
  int lo = 0, hi = P.B;  // the first b with cu[b + 1] > row
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (P.cu[mid + 1] > row) hi = mid; else lo = mid + 1;
  }
  if (lo == P.B) return -1;
  const int first = max(P.cu[lo], 0);
  return first <= row ? first : -1;
}

template <int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(PromptParams P) {
  __shared__ float q[4][D];
  const long long i = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (i >= static_cast<long long>(P.T) * P.hq) return;
  const int row = static_cast<int>(i / P.hq), head = static_cast<int>(i % P.hq);
  const int r0 = sequence_of(P, row);
  if (r0 >= 0) prompt_row<D>(P, r0, row, head, q[threadIdx.x >> 5]);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& P, int D, int, cudaStream_t stream) {
  const long long rows = static_cast<long long>(P.T) * P.hq;
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  if (D == 64)
    prompt_rows_kernel<64><<<grid, 128, 0, stream>>>(P);
  else
    prompt_rows_kernel<128><<<grid, 128, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace sv
