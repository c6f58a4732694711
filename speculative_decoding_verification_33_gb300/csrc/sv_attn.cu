// Causal attention of each sequence's new tokens over the 4-bit paged cache (spec_kv4_attention).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

#include "spec_kv.h"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kAtWarps = 4;

__device__ __forceinline__ float e2m1(uint32_t c) {
  const float m = (c & 6u) ? ldexpf(1.f + 0.5f * static_cast<float>(c & 1u),
                                    static_cast<int>((c >> 1) & 3u) - 1)
                           : 0.5f * static_cast<float>(c & 1u);
  return (c & 8u) ? -m : m;
}
__device__ __forceinline__ float e4m3(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xFFFFu)));
}

// A CTA per query row and head; its warps take tokens in turn, a lane D / 32 values of each.
template <int D>
__global__ void __launch_bounds__(32 * kAtWarps) attn_row_kernel(AttnParams P) {
  constexpr int N = D / 32;
  const int t = blockIdx.x / P.hq, h = blockIdx.x - t * P.hq, hk = h / P.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int b = -1;
  for (int i = 0; i < P.B; ++i)
    if (P.cu[i] <= t && t < P.cu[i + 1]) b = i;
  if (b < 0) return;
  const int n = P.cu[b + 1] - P.cu[b];
  int len = P.lens[b];
  len = max(0, min(len, P.max_blocks * P.ps));
  const int seen = min(len, len - n + (t - P.cu[b]) + 1);
  const int d0 = lane * N;
  float q[N], o[N];
  for (int i = 0; i < N; ++i) {
    q[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(P.q)[t * P.qs + static_cast<long long>(h) * D + d0 + i]);
    o[i] = 0.f;
  }
  float m = -FLT_MAX, l = 0.f;
  for (int k = warp; k < seen; k += kAtWarps) {
    const int page = P.table[static_cast<long long>(b) * P.max_blocks + k / P.ps];
    float s = 0.f, v[N];
    if (page < 0 || page >= P.num_pages) {
      s = NAN;
      for (int i = 0; i < N; ++i) v[i] = 0.f;
    } else {
      const unsigned char* blk =
          P.cache + ((static_cast<long long>(page) * P.hkv + hk) * (P.ps / 16) + k % P.ps / 16) *
                        KvBlock<D>::kBytes;
      const int i16 = k & 15, p = i16 >> 1;
      const float sk = e4m3(blk[KvBlock<D>::kKeyScales + i16 * (D / 16) + d0 / 16]);
      const float sv_ = e4m3(blk[KvBlock<D>::kValScales + (p * (D / 16) + d0 / 16) * 2 + (i16 & 1)]);
      for (int i = 0; i < N; ++i) {
        const int d = d0 + i;
        const uint32_t kc = blk[KvBlock<D>::kKeyCodes + i16 * (D / 2) + d / 2] >> (4 * (d & 1));
        s += q[i] * (e2m1(kc & 15u) * sk);
        const uint32_t vc = blk[KvBlock<D>::kValCodes + p * D +
                                KvBlock<D>::place(p, d / KvBlock<D>::kChunk) * KvBlock<D>::kChunk +
                                d % KvBlock<D>::kChunk] >> (4 * (i16 & 1));
        v[i] = e2m1(vc & 15u) * sv_;
      }
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    }
    s *= P.c;
    const float m2 = fmaxf(m, s), f = ex2_fast(m - m2), w = ex2_fast(s - m2);
    m = m2;
    l = l * f + w;
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + w * v[i];
  }
  __shared__ float sm[kAtWarps], sl[kAtWarps], so[kAtWarps][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int i = 0; i < N; ++i) so[warp][d0 + i] = o[i];
  __syncthreads();
  if (warp) return;
  float M = -FLT_MAX, L = 0.f, r[N] = {};
  for (int w = 0; w < kAtWarps; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < kAtWarps; ++w) {
    const float f = ex2_fast(sm[w] - M);
    L += sl[w] * f;
    for (int i = 0; i < N; ++i) r[i] += so[w][d0 + i] * f;
  }
  const float inv = L == 0.f ? 0.f : P.vs / L;
  for (int i = 0; i < N; ++i)
    static_cast<__nv_bfloat16*>(P.out)[(static_cast<long long>(t) * P.hq + h) * D + d0 + i] =
        __float2bfloat16_rn(r[i] * inv);
  if (lane == 0 && P.lse)
    P.lse[static_cast<long long>(t) * P.hq + h] =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_attention(const AttnParams& P, int D, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(P.T) * static_cast<unsigned>(P.hq);
  if (D == 128)
    attn_row_kernel<128><<<grid, 32 * kAtWarps, 0, stream>>>(P);
  else
    attn_row_kernel<64><<<grid, 32 * kAtWarps, 0, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace sv
