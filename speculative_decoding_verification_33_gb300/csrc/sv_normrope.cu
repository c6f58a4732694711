// Norms of queries and keys per head and the rotation by position (spec_qk_norm_rope).
//
// Every value is read once and written once; the norm and the rotation happen in registers in
// between, so the pass is bound by HBM. A thread holds two 16-byte vectors of a head, chosen so
// that both halves of each rotated pair are its own: vectors j and j + rot/2 for halves, two
// neighbours for interleaved pairs. D / 16 bf16 threads share a head's sum of squares by
// shuffles. A CTA takes a few tokens, computes their sines and cosines once, and runs through the
// heads. 32767 tokens of 28 + 4 heads of 128 in bf16 take 97 us, 5.5 TB/s or 0.82 of the measured
// copy rate; 8 tokens 2.8 us, which is the launch; 1153 tokens of 16 + 2 heads of 64 in float32,
// interleaved, 5.4 us (1.6 us of bytes: all of them fit the L2, the launch and one wave bound it).
//
// The angle position * inv_freq needs more bits than float32 has (2^-24 of a position of 10^6 is
// a twentieth of a turn) but only its fraction of a turn matters: inv_freq / 2 pi is held as a 64-bit
// fixed-point fraction of a turn, to nearest. Its product with the position, modulo 2^64, is the angle's
// fraction, off by position * 2^-65 turns at most. The nearest quarter turn goes into signs, the rest, at
// most an eighth and rounded to 2^-32 turns, through sincospif.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "spec_kv.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrMaxD = 512;

struct NormRopeParams {
  int T, hq, hk, D, rot, inter;
  long long qs, ks, oqs, oks;  // token strides in elements
  const void *q, *k, *wq, *wk;
  const int32_t* pos;
  const double* freq;
  float eps;
  void *oq, *ok;
  int tokens;   // tokens of a CTA
  int splits;   // CTAs that share a token group's heads
};

// Fraction of a turn per position, times 2^64, to nearest; 0 for |freq| >= 2^54. In integers: the 53 bits
// of freq times the first 128 of 2 / pi (a quarter turn is pi / 2), of which 64 are taken from where freq's
// exponent has them. In double the product's rounding, some 2^-56 turns for a frequency of 1, would be
// 2^-25 turns at position 2^31, and with its error carried along 1153 tokens take 6.0 us instead of 5.4:
// double arithmetic is slow here.
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(freq));
  const int exponent = static_cast<int>(bits >> 52) & 0x7FF;  // freq = m 2^(exponent - 1075)
  const unsigned long long m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const unsigned long long high = 0xA2F9836E4E441529ull, low = 0xFC2757D1F534DDC0ull;  // 2 / pi 2^128
  const int at = 1140 - exponent;  // the result's bits of m * 2 / pi * 2^128, and one for rounding
  if (at < 64 || at >= 192) return 0;
  // bits 64 to 127 and 128 to 191
  const unsigned long long p1 = m * high + __umul64hi(m, low);
  const unsigned long long p2 = __umul64hi(m, high) + (p1 < m * high);
  const unsigned long long a = at < 128 ? p1 : p2, b = at < 128 ? p2 : 0;
  const int off = at & 63;
  const unsigned long long g = (a >> off) | ((b << 1) << (63 - off));
  const unsigned long long f = ((g >> 1) | ((b >> off) << 63)) + (g & 1);
  return bits >> 63 ? 0 - f : f;
}

__device__ __forceinline__ float2 cos_sin(unsigned long long fraction, int pos) {
  const unsigned long long f = fraction * static_cast<unsigned long long>(static_cast<long long>(pos));
  const int hi = static_cast<int>(static_cast<uint32_t>((f + 0x80000000ull) >> 32));  // 2^-32 turns
  const int quarter = static_cast<int>((static_cast<uint32_t>(hi) + 0x20000000u) >> 30);
  const int rest = hi - static_cast<int>(static_cast<uint32_t>(quarter) << 30);
  float s, c;
  sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
  const float c2 = (quarter & 1) ? s : c, s2 = (quarter & 1) ? c : s;
  return make_float2(((quarter + 1) & 2) ? -c2 : c2, (quarter & 2) ? -s2 : s2);
}

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(uint4 a, float (&x)[4]) {
  x[0] = __uint_as_float(a.x);
  x[1] = __uint_as_float(a.y);
  x[2] = __uint_as_float(a.z);
  x[3] = __uint_as_float(a.w);
}
__device__ __forceinline__ void unpack(uint4 a, float (&x)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// LPH threads a head, each with two 16-byte vectors. Such a group stays with one token and takes
// its heads in turn, so that sines, cosines and weights stay in registers; the next head is loaded
// while this one is worked on.
template <typename T, int LPH>
__global__ void __launch_bounds__(kNrThreads, 4) norm_rope_kernel(NormRopeParams P) {
  constexpr int N = Vec<T>::n, G = kNrThreads / LPH;
  extern __shared__ __align__(16) float2 cs[];  // per token: cosine, sine of each thread's pairs
  const int half = P.rot / 2;
  const int block = blockIdx.x / P.splits, split = blockIdx.x - block * P.splits;
  const int t0 = block * P.tokens, nt = min(P.tokens, P.T - t0);
  const int lane = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int per = G / P.tokens;  // groups of a token
  const int t = group / per;
  const unsigned mask = (LPH == 32 ? 0xFFFFFFFFu : (1u << LPH) - 1u)
                        << ((threadIdx.x & 31) & ~(LPH - 1));  // the threads of this head
  // vectors of this thread: (lane, lane + rotated half) while they last, else neighbours
  const int hv = P.inter ? 0 : half / N;
  const bool halves = lane < hv;
  const int va = halves ? lane : 2 * lane, vb = halves ? lane + hv : 2 * lane + 1;
  // interleaved: whole vectors are rotated or not
  const bool pair_a = P.inter && va * N < P.rot, pair_b = P.inter && vb * N < P.rot;
  // heads of q, then of k: this group's are split * per + group % per and every (splits * per)-th on
  int h = split * per + group % per;
  const int step = P.splits * per;
  const long long row = t0 + min(t, nt - 1);
  auto source = [&](bool k, int head) {
    return reinterpret_cast<const uint4*>(static_cast<const T*>(k ? P.k : P.q) +
                                          row * (k ? P.ks : P.qs) + static_cast<long long>(head) * P.D);
  };
  // the next head is on its way at any time, the first one while the sines are computed
  uint4 na = make_uint4(0u, 0u, 0u, 0u), nb = na;
  auto fetch = [&](int head) {  // of q, then of k
    if (head >= P.hq + P.hk) return;
    const uint4* x = source(head >= P.hq, head < P.hq ? head : head - P.hq);
    na = __ldcs(x + va);
    nb = __ldcs(x + vb);
  };
  fetch(h);
  unsigned long long turn = 0;
  for (int i = threadIdx.x, last = -1; i < nt * half; i += kNrThreads) {
    const int t = i / half, j = i - t * half;
    if (j != last) turn = turn_fraction(P.freq[j]);  // the same j again where half divides the CTA
    last = j;
    // pair j % N of thread j / N, so that a head's threads read side by side
    cs[((t * (N / 2) + j % N / 2) * LPH + j / N) * 2 + j % 2] = cos_sin(turn, P.pos[t0 + t]);
  }
  __syncthreads();
  if (t >= nt) return;
  const float4* angles = reinterpret_cast<const float4*>(cs) + t * (N / 2) * LPH + lane;
  const float inv_d = 1.f / static_cast<float>(P.D);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = which ? P.hk : P.hq;
    if (h < heads) {
      const uint4* w = static_cast<const uint4*>(which ? P.wk : P.wq);
      uint4 ra = make_uint4(0u, 0u, 0u, 0u), rb = ra;
      if (w) {
        ra = __ldg(w + va);
        rb = __ldg(w + vb);
      }
      T* y = static_cast<T*>(which ? P.ok : P.oq) + row * (which ? P.oks : P.oqs) +
             static_cast<long long>(h) * P.D;
      const int hop = step * P.D;
#pragma unroll 1
      for (; h < heads; h += step) {
        float a[N], b[N];
        unpack(na, a);
        unpack(nb, b);
        fetch((which ? P.hq : 0) + h + step);
        float sum = 0.f, sum2 = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          sum = fmaf(a[i], a[i], sum);
          sum2 = fmaf(b[i], b[i], sum2);
        }
        sum += sum2;
#pragma unroll
        for (int d = LPH / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(mask, sum, d, LPH);
        const float r = rsqrtf(fmaf(sum, inv_d, P.eps));
        if (w) {
          float wa[N], wb[N];
          unpack(ra, wa);
          unpack(rb, wb);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            a[i] *= r * wa[i];
            b[i] *= r * wb[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            a[i] *= r;
            b[i] *= r;
          }
        }
        if (halves) {
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float4 f = angles[i / 2 * LPH];
            float y0 = a[i] * f.x - b[i] * f.y, y1 = b[i] * f.x + a[i] * f.y;
            a[i] = y0;
            b[i] = y1;
            y0 = a[i + 1] * f.z - b[i + 1] * f.w;
            y1 = b[i + 1] * f.z + a[i + 1] * f.w;
            a[i + 1] = y0;
            b[i + 1] = y1;
          }
        }
        if (pair_a || pair_b) {
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float4 f = angles[i / 2 * LPH];  // two pairs: of a, then of b
            float* x = i < N / 2 ? a : b;
            const int k = 2 * i % N;
            if (i < N / 2 ? pair_a : pair_b) {
              float y0 = x[k] * f.x - x[k + 1] * f.y, y1 = x[k + 1] * f.x + x[k] * f.y;
              x[k] = y0;
              x[k + 1] = y1;
              y0 = x[k + 2] * f.z - x[k + 3] * f.w;
              y1 = x[k + 3] * f.z + x[k + 2] * f.w;
              x[k + 2] = y0;
              x[k + 3] = y1;
            }
          }
        }
        __stcs(reinterpret_cast<uint4*>(y) + va, pack(a));
        __stcs(reinterpret_cast<uint4*>(y) + vb, pack(b));
        y += hop;
      }
    }
    h -= heads;
  }
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Any even D and rot, any alignment: a warp a head, a pair of values at a time a lane.
template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_rope_any_kernel(NormRopeParams P) {
  const int heads = P.hq + P.hk, half = P.rot / 2;
  const long long item = static_cast<long long>(blockIdx.x) * (kNrThreads / 32) + threadIdx.x / 32;
  if (item >= static_cast<long long>(P.T) * heads) return;
  const int lane = threadIdx.x % 32;
  const long long row = item / heads;
  const int h = static_cast<int>(item - row * heads);
  const bool is_q = h < P.hq;
  const int hh = is_q ? h : h - P.hq;
  const T* x = static_cast<const T*>(is_q ? P.q : P.k) + row * (is_q ? P.qs : P.ks) +
               static_cast<long long>(hh) * P.D;
  T* y = static_cast<T*>(is_q ? P.oq : P.ok) + row * (is_q ? P.oqs : P.oks) +
         static_cast<long long>(hh) * P.D;
  const T* w = static_cast<const T*>(is_q ? P.wq : P.wk);
  constexpr int kPairs = kNrMaxD / 64;  // pairs of a lane
  float a[kPairs], b[kPairs];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int j = lane + 32 * i;  // pair; the first `half` are rotated
    if (j >= P.D / 2) break;
    const int ia = !P.inter && j < half ? j : 2 * j, ib = !P.inter && j < half ? j + half : 2 * j + 1;
    a[i] = as_float(x[ia]);
    b[i] = as_float(x[ib]);
    sum += a[i] * a[i] + b[i] * b[i];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  const float r = 1.0f / sqrtf(sum / static_cast<float>(P.D) + P.eps);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int j = lane + 32 * i;
    if (j >= P.D / 2) break;
    const int ia = !P.inter && j < half ? j : 2 * j, ib = !P.inter && j < half ? j + half : 2 * j + 1;
    float y0 = a[i] * r * (w ? as_float(w[ia]) : 1.f), y1 = b[i] * r * (w ? as_float(w[ib]) : 1.f);
    if (j < half) {
      const float2 f = cos_sin(turn_fraction(P.freq[j]), P.pos[row]);
      const float z0 = y0 * f.x - y1 * f.y, z1 = y1 * f.x + y0 * f.y;
      y0 = z0;
      y1 = z1;
    }
    put(y + ia, y0);
    put(y + ib, y1);
  }
}

template <typename T>
cudaError_t launch_norm_rope(const NormRopeParams& Q, bool fast, cudaStream_t s) {
  NormRopeParams P = Q;
  const int heads = P.hq + P.hk;
  if (!fast) {
    const long long warps = static_cast<long long>(P.T) * heads;
    norm_rope_any_kernel<T><<<static_cast<unsigned>((warps + kNrThreads / 32 - 1) / (kNrThreads / 32)),
                              kNrThreads, 0, s>>>(P);
    return cudaGetLastError();
  }
  const int lph = P.D / (2 * Vec<T>::n), groups = kNrThreads / lph;
  // Up to 8 tokens a CTA, as many as leave 8 CTAs a multiprocessor; with few tokens the heads of
  // each are shared out so that a group has one.
  P.tokens = 1;
  while (P.tokens < 8 && P.tokens < groups && P.T / (2 * P.tokens) >= 8 * 152) P.tokens *= 2;
  P.splits = P.T < 4 * 152 ? (heads + groups - 1) / groups : 1;
  const unsigned grid = static_cast<unsigned>((P.T + P.tokens - 1) / P.tokens * static_cast<long long>(P.splits));
  const size_t smem = static_cast<size_t>(P.tokens) * (P.D / 2) * sizeof(float2);
  switch (lph) {
    case 4: norm_rope_kernel<T, 4><<<grid, kNrThreads, smem, s>>>(P); break;
    case 8: norm_rope_kernel<T, 8><<<grid, kNrThreads, smem, s>>>(P); break;
    case 16: norm_rope_kernel<T, 16><<<grid, kNrThreads, smem, s>>>(P); break;
    case 32: norm_rope_kernel<T, 32><<<grid, kNrThreads, smem, s>>>(P); break;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_qk_norm_rope(int T, int Hq, int Hkv, int D, int rot, int interleaved,
                                       sv_dtype dtype, const void* q, long long q_token_stride,
                                       const void* k, long long k_token_stride,
                                       const void* q_weight, const void* k_weight,
                                       const int32_t* positions, const double* inv_freq,
                                       float eps, void* out_q, long long out_q_token_stride,
                                       void* out_k, long long out_k_token_stride, void* stream) {
  if (T < 0 || Hq < 1 || Hkv < 0 || D < 2 || D % 2 || rot < 0 || rot > D || rot % 2)
    return SV_ERR_INVALID_ARG;
  if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_INVALID_ARG;
  if (!(std::isfinite(eps) && eps >= 0.f)) return SV_ERR_INVALID_ARG;
  const long long rq = static_cast<long long>(Hq) * D, rk = static_cast<long long>(Hkv) * D;
  if (q_token_stride < rq || out_q_token_stride < rq) return SV_ERR_INVALID_ARG;
  if (Hkv > 0 && (k_token_stride < rk || out_k_token_stride < rk)) return SV_ERR_INVALID_ARG;
  if (D > sv::kNrMaxD) return SV_ERR_UNSUPPORTED;
  if (T == 0) return SV_OK;
  if (!q || !out_q || (Hkv > 0 && (!k || !out_k))) return SV_ERR_INVALID_ARG;
  if (rot > 0 && (!positions || !inv_freq)) return SV_ERR_INVALID_ARG;
  if (q == out_q && q_token_stride != out_q_token_stride) return SV_ERR_INVALID_ARG;
  if (Hkv > 0 && k == out_k && k_token_stride != out_k_token_stride) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * (Hq + static_cast<long long>(Hkv)) > (1LL << 33))
    return SV_ERR_UNSUPPORTED;  // the grid's size
  sv::NormRopeParams P;
  P.T = T;
  P.hq = Hq;
  P.hk = Hkv;
  P.D = D;
  P.rot = rot;
  P.inter = interleaved ? 1 : 0;
  P.qs = q_token_stride;
  P.ks = k_token_stride;
  P.oqs = out_q_token_stride;
  P.oks = out_k_token_stride;
  P.q = q;
  P.k = k;
  P.wq = q_weight;
  P.wk = k_weight;
  P.pos = positions;
  P.freq = inv_freq;
  P.eps = eps;
  P.oq = out_q;
  P.ok = out_k;
  P.tokens = P.splits = 1;
  // whole 16-byte vectors, both vectors of a thread rotated the same way, a power of two threads
  const int n = dtype == SV_DTYPE_BF16 ? 8 : 4;
  const size_t elt = dtype == SV_DTYPE_BF16 ? 2 : 4;
  auto aligned = [&](const void* p, long long stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
           (stride * static_cast<long long>(elt)) % 16 == 0;
  };
  const int lph = D / (2 * n);
  bool fast = D % (2 * n) == 0 && (lph == 4 || lph == 8 || lph == 16 || lph == 32) &&
              (P.inter ? rot : rot / 2) % n == 0 && aligned(q, q_token_stride) &&
              aligned(out_q, out_q_token_stride) && aligned(q_weight, 0) && aligned(k_weight, 0);
  if (Hkv > 0) fast = fast && aligned(k, k_token_stride) && aligned(out_k, out_k_token_stride);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SV_DTYPE_BF16 ? sv::launch_norm_rope<__nv_bfloat16>(P, fast, s)
                                               : sv::launch_norm_rope<float>(P, fast, s);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
