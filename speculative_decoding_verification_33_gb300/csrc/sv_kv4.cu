// Keys and values into the 4-bit paged cache (spec_kv4_append).
//
// A thread takes 16 neighbouring values of one token and head, which share a scale: their maximum
// needs no other thread. Keys then are 8 bytes of codes and a scale byte. A byte of value codes
// holds two tokens, the even slot low: where the call brings both tokens of a pair one after the
// other, the even token's thread quantises both and stores 16 bytes; a token alone sets its four
// bits of each byte with a pair of atomics on 32-bit words, which leaves the other token's bits
// alone, whoever else writes the word. Bits of different tokens never meet, so the order of the
// atomics does not matter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "spec_kv.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr int kApThreads = 256;

struct AppendParams {
  int T, H, ps, num_pages;
  long long ks, vs;  // token strides of k and v, in elements
  const void *k, *v;
  const int64_t* slots;
  float gk, gv, ik, iv;  // tensor scales, and float32(1 / (6 g))
  unsigned char* cache;
  __nv_bfloat16 *ok, *ov;
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = a.x;
    x[4 * i + 1] = a.y;
    x[4 * i + 2] = a.z;
    x[4 * i + 3] = a.w;
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// float -> e4m3 bits, nearest even, held at 448
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xFFFFu)));
}
// Two values -> a byte of e2m1 codes, `lo` in the low four bits; nearest even, held at 6
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e2m1x2(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(b));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// 16 values -> 8 bytes of codes (value 2j low, 2j + 1 high, in byte j) and the scale's bits
__device__ __forceinline__ uint2 quantise(const float (&x)[16], float inv6g, float g,
                                          uint32_t* scale_bits) {
  float m = 0.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    m = fmaxf(m, fabsf(x[i]));
    fine &= fabsf(x[i]) <= 3.402823466e38f;
  }
  const uint32_t bits = fine ? to_e4m3(fminf(m * inv6g, 448.f)) : 0x7Fu;
  *scale_bits = bits;
  const float s = from_e4m3(bits) * g;
  uint2 codes = make_uint2(0u, 0u);
  if (s > 0.f) {  // neither zero nor NaN
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = to_e2m1x2(x[2 * j] / s, x[2 * j + 1] / s);
      if (j < 4) codes.x |= c << (8 * j); else codes.y |= c << (8 * (j - 4));
    }
  }
  return codes;
}

// The values that codes stand for, as bf16
__device__ __forceinline__ void store_values(__nv_bfloat16* to, uint2 codes, uint32_t scale_bits,
                                             float g) {
  const float s = from_e4m3(scale_bits) * g;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = from_e2m1x2(((j < 4 ? codes.x : codes.y) >> (8 * (j & 3))) & 0xFFu);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// The four-bit codes 4k .. 4k + 3 of `codes`, each in the low half of a byte
__device__ __forceinline__ uint32_t spread(uint2 codes, int k) {
  const uint32_t w = ((k < 2 ? codes.x : codes.y) >> (16 * (k & 1))) & 0xFFFFu;
  return (w & 0xFu) | ((w & 0xF0u) << 4) | ((w & 0xF00u) << 8) | ((w & 0xF000u) << 12);
}

template <typename T, int D>
__global__ void __launch_bounds__(kApThreads) append_kernel(AppendParams P) {
  constexpr int S = D / 16;  // scales of a token
  const long long items = static_cast<long long>(P.T) * P.H * S;
  const long long it = static_cast<long long>(blockIdx.x) * kApThreads + threadIdx.x;
  if (it >= 2 * items) return;
  const bool is_v = it >= items;
  const long long r = is_v ? it - items : it;
  const int sb = static_cast<int>(r % S);
  const long long th = r / S;
  const int h = static_cast<int>(th % P.H);
  const int t = static_cast<int>(th / P.H);
  const long long slot = P.slots[t];
  const long long most = static_cast<long long>(P.num_pages) * P.ps;
  const bool writes = slot >= 0 && slot < most;
  const int nb = P.ps / 16;
  auto block_of = [&](long long s) {
    const long long page = s / P.ps;
    const int in = static_cast<int>(s - page * P.ps);
    return P.cache + ((page * P.H + h) * nb + (in >> 4)) * KvBlock<D>::kBytes;
  };
  const long long out_at = (static_cast<long long>(t) * P.H + h) * D + 16 * sb;
  float x[16];
  uint32_t sc;
  if (!is_v) {
    load16(static_cast<const T*>(P.k) + t * P.ks + static_cast<long long>(h) * D + 16 * sb, x);
    const uint2 codes = quantise(x, P.ik, P.gk, &sc);
    if (writes) {
      unsigned char* blk = block_of(slot);
      const int i = static_cast<int>(slot & 15);
      *reinterpret_cast<uint2*>(blk + KvBlock<D>::kKeyCodes + i * (D / 2) + 8 * sb) = codes;
      blk[KvBlock<D>::kKeyScales + i * S + sb] = static_cast<unsigned char>(sc);
    }
    if (P.ok) store_values(P.ok + out_at, codes, sc, P.gk);
    return;
  }
  const bool with_next = writes && !(slot & 1) && slot + 1 < most && t + 1 < P.T &&
                         P.slots[t + 1] == slot + 1;
  const bool with_prev = writes && (slot & 1) && t > 0 && P.slots[t - 1] == slot - 1;
  if (with_prev) return;  // the even token's thread does this one too
  const T* src = static_cast<const T*>(P.v) + t * P.vs + static_cast<long long>(h) * D + 16 * sb;
  load16(src, x);
  const uint2 codes = quantise(x, P.iv, P.gv, &sc);
  if (P.ov) store_values(P.ov + out_at, codes, sc, P.gv);
  if (!writes) return;
  unsigned char* blk = block_of(slot);
  const int p = static_cast<int>(slot & 15) >> 1;
  unsigned char* line = blk + KvBlock<D>::kValCodes + p * D;
  unsigned char* scales = blk + KvBlock<D>::kValScales + (p * S + sb) * 2;
  uint32_t w[4];
  if (with_next) {
    uint32_t sc2;
    load16(src + P.vs, x);
    const uint2 odd = quantise(x, P.iv, P.gv, &sc2);
    if (P.ov) store_values(P.ov + out_at + static_cast<long long>(P.H) * D, odd, sc2, P.gv);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = spread(codes, k) | (spread(odd, k) << 4);
    *reinterpret_cast<uint16_t*>(scales) = static_cast<uint16_t>(sc | (sc2 << 8));
    if (D == 128) {
      *reinterpret_cast<uint4*>(line + 16 * KvBlock<D>::place(p, sb)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    } else {  // a scale covers two chunks of 8 bytes
      *reinterpret_cast<uint2*>(line + 8 * KvBlock<D>::place(p, 2 * sb)) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(line + 8 * KvBlock<D>::place(p, 2 * sb + 1)) =
          make_uint2(w[2], w[3]);
    }
    return;
  }
  const int sh = (slot & 1) ? 4 : 0;
  scales[slot & 1] = static_cast<unsigned char>(sc);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = D == 128 ? 16 * KvBlock<D>::place(p, sb) + 4 * k
                            : 8 * KvBlock<D>::place(p, 2 * sb + (k >> 1)) + 4 * (k & 1);
    uint32_t* word = reinterpret_cast<uint32_t*>(line + at);
    atomicAnd(word, ~(0x0F0F0F0Fu << sh));
    atomicOr(word, spread(codes, k) << sh);
  }
}

template <typename T, int D>
cudaError_t launch_append(const AppendParams& P, cudaStream_t s) {
  const long long threads = 2LL * P.T * P.H * (D / 16);
  const long long grid = (threads + kApThreads - 1) / kApThreads;
  append_kernel<T, D><<<static_cast<unsigned>(grid), kApThreads, 0, s>>>(P);
  return cudaGetLastError();
}

bool row_aligned(const void* p, long long stride, size_t elt) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
         (stride * static_cast<long long>(elt)) % 16 == 0;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_kv4_page_bytes(int page_size, int D) {
  if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(D)) return 0;
  return static_cast<size_t>(page_size) * static_cast<size_t>(D + D / 8);
}

extern "C" sv_status spec_kv4_append(int T, int Hkv, int D, int page_size, int num_pages,
                                     sv_dtype dtype, const void* k, long long k_token_stride,
                                     const void* v, long long v_token_stride,
                                     const int64_t* slots, float k_scale, float v_scale,
                                     void* cache, void* out_k, void* out_v, void* stream) {
  if (T < 0 || Hkv < 1 || D < 1 || num_pages < 1) return SV_ERR_INVALID_ARG;
  if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_INVALID_ARG;
  if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
    return SV_ERR_INVALID_ARG;
  if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(D)) return SV_ERR_UNSUPPORTED;
  const long long row = static_cast<long long>(Hkv) * D;
  if (k_token_stride < row || v_token_stride < row) return SV_ERR_INVALID_ARG;
  if (T == 0) return SV_OK;
  if (!k || !v || !slots || !cache) return SV_ERR_INVALID_ARG;
  const size_t elt = dtype == SV_DTYPE_BF16 ? 2 : 4;
  if (!sv::row_aligned(k, k_token_stride, elt) || !sv::row_aligned(v, v_token_stride, elt) ||
      !sv::row_aligned(cache, 0, 1) || !sv::row_aligned(out_k, 0, 1) ||
      !sv::row_aligned(out_v, 0, 1))
    return SV_ERR_INVALID_ARG;
  if (2LL * T * Hkv * (D / 16) > (1LL << 38)) return SV_ERR_UNSUPPORTED;  // the grid's size
  sv::AppendParams P;
  P.T = T;
  P.H = Hkv;
  P.ps = page_size;
  P.num_pages = num_pages;
  P.ks = k_token_stride;
  P.vs = v_token_stride;
  P.k = k;
  P.v = v;
  P.slots = slots;
  P.gk = k_scale;
  P.gv = v_scale;
  P.ik = static_cast<float>(1.0 / (6.0 * static_cast<double>(k_scale)));
  P.iv = static_cast<float>(1.0 / (6.0 * static_cast<double>(v_scale)));
  P.cache = static_cast<unsigned char*>(cache);
  P.ok = static_cast<__nv_bfloat16*>(out_k);
  P.ov = static_cast<__nv_bfloat16*>(out_v);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SV_DTYPE_BF16)
    e = D == 128 ? sv::launch_append<__nv_bfloat16, 128>(P, s)
                 : sv::launch_append<__nv_bfloat16, 64>(P, s);
  else
    e = D == 128 ? sv::launch_append<float, 128>(P, s) : sv::launch_append<float, 64>(P, s);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
