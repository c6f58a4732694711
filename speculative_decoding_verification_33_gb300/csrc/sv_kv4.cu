// Keys and values into the 4-bit paged cache (spec_kv4_append).
//
// A thread takes 16 neighbouring values of one token and head, which share a scale: their maximum
// needs no other thread. Keys then are 8 bytes of codes and a scale byte. A byte of value codes
// holds two tokens, the even slot low: where the call brings both tokens of a pair one after the
// other, the even token's thread quantises both and stores 16 bytes; a token alone sets its four
// bits of each byte with a pair of atomics on 32-bit words, which leaves the other token's bits
// alone, whoever else writes the word. Bits of different tokens never meet, so the order of the
// atomics does not matter.
//
// 65013 tokens of 8 heads of 128 in bf16 (608 MB read and written, the values as they are held
// among them) take 119 us, 0.75 of the measured copy rate; the quantisation's instructions and the
// scattered lines of 16 to 64 bytes share the rest. 384 tokens take 3.2 us, which is the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "spec_kv.h"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kApThreads = 256;

struct AppendParams {
  int T, H, num_pages;
  int ps_log;  // page_size = 2^ps_log
  int plain;   // tensor scales near enough to 1 for the quotient's short form
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
// Eight values -> four bytes of e2m1 codes, value 2j in the low four bits of byte j; nearest even,
// held at 6
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}
// ... and back, as float16 pairs
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// 16 values -> 8 bytes of codes (value 2j low, 2j + 1 high, in byte j) and the scale's bits. The codes
// are those of the quotients x / s of IEEE division. Where nothing can overflow (`plain`: the tensor scale
// is within 2^+-60, so the scale s = e4m3 * g and 1 / s are normal, and |x| < 9 s, the bound of the smallest
// scale, unless the block's scale is held at 448) they come from one division for the block and
// Markstein's correction for each value: with y = RN(1 / s) and q = RN(x y), RN(q + (x - q s) y), two
// fused operations, is RN(x / s) if q is within a unit in the last place of x / s (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990). At the thresholds
// between codes, whose mantissas are at most 1.75, x y is off by less than 0.9 units: where x / s lies next
// to the middle of two floats, q is one of these two and the theorem holds. Elsewhere q may be off by 1.5
// units and the corrected sum by 3 * 2^-24 units before its rounding, which reaches no middle. The sum is
// written as q - (q s - x) y: it keeps the sign of a zero, as x / s does, where q + (x - q s) y gives +0
// for x = -0.
// 16 divisions made the kernel issue-bound: 65013 tokens of 8 heads took 149 us instead of 119.
__device__ __forceinline__ uint2 quantise(const float (&x)[16], float inv6g, float g, bool plain,
                                          uint32_t* scale_bits) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) m = max_nan(m, fabsf(x[i]));
  const uint32_t bits = m <= 3.402823466e38f ? to_e4m3(fminf(m * inv6g, 448.f)) : 0x7Fu;
  *scale_bits = bits;
  const float s = from_e4m3(bits) * g;
  uint2 codes = make_uint2(0u, 0u);
  if (s > 0.f) {  // neither zero nor NaN
    float t[16];
    if (plain && bits < 0x7Eu) {
      const float y = 1.f / s;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float q = x[i] * y;
        t[i] = fmaf(-fmaf(q, s, -x[i]), y, q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = x[i] / s;
    }
    codes = make_uint2(to_e2m1x8(t), to_e2m1x8(t + 8));
  }
  return codes;
}

// The values that codes stand for, as bf16
__device__ __forceinline__ void store_values(__nv_bfloat16* to, uint2 codes, uint32_t scale_bits,
                                             float g) {
  const float s = from_e4m3(scale_bits) * g;
  uint32_t w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f[4];
    from_e2m1x8(h ? codes.y : codes.x, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
      const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * s, v.y * s);
      w[4 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
    }
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
  const uint32_t items = static_cast<uint32_t>(P.T) * P.H * S;
  const uint32_t r = blockIdx.x * kApThreads + threadIdx.x;
  if (r >= items) return;
  const bool is_v = blockIdx.y;
  const int sb = static_cast<int>(r % S);
  const uint32_t th = r / S;
  const int t = static_cast<int>(th / static_cast<uint32_t>(P.H));
  const int h = static_cast<int>(th - static_cast<uint32_t>(t) * P.H);
  const long long slot = P.slots[t];
  const long long most = static_cast<long long>(P.num_pages) << P.ps_log;
  const bool writes = slot >= 0 && slot < most;
  auto block_of = [&](long long s) {
    const int in = static_cast<int>(s) & ((1 << P.ps_log) - 1);
    return P.cache + ((((s >> P.ps_log) * P.H + h) << (P.ps_log - 4)) + (in >> 4)) * KvBlock<D>::kBytes;
  };
  const long long out_at = static_cast<long long>(th) * D + 16 * sb;
  float x[16];
  uint32_t sc;
  if (!is_v) {
    load16(static_cast<const T*>(P.k) + t * P.ks + static_cast<long long>(h) * D + 16 * sb, x);
    const uint2 codes = quantise(x, P.ik, P.gk, P.plain, &sc);
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
  const uint2 codes = quantise(x, P.iv, P.gv, P.plain, &sc);
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
    const uint2 odd = quantise(x, P.iv, P.gv, P.plain, &sc2);
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
  const long long threads = static_cast<long long>(P.T) * P.H * (D / 16);
  const dim3 grid(static_cast<unsigned>((threads + kApThreads - 1) / kApThreads), 2);  // keys, values
  append_kernel<T, D><<<grid, kApThreads, 0, s>>>(P);
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
  if (static_cast<long long>(T) * Hkv * (D / 16) >= (1LL << 31)) return SV_ERR_UNSUPPORTED;  // 32-bit items
  sv::AppendParams P;
  P.T = T;
  P.H = Hkv;
  P.ps_log = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  const float lo = 8.6736174e-19f, hi = 1.1529215e18f;  // 2^-60, 2^60
  P.plain = k_scale >= lo && k_scale <= hi && v_scale >= lo && v_scale <= hi;
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
