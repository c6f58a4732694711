// Keys and values into the 8-bit paged cache (spec_kv8_append).
//
// A block of 16 tokens of a head shares an exponent, so whoever writes one of its tokens has to see them
// all: a warp takes all tokens of the call that fall into one block (they lie together), for one head
// and keys or values. It loads their rows in the order of their places, eight values a lane, takes the
// maximum, joins it with the exponent that the block has, and writes codes. Only where the exponent grows
// or the block starts afresh does it touch the block's other places. Rows of D = 128 are 16 lanes, so that
// an instruction covers the two tokens of a pair; the two lanes that hold the same values of both exchange
// them, and each writes one pair's 16 bytes.
//
// Codes come from a product and a sum: x 2^-e + 1.5 * 2^23 + 128 is rounded to an integer, to nearest
// with ties to even, and its low byte is the code plus 128. The product with a power of two is exact.
//
// What bounds it: HBM for prompts (13 of 5001 tokens, 8 heads of 128, bf16: 114 us, 0.86 of the measured copy
// rate; blocks of 128 threads at 64 registers took 118 where 256 at 80 took 126, and old codes rounded in a
// loop of their own 114); for small calls the chain of slots, rows, maximum and stores of one block.
// Steps whose places bring nothing are left out (one token of each of 384 sequences, 8 heads: 11.0 -> 7.8 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_kv.h"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr int kThreads8 = 128;
constexpr float kMagic = 12582912.f + 128.f;  // 1.5 * 2^23: its unit in the last place is 1

struct Append8Params {
  int T, H, num_pages;
  int ps_log;     // page_size = 2^ps_log
  int group_log;  // a warp looks at 2^group_log tokens for the first one of a block
  long long ks, vs;
  const void *k, *v;
  const int64_t* slots;
  unsigned char* cache;
  __nv_bfloat16 *ok, *ov;
};

// Eight values of a row
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&a.x)[i >> 1];
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  // bits of the largest magnitude, those of NaN and infinity above all others
  __device__ __forceinline__ uint32_t most() const {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t x = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
    return max(x & 0xFFFF0000u, x << 16);
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? (&a.x)[i & 3] : (&b.x)[i & 3]; }
  __device__ __forceinline__ uint32_t most() const {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x = max(x, __float_as_uint(get(i)) & 0x7FFFFFFFu);
    return x;
  }
};

__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }  // -126..127

// The smallest exponent of kKv8Low..kKv8High whose codes reach the magnitude with these bits:
// f * 2^p <= 127 * 2^e with f of 1..2 is f <= 127/64 for e = p - 6
__device__ __forceinline__ int exponent_for(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 133 + ((bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return min(max(e, kKv8Low), kKv8High);
}

// Low bytes of four floats' bits
__device__ __forceinline__ uint32_t low_bytes(const float* t) {
  const uint32_t a = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}
// Codes of four bytes, as floats
__device__ __forceinline__ void codes_of(uint32_t w, float* c) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)) - (8388608.f + 128.f);
}
// [a0 b0 a1 b1 a2 b2 a3 b3] of the bytes of two words
__device__ __forceinline__ uint2 interleave(uint32_t a, uint32_t b) {
  return make_uint2(__byte_perm(a, b, 0x5140), __byte_perm(a, b, 0x7362));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads8, sizeof(T) == 2 ? 8 : 5) append8_kernel(Append8Params P) {
  using B = Kv8Block<D>;
  constexpr int LP = D / 8;    // lanes of a token
  constexpr int TP = 32 / LP;  // tokens at a time
  constexpr int N = 16 / TP;
  __shared__ unsigned char s_from[kThreads8 / 32][16];
  const int lane = threadIdx.x & 31;
  unsigned char* from = s_from[threadIdx.x >> 5];
  const long long warp = static_cast<long long>(blockIdx.x) * (kThreads8 / 32) + (threadIdx.x >> 5);
  const bool is_v = blockIdx.y & 1;
  const int h = blockIdx.y >> 1;
  const long long t0 = warp << P.group_log;
  if (t0 >= P.T) return;
  const long long most = static_cast<long long>(P.num_pages) << P.ps_log;
  __nv_bfloat16* out = is_v ? P.ov : P.ok;
  auto block_no = [&](long long s) { return s >= 0 && s < most ? s >> 4 : -1LL; };

  // The tokens of this group that are the first of a block: the last token before it that is written, of the
  // 32 before, is of another block. Tokens that are not written stand for themselves, and for
  // nothing where no values are wanted.
  uint32_t starts = 0;
  const long long slot0 = t0 + lane < P.T ? P.slots[t0 + lane] : -1;  // of 64 tokens
  const long long slot1 = P.group_log && t0 + 32 + lane < P.T ? P.slots[t0 + 32 + lane] : -1;
  {
    const long long t = t0 + lane;
    const long long now = block_no(slot0);
    const long long before = t >= 32 ? block_no(P.slots[t - 32]) : -1;
    const uint32_t is_now = __ballot_sync(0xFFFFFFFFu, now >= 0), is_before = __ballot_sync(0xFFFFFFFFu, before >= 0);
    const uint32_t lower = (1u << lane) - 1u;
    const uint32_t below = is_now & lower, above = is_before & ~lower;
    const int last = 31 - __clz(below ? below : above);
    const long long one = __shfl_sync(0xFFFFFFFFu, now, last & 31), other = __shfl_sync(0xFFFFFFFFu, before, last & 31);
    const bool goes_on = now >= 0 && (below ? one == now : above && other == now);
    starts = __ballot_sync(0xFFFFFFFFu, lane < (1 << P.group_log) && t < P.T && !goes_on && (now >= 0 || out));
  }
  const T* src = static_cast<const T*>(is_v ? P.v : P.k);
  const long long stride = is_v ? P.vs : P.ks;
  const int j0 = lane / LP, l = lane % LP;  // token of the instruction, place in its row

  while (starts) {
    __syncwarp();  // `from` is read
    const int off = __ffs(starts) - 1;  // below 2^group_log
    const long long t = t0 + off;
    starts &= starts - 1;
    // lane i: the token t + i, if it is of the same block and no token of another one comes before
    const long long near = __shfl_sync(0xFFFFFFFFu, slot0, (off + lane) & 31);
    const long long far = __shfl_sync(0xFFFFFFFFu, slot1, (off + lane) & 31);
    const long long slot = off + lane < 32 ? near : far;
    const long long no = block_no(slot), blk = __shfl_sync(0xFFFFFFFFu, no, 0);
    const uint32_t ends = __ballot_sync(0xFFFFFFFFu, no >= 0 && no != blk);
    const bool mine = blk < 0 ? lane == 0 : no == blk && !(ends & ((1u << lane) - 1u));
    const int place = blk >= 0 ? static_cast<int>(slot & 15) : 0;
    if (mine) from[place] = static_cast<unsigned char>(lane);  // which of them comes to a place
    const uint32_t there = __reduce_or_sync(0xFFFFFFFFu, mine ? 1u << place : 0u);  // the places written
    __syncwarp();

    Row8<T> x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int p = TP * j + j0;
      x[j].zero();
      if ((there >> p) & 1u) x[j].load(src + (t + from[p]) * stride + static_cast<long long>(h) * D + 8 * l);
    }
    unsigned char* to = nullptr;
    int had = kKv8Low;
    uint32_t marks = 0;
    if (blk >= 0) {
      const int bpp_log = P.ps_log - 4;
      to = P.cache + ((((blk >> bpp_log) * P.H + h) << bpp_log) + (blk & ((1 << bpp_log) - 1))) * B::kBytes;
      had = min(max(static_cast<int>(reinterpret_cast<const signed char*>(to + B::kHead)[is_v]), kKv8Low),
                kKv8High);
      marks = reinterpret_cast<const uint16_t*>(to + B::kHead + 4)[is_v];
    }
    const bool fresh = blk < 0 || (there & 1u);

    // Steps whose places bring nothing are left out, the same ones in all lanes
    auto any = [&](uint32_t places, int j) { return (places >> (TP * j)) & ((1u << TP) - 1u); };
    // marks, and the largest magnitude of the tokens without one
    uint32_t bad = 0, top = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!any(there, j)) continue;
      const uint32_t m = x[j].most();
      const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, m >= 0x7F800000u);
      const bool marked = (lanes >> (lane - l)) & ((1ull << LP) - 1);
#pragma unroll
      for (int i = 0; i < TP; ++i)
        if ((lanes >> (i * LP)) & ((1u << LP) - 1)) bad |= 1u << (TP * j + i);
      if (marked) x[j].zero(); else top = max(top, m);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    const int need = exponent_for(top);
    const int e = fresh ? need : max(need, had);
    const bool again = !fresh && e > had;  // the other places' codes are rounded again
    const float scale = two_to(-e), step = two_to(e);
    if (again) {  // all codes that are there, for the tokens of this call are written after them
      const float down = two_to(max(had - e, -126));
      unsigned char* codes = to + (is_v ? B::kValCodes : B::kKeyCodes) + 16 * lane;
#pragma unroll 1
      for (int at = 0; at < 16 * D; at += 512) {
        uint4 w = *reinterpret_cast<const uint4*>(codes + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[4];
          codes_of((&w.x)[q], y);
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = fmaxf(y[i] * down, -127.f) + kMagic;
          (&w.x)[q] = low_bytes(y);
        }
        *reinterpret_cast<uint4*>(codes + at) = w;
      }
      __syncwarp();
    }

    // codes plus 128, eight a lane; `known`: places whose bytes are to be written
    uint2 c[N];
    const uint32_t known = fresh ? 0xFFFFu : there;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int p = TP * j + j0;
      c[j] = make_uint2(0u, 0u);
      if (!any(known, j)) continue;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = x[j].get(i) * scale;
        if (e == kKv8High) v = fminf(fmaxf(v, -127.f), 127.f);
        y[i] = v + kMagic;
      }
      c[j] = make_uint2(low_bytes(y), low_bytes(y + 4));
      if (out && ((there >> p) & 1u)) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn((y[2 * i] - kMagic) * step, (y[2 * i + 1] - kMagic) * step);
          w[i] = (bad >> p) & 1u ? 0x7FFF7FFFu : *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(out + ((t + from[p]) * P.H + h) * D + 8 * l) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (blk < 0) continue;

    if (!is_v) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int p = TP * j + j0;
        if (any(known, j) && ((known >> p) & 1u))
          *reinterpret_cast<uint2*>(to + B::kKeyCodes + p * D + 16 * B::key_place(p, l >> 1) + 8 * (l & 1)) = c[j];
      }
    } else {
      // pairs: of two instructions, lanes of even tokens write the first one's, those of odd ones the second's
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        if (!any(known, j) && !any(known, j + 1)) continue;
        const bool odd = j0 & 1;
        const uint2 give = odd ? c[j] : c[j + 1], keep = odd ? c[j + 1] : c[j];
        uint2 got;
        got.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, LP);
        got.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, LP);
        const int pair = (TP * (odd ? j + 1 : j) + j0) >> 1;
        const uint2 ev = odd ? got : keep, od = odd ? keep : got;
        unsigned char* line = to + B::kValCodes + pair * 2 * D + 16 * B::val_place(pair, l);
        const uint2 lo = interleave(ev.x, od.x), hi = interleave(ev.y, od.y);
        const uint32_t both = (known >> (2 * pair)) & 3u;
        if (both == 3u) {
          *reinterpret_cast<uint4*>(line) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else if (both) {  // the other token's bytes stay
          const int at = both >> 1;
          const uint2 one = at ? od : ev;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            line[2 * i + at] = static_cast<unsigned char>((i < 4 ? one.x : one.y) >> (8 * (i & 3)));
        }
      }
    }
    if (lane == 0) {
      reinterpret_cast<signed char*>(to + B::kHead)[is_v] = static_cast<signed char>(e);
      reinterpret_cast<uint16_t*>(to + B::kHead + 4)[is_v] =
          static_cast<uint16_t>((fresh ? 0u : marks & ~there) | bad);
    }
  }
}

template <typename T, int D>
cudaError_t launch_append8(const Append8Params& P, cudaStream_t s) {
  const long long warps = (P.T + (1LL << P.group_log) - 1) >> P.group_log;
  const dim3 grid(static_cast<unsigned>((warps + kThreads8 / 32 - 1) / (kThreads8 / 32)), 2 * P.H);
  append8_kernel<T, D><<<grid, kThreads8, 0, s>>>(P);
  return cudaGetLastError();
}

bool row_aligned8(const void* p, long long stride, size_t elt) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * static_cast<long long>(elt)) % 16 == 0;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_kv8_page_bytes(int page_size, int D) {
  if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(D)) return 0;
  return static_cast<size_t>(page_size) * static_cast<size_t>(2 * D + 1);
}

extern "C" sv_status spec_kv8_append(int T, int Hkv, int D, int page_size, int num_pages,
                                     sv_dtype dtype, const void* k, long long k_token_stride,
                                     const void* v, long long v_token_stride,
                                     const int64_t* slots, void* cache, void* out_k, void* out_v,
                                     void* stream) {
  if (T < 0 || Hkv < 1 || D < 1 || num_pages < 1) return SV_ERR_INVALID_ARG;
  if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_INVALID_ARG;
  if (!sv::kv_page_size_ok(page_size) || !sv::kv_head_dim_ok(D)) return SV_ERR_UNSUPPORTED;
  const long long row = static_cast<long long>(Hkv) * D;
  if (k_token_stride < row || v_token_stride < row) return SV_ERR_INVALID_ARG;
  if (T == 0) return SV_OK;
  if (!k || !v || !slots || !cache) return SV_ERR_INVALID_ARG;
  const size_t elt = dtype == SV_DTYPE_BF16 ? 2 : 4;
  if (!sv::row_aligned8(k, k_token_stride, elt) || !sv::row_aligned8(v, v_token_stride, elt) ||
      !sv::row_aligned8(cache, 0, 1) || !sv::row_aligned8(out_k, 0, 1) || !sv::row_aligned8(out_v, 0, 1))
    return SV_ERR_INVALID_ARG;
  if (Hkv > 32767) return SV_ERR_UNSUPPORTED;  // the grid's second dimension
  sv::Append8Params P;
  P.T = T;
  P.H = Hkv;
  P.num_pages = num_pages;
  P.ps_log = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  // Tokens of a warp: many are few warps, and blocks that begin among them follow one another. Measured for 8
  // heads of 128, groups of 1, 2, 4 and 16 tokens: 384 tokens in a run 5.2, 4.7, 4.2, 4.2 us, six to a block
  // 5.2, 4.1, 4.1, 6.7, one to a block 7.8, 7.9, 9.2, 23.8; 1024 tokens 7.7, 6.1, 4.7, 4.6, then 8.6, 7.9,
  // 6.2, 7.7, then 14.9, 14.4, 14.4, 26.1; 4096 tokens 19.5, 13.9, 11.3, 8.2, then 23.5, 19.1, 15.4, 14.4, then
  // 49.2, 44.2, 42.6, 46.6.
  const long long rows = static_cast<long long>(T) * Hkv;
  P.group_log = rows < (1 << 13) ? 1 : rows < (1 << 15) ? 2 : 4;
  P.ks = k_token_stride;
  P.vs = v_token_stride;
  P.k = k;
  P.v = v;
  P.slots = slots;
  P.cache = static_cast<unsigned char*>(cache);
  P.ok = static_cast<__nv_bfloat16*>(out_k);
  P.ov = static_cast<__nv_bfloat16*>(out_v);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SV_DTYPE_BF16)
    e = D == 128 ? sv::launch_append8<__nv_bfloat16, 128>(P, s) : sv::launch_append8<__nv_bfloat16, 64>(P, s);
  else
    e = D == 128 ? sv::launch_append8<float, 128>(P, s) : sv::launch_append8<float, 64>(P, s);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
