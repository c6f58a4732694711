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
#include "spec_kv.h"
#include "sv_attn_mma.cuh"

namespace sv {
namespace {

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

// What attn_kernel asks of a format.
template <int D_>
struct Kv4 {
  static constexpr int D = D_;
  static constexpr bool kHeads = false;  // blocks have exponents and marks of their own
  static constexpr int kBlock = KvBlock<D>::kBytes;
  static constexpr int kSteps = 2;  // steps of the inner dimension of one call of Keys::operands
  using Keys = KeyCodes<D>;
  using Values = ValueCodes<D>;
  struct Head {
    __device__ __forceinline__ void load(const unsigned char*, bool) {}
  };
  static __device__ __forceinline__ uint32_t marks(const unsigned char*) { return 0; }
  // the first of a thread's values of the outputs
  static __device__ __forceinline__ int first_value(int g, int h) { return (D / 8) * g + (D / 16) * h; }
  // Blocks of a unit for each warp of a pair. With one tile of rows there are registers for two: half
  // the barriers, 122 us (now 114) instead of 135 for 524301 tokens of 8 heads and 4 rows, 58 instead of 61 for
  // 64 sequences of up to 8192. With two tiles that takes 160 instead of 168 us and 75 instead of
  // 72.5, and for 256 sequences of up to 1024 tokens 78 instead of 68.
  template <int NT>
  static constexpr int kOwn = NT == 1 ? 2 : 1;
  template <int NT>
  static constexpr int kStages = (kOwn<NT> == 1 ? 3 : 2) * (128 / D);
  // Work as it is cut: 524301 tokens of 8 heads take 135, 168, 215 and 287 us with 1 to 4 tiles and
  // one block a warp. With an item's start and end for nothing, 64 sequences of up to 8192 tokens, 24
  // rows a head, take 113 us and 256 of up to 1024 tokens 135 us; for 96, 89 and 86 us.
  static constexpr int kOver = 96;
  static __host__ __device__ constexpr int cost(int tiles) {
    return tiles <= 1 ? 5 : tiles == 2 ? 6 : tiles == 3 ? 8 : 10;
  }
  // Every pair of a CTA gets three units or so at least: with one, more pieces are to be joined, and
  // one request of 4000 tokens, 24 rows a head, takes 21.9 us instead of 17.6
  template <int NT>
  static constexpr int kLeast = 12 / kOwn<NT>;
};

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
    case 1: return launch_tiles<Kv4<D>, 1>(P, sms, stream);
    case 2: return launch_tiles<Kv4<D>, 2>(P, sms, stream);
    case 3: return launch_tiles<Kv4<D>, 3>(P, sms, stream);
  }
  if constexpr (kMaxRows<D> > 24) return launch_tiles<Kv4<D>, 4>(P, sms, stream);
  return cudaErrorInvalidValue;  // not reached
}

}  // namespace

size_t attention_workspace_bytes(int sms) {
  // two pieces a CTA, of at most kPieceRows rows with one CTA an SM, half as many with two
  return kAttnHeader + static_cast<size_t>(sms) * 2 * kPieceRows * (128 + 2) * sizeof(float);
}

cudaError_t launch_attention(const AttnParams& P, int D, int max_new, int sms,
                             cudaStream_t stream) {
  const long long all = std::max(1LL, static_cast<long long>(max_new) * P.group);
  if (D == 64) return launch_dim<64>(P, all, sms, stream);
  return all <= kMaxRows<128> ? launch_dim<128>(P, all, sms, stream) : launch_attention_tc(P, sms, stream);
}

}  // namespace sv
