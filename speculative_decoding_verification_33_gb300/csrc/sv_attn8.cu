// Causal attention of each sequence's new tokens over the 8-bit paged cache (spec_kv8_attention), with
// the kernel of sv_attn_mma.cuh; sv_attn.cu explains its structure.
//
// Codes become float16 in two instructions a pair: a byte under 0x64 is 1024 + code + 128, less 1152 the
// code, exact. A word of key codes is four neighbouring values of a token, what a step of the inner
// dimension takes of a thread; value codes lie as pairs of tokens, so that two bytes are one operand
// register. The exponents of a block cost no operand anything. That of its keys joins the factor of the
// scores. That of its values joins the exponent of the weights: with t = score + e (base 2) and M the running
// maximum of t, outputs are sums of 2^(t - M) code, and the softmax's sum is that of 2^(t - M) 2^-e, which is
// sum of 2^(score - M): maxima and the log-sum stay as they are, and joins but for the sums' range (times_two_to in
// sv_attn.cuh).
//
// What bounds it, as with 4 bits, is latency: with 20 rows of 524301 tokens, 8 heads of 128, it takes 234 us,
// 0.68 of the measured copy rate, with 0.53 of the issue slots and 0.36 of the tensor pipe used, and fixed
// latencies and the pairs' barriers the largest stalls; 64 sequences of up to 8192 tokens and up to 24 rows
// 104 us. The cut of the work (kOver, kLeast) is at its best here: kOver 48 and 200 take 106 and 107 us for
// these, kLeast 4 and 16 12.9 and 12.8 us for one row of 4097 tokens where 12 takes 11.8. Exponents of values of the
// whole range cost 1 to 4 %: without what add_quiet and times_two_to do these take 231 and 103 us, and 100 sequences
// of up to 4000 tokens, 32 rows of heads of 64, 25.6 instead of 26.7.
#include "spec_kv.h"
#include "sv_attn_mma.cuh"

namespace sv {
namespace {

// Bytes of `w` under 0x64, less 1152: codes as float16. `sel` picks two bytes.
template <uint32_t sel>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(0xE480E480u));
  return r;
}

// A thread's key codes of the tokens g and g + 8 of a block: values c D/4 .. c D/4 + D/4 - 1
template <int D>
struct KeyCodes8 {
  uint32_t a[D / 16], b[D / 16];
  __device__ __forceinline__ void load(const unsigned char* blk, int g, int c) {
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const unsigned char* p = blk + g * D + 16 * Kv8Block<D>::key_place(g, D / 64 * c + i);
      *reinterpret_cast<uint4*>(a + 4 * i) = *reinterpret_cast<const uint4*>(p);
      *reinterpret_cast<uint4*>(b + 4 * i) = *reinterpret_cast<const uint4*>(p + 8 * D);
    }
  }
  __device__ __forceinline__ void operands(int i, uint32_t (&f)[1][4]) const {
    f[0][0] = code_pair<0x4140>(a[i]);
    f[0][1] = code_pair<0x4140>(b[i]);
    f[0][2] = code_pair<0x4342>(a[i]);
    f[0][3] = code_pair<0x4342>(b[i]);
  }
};

// Half h of a thread's values of a block: D / 16 values of the token pairs c and c + 4
template <int D>
struct ValueCodes8 {
  static constexpr int N = D / 32;  // words of one pair's codes
  uint32_t a[N], b[N];
  __device__ __forceinline__ void load(const unsigned char* blk, int g, int c, int h) {
    const unsigned char* p = blk + Kv8Block<D>::kValCodes + c * 2 * D;
    if (D == 128) {
      p += 16 * Kv8Block<D>::val_place(c, 8 * h + g);
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(p);
      *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(p + 8 * D);
    } else {
      p += 16 * Kv8Block<D>::val_place(c, 4 * h + (g >> 1)) + 8 * (g & 1);
      *reinterpret_cast<uint2*>(a) = *reinterpret_cast<const uint2*>(p);
      *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(p + 8 * D);
    }
  }
  __device__ __forceinline__ void operands(uint32_t (&f)[D / 32][4]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[i][0] = code_pair<0x4140>(a[i]);
      f[i][1] = code_pair<0x4342>(a[i]);
      f[i][2] = code_pair<0x4140>(b[i]);
      f[i][3] = code_pair<0x4342>(b[i]);
    }
  }
};

// The head of a block: exponents, and marks of its keys (low half) and values.
struct Head8 {
  float scale, lift, undo;  // 2^e of the keys; e of the values, 2^-e
  int e;                    // of the values
  uint32_t marks;
  template <int D>
  __device__ __forceinline__ void read(const unsigned char* blk, bool lost) {
    uint2 w = *reinterpret_cast<const uint2*>(blk + Kv8Block<D>::kHead);
    if (lost) w = make_uint2(0u, 0u);
    const int ek = static_cast<signed char>(w.x & 0xFFu), ev = static_cast<signed char>((w.x >> 8) & 0xFFu);
    scale = __int_as_float((ek + 127) << 23);
    e = ev;
    lift = static_cast<float>(ev);
    undo = __int_as_float((127 - ev) << 23);
    marks = w.y;
  }
  // Factors of the scores of two rows: held, so that a sum of 0 stays 0 and no other gets smaller than
  // what decides the softmax by itself
  __device__ __forceinline__ float2 key_scale(float2 qc) const {
    const float most = 1.2676506e30f;  // 2^100
    return make_float2(fminf(fmaxf(qc.x * scale, -most), most), fminf(fmaxf(qc.y * scale, -most), most));
  }
};

template <int D_>
struct Kv8 {
  static constexpr int D = D_;
  static constexpr bool kHeads = true;
  static constexpr int kBlock = Kv8Block<D>::kBytes;
  static constexpr int kSteps = 1;
  using Keys = KeyCodes8<D>;
  using Values = ValueCodes8<D>;
  static __device__ __forceinline__ uint2 head(const unsigned char* blk) {
    return *reinterpret_cast<const uint2*>(blk + Kv8Block<D_>::kHead);
  }
  static __device__ __forceinline__ int lift(uint2 head) { return static_cast<signed char>((head.x >> 8) & 0xFFu); }
  struct Head : Head8 {
    __device__ __forceinline__ void load(const unsigned char* blk, bool lost) { read<D_>(blk, lost); }
  };
  static __device__ __forceinline__ uint32_t marks(const unsigned char* blk) {
    return *reinterpret_cast<const uint32_t*>(blk + Kv8Block<D_>::kHead + 4);
  }
  static __device__ __forceinline__ int first_value(int g, int h) { return (D / 2) * h + (D / 16) * g; }
  template <int NT>
  static constexpr int kOwn = 1;
  template <int NT>
  static constexpr int kStages = 2 * (128 / D);
  static constexpr int kOver = 96;
  static __host__ __device__ constexpr int cost(int tiles) {
    return tiles <= 1 ? 5 : tiles == 2 ? 6 : tiles == 3 ? 8 : 10;
  }
  template <int NT>
  static constexpr int kLeast = 12;
};

// Rows of a tile, at most: with 32 of D = 128 the kernel spills.
template <int D>
constexpr int kMaxRows8 = D == 128 ? 24 : 32;

// Rows a head, at most, for this kernel; those past a tile read the cache once more. It works for the rows that
// a sequence has, sv_attn8_tc.cu for 128. Measured in us, here / there, for 8 sequences of 16384 tokens and
// for 64 of up to 8192 with up to that many rows. D = 128, 8 heads: 24 rows 73 / 97 and 96 / 143; 32 rows
// 105 / 99 and 125 / 146; 48 rows 125 / 101 and 150 / 154; 64 rows 175 / 104 and 193 / 159; 20 rows of one
// sequence of 524301 tokens 232 / 335. D = 64, 2 heads: 32 rows 26 / 33; 64 rows 37 / 36 and 41 / 45; 96
// rows 46 / 40 and 53 / 48.
template <int D>
constexpr int kRegisterRows = D == 128 ? 32 : 64;

template <int D>
cudaError_t launch_dim8(const AttnParams& P, long long all, int sms, cudaStream_t stream) {
  // rows of a tile: a sequence's rows in as few tiles as hold them, evenly
  const long long tiles = (all + kMaxRows8<D> - 1) / kMaxRows8<D>;
  switch (((all + tiles - 1) / tiles + 7) / 8) {
    case 1: return launch_tiles<Kv8<D>, 1>(P, sms, stream);
    case 2: return launch_tiles<Kv8<D>, 2>(P, sms, stream);
    case 3: return launch_tiles<Kv8<D>, 3>(P, sms, stream);
  }
  if constexpr (kMaxRows8<D> > 24) return launch_tiles<Kv8<D>, 4>(P, sms, stream);
  return cudaErrorInvalidValue;  // not reached
}

}  // namespace

cudaError_t launch_attention8(const AttnParams& P, int D, int max_new, int sms, cudaStream_t stream) {
  const long long all = std::max(1LL, static_cast<long long>(max_new) * P.group);
  if (all > (D == 64 ? kRegisterRows<64> : kRegisterRows<128>)) return launch_attention8_tc(P, D, all, sms, stream);
  return D == 64 ? launch_dim8<64>(P, all, sms, stream) : launch_dim8<128>(P, all, sms, stream);
}

}  // namespace sv
