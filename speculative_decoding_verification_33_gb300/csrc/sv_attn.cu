// Causal attention of each sequence's new tokens over the 4-bit paged cache (spec_kv4_attention).
//
// Everything that a sequence's rows (new tokens x query heads of one key/value head) need of the
// cache is read once for all of them: a block of 16 tokens is 18 D bytes, its products with R
// rows 64 D R operations. The unit of work is two blocks for one tile of R = 8 NT rows. All
// units of the call, sequence after sequence, are cut into equal runs, one per persistent CTA, so that the
// load is even whatever the lengths are; a head that is cut has its pieces joined by the last
// CTA that finishes one of them, in their order, so results do not depend on timing. The warps
// of a CTA take its units in turn, each with running maximum, sum and output of its own in
// registers, joined at the end of a run of the same head.
//
// Transposed products: scores^T = K q^T with 16 tokens as the rows of the matrix instruction
// (m16n8k16) and 8 query rows as its columns, outputs^T = V^T p^T with 16 values as rows. So few
// query rows waste nothing, and codes go from the cache's bytes to operands in registers: a
// byte of key codes is a pair of one token's values, a byte of value codes one value of two
// tokens, which is what the instruction takes in one register either way. e2m1 * e4m3 has at
// most 6 significant bits, exact in float16. The order of the inner dimension is free as long as both
// operands share it: thread c of a token takes values c D/4 .. c D/4 + D/4 - 1, in one load.
//
// Each warp streams its blocks through a ring in shared memory with bulk copies that it issues
// itself, some blocks ahead; no barrier spans the warps until a head ends.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "spec_kv.h"
#include "sv_kv.h"
#include "sv_ptx.cuh"

namespace sv {
namespace {

constexpr long long kWaitCycles = 4000000000LL;  // about 2 s: a copy that never came
constexpr float kLift = 7.f;    // weights are held times 2^7: float16 has more room above 1 than below
constexpr float kSlack = 15.f;  // and may grow to 2^15 before the running maximum is moved

constexpr int kUnit = 32;  // tokens of a unit: two blocks

template <int D, int NT>
struct AttnShape {
  static constexpr int kWarps = NT == 2 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPerSm = NT == 1 ? 2 : 1;   // CTAs an SM, by registers
  static constexpr int kRows = 8 * NT;
  static constexpr bool kJoint = D == 64 || NT == 1 || NT == 3;  // by registers
  static constexpr int kBlock = KvBlock<D>::kBytes;
  static constexpr int kStages = (NT <= 2 ? 2 : 3) * (128 / D);
  static constexpr int kStage = 2 * kBlock;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQ = NT * (D / 16) * 32 * 8;
  static constexpr int kOutStride = D + 4;  // floats of a row of the joining buffer
  static constexpr int kOut = kWarps * 8 * kOutStride * 4;
  static constexpr int kStat = 2 * kWarps * kRows * 4;
  static constexpr int kSmem = kRing + kQ + kOut + kStat + kRows * 8 + kWarps * kStages * 8;
  static constexpr int kPart = kRows * (D + 2);  // floats of one piece's results
};

// Where a run of units lies: item (sequence b, head h, row tile rt) with its nu units.
struct Walk {
  long long base;  // the item's first unit
  int b, h, rt;
  int rts, nu, len, n, r0;
};

__device__ __forceinline__ void load_seq(const AttnParams& P, int rows_tile, int b, Walk& w) {
  const int c0 = min(max(P.cu[b], 0), P.T), c1 = min(max(P.cu[b + 1], c0), P.T);
  w.b = b;
  w.r0 = c0;
  w.n = c1 - c0;
  w.len = min(max(P.lens[b], 0), P.max_blocks * P.ps);
  w.rts = (w.n * P.group + rows_tile - 1) / rows_tile;
  w.nu = max(1, (w.len + kUnit - 1) / kUnit);
}
__device__ __forceinline__ long long seq_units(const AttnParams& P, const Walk& w) {
  return static_cast<long long>(w.rts) * P.hkv * w.nu;
}
__device__ __forceinline__ void next_item(const AttnParams& P, int rows_tile, Walk& w) {
  w.base += w.nu;
  if (++w.rt < w.rts) return;
  w.rt = 0;
  if (++w.h < P.hkv) return;
  w.h = 0;
  int b = w.b;
  do {
    if (++b >= P.B) {
      w.b = P.B;
      w.nu = 1 << 30;  // nothing follows
      return;
    }
    load_seq(P, rows_tile, b, w);
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Keys of a block's 16 tokens as operands: token g in registers 0 and 2 of a step, g + 8 in 1 and 3
template <int D>
__device__ __forceinline__ void key_operands(const unsigned char* sb, int g, int c,
                                             uint32_t (&f)[D / 16][4]) {
  constexpr int N = D / 32;  // words of a thread's codes of one token
  uint32_t ka[N], kb[N], sa[2], sc[2];
  if (D == 128) {
    *reinterpret_cast<uint4*>(ka) = *reinterpret_cast<const uint4*>(sb + g * 64 + c * 16);
    *reinterpret_cast<uint4*>(kb) = *reinterpret_cast<const uint4*>(sb + g * 64 + 512 + c * 16);
    const uint32_t x = e4m3x2(*reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kKeyScales + g * 8 + 2 * c));
    const uint32_t y = e4m3x2(*reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kKeyScales + 64 + g * 8 + 2 * c));
    sa[0] = __byte_perm(x, x, 0x1010);
    sa[1] = __byte_perm(x, x, 0x3232);
    sc[0] = __byte_perm(y, y, 0x1010);
    sc[1] = __byte_perm(y, y, 0x3232);
  } else {
    *reinterpret_cast<uint2*>(ka) = *reinterpret_cast<const uint2*>(sb + g * 32 + c * 8);
    *reinterpret_cast<uint2*>(kb) = *reinterpret_cast<const uint2*>(sb + g * 32 + 256 + c * 8);
    const uint32_t x = sb[KvBlock<D>::kKeyScales + g * 4 + c];
    const uint32_t y = sb[KvBlock<D>::kKeyScales + 32 + g * 4 + c];
    sa[0] = sa[1] = e4m3x2(x | (x << 8));
    sc[0] = sc[1] = e4m3x2(y | (y << 8));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {  // 8 values, two steps of the inner dimension
    uint32_t a[4], b[4];
    e2m1x8(ka[i], a);
    e2m1x8(kb[i], b);
    const int k = D == 128 ? i / 2 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[2 * i + h][0] = mul_f16x2(a[2 * h], sa[k]);
      f[2 * i + h][1] = mul_f16x2(b[2 * h], sc[k]);
      f[2 * i + h][2] = mul_f16x2(a[2 * h + 1], sa[k]);
      f[2 * i + h][3] = mul_f16x2(b[2 * h + 1], sc[k]);
    }
  }
}

// Values of a block as operands, D / 8 values of the token pairs c and c + 4. A token that some
// row does not see must not reach it as 0 * NaN: in a masked block its scale is taken as 0 where the
// cache holds nothing (past the length) or a NaN; `nan_at` bit i then says that token i, which
// some rows see, has a NaN scale among this thread's values.
template <int D>
__device__ __forceinline__ void value_operands(const unsigned char* sb, int g, int c, bool masked,
                                               int t0, int len, int all_see,
                                               uint32_t (&f)[D / 16][4], uint32_t& nan_at) {
  constexpr int N = D / 32;  // words of a thread's codes of one token pair
  uint32_t va[N], vb[N], fa, fb;
  if (D == 128) {
    const int at = c * 128 + 16 * KvBlock<D>::place(c, g);
    *reinterpret_cast<uint4*>(va) = *reinterpret_cast<const uint4*>(sb + KvBlock<D>::kValCodes + at);
    *reinterpret_cast<uint4*>(vb) = *reinterpret_cast<const uint4*>(sb + KvBlock<D>::kValCodes + 512 + at);
    fa = *reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kValScales + c * 16 + 2 * g);
    fb = *reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kValScales + 64 + c * 16 + 2 * g);
  } else {
    const int at = c * 64 + 8 * KvBlock<D>::place(c, g);
    *reinterpret_cast<uint2*>(va) = *reinterpret_cast<const uint2*>(sb + KvBlock<D>::kValCodes + at);
    *reinterpret_cast<uint2*>(vb) = *reinterpret_cast<const uint2*>(sb + KvBlock<D>::kValCodes + 256 + at);
    fa = *reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kValScales + c * 8 + 2 * (g >> 1));
    fb = *reinterpret_cast<const uint16_t*>(sb + KvBlock<D>::kValScales + 32 + c * 8 + 2 * (g >> 1));
  }
  if (masked) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 2 * c + (k & 1) + 8 * (k >> 1), sh = 8 * (k & 1);
      uint32_t& s = k < 2 ? fa : fb;
      const bool bad = ((s >> sh) & 0x7Fu) == 0x7Fu;
      if (t0 + i >= len || (bad && t0 + i >= all_see)) s &= ~(0xFFu << sh);
      if (bad && t0 + i < len && t0 + i >= all_see) nan_at |= 1u << i;
    }
  }
  fa = e4m3x2(fa);
  fb = e4m3x2(fb);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t a[4], b[4];
    e2m1x8(va[i], a);
    e2m1x8(vb[i], b);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[2 * i + h][0] = mul_f16x2(a[2 * h], fa);
      f[2 * i + h][1] = mul_f16x2(a[2 * h + 1], fa);
      f[2 * i + h][2] = mul_f16x2(b[2 * h], fb);
      f[2 * i + h][3] = mul_f16x2(b[2 * h + 1], fb);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(AttnShape<D, NT>::kThreads, AttnShape<D, NT>::kPerSm)
    attn_kernel(AttnParams P) {
  using S = AttnShape<D, NT>;
  constexpr int W = S::kWarps, NS = S::kStages, R = S::kRows, KS = D / 16, MT = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  uint2* sq = reinterpret_cast<uint2*>(smem + S::kRing);  // query operands [NT][KS][lane]
  float* so = reinterpret_cast<float*>(smem + S::kRing + S::kQ);
  float* swm = so + S::kOut / 4;                    // [W][R] running maxima
  float* swl = swm + W * R;                         // [W][R] sums
  int* svis = reinterpret_cast<int*>(swl + W * R);  // [R] tokens that a row sees
  float* sqc = reinterpret_cast<float*>(svis + R);  // [R] score of a product of the operands
  uint64_t* bars = reinterpret_cast<uint64_t*>(sqc + R);
  __shared__ long long s_scan[W];
  __shared__ long long s_start[2];
  __shared__ int s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  if (tid < W * NS) {
    mbar_init(&bars[tid], 1);
    fence_mbar_init();
  }

  // ---- this CTA's run of units
  Walk w;
  long long u0, u1, U;
  long long ctas;
  {
    const int per = (P.B + S::kThreads - 1) / S::kThreads;
    const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      load_seq(P, R, b, w);
      mine += seq_units(P, w);
    }
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    long long before = 0;
    U = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const long long p = s_scan[i];
      if (i < warp) before += p;
      U += p;
    }
    before += x - mine;
    // every warp of a CTA gets a unit at least
    ctas = min(static_cast<long long>(gridDim.x), (U + W - 1) / W);
    if (blockIdx.x >= ctas) return;
    u0 = U * blockIdx.x / ctas;
    u1 = U * (blockIdx.x + 1) / ctas;
    if (u0 >= before && u0 < before + mine) {
      for (int b = b0; b < b1; ++b) {
        load_seq(P, R, b, w);
        const long long n = seq_units(P, w);
        if (u0 < before + n) {
          s_start[0] = b;
          s_start[1] = before;
          break;
        }
        before += n;
      }
    }
    __syncthreads();
    load_seq(P, R, static_cast<int>(s_start[0]), w);
    const long long item = (u0 - s_start[1]) / w.nu;
    w.h = static_cast<int>(item / w.rts);
    w.rt = static_cast<int>(item - static_cast<long long>(w.h) * w.rts);
    w.base = s_start[1] + item * w.nu;
  }

  // ---- the warp's producer: copies of its units, kStages ahead
  unsigned char* my_ring = ring + warp * NS * S::kStage;
  uint64_t* my_bar = bars + warp * NS;
  const int bpp_log = 31 - __clz(P.ps >> 4);  // blocks of a page: a power of two
  Walk pw = w;
  long long pu = u0 + warp;
  int page[2] = {-1, -1};          // pages of unit pu's blocks; -1: nothing to copy
  uint32_t absent = 0, phase = 0;  // per stage and block: not copied; per stage: next copy's parity
  bool dead = false;
  auto fetch_pages = [&]() {
    page[0] = page[1] = -1;
    if (pu >= u1) return;
    while (pu >= pw.base + pw.nu) next_item(P, R, pw);
    const int blk = 2 * static_cast<int>(pu - pw.base);
    const int32_t* row = P.table + static_cast<long long>(pw.b) * P.max_blocks;
    if (16 * blk < pw.len) page[0] = row[blk >> bpp_log];
    if (16 * blk + 16 < pw.len) page[1] = bpp_log ? page[0] : row[blk + 1];
  };
  auto issue = [&](int stage) {  // copy unit pu into the stage, move on to the next unit
    if (pu >= u1) return;
    const bool h0 = static_cast<unsigned>(page[0]) < static_cast<unsigned>(P.num_pages) && !dead;
    const bool h1 = static_cast<unsigned>(page[1]) < static_cast<unsigned>(P.num_pages) && !dead;
    absent = (absent & ~(3u << (2 * stage))) | ((h0 ? 0u : 1u) | (h1 ? 0u : 2u)) << (2 * stage);
    if (lane == 0 && (h0 || h1)) {
      mbar_arrive_expect_tx(&my_bar[stage], (h0 + h1) * S::kBlock);
      const int in_page = 2 * static_cast<int>(pu - pw.base) & ((1 << bpp_log) - 1);
      unsigned char* to = my_ring + stage * S::kStage;
      if (bpp_log) {  // neighbours in one page
        bulk_g2s(to, P.cache + (((static_cast<long long>(page[0]) * P.hkv + pw.h) << bpp_log) + in_page) * S::kBlock,
                 (h0 + h1) * S::kBlock, &my_bar[stage]);
      } else {
        if (h0)
          bulk_g2s(to, P.cache + (static_cast<long long>(page[0]) * P.hkv + pw.h) * S::kBlock,
                   S::kBlock, &my_bar[stage]);
        if (h1)
          bulk_g2s(to + S::kBlock, P.cache + (static_cast<long long>(page[1]) * P.hkv + pw.h) * S::kBlock,
                   S::kBlock, &my_bar[stage]);
      }
    }
    pu += W;
    fetch_pages();
  };
  fetch_pages();
  for (int i = 0; i < NS; ++i) issue(i);

  // ---- items of the run
  long long cu = u0 + warp;  // next unit of this warp
  int stage = 0;
  while (w.base < u1) {
    const long long ua = max(w.base, u0), ub = min(w.base + w.nu, u1);
    const int rows = min(R, w.n * P.group - w.rt * R);  // rows of this tile
    const int tiles = (rows + 7) >> 3;
    // queries as float16 operands: each row times a power of two that brings its largest value
    // to 2^14 .. 2^15, so that a value down to 2^-28 of that one is exact; undone in the scores
    for (int i = tid; i < R * (D / 8); i += S::kThreads) {
      const int r = i / (D / 8), j = i % (D / 8);
      const int row = w.rt * R + min(r, rows - 1);
      const int tok = row / P.group, hh = w.h * P.group + row % P.group;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows)
        raw = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) +
                                                   (w.r0 + tok) * P.qs +
                                                   static_cast<long long>(hh) * D) + j);
      const uint32_t x[4] = {raw.x, raw.y, raw.z, raw.w};
      unsigned most = 0;  // largest finite magnitude's bits
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const unsigned v = (x[k >> 1] >> (16 * (k & 1))) & 0x7FFFu;
        if (v < 0x7F80u) most = max(most, v);
      }
#pragma unroll
      for (int d = D / 16; d > 0; d >>= 1)
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d, D / 8));
      const int k = min(14 - (static_cast<int>(most >> 7) - 127), 100);
      const float up = __int_as_float((k + 127) << 23);
      if (j == 0) {
        svis[r] = w.len - w.n + tok + 1;
        sqc[r] = P.c * __int_as_float((127 - k) << 23);
      }
      uint32_t h[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        h[n] = pack_f16(__uint_as_float(x[n] << 16) * up, __uint_as_float(x[n] & 0xFFFF0000u) * up);
      // values 8j .. 8j + 7: thread 8j / (D/4) of the row, steps s and s + 1 of the inner dimension
      const int s = 8 * j % (D / 4) / 4;
      uint2* to = sq + ((r >> 3) * KS + s) * 32 + (r & 7) * 4 + 8 * j / (D / 4);
      to[0] = make_uint2(h[0], h[1]);
      to[32] = make_uint2(h[2], h[3]);
    }
    __syncthreads();
    const int all_see = svis[0];  // tokens that every row of the tile sees

    float O[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[t][j][k] = 0.f;
      m[t][0] = m[t][1] = -FLT_MAX;
      l[t][0] = l[t][1] = 0.f;
    }

    // The warp's units of this item, for TN tiles of rows: no branch on the tile inside
    auto run = [&](auto tn) {
      constexpr int TN = decltype(tn)::value;
      for (; cu < ub; cu += W) {
        const unsigned char* sb = my_ring + stage * S::kStage;
        const int t0 = static_cast<int>(cu - w.base) * kUnit;
        uint32_t lost = (absent >> (2 * stage)) & 3u;  // blocks that are not there
        if (lost != 3u) {
          const bool ok = mbar_wait_bounded(&my_bar[stage], (phase >> stage) & 1u, kWaitCycles);
          phase ^= 1u << stage;
          if (__any_sync(0xFFFFFFFFu, !ok)) {
            if (lane == 0) atomicOr(P.err, 1u);
            dead = true;
            lost = 3u;
          }
        }
        const bool masked = t0 + kUnit > all_see || lost;

        // scores of 32 tokens and the tile's rows
        float s[2][TN][4];
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int t = 0; t < TN; ++t) s[hb][t][0] = s[hb][t][1] = s[hb][t][2] = s[hb][t][3] = 0.f;
        if constexpr (S::kJoint) {  // a query operand loaded once for both blocks
          uint32_t kf[2][KS][4];
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) key_operands<D>(sb + hb * S::kBlock, g, c, kf[hb]);
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int t = 0; t < TN; ++t) {
              const uint2 q = sq[(t * KS + i) * 32 + lane];
#pragma unroll
              for (int hb = 0; hb < 2; ++hb)
                mma16816(s[hb][t], kf[hb][i][0], kf[hb][i][1], kf[hb][i][2], kf[hb][i][3], q.x, q.y);
            }
        } else {  // half the registers
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            uint32_t kf[KS][4];
            key_operands<D>(sb + hb * S::kBlock, g, c, kf);
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
              for (int t = 0; t < TN; ++t) {
                const uint2 q = sq[(t * KS + i) * 32 + lane];
                mma16816(s[hb][t], kf[i][0], kf[i][1], kf[i][2], kf[i][3], q.x, q.y);
              }
          }
        }
        // exponents: score * factor of the row - maximum of the row
        float x[2][TN][4];
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < TN; ++t) {
          const float2 qc = *reinterpret_cast<const float2*>(sqc + 8 * t + 2 * c);
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[hb][t][k] = fmaf(s[hb][t][k], k & 1 ? qc.y : qc.x, -m[t][k & 1]);
        }
        uint32_t hidden = 0;  // a bit a score: tokens that the row does not see
        if (masked) {
#pragma unroll
          for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int hb = 0; hb < 2; ++hb)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (t0 + 16 * hb + g + 8 * (k >> 1) >= svis[8 * t + 2 * c + (k & 1)]) {
                  x[hb][t][k] = -INFINITY;
                  hidden |= 1u << (8 * t + 4 * hb + k);
                } else if ((lost >> hb) & 1u) {
                  x[hb][t][k] = s[hb][t][k] = NAN;
                }
        }
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
          for (int hb = 0; hb < 2; ++hb)
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, x[hb][t][k]);
        if (__any_sync(0xFFFFFFFFu, top > kSlack)) {  // a new maximum of some row
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            const float2 qc = *reinterpret_cast<const float2*>(sqc + 8 * t + 2 * c);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = e ? qc.y : qc.x;
              float z[4], y = -INFINITY;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int i = e + 2 * (k & 1);
                z[k] = (hidden >> (8 * t + 4 * (k >> 1) + i)) & 1u ? -INFINITY : s[k >> 1][t][i] * f;
                y = fmaxf(y, z[k]);
              }
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
              y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
              y = fmaxf(m[t][e], y - kLift);
              const float down = ex2_fast(m[t][e] - y);
              m[t][e] = y;
              l[t][e] *= down;
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                O[t][j][e] *= down;
                O[t][j][e + 2] *= down;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k >> 1][t][e + 2 * (k & 1)] = z[k] - y;
            }
          }
        }
        uint32_t p[2][TN][2];
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[hb][t][k] = ex2_fast(x[hb][t][k]);
              l[t][k & 1] += x[hb][t][k];
            }
            p[hb][t][0] = transpose8x8(pack_f16(x[hb][t][0], x[hb][t][1]));
            p[hb][t][1] = transpose8x8(pack_f16(x[hb][t][2], x[hb][t][3]));
          }

        // outputs
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
          if (masked && ((lost >> hb) & 1u)) continue;  // its rows are NaN already
          uint32_t nan_at = 0;
          uint32_t vf[MT][4];
          value_operands<D>(sb + hb * S::kBlock, g, c, masked, t0 + 16 * hb, w.len, all_see, vf, nan_at);
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int t = 0; t < TN; ++t)
              mma16816(O[t][j], vf[j][0], vf[j][1], vf[j][2], vf[j][3], p[hb][t][0], p[hb][t][1]);
          if (masked && __any_sync(0xFFFFFFFFu, nan_at != 0)) {
            nan_at |= __shfl_xor_sync(0xFFFFFFFFu, nan_at, 1);
            nan_at |= __shfl_xor_sync(0xFFFFFFFFu, nan_at, 2);
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int seen = svis[8 * t + 2 * c + e] - t0 - 16 * hb;
                const uint32_t sees = seen >= 16 ? 0xFFFFu : seen > 0 ? (1u << seen) - 1u : 0u;
                if (nan_at & sees) {
#pragma unroll
                  for (int j = 0; j < MT; ++j) O[t][j][e] = O[t][j][e + 2] = NAN;
                }
              }
          }
        }
        __syncwarp();
        issue(stage);
        stage = stage + 1 == NS ? 0 : stage + 1;
      }
    };
    if constexpr (NT == 1) {
      run(std::integral_constant<int, 1>());
    } else if constexpr (NT == 2) {
      if (tiles == 1) run(std::integral_constant<int, 1>());
      else run(std::integral_constant<int, 2>());
    } else if constexpr (NT == 3) {
      if (tiles <= 2) run(std::integral_constant<int, 2>());
      else run(std::integral_constant<int, 3>());
    } else {
      if (tiles <= 2) run(std::integral_constant<int, 2>());
      else if (tiles == 3) run(std::integral_constant<int, 3>());
      else run(std::integral_constant<int, 4>());
    }

    // ---- join the warps
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[t][e];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        if (g == 0) {
          swm[warp * R + 8 * t + 2 * c + e] = m[t][e];
          swl[warp * R + 8 * t + 2 * c + e] = x;
        }
      }
    const bool whole = ua == w.base && ub == w.base + w.nu;
    // a piece's place: a CTA has at most two, one from its start and one to its end
    const int my_slot = 2 * blockIdx.x + (ua == u0 ? 0 : 1);
    float* my_part = P.part + static_cast<long long>(my_slot) * S::kPart;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t >= tiles) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = -FLT_MAX;
#pragma unroll
        for (int i = 0; i < W; ++i) M = fmaxf(M, swm[i * R + 8 * t + 2 * c + e]);
        const float f = ex2_fast(m[t][e] - M);
        // row 2c + e lies at place c + 4e: rows of neighbouring threads 4 banks apart
        float* to = so + (warp * 8 + c + 4 * e) * S::kOutStride + (D / 8) * g;
#pragma unroll
        for (int j = 0; j < MT; j += 2) {
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(O[t][j][e] * f, O[t][j][e + 2] * f, O[t][j + 1][e] * f,
                          O[t][j + 1][e + 2] * f);
        }
      }
      __syncthreads();
      for (int i = tid; i < 8 * D / 4; i += S::kThreads) {
        const int place = i / (D / 4), d = 4 * (i % (D / 4)), r = 8 * t + 2 * (place & 3) + (place >> 2);
        if (r >= rows) continue;
        float M = -FLT_MAX, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < W; ++k) M = fmaxf(M, swm[k * R + r]);
#pragma unroll
        for (int k = 0; k < W; ++k) {
          L += swl[k * R + r] * ex2_fast(swm[k * R + r] - M);
          const float4 x = *reinterpret_cast<const float4*>(so + (k * 8 + place) * S::kOutStride + d);
          o.x += x.x;
          o.y += x.y;
          o.z += x.z;
          o.w += x.w;
        }
        if (whole) {
          const float inv = L == 0.f ? 0.f : P.vs / L;
          const int row = w.rt * R + r;
          const long long at = static_cast<long long>(w.r0 + row / P.group) * P.hq +
                               w.h * P.group + row % P.group;
          const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
          const __nv_bfloat162 b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + at * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          if (d == 0 && P.lse)
            P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(my_part + r * D + d) = o;
          if (d == 0) {
            my_part[R * D + r] = M;
            my_part[R * D + R + r] = L;
          }
        }
      }
      __syncthreads();
    }
    if (!whole) {
      // pieces of this item lie with CTAs first .. last; the last of them to arrive joins them
      const int first = static_cast<int>(((w.base + 1) * ctas + U - 1) / U) - 1;
      const int last = static_cast<int>(((w.base + w.nu) * ctas + U - 1) / U) - 1;
      __threadfence();
      __syncthreads();
      if (tid == 0)
        s_last = atomicAdd(&P.arrived[first], 1u) == static_cast<unsigned>(last - first);
      __syncthreads();
      if (s_last) {
        __threadfence();
        const long long first_u0 = U * first / ctas;
        const int slot0 = 2 * first + (first_u0 == max(w.base, first_u0) ? 0 : 1);
        for (int i = tid; i < rows * (D / 4); i += S::kThreads) {
          const int r = i / (D / 4), d = 4 * (i % (D / 4));
          float M = -FLT_MAX, L = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = first; k <= last; ++k)
            M = fmaxf(M, __ldcg(P.part + static_cast<long long>(k == first ? slot0 : 2 * k) * S::kPart + R * D + r));
#pragma unroll 4
          for (int k = first; k <= last; ++k) {
            const float* part = P.part + static_cast<long long>(k == first ? slot0 : 2 * k) * S::kPart;
            const float f = ex2_fast(__ldcg(part + R * D + r) - M);
            L += __ldcg(part + R * D + R + r) * f;
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + r * D + d));
            o.x += x.x * f;
            o.y += x.y * f;
            o.z += x.z * f;
            o.w += x.w * f;
          }
          const float inv = L == 0.f ? 0.f : P.vs / L;
          const int row = w.rt * R + r;
          const long long at = static_cast<long long>(w.r0 + row / P.group) * P.hq +
                               w.h * P.group + row % P.group;
          const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
          const __nv_bfloat162 b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + at * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
          if (d == 0 && P.lse)
            P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        }
        if (tid == 0) P.arrived[first] = 0;  // ready for the next call
      }
    }
    next_item(P, R, w);
  }
}

template <int D, int NT>
cudaError_t launch_tiles(const AttnParams& P, int sms, cudaStream_t stream) {
  using S = AttnShape<D, NT>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn_kernel<D, NT><<<sms * S::kPerSm, S::kThreads, S::kSmem, stream>>>(P);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const AttnParams& P, int rows, int sms, cudaStream_t stream) {
  switch ((rows + 7) / 8) {
    case 0:
    case 1: return launch_tiles<D, 1>(P, sms, stream);
    case 2: return launch_tiles<D, 2>(P, sms, stream);
    case 3: return launch_tiles<D, 3>(P, sms, stream);
    default: return launch_tiles<D, 4>(P, sms, stream);
  }
}

}  // namespace

size_t attention_workspace_bytes(int sms) {
  // two pieces a CTA, the most with one CTA an SM and 32 rows
  return kAttnHeader + static_cast<size_t>(sms) * 2 * 32 * (128 + 2) * sizeof(float);
}

cudaError_t launch_attention(const AttnParams& P, int D, int max_new, int sms,
                             cudaStream_t stream) {
  // rows of a tile: a sequence's rows in as few tiles of up to 32 as hold them, evenly
  const long long all = std::max(1LL, static_cast<long long>(max_new) * P.group);
  const long long tiles = (all + 31) / 32;
  const int rows = static_cast<int>((all + tiles - 1) / tiles);
  return D == 128 ? launch_dim<128>(P, rows, sms, stream) : launch_dim<64>(P, rows, sms, stream);
}

}  // namespace sv
