// Attention over the 4-bit cache for many rows a head (D = 128), on the fifth-generation tensor cores.
//
// With 9 new tokens and 7 query heads a key/value head a cached value meets 63 rows, and the
// products, not the bytes, bound the kernel of register operands (sv_attn.cu): a warp's matrix
// instruction does 1024 multiplications a cycle and SM, tcgen05 four times that. Here a CTA takes
// 128 tokens at a time:
//   scores^T [128 tokens x N rows] = K [128 x 128, tensor memory] q^T [shared memory]
//   outputs^T [128 values x N rows] += V^T [128 x 128 tokens, shared memory] p^T [shared memory]
// with both results in tensor memory. K goes there as float16, a token a lane, so that it costs
// the shared memory no bandwidth; a byte of value codes is one value of two tokens, which is what
// a row of V^T holds side by side. A thread that has read a token's scores from its lane keeps the
// sums of its weights; the running maximum of a row is moved when a score exceeds it by 2^8
// (kSlack - kLift), a few times in a run, and only then are outputs read back and scaled.
//
// One CTA an SM, its warps specialised, two tiles in flight between any two of them: one copies
// blocks in, one issues products, four unpack keys, four unpack values, sixteen take scores to
// weights, each four of these a quarter of the rows, and one walks through the heads ahead of all
// others. The first form, eight warps that did all of it in turn behind barriers of the CTA, two CTAs
// an SM, took 363 us for 524301 tokens and 20 rows of 8 heads: its warps waited for the one that
// issued products. The work is cut and joined as in sv_attn.cu, in units of 128 tokens.
//
// What bounds it is the way of a tile through the weights' warps, from scores in tensor memory to
// weights in shared memory (about 2050 cycles for 32 rows, 2400 for 64; the products take 1000, the
// copies 700): leaving out the conversions of keys or values in an experiment changed nothing. All
// sixteen warps work on the same tile, so that its waits overlap with no other's. 256 sequences of up to
// 8192 tokens, 63 rows on each of 4 heads, take 218 us (438 in the kernel of register operands when that
// was measured), 0.29 of the measured copy rate; 524301 tokens of 8 heads with 64 rows 269 us; a prompt
// of 4096 tokens, 32 + 8 heads, 0.91 ms, 150 TFLOP/s of what its rows see: every tile of rows takes
// all tokens of its sequence.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <type_traits>
#include <utility>

#include "spec_kv.h"
#include "sv_attn.cuh"
#include "sv_kv.h"
#include "sv_ptx.cuh"
#include "sv_tc.cuh"

namespace sv {
namespace {

constexpr int D = 128;
// warps: copies, products, keys (4), values (4), weights (4 x 4), items; the warps that reach tensor
// memory come in fours, since a warp reaches the lanes of its index modulo 4
constexpr int kWarpKeys = 2, kWarpValues = 6, kWarpWeights = 10, kWarpItems = 26, kTcWarps = 27;
constexpr int kTcWThreads = 32 * (kWarpItems - kWarpWeights);
constexpr int kTcThreads = 32 * kTcWarps;
constexpr int kTcUnit = 128;   // tokens
// Work as it is cut. A tile costs much the same for 32 rows and for 64. An item's start and end cost
// as much as three tiles: counted so, 256 sequences of up to 8192 tokens, 63 rows a head, take 219 us
// (222 counted as four, 225 as five), and not counting them cost 23 us more than counting four.
struct TcWork {
  static constexpr int kRows = kTcMaxRows, kUnit = kTcUnit, kDearest = 4, kOver = 12, kLeast = 2;
  static __device__ __forceinline__ int weight(int) { return 4; }
};
constexpr int kTcStages = 4;   // tiles of the cache's bytes on their way
constexpr int kTcBlock = KvBlock<D>::kBytes;
constexpr int kTcStage = 8 * kTcBlock;
constexpr int kSlabV = 128 * 128;          // 128 values x 64 tokens of float16
constexpr int kSlabR = kTcMaxRows * 128;   // rows x 64 values or tokens
constexpr int kTcV = 2 * kSlabV, kTcQ = 2 * kSlabR;  // each twice
constexpr int kTcP = 128 * 2 * kTcMaxRows;  // weights, 64 rows of a token side by side; twice
static_assert(kTcMaxRows == 64, "a token's weights are a line of 128 bytes");
constexpr int kTcSmem = 1024 + 2 * (kTcV + kTcQ + kTcP) + kTcStages * kTcStage;
// tensor memory columns: keys and scores twice, outputs
constexpr uint32_t kColK = 0, kColS = 128, kColO = 256, kTcCols = 512;
constexpr int kTcPart = kTcMaxRows * (D + 2);
static_assert(kTcSmem + 8 * 1024 <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The low word of a shared-memory operand's descriptor (smem_desc_sw128); its high word is the
// same for every operand here. One thread issues all products, so what it computes for each counts.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A[tmem] * B[smem]^T, one step of 16, float16 operands; issued by one thread.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// The same with A in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}

// Stores at a register's address plus a constant.
template <int off>
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0+%1], {%2, %3, %4, %5};" ::"r"(at), "n"(off), "r"(a), "r"(b), "r"(c),
               "r"(d));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// f(0), ..., f(N - 1) with constants as arguments
template <int... I, class F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N>
using Upto = std::make_integer_sequence<int, N>;

// 32 columns of this warp's lanes from r, complete (for this thread) after tmem_wait_st.
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const float2 (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
               "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Columns t and t + 32 and the seven after each, the row groups of this warp: asked for, and there
// (nothing may be done with r in between).
__device__ __forceinline__ void tmem_ld_start(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(t), "r"(t + 32));
}
__device__ __forceinline__ void tmem_ld_finish(uint32_t (&r)[16], float2 (&v)[2][4]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[k][j] = make_float2(__uint_as_float(r[8 * k + 2 * j]), __uint_as_float(r[8 * k + 2 * j + 1]));
}
__device__ __forceinline__ void tmem_ld_groups(uint32_t t, float2 (&v)[2][4]) {
  uint32_t r[16];
  tmem_ld_start(t, r);
  tmem_ld_finish(r, v);
}

// Two floats at a time
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sums of 16 values over the warp's lanes: lane i < 16 gets the sum of value i.
__device__ __forceinline__ float warp_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int n = 8; n > 0; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, send, n);
    }
  }
  return v[0] + __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);
}

// An item of the run, or the part of it that the run has: its units unit .. end - 1.
struct TcItem {
  Walk w;
  long long out0;  // the output's row that S.at counts from
  int unit, end, rows;
  int all_see;     // tokens that every row sees
  bool whole;
};

// Tiles whose tokens with a NaN scale are kept. The values' warps note those of tile t, over those of
// tile t - kNanTiles, once the products of tile t - 3 are done, so once the weights of tile t - 3 are
// there; the weights' warps read those of tile i before they hand over the weights of tile i + 2, or, of
// an item's last two tiles, those of the next item's first one, i + 1 or i + 2. So any number above 4
// keeps what is still to be read; a power of two makes the place cheap.
constexpr int kNanTiles = 8;

// What the roles share. Tile t uses buffer t & 1 of everything that is held twice.
struct TcShared {
  uint64_t raw_full[kTcStages], raw_empty[kTcStages];  // the cache's bytes
  uint64_t k_full[2];             // keys unpacked
  uint64_t s_full[2];             // scores there: the keys are spent, and so is all that products
                                  // issued before them read
  uint64_t vp_full[2];            // values unpacked and weights there (and the scores read)
  uint64_t pv_done[2];            // values and weights spent, outputs up to date
  uint64_t q_full[2], q_empty[2];  // queries of an item, twice as well
  uint64_t item_full[4];           // the item itself
  TcItem items[4];
  uint64_t end;
  uint32_t tmem;
  uint32_t lost[16];              // per tile modulo 16: blocks that are not there
  Run run;
  Walk first;
  longlong2 scan[kTcWarps];
  alignas(16) float qc[2][kTcMaxRows];  // per row: score of a product of the operands
  int vis[2][kTcMaxRows];         // tokens that it sees
  alignas(16) float nm[kTcMaxRows];  // running maxima, negated
  alignas(16) float down[kTcMaxRows];
  float part[4][kTcMaxRows];      // per quarter of a tile's tokens: maxima, sums
  alignas(16) int at[4][kTcMaxRows];  // its row of the output, from the item's first (of four items)
  uint32_t nan[kNanTiles][8][4];  // per tile modulo kNanTiles and 16 values: tokens with a NaN scale
  int nans[kNanTiles];            // the tile that this speaks of, plus one
  int last;
};

static_assert(offsetof(TcShared, qc) % 16 == 0 && offsetof(TcShared, at) % 16 == 0 &&
                  offsetof(TcShared, down) % 16 == 0 && offsetof(TcShared, nm) % 16 == 0, "read as float4");

__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(AttnParams P) {
  constexpr int R = kTcMaxRows;
  extern __shared__ unsigned char dsm[];
  __shared__ __align__(16) TcShared S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* base = dsm + ((1024u - (smem_u32(dsm) & 1023u)) & 1023u);
  unsigned char* sval = base;
  unsigned char* sq = sval + 2 * kTcV;
  unsigned char* sp = sq + 2 * kTcQ;
  unsigned char* ring = sp + 2 * kTcP;

  if (tid == 0) {
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 4);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.vp_full[i], 20);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.q_full[i], 4);
      mbar_init(&S.q_empty[i], 16);
    }
    mbar_init(&S.end, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.item_full[i], 1);
      S.items[i] = TcItem{};  // what a role reads that gave up waiting: it goes on to its end
      S.items[i].end = S.items[i].rows = 1;
    }
    fence_mbar_init();
    for (int i = 0; i < kNanTiles; ++i) S.nans[i] = 0;
  }
  if (!find_run<kTcThreads, TcWork>(P, S.scan, &S.run, &S.first)) return;
  if (warp == 1) tmem_alloc(&S.tmem, kTcCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int tiles = static_cast<int>(S.run.u1 - S.run.u0);
  // Every wait has a limit. A role that met it waits no more and runs through to its end, so that
  // nobody waits for it for good; what comes out is not used. It hands on nothing that somebody may still
  // use: no stage whose copy may be on its way (raw_empty), no place of an item that is read.
  int tries = kWaitTries;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_u32(bar), p = parity & 1u;
    int left = tries;
    while (!mbar_try(at, p))
      if (--left <= 0) {
        tries = 0;
        break;
      }
  };
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    wait(bar, parity);
    __syncwarp();
  };
  auto arrive_warp = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto give_back = [&](int stage) {
    __syncwarp();
    if (lane == 0 && tries > 0) mbar_arrive(&S.raw_empty[stage]);
  };

  if (warp == 0) {
    // ---- copies. Where the blocks lie is looked up four tiles at a time, a lane a block, and a
    // round before it is needed, so that no copy waits for a page number.
    const int bpp_log = 31 - __clz(P.ps >> 4);  // blocks of a page: a power of two
    const int mine = lane >> 3, block = lane & 7;
    Walk w = S.first;
    int unit = static_cast<int>(S.run.u0 - w.base);
    int issued = 0, next_at = 0;
    int next_page = -1;
    unit += mine;  // of this lane's tile
    auto look_up = [&](int t) {
      next_page = -1;
      while (unit >= w.nu) {
        unit -= w.nu;
        next_item<TcWork>(P, w);
      }
      const int blk = 8 * unit + block;
      if (t + mine < tiles && 16 * blk < w.len) {
        next_page = P.table[static_cast<long long>(w.b) * P.max_blocks + (blk >> bpp_log)];
        next_at = (w.h << bpp_log) + (blk & ((1 << bpp_log) - 1));
      }
      unit += 4;
    };
    look_up(0);
    for (int t0 = 0; t0 < tiles; t0 += 4) {
      const int page = next_page, at = next_at;
      look_up(t0 + 4);
      const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(P.num_pages);
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, there);
      for (int i = 0; i < 4 && t0 + i < tiles; ++i) {
        const int t = t0 + i, stage = t % kTcStages;
        const uint32_t mask = (all >> (8 * i)) & 0xFFu;
        if (t >= kTcStages) wait_warp(&S.raw_empty[stage], t / kTcStages - 1);
        if (!__all_sync(0xFFFFFFFFu, tries > 0)) break;
        if (lane == 0) {
          S.lost[t & 15] = ~mask & 0xFFu;
          if (mask)
            mbar_arrive_expect_tx(&S.raw_full[stage], __popc(mask) * kTcBlock);
          else
            mbar_arrive(&S.raw_full[stage]);
        }
        __syncwarp();
        const bool whole = bpp_log == 3 && mask == 0xFFu;  // one page: neighbours
        if (there && mine == i && (!whole || block == 0))
          bulk_g2s(ring + stage * kTcStage + block * kTcBlock,
                   P.cache + (((static_cast<long long>(page) * P.hkv) << bpp_log) + at) * kTcBlock,
                   whole ? kTcStage : kTcBlock, &S.raw_full[stage]);
        ++issued;
      }
    }
    // no copy is in flight when the CTA ends, whoever gave up
    for (int i = max(0, issued - kTcStages); i < issued; ++i)
      if (!mbar_wait_bounded(&S.raw_full[i % kTcStages], (i / kTcStages) & 1, kWaitCycles)) tries = 0;
  } else if (warp == 1) {
    // ---- products, issued by an elected thread (a thread that the compiler knows to be one: picked
    // by its number it costs 96 to 111 cycles a product whatever its size, elected 39 with 32 rows)
    int t = 0;
    uint32_t idesc = 0, pv_idesc = 0;
    bool pv_first = false;
    const uint32_t a_val = desc_lo(smem_u32(sval)), a_q = desc_lo(smem_u32(sq)), a_p = desc_lo(smem_u32(sp));
    auto outputs = [&](int i) {  // of tile i
      const int b = i & 1;
      wait_warp(&S.vp_full[b], i >> 1);
      tc_fence_after();
      const uint32_t a = a_val + b * (kTcV >> 4), p = a_p + b * (kTcP >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ss(tmem + kColO, a + (((kk >> 2) * kSlabV + 32 * (kk & 3)) >> 4),
                    p + ((kk * 16 * 128) >> 4), pv_idesc, !pv_first || kk > 0);
        tc_commit(&S.pv_done[b]);
      }
      __syncwarp();
    };
    for (int item = 0; t < tiles; ++item) {
      // the last item's outputs do not wait for queries
      bool late = t > 0 && !mbar_test(&S.q_full[item & 1], (item >> 1) & 1);
      if (__any_sync(0xFFFFFFFFu, late)) {
        outputs(t - 1);
        late = true;
      }
      wait_warp(&S.q_full[item & 1], item >> 1);
      const int end = S.items[item & 3].end, rows = S.items[item & 3].rows;
      // float16 operands, float32 sums, 128 x (rows to a multiple of 16)
      idesc = (1u << 4) | (static_cast<uint32_t>((rows + 15) / 16 * 2) << 17) |
              (static_cast<uint32_t>(128 >> 4) << 24);
      const uint32_t q = a_q + (item & 1) * (kTcQ >> 4);
      bool first = true;
      for (int unit = S.items[item & 3].unit; unit < end; ++unit, ++t, first = false) {
        const int b = t & 1;
        // the scores of tile t - 2 have been read: its weights were there
        wait_warp(&S.k_full[b], t >> 1);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc_mma_ts(tmem + kColS + 64 * b, tmem + kColK + 64 * b + 8 * kk,
                      q + (((kk >> 2) * kSlabR + 32 * (kk & 3)) >> 4), idesc, kk > 0);
          tc_commit(&S.s_full[b]);
        }
        __syncwarp();
        if (t > 0 && !(first && late)) outputs(t - 1);
        pv_idesc = idesc | (1u << 16);  // weights lie token by token
        pv_first = first;
      }
    }
    outputs(t - 1);
    // all products are done before the memory goes
    if (elect_one()) tc_commit(&S.end);
    __syncwarp();
    if (!mbar_wait_bounded(&S.end, 0, kWaitCycles)) tries = 0;
  } else if (warp < kWarpValues) {
    // ---- keys: a thread a token
    constexpr int QV = D / 8, QPER = R * QV / 128;
    const int q = warp & 3, tok = 32 * q + lane, kid = tid - 32 * kWarpKeys;
    const uint32_t to = tmem + (static_cast<uint32_t>(q) << 21) + kColK;
    int t = 0;
    for (int item = 0; t < tiles; ++item) {
      wait_warp(&S.item_full[item & 3], item >> 2);
      const TcItem& it = S.items[item & 3];
      const Walk& w = it.w;
      const int end = it.end, rows = it.rows, qb = item & 1, row0 = w.rt * R, i0 = row0 / P.group;
      // queries in rows of 64 values (128 bytes), in the 128-byte swizzle
      uint4 raw[QPER];
#pragma unroll
      for (int n = 0; n < QPER; ++n) {
        const int r = 8 * n + kid / QV;
        raw[n] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int row = w.rt * R + r, i = row / P.group, head = w.h * P.group + row % P.group;
          raw[n] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.q) +
                                                        (w.r0 + i) * P.qs +
                                                        static_cast<long long>(head) * D) + kid % QV);
        }
      }
#pragma unroll
      for (int n = 0; n < QPER; ++n) {
        if (8 * n >= rows) break;
        const int r = 8 * n + kid / QV, j = kid % QV;
        unsigned most = largest_finite(raw[n]);
#pragma unroll
        for (int d = QV / 2; d > 0; d >>= 1)
          most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d, QV));
        float undo;
        const float up = query_scale(most, P.c, &undo);
        if (j == 0) {
          const int row = row0 + min(r, rows - 1), i = row / P.group;
          S.vis[qb][r] = w.len - w.n + i + 1;
          S.at[item & 3][r] = (i - i0) * P.hq + row - i * P.group;
          S.qc[qb][r] = undo;
        }
        uint32_t f[4];
        query_f16(raw[n], up, f);
        *reinterpret_cast<uint4*>(sq + qb * kTcQ + (j >> 3) * kSlabR + r * 128 +
                                  (((j & 7) ^ (r & 7)) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
      }
      fence_proxy_async();
      arrive_warp(&S.q_full[qb]);
      for (int unit = it.unit; unit < end; ++unit, ++t) {
        const int stage = t % kTcStages, b = t & 1;
        wait_warp(&S.raw_full[stage], t / kTcStages);
        const unsigned char* blk = ring + stage * kTcStage + (tok >> 4) * kTcBlock;
        // four vectors a token; neighbours start at different ones, which keeps the banks apart
        const int turn = (lane >> 1) & 3;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const uint4*>(blk + (tok & 15) * 64 + 16 * (i ^ turn));
        const uint2 sc = *reinterpret_cast<const uint2*>(blk + KvBlock<D>::kKeyScales + (tok & 15) * 8);
        give_back(stage);
        auto swap = [&](uint4& a, uint4& c, bool s) {
          const uint4 y = a;
          a = make_uint4(s ? c.x : a.x, s ? c.y : a.y, s ? c.z : a.z, s ? c.w : a.w);
          c = make_uint4(s ? y.x : c.x, s ? y.y : c.y, s ? y.z : c.z, s ? y.w : c.w);
        };
        swap(x[0], x[1], turn & 1);
        swap(x[2], x[3], turn & 1);
        swap(x[0], x[2], turn & 2);
        swap(x[1], x[3], turn & 2);
        if (t >= 2) wait_warp(&S.s_full[b], (t >> 1) - 1);  // this buffer's products are done
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t s4 = half ? sc.y : sc.x;
          const uint32_t s01 = e4m3x2(s4), s23 = e4m3x2(s4 >> 16);
          const uint32_t f[4] = {__byte_perm(s01, s01, 0x1010), __byte_perm(s01, s01, 0x3232),
                                 __byte_perm(s23, s23, 0x1010), __byte_perm(s23, s23, 0x3232)};
          const uint4 lo = x[2 * half], hi = x[2 * half + 1];
          const uint32_t code[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          uint32_t k16[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t y[4];
            e2m1x8(code[i], y);
#pragma unroll
            for (int n = 0; n < 4; ++n) k16[4 * i + n] = mul_f16x2(y[n], f[i >> 1]);
          }
          tmem_st32(to + 64 * b + 32 * half, k16);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&S.k_full[b]);
      }
    }
  } else if (warp < kWarpWeights) {
    // ---- values: a thread 16 values (a scale's) of 8 tokens. Codes: 8 threads side by side read a
    // pair's line of 128 bytes; operands: 8 threads side by side write 8 different 16-byte places of
    // a row of 64 tokens.
    const int vid = tid - 32 * kWarpValues, vg = lane & 7, vv = 4 * (warp - kWarpValues) + (lane >> 3);
    const int vt = (((lane & 7) + vv) & 7) | (vv & 8);  // group of 8 tokens
    const int code_at = (vt >> 1) * kTcBlock + KvBlock<D>::kValCodes + (vt & 1) * 4 * D;
    const int scale_at = (vt >> 1) * kTcBlock + KvBlock<D>::kValScales + (vt & 1) * 64 + 2 * vg;
    const uint32_t v_to = smem_u32(sval) + (vt >> 3) * kSlabV + 16 * vg * 128 + ((vt & 7) << 4);
    int t = 0;
    for (int item = 0; t < tiles; ++item) {
      wait_warp(&S.item_full[item & 3], item >> 2);
      const int end = S.items[item & 3].end, len = S.items[item & 3].w.len;
      const int all_see = S.items[item & 3].all_see;
      for (int unit = S.items[item & 3].unit; unit < end; ++unit, ++t) {
        const int stage = t % kTcStages, b = t & 1, t0 = unit * kTcUnit;
        wait_warp(&S.raw_full[stage], t / kTcStages);
        const unsigned char* src = ring + stage * kTcStage;
        uint4 x[4];
        uint32_t sc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = *reinterpret_cast<const uint4*>(src + code_at + i * D + 16 * (vg ^ (2 * i)));
          sc[i] = *reinterpret_cast<const uint16_t*>(src + scale_at + 16 * i);
        }
        const uint32_t lost = S.lost[t & 15];
        give_back(stage);
        if (t0 + kTcUnit > all_see || lost) {
          // see sv_attn.cu: what some row does not see must not reach it as 0 * NaN
          if (vid < 32) S.nan[t & (kNanTiles - 1)][vid >> 2][vid & 3] = 0;
          named_sync(5, 128);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int k = 8 * vt + 2 * i + n, sh = 8 * n;
              const bool bad = ((sc[i] >> sh) & 0x7Fu) == 0x7Fu;
              if (t0 + k >= len || ((lost >> (k >> 4)) & 1u)) {
                sc[i] &= ~(0xFFu << sh);
              } else if (bad && t0 + k >= all_see) {
                sc[i] &= ~(0xFFu << sh);
                atomicOr(&S.nan[t & (kNanTiles - 1)][vg][k >> 5], 1u << (k & 31));
                S.nans[t & (kNanTiles - 1)] = t + 1;
              }
            }
        }
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = e4m3x2(sc[i]);
        if (t >= 2) wait_warp(&S.pv_done[b], (t >> 1) - 1);  // this buffer's products are done
        const uint32_t dst = v_to + b * kTcV;
        each(Upto<4>(), [&](auto part_) {  // 4 values
          constexpr int part = decltype(part_)::value;
          uint32_t v16[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t y[4];
            e2m1x8(part == 0 ? x[i].x : part == 1 ? x[i].y : part == 2 ? x[i].z : x[i].w, y);
#pragma unroll
            for (int n = 0; n < 4; ++n) v16[n][i] = mul_f16x2(y[n], f[i]);
          }
          each(Upto<4>(), [&](auto n_) {
            constexpr int n = decltype(n_)::value, d = 4 * part + n;
            // (vt ^ d) % 8 is the place in the swizzled row
            st_shared_v4<d * 128>(dst ^ ((d & 7) << 4), v16[n][0], v16[n][1], v16[n][2], v16[n][3]);
          });
        });
        fence_proxy_async();
        arrive_warp(&S.vp_full[b]);
      }
    }
  } else if (warp == kWarpItems) {
    // ---- items: one thread walks through them, ahead of all others, so that nobody waits for a
    // sequence's lengths. An item takes the place of the fourth before it, which nobody reads any
    // more once the weights of the second before it are done.
    if (lane == 0) {
      Walk w = S.first;
      int unit = static_cast<int>(S.run.u0 - w.base), t = 0;
      for (int item = 0;; ++item) {
        if (item >= 2) wait(&S.q_empty[item & 1], (item >> 1) - 1);
        const int end = static_cast<int>(min(static_cast<long long>(w.nu), S.run.u1 - w.base));
        if (tries > 0) {
          TcItem& it = S.items[item & 3];
          it.w = w;
          it.unit = unit;
          it.end = end;
          it.rows = min(R, w.n * P.group - w.rt * R);
          const int i0 = w.rt * R / P.group;
          it.all_see = w.len - w.n + i0 + 1;
          it.out0 = static_cast<long long>(w.r0 + i0) * P.hq + w.h * P.group;
          it.whole = w.base >= S.run.u0 && end == w.nu;
        }
        mbar_arrive(&S.item_full[item & 3]);
        t += end - unit;
        if (t >= tiles) break;
        next_item<TcWork>(P, w);
        unit = 0;
      }
    }
  } else {
    // ---- weights: a thread a token, a quarter of the rows: 8 (4 k + hh) + j
    const int wid = tid - 32 * kWarpWeights, hh = wid >> 7, hid = wid & 127;
    const int q = warp & 3, tok = 32 * q + lane;
    const uint32_t mine = tmem + (static_cast<uint32_t>(q) << 21);
    // 8 rows of a token are 16 bytes, in the 128-byte swizzle; the other 8 lie 64 bytes away
    const uint32_t p_to = smem_u32(sp) + tok * 128 + ((hh ^ (tok & 7)) << 4);
    const int my_row = 8 * (4 * (hid >> 3) + hh) + (hid & 7);  // hid < 16: a row of this quarter
    const int lane_row = 8 * (4 * (lane >> 3) + hh) + (lane & 7);  // lane < 16
    int t = 0;
    for (int item = 0; t < tiles; ++item) {
      const int qb = item & 1;
      if (hid < 16) S.nm[my_row] = FLT_MAX;
      wait_warp(&S.q_full[qb], item >> 1);
      named_sync(1 + hh, 128);
      const TcItem& it = S.items[item & 3];
      const int end = it.end, rows = it.rows, all_see = it.all_see;
      const float4* qc4 = reinterpret_cast<const float4*>(S.qc[qb] + 8 * hh);  // groups of 8 rows, 32 apart
      const float4* nm4 = reinterpret_cast<const float4*>(S.nm + 8 * hh);
      // Rows that see a NaN value get NaN in its 16 values at the item's end: of tile i (unit u of the
      // item), a bit a row. What the values' warps left for it is there once its products are done,
      // and stays until it has been read (see kNanTiles).
      auto nan_rows = [&](int i, int u) {
        uint32_t hits = 0;
        if (S.nans[i & (kNanTiles - 1)] != i + 1) return hits;
        for (int k = 0; k < 16; ++k) {
          const int r = 8 * (4 * (k >> 3) + hh) + (k & 7);
          if (r >= rows) break;
          const int seen = S.vis[qb][r] - u * kTcUnit;
          for (int n = 0; n < 4; ++n) {
            const int here = seen - 32 * n;
            const uint32_t sees = here >= 32 ? 0xFFFFFFFFu : here > 0 ? (1u << here) - 1u : 0u;
            if (S.nan[i & (kNanTiles - 1)][tok >> 4][n] & sees) hits |= 1u << k;
          }
        }
        return hits;
      };
      uint32_t poison = 0, past = 0;  // such rows; a bit a tile of the item: masked, the last one lowest
      float2 l[2][4];  // sums of this token's weights
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) l[k][j] = make_float2(0.f, 0.f);
      bool first = true;
      for (int unit = it.unit; unit < end; ++unit, ++t, first = false) {
        const int b = t & 1, t0 = unit * kTcUnit;
        wait_warp(&S.s_full[b], t >> 1);
        tc_fence_after();
        bool masked;
        // Scores less their rows' maxima. If one of them is too large they are read once more, and
        // the maxima are moved, as an item's first are in any case.
        float2 z[2][4];
        for (bool move = first;;) {
          // what they are multiplied with is read while they come
          uint32_t raw[16];
          tmem_ld_start(mine + kColS + 64 * b + 8 * hh, raw);
          const uint32_t lost = S.lost[t & 15];
          const float4 f[2][2] = {{qc4[0], qc4[1]}, {qc4[8], qc4[9]}};
          tmem_ld_finish(raw, z);
          masked = t0 + kTcUnit > all_see || lost;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (8 * (4 * k + hh) >= rows) break;
            const float4 a = f[k][0], c = f[k][1];
            // rounded before the maximum is taken
            z[k][0] = mul2(z[k][0], make_float2(a.x, a.y));
            z[k][1] = mul2(z[k][1], make_float2(a.z, a.w));
            z[k][2] = mul2(z[k][2], make_float2(c.x, c.y));
            z[k][3] = mul2(z[k][3], make_float2(c.z, c.w));
          }
          if (masked) {
            const bool here = !((lost >> (tok >> 4)) & 1u);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = 8 * (4 * k + hh) + 2 * j;
                if (r < rows && t0 + tok >= S.vis[qb][r]) z[k][j].x = -INFINITY;
                else if (!here) z[k][j].x = NAN;
                if (r + 1 < rows && t0 + tok >= S.vis[qb][r + 1]) z[k][j].y = -INFINITY;
                else if (!here) z[k][j].y = NAN;
              }
          }
          if (move) {
            float y = -INFINITY;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              if (8 * (4 * k + hh) < rows) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float x0 = warp_max(z[k][j].x), x1 = warp_max(z[k][j].y);
                  if (lane == 8 * k + 2 * j) y = x0;
                  if (lane == 8 * k + 2 * j + 1) y = x1;
                }
              }
            if (lane < 16) S.part[q][lane_row] = y;
            named_sync(1 + hh, 128);
            if (hid < 16) {
              const float old = -S.nm[my_row];
              y = fmaxf(fmaxf(S.part[0][my_row], S.part[1][my_row]),
                        fmaxf(S.part[2][my_row], S.part[3][my_row]));
              const float now = fmaxf(old, y - kLift);
              S.down[my_row] = ex2_fast(old - now);
              S.nm[my_row] = -now;
            }
            named_sync(1 + hh, 128);
            const float2* down2 = reinterpret_cast<const float2*>(S.down + 8 * hh);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j) l[k][j] = mul2(l[k][j], down2[16 * k + j]);
            if (!first) {
              wait_warp(&S.pv_done[(t - 1) & 1], (t - 1) >> 1);
              tc_fence_after();
              float2 o[2][4];
              tmem_ld_groups(mine + kColO + 8 * hh, o);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int r0 = 8 * (4 * k + hh);
                if (r0 >= rows) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][j] = mul2(o[k][j], down2[16 * k + j]);
                tmem_st8(mine + kColO + r0, o[k]);
              }
              tmem_wait_st();
            }
          }
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (8 * (4 * k + hh) >= rows) break;
            const float4 a = nm4[8 * k], c = nm4[8 * k + 1];
            z[k][0] = add2(z[k][0], make_float2(a.x, a.y));
            z[k][1] = add2(z[k][1], make_float2(a.z, a.w));
            z[k][2] = add2(z[k][2], make_float2(c.x, c.y));
            z[k][3] = add2(z[k][3], make_float2(c.z, c.w));
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max3(top, z[k][j].x, z[k][j].y);
          }
          if (move || !named_sync_or(1 + hh, 128, top > kSlack)) break;
          move = true;
        }
        if (past & 2u) poison |= nan_rows(t - 2, unit - 2);
        past = (past << 1) | (masked ? 1u : 0u);
        // the products that read this buffer last were issued before these scores'
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (8 * (4 * k + hh) >= rows) break;
          uint32_t p16[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 p = make_float2(ex2_fast(z[k][j].x), ex2_fast(z[k][j].y));
            l[k][j] = add2(l[k][j], p);
            p16[j] = pack_f16(p.x, p.y);
          }
          st_shared_v4<0>((p_to + b * kTcP) ^ (64 * k), p16[0], p16[1], p16[2], p16[3]);
        }
        fence_proxy_async();
        tc_fence_before();
        arrive_warp(&S.vp_full[b]);
      }

      // the item's results, or this piece of them
      wait_warp(&S.pv_done[(t - 1) & 1], (t - 1) >> 1);
      tc_fence_after();
      float2 o2[2][4];
      tmem_ld_groups(mine + kColO + 8 * hh, o2);
      tc_fence_before();
      float o[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[k][j] = j & 1 ? o2[k][j >> 1].y : o2[k][j >> 1].x;
      if (past & 2u) poison |= nan_rows(t - 2, end - 2);
      if (past & 1u) poison |= nan_rows(t - 1, end - 1);
      if (poison) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((poison >> (8 * k + j)) & 1u) o[k][j] = NAN;
      }
      arrive_warp(&S.q_empty[qb]);
      {
        float v[16];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[8 * k + j] = j & 1 ? l[k][j >> 1].y : l[k][j >> 1].x;
        const float sum = warp_sums(v, lane);
        if (lane < 16) S.part[q][lane_row] = sum;
      }
      named_sync(1 + hh, 128);
      const bool whole = it.whole;
      float* part = P.part + static_cast<long long>(2 * blockIdx.x + (it.w.base < S.run.u0 ? 0 : 1)) * kTcPart;
      if (hid < 16 && my_row < rows) {  // a thread a row: its sum, its factor
        const float L = S.part[0][my_row] + S.part[1][my_row] + S.part[2][my_row] + S.part[3][my_row];
        if (whole) {
          S.down[my_row] = L == 0.f ? 0.f : P.vs / L;
          store_lse(P, it.out0 + S.at[item & 3][my_row], -S.nm[my_row], L);
        } else {
          part[R * D + my_row] = -S.nm[my_row];
          part[R * D + R + my_row] = L;
        }
      }
      named_sync(1 + hh, 128);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(P.out) + it.out0 * D + tok;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r0 = 8 * (4 * k + hh);
        if (r0 >= rows) break;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = r0 + 4 * n;
          if (r >= rows) break;
          const float* x = o[k] + 4 * n;
          if (whole) {
            const float4 f = *reinterpret_cast<const float4*>(S.down + r);
            const int4 at = *reinterpret_cast<const int4*>(S.at[item & 3] + r);
            out[static_cast<long long>(at.x) * D] = __float2bfloat16_rn(x[0] * f.x);
            if (r + 1 < rows) out[static_cast<long long>(at.y) * D] = __float2bfloat16_rn(x[1] * f.y);
            if (r + 2 < rows) out[static_cast<long long>(at.z) * D] = __float2bfloat16_rn(x[2] * f.z);
            if (r + 3 < rows) out[static_cast<long long>(at.w) * D] = __float2bfloat16_rn(x[3] * f.w);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) part[(r + j) * D + tok] = x[j];
          }
        }
      }
      if (!whole)
        join_pieces<kTcWThreads, R, D, 4>(P, it.w, S.run, rows, wid, &S.last, [] { named_sync(6, kTcWThreads); });
      named_sync(1 + hh, 128);  // maxima and sums may change
    }
  }
  if (tries <= 0) atomicOr(P.err, 1u);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
}

}  // namespace

cudaError_t launch_attention_tc(const AttnParams& P, int sms, cudaStream_t stream) {
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  attn_tc_kernel<<<sms, kTcThreads, kTcSmem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace sv
