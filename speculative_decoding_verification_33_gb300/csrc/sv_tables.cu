// Block tables and slot maps of a paged cache from request lengths (spec_block_tables), one launch.
//
// The work is a few prefix sums over the sequences (pages taken, pages put back, tokens) and then
// independent writes: 16 bytes a token, one table entry a new page. It is bound by latency, so
// nothing is handed from one CTA to another: every CTA takes the prefix sums of all sequences
// itself (their lengths are a few KB in L2), keeps what the tokens need in shared memory, and
// writes its share of the tokens and pages. Pages that this call puts back are never taken by
// it, so no CTA reads a ring entry or a table entry that another one writes.
//
// On the device: 3.3 us for 8 sequences, 7.3 us for 1024 (their lengths are read by every CTA, in
// chains of loads and scans that nothing shortens), 5.9 us for 256 with prompts of up to 16384
// tokens (4.8 MB of positions, slots and owners: 0.7 us of HBM). A launch that does nothing is
// about 2.5 us of that.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "spec_kv.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr int kTbTokens = 2;  // consecutive tokens a thread writes

struct TablesParams {
  int B, ps_log, max_blocks, max_tokens, ring_size;
  const int32_t *ctx, *acc, *nw, *held;
  int32_t *table, *ring;
  const int64_t* counters;
  int32_t *o_ctx, *o_held, *o_kv, *o_status, *o_cu, *o_pos, *o_seq;
  int64_t *o_counters, *o_slots;
};

// One sequence of the call, from its lengths alone.
struct Seq {
  long long c, n, grow, shrink;
  int held, bad;
};

__device__ __forceinline__ Seq load_seq(const TablesParams& P, int b) {
  Seq s;
  const int ctx = P.ctx[b], nw = P.nw[b], a = P.acc ? P.acc[b] : -1;
  s.held = P.held[b];
  const bool done = nw < 0;
  s.c = done ? 0 : static_cast<long long>(ctx) + (a >= 0 ? static_cast<long long>(a) + 1 : 0);
  s.n = done ? 0 : nw;
  const long long need = (s.c + s.n + (1LL << P.ps_log) - 1) >> P.ps_log;
  s.bad = s.held < 0 || s.held > P.max_blocks ||
          (!done && (ctx < 0 || s.c > (static_cast<long long>(s.held) << P.ps_log) || need > P.max_blocks));
  if (s.bad) {
    s.c = ctx;
    s.n = s.grow = s.shrink = 0;
  } else {
    s.grow = need > s.held ? need - s.held : 0;
    s.shrink = need < s.held ? s.held - need : 0;
  }
  return s;
}

// Sums held at 2^31 - 1: every limit that they are compared with (free pages, token places) is smaller,
// so what is past it stays past it.
constexpr uint32_t kMost = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kMost); }
__device__ __forceinline__ uint32_t held_at_most(long long a) {
  return a > static_cast<long long>(kMost) ? kMost : static_cast<uint32_t>(a);
}

// Exclusive prefix sums of N values over the CTA's threads; total[] the sums. `part` holds N values a
// warp; the call starts with a barrier, so that it may be used again.
template <int THREADS, int N>
__device__ __forceinline__ void block_scan(uint32_t (&v)[N], uint32_t (*part)[N], uint32_t (&total)[N]) {
  constexpr int W = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x[i], d);
      if (lane >= d) x[i] = add(x[i], y);
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x[i], 1);
    v[i] = lane ? y : 0;  // before this thread, within the warp
  }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < N; ++i) part[warp][i] = x[i];
  __syncthreads();
  uint32_t p[N];  // each warp sums up the warps
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = lane < W ? part[lane][i] : 0;
#pragma unroll
  for (int d = 1; d < W; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, p[i], d);
      if (lane >= d) p[i] = add(p[i], y);
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = __shfl_sync(0xFFFFFFFFu, p[i], W - 1);
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, p[i], warp ? warp - 1 : 0);
    if (warp) v[i] = add(v[i], before);
  }
}

// A sequence a thread as far as the threads go: its lengths are then read once.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) tables_kernel(TablesParams P) {
  // per sequence: first token of the round, tokens before the round, pages held before and
  // after the call, rank of its first queue entry taken or put back
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;
  int32_t* s_c = sm + P.B + 1;
  int32_t* s_held = s_c + P.B;
  int32_t* s_now = s_held + P.B;
  int32_t* s_rank = s_now + P.B;
  __shared__ uint32_t part[THREADS / 32][3];

  const int tid = threadIdx.x;
  const int per = (P.B + THREADS - 1) / THREADS;
  const int b0 = min(P.B, tid * per), b1 = min(P.B, b0 + per);
  const long long cap = P.ring_size;
  Seq one;
  if (b0 < b1) one = load_seq(P, b0);
  const long long head = P.counters[0], tail = P.counters[1];
  long long live = tail - head;
  live = live < 0 ? 0 : live > cap ? cap : live;
  auto wrap = [&](long long i) {  // i modulo cap
    if (i >= 0) return i - divide(i, cap) * cap;
    i %= cap;
    return i < 0 ? i + cap : i;
  };
  const long long h0 = wrap(head), t0 = wrap(tail);

  auto sequence = [&](int b) { return b == b0 ? one : load_seq(P, b); };
  uint32_t sums[3] = {0, 0, 0}, all[3];  // pages taken, pages put back, tokens
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(b);
    sums[0] = add(sums[0], held_at_most(s.grow));
    sums[1] = add(sums[1], held_at_most(s.shrink));
    sums[2] = add(sums[2], held_at_most(s.n));
  }
  block_scan<THREADS>(sums, part, all);
  const long long grow0 = sums[0], shrink0 = sums[1], all_grow = all[0], all_shrink = all[1];
  long long n0 = sums[2], all_n = all[2];
  uint32_t(*part1)[1] = reinterpret_cast<uint32_t(*)[1]>(part);
  if (all_grow > live) {  // tokens of the sequences whose pages run out do not count
    long long g = grow0;
    uint32_t n[1] = {0}, total[1];
    for (int b = b0; b < b1; ++b) {
      const Seq s = sequence(b);
      g += s.grow;
      n[0] = add(n[0], s.grow > 0 && g > live ? 0 : held_at_most(s.n));
    }
    block_scan<THREADS>(n, part1, total);
    n0 = n[0];
    all_n = total[0];
  }
  // ranks of the scheduled tokens: n0 unless some do not fit in the token arrays
  long long u0 = n0, all_u = all_n;
  if (all_n > P.max_tokens) {
    long long g = grow0, m = n0;
    uint32_t u[1] = {0}, total[1];
    for (int b = b0; b < b1; ++b) {
      const Seq s = sequence(b);
      g += s.grow;
      const long long nb = s.grow > 0 && g > live ? 0 : s.n;
      m += nb;
      u[0] = add(u[0], m > P.max_tokens ? 0 : held_at_most(nb));
    }
    block_scan<THREADS>(u, part1, total);
    u0 = u[0];
    all_u = total[0];
  }

  // the sequences: what the tokens need into shared memory, the outputs from CTA 0
  long long g = grow0, f = shrink0, m = n0, u = u0, taken = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(b);
    const long long g_before = g;
    g += s.grow;
    const bool lacks = s.grow > 0 && g > live;
    const long long nb = lacks ? 0 : s.n;
    m += nb;
    const bool full = nb > 0 && m > P.max_tokens;
    const int sched = static_cast<int>(full ? 0 : nb);
    const bool takes = s.grow > 0 && !lacks;
    const long long now = lacks ? s.held : s.held + s.grow - s.shrink;
    s_cu[b] = static_cast<int32_t>(u);
    s_c[b] = static_cast<int32_t>(s.c);
    s_held[b] = s.held;
    s_now[b] = static_cast<int32_t>(now);
    s_rank[b] = static_cast<int32_t>(takes ? g_before : f);
    if (takes) taken += s.grow;
    u += sched;
    f += s.shrink;
    if (blockIdx.x == 0) {
      P.o_ctx[b] = static_cast<int32_t>(s.c);
      P.o_held[b] = static_cast<int32_t>(now);
      P.o_kv[b] = static_cast<int32_t>(s.c + sched);
      P.o_status[b] = s.bad ? -2 : lacks ? -1 : full ? -3 : sched > 0 ? 1 : 0;
      P.o_cu[b] = s_cu[b];
    }
  }
  if (blockIdx.x == 0) {
    uint32_t sum[1] = {held_at_most(taken)}, all_taken[1];
    block_scan<THREADS>(sum, part1, all_taken);
    if (tid == 0) {
      P.o_counters[0] = head + all_taken[0];
      P.o_counters[1] = tail + all_shrink;
      P.o_cu[P.B] = static_cast<int32_t>(all_u);
    }
  }
  if (tid == 0) s_cu[P.B] = static_cast<int32_t>(all_u);
  __syncthreads();

  // table entries of new pages, ring entries of pages put back: a warp a sequence, four loads in
  // flight (a prompt takes hundreds of pages)
  const int lane = tid & 31;
  for (int b = blockIdx.x * (THREADS / 32) + (tid >> 5); b < P.B;
       b += gridDim.x * (THREADS / 32)) {
    const int held = s_held[b], now = s_now[b];
    int32_t* row = P.table + static_cast<long long>(b) * P.max_blocks;
    const bool takes = now > held;
    const long long rank = s_rank[b];
    int count = takes ? now - held : held - now;
    // only counters that are not this ring's can ask for more places than it has
    if (!takes) count = static_cast<int>(max(0LL, min(static_cast<long long>(count), cap - live - rank)));
    for (int j0 = lane; j0 < count; j0 += 128) {
      int32_t page[4];
      long long at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 32 * k;
        at[k] = (takes ? h0 : t0) + rank + j;
        at[k] -= at[k] >= cap ? cap : 0;
        if (j < count) page[k] = takes ? P.ring[at[k]] : row[now + j];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 32 * k;
        if (j < count) (takes ? row[held + j] : P.ring[at[k]]) = page[k];
      }
    }
  }

  // the tokens
  const int total = static_cast<int>(all_u);
  const long long step = static_cast<long long>(gridDim.x) * THREADS * kTbTokens;
  for (long long base = (static_cast<long long>(blockIdx.x) * THREADS + tid) * kTbTokens;
       base < P.max_tokens; base += step) {
    int b = 0;
    if (base < total) {  // last sequence that starts at or before the token
      int lo = 0, hi = P.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= base) lo = mid; else hi = mid;
      }
      b = lo;
    }
    // where each token's page number stands, then all of them, then the results
    const int32_t* at[kTbTokens];
    int pos[kTbTokens], seq[kTbTokens], page[kTbTokens];
#pragma unroll
    for (int j = 0; j < kTbTokens; ++j) {
      const long long t = base + j;
      at[j] = nullptr;
      pos[j] = 0;
      seq[j] = -1;
      if (t >= total) continue;
      while (s_cu[b + 1] <= t) ++b;
      seq[j] = b;
      pos[j] = s_c[b] + static_cast<int>(t - s_cu[b]);
      const int blk = pos[j] >> P.ps_log, held = s_held[b];
      long long i = h0 + s_rank[b] + (blk - held);
      i -= i >= cap ? cap : 0;
      at[j] = blk < held ? P.table + static_cast<long long>(b) * P.max_blocks + blk : P.ring + i;
    }
#pragma unroll
    for (int j = 0; j < kTbTokens; ++j) page[j] = at[j] ? *at[j] : -1;
#pragma unroll
    for (int j = 0; j < kTbTokens; ++j) {
      const long long t = base + j;
      if (t >= P.max_tokens) break;
      P.o_slots[t] = page[j] < 0 ? -1
                                 : (static_cast<long long>(page[j]) << P.ps_log) +
                                       (pos[j] & ((1 << P.ps_log) - 1));
      P.o_pos[t] = pos[j];
      P.o_seq[t] = seq[j];
    }
  }
}

template <int THREADS>
cudaError_t launch_tables(const TablesParams& P, cudaStream_t stream) {
  // a CTA for every THREADS * kTbTokens tokens or 64 sequences, at most two a multiprocessor
  const long long want = 1 + std::max((P.max_tokens - 1) / (THREADS * kTbTokens), (P.B - 1) / 64);
  const int grid = static_cast<int>(std::max(1LL, std::min<long long>(want, 304)));
  const size_t smem = (5 * static_cast<size_t>(P.B) + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        tables_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  tables_kernel<THREADS><<<grid, THREADS, smem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sv

extern "C" sv_status spec_block_tables(
    int B, int page_size, int max_blocks, int max_tokens, const int32_t* ctx_lens,
    const int32_t* accept_len, const int32_t* new_lens, int32_t* block_table, const int32_t* held,
    int32_t* ring, int ring_size, const int64_t* counters, int32_t* out_ctx_lens,
    int32_t* out_held, int64_t* out_counters, int32_t* out_kv_lens, int32_t* out_status,
    int32_t* out_cu_new, int64_t* out_slots, int32_t* out_positions, int32_t* out_seq_ids,
    void* stream) {
  if (B < 0 || max_blocks < 1 || max_tokens < 0 || ring_size < 1) return SV_ERR_INVALID_ARG;
  if (!sv::kv_page_size_ok(page_size)) return SV_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks) * page_size >= (1LL << 31)) return SV_ERR_INVALID_ARG;
  if (!counters || !out_counters || !out_cu_new || !ring) return SV_ERR_INVALID_ARG;
  if (counters == out_counters) return SV_ERR_INVALID_ARG;
  if (B > 0) {
    if (!ctx_lens || !new_lens || !block_table || !held || !out_ctx_lens || !out_held ||
        !out_kv_lens || !out_status)
      return SV_ERR_INVALID_ARG;
    // every CTA reads all lengths while CTA 0 writes the new ones
    const void* in[4] = {ctx_lens, accept_len, new_lens, held};
    const void* out[4] = {out_ctx_lens, out_held, out_kv_lens, out_status};
    for (const void* i : in)
      for (const void* o : out)
        if (i && i == o) return SV_ERR_INVALID_ARG;
  }
  if (max_tokens > 0 && (!out_slots || !out_positions || !out_seq_ids)) return SV_ERR_INVALID_ARG;
  if (B > sv::kTablesMaxB) return SV_ERR_UNSUPPORTED;
  // a sum held at 2^31 - 1 must be past its limit
  if (max_tokens == INT_MAX || ring_size == INT_MAX) return SV_ERR_UNSUPPORTED;
  sv::TablesParams P;
  P.B = B;
  P.ps_log = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  P.max_blocks = max_blocks;
  P.max_tokens = max_tokens;
  P.ring_size = ring_size;
  P.ctx = ctx_lens;
  P.acc = accept_len;
  P.nw = new_lens;
  P.held = held;
  P.table = block_table;
  P.ring = ring;
  P.counters = counters;
  P.o_ctx = out_ctx_lens;
  P.o_held = out_held;
  P.o_kv = out_kv_lens;
  P.o_status = out_status;
  P.o_cu = out_cu_new;
  P.o_pos = out_positions;
  P.o_seq = out_seq_ids;
  P.o_counters = out_counters;
  P.o_slots = out_slots;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = B <= 128   ? sv::launch_tables<128>(P, st)
                                                          : sv::launch_tables<512>(P, st);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
