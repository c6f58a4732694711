// Shared by the cache operators (sv_tables.cu, sv_normrope.cu, sv_kv4.cu, sv_kv8.cu, sv_attn.cu, ...): the
// layouts of the 4-bit and the 8-bit cache and the host-side interface of the attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace sv {

constexpr int kTablesMaxB = 8192;  // 20 bytes of shared memory a sequence

inline bool kv_page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }
inline bool kv_head_dim_ok(int D) { return D == 64 || D == 128; }

// Byte offsets inside one block of 16 tokens of one head (see include/spec_kv.h).
template <int D>
struct KvBlock {
  static constexpr int kKeyCodes = 0;
  static constexpr int kKeyScales = 8 * D;
  static constexpr int kValCodes = 9 * D;
  static constexpr int kValScales = 17 * D;
  static constexpr int kBytes = 18 * D;
  static constexpr int kChunk = D / 8;  // bytes of one chunk of a value pair's codes
  // place of chunk g of pair p
  static __host__ __device__ constexpr int place(int p, int g) {
    return D == 128 ? g ^ ((p & 3) << 1) : g ^ (((p >> 1) & 1) << 2);
  }
};

// The same of the 8-bit cache.
template <int D>
struct Kv8Block {
  static constexpr int kKeyCodes = 0;
  static constexpr int kValCodes = 16 * D;
  static constexpr int kHead = 32 * D;  // int8 exponents of keys and values; at 4 and 6 uint16 marks
  static constexpr int kBytes = 32 * D + 16;
  // place of 16-byte chunk j of token i's key codes, and of token pair p's value codes
  static __host__ __device__ constexpr int key_place(int i, int j) { return D == 128 ? j ^ (i & 1) : j; }
  static __host__ __device__ constexpr int val_place(int p, int j) { return j ^ ((p & 3) << 1); }
};
constexpr int kKv8Low = -60, kKv8High = 121;  // exponents

#ifdef __CUDACC__
// a / b for a >= 0, b > 0: the 64-bit division takes some hundred instructions, few calls need it
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

#endif

// Attention of new tokens over the cache (sv_attn.cu).
struct AttnParams {
  int B, T, hq, hkv, group;  // group = hq / hkv
  int ps, num_pages, max_blocks;
  long long qs;  // token stride of q in elements
  const void* q;
  const unsigned char* cache;
  const int32_t *table, *lens, *cu;
  float c;    // scale * k_scale * log2(e)
  float vs;   // v_scale
  void* out;
  float* lse;
  // workspace: error word, arrivals at the items cut between CTAs (zero between calls), pieces
  unsigned* err;
  unsigned* arrived;
  float* part;
};

constexpr size_t kAttnHeader = 4096;  // bytes before the pieces: error word at 0, arrivals from 256
constexpr int kAttnMaxCtas = (4096 - 256) / 4;

constexpr int kPieceRows = 256;
constexpr int kTcMaxRows = 64;  // rows of a tile of the tcgen05 kernel (sv_attn_tc.cu), D = 128
cudaError_t launch_attention_tc(const AttnParams& P, int sms, cudaStream_t stream);

// Bytes of the attention workspace on a device with `sms` multiprocessors; its header is zeroed once.
size_t attention_workspace_bytes(int sms);
cudaError_t launch_attention(const AttnParams& P, int D, int max_new, int sms,
                             cudaStream_t stream);
// The same over the 8-bit cache (sv_attn8.cu); k_scale and v_scale count as 1.
cudaError_t launch_attention8(const AttnParams& P, int D, int max_new, int sms, cudaStream_t stream);
// ... for `rows` rows a head or so, many of them (sv_attn8_tc.cu)
cudaError_t launch_attention8_tc(const AttnParams& P, int D, long long rows, int sms, cudaStream_t stream);

// Causal attention over whole prompts (sv_prompt.cu).
struct PromptParams {
  int B, T, hq, hkv, group;
  long long qs, ks, vs;  // token strides in elements
  const void *q, *k, *v;
  const int32_t* cu;
  float c;  // scale * log2(e)
  void* out;
  float* lse;
  // workspace: error word; counters of items fetched and of CTAs at their end (zero between calls)
  unsigned *err, *queue;
};
cudaError_t launch_prompt(const PromptParams& P, int D, int sms, cudaStream_t stream);

}  // namespace sv
