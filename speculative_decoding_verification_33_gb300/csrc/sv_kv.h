// Shared by the cache operators (sv_tables.cu, sv_normrope.cu, sv_kv4.cu, sv_attn.cu): the layout of the
// 4-bit cache and the host-side interface of the attention kernels.
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

constexpr int kTcMaxRows = 64;  // rows of a tile of the tcgen05 kernel (sv_attn_tc.cu), D = 128
cudaError_t launch_attention_tc(const AttnParams& P, int sms, cudaStream_t stream);

// Bytes of the attention workspace on a device with `sms` multiprocessors; its header is zeroed once.
size_t attention_workspace_bytes(int sms);
cudaError_t launch_attention(const AttnParams& P, int D, int max_new, int sms,
                             cudaStream_t stream);

}  // namespace sv
