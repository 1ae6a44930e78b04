// Internal interfaces of the paged FP4 key/value cache: its byte layout, the kernels' parameters
// and the launch functions (sharq_api.cu calls them after its checks).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace sharq {

// ---------------------------------------------------------------- the cache's bytes
// A page holds page_size tokens of every key head; the bytes of (page, head) are contiguous and
// consist of page_size / 16 groups of 16 tokens. A group is one contiguous block
//   K codes   16 rows x D/2 bytes, row by row, the lower element in the low nibble
//   V codes   16 x D/2 bytes in the order of the value product's matrix fragments
//   K scales  16 x D/B bytes, row by row
//   V scales  16 x D/B bytes in fragment order
// so 16 tokens of one head are one copy whatever the page size. Token r = 8h + 2t + j of a group
// (h, j in 0..1, t in 0..3) is contraction slot (2t + j) + 8h of a 16-wide matrix step, and a run
// g of D/8 consecutive elements belongs to the lanes 4g..4g+3: lane 4g + t finds the four tokens
// that it holds of a step in 16 (D = 64) or 2 x 16 (D = 128) consecutive bytes.
struct KvLayout {
  int k_codes, v_codes, k_scales, v_scales, bytes;
};
__host__ __device__ constexpr int kv_block(int fmt) { return fmt == 0 ? 16 : 32; }
__host__ __device__ constexpr KvLayout kv_group(int d, int fmt) {
  return KvLayout{0, 8 * d, 16 * d, 16 * d + 16 * (d / kv_block(fmt)), 16 * d + 32 * (d / kv_block(fmt))};
}
// byte, inside the V codes, of the D/16 bytes of (row r, run g)
__host__ __device__ constexpr int kv_v_place(int d, int r, int g) {
  return d == 128 ? (64 * (r >> 3) + 2 * (4 * g + ((r >> 1) & 3)) + (r & 1)) * 8
                  : (4 * (4 * g + ((r >> 1) & 3)) + 2 * (r >> 3) + (r & 1)) * 4;
}
// byte, inside the V scales, of block b of row r
__host__ __device__ constexpr int kv_v_scale_place(int r, int b) {
  return (4 * b + ((r >> 1) & 3)) * 4 + 2 * (r >> 3) + (r & 1);
}
// MXFP4 block exponents of the cache: 2^-23 .. 2^13, so that every value is a float16
constexpr int kKvExpMin = 127 - 23, kKvExpMax = 127 + 13;

struct KvCacheView {
  uint8_t *pages;
  const float *k_scale, *v_scale;  // [kv_heads] or null (1)
  int num_pages, page_shift, kv_heads;
};

struct KvBatchView {
  const int *cu_q;        // [n_seq + 1]
  const int *kv_len;      // [n_seq]
  const int *page_table;  // [n_seq][max_pages]
  int n_seq, max_pages, max_q, tokens;
};

struct AppendParams {
  const uint16_t *qkv;
  long long row_stride;
  const uint16_t *q_gamma, *k_gamma;
  const float *inv_freq;
  uint16_t *q_out;
  float eps;
  int q_heads, rot_half, interleaved;
  KvBatchView b;
  KvCacheView c;
};

struct ReadParams {
  void *k_out, *v_out;
  int out_f32;
  KvBatchView b;
  KvCacheView c;
};

struct AttnParams {
  const uint16_t *q;
  long long q_stride;
  uint16_t *y;   // [tokens][q_heads][D]
  float *lse;    // [tokens][q_heads] or null
  float scale_log2;  // softmax scale * log2(e)
  int q_heads, group;  // group = q_heads / kv_heads
  uint32_t group_inv;  // ceil(2^32 / group): row / group = high word of row * group_inv, group > 1, row < 2^32 / group
  int causal, window;  // window 0: none
  uint8_t *workspace;
  unsigned long long limit_ns;  // of the bounded waits
  KvBatchView b;
  KvCacheView c;
};

struct NormResidualParams {
  const uint16_t *y, *post_gamma, *gate, *residual, *pre_gamma;
  uint16_t *residual_out, *h_out;
  float alpha, eps;
  double inv_k;  // 1 / k
  int tokens, k, rows_per_gate;
};

// A kernel's dynamic shared-memory limit, set once per device (1 us of every launch otherwise).
struct SmemOnce {
  std::atomic<uint64_t> devices{0};
  template <class Kernel>
  cudaError_t set(Kernel kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

cudaError_t launch_kv_append(const AppendParams &p, int d, int fmt, cudaStream_t st);
cudaError_t launch_kv_read(const ReadParams &p, int d, int fmt, cudaStream_t st);
cudaError_t launch_attention(const AttnParams &p, int d, int fmt, cudaStream_t st);
// The attention workspace: counters (zero between calls), then parts of cut items.
constexpr int kAttnCounterBytes = 32768;
size_t attention_tiles_workspace(const AttnParams &p, int d);
cudaError_t launch_attention_tiles(const AttnParams &p, int d, int fmt, cudaStream_t st);
cudaError_t read_and_clear_attn_status(uint32_t *status);
cudaError_t read_and_clear_attn_rows_status(uint32_t *status);
size_t attention_workspace(const AttnParams &p, int d);
cudaError_t launch_norm_residual(const NormResidualParams &p, cudaStream_t st);

}  // namespace sharq
