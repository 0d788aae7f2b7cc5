// Internal interfaces between the C ABI layer and the serving kernels (rotary
// positions, the FP8 KV cache, attention over the cache).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace fpattn {

// bf16 rows [B, T, H, d]; strides in elements.
struct Rows {
  void* data;
  int B, T, H, d;
  long long sb, st, sh;
};

struct RotaryTable {
  const unsigned long long* turns;  // device, dim / 2
  int dim;                          // 0: no rotation
  int interleaved;
  float magnitude;
};

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* exps;
  int num_pages, H, page_size, d;
};

struct CacheAttnArgs {
  KvCache cache;
  const void* q;
  long long q_sb, q_st, q_sh;
  const int* q_start;  // or null
  int B, Tmax, rows_total, Hq;
  const int* page_table;
  int max_pages;
  long long page_table_stride;
  const int* lengths;
  int causal;
  const long long* tree;
  int tree_words;
  long long tree_sb;
  float scale;  // softmax scale, > 0
  void* out;
  float* lse;
  void* workspace;
};

cudaError_t launch_rotary(const Rows& x, const RotaryTable& tab, const long long* positions, bool per_b,
                          bool transpose, const Rows& out, cudaStream_t st);
cudaError_t launch_cache_write(const KvCache& c, const Rows& k, const Rows& v, const long long* slots,
                               const RotaryTable& tab, const long long* positions, const Rows* q, const Rows* q_out,
                               int* nonfinite, cudaStream_t st);
cudaError_t launch_cache_read(const KvCache& c, const long long* slots, const Rows& k, const Rows& v,
                              cudaStream_t st);
cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t st);
// The most units of work the launch above may plan (it counts them in 32 bits).
double cache_attention_units(const CacheAttnArgs& a);
// Bytes of device workspace the launch above needs for these sizes.
size_t cache_attention_workspace(const CacheAttnArgs& a);
// Error word of the cache attention's bounded waits.
cudaError_t read_cache_attn_error(cudaStream_t st, int clear, int* code);

}  // namespace fpattn
