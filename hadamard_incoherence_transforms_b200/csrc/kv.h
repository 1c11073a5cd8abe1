// Launcher interface of the rotated key/value cache (host-side C++).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace hit {

// The cache, the call's sequences and the rotary positions (see hit.h).
struct KvArgs {
  uint8_t* k_codes = nullptr;
  uint8_t* v_codes = nullptr;
  float* k_scales = nullptr;
  float* v_scales = nullptr;
  const int32_t* table = nullptr;
  const int32_t* lens = nullptr;
  const int32_t* cu = nullptr;
  const int8_t* k_signs = nullptr;
  const int8_t* v_signs = nullptr;
  const float* inv_freq = nullptr;
  const int32_t* positions = nullptr;
  const int8_t* rope_axis = nullptr;
  int64_t pages = 0, ld_table = 0, ld_pos = 0;
  int64_t tokens = 0;
  int hk = 1, log_page = 0, seqs = 0, max_pages = 0;
  int n_freq = 0, interleaved = 0, rope_axes = 1;
  int head_dim = 0, bits = 0;
};

// Dense keys and values (either may be NULL for reading).
struct KvDense {
  const void* k = nullptr;
  const void* v = nullptr;
  int64_t k_ts = 0, k_hs = 0, v_ts = 0, v_hs = 0;
};
cudaError_t launch_kv_append(const KvArgs& a, const KvDense& x, int dt, cudaStream_t st);
// zero: rows of tokens that belong to no sequence are set to zero
cudaError_t launch_kv_read(const KvArgs& a, const KvDense& y, int dt, bool zero, cudaStream_t st);
// All rows [tokens, heads, head_dim] of out.
cudaError_t launch_kv_zero(void* out, int64_t tokens, int heads, int head_dim, int64_t ts, int64_t hs, int dt,
                           cudaStream_t st);

struct KvAttn {
  const void* q = nullptr;
  void* out = nullptr;
  int64_t q_ts = 0, q_hs = 0, o_ts = 0, o_hs = 0;
  int heads = 0, group = 1;  // query heads; of one key/value head
  int q_f32 = 0, o_f32 = 0, causal = 1;
  int wide = 0;  // every row of out starts on a 32-byte boundary
  int zero = 0;  // the launch sets the rows of tokens that belong to no sequence to zero
  int64_t rows_lo = 0, rows_hi = INT64_MAX;  // sequences with this many query rows (token * group) belong to the launch
  float scale = 1.0f;
  int64_t window = 0;
  int64_t max_new = 1;
  void* ws = nullptr;
};
size_t kv_few_bytes(int head_dim);  // workspace
cudaError_t launch_kv_few(const KvArgs& a, const KvAttn& t, cudaStream_t st);
size_t kv_prompt_bytes(int64_t tokens, int heads, int head_dim);
cudaError_t launch_kv_prompt_queries(const KvArgs& a, const KvAttn& t, cudaStream_t st);
cudaError_t launch_kv_prompt(const KvArgs& a, const KvAttn& t, cudaStream_t st);
cudaError_t wait_timeouts_kv(unsigned long long* count, bool reset);

}  // namespace hit
