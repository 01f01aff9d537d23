// cache_internal.h -- launchers of the paged 8-bit cache, shared by its ABI layer and kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/alhr_cache.h"

namespace alhr {

constexpr int kMaxRequests = 8192;  // the plan keeps two words a request in shared memory

struct PlanArgs {
  int requests, max_blocks, block_size, blocks, tokens, free_count;
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* free_first;
  int32_t* q_start;
  int32_t* seq_len;
  int64_t* slots;
  int32_t* positions;
  int32_t* free_next;
  uint32_t* dev_err;
};

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int blocks, heads, bs, bs_log;
};

struct StoreArgs {
  CacheView c;
  const void* x[2];  // keys, values
  long long token_stride[2], head_stride[2];
  int tokens;
  const int64_t* slots;
  uint32_t* dev_err;
};

struct LoadArgs {
  CacheView c;
  void* x[2];
  int tokens;
  const int64_t* slots;
  uint32_t* dev_err;
};

struct AttendArgs {
  CacheView c;
  const void* q;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* ctx_len;
  const int32_t* seq_len;
  const int32_t* q_start;
  long long q_token_stride, q_head_stride;
  int requests, tokens, q_heads, group, max_blocks, max_q, fp16;
  float scale_log2;  // scale * log2 e: the kernels work with powers of two
  void* workspace;
  uint32_t* dev_err;
};

struct SelectArgs {
  CacheView c;
  const void* q;
  float* out;
  const int32_t* table;
  const int32_t* ctx_len;
  const int32_t* seq_len;
  const int32_t* idx;
  const int32_t* count;
  int q_heads, group, nq, max_keys, max_blocks, type;
  int rows;  // batch * q_heads * nq
  float scale_log2;
  uint32_t* dev_err;
};

cudaError_t launch_plan_blocks(const PlanArgs& a, int sms, cudaStream_t st);
cudaError_t launch_store_cache(const StoreArgs& a, int d, int code, int type, cudaStream_t st);
cudaError_t launch_load_cache(const LoadArgs& a, int d, int code, int type, cudaStream_t st);
size_t attend_cache_workspace(int sms, int d, long long max_rows);
cudaError_t launch_attend_cache(const AttendArgs& a, int d, int code, int sms, cudaStream_t st);
size_t decode_workspace(int sms, int d);
cudaError_t launch_decode(const AttendArgs& a, int d, int code, int sms, int row_limit,
                          cudaStream_t st);
cudaError_t launch_decode_join(const AttendArgs& a, int d, int sms, cudaStream_t st);
size_t chunk_workspace(int sms, int d);
cudaError_t launch_chunk(const AttendArgs& a, int d, int code, int sms, int row_limit,
                         cudaStream_t st);
cudaError_t launch_chunk_join(const AttendArgs& a, int d, int sms, cudaStream_t st);
cudaError_t launch_attend_selected(const SelectArgs& a, int d, int code, cudaStream_t st);

}  // namespace alhr
