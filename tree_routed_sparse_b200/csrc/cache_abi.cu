// cache_abi.cu -- C ABI of the paged 8-bit cache: argument checks and launches.
//
// As in alhr_abi.cu every argument is checked on the host before anything is launched.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "cache_internal.h"

namespace {

using alhr::kMaxRequests;
constexpr int kMaxGroup = 64;
constexpr int kMaxHeads = 65535;           // a grid's second axis
constexpr int64_t kMaxLength = 1 << 30;    // tokens of a block table's row: sums of two stay 32 bits

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool good_block_size(int32_t b) { return b == 16 || b == 32 || b == 64 || b == 128; }

alhr_status check_cache(const alhr_cache* c) {
  if (!c) return ALHR_ERR_INVALID_ARG;
  if (c->blocks < 1 || c->heads < 1) return ALHR_ERR_INVALID_ARG;
  if (!good_block_size(c->block_size)) return ALHR_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return ALHR_ERR_UNSUPPORTED;
  if (c->code != ALHR_CODE_INT8 && c->code != ALHR_CODE_E4M3) return ALHR_ERR_INVALID_ARG;
  if (c->heads > kMaxHeads) return ALHR_ERR_UNSUPPORTED;
  const int64_t rows_per_head = int64_t(c->blocks) * c->block_size;
  if (rows_per_head > INT32_MAX || rows_per_head * c->heads > INT32_MAX)
    return ALHR_ERR_UNSUPPORTED;
  return ALHR_OK;
}

alhr_status check_cache_memory(const alhr_cache* c) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return ALHR_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->k_scale) || !aligned4(c->v_scale))
    return ALHR_ERR_INVALID_ARG;
  return ALHR_OK;
}

int log2_of(int32_t v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

alhr::CacheView view_of(const alhr_cache* c) {
  alhr::CacheView v{};
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.blocks = c->blocks;
  v.heads = c->heads;
  v.bs = c->block_size;
  v.bs_log = log2_of(c->block_size);
  return v;
}

int type_bytes(int32_t type) {
  switch (type) {
    case ALHR_TYPE_BF16:
    case ALHR_TYPE_FP16: return 2;
    case ALHR_TYPE_FP32: return 4;
    case ALHR_TYPE_INT8: return 1;
    default: return 0;
  }
}

// The kernels work with powers of two: scale * log2 e.
float log2_scale(float scale) { return float(double(scale) * 1.4426950408889634); }

alhr_status check_queries(const alhr_cache* c, const alhr_cache_queries* q) {
  const alhr_status s = check_cache(c);
  if (s != ALHR_OK) return s;
  if (!q) return ALHR_ERR_INVALID_ARG;
  if (q->requests < 0 || q->tokens < 0 || q->max_q < 0 || q->q_heads < 1 || q->max_blocks < 1)
    return ALHR_ERR_INVALID_ARG;
  if (q->q_heads % c->heads != 0) return ALHR_ERR_INVALID_ARG;
  if (q->type != ALHR_TYPE_BF16 && q->type != ALHR_TYPE_FP16) return ALHR_ERR_INVALID_ARG;
  if (q->q_token_stride % 8 != 0 || q->q_head_stride % 8 != 0) return ALHR_ERR_INVALID_ARG;
  if (!std::isfinite(log2_scale(q->scale))) return ALHR_ERR_INVALID_ARG;
  if (q->q_heads / c->heads > kMaxGroup || q->requests > kMaxRequests) return ALHR_ERR_UNSUPPORTED;
  if (int64_t(q->tokens) * q->q_heads > INT32_MAX) return ALHR_ERR_UNSUPPORTED;
  if (int64_t(q->max_blocks) * c->block_size > kMaxLength) return ALHR_ERR_UNSUPPORTED;
  return ALHR_OK;
}

alhr_status from_cuda(cudaError_t e) { return e == cudaSuccess ? ALHR_OK : ALHR_ERR_CUDA; }

// Multiprocessors of the current device, 0 on an error. Asked once for each device and thread.
int multiprocessors() {
  static thread_local int known[128] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 128 && known[dev]) return known[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 128) known[dev] = n;
  return n;
}

}  // namespace

extern "C" {

alhr_status alhr_plan_blocks(int32_t requests, int32_t max_blocks, int32_t block_size,
                             int32_t blocks, int32_t tokens, int32_t free_count,
                             const int32_t* ctx_len, const int32_t* new_len,
                             int32_t* block_table, const int32_t* free_blocks,
                             const int32_t* free_first, int32_t* q_start, int32_t* seq_len,
                             int64_t* slots, int32_t* positions, int32_t* free_next,
                             uint32_t* dev_err, void* stream) {
  if (requests < 0 || max_blocks < 1 || blocks < 1 || tokens < 0 || free_count < 0)
    return ALHR_ERR_INVALID_ARG;
  if (!good_block_size(block_size)) return ALHR_ERR_UNSUPPORTED;
  if (requests > kMaxRequests) return ALHR_ERR_UNSUPPORTED;
  if (int64_t(max_blocks) * block_size > kMaxLength) return ALHR_ERR_UNSUPPORTED;
  if (!free_first || !free_next || !q_start) return ALHR_ERR_INVALID_ARG;
  if (requests > 0 && (!ctx_len || !new_len || !block_table || !seq_len))
    return ALHR_ERR_INVALID_ARG;
  if (tokens > 0 && (!slots || !positions)) return ALHR_ERR_INVALID_ARG;
  if (free_count > 0 && !free_blocks) return ALHR_ERR_INVALID_ARG;
  // every CTA reads these while another one may have written its outputs already
  if (free_next == free_first || (requests > 0 && (seq_len == ctx_len || seq_len == new_len)))
    return ALHR_ERR_INVALID_ARG;
  const int sms = multiprocessors();
  if (!sms) return ALHR_ERR_CUDA;
  const alhr::PlanArgs a{requests, max_blocks, block_size, blocks,  tokens,  free_count,
                         ctx_len,  new_len,    block_table, free_blocks, free_first, q_start,
                         seq_len,  slots,      positions,  free_next, dev_err};
  return from_cuda(alhr::launch_plan_blocks(a, sms, static_cast<cudaStream_t>(stream)));
}

alhr_status alhr_store_cache(const alhr_cache* cache, const void* K, const void* V, int32_t type,
                             int32_t tokens, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                             uint32_t* dev_err, void* stream) {
  alhr_status s = check_cache(cache);
  if (s != ALHR_OK) return s;
  if (type != ALHR_TYPE_BF16 && type != ALHR_TYPE_FP16 && type != ALHR_TYPE_FP32)
    return ALHR_ERR_INVALID_ARG;
  if (tokens < 0) return ALHR_ERR_INVALID_ARG;
  const int64_t step = 16 / type_bytes(type);
  if (k_token_stride % step || k_head_stride % step || v_token_stride % step ||
      v_head_stride % step)
    return ALHR_ERR_INVALID_ARG;
  if (tokens == 0) return ALHR_OK;
  s = check_cache_memory(cache);
  if (s != ALHR_OK) return s;
  if (!K || !V || !slots || !aligned16(K) || !aligned16(V)) return ALHR_ERR_INVALID_ARG;
  alhr::StoreArgs a{};
  a.c = view_of(cache);
  a.x[0] = K; a.x[1] = V;
  a.token_stride[0] = k_token_stride; a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride; a.head_stride[1] = v_head_stride;
  a.tokens = tokens; a.slots = slots; a.dev_err = dev_err;
  return from_cuda(alhr::launch_store_cache(a, cache->d, cache->code, type,
                                            static_cast<cudaStream_t>(stream)));
}

alhr_status alhr_load_cache(const alhr_cache* cache, void* K, void* V, int32_t type,
                            int32_t tokens, const int64_t* slots, uint32_t* dev_err,
                            void* stream) {
  alhr_status s = check_cache(cache);
  if (s != ALHR_OK) return s;
  if (type != ALHR_TYPE_BF16 && type != ALHR_TYPE_FP16 && type != ALHR_TYPE_FP32)
    return ALHR_ERR_INVALID_ARG;
  if (tokens < 0) return ALHR_ERR_INVALID_ARG;
  if (tokens == 0) return ALHR_OK;
  s = check_cache_memory(cache);
  if (s != ALHR_OK) return s;
  if (!K || !V || !slots || !aligned16(K) || !aligned16(V)) return ALHR_ERR_INVALID_ARG;
  alhr::LoadArgs a{};
  a.c = view_of(cache);
  a.x[0] = K; a.x[1] = V;
  a.tokens = tokens; a.slots = slots; a.dev_err = dev_err;
  return from_cuda(alhr::launch_load_cache(a, cache->d, cache->code, type,
                                           static_cast<cudaStream_t>(stream)));
}

static size_t workspace_of(const alhr_cache* c, const alhr_cache_queries* q, int sms) {
  const int64_t most = q->max_q == 0 || q->max_q > q->tokens ? q->tokens : q->max_q;
  return alhr::attend_cache_workspace(sms, c->d, most * (q->q_heads / c->heads));
}

size_t alhr_attend_cache_workspace(const alhr_cache* cache, const alhr_cache_queries* queries) {
  if (check_queries(cache, queries) != ALHR_OK) return 0;
  const int sms = multiprocessors();
  return sms ? workspace_of(cache, queries, sms) : 0;
}

alhr_status alhr_attend_cache(const alhr_cache* cache, const alhr_cache_queries* queries,
                              const void* Q, const int32_t* block_table, const int32_t* ctx_len,
                              const int32_t* seq_len, const int32_t* q_start, void* out,
                              float* lse, void* workspace, size_t workspace_bytes,
                              uint32_t* dev_err, void* stream) {
  alhr_status s = check_queries(cache, queries);
  if (s != ALHR_OK) return s;
  if (queries->tokens == 0 || queries->requests == 0) return ALHR_OK;  // nothing to write
  s = check_cache_memory(cache);
  if (s != ALHR_OK) return s;
  if (!Q || !block_table || !ctx_len || !seq_len || !q_start || !out) return ALHR_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace)) return ALHR_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(out)) return ALHR_ERR_INVALID_ARG;
  const int sms = multiprocessors();
  if (!sms) return ALHR_ERR_CUDA;
  if (workspace_bytes < workspace_of(cache, queries, sms)) return ALHR_ERR_INVALID_ARG;
  alhr::AttendArgs a{};
  a.c = view_of(cache);
  a.q = Q; a.out = out; a.lse = lse;
  a.table = block_table; a.ctx_len = ctx_len; a.seq_len = seq_len; a.q_start = q_start;
  a.q_token_stride = queries->q_token_stride; a.q_head_stride = queries->q_head_stride;
  a.requests = queries->requests; a.tokens = queries->tokens; a.q_heads = queries->q_heads;
  a.group = queries->q_heads / cache->heads; a.max_blocks = queries->max_blocks;
  a.max_q = queries->max_q == 0 ? queries->tokens : queries->max_q;
  a.fp16 = queries->type == ALHR_TYPE_FP16;
  a.scale_log2 = log2_scale(queries->scale);
  a.workspace = workspace; a.dev_err = dev_err;
  return from_cuda(alhr::launch_attend_cache(a, cache->d, cache->code, sms,
                                             static_cast<cudaStream_t>(stream)));
}

alhr_status alhr_attend_cache_selected(const alhr_cache* cache,
                                       const alhr_cache_selection* queries, const void* Q,
                                       const int32_t* block_table, const int32_t* ctx_len,
                                       const int32_t* seq_len, const int32_t* idx,
                                       const int32_t* count, float* out, uint32_t* dev_err,
                                       void* stream) {
  alhr_status s = check_cache(cache);
  if (s != ALHR_OK) return s;
  if (!queries) return ALHR_ERR_INVALID_ARG;
  const alhr_cache_selection& q = *queries;
  if (q.batch < 1 || q.q_heads < 1 || q.nq < 0 || q.max_keys < 1 || q.max_blocks < 1)
    return ALHR_ERR_INVALID_ARG;
  if (q.q_heads % cache->heads != 0 || !std::isfinite(log2_scale(q.scale)))
    return ALHR_ERR_INVALID_ARG;
  if (q.type != ALHR_TYPE_INT8 && q.type != ALHR_TYPE_BF16 && q.type != ALHR_TYPE_FP16)
    return ALHR_ERR_INVALID_ARG;
  if (q.max_keys > 96 || q.q_heads / cache->heads > kMaxGroup) return ALHR_ERR_UNSUPPORTED;
  if (int64_t(q.batch) * q.q_heads > INT32_MAX ||
      int64_t(q.batch) * q.q_heads * q.nq > INT32_MAX ||
      int64_t(q.max_blocks) * cache->block_size > kMaxLength)
    return ALHR_ERR_UNSUPPORTED;
  if (q.nq == 0) return ALHR_OK;  // nothing to read or write
  s = check_cache_memory(cache);
  if (s != ALHR_OK) return s;
  if (!Q || !block_table || !ctx_len || !seq_len || !idx || !count || !out)
    return ALHR_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(out)) return ALHR_ERR_INVALID_ARG;
  alhr::SelectArgs a{};
  a.c = view_of(cache);
  a.q = Q; a.out = out; a.table = block_table; a.ctx_len = ctx_len; a.seq_len = seq_len;
  a.idx = idx; a.count = count;
  a.q_heads = q.q_heads; a.group = q.q_heads / cache->heads; a.nq = q.nq;
  a.max_keys = q.max_keys; a.max_blocks = q.max_blocks; a.type = q.type;
  a.rows = q.batch * q.q_heads * q.nq;
  a.scale_log2 = log2_scale(q.scale);
  a.dev_err = dev_err;
  return from_cuda(
      alhr::launch_attend_selected(a, cache->d, cache->code, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
