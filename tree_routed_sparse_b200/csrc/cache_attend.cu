// cache_attend.cu -- attention over all visible keys of each request, from the 8-bit cache.
//
// The simplest form: one warp takes one query row and walks its keys one by one, with the running
// maximum m and sum l of the softmax and fp32 sums.
#include <cmath>

#include "cache_device.cuh"

namespace alhr {

namespace {

constexpr int kRowWarps = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// State of one row: lane holds numbers [lane * E, lane * E + E) of q and of the sum.
template <int D, int CODE>
struct Row {
  static constexpr int E = D / 32;
  float q[E], o[E], m, l;
  __device__ void start() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
  }
  __device__ void key(const CacheView& c, int block, int head, int off, int lane, float scale) {
    const long long at = (block_row(c, block, head) + off) * D + lane * E;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) dot += q[i] * decode<CODE>(__ldg(c.k + at + i));
    const long long si = static_cast<long long>(block) * c.heads + head;
    const float s = warp_sum(dot) * __ldg(c.k_scale + si) * scale;
    const float mn = fmaxf(m, s), keep = exp2f(m - mn), p = exp2f(s - mn);
    const float w = p * __ldg(c.v_scale + si);
    l = l * keep + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * decode<CODE>(__ldg(c.v + at + i));
  }
};

template <int D, int CODE>
__global__ void __launch_bounds__(kRowWarps * 32) attend_selected_kernel(const SelectArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  for (long long u = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
       u < a.rows; u += static_cast<long long>(gridDim.x) * kRowWarps) {
    const int t = static_cast<int>(u % a.nq);
    const long long bh = u / a.nq;
    const int b = static_cast<int>(bh / a.q_heads), h = static_cast<int>(bh % a.q_heads);
    const long long cap = static_cast<long long>(a.max_blocks) << a.c.bs_log;
    const long long pos = static_cast<long long>(__ldg(a.ctx_len + b)) + t;
    const long long see = min(min(pos + 1, static_cast<long long>(__ldg(a.seq_len + b))), cap);
    Row<D, CODE> row;
    const long long qa = u * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      row.q[i] = a.type == ALHR_TYPE_INT8
                     ? static_cast<float>(static_cast<const int8_t*>(a.q)[qa + i])
                 : a.type == ALHR_TYPE_FP16
                     ? __half2float(static_cast<const __half*>(a.q)[qa + i])
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[qa + i]);
    row.start();
    const int count = min(__ldg(a.count + u), a.max_keys);
    bool bad = false, out_of_range = false;
    for (int e = 0; e < count; ++e) {
      const int j = __ldg(a.idx + u * a.max_keys + e);
      if (j < 0 || j >= see) { out_of_range = true; continue; }
      const int block = __ldg(a.table + (long long)b * a.max_blocks + (j >> a.c.bs_log));
      if (block < 0 || block >= a.c.blocks) { bad = true; continue; }
      row.key(a.c, block, h / a.group, j & (a.c.bs - 1), lane, a.scale_log2);
    }
    if (bad && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
    if (out_of_range && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_INDEX);
    const float inv = row.l > 0.f ? 1.f / row.l : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) a.out[qa + i] = row.o[i] * inv;
  }
}

unsigned grid_of(long long rows) {
  const long long g = (rows + kRowWarps - 1) / kRowWarps;
  return static_cast<unsigned>(g < (1 << 20) ? g : (1 << 20));
}

}  // namespace

// Rows of one key head up to which a request is decoded (cache_decode.cu) and from which on it is
// taken as a chunk (cache_chunk.cu): a key tile costs the chunk kernel the same for 1 to 128 rows,
// the decoding one in proportion to groups of 16.
constexpr int kFewRows = 16;

// max_rows: the most rows of one key head that a request may have.
size_t attend_cache_workspace(int sms, int d, long long max_rows) {
  const size_t few = decode_workspace(sms, d), many = chunk_workspace(sms, d);
  return max_rows > kFewRows && many > few ? many : few;
}

cudaError_t launch_attend_cache(const AttendArgs& a, int d, int code, int sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.max_q < a.tokens ? a.max_q : a.tokens) * a.group;
  if (rows <= kFewRows) return launch_decode(a, d, code, sms, 0x7fffffff, st);
  // the two take turns with the workspace
  const cudaError_t e = launch_decode(a, d, code, sms, kFewRows, st);
  return e != cudaSuccess ? e : launch_chunk(a, d, code, sms, kFewRows, a.workspace, st);
}

cudaError_t launch_attend_selected(const SelectArgs& a, int d, int code, int, cudaStream_t st) {
  const unsigned grid = grid_of(a.rows);
  auto kernel = d == 64 ? (code == ALHR_CODE_INT8 ? attend_selected_kernel<64, ALHR_CODE_INT8>
                                                  : attend_selected_kernel<64, ALHR_CODE_E4M3>)
                        : (code == ALHR_CODE_INT8 ? attend_selected_kernel<128, ALHR_CODE_INT8>
                                                  : attend_selected_kernel<128, ALHR_CODE_E4M3>);
  kernel<<<grid, kRowWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace alhr
