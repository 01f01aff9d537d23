// cache_attend.cu -- which kernel takes which requests of an attention over all keys.
#include "cache_internal.h"

namespace alhr {

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

}  // namespace alhr
