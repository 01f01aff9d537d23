// cache_attend.cu -- which kernel takes which requests of an attention over all keys.
#include "cache_internal.h"

namespace alhr {

// Rows of one key head up to which a request is decoded (cache_decode.cu) and from which on it is
// taken as a chunk (cache_chunk.cu): a key tile costs the chunk kernel the same for 1 to 128 rows,
// the decoding one in proportion to groups of 16. Measured, 16 requests of 16,384 int8 keys x 8 key
// heads, microseconds of the one and the other kernel:
//   rows        8          16         17 to 32     48         64         96         128
//   d = 64      62 / 199   77 / 199   128 / 200    181 / 199  233 / 200  343 / 202  450 / 203
//   d = 128     98 / 287   117 / 287  203 / 289    295 / 289  381 / 289  563 / 292  748 / 297
// So they meet near 48 rows: at 17 to 47 the chunk kernel is the slower one, by 1.6 and 1.4 times
// at 32, and neither is near the 41 and 82 us that the codes alone take.
constexpr int kFewRows = 16;

// max_rows: the most rows of one key head that a request may have.
size_t attend_cache_workspace(int sms, int d, long long max_rows) {
  return decode_workspace(sms, d) + (max_rows > kFewRows ? chunk_workspace(sms, d) : 0);
}

cudaError_t launch_attend_cache(const AttendArgs& a, int d, int code, int sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.max_q < a.tokens ? a.max_q : a.tokens) * a.group;
  const bool chunks = rows > kFewRows;
  cudaError_t e = launch_decode(a, d, code, sms, chunks ? kFewRows : 0x7fffffff, st);
  if (chunks && e == cudaSuccess) {
    AttendArgs b = a;
    b.workspace = static_cast<char*>(a.workspace) + decode_workspace(sms, d);
    e = launch_chunk(b, d, code, sms, kFewRows, st);
    if (e == cudaSuccess) e = launch_chunk_join(b, d, sms, st);
  }
  return e != cudaSuccess ? e : launch_decode_join(a, d, sms, st);
}

}  // namespace alhr
