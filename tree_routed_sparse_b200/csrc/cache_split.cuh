// cache_split.cuh -- equal pieces of one list of key tiles, and the join of the units they cut.
#pragma once

#include <cmath>

#include "cache_mma.cuh"

namespace alhr {

// Rows and visible keys of one request, inside the arrays whatever the device memory holds.
struct RequestRange {
  int q_lo, tokens, ctx, see;
  __device__ __forceinline__ RequestRange(const AttendArgs& a, int r) {
    q_lo = min(max(__ldg(a.q_start + r), 0), a.tokens);
    tokens = min(max(__ldg(a.q_start + r + 1), q_lo), a.tokens) - q_lo;
    ctx = __ldg(a.ctx_len + r);
    const long long cap = static_cast<long long>(a.max_blocks) << a.c.bs_log;
    const long long end = min(min(static_cast<long long>(ctx) + tokens,
                                  static_cast<long long>(__ldg(a.seq_len + r))), cap);
    see = static_cast<int>(max(end, 0LL));
  }
};

// `tiles` tiles in `pieces` pieces: piece i begins at tile first(i).
struct Split {
  long long tiles;
  int pieces;
  __device__ __forceinline__ long long first(int i) const { return tiles * i / pieces; }
  __device__ __forceinline__ int piece_of(long long tile) const {
    return static_cast<int>(((tile + 1) * pieces - 1) / tiles);
  }
};

// The list of a CTA whose thread t has `mine` tiles (a run of requests): start[t] is where they
// begin. A short list is cut into single tiles, so that every piece it has holds one at least.
template <int THREADS>
__device__ __forceinline__ Split make_split(long long mine, long long* start, long long* warp_sum,
                                            long long most_pieces) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    before += w < warp ? warp_sum[w] : 0;
    all += warp_sum[w];
  }
  start[threadIdx.x] = before + incl - mine;
  __syncthreads();
  return Split{all, static_cast<int>(min(most_pieces, all))};
}

// The last thread whose tiles begin at or before `tile`: threads without any share their start
// with the next one, so that it has some.
template <int THREADS>
__device__ __forceinline__ int chunk_of(const long long* start, long long tile) {
  int lo = 0, hi = THREADS - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A unit that begins in a piece and ends in a later one: its rows, and the piece that ends it
// (-1: the piece has no such unit).
struct JoinMeta {
  int r, h, row0, rows, last;
};

struct JoinSpace {
  JoinMeta* meta;  // [pieces]
  float* part;     // [pieces][2] of y [ROWS][D], R [ROWS], l [ROWS]: of a unit that began in an
                   // earlier piece, of one that begins here
};

// l 2^r with l in [2^to, 2^(to + 1)).
__device__ __forceinline__ void settle(float& r, float& l, int to) {
  if (l > 0.f) {  // not 0 (no key), not NaN
    const int k = min(static_cast<int>(__float_as_uint(l) >> 23) - 127 - to, 126);
    l *= power_of_two(-k);
    r += static_cast<float>(k);
  }
}
// A piece leaves its own answer y = sum p v / sum p, and sum p = l 2^R with l about 2^-12: the weights
// l_i 2^(R_i - max R) of up to 2^11 pieces add up to no more than 1, so that the sum of y_i times
// weight is in range where the values are.
constexpr int kPartLog = -12;

inline size_t join_bytes(int pieces, int rows, int d) {
  return static_cast<size_t>(pieces) * (32 + 2 * static_cast<size_t>(rows) * (d + 2) * sizeof(float));
}
inline JoinSpace join_space(void* workspace, int pieces) {
  return JoinSpace{static_cast<JoinMeta*>(workspace),
                   reinterpret_cast<float*>(static_cast<char*>(workspace) + pieces * 32)};
}

// The next kernel of the stream may be set up while this one runs (it waits before it reads what
// this one writes).
__device__ __forceinline__ void let_next_begin() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// Launches a kernel that waits for the previous one of the stream by itself.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                          cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

constexpr int kJoinWarps = 8;

// Joins the partial sums of the units that span pieces, one CTA for each piece in which such a unit
// begins. Up to eight warps share a row: each joins every k-th partial (the lanes take 32 weights
// l_i 2^(R_i - max R) at a time, so that the loads of y do not wait for one another), then their
// sums are added in the order of the warps.
template <int D, int ROWS>  // ROWS <= 16
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttendArgs a,
                                                               const JoinSpace space) {
  wait_for_previous();
  constexpr int E = D / 32, kStep = ROWS * (D + 2);
  const int piece = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const JoinMeta p = space.meta[piece];
  const int rows = p.rows;
  if (p.last < 0) return;
  int shared_by = 1;  // warps of a row
  while (rows * shared_by * 2 <= kJoinWarps) shared_by *= 2;
  __shared__ float sums[kJoinWarps][D + 2];
  const int n = p.last - piece + 1, sub = warp % shared_by;
  // partials: slot 1 of this piece, slot 0 of the pieces behind it
  auto part = [&](int i) {
    return space.part + (static_cast<long long>(piece + i) * 2 + (i == 0 ? 1 : 0)) * kStep;
  };
  for (int r = warp / shared_by; r < rows; r += kJoinWarps / shared_by) {
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, part(i)[ROWS * D + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float acc[E], l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int mine = (n - sub + shared_by - 1) / shared_by;  // partials sub, sub + shared_by, ...
    for (int i0 = 0; i0 < mine; i0 += 32) {
      float f = 0.f;
      if (i0 + lane < mine) {
        const float* x = part(sub + (i0 + lane) * shared_by) + ROWS * D + r;
        f = exp2_fast(x[0] - base) * x[ROWS];
        l += f;
      }
      const int some = min(32, mine - i0);
#pragma unroll 8
      for (int i = 0; i < some; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        const float* x = part(sub + (i0 + i) * shared_by) + r * D + lane * E;
        if constexpr (E == 4) {
          const float4 y = *reinterpret_cast<const float4*>(x);
          acc[0] = fmaf(y.x, w, acc[0]);
          acc[1] = fmaf(y.y, w, acc[1]);
          acc[2] = fmaf(y.z, w, acc[2]);
          acc[3] = fmaf(y.w, w, acc[3]);
        } else {
          const float2 y = *reinterpret_cast<const float2*>(x);
          acc[0] = fmaf(y.x, w, acc[0]);
          acc[1] = fmaf(y.y, w, acc[1]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (shared_by > 1) {  // then every warp has one row at most, and all of them come here
#pragma unroll
      for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
      if (lane == 0) sums[warp][D] = l;
      // the warps of rows that there are
      asm volatile("bar.sync 1, %0;\n" ::"r"(rows * shared_by * 32) : "memory");
      if (sub == 0) {
        for (int k = 1; k < shared_by; ++k) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += sums[warp + k][lane * E + e];
          l += sums[warp + k][D];
        }
      }
    }
    if (sub == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no key; NaN stays
      const int rr = p.row0 + r, tok = rr / a.group;
      const int q_lo = min(max(__ldg(a.q_start + p.r), 0), a.tokens);
      const long long at = static_cast<long long>(q_lo + tok) * a.q_heads + p.h * a.group +
                           (rr - tok * a.group);
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * D + lane * E + e) =
            pack2(acc[e] * inv, acc[e + 1] * inv, a.fp16);
      if (a.lse && lane == 0)
        a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// The same for units of many rows, of which most span two or three pieces: a thread takes four
// numbers of two rows through all partials, with a running max R, so that a row costs two dependent
// trips to memory (the unit, its partials) and all rows of a CTA make them together: 9 us for 144
// units of 256 rows in 31 tiles a piece, d = 64, where a warp for each pair of rows took 20 and two
// passes over the partials 12. (y with the rows innermost would be written in whole lines, 1 us less
// in a chunk's CTAs, and read in parts of lines here, 3 us more.)
template <int D, int ROWS>
__global__ void __launch_bounds__(256) join_rows_kernel(const AttendArgs a, const JoinSpace space) {
  wait_for_previous();
  constexpr int kLanes = D / 4, kAtOnce = 256 / kLanes, kEach = 2, kHere = kEach * kAtOnce;
  constexpr long long kStep = ROWS * (D + 2);
  const int piece = blockIdx.x, row0 = blockIdx.y * kHere + threadIdx.x / kLanes;
  const JoinMeta p = space.meta[piece];
  if (p.last < 0 || static_cast<int>(blockIdx.y) * kHere >= p.rows) return;
  const int n = p.last - piece + 1, col = threadIdx.x % kLanes * 4;
  // partials: slot 1 of this piece, slot 0 of the pieces behind it
  const float* const slots = space.part + piece * 2 * kStep;
  auto part = [&](int i) { return slots + (i == 0 ? kStep : 2 * i * kStep); };
  float m[kEach], l[kEach], acc[kEach][4];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
  }
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* const x = part(i);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int row = row0 + k * kAtOnce;
      const float4 y = *reinterpret_cast<const float4*>(x + row * D + col);
      const float mi = x[ROWS * D + row], li = x[ROWS * D + ROWS + row];
      const float mn = fmaxf(m[k], mi), base = mn == -INFINITY ? 0.f : mn;
      const float keep = exp2_fast(m[k] - base), w = exp2_fast(mi - base) * li;
      m[k] = mn;
      l[k] = fmaf(l[k], keep, w);
      acc[k][0] = fmaf(y.x, w, acc[k][0] * keep);
      acc[k][1] = fmaf(y.y, w, acc[k][1] * keep);
      acc[k][2] = fmaf(y.z, w, acc[k][2] * keep);
      acc[k][3] = fmaf(y.w, w, acc[k][3] * keep);
    }
  }
  const int q_lo = min(max(__ldg(a.q_start + p.r), 0), a.tokens);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int row = row0 + k * kAtOnce;
    if (row >= p.rows) continue;
    const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];  // no key; NaN stays
    const int rr = p.row0 + row, tok = rr / a.group;
    const long long at = static_cast<long long>(q_lo + tok) * a.q_heads + p.h * a.group +
                         (rr - tok * a.group);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + col) =
        make_uint2(pack2(acc[k][0] * inv, acc[k][1] * inv, a.fp16),
                   pack2(acc[k][2] * inv, acc[k][3] * inv, a.fp16));
    if (a.lse && col == 0)
      a.lse[at] = l[k] == 0.f ? -INFINITY : (m[k] + log2f(l[k])) * 0.6931471805599453f;
  }
}

template <int D, int ROWS>
cudaError_t launch_join(const AttendArgs& a, const JoinSpace& space, int pieces, cudaStream_t st) {
  if constexpr (ROWS > 16)
    return launch_behind(join_rows_kernel<D, ROWS>, dim3(pieces, ROWS / (512 / (D / 4))), 256, 0, st, a, space);
  else
    return launch_behind(join_kernel<D, ROWS>, dim3(pieces), kJoinWarps * 32, 0, st, a, space);
}

}  // namespace alhr
