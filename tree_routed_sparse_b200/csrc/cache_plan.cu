// cache_plan.cu -- block table, slots and row offsets of one step, from the request lengths.
//
// Two prefix sums over the requests (token rows, missing blocks) place everything:
//   q_start[r] = sum n,  first free entry of r = free_first + sum (ceil((c+n)/bs) - ceil(c/bs)).
// The sums are short (at most 8192 requests, 64 KB of lengths from L2) and the rows they place may
// be many, so every CTA forms them for itself in shared memory and then writes its share of the
// rows: one launch, no exchange between CTAs. A row's block comes from the free list directly when
// its request gets the block in this very step, so no CTA reads what another one writes. Measured:
// 6.3 us for 64 requests of one token, 9.6 us for 1500 requests and 50,000 tokens; a launch and three
// dependent trips to memory are what it is made of.
#include "cache_device.cuh"

namespace alhr {

namespace {

constexpr int kPlanThreads = 512;

struct Lengths {
  int ctx, held, total, end;  // tokens in the cache, blocks they fill, blocks wanted, tokens wanted
};

__device__ __forceinline__ int blocks_of(int tokens, int bs) {
  return static_cast<int>((static_cast<long long>(tokens) + bs - 1) / bs);
}

__device__ __forceinline__ Lengths request_lengths(const PlanArgs& a, int cap, int r, int rows) {
  Lengths l;
  l.ctx = min(max(__ldg(a.ctx_len + r), 0), cap);
  l.end = static_cast<int>(min(static_cast<long long>(l.ctx) + rows, static_cast<long long>(cap)));
  l.held = blocks_of(l.ctx, a.block_size);
  l.total = blocks_of(l.end, a.block_size);
  return l;
}

// Exclusive sum over the block of one value a thread; *all receives the total.
__device__ __forceinline__ long long block_exclusive(long long v, long long* all) {
  __shared__ long long part[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();  // part is free of an earlier use
  if (lane == 31) part[warp] = s;
  __syncthreads();
  long long before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const long long p = part[w];
    before += w < warp ? p : 0;
    sum += p;
  }
  *all = sum;
  return before + s - v;
}

// Two words a request and the end of the last one.
constexpr int plan_smem_bytes(int requests) {
  return (2 * requests + 1) * static_cast<int>(sizeof(int));
}

__global__ void __launch_bounds__(kPlanThreads) plan_blocks_kernel(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* start = plan_smem;                   // [requests + 1]
  int* base = plan_smem + a.requests + 1;   // [requests] first free entry of each request
  const int R = a.requests, bs = a.block_size, tid = threadIdx.x;
  const int cap = static_cast<int>(min(static_cast<long long>(a.max_blocks) * bs, 0x7fffffffLL));
  const int first = min(max(__ldg(a.free_first), 0), a.free_count);
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  bool cut = false;

  long long rows = 0, all;
  for (int r = r0; r < r1; ++r) rows += max(__ldg(a.new_len + r), 0);
  long long at = block_exclusive(rows, &all);
  if (all > a.tokens) cut = true;
  for (int r = r0; r < r1; ++r) {
    start[r] = static_cast<int>(min(at, static_cast<long long>(a.tokens)));
    at += max(__ldg(a.new_len + r), 0);
  }
  if (tid == 0) start[R] = static_cast<int>(min(all, static_cast<long long>(a.tokens)));
  __syncthreads();

  long long need = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = start[r + 1] - start[r];
    const Lengths l = request_lengths(a, cap, r, n);
    need += l.total - l.held;
    if (l.end - l.ctx < n) cut = true;
  }
  at = first + block_exclusive(need, &all);
  if (first + all > a.free_count) cut = true;
  for (int r = r0; r < r1; ++r) {
    const Lengths l = request_lengths(a, cap, r, start[r + 1] - start[r]);
    base[r] = static_cast<int>(min(at, static_cast<long long>(a.free_count)));
    at += l.total - l.held;
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    if (tid == 0) {
      *a.free_next = static_cast<int>(min(first + all, static_cast<long long>(a.free_count)));
      a.q_start[R] = start[R];
    }
    if (cut) cache_flag(a.dev_err, ALHR_DEVERR_CAPACITY);
  }
  // the requests' own outputs and new table entries: one request a warp
  bool bad = false;
  const int lane = tid & 31;
  for (int r = blockIdx.x * (kPlanThreads / 32) + (tid >> 5); r < R;
       r += gridDim.x * (kPlanThreads / 32)) {
    const Lengths l = request_lengths(a, cap, r, start[r + 1] - start[r]);
    const int had = min(l.total - l.held, a.free_count - base[r]);  // blocks the list still has
    if (lane == 0) {
      a.q_start[r] = start[r];
      const long long room = static_cast<long long>(l.held + had) * bs;
      a.seq_len[r] = static_cast<int>(min(static_cast<long long>(l.end), room));
    }
    int32_t* row = a.table + static_cast<long long>(r) * a.max_blocks;
    for (int j = l.held + lane; j < l.total; j += 32) {
      int block = j - l.held < had ? __ldg(a.free_blocks + base[r] + (j - l.held)) : -1;
      if (j - l.held < had && (block < 0 || block >= a.blocks)) { block = -1; bad = true; }
      row[j] = block;
    }
  }
  // the token rows
  for (long long t = static_cast<long long>(blockIdx.x) * kPlanThreads + tid; t < a.tokens;
       t += static_cast<long long>(gridDim.x) * kPlanThreads) {
    long long slot = -1;
    int pos = -1;
    if (t < start[R]) {
      int lo = 0, hi = R - 1;  // the last r with start[r] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const Lengths l = request_lengths(a, cap, lo, start[lo + 1] - start[lo]);
      const long long p = static_cast<long long>(l.ctx) + t - start[lo];
      pos = static_cast<int>(min(p, 0x7fffffffLL));
      if (p < l.end) {
        const int j = static_cast<int>(p) / bs;
        const int e = base[lo] + (j - l.held);
        const bool there = j < l.held;
        int block = -1;
        if (there) block = __ldg(a.table + static_cast<long long>(lo) * a.max_blocks + j);
        else if (e < a.free_count) block = __ldg(a.free_blocks + e);
        if (block >= 0 && block < a.blocks)
          slot = static_cast<long long>(block) * bs + static_cast<int>(p) % bs;
        else if (there || e < a.free_count)
          bad = true;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  if (__syncthreads_or(bad) && tid == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
}

}  // namespace

cudaError_t launch_plan_blocks(const PlanArgs& a, int sms, cudaStream_t st) {
  // One limit for every call, whatever its size: it belongs to the kernel, not to the call, and
  // another thread may be between its own limit and its launch.
  static thread_local bool configured[128] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        plan_blocks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, plan_smem_bytes(kMaxRequests));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) configured[dev] = true;
  }
  // a CTA for every 1024 rows or 64 requests, at most one a multiprocessor
  const long long by_rows = (static_cast<long long>(a.tokens) + 1023) / 1024;
  const long long by_requests = (a.requests + 63) / 64;
  const int grid = static_cast<int>(
      max(1LL, min(static_cast<long long>(sms), by_rows > by_requests ? by_rows : by_requests)));
  plan_blocks_kernel<<<grid, kPlanThreads, plan_smem_bytes(a.requests), st>>>(a);
  return cudaGetLastError();
}

}  // namespace alhr
