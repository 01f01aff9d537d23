// cache_chunk.cu -- attention of many query rows a request over all of its keys (prompts, chunks).
//
// Mathematics as in cache_decode.cu: x_j = s_j log2 e + log2 v_scale_j, weights 2^(x_j - M) times
// value codes, l = sum w_j / v_scale_j, or from the scores alone behind a value scale that is not
// between 2^-48 and 2^28.
//
// What bounds it: the two products, 4 d flops a row and key, and one power of two a row and key; at
// d = 128 the tensor core, the special-function unit and the operands' way through shared memory
// need the same time (2048 cycles for 256 rows and 128 keys), at d = 64 the powers of two do. The
// rows' own work is what it comes to: measured 1.14 ms for 2 x 2048 rows x 32 heads behind 14,336
// keys at d = 128 (904 TFLOP/s, 0.55 of the measured bf16 rate; the tensor core works 41 % of the
// time, the special-function unit 43 %), 0.97 with the rows' work alone (when the whole took 1.12).
// Score columns for each half of a key tile, so that scores never wait for weights, took 1.15 ms
// then. Units whose value scales are not near 1 take 2.4 ms in this case (three passes over the scores).
//
// One CTA a multiprocessor takes 256 query rows (two tiles of 128) of one key head and walks key
// tiles of 128. Eight warps load codes to registers, widen them to halves (exact) and write them to
// shared memory in the core-matrix layout of tcgen05 (8 rows of 16 bytes): for the keys (rows of
// the second operand) K-major, and the same bytes read MN-major are the values' operand, so nothing
// is transposed. The rows' warps, a thread a row, hold the rest: one lane of each tile of rows asks
// for its products, S_i = Q_i K^T into tensor memory and O_i += P_i V with P_i read from tensor
// memory, where the rows' threads put it in place of S_i. While the tensor core works on one tile
// of rows the threads of the other one take their powers of two. A warp of its own for the products
// was slower (1.15 ms against 1.11): it has to be woken twice a tile. Rows of a request are (token,
// head of the group) pairs, so that grouped heads share every key tile.
//
// As in cache_decode.cu the key tiles of all units form one list of which every CTA takes an
// equal, contiguous piece; units that span pieces leave partial sums that a second kernel joins.
//
// Every wait is bounded; when one runs out (not expected) the CTA sets ALHR_DEVERR_TIMEOUT and stops
// waiting (its rows' output is then not to be used), lets its products in flight end (bounded) and
// frees its tensor memory.
#include <cmath>

#include "cache_mma.cuh"
#include "cache_split.cuh"

namespace alhr {

namespace {

constexpr int kRows = 256;       // query rows of a unit: two tiles of 128
constexpr int kKeys = 128;       // keys of a tile
// Warps 0-3, 4-7: the two tiles of rows; 8-11: keys; 12-15: values.
constexpr int kChunkThreads = 512;
constexpr uint32_t kWaits = 1u << 24;
constexpr float kTopLog = 7.f;   // log2 of the largest weight when M is set
// Registers of a thread of the rows' and the codes' warps: 2 * 160 + 2 * 96 = 4 * 128, what the
// block is launched with.
constexpr int kRowRegs = 160, kCodeRegs = 96;

template <int D>
struct ChunkSmem {
  static constexpr int kTile = 128 * D * 2;      // 128 rows of halves
  static constexpr int q = 0;                    // two tiles
  static constexpr int k = 2 * kTile;            // two tiles
  static constexpr int v = 4 * kTile;            // two tiles
  // [4][8] of {k scale, log2 v scale, 1 / v scale}; {0, -infinity, 0} for a group that is not there,
  // -infinity in the last place for one whose value scale is not near 1
  static constexpr int scales = 6 * kTile;
  static constexpr int bars = scales + 4 * 8 * 16;
  static constexpr int misc = bars + 32 * 8;
  static constexpr int bytes = misc + 64;
};

enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kTurn = 8, kSFull = 10, kPFull = 12,
           kQFull = 14, kODone = 16, kDrain = 18 };

__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// The warp waits for the completion of the phase of this parity. When the wait runs out, *stop is
// set and every later wait of the block returns at once: its roles then run to the end of their
// loops with whatever the buffers hold (all inside them), together as always.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  if (!done) {
#pragma unroll 1
    for (uint32_t i = 0; i < kWaits; ++i) {
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
          " selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(done)
          : "r"(bar), "r"(parity)
          : "memory");
      if (done || ((i & 15u) == 15u && *stop)) break;
    }
    if (!done) *stop = 1;
  }
  __syncwarp();
}

// Shared-memory operand descriptor without swizzle: start address, leading and stride byte offset.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46;
}

// Instruction descriptor of kind::f16: fp32 sums, halves, M = 128, N columns; bit 16: the second
// operand is MN-major.
constexpr uint32_t product_desc(int n, bool mn_major) {
  return (1u << 4) | (mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// True in one lane of a warp that is together; the compiler knows what it guards to be uniform.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void commit_to(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_shared() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t (&v)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&v)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// {R, l} of a row with the scores of one tile.
__device__ __forceinline__ float2 sum_scores(const float4* sc, uint32_t s_col, int seen, float qs,
                                             float rmax, float l) {
#pragma unroll 1
  for (int u = 0; u < 8; ++u) {
    const float4 f = sc[u];
    const int here = f.z == 0.f ? 0 : seen - u * 16;  // 0: a group that is not there
    uint32_t v[16];
    tmem_ld16(v, s_col + u * 16);
    wait_ld();
    const float f1 = qs * f.x;
    float most = -INFINITY;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float x = k < here ? __uint_as_float(v[k]) * f1 : -INFINITY;
      v[k] = __float_as_uint(x);
      most = fmaxf(most, x);
    }
    const float r = fmaxf(rmax, most), from = r == -INFINITY ? 0.f : r;
    l *= exp2_fast(rmax - from);
#pragma unroll
    for (int k = 0; k < 16; ++k) l += exp2_fast(__uint_as_float(v[k]) - from);
    rmax = r;
  }
  return make_float2(rmax, l);
}

// Two fp32 numbers an instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int REGS>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS));
}

// One request of the list: more than row_limit rows; groups of kRows rows, each with the key tiles
// that its last row sees.
struct ChunkRequest {
  int q_lo, rows, ctx, see, groups;
  __device__ __forceinline__ void load(const AttendArgs& a, int r, int row_limit) {
    const RequestRange q(a, r);
    q_lo = q.q_lo;
    ctx = q.ctx;
    see = q.see;
    rows = q.tokens * a.group;
    groups = rows > row_limit ? (rows + kRows - 1) / kRows : 0;
  }
  __device__ __forceinline__ int tiles(const AttendArgs& a, int group) const {
    const int last = min((group + 1) * kRows, rows) - 1;
    const long long end = min(static_cast<long long>(ctx) + last / a.group + 1,
                              static_cast<long long>(see));
    return max(1, static_cast<int>((end + kKeys - 1) / kKeys));
  }
  __device__ __forceinline__ long long per_head(const AttendArgs& a) const {
    long long n = 0;
#pragma unroll 1
    for (int g = 0; g < groups; ++g) n += tiles(a, g);
    return n;
  }
};

struct ChunkCursor {
  ChunkRequest q;
  int r, h, group, tile, tiles;
  __device__ __forceinline__ int rows_here() const { return min(kRows, q.rows - group * kRows); }
};

// The unit behind *c's, where c is the calling warp's own cursor in shared memory (it is looked at
// when a unit ends only, and registers are short).
__device__ __forceinline__ ChunkCursor next_unit(const AttendArgs& a, ChunkCursor* cursor,
                                                 int row_limit) {
  ChunkCursor c = *cursor;
  c.tile = 0;
  if (++c.group == c.q.groups) {
    c.group = 0;
    if (++c.h == a.c.heads) {
      c.h = 0;
      do {
        if (++c.r >= a.requests) {  // not reached: the list has ended before
          c.r = a.requests - 1;
          c.q.groups = 1;
          break;
        }
        c.q.load(a, c.r, row_limit);
      } while (c.q.groups == 0);
    }
  }
  c.tiles = c.q.tiles(a, c.group);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *cursor = c;
  __syncwarp();
  return c;
}

template <int D, int CODE>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ JoinSpace space,
                 const int row_limit) {
  using L = ChunkSmem<D>;
  constexpr int kCols = D / 8;  // 16-byte columns of a row of halves
  // At d = 128 the two tiles of rows take turns with the tensor core and so stay out of step (1.11
  // ms against 1.13 for 2 x 2048 rows x 32 heads behind 14,336 keys); at d = 64 its products are
  // short and waiting for a turn costs more (258 us against 277 for prompts of 301 to 4096 tokens).
  constexpr bool kTurns = D == 128;
  extern __shared__ __align__(1024) unsigned char chunk_smem[];
  __shared__ long long chunk_start[kChunkThreads];
  __shared__ long long warp_sum[kChunkThreads / 32];
  __shared__ ChunkCursor cursors[kChunkThreads / 32];
  const uint32_t smem = shared_u32(chunk_smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t bars = smem + L::bars;
  auto bar = [&](int which, int i = 0) { return bars + (which + i) * 8; };
  volatile int* stop = reinterpret_cast<volatile int*>(chunk_smem + L::misc);
  let_next_begin();
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(chunk_smem + L::misc + 16);

  // ---- the tile list
  const int per = (a.requests + kChunkThreads - 1) / kChunkThreads;
  ChunkCursor cur;
  long long sum = 0;
  for (int r = tid * per; r < min(a.requests, (tid + 1) * per); ++r) {
    cur.q.load(a, r, row_limit);
    sum += cur.q.per_head(a) * a.c.heads;
  }
  const Split split = make_split<kChunkThreads>(sum, chunk_start, warp_sum, gridDim.x);
  const int piece = blockIdx.x;
  const long long begin = piece < split.pieces ? split.first(piece) : 0;
  const long long end = piece < split.pieces ? split.first(piece + 1) : 0;
  JoinMeta* meta = space.meta + piece;
  if (tid == 0) meta->last = -1;
  if (begin >= end) {
    wait_for_previous();
    return;
  }
  {
    const int c = chunk_of<kChunkThreads>(chunk_start, begin);
    long long at = chunk_start[c], head = 0;
    cur.r = c * per;
    for (;;) {
      cur.q.load(a, cur.r, row_limit);
      head = cur.q.per_head(a);
      if (begin < at + head * a.c.heads) break;
      at += head * a.c.heads;
      if (++cur.r >= a.requests) return;  // not reached: `begin` is inside the list
    }
    long long rest = begin - at;
    cur.h = static_cast<int>(rest / head);
    rest -= cur.h * head;
    cur.group = 0;
    while (rest >= (cur.tiles = cur.q.tiles(a, cur.group))) {
      rest -= cur.tiles;
      ++cur.group;
    }
    cur.tile = static_cast<int>(rest);
  }
  const int count = static_cast<int>(min(end - begin, 0x7fffffffLL));
  if (lane == 0) cursors[warp] = cur;
  ChunkCursor* const cursor = &cursors[warp];

  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     shared_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(bar(kKFull, i), 4);
      bar_init(bar(kKEmpty, i), 2);
      bar_init(bar(kVFull, i), 4);
      bar_init(bar(kVEmpty, i), 2);
      bar_init(bar(kTurn, i), 1);
      bar_init(bar(kSFull, i), 2);
      bar_init(bar(kPFull, i), 4);
      bar_init(bar(kQFull, i), 4);
      bar_init(bar(kODone, i), 1);
      bar_init(bar(kDrain, i), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    *stop = 0;
    bar_arrive(bar(kTurn, 0));  // the first tile of rows begins
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ================ rows: thread (i, lane of the tile) holds one query row
    more_registers<kRowRegs>();
    const int i = warp >> 2, rt = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + i * 128, o_col = tmem + lanes + 256 + i * D;
    const unsigned char* scales = chunk_smem + L::scales;
    float m = -INFINITY, l = 0.f, qs = 0.f;
    float rmax = 0.f;  // R, while `wide`
    bool wide = false;
    int seen = 0, row = 0;  // columns < seen of the tile are visible
    // this row's queries to shared memory, scaled by a power of two so that halves hold them
    auto load_q = [&](const ChunkCursor& cur) {
      row = cur.group * kRows + i * 128 + rt;
      m = -INFINITY;
      l = 0.f;
      seen = 0x7fffffff;  // a row behind the last one masks nothing and is not written
      uint4 raw[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) raw[c] = make_uint4(0u, 0u, 0u, 0u);
      if (row < cur.q.rows) {
        const int tok = row / a.group;
        seen = static_cast<int>(max(min(static_cast<long long>(cur.q.ctx) + tok + 1,
                                        static_cast<long long>(cur.q.see)), 0LL));
        const uint4* p = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + (cur.q.q_lo + tok) * a.q_token_stride +
            (cur.h * a.group + (row - tok * a.group)) * a.q_head_stride);
#pragma unroll
        for (int c = 0; c < kCols; ++c) raw[c] = __ldg(p + c);
      }
      // magnitudes of both types order like their bits
      uint32_t hi = 0;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        hi = __vmaxu2(hi, __vmaxu2(__vmaxu2(raw[c].x & 0x7fff7fffu, raw[c].y & 0x7fff7fffu),
                                   __vmaxu2(raw[c].z & 0x7fff7fffu, raw[c].w & 0x7fff7fffu)));
      }
      hi = max(hi & 0xffffu, hi >> 16);
      const float top = a.fp16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(hi)))
                               : __uint_as_float(hi << 16);
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 126);
      // a negative factor of the scores goes into the queries: what follows takes the largest
      // score as the largest product
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23),
                                 a.scale_log2);
      qs = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23) * fabsf(a.scale_log2);
      const uint32_t dst = smem + L::q + i * L::kTile + (rt >> 3) * (kCols * 128) + (rt & 7) * 16;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float y[8];
        if (a.fp16) unpack8<ALHR_TYPE_FP16>(raw[c], raw[c], y);
        else unpack8<ALHR_TYPE_BF16>(raw[c], raw[c], y);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(dst + c * 128),
                     "r"(pack2(y[0] * up, y[1] * up, true)), "r"(pack2(y[2] * up, y[3] * up, true)),
                     "r"(pack2(y[4] * up, y[5] * up, true)), "r"(pack2(y[6] * up, y[7] * up, true))
                     : "memory");
      }
      fence_shared();
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kQFull, i));
    };
    // ---- products, asked for by one lane of the tile's first warp
    const bool asks = (warp & 3) == 0;
    constexpr uint32_t kRowGroup = kCols * 128;  // bytes between groups of eight rows
    constexpr uint32_t kScore = product_desc(128, false), kSum = product_desc(D, true);
    const uint32_t s_at = tmem + i * 128, o_at = tmem + 256 + i * D;
    auto ask_scores = [&](int j) {  // of key tile j; the warp's elected lane
      const uint64_t q = operand_desc(smem + L::q + i * L::kTile, 128, kRowGroup);
      const uint64_t k = operand_desc(smem + L::k + (j & 1) * L::kTile, 128, kRowGroup);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) product_ss(s_at, q + s * 16, k + s * 16, kScore, s > 0);
      commit_to(bar(kSFull, i));
      commit_to(bar(kKEmpty, j & 1));
      bar_arrive(bar(kSFull, i));  // hands on that the tile's scales are there
    };
    bool first = true, fresh = true, from_start = true, busy = false;
    int units = 0, q_units = 0, left = 0;  // key tiles of the unit that are still to come
    uint32_t s_phase = 0, p_phase = 0;
    for (int j = 0;; ++j) {
      if (fresh) {
        // ---- the unit before (or this piece of it) has ended, another one begins
        const ChunkCursor was = *cursor;
        const int was_row = row;
        const float was_l = l, was_r = wide ? rmax : m;
        const float up = wide ? exp2_fast(m - rmax) : 1.f;
        const bool was_busy = busy, to_end = left == 0, started = from_start;
        if (j > 0 && tid == 0 && started && !to_end) {
          meta->r = was.r;
          meta->h = was.h;
          meta->row0 = was.group * kRows;
          meta->rows = was.rows_here();
          meta->last = split.piece_of(end - 1 + left);
        }
        first = true;
        fresh = false;
        wide = false;
        if (j < count) {
          ChunkCursor now = was;
          if (j > 0) now = next_unit(a, cursor, row_limit);
          from_start = now.tile == 0;
          left = now.tiles - now.tile;
          busy = now.rows_here() > i * 128;  // the second tile of rows may be empty
          // S of the last tile is here, so nothing reads the queries before any more
          if (busy) load_q(now);
          seen -= now.tile * kKeys;
          if (asks) {
            warp_wait(bar(kKFull, j & 1), (j >> 1) & 1, stop);
            if (busy) {
              warp_wait(bar(kQFull, i), q_units & 1, stop);
              ++q_units;
              fence_after();
              if (elected()) ask_scores(j);
              __syncwarp();
            } else if (lane == 0) {
              bar_arrive(bar(kKEmpty, j & 1));
            }
          }
        }
        if (j > 0 && was_busy) {
          warp_wait(bar(kODone, i), units & 1, stop);
          ++units;
          fence_after();
          const bool on = was_row < was.q.rows, whole = started && to_end;
          const int tok = was_row / a.group;
          const long long at = static_cast<long long>(was.q.q_lo + tok) * a.q_heads +
                               was.h * a.group + (was_row - tok * a.group);
          const float inv = was_l == 0.f ? 0.f : up / was_l;  // no key; NaN stays
          float* part = space.part + (static_cast<long long>(piece) * 2 + (started ? 1 : 0)) *
                                         (kRows * (D + 2));
          const int pr = i * 128 + rt;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(v, o_col + c * 32);
            wait_ld();
            if (on && whole) {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + c * 32);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack2(__uint_as_float(v[k * 8 + 2 * e]) * inv,
                               __uint_as_float(v[k * 8 + 2 * e + 1]) * inv, a.fp16);
                dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else if (on) {
              float4* dst = reinterpret_cast<float4*>(part + pr * D + c * 32);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dst[k] = make_float4(__uint_as_float(v[4 * k]) * inv,
                                     __uint_as_float(v[4 * k + 1]) * inv,
                                     __uint_as_float(v[4 * k + 2]) * inv,
                                     __uint_as_float(v[4 * k + 3]) * inv);
            }
          }
          if (on && whole) {
            if (a.lse)
              a.lse[at] = was_l == 0.f ? -INFINITY : (was_r + log2f(was_l)) * 0.6931471805599453f;
          } else if (on) {
            float r = was_r, sum = was_l;
            settle(r, sum, kPartLog);
            part[kRows * D + pr] = r;
            part[kRows * D + kRows + pr] = sum;
          }
          __syncwarp();
          fence_before();
        }
      }
      if (j == count) break;
      if (busy) {
        warp_wait(bar(kSFull, i), s_phase, stop);
        s_phase ^= 1u;
        fence_after();
        const bool cut = __any_sync(0xffffffffu, seen < kKeys);
        const float4* sc = reinterpret_cast<const float4*>(scales) + (j & 3) * 8;
        // Nearly always M stays as it is: weights are taken with it at once, and held until it is
        // known that none is above 2^15. The tile in which M has to grow, the first one of a unit
        // and those that a mask cuts take two passes over the scores; so does one with a value
        // scale that is not near 1 (it makes the sum -infinity or NaN), and every one behind it.
        bool done = false;
        if (!first && !cut && !wide) {
          uint32_t p[64];
          float sum = l, most = m == -INFINITY ? INFINITY : 0.f;
          uint32_t v[2][32];
          tmem_ld32(v[0], s_col);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            wait_ld();
            if (c < 3) tmem_ld32(v[(c + 1) & 1], s_col + (c + 1) * 32);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float4 f = sc[c * 2 + u];
              const float f1 = qs * f.x, f0 = f.y - m;
              const uint64_t f11 = pair(f1, f1), f00 = pair(f0, f0);
              uint64_t part = 0;
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const uint32_t* w = &v[c & 1][u * 16 + k];
                float x0, x1;
                unpair(fma2(pair(__uint_as_float(w[0]), __uint_as_float(w[1])), f11, f00), x0, x1);
                x0 = exp2_fast(x0);
                x1 = exp2_fast(x1);
                part = add2(part, pair(x0, x1));
                p[c * 16 + u * 8 + k / 2] = pack2(x0, x1, true);
              }
              float lo, hi;
              unpair(part, lo, hi);
              lo += hi;
              most = fmaxf(most, lo);
              sum = fmaf(lo, f.z, sum);
            }
          }
          done = __all_sync(0xffffffffu, most <= 32768.f && sum >= 0.f);
          if (done) {
            l = sum;
            uint32_t half[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int k = 0; k < 32; ++k) half[k] = p[h * 32 + k];
              tmem_st32(s_col + h * 32, half);
            }
          }
        }
        if (!done) {
          // by 32 columns: most of what a mask cuts is seen by the whole warp or by none of it
          float top = -INFINITY;  // the largest x of the row
          bool far = false;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int here = seen - c * 32;
            if (!__any_sync(0xffffffffu, here > 0)) break;
            uint32_t v[32];
            tmem_ld32(v, s_col + c * 32);
            wait_ld();
            if (__any_sync(0xffffffffu, here < 32)) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k >= here) v[k] = 0xff800000u;  // -infinity
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float x = __uint_as_float(v[u * 16]);
#pragma unroll
              for (int k = 1; k < 16; ++k) x = fmaxf(x, __uint_as_float(v[u * 16 + k]));
              const float4 f = sc[c * 2 + u];
              far |= f.z < 0.f;
              // -infinity stays where the factor is 0
              top = fmaxf(top, x == -INFINITY ? x : fmaf(x, qs * f.x, f.y));
            }
          }
          if (__builtin_expect(far && !wide, 0)) {
            wide = true;
            rmax = m;  // l is in units of 2^M so far
            settle(rmax, l, 0);
          }
          if (__builtin_expect(wide, 0)) {  // l and R from the scores
            const float2 y = sum_scores(sc, s_col, seen, qs, rmax, l);
            rmax = y.x;
            l = y.y;
          }
          const bool grow = top > m + kTopLog + 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = fmaxf(m, top - kTopLog);
            const float keep = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
            m = mn;
            if (!wide) l *= keep;
            if (!first) {
              // the product before this tile's scores is complete: they were issued after it
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(v, o_col + c * 32);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * keep);
                tmem_st32(o_col + c * 32, v);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const int here = seen - c * 32;
            uint32_t p[16];
            if (!__any_sync(0xffffffffu, here > 0)) {
#pragma unroll
              for (int k = 0; k < 16; ++k) p[k] = 0u;
            } else {
              uint32_t v[32];
              tmem_ld32(v, s_col + c * 32);
              wait_ld();
              if (__any_sync(0xffffffffu, here < 32)) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (k >= here) v[k] = 0xff800000u;
              }
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float4 f = sc[c * 2 + u];
                // not 0: a masked score stays -infinity (the largest, 2^29, times 1e-37 is nothing)
                const float f1 = fmaxf(qs * f.x, 1e-37f), f0 = f.y - base;
                float part = 0.f;
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float x0 = exp2_fast(fmaf(__uint_as_float(v[u * 16 + k]), f1, f0));
                  const float x1 = exp2_fast(fmaf(__uint_as_float(v[u * 16 + k + 1]), f1, f0));
                  part += x0 + x1;
                  p[u * 8 + k / 2] = pack2(x0, x1, true);
                }
                if (!wide) l = fmaf(part, f.z, l);
              }
            }
            tmem_st16(s_col + c * 16, p);  // over scores that have been read
          }
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(kPFull, i));
      }
      --left;
      fresh = left == 0 || j + 1 == count;
      seen -= kKeys;
      if (asks) {
        // The sum of this tile and the scores of the next one, in turn with the other tile of rows:
        // its rows take their weights while these products run. Keys and values are there before
        // the weights are.
        if (!fresh) warp_wait(bar(kKFull, (j + 1) & 1), ((j + 1) >> 1) & 1, stop);
        warp_wait(bar(kVFull, j & 1), (j >> 1) & 1, stop);
        if (busy) warp_wait(bar(kPFull, i), p_phase, stop);
        if (kTurns) warp_wait(bar(kTurn, i), j & 1, stop);
        if (busy) {
          p_phase ^= 1u;
          fence_after();
          if (elected()) {
            const uint64_t v = operand_desc(smem + L::v + (j & 1) * L::kTile, kRowGroup, 128);
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s)
              product_ts(o_at, s_at + s * 8, v + s * (2 * kRowGroup / 16), kSum, !first || s > 0);
            commit_to(bar(kVEmpty, j & 1));
            if (fresh) commit_to(bar(kODone, i));
            else ask_scores(j + 1);
            bar_arrive(bar(kTurn, 1 - i));
          }
          __syncwarp();
        } else if (lane == 0) {
          bar_arrive(bar(kVEmpty, j & 1));
          if (!fresh) bar_arrive(bar(kKEmpty, (j + 1) & 1));
          bar_arrive(bar(kTurn, 1 - i));
        }
      }
      first = false;
    }
    __syncwarp();
    if (asks && *stop) {  // products in flight end before the tensor memory is freed
      if (elected()) commit_to(bar(kDrain, i));
      __syncwarp();
      volatile int none = 0;
      warp_wait(bar(kDrain, i), 0, &none);
    }
  } else {
    // ================ codes to halves: keys (and the scales) or values
    fewer_registers<kCodeRegs>();
    const int w = warp & 3;
    const bool keys = warp < 12;
    const uint8_t* const codes = keys ? a.c.k : a.c.v;
    const uint32_t full = bar(keys ? kKFull : kVFull), empty = bar(keys ? kKEmpty : kVEmpty);
    const int kr = lane & 7, kc = lane >> 3;       // row of eight, 16-byte piece of 64
    constexpr int kHalves = D / 64;                // pieces kc, kc + 4
    const uint32_t dst0 = smem + (keys ? L::k : L::v) + w * 4 * (kCols * 128) + kc * 256 + kr * 16;
    bool bad = false;
    // the tile whose codes are asked for, this warp's 32 keys of it
    int key0 = cur.tile * kKeys + w * 32, key_end = cur.q.see, left = cur.tiles - cur.tile;
    int head = cur.h;
    const int32_t* table = a.table + static_cast<long long>(cur.r) * a.max_blocks;
    int blk_next[2];  // table entries of its two 16-key groups, -1 where no key is visible
    auto look_up = [&]() {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        blk_next[u] = key0 + u * 16 < key_end ? __ldg(table + ((key0 + u * 16) >> a.c.bs_log)) : -1;
    };
    uint4 raw[4 * kHalves];
    float ks = 0.f, vs = 0.f;  // lanes 0, 1: scales of the two groups, and whether they count
    bool there = false;
    look_up();
#pragma unroll 1
    for (int j = -1; j < count; ++j) {  // tile j is widened, tile j + 1 asked for
      const int b = j & 1;
      if (j >= 0) {
        if (j >= 2) {
          warp_wait(empty + b * 8, ((j >> 1) - 1) & 1, stop);
        }
        const uint32_t dst = dst0 + b * L::kTile;
#pragma unroll
        for (int rg = 0; rg < 4; ++rg)
#pragma unroll
          for (int hh = 0; hh < kHalves; ++hh) {
            const uint4 x = raw[rg * kHalves + hh];
            uint32_t y[8];
            widen4<CODE>(x.x, y[0], y[1]);
            widen4<CODE>(x.y, y[2], y[3]);
            widen4<CODE>(x.z, y[4], y[5]);
            widen4<CODE>(x.w, y[6], y[7]);
            const uint32_t at = dst + (rg * kCols + hh * 8) * 128;
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(y[0]), "r"(y[1]),
                         "r"(y[2]), "r"(y[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at + 128), "r"(y[4]),
                         "r"(y[5]), "r"(y[6]), "r"(y[7])
                         : "memory");
          }
        if (keys && lane < 2) {
          const float log_v = vs >= kTinyScale ? __log2f(vs) : -INFINITY;
          float4 f = make_float4(ks, log_v, __frcp_rn(vs), 0.f);
          if (!is_near(vs)) f.z = -INFINITY;
          if (!there) f = make_float4(0.f, -INFINITY, 0.f, 0.f);
          // four tiles of scales: the rows are done with those of tile j - 3 before the scores of
          // tile j - 2 are asked for, which the wait above has seen
          reinterpret_cast<float4*>(chunk_smem + L::scales)[(j & 3) * 8 + w * 2 + lane] = f;
        }
        fence_shared();
        __syncwarp();
        if (lane == 0) bar_arrive(full + b * 8);
      }
      if (j + 1 < count) {
        int blk[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          blk[u] = blk_next[u];
          if (blk[u] < 0 || blk[u] >= a.c.blocks) {
            if (key0 + u * 16 < key_end) bad = true;
            blk[u] = -1;
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = key0 + u * 16;
          const long long row = block_row(a.c, max(blk[u], 0), head) + (key & (a.c.bs - 1)) + kr;
          const uint8_t* p = codes + row * D + kc * 16;
          const int rows = blk[u] < 0 ? 0 : key_end - key - kr;  // this lane's rows 0 and 8
#pragma unroll
          for (int rg = 0; rg < 2; ++rg)
#pragma unroll
            for (int hh = 0; hh < kHalves; ++hh)
              raw[(u * 2 + rg) * kHalves + hh] =
                  rows > rg * 8 ? __ldg(reinterpret_cast<const uint4*>(p + rg * 8 * D + hh * 64))
                                : make_uint4(0u, 0u, 0u, 0u);
        }
        if (keys && lane < 2) {
          const int mine = lane == 0 ? blk[0] : blk[1];
          const long long si = static_cast<long long>(max(mine, 0)) * a.c.heads + head;
          there = mine >= 0;
          ks = there ? __ldg(a.c.k_scale + si) : 0.f;
          vs = there ? __ldg(a.c.v_scale + si) : 0.f;
        }
        if (j + 2 < count) {
          key0 += kKeys;
          if (--left == 0) {
            const ChunkCursor c = next_unit(a, cursor, row_limit);
            key0 = w * 32;
            key_end = c.q.see;
            left = c.tiles;
            head = c.h;
            table = a.table + static_cast<long long>(c.r) * a.max_blocks;
          }
          look_up();
        }
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (tid == 0 && *stop) cache_flag(a.dev_err, ALHR_DEVERR_TIMEOUT);
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512)
                 : "memory");
  wait_for_previous();  // what follows this kernel follows the one before it too
}

template <int D, int CODE>
cudaError_t chunk_as(const AttendArgs& a, int sms, int row_limit, cudaStream_t st) {
  static thread_local bool configured[128] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        chunk_kernel<D, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkSmem<D>::bytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) configured[dev] = true;
  }
  return launch_behind(chunk_kernel<D, CODE>, dim3(sms), kChunkThreads, ChunkSmem<D>::bytes, st, a,
                       join_space(a.workspace, sms), row_limit);
}

}  // namespace

size_t chunk_workspace(int sms, int d) { return join_bytes(sms, kRows, d); }

// Requests of more than row_limit rows (of one key head); the join has to follow. The kernel may
// begin before the previous one of the stream has ended, whose results it does not read, and ends
// behind it. A CTA of either fills a multiprocessor (198 KB of shared memory, 65,536 registers), so
// only the one's end and the other's start overlap.
cudaError_t launch_chunk(const AttendArgs& a, int d, int code, int sms, int row_limit,
                         cudaStream_t st) {
  if (d == 64)
    return code == ALHR_CODE_INT8 ? chunk_as<64, ALHR_CODE_INT8>(a, sms, row_limit, st)
                                  : chunk_as<64, ALHR_CODE_E4M3>(a, sms, row_limit, st);
  return code == ALHR_CODE_INT8 ? chunk_as<128, ALHR_CODE_INT8>(a, sms, row_limit, st)
                                : chunk_as<128, ALHR_CODE_E4M3>(a, sms, row_limit, st);
}

cudaError_t launch_chunk_join(const AttendArgs& a, int d, int sms, cudaStream_t st) {
  const JoinSpace space = join_space(a.workspace, sms);
  return d == 64 ? launch_join<64, kRows>(a, space, sms, st)
                 : launch_join<128, kRows>(a, space, sms, st);
}

}  // namespace alhr
