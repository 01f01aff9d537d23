// cache_decode.cu -- attention of few query rows a request over all of its keys (decode).
//
// Mathematics: with x_j = s_j log2 e + log2 v_scale_j (s_j the scaled score) and M near the running
// maximum of x, the weights w_j = 2^(x_j - M) multiply the value codes, O = sum w_j vcode_j, and
// l = sum w_j / v_scale_j is the softmax's sum: out = O / l. Taking the block's value scale into
// the exponent keeps the weights of blocks with very different scales in the range of a half: M is
// chosen so that the largest weight lies in [2^7, 2^15], and weights down to 2^-21 of it are
// rounded at 2^-11 of themselves. l is summed from the fp32 weights. That holds while all value
// scales are between 2^-48 and 2^28; from the first tile on that has another one (zeros are stored
// with 2^-100) the unit sums l = sum 2^(s_j log2 e - R) from the scores, R their running maximum, and
// out = 2^(M - R) O / l: a head of zeros takes the second power of two for every key.
//
// What bounds it: the codes have to be read once, 2 d bytes a key and head; everything else is
// there to keep the memory busy. Replayed from a graph: 64 sequences of up to 16,384 int8 keys, 32
// query heads over 8, d = 128: 191 us, 6.2 TB/s; 4 sequences x 8 heads x 262,144 e4m3 keys: 342 us, 6.3
// TB/s; 0.94 and 0.96 of the copy rate (both inputs are larger than L2). One call at a time for
// seconds, at lower clocks: 216 and 334 us. With every value scale at 2^-100 (second powers of two):
// 213 and 323 us. The tiles of all (request, key head, row group)
// units form one list, and each warp of the GPU takes an equal, contiguous piece of it: no unit is
// too short or too long, and no warp waits for another one. A warp copies its tiles (32 keys at d =
// 128, 64 at d = 64: 8 KB) kStages ahead into its own piece of shared memory, 192 KB of copies in
// flight a multiprocessor, reads the values transposed (203 -> 190 us against interleaving bytes of
// key pairs in registers), converts the codes to halves in registers and uses the warp-wide matrix
// product, which costs the same for one query row as for eight. A unit inside one warp's piece is written at
// once; one that spans pieces leaves partial sums (O, M, l), which a second kernel joins in the
// order of the pieces.
#include "cache_split.cuh"

namespace alhr {

namespace {

constexpr int kDecodeWarps = 8;  // of one CTA a multiprocessor
constexpr int kStages = 3;
constexpr float kTopLog = 7.f;    // log2 of the largest weight when M is set
constexpr int kStageBytes = 8192;  // codes of one tile, keys and values

template <int D>
struct Tile {
  static constexpr int kKeys = kStageBytes / (2 * D);
  static constexpr int kSubs = kKeys / 16;         // groups of 16 keys: one block each
  static constexpr int kScaleBytes = kSubs * 16;   // {k scale, v scale, there} of each group
  static constexpr int kStride = kStageBytes + 64;
  static_assert(kScaleBytes <= 64, "scales behind the codes");
};

// Key of the tile's 16-key group that row m (0..7) of the scores stands for; row m + 8 stands for the
// key two behind it. The transposed read of the values gives a lane four consecutive keys, the
// product wants them as two pairs eight apart: the scores' rows are in that order from the start.
__device__ __forceinline__ int key_of(int m) { return 4 * (m >> 1) + (m & 1); }

// 16-byte piece c of row `row`, where it lies in shared memory.
template <int D>
__device__ __forceinline__ int piece_offset(int row, int c) {
  return D == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

// One request as the list sees it.
template <int D, int ROWS>
struct Request {
  int q_lo, rows, ctx, see, tiles, groups;
  __device__ __forceinline__ void load(const AttendArgs& a, int r, int row_limit) {
    const RequestRange q(a, r);
    q_lo = q.q_lo;
    ctx = q.ctx;
    see = q.see;
    rows = q.tokens * a.group;
    groups = rows > row_limit ? 0 : (rows + ROWS - 1) / ROWS;
    tiles = max(1, (see + Tile<D>::kKeys - 1) / Tile<D>::kKeys);
  }
  __device__ __forceinline__ long long work(int heads) const {
    return static_cast<long long>(groups) * tiles * heads;
  }
};

template <int D, int ROWS>
struct Cursor {
  Request<D, ROWS> q;
  int r, h, group, tile;
  __device__ __forceinline__ void step(const AttendArgs& a, int row_limit) {
    if (++tile < q.tiles) return;
    tile = 0;
    if (++group < q.groups) return;
    group = 0;
    if (++h < a.c.heads) return;
    h = 0;
    do {
      if (++r >= a.requests) {  // not reached: the list has ended before
        r = a.requests - 1;
        return;
      }
      q.load(a, r, row_limit);
    } while (q.groups == 0);
  }
};

__device__ __forceinline__ float group_max(float v) {  // over the lanes of equal lane % 4
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float group_add(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, int CODE, int NT>
__global__ void __launch_bounds__(kDecodeWarps * 32, 1)
    decode_kernel(const AttendArgs a, const JoinSpace space, const int row_limit) {
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;              // products over d of one 16-key group
  constexpr int SUBS = Tile<D>::kSubs;
  constexpr int LPR = D / 16;             // 16-byte pieces of a row
  constexpr int RPI = 32 / LPR;           // rows one copy of the warp covers
  extern __shared__ __align__(128) unsigned char decode_smem[];
  __shared__ long long chunk_start[kDecodeWarps * 32];
  __shared__ long long warp_sum[kDecodeWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  let_next_begin();

  // ---- the tile list: every thread sums a run of requests
  const int per = (a.requests + kDecodeWarps * 32 - 1) / (kDecodeWarps * 32);
  Cursor<D, ROWS> load;
  long long sum = 0;
  for (int r = tid * per; r < min(a.requests, (tid + 1) * per); ++r) {
    load.q.load(a, r, row_limit);
    sum += load.q.work(a.c.heads);
  }
  const Split split = make_split<kDecodeWarps * 32>(sum, chunk_start, warp_sum,
                                                    static_cast<long long>(gridDim.x) * kDecodeWarps);
  // pieces beside one another in the list lie on different multiprocessors
  const int piece = warp * gridDim.x + blockIdx.x;
  const long long begin = piece < split.pieces ? split.first(piece) : 0;
  const long long end = piece < split.pieces ? split.first(piece + 1) : 0;
  JoinMeta* meta = space.meta + piece;
  if (lane == 0) meta->last = -1;
  if (begin >= end) return;

  // ---- where this piece begins
  {
    const int c = chunk_of<kDecodeWarps * 32>(chunk_start, begin);
    long long at = chunk_start[c];
    load.r = c * per;
    for (;;) {
      load.q.load(a, load.r, row_limit);
      const long long w = load.q.work(a.c.heads);
      if (begin < at + w) break;
      at += w;
      if (++load.r >= a.requests) return;  // not reached: `begin` is inside the list
    }
    long long rest = begin - at;
    const long long per_head = static_cast<long long>(load.q.groups) * load.q.tiles;
    load.h = static_cast<int>(rest / per_head);
    rest -= load.h * per_head;
    load.group = static_cast<int>(rest / load.q.tiles);
    load.tile = static_cast<int>(rest - static_cast<long long>(load.group) * load.q.tiles);
  }
  Cursor<D, ROWS> cur = load;

  // ---- copies, kStages tiles ahead
  const uint32_t ring = shared_u32(decode_smem) + warp * (kStages * Tile<D>::kStride);
  const int crow = lane / LPR, cpiece = lane % LPR;
  const uint32_t place0 = piece_offset<D>(crow, cpiece), place1 = piece_offset<D>(RPI + crow, cpiece);
  bool bad = false;
  // block of 16-key group `lane` of the loader's tile; -1: no visible key in it; -2: a bad number
  auto fetch_block = [&]() {
    int block = -1;
    const int key = load.tile * Tile<D>::kKeys + lane * 16;
    if (lane < SUBS && key < load.q.see) {
      block = __ldg(a.table + static_cast<long long>(load.r) * a.max_blocks + (key >> a.c.bs_log));
      if (block < 0 || block >= a.c.blocks) block = -2;
    }
    return block;
  };
  int next_block = fetch_block();
  auto issue = [&](int stage) {
    const uint32_t base = ring + stage * Tile<D>::kStride;
    bad |= next_block == -2;
#pragma unroll
    for (int s = 0; s < SUBS; ++s) {
      const int block = __shfl_sync(0xffffffffu, next_block, s);
      const int key0 = load.tile * Tile<D>::kKeys + s * 16;
      const int there = block >= 0 ? min(16, load.q.see - key0) : 0;  // rows of the group to copy
      const long long src = (block_row(a.c, max(block, 0), load.h) + (key0 & (a.c.bs - 1))) * D;
      const uint8_t* const k = a.c.k + src + lane * 16;
      const uint8_t* const v = a.c.v + src + lane * 16;
      const uint32_t dst = base + s * 16 * D;
      if (there == 16) {  // the same place a row group later, but for the order of the pieces
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const uint32_t at = dst + (i & 1 ? place1 : place0) + (i & ~1) * 512;
          copy16(at, k + i * 512, 16);
          copy16(at + kStageBytes / 2, v + i * 512, 16);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < 16 / RPI; ++i) {
          const int n = i * RPI + crow < there ? 16 : 0;
          const uint32_t at = dst + (i & 1 ? place1 : place0) + (i & ~1) * 512;
          copy16(at, n ? k + i * 512 : a.c.k, n);
          copy16(at + kStageBytes / 2, n ? v + i * 512 : a.c.v, n);
        }
      }
    }
    if (lane < SUBS) {
      const long long si =
          static_cast<long long>(max(next_block, 0)) * a.c.heads + load.h;
      const uint32_t dst = base + kStageBytes + lane * 16;
      const int n = next_block >= 0 ? 4 : 0;
      copy4(dst, a.c.k_scale + si, n);
      copy4(dst + 4, a.c.v_scale + si, n);
      asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(dst + 8), "r"(next_block >= 0 ? 1 : 0) : "memory");
    }
  };
  long long loaded = begin;
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) {
    if (loaded < end) {
      issue(s);
      if (++loaded < end) {
        load.step(a, row_limit);
        next_block = fetch_block();
      }
    }
    copy_commit();
  }

  // ---- the unit's queries
  uint32_t qf[NT][KS][2];
  float qscale[NT][2];  // factor of the scores of columns 2 t, 2 t + 1
  int see[NT][2];       // visible keys of those columns' rows
  float o[NT][KS][4], m[NT][2], l[NT][2];
  float rmax[NT][2];    // R, while `wide`
  bool wide = false;
  int see_min;
  auto begin_unit = [&]() {
    const int row0 = cur.group * ROWS;
    wide = false;
    see_min = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + n * 8 + g;
      float x[D / 4];
      float top = 0.f;
      if (row < cur.q.rows) {
        const int tok = row / a.group;
        const long long at = (cur.q.q_lo + tok) * a.q_token_stride +
                             (cur.h * a.group + (row - tok * a.group)) * a.q_head_stride + t * (D / 4);
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 w = __ldg(p + i);
          float y[8];
          if (a.fp16) unpack8<ALHR_TYPE_FP16>(w, w, y);
          else unpack8<ALHR_TYPE_BF16>(w, w, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[8 * i + j] = y[j];
            top = fmaxf(top, fabsf(y[j]));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
      }
      // a row is scaled by the power of two that brings its largest number to [2^14, 2^15), so
      // that its halves are exact down to 2^-28 of it
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 126);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[n][s][0] = pack2(x[4 * s] * up, x[4 * s + 1] * up, true);
        qf[n][s][1] = pack2(x[4 * s + 2] * up, x[4 * s + 3] * up, true);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qscale[n][c] = __shfl_sync(0xffffffffu, down, 4 * (2 * t + c)) * a.scale_log2;
        const int cr = row0 + n * 8 + 2 * t + c;
        const long long pos = static_cast<long long>(cur.q.ctx) + cr / a.group + 1;
        see[n][c] = cr < cur.q.rows
                        ? static_cast<int>(max(min(pos, static_cast<long long>(cur.q.see)), 0LL)) : 0;
        if (cr < cur.q.rows) see_min = min(see_min, see[n][c]);
        m[n][c] = -INFINITY;
        l[n][c] = 0.f;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][s][i] = 0.f;
    }
    see_min = __reduce_min_sync(0xffffffffu, see_min);
  };

  // l and R of a tile from its scores, where the value scales are far apart
  auto sum_scores = [&](const float (&s)[SUBS][NT][4], uint32_t scales, int key0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x[SUBS][2], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
          const uint4 sc = lds128(scales + u * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool on = sc.z && key0 + u * 16 + key_of(g) + i * 2 < see[n][c];
            x[u][i] = on ? s[u][n][2 * i + c] * (qscale[n][c] * __uint_as_float(sc.x)) : -INFINITY;
            top = fmaxf(top, x[u][i]);
          }
        }
        const float r = fmaxf(rmax[n][c], group_max(top));
        const float from = r == -INFINITY ? 0.f : r;
        float sum = l[n][c] * exp2_fast(rmax[n][c] - from);
#pragma unroll
        for (int u = 0; u < SUBS; ++u) sum += exp2_fast(x[u][0] - from) + exp2_fast(x[u][1] - from);
        l[n][c] = sum;
        rmax[n][c] = r;
      }
  };

  // column c of column group n: row, sums over the keys of all lanes
  auto end_unit = [&](bool from_start, bool to_end) {
    const int row0 = cur.group * ROWS;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float sum_l = group_add(l[n][c]);
        const int col = n * 8 + 2 * t + c, row = row0 + col;
        if (row >= cur.q.rows) continue;
        const float base = wide ? rmax[n][c] : m[n][c];
        // no key; NaN stays
        const float inv = sum_l == 0.f ? 0.f : (wide ? exp2_fast(m[n][c] - base) : 1.f) / sum_l;
        // numbers 16 k + g and 16 k + 8 + g of the row
        if (from_start && to_end) {
          const int tok = row / a.group;
          const long long at = static_cast<long long>(cur.q.q_lo + tok) * a.q_heads +
                               cur.h * a.group + (row - tok * a.group);
          uint16_t* const p = static_cast<uint16_t*>(a.out) + at * D + g;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t w = pack2(o[n][k][c] * inv, o[n][k][2 + c] * inv, a.fp16);
            p[16 * k] = static_cast<uint16_t>(w);
            p[16 * k + 8] = static_cast<uint16_t>(w >> 16);
          }
          if (a.lse && g == 0)
            a.lse[at] = sum_l == 0.f ? -INFINITY : (base + log2f(sum_l)) * 0.6931471805599453f;
        } else {
          float* const part = space.part +
                              (static_cast<long long>(piece) * 2 + (from_start ? 1 : 0)) *
                                  (ROWS * (D + 2));
          float* const p = part + col * D + g;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            p[16 * k] = o[n][k][c] * inv;
            p[16 * k + 8] = o[n][k][2 + c] * inv;
          }
          if (g == 0) {
            float r = base, sum = sum_l;
            settle(r, sum, kPartLog);
            part[ROWS * D + col] = r;
            part[ROWS * D + ROWS + col] = sum;
          }
        }
      }
    }
    if (from_start && !to_end && lane == 0) {
      meta->r = cur.r;
      meta->h = cur.h;
      meta->row0 = row0;
      meta->rows = min(ROWS, cur.q.rows - row0);
      // the unit's last tile: this piece ends inside the unit, at list position `end`
      meta->last = split.piece_of(end - 1 + (cur.q.tiles - 1 - cur.tile));
    }
  };

  begin_unit();
  bool from_start = cur.tile == 0;
  int stage = 0;
  for (long long f = begin; f < end; ++f) {
    copy_wait<kStages - 1>();
    __syncwarp();
    const uint32_t base = ring + stage * Tile<D>::kStride;
    // scores
    float s[SUBS][NT][4];
    float add[SUBS], inv_vs[SUBS], ks[SUBS];
    bool far = false;
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][n][i] = 0.f;
      const int r0 = u * 16 + key_of(g);
      uint32_t w0[D / 16], w1[D / 16];  // D / 4 codes of two keys
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 x = lds128(base + piece_offset<D>(r0, t * (D / 64) + i));
        const uint4 y = lds128(base + piece_offset<D>(r0 + 2, t * (D / 64) + i));
        w0[4 * i] = x.x; w0[4 * i + 1] = x.y; w0[4 * i + 2] = x.z; w0[4 * i + 3] = x.w;
        w1[4 * i] = y.x; w1[4 * i + 1] = y.y; w1[4 * i + 2] = y.z; w1[4 * i + 3] = y.w;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a0, a1, a2, a3;
        widen4<CODE>(w0[k], a0, a2);
        widen4<CODE>(w1[k], a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(s[u][n], a0, a1, a2, a3, qf[n][k][0], qf[n][k][1]);
      }
      const uint4 sc = lds128(base + kStageBytes + u * 16);
      const float v = __uint_as_float(sc.y);
      ks[u] = __uint_as_float(sc.x);
      add[u] = sc.z ? __log2f(v) : -INFINITY;
      inv_vs[u] = sc.z ? rcp_fast(v) : 0.f;
      far |= sc.z && !is_near(v);
    }
    const int key0 = cur.tile * Tile<D>::kKeys;
    if (wide || far) {
      if (!wide) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // l is in units of 2^M so far
            l[n][c] = group_add(l[n][c]);
            rmax[n][c] = m[n][c];
            settle(rmax[n][c], l[n][c], 0);
            if (g) l[n][c] = 0.f;
          }
        wide = true;
      }
      sum_scores(s, base + kStageBytes, key0);
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        const uint4 sc = lds128(base + kStageBytes + u * 16);
        const float v = __uint_as_float(sc.y);
        add[u] = sc.z && v >= kTinyScale ? __log2f(v) : -INFINITY;
        inv_vs[u] = 0.f;  // l is complete
      }
    }
#pragma unroll
    for (int u = 0; u < SUBS; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float f1 = qscale[n][c] * ks[u];
          s[u][n][c] = fmaf(s[u][n][c], f1, add[u]);
          s[u][n][2 + c] = fmaf(s[u][n][2 + c], f1, add[u]);
        }
    if (key0 + Tile<D>::kKeys > see_min) {  // some row does not see the whole tile
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        const int k0 = key0 + u * 16 + key_of(g);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + (i >> 1) * 2 >= see[n][i & 1]) s[u][n][i] = -INFINITY;
      }
    }
    // M moves only when it has to: the largest weight is between 2^7 and 2^15
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(s[0][n][c], s[0][n][2 + c]);
#pragma unroll
        for (int u = 1; u < SUBS; ++u) x = fmaxf(x, fmaxf(s[u][n][c], s[u][n][2 + c]));
        grow |= x > m[n][c] + kTopLog + 8.f;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(s[0][n][c], s[0][n][2 + c]);
#pragma unroll
          for (int u = 1; u < SUBS; ++u) x = fmaxf(x, fmaxf(s[u][n][c], s[u][n][2 + c]));
          const float mn = fmaxf(m[n][c], group_max(x) - kTopLog);
          const float keep = mn == -INFINITY ? 1.f : exp2_fast(m[n][c] - mn);
          m[n][c] = mn;
          if (!wide) l[n][c] *= keep;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[n][k][c] *= keep;
            o[n][k][2 + c] *= keep;
          }
        }
    }
    // weights, as the second product's operand
    uint32_t pf[SUBS][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
      const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int u = 0; u < SUBS; ++u) {
        const float p0 = exp2_fast(s[u][n][0] - m0), p1 = exp2_fast(s[u][n][1] - m1);
        const float p2 = exp2_fast(s[u][n][2] - m0), p3 = exp2_fast(s[u][n][3] - m1);
        l[n][0] = fmaf(p0 + p2, inv_vs[u], l[n][0]);
        l[n][1] = fmaf(p1 + p3, inv_vs[u], l[n][1]);
        pf[u][n][0] = transpose8x8(pack2(p0, p1, true));
        pf[u][n][1] = transpose8x8(pack2(p2, p3, true));
      }
    }
    // values: the transposed read gives lane (g, t) keys 4 t .. 4 t + 3 of numbers g and g + 8 of two
    // 16-byte pieces
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        uint32_t v[4];
        read_transposed(v, base + kStageBytes / 2 +
                               piece_offset<D>(u * 16 + (lane & 15), 2 * i + (lane >> 4)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a0, a1, a2, a3;
          widen4<CODE>(v[2 * h], a0, a2);
          widen4<CODE>(v[2 * h + 1], a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(o[n][2 * i + h], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (loaded < end) {
      issue(stage);
      if (++loaded < end) {
        load.step(a, row_limit);
        next_block = fetch_block();
      }
    }
    copy_commit();
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool to_end = cur.tile + 1 == cur.q.tiles;
    if (to_end || f + 1 == end) {
      end_unit(from_start, to_end);
      from_start = true;
      if (f + 1 < end) {
        cur.step(a, row_limit);
        begin_unit();
      }
    } else {
      ++cur.tile;
    }
  }
  copy_wait<0>();
  if (__any_sync(0xffffffffu, bad) && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
}

template <int D, int CODE, int NT>
cudaError_t decode_as(const AttendArgs& a, int sms, int row_limit, cudaStream_t st) {
  static thread_local bool configured[128] = {};
  constexpr int kSmem = kDecodeWarps * kStages * Tile<D>::kStride;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 128 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        decode_kernel<D, CODE, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) configured[dev] = true;
  }
  decode_kernel<D, CODE, NT><<<sms, kDecodeWarps * 32, kSmem, st>>>(
      a, join_space(a.workspace, sms * kDecodeWarps), row_limit);
  return cudaGetLastError();
}

template <int D, int CODE>
cudaError_t decode_with(const AttendArgs& a, int sms, int row_limit, bool one, cudaStream_t st) {
  return one ? decode_as<D, CODE, 1>(a, sms, row_limit, st)
             : decode_as<D, CODE, 2>(a, sms, row_limit, st);
}

// Whether no request has more than eight rows, so that one column group of the product holds them.
bool one_group(const AttendArgs& a) {
  return static_cast<long long>(a.max_q < a.tokens ? a.max_q : a.tokens) * a.group <= 8;
}

}  // namespace

size_t decode_workspace(int sms, int d) { return join_bytes(sms * kDecodeWarps, 16, d); }

// Requests of at most row_limit rows (of one key head); the join has to follow.
cudaError_t launch_decode(const AttendArgs& a, int d, int code, int sms, int row_limit,
                          cudaStream_t st) {
  const bool one = one_group(a);
  if (d == 64)
    return code == ALHR_CODE_INT8 ? decode_with<64, ALHR_CODE_INT8>(a, sms, row_limit, one, st)
                                  : decode_with<64, ALHR_CODE_E4M3>(a, sms, row_limit, one, st);
  return code == ALHR_CODE_INT8 ? decode_with<128, ALHR_CODE_INT8>(a, sms, row_limit, one, st)
                                : decode_with<128, ALHR_CODE_E4M3>(a, sms, row_limit, one, st);
}

cudaError_t launch_decode_join(const AttendArgs& a, int d, int sms, cudaStream_t st) {
  const int pieces = sms * kDecodeWarps;
  const JoinSpace space = join_space(a.workspace, pieces);
  if (one_group(a))
    return d == 64 ? launch_join<64, 8>(a, space, pieces, st)
                   : launch_join<128, 8>(a, space, pieces, st);
  return d == 64 ? launch_join<64, 16>(a, space, pieces, st)
                 : launch_join<128, 16>(a, space, pieces, st);
}

}  // namespace alhr
