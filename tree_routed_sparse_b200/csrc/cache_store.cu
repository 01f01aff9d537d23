// cache_store.cu -- new tokens into the paged 8-bit cache, and its numbers back.
//
// Both are bound by memory: a stored number is read once (2 bytes) and written once (1 byte), a
// loaded one the other way round. Measured (replayed from a graph, L2 warm), keys and values of 17.9 K
// tokens x 8 heads, d = 128, e4m3 blocks of 16: 29 us stored, 25 us read back, 52 us together (4.3
// TB/s, 0.65 of the copy rate). One appended token of 64 sequences, int8 blocks of 64: 3.1 us where no
// block's scale grows, 10.3 us where every one's does (up to 63 rows a block are read and written
// again, one pass behind the other), and 3.6 us for reading the blocks back.
//
// store: one warp takes one run (rows of consecutive slots of one block) of one head, keys or
// values: the run's largest magnitude, the block's new scale, the codes of the rows before the run
// if the scale grew, the codes of the run. A pass covers 32 / (d / 8) rows, eight numbers a lane;
// the first eight passes (four of fp32) stay in registers between the maximum and the codes, the
// rest are read again (from L2). The quotient x / s is one rounding of the exact one, by Markstein's correction
// of x * (1 / s) (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): three operations where a division takes about ten.
#include <cuda_fp8.h>

#include "cache_mma.cuh"

namespace alhr {

namespace {

constexpr int kStoreWarps = 4;

template <int T>
struct Raw8 {
  uint4 a[T == ALHR_TYPE_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, long long at) {
    if constexpr (T == ALHR_TYPE_FP32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
      a[0] = __ldg(p);
      a[1] = __ldg(p + 1);
    } else {
      a[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    }
  }
  __device__ __forceinline__ void numbers(float (&x)[8]) const {
    unpack8<T>(a[0], a[T == ALHR_TYPE_FP32 ? 1 : 0], x);
  }
};

// Eight finite numbers as codes: nearest, ties to even, saturated.
template <int CODE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (CODE == ALHR_CODE_INT8) {
      // x + 1.5 * 2^23 holds the rounded number in its low bits
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = __float_as_uint(fminf(fmaxf(x[4 * i + j], -127.f), 127.f) + 12582912.f);
      w[i] = prmt(prmt(c[0], c[1], 0x0040), prmt(c[2], c[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]),
                                                   __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, float* x) {
  uint32_t lo, hi;
  widen4<CODE>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// per: tokens a warp looks through for the beginnings of runs.
template <int D, int CODE, int T>
__global__ void __launch_bounds__(kStoreWarps * 32, 6) store_kernel(const StoreArgs a, const int per) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows a pass
  constexpr int kKept = T == ALHR_TYPE_FP32 ? 4 : 8;  // passes kept in registers (32 of them)
  constexpr float kFull = CODE == ALHR_CODE_INT8 ? 127.f : 256.f;
  const int lane = threadIdx.x & 31;
  const int bs = a.c.bs, heads = a.c.heads;
  const long long slots_end = static_cast<long long>(a.c.blocks) << a.c.bs_log;
  // blockIdx.y, warp: head, keys or values; blockIdx.x: tokens
  const int hw = blockIdx.y * kStoreWarps + (threadIdx.x >> 5);
  if (hw >= 2 * heads) return;
  const int which = hw >= heads, h = hw - which * heads;
  const void* const x = which ? a.x[1] : a.x[0];
  const long long step = which ? a.token_stride[1] : a.token_stride[0];
  const long long head_at = (which ? a.head_stride[1] : a.head_stride[0]) * h;
  const int sub = lane % kLanes, row = lane / kLanes;
  const long long t0 = static_cast<long long>(blockIdx.x) * per;
  const int look = static_cast<int>(min(static_cast<long long>(per), a.tokens - t0));

  // lane i: the slot of token t0 + i, and whether a run begins there (one of the first `look`)
  long long slot = -1;
  bool leads = false;
  if (t0 + lane < a.tokens) slot = __ldg(a.slots + t0 + lane);
  const long long before = t0 > 0 ? __ldg(a.slots + t0 - 1) : -1;  // the same for every lane
  const long long above = __shfl_up_sync(0xffffffffu, slot, 1);
  if (lane < look) {
    if (slot < 0 || slot >= slots_end) {
      if (slot != -1) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
    } else {
      const long long prev = lane ? above : before;
      leads = (slot & (bs - 1)) == 0 || t0 + lane == 0 || prev + 1 != slot;
    }
  }
  for (unsigned left = __ballot_sync(0xffffffffu, leads); left; left &= left - 1) {
    const int at = __ffs(left) - 1;
    const long long s0 = __shfl_sync(0xffffffffu, slot, at);
    const long long t = t0 + at;
    const int off = static_cast<int>(s0 & (bs - 1));
    const int most = static_cast<int>(min(static_cast<long long>(bs - off), a.tokens - t));
    // rows of the run: those among the lanes' tokens, then further ones
    const unsigned here =
        __ballot_sync(0xffffffffu, lane >= at && lane - at < most && slot == s0 + (lane - at)) >> at;
    int n = here == 0xffffffffu ? 32 : __ffs(~here) - 1;
    if (at + n == 32) {
      for (int i = n; i < most; i += 32) {
        const bool on = i + lane < most && __ldg(a.slots + t + i + lane) == s0 + i + lane;
        const unsigned m = __ballot_sync(0xffffffffu, on);
        n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        if (m != 0xffffffffu) break;
      }
    }
    const int block = static_cast<int>(s0 >> a.c.bs_log);
    const long long x0 = t * step + head_at + sub * 8;

    Raw8<T> kept[kKept];
#pragma unroll
    for (int p = 0; p < kKept; ++p)
      if (p * kRows + row < n) kept[p].load(x, x0 + (p * kRows + row) * step);
    float amax = 0.f;
    bool odd = false;
    auto largest = [&](const Raw8<T>& r) {
      float v[8];
      r.numbers(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(v[j]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
        else odd = true;
      }
    };
#pragma unroll
    for (int p = 0; p < kKept; ++p)
      if (p * kRows + row < n) largest(kept[p]);
#pragma unroll 4
    for (int i = kKept * kRows + row; i < n; i += kRows) {
      Raw8<T> r;
      r.load(x, x0 + i * step);
      largest(r);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    odd = __any_sync(0xffffffffu, odd);
    if (odd && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_NONFINITE);

    float* scale = (which ? a.c.v_scale : a.c.k_scale) + static_cast<long long>(block) * heads + h;
    const float old = off == 0 ? 0.f : *scale;
    const float s = fmaxf(fmaxf(old, __fdiv_rn(amax, kFull)), kTinyScale);
    uint8_t* codes = (which ? a.c.v : a.c.k) + block_row(a.c, block, h) * D + sub * 8;
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = s;
    if (s > old && off > 0) {
      const float f = __fdiv_rn(old, s);
      for (int i = row; i < off; i += kRows) {
        uint2* p = reinterpret_cast<uint2*>(codes + static_cast<long long>(i) * D);
        const uint2 c = *p;
        float v[8];
        decode4<CODE>(c.x, v);
        decode4<CODE>(c.y, v + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], f);
        *p = encode8<CODE>(v);
      }
    }
    const float inv = __frcp_rn(s);
    auto put = [&](const Raw8<T>& r, int i) {
      float v[8];
      r.numbers(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[j], q = __fmul_rn(x, inv);
        v[j] = __fmaf_rn(__fmaf_rn(-q, s, x), inv, q);
      }
      // The correction makes NaN of an infinity: it becomes a quotient that saturates, NaN becomes
      // 0. A branch of the warp's: selects in the loop above cost every run (56 us for 51).
      if (odd) {
        float x[8];
        r.numbers(x);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(fabsf(x[j]) <= 3.402823466e38f)) v[j] = x[j] == x[j] ? copysignf(512.f, x[j]) : 0.f;
      }
      *reinterpret_cast<uint2*>(codes + static_cast<long long>(off + i) * D) = encode8<CODE>(v);
    };
#pragma unroll
    for (int p = 0; p < kKept; ++p)
      if (p * kRows + row < n) put(kept[p], p * kRows + row);
#pragma unroll 4
    for (int i = kKept * kRows + row; i < n; i += kRows) {
      Raw8<T> r;
      r.load(x, x0 + i * step);
      put(r, i);
    }
  }
}

// Threads (piece, token): eight numbers of one head, keys or values, of kTokens tokens each, whose
// loads do not wait for one another.
constexpr int kTokens = 4;

template <int D, int CODE, int T>
__global__ void __launch_bounds__(256) load_kernel(const LoadArgs a) {
  constexpr int kPieces = D / 8;
  const int heads = a.c.heads, all = 2 * heads * kPieces;
  const long long slots_end = static_cast<long long>(a.c.blocks) << a.c.bs_log;
  const long long t0 = (static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y) * kTokens;
  long long slot[kTokens];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    slot[i] = t0 + i < a.tokens ? __ldg(a.slots + t0 + i) : -1;
    if (slot[i] < 0 || slot[i] >= slots_end) {
      bad |= slot[i] != -1;
      slot[i] = -1;
    }
  }
  if (bad && threadIdx.x == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
  for (int p = threadIdx.x; p < all; p += blockDim.x) {
    const int sub = p % kPieces, hw = p / kPieces;
    const int which = hw >= heads, h = hw - which * heads;
    void* const to = which ? a.x[1] : a.x[0];
    const uint8_t* const codes = (which ? a.c.v : a.c.k) + sub * 8;
    const float* const scales = (which ? a.c.v_scale : a.c.k_scale) + h;
    uint2 c[kTokens];
    float s[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      c[i] = make_uint2(0u, 0u);
      s[i] = 0.f;
      if (slot[i] >= 0) {
        const int block = static_cast<int>(slot[i] >> a.c.bs_log);
        const int off = static_cast<int>(slot[i] & (a.c.bs - 1));
        c[i] = __ldg(reinterpret_cast<const uint2*>(codes + (block_row(a.c, block, h) + off) * D));
        s[i] = __ldg(scales + static_cast<long long>(block) * heads);
      }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (t0 + i >= a.tokens) break;
      float v[8];
      decode4<CODE>(c[i].x, v);
      decode4<CODE>(c[i].y, v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = slot[i] >= 0 ? __fmul_rn(v[j], s[i]) : 0.f;
      const long long at = ((t0 + i) * heads + h) * D + sub * 8;
      if constexpr (T == ALHR_TYPE_FP32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(to) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        constexpr bool kHalf = T == ALHR_TYPE_FP16;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + at) =
            make_uint4(pack2(v[0], v[1], kHalf), pack2(v[2], v[3], kHalf), pack2(v[4], v[5], kHalf),
                       pack2(v[6], v[7], kHalf));
      }
    }
  }
}

template <int D, int CODE, int T>
cudaError_t store_as(const StoreArgs& a, cudaStream_t st) {
  // One token a warp while that leaves the GPU room (each may be a run of its own), else 16. Neither
  // is the better one for every call of a size. Microseconds at one token and at 16 a warp, 8 heads,
  // d = 128, bf16 into int8 blocks of 64, by the number of tokens:
  //                                512          1024         2048         4096         large
  //   one token a sequence         8.2 / 26.2   13.4 / 27.1  25.2 / 29.4  47.8 / 56.2  93.5 / 86.1 (8192)
  //   whole blocks                 13.3 / 12.3  15.6 / 12.8  20.5 / 18.2  28.2 / 23.0  87.7 / 44.6 (16,384)
  // The step lies at 1024 tokens of 8 heads: single tokens behind it pay for the prompts (27 us for
  // 14.6 at 1100).
  const long long warps = static_cast<long long>(a.tokens) * a.c.heads * 2;
  const int per = warps <= 16384 ? 1 : 16;
  const dim3 grid(static_cast<unsigned>((a.tokens + per - 1) / per),
                  static_cast<unsigned>((2 * a.c.heads + kStoreWarps - 1) / kStoreWarps));
  if (grid.y > 65535u) return cudaErrorInvalidConfiguration;
  store_kernel<D, CODE, T><<<grid, kStoreWarps * 32, 0, st>>>(a, per);
  return cudaGetLastError();
}

template <int D, int CODE, int T>
cudaError_t load_as(const LoadArgs& a, cudaStream_t st) {
  const int pieces = 2 * a.c.heads * (D / 8);
  unsigned x = 32;
  while (x < 256 && x < static_cast<unsigned>(pieces)) x *= 2;
  const dim3 threads(x, 256 / x);
  const unsigned each = threads.y * kTokens;
  const unsigned grid = (static_cast<unsigned>(a.tokens) + each - 1) / each;
  load_kernel<D, CODE, T><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

#define ALHR_BY_TYPE(fn, D, CODE)                                       \
  (type == ALHR_TYPE_BF16   ? fn<D, CODE, ALHR_TYPE_BF16>(a, st)         \
   : type == ALHR_TYPE_FP16 ? fn<D, CODE, ALHR_TYPE_FP16>(a, st)         \
                            : fn<D, CODE, ALHR_TYPE_FP32>(a, st))
#define ALHR_BY_CODE(fn, D) \
  (code == ALHR_CODE_INT8 ? ALHR_BY_TYPE(fn, D, ALHR_CODE_INT8) : ALHR_BY_TYPE(fn, D, ALHR_CODE_E4M3))

cudaError_t launch_store_cache(const StoreArgs& a, int d, int code, int type, cudaStream_t st) {
  return d == 64 ? ALHR_BY_CODE(store_as, 64) : ALHR_BY_CODE(store_as, 128);
}

cudaError_t launch_load_cache(const LoadArgs& a, int d, int code, int type, cudaStream_t st) {
  return d == 64 ? ALHR_BY_CODE(load_as, 64) : ALHR_BY_CODE(load_as, 128);
}

}  // namespace alhr
