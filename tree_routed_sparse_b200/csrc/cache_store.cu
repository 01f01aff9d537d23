// cache_store.cu -- new tokens into the paged 8-bit cache, and its numbers back.
//
// store: one warp takes one run (rows of consecutive slots of one block) of one head, keys or
// values: the run's largest magnitude, the block's new scale, the codes of the rows before the run
// if the scale grew, the codes of the run. Each pass covers 32 / (d / 8) rows, eight numbers a
// lane.
#include "cache_device.cuh"

namespace alhr {

namespace {

constexpr int kStoreWarps = 4;

template <int T>
__device__ __forceinline__ void load8(const void* base, long long at, float (&x)[8]) {
  if constexpr (T == ALHR_TYPE_FP32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    unpack8<T>(__ldg(p), __ldg(p + 1), x);
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    unpack8<T>(a, a, x);
  }
}

template <int CODE>
__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i >> 2] |= static_cast<uint32_t>(encode<CODE>(x[i])) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

template <int CODE>
__device__ __forceinline__ void decode8(const uint2& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = decode<CODE>(static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3))));
}

template <int D, int CODE, int T>
__global__ void __launch_bounds__(kStoreWarps * 32) store_kernel(const StoreArgs a) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows a pass
  constexpr float kFull = CODE == ALHR_CODE_INT8 ? 127.f : 256.f;
  const int lane = threadIdx.x & 31;
  const int bs = a.c.bs, heads = a.c.heads;
  const long long slots_end = static_cast<long long>(a.c.blocks) << a.c.bs_log;
  const long long units = static_cast<long long>(a.tokens) * heads * 2;
  for (long long u = static_cast<long long>(blockIdx.x) * kStoreWarps + (threadIdx.x >> 5);
       u < units; u += static_cast<long long>(gridDim.x) * kStoreWarps) {
    const int t = static_cast<int>(u / (2 * heads));
    const int hw = static_cast<int>(u - static_cast<long long>(t) * 2 * heads);
    const int which = hw >= heads, h = hw - which * heads;
    const long long slot = __ldg(a.slots + t);
    if (slot < 0 || slot >= slots_end) {
      if (slot != -1 && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
      continue;
    }
    const int off = static_cast<int>(slot & (bs - 1));
    if (off != 0 && t > 0 && __ldg(a.slots + t - 1) + 1 == slot) continue;  // inside a run
    int n = 0;  // rows of the run
    const int most = min(bs - off, a.tokens - t);
    for (int i = 0; i < most; i += 32) {
      const bool on = i + lane < most && __ldg(a.slots + t + i + lane) == slot + i + lane;
      const unsigned m = __ballot_sync(0xffffffffu, on);
      n += m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      if (m != 0xffffffffu) break;
    }
    const int block = static_cast<int>(slot >> a.c.bs_log);
    const int sub = lane % kLanes, row = lane / kLanes;
    const void* x = a.x[which];
    const long long x0 = static_cast<long long>(t) * a.token_stride[which] +
                         static_cast<long long>(h) * a.head_stride[which] + sub * 8;
    const long long step = a.token_stride[which];

    float amax = 0.f;
    bool odd = false;
    for (int i = row; i < n; i += kRows) {
      float v[8];
      load8<T>(x, x0 + i * step, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(v[j]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
        else odd = true;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (__any_sync(0xffffffffu, odd) && lane == 0) cache_flag(a.dev_err, ALHR_DEVERR_NONFINITE);

    float* scale = (which ? a.c.v_scale : a.c.k_scale) + static_cast<long long>(block) * heads + h;
    const float old = off == 0 ? 0.f : *scale;
    const float s = fmaxf(fmaxf(old, __fdiv_rn(amax, kFull)), 7.888609052e-31f);  // 2^-100
    uint8_t* codes = (which ? a.c.v : a.c.k) + block_row(a.c, block, h) * D + sub * 8;
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = s;
    if (s > old && off > 0) {
      const float f = __fdiv_rn(old, s);
      for (int i = row; i < off; i += kRows) {
        uint2* p = reinterpret_cast<uint2*>(codes + static_cast<long long>(i) * D);
        float v[8];
        decode8<CODE>(*p, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], f);
        *p = encode8<CODE>(v);
      }
    }
    for (int i = row; i < n; i += kRows) {
      float v[8];
      load8<T>(x, x0 + i * step, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(v[j], s);
      *reinterpret_cast<uint2*>(codes + static_cast<long long>(off + i) * D) = encode8<CODE>(v);
    }
  }
}

template <int D, int CODE, int T>
__global__ void __launch_bounds__(256) load_kernel(const LoadArgs a) {
  constexpr int kLanes = D / 8;
  const int heads = a.c.heads;
  const long long slots_end = static_cast<long long>(a.c.blocks) << a.c.bs_log;
  const long long units = static_cast<long long>(a.tokens) * heads * 2 * kLanes;
  bool bad = false;
  for (long long u = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; u < units;
       u += static_cast<long long>(gridDim.x) * 256) {
    const int sub = static_cast<int>(u % kLanes);
    const long long rest = u / kLanes;
    const int hw = static_cast<int>(rest % (2 * heads));
    const long long t = rest / (2 * heads);
    const int which = hw >= heads, h = hw - which * heads;
    const long long slot = __ldg(a.slots + t);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (slot >= 0 && slot < slots_end) {
      const int block = static_cast<int>(slot >> a.c.bs_log);
      const int off = static_cast<int>(slot & (a.c.bs - 1));
      const uint8_t* codes =
          (which ? a.c.v : a.c.k) + (block_row(a.c, block, h) + off) * D + sub * 8;
      const float s =
          __ldg((which ? a.c.v_scale : a.c.k_scale) + static_cast<long long>(block) * heads + h);
      decode8<CODE>(__ldg(reinterpret_cast<const uint2*>(codes)), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], s);
    } else if (slot != -1) {
      bad = true;
    }
    const long long at = (t * heads + h) * D + sub * 8;
    if constexpr (T == ALHR_TYPE_FP32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.x[which]) + at);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      constexpr bool kHalf = T == ALHR_TYPE_FP16;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x[which]) + at) =
          make_uint4(pack2(v[0], v[1], kHalf), pack2(v[2], v[3], kHalf), pack2(v[4], v[5], kHalf),
                     pack2(v[6], v[7], kHalf));
    }
  }
  if (bad) cache_flag(a.dev_err, ALHR_DEVERR_BLOCK);
}

template <int D, int CODE, int T>
cudaError_t store_as(const StoreArgs& a, cudaStream_t st) {
  const long long units = static_cast<long long>(a.tokens) * a.c.heads * 2;
  const long long grid = (units + kStoreWarps - 1) / kStoreWarps;
  store_kernel<D, CODE, T>
      <<<static_cast<unsigned>(grid < (1 << 20) ? grid : (1 << 20)), kStoreWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D, int CODE, int T>
cudaError_t load_as(const LoadArgs& a, cudaStream_t st) {
  const long long units = static_cast<long long>(a.tokens) * a.c.heads * 2 * (D / 8);
  const long long grid = (units + 255) / 256;
  load_kernel<D, CODE, T>
      <<<static_cast<unsigned>(grid < (1 << 20) ? grid : (1 << 20)), 256, 0, st>>>(a);
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
