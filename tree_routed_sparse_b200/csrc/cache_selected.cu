// cache_selected.cu -- attention of each query over its own selected positions (at most 96).
//
// Mathematics: s_j = (q . kcode_j) k_scale_j scale log2 e, p_j = 2^(s_j - max s), l = sum p_j,
// out = sum p_j v_scale_j vcode_j / l, in fp32.
//
// What bounds it: 2 d bytes a selected key, gathered (from L2 where sequences are re-read), and
// the widening of the codes. One warp takes one query. Each lane looks up the pages of its keys
// once; then groups of 16 keys go from global memory straight into the operand registers of the
// warp-wide matrix product: K rows times the query (in all eight columns, so that every lane has
// the scores of its keys), and values times weights. A weight is used as two halves, its rounding
// and what that left (2^-22 of it together), which lie in neighbouring columns and are added at
// the end: the output is as exact as one with fp32 weights at the cost of one product.
// Measured: 2 x 8 x 16,384 queries of up to 96 of 16,384 keys, d = 64: 590 us (3.2 GB gathered, 5.4
// TB/s; 1.6 K warp instructions a query, 0.67 of the issue slots); 64 x 8 queries, d = 128: 10 us.
// int8 scores by four-product integer instructions were slower (739 us: they issue at a fraction of
// the products' rate), and so were fewer warps with more registers (692 us at 16 warps a
// multiprocessor, 588 at 32).
#include <cmath>

#include "cache_mma.cuh"

namespace alhr {

namespace {

constexpr int kSelWarps = 4;
constexpr int kSelKeys = 96, kSelGroups = kSelKeys / 16;

struct SelKey {
  int row;        // code row of the key's head; of another key of the query where this one is skipped
  int on;         // 0: skipped
  float k_scale, v_scale;
};

template <int D, int CODE>
__global__ void __launch_bounds__(kSelWarps * 32, D == 64 ? 8 : 6) selected_kernel(const SelectArgs a) {
  constexpr int KS = D / 16;   // products over d of one 16-key group
  constexpr int W = D / 32;    // words of values a lane takes of a key
  __shared__ SelKey keys[kSelWarps][kSelKeys];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  SelKey* const mine = keys[warp];
  for (long long u = static_cast<long long>(blockIdx.x) * kSelWarps + warp; u < a.rows;
       u += static_cast<long long>(gridDim.x) * kSelWarps) {
    const int bh = static_cast<int>(u) / a.nq;  // rows are below 2^31
    const int row_t = static_cast<int>(u) - bh * a.nq;
    const int b = bh / a.q_heads, h = (bh - b * a.q_heads) / a.group;
    const int count = min(max(__ldg(a.count + u), 0), a.max_keys);
    const long long cap = static_cast<long long>(a.max_blocks) << a.c.bs_log;
    const long long pos = static_cast<long long>(__ldg(a.ctx_len + b)) + row_t;
    const long long see = min(min(pos + 1, static_cast<long long>(__ldg(a.seq_len + b))), cap);
    // ---- where the keys lie
    uint32_t flags = 0;
    int spare = -1, behind = 0;  // behind: groups of 32 entries before the first that has a key
#pragma unroll
    for (int i = 0; i < kSelKeys / 32; ++i) {
      const int e = i * 32 + lane;
      SelKey k{-1, 0, 0.f, 0.f};
      if (e < count) {
        const int j = __ldg(a.idx + u * a.max_keys + e);
        if (j >= 0 && j < see) {
          const int block =
              __ldg(a.table + static_cast<long long>(b) * a.max_blocks + (j >> a.c.bs_log));
          if (block >= 0 && block < a.c.blocks) {
            const long long si = static_cast<long long>(block) * a.c.heads + h;
            k.row = static_cast<int>((si << a.c.bs_log) + (j & (a.c.bs - 1)));
            k.on = 1;
            k.k_scale = __ldg(a.c.k_scale + si);
            k.v_scale = __ldg(a.c.v_scale + si);
          } else {
            flags |= ALHR_DEVERR_BLOCK;
          }
        } else {
          flags |= ALHR_DEVERR_INDEX;
        }
      }
      // a skipped key reads the row of one that is not (in bounds, and as finite as the rest)
      const unsigned some = __ballot_sync(0xffffffffu, k.on);
      if (some) spare = __shfl_sync(0xffffffffu, k.row, __ffs(some) - 1);
      if (spare < 0) behind = i + 1;
      if (!k.on) k.row = max(spare, 0);
      mine[e] = k;
    }
    if (spare >= 0)
      for (int i = 0; i < behind; ++i) mine[i * 32 + lane].row = spare;
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0) cache_flag(a.dev_err, flags);
    // ---- the query: lane t holds numbers 16 (4 j + t) .. + 15, scaled by a power of two
    uint32_t qf[KS][2];
    float qs;
    {
      float x[D / 4];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const long long at = u * D + (j * 4 + t) * 16;
        if (a.type == ALHR_TYPE_INT8) {
          const uint4 w =
              __ldg(reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.q) + at));
          const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[j * 16 + i] = static_cast<float>(static_cast<int8_t>(v[i >> 2] >> (8 * (i & 3))));
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 w = __ldg(p + i);
            float y[8];
            if (a.type == ALHR_TYPE_FP16) unpack8<ALHR_TYPE_FP16>(w, w, y);
            else unpack8<ALHR_TYPE_BF16>(w, w, y);
#pragma unroll
            for (int c = 0; c < 8; ++c) x[j * 16 + i * 8 + c] = y[c];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e2 = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100), 126);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e2) << 23);
      qs = __uint_as_float(static_cast<uint32_t>(127 - 14 + e2) << 23) * a.scale_log2;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[s][0] = pack2(x[4 * s] * up, x[4 * s + 1] * up, true);
        qf[s][1] = pack2(x[4 * s + 2] * up, x[4 * s + 3] * up, true);
      }
    }
    __syncwarp();
    // ---- scores of keys 16 i + g and 16 i + 8 + g
    float s[kSelGroups][2];
    const int groups = (count + 15) >> 4;
#pragma unroll
    for (int i = 0; i < kSelGroups; ++i) {
      s[i][0] = s[i][1] = -INFINITY;
      if (i < groups) {
        const SelKey k0 = mine[i * 16 + g], k1 = mine[i * 16 + 8 + g];
        uint4 w0[D / 64], w1[D / 64];
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const int piece = (j * 4 + t) * 16;
          w0[j] = __ldg(reinterpret_cast<const uint4*>(
              a.c.k + static_cast<long long>(k0.row) * D + piece));
          w1[j] = __ldg(reinterpret_cast<const uint4*>(
              a.c.k + static_cast<long long>(k1.row) * D + piece));
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const uint32_t v0[4] = {w0[j].x, w0[j].y, w0[j].z, w0[j].w};
          const uint32_t v1[4] = {w1[j].x, w1[j].y, w1[j].z, w1[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a0, a1, a2, a3;
            widen4<CODE>(v0[k], a0, a2);
            widen4<CODE>(v1[k], a1, a3);
            mma16816(c, a0, a1, a2, a3, qf[j * 4 + k][0], qf[j * 4 + k][1]);
          }
        }
        if (k0.on) s[i][0] = c[0] * (qs * k0.k_scale);
        if (k1.on) s[i][1] = c[2] * (qs * k1.k_scale);
      }
    }
    // ---- weights
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSelGroups; ++i) m = fmaxf(m, fmaxf(s[i][0], s[i][1]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, most = 0.f;
#pragma unroll
    for (int i = 0; i < kSelGroups; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float p = exp2_fast(s[i][c] - base);
        l += p;
        s[i][c] = i < groups ? p * mine[i * 16 + 8 * c + g].v_scale : 0.f;
        most = fmaxf(most, s[i][c]);
      }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, o);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    // the largest weight goes to [2^14, 2^15), exactly
    const int ew = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 126);
    const float wup = __uint_as_float(static_cast<uint32_t>(127 + 14 - ew) << 23);
    const float wdown = __uint_as_float(static_cast<uint32_t>(127 - 14 + ew) << 23);
    float o[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k][i] = 0.f;
#pragma unroll
    for (int i = 0; i < kSelGroups; ++i) {
      if (i < groups) {
        uint32_t pf[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float w = s[i][c] * wup;
          const float hi = __half2float(__float2half_rn(w));
          pf[c] = transpose8x8(pack2(hi, w - hi, true));
        }
        uint32_t v[4][W];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = mine[i * 16 + 2 * t + (r & 1) + (r >> 1) * 8].row;
          const uint8_t* p = a.c.v + static_cast<long long>(row) * D + g * (D / 8);
          if constexpr (D == 128) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
            v[r][0] = w.x; v[r][1] = w.y; v[r][2] = w.z; v[r][3] = w.w;
          } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
            v[r][0] = w.x; v[r][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
          widen4<CODE>(prmt(v[0][w], v[1][w], 0x5140), x0, x1);
          widen4<CODE>(prmt(v[0][w], v[1][w], 0x7362), x2, x3);
          widen4<CODE>(prmt(v[2][w], v[3][w], 0x5140), y0, y1);
          widen4<CODE>(prmt(v[2][w], v[3][w], 0x7362), y2, y3);
          mma16816(o[2 * w], x0, x1, y0, y1, pf[0], pf[1]);
          mma16816(o[2 * w + 1], x2, x3, y2, y3, pf[0], pf[1]);
        }
      }
    }
    // ---- numbers g D / 8 .. + D / 8 - 1 of the output, every t has them: t writes its share
    const float inv = wdown / l;
    float* out = a.out + u * D + g * (D / 8);
#pragma unroll
    for (int k = 0; k < KS / 2; ++k) {
      float4 y = make_float4((o[2 * k][0] + o[2 * k][1]) * inv, (o[2 * k][2] + o[2 * k][3]) * inv,
                             (o[2 * k + 1][0] + o[2 * k + 1][1]) * inv,
                             (o[2 * k + 1][2] + o[2 * k + 1][3]) * inv);
      if (l == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);  // no key; NaN stays
      if (t == k) reinterpret_cast<float4*>(out)[k] = y;
    }
    __syncwarp();  // every lane has read the keys
  }
}

template <int D, int CODE>
cudaError_t selected_as(const SelectArgs& a, cudaStream_t st) {
  const long long grid = (static_cast<long long>(a.rows) + kSelWarps - 1) / kSelWarps;
  selected_kernel<D, CODE>
      <<<static_cast<unsigned>(grid < (1 << 20) ? grid : (1 << 20)), kSelWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_selected(const SelectArgs& a, int d, int code, cudaStream_t st) {
  if (d == 64)
    return code == ALHR_CODE_INT8 ? selected_as<64, ALHR_CODE_INT8>(a, st)
                                  : selected_as<64, ALHR_CODE_E4M3>(a, st);
  return code == ALHR_CODE_INT8 ? selected_as<128, ALHR_CODE_INT8>(a, st)
                                : selected_as<128, ALHR_CODE_E4M3>(a, st);
}

}  // namespace alhr
