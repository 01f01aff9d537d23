// cache_mma.cuh -- 8-bit codes as operands of the warp-wide 16-bit matrix product.
//
// Scores are taken transposed, S^T [16 keys x 8 rows] = K [16 x d] . Q^T [d x 8 rows], and so is
// the sum, O^T [d x 8 rows] = V^T [d x 16 keys] . P^T [16 keys x 8 rows]: the 8-bit operand is the
// 16-row one, so that one to eight query rows fill the product's eight columns.
// A code becomes a half exactly (int8: 8 bits, e4m3: 4 bits of significand), in registers.
#pragma once

#include "cache_device.cuh"

namespace alhr {

// D[16 x 8] += A[16 x 16] B[16 x 8], halves, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of halves held by the warp, lane 4 i + j with columns 2 j, 2 j + 1
// of row i.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Four codes (bytes b0..b3 of w) as two pairs of halves {b0, b1}, {b2, b3}.
// int8: with the sign bit flipped a code is x + 128 in 0..255; as the low byte of 0x64.. it is the
// half 1024 + 128 + x, and one subtraction of 1152 leaves x.
template <int CODE>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (CODE == ALHR_CODE_INT8) {
    w ^= 0x80808080u;
    const uint32_t l = prmt(w, 0x64646464u, 0x4140), h = prmt(w, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&l), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
        " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint32_t shared_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 (or 4) bytes from global to shared memory; bytes = 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// Two 16 x 16 matrices of bytes, lanes 0-15 and 16-31 giving the addresses of their rows of 16
// bytes: lane 4 i + j gets rows 4 j .. 4 j + 3 of column i and of column i + 8 of each.
__device__ __forceinline__ void read_transposed(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// ---- value scales in the exponent (cache_decode.cu, cache_chunk.cu)
// Value scales below this count as 0: such a key has its share of the softmax and no value.
constexpr float kTinyScale = 7.888609052e-31f;  // 2^-100
// Where all value scales of a unit are inside these bounds, the sum of its weights over the scales is
// below 2^(15 + 48) for each of up to 2^30 keys, and what it loses of weights below 2^-126 is 2^(-126
// + 48) a key against 2^(7 - 28) for the key that set M: nothing that 32 bits hold.
constexpr float kNearLow = 3.552713678800501e-15f, kNearHigh = 268435456.f;  // 2^-48, 2^28
__device__ __forceinline__ bool is_near(float v_scale) {
  return v_scale >= kNearLow && v_scale <= kNearHigh;
}

__device__ __forceinline__ float power_of_two(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

}  // namespace alhr
