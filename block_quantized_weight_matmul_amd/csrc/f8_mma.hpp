// f8_mma.hpp -- the group sum of e4m3 operands on the matrix cores, shared by the products.
//
//   y[t][r] = sum_g sx[g][t] * sw[g][r] * sum_{k in group g} xq[t][k] * wq[r][k]
//
// The inner sum of a group runs on the matrix cores, and the group's two scales multiply the finished sum in fp32 on the
// vector units.  Which cores depends on the output's type:
//   16-bit outputs  v_mfma_f32_16x16x128_f8f6f4, whose depth is the group.  It takes the codes as they are, but it
//                   aligns the products of every 8 values to 13 bits below their largest exponent (measured: a product
//                   2^-14 of its octet's largest is lost).  Of the outputs' root mean square that is 1.4e-5 on normal
//                   data and 6e-5 to 7e-5 with one channel 300 times larger, beside 2.1e-4 for an output's rounding to
//                   fp16 and 1.7e-3 to bf16 (512 and 16 tokens of 1024 x 2560).
//   fp32 outputs    v_mfma_f32_16x16x32_f16 on the codes converted to fp16, which holds every e4m3 value: the same sums
//                   kept to 24 bits (1e-7), at half the rate and two conversions a register.
// Weight rows are the A rows of the instruction and tokens its columns, so that a lane holds 4 consecutive outputs of one
// token and its token scale is one register.  The 128 values of a group may reach the instruction in any order as long as
// both operands use the same one: lane (row l & 15, quarter l >> 4) takes bytes 32 * quarter .. + 31 of its row.
#pragma once

#include "f8.hpp"

namespace qmm {

// (scale operands that are the constant 0 select the instruction without scales)
__device__ __forceinline__ f32x4 mfma(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// A lane's 32 codes of an operand as the matrix cores take them, and the group's sum.
template <bool EXACT> struct Frag;
template <> struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) { v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <> struct Frag<true> {
  half8 v[4];
  __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = i < 2 ? lo[2 * i] : hi[2 * i - 4], b = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
      const half2v p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false), q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
      const half2v r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false), t = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
      v[i] = half8{p[0], p[1], q[0], q[1], r[0], r[1], t[0], t[1]};
    }
  }
};
__device__ __forceinline__ f32x4 group_sum(const Frag<false>& a, const Frag<false>& b) {
  return mfma(a.v, b.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
}
__device__ __forceinline__ f32x4 group_sum(const Frag<true>& a, const Frag<true>& b) {
  f32x4 c{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// The 32 x 32 shape of the tiled kernels: half the operand reads of a 16 x 16 product, which leaves the vector units
// room for the scales (registers only, 2 waves a SIMD: 3.5 PFLOP/s with them, 96% of the cores' rate at the clock the
// power allows, against 3.2 and 64% with the 16 x 16 shape).  Lane (row l & 31, half l >> 5) takes the 16-byte pieces
// 4 m + 2 half, + 1 of its row for m = 0, 1; of a sum it holds column l & 31, rows 8 (i / 4) + 4 half + i % 4, i < 16.
template <bool EXACT> struct Frag32;
template <> struct Frag32<false> {
  i32x8 v[2];
  __device__ __forceinline__ void set(int m, i32x4 lo, i32x4 hi) { v[m] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <> struct Frag32<true> {
  Frag<true> v[2];
  __device__ __forceinline__ void set(int m, i32x4 lo, i32x4 hi) { v[m].set(lo, hi); }
};
__device__ __forceinline__ f32x16 group_sum(const Frag32<false>& a, const Frag32<false>& b) {
  f32x16 c{};
  c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v[0], b.v[0], c, 0, 0, 0, 0, 0, 0);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.v[1], b.v[1], c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 group_sum(const Frag32<true>& a, const Frag32<true>& b) {
  f32x16 c{};
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_f16(a.v[i / 4].v[i % 4], b.v[i / 4].v[i % 4], c, 0, 0, 0);
  return c;
}

// The two scales of a group as the smaller and the larger (a NaN stays one of them).  Their product leaves fp32's range
// where both are small or both large, though the sum times both does not: p * lo keeps its bits, since |p| >= 2^-18 and
// lo >= 2^-80, and overflows only where the result does.
__device__ __forceinline__ float2 scale_order(float a, float b) { return a < b ? make_float2(a, b) : make_float2(b, a); }

template <int OT>
__device__ __forceinline__ void store4(typename Elem<OT>::T* p, f32x4 v, int n, bool vec) {
  typedef typename Elem<OT>::T T;
  if (vec && n >= 4) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = to_elem<OT>(v[i]);
    *reinterpret_cast<T4*>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = to_elem<OT>(v[i]);
  }
}

inline int store_vec(const void* y, int64_t M, int ot) {
  const int64_t b = ot == DT_F32 ? 16 : 8;
  return reinterpret_cast<uintptr_t>(y) % b == 0 && M % 4 == 0;
}

}  // namespace qmm
