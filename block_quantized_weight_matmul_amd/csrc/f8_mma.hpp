// f8_mma.hpp -- the group sum of e4m3 operands on the matrix cores, shared by the products.
//
//   y[t][r] = sum_g sx[g][t] * sw[g][r] * sum_{k in group g} xq[t][k] * wq[r][k]
//
// The inner sum of a group runs on the matrix cores, and the group's two scales multiply the finished sum in fp32 on the
// vector units.  Which cores depends on the output's type:
//   16-bit outputs  v_mfma_f32_16x16x128_f8f6f4, whose depth is the group.  It takes the codes as they are, but it
//                   aligns the products of every 8 values to 13 bits below their largest exponent (measured: a product
//                   2^-14 of its octet's largest is lost), an error of 1.5e-5 of the result on normal data and 6e-5 on
//                   data of a wide range: 1/16 of half a step of fp16, 1/130 of bf16's.
//   fp32 outputs    v_mfma_f32_16x16x32_f16 on the codes converted to fp16, which holds every e4m3 value: the same sums
//                   kept to 24 bits (1e-8), at half the rate and two conversions a register.
// Weight rows are the A rows of
// the instruction and tokens its columns, so that a lane holds 4 consecutive outputs of one token and its token scale
// is one register.  The 128 values of a group may reach the instruction in any order as long as both operands use the
// same one: lane (row l & 15, quarter l >> 4) takes bytes 32 * quarter .. + 31 of its row.
#pragma once

#include "f8.hpp"

namespace qmm {

constexpr int kUnitScale = 0x7F7F7F7F;  // e8m0 exponents of 1: the instruction's own scales are not used

__device__ __forceinline__ f32x4 mfma(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, kUnitScale, 0, kUnitScale);
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
