// f8.hpp -- e4m3 values with a scale for each block of 128: device helpers of the quantizers and products, and
// the launch interface between the C ABI (f8_api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

// Element types of the calls' 16- and 32-bit tensors (the values of qmm_dtype).
enum { DT_F32 = 0, DT_F16 = 1, DT_BF16 = 2 };

constexpr int kF8Block = 128;             // values per scale along K; rows per scale of a weight block
constexpr float kF8Max = 448.0f;          // largest e4m3 value
constexpr float kF8MinScale = 0x1p-80f;   // smallest scale: keeps remainders of the quotient exact
constexpr int64_t kF8MaxRows = int64_t(1) << 24;  // rows of a call's tokens, weights and outputs
constexpr int64_t kF8MaxK = int64_t(1) << 22;     // padded K of a call: a tile's rows stay in 32-bit offsets
constexpr int64_t kRouteMaxExperts = 1024;
constexpr int64_t kRouteMaxPairs = int64_t(1) << 22;

inline __host__ __device__ int64_t f8_pad(int64_t n) { return (n + kF8Block - 1) / kF8Block * kF8Block; }

struct F8Desc {
  const uint8_t* codes;  // [n_experts][M][Kp], Kp = f8_pad(K)
  const float* scales;   // [n_experts][f8_pad(M) / 128][Kp / 128]
  int64_t n_experts, M, K, Kp;
  int cus;
};

// Routing plan: int32 arrays in one device buffer (route.hip builds it, the expert products read it).  Pairs are
// sorted by bucket, ascending inside one: buckets 0 .. E-1 the experts, E the empty slots (id -1), E+1 ids that
// name no expert.  map[t] lists, per token tile of kPlanTiles[t] pairs, (bucket, first position, end position).
constexpr int kPlanTileKinds = 3;
constexpr int kPlanTiles[kPlanTileKinds] = {32, 64, 128};
struct PlanDesc {
  int64_t pairs, E;
  // int32 offsets in the buffer; totals: tiles of each kind
  int64_t counts, offsets, tile128, totals, order, map[kPlanTileKinds], scratch, total;
  int64_t cap[kPlanTileKinds];                                                    // entries of each map
};
PlanDesc plan_desc(int64_t pairs, int64_t E);
hipError_t launch_route_plan(const int32_t* ids, int64_t pairs, int64_t E, int32_t* plan, hipStream_t s);

// Quantizers.  codes_r / scales_r: groups of 128 along K ([N][Kp], [Kp / 128][N]); codes_c / scales_c: groups of
// 128 along the rows ([K][Np], [Np / 128][K]); either may be null.  plan: rows are the plan's pairs, each expert's
// padded to 128 on their own (Np = 128 * cap[3]); pair p reads row p / slots.
struct F8QuantArgs {
  const void* x;
  int64_t ldx, N, K;
  uint8_t* codes_r;
  float* scales_r;
  uint8_t* codes_c;
  float* scales_c;
  const int32_t* plan;  // null: dense
  PlanDesc pd;
  int slots;  // rows of x a pair shares: pair / slots
};
hipError_t launch_f8_quantize(const F8QuantArgs& a, int dt, hipStream_t s);
// Weights: one scale per 128 x 128 block; codes_t / scales_t (may be null): the transposed matrix' codes.
hipError_t launch_f8_quantize_weight(const void* w, int dt, int64_t E, int64_t M, int64_t K, uint8_t* codes,
                                     float* scales, uint8_t* codes_t, float* scales_t, hipStream_t s);
hipError_t launch_f8_transpose(const F8Desc& m, uint8_t* codes_t, float* scales_t, hipStream_t s);
hipError_t launch_f8_dequantize(const F8Desc& m, int64_t expert, void* out, int dt, hipStream_t s);

// Products.  Dense: y[N][M] = x W^T of quantized tokens (codes_r / scales_r layout).
size_t f8_gemm_workspace_bytes(const F8Desc& m, int64_t N);
hipError_t launch_f8_gemm(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t N, void* y, int yt, void* ws,
                          hipStream_t s);
// Fused quantization for few tokens: whether a raw call of N tokens takes one launch, and that launch.
bool f8_linear_fused(const F8Desc& m, int64_t N);
hipError_t launch_f8_linear(const F8Desc& m, const void* x, int xt, int64_t ldx, int64_t N, void* y, int yt,
                            hipStream_t s);
// the kernel of few tokens, of quantized ones: whether a call takes it, and its launch
bool f8_few_tokens(const F8Desc& m, int64_t N);
hipError_t launch_f8_few(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t N, void* y, int yt, hipStream_t s);
// Expert-indexed: rows of x are tokens (slots = S) or pairs (slots = 1); y [pairs][M].
hipError_t launch_f8_gemm_id(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t pairs, int slots,
                             const int32_t* plan, void* y, int yt, hipStream_t s);
bool f8_linear_id_fused(const F8Desc& m, int64_t pairs);
hipError_t launch_f8_linear_id(const F8Desc& m, const void* x, int xt, int64_t pairs, int slots, const int32_t* ids,
                               void* y, int yt, hipStream_t s);
// Weight gradients: dw[M][K] = g^T x over N tokens, both quantized along the tokens (codes_c layout); with a plan
// dw[E][M][K], each expert over its own pairs.
struct F8WgradArgs {
  const uint8_t* gc;
  const float* gs;
  const uint8_t* xc;
  const float* xs;
  int64_t M, K, Np;
  void* dw;
  int dt;
  const int32_t* plan;
  PlanDesc pd;
  int cus;
  void* ws;  // dense: f8_wgrad_workspace_bytes
};
size_t f8_wgrad_workspace_bytes(int64_t Np, int64_t M, int64_t K, int cus);
hipError_t launch_f8_wgrad(const F8WgradArgs& a, hipStream_t s);

// Router.
struct RouteArgs {
  const void* logits;
  int lt;
  int64_t N;
  int E, S, normalise;
  float coef;
  const uint8_t* valid;  // null: every row
  int32_t* ids;
  float* weights;
  int32_t* counts;  // [E + 1]: tokens per expert, then rows with an expert
  float* psum;      // [E]
  float* loss;      // null: none
  void* ws;
};
size_t route_workspace_bytes(int64_t N, int64_t E);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_balance_loss(const int32_t* counts, const float* psum, int E, int S, float coef, float* loss,
                               hipStream_t s);
struct RouteBackwardArgs {
  const void* logits;
  int lt;
  int64_t N;
  int E, S, normalise;
  float coef;
  const uint8_t* valid;
  const int32_t* ids;
  const float* dweights;  // null: none
  const int32_t* counts;
  const float* dloss;     // null: none
  void* dlogits;
};
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s);
// out[t] = sum_s w[t][s] y[t][s] (w null: plain sum)
hipError_t launch_route_combine(const void* y, int yt, const void* w, int wt, int64_t N, int S, int64_t M, void* out,
                                hipStream_t s);
hipError_t launch_route_combine_backward(const void* y, int yt, const void* w, int wt, int64_t N, int S, int64_t M,
                                         const void* dout, void* dy, void* dw, hipStream_t s);

// A launch has fewer than 2^32 threads along x: one with more ends without an error and leaves outputs as they were (with
// 2^32 exactly it is refused).  Grid of `blocks` workgroups, numbered by block_index(), in `many` layers along z, those
// past 2^31 threads along y.  Workgroups from `blocks` on have nothing to do.
inline dim3 long_grid(int64_t blocks, int threads = 256, int64_t many = 1) {
  const int64_t most = (int64_t(1) << 31) / threads, x = blocks < most ? blocks : most;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x), static_cast<unsigned>(many));
}
inline bool fits_grid(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

#ifdef __HIPCC__
__device__ __forceinline__ int64_t block_index() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

// ---- device helpers ----------------------------------------------------------------------------

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int DT> struct Elem;
template <> struct Elem<DT_F32> { typedef float T; };
template <> struct Elem<DT_F16> { typedef _Float16 T; };
template <> struct Elem<DT_BF16> { typedef __bf16 T; };

// 8 consecutive elements as fp32.  p is aligned to its elements only: vector loads of this GPU take any address, and a
// 16-byte aligned one costs the same through either form.
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* p, float* v) {
  typedef typename Elem<DT>::T T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef T8 T8u __attribute__((aligned(sizeof(T))));
  const T8 a = *reinterpret_cast<const T8u*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(a[i]);
}
// Columns c .. c + 7 of a row of K as they are, zeros from K on.  Nothing is computed from them in the branches, where the
// wave would wait for the load before it issues the next.
template <int DT> struct Raw8 {
  typedef typename Elem<DT>::T T;
  typedef T V __attribute__((ext_vector_type(8)));
  V v;
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t K) {
    typedef V Vu __attribute__((aligned(sizeof(T))));
    if (c + 8 <= K) {
      v = *reinterpret_cast<const Vu*>(row + c);
    } else {
      T t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = row[c + i < K ? c + i : K - 1];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < K ? t[i] : static_cast<T>(0.0f);
    }
  }
  __device__ __forceinline__ void widen(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(v[i]);
  }
};
template <int DT>
__device__ __forceinline__ void load_row8(const typename Elem<DT>::T* row, int64_t c, int64_t K, float* v) {
  Raw8<DT> r;
  r.load(row, c, K);
  r.widen(v);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale of a block whose largest |x| has these bits: max(a / 448, 2^-80), NaN if the block holds an Inf or a NaN.
__device__ __forceinline__ float f8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  // a / 448 correctly rounded: the product with the rounded inverse, corrected once by the exact remainder
  const float a = __uint_as_float(amax_bits), c = 1.0f / kF8Max, r = a * c;
  return fmaxf(fmaf(fmaf(-kF8Max, r, a), c, r), kF8MinScale);
}
// 1 / s to one step of fp32 (s is normal, and so is its inverse)
__device__ __forceinline__ float f8_inverse(float s) { return __builtin_amdgcn_rcpf(s); }

// x / s ready for the hardware's one rounding to e4m3 (rs = f8_inverse(s)), in two forms.  Rounding the rounded quotient
// would round twice and miss the definition wherever it lands on the middle of two codes.
//
// 16-bit values: 448 x / amax often is a middle, where the rounding of the scale decides.  x * rs, within 2 steps of fp32,
// tells between which two codes the quotient lies, or beside the code that both it and the quotient round to; the sign of
// x - middle * s, which one fma gives exactly, tells on which side of their middle.  What is returned is the middle or
// 2^-12 beside it, less than the way to either code.  Codes of |q| >= 2^-6 have 3 bits behind the leading one, so the
// middle has the low 20 bits 0x80000; smaller ones are 2^-9 apart, as from 2^-6 to 2^-5, and take that way in waves that
// hold any.
__device__ __forceinline__ float f8_middle(float q) { return __uint_as_float((__float_as_uint(q) & 0xFFF00000u) | 0x80000u); }
__device__ __forceinline__ float f8_beside(float middle, float x, float s) {
  const float side = fmaf(-middle, s, x) * 0x1p125f;  // a multiple of 2^-133, so 0 or more than 2^-12
  return middle + __builtin_amdgcn_fmed3f(side, -0x1p-12f, 0x1p-12f);
}

// 32-bit values: q is the neighbour of x / s in fp32 (one correction of x * rs by the exact remainder); an inexact q takes
// the odd one of the two fp32 neighbours of the quotient, which an e4m3 rounding (4 of 24 bits) cannot tell from the
// quotient itself.
__device__ __forceinline__ float f8_quotient(float x, float s, float rs) {
  float q = x * rs;
  q = fmaf(fmaf(-q, s, x), rs, q);
  const float r = fmaf(-q, s, x);
  const uint32_t b = __float_as_uint(q);
  const uint32_t below = (__float_as_uint(r) ^ b) >> 31;  // 1: the quotient is nearer to zero than q
  const uint32_t odd = r == 0.0f ? b : (b - below) | 1u;
  return __uint_as_float((odd & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));  // the correction loses a -0
}

// Eight quotients at once.  32-bit values: x * rs is within 2 steps of fp32 of x / s; its e4m3 rounding can only differ from
// the quotient's next to a middle, and only a wave that holds a value within 4 steps of one, or a smaller one than 2^-6,
// takes the exact form: 5 operations a value, not 12.  The form for 16-bit values has 7 and no such branch: 4096 x 4096 in
// bf16 both ways 22.5 -> 20.6 us, where 777 x 515 in fp32 would go from 7.8 to 10.2.
template <int DT>
__device__ __forceinline__ void f8_quotients(const float* x, const float* s, const float* rs, float* q) {
  if constexpr (DT == DT_F32) {
    uint32_t off = ~0u, small = ~0u;  // distance from the nearest middle, plus 4 steps; the least |q| but 0, which is exact
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = x[i] * rs[i];
      off = min(off, (__float_as_uint(q[i]) + (4 - 0x80000)) & 0xFFFFFu);
      small = min(small, (__float_as_uint(q[i]) << 1) - 1u);
    }
    // (a NaN scale leaves q NaN either way)
    if (off <= 8u || small < (0x3C800000u << 1) - 1u) {  // 2^-6
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = f8_quotient(x[i], s[i], rs[i]);
    }
  } else {
    float a[8], least = INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = x[i] * rs[i];
      least = fminf(least, fabsf(a[i]));
      q[i] = f8_beside(f8_middle(a[i]), x[i], s[i]);
    }
    if (least < 0x1p-6f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float up = __builtin_copysignf(0x1p-6f, x[i]), most = __builtin_copysignf(0x1.fffffep-6f, x[i]);
        const float t = a[i] + up, m = f8_middle(fabsf(t) < 0x1p-5f ? t : most) - up;
        q[i] = fabsf(a[i]) < 0x1p-6f ? f8_beside(m, x[i], s[i]) : q[i];
      }
    }
  }
}

// four codes in one word, lowest byte first
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

template <int DT>
__device__ __forceinline__ typename Elem<DT>::T to_elem(float v) { return static_cast<typename Elem<DT>::T>(v); }
#endif

}  // namespace qmm
