// route.hip -- the expert router (softmax, the S largest, tokens per expert, balance loss, gradients), the plan that
// sorts (token, slot) pairs by expert for the expert-indexed products, and the weighted sum of the slots' outputs.
//
// Router: 16 lanes (one DPP row) hold a token, V experts a lane, so that a reduction over the experts is four DPP steps;
// nothing but the logits is read.  A lane's experts lie in runs of 16 bytes of logits with the other lanes' runs between:
// loads and stores of V consecutive experts a lane took 1.2 times as long at 400 experts.  Sums over tokens (probabilities
// per expert) go through one partial per workgroup, added in a fixed order: the same input gives the same bits.
#include <algorithm>

#include "f8.hpp"

namespace qmm {

namespace {

constexpr float kNegInf = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ int dpp(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false); }
template <int CTRL>
__device__ __forceinline__ float dppf(float v) { return __int_as_float(dpp<CTRL>(__float_as_int(v))); }

// reductions over the 16 lanes of a DPP row (row_ror 8, 4, 2, 1); every lane gets the result
__device__ __forceinline__ float max16f(float v) {
  v = fmaxf(v, dppf<0x128>(v));
  v = fmaxf(v, dppf<0x124>(v));
  v = fmaxf(v, dppf<0x122>(v));
  return fmaxf(v, dppf<0x121>(v));
}
__device__ __forceinline__ float sum16f(float v) {
  v += dppf<0x128>(v);
  v += dppf<0x124>(v);
  v += dppf<0x122>(v);
  return v + dppf<0x121>(v);
}

// e^x to 2 steps of fp32: 2^t with t = x log2(e) rounded, corrected by what the rounding left.  NaN stays NaN.
__device__ __forceinline__ float fast_exp(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  x = x < -150.0f ? -150.0f : x;  // 0 in fp32, and no infinity in the correction
  const float t = x * kLog2e, r = fmaf(x, kLog2eLow, fmaf(x, kLog2e, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return fmaf(y, r * kLn2, y);
}

// Logits as keys that order like (value, lower index first), with a largest and a smallest of two in one instruction
// each; kNone, below every key that can be chosen, stands for -inf and NaN.  -0 counts as +0.  16-bit logits: the value's
// bits made monotonic above the complement of the expert.
template <int LT> struct Key {
  typedef uint32_t T;
  static constexpr T kNone = 0u;
  static __device__ __forceinline__ T make(float v, int e) {
    const uint32_t b = bits(v + 0.0f), k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return v > kNegInf ? (k & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(e)) : kNone;
  }
  static __device__ __forceinline__ int expert(T key) { return static_cast<int>(0xFFFFu - (key & 0xFFFFu)); }
  static __device__ __forceinline__ float value(T key) {
    const uint32_t b = (key & 0xFFFF0000u) ^ (key & 0x80000000u ? 0x80000000u : 0xFFFF0000u);
    if constexpr (LT == DT_F16) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b >> 16)));
    else return __uint_as_float(b);
  }
  // the 16-bit logit above 16 zeros
  static __device__ __forceinline__ uint32_t bits(float v) {
    if constexpr (LT == DT_F16) return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(v))) << 16;
    else return __float_as_uint(v);
  }
  static __device__ __forceinline__ T larger(T a, T b) { return max(a, b); }
  static __device__ __forceinline__ T smaller(T a, T b) { return min(a, b); }
  template <int CTRL> static __device__ __forceinline__ T ror(T v) { return static_cast<T>(dpp<CTRL>(static_cast<int>(v))); }
};
// 32-bit logits: the value as a double, whose 29 spare bits have room for the expert.  +inf is 2^200, to stay a number.
template <> struct Key<DT_F32> {
  typedef double T;
  static constexpr T kNone = -__builtin_inf();
  static constexpr uint32_t kMask = 1023;  // experts
  static __device__ __forceinline__ T make(float v, int e) {
    const double d = fmin(static_cast<double>(v + 0.0f), 0x1p200);
    const uint64_t b = __builtin_bit_cast(uint64_t, d) | static_cast<uint32_t>(v < 0.0f ? e : kMask - e);
    return v > kNegInf ? __builtin_bit_cast(double, b) : kNone;
  }
  static __device__ __forceinline__ int expert(T key) {
    const uint32_t low = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, key)) & kMask;
    return static_cast<int>(__builtin_bit_cast(int64_t, key) < 0 ? low : kMask - low);
  }
  static __device__ __forceinline__ float value(T key) {
    return static_cast<float>(__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~static_cast<uint64_t>(kMask)));
  }
  static __device__ __forceinline__ T larger(T a, T b) { return fmax(a, b); }
  static __device__ __forceinline__ T smaller(T a, T b) { return fmin(a, b); }
  template <int CTRL> static __device__ __forceinline__ T ror(T v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp<CTRL>(static_cast<int>(b)), hi = dpp<CTRL>(static_cast<int>(b >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  }
};
static_assert(kRouteMaxExperts <= 1024, "an expert's index has 10 bits");

// Which experts a lane holds: its logit i is expert lane * kRun + offset(i), rising with i.
template <int LT, int V> struct Spread {
  static constexpr int kRun = std::min<int>(V, 16 / sizeof(typename Elem<LT>::T));
  static __device__ __forceinline__ constexpr int offset(int i) { return i / kRun * (16 * kRun) + i % kRun; }
  static __device__ __forceinline__ int expert(int lane, int i) { return lane * kRun + offset(i); }
};

// The largest logits of 16 lanes, one a call, ties to the lower expert.  next() returns the expert (-1: none is left) and
// its logit; the same in all 16 lanes.  With LIST every lane has its L = min(V, 8) largest sorted, L of them being enough
// for L calls, and a call compares the lanes' first; without, a call looks through all V.
template <int LT, int V, bool LIST> struct Chooser {
  typedef Key<LT> K;
  typedef typename K::T T;
  static constexpr int L = LIST ? std::min(V, 8) : V;
  T k[L];

  // Batcher's merge exchange: falling order
  template <int N> static __device__ __forceinline__ void exchange(T (&x)[N], int i, int j) {
    const T a = x[i], b = x[j];
    x[i] = K::larger(a, b);
    x[j] = K::smaller(a, b);
  }
  static __device__ __forceinline__ void sort(T (&x)[L]) {
#pragma unroll
    for (int p = 1; p < L; p *= 2)
#pragma unroll
      for (int q = p; q >= 1; q /= 2)
#pragma unroll
        for (int j = q % p; j < L - q; j += 2 * q)
#pragma unroll
          for (int i = 0; i < q; ++i)
            if (i + j + q < L && (i + j) / (2 * p) == (i + j + q) / (2 * p)) exchange(x, i + j, i + j + q);
  }

  __device__ __forceinline__ Chooser(const float* l, int lane) {
#pragma unroll
    for (int i = 0; i < L; ++i) k[i] = K::make(l[i], Spread<LT, V>::expert(lane, i));
    if constexpr (LIST) {
      sort(k);
#pragma unroll
      for (int g = L; g < V; g += L) {
        T more[L];
#pragma unroll
        for (int i = 0; i < L; ++i) more[i] = K::make(l[g + i], Spread<LT, V>::expert(lane, g + i));
        sort(more);
        // the L largest of both, first rising then falling; then sorted by halves
#pragma unroll
        for (int i = 0; i < L; ++i) k[i] = K::larger(k[i], more[L - 1 - i]);
#pragma unroll
        for (int h = L / 2; h >= 1; h /= 2)
#pragma unroll
          for (int i = 0; i < L; ++i)
            if (!(i & h)) exchange(k, i, i + h);
      }
    }
  }
  __device__ __forceinline__ int next(float& value) {
    T m = k[0];
    if constexpr (!LIST) {
#pragma unroll
      for (int i = 1; i < L; ++i) m = K::larger(m, k[i]);
    }
    m = K::larger(m, K::template ror<0x128>(m));
    m = K::larger(m, K::template ror<0x124>(m));
    m = K::larger(m, K::template ror<0x122>(m));
    m = K::larger(m, K::template ror<0x121>(m));
    if constexpr (LIST) {
      const bool mine = k[0] == m;
#pragma unroll
      for (int i = 0; i < L; ++i) k[i] = !mine ? k[i] : i + 1 < L ? k[i + 1] : K::kNone;
    } else {
#pragma unroll
      for (int i = 0; i < L; ++i) k[i] = k[i] == m ? K::kNone : k[i];
    }
    if (m == K::kNone) return -1;
    value = K::value(m);
    return K::expert(m);
  }
};

// LDS operations of a wave's lanes before this are done before those after it; a team lies inside a wave
__device__ __forceinline__ void in_wave() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The lane's logits of row t; experts from E on are -inf.  A row's last run is read into the next row, but where no row
// follows that has as much: there the logits are read one by one.
template <int LT, int V>
__device__ __forceinline__ void load_logits(const void* logits, int64_t N, int E, int64_t t, int lane, float* v) {
  typedef typename Elem<LT>::T T;
  typedef Spread<LT, V> Sp;
  typedef T Run __attribute__((ext_vector_type(Sp::kRun)));
  typedef Run RunU __attribute__((aligned(sizeof(T))));
  const T* row = static_cast<const T*>(logits) + t * E;
  if ((N - t) * E >= (E + Sp::kRun - 1) / Sp::kRun * Sp::kRun) {
#pragma unroll
    for (int i = 0; i < V; i += Sp::kRun) {
      const int e = Sp::expert(lane, i);
      const Run r = *reinterpret_cast<const RunU*>(row + (e < E ? e : 0));
#pragma unroll
      for (int k = 0; k < Sp::kRun; ++k) v[i + k] = static_cast<float>(r[k]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = static_cast<float>(row[std::min(Sp::expert(lane, i), E - 1)]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = Sp::expert(lane, i) < E ? v[i] : kNegInf;
}

// Threads of a workgroup: one register of every kind per expert of a lane, so many experts leave room for fewer waves.
constexpr int route_threads(int V) { return V <= 8 ? 1024 : V <= 32 ? 512 : 256; }
// Slot s lives in lane s & 15, register s >> 4: one register (SR) up to 16 slots, four up to 64.
constexpr int kRouteOneBlock = 128;   // rows that one workgroup routes and sums by itself

// Sum of v over the workgroup's threads, in a fixed order, in thread 0.  red: 16 floats of LDS.
__device__ __forceinline__ float block_sum(float v, float* red, int threads) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  if (threadIdx.x == 0)
    for (int i = 0; i < threads / 64; ++i) s += red[i];
  return s;
}

// Expert e's part of sum_e f_e P_e times T, f_e = E counts_e / (S T).
__device__ __forceinline__ float loss_part(int count, float psum, float T, int E, int S) {
  return T > 0.0f ? static_cast<float>(count) * E / (S * T) * psum : 0.0f;
}

// 16384 x 128 in bf16, S = 8: 7.0 us, 4 MB read; bound by vector operations (keys, sorting, exponentials: some 400 a wave
// of four tokens) and the latency of one pass.  12000 x 400: 14.8 us in bf16, 18.4 in fp32.
//
// part, part_n: the workgroups' sums over their rows, [E] and [E + 1] each.  A single workgroup writes the results itself.
template <int LT, int V, int SR, bool LIST>
__global__ __launch_bounds__(route_threads(V)) void k_route(RouteArgs a, float* part, int32_t* part_n) {
  constexpr int kRouteThreads = route_threads(V), kRouteTeams = kRouteThreads / 16;
  extern __shared__ int32_t sh[];  // [E + 1] counts, then [waves][16 * V] probability sums
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4, E = static_cast<int>(a.E);
  float* shp = reinterpret_cast<float*>(sh + a.E + 1);
  for (int i = threadIdx.x; i <= a.E; i += kRouteThreads) sh[i] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteTeams;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTeams + team; t < a.N; t += step) {
    float l[V];
    load_logits<LT, V>(a.logits, a.N, E, t, lane, l);
    if (a.valid && !a.valid[t]) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = kNegInf;
    }
    Chooser<LT, V, LIST> choose(l, lane);
    float top = kNegInf, chosen[SR];
    int ids[SR];
#pragma unroll
    for (int k = 0; k < SR; ++k) { chosen[k] = kNegInf; ids[k] = -1; }
    for (int s = 0; s < a.S; ++s) {
      float m = kNegInf;
      const int e = choose.next(m);
      if (s == 0 && e >= 0) top = m;
#pragma unroll
      for (int k = 0; k < SR; ++k)
        if (s == k * 16 + lane) { chosen[k] = m; ids[k] = e; }
    }
    const bool alive = top > kNegInf;
    if (!alive) {
      top = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = kNegInf;
    }
    float z = 0.0f, p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = fast_exp(l[i] - top);
      z += p[i];
    }
    z = sum16f(z);
    const float rz = alive ? 1.0f / z : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] = fmaf(p[i], rz, psum[i]);
    float total = 0.0f, w[SR];
#pragma unroll
    for (int k = 0; k < SR; ++k) {
      w[k] = ids[k] >= 0 ? fast_exp(chosen[k] - top) : 0.0f;
      total += w[k];
    }
    total = a.normalise ? sum16f(total) : z;
    // a NaN among the logits makes the row's probabilities NaN, normalised or not
    if (!(z == z)) total = z;
#pragma unroll
    for (int k = 0; k < SR; ++k) {
      const int s = k * 16 + lane;
      if (s < a.S) {
        a.ids[t * a.S + s] = ids[k];
        a.weights[t * a.S + s] = ids[k] >= 0 ? w[k] / total : 0.0f;
        if (ids[k] >= 0) atomicAdd(&sh[ids[k]], 1);
      }
    }
    if (lane == 0 && alive) atomicAdd(&sh[a.E], 1);
  }
  // the wave's four tokens, then the waves
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] += __shfl_xor(psum[i], 16);
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] += __shfl_xor(psum[i], 32);
  if ((team & 3) == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) shp[(team >> 2) * (16 * V) + Spread<LT, V>::expert(lane, i)] = psum[i];
  }
  __syncthreads();
  if (gridDim.x == 1) {
    __shared__ float red[16];
    const float T = static_cast<float>(sh[a.E]);
    float v = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kRouteTeams / 4; ++k) s += shp[k * (16 * V) + e];
      a.psum[e] = s;
      a.counts[e] = sh[e];
      v += loss_part(sh[e], s, T, a.E, a.S);
    }
    if (threadIdx.x == 0) a.counts[a.E] = sh[a.E];
    if (a.loss) {
      v = block_sum(v, red, kRouteThreads);
      if (threadIdx.x == 0) *a.loss = T > 0.0f ? a.coef * v / T : 0.0f;
    }
    return;
  }
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kRouteTeams / 4; ++k) s += shp[k * (16 * V) + e];
    part[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
  }
  for (int i = threadIdx.x; i <= a.E; i += kRouteThreads) part_n[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + i] = sh[i];
}

constexpr int kSumCols = 32, kSumSegs = 32;

// Adds the workgroups' partials: a workgroup takes 32 experts, a thread every 32nd partial of one, and the threads' sums
// are added in order.  The loss, which needs all of them, is a launch of its own: one workgroup for everything waited 17
// us for 256 partials of 128 experts, and a last workgroup that knows itself by a counter 14 us, most of it the fence
// that makes the other dies' sums visible.  This way it is 3.1 us and 1.6.
__global__ __launch_bounds__(kSumCols * kSumSegs) void k_route_sum(const float* part, const int32_t* part_n, int blocks,
                                                                   int E, int32_t* counts, float* psum) {
  __shared__ float sp[kSumSegs][kSumCols + 1];
  __shared__ int32_t sn[kSumSegs][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, seg = threadIdx.x / kSumCols, e = blockIdx.x * kSumCols + col, E1 = E + 1;
  float s = 0.0f;
  int n = 0;
  const float* p = part + std::min(e, E - 1);  // no branch, so that the loads do not wait for each other
  const int32_t* pn = part_n + std::min(e, E);
#pragma unroll 8
  for (int b = seg; b < blocks; b += kSumSegs) {
    s += p[static_cast<int64_t>(b) * E];
    n += pn[static_cast<int64_t>(b) * E1];
  }
  sp[seg][col] = s;
  sn[seg][col] = n;
  __syncthreads();
  if (seg == 0 && e < E1) {
    for (int k = 1; k < kSumSegs; ++k) {
      s += sp[k][col];
      n += sn[k][col];
    }
    counts[e] = n;
    if (e < E) psum[e] = s;
  }
}

__global__ __launch_bounds__(1024) void k_route_none(RouteArgs a) {
  for (int e = threadIdx.x; e <= a.E; e += 1024) {
    a.counts[e] = 0;
    if (e < a.E) a.psum[e] = 0.0f;
  }
  if (a.loss && threadIdx.x == 0) *a.loss = 0.0f;
}

__global__ __launch_bounds__(1024) void k_balance_loss(const int32_t* counts, const float* psum, int E, int S, float coef,
                                                       float* loss) {
  __shared__ float red[16];
  const float T = static_cast<float>(counts[E]);
  float v = 0.0f;
  for (int e = threadIdx.x; e < E; e += 1024) v += loss_part(counts[e], psum[e], T, E, S);
  v = block_sum(v, red, 1024);
  if (threadIdx.x == 0) *loss = T > 0.0f ? coef * v / T : 0.0f;
}

// tokens of a workgroup: their rows of LDS stay under 64 KB
constexpr int route_backward_teams(int V) { return V <= 32 ? 16 : 8; }

// dl = p (dp - sum p dp), dp_e = dloss coef f_e / T + the chosen slots' gradients; p again from the logits.  The slots'
// gradients reach the lanes that hold their experts through a row of LDS that holds the loss's part between tokens.
// 16384 x 128 in bf16 5.7 us for 8.4 MB: vector operations and the latency of one pass.  Three waves a SIMD for 257 .. 512
// experts: 12000 x 400 in bf16 14.0 -> 12.5 us; fp32 has more to spill, 15.0 -> 16.0.
template <int LT, int V, int SR>
__global__ __launch_bounds__(16 * route_backward_teams(V), LT != DT_F32 && V == 32 ? 3 : 1)
void k_route_backward(RouteBackwardArgs a) {
  constexpr int kRouteTeams = route_backward_teams(V);
  typedef typename Elem<LT>::T T;
  typedef Spread<LT, V> Sp;
  __shared__ __align__(16) float balance[16 * V], given[kRouteTeams][16 * V];
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4, E = static_cast<int>(a.E);
  float* mine = given[team];
  {
    const float n = a.dloss ? static_cast<float>(a.counts[E]) : 0.0f;
    const float k = n > 0.0f ? a.dloss[0] * a.coef / n * (E / (a.S * n)) : 0.0f;
    for (int e = threadIdx.x; e < 16 * V; e += 16 * kRouteTeams)
      balance[e] = k != 0.0f ? k * static_cast<float>(a.counts[std::min(e, E)]) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i * 16 + lane] = balance[i * 16 + lane];
    in_wave();
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteTeams;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTeams + team; t < a.N; t += step) {
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    T* out = static_cast<T*>(a.dlogits) + t * a.E;
    float l[V], p[V], dp[V];
    load_logits<LT, V>(a.logits, a.N, E, t, lane, l);
    float w[SR], d[SR];
    int id[SR];
#pragma unroll
    for (int k = 0; k < SR; ++k) {
      const int s = k * 16 + lane;
      const bool some = a.dweights && s < a.S;
      id[k] = some ? a.ids[t * a.S + s] : -1;
      d[k] = some ? a.dweights[t * a.S + s] : 0.0f;
      if (id[k] < 0 || id[k] >= a.E) { id[k] = -1; d[k] = 0.0f; }
    }
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);  // fmaxf passes over a NaN
    top = max16f(top);
    const bool alive = top > kNegInf && !(a.valid && !a.valid[t]);
    if (!alive) {
      top = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = kNegInf;
    }
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = fast_exp(l[i] - top);
      z += p[i];
    }
    z = sum16f(z);
    const float rz = alive ? 1.0f / z : 0.0f;
    if (a.dweights && alive) {
      float total = 0.0f, dot = 0.0f;
#pragma unroll
      for (int k = 0; k < SR; ++k) {
        w[k] = id[k] >= 0 ? fast_exp(static_cast<float>(row[id[k]]) - top) : 0.0f;
        total += w[k];
        dot = fmaf(w[k], d[k], dot);
      }
      if (a.normalise) {
        total = sum16f(total);
        dot = sum16f(dot) / total;
        const float f = z / total;
#pragma unroll
        for (int k = 0; k < SR; ++k) d[k] = (d[k] - dot) * f;
      }
#pragma unroll
      for (int k = 0; k < SR; ++k)
        if (id[k] >= 0) atomicAdd(&mine[id[k]], d[k]);
      in_wave();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = alive ? mine[Sp::expert(lane, i)] : 0.0f;
    in_wave();
#pragma unroll
    for (int k = 0; k < SR; ++k)
      if (id[k] >= 0) mine[id[k]] = balance[id[k]];
    in_wave();
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= rz;
      dot = fmaf(p[i], dp[i], dot);
    }
    dot = sum16f(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = p[i] * (dp[i] - dot);
    typedef T Run __attribute__((ext_vector_type(Sp::kRun)));
    typedef Run RunU __attribute__((aligned(sizeof(T))));
#pragma unroll
    for (int i = 0; i < V; i += Sp::kRun) {
      const int e = Sp::expert(lane, i);
      Run o;
#pragma unroll
      for (int k = 0; k < Sp::kRun; ++k) o[k] = to_elem<LT>(dp[i + k]);
      if (e + Sp::kRun <= E) {
        *reinterpret_cast<RunU*>(out + e) = o;
      } else {
#pragma unroll
        for (int k = 0; k < Sp::kRun; ++k)
          if (e + k < E) out[e + k] = o[k];
      }
    }
  }
}

// ---- plan ---------------------------------------------------------------------------------------

__device__ __forceinline__ int bucket_of(int id, int E) { return id >= 0 && id < E ? id : id == -1 ? E : E + 1; }

constexpr int kPlanThreads = 1024;
constexpr int kPlanBlocks = 256;
constexpr int64_t kPlanOneLaunch = 32768;
constexpr int kMaxBuckets = static_cast<int>(kRouteMaxExperts) + 2;

// pairs per workgroup of the counting and scattering kernels, a multiple of 1024
__host__ __device__ inline int64_t plan_chunk(int64_t pairs) {
  const int64_t per = (pairs + kPlanBlocks - 1) / kPlanBlocks;
  return (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

// What the plan's kernels hold in LDS.
struct PlanShared {
  int32_t offs[kMaxBuckets + 1], cnt[kMaxBuckets], tiles[kPlanTileKinds][kMaxBuckets + 1];
  int32_t base[kMaxBuckets];
  int32_t wsum[kPlanTileKinds + 1][kPlanThreads / 64];
  int32_t part[kPlanThreads];
  uint16_t in_wave[kPlanThreads / 64][kMaxBuckets];
};

// counts of the pairs p0 .. p1 - 1 per bucket, in hist
__device__ void plan_count(const int32_t* ids, int64_t p0, int64_t p1, int E, int32_t* hist) {
  for (int b = threadIdx.x; b < E + 2; b += kPlanThreads) hist[b] = 0;
  __syncthreads();
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kPlanThreads) atomicAdd(&hist[bucket_of(ids[p], E)], 1);
  __syncthreads();
}

// From cnt: the buckets' first pairs (offs) and first tiles of each kind (tiles), exclusive prefix sums with the total
// behind; two buckets a thread, all five sums in one pass.
__device__ void plan_prefix(PlanShared& sh, int B) {
  constexpr int A = kPlanTileKinds + 1;
  const int i = 2 * threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = i < B ? sh.cnt[i] : 0, c1 = i + 1 < B ? sh.cnt[i + 1] : 0;
  int x[A], s[A];
#pragma unroll
  for (int k = 0; k < A; ++k) {
    const int T = k < kPlanTileKinds ? kPlanTiles[k] : 1;
    x[k] = (c0 + T - 1) / T;
    s[k] = x[k] + (c1 + T - 1) / T;
  }
  int incl[A];
#pragma unroll
  for (int k = 0; k < A; ++k) incl[k] = s[k];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
#pragma unroll
    for (int k = 0; k < A; ++k) {
      const int u = __shfl_up(incl[k], o);
      if (lane >= o) incl[k] += u;
    }
  }
  if (lane == 63)
#pragma unroll
    for (int k = 0; k < A; ++k) sh.wsum[k][wave] = incl[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < A; ++k) {
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) {
      if (w < wave) before += sh.wsum[k][w];
      all += sh.wsum[k][w];
    }
    const int ex = before + incl[k] - s[k];
    int32_t* out = k < kPlanTileKinds ? sh.tiles[k] : sh.offs;
    if (i < B) out[i] = ex;
    if (i + 1 < B) out[i + 1] = ex + x[k];
    if (threadIdx.x == 0) out[B] = all;
  }
  __syncthreads();
}

// The tiles' lists: half of the workgroup's threads to the smallest tiles, which are as many as the others together, a
// quarter to each of those; the workgroups in turn.
__device__ void plan_tiles(const PlanShared& sh, const PlanDesc& d, int32_t* plan) {
  constexpr int kQuarter = kPlanThreads / 4;
  const int B = static_cast<int>(d.E) + 2, quarter = threadIdx.x / kQuarter, t = std::max(quarter - 1, 0);
  const int T = kPlanTiles[0] << t, each = t == 0 ? 2 * kQuarter : kQuarter, at = threadIdx.x % each;
  int64_t cap = 0, map = 0;
#pragma unroll
  for (int k = 0; k < kPlanTileKinds; ++k)
    if (k == t) { cap = d.cap[k]; map = d.map[k]; }
  const int32_t* tiles = sh.tiles[t];
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * each + at; i < cap; i += static_cast<int64_t>(gridDim.x) * each) {
    int32_t* m = plan + map + 3 * i;
    if (i >= tiles[B]) {
      m[0] = -1;
      m[1] = 0;
      m[2] = 0;
      continue;
    }
    int lo = 0, hi = B - 1;  // the last bucket whose first tile is at or before i: the one that has it
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tiles[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    m[0] = lo;
    m[1] = sh.offs[lo] + (static_cast<int>(i) - tiles[lo]) * T;
    m[2] = sh.offs[lo + 1];
  }
}
static_assert(kPlanTileKinds == 3 && kPlanTiles[1] == 2 * kPlanTiles[0] && kPlanTiles[2] == 4 * kPlanTiles[0],
              "each kind of tile is twice the one before");

// Pairs p0 .. p1 - 1 to their places, in order inside a bucket: base, then the waves in order, then lanes.
__device__ void plan_scatter(const int32_t* ids, int64_t p0, int64_t p1, int E, int32_t* order, PlanShared& sh) {
  const int B = E + 2, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int b = threadIdx.x; b < B; b += kPlanThreads)
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) sh.in_wave[w][b] = 0;
  __syncthreads();
  for (int64_t q = p0; q < p1; q += kPlanThreads) {
    const int64_t p = q + threadIdx.x;
    const bool here = p < p1;
    const int b = here ? bucket_of(ids[p], E) : kMaxBuckets;
    uint64_t same = __ballot(here);
#pragma unroll
    for (int i = 0; i < 11; ++i) {
      const uint64_t set = __ballot((b >> i) & 1);
      same &= (b >> i) & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (here && rank == 0) sh.in_wave[wave][b] = static_cast<uint16_t>(__popcll(same));
    __syncthreads();
    if (here) {
      int at = sh.base[b] + rank;
      for (int w = 0; w < wave; ++w) at += sh.in_wave[w][b];
      order[at] = static_cast<int32_t>(p);
    }
    if (q + kPlanThreads >= p1) break;
    __syncthreads();
    for (int i = threadIdx.x; i < B; i += kPlanThreads) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kPlanThreads / 64; ++w) {
        n += sh.in_wave[w][i];
        sh.in_wave[w][i] = 0;
      }
      sh.base[i] += n;
    }
    __syncthreads();
  }
}

// Up to kPlanOneLaunch pairs: every workgroup counts all of them, those before its own kPlanThreads apart.  128 experts:
// 8.6 us for 16384 pairs and 10.5 for 32768, where three launches took 19 and 19; at 131072, where these take 18.6, it
// took 2 us more than they.
__global__ __launch_bounds__(kPlanThreads) void k_plan_small(const int32_t* ids, PlanDesc d, int32_t* plan) {
  __shared__ PlanShared sh;
  const int E = static_cast<int>(d.E), B = E + 2, pairs = static_cast<int>(d.pairs);
  const int p0 = blockIdx.x * kPlanThreads;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) sh.base[b] = sh.cnt[b] = 0;
  __syncthreads();
  constexpr int kEach = 8;  // loads that do not wait for each other
  for (int p = threadIdx.x; p < pairs; p += kEach * kPlanThreads) {
    int id[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) id[i] = ids[std::min(p + i * kPlanThreads, pairs - 1)];
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (p + i * kPlanThreads < pairs) atomicAdd((p + i * kPlanThreads < p0 ? sh.base : sh.cnt) + bucket_of(id[i], E), 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kPlanThreads) sh.cnt[b] += sh.base[b];
  __syncthreads();
  plan_prefix(sh, B);
  for (int b = threadIdx.x; b < B; b += kPlanThreads) sh.base[b] += sh.offs[b];
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= B; b += kPlanThreads) {
      if (b < B) plan[d.counts + b] = sh.cnt[b];
      plan[d.offsets + b] = sh.offs[b];
      plan[d.tile128 + b] = sh.tiles[kPlanTileKinds - 1][b];
    }
    if (threadIdx.x < kPlanTileKinds) plan[d.totals + threadIdx.x] = sh.tiles[threadIdx.x][B];
  }
  plan_tiles(sh, d, plan);
  plan_scatter(ids, p0, std::min(p0 + kPlanThreads, pairs), E, plan + d.order, sh);
}

// More: counts per chunk; their prefixes, by one workgroup; places and lists.
__global__ __launch_bounds__(kPlanThreads) void k_plan_count(const int32_t* ids, PlanDesc d, int32_t* plan) {
  __shared__ int32_t hist[kMaxBuckets];
  const int E = static_cast<int>(d.E), B = E + 2;
  const int64_t chunk = plan_chunk(d.pairs), p0 = blockIdx.x * chunk;
  plan_count(ids, p0, std::min(p0 + chunk, d.pairs), E, hist);
  for (int b = threadIdx.x; b < B; b += kPlanThreads) plan[d.scratch + static_cast<int64_t>(blockIdx.x) * B + b] = hist[b];
}

// Turns the chunks' counts into their exclusive prefixes, bucket by bucket.  Threads (segment, bucket) hold runs of the
// chunks; the loads of a run do not wait for each other.
__global__ __launch_bounds__(kPlanThreads) void k_plan_scan(PlanDesc d, int32_t* plan, int blocks) {
  __shared__ PlanShared sh;
  const int B = static_cast<int>(d.E) + 2, wide = std::min(B, kPlanThreads);
  const int segs = std::max(1, kPlanThreads / B), per = (blocks + segs - 1) / segs;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x) % wide, seg = threadIdx.x / wide;
    const bool mine = b < B && seg < segs;
    const int k0 = seg * per, k1 = std::min(blocks, k0 + per);
    int32_t* h = plan + d.scratch + b;
    int n = 0;
    if (mine)
#pragma unroll 8
      for (int k = k0; k < k1; ++k) n += h[static_cast<int64_t>(k) * B];
    sh.part[threadIdx.x] = n;
    __syncthreads();
    if (mine) {
      int before = 0;
      for (int s = 0; s < seg; ++s) before += sh.part[s * wide + static_cast<int>(threadIdx.x) % wide];
      if (seg == segs - 1) sh.cnt[b] = plan[d.counts + b] = before + n;
#pragma unroll 8
      for (int k = k0; k < k1; ++k) {
        const int c = h[static_cast<int64_t>(k) * B];
        h[static_cast<int64_t>(k) * B] = before;
        before += c;
      }
    }
    __syncthreads();
  }
  plan_prefix(sh, B);
  for (int b = threadIdx.x; b <= B; b += kPlanThreads) {
    plan[d.offsets + b] = sh.offs[b];
    plan[d.tile128 + b] = sh.tiles[kPlanTileKinds - 1][b];
  }
  if (threadIdx.x < kPlanTileKinds) plan[d.totals + threadIdx.x] = sh.tiles[threadIdx.x][B];
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_scatter(const int32_t* ids, PlanDesc d, int32_t* plan) {
  __shared__ PlanShared sh;
  const int E = static_cast<int>(d.E), B = E + 2;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) {
    sh.cnt[b] = plan[d.counts + b];
    sh.base[b] = plan[d.offsets + b] + plan[d.scratch + static_cast<int64_t>(blockIdx.x) * B + b];
  }
  __syncthreads();
  plan_prefix(sh, B);
  plan_tiles(sh, d, plan);
  const int64_t chunk = plan_chunk(d.pairs), p0 = blockIdx.x * chunk;
  plan_scatter(ids, p0, std::min(p0 + chunk, d.pairs), E, plan + d.order, sh);
}

// ---- weighted sum of the slots ------------------------------------------------------------------

// WT: type of the weights, -1 for none (a plain sum).  8 columns a thread.  A slot of weight 0 is left out whatever its row
// holds: an empty slot's row is NaN where the block formats made it.  Bound by memory: 2048 x 8 x 4096 in bf16 22.8 us, 6.6
// TB/s.
template <int YT, int WT, bool VEC>
__global__ __launch_bounds__(256) void k_combine(const typename Elem<YT>::T* y, const void* w, int64_t N, int S, int64_t M,
                                                 typename Elem<YT>::T* out) {
  typedef typename Elem<YT>::T T;
  const int64_t cols = (M + 7) / 8, i = block_index() * 256 + threadIdx.x;
  if (i >= N * cols) return;
  const int64_t t = i / cols, c = i % cols * 8;
  float o[8] = {};
  for (int s = 0; s < S; ++s) {
    float v[8], k = 1.0f;
    const T* row = y + (t * S + s) * M + c;
    if (VEC) {
      load8<YT>(row, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < M ? static_cast<float>(row[e]) : 0.0f;
    }
    if constexpr (WT >= 0) k = static_cast<float>(static_cast<const typename Elem<WT < 0 ? 0 : WT>::T*>(w)[t * S + s]);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = fmaf(k, k == 0.0f ? 0.0f : v[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (VEC || c + e < M) out[t * M + c + e] = to_elem<YT>(o[e]);
}

// One token a workgroup, its slots dealt to the waves: dy = w dout (one rounding to fp32, one to the type), dw = <y, dout>.
// Bound by memory: 2048 x 8 x 4096 in bf16 54 us, 5.3 TB/s.
template <int YT, int WT, bool VEC>
__global__ __launch_bounds__(256) void k_combine_backward(const typename Elem<YT>::T* y, const typename Elem<WT>::T* w, int64_t N,
                                                          int S, int64_t M, const typename Elem<YT>::T* dout,
                                                          typename Elem<YT>::T* dy, typename Elem<WT>::T* dw) {
  const int64_t t = block_index();
  if (t >= N) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int s = wave; s < S; s += 4) {
    const float k = static_cast<float>(w[t * S + s]);
    const int64_t row = (t * S + s) * M;
    float dot = 0.0f;
    for (int64_t c = lane * 8; c < M; c += 512) {
      float g[8], v[8];
      if (VEC) {
        load8<YT>(dout + t * M + c, g);
        load8<YT>(y + row + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          g[e] = c + e < M ? static_cast<float>(dout[t * M + c + e]) : 0.0f;
          v[e] = c + e < M ? static_cast<float>(y[row + c + e]) : 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dot = fmaf(v[e], g[e], dot);
        if (VEC || c + e < M) dy[row + c + e] = to_elem<YT>(k * g[e]);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
    if (lane == 0) dw[t * S + s] = to_elem<WT>(dot);
  }
}

int lanes_values(int64_t E) {
  int v = 1;
  while (v * 16 < E) v *= 2;
  return v;
}

// workgroups of the router: each leaves one partial
int route_blocks(int64_t N, int64_t E) {
  const int teams = route_threads(lanes_values(E)) / 16;
  return N <= kRouteOneBlock ? 1 : static_cast<int>(std::min<int64_t>((N + teams - 1) / teams, 256));
}

template <int LT, int V>
hipError_t launch_v(const RouteArgs& a, hipStream_t st) {
  if (a.N == 0) {
    k_route_none<<<1, 1024, 0, st>>>(a);
    return hipGetLastError();
  }
  const int nb = route_blocks(a.N, a.E);
  float* part = static_cast<float*>(a.ws);
  int32_t* part_n = reinterpret_cast<int32_t*>(part + static_cast<int64_t>(nb) * a.E);
  constexpr int kThreads = route_threads(V);
  const size_t lds = (a.E + 1) * 4 + static_cast<size_t>(kThreads / 64) * 16 * V * 4;
  // Sorting pays from 4 calls on: 12000 x 400 in bf16 with S = 1, 4 and 8 12.8, 13.8 and 14.8 us with lists, 11.7, 13.8 and
  // 20.7 without; in fp32 14.6 and 18.4 against 12.9 and 26 with S = 1 and 8.
  if (V <= 8 || (a.S >= 4 && a.S <= 8)) {
    if (a.S <= 16) k_route<LT, V, 1, true><<<nb, kThreads, lds, st>>>(a, part, part_n);
    else k_route<LT, V, 4, V <= 8><<<nb, kThreads, lds, st>>>(a, part, part_n);
  } else {
    if (a.S <= 16) k_route<LT, V, 1, V <= 8><<<nb, kThreads, lds, st>>>(a, part, part_n);
    else k_route<LT, V, 4, V <= 8><<<nb, kThreads, lds, st>>>(a, part, part_n);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || nb == 1) return e;
  k_route_sum<<<(a.E + kSumCols) / kSumCols, kSumCols * kSumSegs, 0, st>>>(part, part_n, nb, a.E, a.counts, a.psum);
  const hipError_t es = hipGetLastError();
  if (es != hipSuccess || !a.loss) return es;
  return launch_balance_loss(a.counts, a.psum, a.E, a.S, a.coef, a.loss, st);
}

template <int LT, int V>
hipError_t launch_v(const RouteBackwardArgs& a, hipStream_t st) {
  constexpr int kTeams = route_backward_teams(V);
  const int nb = static_cast<int>(std::min<int64_t>((a.N + kTeams - 1) / kTeams, 2048));
  if (a.S <= 16) k_route_backward<LT, V, 1><<<nb, 16 * kTeams, 0, st>>>(a);
  else k_route_backward<LT, V, 4><<<nb, 16 * kTeams, 0, st>>>(a);
  return hipGetLastError();
}

template <int LT, class A>
hipError_t dispatch_v(const A& a, hipStream_t st) {
  switch (lanes_values(a.E)) {
    case 1: return launch_v<LT, 1>(a, st);
    case 2: return launch_v<LT, 2>(a, st);
    case 4: return launch_v<LT, 4>(a, st);
    case 8: return launch_v<LT, 8>(a, st);
    case 16: return launch_v<LT, 16>(a, st);
    case 32: return launch_v<LT, 32>(a, st);
    case 64: return launch_v<LT, 64>(a, st);
    default: return hipErrorInvalidValue;
  }
}

template <class A>
hipError_t dispatch(const A& a, hipStream_t st) {
  switch (a.lt) {
    case DT_F32: return dispatch_v<DT_F32>(a, st);
    case DT_F16: return dispatch_v<DT_F16>(a, st);
    case DT_BF16: return dispatch_v<DT_BF16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

template <int YT, int WT>
hipError_t combine_t(const void* y, const void* w, int64_t N, int S, int64_t M, void* out, hipStream_t st) {
  typedef typename Elem<YT>::T T;
  const int esz = YT == DT_F32 ? 4 : 2;
  const bool vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && M % 8 == 0 && (M * esz) % 16 == 0;
  const dim3 g = long_grid((N * ((M + 7) / 8) + 255) / 256);
  if (vec) k_combine<YT, WT, true><<<g, 256, 0, st>>>(static_cast<const T*>(y), w, N, S, M, static_cast<T*>(out));
  else k_combine<YT, WT, false><<<g, 256, 0, st>>>(static_cast<const T*>(y), w, N, S, M, static_cast<T*>(out));
  return hipGetLastError();
}

template <int YT, int WT>
hipError_t combine_backward_t(const void* y, const void* w, int64_t N, int S, int64_t M, const void* dout, void* dy, void* dw,
                              hipStream_t st) {
  typedef typename Elem<YT>::T T;
  typedef typename Elem<WT>::T W;
  const bool vec = (reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(dout)) % 16 == 0 && M % 8 == 0;
  if (vec)
    k_combine_backward<YT, WT, true><<<long_grid(N), 256, 0, st>>>(
        static_cast<const T*>(y), static_cast<const W*>(w), N, S, M, static_cast<const T*>(dout), static_cast<T*>(dy),
        static_cast<W*>(dw));
  else
    k_combine_backward<YT, WT, false><<<long_grid(N), 256, 0, st>>>(
        static_cast<const T*>(y), static_cast<const W*>(w), N, S, M, static_cast<const T*>(dout), static_cast<T*>(dy),
        static_cast<W*>(dw));
  return hipGetLastError();
}

}  // namespace

PlanDesc plan_desc(int64_t pairs, int64_t E) {
  PlanDesc d{};
  d.pairs = pairs;
  d.E = E;
  const int64_t B = E + 2;
  d.counts = 0;
  d.offsets = d.counts + B;
  d.tile128 = d.offsets + B + 1;
  d.totals = d.tile128 + B + 1;
  d.order = d.totals + kPlanTileKinds;
  int64_t at = d.order + pairs;
  for (int t = 0; t < kPlanTileKinds; ++t) {
    d.map[t] = at;
    // every bucket with pairs adds at most one part-filled tile
    d.cap[t] = pairs / kPlanTiles[t] + std::min(B, pairs);
    at += 3 * d.cap[t];
  }
  d.scratch = at;
  const int64_t blocks = pairs > kPlanOneLaunch ? (pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs) : 0;
  d.total = at + blocks * B;
  return d;
}

hipError_t launch_route_plan(const int32_t* ids, int64_t pairs, int64_t E, int32_t* plan, hipStream_t st) {
  const PlanDesc d = plan_desc(pairs, E);
  if (pairs <= kPlanOneLaunch) {
    const int blocks = static_cast<int>(std::max<int64_t>(1, (pairs + kPlanThreads - 1) / kPlanThreads));
    k_plan_small<<<blocks, kPlanThreads, 0, st>>>(ids, d, plan);
    return hipGetLastError();
  }
  const int blocks = static_cast<int>((pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs));
  k_plan_count<<<blocks, kPlanThreads, 0, st>>>(ids, d, plan);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_plan_scan<<<1, kPlanThreads, 0, st>>>(d, plan, blocks);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_plan_scatter<<<blocks, kPlanThreads, 0, st>>>(ids, d, plan);
  return hipGetLastError();
}

size_t route_workspace_bytes(int64_t N, int64_t E) {
  const int nb = N > 0 ? route_blocks(N, E) : 0;
  return nb > 1 ? static_cast<size_t>(nb) * static_cast<size_t>(2 * E + 1) * 4 : 0;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t st) { return dispatch(a, st); }
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t st) { return dispatch(a, st); }

hipError_t launch_balance_loss(const int32_t* counts, const float* psum, int E, int S, float coef, float* loss,
                               hipStream_t st) {
  k_balance_loss<<<1, 1024, 0, st>>>(counts, psum, E, S, coef, loss);
  return hipGetLastError();
}

hipError_t launch_route_combine(const void* y, int yt, const void* w, int wt, int64_t N, int S, int64_t M, void* out,
                                hipStream_t st) {
  if (yt == DT_F32) return w ? combine_t<DT_F32, DT_F32>(y, w, N, S, M, out, st) : combine_t<DT_F32, -1>(y, w, N, S, M, out, st);
  if (yt == DT_F16) {
    if (!w) return combine_t<DT_F16, -1>(y, w, N, S, M, out, st);
    return wt == DT_F32 ? combine_t<DT_F16, DT_F32>(y, w, N, S, M, out, st) : combine_t<DT_F16, DT_F16>(y, w, N, S, M, out, st);
  }
  if (!w) return combine_t<DT_BF16, -1>(y, w, N, S, M, out, st);
  return wt == DT_F32 ? combine_t<DT_BF16, DT_F32>(y, w, N, S, M, out, st) : combine_t<DT_BF16, DT_BF16>(y, w, N, S, M, out, st);
}

hipError_t launch_route_combine_backward(const void* y, int yt, const void* w, int wt, int64_t N, int S, int64_t M,
                                         const void* dout, void* dy, void* dw, hipStream_t st) {
  if (yt == DT_F32) return combine_backward_t<DT_F32, DT_F32>(y, w, N, S, M, dout, dy, dw, st);
  if (yt == DT_F16)
    return wt == DT_F32 ? combine_backward_t<DT_F16, DT_F32>(y, w, N, S, M, dout, dy, dw, st)
                        : combine_backward_t<DT_F16, DT_F16>(y, w, N, S, M, dout, dy, dw, st);
  return wt == DT_F32 ? combine_backward_t<DT_BF16, DT_F32>(y, w, N, S, M, dout, dy, dw, st)
                      : combine_backward_t<DT_BF16, DT_BF16>(y, w, N, S, M, dout, dy, dw, st);
}

}  // namespace qmm
