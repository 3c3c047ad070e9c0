// f8_few.hip -- e4m3 products of few tokens, bound by reading the weights once.
//
// A workgroup owns up to 16 weight rows and divides K among its waves (wave v takes groups v, v + KS, ..): a wave loads
// its groups' codes straight into the registers of the matrix instruction (16 rows x 128 bytes, whole cache lines),
// keeps its partial outputs, and the workgroup adds the waves' partials in wave order through LDS.  Nothing but the
// partials and, for raw tokens, the tokens' codes passes through LDS.  Two batches of groups are in flight per wave.
// One token of 4096 x 2560 takes 3.6 us (10.5 MB, an empty launch 1.5), of 2560 x 9728 8.1 (25 MB).  The expert form: 32
// pairs of 128 experts of 4096 x 512 13.6 us for 62 MB.
#include <algorithm>

#include "f8.hpp"
#include "f8_mma.hpp"

namespace qmm {

namespace {

constexpr int kBatch = 4;
constexpr int kFusedLds = 48 << 10;  // token codes a workgroup quantizes for itself

__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x124, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x122, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x121, 0xF, 0xF, false)));
  return v;
}

// A team of 16 lanes quantizes one (row, group) of a token into LDS: codes [g][row][128], 16-byte pieces xored with
// bits 1..3 of the row (two rows fill the 64 banks, so 16 lanes that read one piece of 16 rows use every bank once),
// scales [g][row].
template <int XT>
__device__ __forceinline__ void load_group(const typename Elem<XT>::T* row, int g, int64_t K, Raw8<XT>& r) {
  r.load(row, static_cast<int64_t>(g) * kF8Block + (threadIdx.x & 15) * 8, K);
}
template <int XT>
__device__ __forceinline__ void store_group(const Raw8<XT>& r, int w, int t, uint8_t* codes, float* scales) {
  const int lane = threadIdx.x & 15;
  float v[8];
  r.widen(v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  const float s = f8_scale(max16(m)), rs = f8_inverse(s);
  float q[8], ss[8], rr[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { ss[i] = s; rr[i] = rs; }
  f8_quotients<XT>(v, ss, rr, q);
  *reinterpret_cast<uint2*>(codes + static_cast<size_t>(w) * 128 + (((lane >> 1) ^ (t >> 1 & 7)) * 16) + (lane & 1) * 8) =
      make_uint2(f8_pack4(q[0], q[1], q[2], q[3]), f8_pack4(q[4], q[5], q[6], q[7]));
  if (lane == 0) scales[w] = s;
}
// the two pieces of a row that quarter q of the lanes multiplies
__device__ __forceinline__ void read_codes(const uint8_t* p, int t, int q, i32x4& lo, i32x4& hi) {
  lo = *reinterpret_cast<const i32x4*>(p + 16 * ((2 * q) ^ (t >> 1 & 7)));
  hi = *reinterpret_cast<const i32x4*>(p + 16 * ((2 * q + 1) ^ (t >> 1 & 7)));
}

struct FewArgs {
  const uint8_t* w;
  const float* ws;
  const void* x;      // raw tokens (RAW) or codes [N][Kp]
  const float* xs;    // [G][N] (not RAW)
  void* y;
  int64_t M, K, Kp, ldx;
  int N, G, waves, vec_y;
  int rows;           // of a workgroup, 4 .. 16
};

// RAW: element type of raw tokens, -1 for quantized ones.  B: groups of a batch.  W: most waves of a workgroup (128
// registers a lane at 16, 256 at 8).
template <int NT, int RAW, int OT, int B, int W>
__global__ __launch_bounds__(64 * W) void k_f8_few(FewArgs a) {
  extern __shared__ __align__(16) uint8_t sh[];
  constexpr bool kExact = OT == DT_F32;
  constexpr int kTokens = RAW >= 0 ? 1 : NT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row = lane & 15, q = lane >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int KS = a.waves, last = a.G - 1;

  // raw tokens first: everything waits for them, and loads return in order
  constexpr int kItems = 4;
  typedef typename Elem<RAW < 0 ? 0 : RAW>::T X;
  Raw8<RAW < 0 ? 0 : RAW> v[RAW >= 0 ? kItems : 1];
  const int items = a.N * a.G, teams = KS * 4, team = threadIdx.x >> 4;
  if constexpr (RAW >= 0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int w = std::min(team + i * teams, items - 1), g = w / a.N;
      if (i * teams < items) load_group<RAW>(static_cast<const X*>(a.x) + (w - g * a.N) * a.ldx, g, a.K, v[i]);
    }
  }

  const int64_t rl = std::min<int64_t>(r0 + a.rows, a.M) - 1;  // the last row; it may lie in another row block's scales
  const uint8_t* wrow = a.w + std::min<int64_t>(r0 + row, rl) * a.Kp + q * 32;
  const float *wsc = a.ws + r0 / 128 * a.G, *wsc2 = a.ws + rl / 128 * a.G;
  const int upto = static_cast<int>(rl / 128 * 128 - r0) - q * 4;  // this lane's outputs from here on have the second
  const uint8_t* trow[kTokens];
  const float* tsc[kTokens];
  if constexpr (RAW < 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = std::min(j * 16 + row, a.N - 1);
      trow[j] = static_cast<const uint8_t*>(a.x) + t * a.Kp + q * 32;
      tsc[j] = a.xs + t;
    }
  }
  // A group past the last is the last one again, its part multiplied by zero (what is NaN there is NaN anyway).
  struct Batch {
    i32x4 lo[B], hi[B], tlo[B][kTokens], thi[B][kTokens];
    float sw[B], sw2[B], sx[B][kTokens];
  } b0, b1;
  auto load = [&](Batch& b, int i0) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const int64_t g = std::min(i0 + u * KS, last);
      b.lo[u] = *reinterpret_cast<const i32x4*>(wrow + g * 128);
      b.hi[u] = *reinterpret_cast<const i32x4*>(wrow + g * 128 + 16);
      b.sw[u] = wsc[g];
      b.sw2[u] = wsc2[g];
      if constexpr (RAW < 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          b.tlo[u][j] = *reinterpret_cast<const i32x4*>(trow[j] + g * 128);
          b.thi[u][j] = *reinterpret_cast<const i32x4*>(trow[j] + g * 128 + 16);
          b.sx[u][j] = tsc[j][g * a.N];
        }
      }
    }
  };
  load(b0, wave);
  if (wave + B * KS <= last) load(b1, wave + B * KS);

  uint8_t* codes = sh;
  float* scales = reinterpret_cast<float*>(sh + static_cast<size_t>(a.N) * a.Kp);
  if constexpr (RAW >= 0) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int w = team + i * teams;
      if (w < items) store_group<RAW>(v[i], w, w % a.N, codes, scales);
    }
    for (int w = team + kItems * teams; w < items; w += teams) {
      const int g = w / a.N;
      load_group<RAW>(static_cast<const X*>(a.x) + (w - g * a.N) * a.ldx, g, a.K, v[0]);
      store_group<RAW>(v[0], w, w - g * a.N, codes, scales);
    }
    __syncthreads();
  }

  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Batch& b, int i0) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      const bool real = i0 + u * KS <= last;
      const float sw = real ? b.sw[u] : 0.0f, sw2 = real ? b.sw2[u] : 0.0f;
      Frag<kExact> A;
      A.set(b.lo[u], b.hi[u]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Frag<kExact> T;
        float s;
        if constexpr (RAW >= 0) {
          const int g = std::min(i0 + u * KS, last), t = std::min(row, a.N - 1);
          i32x4 lo, hi;
          read_codes(codes + (static_cast<size_t>(g) * a.N + t) * 128, t, q, lo, hi);
          T.set(lo, hi);
          s = scales[g * a.N + t];
        } else {
          T.set(b.tlo[u][j], b.thi[u][j]);
          s = b.sx[u][j];
        }
        const f32x4 p = group_sum(A, T);
        const float2 o1 = scale_order(s, sw), o2 = scale_order(s, sw2);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(p[e] * (e < upto ? o1.x : o2.x), e < upto ? o1.y : o2.y, acc[j][e]);
      }
    }
  };
  for (int i0 = wave; i0 <= last; i0 += 2 * B * KS) {
    multiply(b0, i0);
    if (i0 + 2 * B * KS <= last) load(b0, i0 + 2 * B * KS);
    if (i0 + B * KS <= last) multiply(b1, i0 + B * KS);
    if (i0 + 3 * B * KS <= last) load(b1, i0 + 3 * B * KS);
  }

  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(sh);  // [wave][NT][lane]
#pragma unroll
  for (int j = 0; j < NT; ++j) part[(wave * NT + j) * 64 + lane] = acc[j];
  __syncthreads();
  typedef typename Elem<OT>::T T;
  for (int j = wave; j < NT; j += KS) {
    f32x4 sum = part[j * 64 + lane];
    for (int k = 1; k < KS; ++k) sum += part[(k * NT + j) * 64 + lane];
    const int t = j * 16 + row;
    const int64_t r = r0 + q * 4, left = rl + 1 - r;
    if (t < a.N && left > 0)
      store4<OT>(static_cast<T*>(a.y) + static_cast<int64_t>(t) * a.M + r, sum, left < 4 ? static_cast<int>(left) : 4, a.vec_y);
  }
}

// ---- experts -------------------------------------------------------------------------------------

constexpr int kIdThreads = 256;
constexpr int kIdPairs = 256;     // pairs of a fused call: one a thread
constexpr int kIdRows = 64;       // rows of a workgroup, 16 a wave

struct FewIdArgs {
  const uint8_t* w;
  const float* ws;
  const void* x;
  const int32_t* ids;
  void* y;
  int64_t M, K, Kp;
  int E, pairs, slots, G, vec_y;
};

// grid (row slices, distinct experts at most): workgroup (s, j) finds the j-th distinct expert among the ids (in order of
// first appearance) and its pairs, quantizes their tokens 16 at a time and multiplies its rows by them.  Slice s of j = 0
// also fills the rows of empty slots and of ids that name no expert.
template <int XT, int OT>
__global__ __launch_bounds__(kIdThreads) void k_f8_few_id(FewIdArgs a) {
  extern __shared__ __align__(16) uint8_t sh[];
  __shared__ int32_t first[kRouteMaxExperts];
  __shared__ int32_t mine[kIdPairs];
  __shared__ int32_t before[4], expert;
  typedef typename Elem<XT>::T T;
  typedef typename Elem<OT>::T O;
  constexpr bool kExact = OT == DT_F32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, row = lane & 15, q = lane >> 4;
  const int64_t s0 = static_cast<int64_t>(blockIdx.x) * kIdRows;
  O* y = static_cast<O*>(a.y);

  const int id = tid < a.pairs ? a.ids[tid] : -1;
  const bool real = tid < a.pairs && id >= 0 && id < a.E;
  for (int e = tid; e < a.E; e += kIdThreads) first[e] = kIdPairs;
  if (tid == 0) expert = -1;
  __syncthreads();
  if (real) atomicMin(&first[id], tid);
  __syncthreads();
  const bool lead = real && first[id] == tid;
  const uint64_t leads = __ballot(lead);
  if (lane == 0) before[wave] = __popcll(leads);
  __syncthreads();
  int rank = __popcll(leads & ((1ull << lane) - 1));
  for (int k = 0; k < wave; ++k) rank += before[k];
  if (lead && rank == static_cast<int>(blockIdx.y)) expert = id;
  __syncthreads();
  if (blockIdx.y == 0) {
    const int rows = static_cast<int>(std::min<int64_t>(kIdRows, a.M - s0));
    for (int p = wave; p < a.pairs; p += kIdThreads / 64) {
      const int other = a.ids[p];
      if (other >= 0 && other < a.E) continue;
      const float v = other == -1 ? 0.0f : __uint_as_float(0x7FC00000u);
      if (lane < rows) y[static_cast<int64_t>(p) * a.M + s0 + lane] = to_elem<OT>(v);
    }
  }
  const int e = expert;
  if (e < 0) return;  // fewer distinct experts than workgroups
  const bool own = real && id == e;
  const uint64_t owns = __ballot(own);
  if (lane == 0) before[wave] = __popcll(owns);
  __syncthreads();
  int at = __popcll(owns & ((1ull << lane) - 1)), all = 0;
  for (int k = 0; k < 4; ++k) {
    if (k < wave) at += before[k];
    all += before[k];
  }
  if (own) mine[at] = tid;

  const int64_t r0 = s0 + wave * 16;
  const uint8_t* wrow = a.w + (static_cast<int64_t>(e) * a.M + std::min<int64_t>(r0 + row, a.M - 1)) * a.Kp + q * 32;
  const float* wsc = a.ws + (static_cast<int64_t>(e) * ((a.M + 127) / 128) + std::min<int64_t>(r0, a.M - 1) / 128) * a.G;
  const int last = a.G - 1;
  i32x4 lo[kBatch], hi[kBatch];
  auto load = [&](int g0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t g = std::min(g0 + u, last);
      lo[u] = *reinterpret_cast<const i32x4*>(wrow + g * 128);
      hi[u] = *reinterpret_cast<const i32x4*>(wrow + g * 128 + 16);
    }
  };
  load(0);
  __syncthreads();

  float* scales = reinterpret_cast<float*>(sh + 16 * a.Kp);
  for (int p0 = 0; p0 < all; p0 += 16) {
    const int n = std::min(16, all - p0);
    if (p0) {
      load(0);
      __syncthreads();  // the codes of the pass before are read
    }
    const T* x = static_cast<const T*>(a.x);
    for (int w = tid >> 4; w < n * a.G; w += kIdThreads / 16) {
      const int g = w / n, u = w - g * n;
      Raw8<XT> v;
      load_group<XT>(x + static_cast<int64_t>(mine[p0 + u] / a.slots) * a.K, g, a.K, v);
      store_group<XT>(v, w, u, sh, scales);
    }
    __syncthreads();
    const int t = std::min(row, n - 1);
    f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
    for (int g0 = 0; g0 <= last; g0 += kBatch) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int g = std::min(g0 + u, last);
        const float sw = g0 + u <= last ? wsc[g] : 0.0f;
        const uint8_t* p = sh + (g * n + t) * 128;
        Frag<kExact> A, B;
        i32x4 tlo, thi;
        read_codes(p, t, q, tlo, thi);
        A.set(lo[u], hi[u]);
        B.set(tlo, thi);
        const f32x4 v = group_sum(A, B);
        const float2 s = scale_order(scales[g * n + t], sw);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(v[i] * s.x, s.y, acc[i]);
      }
      if (g0 + kBatch <= last) load(g0 + kBatch);
    }
    const int64_t r = r0 + q * 4, left = a.M - r;
    if (row < n && left > 0)
      store4<OT>(y + static_cast<int64_t>(mine[p0 + row]) * a.M + r, acc, left < 4 ? static_cast<int>(left) : 4, a.vec_y);
  }
}

template <int NT, int RAW, int OT, int B, int W>
hipError_t few_run(FewArgs a, hipStream_t st) {
  a.waves = std::min(W, (a.G + 1) / 2);
  const int64_t blocks = (a.M + a.rows - 1) / a.rows;
  const size_t codes = RAW >= 0 ? static_cast<size_t>(a.N) * (a.Kp + a.G * 4) : 0;
  const size_t lds = std::max(codes, static_cast<size_t>(a.waves) * NT * 1024);
  k_f8_few<NT, RAW, OT, B, W><<<static_cast<unsigned>(blocks), 64 * a.waves, lds, st>>>(a);
  return hipGetLastError();
}

template <int RAW, int OT>
hipError_t few_tokens(const FewArgs& a, hipStream_t st) {
  // Batches no longer than two of them need to cover a wave's groups: a load past the last group is a wasted one (20
  // groups, 4096 rows, one token: 3.6 us with 16 waves and batches of 2, 4.0 with 8 waves, 4.4 and 5.3 with batches of 4
  // and 6).  Rows of quantized tokens too long for two batches of 16 waves take 8 waves with 10 groups in flight each
  // (2560 x 9728, 16 tokens: 11.9 us against 12.9).
  if constexpr (RAW >= 0) {
    return a.G <= 64 ? few_run<1, RAW, OT, 2, 16>(a, st) : few_run<1, RAW, OT, 3, 16>(a, st);
  } else {
    if (a.N > 16) return few_run<2, RAW, OT, 2, 8>(a, st);
    return a.G <= 64 ? few_run<1, RAW, OT, 2, 16>(a, st) : few_run<1, RAW, OT, 5, 8>(a, st);
  }
}

template <int RAW>
hipError_t few_out(const FewArgs& a, int yt, hipStream_t st) {
  switch (yt) {
    case DT_F32: return few_tokens<RAW, DT_F32>(a, st);
    case DT_F16: return few_tokens<RAW, DT_F16>(a, st);
    case DT_BF16: return few_tokens<RAW, DT_BF16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

FewArgs few_args(const F8Desc& m, int64_t N, void* y, int yt) {
  FewArgs a{};
  a.w = m.codes;
  a.ws = m.scales;
  a.y = y;
  a.M = m.M;
  a.K = m.K;
  a.Kp = m.Kp;
  a.N = static_cast<int>(N);
  a.G = static_cast<int>(m.Kp / kF8Block);
  // Fewer than 16 rows where 16 would leave CUs idle (2560 x 9728, 1 and 16 tokens: 8.9 and 12.2 us with 16 rows, 8.1 and
  // 11.2 with 10; 512 x 4096: 4.9 and 6.3, 4.4 and 5.7 with 4).
  a.rows = static_cast<int>(std::min<int64_t>(16, std::max<int64_t>(4, (m.M + m.cus - 1) / m.cus)));
  a.vec_y = a.rows % 4 == 0 && store_vec(y, m.M, yt);
  return a;
}

template <int XT>
hipError_t few_id_out(const FewIdArgs& a, int yt, dim3 grid, size_t lds, hipStream_t st) {
  switch (yt) {
    case DT_F32: k_f8_few_id<XT, DT_F32><<<grid, kIdThreads, lds, st>>>(a); break;
    case DT_F16: k_f8_few_id<XT, DT_F16><<<grid, kIdThreads, lds, st>>>(a); break;
    case DT_BF16: k_f8_few_id<XT, DT_BF16><<<grid, kIdThreads, lds, st>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

// Above 16 tokens a workgroup's 8 waves fill a CU's registers, so that more than one workgroup a CU makes another round, and
// long rows outlast the tiled kernel that divides K: 17 and 32 tokens of 4096 x 2560 take 5.9 and 6.9 us here and 7.8 in
// tiles, of 5120 x 2560 9.4 and 11.4 against 7.9 and 9.1, of 1280 x 9728 13.4 and 17.0 against 11.7.  Above 32 tokens
// (4096 x 2560, 64: 9.9 us) the tiles read them less often.
bool f8_few_tokens(const F8Desc& m, int64_t N) { return N <= 16 || (N <= 32 && m.M <= 16 * m.cus && m.Kp <= 4096); }

hipError_t launch_f8_few(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t N, void* y, int yt, hipStream_t st) {
  FewArgs a = few_args(m, N, y, yt);
  a.x = xc;
  a.xs = xs;
  return few_out<-1>(a, yt, st);
}

bool f8_linear_fused(const F8Desc& m, int64_t N) {
  return N <= 16 && N * (m.Kp + m.Kp / kF8Block * 4) <= 16384;
}

hipError_t launch_f8_linear(const F8Desc& m, const void* x, int xt, int64_t ldx, int64_t N, void* y, int yt,
                            hipStream_t st) {
  FewArgs a = few_args(m, N, y, yt);
  a.x = x;
  a.ldx = ldx;
  switch (xt) {
    case DT_F32: return few_out<DT_F32>(a, yt, st);
    case DT_F16: return few_out<DT_F16>(a, yt, st);
    case DT_BF16: return few_out<DT_BF16>(a, yt, st);
    default: return hipErrorInvalidValue;
  }
}

bool f8_linear_id_fused(const F8Desc& m, int64_t pairs) {
  return pairs <= kIdPairs && 16 * (m.Kp + m.Kp / kF8Block * 4) <= kFusedLds;
}

hipError_t launch_f8_linear_id(const F8Desc& m, const void* x, int xt, int64_t pairs, int slots, const int32_t* ids, void* y,
                               int yt, hipStream_t st) {
  FewIdArgs a{};
  a.w = m.codes;
  a.ws = m.scales;
  a.x = x;
  a.ids = ids;
  a.y = y;
  a.M = m.M;
  a.K = m.K;
  a.Kp = m.Kp;
  a.E = static_cast<int>(m.n_experts);
  a.pairs = static_cast<int>(pairs);
  a.slots = slots;
  a.G = static_cast<int>(m.Kp / kF8Block);
  a.vec_y = store_vec(y, m.M, yt);
  const int64_t slices = (m.M + kIdRows - 1) / kIdRows;
  const dim3 grid(static_cast<unsigned>(slices), static_cast<unsigned>(std::min<int64_t>(pairs, m.n_experts)));
  const size_t lds = 16 * static_cast<size_t>(m.Kp + a.G * 4);
  switch (xt) {
    case DT_F32: return few_id_out<DT_F32>(a, yt, grid, lds, st);
    case DT_F16: return few_id_out<DT_F16>(a, yt, grid, lds, st);
    case DT_BF16: return few_id_out<DT_BF16>(a, yt, grid, lds, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qmm
