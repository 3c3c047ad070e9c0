// route.hip -- the expert router (softmax, the S largest, tokens per expert, balance loss, gradients), the plan that
// sorts (token, slot) pairs by expert for the expert-indexed products, and the weighted sum of the slots' outputs.
//
// Router: 16 lanes (one DPP row) hold a token, V consecutive experts a lane, so that a reduction over the experts is
// four DPP steps; nothing but the logits is read.  Sums over tokens (probabilities per expert) go through one partial
// per workgroup, added in a fixed order: the same input gives the same bits.
#include <algorithm>
#include <climits>

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
__device__ __forceinline__ int min16i(int v) {
  v = min(v, dpp<0x128>(v));
  v = min(v, dpp<0x124>(v));
  v = min(v, dpp<0x122>(v));
  return min(v, dpp<0x121>(v));
}
__device__ __forceinline__ float sum16f(float v) {
  v += dppf<0x128>(v);
  v += dppf<0x124>(v);
  v += dppf<0x122>(v);
  return v + dppf<0x121>(v);
}

// V logits of this lane from expert lane * V on; experts from E on are -inf
template <int LT, int V>
__device__ __forceinline__ void load_logits(const typename Elem<LT>::T* row, int lane, int E, float* v) {
  if (V >= 8 && lane * V + V <= E) {
#pragma unroll
    for (int i = 0; i < V; i += 8) load8<LT>(row + lane * V + i, v + i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lane * V + i < E ? static_cast<float>(row[lane * V + i]) : kNegInf;
  }
}

constexpr int kRouteThreads = 256;
constexpr int kRouteTeams = kRouteThreads / 16;
constexpr int kMaxSlotRegs = 4;  // slot s lives in lane s & 15, register s >> 4

template <int LT, int V>
__global__ __launch_bounds__(kRouteThreads) void k_route(RouteArgs a, float* part, int32_t* part_n) {
  extern __shared__ int32_t sh[];  // [E + 1] counts, then [waves][16 * V] probability sums
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  float* shp = reinterpret_cast<float*>(sh + a.E + 1);
  for (int i = threadIdx.x; i <= a.E; i += kRouteThreads) sh[i] = 0;
  __syncthreads();
  float psum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) psum[i] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteTeams;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTeams + team; t < a.N; t += step) {
    float v[V], l[V];
    load_logits<LT, V>(static_cast<const typename Elem<LT>::T*>(a.logits) + t * a.E, lane, a.E, l);
    if (a.valid && !a.valid[t]) {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = kNegInf;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = l[i] == l[i] ? l[i] : kNegInf;  // a NaN is never chosen
    float top = 0.0f, chosen[kMaxSlotRegs];
    int ids[kMaxSlotRegs];
#pragma unroll
    for (int k = 0; k < kMaxSlotRegs; ++k) { chosen[k] = kNegInf; ids[k] = -1; }
    for (int s = 0; s < a.S; ++s) {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
      m = max16f(m);
      if (s == 0) top = m;
      int at = INT_MAX;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = v[i] == m ? lane * V + i : at;
      at = min16i(at);
      const bool some = m > kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = lane * V + i == at ? kNegInf : v[i];
#pragma unroll
      for (int k = 0; k < kMaxSlotRegs; ++k)
        if (s == k * 16 + lane && some) { chosen[k] = m; ids[k] = at; }
    }
    const bool alive = top > kNegInf;
    float z = 0.0f, p[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = alive ? expf(l[i] - top) : 0.0f;
      z += p[i];
    }
    z = sum16f(z);
    const float rz = alive ? 1.0f / z : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) psum[i] = fmaf(p[i], rz, psum[i]);
    float total = 0.0f, w[kMaxSlotRegs];
#pragma unroll
    for (int k = 0; k < kMaxSlotRegs; ++k) {
      w[k] = ids[k] >= 0 ? expf(chosen[k] - top) : 0.0f;
      total += w[k];
    }
    total = a.normalise ? sum16f(total) : z;
    // a NaN among the logits makes the row's probabilities NaN, normalised or not
    if (!(z == z)) total = z;
#pragma unroll
    for (int k = 0; k < kMaxSlotRegs; ++k) {
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
  for (int i = 0; i < V; ++i) {
    psum[i] += __shfl_xor(psum[i], 16);
    psum[i] += __shfl_xor(psum[i], 32);
    if ((team & 3) == 0) shp[(team >> 2) * (16 * V) + lane * V + i] = psum[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kRouteTeams / 4; ++k) s += shp[k * (16 * V) + e];
    part[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
  }
  for (int i = threadIdx.x; i <= a.E; i += kRouteThreads) part_n[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + i] = sh[i];
}

// loss = coef * sum_e f_e P_e, f_e = E counts_e / (S T), P_e = psum_e / T; 0 when no row has an expert.
// Every thread of a 1024-thread workgroup calls it; red: 16 floats of LDS.
__device__ void balance_loss(const int32_t* counts, const float* psum, int E, int S, float coef, float* loss, float* red) {
  const float T = static_cast<float>(counts[E]);
  float v = 0.0f;
  for (int e = threadIdx.x; e < E; e += 1024)
    v += T > 0.0f ? static_cast<float>(counts[e]) * E / (S * T) * psum[e] : 0.0f;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < 16; ++i) s += red[i];
    *loss = T > 0.0f ? coef * s / T : 0.0f;
  }
}

// Adds the workgroups' partials: thread (segment, expert) adds a run of them, the segments' sums are added in order.
__global__ __launch_bounds__(1024) void k_route_sum(const float* part, const int32_t* part_n, int blocks, RouteArgs a) {
  __shared__ float sp[1024];
  __shared__ int32_t sn[1024];
  __shared__ float psum[kRouteMaxExperts];
  __shared__ int32_t counts[kRouteMaxExperts + 1];
  __shared__ float red[16];
  const int E1 = a.E + 1;
  int segs = 1024 / E1;
  if (segs < 1) segs = 1;
  const int per = (blocks + segs - 1) / segs;
  for (int e0 = 0; e0 < E1; e0 += 1024) {
    const int e = e0 + static_cast<int>(threadIdx.x) % (E1 < 1024 ? E1 : 1024), seg = E1 < 1024 ? threadIdx.x / E1 : 0;
    float s = 0.0f;
    int n = 0;
    if (e < E1 && seg < segs) {
      const int end = min(blocks, (seg + 1) * per);
#pragma unroll 8
      for (int b = seg * per; b < end; ++b) {
        if (e < a.E) s += part[static_cast<int64_t>(b) * a.E + e];
        n += part_n[static_cast<int64_t>(b) * E1 + e];
      }
    }
    sp[threadIdx.x] = s;
    sn[threadIdx.x] = n;
    __syncthreads();
    if (e < E1 && seg == 0) {
      for (int k = 1; k < segs; ++k) {
        s += sp[k * E1 + e];
        n += sn[k * E1 + e];
      }
      a.counts[e] = n;
      counts[e] = n;
      if (e < a.E) {
        a.psum[e] = s;
        psum[e] = s;
      }
    }
    __syncthreads();
  }
  if (a.loss) balance_loss(counts, psum, a.E, a.S, a.coef, a.loss, red);
}

__global__ __launch_bounds__(1024) void k_balance_loss(const int32_t* counts, const float* psum, int E, int S, float coef,
                                                       float* loss) {
  __shared__ float red[16];
  balance_loss(counts, psum, E, S, coef, loss, red);
}

// dl = p (dp - sum p dp), dp_e = dloss coef f_e / T + the chosen slots' gradients; p again from the logits.
template <int LT, int V>
__global__ __launch_bounds__(kRouteThreads) void k_route_backward(RouteBackwardArgs a) {
  typedef typename Elem<LT>::T T;
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
  float c[V];
  {
    const float n = a.dloss ? static_cast<float>(a.counts[a.E]) : 0.0f;
    const float k = n > 0.0f ? a.dloss[0] * a.coef / n : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      c[i] = n > 0.0f && e < a.E ? k * (static_cast<float>(a.counts[e]) * a.E / (a.S * n)) : 0.0f;
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteTeams;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteTeams + team; t < a.N; t += step) {
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    T* out = static_cast<T*>(a.dlogits) + t * a.E;
    float l[V], p[V], dp[V];
    load_logits<LT, V>(row, lane, a.E, l);
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);  // fmaxf passes over a NaN
    top = max16f(top);
    const bool alive = top > kNegInf && !(a.valid && !a.valid[t]);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = alive ? expf(l[i] - top) : 0.0f;
      z += p[i];
      dp[i] = c[i];
    }
    z = sum16f(z);
    const float rz = alive ? 1.0f / z : 0.0f;
    if (a.dweights && alive) {
      float w[kMaxSlotRegs], d[kMaxSlotRegs], total = 0.0f, dot = 0.0f;
      int id[kMaxSlotRegs];
#pragma unroll
      for (int k = 0; k < kMaxSlotRegs; ++k) {
        const int s = k * 16 + lane;
        id[k] = s < a.S ? a.ids[t * a.S + s] : -1;
        const bool some = id[k] >= 0 && id[k] < a.E;
        w[k] = some ? expf(static_cast<float>(row[id[k]]) - top) : 0.0f;
        d[k] = some ? a.dweights[t * a.S + s] : 0.0f;
        total += w[k];
        dot = fmaf(w[k], d[k], dot);
      }
      if (a.normalise) {
        total = sum16f(total);
        dot = sum16f(dot) / total;
        const float f = z / total;
#pragma unroll
        for (int k = 0; k < kMaxSlotRegs; ++k) d[k] = (d[k] - dot) * f;
      }
      for (int s = 0; s < a.S; ++s) {
        int e = -1;
        float ds = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxSlotRegs; ++k)
          if (s >> 4 == k) { e = id[k]; ds = d[k]; }
        e = __shfl(e, s & 15, 16);
        ds = __shfl(ds, s & 15, 16);
#pragma unroll
        for (int i = 0; i < V; ++i) dp[i] += lane * V + i == e ? ds : 0.0f;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= rz;
      dot = fmaf(p[i], dp[i], dot);
    }
    dot = sum16f(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = p[i] * (dp[i] - dot);
    if (V >= 8 && lane * V + V <= a.E) {
#pragma unroll
      for (int i = 0; i < V; i += 8) {
        typedef T T8 __attribute__((ext_vector_type(8)));
        typedef T8 T8u __attribute__((aligned(sizeof(T))));
        T8 o;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = to_elem<LT>(dp[i + k]);
        *reinterpret_cast<T8u*>(out + lane * V + i) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i < a.E) out[lane * V + i] = to_elem<LT>(dp[i]);
    }
  }
}

// ---- plan ---------------------------------------------------------------------------------------

__device__ __forceinline__ int bucket_of(int id, int E) { return id >= 0 && id < E ? id : id == -1 ? E : E + 1; }

constexpr int kPlanThreads = 1024;
constexpr int kPlanBlocks = 256;
constexpr int kMaxBuckets = static_cast<int>(kRouteMaxExperts) + 2;

// pairs per workgroup of the counting and scattering kernels, a multiple of 1024
__host__ __device__ inline int64_t plan_chunk(int64_t pairs) {
  const int64_t per = (pairs + kPlanBlocks - 1) / kPlanBlocks;
  return (per + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_count(const int32_t* ids, PlanDesc d, int32_t* plan) {
  __shared__ int32_t hist[kMaxBuckets];
  const int E = static_cast<int>(d.E), B = E + 2;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) hist[b] = 0;
  __syncthreads();
  const int64_t chunk = plan_chunk(d.pairs), p0 = blockIdx.x * chunk, p1 = std::min(p0 + chunk, d.pairs);
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kPlanThreads) atomicAdd(&hist[bucket_of(ids[p], E)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kPlanThreads) plan[d.scratch + static_cast<int64_t>(blockIdx.x) * B + b] = hist[b];
}

// exclusive prefix sums of n <= 2 * 1024 values in LDS, v[n] the total (n + 1 <= 2048 + 1 entries); every thread calls
__device__ void scan(int32_t* v, int n, int32_t* wsum) {
  const int i = 2 * threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int x = i < n ? v[i] : 0, y = i + 1 < n ? v[i + 1] : 0;
  int s = x + y;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kPlanThreads / 64; ++k) {
    if (k < wave) before += wsum[k];
    all += wsum[k];
  }
  const int ex = before + s - x - y;
  if (i < n) v[i] = ex;
  if (i + 1 < n) v[i + 1] = ex + x;
  if (threadIdx.x == 0) v[n] = all;
  __syncthreads();
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_scan(PlanDesc d, int32_t* plan, int blocks) {
  __shared__ int32_t offs[kMaxBuckets + 1], cnt[kMaxBuckets], tiles[kMaxBuckets + 1], wsum[kPlanThreads / 64];
  const int B = static_cast<int>(d.E) + 2;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) {
    int32_t* h = plan + d.scratch + b;
    int n = 0;
    for (int k = 0; k < blocks; ++k) {
      const int c = h[static_cast<int64_t>(k) * B];
      h[static_cast<int64_t>(k) * B] = n;
      n += c;
    }
    cnt[b] = n;
    offs[b] = n;
    plan[d.counts + b] = n;
  }
  __syncthreads();
  scan(offs, B, wsum);
  for (int b = threadIdx.x; b <= B; b += kPlanThreads) plan[d.offsets + b] = offs[b];
  for (int t = 0; t < kPlanTileKinds; ++t) {
    const int T = kPlanTiles[t];
    for (int b = threadIdx.x; b < B; b += kPlanThreads) tiles[b] = (cnt[b] + T - 1) / T;
    __syncthreads();
    scan(tiles, B, wsum);
    if (t == kPlanTileKinds - 1)
      for (int b = threadIdx.x; b <= B; b += kPlanThreads) plan[d.tile128 + b] = tiles[b];
    const int total = tiles[B];
    for (int64_t i = threadIdx.x; i < d.cap[t]; i += kPlanThreads) {
      int32_t* m = plan + d.map[t] + 3 * i;
      if (i >= total) {
        m[0] = -1;
        m[1] = 0;
        m[2] = 0;
        continue;
      }
      int lo = 0, hi = B - 1;  // the last bucket whose first tile is at or before i and that has tiles
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tiles[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      m[0] = lo;
      m[1] = offs[lo] + (static_cast<int>(i) - tiles[lo]) * T;
      m[2] = offs[lo + 1];
    }
    __syncthreads();
  }
}

// Pairs to their places, in order inside a bucket: base of the workgroup's chunk, then the waves in order, then lanes.
__global__ __launch_bounds__(kPlanThreads) void k_plan_scatter(const int32_t* ids, PlanDesc d, int32_t* plan) {
  __shared__ int32_t base[kMaxBuckets];
  __shared__ uint16_t in_wave[kPlanThreads / 64][kMaxBuckets];
  const int E = static_cast<int>(d.E), B = E + 2, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int b = threadIdx.x; b < B; b += kPlanThreads) {
    base[b] = plan[d.offsets + b] + plan[d.scratch + static_cast<int64_t>(blockIdx.x) * B + b];
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) in_wave[w][b] = 0;
  }
  __syncthreads();
  const int64_t chunk = plan_chunk(d.pairs), p0 = blockIdx.x * chunk, p1 = std::min(p0 + chunk, d.pairs);
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
    if (here && rank == 0) in_wave[wave][b] = static_cast<uint16_t>(__popcll(same));
    __syncthreads();
    if (here) {
      int at = base[b] + rank;
      for (int w = 0; w < wave; ++w) at += in_wave[w][b];
      plan[d.order + at] = static_cast<int32_t>(p);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < B; i += kPlanThreads) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kPlanThreads / 64; ++w) {
        n += in_wave[w][i];
        in_wave[w][i] = 0;
      }
      base[i] += n;
    }
    __syncthreads();
  }
}

// ---- weighted sum of the slots ------------------------------------------------------------------

// WT: type of the weights, -1 for none (a plain sum).  8 columns a thread.
template <int YT, int WT, bool VEC>
__global__ __launch_bounds__(256) void k_combine(const typename Elem<YT>::T* y, const void* w, int64_t N, int S, int64_t M,
                                                 typename Elem<YT>::T* out) {
  typedef typename Elem<YT>::T T;
  const int64_t cols = (M + 7) / 8, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
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
    for (int e = 0; e < 8; ++e) o[e] = fmaf(k, v[e], o[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (VEC || c + e < M) out[t * M + c + e] = to_elem<YT>(o[e]);
}

// One token a workgroup, its slots dealt to the waves: dy = w dout (one rounding to fp32, one to the type), dw = <y, dout>.
template <int YT, int WT, bool VEC>
__global__ __launch_bounds__(256) void k_combine_backward(const typename Elem<YT>::T* y, const typename Elem<WT>::T* w, int S,
                                                          int64_t M, const typename Elem<YT>::T* dout,
                                                          typename Elem<YT>::T* dy, typename Elem<WT>::T* dw) {
  const int64_t t = blockIdx.x;
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
int route_blocks(int64_t N) { return static_cast<int>(std::min<int64_t>((N + kRouteTeams - 1) / kRouteTeams, 256)); }

template <int LT, int V>
hipError_t launch_v(const RouteArgs& a, hipStream_t st) {
  const int nb = route_blocks(a.N);
  float* part = static_cast<float*>(a.ws);
  int32_t* part_n = reinterpret_cast<int32_t*>(part + static_cast<int64_t>(nb) * a.E);
  const size_t lds = (a.E + 1) * 4 + static_cast<size_t>(kRouteTeams / 4) * 16 * V * 4;
  if (nb > 0) {
    k_route<LT, V><<<nb, kRouteThreads, lds, st>>>(a, part, part_n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_route_sum<<<1, 1024, 0, st>>>(part, part_n, nb, a);
  return hipGetLastError();
}

template <int LT, int V>
hipError_t launch_v(const RouteBackwardArgs& a, hipStream_t st) {
  const int nb = static_cast<int>(std::min<int64_t>((a.N + kRouteTeams - 1) / kRouteTeams, 2048));
  k_route_backward<LT, V><<<nb, kRouteThreads, 0, st>>>(a);
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
  const int64_t blocks = (N * ((M + 7) / 8) + 255) / 256;
  if (blocks > INT_MAX) return hipErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(blocks);
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
    k_combine_backward<YT, WT, true><<<static_cast<unsigned>(N), 256, 0, st>>>(
        static_cast<const T*>(y), static_cast<const W*>(w), S, M, static_cast<const T*>(dout), static_cast<T*>(dy),
        static_cast<W*>(dw));
  else
    k_combine_backward<YT, WT, false><<<static_cast<unsigned>(N), 256, 0, st>>>(
        static_cast<const T*>(y), static_cast<const W*>(w), S, M, static_cast<const T*>(dout), static_cast<T*>(dy),
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
  d.order = d.tile128 + B + 1;
  int64_t at = d.order + pairs;
  for (int t = 0; t < kPlanTileKinds; ++t) {
    d.map[t] = at;
    // every bucket with pairs adds at most one part-filled tile
    d.cap[t] = pairs / kPlanTiles[t] + std::min(B, pairs);
    at += 3 * d.cap[t];
  }
  d.scratch = at;
  const int64_t blocks = pairs > 0 ? (pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs) : 0;
  d.total = at + blocks * B;
  return d;
}

hipError_t launch_route_plan(const int32_t* ids, int64_t pairs, int64_t E, int32_t* plan, hipStream_t st) {
  const PlanDesc d = plan_desc(pairs, E);
  const int blocks = pairs > 0 ? static_cast<int>((pairs + plan_chunk(pairs) - 1) / plan_chunk(pairs)) : 0;
  hipError_t e = hipSuccess;
  if (pairs > 0) {
    k_plan_count<<<blocks, kPlanThreads, 0, st>>>(ids, d, plan);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_plan_scan<<<1, kPlanThreads, 0, st>>>(d, plan, blocks);
  e = hipGetLastError();
  if (e != hipSuccess || pairs == 0) return e;
  k_plan_scatter<<<blocks, kPlanThreads, 0, st>>>(ids, d, plan);
  return hipGetLastError();
}

size_t route_workspace_bytes(int64_t N, int64_t E) {
  return N > 0 ? static_cast<size_t>(route_blocks(N)) * static_cast<size_t>(2 * E + 1) * 4 : 0;
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
