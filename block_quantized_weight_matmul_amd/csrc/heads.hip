// heads.hip -- norms and rotation of query and key heads, and the paged cache: written (quantized where its type is
// e4m3) and read back.
#include <algorithm>

#include "attn.hpp"

namespace qmm {

namespace {

typedef f32x4 f32x4u __attribute__((aligned(4)));

template <int DT> struct Quad { typedef typename Elem<DT>::T V __attribute__((ext_vector_type(4))); };

// four elements as they are (aligned to the elements only)
template <int DT>
__device__ __forceinline__ typename Quad<DT>::V load4(const typename Elem<DT>::T* p) {
  typedef typename Quad<DT>::V Vu __attribute__((aligned(sizeof(typename Elem<DT>::T))));
  return *reinterpret_cast<const Vu*>(p);
}
template <int DT>
__device__ __forceinline__ void store4(typename Elem<DT>::T* p, const float* v) {
  typedef typename Quad<DT>::V V;
  typedef V Vu __attribute__((aligned(sizeof(typename Elem<DT>::T))));
  V w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = static_cast<typename Elem<DT>::T>(v[i]);
  *reinterpret_cast<Vu*>(p) = w;
}

// A lane's eight weights for queries and for keys (null: ones), of a type known at run time: one branch around all loads, so
// that they are in flight together.
template <int DT>
__device__ __forceinline__ void load_weights(const void* qw, const void* kw, int a, int b, float* q, float* k) {
  typedef typename Elem<DT>::T T;
  const void* some = qw ? qw : kw;
  const T *pq = static_cast<const T*>(qw ? qw : some), *pk = static_cast<const T*>(kw ? kw : some);
  const typename Quad<DT>::V v[4] = {load4<DT>(pq + a), load4<DT>(pq + b), load4<DT>(pk + a), load4<DT>(pk + b)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = static_cast<float>(v[0][i]);
    q[4 + i] = static_cast<float>(v[1][i]);
    k[i] = static_cast<float>(v[2][i]);
    k[4 + i] = static_cast<float>(v[3][i]);
  }
}

// sine and cosine of an angle of any size, to fp32's rounding: the angle less a multiple of pi / 2 (a two-part constant;
// fma keeps the first difference exact), then the Taylor series on [-pi/4, pi/4], whose remainder is below 3e-14
__device__ __forceinline__ void turn(double angle, float& sine, float& cosine) {
  const double n = __builtin_rint(angle * 0.63661977236758134308);
  double r = fma(-n, 0x1.921fb54442d18p+0, angle);
  r = fma(-n, 0x1.1a62633145c07p-54, r);
  const double x = r * r;
  double s = 1.0 / 6227020800.0;
  s = fma(s, x, -1.0 / 39916800.0);
  s = fma(s, x, 1.0 / 362880.0);
  s = fma(s, x, -1.0 / 5040.0);
  s = fma(s, x, 1.0 / 120.0);
  s = fma(s, x, -1.0 / 6.0);
  s = fma(s * x, r, r);
  double c = -1.0 / 87178291200.0;
  c = fma(c, x, 1.0 / 479001600.0);
  c = fma(c, x, -1.0 / 3628800.0);
  c = fma(c, x, 1.0 / 40320.0);
  c = fma(c, x, -1.0 / 720.0);
  c = fma(c, x, 1.0 / 24.0);
  c = fma(c, x, -0.5);
  c = fma(c, x, 1.0);
  const int quarter = static_cast<int>(static_cast<int64_t>(n)) & 3;
  const float fs = static_cast<float>(s), fc = static_cast<float>(c);
  const float a = quarter & 1 ? fc : fs, b = quarter & 1 ? fs : fc;
  sine = quarter & 2 ? -a : a;
  cosine = (quarter + 1) & 2 ? -b : b;
}

// A head's rows in a cache: where slot `slot` of head h lies.
struct SlotRow {
  int64_t row;  // in rows of D
  bool there;
};
__device__ __forceinline__ SlotRow slot_row(const CacheDesc& c, int32_t slot, int h) {
  const int64_t page = slot >> c.shift, at = slot & ((1 << c.shift) - 1);
  return {((page * c.heads + h) << c.shift) + at, slot >= 0 && page < c.pages};
}

// Eight values of a lane of a team that holds a head, to row `row` of a cache of type CT: columns a .. a + 3 and b .. b +
// 3.  DT: the type the values were rounded to, which decides the form of the quotient.
template <int CT, int DT, int L>
__device__ __forceinline__ void to_cache(const float* v, uint8_t* data, float* scales, const SlotRow& r, int D, int a,
                                         int b, bool mine) {
  if constexpr (CT == DT_E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    const float s = f8_scale(team_max<L>(mine ? m : 0u)), rs = f8_inverse(s);
    float q[8], ss[8], rr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { ss[i] = s; rr[i] = rs; }
    f8_quotients<DT>(v, ss, rr, q);
    if (r.there && mine) {
      uint8_t* d = data + r.row * D;
      *reinterpret_cast<uint32_t*>(d + a) = f8_pack4(q[0], q[1], q[2], q[3]);
      *reinterpret_cast<uint32_t*>(d + b) = f8_pack4(q[4], q[5], q[6], q[7]);
      if (a == 0) scales[r.row] = s;
    }
  } else {
    if (r.there && mine) {
      typename Elem<CT>::T* d = reinterpret_cast<typename Elem<CT>::T*>(data) + r.row * D;
      store4<CT>(d + a, v);
      store4<CT>(d + b, v + 4);
    }
  }
}

// 1 / sqrt(m) to about half a step: the hardware's is good to one, and a Newton step halves that.  (A root of a number too
// small for it takes the division, by a lane's own number: the vote is a branch, and no token's bits depend on the ones beside
// it.)
__device__ __forceinline__ float inverse_root(float m) {
  float r = __builtin_amdgcn_rsqf(m);
  r = m < INFINITY ? fmaf(fmaf(-m * r, r, 1.0f), 0.5f * r, r) : r;
  if (__any(m < 0x1p-100f)) r = m < 0x1p-100f ? 1.0f / sqrtf(m) : r;
  return r;
}

// Norms and rotation.  A team of L lanes takes a token, and the launch's layers along z a share of the heads each.  A lane
// holds eight columns of a head, the two members of each of its four pairs among them (halves of the rotated part, or
// neighbours), so that a rotation needs no other lane, and the four angles serve every head of the token.
//
//   y = x * w / sqrt(mean(x^2) + eps);   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq
//
// Bound by memory: 8192 tokens of 32 + 8 heads of 128 in bf16 take 37.7 us, 4.45 TB/s of what is read and written (heads chosen
// by each lane, with their branches, 67; a weight behind a branch of its own 46).  A decode step's launch is latency, 4.3 us.
//
// Sums in fp32, the angle and its reduction in 64 bits (a position of 2^20 loses all of a fast pair's angle in 32), one
// rounding at the end.  CACHE: keys and values go to their slots; a key is rounded to the queries' type first, so that the
// call leaves the bits of the two calls it stands for.
template <int XT, int QT, int CT, bool CACHE, int L>
__global__ __launch_bounds__(256) void k_heads(HeadsArgs a) {
  constexpr int kTeams = 256 / L, kAhead = 4;
  typedef typename Elem<XT>::T X;
  typedef typename Quad<XT>::V V4;
  const int lane = threadIdx.x % L;
  const int64_t t = block_index() * kTeams + threadIdx.x / L;
  if (t >= a.T) return;  // whole teams: no lane of this one is asked for
  const int heads = a.Hq + a.H + (CACHE ? a.H : 0), per = (heads + gridDim.z - 1) / gridDim.z;
  const int h0 = blockIdx.z * per, h1 = min(heads, h0 + per);
  if (h0 >= h1) return;
  const int D = a.D, R = a.R;
  const bool mine = lane * 8 < D, turned = lane * 8 < R, halves = !a.interleaved;
  const int pair0 = turned ? lane * 4 : 0;
  // the eight columns: ca .. ca + 3, cb .. cb + 3
  const int ca = !mine ? 0 : turned && halves ? pair0 : lane * 8;
  const int cb = !mine ? 0 : turned && halves ? R / 2 + pair0 : lane * 8 + 4;

  const X* const q = static_cast<const X*>(a.q.p) + t * a.q.st;
  const X* const k = static_cast<const X*>(a.k.p) + t * a.k.st - a.Hq * a.k.sh;
  const X* const v = CACHE ? static_cast<const X*>(a.v.p) + t * a.v.st - (a.Hq + a.H) * a.v.sh : nullptr;
  V4 lo[kAhead], hi[kAhead];
  auto load = [&](int h) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int g = min(h + n, h1 - 1);
      const X* p = g < a.Hq ? q + g * a.q.sh : !CACHE || g < a.Hq + a.H ? k + g * a.k.sh : v + g * a.v.sh;
      lo[n] = load4<XT>(p + ca);
      hi[n] = load4<XT>(p + cb);
    }
  };
  load(h0);
  int32_t slot = -1;
  if constexpr (CACHE) slot = a.slots[t];
  float qw[8], kw[8];
  if (a.qw || a.kw) {
    if (a.wt == DT_F32) load_weights<DT_F32>(a.qw, a.kw, ca, cb, qw, kw);
    else if (a.wt == DT_F16) load_weights<DT_F16>(a.qw, a.kw, ca, cb, qw, kw);
    else load_weights<DT_BF16>(a.qw, a.kw, ca, cb, qw, kw);
  }
  float sine[4], cosine[4];  // while the first heads are on their way
  if (a.inv_freq) {
    const double p = a.positions[t];
    const f32x4 f = *reinterpret_cast<const f32x4u*>(a.inv_freq + pair0);
#pragma unroll
    for (int i = 0; i < 4; ++i) turn(p * static_cast<double>(f[i]), sine[i], cosine[i]);
  }
  const float share = 1.0f / static_cast<float>(D);

  // one head, normed and rotated
  auto norm_turn = [&](const V4& x0, const V4& x1, bool normed, const float* w, float* y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = static_cast<float>(x0[i]);
      y[4 + i] = static_cast<float>(x1[i]);
    }
    if (normed) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
      const float r = inverse_root(fmaf(team_sum<L>(mine ? sum : 0.0f), share, a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * r * w[i];
    }
    if (a.inv_freq) {
      float z[8];
      if (halves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[i] = fmaf(y[i], cosine[i], -(y[4 + i] * sine[i]));
          z[4 + i] = fmaf(y[4 + i], cosine[i], y[i] * sine[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[2 * i] = fmaf(y[2 * i], cosine[i], -(y[2 * i + 1] * sine[i]));
          z[2 * i + 1] = fmaf(y[2 * i + 1], cosine[i], y[2 * i] * sine[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = turned ? z[i] : y[i];
    }
  };
  typedef typename Elem<QT>::T Q;
  Q* const qo = static_cast<Q*>(a.qo) + t * a.Hq * D;
  Q* const ko = CACHE ? nullptr : static_cast<Q*>(a.ko) + (t * a.H - a.Hq) * D;

  for (int h = h0; h < h1; h += kAhead) {
    V4 x0[kAhead], x1[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) x0[n] = lo[n], x1[n] = hi[n];
    if (h + kAhead < h1) load(h + kAhead);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int g = h + n;
      if (g >= h1) break;
      float y[8];
      if (g < a.Hq) {
        norm_turn(x0[n], x1[n], a.qw != nullptr, qw, y);
        if (mine) {
          store4<QT>(qo + g * D + ca, y);
          store4<QT>(qo + g * D + cb, y + 4);
        }
      } else if (!CACHE || g < a.Hq + a.H) {
        norm_turn(x0[n], x1[n], a.kw != nullptr, kw, y);
        if constexpr (CACHE) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = static_cast<float>(static_cast<Q>(y[i]));
          to_cache<CT, QT, L>(y, a.cache.k, a.cache.ks, slot_row(a.cache, slot, g - a.Hq), D, ca, cb, mine);
        } else if (mine) {
          store4<QT>(ko + g * D + ca, y);
          store4<QT>(ko + g * D + cb, y + 4);
        }
      } else if constexpr (CACHE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = static_cast<float>(x0[n][i]);
          y[4 + i] = static_cast<float>(x1[n][i]);
        }
        to_cache<CT, XT, L>(y, a.cache.v, a.cache.vs, slot_row(a.cache, slot, g - a.Hq - a.H), D, ca, cb, mine);
      }
    }
  }
}

// Keys and values of T tokens to their slots: a team of L lanes takes a token's head, of both; the launch's layers along z are
// the heads.  Bound by memory: 32768 tokens of 8 heads of 128, bf16 to e4m3, 36 us, 5.6 TB/s (a head found by a division 40.5;
// in a 16-bit cache 41.9 and 40.5); few tokens are latency, 2 to 3 us.
template <int XT, int CT, int L>
__global__ __launch_bounds__(256) void k_cache_write(CacheDesc c, HeadRows k, HeadRows v, int64_t T, const int32_t* slots) {
  typedef typename Elem<XT>::T X;
  const int lane = threadIdx.x % L, D = c.D;
  const int64_t t = block_index() * (256 / L) + threadIdx.x / L;
  if (t >= T) return;
  const int h = blockIdx.z;
  const bool mine = lane * 8 < D;
  const int at = mine ? lane * 8 : 0;
  float kv[8], vv[8];
  load8<XT>(static_cast<const X*>(k.p) + t * k.st + h * k.sh + at, kv);
  load8<XT>(static_cast<const X*>(v.p) + t * v.st + h * v.sh + at, vv);
  const SlotRow r = slot_row(c, slots[t], h);
  to_cache<CT, XT, L>(kv, c.k, c.ks, r, D, at, at + 4, mine);
  to_cache<CT, XT, L>(vv, c.v, c.vs, r, D, at, at + 4, mine);
}

// Packed rows from the cache: a team of L lanes takes a row and a share of its heads, four at a time, for that many loads on
// their way.  Bound by memory: 52553 tokens of 8 heads of 128, e4m3 to bf16, 63.5 us, 5.1 TB/s of what is read and written.
template <int CT, int OT, int L>
__global__ __launch_bounds__(256) void k_cache_read(CacheDesc c, const int32_t* table, int64_t B, int64_t W,
                                                    const int32_t* starts, int64_t total, void* ko, void* vo) {
  constexpr int kTeams = 256 / L;
  typedef typename Elem<OT>::T O;
  const int lane = threadIdx.x % L, D = c.D, H = c.heads;
  const int64_t first = block_index() * kTeams, row = first + threadIdx.x / L;
  int64_t b = count_first(B, [&](int64_t i) { return starts[i + 1] <= first; });
  if (row >= total) return;
  // the workgroup's rows may end a sequence, and any number of empty ones follow
  int64_t more = 1;
  for (; b + more <= B && starts[b + more] <= row; more *= 2) b += more;
  while (more /= 2)
    if (b + more <= B && starts[b + more] <= row) b += more;
  if (b >= B) return;                         // behind the last sequence
  const int64_t t = row - starts[b];
  if (t < 0) return;                          // before the first
  const int64_t column = t >> c.shift;
  const int64_t page = column < W ? table[b * W + column] : -1;
  const bool there = page >= 0 && page < c.pages;
  const int64_t base = ((there ? page * H : 0) << c.shift) + (t & ((1 << c.shift) - 1));
  const bool mine = lane * 8 < D;
  const int at = mine ? lane * 8 : 0;
  const int h0 = blockIdx.z, step = gridDim.z;
  constexpr int kAhead = 4;
  for (int h = h0; h < H; h += kAhead * step) {
    float kx[kAhead][8], vx[kAhead][8];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int64_t r = base + (static_cast<int64_t>(min(h + n * step, H - 1)) << c.shift);
      if constexpr (CT == DT_E4M3) {
        const uint2 kc = *reinterpret_cast<const uint2*>(c.k + r * D + at), vc = *reinterpret_cast<const uint2*>(c.v + r * D + at);
        const float ks = c.ks[r], vs = c.vs[r];
        const uint32_t kw[2] = {kc.x, kc.y}, vw[2] = {vc.x, vc.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto k0 = __builtin_amdgcn_cvt_pk_f32_fp8(kw[i], false), k1 = __builtin_amdgcn_cvt_pk_f32_fp8(kw[i], true);
          const auto v0 = __builtin_amdgcn_cvt_pk_f32_fp8(vw[i], false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8(vw[i], true);
          kx[n][4 * i] = k0[0] * ks, kx[n][4 * i + 1] = k0[1] * ks, kx[n][4 * i + 2] = k1[0] * ks, kx[n][4 * i + 3] = k1[1] * ks;
          vx[n][4 * i] = v0[0] * vs, vx[n][4 * i + 1] = v0[1] * vs, vx[n][4 * i + 2] = v1[0] * vs, vx[n][4 * i + 3] = v1[1] * vs;
        }
      } else {
        load8<CT>(reinterpret_cast<const typename Elem<CT>::T*>(c.k) + r * D + at, kx[n]);
        load8<CT>(reinterpret_cast<const typename Elem<CT>::T*>(c.v) + r * D + at, vx[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (h + n * step >= H || !mine) break;
      if (!there) {
#pragma unroll
        for (int i = 0; i < 8; ++i) kx[n][i] = vx[n][i] = __uint_as_float(0x7FC00000u);
      }
      const int64_t o = (row * H + h + n * step) * D + at;
      store4<OT>(static_cast<O*>(ko) + o, kx[n]);
      store4<OT>(static_cast<O*>(ko) + o + 4, kx[n] + 4);
      store4<OT>(static_cast<O*>(vo) + o, vx[n]);
      store4<OT>(static_cast<O*>(vo) + o + 4, vx[n] + 4);
    }
  }
}

template <int DT> struct Int { static constexpr int value = DT; };

// f(Int<DT>) for one of the three element types
template <typename F>
hipError_t with_type(int dt, F f) {
  if (dt == DT_F32) return f(Int<DT_F32>{});
  if (dt == DT_F16) return f(Int<DT_F16>{});
  return f(Int<DT_BF16>{});
}
// f(Int<lanes>) for the team that holds D columns, eight a lane
template <typename F>
hipError_t with_team(int D, F f) {
  if (D <= 64) return f(Int<8>{});
  if (D <= 128) return f(Int<16>{});
  return f(Int<32>{});
}

}  // namespace

hipError_t launch_heads(const HeadsArgs& a, int xt, int qt, hipStream_t s) {
  const bool cache = a.slots != nullptr;
  const int heads = a.Hq + a.H + (cache ? a.H : 0);
  return with_team(a.D, [&](auto l) {
    constexpr int L = decltype(l)::value;
    // A token's heads are divided among layers until the teams fill four waves of every SIMD, at least four heads each, one
    // round of loads; each layer makes the tokens' angles anew.
    const int64_t want = 256 * 16 * (64 / L), most = (heads + 3) / 4;
    const int64_t layers = std::min(most, (want + a.T - 1) / a.T);
    const int64_t blocks = (a.T + 256 / L - 1) / (256 / L);
    return with_type(xt, [&](auto x) {
      constexpr int XT = decltype(x)::value;
      auto go = [&](auto q, auto c, auto w) {
        hipLaunchKernelGGL((k_heads<XT, decltype(q)::value, decltype(c)::value, decltype(w)::value != 0, L>),
                           long_grid(blocks, 256, layers), dim3(256), 0, s, a);
        return hipGetLastError();
      };
      if (!cache) return with_type(qt, [&](auto q) { return go(q, q, Int<0>{}); });
      if (a.cache.type == DT_E4M3) return with_type(qt, [&](auto q) { return go(q, Int<DT_E4M3>{}, Int<1>{}); });
      return a.cache.type == DT_F16 ? go(Int<DT_F16>{}, Int<DT_F16>{}, Int<1>{}) : go(Int<DT_BF16>{}, Int<DT_BF16>{}, Int<1>{});
    });
  });
}

hipError_t launch_cache_write(const CacheDesc& c, const HeadRows& k, const HeadRows& v, int xt, int64_t T,
                              const int32_t* slots, hipStream_t s) {
  return with_team(c.D, [&](auto l) {
    constexpr int L = decltype(l)::value;
    const int64_t blocks = (T + 256 / L - 1) / (256 / L);
    return with_type(xt, [&](auto x) {
      constexpr int XT = decltype(x)::value;
      auto go = [&](auto ct) {
        hipLaunchKernelGGL((k_cache_write<XT, decltype(ct)::value, L>), long_grid(blocks, 256, c.heads), dim3(256), 0, s, c, k, v, T, slots);
        return hipGetLastError();
      };
      if (c.type == DT_E4M3) return go(Int<DT_E4M3>{});
      return c.type == DT_F16 ? go(Int<DT_F16>{}) : go(Int<DT_BF16>{});
    });
  });
}

hipError_t launch_cache_read(const CacheDesc& c, const int32_t* table, int64_t B, int64_t W, const int32_t* starts,
                             int64_t total, void* k, void* v, int ot, hipStream_t s) {
  return with_team(c.D, [&](auto l) {
    constexpr int L = decltype(l)::value;
    const int64_t blocks = (total + 256 / L - 1) / (256 / L);
    const int64_t quads = (c.heads + 3) / 4;
    const int64_t share = blocks >= 4 * c.cus ? 1 : quads;  // few rows: four heads a team
    return with_type(ot, [&](auto o) {
      constexpr int OT = decltype(o)::value;
      auto go = [&](auto ct) {
        hipLaunchKernelGGL((k_cache_read<decltype(ct)::value, OT, L>), long_grid(blocks, 256, share), dim3(256), 0, s, c, table,
                           B, W, starts, total, k, v);
        return hipGetLastError();
      };
      if (c.type == DT_E4M3) return go(Int<DT_E4M3>{});
      return c.type == DT_F16 ? go(Int<DT_F16>{}) : go(Int<DT_BF16>{});
    });
  });
}

}  // namespace qmm
