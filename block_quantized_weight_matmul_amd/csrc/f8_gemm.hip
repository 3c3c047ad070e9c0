// f8_gemm.hip -- products of e4m3 operands with one scale per 128 values of K.
//
// Tiled kernel for many tokens; the arithmetic and the choice of matrix cores are f8_mma.hpp's, few tokens f8_few.hip's.
#include <algorithm>
#include <climits>

#include "f8.hpp"
#include "f8_mma.hpp"

namespace qmm {

namespace {

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes a lane straight into LDS: lane i's at dst + 16 i (dst: the wave's base)
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, voff, soff, 0, 0);
}
enum { MODE_DENSE = 0, MODE_ID = 1, MODE_WGRAD = 2 };

struct GemmArgs {
  const uint8_t* w;   // A rows: codes [M][pitch] (MODE_ID: of every expert)
  const float* ws;    // scales: [blocks of M][G] (WGRAD: [G][M])
  const uint8_t* x;   // B rows (tokens): codes [N][pitch]
  const float* xs;    // [G][N]
  void* y;            // [N][M] (ID: [pairs][M]; WGRAD with a plan: [E][N][M])
  int64_t M, N, pitch;
  int G;              // groups along the reduction
  int tiles_m, tiles_n;
  const int32_t* plan;
  PlanDesc pd;
  int map;            // index of the token tile's map in the plan
  int slots;          // MODE_ID: pairs that share a token row
  int vec;            // outputs of 4 consecutive rows may be stored at once
};

// One workgroup: TM rows x TN tokens, its waves in a WM x WN grid; K in stages of one group, two stages in LDS.
// A stage's rows are 128 bytes; their eight 16-byte pieces are stored xored with the row's low bits, so that the 8
// lanes of a read phase (8 rows, one piece) use every bank once.
template <int TM, int TN, int WM, int WN, int MODE, int OT>
__global__ __launch_bounds__(64 * WM * WN) void k_f8_gemm(GemmArgs a) {
  constexpr int NT = 64 * WM * WN, RT = TM / WM / 16, CT = TN / WN / 16;
  constexpr int AI = TM * 8 / NT, BI = TN * 8 / NT;  // 16-byte pieces a thread stages
  static_assert(AI * NT == TM * 8 && BI * NT == TN * 8, "tile");
  constexpr bool kRowScale = MODE == MODE_WGRAD;
  constexpr int kStage = (TM + TN) * 128 + TN * 4 + (kRowScale ? TM * 4 : 0);
  __shared__ __align__(128) uint8_t lds[2][kStage];
  typedef typename Elem<OT>::T T;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % WM, wn = wave / WM;
  int64_t bid = blockIdx.x;
  const int tm = static_cast<int>(bid % a.tiles_m);
  bid /= a.tiles_m;
  const int64_t r0 = static_cast<int64_t>(tm) * TM;
  int64_t M = a.M, N = a.N;
  const uint8_t* w = a.w;
  const float* wsc = a.ws;
  T* y = static_cast<T*>(a.y);
  int g0 = 0, g1 = a.G;
  int64_t t0;
  int first = 0, count = 0;  // MODE_ID: the tile's pairs
  if constexpr (MODE == MODE_ID) {
    const int32_t* mp = a.plan + a.pd.map[a.map] + 3 * bid;
    const int bucket = mp[0];
    first = mp[1];
    count = mp[2] - first;
    if (bucket < 0) return;
    count = count < TN ? count : TN;
    if (bucket >= a.pd.E) {  // empty slots: zeros; ids that name no expert: NaN
      const float v = bucket == a.pd.E ? 0.0f : __uint_as_float(0x7FC00000u);
      const int rows = static_cast<int>(M - r0 < TM ? M - r0 : TM);
      for (int i = tid; i < count * rows; i += NT)
        y[static_cast<int64_t>(a.plan[a.pd.order + first + i / rows]) * M + r0 + i % rows] = to_elem<OT>(v);
      return;
    }
    w += static_cast<int64_t>(bucket) * M * a.pitch;
    wsc += static_cast<int64_t>(bucket) * ((M + 127) / 128) * a.G;
    t0 = 0;
  } else if constexpr (MODE == MODE_WGRAD) {
    t0 = (bid % a.tiles_n) * TN;
    if (a.plan) {
      const int64_t e = bid / a.tiles_n;
      g0 = a.plan[a.pd.tile128 + e];
      g1 = a.plan[a.pd.tile128 + e + 1];
      y += e * M * N;
    }
  } else {
    t0 = bid * TN;
  }

  // what this thread stages: offsets from the tile's first row
  const int64_t last_m = M - 1 - r0;
  const __amdgpu_buffer_rsrc_t rw = rsrc(w + r0 * a.pitch, static_cast<uint32_t>(std::min<int64_t>(TM, M - r0) * a.pitch));
  __amdgpu_buffer_rsrc_t rx, rxs;
  uint32_t aoff[AI], boff[BI];
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int p = i * NT + tid, row = p >> 3;
    aoff[i] = static_cast<uint32_t>((row < last_m ? row : last_m) * a.pitch) + 16 * ((p ^ row) & 7);
  }
  if constexpr (MODE == MODE_ID) {
    rx = rsrc(a.x, static_cast<uint32_t>(N * a.pitch));
    rxs = rsrc(a.xs, static_cast<uint32_t>(N * a.G * 4));
  } else {
    rx = rsrc(a.x + t0 * a.pitch, static_cast<uint32_t>(std::min<int64_t>(TN, N - t0) * a.pitch));
    rxs = rx;
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int p = i * NT + tid, row = p >> 3;
    int64_t src;
    if constexpr (MODE == MODE_ID) src = a.plan[a.pd.order + first + (row < count ? row : count - 1)] / a.slots;
    else src = row < N - 1 - t0 ? row : N - 1 - t0;
    boff[i] = static_cast<uint32_t>(src * a.pitch) + 16 * ((p ^ row) & 7);
  }
  // scales: thread i < TN the token's, the next TM (WGRAD) the row's
  int64_t soff = 0;
  const bool sx_thread = tid < TN;
  if constexpr (MODE == MODE_ID) {
    if (sx_thread) soff = a.plan[a.pd.order + first + (tid < count ? tid : count - 1)] / a.slots;
  } else {
    if (sx_thread) soff = t0 + tid < N ? t0 + tid : N - 1;
  }
  const float* srow_x = a.xs + soff;
  const float* srow_w = kRowScale && tid < TM ? wsc + (r0 + tid < M ? r0 + tid : M - 1) : nullptr;
  (void)rxs;

  auto stage = [&](int buf, int g) {
    uint8_t* d = lds[buf];
    const uint32_t ks = static_cast<uint32_t>(g) * 128u;
#pragma unroll
    for (int i = 0; i < AI; ++i) load_lds16(rw, d + (i * NT + wave * 64) * 16, aoff[i], ks);
#pragma unroll
    for (int i = 0; i < BI; ++i) load_lds16(rx, d + TM * 128 + (i * NT + wave * 64) * 16, boff[i], ks);
  };
  float nsx = 0.0f, nsw = 0.0f;
  auto fetch_scales = [&](int g) {
    if (sx_thread) nsx = srow_x[static_cast<int64_t>(g) * N];
    if (kRowScale && tid < TM) nsw = srow_w[static_cast<int64_t>(g) * M];
  };
  auto put_scales = [&](int buf) {
    float* s = reinterpret_cast<float*>(lds[buf] + (TM + TN) * 128);
    if (sx_thread) s[tid] = nsx;
    if (kRowScale && tid < TM) s[TN + tid] = nsw;
  };

  f32x4 acc[RT][CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // a wave's rows lie in one 128-row block of the weights (TM / WM divides 128)
  static_assert(128 % (TM / WM) == 0, "a wave's rows share their scales");
  const float* wblock = wsc + (kRowScale ? 0 : ((r0 + wm * (TM / WM)) / 128) * static_cast<int64_t>(a.G));
  const bool wave_rows = r0 + wm * (TM / WM) < M;

  if (g0 < g1) {
    stage(0, g0);
    fetch_scales(g0);
    put_scales(0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  for (int g = g0; g < g1; ++g) {
    const int buf = (g - g0) & 1;
    if (g + 1 < g1) {
      stage(buf ^ 1, g + 1);
      fetch_scales(g + 1);
    }
    const uint8_t* A = lds[buf] + wm * (TM / WM) * 128;
    const uint8_t* B = lds[buf] + TM * 128 + wn * (TN / WN) * 128;
    const float* S = reinterpret_cast<const float*>(lds[buf] + (TM + TN) * 128);
    const int row = lane & 15, q = lane >> 4;
    const int c0 = 16 * ((2 * q) ^ (row & 7)), c1 = 16 * ((2 * q + 1) ^ (row & 7));
    float wscale = 1.0f;
    if (!kRowScale && wave_rows) wscale = wblock[g];
    Frag<OT == DT_F32> b[CT];
    float s[CT];
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(B + (j * 16 + row) * 128 + c0);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(B + (j * 16 + row) * 128 + c1);
      b[j].set(lo, hi);
      s[j] = S[wn * (TN / WN) + j * 16 + row] * wscale;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(A + (i * 16 + row) * 128 + c0);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(A + (i * 16 + row) * 128 + c1);
      Frag<OT == DT_F32> av;
      av.set(lo, hi);
      f32x4 rs{1.0f, 1.0f, 1.0f, 1.0f};
      if (kRowScale) rs = *reinterpret_cast<const f32x4*>(S + TN + wm * (TM / WM) + i * 16 + q * 4);
#pragma unroll
      for (int j = 0; j < CT; ++j) {
        const f32x4 p = group_sum(av, b[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = fmaf(p[e], kRowScale ? s[j] * rs[e] : s[j], acc[i][j][e]);
      }
    }
    if (g + 1 < g1) put_scales(buf ^ 1);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }

#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int t = wn * (TN / WN) + j * 16 + (lane & 15);
    int64_t yrow;
    if constexpr (MODE == MODE_ID) {
      if (t >= count) continue;
      yrow = a.plan[a.pd.order + first + t];
    } else {
      yrow = t0 + t;
      if (yrow >= N) continue;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t r = r0 + wm * (TM / WM) + i * 16 + (lane >> 4) * 4;
      const int64_t left = M - r;
      if (left > 0) store4<OT>(y + yrow * M + r, acc[i][j], left < 4 ? static_cast<int>(left) : 4, a.vec);
    }
  }
}

template <int TM, int TN, int WM, int WN, int MODE>
hipError_t run_tile(const GemmArgs& a, int ot, int64_t blocks, hipStream_t st) {
  if (blocks > INT_MAX) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * WM * WN);
  switch (ot) {
    case DT_F32: k_f8_gemm<TM, TN, WM, WN, MODE, DT_F32><<<grid, block, 0, st>>>(a); break;
    case DT_F16: k_f8_gemm<TM, TN, WM, WN, MODE, DT_F16><<<grid, block, 0, st>>>(a); break;
    case DT_BF16: k_f8_gemm<TM, TN, WM, WN, MODE, DT_BF16><<<grid, block, 0, st>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

size_t f8_gemm_workspace_bytes(const F8Desc&, int64_t) { return 0; }

hipError_t launch_f8_gemm(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t N, void* y, int yt, void*,
                          hipStream_t st) {
  if (f8_few_tokens(m, N)) return launch_f8_few(m, xc, xs, N, y, yt, st);
  GemmArgs a{};
  a.w = m.codes;
  a.ws = m.scales;
  a.x = xc;
  a.xs = xs;
  a.y = y;
  a.M = m.M;
  a.N = N;
  a.pitch = m.Kp;
  a.G = static_cast<int>(m.Kp / kF8Block);
  a.vec = store_vec(y, m.M, yt);
  a.tiles_m = static_cast<int>((m.M + 127) / 128);
  a.tiles_n = static_cast<int>((N + 127) / 128);
  return run_tile<128, 128, 2, 2, MODE_DENSE>(a, yt, static_cast<int64_t>(a.tiles_m) * a.tiles_n, st);
}

hipError_t launch_f8_gemm_id(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t pairs, int slots,
                             const int32_t* plan, void* y, int yt, hipStream_t st) {
  GemmArgs a{};
  a.w = m.codes;
  a.ws = m.scales;
  a.x = xc;
  a.xs = xs;
  a.y = y;
  a.M = m.M;
  a.N = pairs / slots;
  a.pitch = m.Kp;
  a.G = static_cast<int>(m.Kp / kF8Block);
  a.vec = store_vec(y, m.M, yt);
  a.plan = plan;
  a.pd = plan_desc(pairs, m.n_experts);
  a.slots = slots;
  a.tiles_m = static_cast<int>((m.M + 127) / 128);
  a.map = 3;
  return run_tile<128, 128, 2, 2, MODE_ID>(a, yt, static_cast<int64_t>(a.tiles_m) * a.pd.cap[3], st);
}

hipError_t launch_f8_wgrad(const F8WgradArgs& w, hipStream_t st) {
  GemmArgs a{};
  a.w = w.xc;
  a.ws = w.xs;
  a.x = w.gc;
  a.xs = w.gs;
  a.y = w.dw;
  a.M = w.K;
  a.N = w.M;
  a.pitch = w.Np;
  a.G = static_cast<int>(w.Np / kF8Block);
  a.vec = store_vec(w.dw, w.K, w.dt);
  a.plan = w.plan;
  a.pd = w.pd;
  a.tiles_m = static_cast<int>((w.K + 127) / 128);
  a.tiles_n = static_cast<int>((w.M + 127) / 128);
  const int64_t E = w.plan ? w.pd.E : 1;
  return run_tile<128, 128, 2, 2, MODE_WGRAD>(a, w.dt, static_cast<int64_t>(a.tiles_m) * a.tiles_n * E, st);
}

}  // namespace qmm
