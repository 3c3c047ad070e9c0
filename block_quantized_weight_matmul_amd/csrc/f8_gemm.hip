// f8_gemm.hip -- products of e4m3 operands with one scale per 128 values of K.
//
// Tiled kernel for many tokens; the arithmetic and the choice of matrix cores are f8_mma.hpp's, few tokens f8_few.hip's.
#include <algorithm>
#include <cmath>

#include "f8.hpp"
#include "f8_mma.hpp"

namespace qmm {

namespace {

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, voff, soff, 0, 0);
}
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
  int share;          // groups of a workgroup where the reduction is divided (gridDim.y > 1)
  int vec;            // 16 bytes of consecutive outputs may be stored at once
};

// waves a SIMD that the LDS of a tile's stages leaves room for
constexpr int tile_waves(int TM, int TN) { return TM + TN > 192 ? 2 : TM + TN > 128 ? 3 : 4; }

// One workgroup: TM rows x TN tokens, its waves in a WM x WN grid; K in stages of one group, two stages in LDS.
// A stage's rows are 128 bytes, two to the 64 banks; their eight 16-byte pieces are stored xored with bits 1..3 of the
// row, so that 16 lanes that read one piece of 16 rows use every bank once (xored with bits 0..2, the reads took twice
// the cycles, and a 256 x 256 stage 4190 instead of 3570).
//
// The second bound, waves per SIMD, keeps the compiler at 256 registers or fewer: above, it puts the sums of the matrix
// cores into the accumulation registers, which the vector units cannot read.
// EXACT: the cores of an fp32 output (f8_mma.hpp); ST: the type stored.
//
// 16-bit outputs: 4096 x 4096 x 2560 47 us, 1.83 PFLOP/s; 8192^3 481 us, 2.29; dW of the former 66 us; 128 experts of 4096
// x 512 and 16384 pairs 100 us, whose 400 MB are most of it.  A 256 x 256 stage takes 3500 cycles for 2048 of matrix
// instructions: 192 KB read from LDS and 64 KB put there, at 128 bytes a cycle as many, and the fma of the group sums
// (promotion) do not hide behind them entirely, and power holds the clock at 1.7 to 2.1 GHz.
template <int TM, int TN, int WM, int WN, int MODE, bool EXACT, int ST>
__global__ __launch_bounds__(64 * WM * WN, tile_waves(TM, TN)) void k_f8_gemm(GemmArgs a) {
  constexpr int NT = 64 * WM * WN, RT = TM / WM / 32, CT = TN / WN / 32;
  constexpr int AI = TM * 8 / NT, BI = TN * 8 / NT;  // 16-byte pieces a thread stages
  static_assert(AI * NT == TM * 8 && BI * NT == TN * 8, "tile");
  constexpr bool kRowScale = MODE == MODE_WGRAD, kId = MODE == MODE_ID;
  constexpr int W = WM * WN;
  constexpr int TS = TN < 64 ? 64 : TN;                // room of the token scales: whole loads of 64
  constexpr int kScales = TS + (kRowScale ? TM : 64);  // then the rows' or the row blocks'
  constexpr int kUnitsPer = (kScales / 64 + W - 1) / W;  // loads of 64 scales a wave; those past the last repeat it
  constexpr int kStage = (TM + TN) * 128 + kUnitsPer * W * 256;
  constexpr int kRows = RT * 32, kPitch = kRows * static_cast<int>(sizeof(typename Elem<ST>::T)) + 16;  // of a wave's outputs
  // The two stages, and after the loop the waves' outputs.  One array: with a second one the compiler waits for a stage's
  // loads before any read of the other stage (51 -> 43 us for 8 experts of 2048 x 2560 and 4096 pairs).
  __shared__ __align__(128) uint8_t lds[2 * kStage];
  typedef typename Elem<ST>::T T;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  // Tile indices, kept in scalar registers: divisions leave them in vector registers, and every staging load would then
  // loop over the lanes' copies of its descriptor.
  auto scalar = [](unsigned v) { return static_cast<unsigned>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); };
  unsigned bid = blockIdx.x, tm;
  if constexpr (MODE == MODE_DENSE) {
    // Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, kGroup row tiles by all token tiles after
    // another, so that the tiles it works on share their operands in its L2.
    constexpr unsigned kXcds = 8, kGroup = 1024 / TM;
    const unsigned n = gridDim.x, per = n / kXcds, more = n % kXcds, x = bid % kXcds;
    bid = x * per + std::min(x, more) + bid / kXcds;
    const unsigned in = kGroup * static_cast<unsigned>(a.tiles_n), gm = scalar(bid / in) * kGroup, off = bid - gm / kGroup * in;
    const unsigned wide = std::min(kGroup, static_cast<unsigned>(a.tiles_m) - gm);
    bid = scalar(off / wide);
    tm = gm + off - bid * wide;
  } else if constexpr (kId) {
    // An XCD takes a run of the listed tiles: the token tiles of an expert share its weights in one L2.
    const unsigned rows = static_cast<unsigned>(a.tiles_m);
    const unsigned n = scalar(static_cast<unsigned>(a.plan[a.pd.totals + a.map])) * rows, per = (n + 7) / 8, k = bid / 8;
    bid = bid % 8 * per + k;
    if (k >= per || bid >= n) return;
    const unsigned tile = scalar(bid / rows);
    tm = bid - tile * rows;
    bid = tile;
  } else {
    const unsigned rest = scalar(bid / static_cast<unsigned>(a.tiles_m));
    tm = bid - rest * static_cast<unsigned>(a.tiles_m);
    bid = rest;
  }
  const int64_t r0 = static_cast<int64_t>(tm) * TM;
  const int64_t M = a.M, N = a.N;
  const uint8_t* w = a.w;
  const float* wsc = a.ws;
  T* y = static_cast<T*>(a.y);
  int g0 = 0, g1 = a.G;
  int64_t t0;
  int first = 0, count = 0;  // MODE_ID: the tile's pairs
  auto share = [&]() {  // of the reduction, the sums to a slab of their own
    g0 = static_cast<int>(blockIdx.y) * a.share;
    g1 = std::min(a.G, g0 + a.share);
    y += static_cast<int64_t>(blockIdx.y) * M * N;
  };
  if constexpr (kId) {
    const int32_t* mp = a.plan + a.pd.map[a.map] + 3 * static_cast<int64_t>(bid);
    const int bucket = static_cast<int>(scalar(static_cast<unsigned>(mp[0])));
    first = static_cast<int>(scalar(static_cast<unsigned>(mp[1])));
    count = static_cast<int>(scalar(static_cast<unsigned>(mp[2]))) - first;
    count = count < TN ? count : TN;
    if (bucket >= a.pd.E) {  // empty slots: zeros; ids that name no expert: NaN
      const float v = bucket == a.pd.E ? 0.0f : __uint_as_float(0x7FC00000u);
      const int rows = static_cast<int>(std::min<int64_t>(M - r0, TM));
      for (int i = tid; i < count * rows; i += NT)
        y[static_cast<int64_t>(a.plan[a.pd.order + first + i / rows]) * M + r0 + i % rows] = to_elem<ST>(v);
      return;
    }
    w += static_cast<int64_t>(bucket) * M * a.pitch;
    wsc += static_cast<int64_t>(bucket) * ((M + 127) / 128) * a.G;
    t0 = 0;
  } else if constexpr (MODE == MODE_WGRAD) {
    const unsigned e = scalar(bid / static_cast<unsigned>(a.tiles_n));
    t0 = static_cast<int64_t>(bid - e * static_cast<unsigned>(a.tiles_n)) * TN;
    if (a.plan) {
      g0 = static_cast<int>(scalar(static_cast<unsigned>(a.plan[a.pd.tile128 + e])));
      g1 = static_cast<int>(scalar(static_cast<unsigned>(a.plan[a.pd.tile128 + e + 1])));
      y += static_cast<int64_t>(e) * M * N;
    } else if (gridDim.y > 1) {
      share();
    }
  } else {
    t0 = static_cast<int64_t>(bid) * TN;
    if (gridDim.y > 1) share();
  }

  // What this thread stages: 16-byte pieces, offsets from the tile's first row (rows past the end repeat the last), and
  // scales, 64 to a wave's load.
  const __amdgpu_buffer_rsrc_t rx =
      kId ? rsrc(a.x, static_cast<uint32_t>(N * a.pitch))
                      : rsrc(a.x + t0 * a.pitch, static_cast<uint32_t>(std::min<int64_t>(TN, N - t0) * a.pitch));
  auto token = [&](int i) -> int64_t {  // tile row i: its row of x, from t0
    if constexpr (kId) return a.plan[a.pd.order + first + (i < count ? i : count - 1)] / a.slots;
    else return i < N - 1 - t0 ? i : N - 1 - t0;
  };
  uint32_t aoff[AI], boff[BI], soff[kUnitsPer];
  const float* sbase[kUnitsPer];
  int64_t sstep[kUnitsPer];
  uint32_t sbytes[kUnitsPer];
  const int64_t last_m = M - 1 - r0;
  const __amdgpu_buffer_rsrc_t rw = rsrc(w + r0 * a.pitch, static_cast<uint32_t>(std::min<int64_t>(TM, M - r0) * a.pitch));
#pragma unroll
  for (int i = 0; i < AI; ++i) {
    const int p = i * NT + tid, row = p >> 3;
    aoff[i] = static_cast<uint32_t>((row < last_m ? row : last_m) * a.pitch) + 16 * ((p ^ (row >> 1)) & 7);
  }
#pragma unroll
  for (int i = 0; i < BI; ++i) {
    const int p = i * NT + tid, row = p >> 3;
    boff[i] = static_cast<uint32_t>(token(row) * a.pitch) + 16 * ((p ^ (row >> 1)) & 7);
  }
#pragma unroll
  for (int k = 0; k < kUnitsPer; ++k) {
    const int u = k * W + wave, i = std::min(u * 64 + lane, kScales - 1);
    const bool tokens = u * 64 < TS;  // the same for a whole wave
    if (tokens) soff[k] = 4 * static_cast<uint32_t>(t0 + token(std::min(i, TN - 1)));
    else if (kRowScale) soff[k] = 4 * static_cast<uint32_t>(r0 + (i - TS < last_m ? i - TS : last_m));
    else soff[k] = 4 * static_cast<uint32_t>(std::min<int64_t>(i - TS, (M - 1) / 128 - r0 / 128) * a.G);
    sbase[k] = tokens ? a.xs : kRowScale ? wsc : wsc + r0 / 128 * a.G;
    sstep[k] = tokens ? N : kRowScale ? M : 1;
    // the last row block's scales end at its G-th: a base advanced by g leaves G - g of them
    sbytes[k] = tokens || kRowScale ? 0u : static_cast<uint32_t>(((M + 127) / 128 - r0 / 128) * a.G * 4);
  }

  // a descriptor in scalar registers, whichever its parts are in
  auto uniform = [&](const void* p, uint32_t bytes) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t u = static_cast<uint64_t>(scalar(static_cast<unsigned>(v >> 32))) << 32 | scalar(static_cast<unsigned>(v));
    return rsrc(reinterpret_cast<const void*>(u), scalar(bytes));
  };
  auto stage = [&](int buf, int g) {
    uint8_t* d = lds + buf * kStage;
    const uint32_t ks = static_cast<uint32_t>(g) * 128u;
#pragma unroll
    for (int i = 0; i < AI; ++i) load_lds16(rw, d + (i * NT + wave * 64) * 16, aoff[i], ks);
#pragma unroll
    for (int i = 0; i < BI; ++i) load_lds16(rx, d + TM * 128 + (i * NT + wave * 64) * 16, boff[i], ks);
#pragma unroll
    for (int k = 0; k < kUnitsPer; ++k)
      load_lds4(uniform(sbase[k] + g * sstep[k], sbytes[k] ? sbytes[k] - 4 * g : static_cast<uint32_t>(sstep[k]) * 4),
                d + (TM + TN) * 128 + (k * W + wave) * 256, soff[k], 0);
  };

  f32x16 acc[RT][CT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[i][j] = f32x16{};

  // a wave's rows lie in one 128-row block of the weights
  static_assert(128 % (TM / WM) == 0, "a wave's rows share their scales");
  const int row = lane & 31, half = lane >> 5;
  uint32_t piece[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    piece[m][0] = row * 128 + 16 * ((4 * m + 2 * half) ^ (row >> 1 & 7));
    piece[m][1] = row * 128 + 16 * ((4 * m + 2 * half + 1) ^ (row >> 1 & 7));
  }
  typedef Frag32<EXACT> F;
  auto read_frag = [&](F& f, const uint8_t* p) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
      f.set(m, *reinterpret_cast<const i32x4*>(p + piece[m][0]), *reinterpret_cast<const i32x4*>(p + piece[m][1]));
  };
  const uint8_t* Abase = lds + wm * (TM / WM) * 128;
  const uint8_t* Bbase = lds + (TM + wn * (TN / WN)) * 128;
  const float* Sbase = reinterpret_cast<const float*>(lds + (TM + TN) * 128);
  // Scales.  The sweep over the groups multiplies a group's sum by its token's and its row block's scale in one step
  // (kRowScale: by one after the other), which is right unless their product leaves fp32's normal range (the sum times the
  // token's may overflow).  A wave that met such scales, from operands with both largest values around 2^-55 or a product
  // of them above 2^145, makes its outputs anew behind the sweep, the scales in order of size.  Two blocks of the smallest
  // scale, 2^-80, which zeros have, do not count: what they add is below 2^-135.  That costs the others 0 to 2% (8192^3
  // 474 -> 477 us).  Asking at the start of every stage made each wait for its scales (480 us); a second sweep by the
  // whole workgroup had it agree on one (experts +3%); telling zeros in the sweep took 7% of small tiles.
  F b[CT];
  float sc[CT];
  uint32_t least = ~0u, most = 0u;  // bits of the smallest and the largest factor; a NaN is large
  auto read_b = [&](int buf) {
    const float* S = Sbase + buf * (kStage / 4);
    const float wscale = kRowScale ? 1.0f : S[TS + wm * (TM / WM) / 128];
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      read_frag(b[j], Bbase + buf * kStage + j * 4096);
      sc[j] = S[wn * (TN / WN) + j * 32 + row] * wscale;
    }
  };
  auto read_rs = [&](f32x4* rs, int buf, int i) {
    if (kRowScale) {
      const float* S = Sbase + buf * (kStage / 4) + TS + wm * (TM / WM) + i * 32 + half * 4;
#pragma unroll
      for (int k = 0; k < 4; ++k) rs[k] = *reinterpret_cast<const f32x4*>(S + 8 * k);
    }
  };
  auto add = [&](f32x16& to, const f32x16& p, float s, const f32x4* rs) {
#pragma unroll
    for (int e = 0; e < 16; ++e) to[e] = kRowScale ? fmaf(p[e] * s, rs[e / 4][e % 4], to[e]) : fmaf(p[e], s, to[e]);
  };

  // Outputs leave through LDS, 32 tokens of the wave's rows at a time: a lane holds 4 rows of one token, and stores
  // straight from there would be 16 bytes a token (10 us of the 60 at 4096 x 4096 outputs).
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  static_assert(W * 32 * kPitch <= 2 * kStage, "the waves' regions fit the stages");
  uint8_t* mine = lds + wave * (32 * kPitch);
  constexpr int kLanes = kRows / kVec;             // lanes that store one token's rows
  constexpr int kStores = 32 * kLanes / 64;        // stores of a lane for 32 tokens
  // MODE_ID: the output rows of this lane's tokens, looked up before the loop (a lookup in it waits for the stage's loads)
  int32_t orow[kId ? CT * kStores : 1];
  if constexpr (kId) {
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int n = 0; n < kStores; ++n) {
        const int t = wn * (TN / WN) + j * 32 + n * (64 / kLanes) + lane / kLanes;
        orow[j * kStores + n] = a.plan[a.pd.order + first + std::min(t, count - 1)];
      }
  }
  auto store = [&]() {
    const int64_t rw0 = r0 + wm * kRows;
    const int rows = static_cast<int>(std::min<int64_t>(kRows, M - rw0));  // may be negative
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      const int tj = wn * (TN / WN) + j * 32;
      int tokens = kId ? count - tj : static_cast<int>(std::min<int64_t>(32, N - t0 - tj));
      tokens = std::min(tokens, 32);
      auto out = [&](int t) -> T* {
        if constexpr (kId) return y + static_cast<int64_t>(a.plan[a.pd.order + first + tj + t]) * M + rw0;
        else return y + (t0 + tj + t) * M + rw0;
      };
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          typedef T T4 __attribute__((ext_vector_type(4)));
          T4 o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = to_elem<ST>(acc[i][j][4 * k + e]);
          *reinterpret_cast<T4*>(mine + row * kPitch + (i * 32 + k * 8 + half * 4) * sizeof(T)) = o;
        }
      __builtin_amdgcn_wave_barrier();
      if (a.vec) {  // M is a multiple of kVec and rows are 16-byte aligned
        // every read before any store: a read of LDS waits for the memory operations before it
        const int c = lane % kLanes * kVec;
        uint4 v[kStores];
#pragma unroll
        for (int n = 0; n < kStores; ++n)
          v[n] = *reinterpret_cast<const uint4*>(mine + (n * (64 / kLanes) + lane / kLanes) * kPitch + c * sizeof(T));
#pragma unroll
        for (int n = 0; n < kStores; ++n) {
          const int t = n * (64 / kLanes) + lane / kLanes;
          T* o = kId ? y + static_cast<int64_t>(orow[kId ? j * kStores + n : 0]) * M + rw0 : out(t);
          if (t < tokens && c < rows) *reinterpret_cast<uint4*>(o + c) = v[n];
        }
      } else {
        for (int n = lane; n < 32 * kRows; n += 64) {
          const int t = n / kRows, c = n % kRows;
          if (t < tokens && c < rows) out(t)[c] = *reinterpret_cast<const T*>(mine + t * kPitch + c * sizeof(T));
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  if (g0 < g1) stage(0, g0);
  for (int g = g0; g < g1; ++g) {
    const int buf = (g - g0) & 1;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the stage's loads, issued a whole stage ago
    __syncthreads();
    if (g + 1 < g1) stage(buf ^ 1, g + 1);
    read_b(buf);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      F av;
      f32x4 rs[4];
      read_frag(av, Abase + buf * kStage + i * 4096);
      read_rs(rs, buf, i);
#pragma unroll
      for (int j = 0; j < CT; ++j) add(acc[i][j], group_sum(av, b[j]), sc[j], rs);
    }
    __builtin_amdgcn_sched_barrier(0);  // the scales are looked at behind the products
#pragma unroll
    for (int j = 0; j < CT; ++j) {
      if (!kRowScale) least = min(least, __float_as_uint(sc[j]));
      most = max(most, __float_as_uint(sc[j]));
    }
  }
  bool ordered = __any(kRowScale ? most > 0x71800000u : least < 0x00800000u || most >= 0x7F800000u);  // 2^100; 2^-126, infinity
  if (ordered) {  // unless from zeros and NaN alone
    bool out = false;
    const float* sa = wsc + std::min((r0 + wm * (TM / WM)) / 128, (M - 1) / 128) * a.G;
#pragma unroll 1
    for (int i = lane; i < TN / WN; i += 64) {
      const float* st = a.xs + t0 + token(wn * (TN / WN) + i);
#pragma unroll 4
      for (int64_t g = g0; g < g1; ++g) {
        const float s = st[g * N], f = kRowScale ? s : s * sa[g];
        out |= kRowScale ? s > 0x1p100f : (f < 0x1p-126f && fmaxf(s, sa[g]) > kF8MinScale) || f > 0x1.fffffep127f;
      }
    }
    ordered = __any(out);
  }
  if (ordered) {
    // 32 x 32 outputs at a time, straight from and to global memory, in few registers
#pragma unroll 1
    for (int ij = 0; ij < RT * CT; ++ij) {
      const int ra = wm * (TM / WM) + ij / CT * 32, tb = wn * (TN / WN) + ij % CT * 32 + row;  // first row; token
      auto at = [&](int r) { return r0 + (r < last_m ? r : last_m); };  // rows past the end repeat the last
      const int64_t t = t0 + token(std::min(tb, TN - 1));
      const uint8_t *pa = w + at(ra + row) * a.pitch + 32 * half, *pb = a.x + t * a.pitch + 32 * half;
      const float* sa = wsc + std::min((r0 + ra) / 128, (M - 1) / 128) * a.G;  // not kRowScale
      f32x16 sum{};
#pragma unroll 1
      for (int64_t g = g0; g < g1; ++g) {
        F fa, fb;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint8_t *qa = pa + g * 128 + 64 * m, *qb = pb + g * 128 + 64 * m;
          fa.set(m, *reinterpret_cast<const i32x4*>(qa), *reinterpret_cast<const i32x4*>(qa + 16));
          fb.set(m, *reinterpret_cast<const i32x4*>(qb), *reinterpret_cast<const i32x4*>(qb + 16));
        }
        const f32x16 p = group_sum(fa, fb);
        const float s = a.xs[g * N + t];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          i32x4 rs;
          if (kRowScale)  // 0 past the last row
            rs = __builtin_amdgcn_raw_buffer_load_b128(uniform(wsc + g * M, static_cast<uint32_t>(M) * 4),
                                                       4 * static_cast<uint32_t>(r0 + ra + 8 * k + 4 * half), 0, 0);
          else
            rs = __float_as_int(sa[g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 o = scale_order(s, __int_as_float(rs[e]));
            sum[4 * k + e] = fmaf(p[4 * k + e] * o.x, o.y, sum[4 * k + e]);
          }
        }
      }
      const bool mine_t = kId ? tb < count : t0 + tb < N;
      T* out = y + (kId ? static_cast<int64_t>(a.plan[a.pd.order + first + std::min(tb, count - 1)]) : t0 + tb) * M;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t r = r0 + ra + e / 4 * 8 + half * 4 + e % 4;
        if (mine_t && r < M) out[r] = to_elem<ST>(sum[e]);
      }
    }
  }
  __syncthreads();
  if (!ordered) store();
}

template <int TM, int TN, int WM, int WN, int MODE>
hipError_t run_tile(const GemmArgs& a, int ot, int64_t blocks, hipStream_t st) {
  if (!fits_grid(blocks, 64 * WM * WN)) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * WM * WN);
  switch (ot) {
    case DT_F32:
      // (an fp32 output's operands are twice as wide in registers: no 256 x 256 tile)
      if constexpr (TM * TN <= 128 * 128) k_f8_gemm<TM, TN, WM, WN, MODE, true, DT_F32><<<grid, block, 0, st>>>(a);
      else return hipErrorInvalidValue;
      break;
    case DT_F16: k_f8_gemm<TM, TN, WM, WN, MODE, false, DT_F16><<<grid, block, 0, st>>>(a); break;
    case DT_BF16: k_f8_gemm<TM, TN, WM, WN, MODE, false, DT_BF16><<<grid, block, 0, st>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// y = the sum of the slabs [splits][n], in order
template <int OT>
__global__ __launch_bounds__(256) void k_f8_join(const float* slabs, int splits, int64_t n, typename Elem<OT>::T* y) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 4 <= n && n % 4 == 0) {
    f32x4 v = *reinterpret_cast<const f32x4*>(slabs + i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(slabs + s * n + i);
    store4<OT>(y + i, v, 4, reinterpret_cast<uintptr_t>(y) % (4 * sizeof(*y)) == 0);
  } else {
    for (int64_t k = i; k < n && k < i + 4; ++k) {
      float v = slabs[k];
      for (int s = 1; s < splits; ++s) v += slabs[s * n + k];
      y[k] = to_elem<OT>(v);
    }
  }
}

template <int TM, int TN, int MODE>
hipError_t run_split(const GemmArgs& a, bool exact, int64_t blocks, int splits, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(splits)), block(256);
  if (exact) k_f8_gemm<TM, TN, 2, 2, MODE, true, DT_F32><<<grid, block, 0, st>>>(a);
  else k_f8_gemm<TM, TN, 2, 2, MODE, false, DT_F32><<<grid, block, 0, st>>>(a);
  return hipGetLastError();
}

int store_vec16(const void* y, int64_t M, int ot) {
  return reinterpret_cast<uintptr_t>(y) % 16 == 0 && M % (ot == DT_F32 ? 4 : 8) == 0;
}

// The tiles, the workgroups of each that a CU holds at once, and what one stage (128 values of K) of 1 .. per_cu of
// them costs there, in us, from launches of 1 .. 8 of them a CU and 8, 20 and 60 stages with a 16-bit output.  A call takes
// the tile with the least estimated time, which is within 12% of the measured one at 20 stages; it is the last round of a
// launch, its CUs part-filled, that decides (dx of 4096 x 2560, 32 stages: 256 x 256 tiles 60 us, 256 x 192 53, 128 x 128
// 67, 64 x 64 74; 512 x 4096: 256 x 256 33, 128 x 128 20, 64 x 64 14; 2048 x 9728, 20 stages: 256 x 192 65, 128 x 128 62).
struct TileKind {
  int tm, tn, per_cu;
  float round;   // prologue and epilogue of a round
  float us[4];
};
enum { TILE_256 = 0, TILE_128 = 1, TILE_128_64 = 2, TILE_64 = 3, TILE_128_32 = 4, TILE_256_192 = 5 };
constexpr TileKind kTiles[] = {
    {256, 256, 1, 8.0f, {1.95f}},
    {128, 128, 2, 2.0f, {0.85f, 1.21f}},
    {128, 64, 3, 1.5f, {0.52f, 0.79f, 1.07f}},
    {64, 64, 4, 1.0f, {0.33f, 0.48f, 0.75f, 0.99f}},
    {128, 32, 4, 1.5f, {0.50f, 0.80f, 1.10f, 1.40f}},  // experts only
    {256, 192, 1, 7.0f, {1.50f}},
};

// tiles: workgroups of a launch, of `stages` stages each
float tile_cost(const TileKind& k, double tiles, double stages, int cus) {
  const double per = std::ceil(tiles / cus);
  const double full = std::floor(per / k.per_cu);
  const int rest = static_cast<int>(per - full * k.per_cu);
  return static_cast<float>(full * (k.us[k.per_cu - 1] * stages + k.round) + (rest > 0 ? k.us[rest - 1] * stages + k.round : 0.0));
}

// How a dense product of M rows, N tokens and `many` matrices runs: its tile, and the shares that K is divided into
// (1: not at all).  Shares make their sums in slabs of fp32 that k_f8_join adds: worth it where the tiles leave CUs idle
// and K is long (2560 x 9728, 64 tokens: 27 us undivided, 40 workgroups of 76 stages, 12.7 divided; dW of 128 x 2560 over
// 16384 tokens 59 and 20).
struct DensePlan {
  int kind, splits;
};
constexpr int kMinShare = 4;                              // stages
constexpr int64_t kMaxSlabs = int64_t(64) << 20;          // bytes
DensePlan dense_plan(int64_t M, int64_t N, int64_t many, double stages, bool f32, bool may_split, int cus) {
  const int kinds[] = {TILE_128, TILE_128_64, TILE_64, TILE_256, TILE_256_192};
  DensePlan best{TILE_128, 1};
  float cost = INFINITY;
  for (int i = 0; i < (f32 ? 3 : 5); ++i) {
    const TileKind& k = kTiles[kinds[i]];
    const double tiles = static_cast<double>((M + k.tm - 1) / k.tm) * static_cast<double>((N + k.tn - 1) / k.tn) * static_cast<double>(many);
    for (int s = 1; s <= 16; s *= 2) {
      if (s > 1 && (!may_split || kinds[i] == TILE_256 || kinds[i] == TILE_256_192 || kinds[i] == TILE_128 || stages < s * kMinShare || s * M * N * 4 > kMaxSlabs)) break;
      // a second launch, and the slabs written and read
      const float c = tile_cost(k, tiles * s, std::ceil(stages / s), cus) + (s > 1 ? 3.0f + static_cast<float>(s * M * N) * 8 / 4e6f : 0.0f);
      if (c < cost) {
        cost = c;
        best = {kinds[i], s};
      }
    }
  }
  return best;
}

template <int MODE>
hipError_t run_dense(GemmArgs& a, int ot, int64_t many, const DensePlan& plan, float* slabs, hipStream_t st) {
  const TileKind& k = kTiles[plan.kind];
  a.tiles_m = static_cast<int>((a.M + k.tm - 1) / k.tm);
  a.tiles_n = static_cast<int>((a.N + k.tn - 1) / k.tn);
  const int64_t blocks = static_cast<int64_t>(a.tiles_m) * a.tiles_n * many;
  if (plan.splits > 1) {
    if (!fits_grid(blocks, 256)) return hipErrorInvalidConfiguration;
    void* y = a.y;
    const int64_t n = a.M * a.N;
    a.y = slabs;
    a.vec = store_vec16(slabs, a.M, DT_F32);
    a.share = (a.G + plan.splits - 1) / plan.splits;
    const int splits = (a.G + a.share - 1) / a.share;  // every share has groups
    const hipError_t e = plan.kind == TILE_64 ? run_split<64, 64, MODE>(a, ot == DT_F32, blocks, splits, st)
                                              : run_split<128, 64, MODE>(a, ot == DT_F32, blocks, splits, st);
    if (e != hipSuccess) return e;
    const unsigned grid = static_cast<unsigned>((n + 1023) / 1024);
    switch (ot) {
      case DT_F32: k_f8_join<DT_F32><<<grid, 256, 0, st>>>(slabs, splits, n, static_cast<float*>(y)); break;
      case DT_F16: k_f8_join<DT_F16><<<grid, 256, 0, st>>>(slabs, splits, n, static_cast<_Float16*>(y)); break;
      default: k_f8_join<DT_BF16><<<grid, 256, 0, st>>>(slabs, splits, n, static_cast<__bf16*>(y)); break;
    }
    return hipGetLastError();
  }
  switch (plan.kind) {
    case TILE_256: return run_tile<256, 256, 2, 4, MODE>(a, ot, blocks, st);
    case TILE_256_192: return run_tile<256, 192, 4, 2, MODE>(a, ot, blocks, st);
    case TILE_128: return run_tile<128, 128, 2, 2, MODE>(a, ot, blocks, st);
    case TILE_128_64: return run_tile<128, 64, 2, 2, MODE>(a, ot, blocks, st);
    default: return run_tile<64, 64, 2, 2, MODE>(a, ot, blocks, st);
  }
}

// expert products: the pairs of each expert in tiles of their own
hipError_t run_experts(GemmArgs& a, int ot, int cus, hipStream_t st) {
  const int kinds[] = {TILE_128, TILE_128_64, TILE_64, TILE_128_32};
  double tiles[4];
  const double experts = static_cast<double>(std::min(a.pd.E, a.pd.pairs));
  for (int i = 0; i < 4; ++i) {
    const TileKind& k = kTiles[kinds[i]];
    // about half a tile of each expert is padding
    tiles[i] = static_cast<double>((a.M + k.tm - 1) / k.tm) * (static_cast<double>(a.pd.pairs) / k.tn + experts * 0.5);
  }
  int kind = kinds[0];
  float least = INFINITY;
  for (int i = 0; i < 4; ++i) {
    const float c = tile_cost(kTiles[kinds[i]], tiles[i], a.G, cus);
    if (c < least) {
      least = c;
      kind = kinds[i];
    }
  }
  const TileKind& k = kTiles[kind];
  a.tiles_m = static_cast<int>((a.M + k.tm - 1) / k.tm);
  a.map = 0;
  while (kPlanTiles[a.map] != k.tn) ++a.map;
  const int64_t blocks = static_cast<int64_t>(a.tiles_m) * a.pd.cap[a.map] + 7;  // a run of the listed ones for each XCD
  switch (kind) {
    case TILE_128: return run_tile<128, 128, 2, 2, MODE_ID>(a, ot, blocks, st);
    case TILE_128_64: return run_tile<128, 64, 2, 2, MODE_ID>(a, ot, blocks, st);
    case TILE_64: return run_tile<64, 64, 2, 2, MODE_ID>(a, ot, blocks, st);
    default: return run_tile<128, 32, 4, 1, MODE_ID>(a, ot, blocks, st);
  }
}

}  // namespace

// room for the slabs of a product of M x N outputs, for either kind of output
static size_t slab_bytes(int64_t M, int64_t N, int64_t stages, int cus) {
  int splits = 1;
  for (int f32 = 0; f32 < 2; ++f32)
    splits = std::max(splits, dense_plan(M, N, 1, static_cast<double>(stages), f32, true, cus).splits);
  return splits > 1 ? static_cast<size_t>(splits) * M * N * 4 : 0;
}

size_t f8_gemm_workspace_bytes(const F8Desc& m, int64_t N) {
  return f8_few_tokens(m, N) ? 0 : slab_bytes(m.M, N, m.Kp / kF8Block, m.cus);
}

size_t f8_wgrad_workspace_bytes(int64_t Np, int64_t M, int64_t K, int cus) {
  return Np > 0 ? slab_bytes(K, M, Np / kF8Block, cus) : 0;
}

hipError_t launch_f8_gemm(const F8Desc& m, const uint8_t* xc, const float* xs, int64_t N, void* y, int yt, void* ws,
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
  a.vec = store_vec16(y, m.M, yt);
  return run_dense<MODE_DENSE>(a, yt, 1, dense_plan(m.M, N, 1, a.G, yt == DT_F32, true, m.cus), static_cast<float*>(ws), st);
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
  a.vec = store_vec16(y, m.M, yt);
  a.plan = plan;
  a.pd = plan_desc(pairs, m.n_experts);
  a.slots = slots;
  return run_experts(a, yt, m.cus, st);
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
  a.vec = store_vec16(w.dw, w.K, w.dt);
  a.plan = w.plan;
  a.pd = w.pd;
  const int64_t E = w.plan ? w.pd.E : 1;
  const DensePlan plan = dense_plan(a.M, a.N, E, std::max(1.0, static_cast<double>(a.G) / E), w.dt == DT_F32,
                                    !w.plan, w.cus);
  return run_dense<MODE_WGRAD>(a, w.dt, E, plan, static_cast<float*>(w.ws), st);
}

}  // namespace qmm
