// f8_quant.hip -- quantizers to e4m3 with a scale per block of 128, the transposition of quantized weights, and
// their decoding.
//
// A block's scale is s = max(fp32(max |x| / 448), 2^-80); a code is the e4m3 value nearest to the real quotient
// x / s (ties to even).  All four forms read their input once and are bound by memory: 2 or 4 bytes in and 1 out
// per value (the division, made exact by its remainder, is ~10 fp32 operations).
#include <climits>

#include "f8.hpp"

namespace qmm {

namespace {

// largest of v over the 16 lanes of a DPP row
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x128, 0xF, 0xF, false)));  // row_ror:8
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x124, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x122, 0xF, 0xF, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x121, 0xF, 0xF, false)));
  return v;
}

template <int DT>
__device__ __forceinline__ uint2 codes8(const float* v, float s, float rs) {
  float q[8], ss[8], rr[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { ss[i] = s; rr[i] = rs; }
  f8_quotients<DT>(v, ss, rr, q);
  return make_uint2(f8_pack4(q[0], q[1], q[2], q[3]), f8_pack4(q[4], q[5], q[6], q[7]));
}

// Groups along K only: 16 lanes hold one token's group, 8 values each; a workgroup takes 16 tokens of one group, so
// that their scales (group-major) are one 64-byte store.  Bound by memory: 4096 x 4096 in bf16 10.1 us, 5.0 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void k_f8_quant_rows(F8QuantArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (t >= a.N) return;
  const int64_t g = blockIdx.y;
  const int64_t c = g * kF8Block + lane * 8;
  float v[8];
  load_row8<DT>(static_cast<const typename Elem<DT>::T*>(a.x) + t * a.ldx, c, a.K, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  const float s = f8_scale(max16(m));
  *reinterpret_cast<uint2*>(a.codes_r + t * f8_pad(a.K) + c) = codes8<DT>(v, s, f8_inverse(s));
  if (lane == 0) a.scales_r[g * a.N + t] = s;
}

// Transposed write of a 128 x 128 tile of codes through LDS: column by column of 128 bytes, whose 8-byte pieces are
// xored with the column's lane, so that 16 lanes that write one piece of 16 columns, or read the 16 pieces of one, use
// every bank once.  Rows r .. of column lane * 8 + j (r a multiple of the store's size):
__device__ __forceinline__ uint8_t* lds_piece(uint8_t* tile, int col, int r) {
  return tile + col * 128 + (((r >> 3) ^ (col >> 3)) * 8) + (r & 7);
}

// A tile's threads are teams of 16 lanes; a thread holds R rows x 8 columns.  4 rows a thread keep half the values in
// registers that 8 would, and twice the threads on a tile (777 x 515 fp32, 35 tiles, 11.6 -> 6.3 us).  2 suit the two
// quotients a value of rows and columns at once (4096 x 4096 in bf16 20.0 -> 18.8 us, 777 x 515 in fp32 6.5 -> 6.6), not
// one (columns alone 12.9 -> 14.6; weights of 4096 x 2560 10.8 -> 12.0).
constexpr int tile_rows(bool rows, bool cols) { return rows && cols ? 2 : 4; }
constexpr int tile_threads(int R) { return 128 / R * 16; }

// codes of R rows of one column, transposed from R words of 4 columns each, at dst
template <int R>
__device__ __forceinline__ void store_column(uint8_t* dst, uint32_t w) {
  if constexpr (R == 4) *reinterpret_cast<uint32_t*>(dst) = w;
  else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w);
}
template <int R>
__device__ __forceinline__ uint32_t column(const uint2* q, int j) {
  uint32_t w = 0;
#pragma unroll
  for (int p = 0; p < R; ++p) w |= (((j < 4 ? q[p].x : q[p].y) >> (8 * (j & 3))) & 0xFFu) << (8 * p);
  return w;
}

// A 128 x 128 tile in registers.  ROWS: one scale per row of the tile; COLS: one per column, codes transposed; neither:
// one for the tile, codes as they stand and (codes_c given) transposed.  Weights are bound by memory (8 x 2048 x 2560 fp32
// with the transpose 39 us, 6.4 TB/s), rows and columns at once by vector operations (4096 x 4096 bf16 18.8 us, 3.6 TB/s).
template <int DT, bool ROWS, bool COLS>
__global__ __launch_bounds__(tile_threads(tile_rows(ROWS, COLS))) void k_f8_quant_tile(F8QuantArgs a, int64_t w_rows_pad) {
  typedef typename Elem<DT>::T T;
  constexpr int R = tile_rows(ROWS, COLS), kTileThreads = tile_threads(R);
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ uint32_t cmax[kTileThreads / 64][128];
  __shared__ float2 cscale[128];  // scale and its inverse
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int64_t Kp = f8_pad(a.K);
  const int64_t N = a.N, tiles = a.plan ? a.pd.cap[kPlanTileKinds - 1] : (N + kF8Block - 1) / kF8Block;
  const unsigned tiles_k = static_cast<unsigned>(Kp / kF8Block), b = static_cast<unsigned>(block_index());
  const int64_t g = b % tiles_k;  // tile along K
  const int64_t j = b / tiles_k;  // tile along the rows
  if (j >= tiles) return;
  const T* x = static_cast<const T*>(a.x);
  const int64_t e = blockIdx.z;  // expert of a weight
  if (!ROWS && !COLS) x += e * a.N * a.K;
  const int64_t c = g * kF8Block + lane * 8;
  const int r0 = team * R;
  Raw8<DT> raw[R];
  float v[R][8];
  int64_t src[R];  // row of x, -1 past the end
  if (a.plan) {
    const int32_t* mp = a.plan + a.pd.map[kPlanTileKinds - 1] + 3 * j;
    const int bucket = mp[0], first = mp[1], end = mp[2];
    if (bucket < 0 || bucket >= a.pd.E) return;  // no expert's pairs: no product reads this group
#pragma unroll
    for (int p = 0; p < R; ++p) src[p] = a.plan[a.pd.order + std::min(first + r0 + p, end - 1)] / a.slots;
#pragma unroll
    for (int p = 0; p < R; ++p)
      if (first + r0 + p >= end) src[p] = -1;
  } else {
#pragma unroll
    for (int p = 0; p < R; ++p) {
      src[p] = j * kF8Block + r0 + p;
      if (src[p] >= N) src[p] = -1;
    }
  }
#pragma unroll
  for (int p = 0; p < R; ++p) raw[p].load(x + std::max<int64_t>(src[p], 0) * a.ldx, c, a.K);  // absent: row 0
#pragma unroll
  for (int p = 0; p < R; ++p) {
    raw[p].widen(v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = src[p] >= 0 ? v[p][i] : 0.0f;
  }
  if (ROWS) {
#pragma unroll
    for (int p = 0; p < R; ++p) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[p][i]));
      const float s = f8_scale(max16(m));
      const int64_t r = j * kF8Block + r0 + p;
      if (r < N) {
        *reinterpret_cast<uint2*>(a.codes_r + r * Kp + c) = codes8<DT>(v[p], s, f8_inverse(s));
        if (lane == 0) a.scales_r[g * N + r] = s;
      }
    }
  }
  const int64_t Np = COLS ? tiles * kF8Block : w_rows_pad;
  if (COLS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < R; ++p) m = max(m, abs_bits(v[p][i]));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
      if ((team & 3) == 0) cmax[wave][lane * 8 + i] = m;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      uint32_t m = 0;
#pragma unroll
      for (int t = 0; t < kTileThreads / 64; ++t) m = max(m, cmax[t][threadIdx.x]);
      const float s = f8_scale(m);
      cscale[threadIdx.x] = make_float2(s, f8_inverse(s));
      const int64_t k = g * kF8Block + threadIdx.x;
      if (k < a.K) a.scales_c[j * a.K + k] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i += 8 / R) {
      float col[8], q[8], s[8], rs[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 sr = cscale[lane * 8 + i + n / R];
        col[n] = v[n % R][i + n / R];
        s[n] = sr.x;
        rs[n] = sr.y;
      }
      f8_quotients<DT>(col, s, rs, q);
      const uint32_t w[2] = {f8_pack4(q[0], q[1], q[2], q[3]), f8_pack4(q[4], q[5], q[6], q[7])};
#pragma unroll
      for (int n = 0; n < 8 / R; ++n) store_column<R>(lds_piece(tile, lane * 8 + i + n, r0), w[n * R / 4] >> (n * R % 4 * 8));
    }
  }
  if (!ROWS && !COLS) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < R; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[p][i]));
    m = max16(m);
    if (lane == 0) cmax[0][team] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int t = 0; t < kTileThreads / 16; ++t) m = max(m, cmax[0][t]);
    const float s = f8_scale(m), rs = f8_inverse(s);
    const int64_t G = Kp / kF8Block, blocks = f8_pad(N) / kF8Block;
    uint2 q[R];
#pragma unroll
    for (int p = 0; p < R; ++p) {
      q[p] = codes8<DT>(v[p], s, rs);
      const int64_t r = j * kF8Block + r0 + p;
      if (r < N) *reinterpret_cast<uint2*>(a.codes_r + (e * N + r) * Kp + c) = q[p];
    }
    if (threadIdx.x == 0) a.scales_r[(e * blocks + j) * G + g] = s;
    if (!a.codes_c) return;
    if (threadIdx.x == 0) a.scales_c[(e * G + g) * blocks + j] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) store_column<R>(lds_piece(tile, lane * 8 + i, r0), column<R>(q, i));
  }
  if (COLS || !ROWS) {
    __syncthreads();
    const int64_t row0 = COLS ? 0 : e * a.K;
#pragma unroll
    for (int p = 0; p < 128 / (kTileThreads / 16); ++p) {
      const int col = p * (kTileThreads / 16) + team;
      const int64_t k = g * kF8Block + col;
      if (k < a.K)
        *reinterpret_cast<uint2*>(a.codes_c + (row0 + k) * Np + j * kF8Block + lane * 8) =
            *reinterpret_cast<const uint2*>(lds_piece(tile, col, lane * 8));
    }
  }
}

// The codes of the transposed matrix: the same bytes, tile by tile (8192 x 8192 21 us, 6.3 TB/s).
__global__ __launch_bounds__(tile_threads(4)) void k_f8_transpose(const uint8_t* codes, const float* scales, int64_t M,
                                                               int64_t K, uint8_t* codes_t, float* scales_t) {
  constexpr int kTileRows = 4, kTileThreads = tile_threads(kTileRows);
  __shared__ __align__(16) uint8_t tile[128 * 128];
  const int lane = threadIdx.x & 15, team = threadIdx.x >> 4, r0 = team * kTileRows;
  const int64_t Kp = f8_pad(K), Mp = f8_pad(M), G = Kp / kF8Block, R = Mp / kF8Block;
  const unsigned b = static_cast<unsigned>(block_index());
  const int64_t g = b % static_cast<unsigned>(G), j = b / static_cast<unsigned>(G), e = blockIdx.z;
  if (j >= R) return;
  uint2 q[kTileRows];
#pragma unroll
  for (int p = 0; p < kTileRows; ++p) {
    const int64_t r = j * kF8Block + r0 + p;
    q[p] = r < M ? *reinterpret_cast<const uint2*>(codes + (e * M + r) * Kp + g * kF8Block + lane * 8) : make_uint2(0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) store_column<kTileRows>(lds_piece(tile, lane * 8 + i, r0), column<kTileRows>(q, i));
  if (threadIdx.x == 0) scales_t[(e * G + g) * R + j] = scales[(e * R + j) * G + g];
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 128 / (kTileThreads / 16); ++p) {
    const int col = p * (kTileThreads / 16) + team;
    const int64_t k = g * kF8Block + col;
    if (k < K)
      *reinterpret_cast<uint2*>(codes_t + (e * K + k) * Mp + j * kF8Block + lane * 8) =
          *reinterpret_cast<const uint2*>(lds_piece(tile, col, lane * 8));
  }
}

// Decoded weights: code times scale, exact in fp32 up to its one rounding, rounded once more to a 16-bit output.  Eight
// columns a thread, in one store (a column a thread took 95 us for 8192 x 8192 to bf16, this 31: 6.4 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void k_f8_dequantize(const uint8_t* codes, const float* scales, int64_t M, int64_t K,
                                                       typename Elem<DT>::T* out) {
  typedef typename Elem<DT>::T T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  typedef T8 T8u __attribute__((aligned(sizeof(T))));
  const int64_t Kp = f8_pad(K), i = (block_index() * 256 + threadIdx.x) * 8;
  if (i >= M * Kp) return;
  const int64_t r = i / Kp, k = i - r * Kp;
  const uint2 w = *reinterpret_cast<const uint2*>(codes + i);
  const float s = scales[r / kF8Block * (Kp / kF8Block) + k / kF8Block];
  T8 o;
#pragma unroll
  for (int n = 0; n < 8; ++n) o[n] = to_elem<DT>(__builtin_amdgcn_cvt_f32_fp8(n < 4 ? w.x >> (8 * n) : w.y >> (8 * n - 32), 0) * s);
  T* dst = out + r * K + k;
  if (k + 8 <= K) {
    *reinterpret_cast<T8u*>(dst) = o;
  } else {
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (k + n < K) dst[n] = o[n];
  }
}

template <int DT, bool ROWS, bool COLS>
hipError_t run_tiles(const F8QuantArgs& a, int64_t tiles, int64_t E, int64_t rows_pad, hipStream_t st) {
  if (tiles > INT_MAX) return hipErrorInvalidValue;
  constexpr int kThreads = tile_threads(tile_rows(ROWS, COLS));
  k_f8_quant_tile<DT, ROWS, COLS><<<long_grid(tiles, kThreads, E), kThreads, 0, st>>>(a, rows_pad);
  return hipGetLastError();
}

template <int DT>
hipError_t quantize_dt(const F8QuantArgs& a, hipStream_t st) {
  const int64_t G = f8_pad(a.K) / kF8Block;
  if (!a.codes_c) {
    const dim3 grid(static_cast<unsigned>((a.N + 15) / 16), static_cast<unsigned>(G));
    k_f8_quant_rows<DT><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
  }
  const int64_t tiles = a.plan ? a.pd.cap[kPlanTileKinds - 1] : (a.N + kF8Block - 1) / kF8Block;
  return a.codes_r ? run_tiles<DT, true, true>(a, tiles * G, 1, 0, st) : run_tiles<DT, false, true>(a, tiles * G, 1, 0, st);
}

template <int DT>
hipError_t quantize_weight_dt(const F8QuantArgs& a, int64_t E, hipStream_t st) {
  return run_tiles<DT, false, false>(a, f8_pad(a.K) / kF8Block * (f8_pad(a.N) / kF8Block), E, f8_pad(a.N), st);
}

}  // namespace

hipError_t launch_f8_quantize(const F8QuantArgs& a, int dt, hipStream_t st) {
  switch (dt) {
    case DT_F32: return quantize_dt<DT_F32>(a, st);
    case DT_F16: return quantize_dt<DT_F16>(a, st);
    case DT_BF16: return quantize_dt<DT_BF16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_f8_quantize_weight(const void* w, int dt, int64_t E, int64_t M, int64_t K, uint8_t* codes,
                                     float* scales, uint8_t* codes_t, float* scales_t, hipStream_t st) {
  F8QuantArgs a{};
  a.x = w;
  a.ldx = K;
  a.N = M;
  a.K = K;
  a.codes_r = codes;
  a.scales_r = scales;
  a.codes_c = codes_t;
  a.scales_c = scales_t;
  switch (dt) {
    case DT_F32: return quantize_weight_dt<DT_F32>(a, E, st);
    case DT_F16: return quantize_weight_dt<DT_F16>(a, E, st);
    case DT_BF16: return quantize_weight_dt<DT_BF16>(a, E, st);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_f8_transpose(const F8Desc& m, uint8_t* codes_t, float* scales_t, hipStream_t st) {
  const int64_t tiles = m.Kp / kF8Block * (f8_pad(m.M) / kF8Block);
  if (tiles > INT_MAX) return hipErrorInvalidValue;
  k_f8_transpose<<<long_grid(tiles, tile_threads(4), m.n_experts), tile_threads(4), 0, st>>>(m.codes, m.scales, m.M, m.K, codes_t, scales_t);
  return hipGetLastError();
}

hipError_t launch_f8_dequantize(const F8Desc& m, int64_t expert, void* out, int dt, hipStream_t st) {
  const uint8_t* c = m.codes + expert * m.M * m.Kp;
  const float* s = m.scales + expert * (f8_pad(m.M) / kF8Block) * (m.Kp / kF8Block);
  const dim3 grid = long_grid((m.M * m.Kp / 8 + 255) / 256);
  switch (dt) {
    case DT_F32: k_f8_dequantize<DT_F32><<<grid, 256, 0, st>>>(c, s, m.M, m.K, static_cast<float*>(out)); break;
    case DT_F16: k_f8_dequantize<DT_F16><<<grid, 256, 0, st>>>(c, s, m.M, m.K, static_cast<_Float16*>(out)); break;
    case DT_BF16: k_f8_dequantize<DT_BF16><<<grid, 256, 0, st>>>(c, s, m.M, m.K, static_cast<__bf16*>(out)); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace qmm
