// attend.hip -- attention of one new token per sequence over the paged cache.
//
//   out[b, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - max),  j over the sequence's tokens
//
// Bound by reading the cache once.  The query heads that share a key head are the 16 columns of one matrix product (more
// than 16: further row tiles), so a token's keys and values are read once for all of them.  A sequence is divided into
// `splits` pieces of whole 32-token tiles, a piece among the four waves of a workgroup; each wave keeps its own running
// maximum, sum and output, which are joined in wave order through LDS and, where there is more than one piece, in piece
// order by a second small launch.
#include "attn.hpp"

namespace qmm {

namespace {

constexpr int kWaves = 4, kTile = 32;  // waves of a workgroup, tokens of a wave's tile
constexpr int kRows = 16;              // query heads of a workgroup

template <int QT> struct Half8 { typedef typename Elem<QT>::T V __attribute__((ext_vector_type(8))); };
template <int QT> using H8 = typename Half8<QT>::V;

__device__ __forceinline__ f32x4 mma(H8<DT_F16> a, H8<DT_F16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(H8<DT_BF16> a, H8<DT_BF16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// eight e4m3 codes as 16-bit values (each is one exactly)
template <int QT>
__device__ __forceinline__ H8<QT> widen(uint32_t lo, uint32_t hi) {
  H8<QT> r;
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (QT == DT_F16) {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[i], 1.0f, true);
      r[4 * i] = a[0], r[4 * i + 1] = a[1], r[4 * i + 2] = b[0], r[4 * i + 3] = b[1];
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
      const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
      r[4 * i] = a[0], r[4 * i + 1] = a[1], r[4 * i + 2] = b[0], r[4 * i + 3] = b[1];
    }
  }
  return r;
}

// over the four lanes that hold a column of a 16 x 16 product
__device__ __forceinline__ float column_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Pieces of a sequence: whole tiles for every wave.
__device__ __forceinline__ int64_t piece_of(int64_t len, int splits) {
  const int64_t step = kWaves * kTile;
  return ((len + splits - 1) / splits + step - 1) / step * step;
}

// Rows of a wave's tile in LDS: DP columns of `size` bytes each, in 16-byte pieces xored with a function of the row, so
// that the reads of one piece of many rows (keys) and of two neighbouring pieces of four or eight rows (values, transposed
// on the way) use different banks.
template <int ROW>  // bytes
struct Rows {
  static constexpr int kPieces = ROW / 16;
  __device__ static __forceinline__ int key(int row, int piece) {
    const int x = ROW >= 256 ? row & 15 : ROW == 128 ? (row >> 1 ^ row >> 3) & 7 : (row >> 2) & 3;
    return row * ROW + ((piece ^ x) * 16);
  }
  __device__ static __forceinline__ int value(int row, int piece) {
    const int x = ROW >= 256 ? 2 * row & 15 : ROW == 128 ? (row >> 1 ^ row >> 3) & 7 : (row >> 2) & 3;
    return row * ROW + ((piece ^ x) * 16);
  }
};

// QT: type of the queries and outputs; CT: QT or DT_E4M3; DP: columns, D rounded up to 64, 128 or 256.
//
// Scores are computed transposed, S^T = K Q^T (tokens x heads): a lane then holds, for one head, the scores of the eight
// tokens that its operand of O^T = V^T P^T takes, in the order in which that product's other operand, V^T, can be read
// from row-major LDS by transposing reads; the probabilities never leave their lane.
//
// P is fed to the matrix cores as the sum of two 16-bit numbers, its rounding and the rest (2^-17 of it in bf16): the
// cores have time to spare here, and one rounding of P to bf16 would add as much to the output's error as the output's
// own rounding.  With an e4m3 cache the tokens' scales of the values multiply P, in bf16, which has fp32's range.
template <int QT, int CT, int DP>
__global__ __launch_bounds__(64 * kWaves, DP == 256 ? 1 : 2) void k_attend(AttendArgs a) {
  constexpr bool kCodes = CT == DT_E4M3;
  constexpr int PT = kCodes ? DT_BF16 : QT;            // type of P and V on the matrix cores
  constexpr int kSize = kCodes ? 1 : 2, kRow = DP * kSize;
  constexpr int kLoads = kRow * 16 / 1024;             // of a wave, for 16 tokens
  constexpr int kBlocks = kTile / 16, kOut = DP / 16;
  constexpr float kLift = PT == DT_F16 ? 8.0f : 0.0f;  // P in fp16 times 2^8: small ones keep their bits
  typedef typename Elem<QT>::T Q;
  typedef typename Elem<PT>::T P;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kWaves][2][kTile * kRow];
  __shared__ float sums[kWaves][2][kRows];

  const CacheDesc& c = a.cache;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const int D = c.D, H = c.heads, G = a.Hq / H, tiles = (G + kRows - 1) / kRows;
  const int split = blockIdx.x, h = blockIdx.y / tiles, g0 = (blockIdx.y % tiles) * kRows;
  const int64_t b = blockIdx.z;
  const int rows = min(kRows, G - g0);                 // heads here
  const int64_t room = a.W << c.shift;
  int64_t len = a.lengths[b];
  len = len < 0 ? 0 : len > room ? room : len;
  const int64_t piece = piece_of(len, a.splits), t0 = split * piece, t1 = min(len, t0 + piece);
  if (t0 >= len && split > 0) return;                  // the join reads the pieces that there are
  const int32_t* table = a.table + b * a.W;

  // queries: column col of the products, 8 columns of the head at a time
  H8<QT> q[DP / 32];
  {
    const Q* p = static_cast<const Q*>(a.q.p) + b * a.q.st + (h * G + g0 + min(col, rows - 1)) * a.q.sh;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
      // codes: a 16-byte piece of a row holds the operands of two steps
      const int d = kCodes ? (j / 2) * 64 + quarter * 16 + (j % 2) * 8 : j * 32 + quarter * 8;
      typedef H8<QT> Qu __attribute__((aligned(sizeof(Q))));
      q[j] = *reinterpret_cast<const Qu*>(p + (d < D ? d : 0));
      if (d >= D || col >= rows) q[j] = H8<QT>{};
    }
  }

  uint8_t* const lk = lds[wave][0];
  uint8_t* const lv = lds[wave][1];
  // a lane's share of 16 tokens' rows, which lie one after another in a page: 16-byte pieces lane, lane + 64, ..
  const int pieces = D * kSize / 16;                   // of a row
  int at[kLoads], row_of[kLoads], piece_at[kLoads];
  bool some[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int i = n * 64 + lane;
    row_of[n] = DP == D ? i / (kRow / 16) : i / pieces;
    piece_at[n] = i - row_of[n] * pieces;
    some[n] = i < 16 * pieces;
    at[n] = some[n] ? i * 16 : 0;
  }
  if (D < DP) {  // columns past D: zeros, once
    for (int i = lane; i < kTile * kRow / 16; i += 64) {
      reinterpret_cast<uint4*>(lk)[i] = uint4{};
      reinterpret_cast<uint4*>(lv)[i] = uint4{};
    }
  }

  const float factor = a.scale * 1.44269504088896340736f;
  const int count = t1 > t0 ? static_cast<int>((t1 - t0 + kTile - 1) / kTile) : 0;
  bool bad = false;
  uint4 kr[kBlocks][kLoads], vr[kBlocks][kLoads];
  f32x4 ks[kBlocks], vs[kBlocks];

  // where a tile's 16-token block lies; a block past the sequence's last one repeats that
  auto block_base = [&](int64_t t) -> int64_t {
    t = min(t, (len - 1) & ~int64_t(15));
    int64_t page = table[t >> c.shift];
    if (page < 0 || page >= c.pages) bad = true, page = 0;
    return ((page * H + h) << c.shift) + (t & ((int64_t(1) << c.shift) - 1));
  };
  auto load_rows = [&](const uint8_t* data, const int64_t* base, uint4 (*r)[kLoads]) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        r[k][n] = *reinterpret_cast<const uint4*>(data + base[k] * (D * kSize) + at[n]);
  };
  auto load_scales = [&](const float* data, const int64_t* base, f32x4* r) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) r[k] = *reinterpret_cast<const f32x4*>(data + base[k] + quarter * 4);
  };

  int64_t base[kBlocks];
  if (wave < count) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) base[k] = block_base(t0 + wave * kTile + k * 16);
    load_rows(c.k, base, kr);
    load_rows(c.v, base, vr);
    if constexpr (kCodes) load_scales(c.ks, base, ks), load_scales(c.vs, base, vs);
  }

  float most = -INFINITY, total = 0.0f;  // of column col, over the scores this wave has seen
  f32x4 o[kOut];
#pragma unroll
  for (int d = 0; d < kOut; ++d) o[d] = f32x4{};

  for (int i = wave; i < count; i += kWaves) {
    const int64_t t = t0 + static_cast<int64_t>(i) * kTile;
    const int left = static_cast<int>(min(len - t, int64_t(kTile)));  // tokens of this tile
    const bool more = i + kWaves < count;
    f32x4 kscale[kBlocks], vscale[kBlocks];
    if constexpr (kCodes) {
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) kscale[k] = ks[k], vscale[k] = vs[k];
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        if (some[n]) {
          uint4 v = vr[k][n];
          if (left < kTile && k * 16 + row_of[n] >= left) v = uint4{};  // what a page holds past the sequence stays out
          *reinterpret_cast<uint4*>(lk + Rows<kRow>::key(k * 16 + row_of[n], piece_at[n])) = kr[k][n];
          *reinterpret_cast<uint4*>(lv + Rows<kRow>::value(k * 16 + row_of[n], piece_at[n])) = v;
        }
    if (more) {
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) base[k] = block_base(t + kWaves * kTile + k * 16);
      load_rows(c.k, base, kr);
      load_rows(c.v, base, vr);
      if constexpr (kCodes) load_scales(c.ks, base, ks), load_scales(c.vs, base, vs);
    }

    // scores: lane holds column col, tokens 16 k + 4 quarter + 0 .. 3
    f32x4 s[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      s[k] = f32x4{};
      if constexpr (kCodes) {
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          const uint4 w = *reinterpret_cast<const uint4*>(lk + Rows<kRow>::key(k * 16 + col, 4 * j + quarter));
          s[k] = mma(widen<QT>(w.x, w.y), q[2 * j], s[k]);
          s[k] = mma(widen<QT>(w.z, w.w), q[2 * j + 1], s[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < DP / 32; ++j)
          s[k] = mma(*reinterpret_cast<const H8<QT>*>(lk + Rows<kRow>::key(k * 16 + col, 4 * j + quarter)), q[j], s[k]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[k][e] *= kCodes ? factor * kscale[k][e] : factor;
        if (left < kTile && k * 16 + quarter * 4 + e >= left) s[k][e] = -INFINITY;
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int e = 1; e < 4 * kBlocks; ++e) top = fmaxf(top, s[e / 4][e % 4]);
    top = fmaxf(most, column_max(top));
    const float zero = top == -INFINITY ? 0.0f : top;  // nothing but -inf so far: exp of it is 0
    const float shrink = __builtin_amdgcn_exp2f(most - zero);
    most = top;
    H8<PT> hi, lo;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4 * kBlocks; ++e) {
      float p = __builtin_amdgcn_exp2f(s[e / 4][e % 4] - zero + kLift);
      sum += p;
      if constexpr (kCodes) {
        p *= vscale[e / 4][e % 4];
        if (left < kTile && e / 4 * 16 + quarter * 4 + e % 4 >= left) p = 0.0f;  // the scale may be NaN
      }
      const P r = static_cast<P>(p);
      hi[e] = r;
      lo[e] = static_cast<P>(p - static_cast<float>(r));
    }
    total = total * shrink + sum;
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
      o[d] *= shrink;
      H8<PT> v;
      if constexpr (kCodes) {
        const int r = (lane & 15) >> 1, row = (r & 4) * 4 + quarter * 4 + (r & 3);
        const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2*)(lv + Rows<kRow>::value(row, d) + (lane & 1) * 8));
        v = widen<PT>(w[0], w[1]);
      } else {
        const int r = quarter * 4 + ((lane & 15) >> 2), p = 2 * d + ((lane & 3) >> 1);
        union { i16x4 w[2]; H8<PT> v; } u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          u.w[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) i16x4*)(lv + Rows<kRow>::value(k * 16 + r, p) + (lane & 1) * 8));
        v = u.v;
      }
      o[d] = mma(v, hi, o[d]);
      o[d] = mma(v, lo, o[d]);
    }
  }
  total = column_sum(total);
  if (bad) total = __uint_as_float(0x7FC00000u);  // a table entry that names no page

  // join the waves: outputs of head `col`, columns 16 d + 4 quarter + 0 .. 3
  if (quarter == 0) sums[wave][0][col] = most, sums[wave][1][col] = total;
  __syncthreads();  // also: the tiles are done with
  float best = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) best = fmaxf(best, sums[w][0][col]);
  const float mine = most == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(most - best);
  static_assert(sizeof(lds) >= kWaves * kRows * DP * 4, "the outputs fit the tiles' room");
  float* part = reinterpret_cast<float*>(lds) + wave * kRows * DP;
#pragma unroll
  for (int d = 0; d < kOut; ++d) *reinterpret_cast<f32x4*>(part + col * DP + d * 16 + quarter * 4) = o[d] * mine;
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (DP / 4); i += 64 * kWaves) {
    const int r = i / (DP / 4), d = i % (DP / 4) * 4;
    if (d >= D) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sums[w][0][r]);
    float sum = 0.0f;
    f32x4 v{};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float m = sums[w][0][r], l = sums[w][1][r];
      sum += m == -INFINITY && l == 0.0f ? 0.0f : l * (m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top));
      v += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds) + (w * kRows + r) * DP + d);
    }
    const int64_t head = b * a.Hq + h * G + g0 + r;
    if (a.splits == 1) {
      Q* out = static_cast<Q*>(a.out) + head * D + d;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = static_cast<Q>(v[e] * inv);
    } else {
      *reinterpret_cast<f32x4*>(a.ws + (head * a.splits + split) * D + d) = v;
      if (d == 0) {
        float* ml = a.ws + a.B * a.Hq * a.splits * D + (head * a.splits + split) * 2;
        ml[0] = top;
        ml[1] = sum;
      }
    }
  }
}

// The pieces of a sequence joined, in piece order: a workgroup takes a head of a sequence.
template <int QT>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
  __shared__ float weight[256];
  __shared__ float part[4][kMaxHeadDim];
  __shared__ float red[8];
  typedef typename Elem<QT>::T Q;
  const int D = a.cache.D, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t head = block_index(), b = head / a.Hq;
  const int64_t room = a.W << a.cache.shift;
  int64_t len = a.lengths[b];
  len = len < 0 ? 0 : len > room ? room : len;
  const int64_t piece = piece_of(len, a.splits);
  const int n = len == 0 ? 1 : static_cast<int>((len + piece - 1) / piece);  // an empty sequence has an empty piece
  const float* ml = a.ws + a.B * a.Hq * a.splits * D + head * a.splits * 2;
  const float m = tid < n ? ml[2 * tid] : -INFINITY, l = tid < n ? ml[2 * tid + 1] : 0.0f;
  float top = m;
  for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  if (lane == 0) red[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float w = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  float sum = l != l ? l : l * w;  // NaN also where nothing else is
  for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
  if (lane == 0) red[4 + wave] = sum;
  weight[tid] = w;
  __syncthreads();
  sum = (red[4] + red[5]) + (red[6] + red[7]);
  const float* o = a.ws + head * a.splits * D;
  for (int d = lane * 4; d < D; d += 256) {
    f32x4 v{};
    for (int s = wave; s < n; s += 4)
      if (weight[s] != 0.0f) v += weight[s] * *reinterpret_cast<const f32x4*>(o + static_cast<int64_t>(s) * D + d);
    *reinterpret_cast<f32x4*>(&part[wave][d]) = v;
  }
  __syncthreads();
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (tid < D) {
    const float v = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    static_cast<Q*>(a.out)[head * D + tid] = static_cast<Q>(v * inv);
  }
}

template <int QT, int CT>
hipError_t attend(const AttendArgs& a, hipStream_t s) {
  const int G = a.Hq / a.cache.heads, tiles = (G + kRows - 1) / kRows;
  const dim3 grid(a.splits, a.cache.heads * tiles, static_cast<unsigned>(a.B));
  if (a.cache.D <= 64) hipLaunchKernelGGL((k_attend<QT, CT, 64>), grid, dim3(64 * kWaves), 0, s, a);
  else if (a.cache.D <= 128) hipLaunchKernelGGL((k_attend<QT, CT, 128>), grid, dim3(64 * kWaves), 0, s, a);
  else hipLaunchKernelGGL((k_attend<QT, CT, 256>), grid, dim3(64 * kWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((k_attend_join<QT>), long_grid(a.B * a.Hq), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Pieces a sequence is divided into: enough workgroups for two on every compute unit, none of fewer than a tile for every
// wave by the bound on the lengths, 256 at most.
int attend_splits(const CacheDesc& c, int64_t B, int Hq, int64_t bound) {
  const int64_t G = Hq / c.heads, units = B * c.heads * ((G + kRows - 1) / kRows);
  int64_t n = (2 * c.cus + units - 1) / units;
  const int64_t most = (bound + kWaves * kTile - 1) / (kWaves * kTile);
  n = n < most ? n : most;
  return static_cast<int>(n < 1 ? 1 : n > 256 ? 256 : n);
}

hipError_t launch_attend(const AttendArgs& a, int qt, hipStream_t s) {
  if (a.cache.type == DT_E4M3) return qt == DT_F16 ? attend<DT_F16, DT_E4M3>(a, s) : attend<DT_BF16, DT_E4M3>(a, s);
  return qt == DT_F16 ? attend<DT_F16, DT_F16>(a, s) : attend<DT_BF16, DT_BF16>(a, s);
}

}  // namespace qmm
