// attend.hip -- attention of one new token per sequence over the paged cache.
//
//   out[b, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - max),  j over the sequence's tokens
//
// Bound by reading the cache once: 64 sequences of 2048 to 8192 tokens, 32 / 8 heads of 128, bf16, take 252 us (5.4 TB/s), 2
// of up to 131072 in e4m3 80 us (4.7 TB/s), and one of 777 tokens the latency of two launches, 8.7 us.
//
// The query heads that share a key head are the 16 columns of one matrix product (more than 16: further row tiles), so a
// token's keys and values are read once for all of them.  A sequence is divided into `splits` pieces of whole 32-token
// tiles, a piece among the four or eight waves of a workgroup; each wave keeps its own running maximum, sum and output,
// which are joined in wave order through LDS and, where there is more than one piece, in piece order by a second small
// launch.
#include <algorithm>

#include "attn.hpp"

namespace qmm {

namespace {

constexpr int kWaves = 4, kTile = 32;  // waves of a workgroup (or twice as many), tokens of a wave's tile
constexpr int kRows = 16;              // query heads of a workgroup

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// A wave's tile in LDS, rows of ROW bytes in 16-byte pieces xored with a function of the row, so that the reads of one piece
// of 16 rows (keys) and of two neighbouring pieces of four rows (values, transposed on the way; of codes one piece of eight
// rows) use different banks.  Keys and values share it, and with it the pieces past D, which stay zeros.
template <int ROW>
__device__ __forceinline__ int tile_at(int row, int piece) {
  const int x = ROW >= 256 ? (2 * row | (row >> 3 & 1)) & 15 : ROW == 128 ? (row >> 1 ^ row >> 3) & 7 : (row >> 2) & 3;
  return row * ROW + (piece ^ x) * 16;
}

// LDS by byte address: the piece of the same row whose number differs by the bits of `by`, which is one xor.  `fresh` keeps
// the compiler from making the addresses of all pieces ahead of the loop, which would cost it a register each.
#define LDS_AS __attribute__((address_space(3)))
template <typename T>
__device__ __forceinline__ LDS_AS T* lds_piece(uint32_t at, int by) {
  return reinterpret_cast<LDS_AS T*>(at ^ static_cast<uint32_t>(by * 16));
}
__device__ __forceinline__ uint32_t lds_address(const void* p) { return reinterpret_cast<uintptr_t>((LDS_AS const void*)p); }
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// What the infinite values among columns d .. d + 3 of tokens t0 .. t1 - 1 of key head h add up to, 0 where there are none (an
// infinity of each sign, or a NaN: NaN): the largest 16 bits, taken as signed numbers and as unsigned ones, tell.  Four blocks of
// 16 tokens, which lie one after another in a page, are on their way at a time.  A rare sweep: 2 x 131072 tokens that hold an
// infinity take 573 us, not 188.
template <int QT>
__device__ __forceinline__ f32x4 infinite_values(const CacheDesc& c, const int32_t* table, int h, int64_t t0, int64_t t1, int d) {
  constexpr int kAhead = 4;
  constexpr int kInf = QT == DT_F16 ? 0x7C00 : 0x7F80;
  typedef int16_t I4 __attribute__((ext_vector_type(4)));
  typedef uint16_t U4 __attribute__((ext_vector_type(4)));
  const uint16_t* const values = reinterpret_cast<const uint16_t*>(c.v) + d;
  I4 above{};  // 0: nothing infinite
  U4 below{};
  for (int64_t t = t0; t < t1; t += 16 * kAhead) {
    U4 v[kAhead][16];
    int32_t page[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) page[k] = table[min(t + 16 * k, t1 - 1) >> c.shift];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // a page that is none makes the outputs NaN elsewhere; past the last token its row is read again
      const int64_t at = page[k] >= 0 && page[k] < c.pages ? page[k] : 0, first = min(t + 16 * k, t1 - 1);
      const int last = static_cast<int>(min(t1 - 1 - first, int64_t(15)));
      const int64_t row = ((at * c.heads + h) << c.shift) + (first & ((int64_t(1) << c.shift) - 1));
#pragma unroll
      for (int i = 0; i < 16; ++i) v[k][i] = *reinterpret_cast<const U4*>(values + (row + min(i, last)) * c.D);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        union { U4 u; I4 i; } x;
        x.u = v[k][i];
        above = __builtin_elementwise_max(above, x.i);
        below = __builtin_elementwise_max(below, x.u);
      }
  }
  f32x4 sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int up = above[e], down = below[e] - 0x8000;
    sum[e] = (up >= kInf ? INFINITY : 0.0f) + (down >= kInf ? -INFINITY : 0.0f);
    if (up > kInf || down > kInf) sum[e] = __uint_as_float(0x7FC00000u);
  }
  return sum;
}

// Whether two waves' registers find room in a SIMD: all but those of the widest 16-bit rows (64 x 4000 tokens of 16 / 4 heads of
// 192 119 -> 110 us, in e4m3 of 256 112 -> 81).
constexpr bool two_a_simd(int type, int D) { return D <= 192 || type == DT_E4M3; }

// QT: type of the queries and outputs; CT: QT or DT_E4M3; COLS: columns of the products, D rounded up to 32, 64, 96, 128, 192
// or 256.
//
// Scores are computed transposed, S^T = K Q^T (tokens x heads): a lane then holds, for one head, the scores of the eight
// tokens that its operand of O^T = V^T P^T takes, in the order in which that product's other operand, V^T, can be read
// from row-major LDS by transposing reads; the probabilities never leave their lane.
//
// P is fed to the matrix cores as the sum of two 16-bit numbers, its rounding and the rest (2^-17 of it in bf16): the
// cores have time to spare here, and one rounding of P to bf16 would add as much to the output's error as the output's
// own rounding.  With an e4m3 cache the tokens' scales of the values multiply P, in bf16, which has fp32's range.
template <int QT, int CT, int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES, two_a_simd(CT, COLS) ? 2 : 1) void k_attend(AttendArgs a) {
  constexpr bool kCodes = CT == DT_E4M3;
  constexpr int PT = kCodes ? DT_BF16 : QT;            // type of P and V on the matrix cores
  constexpr int DP = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;  // of a row in LDS
  constexpr int kSize = kCodes ? 1 : 2, kRow = DP * kSize;
  constexpr int kLoads = (COLS * kSize * 16 + 1023) / 1024;  // of a wave, for 16 tokens
  constexpr int kBlocks = kTile / 16, kOut = COLS / 16;
  constexpr float kLift = PT == DT_F16 ? 8.0f : 0.0f;  // P in fp16 times 2^8: small ones keep their bits
  typedef typename Elem<QT>::T Q;
  typedef typename Elem<PT>::T P;
  // a wave's tile, first its keys, then its values; at the end its outputs
  constexpr int kRoom = kTile * kRow > kRows * DP * 4 ? kTile * kRow : kRows * DP * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[WAVES][kRoom];
  __shared__ float sums[WAVES][2][kRows];

  const CacheDesc& c = a.cache;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const int D = c.D, H = c.heads, G = a.G;
  // Pieces vary slowest: workgroup i runs on die i mod 8, and where the bound is far above the lengths it is the first pieces that
  // there are (fastest, 64 x 8192 tokens of a table that reaches 131072 ran on one die of eight: 254 us, not 1539).
  const int split = blockIdx.z, h = a.tiles == 1 ? blockIdx.x : blockIdx.x / a.tiles, g0 = (blockIdx.x - h * a.tiles) * kRows;
  const int64_t b = blockIdx.y;
  const int rows = min(kRows, G - g0);                 // heads here
  const int64_t room = a.W << c.shift;
  const int64_t t0 = split * a.piece;
  const int32_t* table = a.table + b * a.W;
  // the first tile's pages are asked for before the length is known; a place past the table reads its last entry
  auto page_at = [&](int64_t t) { return table[min(t >> c.shift, a.W - 1)]; };
  int32_t page[kBlocks];
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) page[k] = a.W ? page_at(t0 + wave * kTile + k * 16) : 0;
  int64_t len = a.lengths[b];
  len = len < 0 ? 0 : len > room ? room : len;
  if (t0 >= len && split > 0) return;                  // the join reads the pieces that there are
  const int64_t t1 = split + 1 == a.splits ? len : min(len, t0 + a.piece);

  // queries: column col of the products, 8 columns of the head at a time
  constexpr int kSteps = kCodes ? DP / 32 : COLS / 32;  // of 32 columns; a piece of codes holds two
  H8<QT> q[kSteps];
  {
    const Q* p = static_cast<const Q*>(a.q.p) + b * a.q.st + (h * G + g0 + min(col, rows - 1)) * a.q.sh;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      // codes: a 16-byte piece of a row holds the operands of two steps
      const int d = kCodes ? (j / 2) * 64 + quarter * 16 + (j % 2) * 8 : j * 32 + quarter * 8;
      typedef H8<QT> Qu __attribute__((aligned(sizeof(Q))));
      q[j] = *reinterpret_cast<const Qu*>(p + (d < D ? d : 0));
      if (d >= D || col >= rows) q[j] = H8<QT>{};
    }
  }

  uint8_t* const mine_lds = lds[wave];
  // a lane's share of 16 tokens' rows, which lie one after another in a page: 16-byte pieces lane, lane + 64, ..
  const int pieces = D * kSize / 16;                   // of a row
  const int inverse = (65536 + pieces - 1) / pieces;   // i / pieces = i * inverse >> 16 for i < 512
  int at[kLoads], row_of[kLoads], piece_at[kLoads];
  bool some[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int i = n * 64 + lane;
    some[n] = i < 16 * pieces;
    row_of[n] = some[n] ? i * inverse >> 16 : 0;
    piece_at[n] = some[n] ? i - row_of[n] * pieces : 0;
    at[n] = some[n] ? i * 16 : 0;
  }
  if (D < DP) {  // columns past D: zeros, once
    for (int i = lane; i < kTile * kRow / 16; i += 64) reinterpret_cast<u32x4*>(mine_lds)[i] = u32x4{};
  }

  // where the lane reads: keys, a token a lane; values, eight bytes of which the transposing read makes its operand
  const int vrow = kCodes ? ((lane & 8) * 2 + quarter * 4 + (lane >> 1 & 3)) : quarter * 4 + ((lane & 15) >> 2);
  uint32_t key_at[kBlocks], value_at[kBlocks];  // (codes: one read for both blocks)
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    key_at[k] = lds_address(mine_lds) + tile_at<kRow>(k * 16 + col, quarter);
    value_at[k] = lds_address(mine_lds) + tile_at<kRow>(kCodes ? vrow : k * 16 + vrow, kCodes ? 0 : (lane & 3) >> 1) + (lane & 1) * 8;
  }

  const float factor = a.scale * 1.44269504088896340736f;
  const int count = t1 > t0 ? static_cast<int>((t1 - t0 + kTile - 1) / kTile) : 0;
  bool bad = false;
  u32x4 kr[kBlocks][kLoads], vr[kBlocks][kLoads];
  f32x4 ks[kBlocks], vs[kBlocks];

  // where a tile's 16-token block lies; what is past the sequence's last block is not looked at: any page will do
  auto block_base = [&](int64_t t, int64_t page) -> int64_t {
    if (page < 0 || page >= c.pages) bad |= t < len, page = 0;
    return ((page * H + h) << c.shift) + (t & ((int64_t(1) << c.shift) - 1));
  };
  auto load_rows = [&](const uint8_t* data, const int64_t (&base)[kBlocks], u32x4 (&r)[kBlocks][kLoads]) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        r[k][n] = *reinterpret_cast<const u32x4*>(data + base[k] * (D * kSize) + at[n]);
  };
  auto load_scales = [&](const float* data, const int64_t (&base)[kBlocks], f32x4 (&r)[kBlocks]) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) r[k] = *reinterpret_cast<const f32x4*>(data + base[k] + quarter * 4);
  };

  int64_t base[kBlocks];
  if (wave < count) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      base[k] = block_base(t0 + wave * kTile + k * 16, page[k]);
      page[k] = page_at(t0 + (wave + WAVES) * kTile + k * 16);
    }
    load_rows(c.k, base, kr);
    load_rows(c.v, base, vr);
    if constexpr (kCodes) load_scales(c.ks, base, ks), load_scales(c.vs, base, vs);
  }

  float most = -INFINITY, total = 0.0f;  // of column col, over the scores this wave has seen
  f32x4 o[kOut];
#pragma unroll
  for (int d = 0; d < kOut; ++d) o[d] = f32x4{};

  for (int i = wave; i < count; i += WAVES) {
    const int64_t t = t0 + static_cast<int64_t>(i) * kTile;
    const int left = static_cast<int>(min(len - t, int64_t(kTile)));  // tokens of this tile
    const bool more = i + WAVES < count;
    f32x4 kscale[kBlocks], vscale[kBlocks];
    if constexpr (kCodes) {
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) kscale[k] = ks[k], vscale[k] = vs[k];
    }
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        if (some[n]) *reinterpret_cast<u32x4*>(mine_lds + tile_at<kRow>(k * 16 + row_of[n], piece_at[n])) = kr[k][n];
    if (more) {
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) {
        base[k] = block_base(t + WAVES * kTile + k * 16, page[k]);
        page[k] = page_at(t + 2 * WAVES * kTile + k * 16);  // a tile ahead
      }
      load_rows(c.k, base, kr);
      if constexpr (kCodes) load_scales(c.ks, base, ks), load_scales(c.vs, base, vs);
    }

    // scores: lane holds column col, tokens 16 k + 4 quarter + 0 .. 3
    f32x4 s[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      s[k] = f32x4{};
      const uint32_t key = fresh(key_at[k]);
      if constexpr (kCodes) {
#pragma unroll
        for (int j = 0; j < kSteps / 2; ++j) {
          const u32x4 w = *lds_piece<const u32x4>(key, 4 * j);
          s[k] = mma(widen<QT>(w.x, w.y), q[2 * j], s[k]);
          s[k] = mma(widen<QT>(w.z, w.w), q[2 * j + 1], s[k]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
          s[k] = mma(*lds_piece<const H8<QT>>(key, 4 * j), q[j], s[k]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[k][e] *= kCodes ? factor * kscale[k][e] : factor;
        if (left < kTile && k * 16 + quarter * 4 + e >= left) s[k][e] = -INFINITY;
      }
    }
    // every read of the keys lies before this in the wave's order, as do the products that wait for them
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        if (some[n]) {
          u32x4 v = vr[k][n];
          if (left < kTile && k * 16 + row_of[n] >= left) v = u32x4{};  // what a page holds past the sequence stays out
          *reinterpret_cast<u32x4*>(mine_lds + tile_at<kRow>(k * 16 + row_of[n], piece_at[n])) = v;
        }
    if (more) load_rows(c.v, base, vr);
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
    const uint32_t value[kBlocks] = {fresh(value_at[0]), fresh(value_at[1])};
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
      o[d] *= shrink;
      H8<PT> v;
      if constexpr (kCodes) {
        const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(lds_piece<i32x2>(value[0], d));
        v = widen<PT>(w[0], w[1]);
      } else {
        union { i16x4 w[kBlocks]; H8<PT> v; } x;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k)
          x.w[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_piece<i16x4>(value[k], 2 * d));
        v = x.v;
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
  for (int w = 0; w < WAVES; ++w) best = fmaxf(best, sums[w][0][col]);
  const float mine = most == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(most - best);
  float* part = reinterpret_cast<float*>(mine_lds);
#pragma unroll
  for (int d = 0; d < kOut; ++d) *reinterpret_cast<f32x4*>(part + col * DP + d * 16 + quarter * 4) = o[d] * mine;
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (DP / 4); i += 64 * WAVES) {
    const int r = i / (DP / 4), d = i % (DP / 4) * 4;
    if (d >= D) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sums[w][0][r]);
    float sum = 0.0f;
    f32x4 v{};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const float m = sums[w][0][r], l = sums[w][1][r];
      sum += m == -INFINITY && l == 0.0f ? 0.0f : l * (m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top));
      v += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds[w]) + r * DP + d);
    }
    if constexpr (!kCodes) {  // (codes have no infinity)
      const f32x4 x = v * 0.0f;
      if (x[0] + x[1] + x[2] + x[3] != 0.0f && sum == sum) {
        // Infinite values: with rests of P that are 0 or negative they have become NaN.
        const f32x4 y = infinite_values<QT>(c, table, h, t0, t1, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = y[e] == 0.0f ? v[e] : y[e];
      }
    }
    const int64_t head = b * a.Hq + h * G + g0 + r;
    if (a.splits == 1) {
      Q* out = static_cast<Q*>(a.out) + head * D + d;
      const float inv = 1.0f / sum;  // no sum: zeros, whatever the values are
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = static_cast<Q>(sum == 0.0f ? 0.0f : v[e] * inv);
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

// over a wave, the same bits in every lane
template <typename F>
__device__ __forceinline__ float over_wave(float v, F f) {
  const auto g = [&](uint32_t a, uint32_t b) { return __float_as_uint(f(__uint_as_float(a), __uint_as_float(b))); };
  const uint32_t u = team<32>(__float_as_uint(v), g);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(g(r[0], r[1]));
}

// The pieces of a sequence joined: a workgroup takes a head of a sequence, teams of L lanes every (256 / L)-th piece, and
// the teams' sums are added in order.  Bound by latency: every wave looks at all maxima and sums itself, and the first pieces
// are asked for before it is known which there are.
template <int QT, int L>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a) {
  constexpr int kTeams = 256 / L, kAhead = 4;
  __shared__ f32x4 part[kTeams][L];
  typedef typename Elem<QT>::T Q;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int D = a.cache.D, tid = threadIdx.x, lane = tid & 63;
  const uint32_t index = static_cast<uint32_t>(block_index());  // B * Hq < 2^30
  if (index >= static_cast<uint32_t>(a.B * a.Hq)) return;       // the grid may have more workgroups than there are heads
  const int64_t head = index, b = index / static_cast<uint32_t>(a.Hq);
  const int team = tid / L, d = tid % L * 4;
  const float* const o = a.ws + head * a.splits * D + (d < D ? d : 0);
  const f32x2* const ml = reinterpret_cast<const f32x2*>(a.ws + a.B * a.Hq * a.splits * D) + head * a.splits;
  f32x4 x[kAhead];
  float at[kAhead];  // the pieces' maxima
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t p = min(s + i * kTeams, a.splits - 1);
      x[i] = *reinterpret_cast<const f32x4*>(o + p * D);
      at[i] = ml[p][0];
    }
  };
  f32x2 of[4];  // of pieces lane, lane + 64, ..: up to 256
#pragma unroll
  for (int k = 0; k < 4; ++k) of[k] = k * 64 < a.splits ? ml[min(k * 64 + lane, a.splits - 1)] : f32x2{-INFINITY, 0.0f};
  load(team);
  const int64_t room = a.W << a.cache.shift;
  int64_t len = a.lengths[b];
  len = len < 0 ? 0 : len > room ? room : len;
  // pieces that there are: one at least, of an empty sequence too
  const int n = static_cast<int>(min(max((len + a.piece - 1) / a.piece, int64_t(1)), int64_t(a.splits)));
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k * 64 + lane >= n) of[k] = f32x2{-INFINITY, 0.0f};
    top = fmaxf(top, of[k][0]);
  }
  top = over_wave(top, [](float u, float v) { return fmaxf(u, v); });
  const auto weight = [&](float m) { return m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top); };
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) sum += of[k][1] != of[k][1] ? of[k][1] : of[k][1] * weight(of[k][0]);  // NaN also where nothing else is
  sum = over_wave(sum, [](float u, float v) { return u + v; });
  f32x4 v{};
  for (int s = team; s < n; s += kAhead * kTeams) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const float w = weight(at[i]);
      if (s + i * kTeams < n) v += w * x[i];  // (also where w is 0: what is infinite or NaN there has been seen)
    }
    if (s + kAhead * kTeams < n) load(s + kAhead * kTeams);
  }
  part[team][tid % L] = v;
  __syncthreads();
  if (team == 0 && d < D) {
#pragma unroll
    for (int i = 1; i < kTeams; ++i) v += part[i][tid];
    const float inv = 1.0f / sum;
    Q* out = static_cast<Q*>(a.out) + head * D + d;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = static_cast<Q>(sum == 0.0f ? 0.0f : v[e] * inv);
  }
}

template <int QT, int CT, int COLS>
hipError_t attend(const AttendArgs& a, hipStream_t s) {
  const dim3 grid(a.cache.heads * a.tiles, static_cast<unsigned>(a.B), a.splits), threads(64 * a.waves);
  if constexpr (two_a_simd(CT, COLS)) {
    if (a.waves > kWaves) hipLaunchKernelGGL((k_attend<QT, CT, COLS, 2 * kWaves>), grid, threads, 0, s, a);
  }
  if (a.waves == kWaves) hipLaunchKernelGGL((k_attend<QT, CT, COLS, kWaves>), grid, threads, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  constexpr int L = COLS <= 64 ? 16 : COLS <= 128 ? 32 : 64;
  hipLaunchKernelGGL((k_attend_join<QT, L>), long_grid(a.B * a.Hq), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int QT, int CT>
hipError_t attend_of(const AttendArgs& a, hipStream_t s) {
  const int D = a.cache.D;
  if (D <= 32) return attend<QT, CT, 32>(a, s);
  if (D <= 64) return attend<QT, CT, 64>(a, s);
  if (D <= 96) return attend<QT, CT, 96>(a, s);
  if (D <= 128) return attend<QT, CT, 128>(a, s);
  return D <= 192 ? attend<QT, CT, 192>(a, s) : attend<QT, CT, 256>(a, s);
}

}  // namespace

// Pieces: so long that sequences of the bound's length give two workgroups a compute unit, as many as reside (four: 64 x
// 8192 tokens 251 -> 255 us, 2 x 131072 codes 78 -> 89: each piece begins with two round trips to memory), but not
// longer than 8192 tokens, so that one sequence much longer than the others does not end alone; whole tiles for every
// wave, and at most 256 a sequence.  Up to two tiles a wave are one piece: 200 tokens of 8 heads 7.3 us, in two pieces and
// joined 8.9; 777 tokens in pieces of one tile a wave 10.4, of two 12.0.
//
// Two pieces become one of a workgroup with twice the waves, and need no join: 32 x 300 tokens of 8 heads 16.2 -> 10.8 us,
// 32 x 2000 42.7 -> 38.1, 48 x 4000 119 -> 105, 64 x 10000 332 -> 298; in codes 14.5 -> 9.3, 29.4 -> 25.8, 64 -> 70 and 220
// -> 167.  So do, two by two, long ones of 16-bit caches (2 x 131072 tokens 140 -> 126 us, 8 x 16384 78 -> 73; codes 86 ->
// 86 and 49 -> 52; pieces below 512 tokens: 777 tokens 9.0 -> 10.3) where it is the sequences that are too few, not the
// pieces too long (64 x 20000 581 -> 599).
AttendSplit attend_split(const CacheDesc& c, int64_t B, int Hq, int64_t bound) {
  constexpr int64_t kMost = 8192, kStep = kWaves * kTile;
  const int64_t G = Hq / c.heads, units = B * c.heads * ((G + kRows - 1) / kRows);
  const int64_t few = (2 * c.cus + units - 1) / units;
  int64_t n = bound <= 2 * kStep ? 1 : std::min<int64_t>(std::max(few, (bound + kMost - 1) / kMost), 256);
  const bool twice = two_a_simd(c.type, c.D) && (n == 2 || (n > 2 && few > 1 && c.type != DT_E4M3 && bound >= 512 * n));
  const int64_t step = twice ? 2 * kStep : kStep;
  if (twice) n = (n + 1) / 2;
  const int64_t piece = std::max<int64_t>((bound + n * step - 1) / (n * step), 1) * step;
  return {static_cast<int>(std::max<int64_t>((bound + piece - 1) / piece, 1)), piece, twice ? 2 * kWaves : kWaves};
}

hipError_t launch_attend(AttendArgs a, int qt, hipStream_t s) {
  a.G = a.Hq / a.cache.heads;
  a.tiles = (a.G + kRows - 1) / kRows;
  if (a.cache.type == DT_E4M3) return qt == DT_F16 ? attend_of<DT_F16, DT_E4M3>(a, s) : attend_of<DT_BF16, DT_E4M3>(a, s);
  return qt == DT_F16 ? attend_of<DT_F16, DT_F16>(a, s) : attend_of<DT_BF16, DT_BF16>(a, s);
}

}  // namespace qmm
