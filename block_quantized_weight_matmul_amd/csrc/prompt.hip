// prompt.hip -- attention of whole prompts: packed sequences, grouped heads, causal.
//
//   out[i, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q_i.k_j - max),  j <= i + (m - n)  (m keys, n queries)
//
// Bound by the matrix cores, of which the card's power allows a part: 8192 tokens, 32 / 8 heads of 128, bf16, take 505 us in a
// long run, 1.09 PFLOP/s at 1.9 GHz (with zeros for inputs 440 us; in the first tenth of a second after idling 550 to 610), 16
// packed prompts of 50 to 1024 queries with up to 1024 keys before them 168 us (180 to 205); of many short sequences by memory:
// 128 of 64 tokens 38 us, 4.4 TB/s.
//
// A workgroup takes 128 rows, queries of up to four heads that share a key head, and sweeps the keys they may see in tiles
// of 64: keys and values go straight into LDS, two tiles deep, while the waves, 32 queries of one head each, work on the
// tile before.  Where such workgroups are few, each has twice the waves and sweeps two tiles at a time.
#include <algorithm>
#include <type_traits>

#include "attn.hpp"

namespace qmm {

namespace {

typedef __attribute__((address_space(3))) void lds_void;

constexpr int kRows = 128, kWaves = 4;  // of a workgroup: queries times heads, waves that they are divided among
constexpr int kKeys = 64;               // of a tile
constexpr int kCus = 256;               // compute units of the card (a call without a handle knows no other number)

template <int QT> struct Half8 { typedef typename Elem<QT>::T V __attribute__((ext_vector_type(8))); };
template <int QT> using H8 = typename Half8<QT>::V;

__device__ __forceinline__ f32x16 mma(H8<DT_F16> a, H8<DT_F16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(H8<DT_BF16> a, H8<DT_BF16> b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}
// 16 bytes a lane straight into LDS: lane i's at dst + 16 i (dst: the wave's base)
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, voff, 0, 0, 0);
}

// Four rows' elements of a column, transposed on the way from LDS.  `restrict`: the compiler takes a read through a pointer
// that it knows nothing of for one of what is on its way into LDS, and waits for the next tile.
__device__ __forceinline__ i16x4 read_transposed(__attribute__((address_space(3))) i16x4* __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

// 16-bit values with zeros for infinities and NaN
template <int DT>
__device__ __forceinline__ i16x4 finite_or_zero(i16x4 v) {
  constexpr short kExponent = DT == DT_F16 ? 0x7C00 : 0x7F80;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (v[i] & kExponent) == kExponent ? short(0) : v[i];
  return v;
}

// the larger (the sum) of a value and the one of the lane 32 further
__device__ __forceinline__ float both_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float both_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// scores so large that the rounding of the maximum, which the fma of a score does not share, would show
__device__ __forceinline__ bool far_out(float most) { return fabsf(most) > 0x1p20f && fabsf(most) < INFINITY; }

// The lane's number (or the like) as a value that the compiler knows nothing of, so that addresses are made where they are used:
// kept over the loop they would cost it registers that it does not have.
__device__ __forceinline__ int again(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A tile of 64 rows of DP columns in LDS, in 16-byte pieces xored with a function of the row: 16 lanes that read one piece
// of 16 rows (keys), and 32 that read four neighbouring pieces of four rows (values), use every bank once.
template <int DP>
struct Tile {
  static constexpr int kRow = DP * 2, kPieces = kRow / 16;
  __device__ static __forceinline__ int key(int row, int piece) { return piece ^ (DP >= 128 ? row & 15 : row >> 1 & 7); }
  __device__ static __forceinline__ int value(int row, int piece) {
    return piece ^ (DP >= 128 ? 4 * (row & 3) : 4 * (row >> 1 & 1));
  }
};

// The tile of queries of a workgroup.
struct Work {
  int64_t q0, k0;  // first row of the sequence's queries, of its keys
  int n, m;        // their numbers, up to 2^30
  int first;       // first query of the tile
  bool some;
};
// Starts are taken as they come, kept within [0, total]: no row outside the tensors is touched whatever they hold.
__device__ __forceinline__ int64_t start_at(const int32_t* s, int64_t i, int64_t total) {
  const int64_t v = s[i];
  return v < 0 ? 0 : v > total ? total : v;
}
// Sequence b's tiles, of 1 << shift queries, have the indexes from (start_b >> shift) + b on: the next one's begin late enough
// for all of them, one index or none is left over, and no sum over the sequences before is needed.
__device__ __forceinline__ Work find_work(const PromptArgs& a, int64_t index, int shift) {
  Work w{};
  int64_t b;
  if (a.B < 64) {  // all starts in the wave's registers: one round trip to memory, not two
    const int lane = threadIdx.x & 63, at = min(lane, static_cast<int>(a.B));
    const int qs = static_cast<int>(start_at(a.q_starts, at, a.Tq)), ks = static_cast<int>(start_at(a.k_starts, at, a.Tk));
    const int i = __popcll(__ballot(lane < a.B && (qs >> shift) + lane <= index)) - 1;
    if (i < 0) return w;
    w.q0 = __builtin_amdgcn_readlane(qs, i);
    w.n = __builtin_amdgcn_readlane(qs, i + 1) - static_cast<int>(w.q0);
    w.k0 = __builtin_amdgcn_readlane(ks, i);
    w.m = max(__builtin_amdgcn_readlane(ks, i + 1) - static_cast<int>(w.k0), 0);
    b = i;
  } else {
    b = count_first(a.B, [&](int64_t i) { return (start_at(a.q_starts, i, a.Tq) >> shift) + i <= index; }) - 1;
    if (b < 0) return w;
    w.q0 = start_at(a.q_starts, b, a.Tq);
    w.n = static_cast<int>(start_at(a.q_starts, b + 1, a.Tq) - w.q0);
    w.k0 = start_at(a.k_starts, b, a.Tk);
    w.m = static_cast<int>(max(start_at(a.k_starts, b + 1, a.Tk) - w.k0, int64_t(0)));
  }
  const int all = (w.n + (1 << shift) - 1) >> shift, mine = static_cast<int>(index - ((w.q0 >> shift) + b));
  // the last tile, which sees the most keys, first
  w.first = (all - 1 - mine) << shift;
  w.some = w.n > 0 && mine >= 0 && mine < all;  // (below 0 only where starts decrease)
  return w;
}

// DT: type of everything but the sums; COLS: columns of the products, D rounded up to 32, 64, 96, 128, 192 or 256 (of 64,
// 128 or 256 alone: 4096 tokens of 32 heads of 80 117 -> 129 us, 32 heads of 32 74 -> 84, 16 heads of 160 146 -> 171).
//
// Scores are computed transposed, S^T = K Q^T (keys x queries): a lane then holds, for one query, the scores of the keys
// that its operand of O^T = V^T P^T takes, in the order in which that product's other operand, V^T, can be read from
// row-major LDS by transposing reads; the probabilities never leave their lane, and a row's maximum takes one exchange
// between two lanes.
//
// P is rounded to DT once: up to 2^-8 of a term in bf16 (2^-11 in fp16), with independent signs, which stays below the output's
// own rounding and adds to it: against fp64 2.3e-3 of the root mean square, not 1.7e-3 (16 packed prompts), 2.1e-3, not 1.6e-3
// (8192 tokens).  P as two numbers leaves the output's rounding alone and takes half as many products again: 168 -> 222 us, 505
// -> 696.
//
// PARTS: as often a workgroup has four waves for its rows, and each four take every PARTS-th tile of keys.
template <int DT, int COLS, int PARTS>
__global__ __launch_bounds__(64 * kWaves * PARTS, COLS > 128 ? 1 : 2) void k_prompt(PromptArgs a) {
  constexpr int DP = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;  // of a row in LDS
  typedef typename Elem<DT>::T T;
  typedef Tile<DP> L;
  constexpr int kBytes = kKeys * L::kRow, kLoads = kBytes / 1024 / kWaves, kOut = COLS / 32;
  constexpr int kPer = 64 / L::kPieces > 0 ? 64 / L::kPieces : 1;  // rows of a load of a wave
  static_assert(L::kPieces <= 64, "a load holds whole rows");
  // The maximum that P is relative to is moved, and with it every output so far, only where a score exceeds it by 2^kSlack:
  // P is at most 2^(kLift + kSlack), and in fp16 keeps small probabilities' bits by 2^kLift.
  constexpr float kSlack = 8.0f, kLift = DT == DT_F16 ? 6.0f : 0.0f;
  // One array: with a second one the compiler tells what is loaded into LDS apart by its variable, and makes every read of
  // `lds` wait for the loads of the next tile.
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * kBytes * PARTS + 16];
  int& met = *reinterpret_cast<int*>(lds + 4 * kBytes * PARTS);

  // key heads vary fastest: workgroup i runs on die i mod 8, so that a key head's rows stay in one die's L2 cache
  const int share = blockIdx.x / a.H, kv = blockIdx.x - share * a.H;
  const int rows = kRows >> a.group;  // queries of a head
  const Work w = find_work(a, static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y, __builtin_ctz(kRows) - a.group);
  if (!w.some) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6 & kWaves - 1);
  const int part = PARTS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * kWaves));
  uint8_t* const room = lds + part * 4 * kBytes;  // of this part's waves
  const int head0 = kv * a.G + (share << a.group), head = head0 + (wave & (1 << a.group) - 1);
  const float factor = a.scale * 1.44269504088896340736f;
  const int shift = w.m - w.n;  // query i sees keys 0 .. i + shift
  const int i0 = w.first + (wave >> a.group) * 32;
  const int last = min(w.n, w.first + rows) - 1;
  int end = a.causal ? min(w.m, last + shift + 1) : w.m;  // keys that some row here sees
  if (end < 0) end = 0;
  const int mine = a.causal ? min(w.m, i0 + 31 + shift + 1) : w.m;   // of this wave's rows
  const int whole = a.causal ? min(w.m, i0 + shift + 1) : w.m;       // keys that all of its rows see
  const int whole_all = a.causal ? min(w.m, w.first + shift + 1) : w.m;
  const int count = (end + kKeys - 1) / kKeys;
  if (threadIdx.x == 0) met = 0;

  // loads of a tile: this wave's lanes take pieces of rows (wave * kLoads + n) * kPer ..; a lane whose piece lies past D
  // reads past the descriptor's end, which gives zeros, as do rows past the last key
  const uint32_t kst = static_cast<uint32_t>(a.k.st * 2), vst = static_cast<uint32_t>(a.v.st * 2);
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int n = 0; n < kLoads; ++n) {
    const int row = (wave * kLoads + n) * kPer + lane / L::kPieces, p = lane % L::kPieces;
    const int kp = L::key(row, p), vp = L::value(row, p);  // the xor is its own inverse
    koff[n] = kp * 8 < a.D ? row * kst + kp * 16 : 0x7FFFFFF0u;
    voff[n] = vp * 8 < a.D ? row * vst + vp * 16 : 0x7FFFFFF0u;
  }
  const T* const kbase = static_cast<const T*>(a.k.p) + w.k0 * a.k.st + kv * a.k.sh;
  const T* const vbase = static_cast<const T*>(a.v.p) + w.k0 * a.v.st + kv * a.v.sh;
  auto load_tile = [&](int i, int buffer) {
    const int64_t j = static_cast<int64_t>(i) * kKeys;
    const uint32_t left = min(w.m - i * kKeys, kKeys);
    const __amdgpu_buffer_rsrc_t kr = rsrc(kbase + j * a.k.st, (left - 1) * kst + a.D * 2);
    const __amdgpu_buffer_rsrc_t vr = rsrc(vbase + j * a.v.st, (left - 1) * vst + a.D * 2);
    uint8_t* d = room + buffer * 2 * kBytes + wave * kLoads * 1024;
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load_lds16(kr, d + n * 1024, koff[n]);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) load_lds16(vr, d + kBytes + n * 1024, voff[n]);
  };

  // Queries and outputs pass through the second tile's room, so that their rows are read and written whole (not as the
  // products have them, 16 or 32 bytes of a row at a time: 128 sequences of 64 tokens 48 -> 37 us, 16 of 1000 203 -> 191): a
  // wave's 32 rows, 16-byte piece lane % kPieces of row lane / kPieces and of every kPer-th after it.
  typedef H8<DT> H8u __attribute__((aligned(sizeof(T))));
  const auto rows_at = [&](uint8_t* base, int row, int piece) { return base + row * L::kRow + L::key(row, piece) * 16; };
  H8<DT> q[COLS / 16];
  {
    const int lane = again(threadIdx.x & 63), col = lane & 31, half = lane >> 5;
    uint8_t* const own = room + 2 * kBytes + wave * 32 * L::kRow;
    const T* const p = static_cast<const T*>(a.q.p) + w.q0 * a.q.st + head * a.q.sh;
    const int piece = lane % L::kPieces;
    constexpr int kAtOnce = 32 / kPer < 8 ? 32 / kPer : 8;  // (more of 256 columns take registers from the loop)
#pragma unroll
    for (int n0 = 0; n0 < 32 / kPer; n0 += kAtOnce) {
      H8<DT> x[kAtOnce];
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n) {
        const int row = (n0 + n) * kPer + lane / L::kPieces;
        x[n] = *reinterpret_cast<const H8u*>(p + min(i0 + row, w.n - 1) * a.q.st + (piece * 8 < a.D ? piece * 8 : 0));
        if (piece * 8 >= a.D) x[n] = H8<DT>{};
      }
      if (n0 + kAtOnce >= 32 / kPer && part < count) load_tile(part, 0);
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n)
        *reinterpret_cast<H8<DT>*>(rows_at(own, (n0 + n) * kPer + lane / L::kPieces, piece)) = x[n];
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < COLS / 16; ++j) q[j] = *reinterpret_cast<const H8<DT>*>(rows_at(own, col, 2 * j + half));
  }

  float most = -INFINITY, zero = 0.0f, total = 0.0f;  // of query col; the sum over this lane's keys only
  bool huge = false;
  f32x16 o[kOut];
#pragma unroll
  for (int d = 0; d < kOut; ++d) o[d] = f32x16{};

  auto sweep = [&](auto careful) {
    constexpr bool kCareful = decltype(careful)::value;
    for (int n = 0; n * PARTS < count; ++n) {
      const int i = n * PARTS + part;
      const int lane = kCareful ? again(threadIdx.x & 63) : threadIdx.x & 63;
      const int col = lane & 31, half = lane >> 5;
      if constexpr (kCareful) {
        __syncthreads();  // the tile before, and the probabilities beside it, are done with
        if (i < count) load_tile(i, n & 1);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this tile's loads, issued a tile ago
      __syncthreads();
      if (!kCareful && i + PARTS < count) load_tile(i + PARTS, n + 1 & 1);
      if (PARTS > 1 && i >= count) continue;
      const uint8_t* const lk = room + (n & 1) * 2 * kBytes;
      const uint8_t* const lv = lk + kBytes;
      const int j0 = i * kKeys;
      if (!kCareful && a.causal && j0 + kKeys > whole_all) {  // rows see parts of this tile: infinities and NaN among its values
        uint32_t worst = 0;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
          const uint4 x = *reinterpret_cast<const uint4*>(lv + (wave * kLoads + n) * 1024 + lane * 16);
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) worst = max(worst, max(y[e] << 1 & 0xFFFFu, y[e] >> 15 & 0xFFFEu));
        }
        if (__any(worst >= (DT == DT_F16 ? 0xF800u : 0xFF00u))) met = 1;
      }
      if (j0 >= mine) continue;  // this wave's rows see nothing of it (nor of later ones)

      f32x16 s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s[k] = f32x16{};
        const int row = k * 32 + col;
#pragma unroll
        for (int j = 0; j < COLS / 16; ++j)
          s[k] = mma(*reinterpret_cast<const H8<DT>*>(lk + row * L::kRow + L::key(row, 2 * j + half) * 16), q[j], s[k]);
      }
      // four reads ahead of the products (one or two, as the compiler has it: 2048 queries of 8 heads 43.0 -> 40.7 us, 8192 of 32
      // 526 -> 519; eight: 41.9)
      __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
      for (int n = 0; n < COLS / 8 - 4; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
      if (j0 + kKeys > whole) {
        const int seen = min(w.m, a.causal ? i0 + col + shift + 1 : w.m) - j0;  // keys of the tile that row col sees
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (k * 32 + e / 4 * 8 + half * 4 + e % 4 >= seen) s[k][e] = -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, s[k][e]);
      top = both_max(top) * factor;  // factor > 0
      // The votes are branches: a row's maximum moves, and its scores are scaled ahead, by what the row itself sees, so that its
      // output has the same bits whatever the rows beside it see.
      if (__any(top > most + kSlack)) {
        top = top > most + kSlack ? top : most;
        zero = top == -INFINITY ? 0.0f : top;  // nothing but -inf so far: exp of it is 0
        const float shrink = __builtin_amdgcn_exp2f(most - zero);
        most = top;
        total *= shrink;
#pragma unroll
        for (int d = 0; d < kOut; ++d) o[d] *= shrink;
        huge = __any(far_out(most));
      }
      float f = factor;
      if (huge) {
        const bool own = far_out(most);
#pragma unroll
        for (int k = 0; k < 2; ++k) s[k] *= own ? factor : 1.0f;
        f = own ? 1.0f : factor;
      }
      const bool clean = kCareful && j0 + kKeys > whole;
      if constexpr (kCareful) {
        if (clean) {
          // Key by key, the values that are not finite, each added to the rows that see it; the products below take zeros for
          // them.  The probabilities pass through the other tile's room.
          T* const pw = reinterpret_cast<T*>(room + (n + 1 & 1) * 2 * kBytes) + wave * kKeys * 32;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              pw[(k * 32 + e / 4 * 8 + half * 4 + e % 4) * 32 + col] =
                  static_cast<T>(__builtin_amdgcn_exp2f(fmaf(s[k][e], f, kLift - zero)));
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          const int seen = min(w.m, i0 + col + shift + 1) - j0;
#pragma unroll 1
          for (int j = 0; j < kKeys; ++j) {
            if (j >= seen) continue;
            const float x = static_cast<float>(pw[j * 32 + col]);
#pragma unroll
            for (int d = 0; d < kOut * 4; ++d) {
              typedef T V4 __attribute__((ext_vector_type(4)));
              const V4 v = *reinterpret_cast<const V4*>(lv + j * L::kRow + L::value(j, d) * 16 + half * 8);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = static_cast<float>(v[e]);
                if (!(fabsf(y) < INFINITY)) o[d / 4][d % 4 * 4 + e] = fmaf(x, y, o[d / 4][d % 4 * 4 + e]);
              }
              __builtin_amdgcn_sched_barrier(0);  // a read at a time: registers again
            }
          }
        }
      }
      // ahead of the SIMD's other wave while the matrix cores have work (8192 tokens 538 -> 527 us)
      __builtin_amdgcn_s_setprio(1);
      // Step by step, so that the next step's exponentials run beside this one's products (all of P first: 2048 queries of 8 heads
      // 45.0 us, not 43.0).  Key slots of step u: 16 u + 4 half + 0 .. 3 and 8 more, as the scores lie
      H8<DT> vf[2][kOut];
      auto read_values = [&](int u) {
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
          union { i16x4 w[2]; H8<DT> v; } x;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = u * 16 + e * 8 + half * 4 + (lane & 15) / 4, piece = d * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1);
            x.w[e] = read_transposed(
                (__attribute__((address_space(3))) i16x4*)(lv + row * L::kRow + L::value(row, piece) * 16 + (lane & 1) * 8));
            if (clean) x.w[e] = finite_or_zero<DT>(x.w[e]);
          }
          vf[u & 1][d] = x.v;
        }
      };
      read_values(0);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        H8<DT> p;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __builtin_amdgcn_exp2f(fmaf(s[u / 2][u % 2 * 8 + e], f, kLift - zero));
          total += x;
          p[e] = static_cast<T>(x);
        }
        if (u < 3) read_values(u + 1);
#pragma unroll
        for (int d = 0; d < kOut; ++d) o[d] = mma(vf[u & 1][d], p, o[d]);
      }
      __builtin_amdgcn_s_setprio(0);
    }
  };
  sweep(std::false_type{});
  __syncthreads();
  if (met) {
    // An infinity or a NaN among the values of a tile which some of the rows see in part: a product of matrices has added 0 *
    // Inf = NaN to the others.  Once more, with such values of such tiles left to the rows that see them: the others' outputs
    // have the bits that any finite value there would have given them.
    most = -INFINITY, zero = total = 0.0f;
    huge = false;
#pragma unroll
    for (int d = 0; d < kOut; ++d) o[d] = f32x16{};
    sweep(std::true_type{});
    __syncthreads();
  }
  total = both_sum(total);
  if constexpr (PARTS == 2) {  // the second part's sums to the first
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(lds) + wave * 128 + lane;
    float* const rest = reinterpret_cast<float*>(lds + 4 * kBytes) + wave * kOut * 16 * 64 + lane;
    if (part) {
      sums[0] = most, sums[64] = total;
#pragma unroll
      for (int d = 0; d < kOut * 16; ++d) rest[d * 64] = o[d / 16][d % 16];
    }
    __syncthreads();
    if (part) return;
    const float top = fmaxf(most, sums[0]);
    const float w0 = most == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(most - top);
    const float w1 = sums[0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(sums[0] - top);
    total = total * w0 + sums[64] * w1;
#pragma unroll
    for (int d = 0; d < kOut * 16; ++d) o[d / 16][d % 16] = o[d / 16][d % 16] * w0 + rest[d * 64] * w1;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  if (__any(total == 0.0f)) {  // no sum: zeros, whatever the values are
#pragma unroll
    for (int d = 0; d < kOut; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = total == 0.0f ? 0.0f : o[d][e];
  }
  uint8_t* const own = lds + 2 * kBytes + wave * 32 * L::kRow;
  const int lane1 = again(threadIdx.x & 63), col1 = lane1 & 31, half1 = lane1 >> 5;
#pragma unroll
  for (int d = 0; d < kOut; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      typedef T V4 __attribute__((ext_vector_type(4)));
      V4 v;
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = static_cast<T>(o[d][4 * e + x] * inv);
      *reinterpret_cast<V4*>(rows_at(own, col1, d * 4 + e) + half1 * 8) = v;
    }
  T* const out = static_cast<T*>(a.out) + (w.q0 * a.Hq + head) * a.D;
#pragma unroll
  for (int n = 0; n < 32 / kPer; ++n) {
    const int row = n * kPer + lane1 / L::kPieces, piece = lane1 % L::kPieces;
    const H8<DT> v = *reinterpret_cast<const H8<DT>*>(rows_at(own, row, piece));
    if (i0 + row < w.n && piece * 8 < a.D)
      *reinterpret_cast<H8u*>(out + static_cast<int64_t>(i0 + row) * a.Hq * a.D + piece * 8) = v;
  }
}

template <int DT, int COLS, int PARTS>
hipError_t launch(const PromptArgs& a, hipStream_t s) {
  const int64_t tiles = a.Tq / (kRows >> a.group) + a.B, y = std::min<int64_t>(tiles, 65535);  // their indexes (find_work)
  const dim3 grid(a.Hq >> a.group, static_cast<unsigned>(y), static_cast<unsigned>((tiles + y - 1) / y));
  hipLaunchKernelGGL((k_prompt<DT, COLS, PARTS>), grid, dim3(64 * kWaves * PARTS), 0, s, a);
  return hipGetLastError();
}

// Few workgroups: the longest sweep is what a call waits for, and two parts halve it (a workgroup then has a compute unit to
// itself).  Where a unit is left for each and the sequences have a few tiles: 512 tokens of 16 heads 14.0 -> 13.1 us, 2048
// of 8 heads 40.5 -> 32.7, 4096 75 -> 60; 128 of 16 heads 7.6 -> 8.2, 16 of those 10.4 -> 16.0.  And where two would share a
// unit, one of which sweeps much longer than the other, in long sequences without much of a prefix: 2048 tokens of 32 heads
// 53.7 -> 47.1, 8192 of 8 180 -> 146; four of 512 of 32 heads 21.6 -> 26.2.  More workgroups than that keep the units busy:
// 4096 tokens of 32 heads 139 -> 152.  (Lengths by their mean, all that the host knows: a long sequence among many short ones
// counts as short.)
template <int DT, int COLS>
hipError_t prompt(const PromptArgs& a, hipStream_t s) {
  if constexpr (COLS <= 128) {
    const int64_t rows = a.Tq * a.Hq;
    if (rows <= kRows * kCus ? a.Tk >= 256 * a.B
                             : rows <= 2 * kRows * kCus && a.causal && a.Tk >= 1024 * a.B && a.Tk < 2 * a.Tq)
      return launch<DT, COLS, 2>(a, s);
  }
  return launch<DT, COLS, 1>(a, s);
}

template <int DT>
hipError_t prompt_of(const PromptArgs& a, hipStream_t s) {
  if (a.D <= 32) return prompt<DT, 32>(a, s);
  if (a.D <= 64) return prompt<DT, 64>(a, s);
  if (a.D <= 96) return prompt<DT, 96>(a, s);
  if (a.D <= 128) return prompt<DT, 128>(a, s);
  return a.D <= 192 ? prompt<DT, 192>(a, s) : prompt<DT, 256>(a, s);
}

}  // namespace

hipError_t launch_prompt(PromptArgs a, int dt, hipStream_t s) {
  // The query heads of a key head share a workgroup, four or two where their number allows it, so that its queries, 32 or 64
  // of each, end later in fewer tiles that they see in part.
  a.G = a.Hq / a.H;
  a.group = a.G % 4 == 0 ? 2 : a.G % 2 == 0 ? 1 : 0;
  return dt == DT_F16 ? prompt_of<DT_F16>(a, s) : prompt_of<DT_BF16>(a, s);
}

}  // namespace qmm
