// attn.hpp -- a decoder layer between its projections: norms and rotation of the heads, the paged key-value cache, and
// attention.  Device helpers, and the launch interface between the C ABI (attn_api.hip) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "f8.hpp"

namespace qmm {

enum { DT_E4M3 = 3 };  // QMM_E4M3: codes of a cache

constexpr int kMaxHeadDim = 256;
constexpr int64_t kMaxHeads = 1024;
constexpr int kMinPage = 16, kMaxPage = 4096;
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // tokens of a call, slots of a cache

// k, v [pages][heads][page][D], scales [pages][heads][page]; page = 1 << shift
struct CacheDesc {
  uint8_t *k, *v;
  float *ks, *vs;  // null unless type == DT_E4M3
  int type;
  int64_t pages;
  int shift, heads, D;
  int cus;
};

// x [T][heads][D]: strides in elements, the last axis contiguous
struct HeadRows {
  const void* p;
  int64_t st, sh;
};

struct HeadsArgs {
  HeadRows q, k, v;  // v.p is null unless the call writes a cache
  int64_t T;
  int Hq, H, D, R;
  const int32_t* positions;
  const float* inv_freq;     // null: no rotation
  const void *qw, *kw;       // null: no norm
  int wt;
  float eps;
  int interleaved;
  void *qo, *ko;             // contiguous
  CacheDesc cache;
  const int32_t* slots;
};
// xt: type of q, k, v; qt: of qo and ko.  With a.slots the keys and values go to a.cache instead of ko.
hipError_t launch_heads(const HeadsArgs& a, int xt, int qt, hipStream_t s);

hipError_t launch_cache_write(const CacheDesc& c, const HeadRows& k, const HeadRows& v, int xt, int64_t T,
                              const int32_t* slots, hipStream_t s);
hipError_t launch_cache_read(const CacheDesc& c, const int32_t* table, int64_t B, int64_t W, const int32_t* starts,
                             int64_t total, void* k, void* v, int ot, hipStream_t s);

struct AttendArgs {
  CacheDesc cache;
  HeadRows q;  // [B][Hq][D]
  int64_t B;
  int Hq;
  const int32_t* table;  // [B][W]
  int64_t W;
  const int32_t* lengths;
  float scale;  // of the scores
  void* out;    // [B][Hq][D]
  int splits;     // pieces of a sequence, of `piece` tokens each, the last of all that is left
  int64_t piece;
  int waves;      // of a workgroup
  int G, tiles;   // query heads of a key head, row tiles of them (set by the launch)
  float* ws;    // splits > 1: partial outputs [B][Hq][splits][D], then (maximum, sum) [B][Hq][splits]
};
struct AttendSplit {
  int splits;
  int64_t piece;
  int waves;
};
AttendSplit attend_split(const CacheDesc& c, int64_t B, int Hq, int64_t bound);
hipError_t launch_attend(AttendArgs a, int qt, hipStream_t s);

struct PromptArgs {
  HeadRows q, k, v;
  int64_t B, Tq, Tk;
  int Hq, H, D;
  const int32_t *q_starts, *k_starts;
  int causal;
  float scale;
  void* out;  // [Tq][Hq][D]
  int G, group;  // query heads of a key head; 1 << group of them share a workgroup (both set by the launch)
};
hipError_t launch_prompt(PromptArgs a, int dt, hipStream_t s);

#ifdef __HIPCC__

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Sum or maximum over the L lanes of a team (8, 16 or 32 neighbours), the same bits in every lane.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
template <int L, typename F>
__device__ __forceinline__ uint32_t team(uint32_t v, F f) {
  static_assert(L == 8 || L == 16 || L == 32, "teams of half a row, a row or two rows");
  if constexpr (L == 8) {
    v = f(v, dpp<0xB1>(v));   // lanes xor 1
    v = f(v, dpp<0x4E>(v));   // xor 2
    v = f(v, dpp<0x141>(v));  // 7 - lane, of eight: the other four hold one value
  } else {
    v = f(v, dpp<0x128>(v));  // rotations of a row of 16 lanes by 8, 4, 2, 1
    v = f(v, dpp<0x124>(v));
    v = f(v, dpp<0x122>(v));
    v = f(v, dpp<0x121>(v));
    if constexpr (L == 32) {
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      v = f(r[0], r[1]);
    }
  }
  return v;
}
template <int L>
__device__ __forceinline__ float team_sum(float v) {
  return __uint_as_float(team<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  return team<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// The number of i < n for which f holds, f first true and then false: a search by 64 lanes at a time, the same in every
// lane of the wave.  (Of an f that is not so, some number 0 .. n.)
template <typename F>
__device__ __forceinline__ int64_t count_first(int64_t n, F f) {
  const int lane = threadIdx.x & 63;
  int64_t at = 0;
  while (n > 0) {
    const int64_t step = (n + 63) / 64, i = lane * step;
    const int some = __popcll(__ballot(i < n && f(at + i)));
    if (some == 0) break;
    const int64_t known = (some - 1) * step + 1;  // f holds up to here
    at += known;
    n = min(n - known, step - 1);
  }
  return at;
}

#endif  // __HIPCC__

}  // namespace qmm
