// attn_api.hip -- the C ABI of the head norms, the paged cache and attention (include/qmm.h): argument checks, device
// checks and dispatch.  No device memory is allocated here and nothing synchronises.
#include <math.h>
#include <string.h>

#include <new>

#include "api_common.hpp"
#include "attn.hpp"

struct qmm_cache {
  qmm::CacheDesc d;
  int device;
};

namespace {

using qmm::aligned;
using qmm::check_dtype;
using qmm::check_ptr;
using qmm::check_range;
using qmm::check_ws;
using qmm::fail;
using qmm::hip_fail;
using qmm::HeadRows;
using qmm::ll;
using qmm::ok;
using qmm::size_of;
using qmm::stream_of;

constexpr int64_t kMaxStride = int64_t(1) << 40;

qmm_status check_device(const qmm_cache* h) {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev != h->device) return fail(QMM_E_DEVICE, "current device %d is not the cache's device %d", dev, h->device);
  return QMM_OK;
}

// rows that are only read may be shared by heads (stride 0) and lie in any order
qmm_status check_rows(const HeadRows& r, int type, const char* what) {
  QMM_TRY(check_ptr(r.p, size_of(type), what));
  if (r.st < 0 || r.sh < 0 || r.st > kMaxStride || r.sh > kMaxStride)
    return fail(QMM_E_SHAPE, "strides of %s outside [0, 2^40]", what);
  return QMM_OK;
}

qmm_status check_head(int64_t D) {
  QMM_TRY(check_range(D, 16, qmm::kMaxHeadDim, "D"));
  return D % 16 == 0 ? QMM_OK : fail(QMM_E_SHAPE, "D=%lld is not a multiple of 16", static_cast<ll>(D));
}

// norms and rotation: weights, angles, and the tensors that the call reads and writes
qmm_status check_heads(const qmm::HeadsArgs& a, int xt, int64_t Hq, int64_t H, int64_t D, int64_t R) {
  QMM_TRY(check_dtype(xt, "input"));
  QMM_TRY(check_dtype(a.wt, "weight"));
  QMM_TRY(check_range(a.T, 0, qmm::kMaxTokens, "T"));
  QMM_TRY(check_range(Hq, 0, qmm::kMaxHeads, "query heads"));
  QMM_TRY(check_range(H, 0, qmm::kMaxHeads, "key heads"));
  if (Hq + H == 0) return fail(QMM_E_SHAPE, "no heads");
  QMM_TRY(check_head(D));
  if (R < 0 || R > D || R % 8) return fail(QMM_E_SHAPE, "R=%lld is not a multiple of 8 up to D", static_cast<ll>(R));
  if (!(a.eps >= 0.0f) || a.eps > 3e38f) return fail(QMM_E_ARG, "eps must be finite and not negative");
  if (a.interleaved != 0 && a.interleaved != 1) return fail(QMM_E_ARG, "interleaved must be 0 or 1");
  if (a.T == 0) return QMM_OK;
  if (Hq) QMM_TRY(check_rows(a.q, xt, "q"));
  if (H) QMM_TRY(check_rows(a.k, xt, "k"));
  if (R) {
    QMM_TRY(check_ptr(a.positions, 4, "positions"));
    QMM_TRY(check_ptr(a.inv_freq, 4, "inv_freq"));
  }
  if (a.qw && !aligned(a.qw, size_of(a.wt))) return fail(QMM_E_ALIGN, "q_weight must be element-aligned");
  if (a.kw && !aligned(a.kw, size_of(a.wt))) return fail(QMM_E_ALIGN, "k_weight must be element-aligned");
  return QMM_OK;
}

qmm::HeadsArgs heads_args(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh, int64_t T,
                          int64_t Hq, int64_t H, int64_t D, const void* qw, const void* kw, int wt, float eps,
                          const int32_t* positions, const float* inv_freq, int64_t R, int interleaved) {
  qmm::HeadsArgs a{};
  a.q = {q, q_st, q_sh};
  a.k = {k, k_st, k_sh};
  a.T = T;
  a.Hq = static_cast<int>(Hq);
  a.H = static_cast<int>(H);
  a.D = static_cast<int>(D);
  a.R = static_cast<int>(R);
  a.positions = positions;
  a.inv_freq = R ? inv_freq : nullptr;
  a.qw = qw;
  a.kw = kw;
  a.wt = wt;
  a.eps = eps;
  a.interleaved = interleaved;
  return a;
}

qmm_status check_scale(float scale) {
  return scale > 0.0f && scale <= 3e38f ? QMM_OK : fail(QMM_E_ARG, "scale must be positive and finite");
}

qmm_status check_attend(const qmm_cache* h, int64_t B, int64_t Hq, int64_t max_length) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_range(B, 0, 65535, "B"));
  QMM_TRY(check_range(Hq, 1, 8192, "query heads"));
  if (Hq % h->d.heads) return fail(QMM_E_SHAPE, "%lld query heads are no multiple of the cache's %d", static_cast<ll>(Hq), h->d.heads);
  return check_range(max_length, 0, int64_t(1) << 31, "max_length");
}

size_t attend_bytes(const qmm::CacheDesc& d, int64_t B, int64_t Hq, int splits) {
  return splits == 1 ? 0 : static_cast<size_t>(B * Hq * splits) * (d.D + 2) * 4;
}

}  // namespace

extern "C" {

qmm_status qmm_cache_create(qmm_cache** out, void* k, void* v, float* k_scales, float* v_scales, qmm_dtype type,
                            int64_t pages, int64_t page, int64_t heads, int64_t D) {
  if (!out) return fail(QMM_E_ARG, "out is NULL");
  *out = nullptr;
  if (type != QMM_F16 && type != QMM_BF16 && type != QMM_E4M3) return fail(QMM_E_TYPE, "unknown cache type %d", type);
  QMM_TRY(check_ptr(k, 16, "k"));
  QMM_TRY(check_ptr(v, 16, "v"));
  if (type == QMM_E4M3) {
    QMM_TRY(check_ptr(k_scales, 16, "k_scales"));
    QMM_TRY(check_ptr(v_scales, 16, "v_scales"));
  } else if (k_scales || v_scales) {
    return fail(QMM_E_ARG, "only an e4m3 cache has scales");
  }
  QMM_TRY(check_range(page, qmm::kMinPage, qmm::kMaxPage, "page"));
  if (page & (page - 1)) return fail(QMM_E_SHAPE, "page=%lld is not a power of two", static_cast<ll>(page));
  QMM_TRY(check_range(pages, 1, qmm::kMaxTokens / page, "pages"));
  QMM_TRY(check_range(heads, 1, qmm::kMaxHeads, "heads"));
  QMM_TRY(check_head(D));
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(QMM_E_DEVICE, "no HIP device: %s", hipGetErrorString(e));
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(QMM_E_DEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return fail(QMM_E_DEVICE, "device %d is %s, this library is built for gfx950", dev, prop.gcnArchName);
  qmm_cache* h = new (std::nothrow) qmm_cache;
  if (!h) return fail(QMM_E_ARG, "out of host memory");
  h->d = {};
  h->d.k = static_cast<uint8_t*>(k);
  h->d.v = static_cast<uint8_t*>(v);
  h->d.ks = k_scales;
  h->d.vs = v_scales;
  h->d.type = type;
  h->d.pages = pages;
  while ((int64_t(1) << h->d.shift) < page) ++h->d.shift;
  h->d.heads = static_cast<int>(heads);
  h->d.D = static_cast<int>(D);
  h->d.cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  h->device = dev;
  *out = h;
  return ok();
}

qmm_status qmm_cache_destroy(qmm_cache* h) {
  delete h;
  return ok();
}

qmm_status qmm_cache_write(const qmm_cache* h, const void* k, int64_t k_st, int64_t k_sh, const void* v, int64_t v_st,
                           int64_t v_sh, qmm_dtype xt, int64_t T, const int32_t* slots, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_dtype(xt, "input"));
  QMM_TRY(check_range(T, 0, qmm::kMaxTokens, "T"));
  if (T == 0) return ok();
  const HeadRows kr{k, k_st, k_sh}, vr{v, v_st, v_sh};
  QMM_TRY(check_rows(kr, xt, "k"));
  QMM_TRY(check_rows(vr, xt, "v"));
  QMM_TRY(check_ptr(slots, 4, "slots"));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_cache_write(h->d, kr, vr, xt, T, slots, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "cache write launch");
}

qmm_status qmm_cache_read(const qmm_cache* h, const int32_t* table, int64_t B, int64_t W, const int32_t* starts,
                          int64_t total, void* k, void* v, qmm_dtype ot, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_dtype(ot, "output"));
  QMM_TRY(check_range(B, 0, 1 << 20, "B"));
  QMM_TRY(check_range(W, 0, qmm::kMaxTokens, "table columns"));
  QMM_TRY(check_range(total, 0, qmm::kMaxTokens, "total"));
  if (total == 0 || B == 0) return ok();
  if (W) QMM_TRY(check_ptr(table, 4, "table"));
  QMM_TRY(check_ptr(starts, 4, "starts"));
  QMM_TRY(check_ptr(k, size_of(ot), "k"));
  QMM_TRY(check_ptr(v, size_of(ot), "v"));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_cache_read(h->d, table, B, W, starts, total, k, v, ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "cache read launch");
}

qmm_status qmm_head_norm_rope(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                              qmm_dtype xt, int64_t T, int64_t Hq, int64_t H, int64_t D, const void* q_weight,
                              const void* k_weight, qmm_dtype wt, float eps, const int32_t* positions, const float* inv_freq,
                              int64_t R, int interleaved, void* q_out, void* k_out, qmm_dtype ot, qmm_stream_t stream) {
  qmm::HeadsArgs a = heads_args(q, q_st, q_sh, k, k_st, k_sh, T, Hq, H, D, q_weight, k_weight, wt, eps, positions, inv_freq, R,
                                interleaved);
  QMM_TRY(check_heads(a, xt, Hq, H, D, R));
  QMM_TRY(check_dtype(ot, "output"));
  if (T == 0) return ok();
  if (Hq) QMM_TRY(check_ptr(q_out, size_of(ot), "q_out"));
  if (H) QMM_TRY(check_ptr(k_out, size_of(ot), "k_out"));
  a.qo = q_out;
  a.ko = k_out;
  const hipError_t e = qmm::launch_heads(a, xt, ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "head norm launch");
}

qmm_status qmm_cache_norm_rope_write(const qmm_cache* h, const void* q, int64_t q_st, int64_t q_sh, const void* k,
                                     int64_t k_st, int64_t k_sh, const void* v, int64_t v_st, int64_t v_sh, qmm_dtype xt,
                                     int64_t T, int64_t Hq, const void* q_weight, const void* k_weight, qmm_dtype wt,
                                     float eps, const int32_t* positions, const float* inv_freq, int64_t R, int interleaved,
                                     const int32_t* slots, void* q_out, qmm_dtype ot, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  qmm::HeadsArgs a = heads_args(q, q_st, q_sh, k, k_st, k_sh, T, Hq, h->d.heads, h->d.D, q_weight, k_weight, wt, eps, positions,
                                inv_freq, R, interleaved);
  QMM_TRY(check_heads(a, xt, Hq, h->d.heads, h->d.D, R));
  QMM_TRY(check_dtype(ot, "output"));
  if (h->d.type != QMM_E4M3 && ot != h->d.type) return fail(QMM_E_TYPE, "a 16-bit cache gives queries of its own type");
  if (T == 0) return ok();
  a.v = {v, v_st, v_sh};
  QMM_TRY(check_rows(a.v, xt, "v"));
  QMM_TRY(check_ptr(slots, 4, "slots"));
  if (Hq) QMM_TRY(check_ptr(q_out, size_of(ot), "q_out"));
  QMM_TRY(check_device(h));
  a.cache = h->d;
  a.slots = slots;
  a.qo = q_out;
  const hipError_t e = qmm::launch_heads(a, xt, ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "head norm launch");
}

size_t qmm_cache_attend_workspace_bytes(const qmm_cache* h, int64_t B, int64_t Hq, int64_t max_length) {
  if (check_attend(h, B, Hq, max_length) != QMM_OK || B == 0) return 0;
  return attend_bytes(h->d, B, Hq, qmm::attend_split(h->d, B, static_cast<int>(Hq), max_length).splits);
}

qmm_status qmm_cache_attend(const qmm_cache* h, const void* q, qmm_dtype qt, int64_t q_sb, int64_t q_sh, int64_t B, int64_t Hq,
                            const int32_t* table, int64_t W, const int32_t* lengths, int64_t max_length, float scale,
                            void* out, void* ws, size_t ws_bytes, qmm_stream_t stream) {
  QMM_TRY(check_attend(h, B, Hq, max_length));
  if (qt != QMM_F16 && qt != QMM_BF16) return fail(QMM_E_TYPE, "queries are fp16 or bf16 (got %d)", qt);
  if (h->d.type != QMM_E4M3 && qt != h->d.type) return fail(QMM_E_TYPE, "a 16-bit cache takes queries of its own type");
  QMM_TRY(check_range(W, 0, qmm::kMaxTokens >> h->d.shift, "table columns"));
  QMM_TRY(check_scale(scale));
  if (B == 0) return ok();
  const HeadRows rows{q, q_sb, q_sh};
  QMM_TRY(check_rows(rows, qt, "q"));
  if (W) QMM_TRY(check_ptr(table, 4, "table"));
  QMM_TRY(check_ptr(lengths, 4, "lengths"));
  QMM_TRY(check_ptr(out, size_of(qt), "out"));
  qmm::AttendArgs a{};
  const qmm::AttendSplit split = qmm::attend_split(h->d, B, static_cast<int>(Hq), max_length);
  a.splits = split.splits;
  a.piece = split.piece;
  QMM_TRY(check_ws(ws, ws_bytes, attend_bytes(h->d, B, Hq, a.splits), "ws"));
  QMM_TRY(check_device(h));
  a.cache = h->d;
  a.q = rows;
  a.B = B;
  a.Hq = static_cast<int>(Hq);
  a.table = table;
  a.W = W;
  a.lengths = lengths;
  a.scale = scale;
  a.out = out;
  a.ws = static_cast<float*>(ws);
  const hipError_t e = qmm::launch_attend(a, qt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attend launch");
}

qmm_status qmm_attend_prompt(const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
                             const void* v, int64_t v_st, int64_t v_sh, qmm_dtype dt, const int32_t* q_starts,
                             const int32_t* k_starts, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t H, int64_t D,
                             int causal, float scale, void* out, qmm_stream_t stream) {
  if (dt != QMM_F16 && dt != QMM_BF16) return fail(QMM_E_TYPE, "prompts are fp16 or bf16 (got %d)", dt);
  QMM_TRY(check_range(B, 0, 1 << 20, "B"));
  QMM_TRY(check_range(Tq, 0, qmm::kMaxTokens, "queries"));
  QMM_TRY(check_range(Tk, 0, qmm::kMaxTokens, "keys"));
  QMM_TRY(check_range(H, 1, qmm::kMaxHeads, "key heads"));
  QMM_TRY(check_range(Hq, 1, 8192, "query heads"));
  if (Hq % H) return fail(QMM_E_SHAPE, "%lld query heads are no multiple of %lld key heads", static_cast<ll>(Hq), static_cast<ll>(H));
  QMM_TRY(check_head(D));
  if (causal != 0 && causal != 1) return fail(QMM_E_ARG, "causal must be 0 or 1");
  QMM_TRY(check_scale(scale));
  if (B == 0 || Tq == 0) return ok();
  qmm::PromptArgs a{};
  a.q = {q, q_st, q_sh};
  a.k = {k, k_st, k_sh};
  a.v = {v, v_st, v_sh};
  QMM_TRY(check_rows(a.q, dt, "q"));
  if (Tk) {
    for (HeadRows* r : {&a.k, &a.v}) {
      const char* what = r == &a.k ? "k" : "v";
      QMM_TRY(check_rows(*r, dt, what));
      if (Tk == 1) r->st = D;
      if (r->st < D || r->st > (1 << 23)) return fail(QMM_E_SHAPE, "the token stride of %s is outside [D, 2^23]", what);
      if (!aligned(r->p, 16) || r->st % 8 || r->sh % 8) return fail(QMM_E_ALIGN, "rows of %s must be 16-byte aligned", what);
    }
  }
  QMM_TRY(check_ptr(q_starts, 4, "q_starts"));
  QMM_TRY(check_ptr(k_starts, 4, "k_starts"));
  QMM_TRY(check_ptr(out, size_of(dt), "out"));
  a.B = B;
  a.Tq = Tq;
  a.Tk = Tk;
  a.Hq = static_cast<int>(Hq);
  a.H = static_cast<int>(H);
  a.D = static_cast<int>(D);
  a.q_starts = q_starts;
  a.k_starts = k_starts;
  a.causal = causal;
  a.scale = scale;
  a.out = out;
  const hipError_t e = qmm::launch_prompt(a, dt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "prompt launch");
}

}  // extern "C"
