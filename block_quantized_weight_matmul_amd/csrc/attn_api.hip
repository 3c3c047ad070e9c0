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

// norms and rotation: weights, angles, and the tensors that the call reads; *r is what the launch takes
qmm_status check_heads(const qmm_head_args* a, qmm::HeadsArgs* r) {
  QMM_TRY(check_dtype(a->xt, "input"));
  QMM_TRY(check_dtype(a->wt, "weight"));
  QMM_TRY(check_dtype(a->ot, "output"));
  QMM_TRY(check_range(a->T, 0, qmm::kMaxTokens, "T"));
  QMM_TRY(check_range(a->Hq, 0, qmm::kMaxHeads, "query heads"));
  QMM_TRY(check_range(a->H, 0, qmm::kMaxHeads, "key heads"));
  if (a->Hq + a->H == 0) return fail(QMM_E_SHAPE, "no heads");
  QMM_TRY(check_head(a->D));
  if (a->R < 0 || a->R > a->D || a->R % 8)
    return fail(QMM_E_SHAPE, "R=%lld is not a multiple of 8 up to D", static_cast<ll>(a->R));
  if (!(a->eps >= 0.0f) || a->eps > 3e38f) return fail(QMM_E_ARG, "eps must be finite and not negative");
  if (a->interleaved != 0 && a->interleaved != 1) return fail(QMM_E_ARG, "interleaved must be 0 or 1");
  if (a->T == 0) return QMM_OK;
  r->q = {a->q, a->q_token, a->q_head};
  r->k = {a->k, a->k_token, a->k_head};
  if (a->Hq) {
    QMM_TRY(check_rows(r->q, a->xt, "q"));
    QMM_TRY(check_ptr(a->q_out, size_of(a->ot), "q_out"));
  }
  if (a->H) QMM_TRY(check_rows(r->k, a->xt, "k"));
  if (a->R) {
    QMM_TRY(check_ptr(a->positions, 4, "positions"));
    QMM_TRY(check_ptr(a->inv_freq, 4, "inv_freq"));
  }
  if (a->q_weight && !aligned(a->q_weight, size_of(a->wt))) return fail(QMM_E_ALIGN, "q_weight must be element-aligned");
  if (a->k_weight && !aligned(a->k_weight, size_of(a->wt))) return fail(QMM_E_ALIGN, "k_weight must be element-aligned");
  r->T = a->T;
  r->Hq = static_cast<int>(a->Hq);
  r->H = static_cast<int>(a->H);
  r->D = static_cast<int>(a->D);
  r->R = static_cast<int>(a->R);
  r->positions = a->positions;
  r->inv_freq = a->R ? a->inv_freq : nullptr;
  r->qw = a->q_weight;
  r->kw = a->k_weight;
  r->wt = a->wt;
  r->eps = a->eps;
  r->interleaved = a->interleaved;
  r->qo = a->q_out;
  return QMM_OK;
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

qmm_status qmm_cache_write(const qmm_cache* h, const qmm_cache_write_args* a, qmm_stream_t stream) {
  if (!h || !a) return fail(QMM_E_ARG, "%s is NULL", h ? "a" : "handle");
  QMM_TRY(check_dtype(a->xt, "input"));
  QMM_TRY(check_range(a->T, 0, qmm::kMaxTokens, "T"));
  if (a->T == 0) return ok();
  const HeadRows k{a->k, a->k_token, a->k_head}, v{a->v, a->v_token, a->v_head};
  QMM_TRY(check_rows(k, a->xt, "k"));
  QMM_TRY(check_rows(v, a->xt, "v"));
  QMM_TRY(check_ptr(a->slots, 4, "slots"));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_cache_write(h->d, k, v, a->xt, a->T, a->slots, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "cache write launch");
}

qmm_status qmm_cache_read(const qmm_cache* h, const qmm_cache_read_args* a, qmm_stream_t stream) {
  if (!h || !a) return fail(QMM_E_ARG, "%s is NULL", h ? "a" : "handle");
  QMM_TRY(check_dtype(a->ot, "output"));
  QMM_TRY(check_range(a->B, 0, 1 << 20, "B"));
  QMM_TRY(check_range(a->W, 0, qmm::kMaxTokens, "table columns"));
  QMM_TRY(check_range(a->total, 0, qmm::kMaxTokens, "total"));
  if (a->total == 0 || a->B == 0) return ok();
  if (a->W) QMM_TRY(check_ptr(a->table, 4, "table"));
  QMM_TRY(check_ptr(a->starts, 4, "starts"));
  QMM_TRY(check_ptr(a->k, size_of(a->ot), "k"));
  QMM_TRY(check_ptr(a->v, size_of(a->ot), "v"));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_cache_read(h->d, a->table, a->B, a->W, a->starts, a->total, a->k, a->v, a->ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "cache read launch");
}

qmm_status qmm_head_norm_rope(const qmm_head_args* a, qmm_stream_t stream) {
  if (!a) return fail(QMM_E_ARG, "a is NULL");
  qmm::HeadsArgs r{};
  QMM_TRY(check_heads(a, &r));
  if (a->T == 0) return ok();
  if (a->H) QMM_TRY(check_ptr(a->k_out, size_of(a->ot), "k_out"));
  r.ko = a->k_out;
  const hipError_t e = qmm::launch_heads(r, a->xt, a->ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "head norm launch");
}

qmm_status qmm_cache_norm_rope_write(const qmm_cache* h, const qmm_head_args* a, qmm_stream_t stream) {
  if (!h || !a) return fail(QMM_E_ARG, "%s is NULL", h ? "a" : "handle");
  qmm::HeadsArgs r{};
  QMM_TRY(check_heads(a, &r));
  if (a->H != h->d.heads || a->D != h->d.D)
    return fail(QMM_E_SHAPE, "%lld key heads of %lld; the cache has %d of %d", static_cast<ll>(a->H), static_cast<ll>(a->D),
                h->d.heads, h->d.D);
  if (h->d.type != QMM_E4M3 && a->ot != h->d.type) return fail(QMM_E_TYPE, "a 16-bit cache gives queries of its own type");
  if (a->T == 0) return ok();
  r.v = {a->v, a->v_token, a->v_head};
  QMM_TRY(check_rows(r.v, a->xt, "v"));
  QMM_TRY(check_ptr(a->slots, 4, "slots"));
  QMM_TRY(check_device(h));
  r.cache = h->d;
  r.slots = a->slots;
  const hipError_t e = qmm::launch_heads(r, a->xt, a->ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "head norm launch");
}

size_t qmm_cache_attend_workspace_bytes(const qmm_cache* h, int64_t B, int64_t Hq, int64_t max_length) {
  if (check_attend(h, B, Hq, max_length) != QMM_OK || B == 0) return 0;
  return attend_bytes(h->d, B, Hq, qmm::attend_split(h->d, B, static_cast<int>(Hq), max_length).splits);
}

qmm_status qmm_cache_attend(const qmm_cache* h, const qmm_attend_args* a, qmm_stream_t stream) {
  if (!a) return fail(QMM_E_ARG, "a is NULL");
  QMM_TRY(check_attend(h, a->B, a->Hq, a->max_length));
  if (a->qt != QMM_F16 && a->qt != QMM_BF16) return fail(QMM_E_TYPE, "queries are fp16 or bf16 (got %d)", a->qt);
  if (h->d.type != QMM_E4M3 && a->qt != h->d.type) return fail(QMM_E_TYPE, "a 16-bit cache takes queries of its own type");
  QMM_TRY(check_range(a->W, 0, qmm::kMaxTokens >> h->d.shift, "table columns"));
  QMM_TRY(check_scale(a->scale));
  if (a->B == 0) return ok();
  qmm::AttendArgs r{};
  r.q = {a->q, a->q_token, a->q_head};
  QMM_TRY(check_rows(r.q, a->qt, "q"));
  if (a->W) QMM_TRY(check_ptr(a->table, 4, "table"));
  QMM_TRY(check_ptr(a->lengths, 4, "lengths"));
  QMM_TRY(check_ptr(a->out, size_of(a->qt), "out"));
  const qmm::AttendSplit split = qmm::attend_split(h->d, a->B, static_cast<int>(a->Hq), a->max_length);
  QMM_TRY(check_ws(a->ws, a->ws_bytes, attend_bytes(h->d, a->B, a->Hq, split.splits), "ws"));
  QMM_TRY(check_device(h));
  r.cache = h->d;
  r.B = a->B;
  r.Hq = static_cast<int>(a->Hq);
  r.table = a->table;
  r.W = a->W;
  r.lengths = a->lengths;
  r.scale = a->scale;
  r.out = a->out;
  r.splits = split.splits;
  r.piece = split.piece;
  r.waves = split.waves;
  r.ws = static_cast<float*>(a->ws);
  const hipError_t e = qmm::launch_attend(r, a->qt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attend launch");
}

qmm_status qmm_attend_prompt(const qmm_prompt_args* a, qmm_stream_t stream) {
  if (!a) return fail(QMM_E_ARG, "a is NULL");
  if (a->dt != QMM_F16 && a->dt != QMM_BF16) return fail(QMM_E_TYPE, "prompts are fp16 or bf16 (got %d)", a->dt);
  QMM_TRY(check_range(a->B, 0, 1 << 20, "B"));
  QMM_TRY(check_range(a->Tq, 0, qmm::kMaxTokens, "queries"));
  QMM_TRY(check_range(a->Tk, 0, qmm::kMaxTokens, "keys"));
  QMM_TRY(check_range(a->H, 1, qmm::kMaxHeads, "key heads"));
  QMM_TRY(check_range(a->Hq, 1, 8192, "query heads"));
  if (a->Hq % a->H)
    return fail(QMM_E_SHAPE, "%lld query heads are no multiple of %lld key heads", static_cast<ll>(a->Hq), static_cast<ll>(a->H));
  QMM_TRY(check_head(a->D));
  if (a->causal != 0 && a->causal != 1) return fail(QMM_E_ARG, "causal must be 0 or 1");
  QMM_TRY(check_scale(a->scale));
  if (a->B == 0 || a->Tq == 0) return ok();
  qmm::PromptArgs r{};
  r.q = {a->q, a->q_token, a->q_head};
  r.k = {a->k, a->k_token, a->k_head};
  r.v = {a->v, a->v_token, a->v_head};
  QMM_TRY(check_rows(r.q, a->dt, "q"));
  if (a->Tk) {
    for (HeadRows* x : {&r.k, &r.v}) {
      const char* what = x == &r.k ? "k" : "v";
      QMM_TRY(check_rows(*x, a->dt, what));
      if (a->Tk == 1) x->st = a->D;
      if (a->H == 1) x->sh = 0;
      if (x->st < a->D || x->st > (1 << 23)) return fail(QMM_E_SHAPE, "the token stride of %s is outside [D, 2^23]", what);
      if (!aligned(x->p, 16) || x->st % 8 || x->sh % 8) return fail(QMM_E_ALIGN, "rows of %s must be 16-byte aligned", what);
    }
  }
  QMM_TRY(check_ptr(a->q_starts, 4, "q_starts"));
  QMM_TRY(check_ptr(a->k_starts, 4, "k_starts"));
  QMM_TRY(check_ptr(a->out, size_of(a->dt), "out"));
  r.B = a->B;
  r.Tq = a->Tq;
  r.Tk = a->Tk;
  r.Hq = static_cast<int>(a->Hq);
  r.H = static_cast<int>(a->H);
  r.D = static_cast<int>(a->D);
  r.q_starts = a->q_starts;
  r.k_starts = a->k_starts;
  r.causal = a->causal;
  r.scale = a->scale;
  r.out = a->out;
  const hipError_t e = qmm::launch_prompt(r, a->dt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "prompt launch");
}

}  // extern "C"
