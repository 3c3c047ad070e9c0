// f8_api.hip -- the C ABI of the e4m3 products and the expert router (include/qmm.h): argument checks, device checks
// and dispatch.  No device memory is allocated here and nothing synchronises.
#include <string.h>

#include <new>

#include "api_common.hpp"
#include "f8.hpp"

struct qmm_f8_matrix {
  qmm::F8Desc d;
  int device;
};

namespace {

using qmm::aligned;
using qmm::check_dtype;
using qmm::check_ptr;
using qmm::check_range;
using qmm::check_ws;
using qmm::dtype_ok;
using qmm::fail;
using qmm::hip_fail;
using qmm::ok;
using qmm::f8_pad;
using qmm::ll;
using qmm::size_of;
using qmm::stream_of;

qmm_status check_device(const qmm_f8_matrix* h) {
  int dev = -1;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev != h->device) return fail(QMM_E_DEVICE, "current device %d is not the handle's device %d", dev, h->device);
  return QMM_OK;
}

constexpr int64_t kMaxK = qmm::kF8MaxK - qmm::kF8Block;
constexpr int64_t kMaxWgradTokens = int64_t(1) << 23;

qmm_status check_rows(int64_t ldx, int64_t K) {
  return ldx >= K && ldx <= (int64_t(1) << 40) ? QMM_OK
                                               : fail(QMM_E_SHAPE, "ldx=%lld below K=%lld (or too large)",
                                                      static_cast<ll>(ldx), static_cast<ll>(K));
}

// both or neither of a code and a scale buffer
qmm_status check_out(const void* codes, const float* scales, const char* what, bool optional) {
  if (optional && !codes && !scales) return QMM_OK;
  if (!codes || !scales) return fail(QMM_E_ARG, "%s needs both codes and scales", what);
  if (!aligned(codes, 16)) return fail(QMM_E_ALIGN, "codes must be 16-byte aligned");
  if (!aligned(scales, 4)) return fail(QMM_E_ALIGN, "scales must be 4-byte aligned");
  return QMM_OK;
}

qmm_status check_pairs(int64_t N, int64_t S, int64_t E) {
  QMM_TRY(check_range(S, 1, 64, "S"));
  QMM_TRY(check_range(E, 1, qmm::kRouteMaxExperts, "experts"));
  if (N < 0 || N > qmm::kRouteMaxPairs || N * S > qmm::kRouteMaxPairs)
    return fail(QMM_E_SHAPE, "takes 0..%lld (token, slot) pairs (got %lld x %lld)", static_cast<ll>(qmm::kRouteMaxPairs),
                static_cast<ll>(N), static_cast<ll>(S));
  return QMM_OK;
}

// sizes of an expert-indexed call on h
qmm_status check_id(const qmm_f8_matrix* h, int64_t N, int64_t S, int x_per_slot) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_pairs(N, S, h->d.n_experts));
  if (x_per_slot != 0 && x_per_slot != 1) return fail(QMM_E_ARG, "x_per_slot must be 0 or 1");
  if ((x_per_slot ? N * S : N) * h->d.Kp >= (int64_t(1) << 32))
    return fail(QMM_E_SHAPE, "expert-indexed calls take rows whose codes are below 4 GiB");
  return QMM_OK;
}

size_t token_bytes(int64_t rows, int64_t Kp) {
  return static_cast<size_t>(rows) * Kp + (static_cast<size_t>(rows) * (Kp / qmm::kF8Block) * 4 + 15) / 16 * 16;
}

}  // namespace

extern "C" {

int64_t qmm_f8_padded(int64_t n) { return n <= 0 ? 0 : f8_pad(n); }

qmm_status qmm_f8_create(qmm_f8_matrix** out, const void* codes, const float* scales, int64_t n_experts, int64_t M,
                         int64_t K) {
  if (!out) return fail(QMM_E_ARG, "out is NULL");
  *out = nullptr;
  QMM_TRY(check_ptr(codes, 16, "codes"));
  QMM_TRY(check_ptr(scales, 4, "scales"));
  QMM_TRY(check_range(n_experts, 1, 8192, "n_experts"));
  QMM_TRY(check_range(M, 1, qmm::kF8MaxRows, "M"));
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(QMM_E_DEVICE, "no HIP device: %s", hipGetErrorString(e));
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(QMM_E_DEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return fail(QMM_E_DEVICE, "device %d is %s, this library is built for gfx950", dev, prop.gcnArchName);
  qmm_f8_matrix* h = new (std::nothrow) qmm_f8_matrix;
  if (!h) return fail(QMM_E_ARG, "out of host memory");
  h->d.codes = static_cast<const uint8_t*>(codes);
  h->d.scales = scales;
  h->d.n_experts = n_experts;
  h->d.M = M;
  h->d.K = K;
  h->d.Kp = f8_pad(K);
  h->d.cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  h->device = dev;
  *out = h;
  return ok();
}

qmm_status qmm_f8_destroy(qmm_f8_matrix* h) {
  delete h;
  return ok();
}

qmm_status qmm_f8_quantize(const void* x, qmm_dtype xt, int64_t ldx, int64_t N, int64_t K, void* codes, float* scales,
                           void* codes_t, float* scales_t, qmm_stream_t stream) {
  QMM_TRY(check_dtype(xt, "activation"));
  QMM_TRY(check_range(N, 0, qmm::kF8MaxRows, "N"));
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  QMM_TRY(check_rows(ldx, K));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(x, size_of(xt), "x"));
  QMM_TRY(check_out(codes, scales, "codes", true));
  QMM_TRY(check_out(codes_t, scales_t, "codes_t", true));
  if (!codes && !codes_t) return fail(QMM_E_ARG, "neither codes nor codes_t is given");
  qmm::F8QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.N = N;
  a.K = K;
  a.codes_r = static_cast<uint8_t*>(codes);
  a.scales_r = scales;
  a.codes_c = static_cast<uint8_t*>(codes_t);
  a.scales_c = scales_t;
  a.slots = 1;
  const hipError_t e = qmm::launch_f8_quantize(a, xt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 quantize launch");
}

qmm_status qmm_f8_quantize_weight(const void* w, qmm_dtype wt, int64_t n_experts, int64_t M, int64_t K, void* codes,
                                  float* scales, void* codes_t, float* scales_t, qmm_stream_t stream) {
  QMM_TRY(check_dtype(wt, "weight"));
  QMM_TRY(check_range(n_experts, 1, 8192, "n_experts"));
  QMM_TRY(check_range(M, 1, qmm::kF8MaxRows, "M"));
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  QMM_TRY(check_ptr(w, size_of(wt), "w"));
  QMM_TRY(check_out(codes, scales, "codes", false));
  QMM_TRY(check_out(codes_t, scales_t, "codes_t", true));
  const hipError_t e = qmm::launch_f8_quantize_weight(w, wt, n_experts, M, K, static_cast<uint8_t*>(codes), scales,
                                                      static_cast<uint8_t*>(codes_t), scales_t, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 quantize launch");
}

qmm_status qmm_f8_transpose(const qmm_f8_matrix* h, void* codes_t, float* scales_t, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_out(codes_t, scales_t, "codes_t", false));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_f8_transpose(h->d, static_cast<uint8_t*>(codes_t), scales_t, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 transpose launch");
}

qmm_status qmm_f8_dequantize(const qmm_f8_matrix* h, int64_t expert, void* out, qmm_dtype ot, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  QMM_TRY(check_range(expert, 0, h->d.n_experts - 1, "expert"));
  QMM_TRY(check_dtype(ot, "output"));
  QMM_TRY(check_ptr(out, size_of(ot), "out"));
  QMM_TRY(check_device(h));
  const hipError_t e = qmm::launch_f8_dequantize(h->d, expert, out, ot, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 dequantize launch");
}

size_t qmm_f8_gemm_workspace_bytes(const qmm_f8_matrix* h, int64_t N) {
  if (!h || h->d.n_experts != 1 || N <= 0 || N > qmm::kF8MaxRows) return 0;
  return qmm::f8_gemm_workspace_bytes(h->d, N);
}

size_t qmm_f8_linear_workspace_bytes(const qmm_f8_matrix* h, int64_t N) {
  if (!h || h->d.n_experts != 1 || N <= 0 || N > qmm::kF8MaxRows || qmm::f8_linear_fused(h->d, N)) return 0;
  return token_bytes(N, h->d.Kp) + qmm::f8_gemm_workspace_bytes(h->d, N);
}

qmm_status qmm_f8_gemm(const qmm_f8_matrix* h, const void* codes, const float* scales, int64_t N, void* y, qmm_dtype yt,
                       void* ws, size_t ws_bytes, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  if (h->d.n_experts != 1) return fail(QMM_E_ARG, "qmm_f8_gemm needs a handle with n_experts == 1");
  QMM_TRY(check_dtype(yt, "output"));
  QMM_TRY(check_range(N, 0, qmm::kF8MaxRows, "N"));
  if (N == 0) return ok();
  QMM_TRY(check_out(codes, scales, "tokens", false));
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  QMM_TRY(check_ws(ws, ws_bytes, qmm::f8_gemm_workspace_bytes(h->d, N), "ws"));
  QMM_TRY(check_device(h));
  const hipError_t e =
      qmm::launch_f8_gemm(h->d, static_cast<const uint8_t*>(codes), scales, N, y, yt, ws, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 gemm launch");
}

qmm_status qmm_f8_linear(const qmm_f8_matrix* h, const void* x, qmm_dtype xt, int64_t ldx, int64_t N, void* y,
                         qmm_dtype yt, void* ws, size_t ws_bytes, qmm_stream_t stream) {
  if (!h) return fail(QMM_E_ARG, "handle is NULL");
  if (h->d.n_experts != 1) return fail(QMM_E_ARG, "qmm_f8_linear needs a handle with n_experts == 1");
  QMM_TRY(check_dtype(xt, "activation"));
  QMM_TRY(check_dtype(yt, "output"));
  QMM_TRY(check_range(N, 0, qmm::kF8MaxRows, "N"));
  QMM_TRY(check_rows(ldx, h->d.K));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(x, size_of(xt), "x"));
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  QMM_TRY(check_ws(ws, ws_bytes, qmm_f8_linear_workspace_bytes(h, N), "ws"));
  QMM_TRY(check_device(h));
  const hipStream_t st = stream_of(stream);
  hipError_t e;
  if (qmm::f8_linear_fused(h->d, N)) {
    e = qmm::launch_f8_linear(h->d, x, xt, ldx, N, y, yt, st);
  } else {
    qmm::F8QuantArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.N = N;
    a.K = h->d.K;
    a.codes_r = static_cast<uint8_t*>(ws);
    a.scales_r = reinterpret_cast<float*>(a.codes_r + N * h->d.Kp);
    a.slots = 1;
    e = qmm::launch_f8_quantize(a, xt, st);
    if (e == hipSuccess)
      e = qmm::launch_f8_gemm(h->d, a.codes_r, a.scales_r, N, y, yt, a.codes_r + token_bytes(N, h->d.Kp), st);
  }
  return e == hipSuccess ? ok() : hip_fail(e, "f8 linear launch");
}

size_t qmm_route_plan_bytes(int64_t pairs, int64_t E) {
  if (pairs < 0 || pairs > qmm::kRouteMaxPairs || E < 1 || E > qmm::kRouteMaxExperts) return 0;
  return (static_cast<size_t>(qmm::plan_desc(pairs, E).total) * 4 + 15) / 16 * 16;
}

qmm_status qmm_route_plan(const int32_t* ids, int64_t N, int64_t S, int64_t E, void* plan, size_t plan_bytes,
                          qmm_stream_t stream) {
  QMM_TRY(check_pairs(N, S, E));
  QMM_TRY(check_ws(plan, plan_bytes, qmm_route_plan_bytes(N * S, E), "plan"));
  if (N > 0) QMM_TRY(check_ptr(ids, 4, "ids"));
  const hipError_t e = qmm::launch_route_plan(ids, N * S, E, static_cast<int32_t*>(plan), stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route plan launch");
}

size_t qmm_f8_linear_id_workspace_bytes(const qmm_f8_matrix* h, int64_t N, int64_t S, int x_per_slot) {
  if (!h || N <= 0 || S < 1 || S > 64 || N > qmm::kRouteMaxPairs || N * S > qmm::kRouteMaxPairs ||
      h->d.n_experts > qmm::kRouteMaxExperts ||
      qmm::f8_linear_id_fused(h->d, N * S))
    return 0;
  return token_bytes(x_per_slot ? N * S : N, h->d.Kp) + qmm_route_plan_bytes(N * S, h->d.n_experts);
}

qmm_status qmm_f8_gemm_id(const qmm_f8_matrix* h, const void* codes, const float* scales, int64_t N, int64_t S,
                          int x_per_slot, const void* plan, void* y, qmm_dtype yt, qmm_stream_t stream) {
  QMM_TRY(check_id(h, N, S, x_per_slot));
  QMM_TRY(check_dtype(yt, "output"));
  if (N == 0) return ok();
  QMM_TRY(check_out(codes, scales, "tokens", false));
  QMM_TRY(check_ptr(plan, 16, "plan"));
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  QMM_TRY(check_device(h));
  const hipError_t e =
      qmm::launch_f8_gemm_id(h->d, static_cast<const uint8_t*>(codes), scales, N * S, x_per_slot ? 1 : static_cast<int>(S),
                             static_cast<const int32_t*>(plan), y, yt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 gemm_id launch");
}

qmm_status qmm_f8_linear_id(const qmm_f8_matrix* h, const void* x, qmm_dtype xt, int64_t N, int64_t S, int x_per_slot,
                            const int32_t* ids, void* y, qmm_dtype yt, void* ws, size_t ws_bytes, qmm_stream_t stream) {
  QMM_TRY(check_id(h, N, S, x_per_slot));
  QMM_TRY(check_dtype(xt, "activation"));
  QMM_TRY(check_dtype(yt, "output"));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(x, size_of(xt), "x"));
  QMM_TRY(check_ptr(ids, 4, "ids"));
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  QMM_TRY(check_ws(ws, ws_bytes, qmm_f8_linear_id_workspace_bytes(h, N, S, x_per_slot), "ws"));
  QMM_TRY(check_device(h));
  const hipStream_t st = stream_of(stream);
  const int slots = x_per_slot ? 1 : static_cast<int>(S);
  const int64_t rows = x_per_slot ? N * S : N;
  hipError_t e;
  if (qmm::f8_linear_id_fused(h->d, N * S)) {
    e = qmm::launch_f8_linear_id(h->d, x, xt, N * S, slots, ids, y, yt, st);
  } else {
    qmm::F8QuantArgs a{};
    a.x = x;
    a.ldx = h->d.K;
    a.N = rows;
    a.K = h->d.K;
    a.codes_r = static_cast<uint8_t*>(ws);
    a.scales_r = reinterpret_cast<float*>(a.codes_r + rows * h->d.Kp);
    a.slots = 1;
    int32_t* plan = reinterpret_cast<int32_t*>(a.codes_r + token_bytes(rows, h->d.Kp));
    e = qmm::launch_f8_quantize(a, xt, st);
    if (e == hipSuccess) e = qmm::launch_route_plan(ids, N * S, h->d.n_experts, plan, st);
    if (e == hipSuccess) e = qmm::launch_f8_gemm_id(h->d, a.codes_r, a.scales_r, N * S, slots, plan, y, yt, st);
  }
  return e == hipSuccess ? ok() : hip_fail(e, "f8 linear_id launch");
}

int64_t qmm_f8_routed_tokens(int64_t pairs, int64_t E) {
  if (pairs < 0 || pairs > qmm::kRouteMaxPairs || E < 1 || E > qmm::kRouteMaxExperts) return 0;
  return qmm::kF8Block * qmm::plan_desc(pairs, E).cap[qmm::kPlanTileKinds - 1];
}

qmm_status qmm_f8_quantize_routed(const void* x, qmm_dtype xt, int64_t ldx, int64_t N, int64_t S, int x_per_slot,
                                  int64_t K, int64_t E, const void* plan, void* codes_t, float* scales_t,
                                  qmm_stream_t stream) {
  QMM_TRY(check_dtype(xt, "activation"));
  QMM_TRY(check_pairs(N, S, E));
  if (x_per_slot != 0 && x_per_slot != 1) return fail(QMM_E_ARG, "x_per_slot must be 0 or 1");
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  QMM_TRY(check_rows(ldx, K));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(x, size_of(xt), "x"));
  QMM_TRY(check_ptr(plan, 16, "plan"));
  QMM_TRY(check_out(codes_t, scales_t, "codes_t", false));
  qmm::F8QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.N = x_per_slot ? N * S : N;
  a.K = K;
  a.codes_c = static_cast<uint8_t*>(codes_t);
  a.scales_c = scales_t;
  a.plan = static_cast<const int32_t*>(plan);
  a.pd = qmm::plan_desc(N * S, E);
  a.slots = x_per_slot ? 1 : static_cast<int>(S);
  const hipError_t e = qmm::launch_f8_quantize(a, xt, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 quantize launch");
}

constexpr int kWgradCus = 256;  // of gfx950; only the choice of tiles and shares depends on it

static qmm_status wgrad(const void* gc, const float* gs, const void* xc, const float* xs, int64_t Np, int64_t M, int64_t K,
                        const void* plan, const qmm::PlanDesc* pd, void* dw, int dt, void* ws, qmm_stream_t stream) {
  QMM_TRY(check_ptr(dw, size_of(dt), "dw"));
  if (Np > 0) {
    QMM_TRY(check_out(gc, gs, "g", false));
    QMM_TRY(check_out(xc, xs, "x", false));
  }
  if (pd) QMM_TRY(check_ptr(plan, 16, "plan"));
  qmm::F8WgradArgs a{};
  a.gc = static_cast<const uint8_t*>(gc);
  a.gs = gs;
  a.xc = static_cast<const uint8_t*>(xc);
  a.xs = xs;
  a.M = M;
  a.K = K;
  a.Np = Np;
  a.dw = dw;
  a.dt = dt;
  a.cus = kWgradCus;
  a.ws = ws;
  if (pd) {
    a.plan = static_cast<const int32_t*>(plan);
    a.pd = *pd;
  }
  const hipError_t e = qmm::launch_f8_wgrad(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "f8 wgrad launch");
}

size_t qmm_f8_wgrad_workspace_bytes(int64_t N, int64_t M, int64_t K) {
  if (N <= 0 || N > kMaxWgradTokens || M < 1 || M > qmm::kF8MaxRows || K < 1 || K > kMaxK) return 0;
  return qmm::f8_wgrad_workspace_bytes(f8_pad(N), M, K, kWgradCus);
}

qmm_status qmm_f8_wgrad(const void* g_codes, const float* g_scales, const void* x_codes, const float* x_scales, int64_t N,
                        int64_t M, int64_t K, void* dw, qmm_dtype dt, void* ws, size_t ws_bytes, qmm_stream_t stream) {
  QMM_TRY(check_dtype(dt, "gradient"));
  QMM_TRY(check_range(N, 0, kMaxWgradTokens, "N"));
  QMM_TRY(check_range(M, 1, qmm::kF8MaxRows, "M"));
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  QMM_TRY(check_ws(ws, ws_bytes, qmm_f8_wgrad_workspace_bytes(N, M, K), "ws"));
  return wgrad(g_codes, g_scales, x_codes, x_scales, N > 0 ? f8_pad(N) : 0, M, K, nullptr, nullptr, dw, dt, ws, stream);
}

qmm_status qmm_f8_wgrad_id(const void* g_codes, const float* g_scales, const void* x_codes, const float* x_scales,
                           int64_t N, int64_t S, int64_t M, int64_t K, int64_t E, const void* plan, void* dw, qmm_dtype dt,
                           qmm_stream_t stream) {
  QMM_TRY(check_dtype(dt, "gradient"));
  QMM_TRY(check_pairs(N, S, E));
  QMM_TRY(check_range(M, 1, qmm::kF8MaxRows, "M"));
  QMM_TRY(check_range(K, 1, kMaxK, "K"));
  const qmm::PlanDesc pd = qmm::plan_desc(N * S, E);
  const int64_t Np = qmm::kF8Block * pd.cap[qmm::kPlanTileKinds - 1];
  return wgrad(g_codes, g_scales, x_codes, x_scales, Np, M, K, plan, &pd, dw, dt, nullptr, stream);
}

size_t qmm_route_workspace_bytes(int64_t N, int64_t E) {
  if (N <= 0 || N > qmm::kF8MaxRows || E < 1 || E > qmm::kRouteMaxExperts) return 0;
  return qmm::route_workspace_bytes(N, E);
}

static qmm_status check_route(int64_t N, int64_t E, int64_t S, int normalise) {
  QMM_TRY(check_range(N, 0, qmm::kF8MaxRows, "N"));
  QMM_TRY(check_range(E, 1, qmm::kRouteMaxExperts, "E"));
  QMM_TRY(check_range(S, 1, E < 64 ? E : 64, "S"));
  if (normalise != 0 && normalise != 1) return fail(QMM_E_ARG, "normalise must be 0 or 1");
  return QMM_OK;
}

qmm_status qmm_route(const void* logits, qmm_dtype lt, int64_t N, int64_t E, int64_t S, const uint8_t* valid, int normalise,
                     float coef, int32_t* ids, float* weights, int32_t* counts, float* psum, float* loss, void* ws,
                     size_t ws_bytes, qmm_stream_t stream) {
  QMM_TRY(check_dtype(lt, "logits"));
  QMM_TRY(check_route(N, E, S, normalise));
  QMM_TRY(check_ptr(counts, 4, "counts"));
  QMM_TRY(check_ptr(psum, 4, "psum"));
  if (!aligned(loss, 4)) return fail(QMM_E_ALIGN, "loss must be 4-byte aligned");
  if (N > 0) {
    QMM_TRY(check_ptr(logits, size_of(lt), "logits"));
    QMM_TRY(check_ptr(ids, 4, "ids"));
    QMM_TRY(check_ptr(weights, 4, "weights"));
    QMM_TRY(check_ws(ws, ws_bytes, qmm_route_workspace_bytes(N, E), "ws"));
  }
  qmm::RouteArgs a{logits, lt, N, static_cast<int>(E), static_cast<int>(S), normalise, coef, valid, ids, weights, counts,
                   psum, loss, ws};
  const hipError_t e = qmm::launch_route(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route launch");
}

qmm_status qmm_balance_loss(const int32_t* counts, const float* psum, int64_t E, int64_t S, float coef, float* loss,
                            qmm_stream_t stream) {
  QMM_TRY(check_route(0, E, S, 0));
  QMM_TRY(check_ptr(counts, 4, "counts"));
  QMM_TRY(check_ptr(psum, 4, "psum"));
  QMM_TRY(check_ptr(loss, 4, "loss"));
  const hipError_t e = qmm::launch_balance_loss(counts, psum, static_cast<int>(E), static_cast<int>(S), coef, loss,
                                                stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "balance loss launch");
}

qmm_status qmm_route_backward(const void* logits, qmm_dtype lt, int64_t N, int64_t E, int64_t S, const uint8_t* valid,
                              int normalise, float coef, const int32_t* ids, const float* dweights, const int32_t* counts,
                              const float* dloss, void* dlogits, qmm_stream_t stream) {
  QMM_TRY(check_dtype(lt, "logits"));
  QMM_TRY(check_route(N, E, S, normalise));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(logits, size_of(lt), "logits"));
  QMM_TRY(check_ptr(dlogits, size_of(lt), "dlogits"));
  if (dweights) {
    QMM_TRY(check_ptr(dweights, 4, "dweights"));
    QMM_TRY(check_ptr(ids, 4, "ids"));
  }
  if (dloss) {
    QMM_TRY(check_ptr(dloss, 4, "dloss"));
    QMM_TRY(check_ptr(counts, 4, "counts"));
  }
  qmm::RouteBackwardArgs a{logits, lt, N, static_cast<int>(E), static_cast<int>(S), normalise, coef, valid, ids, dweights,
                           counts, dloss, dlogits};
  const hipError_t e = qmm::launch_route_backward(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route backward launch");
}

static qmm_status check_combine(int yt, bool weighted, int wt, int64_t N, int64_t S, int64_t M) {
  QMM_TRY(check_dtype(yt, "slot output"));
  if (weighted && wt != QMM_F32 && wt != yt) return fail(QMM_E_TYPE, "weights must be fp32 or of y's type (got %d)", wt);
  QMM_TRY(check_range(N, 0, qmm::kF8MaxRows, "N"));
  QMM_TRY(check_range(S, 1, 64, "S"));
  return check_range(M, 1, qmm::kF8MaxRows, "M");
}

qmm_status qmm_route_combine(const void* y, qmm_dtype yt, const void* weights, qmm_dtype wt, int64_t N, int64_t S,
                             int64_t M, void* out, qmm_stream_t stream) {
  QMM_TRY(check_combine(yt, weights != nullptr, wt, N, S, M));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  if (weights) QMM_TRY(check_ptr(weights, size_of(wt), "weights"));
  QMM_TRY(check_ptr(out, size_of(yt), "out"));
  const hipError_t e = qmm::launch_route_combine(y, yt, weights, wt, N, static_cast<int>(S), M, out, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route combine launch");
}

qmm_status qmm_route_combine_backward(const void* y, qmm_dtype yt, const void* weights, qmm_dtype wt, int64_t N, int64_t S,
                                      int64_t M, const void* dout, void* dy, void* dweights, qmm_stream_t stream) {
  QMM_TRY(check_combine(yt, true, wt, N, S, M));
  if (N == 0) return ok();
  QMM_TRY(check_ptr(y, size_of(yt), "y"));
  QMM_TRY(check_ptr(weights, size_of(wt), "weights"));
  QMM_TRY(check_ptr(dout, size_of(yt), "dout"));
  QMM_TRY(check_ptr(dy, size_of(yt), "dy"));
  QMM_TRY(check_ptr(dweights, size_of(wt), "dweights"));
  const hipError_t e = qmm::launch_route_combine_backward(y, yt, weights, wt, N, static_cast<int>(S), M, dout, dy, dweights,
                                                          stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route combine launch");
}

}  // extern "C"
