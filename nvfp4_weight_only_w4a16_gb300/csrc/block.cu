// C ABI of what a block has around the 4-bit products: routing, norm, SwiGLU, the INT8 linear.  As in api.cu: every entry
// point returns a status and never throws; shape and pointer errors are caught here, before anything is enqueued.
#include <cmath>

#include "handle.h"

using namespace nvfp4moe;

namespace {
constexpr int kMaxRows = 1 << 20;  // of a route, norm or INT8 call

nvfp4_moe_status bad(nvfp4_moe* h, nvfp4_moe_status s, const char* what, const char* msg) {
  snprintf(h->last_error, sizeof(h->last_error), "%s: %s", what, msg);
  if (h->log) fprintf(stderr, "[nvfp4_moe] %s\n", h->last_error);
  return s;
}
nvfp4_moe_status launched(nvfp4_moe* h, cudaError_t e, const char* what) {
  return e == cudaSuccess ? NVFP4_MOE_OK : cuda_fail(h, e, what);
}

// A matrix of rows `cols` long: what is wrong with it, or NULL.
const char* rows_error(const void* p, int64_t ld, int cols, int align = 16, int multiple = 8) {
  if (!p) return "NULL pointer";
  if (!aligned(p, align)) return "misaligned rows";
  if (ld < cols || ld % multiple || ld > (1 << 24)) return "a row stride is below the row length, above 2^24 or not a multiple of what it has to be";
  return nullptr;
}

bool act_ok(int t) { return t == NVFP4_MOE_ACT_BF16 || t == NVFP4_MOE_ACT_F16; }
}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
nvfp4_moe_status nvfp4_route_create(const nvfp4_route_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->num_experts > 512) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->groups < 1 || c->groups > 32 || c->num_experts % c->groups) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->top_groups < 1 || c->top_groups > c->groups) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  const int size = c->num_experts / c->groups;
  if (c->group_top < 1 || c->group_top > 2 || c->group_top > size) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->top_k < 1 || c->top_k > 16 || c->top_k > c->top_groups * size) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->score != NVFP4_MOE_SCORE_SOFTMAX && c->score != NVFP4_MOE_SCORE_SIGMOID) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->renormalize != 0 && c->renormalize != 1) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale)) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->logits_dtype != NVFP4_MOE_LOGITS_F32 && c->logits_dtype != NVFP4_MOE_LOGITS_BF16) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s = create_product(nvfp4_moe::kRoute, c->device, 0, 0, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->route = *c;
  *out = h;
  return NVFP4_MOE_OK;
}

}  // extern "C"

namespace {
nvfp4_moe_status check_logits(nvfp4_moe* h, const char* what, int T, const void* p, int64_t ld) {
  if (T < 0 || T > kMaxRows) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "T outside 0..2^20");
  if (T == 0) return NVFP4_MOE_OK;
  if (!p) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "NULL pointer");
  if (!aligned(p, h->route.logits_dtype == NVFP4_MOE_LOGITS_BF16 ? 2 : 4))
    return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "misaligned logits");
  if (ld < h->route.num_experts || ld > (1 << 24))
    return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "a row stride is below the number of experts or above 2^24");
  return NVFP4_MOE_OK;
}
RouteOp route_op(const nvfp4_moe* h, int T, const void* logits, int64_t ld) {
  const nvfp4_route_config& c = h->route;
  RouteOp p{};
  p.logits = logits, p.ld = ld;
  p.bf16 = c.logits_dtype == NVFP4_MOE_LOGITS_BF16;
  p.T = T, p.E = c.num_experts, p.k = c.top_k;
  p.score = c.score == NVFP4_MOE_SCORE_SIGMOID, p.renorm = c.renormalize, p.scale = c.scale;
  p.groups = c.groups, p.top_groups = c.top_groups, p.group_top = c.group_top;
  p.status = h->ws.status;
  p.num_sms = h->num_sms;
  return p;
}
}  // namespace

extern "C" {

nvfp4_moe_status nvfp4_route_forward(nvfp4_moe_t h, int T, const void* logits, int64_t ld, const float* bias,
                                     int32_t* ids, float* weights, int32_t* offsets, int32_t* perm, int32_t* inv,
                                     cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "route_forward";
  if (h->kind != nvfp4_moe::kRoute) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a route handle");
  const nvfp4_moe_status s = check_logits(h, what, T, logits, ld);
  if (s != NVFP4_MOE_OK) return s;
  if (!offsets || (T && (!ids || !weights || !perm || !inv))) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "NULL pointer");
  if (!aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(inv, 4))
    return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "misaligned pointer");
  DeviceGuard g(h->cfg.device);
  if (T == 0) return launched(h, cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (h->route.num_experts + 1), st), what);
  RouteOp p = route_op(h, T, logits, ld);
  p.bias = bias, p.ids = ids, p.weights = weights, p.offsets = offsets, p.perm = perm, p.inv = inv;
  return launched(h, launch_route_forward(p, st), what);
}

nvfp4_moe_status nvfp4_route_backward(nvfp4_moe_t h, int T, const void* logits, int64_t ld, const int32_t* ids,
                                      const float* dweights, void* dlogits, int64_t ld_dl, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "route_backward";
  if (h->kind != nvfp4_moe::kRoute) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a route handle");
  nvfp4_moe_status s = check_logits(h, what, T, logits, ld);
  if (s == NVFP4_MOE_OK) s = check_logits(h, what, T, dlogits, ld_dl);
  if (s != NVFP4_MOE_OK || T == 0) return s;
  if (!ids || !dweights) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "NULL pointer");
  if (!aligned(ids, 4) || !aligned(dweights, 4)) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "misaligned pointer");
  DeviceGuard g(h->cfg.device);
  RouteOp p = route_op(h, T, logits, ld);
  p.ids = const_cast<int32_t*>(ids), p.dweights = dweights, p.dlogits = dlogits, p.ld_dl = ld_dl;
  return launched(h, launch_route_backward(p, st), what);
}

// ---------------------------------------------------------------------------
// Norm
// ---------------------------------------------------------------------------
nvfp4_moe_status nvfp4_norm_create(const nvfp4_norm_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->hidden < 8 || c->hidden > 16384 || c->hidden % 8) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (!(c->eps >= 0.0f) || !std::isfinite(c->eps) || !act_ok(c->act_dtype)) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MOE_ERR_CUDA;
  }
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s =
      create_product(nvfp4_moe::kNorm, c->device, sizeof(float) * norm_backward_parts(c->hidden, sms) * c->hidden, 0, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->norm = *c;
  *out = h;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_norm_forward(nvfp4_moe_t h, int T, const void* x, int64_t ldx, const void* residual,
                                    int64_t ld_res, const void* weight, void* sum, int64_t ld_sum, void* y, int64_t ldy,
                                    int8_t* q, int64_t ldq, float* q_scale, float* rstd, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "norm_forward";
  if (h->kind != nvfp4_moe::kNorm) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a norm handle");
  if (T < 0 || T > kMaxRows) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "T outside 0..2^20");
  if (T == 0) return NVFP4_MOE_OK;
  const int H = h->norm.hidden;
  const char* e = rows_error(x, ldx, H);
  if (!e && residual) e = rows_error(residual, ld_res, H);
  if (!e && residual) e = rows_error(sum, ld_sum, H);
  if (!e && !residual && sum) e = "a sum without a residual";
  if (!e && !y && !q) e = "neither y nor q";
  if (!e && y) e = rows_error(y, ldy, H);
  if (!e && q) e = rows_error(q, ldq, H, 8);
  if (!e && (!weight || (q && !q_scale))) e = "NULL pointer";
  if (!e && (!aligned(weight, 16) || !aligned(q_scale, 4) || !aligned(rstd, 4))) e = "misaligned pointer";
  if (e) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, e);
  DeviceGuard g(h->cfg.device);
  NormOp p{};
  p.x = x, p.ldx = ldx, p.res = residual, p.ldr = ld_res, p.weight = weight;
  p.sum = sum, p.lds = ld_sum, p.y = y, p.ldy = ldy, p.q = q, p.ldq = ldq, p.q_scale = q_scale, p.rstd = rstd;
  p.T = T, p.H = H, p.f16 = h->norm.act_dtype == NVFP4_MOE_ACT_F16, p.num_sms = h->num_sms, p.eps = h->norm.eps;
  return launched(h, launch_norm_forward(p, st), what);
}

nvfp4_moe_status nvfp4_norm_backward(nvfp4_moe_t h, int T, const void* dy, int64_t ld_dy, const void* sum,
                                     int64_t ld_sum, const void* weight, const float* rstd, const void* dsum,
                                     int64_t ld_dsum, void* dx, int64_t ld_dx, float* dweight, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "norm_backward";
  if (h->kind != nvfp4_moe::kNorm) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a norm handle");
  if (T < 0 || T > kMaxRows) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "T outside 0..2^20");
  const int H = h->norm.hidden;
  if (!aligned(dweight, 16)) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "misaligned pointer");
  DeviceGuard g(h->cfg.device);
  if (T == 0) return dweight ? launched(h, cudaMemsetAsync(dweight, 0, sizeof(float) * H, st), what) : NVFP4_MOE_OK;
  const char* e = rows_error(dy, ld_dy, H);
  if (!e) e = rows_error(sum, ld_sum, H);
  if (!e && dsum) e = rows_error(dsum, ld_dsum, H);
  if (!e) e = rows_error(dx, ld_dx, H);
  if (!e && (!weight || !rstd)) e = "NULL pointer";
  if (!e && (!aligned(weight, 16) || !aligned(rstd, 4))) e = "misaligned pointer";
  if (e) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, e);
  NormBackOp p{};
  p.dy = dy, p.ld_dy = ld_dy, p.x = sum, p.ldx = ld_sum, p.weight = weight, p.rstd = rstd;
  p.dsum = dsum, p.ld_dsum = ld_dsum, p.dx = dx, p.ld_dx = ld_dx;
  p.dweight = dweight, p.part = reinterpret_cast<float*>(h->blob), p.status = h->ws.status;
  p.T = T, p.H = H, p.f16 = h->norm.act_dtype == NVFP4_MOE_ACT_F16, p.num_sms = h->num_sms;
  return launched(h, launch_norm_backward(p, st), what);
}

// ---------------------------------------------------------------------------
// SwiGLU
// ---------------------------------------------------------------------------
nvfp4_moe_status nvfp4_swiglu_create(const nvfp4_swiglu_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->inter < 16 || c->inter > 16384 || c->inter % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (!act_ok(c->act_dtype) || !device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s = create_product(nvfp4_moe::kSwiglu, c->device, 0, 0, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->swiglu = *c;
  *out = h;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_swiglu_forward(nvfp4_moe_t h, int R, const void* gate, int64_t ld_gate, const void* up,
                                      int64_t ld_up, void* out, int64_t ld_out, int8_t* codes, float* scales,
                                      cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "swiglu_forward";
  if (h->kind != nvfp4_moe::kSwiglu) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a SwiGLU handle");
  if (R < 0 || R > (1 << 24)) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "R outside 0..2^24");
  if (R == 0) return NVFP4_MOE_OK;
  const int I = h->swiglu.inter;
  const char* e = rows_error(gate, ld_gate, I);
  if (!e) e = rows_error(up, ld_up, I);
  if (!e) e = rows_error(out, ld_out, I);
  if (!e && !codes != !scales) e = "codes without scales, or scales without codes";
  if (!e && (!aligned(codes, 16) || !aligned(scales, 4))) e = "misaligned pointer";
  if (e) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, e);
  DeviceGuard g(h->cfg.device);
  SwigluOp p{};
  p.gate = gate, p.ld_gate = ld_gate, p.up = up, p.ld_up = ld_up, p.h = out, p.ld_h = ld_out;
  p.codes = codes, p.scales = scales;
  p.R = R, p.I = I, p.f16 = h->swiglu.act_dtype == NVFP4_MOE_ACT_F16, p.num_sms = h->num_sms;
  return launched(h, launch_swiglu_forward(p, st), what);
}

nvfp4_moe_status nvfp4_swiglu_backward(nvfp4_moe_t h, int R, const int8_t* codes, const float* scales, const void* dh,
                                       int64_t ld_dh, void* dgate, int64_t ld_dgate, void* dup, int64_t ld_dup,
                                       cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "swiglu_backward";
  if (h->kind != nvfp4_moe::kSwiglu) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not a SwiGLU handle");
  if (R < 0 || R > (1 << 24)) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "R outside 0..2^24");
  if (R == 0) return NVFP4_MOE_OK;
  const int I = h->swiglu.inter;
  const char* e = rows_error(dh, ld_dh, I);
  if (!e) e = rows_error(dgate, ld_dgate, I);
  if (!e) e = rows_error(dup, ld_dup, I);
  if (!e && (!codes || !scales)) e = "NULL pointer";
  if (!e && (!aligned(codes, 16) || !aligned(scales, 4))) e = "misaligned pointer";
  if (e) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, e);
  DeviceGuard g(h->cfg.device);
  SwigluOp p{};
  p.codes = const_cast<int8_t*>(codes), p.scales = const_cast<float*>(scales);
  p.dh = dh, p.ld_dh = ld_dh, p.dgate = dgate, p.ld_dgate = ld_dgate, p.dup = dup, p.ld_dup = ld_dup;
  p.R = R, p.I = I, p.f16 = h->swiglu.act_dtype == NVFP4_MOE_ACT_F16, p.num_sms = h->num_sms;
  return launched(h, launch_swiglu_backward(p, st), what);
}

// ---------------------------------------------------------------------------
// INT8 linear
// ---------------------------------------------------------------------------
nvfp4_moe_status nvfp4_int8_create(const nvfp4_int8_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->out_features < 16 || c->out_features > (1 << 20) || c->out_features % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->in_features < 16 || c->in_features > 16384 || c->in_features % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_tokens < 1 || c->max_tokens > kMaxRows) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->out_dtype < NVFP4_MOE_OUT_BF16 || c->out_dtype > NVFP4_MOE_OUT_F16) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s = create_product(nvfp4_moe::kInt8, c->device, int8_packed_bytes(c->out_features, c->in_features),
                                            2 * c->out_features, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->i8 = *c;
  const size_t bytes = int8_workspace_bytes(c->in_features, c->max_tokens);
  if (bytes) {
    DeviceGuard g(c->device);
    if (cudaMalloc(&h->ws_mem2, bytes) != cudaSuccess) {
      cudaGetLastError();
      nvfp4_moe_destroy(h);
      return NVFP4_MOE_ERR_WORKSPACE;
    }
  }
  *out = h;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_int8_pack(nvfp4_moe_t h, const int8_t* w, const float* w_scale, const float* bias,
                                 cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "int8_pack";
  if (h->kind != nvfp4_moe::kInt8) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not an INT8 handle");
  if (!w || !w_scale) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "NULL input");
  if (!aligned(w, 16) || !aligned(w_scale, 4) || !aligned(bias, 4))
    return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "misaligned input");
  DeviceGuard g(h->cfg.device);
  const int N = h->i8.out_features;
  float* host = new (std::nothrow) float[N];
  if (!host) return bad(h, NVFP4_MOE_ERR_WORKSPACE, what, "out of host memory");
  h->packed = false;  // until all of it is done
  cudaError_t e = cudaMemcpyAsync(host, w_scale, sizeof(float) * N, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  bool finite = true;
  for (int i = 0; e == cudaSuccess && i < N; ++i) finite &= std::isfinite(host[i]);
  delete[] host;
  if (e != cudaSuccess) return cuda_fail(h, e, "int8_pack: reading w_scale");
  if (!finite) return bad(h, NVFP4_MOE_ERR_BAD_SCALE, what, "a scale is not finite");
  e = cudaMemcpyAsync(h->gscale, w_scale, sizeof(float) * N, cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess && bias) e = cudaMemcpyAsync(h->gscale + N, bias, sizeof(float) * N, cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess) e = launch_pack_int8(w, N, h->i8.in_features, h->blob, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, what);
  h->i8_bias = bias != nullptr;
  h->packed = true;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_int8_quantize(nvfp4_moe_t h, int T, const void* x, int x_dtype, int64_t ldx, int8_t* q,
                                     int64_t ldq, float* q_scale, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "int8_quantize";
  if (h->kind != nvfp4_moe::kInt8) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not an INT8 handle");
  if (T < 0 || T > kMaxRows) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "T outside 0..2^20");
  if (!act_ok(x_dtype)) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "unknown type of x");
  if (T == 0) return NVFP4_MOE_OK;
  const int K = h->i8.in_features;
  const char* e = rows_error(x, ldx, K);
  if (!e) e = rows_error(q, ldq, K, 8);
  if (!e && (!q_scale || !aligned(q_scale, 4))) e = "q_scale is NULL or misaligned";
  if (e) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, e);
  DeviceGuard g(h->cfg.device);
  NormOp p{};
  p.x = x, p.ldx = ldx, p.q = q, p.ldq = ldq, p.q_scale = q_scale;
  p.T = T, p.H = K, p.f16 = x_dtype == NVFP4_MOE_ACT_F16, p.num_sms = h->num_sms;
  return launched(h, launch_norm_forward(p, st), what);
}

nvfp4_moe_status nvfp4_int8_forward(nvfp4_moe_t h, int T, const int8_t* x, int64_t ldx, const float* x_scale, void* out,
                                    int64_t ldo, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const char* what = "int8_forward";
  if (h->kind != nvfp4_moe::kInt8) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, "not an INT8 handle");
  if (!h->packed) return bad(h, NVFP4_MOE_ERR_NOT_PACKED, what, "before a successful pack");
  if (T < 0 || T > h->i8.max_tokens) return bad(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, what, "T outside 0..max_tokens");
  if (T == 0) return NVFP4_MOE_OK;
  const int N = h->i8.out_features, K = h->i8.in_features;
  const char* err = rows_error(x, ldx, K, 16, 16);
  if (!err) err = rows_error(out, ldo, N);
  if (!err && (!x_scale || !aligned(x_scale, 4))) err = "x_scale is NULL or misaligned";
  if (err) return bad(h, NVFP4_MOE_ERR_INVALID_ARG, what, err);
  DeviceGuard g(h->cfg.device);
  Int8Product p{};
  p.packed = h->blob, p.w_scale = h->gscale, p.bias = h->i8_bias ? h->gscale + N : nullptr;
  p.N = N, p.K = K, p.T = T;
  p.x = x, p.x_scale = x_scale, p.ldx = ldx, p.out = out, p.ldo = ldo;
  p.out_type = h->i8.out_dtype;
  p.once = h->product_bytes > h->l2_bytes;
  p.num_sms = h->num_sms, p.status = h->ws.status, p.fault = h->fault;
  cudaEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
  const nvfp4_moe_status s = take_events(h, ev);
  if (s != NVFP4_MOE_OK) return s;
  record(ev, 0, 2, st);
  cudaError_t e = cudaSuccess;
  if (T <= kDecodeMaxTokens) {
    e = launch_int8_gemv(p, st);
  } else {
    const int chunk = int8_chunk_tokens(K), Kp = (K + 127) / 128 * 128, size = p.out_type == NVFP4_MOE_OUT_F32 ? 4 : 2;
    for (int t0 = 0; t0 < T && e == cudaSuccess; t0 += chunk) {
      p.T = T - t0 < chunk ? T - t0 : chunk;
      p.x = x + t0 * ldx, p.x_scale = x_scale + t0, p.out = static_cast<uint8_t*>(out) + t0 * ldo * size;
      const Int8Tiling t = int8_tiling(N, K, p.T, h->num_sms);
      CUtensorMap map{};
      if (t.fp16) e = launch_int8_tokens(p, h->ws_mem2, st);
      if (e != cudaSuccess) break;
      if (!(t.fp16 ? encode_rows_map(&map, h->ws_mem2, (uint64_t)p.T, (uint64_t)Kp, (uint32_t)t.box)
                   : encode_bytes_map(&map, p.x, (uint64_t)p.T, (uint64_t)K, (uint32_t)t.box, (uint64_t)ldx)))
        return bad(h, NVFP4_MOE_ERR_CUDA, what, "cuTensorMapEncodeTiled failed");
      e = launch_int8_gemm(p, t, map, st);
    }
  }
  if (e != cudaSuccess) return cuda_fail(h, e, what);
  record(ev, 3, 4, st);
  return NVFP4_MOE_OK;
}

}  // extern "C"
