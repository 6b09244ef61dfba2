// C ABI of the NVFP4 W4A16 MoE layer: handle, validation, dispatch.
// Every entry point returns a status and never throws; shape and pointer
// errors are caught here, before anything is enqueued.
#include <cstdio>
#include <cstdlib>
#include <algorithm>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "handle.h"

using namespace nvfp4moe;

namespace {

struct Carver {
  size_t off = 0;
  std::vector<std::pair<void**, size_t>> items;
  std::vector<bool> is_data;  // rewritten by every forward before it is read (no counter, no constant)
  template <class T>
  void add(T** p, size_t count, bool data = false) {
    items.push_back({reinterpret_cast<void**>(p), count * sizeof(T)});
    is_data.push_back(data);
  }
  size_t layout() {
    off = 0;
    for (auto& it : items) off = ((off + 255) & ~size_t(255)) + it.second;
    return off + 256;
  }
  void assign(uint8_t* base) {
    size_t o = 0;
    for (auto& it : items) {
      o = (o + 255) & ~size_t(255);
      *it.first = base + o;
      o += it.second;
    }
  }
};

int choose_path(const nvfp4_moe* h, int T, int k) {
  if (h->path != NVFP4_MOE_PATH_AUTO) return h->path;
  return (T <= h->cfg.decode_max_tokens && T <= kDecodeMaxTokens &&
          T * (k + h->cfg.num_shared_experts) <= kDecodeMaxTokens * 16)
             ? NVFP4_MOE_PATH_DECODE
             : NVFP4_MOE_PATH_PREFILL;
}

nvfp4_moe_status check_forward_args(nvfp4_moe* h, const void* logits, int T, int top_k, int path) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "not an MoE handle: call its own forward");
  if (!h->packed) return fail(h, NVFP4_MOE_ERR_NOT_PACKED, "forward before a successful pack");
  if (!logits) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "router_logits is NULL");
  if (!aligned(logits, h->cfg.logits_dtype == NVFP4_MOE_LOGITS_BF16 ? 2 : 4))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "router_logits misaligned");
  if (T < 1 || T > h->cfg.max_tokens) return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "T outside 1..max_tokens");
  if (top_k < 1 || top_k > h->cfg.max_top_k || top_k > h->cfg.num_experts)
    return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "top_k outside 1..min(max_top_k, E)");
  if (path == NVFP4_MOE_PATH_DECODE && (T > kDecodeMaxTokens))
    return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "decode path takes at most 16 tokens");
  if (path == NVFP4_MOE_PATH_DECODE && T * (top_k + h->cfg.num_shared_experts) > kDecodeMaxTokens * 16)
    return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "decode path takes at most 256 routed rows");
  return NVFP4_MOE_OK;
}

LayerDims dims_of(const nvfp4_moe* h) {
  LayerDims d{h->cfg.num_experts + h->cfg.num_shared_experts, h->cfg.hidden, h->cfg.inter,
              h->cfg.logits_dtype == NVFP4_MOE_LOGITS_BF16, h->cfg.out_dtype == NVFP4_MOE_OUT_F32,
              h->cfg.num_experts, h->cfg.num_shared_experts, h->linear ? 1 : 0, h->lin_n};
  d.rp = h->rp;
  d.in_scale = h->w4a4 ? h->in_scale : nullptr;
  d.gs = h->w4a4 ? h->gs_eff : h->gscale;
  d.hbound = h->hbound;
  d.checks = h->checks;
  return d;
}

size_t blob_bytes_of(const nvfp4_moe_config& c, bool linear) {
  return linear ? linear_layout(c.hidden, c.inter).stride
                : (size_t)(c.num_experts + c.num_shared_experts) * expert_layout(c.hidden, c.inter).stride;
}

// Handle allocation shared by the MoE layer and the dense linear (c already
// validated; a linear's c holds one expert with hidden = N and inter = K).
nvfp4_moe_status create_handle(const nvfp4_moe_config* c, bool linear, int lin_n, nvfp4_moe_t* out);

// W4A4: tensor scales with the input scales folded in (routed experts: gate and
// up times is_w13, down times is_w2; the shared expert keeps its own).
nvfp4_moe_status upload_gs_eff(nvfp4_moe* h, cudaStream_t st) {
  const int E = h->cfg.num_experts + h->cfg.num_shared_experts, Er = h->cfg.num_experts;
  if (h->gs_host.size() != (size_t)3 * E) return NVFP4_MOE_OK;  // not packed yet: pack uploads it
  std::vector<float> g(h->gs_host);
  for (int e = 0; e < Er; ++e) {
    g[3 * e] *= h->is_host[2 * e];
    g[3 * e + 1] *= h->is_host[2 * e];
    g[3 * e + 2] *= h->is_host[2 * e + 1];
  }
  cudaError_t err = cudaMemcpyAsync(h->gs_eff, g.data(), sizeof(float) * g.size(), cudaMemcpyHostToDevice, st);
  if (err == cudaSuccess) err = cudaStreamSynchronize(st);  // g lives on this frame
  if (err != cudaSuccess) return cuda_fail(h, err, "W4A4 tensor scales upload");
  return NVFP4_MOE_OK;
}

// The decode forward takes the streaming kernel wherever it applies (W4A16
// routed experts); NVFP4_MOE_DECODE_KERNEL=fused keeps the earlier fused
// kernel for comparison.
bool use_stream(const nvfp4_moe* h, const LayerDims& d, int T, int k) {
  static const bool fused = [] {
    const char* s = getenv("NVFP4_MOE_DECODE_KERNEL");
    return s && !strcmp(s, "fused");
  }();
  (void)h;
  return !fused && stream_supported(d, T, k);
}

nvfp4_moe_status run_route(nvfp4_moe* h, const void* logits, const void* x, int T, int k, int path,
                           cudaStream_t st, int logits_bf16 = -1) {
  LayerDims d = dims_of(h);
  if (logits_bf16 >= 0) d.logits_bf16 = logits_bf16;
  cudaError_t e = path != NVFP4_MOE_PATH_DECODE ? launch_route_prefill(d, logits, x, T, k, h->ws, st)
                   : use_stream(h, d, T, k)
                       ? launch_decode_stream(d, h->blob, h->gscale, logits, nullptr, T, k, nullptr, 1, h->num_sms,
                                              h->ws, 0, st)
                       : launch_decode_forward(d, h->blob, h->gscale, logits, nullptr, T, k, nullptr, 1, h->num_sms,
                                               h->ws, 0, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "route launch");
  return NVFP4_MOE_OK;
}

}  // namespace

extern "C" {

const char* nvfp4_moe_status_string(nvfp4_moe_status s) {
  switch (s) {
    case NVFP4_MOE_OK: return "ok";
    case NVFP4_MOE_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_MOE_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case NVFP4_MOE_ERR_NOT_PACKED: return "weights not packed";
    case NVFP4_MOE_ERR_WORKSPACE: return "device allocation failed";
    case NVFP4_MOE_ERR_CUDA: return "CUDA error";
    case NVFP4_MOE_ERR_TIMEOUT: return "device-side wait timed out";
    case NVFP4_MOE_ERR_BAD_SCALE: return "tensor scale is zero, negative, NaN or Inf";
    case NVFP4_MOE_ERR_NOT_IMPLEMENTED: return "not implemented";
    case NVFP4_MOE_ERR_DEVICE_CHECK: return "device-side bounds check fired";
  }
  return "unknown status";
}

const char* nvfp4_moe_last_error(nvfp4_moe_t h) { return h ? h->last_error : "null handle"; }

nvfp4_moe_status nvfp4_moe_create(const nvfp4_moe_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->num_experts > 256) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->hidden < 128 || c->hidden > 16384 || c->hidden % 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->inter < 128 || c->inter > 16384 || c->inter % 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_tokens < 1 || c->max_tokens > (1 << 20)) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_top_k < 1 || c->max_top_k > 16 || c->max_top_k > c->num_experts) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->decode_max_tokens < 0 || c->decode_max_tokens > kDecodeMaxTokens) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->logits_dtype != NVFP4_MOE_LOGITS_F32 && c->logits_dtype != NVFP4_MOE_LOGITS_BF16)
    return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->out_dtype != NVFP4_MOE_OUT_BF16 && c->out_dtype != NVFP4_MOE_OUT_F32) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->num_shared_experts < 0 || c->num_shared_experts > 1) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->num_experts + c->num_shared_experts > 256 || c->max_top_k + c->num_shared_experts > 16)
    return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || c->device < 0 || c->device >= ndev) return NVFP4_MOE_ERR_INVALID_ARG;
  return create_handle(c, false, 0, out);
}

}  // extern "C"

namespace {
nvfp4_moe_status create_handle(const nvfp4_moe_config* c, bool linear, int lin_n, nvfp4_moe_t* out) {
  nvfp4_moe* h = new (std::nothrow) nvfp4_moe();
  if (!h) return NVFP4_MOE_ERR_WORKSPACE;
  h->cfg = *c;
  h->linear = linear;
  h->lin_n = lin_n;
  const char* lg = getenv("NVFP4_MOE_LOG");
  h->log = lg && lg[0] == '1';
  const char* ck = getenv("NVFP4_MOE_CHECKS");
  h->checks = ck && ck[0] == '1';
  const char* fp = getenv("NVFP4_MOE_FORCE_PATH");
  if (fp && !strcmp(fp, "decode")) h->path = NVFP4_MOE_PATH_DECODE;
  if (fp && !strcmp(fp, "prefill")) h->path = NVFP4_MOE_PATH_PREFILL;

  DeviceGuard g(c->device);
  cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, c->device);
  // E: experts in the blob (routed + shared); K: routed-row slots per token
  const int E = c->num_experts + c->num_shared_experts, H = c->hidden, I = c->inter;
  const int K = c->max_top_k + c->num_shared_experts;
  const size_t R = (size_t)c->max_tokens * K;
  const size_t Rm = R < 256 ? 256 : R;
  const size_t maxU = (size_t)std::min(E, kDecodeMaxTokens * K);
  const size_t ncta = ((size_t)c->max_tokens + kRankTokens - 1) / kRankTokens;
  // m-tiles: the MoE's (<= R/128 + E + 1) and the router GEMM's (<= one per SM)
  const size_t max_tiles = std::max(R / kTileRows + E + 1, (size_t)h->num_sms + 2);
  const size_t blob_bytes = blob_bytes_of(*c, linear);
  // a dense linear reads x and writes out directly: no permuted copies, no
  // hidden rows, no FP32 expert outputs
  const size_t RmH = linear ? 1 : Rm * H, RmI = linear ? 1 : Rm * I;

  Carver cv;
  Workspace& w = h->ws;
  cv.add(&w.ids, Rm, true);
  cv.add(&w.wts, Rm, true);
  cv.add(&w.offsets, E + 1, true);
  cv.add(&w.perm, Rm, true);
  cv.add(&w.inv, Rm, true);
  cv.add(&w.tch_expert, E, true);
  cv.add(&w.tch_row0, E, true);
  cv.add(&w.tch_rows, E, true);
  cv.add(&w.num_touched, 1);
  cv.add(&w.x16, (size_t)kDecodeMaxTokens * H, true);
  cv.add(&w.xexp, kDecodeMaxTokens, true);
  cv.add(&w.h, RmI, true);
  cv.add(&w.hmax, Rm);
  cv.add(&w.y, RmH, true);
  cv.add(&w.part_gu, decode_part_floats(h->num_sms, kDecodeMaxTokens), true);
  cv.add(&w.cnt_gu, maxU * (2 * I / 16));
  cv.add(&w.part_dn, decode_part_floats(h->num_sms, kDecodeMaxTokens), true);
  cv.add(&w.cnt_dn, maxU * (H / 16));
  cv.add(&w.done_gu, maxU);
  cv.add(&w.cmb, H / 64);
  cv.add(&w.exit_cnt, 1);
  w.act_rows = kDecodeMaxTokens * K;  // a dense linear: K = 1, its x rows as the "h" rows
  cv.add(&w.act_h, stream_act_h_bytes(I, w.act_rows), true);
  cv.add(&w.act_x, linear ? 16 : stream_act_x_bytes(H), true);
  cv.add(&w.wctr, 1);
  cv.add(&w.done_c, maxU * (I / 64));
  cv.add(&w.x_ready, H / 64);
  cv.add(&w.logit_ready, 1);
  cv.add(&w.blk_counts, ncta * E, true);
  cv.add(&w.blk_base, ncta * E, true);
  cv.add(&w.local_rank, Rm, true);
  cv.add(&w.x_perm, RmH, true);
  cv.add(&w.pexp_x, Rm, true);
  cv.add(&w.pexp_h, Rm, true);
  cv.add(&w.tile_expert, max_tiles, true);
  cv.add(&w.tile_row0, max_tiles, true);
  cv.add(&w.tile_rows, max_tiles, true);
  cv.add(&w.num_tiles, 1, true);
  cv.add(&w.status, 1);
  cv.add(&w.logits, linear ? 1 : (size_t)c->max_tokens * c->num_experts, true);
  cv.add(&w.ones3, 3);
  const char* tr = getenv("NVFP4_MOE_TRACE");
  const bool trace = tr && tr[0] == '1';
  if (trace) cv.add(&w.trace, (size_t)h->num_sms * 16 * 16);
  h->ws_bytes = cv.layout();

  if (cudaMalloc(&h->blob, blob_bytes) != cudaSuccess || cudaMalloc(&h->gscale, sizeof(float) * 3 * E) != cudaSuccess ||
      cudaMalloc(&h->bias, sizeof(float) * E) != cudaSuccess || cudaMalloc(&h->in_scale, sizeof(float) * 2 * E) != cudaSuccess ||
      cudaMalloc(&h->gs_eff, sizeof(float) * 3 * E) != cudaSuccess || cudaMalloc(&h->hbound, sizeof(float) * E) != cudaSuccess ||
      cudaMalloc(&h->ws_mem, h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    nvfp4_moe_destroy(h);
    return NVFP4_MOE_ERR_WORKSPACE;
  }
  cv.assign(static_cast<uint8_t*>(h->ws_mem));
  for (size_t i = 0; i < cv.items.size(); ++i)
    if (cv.is_data[i]) h->data_regions.push_back({static_cast<uint8_t*>(*cv.items[i].first), cv.items[i].second});
  const float ones[3] = {1.0f, 1.0f, 1.0f};
  if (cudaMemset(h->ws_mem, 0, h->ws_bytes) != cudaSuccess ||
      cudaMemcpy(w.ones3, ones, sizeof(ones), cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaGetLastError();
    nvfp4_moe_destroy(h);
    return NVFP4_MOE_ERR_CUDA;
  }
  if (!linear && (!encode_rows_map(&h->maps.x_perm, w.x_perm, Rm, H) || !encode_rows_map(&h->maps.h, w.h, Rm, I))) {
    nvfp4_moe_destroy(h);
    return NVFP4_MOE_ERR_CUDA;
  }
  *out = h;
  return NVFP4_MOE_OK;
}
}  // namespace

extern "C" {

void nvfp4_moe_destroy(nvfp4_moe_t h) {
  if (!h) return;
  {
    DeviceGuard g(h->cfg.device);
    cudaDeviceSynchronize();
    for (cudaEvent_t ev : h->ev_pool) cudaEventDestroy(ev);
    if (h->blob) cudaFree(h->blob);
    if (h->gscale) cudaFree(h->gscale);
    if (h->bias) cudaFree(h->bias);
    if (h->w_router) cudaFree(h->w_router);
    if (h->in_scale) cudaFree(h->in_scale);
    if (h->gs_eff) cudaFree(h->gs_eff);
    if (h->hbound) cudaFree(h->hbound);
    if (h->ws_mem) cudaFree(h->ws_mem);
    if (h->ws_mem2) cudaFree(h->ws_mem2);
    cudaGetLastError();
  }
  delete h;
}

nvfp4_moe_status nvfp4_moe_set_path(nvfp4_moe_t h, int path) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (path < NVFP4_MOE_PATH_AUTO || path > NVFP4_MOE_PATH_PREFILL) return NVFP4_MOE_ERR_INVALID_ARG;
  h->path = path;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_set_profiling(nvfp4_moe_t h, int on) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  h->profiling = on != 0;
  h->ev_used = 0;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_get_stage_times(nvfp4_moe_t h, float* ms, int* count) {
  if (!h || !ms || !count) return NVFP4_MOE_ERR_INVALID_ARG;
  DeviceGuard g(h->cfg.device);
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(h, e, "get_stage_times");
  for (int i = 0; i < 4; ++i) ms[i] = 0.f;
  const int n = (int)(h->ev_used / 5);
  for (int f = 0; f < n; ++f)
    for (int i = 0; i < 4; ++i) {
      float t = 0.f;
      e = cudaEventElapsedTime(&t, h->ev_pool[5 * f + i], h->ev_pool[5 * f + i + 1]);
      if (e != cudaSuccess) return cuda_fail(h, e, "get_stage_times elapsed");
      ms[i] += t;
    }
  *count = n;
  h->ev_used = 0;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_set_scoring(nvfp4_moe_t h, int score_func, int renormalize, float scale,
                                       const float* bias, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_scoring: a dense linear has no routing");
  if (score_func != NVFP4_MOE_SCORE_SOFTMAX && score_func != NVFP4_MOE_SCORE_SIGMOID)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_scoring: unknown score function");
  if (renormalize != 0 && renormalize != 1) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_scoring: renormalize is 0 or 1");
  if (!(scale > 0.0f) || scale > 3.4e38f) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_scoring: scale must be finite > 0");
  if (bias && !aligned(bias, 4)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_scoring: bias misaligned");
  DeviceGuard g(h->cfg.device);
  if (bias) {
    cudaError_t e = cudaMemcpyAsync(h->bias, bias, sizeof(float) * h->cfg.num_experts, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "set_scoring: bias copy");
  }
  h->rp.score = score_func;
  h->rp.renorm = renormalize;
  h->rp.scale = scale;
  h->rp.bias = bias ? h->bias : nullptr;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_set_act_quant(nvfp4_moe_t h, const float* input_scale, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_act_quant: not for a dense-linear handle");
  if (!input_scale) {
    h->w4a4 = false;
    return NVFP4_MOE_OK;
  }
  if (!aligned(input_scale, 4)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_act_quant: misaligned input_scale");
  DeviceGuard g(h->cfg.device);
  const int E = h->cfg.num_experts + h->cfg.num_shared_experts, Er = h->cfg.num_experts;
  std::vector<float> is((size_t)2 * E, 0.0f);
  cudaError_t e = cudaMemcpyAsync(is.data(), input_scale, sizeof(float) * 2 * Er, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "set_act_quant: reading input_scale");
  for (int i = 0; i < 2 * Er; ++i) {
    const float v = is[i];
    if (!(v > 0.0f) || v != v || v > 3.4e38f) {
      h->w4a4 = false;
      return fail(h, NVFP4_MOE_ERR_BAD_SCALE, "set_act_quant: input scale " + std::to_string(i % 2) + " of expert " +
                                                  std::to_string(i / 2) + " is not finite > 0");
    }
  }
  e = cudaMemcpyAsync(h->in_scale, is.data(), sizeof(float) * is.size(), cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "set_act_quant: input_scale upload");
  h->is_host = is;
  h->w4a4 = true;
  return upload_gs_eff(h, st);
}

nvfp4_moe_status nvfp4_moe_debug_poison_workspace(nvfp4_moe_t h, int byte, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (byte < 0 || byte > 255) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_poison_workspace: byte out of range");
  DeviceGuard g(h->cfg.device);
  for (const auto& r : h->data_regions) {
    const cudaError_t e = cudaMemsetAsync(r.first, byte, r.second, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "debug_poison_workspace");
  }
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_decode_status_word(uint32_t flags) {
  if (flags & kFlagTimeout) return NVFP4_MOE_ERR_TIMEOUT;
  if (flags & kFlagBounds) return NVFP4_MOE_ERR_DEVICE_CHECK;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_set_fault(nvfp4_moe_t h, int fault) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (fault < 0 || fault > 1) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_set_fault: unknown fault");
  h->fault = fault;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_pack(nvfp4_moe_t h, const uint8_t* w13_q, const uint8_t* w13_s, const uint8_t* w2_q,
                                const uint8_t* w2_s, const float* gscale, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "not an MoE handle: call its own pack");
  if (!w13_q || !w13_s || !w2_q || !w2_s || !gscale) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "pack: NULL input");
  if (!aligned(w13_q, 16) || !aligned(w2_q, 16) || !aligned(w13_s, 4) || !aligned(w2_s, 4) || !aligned(gscale, 4))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "pack: misaligned input");
  DeviceGuard g(h->cfg.device);
  const int E = h->cfg.num_experts + h->cfg.num_shared_experts;
  std::vector<float> gs((size_t)3 * E);
  h->packed = false;  // until all of it is done
  cudaError_t e = cudaMemcpyAsync(gs.data(), gscale, sizeof(float) * gs.size(), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "pack: reading gscale");
  for (size_t i = 0; i < gs.size(); ++i) {
    const float v = gs[i];
    if (!(v > 0.0f) || v != v || v > 3.4e38f) {
      return fail(h, NVFP4_MOE_ERR_BAD_SCALE,
                  "pack: tensor scale " + std::to_string(i % 3) + " of expert " + std::to_string(i / 3) + " is not finite > 0");
    }
  }
  e = cudaMemcpyAsync(h->gscale, gscale, sizeof(float) * gs.size(), cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess) e = launch_pack(w13_q, w13_s, w2_q, w2_s, h->blob, E, h->cfg.hidden, h->cfg.inter, st);
  if (e == cudaSuccess) e = launch_gateup_bound(w13_q, w13_s, E, h->cfg.hidden, h->cfg.inter, h->hbound, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "pack launch");
  h->gs_host = gs;
  if (h->w4a4) {
    nvfp4_moe_status s2 = upload_gs_eff(h, st);
    if (s2 != NVFP4_MOE_OK) return s2;
  }
  h->packed = true;
  return NVFP4_MOE_OK;
}

}  // extern "C"

namespace {
// One forward.  routed: the logits are computed here from x and the router
// weight (into the workspace) instead of being passed in.
nvfp4_moe_status forward_impl(nvfp4_moe* h, const void* logits, int T, int top_k, const void* x, void* out,
                              cudaStream_t st, bool routed) {
  const int path = choose_path(h, T, top_k);
  nvfp4_moe_status s = check_forward_args(h, routed ? h->ws.logits : logits, T, top_k, path);
  if (s != NVFP4_MOE_OK) return s;
  if (!x || !out) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "x or out is NULL");
  if (!aligned(x, 16) || !aligned(out, 16)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "x or out not 16-byte aligned");
  if (routed && !h->have_router) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "forward_routed before set_router");
  DeviceGuard g(h->cfg.device);
  CUtensorMap x_map{};
  if (routed && T > kDecodeMaxTokens &&
      !encode_rows_map(&x_map, const_cast<void*>(x), (uint64_t)T, (uint64_t)h->cfg.hidden))
    return fail(h, NVFP4_MOE_ERR_CUDA, "forward_routed: cuTensorMapEncodeTiled failed for x");
  if (h->log && !h->logged_path[path]) {
    h->logged_path[path] = true;
    fprintf(stderr, "[nvfp4_moe] forward T=%d top_k=%d -> %s path\n", T, top_k,
            path == NVFP4_MOE_PATH_DECODE ? "decode (grouped GEMV)" : "prefill (tcgen05 grouped GEMM)");
  }
  cudaEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
  s = take_events(h, ev);
  if (s != NVFP4_MOE_OK) return s;
  if (ev[0]) cudaEventRecord(ev[0], st);
  LayerDims d = dims_of(h);
  const float* gsc = h->w4a4 ? h->gs_eff : h->gscale;  // W4A4: input scales folded in
  cudaError_t e;
  // the streaming decode kernel computes the router logits itself (one launch for the layer)
  const bool fused_router = routed && path == NVFP4_MOE_PATH_DECODE && use_stream(h, d, T, top_k);
  if (routed && !fused_router) {  // the router linear, timed with route + permute
    const int Er = h->cfg.num_experts, H = h->cfg.hidden;
    if (T <= kDecodeMaxTokens) {
      e = launch_router_gemv(x, h->w_router, T, Er, H, h->ws.logits, st);
    } else {
      // token tiles small enough to give every SM a unit (16..128 rows)
      int rows = (T + h->num_sms - 1) / h->num_sms;
      rows = std::min(kTileRows, std::max(16, (rows + 15) / 16 * 16));
      e = launch_route_linear(T, rows, h->ws, st);
      if (e == cudaSuccess)
        e = launch_router_gemm(x_map, h->w_router_map, Er, H, h->num_sms, h->ws.ones3, h->ws, h->ws.logits, st);
    }
    if (e != cudaSuccess) return cuda_fail(h, e, "router launch");
  }
  if (routed) {
    logits = h->ws.logits;
    d.logits_bf16 = 0;
  }
  if (path == NVFP4_MOE_PATH_DECODE) {
    // one fused kernel: its time is reported as the gate/up stage
    if (ev[1]) cudaEventRecord(ev[1], st);
    const bool stream = use_stream(h, d, T, top_k);
    e = stream ? launch_decode_stream(d, h->blob, gsc, logits, x, T, top_k, out, 0, h->num_sms, h->ws, h->fault, st,
                                      fused_router ? h->w_router : nullptr)
               : launch_decode_forward(d, h->blob, gsc, logits, x, T, top_k, out, 0, h->num_sms, h->ws, h->fault, st);
    h->last_hsrc = stream ? 1 : 0;
    if (e != cudaSuccess) return cuda_fail(h, e, "decode launch");
    if (ev[2]) cudaEventRecord(ev[2], st);
    if (ev[3]) cudaEventRecord(ev[3], st);
  } else {
    s = run_route(h, logits, x, T, top_k, path, st, d.logits_bf16);
    if (s != NVFP4_MOE_OK) return s;
    if (ev[1]) cudaEventRecord(ev[1], st);
    e = launch_prefill_ffn(d, h->blob, gsc, T, top_k, h->num_sms, h->maps, h->ws, h->fault, ev[2],
                           nullptr, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "expert FFN launch");
    if (ev[3]) cudaEventRecord(ev[3], st);
    e = launch_combine(d, T, top_k, h->ws, out, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "combine launch");
    h->last_hsrc = 2;
  }
  if (ev[4]) cudaEventRecord(ev[4], st);
  h->last_T = T;
  h->last_k = top_k + h->cfg.num_shared_experts;  // routed-row slots per token
  h->last_routed = routed;
  return NVFP4_MOE_OK;
}
}  // namespace

extern "C" {

nvfp4_moe_status nvfp4_moe_forward(nvfp4_moe_t h, const void* logits, int T, int top_k, const void* x, void* out,
                                   cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  return forward_impl(h, logits, T, top_k, x, out, st, false);
}

}  // extern "C"

namespace {
// The device address of host memory the device may read and write in place: page-locked memory
// that CUDA has mapped into the device's address space (under unified addressing, the same
// pointer).  NULL for pageable, managed or device memory.
const void* mapped_host(const void* p) {
  if (!p) return nullptr;
  cudaPointerAttributes attr{};
  if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return nullptr;
  }
  return attr.type == cudaMemoryTypeHost ? attr.devicePointer : nullptr;
}
}  // namespace

extern "C" {

nvfp4_moe_status nvfp4_moe_forward_host(nvfp4_moe_t h, const void* logits, int T, int top_k, const void* x,
                                        void* out, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "forward_host: the handle is a dense linear");
  DeviceGuard g(h->cfg.device);
  // the streaming decode kernel reads logits and x and writes out with plain loads and stores
  // only, so those may live in host memory; the other paths copy x and logits in bulk
  if (choose_path(h, T, top_k) != NVFP4_MOE_PATH_DECODE || !use_stream(h, dims_of(h), T, top_k))
    return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE,
                "forward_host: host buffers are read in place by the W4A16 decode kernel only (T <= decode_max_tokens)");
  const void* dl = mapped_host(logits);
  const void* dx = mapped_host(x);
  void* dout = const_cast<void*>(mapped_host(out));
  if (!dl || !dx || !dout)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "forward_host: logits, x and out must be mapped page-locked host memory");
  return forward_impl(h, dl, T, top_k, dx, dout, st, false);
}

nvfp4_moe_status nvfp4_moe_set_router(nvfp4_moe_t h, const void* w_router, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_router: a dense linear has no router");
  if (!w_router || !aligned(w_router, 16)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "set_router: NULL or misaligned");
  DeviceGuard g(h->cfg.device);
  const size_t n = (size_t)h->cfg.num_experts * h->cfg.hidden * 2;
  if (!h->w_router && cudaMalloc(&h->w_router, n) != cudaSuccess) {
    cudaGetLastError();
    h->w_router = nullptr;
    return fail(h, NVFP4_MOE_ERR_WORKSPACE, "set_router: device allocation failed");
  }
  cudaError_t e = cudaMemcpyAsync(h->w_router, w_router, n, cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "set_router copy");
  if (!encode_rows_map(&h->w_router_map, h->w_router, (uint64_t)h->cfg.num_experts, (uint64_t)h->cfg.hidden, 128))
    return fail(h, NVFP4_MOE_ERR_CUDA, "set_router: cuTensorMapEncodeTiled failed");
  h->have_router = true;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_forward_routed(nvfp4_moe_t h, int T, int top_k, const void* x, void* out,
                                          cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  return forward_impl(h, nullptr, T, top_k, x, out, st, true);
}

nvfp4_moe_status nvfp4_moe_debug_logits(nvfp4_moe_t h, float* logits, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!h->last_T || !h->last_routed)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_logits: no nvfp4_moe_forward_routed yet");
  if (!logits) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_logits: NULL output");
  DeviceGuard g(h->cfg.device);
  cudaError_t e = cudaMemcpyAsync(logits, h->ws.logits, (size_t)h->last_T * h->cfg.num_experts * 4,
                                  cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_logits copy");
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_get_status(nvfp4_moe_t h, uint32_t* nan_logits) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  DeviceGuard g(h->cfg.device);
  DeviceStatus ds{};
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&ds, h->ws.status, sizeof(ds), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->ws.status, 0, sizeof(ds));
  if (e != cudaSuccess) return cuda_fail(h, e, "get_status");
  if (nan_logits) *nan_logits = ds.nan_logits;
  if (ds.flags & kFlagTimeout)
    return fail(h, NVFP4_MOE_ERR_TIMEOUT, "device wait timed out at site " + std::to_string(ds.where));
  if (ds.flags & kFlagBounds)
    return fail(h, NVFP4_MOE_ERR_DEVICE_CHECK, "device bounds check at site " + std::to_string(ds.where));
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_route(nvfp4_moe_t h, const void* logits, int T, int top_k, int32_t* ids,
                                       float* weights, int32_t* offsets, int32_t* perm, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  const int path = choose_path(h, T, top_k);
  nvfp4_moe_status s = check_forward_args(h, logits, T, top_k, path);
  if (s != NVFP4_MOE_OK) return s;
  if (!ids || !weights || !offsets || !perm) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_route: NULL output");
  DeviceGuard g(h->cfg.device);
  s = run_route(h, logits, nullptr, T, top_k, path, st);
  if (s != NVFP4_MOE_OK) return s;
  const size_t n = (size_t)T * (top_k + h->cfg.num_shared_experts);
  cudaError_t e = cudaMemcpyAsync(ids, h->ws.ids, n * 4, cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(weights, h->ws.wts, n * 4, cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(offsets, h->ws.offsets, (h->cfg.num_experts + h->cfg.num_shared_experts + 1) * 4,
                        cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(perm, h->ws.perm, n * 4, cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_route copy");
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_trace(nvfp4_moe_t h, uint64_t* host_dst, size_t n, size_t* n_written) {
  if (!h || !host_dst || !n_written) return NVFP4_MOE_ERR_INVALID_ARG;
  *n_written = 0;
  if (!h->ws.trace) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_trace: create the handle with NVFP4_MOE_TRACE=1");
  DeviceGuard g(h->cfg.device);
  const size_t total = (size_t)h->num_sms * 16 * 16;
  const size_t m = n < total ? n : total;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(host_dst, h->ws.trace, m * 8, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->ws.trace, 0, total * 8);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_trace");
  *n_written = m;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_packed_blob(nvfp4_moe_t h, void* dst, size_t dst_bytes, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!h->packed) return fail(h, NVFP4_MOE_ERR_NOT_PACKED, "debug_packed_blob before pack");
  const size_t n = h->product_bytes ? h->product_bytes : blob_bytes_of(h->cfg, h->linear);
  if (!dst || dst_bytes < n) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_packed_blob: destination too small");
  DeviceGuard g(h->cfg.device);
  cudaError_t e = cudaMemcpyAsync(dst, h->blob, n, cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_packed_blob copy");
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_dequant(nvfp4_moe_t h, int expert, int which, float* w_out, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_NOT_IMPLEMENTED, "debug_dequant: not for a dense-linear handle");
  if (!h->packed) return fail(h, NVFP4_MOE_ERR_NOT_PACKED, "debug_dequant before pack");
  const int base = which & 3, via_bf16 = (which >> 2) & 1;
  if (expert < 0 || expert >= h->cfg.num_experts + h->cfg.num_shared_experts || base > 2 || (which & ~7) || !w_out)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_dequant: bad expert/which/out");
  DeviceGuard g(h->cfg.device);
  cudaError_t e = launch_debug_dequant(h->blob, h->gscale, h->cfg.hidden, h->cfg.inter, expert, base, via_bf16, w_out, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_dequant launch");
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_moe_debug_intermediates(nvfp4_moe_t h, void* hidden, float* y, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->linear) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_intermediates: a dense linear has none");
  if (!h->last_T) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_intermediates before any forward");
  if (!hidden || !y) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "debug_intermediates: NULL output");
  DeviceGuard g(h->cfg.device);
  const size_t n = (size_t)h->last_T * h->last_k;
  cudaError_t e = launch_hidden_to_f32(h->ws, h->last_hsrc, (int)n, h->cfg.inter, static_cast<float*>(hidden), st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(y, h->ws.y, n * h->cfg.hidden * 4, cudaMemcpyDeviceToDevice, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "debug_intermediates copy");
  return NVFP4_MOE_OK;
}

// ---------------------------------------------------------------------------
// Dense W4A16 NVFP4 linear: one matrix, every token, no routing.
// ---------------------------------------------------------------------------
nvfp4_moe_status nvfp4_linear_create(const nvfp4_linear_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->out_features < 16 || c->out_features > 16384 || c->out_features % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->in_features < 128 || c->in_features > 16384 || c->in_features % 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_tokens < 1 || c->max_tokens > (1 << 20)) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->decode_max_tokens < 0 || c->decode_max_tokens > kDecodeMaxTokens) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->out_dtype != NVFP4_MOE_OUT_BF16 && c->out_dtype != NVFP4_MOE_OUT_F32) return NVFP4_MOE_ERR_INVALID_ARG;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || c->device < 0 || c->device >= ndev) return NVFP4_MOE_ERR_INVALID_ARG;
  nvfp4_moe_config m{};
  m.num_experts = 1;
  m.hidden = (c->out_features + 127) / 128 * 128;  // whole 128-row blocks; the padding rows are zero
  m.inter = c->in_features;
  m.max_tokens = c->max_tokens;
  m.max_top_k = 1;
  m.decode_max_tokens = c->decode_max_tokens;
  m.logits_dtype = NVFP4_MOE_LOGITS_F32;
  m.out_dtype = c->out_dtype;
  m.device = c->device;
  m.num_shared_experts = 0;
  return create_handle(&m, true, c->out_features, out);
}

nvfp4_moe_status nvfp4_linear_pack(nvfp4_moe_t h, const uint8_t* w_q, const uint8_t* w_s, const float* gscale,
                                   cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!h->linear || h->kind != nvfp4_moe::kLayerOrLinear)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "not a dense-linear handle: call its own pack");
  if (!w_q || !w_s || !gscale) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "linear_pack: NULL input");
  if (!aligned(w_q, 16) || !aligned(w_s, 4) || !aligned(gscale, 4))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "linear_pack: misaligned input");
  DeviceGuard g(h->cfg.device);
  float gs = 0.f;
  h->packed = false;  // until all of it is done
  cudaError_t e = cudaMemcpyAsync(&gs, gscale, sizeof(float), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "linear_pack: reading gscale");
  if (!(gs > 0.0f) || gs != gs || gs > 3.4e38f)
    return fail(h, NVFP4_MOE_ERR_BAD_SCALE, "linear_pack: the tensor scale is not finite > 0");
  // the kernels read the down-projection scale of "expert" 0: slot 2 of 3
  const float gs3[3] = {gs, gs, gs};
  e = cudaMemcpyAsync(h->gscale, gs3, sizeof(gs3), cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess) e = launch_pack_linear(w_q, w_s, h->blob, h->lin_n, h->cfg.hidden, h->cfg.inter, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);  // gs3 lives on this frame
  if (e != cudaSuccess) return cuda_fail(h, e, "linear_pack launch");
  h->packed = true;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_linear_forward(nvfp4_moe_t h, int T, const void* x, void* out, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!h->linear || h->kind != nvfp4_moe::kLayerOrLinear)
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "not a dense-linear handle: call its own forward");
  if (!h->packed) return fail(h, NVFP4_MOE_ERR_NOT_PACKED, "linear_forward before a successful pack");
  if (T < 1 || T > h->cfg.max_tokens) return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "T outside 1..max_tokens");
  if (!x || !out) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "x or out is NULL");
  if (!aligned(x, 16) || !aligned(out, 16)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "x or out not 16-byte aligned");
  const int path = choose_path(h, T, 1);
  if (path == NVFP4_MOE_PATH_DECODE && T > kDecodeMaxTokens)
    return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "decode path takes at most 16 tokens");
  DeviceGuard g(h->cfg.device);
  PrefillMaps maps{};
  if (path == NVFP4_MOE_PATH_PREFILL && !encode_rows_map(&maps.h, const_cast<void*>(x), (uint64_t)T, h->cfg.inter))
    return fail(h, NVFP4_MOE_ERR_CUDA, "linear_forward: cuTensorMapEncodeTiled failed for x");
  if (h->log && !h->logged_path[path]) {
    h->logged_path[path] = true;
    fprintf(stderr, "[nvfp4_moe] linear forward T=%d -> %s path\n", T,
            path == NVFP4_MOE_PATH_DECODE ? "decode (GEMV)" : "prefill (tcgen05 GEMM)");
  }
  cudaEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
  nvfp4_moe_status s = take_events(h, ev);
  if (s != NVFP4_MOE_OK) return s;
  if (ev[0]) cudaEventRecord(ev[0], st);
  const LayerDims d = dims_of(h);
  cudaError_t e;
  if (path == NVFP4_MOE_PATH_DECODE) {
    if (ev[1]) cudaEventRecord(ev[1], st);
    if (ev[2]) cudaEventRecord(ev[2], st);
    e = stream_supported(d, T, 1)
            ? launch_decode_stream(d, h->blob, h->gscale, nullptr, x, T, 1, out, 0, h->num_sms, h->ws, h->fault, st)
            : launch_decode_forward(d, h->blob, h->gscale, nullptr, x, T, 1, out, 0, h->num_sms, h->ws, h->fault, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "linear decode launch");
  } else {
    e = launch_route_linear(T, kTileRows, h->ws, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "linear tables launch");
    if (ev[1]) cudaEventRecord(ev[1], st);
    e = launch_prefill_ffn(d, h->blob, h->gscale, T, 1, h->num_sms, maps, h->ws, h->fault, ev[2], out, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "linear GEMM launch");
  }
  if (ev[3]) cudaEventRecord(ev[3], st);
  if (ev[4]) cudaEventRecord(ev[4], st);
  h->last_T = T;
  h->last_k = 1;
  h->last_routed = false;
  return NVFP4_MOE_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Products outside the layer: grouped NVFP4 experts, the INT4 linear.
// ---------------------------------------------------------------------------
// A handle with a blob of `bytes`, n_scales tensor scales and a status word, on `device`.
nvfp4_moe_status nvfp4moe::create_product(nvfp4_moe::Kind kind, int device, size_t bytes, int n_scales, nvfp4_moe** out) {
  nvfp4_moe* h = new (std::nothrow) nvfp4_moe();
  if (!h) return NVFP4_MOE_ERR_WORKSPACE;
  h->kind = kind;
  h->linear = true;
  h->cfg.device = device;
  h->product_bytes = bytes;
  const char* lg = getenv("NVFP4_MOE_LOG");
  h->log = lg && lg[0] == '1';
  const char* fp = getenv("NVFP4_MOE_FORCE_PATH");
  if (fp && !strcmp(fp, "decode")) h->path = NVFP4_MOE_PATH_DECODE;
  if (fp && !strcmp(fp, "prefill")) h->path = NVFP4_MOE_PATH_PREFILL;
  DeviceGuard g(device);
  cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, device);
  int l2 = 0;
  cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, device);
  h->l2_bytes = (size_t)l2;
  h->ws_bytes = sizeof(DeviceStatus);
  if (cudaMalloc(&h->blob, bytes) != cudaSuccess || cudaMalloc(&h->gscale, sizeof(float) * n_scales) != cudaSuccess ||
      cudaMalloc(&h->ws_mem, h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    nvfp4_moe_destroy(h);
    return NVFP4_MOE_ERR_WORKSPACE;
  }
  h->ws.status = static_cast<DeviceStatus*>(h->ws_mem);
  if (cudaMemset(h->ws_mem, 0, h->ws_bytes) != cudaSuccess) {
    cudaGetLastError();
    nvfp4_moe_destroy(h);
    return NVFP4_MOE_ERR_CUDA;
  }
  *out = h;
  return NVFP4_MOE_OK;
}

namespace {
nvfp4_moe_status grouped_impl(nvfp4_moe* h, bool backward, int R, const int32_t* offsets, const void* in,
                              int64_t ldi, void* out, int64_t ldo, cudaStream_t st) {
  const char* what = backward ? "grouped_backward" : "grouped_forward";
  const auto bad = [&](nvfp4_moe_status s, const char* msg) { return fail(h, s, std::string(what) + ": " + msg); };
  if (h->kind != nvfp4_moe::kGrouped) return bad(NVFP4_MOE_ERR_INVALID_ARG, "not a grouped handle");
  if (!h->packed) return bad(NVFP4_MOE_ERR_NOT_PACKED, "before a successful pack");
  if (R < 0 || R > h->cfg.max_tokens) return bad(NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "R outside 0..max_rows");
  if (R == 0) return NVFP4_MOE_OK;
  const int N = h->lin_n, K = h->cfg.inter, E = h->cfg.num_experts;
  const int wi = backward ? N : K, wo = backward ? K : N;
  if (!offsets || !in || !out) return bad(NVFP4_MOE_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(offsets, 4) || !aligned(in, 16) || !aligned(out, 16))
    return bad(NVFP4_MOE_ERR_INVALID_ARG, "offsets not 4-byte or rows not 16-byte aligned");
  if (ldi < wi || ldo < wo || ldi % 8 || ldo % 8 || ldi > (1 << 24) || ldo > (1 << 24))
    return bad(NVFP4_MOE_ERR_INVALID_ARG, "a row stride is below the row length, above 2^24 or no multiple of 8");
  if (!backward && h->path == NVFP4_MOE_PATH_DECODE && R > kGemvMaxRows)
    return bad(NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "the decode path takes at most 2048 rows");
  // AUTO streams the weights through the row kernel as long as an expert's rows, were they even, make one tile of it: 8
  // up to K = 4096, then as many as fit beside its rings (5 at 7168, 4 at 8192, 2 at 16384).  It reads and converts a
  // matrix once for each tile, in a little over half of the GEMM's time, so that a second tile loses the gain.  Even
  // counts, us streamed and as GEMM: 128 experts of 1536 x 4096, 8 rows each 77 and 144; 64 of 2048 x 7168, 5 each 85
  // and 158, 6 each 154 and 155; of 2048 x 8192, 4 each 97 and 176, 6 each 176 and 176; of 1024 x 16384, 2 each 99 and
  // 198, 4 each 181 and 198, 8 each 340 and 198; one of 16384 x 16384, 2 rows 29 and 97, 8 rows 90 and 63.  Uneven ones
  // make more tiles: at these limits, popularity by Zipf's law with 1.1, 112 and 131, 111 and 136, 117 and 128, 109 and
  // 153.  The host does not see the offsets; all rows with one expert is the worst (1024 of 1536 x 4096: 76 and 31).
  const bool stream = !backward && (h->path == NVFP4_MOE_PATH_DECODE ||
                                    (h->path == NVFP4_MOE_PATH_AUTO && R <= kGemvMaxRows && R <= E * grouped_gemv_tile_rows(K)));
  DeviceGuard g(h->cfg.device);
  const GroupedTiling tiling = grouped_tiling(E, R, backward ? K / 128 : (N + 127) / 128, backward ? (N + 127) / 128 : K / 128,
                                              h->num_sms);
  CUtensorMap map{};
  if (!stream &&
      !encode_rows_map(&map, const_cast<void*>(in), (uint64_t)R, (uint64_t)wi, (uint32_t)tiling.box, (uint64_t)ldi))
    return fail(h, NVFP4_MOE_ERR_CUDA, std::string(what) + ": cuTensorMapEncodeTiled failed");
  GroupedProduct p{};
  p.blob = h->blob;
  p.gscale = h->gscale;
  p.E = E;
  p.N = N;
  p.K = K;
  p.offsets = offsets;
  p.R = R;
  p.in = in;
  p.ldi = ldi;
  p.out = out;
  p.ldo = ldo;
  p.out_f32 = h->cfg.out_dtype == NVFP4_MOE_OUT_F32;
  p.once = h->product_bytes > h->l2_bytes;
  p.num_sms = h->num_sms;
  p.status = h->ws.status;
  p.fault = h->fault;
  cudaEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
  const nvfp4_moe_status s = take_events(h, ev);
  if (s != NVFP4_MOE_OK) return s;
  record(ev, 0, 2, st);
  const cudaError_t e = stream ? launch_grouped_gemv(p, st) : launch_grouped_gemm(p, backward, tiling, map, st);
  if (e != cudaSuccess) return cuda_fail(h, e, what);
  record(ev, 3, 4, st);
  return NVFP4_MOE_OK;
}
}  // namespace

extern "C" {

nvfp4_moe_status nvfp4_grouped_create(const nvfp4_grouped_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->num_experts < 1 || c->num_experts > 256) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->out_features < 16 || c->out_features > 16384 || c->out_features % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->in_features < 128 || c->in_features > 16384 || c->in_features % 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_rows < 1 || c->max_rows > (1 << 24)) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->out_dtype != NVFP4_MOE_OUT_BF16 && c->out_dtype != NVFP4_MOE_OUT_F32) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  const int Np = (c->out_features + 127) / 128 * 128;
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s =
      create_product(nvfp4_moe::kGrouped, c->device, (size_t)c->num_experts * linear_layout(Np, c->in_features).stride,
                     c->num_experts, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->cfg.num_experts = c->num_experts;
  h->cfg.hidden = Np;
  h->cfg.inter = c->in_features;
  h->cfg.max_tokens = c->max_rows;
  h->cfg.max_top_k = 1;
  h->cfg.out_dtype = c->out_dtype;
  h->lin_n = c->out_features;
  *out = h;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_grouped_pack(nvfp4_moe_t h, const uint8_t* w_q, const uint8_t* w_s, const float* gscale,
                                    cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->kind != nvfp4_moe::kGrouped) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "grouped_pack: not a grouped handle");
  if (!w_q || !w_s || !gscale) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "grouped_pack: NULL input");
  if (!aligned(w_q, 16) || !aligned(w_s, 4) || !aligned(gscale, 4))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "grouped_pack: misaligned input");
  DeviceGuard g(h->cfg.device);
  const int E = h->cfg.num_experts;
  float gs[256];
  h->packed = false;  // until all of it is done
  cudaError_t e = cudaMemcpyAsync(gs, gscale, sizeof(float) * E, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "grouped_pack: reading gscale");
  for (int i = 0; i < E; ++i)
    if (!(gs[i] > 0.0f) || gs[i] > 3.4e38f)
      return fail(h, NVFP4_MOE_ERR_BAD_SCALE,
                  "grouped_pack: the tensor scale of expert " + std::to_string(i) + " is not finite > 0");
  e = cudaMemcpyAsync(h->gscale, gscale, sizeof(float) * E, cudaMemcpyDeviceToDevice, st);
  if (e == cudaSuccess) e = launch_pack_grouped(w_q, w_s, h->blob, E, h->lin_n, h->cfg.hidden, h->cfg.inter, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "grouped_pack launch");
  h->packed = true;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_grouped_forward(nvfp4_moe_t h, int R, const int32_t* offsets, const void* x, int64_t ldx,
                                       void* out, int64_t ldo, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  return grouped_impl(h, false, R, offsets, x, ldx, out, ldo, st);
}

nvfp4_moe_status nvfp4_grouped_backward(nvfp4_moe_t h, int R, const int32_t* offsets, const void* dy, int64_t ld_dy,
                                        void* dx, int64_t ld_dx, cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  return grouped_impl(h, true, R, offsets, dy, ld_dy, dx, ld_dx, st);
}

nvfp4_moe_status nvfp4_int4_create(const nvfp4_int4_config* c, nvfp4_moe_t* out) {
  if (!out) return NVFP4_MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!c) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->out_features < 16 || c->out_features > (1 << 20) || c->out_features % 16) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->in_features < 128 || c->in_features > 16384 || c->in_features % 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->max_tokens < 1 || c->max_tokens > kDecodeMaxTokens) return NVFP4_MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->act_dtype != NVFP4_MOE_ACT_BF16 && c->act_dtype != NVFP4_MOE_ACT_F16) return NVFP4_MOE_ERR_INVALID_ARG;
  if (c->out_f32 != 0 && c->out_f32 != 1) return NVFP4_MOE_ERR_INVALID_ARG;
  if (!device_ok(c->device)) return NVFP4_MOE_ERR_INVALID_ARG;
  nvfp4_moe* h = nullptr;
  const nvfp4_moe_status s = create_product(
      nvfp4_moe::kInt4, c->device, int4_packed_bytes(c->out_features, c->in_features, c->group_size, true), 1, &h);
  if (s != NVFP4_MOE_OK) return s;
  h->i4 = *c;
  *out = h;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_int4_pack(nvfp4_moe_t h, const uint8_t* w_q, const void* scale, const uint8_t* zero,
                                 cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->kind != nvfp4_moe::kInt4) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_pack: not an INT4 handle");
  if (!w_q || !scale) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_pack: NULL input");
  if (!aligned(w_q, 16) || !aligned(scale, 2)) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_pack: misaligned input");
  DeviceGuard g(h->cfg.device);
  h->packed = false;
  int bad = 0;
  int* bad_dev = reinterpret_cast<int*>(h->gscale);  // an INT4 handle has no tensor scale
  cudaError_t e = launch_pack_int4(w_q, scale, zero, h->i4.act_dtype == NVFP4_MOE_ACT_F16, h->i4.out_features,
                                   h->i4.in_features, h->i4.group_size, h->blob, bad_dev, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&bad, bad_dev, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(h, e, "int4_pack");
  if (bad)
    return fail(h, NVFP4_MOE_ERR_BAD_SCALE,
                "int4_pack: " + std::to_string(bad) + " groups have a scale that is not finite or a zero point above 15");
  h->i4_zeros = zero != nullptr;
  h->packed = true;
  return NVFP4_MOE_OK;
}

nvfp4_moe_status nvfp4_int4_forward(nvfp4_moe_t h, int T, const void* x, int64_t ldx, void* out, int64_t ldo,
                                    cudaStream_t st) {
  if (!h) return NVFP4_MOE_ERR_INVALID_ARG;
  if (h->kind != nvfp4_moe::kInt4) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_forward: not an INT4 handle");
  if (!h->packed) return fail(h, NVFP4_MOE_ERR_NOT_PACKED, "int4_forward before a successful pack");
  if (T < 1 || T > h->i4.max_tokens) return fail(h, NVFP4_MOE_ERR_UNSUPPORTED_SHAPE, "int4_forward: T outside 1..max_tokens");
  if (!x || !out) return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_forward: x or out is NULL");
  if (!aligned(x, 16) || !aligned(out, 16))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG, "int4_forward: x or out not 16-byte aligned");
  if (ldx < h->i4.in_features || ldo < h->i4.out_features || ldx % 8 || ldo % 8 || ldx > (1 << 24) || ldo > (1 << 24))
    return fail(h, NVFP4_MOE_ERR_INVALID_ARG,
                "int4_forward: a row stride is below the row length, above 2^24 or no multiple of 8");
  DeviceGuard g(h->cfg.device);
  Int4Product p{};
  p.packed = h->blob;
  p.zeros = h->i4_zeros;
  p.N = h->i4.out_features;
  p.K = h->i4.in_features;
  p.group = h->i4.group_size;
  p.T = T;
  p.act_f16 = h->i4.act_dtype == NVFP4_MOE_ACT_F16;
  p.x = x;
  p.ldx = ldx;
  p.out = out;
  p.ldo = ldo;
  p.out_f32 = h->i4.out_f32;
  p.once = h->product_bytes > h->l2_bytes;
  p.num_sms = h->num_sms;
  p.status = h->ws.status;
  p.fault = h->fault;
  cudaEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
  const nvfp4_moe_status s = take_events(h, ev);
  if (s != NVFP4_MOE_OK) return s;
  record(ev, 0, 2, st);
  const cudaError_t e = launch_int4_gemv(p, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "int4_forward");
  record(ev, 3, 4, st);
  return NVFP4_MOE_OK;
}

}  // extern "C"
