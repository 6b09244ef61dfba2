// The handle behind nvfp4_moe_t, and what the entry points share.
#pragma once
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "../../include/nvfp4_moe.h"
#include "kernels.h"

struct nvfp4_moe {
  nvfp4_moe_config cfg;
  bool linear = false;  // a dense linear (nvfp4_linear_create): cfg holds E = 1, hidden = N padded to 128, inter = K
  int lin_n = 0;        // a dense linear's N (output features)
  // a product's or another operator's handle (nvfp4_grouped_create, nvfp4_int4_create, ..): `linear` is set too, so that
  // no MoE call takes it, and ws holds the status word alone
  enum Kind { kLayerOrLinear, kGrouped, kInt4, kInt8, kRoute, kNorm, kSwiglu } kind = kLayerOrLinear;
  nvfp4_int4_config i4{};
  nvfp4_int8_config i8{};      // blob: the packed matrix; gscale: [2][out_features] scales and, if i8_bias, biases
  bool i8_bias = false;
  nvfp4_route_config route{};
  nvfp4_norm_config norm{};    // blob: the backward's partial sums
  nvfp4_swiglu_config swiglu{};
  size_t product_bytes = 0;  // a product handle's packed matrix (matrices)
  size_t l2_bytes = 0;       // a product handle's device's L2
  bool i4_zeros = false;     // INT4: the last pack had zero points
  nvfp4moe::RouteParams rp{};     // scoring rule (nvfp4_moe_set_scoring); rp.bias points at `bias` when set
  float* bias = nullptr;  // [num_experts] device copy of the choice bias
  void* w_router = nullptr;  // [num_experts][hidden] BF16 router weight (nvfp4_moe_set_router)
  CUtensorMap w_router_map{};  // over w_router, box {64, 128}, 128B swizzle
  bool have_router = false;
  // W4A4 comparison variant (nvfp4_moe_set_act_quant)
  bool w4a4 = false;
  float* in_scale = nullptr;     // [E][2] device input scales (w13, w2); shared expert's unused
  float* gs_eff = nullptr;       // [E][3] device tensor scales with the input scales folded in
  float* hbound = nullptr;       // [E] max_f ||Wg_f|| ||Wu_f|| (written at pack): sizes h's FP16 prescale
  std::vector<std::pair<uint8_t*, size_t>> data_regions;  // workspace buffers every forward rewrites
  int checks = 0;  // NVFP4_MOE_CHECKS=1 at create: kernels check table-derived indices
  std::vector<float> gs_host;    // [E][3] the packed tensor scales
  std::vector<float> is_host;    // [E][2]
  int path = NVFP4_MOE_PATH_AUTO;
  int num_sms = 0;
  bool packed = false;
  bool log = false;
  bool logged_path[3] = {false, false, false};
  uint8_t* blob = nullptr;
  float* gscale = nullptr;
  void* ws_mem = nullptr;
  void* ws_mem2 = nullptr;     // INT8: tokens in FP16
  size_t ws_bytes = 0;
  nvfp4moe::Workspace ws{};
  nvfp4moe::PrefillMaps maps{};
  int last_T = 0, last_k = 0;
  int last_hsrc = 0;  // where the last forward's hidden activations are (launch_hidden_to_f32's src)
  bool last_routed = false;
  int fault = 0;
  bool profiling = false;
  std::vector<cudaEvent_t> ev_pool;  // 5 events per profiled forward
  size_t ev_used = 0;
  char last_error[256] = {0};
};

namespace nvfp4moe {

struct DeviceGuard {
  int prev = -1;
  bool changed = false;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) changed = cudaSetDevice(dev) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (changed) cudaSetDevice(prev);
  }
};

inline nvfp4_moe_status fail(nvfp4_moe* h, nvfp4_moe_status s, const std::string& msg) {
  if (h) snprintf(h->last_error, sizeof(h->last_error), "%s", msg.c_str());
  if (h && h->log) fprintf(stderr, "[nvfp4_moe] %s\n", msg.c_str());
  return s;
}

inline nvfp4_moe_status cuda_fail(nvfp4_moe* h, cudaError_t e, const char* where) {
  cudaGetLastError();  // reported here: left behind, it would be the next kernel launch's
  return fail(h, NVFP4_MOE_ERR_CUDA, std::string(where) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// 2D 16-bit [rows][cols], rows ld elements apart (0: cols), box = 64 columns x box_rows rows, 128B swizzle.
inline bool encode_rows_map(CUtensorMap* map, void* base, uint64_t rows, uint64_t cols, uint32_t box_rows = 16,
                     uint64_t ld = 0) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {(ld ? ld : cols) * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2D bytes [rows][cols], rows ld apart, box = 128 columns x box_rows rows, 128B swizzle.
inline bool encode_bytes_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows,
                             uint64_t ld) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Forward events: 5 per profiled forward (ev[i] stays NULL when profiling is off).
inline nvfp4_moe_status take_events(nvfp4_moe* h, cudaEvent_t (&ev)[5]) {
  if (!h->profiling) return NVFP4_MOE_OK;
  for (int i = 0; i < 5; ++i) {
    if (h->ev_used == h->ev_pool.size()) {
      cudaEvent_t e0;
      if (cudaEventCreate(&e0) != cudaSuccess) return cuda_fail(h, cudaGetLastError(), "event create");
      h->ev_pool.push_back(e0);
    }
    ev[i] = h->ev_pool[h->ev_used++];
  }
  return NVFP4_MOE_OK;
}

inline bool device_ok(int device) {
  int ndev = 0;
  return cudaGetDeviceCount(&ndev) == cudaSuccess && device >= 0 && device < ndev;
}

// Event record around a product: its time counts as the down GEMM stage.
inline void record(cudaEvent_t (&ev)[5], int i0, int i1, cudaStream_t st) {
  for (int i = i0; i <= i1; ++i)
    if (ev[i]) cudaEventRecord(ev[i], st);
}

// A handle with a blob of `bytes` and n_scales tensor scales (either may be 0) and a status word, on `device`.
nvfp4_moe_status create_product(nvfp4_moe::Kind kind, int device, size_t bytes, int n_scales, nvfp4_moe** out);

}  // namespace nvfp4moe
