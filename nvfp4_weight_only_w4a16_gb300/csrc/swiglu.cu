// SwiGLU with its backward pass's inputs kept in 8 bits (nvfp4_swiglu_forward / nvfp4_swiglu_backward):
//   forward : h = silu(g) u, and g and u as round(127 v / peak), peak / 127 per 128 elements of a row
//   backward: dg = dh u s (1 + g (1 - s)), du = dh g s, with s = 1 / (1 + e^-g) and g and u from the codes
//
// Bound by memory: 8 bytes an element either way (two 16-bit rows in or out, one the other way, two bytes of codes;
// 131072 x 1536, 1.6 GB: 248 us forward, 243 backward, 0.98 and 1.0 of the copy rate).
// A thread takes 16 elements of gate and of up, eight threads a block of 128, so that all loads and stores are 16
// bytes wide and a block's peak takes three shuffles.  Few instructions an element count (at 41 the forward took 316 us
// for 131072 x 1536), so exp and the reciprocal are the hardware's approximations (relative error 2^-21 for |g| up to 16,
// next to the result's rounding of 2^-9 or 2^-12), no code is converted to or from an integer (both go by the low bits of
// a float), and the exact rounding of a code takes no test.
#include <algorithm>

#include "kernels.h"
#include "quant8.cuh"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace sg {
constexpr int kThreads = 256, kPer = 16;           // elements per thread
constexpr int kPerSm = 3;                          // CTAs a multiprocessor holds, and is given
constexpr int kBlock = 128, kLanes = kBlock / kPer;  // of a checkpoint's scale; threads per block
}  // namespace sg

struct SwigluArgs {
  const uint8_t *gate, *up, *dh;  // rows of 16-bit elements
  uint8_t *h, *dgate, *dup;
  long long ld_gate, ld_up, ld_dh, ld_h, ld_dgate, ld_dup;  // bytes
  int8_t* codes;                  // [R][2][I]
  float* scales;                  // [R][2][nb]
  long long R;
  int I, nb;                      // nb: blocks of a row
};

// The blocks of eight threads: first, first + stride, ..; walked without divisions.
struct SwigluBlocks {
  long long row, drow;
  int b, db, nb;
  __device__ __forceinline__ explicit SwigluBlocks(int nb_) : nb(nb_) {
    const unsigned first = (blockIdx.x * sg::kThreads + threadIdx.x) / sg::kLanes;
    const unsigned stride = gridDim.x * (sg::kThreads / sg::kLanes);
    row = first / nb, b = (int)(first - (unsigned)row * nb);
    drow = stride / nb, db = (int)(stride - (unsigned)drow * nb);
  }
  __device__ __forceinline__ void next() {
    row += drow, b += db;
    if (b >= nb) b -= nb, ++row;
  }
};

// 1 / (1 + e^-g) by the hardware's 2^x and 1/x.
__device__ __forceinline__ float sigmoid_fast(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

template <bool kF16>
__device__ __forceinline__ void load_elems(const uint8_t* p, bool ok, uint4 (&w)[2]) {
  w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
  if (ok) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    w[1] = *reinterpret_cast<const uint4*>(p + 16);
  }
}

// The codes of a block of which this thread holds 16 elements (raw: as they came), and its scale.
template <bool kF16>
__device__ __forceinline__ uint4 checkpoint(const uint4 (&raw)[2], const float (&v)[sg::kPer], float& scale) {
  unsigned m = max(peak_of(raw[0]), peak_of(raw[1]));
#pragma unroll
  for (int o = 1; o < sg::kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = __float_as_uint(unpack16<kF16>(m).x);
  const float peak = __uint_as_float(m);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  scale = 0.f;
  if (plain_peak(peak)) {
    codes_of_elements(v, peak, c);
    scale = scale_of_peak(peak);
  } else if (m >= 0x7F800000u) {
    scale = __uint_as_float(0x7FC00000u);
  } else if (m) {  // too small, or too large, for FP32 quotients
    scale = peak / 127.0f;
#pragma unroll
    for (int i = 0; i < sg::kPer; ++i) c[i >> 2] |= ((uint32_t)code_of_64(v[i], peak) & 255u) << (8 * (i & 3));
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <bool kF16, bool kKeep>
__global__ void __launch_bounds__(sg::kThreads, sg::kPerSm) swiglu_forward_kernel(SwigluArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int part = threadIdx.x % sg::kLanes;
  SwigluBlocks w(a.nb);
  // whole warps stay, for the shuffles: a warp's four blocks follow one another
  for (;; w.next()) {
    const bool row_ok = w.row < a.R;
    if (!__any_sync(0xffffffffu, row_ok)) break;
    const int e = w.b * sg::kBlock + part * sg::kPer;
    const bool ok = row_ok && e < a.I;
    uint4 g4[2], u4[2];
    load_elems<kF16>(a.gate + w.row * a.ld_gate + 2ll * e, ok, g4);
    load_elems<kF16>(a.up + w.row * a.ld_up + 2ll * e, ok, u4);
    float g[sg::kPer], u[sg::kPer];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float t[8];
      unpack8<kF16>(g4[i], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) g[8 * i + j] = t[j];
      unpack8<kF16>(u4[i], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[8 * i + j] = t[j];
    }
    if (kKeep) {
      float sg_, su;
      const uint4 cg = checkpoint<kF16>(g4, g, sg_), cu = checkpoint<kF16>(u4, u, su);
      if (ok) {
        int8_t* c = a.codes + w.row * 2 * a.I + e;
        *reinterpret_cast<uint4*>(c) = cg;
        *reinterpret_cast<uint4*>(c + a.I) = cu;
        if (part == 0) {
          float* s = a.scales + w.row * 2 * a.nb + w.b;
          s[0] = sg_, s[a.nb] = su;
        }
      }
    }
    if (ok) {
      uint8_t* h = a.h + w.row * a.ld_h + 2ll * e;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = g[8 * i + j] * sigmoid_fast(g[8 * i + j]) * u[8 * i + j];
        *reinterpret_cast<uint4*>(h + 16 * i) = pack8<kF16>(t);
      }
    }
  }
}

template <bool kF16>
__global__ void __launch_bounds__(sg::kThreads, sg::kPerSm) swiglu_backward_kernel(SwigluArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int part = threadIdx.x % sg::kLanes;
  for (SwigluBlocks w(a.nb); w.row < a.R; w.next()) {
    const int e = w.b * sg::kBlock + part * sg::kPer;
    if (e >= a.I) continue;
    const int8_t* c = a.codes + w.row * 2 * a.I + e;
    const float* s = a.scales + w.row * 2 * a.nb + w.b;
    const uint4 cg = *reinterpret_cast<const uint4*>(c), cu = *reinterpret_cast<const uint4*>(c + a.I);
    const float sg_ = s[0], su = s[a.nb];
    uint4 d4[2];
    load_elems<kF16>(a.dh + w.row * a.ld_dh + 2ll * e, true, d4);
    const uint32_t wg[4] = {cg.x, cg.y, cg.z, cg.w}, wu[4] = {cu.x, cu.y, cu.z, cu.w};
    uint8_t* og = a.dgate + w.row * a.ld_dgate + 2ll * e;
    uint8_t* ou = a.dup + w.row * a.ld_dup + 2ll * e;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float d[8], dg[8], du[8];
      unpack8<kF16>(d4[i], d);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float g[4], u[4];
        codes_to_f32(wg[2 * i + k], g);
        codes_to_f32(wu[2 * i + k], u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gv = g[j] * sg_, sig = sigmoid_fast(gv), ds = d[4 * k + j] * sig;
          du[4 * k + j] = ds * gv;
          dg[4 * k + j] = ds * (u[j] * su) * fmaf(gv, 1.0f - sig, 1.0f);
        }
      }
      *reinterpret_cast<uint4*>(og + 16 * i) = pack8<kF16>(dg);
      *reinterpret_cast<uint4*>(ou + 16 * i) = pack8<kF16>(du);
    }
  }
}

template <class K>
static cudaError_t launch_swiglu(K kernel, const SwigluArgs& a, int num_sms, cudaStream_t st) {
  const long long threads = a.R * a.nb * sg::kLanes;
  const long long all = (threads + sg::kThreads - 1) / sg::kThreads;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min(all, (long long)num_sms * sg::kPerSm));
  cfg.blockDim = dim3(sg::kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_swiglu_forward(const SwigluOp& p, cudaStream_t st) {
  SwigluArgs a{};
  a.gate = static_cast<const uint8_t*>(p.gate), a.ld_gate = 2 * p.ld_gate;
  a.up = static_cast<const uint8_t*>(p.up), a.ld_up = 2 * p.ld_up;
  a.h = static_cast<uint8_t*>(p.h), a.ld_h = 2 * p.ld_h;
  a.codes = p.codes, a.scales = p.scales;
  a.R = p.R, a.I = p.I, a.nb = (p.I + sg::kBlock - 1) / sg::kBlock;
  if (p.f16)
    return p.codes ? launch_swiglu(swiglu_forward_kernel<true, true>, a, p.num_sms, st)
                   : launch_swiglu(swiglu_forward_kernel<true, false>, a, p.num_sms, st);
  return p.codes ? launch_swiglu(swiglu_forward_kernel<false, true>, a, p.num_sms, st)
                 : launch_swiglu(swiglu_forward_kernel<false, false>, a, p.num_sms, st);
}

cudaError_t launch_swiglu_backward(const SwigluOp& p, cudaStream_t st) {
  SwigluArgs a{};
  a.dh = static_cast<const uint8_t*>(p.dh), a.ld_dh = 2 * p.ld_dh;
  a.dgate = static_cast<uint8_t*>(p.dgate), a.ld_dgate = 2 * p.ld_dgate;
  a.dup = static_cast<uint8_t*>(p.dup), a.ld_dup = 2 * p.ld_dup;
  a.codes = p.codes, a.scales = p.scales;
  a.R = p.R, a.I = p.I, a.nb = (p.I + sg::kBlock - 1) / sg::kBlock;
  return p.f16 ? launch_swiglu(swiglu_backward_kernel<true>, a, p.num_sms, st)
               : launch_swiglu(swiglu_backward_kernel<false>, a, p.num_sms, st);
}

}  // namespace nvfp4moe
