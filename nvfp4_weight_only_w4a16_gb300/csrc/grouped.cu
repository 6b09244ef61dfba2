// Products of NVFP4 experts over ragged row groups (nvfp4_grouped_forward /
// nvfp4_grouped_backward): a persistent tcgen05 GEMM over
//   forward : y[r][n]  = gs_e sum_k W_e[n][k] x[r][k]
//   backward: dx[r][k] = gs_e sum_n W_e[n][k] dy[r][n]
// for the rows off[e] <= r < off[e+1] of every expert e.
//
// Both directions read the same packed bytes.  The weights are the 128-row M
// operand and the rows the N operand (a multiple of 16, up to 256), so that an
// expert with few rows pays for few columns.  A work unit is one 128-feature
// output block of one token tile; its reduction runs over 128 x 128 weight
// squares: two neighbouring packed tiles (128 weight rows x 64 K each).  A
// square is dequantised to BF16 -- exact: an E2M1 x E4M3 product has at most 6
// significant bits -- into shared memory as rows of 64 K elements (128 B,
// 128B swizzle).  That one image serves both products: read K-major it is the
// forward operand (M = weight row, reduction = K), read M-major it is its
// transpose (M = K element, reduction = weight row).  Only the descriptors, and
// which half of a square makes up a 64-long reduction step, differ.
//
// One CTA per SM, 16 warps: 0 packed-weight producer (bulk copies into a ring),
// 1 MMA issuer, 2 row producer (TMA, zero fill past the matrix), 4-7 epilogue
// (TMEM -> gs -> BF16/FP32 -> global), 8-15 dequantisers.  Two accumulator
// buffers of 256 columns: the epilogue of a unit overlaps the next one's MMAs.
// The row offsets are read on the device; every CTA derives the same unit list
// from them, so nothing is written but the output.
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace gg {
constexpr int kThreads = 512;
constexpr int kDequantWarps = 8, kEpiWarps = 4;
constexpr int kPairBytes = 2 * kTileBytes;  // one 128 x 128 weight square, packed
constexpr int kABytes = 16384;              // half a square in BF16: one 64-long reduction step
constexpr int kMaxStages = 8, kMaxRaw = 16;
constexpr int kSmemMax = 232448;
constexpr int kCtlBytes = 4096;             // tables and barriers in front of the rings
}  // namespace gg

struct GroupedArgs {
  const uint8_t* blob;
  size_t expert_stride;
  const float* gscale;     // [E]
  const int32_t* offsets;  // [E + 1]
  int E, R;
  int NB;                  // 128-feature output blocks
  int steps;               // 128-long reduction steps
  size_t block_stride;     // bytes from one output block's first square to the next one's
  size_t step_stride;      // bytes from one reduction step's square to the next
  int n_out;               // output features
  void* out;
  long long ldo;
  int out_f32;
  int tile_rows;           // rows per token tile, a multiple of 16 up to 256
  int stages, raw_stages;
  DeviceStatus* st;
  int fault;
};

struct GroupedCtl {
  int off[257];
  int tile[257];  // token tiles before expert e; tile[E] = all
  uint64_t raw_full[gg::kMaxRaw], raw_empty[gg::kMaxRaw];
  uint64_t a_full[gg::kMaxStages], b_full[gg::kMaxStages], empty[gg::kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(GroupedCtl) <= gg::kCtlBytes, "control block");

struct GroupedUnit {
  int e, row0, rows, nb;
};

__device__ __forceinline__ GroupedUnit grouped_unit(const GroupedCtl& c, const GroupedArgs& a, int u) {
  const int t = u / a.NB;
  int lo = 0, hi = a.E;  // the expert e with tile[e] <= t < tile[e + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.tile[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int m = c.off[lo + 1] - c.off[lo], nt = c.tile[lo + 1] - c.tile[lo], j = t - c.tile[lo];
  // an expert's tiles are of one size, so that none is a small remainder
  const int per = ((m + nt - 1) / nt + 15) & ~15;
  GroupedUnit r;
  r.e = lo;
  r.row0 = c.off[lo] + j * per;
  r.rows = min(per, m - j * per);
  r.nb = u - t * a.NB;
  return r;
}

// K-major A and B operands use sw128_desc.  M-major A operand, 128B swizzle: 64 M
// elements by 8 reduction rows per 1024-byte atom, the next 8 rows 1024 B on, the
// next 64 M elements one panel (64 rows x 128 B) on.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// 16 weights (8 bytes of codes, one scale) -> 8 BF16 pairs, exact.
__device__ __forceinline__ void dequant16_bf16(uint32_t c0, uint32_t c1, uint32_t s2, uint32_t (&o)[8]) {
  uint32_t v[4];
  e2m1x8_to_f16x2x4(c0, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f16x2_to_bf16x2(hmul2_u32(v[i], s2));
  e2m1x8_to_f16x2x4(c1, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[4 + i] = f16x2_to_bf16x2(hmul2_u32(v[i], s2));
}

template <bool kBackward>
__global__ void __launch_bounds__(gg::kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap, GroupedArgs a) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  GroupedCtl& ctl = *reinterpret_cast<GroupedCtl*>(smem);
  uint8_t* ring = smem + gg::kCtlBytes;
  const int stage_bytes = gg::kABytes + a.tile_rows * 128;
  uint8_t* raw = ring + a.stages * stage_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort_flag;

  for (int i = threadIdx.x; i <= a.E; i += gg::kThreads) ctl.off[i] = a.offsets[i];
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.raw_stages; ++s) {
      mbar_init(ctl.raw_full + s, 1);
      mbar_init(ctl.raw_empty + s, gg::kDequantWarps);
    }
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(ctl.a_full + s, gg::kDequantWarps);
      mbar_init(ctl.b_full + s, 1);
      mbar_init(ctl.empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(ctl.acc_full + b, 1);
      mbar_init(ctl.acc_empty + b, gg::kEpiWarps);
    }
    ctl.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();
  if (warp == 0) {  // token tiles per expert, 8 experts a lane; offsets that do not ascend within 0..R give no tile
    int n[8], sum = 0;
    bool bad = lane == 0 && (ctl.off[0] < 0 || ctl.off[a.E] > a.R);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * lane + i;
      const int m = e < a.E ? ctl.off[e + 1] - ctl.off[e] : 0;
      bad |= e < a.E && ctl.off[e + 1] < ctl.off[e];
      n[i] = (m + a.tile_rows - 1) / a.tile_rows;
      sum += n[i];
    }
    bad = __any_sync(0xffffffffu, bad);
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 8 * lane + i;
      if (e <= a.E) ctl.tile[e] = bad ? 0 : before;
      before += n[i];
    }
    if (lane == 31 && a.E == 256) ctl.tile[256] = bad ? 0 : before;
    if (bad && lane == 0 && blockIdx.x == 0) report(a.st, kFlagBounds, 910);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const int total = ctl.tile[a.E] * a.NB;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- packed weights ----------------
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < total && ok && a.fault != 1; u += gridDim.x) {
        const GroupedUnit w = grouped_unit(ctl, a, u);
        const uint8_t* src = a.blob + (size_t)w.e * a.expert_stride + (size_t)w.nb * a.block_stride;
        for (int s = 0; s < a.steps; ++s, ++it) {
          const int sr = it % a.raw_stages;
          if (!mbar_wait(ctl.raw_empty + sr, ((it / a.raw_stages) & 1u) ^ 1u, abort_flag, a.st, 911)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(ctl.raw_full + sr, gg::kPairBytes);
          bulk_g2s(raw + sr * gg::kPairBytes, src + (size_t)s * a.step_stride, gg::kPairBytes, ctl.raw_full + sr);
        }
      }
      if (!ok) drain_copies(ctl.raw_full, it, a.raw_stages);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      uint32_t ia = 0, j = 0;
      for (int u = blockIdx.x; u < total; u += gridDim.x, ++j) {
        const GroupedUnit w = grouped_unit(ctl, a, u);
        const uint32_t idesc = idesc_bf16(128, (w.rows + 15) & ~15) | (kBackward ? 1u << 15 : 0u);
        const uint32_t buf = j & 1u;
        if (!mbar_wait(ctl.acc_empty + buf, ((j >> 1) & 1u) ^ 1u, abort_flag, a.st, 912)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256u;
        bool ok = true;
        for (int s = 0; s < 2 * a.steps; ++s, ++ia) {
          const int sa = ia % a.stages;
          const uint32_t ph = (ia / a.stages) & 1u;
          if (!mbar_wait(ctl.b_full + sa, ph, abort_flag, a.st, 913) ||
              !mbar_wait(ctl.a_full + sa, ph, abort_flag, a.st, 914)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(ring + sa * stage_bytes);
          const uint64_t ad = kBackward ? sw128_desc_mn(st) : sw128_desc(st);
          const uint64_t bd = sw128_desc(st + gg::kABytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 16 reduction elements: 32 B along a row, or 16 rows of 128 B
            umma_bf16(d, ad + (kBackward ? 128u : 2u) * kk, bd + 2u * kk, idesc, (s | kk) != 0 ? 1u : 0u);
          umma_commit(ctl.empty + sa);
        }
        if (!ok) break;
        umma_commit(ctl.acc_full + buf);
      }
    }
  } else if (warp == 2) {
    // ---------------- rows of x (dy): boxes of 16 rows x 64 reduction elements ----------------
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok && a.fault != 1; u += gridDim.x) {
      const GroupedUnit w = grouped_unit(ctl, a, u);
      const int nbox = (w.rows + 15) >> 4;
      for (int s = 0; s < 2 * a.steps; ++s, ++it) {
        const int sa = it % a.stages;
        int got = 1;
        if (lane == 0) {
          got = mbar_wait(ctl.empty + sa, ((it / a.stages) & 1u) ^ 1u, abort_flag, a.st, 915);
          if (got) mbar_arrive_expect_tx(ctl.b_full + sa, (uint32_t)nbox * 2048u);
        }
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          ok = false;
          break;
        }
        if (lane < nbox)
          tma_2d(ring + sa * stage_bytes + gg::kABytes + lane * 2048, &tmap, s * 64, w.row0 + 16 * lane, ctl.b_full + sa);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) drain_copies(ctl.b_full, it, a.stages);
  } else if (warp >= 8) {
    // ---------------- dequantisers: warp w takes one 16-row sub-block of each 64-long step ----------------
    const int w = warp - 8, q = lane & 3;
    const int slot = seg_pos(lane);
    // forward: step h is tile h (K elements 64 h ..), all 128 rows; backward: rows 64 h .. of both tiles
    const int r = (kBackward ? (w & 3) * 16 : w * 16) + (lane >> 2);
    const uint32_t dst0 = (kBackward ? (uint32_t)(w >> 2) * 8192u : 0u) + (uint32_t)r * 128u;
    const uint32_t x0 = (uint32_t)((2 * q) ^ (r & 7)) * 16u, x1 = (uint32_t)((2 * q + 1) ^ (r & 7)) * 16u;
    uint32_t ir = 0, ia = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
      for (int s = 0; s < a.steps && ok; ++s, ++ir) {
        const int sr = ir % a.raw_stages;
        if (!mbar_wait(ctl.raw_full + sr, (ir / a.raw_stages) & 1u, abort_flag, a.st, 916)) {
          ok = false;
          break;
        }
        uint4 c[2];
        uint32_t sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* tile = raw + sr * gg::kPairBytes + (kBackward ? w >> 2 : h) * kTileBytes;
          const int sb = kBackward ? 4 * h + (w & 3) : w;
          c[h] = *reinterpret_cast<const uint4*>(tile + sb * 512 + slot * 16);
          sc[h] = *reinterpret_cast<const uint16_t*>(tile + kTileCodes + sb * 64 + slot * 2);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ctl.raw_empty + sr);
#pragma unroll
        for (int h = 0; h < 2; ++h, ++ia) {
          const int sa = ia % a.stages;
          if (!mbar_wait(ctl.empty + sa, ((ia / a.stages) & 1u) ^ 1u, abort_flag, a.st, 917)) {
            ok = false;
            break;
          }
          const uint32_t s2 = e4m3x2_to_f16x2(sc[h]);
          const uint32_t p = smem_u32(ring + sa * stage_bytes) + dst0;
          uint32_t o[8];
          dequant16_bf16(c[h].x, c[h].y, dup_lo(s2), o);
          sts128(p + x0, o[0], o[1], o[2], o[3]);
          sts128(p + x1, o[4], o[5], o[6], o[7]);
          dequant16_bf16(c[h].z, c[h].w, dup_hi(s2), o);
          sts128(p + 1024u + x0, o[0], o[1], o[2], o[3]);
          sts128(p + 1024u + x1, o[4], o[5], o[6], o[7]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.a_full + sa);
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: warp w reads TMEM lanes 32 (w % 4) .., one output feature a lane ----------------
    const int i = 32 * (warp & 3) + lane;
    uint32_t j = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++j) {
      const GroupedUnit w = grouped_unit(ctl, a, u);
      const float gs = __ldg(a.gscale + w.e);
      const uint32_t buf = j & 1u;
      if (!mbar_wait(ctl.acc_full + buf, (j >> 1) & 1u, abort_flag, a.st, 918)) break;
      tc_fence_after();
      const uint32_t t = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + buf * 256u;
      const int f = 128 * w.nb + i;
      for (int col = 0; col < w.rows; col += 32) {
        uint32_t v[2][16];
        const bool two = col + 16 < w.rows;
        tmem_ld16_nw(t + (uint32_t)col, v[0]);
        if (two) tmem_ld16_nw(t + (uint32_t)col + 16u, v[1]);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        if (f < a.n_out) {
          const long long base = (long long)(w.row0 + col) * a.ldo + f;
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) {
            if (col + jj < w.rows) {
              const float y = gs * __uint_as_float(v[jj >> 4][jj & 15]);
              if (a.out_f32) reinterpret_cast<float*>(a.out)[base + jj * a.ldo] = y;
              else reinterpret_cast<__nv_bfloat16*>(a.out)[base + jj * a.ldo] = __float2bfloat16_rn(y);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ctl.acc_empty + buf);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// The opt-in shared-memory size, once per device.
static cudaError_t set_grouped_attrs() {
  constexpr int kCached = 64;
  static std::mutex mu;
  static bool done[kCached] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < kCached && done[dev]) return cudaSuccess;
  for (const void* f : {(const void*)grouped_gemm_kernel<false>, (const void*)grouped_gemm_kernel<true>}) {
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, gg::kSmemMax);
    if (e != cudaSuccess) return e;
  }
  if (dev >= 0 && dev < kCached) done[dev] = true;
  return cudaSuccess;
}

cudaError_t launch_grouped_gemm(const GroupedProduct& p, bool backward, const CUtensorMap& rows_map, cudaStream_t st) {
  cudaError_t e = set_grouped_attrs();
  if (e != cudaSuccess) return e;
  const int Np = (p.N + 127) / 128 * 128, nch = p.K / kChunk;
  const size_t row_block = (size_t)nch * kTileBytes;  // one 128-row block's tiles
  GroupedArgs a{};
  a.blob = p.blob;
  a.expert_stride = linear_layout(Np, p.K).stride;
  a.gscale = p.gscale;
  a.offsets = p.offsets;
  a.E = p.E;
  a.R = p.R;
  a.NB = backward ? p.K / 128 : Np / 128;
  a.steps = backward ? Np / 128 : p.K / 128;
  a.block_stride = backward ? (size_t)gg::kPairBytes : row_block;
  a.step_stride = backward ? row_block : (size_t)gg::kPairBytes;
  a.n_out = backward ? p.K : p.N;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.st = p.status;
  a.fault = p.fault;
  // rows per token tile: wide tiles dequantise a weight square once for many rows, narrow ones leave
  // shared memory for a deeper packed ring, which the few-rows end needs to stream weights
  const int avg = p.R / p.E;
  a.tile_rows = avg > 64 ? 256 : avg > 32 ? 128 : 64;
  a.stages = 4;
  const int left = gg::kSmemMax - 1024 - gg::kCtlBytes - a.stages * (gg::kABytes + a.tile_rows * 128);
  a.raw_stages = left / gg::kPairBytes < gg::kMaxRaw ? left / gg::kPairBytes : gg::kMaxRaw;
  const auto fn = backward ? grouped_gemm_kernel<true> : grouped_gemm_kernel<false>;
  fn<<<p.num_sms, gg::kThreads, gg::kSmemMax, st>>>(rows_map, a);
  return cudaGetLastError();
}

}  // namespace nvfp4moe
