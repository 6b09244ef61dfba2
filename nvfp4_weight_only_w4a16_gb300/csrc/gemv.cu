// Matrix-vector products with 4-bit weights for a few rows: the few-rows form of
// the grouped NVFP4 forward, and the INT4 linear with group scales.
//
//   NVFP4: y[r][n] = gs_e sum_k e2m1(W_e[n][k]) s_e[n][k/16] x[r][k]
//   INT4 : y[t][n] = sum_g s[n][g] sum_{k in g} (q[n][k] - z[n][g]) x[t][k]
//
// Bound by the weight bytes, so the weights go from global memory straight into
// registers (16 bytes a lane, a warp reading 512 contiguous bytes), are
// dequantised there into the A fragments of m16n8k16 and multiplied with up to
// 8 * kTiles rows of x held in shared memory; FP32 accumulation.  A warp owns
// one 16-row group of weights and every KS-th 128-element step of K; the KS
// warps of a group are summed through shared memory in a fixed order.  kDepth
// steps are in flight per warp, and the first ones are issued before x is
// staged.  K is taken in slabs whose x fits shared memory.
//
// NVFP4 values are multiplied by their scale in FP16 (exact: at most 6
// significant bits), so x enters as FP16 too, each row of a slab times a power
// of two that brings its largest finite magnitude into [2^13, 2^14); what that
// drops lies 2^-37 below the row's maximum.  INT4 codes q - z are exact in
// BF16 and FP16, x enters as it is, and the scales multiply each group's FP32
// sum: no product is rounded before the sum.
#include "common.cuh"
#include "kernels.h"

namespace nvfp4moe {

namespace gv {
constexpr int kThreads = 256, kWarps = 8;
constexpr int kDepth = 4;  // 128-element K steps in flight per warp
constexpr int kStep = 128;
}  // namespace gv

enum class W4 { kNvfp4, kInt4G32, kInt4G64, kInt4G128 };

struct GemvArgs {
  // NVFP4
  const uint8_t* blob;
  size_t expert_stride;
  const float* gscale;
  const int32_t* offsets;
  int E, R;
  // INT4
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;
  int T;
  // both
  int N, K;
  int KS;          // warps along K per 16-row group: 1, 2, 4, 8
  int slab_steps;  // 128-element steps of x in shared memory, a multiple of kDepth * KS
  int pitch;       // bytes of one x row in shared memory
  const void* x;
  long long ldx;
  void* out;
  long long ldo;
  int out_f32;
  DeviceStatus* st;
};

// ---- the MMA's operand type -------------------------------------------------
template <bool kBf16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One 128-element step of a 16-row group, as loaded: the lane's codes of both
// 64-element chunks and its scales (and zero points).
template <W4 kFmt>
struct StepRaw {
  static constexpr int kGroups = kFmt == W4::kInt4G32 ? 4 : kFmt == W4::kInt4G64 ? 2 : 1;  // per step (INT4)
  uint4 c[2];
  uint32_t s[kFmt == W4::kNvfp4 ? 2 : kGroups];  // INT4: {row r, row r + 8} 16-bit scales per group
  uint32_t z[kFmt == W4::kNvfp4 ? 1 : (kGroups + 1) / 2];  // INT4: {r, r + 8} bytes per group
};

// INT4 layout: codes [N/16][K/64][32 lanes][16 B] -- lane 4 r + t holds the words of row r's elements
// 8 t .. 8 t + 7 and 32 + 8 t .. of the chunk, then row r + 8's; nibble i of a word is element 2 i, nibble
// 4 + i element 2 i + 1.  Scales [N/16][K/128][8 r][128/group][2: row r, row r + 8] 16-bit, zeros alike in bytes.
template <W4 kFmt>
__device__ __forceinline__ void load_step(const GemvArgs& a, const uint8_t* codes, const uint8_t* sc,
                                          const uint8_t* zr, int step, int lane, StepRaw<kFmt>& w) {
  if (kFmt == W4::kNvfp4) {  // codes: the sub-block's bytes in the row block's first tile
    const uint8_t* p = codes + (size_t)(2 * step) * kTileBytes;
    const int slot = seg_pos(lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w.c[h] = ldg_stream(p + h * kTileBytes + slot * 16);
      w.s[h] = __ldg(reinterpret_cast<const uint16_t*>(sc + (size_t)(2 * step + h) * kTileBytes + slot * 2));
    }
  } else {
    constexpr int G = StepRaw<kFmt>::kGroups;
    const uint8_t* p = codes + (size_t)step * 1024 + lane * 16;
    w.c[0] = ldg_stream(p);
    w.c[1] = ldg_stream(p + 512);
    const uint8_t* s = sc + ((size_t)step * 8 + (lane >> 2)) * (G * 4);
    if (G == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
      w.s[0] = v.x;
      w.s[G > 1 ? 1 : 0] = v.y;
      w.s[G > 2 ? 2 : 0] = v.z;
      w.s[G > 3 ? 3 : 0] = v.w;
      if (zr) {
        const uint2 z = __ldg(reinterpret_cast<const uint2*>(zr + ((size_t)step * 8 + (lane >> 2)) * 8));
        w.z[0] = z.x;
        w.z[G > 2 ? 1 : 0] = z.y;
      }
    } else if (G == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
      w.s[0] = v.x;
      w.s[G > 1 ? 1 : 0] = v.y;
      if (zr) w.z[0] = __ldg(reinterpret_cast<const uint32_t*>(zr + ((size_t)step * 8 + (lane >> 2)) * 4));
    } else {
      w.s[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
      if (zr) w.z[0] = __ldg(reinterpret_cast<const uint16_t*>(zr + ((size_t)step * 8 + (lane >> 2)) * 2));
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ float half_of(uint32_t v, int hi) {
  const unsigned short u = (unsigned short)(hi ? v >> 16 : v & 0xFFFFu);
  return kBf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// Pair i of a code word minus the zero point, exact in the operand type:
// magic | q is 128 + q (BF16) or 1024 + q (FP16), and zm holds magic + z twice.
template <bool kBf16>
__device__ __forceinline__ uint32_t int4_pair(uint32_t w, int i, uint32_t zm) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(kBf16 ? 0x43004300u : 0x64006400u));
  uint32_t r;
  if (kBf16) asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zm));
  else asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zm));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t int4_zero_magic(uint32_t z) {  // z: 0..15
  return kBf16 ? 0x43004300u | (z * 0x00010001u) : 0x64006400u | (z * 0x00010001u);
}

// The B fragments' words of one chunk for token g: 8 words (16 elements) in the order the MMAs use them.
template <W4 kFmt>
__device__ __forceinline__ void load_x(const uint8_t* row, int chunk, int t, uint32_t (&x)[8]) {
  const uint8_t* p = row + chunk * 128 + (kFmt == W4::kNvfp4 ? 32 * t : 16 * t);
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint4 b = *reinterpret_cast<const uint4*>(p + (kFmt == W4::kNvfp4 ? 16 : 64));
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// acc += the step's 16 x (8 kTiles) products.  xs: shared x rows, chunk0 the step's first chunk in the slab.
template <W4 kFmt, bool kBf16, int kTiles>
__device__ __forceinline__ void use_step(const StepRaw<kFmt>& w, const uint8_t* xs, int pitch, int chunk0, int rows,
                                         bool zeros, int lane, float (&acc)[kTiles][4]) {
  const int g = lane >> 2, t = lane & 3;
  float part[kTiles][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t x[kTiles][8];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      if (8 * n + g < rows) {
        load_x<kFmt>(xs + (8 * n + g) * pitch, chunk0 + h, t, x[n]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[n][i] = 0u;
      }
    }
    const uint4 c = w.c[h];
    if (kFmt == W4::kNvfp4) {
      const uint32_t s2 = e4m3x2_to_f16x2(w.s[h]);
      const uint32_t slo = dup_lo(s2), shi = dup_hi(s2);
      uint32_t lo[2][4], hi[2][4];
      e2m1x8_to_f16x2x4(c.x, lo[0]);
      e2m1x8_to_f16x2x4(c.y, lo[1]);
      e2m1x8_to_f16x2x4(c.z, hi[0]);
      e2m1x8_to_f16x2x4(c.w, hi[1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t A[4] = {hmul2_u32(lo[j >> 1][2 * (j & 1)], slo), hmul2_u32(hi[j >> 1][2 * (j & 1)], shi),
                               hmul2_u32(lo[j >> 1][2 * (j & 1) + 1], slo), hmul2_u32(hi[j >> 1][2 * (j & 1) + 1], shi)};
#pragma unroll
        for (int n = 0; n < kTiles; ++n) mma_16816<false>(acc[n], A, x[n][2 * j], x[n][2 * j + 1]);
      }
    } else {
      constexpr int G = StepRaw<kFmt>::kGroups;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int run = 2 * h + hf;           // 32-element run of the step
        const int grp = run * G / 4;          // its group
        if (run * G % 4 == 0) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[n][i] = 0.f;
        }
        const uint32_t zz = zeros ? w.z[grp >> 1] >> (16 * (grp & 1)) : 0x0808u;
        const uint32_t zlo = int4_zero_magic<kBf16>(zz & 0xFFu), zhi = int4_zero_magic<kBf16>((zz >> 8) & 0xFFu);
        const uint32_t wl = hf ? c.y : c.x, wh = hf ? c.w : c.z;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t A[4] = {int4_pair<kBf16>(wl, 2 * u, zlo), int4_pair<kBf16>(wh, 2 * u, zhi),
                                 int4_pair<kBf16>(wl, 2 * u + 1, zlo), int4_pair<kBf16>(wh, 2 * u + 1, zhi)};
#pragma unroll
          for (int n = 0; n < kTiles; ++n) mma_16816<kBf16>(part[n], A, x[n][4 * hf + 2 * u], x[n][4 * hf + 2 * u + 1]);
        }
        if ((run + 1) * G % 4 == 0) {
          const float s0 = half_of<kBf16>(w.s[grp], 0), s1 = half_of<kBf16>(w.s[grp], 1);
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            acc[n][0] = fmaf(s0, part[n][0], acc[n][0]);
            acc[n][1] = fmaf(s0, part[n][1], acc[n][1]);
            acc[n][2] = fmaf(s1, part[n][2], acc[n][2]);
            acc[n][3] = fmaf(s1, part[n][3], acc[n][3]);
          }
        }
      }
    }
  }
}

// x rows row0 .. row0 + rows - 1, K elements k0 .. k0 + len - 1, into shared memory as they are.
__device__ __forceinline__ void stage_raw(const void* x, long long ldx, long long row0, int rows, int k0, int len,
                                          uint8_t* xs, int pitch) {
  const int per = len / 8;  // 16-byte pieces of a row
  for (int i = threadIdx.x; i < rows * per; i += gv::kThreads) {
    const int r = i / per, p = i - r * per;
    *reinterpret_cast<uint4*>(xs + r * pitch + p * 16) =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + (row0 + r) * ldx + k0) + p);
  }
}

// The same as FP16 times 2^-p per row, xexp[r] = p.  amax: one word per row, zero on entry and on exit.
__device__ __forceinline__ void stage_f16(const void* x, long long ldx, long long row0, int rows, int k0, int len,
                                          uint8_t* xs, int pitch, unsigned* amax, int* xexp) {
  const int per = len / 8;
  for (int i0 = 0; i0 < rows * per; i0 += gv::kThreads) {
    const int i = i0 + (int)threadIdx.x;
    unsigned m = 0;
    int r = -1;
    if (i < rows * per) {
      r = i / per;
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + (row0 + r) * ldx + k0) +
                            (i - r * per));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // magnitude bits order like the values; infinities and NaN do not count
        const unsigned lo = (w[j] & 0x7FFFu) << 16, hi = w[j] & 0x7FFF0000u;
        if (lo < 0x7F800000u) m = max(m, lo);
        if (hi < 0x7F800000u) m = max(m, hi);
      }
    }
    // one atomic per warp when its lanes share a row
    const int r0 = __shfl_sync(0xffffffffu, r, 0);
    if (__all_sync(0xffffffffu, r == r0)) {
      m = __reduce_max_sync(0xffffffffu, m);
      if ((threadIdx.x & 31) == 0 && r >= 0) atomicMax(amax + r, m);
    } else if (r >= 0) {
      atomicMax(amax + r, m);
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < rows) xexp[threadIdx.x] = prescale_exp(__uint_as_float(amax[threadIdx.x]));
  __syncthreads();
  if ((int)threadIdx.x < rows) amax[threadIdx.x] = 0u;
  for (int i = threadIdx.x; i < rows * per; i += gv::kThreads) {
    const int r = i / per, p = i - r * per;
    const uint4 v =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + (row0 + r) * ldx + k0) + p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int ex = xexp[r];
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(ldexpf(__uint_as_float(w[j] << 16), -ex),
                                          ldexpf(__uint_as_float(w[j] & 0xFFFF0000u), -ex));
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(xs + r * pitch + p * 16) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <W4 kFmt, bool kBf16, int kTiles>
__global__ void __launch_bounds__(gv::kThreads, 2) gemv_kernel(GemvArgs a) {
  extern __shared__ __align__(16) uint8_t xs[];
  __shared__ unsigned amax[8 * kTiles];
  __shared__ int xexp[8 * kTiles];
  __shared__ int unit[3];  // expert, first row, rows
  __shared__ int wsum[gv::kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRows = 8 * kTiles;
  int e = 0, row0 = 0, rows = a.T;
  if (kFmt == W4::kNvfp4) {
    // blockIdx.y -> (expert, tile of at most kRows rows); thread i looks at expert i
    if (threadIdx.x < kRows) amax[threadIdx.x] = 0u;
    if (threadIdx.x == 0) unit[2] = 0;
    const int i = threadIdx.x;
    const int o0 = i < a.E ? __ldg(a.offsets + i) : 0, o1 = i < a.E ? __ldg(a.offsets + i + 1) : 0;
    const bool bad = o0 < 0 || o1 < o0 || o1 > a.R;
    const int nt = (o1 - o0 + kRows - 1) / kRows;
    int before = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) wsum[warp] = before;
    if (__syncthreads_or(bad)) {  // offsets that do not ascend within 0..R: nothing is computed
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) report(a.st, kFlagBounds, 920);
      return;
    }
    before -= nt;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    const int j = (int)blockIdx.y - before;
    if (j >= 0 && j < nt) {
      unit[0] = i;
      unit[1] = o0 + j * kRows;
      unit[2] = min(kRows, o1 - o0 - j * kRows);
    }
    __syncthreads();
    e = unit[0], row0 = unit[1], rows = unit[2];
    if (rows == 0) return;
  }
  const int RG = gv::kWarps / a.KS;
  const int rgroups = a.N / 16;
  const int ks = warp / RG;
  const int rg = blockIdx.x * RG + warp % RG;
  const bool active = rg < rgroups;
  const int steps = a.K / gv::kStep;

  const uint8_t *codes, *sc, *zr = nullptr;
  if (kFmt == W4::kNvfp4) {
    const uint8_t* tile = a.blob + (size_t)e * a.expert_stride + (size_t)(rg >> 3) * (a.K / kChunk) * kTileBytes;
    codes = tile + (rg & 7) * 512;
    sc = tile + kTileCodes + (rg & 7) * 64;
  } else {
    constexpr int G = StepRaw<kFmt>::kGroups;
    codes = a.codes + (size_t)rg * steps * 1024;
    sc = static_cast<const uint8_t*>(a.scales) + (size_t)rg * steps * (32 * G);
    if (a.zeros) zr = a.zeros + (size_t)rg * steps * (16 * G);
  }

  StepRaw<kFmt> buf[gv::kDepth];
#pragma unroll
  for (int d = 0; d < gv::kDepth; ++d)
    if (active && ks + d * a.KS < steps) load_step<kFmt>(a, codes, sc, zr, ks + d * a.KS, lane, buf[d]);

  float acc[kTiles][4], part[kTiles][4];
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = part[n][i] = 0.f;

  for (int s0 = 0; s0 < steps; s0 += a.slab_steps) {
    const int s1 = min(s0 + a.slab_steps, steps);
    if (s0) __syncthreads();  // the previous slab has been used
    if (kFmt == W4::kNvfp4)
      stage_f16(a.x, a.ldx, row0, rows, s0 * gv::kStep, (s1 - s0) * gv::kStep, xs, a.pitch, amax, xexp);
    else
      stage_raw(a.x, a.ldx, 0, rows, s0 * gv::kStep, (s1 - s0) * gv::kStep, xs, a.pitch);
    __syncthreads();
    if (active) {
      for (int s = s0 + ks; s < s1; s += gv::kDepth * a.KS) {
#pragma unroll
        for (int d = 0; d < gv::kDepth; ++d) {
          const int sd = s + d * a.KS;
          if (sd < s1) {
            use_step<kFmt, kBf16, kTiles>(buf[d], xs, a.pitch, 2 * (sd - s0), rows, zr != nullptr, lane,
                                          kFmt == W4::kNvfp4 ? part : acc);
            const int nx = sd + gv::kDepth * a.KS;
            if (nx < steps) load_step<kFmt>(a, codes, sc, zr, nx, lane, buf[d]);
          }
        }
      }
      if (kFmt == W4::kNvfp4) {  // undo the slab's row scales
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * n + 2 * (lane & 3) + (i & 1);
            if (r < rows) acc[n][i] += ldexpf(part[n][i], xexp[r]);
            part[n][i] = 0.f;
          }
      }
    }
  }

  if (a.KS > 1) {  // sum the group's warps in order
    __syncthreads();
    float* red = reinterpret_cast<float*>(xs);
    if (ks > 0) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((warp * kTiles + n) * 4 + i) * 32 + lane] = acc[n][i];
    }
    __syncthreads();
    if (ks == 0) {
      for (int w = warp + RG; w < gv::kWarps; w += RG)
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] += red[((w * kTiles + n) * 4 + i) * 32 + lane];
    }
  }
  if (ks == 0 && active) {
    const float gs = kFmt == W4::kNvfp4 ? __ldg(a.gscale + e) : 1.0f;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * n + 2 * (lane & 3) + (i & 1);
        const int f = 16 * rg + (lane >> 2) + 8 * (i >> 1);
        if (r < rows) {
          const long long o = (long long)(row0 + r) * a.ldo + f;
          const float y = kFmt == W4::kNvfp4 ? gs * acc[n][i] : acc[n][i];
          if (a.out_f32) static_cast<float*>(a.out)[o] = y;
          else if (kFmt == W4::kNvfp4 || kBf16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
          else static_cast<__half*>(a.out)[o] = __float2half_rn(y);
        }
      }
  }
}

// Warps along K (KS): as few as give at least two CTAs a multiprocessor -- a
// wider CTA stages x for more weight rows -- and 8 where the matrix is small.
static int pick_ks(int row_tiles, int N, int num_sms, int ks_max) {
  int ks = 1;
  while (ks < ks_max && (long long)row_tiles * ((N / 16 + gv::kWarps / ks - 1) / (gv::kWarps / ks)) < 2 * num_sms) ks *= 2;
  return ks;
}

// x's shared-memory layout for up to max_rows rows: at most 64 KB, three CTAs' worth a multiprocessor.
static size_t set_slab(GemvArgs& a, int max_rows, int pad) {
  const int steps = a.K / gv::kStep;
  const int most = max_rows <= 8 ? 32 : 16;  // 128-element steps: a multiple of kDepth * KS (KS <= 8, or 4 above 8 rows)
  a.slab_steps = most;
  a.pitch = (steps < most ? steps : most) * gv::kStep * 2 + pad;
  const size_t red = (size_t)gv::kWarps * 32 * 4 * 4 * (max_rows <= 8 ? 1 : 2);  // the K sum reuses it
  const size_t x = (size_t)max_rows * a.pitch;
  return x > red ? x : red;
}

template <W4 kFmt, bool kBf16, int kTiles>
static cudaError_t launch_gemv(const GemvArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  constexpr int kMaxSmem = 8 * kTiles * ((kTiles == 1 ? 32 : 16) * gv::kStep * 2 + 64);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(gemv_kernel<kFmt, kBf16, kTiles>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  gemv_kernel<kFmt, kBf16, kTiles><<<grid, gv::kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_grouped_gemv(const GroupedProduct& p, cudaStream_t st) {
  const int Np = (p.N + 127) / 128 * 128;
  GemvArgs a{};
  a.blob = p.blob;
  a.expert_stride = linear_layout(Np, p.K).stride;
  a.gscale = p.gscale;
  a.offsets = p.offsets;
  a.E = p.E;
  a.R = p.R;
  a.N = p.N;
  a.K = p.K;
  a.x = p.in;
  a.ldx = p.ldi;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.st = p.status;
  const int touched = p.R < p.E ? p.R : p.E;  // at most
  const bool wide = p.R > 8 * p.E;            // some expert has more than 8 rows: tiles of 16
  const int rows = wide ? 16 : 8;
  a.KS = pick_ks(touched, p.N, p.num_sms, wide ? 4 : 8);
  const int RG = gv::kWarps / a.KS;
  const dim3 grid((p.N / 16 + RG - 1) / RG, touched + p.R / rows);
  const size_t smem = set_slab(a, rows, 16);
  return wide ? launch_gemv<W4::kNvfp4, false, 2>(a, grid, smem, st)
              : launch_gemv<W4::kNvfp4, false, 1>(a, grid, smem, st);
}

template <W4 kFmt, bool kBf16>
static cudaError_t launch_int4(GemvArgs& a, int num_sms, cudaStream_t st) {
  const bool wide = a.T > 8;
  a.KS = pick_ks(1, a.N, num_sms, wide ? 4 : 8);
  const int RG = gv::kWarps / a.KS;
  const dim3 grid((a.N / 16 + RG - 1) / RG);
  const size_t smem = set_slab(a, a.T, 64);
  return wide ? launch_gemv<kFmt, kBf16, 2>(a, grid, smem, st) : launch_gemv<kFmt, kBf16, 1>(a, grid, smem, st);
}

cudaError_t launch_int4_gemv(const Int4Product& p, cudaStream_t st) {
  GemvArgs a{};
  a.codes = p.codes;
  a.scales = p.scales;
  a.zeros = p.zeros;
  a.T = p.T;
  a.N = p.N;
  a.K = p.K;
  a.x = p.x;
  a.ldx = p.ldx;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  if (p.act_f16)
    return p.group == 32   ? launch_int4<W4::kInt4G32, false>(a, p.num_sms, st)
           : p.group == 64 ? launch_int4<W4::kInt4G64, false>(a, p.num_sms, st)
                           : launch_int4<W4::kInt4G128, false>(a, p.num_sms, st);
  return p.group == 32   ? launch_int4<W4::kInt4G32, true>(a, p.num_sms, st)
         : p.group == 64 ? launch_int4<W4::kInt4G64, true>(a, p.num_sms, st)
                         : launch_int4<W4::kInt4G128, true>(a, p.num_sms, st);
}

// ---------------------------------------------------------------------------
// INT4 packer: one thread per 16-byte code segment.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t int4_word(uint32_t w) {  // canonical nibble m = element m
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= (((w >> (8 * i)) & 0xFu) << (4 * i)) | (((w >> (8 * i + 4)) & 0xFu) << (16 + 4 * i));
  return o;
}

__global__ void pack_int4_codes_kernel(const uint8_t* __restrict__ w_q, uint8_t* __restrict__ codes, int N, int K) {
  const size_t s = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int nch = K / kChunk;
  if (s >= (size_t)N / 16 * nch * 32) return;
  const int lane = (int)(s & 31);
  const size_t rc = s >> 5;
  const int c = (int)(rc % nch);
  const size_t rg = rc / nch;
  const int t = lane & 3;
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const size_t n = 16 * rg + (lane >> 2) + 8 * (i >> 1);
    const int k = 64 * c + 32 * (i & 1) + 8 * t;
    o[i] = int4_word(*reinterpret_cast<const uint32_t*>(w_q + n * (size_t)(K / 2) + k / 2));
  }
  *reinterpret_cast<uint4*>(codes + s * 16) = make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void pack_int4_scales_kernel(const uint16_t* __restrict__ scale, const uint8_t* __restrict__ zero, int f16,
                                        int N, int K, int group, uint16_t* __restrict__ scales,
                                        uint8_t* __restrict__ zeros, int* __restrict__ bad) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;  // canonical [N][K/group]
  const int ng = K / group;
  if (i >= (size_t)N * ng) return;
  const size_t n = i / ng;
  const int grp = (int)(i - n * ng);
  const int G = 128 / group, step = grp / G, gi = grp - step * G;
  const size_t o = ((((n >> 4) * (K / 128) + step) * 8 + (n & 7)) * G + gi) * 2 + ((n >> 3) & 1);
  const uint16_t s = scale[i];
  const uint16_t inf = f16 ? 0x7C00u : 0x7F80u;
  bool b = (s & inf) == inf;
  scales[o] = s;
  if (zero) {
    const uint8_t z = zero[i];
    b |= z > 15;
    zeros[o] = z;
  }
  if (b) atomicAdd(bad, 1);
}

cudaError_t launch_pack_int4(const uint8_t* w_q, const void* scale, const uint8_t* zero, int act_f16, int N, int K,
                             int group, uint8_t* codes, void* scales, uint8_t* zeros, int* bad, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(bad, 0, sizeof(int), st);
  if (e != cudaSuccess) return e;
  const int thr = 256;
  const size_t nseg = (size_t)N * K / 32, ns = (size_t)N * (K / group);
  pack_int4_codes_kernel<<<(unsigned)((nseg + thr - 1) / thr), thr, 0, st>>>(w_q, codes, N, K);
  pack_int4_scales_kernel<<<(unsigned)((ns + thr - 1) / thr), thr, 0, st>>>(
      static_cast<const uint16_t*>(scale), zero, act_f16, N, K, group, static_cast<uint16_t*>(scales), zeros, bad);
  return cudaGetLastError();
}

}  // namespace nvfp4moe
