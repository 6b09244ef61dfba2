// Matrix-vector products with 4-bit weights for a few rows: the few-rows form of
// the grouped NVFP4 forward, and the INT4 linear with group scales.
//
//   NVFP4: y[r][n] = gs_e sum_k e2m1(W_e[n][k]) s_e[n][k/16] x[r][k]
//   INT4 : y[t][n] = sum_g s[n][g] (sum_{k in g} q[n][k] x[t][k] - z[n][g] sum_{k in g} x[t][k])
//
// Bound by the weight bytes: what counts is how many of them are in flight (a read
// takes about 1.7 us under load, so 96 KB and more a multiprocessor) and how few
// instructions a byte costs.  Each of a CTA's warps streams its weights through a
// ring of its own in shared memory (cp.async, no barrier: a lane reads back what it
// copied itself, but for the scales), turns them into the A fragments of m16n8k16 in
// registers and multiplies them with up to 8 rows of x, also in shared memory; FP32
// accumulation.  The unit of distribution is a granule of kRg 16-row groups over all
// of K: one persistent CTA a multiprocessor takes an equal contiguous run of them,
// kWarps / KS at a time, of which each is shared by KS warps that take every KS-th
// 128-element step of K and are summed through shared memory in a fixed order, one
// barrier each time.  The rings run ahead across that, and across new rows of x.
// Rows of x that do not fit beside the rings are spread over a cluster (INT4): each
// of its CTAs takes a slice of K, and sends its sums to the CTA that stores them,
// which adds them in a fixed order one batch later.  (8192 x 8192, groups of 32, 16
// tokens: 18.6 us against 26.9 as tiles of 4 rows, each with the weights converted
// again; 4096 x 16384, groups of 64: 18.1 against 42.7.  16 rows at a time instead of
// twice 8 was a fifth slower in an earlier form of this kernel: work per weight and
// token outweighs the conversion, and the shorter slices need more batches.)
//
// Both formats run on FP16 operands.  x enters as FP16 times a power of two per row
// that brings its largest finite magnitude into [2^13, 2^14); what that drops lies
// 2^-38 below the row's maximum (INT4: 2^-34, see below).  NVFP4 codes times their scale are exact in FP16
// (at most 6 significant bits).  An INT4 code needs no conversion: its four bits,
// masked in place, are the FP16 subnormal q 2^-22, or q 2^-18 one nibble higher,
// which x's matching elements, staged times 2^-4, make good (their smallest step is 2^4
// times farther up).  The zero point comes off a group's FP32 sum with the sum of x
// over the group, which is staged too.
// The tensor core aligns what it adds by exponents that a subnormal does not show, and
// truncates there.  So the codes lie as high as FP16's ten low bits allow: the packed
// words are rotated left by 2 bits, and the second byte comes down by a rotation in place
// of a shift.  FP32 results of BF16 x are off by 1 to 1.5e-7 of their norm (codes of normal
// weights; FP32 arithmetic 1 to 4e-7), two bits lower by 4 to 6e-7.  FP16's 11 significant
// bits still show (2e-7; 7e-7 with codes next to their zero points), so with an FP32 result
// that case (kCenter) makes q - 8 of every code, a normal number, at one more instruction a
// pair (1024 | 4 q, less 1056), and takes z - 8 off the sums: 1e-7, and a quarter to a third
// more time (131072 x 4096, 4 tokens, 46 -> 62 us).
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace gv {
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kStep = 128;
constexpr int kRg = 2;            // 16-row groups a warp multiplies with the same x: two chains of MMAs
constexpr int kRows = 8;          // rows of x in one MMA: its N
constexpr int kShared = 32 * 32 * 4;  // bytes of a batch's sums, where a cluster adds them: 4 granules'
constexpr int kMaxCluster = 8;
constexpr int kDepth = 3;         // steps in flight per warp, kRg KB of codes each
constexpr int kMaxTiles = 256 + kGemvMaxRows / 2;  // NVFP4: of a call; all but an expert's last have 2 rows or more
constexpr int smem_for(bool nvfp4) { return (nvfp4 ? 180 : 192) * 1024; }  // of rings and x; the rest is static
}  // namespace gv

enum class W4 { kNvfp4, kInt4G32, kInt4G64, kInt4G128 };
__host__ __device__ constexpr int int4_groups(W4 f) {  // of 128 elements of a row
  return f == W4::kInt4G32 ? 4 : f == W4::kInt4G64 ? 2 : 1;
}

struct GemvArgs {
  // NVFP4
  const uint8_t* blob;
  size_t expert_stride;
  const float* gscale;
  const int32_t* offsets;
  int E, R;
  // INT4
  const uint8_t* packed;
  int T;
  // both
  int N, K;
  int S;           // CTAs of a cluster, which share K (1 for NVFP4)
  int tiles;       // INT4: ceil(T / tile_rows)
  int KS;          // warps along the CTA's slice of K per granule: 1, 2, 4, 8, 16
  int tile_rows;   // rows of x per tile, up to 8
  int pitch;       // bytes of one x row in shared memory
  const void* x;
  long long ldx;
  void* out;
  long long ldo;
  int out_f32;
  bool once;       // the weights do not outlast the call in L2
  DeviceStatus* st;
  int fault;       // 1: x is not copied, so that the wait for it ends with a timeout
};

// D += A B (m16n8k16, FP16 in, FP32 out); not volatile, so that the two row groups' chains interleave.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hsub2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The weights' L2 policy.  Matrices larger than L2 are gone before the next call reads them again: L2 gives their lines
// up first, and need not write back or drop what else it holds for them (128 experts of 1536 x 4096, 128 rows, 51.5 ->
// 50.3 us, behind 256 MB of written lines 65 -> 57; INT4 131072 x 4096 47.1 -> 46.2 and 63 -> 55).  Smaller ones may
// still be there (INT4 12576 x 4096: 8.0 us, 8.4 with their lines given up).
__device__ __forceinline__ uint64_t weight_policy(bool once) {
  uint64_t first, normal;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return once ? first : normal;
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() {  // all but the latest kDepth - 1 groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(gv::kDepth - 1) : "memory");
}

// One 128-element step of a granule (two 16-row groups).
//   NVFP4: in the packed tiles, the two groups' codes are 1024 contiguous bytes of each of the step's two tiles and
//   their scales 128; a slot holds [chunk][group][512 B] codes (lane t's at seg_pos(t)), then [chunk][group][64 B] scales.
//   INT4: packed as [N/32][K/128] blocks, one block a slot's contents: [group][chunk][32 lanes][16 B] codes -- lane
//   4 r + t holds the words of row r's elements 8 t .. 8 t + 7 and 32 + 8 t .. of the chunk, then row r + 8's; nibble i
//   of a word is element 2 i, nibble 4 + i element 2 i + 1, and the word is rotated left by 2 bits -- then [group][8 r][128/g][2: row r, row r + 8] 16-bit
//   scales and, if the matrix has any, zero points alike in bytes.
template <W4 kFmt, bool kZeros>
struct Step {
  static constexpr bool kNv = kFmt == W4::kNvfp4;
  static constexpr int kGroups = int4_groups(kFmt);
  static constexpr int kCodes = gv::kRg * 1024;
  static constexpr int kZeroOff = kCodes + 64 * kGroups;
  static constexpr int kBytes = kNv ? kCodes + 256 : kZeroOff + (kZeros ? 32 * kGroups : 0);  // of a slot
  static constexpr int kSlot = (kBytes + 127) & ~127;  // slots start on 128 bytes: off it, a read of 512 takes a turn more
  static constexpr int kStride = kNv ? 2 * kTileBytes : kBytes;  // in memory, from a step to the next
  uint4 c[gv::kRg][2];                     // the lane's codes
  uint32_t s[gv::kRg][kNv ? 2 : kGroups];  // INT4: {row r, row r + 8} 16-bit scales per group
  uint32_t z[gv::kRg][(kGroups + 1) / 2];  // INT4: {r, r + 8} bytes per group

  // Start the copy of a step into a slot.  c: the lane's place in the codes; s (NVFP4): lanes 0..15's in the scales.
  static __device__ __forceinline__ void copy(const uint8_t* c, const uint8_t* s, uint32_t slot, int lane, uint64_t policy) {
    const uint32_t d = slot + lane * 16;
    if (kNv) {
      copy16(d, c, policy);
      copy16(d + 512, c + 512, policy);
      copy16(d + 1024, c + kTileBytes, policy);
      copy16(d + 1536, c + kTileBytes + 512, policy);
      if (lane < 16) copy16(d + kCodes, s, policy);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(d + 512 * i, c + 512 * i, policy);
      if (lane < (kBytes - kCodes) / 16) copy16(d + kCodes, c + kCodes, policy);
    }
  }
  // The lane's part of a landed step.
  __device__ __forceinline__ void read(const uint8_t* slot, int lane) {
    constexpr int G = kGroups;
#pragma unroll
    for (int q = 0; q < gv::kRg; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        c[q][h] = *reinterpret_cast<const uint4*>(slot + (kNv ? 1024 * h + 512 * q + seg_pos(lane) * 16 : 1024 * q + 512 * h + lane * 16));
#pragma unroll
    for (int q = 0; q < gv::kRg; ++q) {
      const uint8_t* sp = slot + kCodes + (kNv ? q * 64 + seg_pos(lane) * 2 : q * 32 * G + (lane >> 2) * 4 * G);
      const uint8_t* zp = slot + kZeroOff + q * 16 * G + (lane >> 2) * 2 * G;
      if (kNv) {
        s[q][0] = *reinterpret_cast<const uint16_t*>(sp);
        s[q][G > 0 ? 1 : 0] = *reinterpret_cast<const uint16_t*>(sp + 128);
      } else if (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(sp);
        s[q][0] = v.x;
        s[q][G > 1 ? 1 : 0] = v.y;
        s[q][G > 2 ? 2 : 0] = v.z;
        s[q][G > 3 ? 3 : 0] = v.w;
        if (kZeros) {
          const uint2 v2 = *reinterpret_cast<const uint2*>(zp);
          z[q][0] = v2.x;
          z[q][G > 2 ? 1 : 0] = v2.y;
        }
      } else if (G == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(sp);
        s[q][0] = v.x;
        s[q][G > 1 ? 1 : 0] = v.y;
        if (kZeros) z[q][0] = *reinterpret_cast<const uint32_t*>(zp);
      } else {
        s[q][0] = *reinterpret_cast<const uint32_t*>(sp);
        if (kZeros) z[q][0] = *reinterpret_cast<const uint16_t*>(zp);
      }
    }
  }
};

template <bool kBf16>
__device__ __forceinline__ float scale_of(uint32_t v, int hi) {
  if (kBf16) return __uint_as_float(hi ? v & 0xFFFF0000u : v << 16);
  return __half2float(__ushort_as_half((unsigned short)(hi ? v >> 16 : v & 0xFFFFu)));
}
__device__ __forceinline__ float byte_of(uint32_t v, int i) {  // 0..255, exactly
  return __uint_as_float(__byte_perm(v, 0x4B000000u, 0x7440 + i)) - 8388608.0f;
}

// acc += the step's (16 kRg) x 8 products.  xl: the lane's x row at the step's first element and the lane's
// position in it; sl: the lane's group sums of x at the step's first group (INT4).
template <W4 kFmt, bool kBf16, bool kZeros, bool kCenter>
__device__ __forceinline__ void use_step(const Step<kFmt, kZeros>& w, const uint8_t* xl, const float* sl,
                                         float (&acc)[gv::kRg][4]) {
  uint32_t x[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // NVFP4: 16 elements a lane and chunk; INT4: 8 elements of either half of the chunk
      const uint4 v = *reinterpret_cast<const uint4*>(xl + h * 128 + p * (kFmt == W4::kNvfp4 ? 16 : 64));
      x[h][4 * p] = v.x, x[h][4 * p + 1] = v.y, x[h][4 * p + 2] = v.z, x[h][4 * p + 3] = v.w;
    }
  if (kFmt == W4::kNvfp4) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < gv::kRg; ++q) {
        const uint32_t s2 = e4m3x2_to_f16x2(w.s[q][h]);
        const uint32_t slo = dup_lo(s2), shi = dup_hi(s2);
        uint32_t lo[2][4], hi[2][4];
        e2m1x8_to_f16x2x4(w.c[q][h].x, lo[0]);
        e2m1x8_to_f16x2x4(w.c[q][h].y, lo[1]);
        e2m1x8_to_f16x2x4(w.c[q][h].z, hi[0]);
        e2m1x8_to_f16x2x4(w.c[q][h].w, hi[1]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_16816(acc[q], hmul2_u32(lo[j >> 1][2 * (j & 1)], slo), hmul2_u32(hi[j >> 1][2 * (j & 1)], shi),
                    hmul2_u32(lo[j >> 1][2 * (j & 1) + 1], slo), hmul2_u32(hi[j >> 1][2 * (j & 1) + 1], shi), x[h][2 * j],
                    x[h][2 * j + 1]);
      }
  } else {
    constexpr int G = int4_groups(kFmt);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float2 sx = *reinterpret_cast<const float2*>(sl + g * gv::kRows);
#pragma unroll
      for (int q = 0; q < gv::kRg; ++q) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int run = g * (4 / G); run < (g + 1) * (4 / G); ++run) {  // 32 elements
          const uint4 c = w.c[q][run >> 1];
          const uint32_t l = run & 1 ? c.y : c.x, h = run & 1 ? c.w : c.z;
          const uint32_t* xr = x[run >> 1] + 4 * (run & 1);
          const uint32_t l8 = __byte_perm(l, 0, 0x0321), h8 = __byte_perm(h, 0, 0x0321);  // rotated right by 8
          // kCenter: 1024 | 4 q less 1056, and 1024 | 64 q less 1536 (0x6400 = 1024, 0x6420 = 1056, 0x6600 = 1536)
          const auto lo = [](uint32_t w) {
            return kCenter ? hsub2_u32((w & 0x003C003Cu) | 0x64006400u, 0x64206420u) : w & 0x003C003Cu;
          };
          const auto hi = [](uint32_t w) {
            return kCenter ? hsub2_u32((w & 0x03C003C0u) | 0x64006400u, 0x66006600u) : w & 0x03C003C0u;
          };
          mma_16816(part, lo(l), lo(h), hi(l), hi(h), xr[0], xr[1]);
          mma_16816(part, lo(l8), lo(h8), hi(l8), hi(h8), xr[2], xr[3]);
        }
        constexpr float kOff = kCenter ? 8.0f : 0.0f;
        float z0 = 8.0f - kOff, z1 = 8.0f - kOff;
        if (kZeros) {
          z0 = byte_of(w.z[q][g >> 1], 2 * (g & 1)) - kOff, z1 = byte_of(w.z[q][g >> 1], 2 * (g & 1) + 1) - kOff;
        }
        const float s0 = scale_of<kBf16>(w.s[q][g], 0), s1 = scale_of<kBf16>(w.s[q][g], 1);
        acc[q][0] = fmaf(s0, fmaf(-z0, sx.x, part[0]), acc[q][0]);
        acc[q][1] = fmaf(s0, fmaf(-z0, sx.y, part[1]), acc[q][1]);
        acc[q][2] = fmaf(s1, fmaf(-z1, sx.x, part[2]), acc[q][2]);
        acc[q][3] = fmaf(s1, fmaf(-z1, sx.y, part[3]), acc[q][3]);
      }
    }
  }
}

// 2^e as a product of two floats, for |e| <= 252.
__device__ __forceinline__ float2 pow2_pair(int e) {
  const int a = e >> 1, b = e - a;
  return make_float2(__int_as_float((127 + a) << 23), __int_as_float((127 + b) << 23));
}
// p such that a row whose largest finite magnitude has these FP32 bits lies below 2^14 times 2^p
// (in [2^13, 2^14) unless it is below FP32's normal range).
__device__ __forceinline__ int row_exponent(unsigned bits) { return bits ? (int)(bits >> 23) - 140 : 0; }

// sum + the two halves of w times s (FP16), in FP32.
__device__ __forceinline__ float add_halves(float sum, uint32_t w, uint16_t s) {
  asm("{\n .reg .f16 l, h;\n mov.b32 {l, h}, %1;\n fma.rn.f32.f16 %0, l, %2, %0;\n fma.rn.f32.f16 %0, h, %2, %0;\n}"
      : "+f"(sum)
      : "r"(w), "h"(s));
  return sum;
}

// x rows into shared memory as FP16 times 2^-p per row; INT4: elements 2, 3, 6 and 7 of every 8 times another
// 2^-4, and 2^-22 (kCenter: 4) times the sums over each group of the matrix into sums[group][8].  In two parts:
// start() copies the rows as they are (bulk copies, by one thread), finish() waits for them, finds each row's p and
// converts in place; a row's 16-byte pieces are shared by kWarps / rows warps.
// (Small loops on purpose: a call's first use of its code comes from memory, and this runs before any product.)
template <W4 kFmt, bool kBf16, bool kCenter>
struct Stage {
  uint8_t* xs;
  int pitch, per, rows;  // pieces of a row (of the CTA's slice)
  int first;             // element the slice begins at
  __device__ __forceinline__ Stage(const GemvArgs& a, uint8_t* x, int step0, int steps)
      : xs(x), pitch(a.pitch), per(steps * (gv::kStep / 8)), rows(0), first(step0 * gv::kStep) {}
  __device__ __forceinline__ void start(const GemvArgs& a, int row0, uint64_t* bar) {  // one thread
    if (a.fault == 1) return;
    mbar_arrive_expect_tx(bar, (uint32_t)(rows * per * 16));
#pragma unroll 1
    for (int r = 0; r < rows; ++r)
      bulk_g2s(xs + r * pitch, static_cast<const uint16_t*>(a.x) + (long long)(row0 + r) * a.ldx + first, (uint32_t)(per * 16), bar);
  }
  static __device__ __forceinline__ float value(uint32_t w, int hi) {
    return kBf16 ? __uint_as_float(hi ? w & 0xFFFF0000u : w << 16)
                 : __half2float(__ushort_as_half((unsigned short)(hi ? w >> 16 : w & 0xFFFFu)));
  }
  // amax: the rows' largest finite magnitudes (FP32 bits, which order alike), zero on entry.  odd: set where one has an
  // element that is not finite.  False, in every thread,
  // when the copies did not land in time (reported).  The barrier after the writes is the caller's.
  __device__ __forceinline__ bool finish(float* sums, unsigned* amax, int* odd, uint64_t* bar, uint32_t parity,
                                         volatile int* abort, DeviceStatus* st) {
    // one answer for a warp: at the limit one lane may still see the copy and another not, and the reductions below
    // need them all
    const bool landed = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, st, 921));
    const int lane = threadIdx.x & 31, warps = gv::kWarps / rows, r = (int)(threadIdx.x >> 5) / warps;
    const int p0 = ((int)(threadIdx.x >> 5) - r * warps) * 32, dp = warps * 32;
    uint8_t* row = xs + r * pitch;
    if (landed && r < rows) {
      constexpr unsigned kInf = kBf16 ? 0x7F80u : 0x7C00u;
      unsigned m = 0;
#pragma unroll 2
      for (int p = p0 + lane; p < per; p += dp) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + p * 16);
        m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
        m = __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
      }
      m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
      if (m >= kInf) {  // once more, of the finite ones
        m = 0;
#pragma unroll 1
        for (int i = 8 * (p0 + lane); i < 8 * per; i += i % 8 == 7 ? 8 * dp - 7 : 1) {
          const unsigned e = reinterpret_cast<const uint16_t*>(row)[i] & 0x7FFFu;
          if (e < kInf) m = max(m, e);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (kFmt != W4::kNvfp4) *odd = 1;
      }
      if (lane == 0) atomicMax(amax + r, __float_as_uint(value(m, 0)));
    }
    if (__syncthreads_or(!landed)) return false;
    if (r >= rows) return true;
    constexpr int kLanes = kFmt == W4::kNvfp4 ? 1 : 16 / int4_groups(kFmt);  // threads per group
    const float2 f2 = pow2_pair(-row_exponent(amax[r]));
#pragma unroll 1
    for (int p = p0 + lane; p - lane < per; p += dp) {  // whole warps, for the shuffles
      const bool ok = p < per;  // rows are multiples of 16 pieces, so half a warp is in or out
      uint4* at = reinterpret_cast<uint4*>(row + (ok ? p : 0) * 16);
      const uint4 v = *at;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // odd pairs of INT4: what the MMA multiplies with q 2^-18
        const float f = kFmt != W4::kNvfp4 && (j & 1) ? f2.y * 0.0625f : f2.y;
        const __half2 h = __floats2half2_rn(value(w[j], 0) * f2.x * f, value(w[j], 1) * f2.x * f);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
        if (kFmt != W4::kNvfp4) sum = add_halves(sum, o[j], j & 1 ? 0x4C00u : 0x3C00u);  // times 16, 1
      }
      if (ok) *at = make_uint4(o[0], o[1], o[2], o[3]);
      if (kFmt != W4::kNvfp4) {  // a group's pieces belong to neighbouring lanes
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (ok && p % kLanes == 0) sums[p / kLanes * gv::kRows + r] = sum * (kCenter ? 4.0f : 0x1p-22f);
      }
    }
    return true;
  }
};

// A CTA's run of granules, u0 .. u1 - 1.  NVFP4: tile * granules + granule, over all CTAs.  INT4: clusters c, c + 1, ..
// c + tiles - 1 take the same granules for one tile of x each, so that they share the weights in L2.
template <bool kNv>
__device__ __forceinline__ void run_of(const GemvArgs& a, int tiles, int granules, int& u0, int& u1) {
  const int n = kNv ? (int)gridDim.x : (int)gridDim.x / a.S / tiles;
  const int c = kNv ? (int)blockIdx.x : (int)blockIdx.x / a.S / tiles;
  const int all = kNv ? tiles * granules : granules;
  const int base = all / n, extra = all - base * n;
  u0 = c * base + min(c, extra);
  u1 = c < n ? u0 + base + (c < extra ? 1 : 0) : u0;
}

// INT4, where a row of x is not all finite.  With an infinity, sum q x less z sum x is infinity less infinity, but the
// definition has s (q - z) x, of either sign.  So each thread looks at the results that it has stored, and adds what is
// not finite of a NaN's row up again, term by term, from x and the packed matrix; all that is finite does not count
// beside it.  G: groups of 128 elements.
// Out of line and after all products, so that they do not pay for it: called where a result is stored it cost
// 131072 x 4096, 4 tokens, 1.6%, this less than 1%.  One thread a result (with an infinity in every token that product
// takes 540 us, 4096 x 4096 with one token 30).
static __device__ __noinline__ void int4_non_finite(const GemvArgs& a, int G, bool bf16, bool zeros) {
  const unsigned inf = bf16 ? 0x7F80u : 0x7C00u;
  const auto value = [&](unsigned b) {
    return bf16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
  };
  constexpr int kSums = 4 * gv::kRg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = a.S == 1 ? 0 : (int)cluster_rank();
  const int rgroups = a.N / 16, granules = (rgroups + gv::kRg - 1) / gv::kRg, RG = gv::kWarps / a.KS;
  const int row0 = (int)blockIdx.x / a.S % a.tiles * a.tile_rows, rows = min(a.tile_rows, a.T - row0);
  const int block = 2048 + G * (zeros ? 96 : 64);
  int u0, u1;
  run_of<false>(a, a.tiles, granules, u0, u1);
  for (int u = u0; u < u1; u += RG)
    for (int j = rank + a.S * warp; j < kSums * min(RG, u1 - u); j += a.S * gv::kWarps) {
      const int s = j % kSums, rg = (u + j / kSums) * gv::kRg + (s >> 2), t = 2 * (lane & 3) + (s & 1);
      const int r = lane >> 2, hf = (s >> 1) & 1;  // row r or r + 8 of the 16-row group
      if (t >= rows || rg >= rgroups) continue;
      const long long o = (long long)(row0 + t) * a.ldo + 16 * rg + r + 8 * hf;
      float* const f = static_cast<float*>(a.out) + o;
      uint16_t* const h = static_cast<uint16_t*>(a.out) + o;
      const float y = a.out_f32 ? *f : value(*h);
      if (y == y) continue;
      const uint16_t* x = static_cast<const uint16_t*>(a.x) + (long long)(row0 + t) * a.ldx;
      const uint8_t* w = a.packed + (size_t)(rg >> 1) * (a.K / gv::kStep) * block;  // the row's blocks; layout: Step
      float sum = 0.f;
      bool any = false;  // else sums of finite values have overflowed, and y stays
      for (int k0 = 0; k0 < a.K && sum == sum; k0 += 64) {  // a chunk, whose loads overlap
        uint4 v[8];
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = reinterpret_cast<const uint4*>(x + k0)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          m = __vmaxu2(__vmaxu2(m, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu)),
                       __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
        if (max(m & 0xFFFFu, m >> 16) < inf) continue;
        any = true;
        const uint8_t* b = w + (size_t)(k0 / gv::kStep) * block;
        for (int k = k0; k < k0 + 64; ++k) {
          if ((x[k] & 0x7FFFu) < inf) continue;
          const uint32_t codes = *reinterpret_cast<const uint32_t*>(
              b + 1024 * (rg & 1) + 512 * ((k >> 6) & 1) + 16 * (4 * r + ((k >> 3) & 3)) + 4 * (2 * hf + ((k >> 5) & 1)));
          const int code = (int)(__funnelshift_r(codes, codes, 2) >> (4 * (((k & 7) >> 1) + 4 * (k & 1)))) & 15;
          const int at = (((rg & 1) * 8 + r) * G + k % gv::kStep * G / gv::kStep) * 2 + hf;
          const float scale = value(reinterpret_cast<const uint16_t*>(b + 2048)[at]);
          sum += scale * (float)(code - (zeros ? b[2048 + 64 * G + at] : 8)) * value(x[k]);
        }
      }
      if (!any) continue;
      if (a.out_f32) *f = sum;
      else *h = bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(sum)) : __half_as_ushort(__float2half_rn(sum));
    }
}

template <W4 kFmt, bool kBf16, bool kZeros, bool kCenter>
__global__ void __launch_bounds__(gv::kThreads, 1) gemv_kernel(const __grid_constant__ GemvArgs a) {
  using S = Step<kFmt, kZeros>;
  constexpr int kSums = 4 * gv::kRg;                // of a lane
  extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings, x rows, then (INT4) the cluster's and the group sums
  __shared__ unsigned amax[2][gv::kRows];           // of this tile and, zero, of the next
  __shared__ short tile_expert[S::kNv ? gv::kMaxTiles : 1];
  __shared__ int tile_row0[S::kNv ? gv::kMaxTiles : 1], wsum[8];
  __shared__ uint8_t tile_count[S::kNv ? gv::kMaxTiles : 1];  // its rows
  __shared__ uint64_t x_bar;  // x rows landed
  __shared__ int abort_flag, odd;  // odd: INT4, x is not all finite
  __shared__ float red[2][gv::kWarps][kSums][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int tiles = a.tiles;
  if (threadIdx.x < 2 * gv::kRows) amax[0][threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    abort_flag = odd = 0;
    mbar_init(&x_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (S::kNv) {
    // Tiles of at most tile_rows rows of one expert; thread i looks at expert i.  The offsets are read here alone, with
    // ordinary loads: the kernel before may write them while this one has begun, so that a read-only load could return
    // an older line, and two reads that differ would put a tile's rows out of its range.
    grid_dependency_wait();
    grid_launch_dependents();
    const int i = threadIdx.x;
    const int o0 = i < a.E ? a.offsets[i] : 0, o1 = i < a.E ? a.offsets[i + 1] : 0;
    const bool bad = o0 < 0 || o1 < o0 || o1 > a.R;
    const int nt = (o1 - o0 + a.tile_rows - 1) / a.tile_rows;
    int before = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31 && warp < 8) wsum[warp] = before;
    if (__syncthreads_or(bad)) {  // offsets that do not ascend within 0..R: nothing is computed
      if (threadIdx.x == 0 && blockIdx.x == 0) report(a.st, kFlagBounds, 920);
      return;
    }
    tiles = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += wsum[w];
      tiles += wsum[w];
    }
    for (int k = 0; k < nt; ++k) {
      tile_expert[before - nt + k] = (short)i;
      tile_row0[before - nt + k] = o0 + k * a.tile_rows;
      tile_count[before - nt + k] = (uint8_t)min(a.tile_rows, o1 - o0 - k * a.tile_rows);
    }
    __syncthreads();
  }
  const int rank = S::kNv || a.S == 1 ? 0 : (int)cluster_rank();
  const int all_steps = a.K / gv::kStep, rgroups = a.N / 16;
  const int step0 = S::kNv ? 0 : rank * (all_steps / a.S) + min(rank, all_steps % a.S);  // this CTA's slice of K
  const int steps = S::kNv ? all_steps : all_steps / a.S + (rank < all_steps % a.S);
  const int granules = (rgroups + gv::kRg - 1) / gv::kRg;  // of a matrix
  const int RG = gv::kWarps / a.KS;                        // granules at a time
  const int ks = warp % a.KS, wg = warp / a.KS;
  int tile = 0, left = 0x7FFFFFFF;  // the tile at the run's next granule, and how many it has from there on
  int u0, u1;
  run_of<S::kNv>(a, tiles, granules, u0, u1);
  if (u0 >= u1) return;
  if (S::kNv) {
    tile = u0 / granules;
    left = granules - (u0 - tile * granules);
  } else {
    tile = (int)blockIdx.x / a.S % tiles;
  }
  if (!S::kNv && a.S > 1) cluster_arrive();  // the first batch waits for it: every CTA has begun
  uint8_t* xs = smem + gv::kWarps * gv::kDepth * S::kSlot;
  float* shared = reinterpret_cast<float*>(xs + (size_t)a.tile_rows * a.pitch);  // S > 1: [2][source][kShared / S]
  float* sums = shared + (!S::kNv && a.S > 1 ? 2 * gv::kShared / 4 : 0);
  Stage<kFmt, kBf16, kCenter> stage(a, xs, step0, steps);
  int row0, rows;
  const auto tile_rows = [&] {  // the rows of `tile`
    row0 = S::kNv ? tile_row0[tile] : tile * a.tile_rows;
    rows = S::kNv ? tile_count[tile] : min(a.tile_rows, a.T - row0);
  };
  tile_rows();
  stage.rows = rows;
  if (S::kNv && threadIdx.x == 0) stage.start(a, row0, &x_bar);

  // ---- the copy side: the warp's next step to copy is number lk of its my_steps in the granule it is at; lnext is
  // where the next batch of granules starts, lleft how many granules the tile has from there on ----
  const int my_steps = (steps - ks + a.KS - 1) / a.KS;
  uint8_t* ring = smem + warp * (gv::kDepth * S::kSlot);
  const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
  int lnext = u0, lk = 0, lslot = 0, lleft = left, ltile = tile;
  const uint8_t *pc = nullptr, *ps = nullptr;
  const int row_block = a.K / kChunk * kTileBytes;
  const int dstep = a.KS * S::kStride;
  const auto next_granule = [&] {  // point the copies at the warp's next granule; false: it has no more
    while (my_steps > 0 && lnext < u1) {
      if (lleft == 0) {
        ++ltile;
        lleft = granules;
      }
      const int n = min(RG, min(lleft, u1 - lnext));
      const int g = (S::kNv ? granules - lleft : lnext) + wg;
      lnext += n;
      lleft -= n;
      if (wg < n) {  // the last batch of a tile or of the run may leave warps idle
        if (S::kNv) {
          const uint8_t* p = a.blob + (size_t)tile_expert[ltile] * a.expert_stride + (size_t)ks * S::kStride +
                             (size_t)(g >> 2) * row_block;
          pc = p + (g & 3) * 1024 + lane * 16;
          ps = p + kTileCodes + (g & 3) * 128 + (lane >> 3) * kTileBytes + (lane & 7) * 16;
        } else {
          pc = a.packed + ((size_t)g * all_steps + step0 + ks) * S::kStride + lane * 16;
        }
        return true;
      }
    }
    return false;
  };
  bool more = true;
  const uint64_t policy = weight_policy(a.once);
  const auto copy_next = [&] {  // one group, empty past the end
    if (more && lk == 0) more = next_granule();
    if (more) {
      S::copy(pc, ps, ring_addr + lslot * S::kSlot, lane, policy);
      lslot = lslot == gv::kDepth - 1 ? 0 : lslot + 1;
      pc += dstep;
      ps += dstep;
      if (++lk == my_steps) lk = 0;
    }
    copies_commit();
  };
#pragma unroll 1
  for (int d = 0; d < gv::kDepth; ++d) copy_next();

  // ---- the product side ----
  if (!S::kNv) {  // the weights, which no kernel writes, are on their way; x may still be in the making
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x == 0) stage.start(a, row0, &x_bar);
  }
  __syncthreads();  // the barrier is initialised
  float gs = 1.0f;
  const uint8_t* xl0 = nullptr;
  const float* sl0 = sums + ks * (S::kGroups * gv::kRows) + 2 * (lane & 3);
  int phase = 0, tphase = 0, slot = 0;
  bool fresh = true;  // x of `tile` is still to be converted
  bool dead = false;  // its copy did not land
  float2 up = make_float2(1.0f, 1.0f);  // the power of two of row 2 (lane & 3) + (warp & 1), the one whose sums the lane adds
  // y, the lane's sum s (row group, element of the accumulator) of a granule, into out
  const auto store = [&](int granule, int s, float y) {
    const int rg = granule * gv::kRg + (s >> 2), r = 2 * (lane & 3) + (s & 1);
    if (r < rows && rg < rgroups) {
      const long long o = (long long)(row0 + r) * a.ldo + 16 * rg + (lane >> 2) + 8 * ((s >> 1) & 1);
      if (a.out_f32) static_cast<float*>(a.out)[o] = y;
      else if (S::kNv || kBf16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
      else static_cast<__half*>(a.out)[o] = __float2half_rn(y);
    }
  };
  // S > 1: row j of a batch's sums is added and stored by CTA j % S, from what every CTA has put into its `shared`
  int pg0 = 0, pj = 0;  // the batch before: its first granule, its rows
  const int slog = 31 - __clz(a.S);  // a source has 32 / S rows of `shared`
  static_assert(gv::kShared == 32 * 128, "rows");
  const auto add_shared = [&] {
    const float* from = shared + (phase ^ 1) * (gv::kShared / 4) + lane;
    for (int j = rank + a.S * warp; j < pj; j += a.S * gv::kWarps) {
      float y = 0.f;
      for (int c = 0; c < a.S; ++c) y += from[((c << (5 - slog)) + (j >> slog)) * 32];
      if (y != y) odd = 1;  // by another CTA's slice; what this thread writes it reads itself
      if (!dead) store(pg0 + j / kSums, j % kSums, y);
    }
  };
  for (int u = u0; u < u1;) {
    if (left == 0) {  // the next tile: its rows of x
      ++tile;
      left = granules;
      tile_rows();
      __syncthreads();  // every warp is done with the last one's
      tphase ^= 1;
      stage.rows = rows;
      if (threadIdx.x == 0) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the reads of the last x, before the copies
        stage.start(a, row0, &x_bar);
      }
      fresh = true;
    }
    if (fresh) {
      if (!stage.finish(sums, amax[tphase], &odd, &x_bar, (uint32_t)tphase, &abort_flag, a.st)) {
        dead = true;
        if (S::kNv || a.S == 1) break;  // a cluster's others wait for this CTA's sums, which then count for nothing
      }
      if (threadIdx.x < gv::kRows) amax[tphase ^ 1][threadIdx.x] = 0u;
      if (S::kNv) gs = __ldg(a.gscale + tile_expert[tile]);
      up = pow2_pair(row_exponent(amax[tphase][2 * (lane & 3) + (warp & 1)]) + (S::kNv ? 0 : kCenter ? -2 : 22));
      // a lane whose token does not exist reads the last one's row: its column of the products is not stored
      xl0 = xs + min(lane >> 2, rows - 1) * a.pitch + (lane & 3) * (S::kNv ? 32 : 16) + ks * 256;
      __syncthreads();
      fresh = false;
    }
    const int n = min(RG, min(left, u1 - u));
    const int g0 = S::kNv ? granules - left : u;
    float acc[gv::kRg][4] = {};
    if (wg < n && !dead) {
      const uint8_t* xl = xl0;
      const float* sl = sl0;
#pragma unroll 1
      for (int k = 0; k < my_steps; ++k) {
        copies_wait();
        __syncwarp();  // the other lanes' copies too
        S w;
        w.read(ring + slot * S::kSlot, lane);
        slot = slot == gv::kDepth - 1 ? 0 : slot + 1;
        __syncwarp();  // read by all before it is filled again
        copy_next();
        use_step<kFmt, kBf16, kZeros, kCenter>(w, xl, sl, acc);
        xl += a.KS * 256;
        sl += a.KS * (S::kGroups * gv::kRows);
      }
    }
    // the batch's sums into out; the next batch's go to the other buffer: one barrier a batch
    const bool cluster = !S::kNv && a.S > 1;
    float(*part)[kSums][32] = red[phase];
#pragma unroll
    for (int s = 0; s < kSums; ++s) part[warp][s][lane] = acc[s >> 2][s & 3];
    if (cluster) {
      cluster_wait();  // the last batch's sums are there, and those of the one before are read
      add_shared();
    }
    __syncthreads();
    static_assert(gv::kWarps % kSums == 0, "a warp's rows j are all even or all odd");
    for (int j = warp; j < kSums * n; j += gv::kWarps) {
      const int g = j / kSums, s = j % kSums;
      float y = 0.f;
      for (int w = 0; w < a.KS; ++w) y += part[g * a.KS + w][s][lane];
      y = y * up.x * up.y;
      if (S::kNv) y *= gs;
      if (cluster)
        st_cluster(shared + phase * (gv::kShared / 4) + ((rank << (5 - slog)) + (j >> slog)) * 32 + lane, j & (a.S - 1), y);
      else store(g0 + g, s, y);
    }
    if (cluster) {
      cluster_arrive();
      pg0 = g0, pj = kSums * n;
    }
    phase ^= 1;
    u += n;
    left -= n;
  }
  if (!S::kNv && a.S > 1) {
    cluster_wait();
    add_shared();
  }
  if (!S::kNv && odd) int4_non_finite(a, S::kGroups, kBf16, kZeros);
  if (dead) {
    if (threadIdx.x == 0 && a.fault != 1) drain_copies(&x_bar, (uint32_t)tphase + 1, 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
}

// Warps along K: few, for few barriers, but as many as keep every warp busy with the CTA's share of granules.
static void set_steps(GemvArgs& a, int steps, long long granules_per_cta, int least = 1) {
  if (granules_per_cta < 1) granules_per_cta = 1;
  float best = 0.f;
  for (int ks = gv::kWarps; ks >= least; ks /= 2) {
    const int spw = (steps + ks - 1) / ks;
    float used = (float)steps / (float)(ks * spw);  // of the warps' steps
    const int rg = gv::kWarps / ks;
    if (granules_per_cta < rg) used *= (float)granules_per_cta / (float)rg;
    if (ks < 4) used *= 0.5f;
    if (used >= best - 0.01f) {
      best = used > best ? used : best;
      a.KS = ks;
    }
  }
}

// The kernel over as many clusters of a.S CTAs as there are granules (of all tiles), or as run at a time.
template <W4 kFmt, bool kBf16, bool kZeros, bool kCenter>
static cudaError_t launch_gemv(const GemvArgs& a, long long granules, size_t smem, int num_sms, cudaStream_t st) {
  static std::mutex mu;
  static int fit[64][gv::kMaxCluster + 1] = {};  // clusters that run at a time, by device and size; 0: not known yet
  const auto kernel = gemv_kernel<kFmt, kBf16, kZeros, kCenter>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(num_sms / a.S * a.S));
  cfg.blockDim = dim3(gv::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)a.S;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.S > 1 ? 2 : 1;
  int n = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64) n = fit[dev][a.S];
    if (n == 0) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, gv::smem_for(kFmt == W4::kNvfp4));
      if (e == cudaSuccess && a.S > 1) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (a.S == 1) n = num_sms;
      if (n < 1) n = 1;
      if (dev < 64) fit[dev][a.S] = n;
    }
  }
  if (n < a.tiles) n = a.tiles;  // one for each tile of x at least
  cfg.gridDim = dim3((unsigned)(granules < n ? granules : n) * a.S);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// NVFP4: two of the longest rows of x fit beside the rings (kMaxTiles).
static_assert(gv::kWarps * gv::kDepth * Step<W4::kNvfp4, false>::kSlot + 2 * (16384 * 2 + 16) <= gv::smem_for(true), "x");

static int nvfp4_pitch(int K) { return K * 2 + 16; }  // 16 bytes apart in the banks: 32-byte pieces of two rows never collide
static constexpr size_t kNvfp4Rings = (size_t)gv::kWarps * gv::kDepth * Step<W4::kNvfp4, false>::kSlot;
int grouped_gemv_tile_rows(int K) {
  const int fit = (int)((gv::smem_for(true) - kNvfp4Rings) / nvfp4_pitch(K));
  return fit < gv::kRows ? fit : gv::kRows;
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
  a.once = p.once;
  a.fault = p.fault;
  a.st = p.status;
  a.S = 1;
  const int granules = (p.N / 16 + gv::kRg - 1) / gv::kRg;
  const int touched = p.R < p.E ? p.R : p.E;
  set_steps(a, p.K / gv::kStep, (long long)touched * granules / p.num_sms);
  a.pitch = nvfp4_pitch(p.K);
  a.tile_rows = grouped_gemv_tile_rows(p.K);
  if (p.R < a.tile_rows) a.tile_rows = p.R;
  return launch_gemv<W4::kNvfp4, true, false, false>(a, (long long)(touched + p.R / a.tile_rows) * granules,
                                                     kNvfp4Rings + (size_t)a.tile_rows * a.pitch, p.num_sms, st);
}

// Shared memory of a CTA that takes `steps` steps of K for `rows` rows of x.
template <W4 kFmt, bool kZeros>
static constexpr size_t int4_smem(int rows, int steps, bool cluster) {
  return (size_t)gv::kWarps * gv::kDepth * Step<kFmt, kZeros>::kSlot + (size_t)rows * (steps * 256 + 64) +
         (size_t)steps * int4_groups(kFmt) * gv::kRows * 4 + (cluster ? 2 * gv::kShared : 0);
}
static_assert(int4_smem<W4::kInt4G32, true>(gv::kRows, 16384 / gv::kStep / gv::kMaxCluster, true) <= gv::smem_for(false), "x");

template <W4 kFmt, bool kBf16, bool kZeros, bool kCenter>
static cudaError_t launch_int4(GemvArgs& a, int num_sms, cudaStream_t st) {
  const int granules = (a.N / 16 + gv::kRg - 1) / gv::kRg, steps = a.K / gv::kStep;
  a.tiles = (a.T + gv::kRows - 1) / gv::kRows;
  a.tile_rows = (a.T + a.tiles - 1) / a.tiles;
  int per = steps;
  a.S = 1;
  while (int4_smem<kFmt, kZeros>(a.tile_rows, per, a.S > 1) > (size_t)gv::smem_for(false)) {  // at kMaxCluster it fits
    a.S *= 2;
    per = (steps + a.S - 1) / a.S;
  }
  a.pitch = per * 256 + 64;  // the lanes' 16-byte pieces of two rows never collide
  set_steps(a, steps / a.S, (long long)granules * a.tiles * a.S / num_sms, a.S > 1 ? 4 : 1);  // 4: a batch fits into kShared
  return launch_gemv<kFmt, kBf16, kZeros, kCenter>(a, (long long)granules * a.tiles,
                                                   int4_smem<kFmt, kZeros>(a.tile_rows, per, a.S > 1), num_sms, st);
}
template <W4 kFmt>
static cudaError_t launch_int4(GemvArgs& a, const Int4Product& p, cudaStream_t st) {
  if (p.act_f16 && p.out_f32)
    return p.zeros ? launch_int4<kFmt, false, true, true>(a, p.num_sms, st) : launch_int4<kFmt, false, false, true>(a, p.num_sms, st);
  if (p.act_f16)
    return p.zeros ? launch_int4<kFmt, false, true, false>(a, p.num_sms, st) : launch_int4<kFmt, false, false, false>(a, p.num_sms, st);
  return p.zeros ? launch_int4<kFmt, true, true, false>(a, p.num_sms, st) : launch_int4<kFmt, true, false, false>(a, p.num_sms, st);
}

cudaError_t launch_int4_gemv(const Int4Product& p, cudaStream_t st) {
  GemvArgs a{};
  a.st = p.status;
  a.packed = p.packed;
  a.T = p.T;
  a.N = p.N;
  a.K = p.K;
  a.x = p.x;
  a.ldx = p.ldx;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.once = p.once;
  a.fault = p.fault;
  return p.group == 32   ? launch_int4<W4::kInt4G32>(a, p, st)
         : p.group == 64 ? launch_int4<W4::kInt4G64>(a, p, st)
                         : launch_int4<W4::kInt4G128>(a, p, st);
}

// ---------------------------------------------------------------------------
// INT4 packer (the layout is described at Step).
// ---------------------------------------------------------------------------
size_t int4_packed_bytes(int N, int K, int group, bool zeros) {
  const size_t blocks = (size_t)((N + 31) / 32) * (K / 128);
  return blocks * (2048 + (128 / group) * (zeros ? 96 : 64));
}

__device__ __forceinline__ uint32_t int4_word(uint32_t w) {  // canonical nibble m = element m
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= (((w >> (8 * i)) & 0xFu) << (4 * i)) | (((w >> (8 * i + 4)) & 0xFu) << (16 + 4 * i));
  return __funnelshift_l(o, o, 2);
}

// One CTA a block of 32 rows x 128 elements; rows past the matrix hold zeros.
__global__ void pack_int4_kernel(const uint8_t* __restrict__ w_q, const uint16_t* __restrict__ scale,
                                 const uint8_t* __restrict__ zero, int f16, int N, int K, int group,
                                 uint8_t* __restrict__ packed, int* __restrict__ bad) {
  const int G = 128 / group, steps = K / 128;
  const int step = blockIdx.x % steps, granule = blockIdx.x / steps;
  uint8_t* dst = packed + (size_t)blockIdx.x * (2048 + G * (zero ? 96 : 64));
  const int tid = threadIdx.x;  // 128 threads: segment [group q][chunk h][lane]
  {
    const int q = tid >> 6, h = (tid >> 5) & 1, lane = tid & 31;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 32 * granule + 16 * q + (lane >> 2) + 8 * (i >> 1);
      const int k = 128 * step + 64 * h + 32 * (i & 1) + 8 * (lane & 3);
      o[i] = n < N ? int4_word(*reinterpret_cast<const uint32_t*>(w_q + (size_t)n * (K / 2) + k / 2)) : 0u;
    }
    *reinterpret_cast<uint4*>(dst + tid * 16) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  const uint16_t inf = f16 ? 0x7C00u : 0x7F80u;
  for (int i = tid; i < 32 * G; i += 128) {  // [q][r][group][half]
    const int hf = i & 1, gi = (i >> 1) % G, r = (i >> 1) / G % 8, q = i / (16 * G);
    const int n = 32 * granule + 16 * q + 8 * hf + r;
    const size_t src = (size_t)n * (K / group) + step * G + gi;
    const uint16_t s = n < N ? scale[src] : 0;
    reinterpret_cast<uint16_t*>(dst + 2048)[i] = s;
    bool b = (s & inf) == inf;
    if (zero) {
      const uint8_t z = n < N ? zero[src] : 0;
      dst[2048 + 64 * G + i] = z;
      b |= z > 15;
    }
    if (b) atomicAdd(bad, 1);
  }
}

cudaError_t launch_pack_int4(const uint8_t* w_q, const void* scale, const uint8_t* zero, int act_f16, int N, int K,
                             int group, uint8_t* packed, int* bad, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(bad, 0, sizeof(int), st);
  if (e != cudaSuccess) return e;
  pack_int4_kernel<<<(unsigned)((N + 31) / 32 * (K / 128)), 128, 0, st>>>(w_q, static_cast<const uint16_t*>(scale), zero,
                                                                          act_f16, N, K, group, packed, bad);
  return cudaGetLastError();
}

}  // namespace nvfp4moe
