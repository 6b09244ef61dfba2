// Root-mean-square norm with the residual's addition (nvfp4_norm_forward / nvfp4_norm_backward), and the 8-bit codes of
// plain rows (nvfp4_int8_quantize).
//   forward : h = x + r rounded to 16 bits; y = w h rstd, rstd = 1 / sqrt(mean(h^2) + eps);
//             code = round(127 w h / max |w h|), its scale max |y| / 127
//   backward: dx = rstd (w dy) - h rstd^3 / H sum(w dy h) + dsum;  dw = sum over the rows of dy h rstd
// The codes do not depend on rstd: they are the rounded quotients of w h and its largest magnitude, both exact products
// of 16-bit numbers, so that the rounding of sums cannot turn a code over.
//
// Bound by memory (16384 x 4096 with the residual, in 16 and 8 bits: 604 MB, 93 us, 0.97 of the copy rate; its gradient,
// 8191 rows, 268 MB, 45 us, 0.89; two rows alone 2.5 us).  A row stays in the registers of the threads that share it (`TP`
// threads of `V` pieces of 8 elements): one read, one reduction, one write.  Rows up to 1024 elements take
// 8 to 32 lanes of a warp and no barrier, longer ones a CTA, whose next row is on its way while this one is reduced.
//
// Sums are FP32; where squares or products leave its range (the mean below 2^-80 or the sum above 2^120, the peak beyond
// 2^+-100) the row's statistics are formed again in 64 bits.  A row whose products are all below 2^-149 counts as zeros.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "kernels.h"
#include "quant8.cuh"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace nm {
constexpr int kSmallThreads = 128;  // of a CTA whose rows fit a warp
}

struct NormArgs {
  const uint8_t *x, *res, *weight;  // 16-bit; res, weight may be NULL (weight: quantisation alone)
  uint8_t *sum, *y;                 // 16-bit, may be NULL
  int8_t* q;                        // may be NULL
  float *q_scale, *rstd;            // rstd may be NULL
  long long ldx, ldr, lds, ldy, ldq;  // bytes
  int T, H;
  float eps;
};

// The sum and the maximum over the TP threads of a row; all get both.  red: 2 x 32 floats, by turns.
template <int TP, class F>
__device__ __forceinline__ void row_reduce(F& sum, F& top, F* red) {
#pragma unroll
  for (int o = 1; o < (TP < 32 ? TP : 32); o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const F t = __shfl_xor_sync(0xffffffffu, top, o);
    top = t > top ? t : top;
  }
  if constexpr (TP > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = sum, red[32 + warp] = top;
    __syncthreads();
    sum = lane < TP / 32 ? red[lane] : F(0);
    top = lane < TP / 32 ? red[32 + lane] : F(0);
#pragma unroll
    for (int o = 1; o < TP / 32; o <<= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const F t = __shfl_xor_sync(0xffffffffu, top, o);
      top = t > top ? t : top;
    }
    sum = __shfl_sync(0xffffffffu, sum, 0);
    top = __shfl_sync(0xffffffffu, top, 0);
  }
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

template <bool kF16, int TP, int V>
// (rows of 4104 to 8192: 6 registers over two CTAs a multiprocessor without the bound)
__global__ void __launch_bounds__(TP <= 32 ? nm::kSmallThreads : TP, TP == 256 ? 2 : 0)
    norm_forward_kernel(NormArgs a) {
  constexpr int kRows = TP <= 32 ? nm::kSmallThreads / TP : 1;  // rows of a CTA at a time
  __shared__ float red[2][64];
  __shared__ double red64[64];
  const int lane = threadIdx.x % TP, pieces = a.H / 8;
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 w4[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = lane + v * TP;
    w4[v] = a.weight && p < pieces ? load16(a.weight + 16ll * p) : make_uint4(0u, 0u, 0u, 0u);
  }
  long long t = (long long)blockIdx.x * kRows + threadIdx.x / TP;
  const long long step = (long long)gridDim.x * kRows;
  uint4 x4[V], r4[V];
  const auto fetch = [&](long long row) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * TP;
      x4[v] = r4[v] = make_uint4(0u, 0u, 0u, 0u);
      if (row < a.T && p < pieces) {
        x4[v] = load16(a.x + row * a.ldx + 16ll * p);
        if (a.res) r4[v] = load16(a.res + row * a.ldr + 16ll * p);
      }
    }
  };
  fetch(t);
  // warps stay together, for the shuffles: their rows are neighbours, and the first is the last to run out
  for (int turn = 0; t - threadIdx.x / TP % (TP < 32 ? 32 / TP : 1) < a.T; t += step, turn ^= 1) {
    const bool row_ok = t < a.T;
    uint4 h4[V];
    float ss = 0.f;
    unsigned peak_bits = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[8], w[8];
      unpack8<kF16>(x4[v], h);
      if (a.res) {
        float r[8];
        unpack8<kF16>(r4[v], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
        h4[v] = pack8<kF16>(h);
        unpack8<kF16>(h4[v], h);
      } else {
        h4[v] = x4[v];
      }
      unpack8<kF16>(w4[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[i], h[i], ss);
        peak_bits = max(peak_bits, magnitude(a.weight ? h[i] * w[i] : h[i]));
      }
    }
    fetch(t + step);
#pragma unroll
    for (int o = 1; o < (TP < 32 ? TP : 32); o <<= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      peak_bits = max(peak_bits, __shfl_xor_sync(0xffffffffu, peak_bits, o));
    }
    if constexpr (TP > 32) {
      const int warp = threadIdx.x >> 5, l = threadIdx.x & 31;
      float* s = red[turn];
      if (l == 0) s[warp] = ss, s[32 + warp] = __uint_as_float(peak_bits);
      __syncthreads();
      ss = l < TP / 32 ? s[l] : 0.f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      peak_bits = __reduce_max_sync(0xffffffffu, l < TP / 32 ? __float_as_uint(s[32 + l]) : 0u);
    }
    const float peak = __uint_as_float(peak_bits), mean = ss / (float)a.H + a.eps;
    float rstd = 1.0f / sqrtf(mean), scale = a.weight ? peak * rstd / 127.0f : peak / 127.0f;
    double peak64 = 0.0;
    float up = 1.0f;  // rstd's second factor, where it is beyond FP32: without eps, of rows below the normal numbers
    bool finite = true;
    // out of FP32's range: its mean, or what its codes are made of (a peak of zero is that of a row of zeros).  Each alone
    // decides what is taken from the 64-bit sums, so that a row is the same whatever its neighbours and outputs are
    const bool far = a.weight && !(mean >= 0x1p-80f && ss <= 0x1p120f), odd = far || (a.q && peak_bits && !plain_peak(peak));
    if (TP < 32 ? __any_sync(0xffffffffu, odd) : odd) {  // a warp's rows go together
      double s64 = 0.0, p64 = 0.0;
      bool bad = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float h[8], w[8];
        unpack8<kF16>(h4[v], h);
        unpack8<kF16>(w4[v], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double p = a.weight ? (double)h[i] * (double)w[i] : (double)h[i];
          s64 += (double)h[i] * (double)h[i];
          bad |= !(fabs(p) <= 1.7e308);
          p64 = fmax(p64, fabs(p));
        }
      }
      if (bad) p64 = INFINITY;
      if (TP > 32) __syncthreads();  // red64 of the row before
      row_reduce<TP>(s64, p64, red64);
      const double mean64 = s64 / a.H + (double)a.eps, r64 = mean64 == 0.0 ? 0.0 : 1.0 / sqrt(mean64);
      if (far) {
        rstd = mean64 == 0.0 ? INFINITY : (float)r64;
        if (rstd == INFINITY) up = (float)(r64 * 0x1p-64);  // 0 for a row of zeros, which stays so
      }
      if (odd) {
        peak64 = p64;
        scale = (float)(a.weight ? p64 * r64 / 127.0 : p64 / 127.0);
        finite = p64 <= 1.7e308;
      }
    }
    if (row_ok) {
      if (lane == 0) {
        if (a.rstd) a.rstd[t] = rstd;
        if (a.q) a.q_scale[t] = finite ? scale : __uint_as_float(0x7FC00000u);
      }
      if (rstd == INFINITY) rstd = 0x1p64f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = lane + v * TP;
        if (p >= pieces) continue;
        float h[8], w[8];
        unpack8<kF16>(h4[v], h);
        unpack8<kF16>(w4[v], w);
        if (a.sum) *reinterpret_cast<uint4*>(a.sum + t * a.lds + 16ll * p) = h4[v];
        if (a.y) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * up * w[i];
          *reinterpret_cast<uint4*>(a.y + t * a.ldy + 16ll * p) = pack8<kF16>(y);
        }
        if (a.q) {
          uint32_t c[2] = {0u, 0u};
          float pr[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) pr[i] = a.weight ? h[i] * w[i] : h[i];
          if (!odd) {
            if (peak_bits) {
              if (!a.weight) codes_of_elements(pr, peak, c);
              else if (kF16) codes_of_products<22>(pr, peak, c);
              else codes_of_products<16>(pr, peak, c);
            }
          } else if (finite && peak64 > 0.0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              c[i >> 2] |= ((uint32_t)code_of_64(a.weight ? (double)h[i] * (double)w[i] : (double)h[i], peak64) & 255u)
                           << (8 * (i & 3));
          }
          *reinterpret_cast<uint2*>(a.q + t * a.ldq + 8ll * p) = make_uint2(c[0], c[1]);
        }
      }
    }
  }
}

struct NormBackArgs {
  const uint8_t *dy, *x, *weight, *dsum;  // dsum may be NULL
  const float* rstd;
  uint8_t* dx;
  float* part;  // [parts][H] this call's partial sums of dw, or NULL
  long long ld_dy, ldx, ld_dsum, ld_dx;  // bytes
  int T, H;
};

template <bool kF16, int TP, int V>
__global__ void __launch_bounds__(nm::kSmallThreads) norm_backward_kernel(NormBackArgs a) {
  constexpr int kRows = nm::kSmallThreads / TP;
  __shared__ float fold[kRows][8 * TP * V];
  const int lane = threadIdx.x % TP, pieces = a.H / 8;
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 w4[V];
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = lane + v * TP;
    w4[v] = p < pieces ? load16(a.weight + 16ll * p) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  long long t = (long long)blockIdx.x * kRows + threadIdx.x / TP;
  const long long step = (long long)gridDim.x * kRows;
  const float inv_h = 1.0f / (float)a.H;
  const auto fetch = [&](long long row, uint4 (&x)[V], uint4 (&d)[V], uint4 (&s)[V], float& r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = lane + v * TP;
      x[v] = d[v] = s[v] = make_uint4(0u, 0u, 0u, 0u);
      if (row < a.T && p < pieces) {
        x[v] = load16(a.x + row * a.ldx + 16ll * p);
        d[v] = load16(a.dy + row * a.ld_dy + 16ll * p);
        if (a.dsum) s[v] = load16(a.dsum + row * a.ld_dsum + 16ll * p);
      }
    }
    r = row < a.T ? a.rstd[row] : 0.f;
  };
  constexpr bool kAhead = V == 1;  // the next row is on its way while this one is reduced, where there are registers for it
  uint4 x_n[V], d_n[V], s_n[V];
  float rstd_n = 0.f;
  if (kAhead) fetch(t, x_n, d_n, s_n, rstd_n);
  for (; t - threadIdx.x / TP % (TP < 32 ? 32 / TP : 1) < a.T; t += step) {
    const bool row_ok = t < a.T;
    uint4 x4[V], d4[V], s4[V];
    float rstd = rstd_n;
    if constexpr (kAhead) {
#pragma unroll
      for (int v = 0; v < V; ++v) x4[v] = x_n[v], d4[v] = d_n[v], s4[v] = s_n[v];
      fetch(t + step, x_n, d_n, s_n, rstd_n);
    } else {
      fetch(t, x4, d4, s4, rstd);
    }
    float c = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float x[8], d[8], w[8];
      unpack8<kF16>(x4[v], x);
      unpack8<kF16>(d4[v], d);
      unpack8<kF16>(w4[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = x[i] * rstd;
        c = fmaf(d[i] * w[i], n, c);
        dw[v][i] = fmaf(d[i], n, dw[v][i]);
      }
    }
#pragma unroll
    for (int o = 1; o < TP; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    c *= inv_h;
    if (row_ok) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int p = lane + v * TP;
        if (p >= pieces) continue;
        float x[8], d[8], w[8], s[8], o[8];
        unpack8<kF16>(x4[v], x);
        unpack8<kF16>(d4[v], d);
        unpack8<kF16>(w4[v], w);
        unpack8<kF16>(s4[v], s);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(rstd, fmaf(-c, x[i] * rstd, d[i] * w[i]), s[i]);
        *reinterpret_cast<uint4*>(a.dx + t * a.ld_dx + 16ll * p) = pack8<kF16>(o);
      }
    }
  }
  // The CTA's rows together, so that the few CTAs that add up the parts have few to read (64000 x 64: 23 us with a part a row,
  // 8 so).
  if (a.part) {
    float* to = fold[threadIdx.x / TP];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) to[8 * (lane + v * TP) + i] = dw[v][i];
    __syncthreads();
    for (int h = threadIdx.x; h < a.H; h += nm::kSmallThreads) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) sum += fold[i][h];
      a.part[(long long)blockIdx.x * a.H + h] = sum;
    }
  }
}

// The same for rows longer than a warp holds.  A warp of its own brings the rows by bulk copies to a ring in shared memory,
// as far ahead as that holds; the others read a row there twice, before and after its sum is known, so that few registers
// are taken and two or three CTAs a multiprocessor hide one another's barriers.  (8191 rows of 4096: 58 us with the rows in
// registers, 25 KB a multiprocessor on their way; 55 with one CTA a multiprocessor and the rows copied from the ring to
// registers; 45 as it is.  2047 rows of 16384, as many bytes, take 65: two such rows fill the ring.)
namespace nm {
constexpr int kRingBytes = 216 * 1024, kMaxSlots = 8;  // of a multiprocessor
}
template <bool kF16, int TP, int V, int kPerSm>
__global__ void __launch_bounds__(TP + 32, kPerSm) norm_backward_ring_kernel(NormBackArgs a, int slots, DeviceStatus* st) {
  extern __shared__ __align__(16) uint8_t ring[];  // [slot][x, dy, dsum][H]
  __shared__ uint64_t full[nm::kMaxSlots], empty[nm::kMaxSlots];
  __shared__ float red[2][TP / 32];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pieces = a.H / 8;
  const uint32_t bytes = 2u * a.H;
  if (tid == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, TP / 32);
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  RingPos pos;
  if (warp == TP / 32) {
    if (lane == 0) {
      uint32_t issued = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < a.T && ok; t += gridDim.x, pos.step(slots)) {
        ok = mbar_wait(empty + pos.slot, pos.phase ^ 1u, &abort_flag, st, 942);
        if (!ok) break;
        uint8_t* to = ring + (size_t)pos.slot * 3 * bytes;
        mbar_arrive_expect_tx(full + pos.slot, bytes * (a.dsum ? 3 : 2));
        bulk_g2s(to, a.x + t * a.ldx, bytes, full + pos.slot);
        bulk_g2s(to + bytes, a.dy + t * a.ld_dy, bytes, full + pos.slot);
        if (a.dsum) bulk_g2s(to + 2 * bytes, a.dsum + t * a.ld_dsum, bytes, full + pos.slot);
        ++issued;
      }
      drain_copies(full, issued, slots);
    }
    return;
  }
  uint4 w4[V];
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = tid + v * TP;
    w4[v] = p < pieces ? load16(a.weight + 16ll * p) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.f;
  }
  const float inv_h = 1.0f / (float)a.H;
  int k = 0;
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x, k ^= 1, pos.step(slots)) {
    const float rstd = a.rstd[t];
    const bool landed = mbar_wait(full + pos.slot, pos.phase, &abort_flag, st, 941);
    const uint8_t* slot = ring + (size_t)pos.slot * 3 * bytes;
    float c = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * TP;
      if (p >= pieces) continue;
      float x[8], d[8], w[8];
      unpack8<kF16>(load16(slot + 16 * p), x);
      unpack8<kF16>(load16(slot + bytes + 16 * p), d);
      unpack8<kF16>(w4[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = x[i] * rstd;
        c = fmaf(d[i] * w[i], n, c);
        dw[v][i] = fmaf(d[i], n, dw[v][i]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (lane == 0) red[k][warp] = c;
    uint32_t lost;  // one answer for all of them
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(lost)
                 : "r"(landed ? 0u : 1u), "n"(TP)
                 : "memory");
    if (lost) return;
    c = lane < TP / 32 ? red[k][lane] : 0.f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    c *= inv_h;
    uint4 out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * TP;
      if (p >= pieces) continue;
      float x[8], d[8], w[8], s[8], o[8];
      unpack8<kF16>(load16(slot + 16 * p), x);
      unpack8<kF16>(load16(slot + bytes + 16 * p), d);
      unpack8<kF16>(a.dsum ? load16(slot + 2 * bytes + 16 * p) : make_uint4(0u, 0u, 0u, 0u), s);
      unpack8<kF16>(w4[v], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(rstd, fmaf(-c, x[i] * rstd, d[i] * w[i]), s[i]);
      out[v] = pack8<kF16>(o);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + pos.slot);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * TP;
      if (p < pieces) *reinterpret_cast<uint4*>(a.dx + t * a.ld_dx + 16ll * p) = out[v];
    }
  }
  if (a.part) {
    float* to = a.part + (long long)blockIdx.x * a.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int p = tid + v * TP;
      if (p >= pieces) continue;
      *reinterpret_cast<float4*>(to + 8 * p) = make_float4(dw[v][0], dw[v][1], dw[v][2], dw[v][3]);
      *reinterpret_cast<float4*>(to + 8 * p + 4) = make_float4(dw[v][4], dw[v][5], dw[v][6], dw[v][7]);
    }
  }
}

// dw[h] = sum of part[i][h], in a fixed order: 32 columns a CTA, 32 runs of rows each.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* part, int parts, int H, float* dw) {
  __shared__ float s[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  float sum = 0.f;
  if (col < H) {
#pragma unroll 10
    for (int i = run; i < parts; i += 32) sum += part[(long long)i * H + col];
  }
  s[run][threadIdx.x & 31] = sum;
  __syncthreads();
  if (run == 0 && col < H) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][threadIdx.x];
    dw[col] = sum;
  }
}

static cudaLaunchConfig_t dependent(dim3 grid, dim3 block, cudaStream_t st, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = block, cfg.stream = st;
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cfg;
}

// Threads a row and pieces a thread for rows of `pieces` 8-element pieces.
struct NormShape {
  int tp, v;
};
static NormShape norm_shape(int pieces, int T, int num_sms) {
  if (pieces <= 8) return {8, 1};
  if (pieces <= 16) return {16, 1};
  // few rows: one piece a thread, for the shortest way through a row
  if (T <= 2 * num_sms) {
    if (pieces <= 32) return {32, 1};
    if (pieces <= 128) return {128, 1};
    if (pieces <= 512) return {512, 1};
    return {1024, 2};
  }
  if (pieces <= 32) return {32, 1};
  if (pieces <= 64) return {32, 2};
  if (pieces <= 128) return {32, 4};
  if (pieces <= 512) return {128, 4};
  if (pieces <= 1024) return {256, 4};
  return {512, 4};
}

template <bool kF16, int TP, int V>
static cudaError_t run_forward(const NormArgs& a, int num_sms, cudaStream_t st) {
  constexpr int threads = TP <= 32 ? nm::kSmallThreads : TP, rows = threads / (TP <= 32 ? TP : threads);
  // As many CTAs as run at a time: the last ones of 8 a multiprocessor, of which registers let 3 run, found the machine half
  // empty (16384 x 4096 97 us, 93 so; 1000 rows 9.8, 8.2).  Long calls whose threads hold four pieces do better with
  // twice as many (65536 x 1024 101 us once, 95 twice; 4096 x 16384 102, 97; the
  // 16384 rows of 4096 alike; but 8000 rows of 4096 48.2, 49.5, and 262144 of 128, one piece a thread, 55.4, 56.5).
  static std::atomic<int> resident{0};  // of a multiprocessor; all devices that run this code are alike
  int per_sm = resident.load(std::memory_order_relaxed);
  if (!per_sm) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_forward_kernel<kF16, TP, V>, threads, 0);
    if (e != cudaSuccess) return e;
    per_sm = std::max(per_sm, 1);
    resident.store(per_sm, std::memory_order_relaxed);
  }
  cudaLaunchAttribute at;
  const int turns = (a.T + rows - 1) / rows, wave = num_sms * per_sm;
  const int grid = std::min(turns, V >= 4 && turns >= 24 * wave ? 2 * wave : wave);
  const cudaLaunchConfig_t cfg = dependent(dim3(grid), dim3(threads), st, &at);
  return cudaLaunchKernelEx(&cfg, norm_forward_kernel<kF16, TP, V>, a);
}
template <bool kF16>
static cudaError_t forward_of(const NormArgs& a, int num_sms, cudaStream_t st) {
  const NormShape s = norm_shape(a.H / 8, a.T, num_sms);
  switch (s.tp * 8 + s.v) {
    case 8 * 8 + 1: return run_forward<kF16, 8, 1>(a, num_sms, st);
    case 16 * 8 + 1: return run_forward<kF16, 16, 1>(a, num_sms, st);
    case 32 * 8 + 1: return run_forward<kF16, 32, 1>(a, num_sms, st);
    case 32 * 8 + 2: return run_forward<kF16, 32, 2>(a, num_sms, st);
    case 32 * 8 + 4: return run_forward<kF16, 32, 4>(a, num_sms, st);
    case 128 * 8 + 1: return run_forward<kF16, 128, 1>(a, num_sms, st);
    case 128 * 8 + 4: return run_forward<kF16, 128, 4>(a, num_sms, st);
    case 256 * 8 + 4: return run_forward<kF16, 256, 4>(a, num_sms, st);
    case 512 * 8 + 1: return run_forward<kF16, 512, 1>(a, num_sms, st);
    case 512 * 8 + 4: return run_forward<kF16, 512, 4>(a, num_sms, st);
    default: return run_forward<kF16, 1024, 2>(a, num_sms, st);
  }
}

cudaError_t launch_norm_forward(const NormOp& p, cudaStream_t st) {
  NormArgs a{};
  a.x = static_cast<const uint8_t*>(p.x), a.ldx = 2 * p.ldx;
  a.res = static_cast<const uint8_t*>(p.res), a.ldr = 2 * p.ldr;
  a.weight = static_cast<const uint8_t*>(p.weight);
  a.sum = static_cast<uint8_t*>(p.sum), a.lds = 2 * p.lds;
  a.y = static_cast<uint8_t*>(p.y), a.ldy = 2 * p.ldy;
  a.q = p.q, a.ldq = p.ldq, a.q_scale = p.q_scale, a.rstd = p.rstd;
  a.T = p.T, a.H = p.H, a.eps = p.eps;
  return p.f16 ? forward_of<true>(a, p.num_sms, st) : forward_of<false>(a, p.num_sms, st);
}

// The backward: rows within a warp as in the forward, longer ones through the ring.
struct NormBackShape {
  int tp, v, rows;  // threads a row, pieces a thread, rows of a CTA at a time
  int per_sm;       // CTAs a multiprocessor
};
// As many CTAs as run at a time, by registers or by the ring (131072 x 256: 56 us with 4, 49 with 6).  Rows of 4104 to 6144
// by 256 threads, two CTAs (6552 x 5120 46 us; one CTA of 512 threads 58; 666 rows of 6144 12.2, 10.9); longer ones that way
// would hold four pieces a thread (4095 x 8192 66 us, 50 as it is).
static NormBackShape norm_back_shape(int pieces) {
  if (pieces <= 8) return {8, 1, 16, 5};
  if (pieces <= 16) return {16, 1, 8, 5};
  if (pieces <= 32) return {32, 1, 4, 6};
  if (pieces <= 64) return {32, 2, 4, 5};
  if (pieces <= 128) return {128, 1, 1, 6};
  if (pieces <= 256) return {256, 1, 1, 3};
  if (pieces <= 512) return {256, 2, 1, 3};
  if (pieces <= 768) return {256, 3, 1, 2};
  if (pieces <= 1024) return {512, 2, 1, 1};
  return {512, 4, 1, 1};
}
int norm_backward_parts(int H, int num_sms) { return num_sms * norm_back_shape(H / 8).per_sm; }  // one a CTA

template <bool kF16, int TP, int V>
static cudaError_t run_backward(const NormBackArgs& a, int grid, cudaStream_t st) {
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent(dim3(grid), dim3(nm::kSmallThreads), st, &at);
  return cudaLaunchKernelEx(&cfg, norm_backward_kernel<kF16, TP, V>, a);
}
template <bool kF16, int TP, int V, int kPerSm>
static cudaError_t run_ring(const NormBackArgs& a, int grid, DeviceStatus* status, cudaStream_t st) {
  constexpr int kCached = 64, kRoom = (nm::kRingBytes / kPerSm - 1024 * (kPerSm - 1)) & ~1023;
  static std::mutex mu;
  static bool done[kCached] = {};  // the opt-in shared-memory size, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(dev >= 0 && dev < kCached && done[dev])) {
      e = cudaFuncSetAttribute((const void*)norm_backward_ring_kernel<kF16, TP, V, kPerSm>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kRoom);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < kCached) done[dev] = true;
    }
  }
  const int slots = std::min(nm::kMaxSlots, kRoom / (6 * a.H));
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = dependent(dim3(grid), dim3(TP + 32), st, &at);
  cfg.dynamicSmemBytes = (size_t)slots * 6 * a.H;
  return cudaLaunchKernelEx(&cfg, norm_backward_ring_kernel<kF16, TP, V, kPerSm>, a, slots, status);
}
template <bool kF16>
static cudaError_t backward_of(const NormBackArgs& a, const NormBackShape& s, int grid, DeviceStatus* status, cudaStream_t st) {
  switch (s.tp * 8 + s.v) {
    case 8 * 8 + 1: return run_backward<kF16, 8, 1>(a, grid, st);
    case 16 * 8 + 1: return run_backward<kF16, 16, 1>(a, grid, st);
    case 32 * 8 + 1: return run_backward<kF16, 32, 1>(a, grid, st);
    case 32 * 8 + 2: return run_backward<kF16, 32, 2>(a, grid, st);
    case 128 * 8 + 1: return run_ring<kF16, 128, 1, 6>(a, grid, status, st);
    case 256 * 8 + 1: return run_ring<kF16, 256, 1, 3>(a, grid, status, st);
    case 256 * 8 + 2: return run_ring<kF16, 256, 2, 3>(a, grid, status, st);
    case 256 * 8 + 3: return run_ring<kF16, 256, 3, 2>(a, grid, status, st);
    case 512 * 8 + 2: return run_ring<kF16, 512, 2, 1>(a, grid, status, st);
    default: return run_ring<kF16, 512, 4, 1>(a, grid, status, st);
  }
}

cudaError_t launch_norm_backward(const NormBackOp& p, cudaStream_t st) {
  NormBackArgs a{};
  a.dy = static_cast<const uint8_t*>(p.dy), a.ld_dy = 2 * p.ld_dy;
  a.x = static_cast<const uint8_t*>(p.x), a.ldx = 2 * p.ldx;
  a.weight = static_cast<const uint8_t*>(p.weight);
  a.dsum = static_cast<const uint8_t*>(p.dsum), a.ld_dsum = 2 * p.ld_dsum;
  a.rstd = p.rstd;
  a.dx = static_cast<uint8_t*>(p.dx), a.ld_dx = 2 * p.ld_dx;
  a.part = p.dweight ? p.part : nullptr;
  a.T = p.T, a.H = p.H;
  const NormBackShape s = norm_back_shape(p.H / 8);
  const int grid = std::min((p.T + s.rows - 1) / s.rows, p.num_sms * s.per_sm);
  cudaError_t e = p.f16 ? backward_of<true>(a, s, grid, p.status, st) : backward_of<false>(a, s, grid, p.status, st);
  if (e != cudaSuccess || !p.dweight) return e;
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg = dependent(dim3((p.H + 31) / 32), dim3(1024), st, &at);
  return cudaLaunchKernelEx(&cfg, norm_dweight_kernel, (const float*)p.part, grid, p.H, p.dweight);
}

}  // namespace nvfp4moe
