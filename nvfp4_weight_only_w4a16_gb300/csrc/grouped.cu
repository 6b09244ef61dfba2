// Products of NVFP4 experts over ragged row groups (nvfp4_grouped_forward /
// nvfp4_grouped_backward): a persistent tcgen05 GEMM over
//   forward : y[r][n]  = gs_e sum_k W_e[n][k] x[r][k]
//   backward: dx[r][k] = gs_e sum_n W_e[n][k] dy[r][n]
// for the rows off[e] <= r < off[e+1] of every expert e.
//
// Both directions read the same packed bytes.  The weights are the M operand and
// the rows the N operand, so that an expert with few rows pays for few columns.
// The reduction runs over 128 x 128 weight squares: two neighbouring packed tiles
// (128 weight rows x 64 K each).  A square is dequantised to BF16 -- exact: an
// E2M1 x E4M3 product has at most 6 significant bits -- into shared memory as rows
// of 64 K elements (128 B, 128B swizzle).  That one image serves both products:
// read K-major it is the forward operand (M = weight row, reduction = K), read
// M-major it is its transpose (M = K element, reduction = weight row).  Only the
// descriptors, and which part of a square a 64-long half step takes, differ.
//
// kCtas = 2: a pair of CTAs on neighbouring multiprocessors works on 256 output
// features (128 each) of one tile of up to 256 rows, M = 256 MMAs: each CTA
// dequantises its own 128 x 128 squares and loads half of the rows, which both
// halves of the MMA read.  kCtas = 1, 128 features, where there is no second block
// to pair with.
//
// One CTA per multiprocessor, 24 warps: 0 packed-weight producer (bulk copies into
// a ring), 1 MMA issuer (the pair's first CTA), 2 row producer (TMA, zero fill past
// the matrix), 4-7 epilogue (TMEM -> gs -> shared -> 16-byte stores), 8-23
// dequantisers in two teams that take turns.  Two accumulator buffers of 256
// columns: the epilogue of a unit overlaps the next one's MMAs.  The row offsets
// are read on the device; every CTA derives the same unit list from them, so
// nothing is written but the output.
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace gg {
constexpr int kThreads = 768;
constexpr int kTeamWarps = 8, kDequantWarps = 2 * kTeamWarps, kEpiWarps = 4;
constexpr int kPairBytes = 2 * kTileBytes;  // one 128 x 128 weight square, packed
constexpr int kHalfBytes = 16384;           // half a square in BF16: 64 long in the reduction
constexpr int kMaxStages = 6, kMaxRaw = 16;
constexpr int kSmemMax = 232448;
constexpr int kCtlBytes = 4096;             // tables and barriers in front of the rings
constexpr int kEpiBytes = 2048;             // per epilogue warp
constexpr int kRingOff = kCtlBytes + kEpiWarps * kEpiBytes;
}  // namespace gg

struct GroupedArgs {
  const uint8_t* blob;
  size_t expert_stride;
  const float* gscale;     // [E]
  const int32_t* offsets;  // [E + 1]
  int E, R;
  int NB;                  // 128-feature output blocks
  int NU;                  // work units across the features: NB or, in pairs, half of it
  int steps;               // 128-long reduction steps
  size_t block_stride;     // bytes from one output block's first square to the next one's
  size_t step_stride;      // bytes from one reduction step's square to the next
  int n_out;               // output features
  void* out;
  long long ldo;
  int out_f32;
  int tile_rows;           // rows per token tile, a multiple of 64 up to 256
  int box;                 // rows per TMA box, divides tile_rows / kCtas
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

template <int kCtas>
__device__ __forceinline__ GroupedUnit grouped_unit(const GroupedCtl& c, const GroupedArgs& a, int u) {
  const int t = u / a.NU;
  int lo = 0, hi = a.E;  // the expert e with tile[e] <= t < tile[e + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.tile[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int m = c.off[lo + 1] - c.off[lo], nt = c.tile[lo + 1] - c.tile[lo], j = t - c.tile[lo];
  // an expert's tiles are of one size, so that none is a small remainder
  constexpr int kRound = 16 * kCtas - 1;
  const int per = ((m + nt - 1) / nt + kRound) & ~kRound;
  GroupedUnit r;
  r.e = lo;
  r.row0 = c.off[lo] + j * per;
  r.rows = min(per, m - j * per);
  r.nb = (u - t * a.NU) * kCtas;
  return r;
}

// M-major A operand, 128B swizzle: 64 M elements by 8 reduction rows per 1024-byte
// atom, the next 8 rows 1024 B on, the next 64 M elements one panel (64 rows x
// 128 B) on.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Two E2M1 x E4M3 products as a BF16 pair: FP16 x FP16 -> FP32 multiplies (exact),
// one packing conversion (exact).
__device__ __forceinline__ uint32_t scaled_pair_bf16(uint32_t codes_f16x2, uint32_t scale_f16) {
  float lo, hi;
  asm("{\n .reg .b16 l, h, s, u;\n mov.b32 {l, h}, %2;\n mov.b32 {s, u}, %3;\n"
      " fma.rn.f32.f16 %0, l, s, 0f00000000;\n fma.rn.f32.f16 %1, h, s, 0f00000000;\n}"
      : "=f"(lo), "=f"(hi)
      : "r"(codes_f16x2), "r"(scale_f16));
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 weights (8 bytes of codes; scale in the low half of s) -> 8 BF16 pairs.
__device__ __forceinline__ void dequant16_bf16(uint32_t c0, uint32_t c1, uint32_t s, uint32_t (&o)[8]) {
  uint32_t v[4];
  e2m1x8_to_f16x2x4(c0, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = scaled_pair_bf16(v[i], s);
  e2m1x8_to_f16x2x4(c1, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[4 + i] = scaled_pair_bf16(v[i], s);
}

template <bool kBackward, int kCtas>
__global__ void __launch_bounds__(gg::kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap, GroupedArgs a) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  GroupedCtl& ctl = *reinterpret_cast<GroupedCtl*>(smem);
  uint8_t* ring = smem + gg::kRingOff;
  // a stage: the operand's two halves, then the rows' two halves (this CTA's share of the tile)
  const int b_half = a.tile_rows / kCtas * 128;
  const int stage_bytes = 2 * gg::kHalfBytes + 2 * b_half;
  uint8_t* raw = ring + a.stages * stage_bytes;
  const uint32_t ring_addr = smem_u32(ring);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
  const int first = blockIdx.x / kCtas, stride = gridDim.x / kCtas;
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.raw_stages; ++s) {
      mbar_init(ctl.raw_full + s, 1);
      mbar_init(ctl.raw_empty + s, gg::kTeamWarps);
    }
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(ctl.a_full + s, kCtas * gg::kTeamWarps);  // waited for by the pair's first CTA
      mbar_init(ctl.b_full + s, 1);                          // the same
      mbar_init(ctl.empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(ctl.acc_full + b, 1);
      mbar_init(ctl.acc_empty + b, kCtas * gg::kEpiWarps);
    }
    ctl.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (kCtas == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = threadIdx.x; i <= a.E; i += gg::kThreads) ctl.off[i] = a.offsets[i];
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
  if (kCtas == 2) cluster_sync_all();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const int total = ctl.tile[a.E] * a.NU;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- packed weights of this CTA's 128 features ----------------
      uint32_t it = 0;
      RingPos p;
      bool ok = true;
      for (int u = first; u < total && ok && a.fault != 1; u += stride) {
        const GroupedUnit w = grouped_unit<kCtas>(ctl, a, u);
        // the last pair of an odd number of blocks: the second CTA computes the first one's block again, unstored
        const int nb = min(w.nb + rank, a.NB - 1);
        const uint8_t* src = a.blob + (size_t)w.e * a.expert_stride + (size_t)nb * a.block_stride;
        for (int s = 0; s < a.steps; ++s, ++it, p.step(a.raw_stages)) {
          if (!mbar_wait(ctl.raw_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 911)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(ctl.raw_full + p.slot, gg::kPairBytes);
          bulk_g2s(raw + p.slot * gg::kPairBytes, src + (size_t)s * a.step_stride, gg::kPairBytes, ctl.raw_full + p.slot);
        }
      }
      if (!ok) drain_copies(ctl.raw_full, it, a.raw_stages);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: the whole warp walks the loop, one lane issues ----------------
    uint32_t j = 0;
    RingPos p;
    if (rank == 0) {
      for (int u = first; u < total; u += stride, ++j) {
        const GroupedUnit w = grouped_unit<kCtas>(ctl, a, u);
        const uint32_t idesc =
            idesc_bf16(128 * kCtas, (w.rows + 16 * kCtas - 1) & ~(16 * kCtas - 1)) | (kBackward ? 1u << 15 : 0u);
        const uint32_t buf = j & 1u;
        if (!mbar_wait_cluster(ctl.acc_empty + buf, ((j >> 1) & 1u) ^ 1u, abort_flag, a.st, 912)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 256u;
        bool ok = true;
        for (int s = 0; s < a.steps; ++s, p.step(a.stages)) {
          if (!mbar_wait_cluster(ctl.b_full + p.slot, p.phase, abort_flag, a.st, 913) ||
              !mbar_wait_cluster(ctl.a_full + p.slot, p.phase, abort_flag, a.st, 914)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = ring_addr + (uint32_t)(p.slot * stage_bytes);
          const uint64_t ad = kBackward ? sw128_desc_mn(st) : sw128_desc(st);
          const uint64_t bd = sw128_desc(st + 2 * gg::kHalfBytes);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 reduction elements: 32 B along a row, or 16 rows of 128 B
              const uint64_t ak = ad + (uint32_t)(kk >> 2) * (gg::kHalfBytes >> 4) + (kBackward ? 128u : 2u) * (kk & 3);
              const uint64_t bk = bd + (uint32_t)(kk >> 2) * (uint32_t)(b_half >> 4) + 2u * (kk & 3);
              if (kCtas == 2) umma_bf16_pair(d, ak, bk, idesc, (s | kk) != 0 ? 1u : 0u);
              else umma_bf16(d, ak, bk, idesc, (s | kk) != 0 ? 1u : 0u);
            }
            if (kCtas == 2) umma_commit_pair(ctl.empty + p.slot);
            else umma_commit(ctl.empty + p.slot);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          if (kCtas == 2) umma_commit_pair(ctl.acc_full + buf);
          else umma_commit(ctl.acc_full + buf);
        }
        __syncwarp();
      }
    }
  } else if (warp == 2) {
    // ---------------- rows of x (dy): this CTA's half of the tile, boxes of 64 reduction elements ----------------
    uint32_t it = 0;
    RingPos p;
    bool ok = true;
    for (int u = first; u < total && ok && a.fault != 1; u += stride) {
      const GroupedUnit w = grouped_unit<kCtas>(ctl, a, u);
      const int share = ((w.rows + 16 * kCtas - 1) & ~(16 * kCtas - 1)) / kCtas;
      const int nbox = (share + a.box - 1) / a.box;
      const int row0 = w.row0 + rank * share;
      for (int s = 0; s < a.steps; ++s, ++it, p.step(a.stages)) {
        if (!mbar_wait(ctl.empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 915)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* dst = ring + p.slot * stage_bytes + 2 * gg::kHalfBytes;
          if (rank == 0) mbar_arrive_expect_tx(ctl.b_full + p.slot, (uint32_t)(kCtas * 2 * nbox * a.box) * 128u);
          const uint32_t bar = kCtas == 2 ? map_rank(ctl.b_full + p.slot, 0) : 0u;
          for (int h = 0; h < 2; ++h)
            for (int b = 0; b < nbox; ++b) {
              if (kCtas == 2) tma_2d_pair(dst + h * b_half + b * a.box * 128, &tmap, s * 128 + h * 64, row0 + b * a.box, bar);
              else tma_2d(dst + h * b_half + b * a.box * 128, &tmap, s * 128 + h * 64, row0 + b * a.box, ctl.b_full + p.slot);
            }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      if (rank == 0) drain_copies(ctl.b_full, it, a.stages);
      else
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // its copies complete on the first CTA's barriers
    }
  } else if (warp >= 8) {
    // ---------------- dequantisers: two teams take turns at the squares; warp w of a team takes one 16-row
    // sub-block of each half, so that its waits and its fence are paid once for 64 weights a lane ----------------
    const int team = (warp - 8) >> 3, w = (warp - 8) & 7, q = lane & 3;
    const int slot = seg_pos(lane);
    // forward: half h is tile h (K elements 64 h ..), all 128 rows; backward: rows 64 h .. of both tiles
    const int r = (kBackward ? (w & 3) * 16 : w * 16) + (lane >> 2);
    const uint32_t dst0 = (kBackward ? (uint32_t)(w >> 2) * 8192u : 0u) + (uint32_t)r * 128u;
    const uint32_t x0 = (uint32_t)((2 * q) ^ (r & 7)) * 16u, x1 = (uint32_t)((2 * q + 1) ^ (r & 7)) * 16u;
    RingPos pr, pa;
    int mine = 0;  // team of the current square
    bool ok = true;
    for (int u = first; u < total && ok; u += stride) {
      for (int s = 0; s < a.steps; ++s, mine ^= 1, pr.step(a.raw_stages), pa.step(a.stages)) {
        if (mine != team) continue;
        if (!mbar_wait(ctl.raw_full + pr.slot, pr.phase, abort_flag, a.st, 916)) {
          ok = false;
          break;
        }
        uint4 c[2];
        uint32_t sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* tile = raw + pr.slot * gg::kPairBytes + (kBackward ? w >> 2 : h) * kTileBytes;
          const int sb = kBackward ? 4 * h + (w & 3) : w;
          c[h] = *reinterpret_cast<const uint4*>(tile + sb * 512 + slot * 16);
          sc[h] = *reinterpret_cast<const uint16_t*>(tile + kTileCodes + sb * 64 + slot * 2);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ctl.raw_empty + pr.slot);
        if (!mbar_wait(ctl.empty + pa.slot, pa.phase ^ 1u, abort_flag, a.st, 917)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t s2 = e4m3x2_to_f16x2(sc[h]);
          const uint32_t p = ring_addr + (uint32_t)(pa.slot * stage_bytes + h * gg::kHalfBytes) + dst0;
          uint32_t o[8];
          dequant16_bf16(c[h].x, c[h].y, s2, o);
          sts128(p + x0, o[0], o[1], o[2], o[3]);
          sts128(p + x1, o[4], o[5], o[6], o[7]);
          dequant16_bf16(c[h].z, c[h].w, s2 >> 16, o);
          sts128(p + 1024u + x0, o[0], o[1], o[2], o[3]);
          sts128(p + 1024u + x1, o[4], o[5], o[6], o[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 2 && rank) mbar_arrive_cluster(map_rank(ctl.a_full + pa.slot, 0));
          else mbar_arrive(ctl.a_full + pa.slot);
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- epilogue: warp w reads TMEM lanes 32 (w % 4) .., one output feature a lane, and turns
    // 32 (FP32: 16) rows x 32 features through shared memory into 16-byte stores ----------------
    const int quarter = warp & 3;
    uint8_t* buf_s = smem + gg::kCtlBytes + quarter * gg::kEpiBytes;
    uint32_t j = 0;
    for (int u = first; u < total; u += stride, ++j) {
      const GroupedUnit w = grouped_unit<kCtas>(ctl, a, u);
      const float gs = __ldg(a.gscale + w.e);
      const uint32_t buf = j & 1u;
      if (!mbar_wait(ctl.acc_full + buf, (j >> 1) & 1u, abort_flag, a.st, 918)) break;
      tc_fence_after();
      const uint32_t t = tmem + ((uint32_t)(32 * quarter) << 16) + buf * 256u;
      const int f0 = 128 * (w.nb + rank) + 32 * quarter;  // beyond n_out for a block computed twice
      if (f0 < a.n_out) {
        for (int col = 0; col < w.rows; col += 32) {
          uint32_t v[2][16];
          tmem_ld16_nw(t + (uint32_t)col, v[0]);
          tmem_ld16_nw(t + (uint32_t)col + 16u, v[1]);  // past the tile's last column: unwritten columns, not stored
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          if (a.out_f32) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                *reinterpret_cast<float*>(buf_s + i * 128 + lane * 4) = gs * __uint_as_float(v[hh][i]);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = 4 * i + (lane >> 3), f = f0 + 4 * (lane & 7), rr = col + 16 * hh + row;
                if (rr < w.rows && f < a.n_out)
                  *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + (long long)(w.row0 + rr) * a.ldo + f) =
                      *reinterpret_cast<const uint4*>(buf_s + row * 128 + (lane & 7) * 16);
              }
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              *reinterpret_cast<__nv_bfloat16*>(buf_s + i * 64 + lane * 2) =
                  __float2bfloat16_rn(gs * __uint_as_float(v[i >> 4][i & 15]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 8 * i + (lane >> 2), f = f0 + 8 * (lane & 3), rr = col + row;
              if (rr < w.rows && f < a.n_out)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (long long)(w.row0 + rr) * a.ldo + f) =
                    *reinterpret_cast<const uint4*>(buf_s + row * 64 + (lane & 3) * 16);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kCtas == 2) mbar_arrive_cluster(map_rank(ctl.acc_empty + buf, 0));
        else mbar_arrive(ctl.acc_empty + buf);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kCtas == 2) cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    if (kCtas == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

typedef void (*GroupedKernel)(const CUtensorMap, GroupedArgs);
static GroupedKernel grouped_kernel(bool backward, bool pair) {
  return backward ? (pair ? grouped_gemm_kernel<true, 2> : grouped_gemm_kernel<true, 1>)
                  : (pair ? grouped_gemm_kernel<false, 2> : grouped_gemm_kernel<false, 1>);
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
  for (int i = 0; i < 4; ++i) {
    e = cudaFuncSetAttribute((const void*)grouped_kernel(i & 1, i & 2), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gg::kSmemMax);
    if (e != cudaSuccess) return e;
  }
  if (dev >= 0 && dev < kCached) done[dev] = true;
  return cudaSuccess;
}

GroupedTiling grouped_tiling(int E, int R, int out_blocks) {
  GroupedTiling t;
  t.ctas = out_blocks > 1 ? 2 : 1;
  // rows per token tile: wide tiles dequantise a weight square once for many rows, narrow ones leave
  // shared memory for a deeper packed ring, which the few-rows end needs to stream weights
  const int avg = R / E;
  t.tile_rows = avg > 64 ? 256 : avg > 32 ? 128 : 64;
  t.box = t.tile_rows / t.ctas < 64 ? t.tile_rows / t.ctas : 64;
  return t;
}

cudaError_t launch_grouped_gemm(const GroupedProduct& p, bool backward, const GroupedTiling& t,
                                const CUtensorMap& rows_map, cudaStream_t st) {
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
  a.NU = (a.NB + t.ctas - 1) / t.ctas;
  a.steps = backward ? Np / 128 : p.K / 128;
  a.block_stride = backward ? (size_t)gg::kPairBytes : row_block;
  a.step_stride = backward ? row_block : (size_t)gg::kPairBytes;
  a.n_out = backward ? p.K : p.N;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.st = p.status;
  a.fault = p.fault;
  a.tile_rows = t.tile_rows;
  a.box = t.box;
  const int stage = 2 * gg::kHalfBytes + 2 * (t.tile_rows / t.ctas) * 128;
  const int room = gg::kSmemMax - 1024 - gg::kRingOff;
  a.stages = stage > 49152 ? (room - 2 * gg::kPairBytes) / stage : 4;
  const int left = (room - a.stages * stage) / gg::kPairBytes;
  a.raw_stages = left < gg::kMaxRaw ? left : gg::kMaxRaw;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.num_sms / t.ctas * t.ctas));
  cfg.blockDim = dim3(gg::kThreads);
  cfg.dynamicSmemBytes = gg::kSmemMax;
  cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)t.ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_kernel(backward, t.ctas == 2), rows_map, a);
}

}  // namespace nvfp4moe
