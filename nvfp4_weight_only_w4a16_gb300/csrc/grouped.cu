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
// to pair with or nothing to gain from it (grouped_tiling).
//
// kSplit: where there are few units, a cluster of 2 or 4 CTAs takes one unit, a
// share of the reduction each.  Then each puts its sums into its shared memory (the
// rings, which are done with), and adds and stores every S-th row from all of theirs,
// in a fixed order.
//
// One CTA per multiprocessor, 24 warps: 0 packed-weight producer (bulk copies into
// a ring), 1 MMA issuer (the pair's first CTA; for narrow tiles 3 too), 2 row
// producer (TMA, zero fill past the matrix), 4-7 epilogue (TMEM -> gs -> shared ->
// 16-byte stores), the rest dequantisers, in teams that take turns.  Two accumulator
// buffers: the epilogue of a unit overlaps the next one's MMAs.  The row offsets are
// read on the device; every CTA derives the same unit list from them, so nothing is
// written but the output.
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace gg {
constexpr int kDequantWarps = 16, kEpiWarps = 4;
constexpr int kThreads = 32 * (8 + kDequantWarps);
constexpr int kPairBytes = 2 * kTileBytes;  // one 128 x 128 weight square, packed
constexpr int kHalfBytes = 16384;           // half a square in BF16: 64 long in the reduction
constexpr int kSmemMax = 232448;
constexpr int kCtlBytes = 4096;             // tables and barriers in front of the rings
constexpr int kEpiBytes = 2048;             // per epilogue warp
constexpr int kRingOff = kCtlBytes + kEpiWarps * kEpiBytes;
constexpr int kMaxStages = 8, kMaxRaw = 16;
constexpr int kMaxSplit = 4;                // CTAs that share a unit
constexpr int kRoom = kSmemMax - 1024 - kRingOff;  // for the rings

// What follows from the CTAs of a unit (1 or 2) and the rows of a token tile (64, 128 or 256): MMA issuers and ring
// depths.
//
// With up to 64 rows the MMAs are so short that issuing them sets the pace, so two warps take turns at the squares,
// each into an accumulator of its own.
//
// The forward's operand goes to tensor memory where that has room beside the accumulators, that is for tiles of up to
// 128 rows: with the operand in shared memory its bandwidth is the bound there (per square 256 of 128-byte accesses to
// write it, 256 to read it, and 400 for the rest, against some 390 cycles that the packed bytes take from memory).
// The transposed operand would have to cross the lanes to get there.
//
// The rows have a ring of their own, deeper than the operand's: they come from L2 some 1500 cycles after they are asked
// for, and with the operand's 4 stages that alone made a square cost 670 cycles (64 rows an expert, E 128, N 1536,
// K 4096: 115 us with no conversion, no MMA and no weights, of 149).
//
// The dequantisers work in teams that take turns at the squares.  Half of what a warp spends on a square is waiting for
// and signalling barriers, so small teams with more of a square to each warp are better: four teams of four warps where
// there are four operand stages and packed slots for them, else two of eight.
//
// A parity wait must not run two phases ahead of its barrier: a team meets every packed slot again itself (their
// number is a multiple of the teams; bulk copies may land out of order), and so does one of two issuers every stage;
// one issuer frees the operand stages in order, so that as many of them as teams are enough.
template <bool kBackward, int kCtas, int kTile>
struct Plan {
  static constexpr bool kTmemA = !kBackward && kCtas == 2 && kTile <= 128;
  static constexpr int kIssuers = kCtas == 2 && kTile == 64 ? 2 : 1;
  static constexpr int kABytes = kTmemA ? 0 : 2 * kHalfBytes;  // an operand stage in shared memory: a square
  static constexpr int kBHalf = kTile / kCtas * 128;           // half a row stage: this CTA's share of the tile
  static constexpr int kBBytes = 2 * kBHalf;
  static constexpr int kStagesA = kTmemA || kTile == 64 ? 4 : kCtas == 1 && kTile == 256 ? 2 : 3;
  static constexpr int kStagesB = kTmemA ? (kTile == 64 ? 8 : 6)
                                  : kCtas == 2 ? (kTile == 64 ? 6 : kTile == 128 ? 5 : 3)
                                               : (kTile == 64 ? 4 : kTile == 128 ? 3 : 2);
  static constexpr int kRings = kStagesA * kABytes + kStagesB * kBBytes;
  static constexpr int kFit = (kRoom - kRings) / kPairBytes;
  static constexpr int kTeams = kStagesA == 4 && kFit >= 4 ? 4 : 2, kTeamWarps = kDequantWarps / kTeams;
  static constexpr int kRaw = kFit / kTeams * kTeams;  // packed slots
  static constexpr int kBox = kTile / kCtas < 64 ? kTile / kCtas : 64;          // rows per TMA box
  // tensor memory: buffer b, issuer h at b kAccBuf + h kAccIssuer; operand stages of 64 columns from kOperand on
  static constexpr uint32_t kAccBuf = kTmemA ? 128 : 256, kAccIssuer = kAccBuf / 2, kOperand = 256;
  static_assert(kRaw >= kTeams && kRaw <= kMaxRaw && kStagesA <= kMaxStages && kStagesB <= kMaxStages && kStagesA >= kTeams, "rings");
  static_assert(kIssuers == 1 || (kStagesA % 2 == 0 && kStagesB % 2 == 0 && kStagesA % kTeams == 0), "two issuers");
  static_assert(kBHalf % 1024 == 0, "128B-swizzled tiles");
};
}  // namespace gg

// The result's type, where the kernel knows it: with tiles of 256 rows that is 1 to 2% faster, with fewer, where the
// dequantisers' code sets the pace, up to 4% slower.
enum class Out { kBf16, kF32, kEither };

struct GroupedArgs {
  const uint8_t* blob;
  size_t expert_stride;
  const float* gscale;     // [E]
  const int32_t* offsets;  // [E + 1]
  int E, R;
  int NB;                  // 128-feature output blocks
  int NU;                  // work units across the features: NB or, in pairs, half of it
  int steps;               // 128-long reduction steps
  int split;               // CTAs that share a unit's (kSplit), else 1
  size_t block_stride;     // bytes from one output block's first square to the next one's
  size_t step_stride;      // bytes from one reduction step's square to the next
  int n_out;               // output features
  void* out;
  long long ldo;
  int out_f32;
  DeviceStatus* st;
  int fault;
  uint32_t zero;           // 0, unknown to the compiler
};

struct GroupedCtl {
  int off[257];
  int tile[257];   // token tiles before expert e; tile[E] = all
  short per[256];  // rows per tile of expert e: its tiles are of one size, so that none is a small remainder
  uint64_t raw_full[gg::kMaxRaw], raw_empty[gg::kMaxRaw];
  uint64_t a_full[gg::kMaxStages], a_empty[gg::kMaxStages], b_full[gg::kMaxStages], b_empty[gg::kMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done[2];  // every MMA of issuer h has completed
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(GroupedCtl) <= gg::kCtlBytes, "control block");

// The units of one CTA (pair): first, first + stride, ..; unit u is feature block(s) u % NU of token tile u / NU.
template <int kCtas>
struct GroupedUnits {
  int u, stride, nu, t, nb, dt, dnb, e;
  __device__ __forceinline__ GroupedUnits(const GroupedCtl& c, const GroupedArgs& a, int first, int step)
      : u(first), stride(step), nu(a.NU) {
    t = u / nu, nb = u - t * nu;
    dt = stride / nu, dnb = stride - dt * nu;
    e = 0;
    int hi = a.E;  // the expert e with tile[e] <= t < tile[e + 1]
    while (hi - e > 1) {
      const int mid = (e + hi) >> 1;
      if (c.tile[mid] <= t) e = mid;
      else hi = mid;
    }
  }
  __device__ __forceinline__ void next(const GroupedCtl& c, int total) {
    u += stride, t += dt, nb += dnb;
    if (nb >= nu) nb -= nu, ++t;
    if (u < total)
      while (c.tile[e + 1] <= t) ++e;
  }
  __device__ __forceinline__ int block() const { return nb * kCtas; }
  __device__ __forceinline__ int rows(const GroupedCtl& c, int& row0) const {
    const int per = c.per[e], j = (t - c.tile[e]) * per;
    row0 = c.off[e] + j;
    return min(per, c.off[e + 1] - c.off[e] - j);
  }
};

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

// 32 registers into 32 columns of the thread's lane; the caller waits.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&o)[4][8]) {
  const uint32_t* w = o[0];
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]), "r"(w[16]), "r"(w[17]), "r"(w[18]),
      "r"(w[19]), "r"(w[20]), "r"(w[21]), "r"(w[22]), "r"(w[23]), "r"(w[24]), "r"(w[25]), "r"(w[26]), "r"(w[27]),
      "r"(w[28]), "r"(w[29]), "r"(w[30]), "r"(w[31])
      : "memory");
}

template <bool kBackward, int kCtas, int kTile, Out kOut, bool kSplit>
__global__ void __launch_bounds__(gg::kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap, GroupedArgs a) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  GroupedCtl& ctl = *reinterpret_cast<GroupedCtl*>(smem);
  uint8_t* ring = smem + gg::kRingOff;
  using Plan = gg::Plan<kBackward, kCtas, kTile>;
  constexpr int kIssuers = Plan::kIssuers, kTeams = Plan::kTeams, kTeamWarps = Plan::kTeamWarps;
  // FP32 results: the two halves of the reduction into an accumulator each, summed in the epilogue, in place of two
  // units' accumulators.  The tensor core truncates where it adds (4e-6 of the result's norm after 4096 terms in one
  // accumulator, E4M3 scales over their whole range, 2e-6 in two), and BF16's rounding hides that.
  const auto f32 = [&] { return kOut == Out::kF32 || (kOut == Out::kEither && a.out_f32); };
  const auto halves = [&] { return kIssuers == 1 && !kSplit && f32(); };  // (split: already fewer terms each)
  constexpr int kStagesA = Plan::kStagesA, kStagesB = Plan::kStagesB, kRaw = Plan::kRaw;
  uint8_t* ring_b = ring + kStagesA * Plan::kABytes;
  uint8_t* raw = ring + Plan::kRings;
  const uint32_t ring_addr = smem_u32(ring), ring_b_addr = smem_u32(ring_b), raw_addr = smem_u32(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(!kSplit || kCtas == 1, "a cluster is a pair or shares a unit");
  const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
  const int first = kSplit ? blockIdx.x / a.split : blockIdx.x / kCtas;
  const int stride = kSplit ? gridDim.x / a.split : gridDim.x / kCtas;  // split: no CTA has a second unit
  const int part = kSplit ? (int)cluster_rank() : 0;
  const int step0 = kSplit ? part * a.steps / a.split : 0;  // this CTA's steps of the reduction
  const int steps = kSplit ? (part + 1) * a.steps / a.split - step0 : a.steps;
  constexpr int kRound = 16 * kCtas;  // the MMA's columns come in these
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(ctl.raw_full + s, 1);
      mbar_init(ctl.raw_empty + s, kTeamWarps);
    }
    for (int s = 0; s < kStagesA; ++s) {
      mbar_init(ctl.a_full + s, kCtas * kTeamWarps);  // waited for by the pair's first CTA
      mbar_init(ctl.a_empty + s, 1);
    }
    for (int s = 0; s < kStagesB; ++s) {
      mbar_init(ctl.b_full + s, 1);  // the same
      mbar_init(ctl.b_empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(ctl.acc_full + b, kIssuers);
      mbar_init(ctl.acc_empty + b, kCtas * gg::kEpiWarps);
      mbar_init(ctl.mma_done + b, 1);
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
      n[i] = (m + kTile - 1) / kTile;
      if (e < a.E && n[i] > 0) ctl.per[e] = (short)(((m + n[i] - 1) / n[i] + kRound - 1) & ~(kRound - 1));
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
  const int squares = first < total ? ((total - first - 1) / stride + 1) * steps : 0;  // of this CTA

  if (warp == 0) {
    // ---------------- packed weights of this CTA's 128 features ----------------
    uint32_t it = 0;
    RingPos p;
    bool ok = true;
    for (GroupedUnits<kCtas> w(ctl, a, first, stride); w.u < total && ok && a.fault != 1; w.next(ctl, total)) {
      // the last pair of an odd number of blocks: the second CTA computes the first one's block again, unstored
      const int nb = min(w.block() + rank, a.NB - 1);
      const uint8_t* src = a.blob + (size_t)w.e * a.expert_stride + (size_t)nb * a.block_stride +
                           (kSplit ? (size_t)step0 * a.step_stride : 0);
      for (int s = 0; s < steps; ++s, ++it, p.step(kRaw), src += a.step_stride) {
        if (!warp_wait(ctl.raw_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 911)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(ctl.raw_full + p.slot, gg::kPairBytes);
          bulk_g2s(raw + p.slot * gg::kPairBytes, src, gg::kPairBytes, ctl.raw_full + p.slot);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) drain_copies(ctl.raw_full, it, kRaw);
  } else if (warp == 1 || (kIssuers == 2 && warp == 3)) {
    // ---------------- MMA issuers: the whole warp walks the loop, one lane issues.  Issuer h takes every kIssuers-th
    // square of the CTA's sequence, into its own accumulator ----------------
    if (rank == 0) {
      const int h = warp >> 1;  // 0, 1
      uint32_t j = 0;
      int base = 0;  // squares before the unit
      bool ok = true;
      for (GroupedUnits<kCtas> w(ctl, a, first, stride); w.u < total && ok; w.next(ctl, total), ++j, base += steps) {
        int row0;
        const uint32_t idesc =
            idesc_bf16(128 * kCtas, (w.rows(ctl, row0) + kRound - 1) & ~(kRound - 1)) | (kBackward ? 1u << 15 : 0u);
        const uint32_t buf = halves() ? 0u : j & 1u;
        if (!warp_wait(ctl.acc_empty + buf, ((halves() ? j : j >> 1) & 1u) ^ 1u, abort_flag, a.st, 912)) break;
        tc_fence_after();
        uint32_t d = tmem + buf * Plan::kAccBuf + (uint32_t)h * Plan::kAccIssuer;
        const int end = base + steps;
        int i = kIssuers == 2 ? base + ((base ^ h) & 1) : base;
        int stop = halves() && steps > 1 ? base + steps / 2 : end;
        uint32_t acc = 0;
        for (; ok; stop = end, d += Plan::kAccBuf, acc = 0) {  // once or twice (a test in the loop itself cost 1.5%)
          for (; i < stop; i += kIssuers) {
            const int sa = i % kStagesA, sb = i % kStagesB;
            if (!warp_wait(ctl.b_full + sb, (uint32_t)(i / kStagesB) & 1u, abort_flag, a.st, 913) ||
                !warp_wait(ctl.a_full + sa, (uint32_t)(i / kStagesA) & 1u, abort_flag, a.st, 914)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t st = ring_addr + (uint32_t)(sa * Plan::kABytes);
            const uint64_t ad = kBackward ? sw128_desc_mn(st) : sw128_desc(st);
            const uint64_t bd = sw128_desc(ring_b_addr + (uint32_t)(sb * Plan::kBBytes));
            const uint32_t at = tmem + Plan::kOperand + (uint32_t)sa * 64u;  // 8 columns per 16 elements
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {  // 16 reduction elements: 32 B along a row, or 16 rows of 128 B
                const uint64_t ak = ad + (uint32_t)(kk >> 2) * (gg::kHalfBytes >> 4) + (kBackward ? 128u : 2u) * (kk & 3);
                const uint64_t bk = bd + (uint32_t)(kk >> 2) * (uint32_t)(Plan::kBHalf >> 4) + 2u * (kk & 3);
                if (Plan::kTmemA) umma_ts_pair(d, at + 8u * kk, bk, idesc, kk ? 1u : acc);
                else if (kCtas == 2) umma_bf16_pair(d, ak, bk, idesc, kk ? 1u : acc);
                else umma_bf16(d, ak, bk, idesc, kk ? 1u : acc);
              }
              if (kCtas == 2) {
                umma_commit_pair(ctl.b_empty + sb);
                umma_commit_pair(ctl.a_empty + sa);
              } else {
                umma_commit(ctl.b_empty + sb);
                umma_commit(ctl.a_empty + sa);
              }
            }
            acc = 1;
            __syncwarp();
          }
          if (stop == end) break;
        }
        if (!ok) break;
        if (elect_one()) {  // (an issuer without a square in the unit: nothing to wait for, and its accumulator is not read)
          if (kCtas == 2) umma_commit_pair(ctl.acc_full + buf);
          else umma_commit(ctl.acc_full + buf);
        }
        __syncwarp();
      }
      // MMAs may still be at work where a role has given up: none may outlive the shared and tensor memory it uses
      if (elect_one()) {
        if (kCtas == 2) umma_commit_pair_own(ctl.mma_done + h);
        else umma_commit(ctl.mma_done + h);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(ctl.mma_done + h, 0) && globaltimer_ns() - t0 <= kWaitTimeoutNs) {}
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    // ---------------- rows of x (dy): this CTA's half of the tile, boxes of 64 reduction elements ----------------
    uint32_t it = 0;
    RingPos p;
    bool ok = true;
    for (GroupedUnits<kCtas> w(ctl, a, first, stride); w.u < total && ok && a.fault != 1; w.next(ctl, total)) {
      int row0;
      const int share = ((w.rows(ctl, row0) + kRound - 1) & ~(kRound - 1)) / kCtas;
      const int nbox = (share + Plan::kBox - 1) / Plan::kBox;
      row0 += rank * share;
      for (int s = step0; s < step0 + steps; ++s, ++it, p.step(kStagesB)) {
        if (!warp_wait(ctl.b_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 915)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* dst = ring_b + p.slot * Plan::kBBytes;
          uint64_t* bar = ctl.b_full + p.slot;
          if (rank == 0) mbar_arrive_expect_tx(bar, (uint32_t)(kCtas * 2 * nbox * Plan::kBox) * 128u);
          const uint32_t bar0 = kCtas == 2 ? map_rank(bar, 0) : 0u;
          for (int h = 0; h < 2; ++h)
            for (int b = 0; b < nbox; ++b) {
              uint8_t* to = dst + h * Plan::kBHalf + b * Plan::kBox * 128;
              if (kCtas == 2) tma_2d_pair(to, &tmap, s * 128 + h * 64, row0 + b * Plan::kBox, bar0);
              else tma_2d(to, &tmap, s * 128 + h * 64, row0 + b * Plan::kBox, bar);
            }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      if (rank == 0) drain_copies(ctl.b_full, it, kStagesB);
      else
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // its copies complete on the first CTA's barriers
    }
  } else if (warp >= 8) {
    // ---------------- dequantisers: the teams take turns at the squares.  A square's work is 8 shares (share w: in
    // shared memory one 16-row sub-block of each half, in tensor memory 32 rows of one half); a warp takes kShares of
    // them, w and w + 4, so that its waits and its fence are paid once ----------------
    constexpr int kShares = 8 / kTeamWarps;
    const int team = (warp - 8) / kTeamWarps, w0 = (warp - 8) % kTeamWarps, q = lane & 3;
    const uint32_t raw_empty0 = smem_u32(ctl.raw_empty);
    const uint32_t full0 = kCtas == 2 ? map_rank(ctl.a_full, 0) : 0u;  // the pair's first CTA's
    RingPos pr, pa;
    pr.slot = pa.slot = team;  // at most the ring's depth
    for (int i = team; i < squares; i += kTeams, pr.step(kRaw, kTeams), pa.step(kStagesA, kTeams)) {
      if (!warp_wait(ctl.raw_full + pr.slot, pr.phase, abort_flag, a.st, 916)) break;
      const uint32_t pair = raw_addr + pr.slot * gg::kPairBytes;
      // The packed slot goes back as soon as it has been read.  A read that is merely issued can be overtaken by the
      // refill (measured: wrong 16-row groups), so the address of the arrival takes in what was read, masked by an
      // argument that is zero.
      uint32_t seen = 0;
      if constexpr (Plan::kTmemA) {
        // thread = one weight row, its TMEM lane: per half 4 groups of 16 elements, 8 bytes and a scale each
        const int r = 32 * (w0 & 3) + lane;
        uint2 c[kShares][4];
        uint32_t sc[kShares][4];
#pragma unroll
        for (int k = 0; k < kShares; ++k) {
          const uint32_t tile = pair + (uint32_t)(((w0 + 4 * k) >> 2) * kTileBytes);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int slot = seg_pos(4 * (lane & 7) + g);
            c[k][g] = lds64(tile + (r >> 4) * 512 + ((r >> 3) & 1) * 8 + slot * 16);
            sc[k][g] = lds8(tile + kTileCodes + (r >> 4) * 64 + ((r >> 3) & 1) + slot * 2);
            seen |= c[k][g].x | c[k][g].y | sc[k][g];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_at(raw_empty0 + pr.slot * 8 + (seen & a.zero));
        if (!warp_wait(ctl.a_empty + pa.slot, pa.phase ^ 1u, abort_flag, a.st, 917)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kShares; ++k) {
          uint32_t o[4][8];
#pragma unroll
          for (int g = 0; g < 4; ++g) dequant16_bf16(c[k][g].x, c[k][g].y, e4m3x2_to_f16x2(sc[k][g]), o[g]);
          tmem_st32(tmem + ((uint32_t)(32 * (w0 & 3)) << 16) + Plan::kOperand + (uint32_t)pa.slot * 64u +
                        32u * (uint32_t)((w0 + 4 * k) >> 2),
                    o);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
      } else {
        uint4 c[kShares][2];
        uint32_t sc[kShares][2];
#pragma unroll
        for (int k = 0; k < kShares; ++k) {
          const int w = w0 + 4 * k;
          // forward: half h is tile h (K elements 64 h ..), all 128 rows; backward: rows 64 h .. of both tiles
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t tile = pair + (uint32_t)((kBackward ? w >> 2 : h) * kTileBytes);
            const int sb = kBackward ? 4 * h + (w & 3) : w;
            c[k][h] = lds128(tile + sb * 512 + seg_pos(lane) * 16);
            sc[k][h] = lds16(tile + kTileCodes + sb * 64 + seg_pos(lane) * 2);
            seen |= c[k][h].x | c[k][h].y | c[k][h].z | c[k][h].w | sc[k][h];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_at(raw_empty0 + pr.slot * 8 + (seen & a.zero));
        if (!warp_wait(ctl.a_empty + pa.slot, pa.phase ^ 1u, abort_flag, a.st, 917)) break;
#pragma unroll
        for (int k = 0; k < kShares; ++k) {
          const int w = w0 + 4 * k;
          const int r = (kBackward ? (w & 3) * 16 : w * 16) + (lane >> 2);
          const uint32_t x0 = (uint32_t)((2 * q) ^ (r & 7)) * 16u, x1 = (uint32_t)((2 * q + 1) ^ (r & 7)) * 16u;
          const uint32_t st = ring_addr + (uint32_t)(pa.slot * Plan::kABytes) + (kBackward ? (uint32_t)(w >> 2) * 8192u : 0u) +
                              (uint32_t)r * 128u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s2 = e4m3x2_to_f16x2(sc[k][h]);
            const uint32_t p = st + h * gg::kHalfBytes;
            uint32_t o[8];
            dequant16_bf16(c[k][h].x, c[k][h].y, s2, o);
            sts128(p + x0, o[0], o[1], o[2], o[3]);
            sts128(p + x1, o[4], o[5], o[6], o[7]);
            dequant16_bf16(c[k][h].z, c[k][h].w, s2 >> 16, o);
            sts128(p + 1024u + x0, o[0], o[1], o[2], o[3]);
            sts128(p + 1024u + x1, o[4], o[5], o[6], o[7]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) {
        if (kCtas == 2 && rank) mbar_arrive_cluster(full0 + pa.slot * 8);
        else mbar_arrive(ctl.a_full + pa.slot);
      }
    }
  } else if (warp >= 4 && kSplit) {
    if (first < total && !warp_wait(ctl.acc_full, 0, abort_flag, a.st, 918) && lane == 0) ctl.abort_flag = 1;
    tc_fence_after();
  } else if (warp >= 4) {
    // ---------------- epilogue: warp w reads TMEM lanes 32 (w % 4) .., one output feature a lane, and turns
    // 32 (FP32: 16) rows x 32 features through shared memory into 16-byte stores ----------------
    const int quarter = warp & 3;
    uint8_t* buf_s = smem + gg::kCtlBytes + quarter * gg::kEpiBytes;
    uint32_t j = 0;
    for (GroupedUnits<kCtas> w(ctl, a, first, stride); w.u < total; w.next(ctl, total), ++j) {
      int row0;
      const int rows = w.rows(ctl, row0);
      const float gs = __ldg(a.gscale + w.e);
      const uint32_t buf = halves() ? 0u : j & 1u;
      if (!warp_wait(ctl.acc_full + buf, (halves() ? j : j >> 1) & 1u, abort_flag, a.st, 918)) break;
      tc_fence_after();
      uint32_t t = tmem + ((uint32_t)(32 * quarter) << 16) + buf * Plan::kAccBuf;
      if (kIssuers == 2 && steps == 1) t += (j & 1u) * Plan::kAccIssuer;  // unit j's only square is the CTA's j-th
      const int f0 = 128 * (w.block() + rank) + 32 * quarter;  // beyond n_out for a block computed twice
      if (f0 < a.n_out) {
        for (int col = 0; col < rows; col += 32) {
          uint32_t v[2][16];
          if ((kIssuers == 2 || halves()) && steps > 1) {  // the sum of two accumulators
            constexpr uint32_t kOther = kIssuers == 2 ? Plan::kAccIssuer : Plan::kAccBuf;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {  // 16 columns at a time: all 32 of both would spill
              uint32_t v1[16];
              tmem_ld16_nw(t + (uint32_t)col + 16u * hh, v[hh]);
              tmem_ld16_nw(t + (uint32_t)col + 16u * hh + kOther, v1);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
              for (int i = 0; i < 16; ++i) v[hh][i] = __float_as_uint(__uint_as_float(v[hh][i]) + __uint_as_float(v1[i]));
            }
          } else {
            tmem_ld16_nw(t + (uint32_t)col, v[0]);
            tmem_ld16_nw(t + (uint32_t)col + 16u, v[1]);  // past the tile's last column: unwritten columns, not stored
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          }
          if (f32()) {
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
                if (rr < rows && f < a.n_out)
                  *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + (long long)(row0 + rr) * a.ldo + f) =
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
              if (rr < rows && f < a.n_out)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (long long)(row0 + rr) * a.ldo + f) =
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
  if constexpr (kSplit) {
    GroupedUnits<kCtas> w(ctl, a, first, stride);
    int row0 = 0;
    const int rows = first < total ? w.rows(ctl, row0) : 0;
    float* sums = reinterpret_cast<float*>(ring);  // [row][128 features]; the copies and MMAs are done with the rings
    if (warp >= 4 && warp < 8 && rows && !*abort_flag) {
      tc_fence_after();
      const uint32_t t = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
      for (int col = 0; col < rows; col += 16) {
        uint32_t v[16];
        tmem_ld16_nw(t + (uint32_t)col, v);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[(col + i) * 128 + 32 * (warp & 3) + lane] = __uint_as_float(v[i]);
      }
      tc_fence_before();
    }
    cluster_sync_all();
    const int f = 128 * w.block() + 4 * lane;
    if (rows && f < a.n_out) {
      const float gs = __ldg(a.gscale + w.e);
      for (int r = warp * a.split + part; r < rows; r += gg::kThreads / 32 * a.split) {
        float4 v[gg::kMaxSplit], y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < gg::kMaxSplit; ++c)
          if (c < a.split) v[c] = ld_cluster(sums + r * 128 + 4 * lane, c);
#pragma unroll
        for (int c = 0; c < gg::kMaxSplit; ++c)
          if (c < a.split) y.x += v[c].x, y.y += v[c].y, y.z += v[c].z, y.w += v[c].w;
        y.x *= gs, y.y *= gs, y.z *= gs, y.w *= gs;
        const long long o = (long long)(row0 + r) * a.ldo + f;
        if (f32()) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = y;
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its sums are read
  }
  if (warp == 1) {
    tc_fence_after();
    if (kCtas == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

typedef void (*GroupedKernel)(const CUtensorMap, GroupedArgs);
struct GroupedVariant {
  GroupedKernel fn[2][2];  // forward, backward; BF16, FP32
  int ctas, box;
};
template <int kCtas, int kTile, bool kSplit>
static constexpr GroupedVariant grouped_variant() {
  constexpr bool known = kTile == 256 && !kSplit;
  constexpr Out b = known ? Out::kBf16 : Out::kEither, f = known ? Out::kF32 : Out::kEither;
  return {{{grouped_gemm_kernel<false, kCtas, kTile, b, kSplit>, grouped_gemm_kernel<false, kCtas, kTile, f, kSplit>},
           {grouped_gemm_kernel<true, kCtas, kTile, b, kSplit>, grouped_gemm_kernel<true, kCtas, kTile, f, kSplit>}},
          kCtas,
          gg::Plan<false, kCtas, kTile>::kBox};
}
static const GroupedVariant kGroupedVariants[] = {
    grouped_variant<1, 64, false>(), grouped_variant<1, 128, false>(), grouped_variant<1, 256, false>(),
    grouped_variant<2, 64, false>(), grouped_variant<2, 128, false>(), grouped_variant<2, 256, false>(),
    grouped_variant<1, 64, true>(),  grouped_variant<1, 128, true>(),  grouped_variant<1, 256, true>()};

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
  for (int i = 0; i < 36; ++i) {
    e = cudaFuncSetAttribute((const void*)kGroupedVariants[i >> 2].fn[i & 1][(i >> 1) & 1], cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gg::kSmemMax);
    if (e != cudaSuccess) return e;
  }
  if (dev >= 0 && dev < kCached) done[dev] = true;
  return cudaSuccess;
}

GroupedTiling grouped_tiling(int E, int R, int out_blocks, int steps, int num_sms) {
  // Rows per token tile: a wide tile dequantises a weight square once for many rows, a narrow one leaves shared memory
  // for deeper rings.  At 128 experts of 1536 x 4096, counts spread by half around the mean (sigma 0.5), forward /
  // backward, us for tiles of 64, 128 and 256 rows: 32 rows an expert 143 / 140, 145 / 146, 187 / 171; 48 167 / 171,
  // 146 / 153, 190 / 175; 96 262 / 260, 172 / 193, 198 / 190; 112 285 / 286, 184 / 204, 200 / 195; 144 345 / 352,
  // 209 / 234, 209 / 205; 256 559 / 573, 332 / 374, 282 / 273.  Popularity by Zipf's law with 1.1 instead: 24 159 / 161,
  // 144 / 155, 175 / 174; 32 172 / 175, 156 / 167, 178 / 177; 64 221 / 223, 170 / 189, 197 / 199; 96 271 / 275, 196 / 216,
  // 206 / 212; so up to 32 rows on average, counts as uneven as that cost the rule, which sees the average, a tenth.
  const int avg = R / E;
  GroupedTiling t;
  const int width = avg > 112 ? 2 : avg > 32 ? 1 : 0;  // of a tile: 64, 128, 256 rows
  // Units too few for half of the multiprocessors share them, as long as a CTA keeps two squares: one expert of
  // 4096 x 4096, 32 rows, 17.7 us as pairs, 13.6 and 10.4 with 2 and 4 CTAs a unit; 2048 x 4096, 64 rows, 18.2, 14.4 and
  // 10.8 (8: 16.9, too few clusters of that size run at a time; of 4, 36 on 152 multiprocessors, and with 37 the time
  // goes from 10.8 to 19.0: hence 15/16).
  const int groups = E < R ? E : R;  // with rows: a unit each, and one for every further full tile, at most
  const long long units = (long long)((R - groups) / (64 << width) + groups) * out_blocks;
  t.units = (int)(units < num_sms ? units : num_sms);
  t.split = 1;
  while (t.split < gg::kMaxSplit && units * 2 * t.split <= (t.split == 1 ? num_sms : num_sms * 15 / 16) && 4 * t.split <= steps)
    t.split *= 2;
  // Pairs only where there are more units than multiprocessors or tiles of 128 rows and more, for which they halve the
  // reads of the rows: 8 experts of 272 x 256, 4 rows each, 7.0 us as pairs, 6.3 without; of 1024 x 1024, 16 rows, 9.0
  // and 8.8; but 2 of 4096 x 4096, 100 rows, 18.6 and 21.4.
  const bool pairs = out_blocks > 1 && (width > 0 || units > num_sms);
  t.variant = width + (t.split > 1 ? 6 : pairs ? 3 : 0);
  t.box = kGroupedVariants[t.variant].box;
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
  const GroupedVariant& v = kGroupedVariants[t.variant];
  a.NU = (a.NB + v.ctas - 1) / v.ctas;
  a.steps = backward ? Np / 128 : p.K / 128;
  a.split = t.split;
  a.block_stride = backward ? (size_t)gg::kPairBytes : row_block;
  a.step_stride = backward ? row_block : (size_t)gg::kPairBytes;
  a.n_out = backward ? p.K : p.N;
  a.out = p.out;
  a.ldo = p.ldo;
  a.out_f32 = p.out_f32;
  a.st = p.status;
  a.fault = p.fault;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(t.split > 1 ? t.units * t.split : p.num_sms / v.ctas * v.ctas));
  cfg.blockDim = dim3(gg::kThreads);
  cfg.dynamicSmemBytes = gg::kSmemMax;
  cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)(t.split > 1 ? t.split : v.ctas);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, v.fn[backward][p.out_f32 != 0], rows_map, a);
}

}  // namespace nvfp4moe
