// Linear with 8-bit integers on both sides (nvfp4_int8_*):
//   y[t][n] = sx[t] sw[n] sum_k xq[t][k] wq[n][k] + bias[n]
//
// The tensor cores of sm_103a that are fast take no integers, so both operands go through as FP16, which holds an 8-bit
// integer exactly; so is a product, and an FP32 sum of up to 1024 of them (below or at 2^24, which the alignment of what a
// tensor core adds does not cut).  Every 1024 terms the sums go to 32-bit integers, so that the whole sum is exact, and
// splitting it over warps and CTAs in any order changes nothing.
//
// The matrix is packed as bytes q + 128, [N / 128][K / 16][128 rows][16 elements], filled up with zeros to whole 128 x 128
// squares: a square is one 16 KB copy, a thread that owns a row reads 16 elements of it at a time without bank conflicts
// (GEMM), and a warp's reads for a fragment of 16 rows are runs of 256 bytes (few tokens).
#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace i8 {
constexpr int kSquare = 16384;  // bytes of a 128 x 128 square
constexpr int kSmemMax = 232448;
}  // namespace i8

// Four bytes q + 128 -> two FP16 pairs q: 1024 + byte by its bits, less 1152.
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
}
__device__ __forceinline__ void bytes_to_f16(const uint4& w, uint32_t (&o)[8]) {
  bytes_to_f16(w.x, o[0], o[1]);
  bytes_to_f16(w.y, o[2], o[3]);
  bytes_to_f16(w.z, o[4], o[5]);
  bytes_to_f16(w.w, o[6], o[7]);
}
__device__ __forceinline__ uint4 biased(uint4 w) {
  w.x ^= 0x80808080u, w.y ^= 0x80808080u, w.z ^= 0x80808080u, w.w ^= 0x80808080u;
  return w;
}

// --------------------------------------------------------------------------------------------------------------------
// Packing
// --------------------------------------------------------------------------------------------------------------------
size_t int8_packed_bytes(int N, int K) {
  return (size_t)((N + 127) / 128) * ((K + 127) / 128) * i8::kSquare;
}
// One thread a 16-byte piece.
__global__ void pack_int8_kernel(const int8_t* w, int N, int K, uint8_t* packed) {
  const long long pieces = (K + 127) / 128 * 8, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long blocks = (N + 127) / 128;
  if (i >= blocks * pieces * 128) return;
  const long long row = i / (128 * pieces) * 128 + i % 128, p = i / 128 % pieces;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (row < N && 16 * p < K) v = *reinterpret_cast<const uint4*>(w + row * K + 16 * p);
  reinterpret_cast<uint4*>(packed)[i] = biased(v);
}
cudaError_t launch_pack_int8(const int8_t* w_q, int N, int K, uint8_t* packed, cudaStream_t st) {
  const long long n = (long long)int8_packed_bytes(N, K) / 16;
  pack_int8_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(w_q, N, K, packed);
  return cudaGetLastError();
}

struct Int8Args {
  const uint8_t* packed;
  const float *w_scale, *bias;
  int N, K, T;
  const int8_t* x;
  const float* x_scale;
  long long ldx;  // bytes
  void* out;
  long long ldo;  // elements
  int out_type;
  bool once;
  DeviceStatus* st;
  int fault;
  // few tokens
  int wk;          // warps along K: 1, 2, 4, 8 or 16
  int slice;       // elements of K a warp takes at a time, a multiple of 64
  int passes;      // of all warps along K
  int batch;       // 16-row groups whose sums shared memory holds
  // GEMM
  int NB, NU;      // 128-feature blocks; units across the features
  int tiles, per;  // token tiles, and tokens of each
  int squares;     // 128-long steps of the reduction
  int split;       // CTAs that share a unit
};

// Two results that follow one another.
__device__ __forceinline__ void store_out(const Int8Args& a, long long at, float y, float z) {
  if (a.out_type == 1) *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(y, z);
  else if (a.out_type == 2) *reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + at) = __floats2half2_rn(y, z);
  else *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) = __floats2bfloat162_rn(y, z);
}

// --------------------------------------------------------------------------------------------------------------------
// Up to 16 tokens.  Bound by the matrix's bytes.
//
// A warp keeps one slice of K (up to 256 elements) of all tokens in registers as B fragments and streams the matrix past
// it, 16 rows at a time, through a ring of its own in shared memory, so there is no barrier.  Eight neighbouring lanes copy
// 128 bytes that follow one another: with each lane copying the 16 bytes that it will use, whose neighbours are 2 KB away,
// a copy took four times the cycles (12576 x 4096, 16 tokens: 21.5 us, now 12.0).  Bound by the matrix's bytes where there
// are enough of them (131072 x 4096, 4 tokens: 86 us, 0.94 of the copy rate; 4096 x 4096, 1 token: 4.3, its bytes 2.5).
// m16n8k16 sums a slice exactly in FP32; its integers are added to the CTA's sums in shared memory by
// atomics, whose order does not matter.  A CTA takes a run of 16-row groups, its warps share K and, where K is short, the
// groups; one barrier a batch of groups, and longer K in passes over the batch.
// --------------------------------------------------------------------------------------------------------------------
namespace i8v {
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kSlice = 256, kBlocks = kSlice / 64;  // 64-element blocks of a slice
constexpr int kStage = 16 * kSlice;                 // bytes: 16 rows of a slice
constexpr int kDepth = 3;
constexpr int kRing = kWarps * kDepth * kStage;
constexpr int kSumBytes = 24576;
constexpr int kMaxRows = (kSumBytes / 4 / 8 - 4) / 16 * 16;  // of a batch
constexpr int kSmem = kRing + kSumBytes + 8 * kMaxRows + 64;
}  // namespace i8v

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kTiles: groups of 8 tokens.
template <int kTiles>
__global__ void __launch_bounds__(i8v::kThreads, 1) int8_gemv_kernel(Int8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  int* sums = reinterpret_cast<int*>(smem + i8v::kRing);  // [token][pitch]
  float* sw = reinterpret_cast<float*>(smem + i8v::kRing + i8v::kSumBytes);  // the batch's scales, and biases
  float* add = sw + i8v::kMaxRows;
  float* sx = add + i8v::kMaxRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * i8v::kDepth * i8v::kStage;
  // a stage's 1 KB for 64 elements of K: rows 0 .. 7, then 8 .. 15, of each 4 pieces of 8 rows, piece p's rows turned by
  // 2 p, so that neither the copies nor the fragments' reads meet in a bank
  const uint32_t to = ring + (lane & 24) * 16 + ((lane + 2 * (lane >> 3)) & 7) * 16;
  const uint32_t from = ring + c * 128 + ((r + 2 * c) & 7) * 16;
  const int pitch = 16 * a.batch + 4;  // a lane's sums, rows r and r + 8 of tokens 2 c and 2 c + 1, in different banks
  const int groups = (a.N + 15) / 16, per = groups / gridDim.x, extra = groups - per * gridDim.x;
  const int g0 = blockIdx.x * per + min((int)blockIdx.x, extra), g1 = g0 + per + ((int)blockIdx.x < extra ? 1 : 0);
  const int streams = i8v::kWarps / a.wk, stream = warp / a.wk;
  const long long block_bytes = (long long)((a.K + 127) / 128) * i8::kSquare;
  uint64_t first, normal;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  const uint64_t policy = a.once ? first : normal;

  // The warp's stages in order: batches, passes, groups.  `at` walks them twice: once to copy, once to use.
  struct At {
    int b0, pass, g;  // the batch's first group; the group
  };
  const auto batch_end = [&](const At& s) { return min(s.b0 + a.batch, g1); };
  const auto valid = [&](const At& s) { return s.b0 < g1; };
  const auto settle = [&](At& s) {  // the stream may have no group in a short batch
    while (valid(s) && s.g >= batch_end(s)) {
      if (++s.pass == a.passes) s.pass = 0, s.b0 += a.batch;
      s.g = s.b0 + stream;
    }
  };
  const auto k_of = [&](int pass) { return (pass * a.wk + warp % a.wk) * a.slice; };  // the slice's first element
  const auto copy = [&](const At& s, int slot) {
    const int k0 = k_of(s.pass);
    const uint8_t* p = a.packed + (s.g >> 3) * block_bytes + (long long)(k0 / 16 + (lane >> 3)) * 2048 + ((s.g & 7) * 16 + (lane & 7)) * 16;
    const uint32_t d = to + slot * i8v::kStage;
#pragma unroll
    for (int b = 0; b < i8v::kBlocks; ++b)
      if (64 * b < a.slice && k0 + 64 * b < a.K) {
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d + b * 1024), "l"(p + b * 8192), "l"(policy) : "memory");
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d + b * 1024 + 512), "l"(p + b * 8192 + 128), "l"(policy) : "memory");
      }
  };
  At ahead{g0, 0, g0 + stream}, now = ahead;
  settle(ahead);
  settle(now);
  int slot_in = 0, slot = 0;
  const auto push = [&] {
    if (valid(ahead)) {
      copy(ahead, slot_in);
      ahead.g += streams;
      settle(ahead);
    }
    slot_in = slot_in == i8v::kDepth - 1 ? 0 : slot_in + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // The matrix is no kernel's output: its copies start before the wait for the kernel before.  One stage of them: what is
  // asked for after two, 20 MB over the machine, comes 3 us later, and the tokens are wanted first (4096 x 4096, 1 token,
  // from memory 8.2 us).
  push();
  for (int i = threadIdx.x; i < 8 * kTiles * pitch; i += i8v::kThreads) sums[i] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  uint32_t x[kTiles][i8v::kBlocks][8];  // B fragments: lane (n = r, c) holds elements 16 c .. 16 c + 15 of each 64 of token n
  const auto load_x = [&](int pass, uint4 (&v)[kTiles][i8v::kBlocks]) {
    const int k0 = k_of(pass);
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int b = 0; b < i8v::kBlocks; ++b) {
        const int t = 8 * n + r, k = k0 + 64 * b + 16 * c;
        v[n][b] = make_uint4(0u, 0u, 0u, 0u);
        if (t < a.T && 64 * b < a.slice && k < a.K) v[n][b] = *reinterpret_cast<const uint4*>(a.x + t * a.ldx + k);
      }
  };
  const auto convert_x = [&](const uint4 (&v)[kTiles][i8v::kBlocks]) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int b = 0; b < i8v::kBlocks; ++b) bytes_to_f16(biased(v[n][b]), x[n][b]);
  };
  int loaded = 0;
  {
    uint4 v[kTiles][i8v::kBlocks];
    load_x(0, v);
    const float s = threadIdx.x < a.T ? a.x_scale[threadIdx.x] : 0.f;
#pragma unroll
    for (int i = 1; i < i8v::kDepth - 1; ++i) push();
    if (threadIdx.x < a.T) sx[threadIdx.x] = s;
    convert_x(v);
  }
  __syncthreads();

  for (int b0 = g0; b0 < g1; b0 += a.batch) {
    const int rows = 16 * (min(b0 + a.batch, g1) - b0), f0 = 16 * b0;
    for (int i = threadIdx.x; i < rows; i += i8v::kThreads)
      if (f0 + i < a.N) sw[i] = a.w_scale[f0 + i], add[i] = a.bias ? a.bias[f0 + i] : 0.f;
    while (valid(now) && now.b0 == b0) {
      if (now.pass != loaded) {
        uint4 v[kTiles][i8v::kBlocks];
        load_x(loaded = now.pass, v);
        convert_x(v);
      }
      push();
      asm volatile("cp.async.wait_group %0;" ::"n"(i8v::kDepth - 1) : "memory");
      __syncwarp();  // every lane's copies
      float acc[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      const int k0 = k_of(now.pass);
#pragma unroll
      for (int b = 0; b < i8v::kBlocks; ++b)
        if (64 * b < a.slice && k0 + 64 * b < a.K) {
          uint32_t lo[8], hi[8];
          // lane (r, c): rows r and r + 8, elements 16 c .. 16 c + 15 of the 64
          bytes_to_f16(lds128(from + slot * i8v::kStage + b * 1024), lo);
          bytes_to_f16(lds128(from + slot * i8v::kStage + b * 1024 + 512), hi);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
              mma_f16(acc[n], lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1], x[n][b][2 * j], x[n][b][2 * j + 1]);
        }
      slot = slot == i8v::kDepth - 1 ? 0 : slot + 1;
      int* s = sums + 2 * c * pitch + (now.g - b0) * 16 + r;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (8 * n + 2 * c + (i & 1) < a.T) atomicAdd(s + (8 * n + (i & 1)) * pitch + 8 * (i >> 1), __float2int_rn(acc[n][i]));
      now.g += streams;
      settle(now);
    }
    __syncthreads();
    // two features a thread
    for (int i = threadIdx.x; i < rows / 2 * a.T; i += i8v::kThreads) {
      const int t = i / (rows / 2), n = 2 * (i - t * (rows / 2));
      int2* at = reinterpret_cast<int2*>(sums + t * pitch + n);
      const int2 v = *at;
      *at = make_int2(0, 0);
      if (f0 + n < a.N)
        store_out(a, t * a.ldo + f0 + n, fmaf((float)v.x, sx[t] * sw[n], add[n]), fmaf((float)v.y, sx[t] * sw[n + 1], add[n + 1]));
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------------------------------------------------------------
// More tokens: a persistent tcgen05 GEMM, the matrix as the M operand and the tokens as the N operand.
//
// The matrix is converted on the way, a square's rows into tensor memory, a thread its own lane.  Up to 64 tokens so are
// the tokens, into 128B-swizzled shared memory; more are written as FP16 to the handle's workspace by a kernel of its own
// first and come by TMA: converted again for every 256 features, by whichever warps, they were what the MMAs waited for
// (16384 tokens of 12576 x 4096 1286 us).
//
// kCtas = 2: a pair of CTAs on 256 features, each with half of the tile's tokens.  192 tokens, and not 256, because tensor
// memory then holds two sets of sums (384 columns) beside four stages of the matrix (128): the sums go to registers every
// 1024 elements, to stay exact, and that passes under the next 1024's MMAs.
//
// A warp takes some 370 cycles for its 32 rows of 64 elements, most of it waiting, and the MMAs of 192 tokens 384.  With
// fewer tokens, where the matrix's bytes are what there is to wait for, two teams of four warps take turns.  So does the
// issuer take 80 cycles a wait and 50 a commit, next to 30 an MMA: with both for every four MMAs it was what all variants
// waited for (460 cycles for 64 elements), and where tensor memory has the room a stage is a whole square.
//
// kSplit: where there are few units, a cluster of CTAs takes one, a share of the reduction each, and adds the integers
// through distributed shared memory.
//
// 16384 tokens of 12576 x 4096 take 952 us by themselves, 1.77 PFLOP/s with the tokens' conversion, and 1046 to 1058 among
// calls that keep the card at its power limit, 1.60 to 1.61; a library's BF16 product runs at 1.74 when sustained.
// --------------------------------------------------------------------------------------------------------------------
namespace i8g {
constexpr int kEpiWarps = 8;
constexpr int kCtlBytes = 2048, kEpiBytes = 2048;  // per epilogue warp
constexpr int kRingOff = kCtlBytes + kEpiWarps * kEpiBytes;
constexpr int kRoom = i8::kSmemMax - 1024 - kRingOff;
constexpr int kSegment = 8;                        // squares whose sums FP32 holds exactly
constexpr int kStagesA = 4;                        // of the matrix, in tensor memory: 32 columns for 64 elements
constexpr int kMaxStages = 4, kMaxRaw = 8, kMaxSplit = 8;

template <int kCtas, int kTile>
struct Plan {
  static constexpr bool kPre = kTile > 64;                   // tokens come in FP16
  static constexpr int kTeams = kTile == 192 ? 1 : 2;        // of four warps that convert the matrix
  static constexpr int kTokenWarps = kPre ? 0 : 4;           // that convert tokens, half of them a team
  // warps: converters of the matrix, epilogue, converters of tokens, matrix producer, token producer, MMA issuer
  static constexpr int kRowWarps = 4 * kTeams, kToken0 = kRowWarps + kEpiWarps, kProducer = kToken0 + kTokenWarps;
  static constexpr int kTokens = kProducer + 1, kIssuer = kTokens + 1, kThreads = 32 * (kIssuer + 1);
  static constexpr int kShare = kTile / kCtas;               // tokens of a CTA
  static constexpr int kBBytes = kShare * 256;               // a stage of them, 128 elements in FP16: two halves of 64
  static constexpr int kXBytes = kPre ? 0 : kShare * 128;    // a raw slot of them, 128 elements in bytes
  static constexpr int kStagesB = kTile == 128 ? 3 : 4;
  static constexpr int kRaw = 6;                             // raw slots, squares
  static constexpr int kHalves = kTile == 192 ? 1 : 2;       // of a square in a stage of the matrix, 64 elements each
  static constexpr uint32_t kOperand = 2 * kTile;            // the matrix's first column in tensor memory
  static constexpr int kRings = kStagesB * kBBytes + kRaw * (kXBytes + i8::kSquare);
  static_assert(kRings <= kRoom && kRaw <= kMaxRaw && kStagesB <= kMaxStages && 2 * kTile + 32 * kHalves * kStagesA <= 512, "rings");
  static_assert(kBBytes % 2048 == 0 && (kPre || (kStagesB == kStagesA && kHalves == 2)), "128B-swizzled tiles");
  // a team meets every slot of a ring again itself: a parity wait must not run two phases ahead of its barrier
  static_assert(kRaw % kTeams == 0 && kStagesA % kTeams == 0 && (kTeams == 1 || kHalves == 2), "teams");
};
}  // namespace i8g

struct Int8Ctl {
  uint64_t raw_full[i8g::kMaxRaw], raw_empty[i8g::kMaxRaw];      // a square (and its tokens' bytes)
  uint64_t a_full[i8g::kStagesA], a_empty[i8g::kStagesA];        // converted stages (and their tokens)
  uint64_t b_full[i8g::kMaxStages], b_empty[i8g::kMaxStages];    // tokens in FP16
  uint64_t acc_full[2], acc_empty[2], mma_done;
  uint32_t tmem;
  int abort_flag;
};
static_assert(sizeof(Int8Ctl) <= i8g::kCtlBytes, "control block");

template <int kCtas, int kTile, bool kSplit>
__global__ void __launch_bounds__((i8g::Plan<kCtas, kTile>::kThreads), 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap x_map, Int8Args a) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  Int8Ctl& ctl = *reinterpret_cast<Int8Ctl*>(smem);
  using Plan = i8g::Plan<kCtas, kTile>;
  uint8_t* ring_b = smem + i8g::kRingOff;
  uint8_t* raw_x = ring_b + Plan::kStagesB * Plan::kBBytes;
  uint8_t* raw_w = raw_x + Plan::kRaw * Plan::kXBytes;
  const uint32_t b_addr = smem_u32(ring_b), x_addr = smem_u32(raw_x), w_addr = smem_u32(raw_w);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(!kSplit || kCtas == 1, "a cluster is a pair or shares a unit");
  const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
  const int part = kSplit ? (int)cluster_rank() : 0;
  const int first = kSplit ? blockIdx.x / a.split : blockIdx.x / kCtas;
  const int stride = kSplit ? gridDim.x / a.split : gridDim.x / kCtas;  // split: no CTA has a second unit
  const int squares = a.squares;
  const int sq0 = kSplit ? part * squares / a.split : 0, sq1 = kSplit ? (part + 1) * squares / a.split : squares;
  const int steps = sq1 - sq0;        // squares
  constexpr int kRound = 16 * kCtas;  // the MMA's columns come in these
  const int total = a.tiles * a.NU;
  volatile int* abort_flag = &ctl.abort_flag;

  if (threadIdx.x == 0) {
    constexpr int kConverters = 4 + Plan::kTokenWarps / Plan::kTeams;  // warps that convert a square
    for (int s = 0; s < Plan::kRaw; ++s) {
      mbar_init(ctl.raw_full + s, 1);
      mbar_init(ctl.raw_empty + s, kConverters);
    }
    for (int s = 0; s < i8g::kStagesA; ++s) {
      mbar_init(ctl.a_full + s, kCtas * kConverters);  // waited for by the pair's first CTA
      mbar_init(ctl.a_empty + s, 1);
    }
    for (int s = 0; s < Plan::kStagesB; ++s) {
      mbar_init(ctl.b_full + s, 1);  // the same
      mbar_init(ctl.b_empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(ctl.acc_full + b, 1);
      mbar_init(ctl.acc_empty + b, kCtas * i8g::kEpiWarps);
    }
    mbar_init(&ctl.mma_done, 1);
    ctl.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == Plan::kIssuer) {
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
  tc_fence_before();
  __syncthreads();
  if (kCtas == 2) cluster_sync_all();  // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // Unit u: feature block(s) u % NU of token tile u / NU.
  const auto tokens_of = [&](int u, int& row0) {
    const int t = u / a.NU;
    row0 = t * a.per;
    return min(a.per, a.T - row0);
  };
  const auto columns = [&](int tokens) { return (tokens + kRound - 1) & ~(kRound - 1); };

  int acc[kTile / 2];  // epilogue: a feature's sums over half of the columns (kSplit: until after the roles have met again)

  if (warp == Plan::kProducer) {
    // ---------------- the matrix's squares, and the bytes of the tokens that meet them ----------------
    uint32_t it = 0;
    RingPos p;
    bool ok = true, waited = false;
    for (int u = first; u < total && ok && a.fault != 1; u += stride) {
      int row0;
      tokens_of(u, row0);
      // the last pair of an odd number of blocks: the second CTA computes the first one's block again, unstored
      const int nb = min(u % a.NU * kCtas + rank, a.NB - 1);
      const uint8_t* src = a.packed + ((long long)nb * squares + sq0) * i8::kSquare;
      for (int s = sq0; s < sq1; ++s, ++it, p.step(Plan::kRaw), src += i8::kSquare) {
        if (!warp_wait(ctl.raw_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 931)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(ctl.raw_full + p.slot, i8::kSquare + Plan::kXBytes);
          bulk_g2s(raw_w + p.slot * i8::kSquare, src, i8::kSquare, ctl.raw_full + p.slot);
        }
        __syncwarp();
        if constexpr (!Plan::kPre) {
          // the tokens may be the kernel before's, the matrix is not
          if (!waited) grid_dependency_wait();
          waited = true;
          if (elect_one()) tma_2d(raw_x + p.slot * Plan::kXBytes, &x_map, s * 128, row0, ctl.raw_full + p.slot);
          __syncwarp();
        }
      }
    }
    if (lane == 0) drain_copies(ctl.raw_full, it, Plan::kRaw);
  } else if (warp == Plan::kTokens) {
    // ---------------- tokens in FP16: this CTA's half of the tile, 128 elements a stage ----------------
    if constexpr (Plan::kPre) {
      grid_dependency_wait();
      uint32_t it = 0;
      RingPos p;
      bool ok = true;
      for (int u = first; u < total && ok && a.fault != 1; u += stride) {
        int row0;
        const int share = columns(tokens_of(u, row0)) / kCtas;
        row0 += rank * share;
        for (int s = sq0; s < sq1; ++s, ++it, p.step(Plan::kStagesB)) {
          if (!warp_wait(ctl.b_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 937)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            uint8_t* dst = ring_b + p.slot * Plan::kBBytes;
            if (rank == 0) mbar_arrive_expect_tx(ctl.b_full + p.slot, (uint32_t)(kCtas * Plan::kBBytes));
            const uint32_t bar0 = kCtas == 2 ? map_rank(ctl.b_full + p.slot, 0) : 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (kCtas == 2) tma_2d_pair(dst + h * (Plan::kBBytes / 2), &x_map, s * 128 + h * 64, row0, bar0);
              else tma_2d(dst + h * (Plan::kBBytes / 2), &x_map, s * 128 + h * 64, row0, ctl.b_full + p.slot);
            }
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        if (rank == 0) drain_copies(ctl.b_full, it, Plan::kStagesB);
        else if (!ok)
          for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // its copies complete on the first CTA's barriers
      }
    }
  } else if (warp == Plan::kIssuer) {
    // ---------------- MMA issuer: the whole warp walks the loop, one lane issues ----------------
    if (rank == 0) {
      uint32_t j = 0;  // segments so far
      RingPos pa, pb;
      bool ok = true;
      for (int u = first; u < total && ok; u += stride) {
        int row0;
        const uint32_t idesc = idesc_f16(128 * kCtas, columns(tokens_of(u, row0)));
        for (int s = 0; s < steps && ok; s += i8g::kSegment, ++j) {
          const uint32_t buf = j & 1u;
          if (!warp_wait(ctl.acc_empty + buf, ((j >> 1) & 1u) ^ 1u, abort_flag, a.st, 932)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + buf * kTile;
          const int end = min(s + i8g::kSegment, steps);
          uint32_t add = 0;
          for (int i = s; i < end && ok; ++i, pb.step(Plan::kStagesB)) {
            if (Plan::kPre && !warp_wait(ctl.b_full + pb.slot, pb.phase, abort_flag, a.st, 938)) {
              ok = false;
              break;
            }
            const uint64_t bd = sw128_desc(b_addr + (uint32_t)(pb.slot * Plan::kBBytes));
#pragma unroll
            for (int g = 0; g < 2 / Plan::kHalves; ++g, pa.step(i8g::kStagesA)) {
              if (!warp_wait(ctl.a_full + pa.slot, pa.phase, abort_flag, a.st, 933)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t at = tmem + Plan::kOperand + (uint32_t)(pa.slot * 32 * Plan::kHalves);  // 8 columns per 16 elements
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4 * Plan::kHalves; ++kk) {
                  const int k = 4 * g + kk;  // of the square's 8
                  const uint64_t bk = bd + (uint32_t)((k >> 2) * (Plan::kBBytes / 2) >> 4) + 2u * (k & 3);
                  if (kCtas == 2) umma_ts_pair(d, at + 8u * kk, bk, idesc, k ? 1u : add);
                  else umma_ts(d, at + 8u * kk, bk, idesc, k ? 1u : add);
                }
                if (kCtas == 2) umma_commit_pair(ctl.a_empty + pa.slot);
                else umma_commit(ctl.a_empty + pa.slot);
                if (Plan::kPre && g == 2 / Plan::kHalves - 1) {
                  if (kCtas == 2) umma_commit_pair(ctl.b_empty + pb.slot);
                  else umma_commit(ctl.b_empty + pb.slot);
                }
              }
              __syncwarp();
            }
            add = 1;
          }
          if (!ok) break;
          if (elect_one()) {
            if (kCtas == 2) umma_commit_pair(ctl.acc_full + buf);
            else umma_commit(ctl.acc_full + buf);
          }
          __syncwarp();
        }
      }
      // no MMA may outlive the shared and tensor memory it uses, also where a role has given up
      if (elect_one()) {
        if (kCtas == 2) umma_commit_pair_own(&ctl.mma_done);
        else umma_commit(&ctl.mma_done);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(&ctl.mma_done, 0) && globaltimer_ns() - t0 <= kWaitTimeoutNs) {}
      }
      __syncwarp();
    }
  } else if (warp < Plan::kRowWarps || warp >= Plan::kToken0) {
    // ---------------- converters: a raw slot makes a stage or two; the teams take turns at the slots ----------------
    const bool rows = warp < Plan::kRowWarps;
    constexpr int kTeamTokens = Plan::kPre ? 1 : Plan::kTokenWarps / Plan::kTeams;  // a team's warps for tokens
    constexpr int kOctets = Plan::kPre ? 1 : Plan::kShare / 8 / kTeamTokens;        // of 8 tokens, of one of them
    const int team = rows ? warp / 4 : (warp - Plan::kToken0) / kTeamTokens;
    const int w0 = rows ? warp % 4 : (warp - Plan::kToken0) % kTeamTokens;
    const uint32_t lanes = (uint32_t)(32 * w0) << 16;
    const uint32_t full0 = kCtas == 2 ? map_rank(ctl.a_full, 0) : 0u;  // the pair's first CTA's
    const int all = first < total ? ((total - first - 1) / stride + 1) * (sq1 - sq0) : 0;  // squares of this CTA
    RingPos raw, p;
    raw.slot = p.slot = team;
    const auto tell = [&] {  // the stage is written
      __syncwarp();
      if (lane == 0) {
        if (kCtas == 2 && rank) mbar_arrive_cluster(full0 + p.slot * 8);
        else mbar_arrive(ctl.a_full + p.slot);
      }
    };
    bool ok = true;
    for (int n = team; n < all && ok; n += Plan::kTeams, raw.step(Plan::kRaw, Plan::kTeams)) {
      if (!warp_wait(ctl.raw_full + raw.slot, raw.phase, abort_flag, a.st, 934)) break;
      if (rows) {
        const uint32_t slot = w_addr + raw.slot * i8::kSquare + (uint32_t)(32 * w0 + lane) * 16u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[4][8];
#pragma unroll
          for (int i = 0; i < 4; ++i) bytes_to_f16(lds128(slot + (4 * h + i) * 2048), v[i]);
          if (Plan::kHalves == 1 || h == 0) {
            if (!warp_wait(ctl.a_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 935)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          tmem_st32(tmem + lanes + Plan::kOperand + (uint32_t)(p.slot * 32 * Plan::kHalves) + (Plan::kHalves == 2 ? 32u * h : 0u), v);
          if (Plan::kHalves == 1 || h == 1) {
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            tell();
            p.step(i8g::kStagesA, Plan::kTeams);
          }
        }
      } else if constexpr (!Plan::kPre) {
        // 8 tokens of 16 elements a quarter of a warp; all lie in banks of their own, going in and coming out.  All
        // reads first: there is no other warp to hide what one takes
        const uint32_t slot = x_addr + raw.slot * Plan::kXBytes;
        uint4 x[2][kOctets];
        const int q = lane >> 3, m = lane & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int o = 0; o < kOctets; ++o)
            x[h][o] = lds128(slot + (uint32_t)(8 * (w0 + kTeamTokens * o) + m) * 128u + (uint32_t)((4 * h + q) ^ m) * 16u);
        if (!warp_wait(ctl.a_empty + p.slot, p.phase ^ 1u, abort_flag, a.st, 939)) break;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int o = 0; o < kOctets; ++o) {
            const uint32_t row = b_addr + (uint32_t)(p.slot * Plan::kBBytes + h * (Plan::kBBytes / 2)) +
                                 (uint32_t)(8 * (w0 + kTeamTokens * o) + m) * 128u;
            uint32_t u[8];
            bytes_to_f16(biased(x[h][o]), u);
            sts128(row + (uint32_t)((2 * q) ^ m) * 16u, u[0], u[1], u[2], u[3]);
            sts128(row + (uint32_t)((2 * q + 1) ^ m) * 16u, u[4], u[5], u[6], u[7]);
          }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tell();
        p.step(i8g::kStagesA, Plan::kTeams);
      }
      // what was read of the slot has been stored since
      if (ok && lane == 0) mbar_arrive(ctl.raw_empty + raw.slot);
    }
  } else {
    // ---------------- epilogue: warp w reads TMEM lanes 32 (w % 4) .., one feature a lane, and half of the columns; two
    // warps a quarter.  32 tokens x 32 features go through shared memory into 16-byte stores ----------------
    const int quarter = warp & 3, half = (warp - Plan::kRowWarps) >> 2;
    const uint32_t t_acc = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(half * (kTile / 2));
    uint8_t* buf_s = smem + i8g::kCtlBytes + (warp - Plan::kRowWarps) * i8g::kEpiBytes;
    if (!kSplit) grid_dependency_wait();  // x's scales, and what the output's memory holds, may be the kernel before's
    uint32_t j = 0;
    bool ok = true;
    for (int u = first; u < total && ok; u += stride) {
      int row0;
      const int tokens = tokens_of(u, row0);
#pragma unroll
      for (int i = 0; i < kTile / 2; ++i) acc[i] = 0;
      for (int s = 0; s < steps; s += i8g::kSegment, ++j) {
        const uint32_t buf = j & 1u;
        if (!warp_wait(ctl.acc_full + buf, (j >> 1) & 1u, abort_flag, a.st, 936)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // (columns past the tile's last: unwritten, not stored)
#pragma unroll
        for (int i = 0; i < kTile / 2; i += 16) {
          uint32_t v[16];
          tmem_ld16_nw(t_acc + buf * kTile + i, v);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int k = 0; k < 16; ++k) acc[i + k] += __float2int_rn(__uint_as_float(v[k]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 2) mbar_arrive_cluster(map_rank(ctl.acc_empty + buf, 0));
          else mbar_arrive(ctl.acc_empty + buf);
        }
      }
      if (!ok || kSplit) break;
      const int f0 = 128 * (u % a.NU * kCtas + rank) + 32 * quarter;  // beyond N for a block computed twice
      if (f0 >= a.N) continue;
      const float sw = f0 + lane < a.N ? __ldg(a.w_scale + f0 + lane) : 0.f;
      const float add = a.bias && f0 + lane < a.N ? __ldg(a.bias + f0 + lane) : 0.f;
      // 16 bytes a lane: FP32 4 tokens of 8 lanes at a time, else 8 of 4
      const bool f32 = a.out_type == 1;
      const int row = f32 ? lane >> 3 : lane >> 2, f = f32 ? 4 * (lane & 7) : 8 * (lane & 3), size = f32 ? 4 : 2;
      const long long step = a.ldo * 16;  // bytes from 4, or 8, tokens to the next
      int left = f0 + f < a.N ? tokens - half * (kTile / 2) - row : 0;
      const float* sx = a.x_scale + row0 + half * (kTile / 2);
      uint8_t* out = static_cast<uint8_t*>(a.out) + ((long long)(row0 + half * (kTile / 2) + row) * a.ldo + f0 + f) * size;
      const uint8_t* from = buf_s + row * (32 * size) + f * size;
#pragma unroll
      for (int col = 0; col < kTile / 2; col += 16) {
        if (half * (kTile / 2) + col >= tokens) break;
        __syncwarp();
        const float sx_lane = half * (kTile / 2) + col + (lane & 15) < tokens ? sx[col + (lane & 15)] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float y = fmaf((float)acc[col + i], sw * __shfl_sync(0xffffffffu, sx_lane, i), add);
          if (f32) *reinterpret_cast<float*>(buf_s + i * 128 + lane * 4) = y;
          else if (a.out_type == 2) *reinterpret_cast<__half*>(buf_s + i * 64 + lane * 2) = __float2half_rn(y);
          else *reinterpret_cast<__nv_bfloat16*>(buf_s + i * 64 + lane * 2) = __float2bfloat16_rn(y);
        }
        __syncwarp();
        // (a loop: as 96 tokens' addresses it would not fit the registers)
#pragma unroll 1
        for (int i = 0; i < 16; i += f32 ? 4 : 8, out += step, left -= f32 ? 4 : 8)
          if (left > 0) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(from + i * (32 * size));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  grid_launch_dependents();
  if (kCtas == 2) cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if constexpr (kSplit) {
    int row0 = 0;
    const int tokens = first < total ? tokens_of(first, row0) : 0;
    int* sums = reinterpret_cast<int*>(ring_b);  // [token][128 features]; the copies and MMAs are done with the rings
    if (warp >= Plan::kRowWarps && warp < Plan::kToken0 && tokens && !*abort_flag) {
      const int half = (warp - Plan::kRowWarps) >> 2, t0 = half * (kTile / 2);
#pragma unroll
      for (int i = 0; i < kTile / 2; ++i)
        if (t0 + i < tokens) sums[(t0 + i) * 128 + 32 * (warp & 3) + lane] = acc[i];
    }
    cluster_sync_all();
    grid_dependency_wait();
    const int f = 128 * (first % a.NU) + 4 * lane;
    if (f < a.N) {
      const float4 sw = *reinterpret_cast<const float4*>(a.w_scale + f);
      const float4 add = a.bias ? *reinterpret_cast<const float4*>(a.bias + f) : make_float4(0.f, 0.f, 0.f, 0.f);
      for (int t = warp * a.split + part; t < tokens; t += Plan::kThreads / 32 * a.split) {
        int4 n = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < i8g::kMaxSplit; ++c)
          if (c < a.split) {
            const float4 v = ld_cluster(reinterpret_cast<const float*>(sums + t * 128 + 4 * lane), c);
            n.x += __float_as_int(v.x), n.y += __float_as_int(v.y), n.z += __float_as_int(v.z), n.w += __float_as_int(v.w);
          }
        const float sx = a.x_scale[row0 + t];
        const float y[4] = {fmaf((float)n.x, sw.x * sx, add.x), fmaf((float)n.y, sw.y * sx, add.y),
                            fmaf((float)n.z, sw.z * sx, add.z), fmaf((float)n.w, sw.w * sx, add.w)};
        const long long o = (long long)(row0 + t) * a.ldo + f;
        if (a.out_type == 1) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
          uint32_t w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
            w[i] = a.out_type == 2 ? *reinterpret_cast<const uint32_t*>(&h) : *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) = make_uint2(w[0], w[1]);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while its sums are read
  }
  if (warp == Plan::kIssuer) {
    tc_fence_after();
    if (kCtas == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// --------------------------------------------------------------------------------------------------------------------
// Launches
// --------------------------------------------------------------------------------------------------------------------
typedef void (*Int8Gemm)(const CUtensorMap, Int8Args);
struct Int8Variant {
  Int8Gemm fn;
  int ctas, tile, threads;
  bool split;
  double square, base;  // us that a square takes a unit, and that a call takes beside its squares, measured
};
template <int kCtas, int kTile, bool kSplit>
static constexpr Int8Variant int8_variant(double square, double base) {
  return {int8_gemm_kernel<kCtas, kTile, kSplit>, kCtas, kTile, i8g::Plan<kCtas, kTile>::kThreads, kSplit, square, base};
}
static const Int8Variant kInt8Variants[] = {int8_variant<1, 64, false>(0.35, 3.2), int8_variant<1, 128, false>(0.48, 3.2),
                                            int8_variant<2, 192, false>(0.53, 4.5), int8_variant<1, 64, true>(0.35, 4.3),
                                            int8_variant<1, 128, true>(0.48, 5.0)};

// Tokens as FP16: a thread 16 elements, zeros from K on.
__global__ void __launch_bounds__(256) int8_tokens_kernel(const int8_t* x, long long ldx, int T, int K, int Kp, uint16_t* out) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int pieces = Kp / 16;
  const long long n = (long long)T * pieces;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int t = (int)(i / pieces), k = 16 * (int)(i - (long long)t * pieces);
    uint32_t v[8];
    bytes_to_f16(biased(k < K ? *reinterpret_cast<const uint4*>(x + t * ldx + k) : make_uint4(0u, 0u, 0u, 0u)), v);
    uint4* o = reinterpret_cast<uint4*>(out + (long long)t * Kp + k);
    o[0] = make_uint4(v[0], v[1], v[2], v[3]);
    o[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

static cudaError_t set_int8_attrs() {  // once per device
  constexpr int kCached = 64;
  static std::mutex mu;
  static bool done[kCached] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < kCached && done[dev]) return cudaSuccess;
  for (const Int8Variant& v : kInt8Variants) {
    e = cudaFuncSetAttribute((const void*)v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, i8::kSmemMax);
    if (e != cudaSuccess) return e;
  }
  e = cudaFuncSetAttribute((const void*)int8_gemv_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, i8::kSmemMax);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)int8_gemv_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, i8::kSmemMax);
  if (e == cudaSuccess && dev >= 0 && dev < kCached) done[dev] = true;
  return e;
}

static Int8Args args_of(const Int8Product& p) {
  Int8Args a{};
  a.packed = p.packed, a.w_scale = p.w_scale, a.bias = p.bias;
  a.N = p.N, a.K = p.K, a.T = p.T;
  a.x = p.x, a.x_scale = p.x_scale, a.ldx = p.ldx;
  a.out = p.out, a.ldo = p.ldo, a.out_type = p.out_type;
  a.once = p.once, a.st = p.status, a.fault = p.fault;
  return a;
}

cudaError_t launch_int8_gemv(const Int8Product& p, cudaStream_t st) {
  cudaError_t e = set_int8_attrs();
  if (e != cudaSuccess) return e;
  Int8Args a = args_of(p);
  const int blocks = (a.K + 63) / 64;
  a.wk = 1;
  while (a.wk < i8v::kWarps && a.wk * i8v::kBlocks < blocks) a.wk *= 2;
  a.passes = (blocks + a.wk * i8v::kBlocks - 1) / (a.wk * i8v::kBlocks);
  a.slice = (blocks + a.wk * a.passes - 1) / (a.wk * a.passes) * 64;
  const int groups = (a.N + 15) / 16, tokens = a.T <= 8 ? 8 : 16;
  const int ctas = std::min(groups, p.num_sms);
  a.batch = std::min((i8v::kSumBytes / 4 / tokens - 4) / 16, (groups + ctas - 1) / ctas);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(i8v::kThreads);
  cfg.dynamicSmemBytes = i8v::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return a.T <= 8 ? cudaLaunchKernelEx(&cfg, int8_gemv_kernel<1>, a) : cudaLaunchKernelEx(&cfg, int8_gemv_kernel<2>, a);
}

int int8_chunk_tokens(int K) {
  const int Kp = (K + 127) / 128 * 128;
  return std::max(192, (1 << 27) / Kp / 192 * 192);
}
size_t int8_workspace_bytes(int K, int max_tokens) {
  return max_tokens > 64 ? sizeof(uint16_t) * ((K + 127) / 128 * 128) * std::min(max_tokens, int8_chunk_tokens(K)) : 0;
}

Int8Tiling int8_tiling(int N, int K, int T, int num_sms) {
  // The variant whose rounds of units take the least time by what was measured of each: its squares, 0.6 us a unit, and its
  // base, with 2 us and the bytes at 6 TB/s where the tokens are converted first.  Of the variants in that order, us, for
  // 12576 x 4096 and 64 tokens 15 / - / -, 128 26 / 21 / 24, 256 37 / 36 / 40, 512 70 / 51 / 42, 2048 - / 172 / 140; for
  // 4096 x 4096 and 64 tokens 15 whole, 10 and 9 with 2 and 4 CTAs a unit; 128 tokens 11 with tiles of 64 and 2 CTAs, 13
  // of 128 and 4.  Clusters of 4 fit the machine 36 at a time, of 8 some 13 (512 x 4096, 192 tokens, 12 units of 8 CTAs
  // 7.5 us, 256 tokens, 16 units, 13.5).
  const int blocks = (N + 127) / 128, squares = (K + 127) / 128;
  Int8Tiling best{};
  double least = 1e300;
  for (int i = 0; i < (int)(sizeof(kInt8Variants) / sizeof(kInt8Variants[0])); ++i) {
    const Int8Variant& v = kInt8Variants[i];
    const long long units = (long long)((blocks + v.ctas - 1) / v.ctas) * ((T + v.tile - 1) / v.tile);
    const bool fp16 = v.tile > 64;
    if (fp16 && T <= 64) continue;  // calls of up to 64 tokens use no workspace
    for (int split = v.split ? 2 : 1; split <= (v.split ? i8g::kMaxSplit : 1); split *= 2) {
      const long long slots = num_sms * (split == 8 ? 11 : split > 1 ? 15 : 16) / 16 / (v.ctas * split);
      if (v.split && (units > slots || 2 * split > squares)) break;
      const long long rounds = (units + slots - 1) / slots;
      const double t = (double)rounds * ((squares + split - 1) / split * v.square + 0.6) + v.base +
                       (fp16 ? 2.0 + (double)T * squares * 128 * 3 / 6e6 : 0.0);
      if (t < least) least = t, best = {i, v.tile / v.ctas, split, fp16};
    }
  }
  return best;
}

cudaError_t launch_int8_gemm(const Int8Product& p, const Int8Tiling& t, const CUtensorMap& x_map, cudaStream_t st) {
  cudaError_t e = set_int8_attrs();
  if (e != cudaSuccess) return e;
  const Int8Variant& v = kInt8Variants[t.variant];
  Int8Args a = args_of(p);
  a.NB = (a.N + 127) / 128;
  a.NU = (a.NB + v.ctas - 1) / v.ctas;
  a.tiles = (a.T + v.tile - 1) / v.tile;
  const int round = 16 * v.ctas;
  a.per = ((a.T + a.tiles - 1) / a.tiles + round - 1) / round * round;  // tiles of one size, so that none is a small rest
  a.tiles = (a.T + a.per - 1) / a.per;
  a.squares = (a.K + 127) / 128;
  a.split = t.split;
  cudaLaunchConfig_t cfg{};
  const int units = a.tiles * a.NU;
  cfg.gridDim = dim3((unsigned)(t.split > 1 ? units * t.split : std::min(units, p.num_sms / v.ctas) * v.ctas));
  cfg.blockDim = dim3((unsigned)v.threads);
  cfg.dynamicSmemBytes = i8::kSmemMax;
  cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)(t.split > 1 ? t.split : v.ctas);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, v.fn, x_map, a);
}

cudaError_t launch_int8_tokens(const Int8Product& p, void* out, cudaStream_t st) {
  const int Kp = (p.K + 127) / 128 * 128;
  const long long threads = (long long)p.T * (Kp / 16);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min((threads + 255) / 256, (long long)p.num_sms * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_tokens_kernel, p.x, p.ldx, p.T, p.K, Kp, static_cast<uint16_t*>(out));
}

}  // namespace nvfp4moe
