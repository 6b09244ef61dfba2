// Routing on its own (nvfp4_route_forward / nvfp4_route_backward): scores, choice, weights and the tables that sort the
// routed rows by expert.
//   s_e = softmax of a token's logits, or 1 / (1 + e^-l_e);  c_e = s_e + bias_e, or the logit where there is no bias
//   groups: a group's value is its largest c, or the sum of its two largest (of s without a bias); the best `top_groups`
//           groups' experts are eligible
//   choice: the k largest c, largest first, the lower index first among equals; weights scale s_j (/ sum of the chosen)
//   tables: the T k routed rows t k + j by expert, ascending within one: offsets, perm, and its inverse
//
// The choice is that of c in 64 bits.  Comparing FP32 scores gives it wherever neighbours in the order are further apart
// than those scores can be wrong (2^-20 of the token's largest score for sigmoids, 2^-17 for softmax, whose sum is over
// all experts); a token where some are not, one in a few hundred on random logits, is chosen again from scores in 64
// bits.  Logits that are compared as they are need no such test.
//
// One warp a token, lane l with experts l V .. l V + V - 1, so that a lane's logits are one or two vector loads and the
// lowest index among equals is the lowest lane's.  A CTA takes a run of tokens; bit t of bits[e] says that its token t
// chose e, so that a row's place among its expert's is a population count, whatever the order the warps came in.  Few
// tokens: one CTA does it all.  Else a second kernel turns the runs' counts into places and a third scatters; the counts
// lie in `inv`, each run's in its own rows' part, which its CTA alone overwrites in the end, so that there is no
// workspace and calls may overlap.
#include <algorithm>

#include "kernels.h"
#include "route_common.cuh"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace rt {
constexpr int kMaxExperts = 512;
constexpr int kThreads = 512;
constexpr int kOneCta = 128;  // tokens up to which one CTA does it all
constexpr int kRun = 256;     // of a run, unless its counts need more
}  // namespace rt

struct RouteArgs {
  const void* logits;
  long long ld;       // elements
  int bf16, vec;      // vec: rows start on 16 bytes
  int T, E, k;
  int score, renorm;
  float scale;
  const float* bias;  // or NULL
  int groups, top_groups, group_top, group_size;
  int runs;           // CTAs' runs of tokens
  int words;          // 32-bit words of a run's bits per expert
  int32_t* ids;
  float* weights;
  int32_t *offsets, *perm, *inv;
  DeviceStatus* st;
  // backward
  const int32_t* cids;
  const float* dw;
  void* dl;
  long long ld_dl;
};

// Tokens t0 .. t1 - 1 of run b: of equal length, the first ones longer by one.
__device__ __forceinline__ void run_of(const RouteArgs& a, int b, int& t0, int& t1) {
  const int base = a.T / a.runs, extra = a.T - base * a.runs;
  t0 = b * base + min(b, extra);
  t1 = t0 + base + (b < extra ? 1 : 0);
}

// Lane's V logits of token t; beyond E: NaN, which no choice takes before a number.
template <int V>
__device__ __forceinline__ void load_lane(const RouteArgs& a, int t, float (&v)[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  const size_t at = (size_t)t * a.ld + e0;
  if (a.vec && e0 + V <= a.E) {
    if (a.bf16) {
      constexpr int kW = V >= 2 ? V / 2 : 1;
      uint32_t w[kW];
      const uint16_t* p = static_cast<const uint16_t*>(a.logits) + at;
      if constexpr (V >= 8) {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
          const uint4 q = reinterpret_cast<const uint4*>(p)[i];
          w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
      } else if constexpr (V == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
      } else if constexpr (V == 2) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        w[0] = *p;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    } else {
      const float* p = static_cast<const float*>(a.logits) + at;
      if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 q = reinterpret_cast<const float4*>(p)[i];
          v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
        }
      } else if constexpr (V == 2) {
        const float2 q = *reinterpret_cast<const float2*>(p);
        v[0] = q.x, v[1] = q.y;
      } else {
        v[0] = *p;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e0 + i < a.E ? load_logit(a.logits, a.bf16, at + i) : __uint_as_float(0x7FC00000u);
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Softmax over all of a token's logits, as the layer's (NaN counts as -inf).
template <class F>
struct Softmax {
  float top;
  F sum;
  int infinities;
};
template <class F, int V>
__device__ __forceinline__ Softmax<F> softmax_of(const float (&l)[V]) {
  Softmax<F> s;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);  // fmaxf drops NaNs
  s.top = warp_max(m);
  s.sum = 0;
  int n = 0;
  const bool finite = s.top != INFINITY && s.top != -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    n += l[i] == INFINITY;
    if (finite && l[i] == l[i]) s.sum += sizeof(F) == 8 ? (F)exp((double)l[i] - (double)s.top) : (F)expf(l[i] - s.top);
  }
  s.sum = warp_sum(s.sum);
  s.infinities = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  return s;
}
template <class F>
__device__ __forceinline__ F score_of(float l, int sigmoid, const Softmax<F>& s, int E) {
  if (l != l) return F(0);
  if (sigmoid) return sizeof(F) == 8 ? F(1.0 / (1.0 + exp(-(double)l))) : F(1.0f / (1.0f + expf(-l)));
  if (s.top == -INFINITY) return F(1) / F(E);
  if (s.top == INFINITY) return l == INFINITY ? F(1) / F(s.infinities) : F(0);
  return sizeof(F) == 8 ? F(exp((double)l - (double)s.top) / s.sum) : F(expf(l - s.top) / (float)s.sum);
}

// The larger two of a pair of sorted pairs.
template <class F>
__device__ __forceinline__ void merge_two(F& a, F& b, F c, F d) {
  const F lo = a < c ? a : c;
  a = a < c ? c : a;
  b = b < d ? d : b;
  b = b < lo ? lo : b;
}

// Lane g < groups: the value of group g over the c of its members (NaN counts as -inf), and the magnitudes that went in.
template <class F, int V>
__device__ __forceinline__ F group_value(const RouteArgs& a, const F (&c)[V], F* size) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  const F none = F(-INFINITY);
  F mine = none;
  for (int g = 0; g < a.groups; ++g) {
    const int lo = g * a.group_size, hi = lo + a.group_size;
    F x = none, y = none;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i >= lo && e0 + i < hi) merge_two(x, y, c[i] == c[i] ? c[i] : none, none);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const F x2 = __shfl_xor_sync(0xffffffffu, x, o), y2 = __shfl_xor_sync(0xffffffffu, y, o);
      merge_two(x, y, x2, y2);
    }
    if (lane == g) mine = a.group_top == 2 ? x + y : x, *size = a.group_top == 2 ? fabs(x) + fabs(y) : fabs(x);
  }
  return mine == mine ? mine : none;  // (infinities of both signs)
}

// The groups kept, one bit each.  `apart`: whether the last one in and the first one out are further apart than they can
// be wrong: `tol`, and 2^-21 of the magnitudes that they are made of.
template <class F>
__device__ __forceinline__ unsigned best_groups(const RouteArgs& a, F mine, F size, F tol, bool* apart) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const F v = __shfl_sync(0xffffffffu, mine, g);
    rank += v > mine || (v == mine && g < lane);
  }
  const bool in = lane < a.groups && rank < a.top_groups;
  const int l = __ffs(__ballot_sync(0xffffffffu, lane < a.groups && rank == a.top_groups - 1)) - 1;
  const int n = __ffs(__ballot_sync(0xffffffffu, lane < a.groups && rank == a.top_groups)) - 1;
  const F gap = __shfl_sync(0xffffffffu, mine, l) - __shfl_sync(0xffffffffu, mine, n);
  const F sizes = __shfl_sync(0xffffffffu, size, l) + __shfl_sync(0xffffffffu, size, n);
  *apart = gap > tol + sizes * F(0x1p-21);
  return __ballot_sync(0xffffffffu, in);
}

// Experts of the lane that may be chosen: bit i.
template <int V>
__device__ __forceinline__ unsigned eligible(const RouteArgs& a, unsigned groups) {
  const int e0 = (threadIdx.x & 31) * V;
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < a.E && (a.top_groups == a.groups || ((groups >> ((e0 + i) / a.group_size)) & 1u))) m |= 1u << i;
  return m;
}

// The value of an order key (NaN for a NaN's).
__device__ __forceinline__ float key_float(uint32_t key) {
  return key == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The k largest keys among those marked in `avail`, by rounds; lane j gets choice j's expert and logit.  `apart`: whether
// every one and the next differ by more than they can be wrong, tol and their own roundings; not looked at for tol < 0.
template <int V>
__device__ __forceinline__ void choose(const RouteArgs& a, const uint32_t (&key)[V], const float (&l)[V], unsigned avail,
                                       float tol, int* id, float* logit, bool* apart) {
  const int lane = threadIdx.x & 31;
  float before = INFINITY;
  bool ok = true;
  for (int j = 0; j <= a.k; ++j) {
    if (j == a.k && tol < 0.f) break;
    uint32_t best = 0;
    int at = -1;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (((avail >> i) & 1u) && (at < 0 || key[i] > best)) best = key[i], at = i;
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const unsigned who = __ballot_sync(0xffffffffu, at >= 0 && best == top);
    if (who == 0) break;  // fewer than k + 1 are eligible
    if (tol >= 0.f) {
      const float v = key_float(top);
      if (j > 0 && !(before - v > tol + (fabsf(before) + fabsf(v)) * 0x1p-22f)) ok = false;
      before = v;
      if (j == a.k) break;
    }
    const int owner = __ffs(who) - 1;
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (at == i) v = l[i];
    const int e = __shfl_sync(0xffffffffu, lane * V + at, owner);
    v = __shfl_sync(0xffffffffu, v, owner);
    if (lane == owner) avail &= ~(1u << at);
    if (lane == j) *id = e, *logit = v;
  }
  *apart = ok;
}

// The choice from scores in 64 bits.
template <int V>
__device__ __noinline__ void choose_64(const RouteArgs& a, const float (&l)[V], int* id, float* logit) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  Softmax<double> sm{0.f, 0.0, 0};
  if (!a.score) sm = softmax_of<double>(l);
  double c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = score_of<double>(l[i], a.score, sm, a.E);
    if (a.bias && e0 + i < a.E) c[i] += (double)a.bias[e0 + i];
    if (l[i] != l[i]) c[i] = __longlong_as_double(0x7FF8000000000000ll);
  }
  unsigned groups = ~0u;
  if (a.top_groups < a.groups) {
    bool apart;
    double rated[V], size = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) rated[i] = a.bias || a.group_top == 2 ? c[i] : (double)l[i];
    const double mine = group_value<double>(a, rated, &size);
    groups = best_groups<double>(a, mine, size, 0.0, &apart);
  }
  if (!a.bias) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = (double)l[i];
  }
  unsigned avail = eligible<V>(a, groups);
  for (int j = 0; j < a.k; ++j) {
    // a number before a NaN, then the larger, then the lower index
    double best = 0.0;
    int at = -1;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (((avail >> i) & 1u) && (at < 0 || c[i] > best || (best != best && c[i] == c[i]))) best = c[i], at = i;
    int e = at < 0 ? 0x7FFFFFFF : e0 + at;
    double v = best;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, e, o);
      const bool none = e == 0x7FFFFFFF, none2 = e2 == 0x7FFFFFFF, nan = v != v, nan2 = v2 != v2;
      const bool same = nan == nan2 && (nan || v == v2);
      const bool take = !none2 && (none || (nan && !nan2) || (nan == nan2 && !nan && v2 > v) || (same && e2 < e));
      if (take) v = v2, e = e2;
    }
    const int owner = e / V, i0 = e - owner * V;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i == i0) x = l[i];
    x = __shfl_sync(0xffffffffu, x, owner);
    if (lane == owner) avail &= ~(1u << i0);
    if (lane == j) *id = e, *logit = x;
  }
}

// Token t's choice: lane j < k gets its j-th expert and weight.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, int* id, float* weight) {
  const int lane = threadIdx.x & 31, e0 = lane * V;
  float l[V];
  load_lane<V>(a, t, l);
  int nan = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) nan += e0 + i < a.E && l[i] != l[i];
  nan = (int)__reduce_add_sync(0xffffffffu, (unsigned)nan);
  if (nan && lane == 0) atomicAdd(&a.st->nan_logits, (unsigned)nan);
  const bool limited = a.top_groups < a.groups, sums = limited && a.group_top == 2;
  Softmax<float> sm{0.f, 0.f, 0};
  if (!a.score && (a.bias || sums || !a.renorm)) sm = softmax_of<float>(l);
  float logit = 0.f;
  bool apart = true;
  {
    uint32_t key[V];
    float tol = -1.f, c[V];
    if (a.bias || sums) {
      float most = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float s = score_of<float>(l[i], a.score, sm, a.E);
        c[i] = a.bias && e0 + i < a.E ? s + a.bias[e0 + i] : s;
        if (l[i] != l[i]) c[i] = l[i];
        most = fmaxf(most, s);
      }
      tol = warp_max(most) * (a.score ? 0x1p-20f : 0x1p-17f);  // NaNs, a NaN bias's too, are never apart
    }
    unsigned groups = ~0u;
    if (limited) {
      float rated[V], size = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) rated[i] = a.bias || sums ? c[i] : l[i];
      bool far;
      const float mine = group_value<float>(a, rated, &size);
      groups = best_groups<float>(a, mine, size, tol < 0.f ? 0.f : 2.0f * tol, &far);
      apart = far || tol < 0.f;  // logits are exact
    }
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = float_key(a.bias ? c[i] : l[i]);
    bool far = true;
    choose<V>(a, key, l, eligible<V>(a, groups), a.bias ? tol : -1.f, id, &logit, &far);
    apart = apart && far;
  }
  if (!apart) {  // (copies, so that the arrays above stay in registers)
    float l2[V], x = 0.f;
    int e = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) l2[i] = l[i];
    choose_64<V>(a, l2, &e, &x);
    *id = e, logit = x;
  }
  float w;
  if (!a.score && a.renorm) {
    w = warp_softmax_k(logit, a.k);
  } else {
    w = lane < a.k ? score_of<float>(logit, a.score, sm, a.E) : 0.f;
    if (a.renorm) {
      float sum = 0.f;
      for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, w, j);
      w = sum > 0.f ? w / sum : 1.0f / (float)a.k;
    }
  }
  *weight = w * a.scale;
}

// Rows of expert e of the run before its token tl: `bits` [E][words].
__device__ __forceinline__ int rows_before(const uint32_t* bits, int words, int e, int tl) {
  const uint32_t* b = bits + e * words;
  int n = 0;
  for (int w = 0; w < (tl >> 5); ++w) n += __popc(b[w]);
  return n + __popc(b[tl >> 5] & ((1u << (tl & 31)) - 1u));
}

// kAll: the only run, tables included.
template <int V, bool kAll>
__global__ void __launch_bounds__(rt::kThreads) route_choose_kernel(RouteArgs a) {
  extern __shared__ uint32_t bits[];  // [E][words]
  __shared__ int scan[32], base[rt::kMaxExperts];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int t0, t1;
  run_of(a, blockIdx.x, t0, t1);
  for (int i = threadIdx.x; i < a.E * a.words; i += blockDim.x) bits[i] = 0u;
  __syncthreads();
  for (int t = t0 + warp; t < t1; t += blockDim.x >> 5) {
    int id = 0;
    float w;
    route_token<V>(a, t, &id, &w);
    if (lane < a.k) {
      a.ids[(size_t)t * a.k + lane] = id;
      a.weights[(size_t)t * a.k + lane] = w;
      atomicOr(bits + id * a.words + ((t - t0) >> 5), 1u << ((t - t0) & 31));
    }
  }
  __syncthreads();
  const int e = threadIdx.x;  // at most one expert a thread
  int n = 0;
  if (e < a.E)
    for (int w = 0; w < a.words; ++w) n += __popc(bits[e * a.words + w]);
  if (!kAll) {
    if (e < a.E) a.inv[(size_t)t0 * a.k + e] = n;
    return;
  }
  int total;
  const int before = block_exclusive_scan(n, scan, &total);
  if (e < a.E) a.offsets[e] = base[e] = before;
  if (e == 0) a.offsets[a.E] = total;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.k; i += blockDim.x) {
    const int id = a.ids[i], p = base[id] + rows_before(bits, a.words, id, i / a.k);
    a.perm[p] = i;
    a.inv[i] = p;
  }
}

// The runs' counts into places: one cluster, each CTA some of the experts, which tell one another their sums.
namespace rt {
constexpr int kScanCtas = 8, kScanThreads = 1024;
}
__global__ void __launch_bounds__(rt::kScanThreads) route_scan_kernel(RouteArgs a) {
  constexpr int kCols = rt::kMaxExperts / rt::kScanCtas, kRows = rt::kScanThreads / kCols;  // 64 columns by 16 stretches
  __shared__ int part[kRows][kCols];
  __shared__ int mine[kCols];
  __shared__ float sums[rt::kScanCtas];  // every CTA's, as bits
  __shared__ int scan[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int cols = (a.E + rt::kScanCtas - 1) / rt::kScanCtas, rank = (int)cluster_rank();
  const int c = threadIdx.x % kCols, r = threadIdx.x / kCols, e = rank * cols + c;
  const bool ok = c < cols && e < a.E;
  const int b0 = (int)((long long)a.runs * r / kRows), b1 = (int)((long long)a.runs * (r + 1) / kRows);
  int n = 0;
  if (ok)
    for (int b = b0; b < b1; ++b) {
      int t0, t1;
      run_of(a, b, t0, t1);
      n += a.inv[(size_t)t0 * a.k + e];
    }
  part[r][c] = n;
  __syncthreads();
  int sum = 0;
  if (r == 0)
    for (int i = 0; i < kRows; ++i) sum += part[i][c];
  int total;
  const int before = block_exclusive_scan(sum, scan, &total);
  if (threadIdx.x < rt::kScanCtas) st_cluster(sums + rank, threadIdx.x, __int_as_float(total));
  if (r == 0) mine[c] = before;
  cluster_sync_all();
  int base = mine[c];
  for (int i = 0; i < rank; ++i) base += __float_as_int(sums[i]);
  if (ok && r == 0) a.offsets[e] = base;
  if (rank == rt::kScanCtas - 1 && threadIdx.x == 0) a.offsets[a.E] = a.T * a.k;
  if (!ok) return;
  for (int i = 0; i < r; ++i) base += part[i][c];
  for (int b = b0; b < b1; ++b) {
    int t0, t1;
    run_of(a, b, t0, t1);
    int32_t* at = a.inv + (size_t)t0 * a.k + e;
    const int v = *at;
    *at = base;
    base += v;
  }
}

__global__ void __launch_bounds__(rt::kThreads) route_scatter_rows_kernel(RouteArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int base[rt::kMaxExperts];
  grid_dependency_wait();
  grid_launch_dependents();
  int t0, t1;
  run_of(a, blockIdx.x, t0, t1);
  const int i0 = t0 * a.k, rows = (t1 - t0) * a.k;
  for (int i = threadIdx.x; i < a.E * a.words; i += blockDim.x) bits[i] = 0u;
  if (threadIdx.x < a.E) base[threadIdx.x] = a.inv[i0 + threadIdx.x];
  __syncthreads();
  for (int i = threadIdx.x; i < rows; i += blockDim.x) {
    const int tl = i / a.k;
    atomicOr(bits + a.ids[i0 + i] * a.words + (tl >> 5), 1u << (tl & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows; i += blockDim.x) {
    const int id = a.ids[i0 + i], p = base[id] + rows_before(bits, a.words, id, i / a.k);
    a.perm[p] = i0 + i;
    a.inv[i0 + i] = p;
  }
}

// dl of a token from the gradient of its weights.  An id outside 0 .. E - 1 counts as no choice.
template <int V>
__global__ void __launch_bounds__(rt::kThreads) route_backward_kernel(RouteArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * V, warps = rt::kThreads / 32;
  for (int t = blockIdx.x * warps + warp; t < a.T; t += gridDim.x * warps) {
    float l[V], d[V];
    load_lane<V>(a, t, l);
    unsigned chosen = 0;
    const int id = lane < a.k ? a.cids[(size_t)t * a.k + lane] : -1;
    const float w = lane < a.k ? a.dw[(size_t)t * a.k + lane] * a.scale : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int at = __shfl_sync(0xffffffffu, id, j) - e0;
      const float v = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at == i && e0 + i < a.E) d[i] = v, chosen |= 1u << i;
    }
    float s[V];  // the scores that the weights are made of
    if (a.score) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = score_of<float>(l[i], 1, Softmax<float>{}, a.E);
    } else {
      // renormalised: the softmax of the chosen logits alone
      float m[V];
#pragma unroll
      for (int i = 0; i < V; ++i) m[i] = !a.renorm || ((chosen >> i) & 1u) ? l[i] : __uint_as_float(0x7FC00000u);
      const Softmax<float> sm = softmax_of<float>(m);
      const bool flat = sm.top == INFINITY || sm.top == -INFINITY;  // weights that do not move with the logits
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = flat ? 0.f : score_of<float>(m[i], 0, sm, a.E);
    }
    if (a.score && a.renorm) {
      float sum = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if ((chosen >> i) & 1u) sum += s[i], dot = fmaf(d[i], s[i], dot);
      sum = warp_sum(sum), dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = ((chosen >> i) & 1u) && sum > 0.f ? (d[i] - dot / sum) / sum : 0.f;
    }
    if (a.score) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = d[i] == 0.f || l[i] != l[i] ? 0.f : d[i] * s[i] * score_of<float>(-l[i], 1, Softmax<float>{}, a.E);
    } else {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) dot = fmaf(d[i], s[i], dot);
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = s[i] * (d[i] - dot);
    }
    const size_t at = (size_t)t * a.ld_dl + e0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E) {
        if (a.bf16) static_cast<__nv_bfloat16*>(a.dl)[at + i] = __float2bfloat16_rn(d[i]);
        else static_cast<float*>(a.dl)[at + i] = d[i];
      }
  }
}

static RouteArgs args_of(const RouteOp& p) {
  RouteArgs a{};
  a.logits = p.logits, a.ld = p.ld, a.bf16 = p.bf16;
  a.vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && p.ld * (p.bf16 ? 2 : 4) % 16 == 0;
  a.T = p.T, a.E = p.E, a.k = p.k;
  a.score = p.score, a.renorm = p.renorm, a.scale = p.scale, a.bias = p.bias;
  a.groups = p.groups, a.top_groups = p.top_groups, a.group_top = p.group_top, a.group_size = p.E / p.groups;
  a.ids = p.ids, a.weights = p.weights, a.offsets = p.offsets, a.perm = p.perm, a.inv = p.inv;
  a.st = p.status;
  a.cids = p.ids, a.dw = p.dweights, a.dl = p.dlogits, a.ld_dl = p.ld_dl;
  return a;
}

typedef void (*RouteKernel)(RouteArgs);
struct RouteKernels {
  RouteKernel all, choose, backward;
};
template <int V>
static RouteKernels kernels_for() {
  return {route_choose_kernel<V, true>, route_choose_kernel<V, false>, route_backward_kernel<V>};
}
static RouteKernels kernels_of(int E) {
  return E <= 32    ? kernels_for<1>()
         : E <= 64  ? kernels_for<2>()
         : E <= 128 ? kernels_for<4>()
         : E <= 256 ? kernels_for<8>()
                    : kernels_for<16>();
}

static cudaError_t launch(RouteKernel f, int grid, int threads, size_t smem, const RouteArgs& a, cudaStream_t st,
                          int cluster = 1) {
  if (smem > 32768) {  // 512 experts and one choice: up to 1024 tokens a run
    const cudaError_t e = cudaFuncSetAttribute((const void*)f, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * rt::kMaxExperts * 32);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid), cfg.blockDim = dim3((unsigned)threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

cudaError_t launch_route_forward(const RouteOp& p, cudaStream_t st) {
  RouteArgs a = args_of(p);
  const RouteKernels f = kernels_of(a.E);
  // Runs: a CTA each, none with fewer tokens than hold its counts in `inv`
  const int least = std::max(32, (a.E + a.k - 1) / a.k);
  const int per = std::max(least, std::min(rt::kRun, (a.T + p.num_sms - 1) / p.num_sms));
  a.runs = a.T <= rt::kOneCta ? 1 : std::max(1, a.T / per);
  a.words = ((a.T + a.runs - 1) / a.runs + 31) / 32;
  const size_t smem = sizeof(uint32_t) * a.E * a.words;
  if (a.runs == 1) return launch(f.all, 1, rt::kThreads, smem, a, st);
  cudaError_t e = launch(f.choose, a.runs, rt::kThreads, smem, a, st);
  if (e == cudaSuccess) e = launch(route_scan_kernel, rt::kScanCtas, rt::kScanThreads, 0, a, st, rt::kScanCtas);
  if (e == cudaSuccess) e = launch(route_scatter_rows_kernel, a.runs, rt::kThreads, smem, a, st);
  return e;
}

cudaError_t launch_route_backward(const RouteOp& p, cudaStream_t st) {
  RouteArgs a = args_of(p);
  const int warps = rt::kThreads / 32;
  return launch(kernels_of(a.E).backward, std::min((a.T + warps - 1) / warps, 4 * p.num_sms), rt::kThreads, 0, a, st);
}

}  // namespace nvfp4moe
