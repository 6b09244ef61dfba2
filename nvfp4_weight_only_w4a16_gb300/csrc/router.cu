// Routing on its own (nvfp4_route_forward / nvfp4_route_backward): scores, choice, weights and the tables that sort the
// routed rows by expert.
//   s_e = softmax of a token's logits, or 1 / (1 + e^-l_e);  c_e = s_e + bias_e, or the logit where there is no bias
//   groups: a group's value is its largest c, or the sum of its two largest (of s without a bias); the best `top_groups`
//           groups' experts are eligible
//   choice: the k largest c, largest first, the lower index first among equals; weights scale s_j (/ sum of the chosen)
//   tables: the T k routed rows t k + j by expert, ascending within one: offsets, perm, and its inverse
//
// The choice is that of c in 64 bits.  Comparing FP32 scores gives it wherever neighbours in the order are further apart
// than those scores can be wrong (2^-20 of a largest sigmoid near 1, more below, and 2^-17 of a softmax's largest); a
// token where some are not is chosen again, its candidates scored in 64 bits, or all experts where more than 32 are in
// doubt (softmax in groups with the border far below the largest score: 16384 x 256 takes 236 us at a standard deviation
// of the logits of 10, 45 at 1).  Logits that are compared as they are need no such test.
//
// One warp a token, lane l with experts l, l + 32, ..  No rounds of warp maxima (at 9 of them, 8 experts chosen of 256, a
// token took some 1800 cycles of latency): the (k + 1)-th largest of the lanes' own maxima is a bound that the k + 1
// largest reach, and few others; those are laid out one to a lane, and each counts how many are ahead of it.
//
// A CTA takes a run of tokens; bit t of bits[e] says that its token t chose e, so that a row's place among its expert's
// is a population count, whatever the order the warps came in.  Few tokens: one CTA does it all.  Else a second kernel
// turns the runs' counts into places and a third scatters; the counts lie in `inv`, each run's in its own rows' part,
// which its CTA alone overwrites in the end, so that there is no workspace and calls may overlap.
//
// 16384 tokens of 256 experts take 800 warp instructions a token as a softmax, 1150 with a bias and groups, issued in two
// thirds of the slots by six warps a scheduler, and 25 and 36 us with the scan and the scatter; their bytes would take 3.
// Few tokens wait for one token's way through a warp and for the launches (2 tokens of 128 experts 4.1 us; 128 of 256 in
// groups 16).
#include <algorithm>
#include <mutex>

#include "kernels.h"
#include "route_common.cuh"
#include "tcgen05.cuh"

namespace nvfp4moe {

namespace rt {
constexpr int kMaxExperts = 512;
constexpr int kThreads = 768;   // of 80 registers; 1024 of 64 spill (16384 x 256 in groups 40.2 us, 39.0); 896 of 72 gain
                                // there (35.8, 36.4) and lose below (8192 tokens 27.3, 25.7)
constexpr int kOneCta = 72;     // tokens up to which one CTA does it all (256 experts in groups, 64 tokens: 15.1 us, 16.2 as
                                // three kernels; 96: 19.8, 16.1)
constexpr int kRun = 256;     // of a run, unless its counts need more
constexpr int kMostShared = 208 * 1024;  // 512 experts: 128 KB of 32 warps' rows and 64 KB of a run's bits
// Sigmoids below this are e^l to a rounding, and what they are renormalised to is the softmax of their logits: it holds
// where they themselves are lost to FP32 (from l = -88.7 down).  Of chosen ones only -inf and NaN are 0 then.
constexpr float kLowSigmoids = 0x1p-25f;
}  // namespace rt

struct RouteArgs {
  const void* logits;
  long long ld;       // elements
  int bf16;
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

// Lane's logits l, l + 32, .. of token t; beyond E: -inf, which no sum or maximum sees.
template <int V>
__device__ __forceinline__ void load_lane(const RouteArgs& a, int t, float (&v)[V]) {
  const int lane = threadIdx.x & 31;
  const size_t at = (size_t)t * a.ld + lane;
  if (a.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lane + 32 * i < a.E ? __uint_as_float((uint32_t)p[32 * i] << 16) : -INFINITY;
  } else {
    const float* p = static_cast<const float*>(a.logits) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = lane + 32 * i < a.E ? p[32 * i] : -INFINITY;
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

// 1 / (1 + e^-l) by the hardware's 2^x and 1/x.
__device__ __forceinline__ float sigmoid_fast(float l) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// The larger two of two sorted pairs, and of a pair and one more.
template <class F>
__device__ __forceinline__ F larger(F a, F b) {
  return a < b ? b : a;
}
template <class F>
__device__ __forceinline__ F smaller(F a, F b) {
  return a < b ? a : b;
}
template <>
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
template <>
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
template <class F>
__device__ __forceinline__ void merge_two(F& a, F& b, F c, F d) {
  b = larger(smaller(a, c), larger(b, d));
  a = larger(a, c);
}
template <class F>
__device__ __forceinline__ void merge_one(F& a, F& b, F c) {
  b = larger(b, smaller(a, c));
  a = larger(a, c);
}

// A warp's part of shared memory.
struct RouteScratch {
  uint32_t key[32];  // candidates: order key, expert
  int id[32];
};

// Lane g < groups: the value of group g over its members' c in shared memory (row [E]; NaN counts as -inf), the
// magnitudes that went in, and the smaller of them.  Every group gets as many lanes as there are for it, which start at different members so as not
// to meet in a bank.
template <class F>
__device__ __forceinline__ F group_value(const RouteArgs& a, const F* row, F* size, F* least) {
  const int lane = threadIdx.x & 31;
  const F none = F(-INFINITY);
  const int bits = 32 - __clz(a.groups - 1), per = 32 >> bits;  // lanes a group (groups >= 2)
  const int g = lane / per, sub = lane % per, turns = (a.group_size + per - 1) / per;
  F x = none, y = none;
  if (g < a.groups)
    for (int j = 0, at = g % turns; j < turns; ++j, at = at + 1 == turns ? 0 : at + 1) {
      const int m = sub + at * per;
      if (m < a.group_size) {
        const F c = row[g * a.group_size + m];
        merge_one(x, y, c == c ? c : none);
      }
    }
  for (int o = 1; o < per; o <<= 1) {
    const F x2 = __shfl_xor_sync(0xffffffffu, x, o), y2 = __shfl_xor_sync(0xffffffffu, y, o);
    merge_two(x, y, x2, y2);
  }
  F value = a.group_top == 2 ? x + y : x;
  if (value != value) value = none;  // infinities of both signs
  const F sizes = a.group_top == 2 ? fabs(x) + fabs(y) : fabs(x);
  const int from = (lane * per) & 31;
  *size = __shfl_sync(0xffffffffu, sizes, from);
  *least = __shfl_sync(0xffffffffu, a.group_top == 2 ? y : x, from);
  return __shfl_sync(0xffffffffu, value, from);
}

// The same where groups are of 32 experts, so that group i is register i of all lanes (groups = V): the lanes halve the
// registers they keep, exchanging the others, with each of the first steps.  c holds no NaN.
template <int V>
__device__ __forceinline__ float group_value_32(const RouteArgs& a, const float (&c)[V], float* size, float* least) {
  const int lane = threadIdx.x & 31;
  float x[V], y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = c[i];
  int o = 16;
#pragma unroll
  for (int n = V / 2; n >= 1; n /= 2, o /= 2) {  // registers kept
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? x[i + n] : x[i], x2 = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i + n], o);
      if (n == V / 2) {
        y[i] = fminf(keep, x2);
        x[i] = fmaxf(keep, x2);
      } else {
        const float keep_y = upper ? y[i + n] : y[i], y2 = __shfl_xor_sync(0xffffffffu, upper ? y[i] : y[i + n], o);
        x[i] = keep, y[i] = keep_y;
        merge_two(x[i], y[i], x2, y2);
      }
    }
  }
#pragma unroll
  for (; o >= 1; o /= 2) {
    const float x2 = __shfl_xor_sync(0xffffffffu, x[0], o), y2 = __shfl_xor_sync(0xffffffffu, y[0], o);
    merge_two(x[0], y[0], x2, y2);
  }
  float value = a.group_top == 2 ? x[0] + y[0] : x[0];
  if (value != value) value = -INFINITY;  // infinities of both signs
  // group g is with the lanes whose first bits, from 16 down, are g's
  const int from = (lane * (32 / V)) & 31;
  *size = __shfl_sync(0xffffffffu, a.group_top == 2 ? fabsf(x[0]) + fabsf(y[0]) : fabsf(x[0]), from);
  *least = __shfl_sync(0xffffffffu, a.group_top == 2 ? y[0] : x[0], from);
  return __shfl_sync(0xffffffffu, value, from);
}

// The groups kept, one bit each.  `near`: the groups, if any, that may be on either side of the border: the last one in
// and the first one out are no further apart than they can be wrong (`tol`, and 2^-21 of the magnitudes that they are made
// of), and these are within twice that.
template <class F>
__device__ __forceinline__ unsigned best_groups(const RouteArgs& a, F mine, F size, F tol, unsigned* near) {
  const int lane = threadIdx.x & 31;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const F v = __shfl_sync(0xffffffffu, mine, g);
    rank += v > mine || (v == mine && g < lane);
  }
  const bool in = lane < a.groups && rank < a.top_groups;
  const int l = __ffs(__ballot_sync(0xffffffffu, lane < a.groups && rank == a.top_groups - 1)) - 1;
  const int n = __ffs(__ballot_sync(0xffffffffu, lane < a.groups && rank == a.top_groups)) - 1;
  const F last = __shfl_sync(0xffffffffu, mine, l), gap = last - __shfl_sync(0xffffffffu, mine, n);
  const F sizes = __shfl_sync(0xffffffffu, size, l) + __shfl_sync(0xffffffffu, size, n);
  const F can = tol + sizes * F(0x1p-21);
  *near = gap > can ? 0u : __ballot_sync(0xffffffffu, lane < a.groups && !(fabs(mine - last) > 2 * can));
  return __ballot_sync(0xffffffffu, in);
}

// The groups of the lane's experts, a byte each, and which of them there are, a bit each.
template <int V>
struct LaneGroups {
  uint32_t w[(V + 3) / 4], all;
  __device__ __forceinline__ explicit LaneGroups(const RouteArgs& a) : all(0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < (V + 3) / 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) w[i / 4] |= (uint32_t)(e / a.group_size) << (8 * (i % 4)), all |= 1u << i;
    }
  }
  // those whose group has its bit set
  __device__ __forceinline__ unsigned among(unsigned groups) const {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m |= ((groups >> ((w[i / 4] >> (8 * (i % 4))) & 31u)) & 1u) << i;
    return m & all;
  }
};

// The value of an order key; NaN for a NaN's (0, or 1 where 0 means none).
__device__ __forceinline__ float key_float(uint32_t key) {
  return key <= 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// Order keys of doubles: larger value, larger key; NaN lowest.
__device__ __forceinline__ unsigned long long double_key(double v) {
  if (v != v) return 0ull;
  if (v == 0.0) return 1ull << 63;
  const unsigned long long b = (unsigned long long)__double_as_longlong(v);
  return b >> 63 ? ~b : b | (1ull << 63);
}

// The softmax's sum in 64 bits.
__device__ __noinline__ Softmax<double> softmax_64(const RouteArgs& a, int t, const Softmax<float>& sm) {
  Softmax<double> r{sm.top, 0.0, sm.infinities};
  if (!a.score && fabsf(sm.top) != INFINITY) {
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
      const float l = load_logit(a.logits, a.bf16, (size_t)t * a.ld + e);
      if (l == l) r.sum += exp((double)l - (double)sm.top);
    }
    r.sum = warp_sum(r.sum);
  }
  return r;
}

// The choice in 64 bits, for the tokens that the fast way leaves open.  Small loops over shared memory (row [E]) on
// purpose: its code is cold, and unrolled over the lane's experts its first use took 20 us, which such a token's CTA
// then took longer than the others.
__device__ __noinline__ void choose_64(const RouteArgs& a, int t, double* row, int* id) {
  const int lane = threadIdx.x & 31;
  const double nan = __longlong_as_double(0x7FF8000000000000ll);
  const size_t at = (size_t)t * a.ld;
  const bool limited = a.top_groups < a.groups, sums = limited && a.group_top == 2;
  Softmax<float> top{-INFINITY, 0.f, 0};
  if (!a.score) {
    int n = 0;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_logit(a.logits, a.bf16, at + e);
      top.top = fmaxf(top.top, l);
      n += l == INFINITY;
    }
    top.top = warp_max(top.top);
    top.infinities = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  }
  const Softmax<double> sm = softmax_64(a, t, top);
  __syncwarp();
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const float l = load_logit(a.logits, a.bf16, at + e);
    double c = l;
    if (a.bias || sums) c = score_of<double>(l, a.score, sm, a.E) + (a.bias ? (double)a.bias[e] : 0.0);
    row[e] = l == l ? c : nan;
  }
  __syncwarp();
  unsigned groups = ~0u;
  if (limited) {
    double size, least;
    unsigned near;
    const double mine = group_value<double>(a, row, &size, &least);
    groups = best_groups<double>(a, mine, size, 0.0, &near);
  }
  unsigned open = 0;
#pragma unroll 1
  for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
    if (!limited || ((groups >> (e / a.group_size)) & 1u)) open |= 1u << i;
    if (!a.bias && sums) row[e] = load_logit(a.logits, a.bf16, at + e);
  }
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0;
    int e = 0x7FFFFFFF;
#pragma unroll 1
    for (int i = 0; open >> i; ++i)
      if ((open >> i) & 1u) {
        const unsigned long long key = double_key(row[lane + 32 * i]) + 1ull;
        if (key > best) best = key, e = lane + 32 * i;
      }
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long b2 = __shfl_xor_sync(0xffffffffu, best, o);
      const int e2 = __shfl_xor_sync(0xffffffffu, e, o);
      if (b2 > best || (b2 == best && e2 < e)) best = b2, e = e2;
    }
    if ((e & 31) == lane) open &= ~(1u << (e >> 5));
    if (lane == j) *id = e;
  }
}

// The groups kept, where those in `near` are too close for FP32: row [E] holds the experts' FP32 c as doubles, and those
// of these groups that may count in their group's value, at least `bound`, are evaluated in 64 bits, one a lane.  False
// where they are more than lanes.
__device__ __noinline__ bool groups_64(const RouteArgs& a, int t, const Softmax<float>& sm, unsigned near, float bound,
                                       RouteScratch& s, double* row, unsigned* groups) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    const bool in = e < a.E && ((near >> (e / a.group_size)) & 1u) && row[e] >= (double)bound;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) s.id[at] = e;
    n += __popc(who);
  }
  __syncwarp();
  if (n > 32) return false;
  const Softmax<double> sm64 = softmax_64(a, t, sm);
  if (lane < n) {
    const int e = s.id[lane];
    row[e] = score_of<double>(load_logit(a.logits, a.bf16, (size_t)t * a.ld + e), a.score, sm64, a.E) + (a.bias ? (double)a.bias[e] : 0.0);
  }
  __syncwarp();
  double size, least;
  unsigned still;
  const double mine = group_value<double>(a, row, &size, &least);
  *groups = best_groups<double>(a, mine, size, 0.0, &still);
  return true;
}

// Token t's choice: lane j < k gets its j-th expert and weight.  row: the warp's [E] doubles; bias [32 V], in shared memory.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int t, const float (&l)[V], const LaneGroups<V>& of, const float* bias, RouteScratch& s,
                                            double* row, int* id, float* weight) {
  const int lane = threadIdx.x & 31;
  float all = 0.f;  // NaN where one is (or infinities of both signs)
#pragma unroll
  for (int i = 0; i < V; ++i) all += l[i];
  const bool odd = __any_sync(0xffffffffu, all != all);
  if (odd) {
    int nan = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) nan += lane + 32 * i < a.E && l[i] != l[i];
    nan = (int)__reduce_add_sync(0xffffffffu, (unsigned)nan);
    if (nan && lane == 0) atomicAdd(&a.st->nan_logits, (unsigned)nan);
  }
  const bool limited = a.top_groups < a.groups, sums = limited && a.group_top == 2;
  Softmax<float> sm{0.f, 0.f, 0};
  if (!a.score && (a.bias || sums || !a.renorm)) sm = softmax_of<float>(l);
  float tol = -1.f, c[V];  // NaN where the logit is
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = l[i] + 0.0f;  // no negative zero
  if (a.bias || sums) {
    // By the hardware's 2^x (2^-22, and half a step of x) and 1/x (a step).  A sigmoid s is off by 2^-24 (7 + 1.5 |l|) s at
    // most for l < 0, and by less than 2^-24 6 for l > 0, so by 2^-24 (7 - 1.5 log s) s for the largest s; a softmax, whose
    // sum of E terms counts too, by 2^-24 43 of the largest.  Both are flushed to 0 below 2^-126.  tol covers two.
    if (a.score) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = sigmoid_fast(c[i]);
    } else if (sm.top != INFINITY && sm.top != -INFINITY) {
      const float inv = __fdividef(1.0f, sm.sum);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = __expf(c[i] - sm.top) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l[i] == l[i] ? score_of<float>(l[i], 0, sm, a.E) : l[i];
    }
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) most = fmaxf(most, c[i]);  // drops NaNs
    most = fmaxf(warp_max(most), 0x1p-126f);
    tol = most * (a.score ? 0x1p-23f * (8.0f - 1.5f * __logf(most)) : 0x1p-17f) + 0x1p-124f;
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] += bias[lane + 32 * i];
    }
  }
  unsigned open = of.all;
  bool exact = true;  // the groups are certain
  if (limited) {
    float size, least, mine;
    if (V > 1 && a.group_size == 32 && a.groups == V) {
      float clean[V];
#pragma unroll
      for (int i = 0; i < V; ++i) clean[i] = c[i] == c[i] ? c[i] : -INFINITY;
      mine = group_value_32<V>(a, clean, &size, &least);
    } else {
      float* r = reinterpret_cast<float*>(row);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.E) r[lane + 32 * i] = c[i];
      __syncwarp();
      mine = group_value<float>(a, r, &size, &least);
    }
    unsigned near, groups = best_groups<float>(a, mine, size, tol < 0.f ? 0.f : 2.0f * tol, &near);
    __syncwarp();
    if (near && tol >= 0.f) {  // (logits are exact)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.E) row[lane + 32 * i] = c[i];
      __syncwarp();
      const float low = -warp_max((near >> lane) & 1u ? -least : -INFINITY);
      exact = groups_64(a, t, sm, near, low - 2.0f * (tol + fabsf(low) * 0x1p-22f), s, row, &groups);
      __syncwarp();
    }
    open = V > 1 && a.group_size == 32 && a.groups == V ? groups : of.among(groups);
  }
  const bool close = a.bias != nullptr;  // the keys are of FP32 scores: look at the gaps
  if (!close && sums) {  // the groups were of scores, the experts are of logits
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i] + 0.0f;
  }
  uint32_t key[V], m = 0;  // order keys: 0 not eligible, 1 NaN
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t b = __float_as_uint(c[i]), k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    key[i] = (open >> i) & 1u ? (c[i] == c[i] ? k : 1u) : 0u;
    m = max(m, key[i]);
  }
  // the bound: the (k + 1)-th largest of the lanes' maxima, less what two scores can be wrong
  uint32_t bound = 0;
  for (int j = 0; j <= a.k; ++j) {
    bound = __reduce_max_sync(0xffffffffu, m);
    const unsigned who = __ballot_sync(0xffffffffu, m == bound);
    if (lane == __ffs(who) - 1) m = 0;
  }
  if (close && bound > 1u) {
    const float v = key_float(bound);
    bound = float_key(v - 2.0f * (tol + fabsf(v) * 0x1p-22f));
  }
  bound = max(bound, 1u);
  int n = 0;  // candidates, in the experts' order
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = key[i] >= bound;
    const unsigned who = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) s.key[at] = key[i], s.id[at] = lane + 32 * i;
    n += __popc(who);
  }
  __syncwarp();
  if (exact && n <= 32) {
    const uint32_t mine = lane < n ? s.key[lane] : 0u;
    const int e = lane < n ? s.id[lane] : 0;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint32_t v = s.key[j];
      rank += v > mine || (v == mine && j < lane);
    }
    __syncwarp();
    bool apart = true;
    if (close) {
      // whether every one of the k + 1 first and the next differ by more than they can be wrong
      if (lane < n) s.key[rank] = mine;
      __syncwarp();
      const float u = key_float(s.key[lane]), v = key_float(s.key[lane < 31 ? lane + 1 : 31]);
      apart = __all_sync(0xffffffffu, lane >= a.k || lane + 1 >= n || u - v > tol + (fabsf(u) + fabsf(v)) * 0x1p-22f);
    }
    if (!apart) {  // again in 64 bits, of the candidates
      const Softmax<double> sm64 = softmax_64(a, t, sm);
      unsigned long long k64 = 0;
      if (lane < n) {
        const float x = load_logit(a.logits, a.bf16, (size_t)t * a.ld + e);
        k64 = double_key(x != x ? (double)x : score_of<double>(x, a.score, sm64, a.E) + (double)a.bias[e]);
      }
      rank = 0;
      for (int j = 0; j < n; ++j) {
        const unsigned long long v = __shfl_sync(0xffffffffu, k64, j);
        rank += v > k64 || (v == k64 && j < lane);
      }
    }
    if (lane < n) s.id[rank] = e;
    __syncwarp();
    if (lane < a.k) *id = s.id[lane];
  } else {
    int e = 0;
    choose_64(a, t, row, &e);
    if (lane < a.k) *id = e;
  }
  __syncwarp();  // the scratch is free again
  const float logit = lane < a.k ? load_logit(a.logits, a.bf16, (size_t)t * a.ld + *id) : 0.f;
  float w;
  if (!a.score && a.renorm) {
    w = warp_softmax_k(logit, a.k);
  } else {
    w = lane < a.k ? score_of<float>(logit, a.score, sm, a.E) : 0.f;
    if (a.renorm) {
      float sum = 0.f;
      for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, w, j);
      w = sum >= rt::kLowSigmoids ? w / sum : warp_softmax_k(logit, a.k);
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
  extern __shared__ double rows_mem[];  // [warps][E], then bits [E][words]
  __shared__ int scan[32], base[rt::kMaxExperts];
  __shared__ float bias[32 * V];
  __shared__ RouteScratch scratch[rt::kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double* row = rows_mem + warp * a.E;
  uint32_t* bits = reinterpret_cast<uint32_t*>(rows_mem + (blockDim.x >> 5) * a.E);
  int t0, t1;
  run_of(a, blockIdx.x, t0, t1);
  const LaneGroups<V> of(a);
  for (int i = threadIdx.x; i < a.E * a.words; i += blockDim.x) bits[i] = 0u;
  for (int i = threadIdx.x; i < 32 * V; i += blockDim.x) bias[i] = a.bias && i < a.E ? a.bias[i] : 0.f;
  __syncthreads();
  const int step = blockDim.x >> 5;
  float next[V];
  if (t0 + warp < t1) load_lane<V>(a, t0 + warp, next);
  for (int t = t0 + warp; t < t1; t += step) {
    int id = 0;
    float w, l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = next[i];
    if (t + step < t1) load_lane<V>(a, t + step, next);
    route_token<V>(a, t, l, of, bias, scratch[warp], row, &id, &w);
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

// The runs' counts into places: one cluster, each CTA some of the experts, which tell one another their sums.  A thread
// has one expert's counts of a stretch of runs.
namespace rt {
constexpr int kScanCtas = 8, kScanThreads = 1024, kScanHeld = 8;
}
__global__ void __launch_bounds__(rt::kScanThreads) route_scan_kernel(RouteArgs a) {
  __shared__ int part[rt::kScanThreads];
  __shared__ float sums[rt::kScanCtas];  // every CTA's, as bits
  __shared__ int scan[32];
  cluster_arrive();  // the sums wait for it: every CTA has begun
  grid_dependency_wait();
  grid_launch_dependents();
  const int cols = (a.E + rt::kScanCtas - 1) / rt::kScanCtas, rank = (int)cluster_rank();
  const int stretches = min(rt::kScanThreads / cols, 64);  // few experts: each thread adds up all of its own's
  const int r = threadIdx.x / cols, c = threadIdx.x - r * cols, e = rank * cols + c;
  const bool ok = r < stretches && e < a.E;
  const int b0 = ok ? a.runs * r / stretches : 0, b1 = ok ? a.runs * (r + 1) / stretches : 0;
  const int base = a.T / a.runs, extra = a.T - base * a.runs;
  const auto at = [&](int b) { return a.inv + (size_t)(b * base + min(b, extra)) * a.k + e; };
  int held[rt::kScanHeld], n = 0;  // the first ones, so that they are not read twice
#pragma unroll
  for (int i = 0; i < rt::kScanHeld; ++i) held[i] = b0 + i < b1 ? *at(b0 + i) : 0;
#pragma unroll
  for (int i = 0; i < rt::kScanHeld; ++i) n += held[i];
  for (int b = b0 + rt::kScanHeld; b < b1; ++b) n += *at(b);
  part[threadIdx.x] = n;
  __syncthreads();
  int sum = 0, before = 0;  // of the expert; of its stretches before this one
  if (ok)
    for (int i = 0; i < stretches; ++i) {
      const int v = part[i * cols + c];
      before += i < r ? v : 0;
      sum += v;
    }
  int total;
  const int lower = block_exclusive_scan(r == 0 ? sum : 0, scan, &total);  // experts of this CTA below; r = 0 comes first
  cluster_wait();
  if (threadIdx.x < rt::kScanCtas) st_cluster(sums + rank, threadIdx.x, __int_as_float(total));
  if (r == 0) part[c] = lower;
  cluster_sync_all();
  if (!ok) return;
  int place = part[c];
  for (int i = 0; i < rank; ++i) place += __float_as_int(sums[i]);
  if (r == 0) a.offsets[e] = place;
  if (r == 0 && e == a.E - 1) a.offsets[a.E] = a.T * a.k;
  place += before;
#pragma unroll
  for (int i = 0; i < rt::kScanHeld; ++i)
    if (b0 + i < b1) {
      *at(b0 + i) = place;
      place += held[i];
    }
  for (int b = b0 + rt::kScanHeld; b < b1; ++b) {
    const int v = *at(b);
    *at(b) = place;
    place += v;
  }
}

__global__ void __launch_bounds__(rt::kThreads) route_scatter_rows_kernel(RouteArgs a) {
  extern __shared__ double rows_mem[];
  uint32_t* bits = reinterpret_cast<uint32_t*>(rows_mem);
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

// dl of a token from the gradient of its weights.  Renormalised weights and sigmoids move with the chosen logits alone:
// lanes j < k form those and lay them into a row of zeros in shared memory.  Plain softmax: s (d - sum d s) of all E, d the
// weights' gradient laid out so.  One slot after the other, so that an expert named twice gets both, in one order.
// An id outside 0 .. E - 1 counts as no choice.
namespace rt {
constexpr int kBackThreads = 256;
}
template <int V>
__global__ void __launch_bounds__(rt::kBackThreads) route_backward_kernel(RouteArgs a) {
  __shared__ float rows[rt::kBackThreads / 32][32 * V];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = rt::kBackThreads / 32;
  const bool sparse = a.score || a.renorm;
  float* row = rows[warp];
  for (int t = blockIdx.x * warps + warp; t < a.T; t += gridDim.x * warps) {
    float l[V];
    if (!sparse) load_lane<V>(a, t, l);
    const int id = lane < a.k ? a.cids[(size_t)t * a.k + lane] : -1;
    float v = lane < a.k ? a.dw[(size_t)t * a.k + lane] * a.scale : 0.f;
    const bool ok = (unsigned)id < (unsigned)a.E;
#pragma unroll
    for (int i = 0; i < V; ++i) row[lane + 32 * i] = 0.f;
    Softmax<float> sm{0.f, 0.f, 0};
    if (sparse) {
      const float x = ok ? load_logit(a.logits, a.bf16, (size_t)t * a.ld + id) : __uint_as_float(0x7FC00000u);
      const bool counts = x == x;
      if (a.score) {
        float s = counts ? score_of<float>(x, 1, sm, a.E) : 0.f;
        const float rest = counts ? score_of<float>(-x, 1, sm, a.E) : 0.f;
        if (a.renorm) {  // of the weights, w rest (d - sum w d): no quotient by a sum that may be as small as a score
          float sum = warp_sum(s);
          if (sum < rt::kLowSigmoids) {
            const float top = warp_max(counts ? x : -INFINITY);
            s = counts && top != -INFINITY ? expf(x - top) : 0.f;
            sum = warp_sum(s);
          }
          s = sum > 0.f ? s / sum : 0.f;
          v -= warp_sum(counts ? v * s : 0.f);
        }
        v = counts && v != 0.f ? v * s * rest : 0.f;
      } else {
        const float top = warp_max(counts ? x : -INFINITY);
        const bool flat = fabsf(top) == INFINITY;  // weights that do not move with the logits
        const float e = counts && !flat ? expf(x - top) : 0.f, sum = warp_sum(e), s = flat ? 0.f : e / sum;
        const float dot = warp_sum(counts ? v * s : 0.f);
        v = counts ? s * (v - dot) : 0.f;
      }
    } else {
      sm.top = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) sm.top = fmaxf(sm.top, l[i]);
      sm.top = warp_max(sm.top);
    }
    __syncwarp();
    for (int j = 0; j < a.k; ++j) {
      if (lane == j && ok) row[id] += v;
      __syncwarp();
    }
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = row[lane + 32 * i];
    if (!sparse) {
      const bool flat = fabsf(sm.top) == INFINITY;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        l[i] = l[i] == l[i] && !flat ? __expf(l[i] - sm.top) : 0.f;
        sm.sum += l[i];
        dot = fmaf(o[i], l[i], dot);
      }
      const float inv = flat ? 0.f : 1.0f / warp_sum(sm.sum);
      dot = warp_sum(dot) * inv;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = l[i] * inv * (o[i] - dot);
    }
    const size_t at = (size_t)t * a.ld_dl + lane;
    if (a.bf16) {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.dl) + at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.E) p[32 * i] = __float2bfloat16_rn(o[i]);
    } else {
      float* p = static_cast<float*>(a.dl) + at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 32 * i < a.E) p[32 * i] = o[i];
    }
    __syncwarp();
  }
}

static RouteArgs args_of(const RouteOp& p) {
  RouteArgs a{};
  a.logits = p.logits, a.ld = p.ld, a.bf16 = p.bf16;
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

static cudaError_t set_route_attrs() {  // once per device
  constexpr int kCached = 64;
  static std::mutex mu;
  static bool done[kCached] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < kCached && done[dev]) return cudaSuccess;
  for (int E = 32; E <= rt::kMaxExperts && e == cudaSuccess; E *= 2) {
    const RouteKernels f = kernels_of(E);
    for (const RouteKernel k : {f.all, f.choose})
      if (e == cudaSuccess) e = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, rt::kMostShared);
  }
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute((const void*)route_scatter_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, rt::kMostShared);
  if (e == cudaSuccess && dev >= 0 && dev < kCached) done[dev] = true;
  return e;
}

static cudaError_t launch(RouteKernel f, int grid, int threads, size_t smem, const RouteArgs& a, cudaStream_t st,
                          int cluster = 1) {
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
  cudaError_t e = set_route_attrs();
  if (e != cudaSuccess) return e;
  RouteArgs a = args_of(p);
  const RouteKernels f = kernels_of(a.E);
  // Runs: a CTA each, none with fewer tokens than hold its counts in `inv`
  const int least = std::max(32, (a.E + a.k - 1) / a.k);
  const int per = std::max(least, std::min(rt::kRun, (a.T + p.num_sms - 1) / p.num_sms));
  a.runs = a.T <= rt::kOneCta ? 1 : std::max(1, a.T / per);
  a.words = ((a.T + a.runs - 1) / a.runs + 31) / 32;
  // warps: one a token up to all of them, and threads enough for an expert each
  const int threads = std::min(rt::kThreads, std::max((a.E + 31) / 32, (a.T + a.runs - 1) / a.runs) * 32);
  const size_t bits = sizeof(uint32_t) * a.E * a.words;
  const size_t smem = bits + sizeof(double) * a.E * (threads / 32);
  if (a.runs == 1) return launch(f.all, 1, threads, smem, a, st);
  e = launch(f.choose, a.runs, threads, smem, a, st);
  if (e == cudaSuccess) e = launch(route_scan_kernel, rt::kScanCtas, rt::kScanThreads, 0, a, st, rt::kScanCtas);
  if (e == cudaSuccess) e = launch(route_scatter_rows_kernel, a.runs, rt::kThreads, bits, a, st);
  return e;
}

cudaError_t launch_route_backward(const RouteOp& p, cudaStream_t st) {
  RouteArgs a = args_of(p);
  const int warps = rt::kBackThreads / 32;
  return launch(kernels_of(a.E).backward, std::min((a.T + warps - 1) / warps, 8 * p.num_sms), rt::kBackThreads, 0, a, st);
}

}  // namespace nvfp4moe
