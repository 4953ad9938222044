// Routing of a mixture of experts by scores: sigmoid or softmax, a bias for balance, expert groups,
// scaled weights; and the gradient of the logits.
//
//   s_te = 1 / (1 + e^-l_te),  or  e^l_te / sum_open e^l      over the open experts (-inf logits are closed)
//   c_te = s_te + b_e          as an FP64 value; a NaN counts as +inf; c = -inf is never chosen (a softmax without
//                              a bias: e^(l - max), the sum being the row's)
//   group g = S adjacent experts, its value the sum of its 1 or 2 largest c; the top_groups groups of
//   the largest values stay (ties: the lower group)
//   S_t = the k largest c among them                          (ties: the lower expert)
//   w_tj = f s / sum_S s,  or  f s                            (the bias chooses, it does not weigh)
//   p_te = s_te / sum_open s_te,  L = coef E sum_e (c_e / R) (1 / n) sum_t p_te
//
// The choice is discontinuous, and rounded scores would make it depend on how a score was computed.  So
// it is defined on FP64 values, and computed in FP32 with a bound on the error: where two values that
// decide something (the choice, its order, the last group kept) lie within the bound of each other, and
// are not the same logit with the same bias, the row is chosen again by their FP64 values (late_row).
//
// A row is held by a warp, 32 / G lanes per group (G rounded up to a power of two), so that a group's
// largest values are found by exchanges among its own lanes.  Counts, ranks and offsets as in
// moe_route.cuh, whose later kernels finish the call.
#pragma once
#include "moe_route.cuh"

namespace tst {

struct ScoreParams {
  RouteParams r;
  const float* bias;        // experts, or null
  int32_t groups, size;     // groups of `size` experts
  int32_t lanes;            // lanes per group: 32 / groups rounded up to a power of two
  int32_t top_groups, best;
  int32_t sigmoid;
  float weight_scale;
};

struct ScoreGradParams {
  RouteGradParams r;
  int32_t size, lanes, groups;
  int32_t sigmoid;
  float weight_scale;
};

// Which experts a lane holds: W adjacent ones in each run of lanes * W of its group.
template <typename T, int VPL>
struct ScoreMap {
  static constexpr int W = VPL < static_cast<int>(16 / sizeof(T)) ? VPL : static_cast<int>(16 / sizeof(T));
  struct alignas(W * sizeof(T)) Pack { T v[W]; };
  int first, sub, lanes, size;   // the group's first expert, the lane's place in it; size 0 for a lane without a group
  __device__ __forceinline__ ScoreMap(int lane, int lanes_, int size_, int groups) : lanes(lanes_) {
    const int g = lane / lanes_;
    sub = lane - g * lanes_;
    first = g * size_;
    size = g < groups ? size_ : 0;
  }
  __device__ __forceinline__ int inside(int v) const { return (v / W) * lanes * W + sub * W + v % W; }   // place in the group
  __device__ __forceinline__ bool has(int v) const { return inside(v) < size; }
  __device__ __forceinline__ int expert(int v) const { return first + inside(v); }
  template <bool VEC>
  __device__ __forceinline__ void load(const T* src, bool on, float (&x)[VPL]) const {
#pragma unroll
    for (int q = 0; q < VPL / W; ++q) {
      const bool in = on && has(q * W);   // VEC: groups are whole packs
      if (VEC) {
        Pack pk;
        if (in) pk = *reinterpret_cast<const Pack*>(src + expert(q * W));
#pragma unroll
        for (int i = 0; i < W; ++i) x[q * W + i] = in ? logit_value<T>(pk.v[i]) : closed_logit();
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          x[q * W + i] = on && has(q * W + i) ? logit_value<T>(src[expert(q * W + i)]) : closed_logit();
      }
    }
  }
  template <bool VEC>
  __device__ __forceinline__ void store(T* dst, const float (&x)[VPL]) const {
#pragma unroll
    for (int q = 0; q < VPL / W; ++q) {
      if (VEC) {
        Pack pk;
#pragma unroll
        for (int i = 0; i < W; ++i) pk.v[i] = static_cast<T>(x[q * W + i]);
        if (has(q * W)) *reinterpret_cast<Pack*>(dst + expert(q * W)) = pk;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (has(q * W + i)) dst[expert(q * W + i)] = static_cast<T>(x[q * W + i]);
      }
    }
  }
};

// 1 / (1 + e^-x), and 1 less that.  With u = 2^-24 their relative errors are (1.5 |x| + 8) u: the exponent's argument is
// rounded (1.5 |x| u), and ex2, the sum and the quotient add the rest.
struct Sigmoid {
  float s, rest;   // and 1 - s
  __device__ __forceinline__ explicit Sigmoid(float x) {
    const float t = RowExp::exp2_approx(-fabsf(x) * kLog2e), d = __fdividef(1.0f, 1.0f + t);
    s = x >= 0.0f ? d : t * d;
    rest = x >= 0.0f ? t * d : d;
  }
};
// the same without 1 - s, in four operations, to the same bound (below 2^-126: 0): 0 for -inf, a NaN for a NaN
__device__ __forceinline__ float fast_sigmoid(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + RowExp::exp2_approx(-x * kLog2e)));
  return r;
}
// e^-min(m, 0) / (1 + e^-x) for x <= m: scores of which the largest is at least 1/2, however far below 0 the logits are
__device__ __forceinline__ float shifted_sigmoid(float x, float m) {
  return x >= 0.0f ? Sigmoid(x).s : __fdividef(__expf(x - fminf(m, 0.0f)), 1.0f + __expf(x));
}
constexpr float kLowest = -3.4028235e38f;
constexpr float kLeastSum = 8.6736174e-19f;   // 2^-60: sums of sigmoids below this are taken again with a shift

// At least this far apart, two values c computed in FP32 are in the order of their FP64 values.  (Sums of two: in
// score_rows_kernel.)  s: the larger score, c: the larger magnitude.  With u = 2^-24: a score is computed with a relative error below 128 u (sigmoid:
// 1.5 |x| u from the exponent's argument, |x| < 80, and 8 u from ex2, the sum and the quotient; softmax:
// 2.4 |x - top| u and (12 + log2 E) u, and e^x that small is weighed by x), an absolute one below 8 u for
// a sigmoid (s (1 - s) |x| < 0.23), and the bias adds u |c|; twice that for a pair, below 2^-120 flushed.
__device__ __forceinline__ float score_gap(bool sigmoid, float s, float c) {
  const float mine = s * 1.52587890625e-5f;   // 2^-16
  return (sigmoid ? fminf(mine, 1.9073486e-6f) : mine) + fabsf(c) * 2.3841858e-7f + 1.5046328e-36f;   // 2^-19, 2^-22, 2^-119
}

// The row's choice on FP64 values, as defined: lane j gets the j-th.
template <typename T, int VPL>
__device__ __noinline__ int choose_exact(const ScoreParams& p, const T* src, int lane) {
  const ScoreMap<T, VPL> map(lane, p.lanes, p.size, p.groups);
  const double shut = -__longlong_as_double(0x7FF0000000000000ll);
  double c[VPL];
  double top = shut, sum = 0.0;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    c[v] = map.has(v) ? static_cast<double>(logit_value<T>(src[map.expert(v)])) : shut;
    if (!(c[v] <= top)) top = c[v];   // a NaN passes on
  }
  uint32_t open = 0u;
#pragma unroll
  for (int v = 0; v < VPL; ++v) open |= (c[v] != shut ? 1u : 0u) << v;
  if (!p.sigmoid) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double o = __shfl_xor_sync(kFullMask, top, d);
      if (!(o <= top)) top = o;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      c[v] = (open >> v) & 1u ? exp(c[v] - top) : 0.0;
      sum += c[v];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
    if (p.bias == nullptr && sum == sum) sum = 1.0;   // as softmax_exact
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    c[v] = p.sigmoid ? 1.0 / (1.0 + exp(-c[v])) : c[v] / sum;
    if (p.bias != nullptr && map.has(v)) c[v] += static_cast<double>(p.bias[map.expert(v)]);
    if (c[v] != c[v]) c[v] = -shut;
    if (!((open >> v) & 1u)) c[v] = shut;
  }
  if (p.groups > 1) {
    double a = shut, b = shut;   // the largest two
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      b = fmax(b, fmin(a, c[v]));
      a = fmax(a, c[v]);
    }
    for (int d = p.lanes >> 1; d > 0; d >>= 1) {
      const double oa = __shfl_xor_sync(kFullMask, a, d), ob = __shfl_xor_sync(kFullMask, b, d);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    const double mine = p.best == 2 && b != shut ? a + b : a;
    const int g = lane / p.lanes;
    int rank = 0;
    for (int i = 0; i < p.groups; ++i) {
      const double o = __shfl_sync(kFullMask, mine, i * p.lanes);
      rank += o > mine || (o == mine && i < g) ? 1 : 0;
    }
    if (rank >= p.top_groups) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) c[v] = shut;
    }
  }
  int chosen = -1;
  for (int j = 0; j < p.r.top_k; ++j) {
    double best = shut;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (c[v] > best) { best = c[v]; at = map.expert(v); }   // a lane's experts rise with v
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const double o = __shfl_xor_sync(kFullMask, best, d);
      const int oat = __shfl_xor_sync(kFullMask, at, d);
      if (o > best || (o == best && oat < at)) { best = o; at = oat; }
    }
    if (best == shut) break;
    if (lane == j) chosen = at;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (map.expert(v) == at && map.has(v)) c[v] = shut;
  }
  return chosen;
}

// A score as defined, of a row without NaN; peak and sum are softmax's.
__device__ __forceinline__ double score_exact(bool sigmoid, float x, double peak, double sum) {
  const double e = exp(sigmoid ? -static_cast<double>(x) : static_cast<double>(x) - peak);
  return (sigmoid ? 1.0 : e) / (sigmoid ? 1.0 + e : sum);
}
// Softmax's top and sum.  Without a bias the scores are compared as defined, before the division: a sum of 1.
template <typename T, int VPL>
__device__ __forceinline__ void softmax_exact(const ScoreParams& p, const ScoreMap<T, VPL>& map, const T* src, double& peak, double& sum) {
  float x[VPL], top = closed_logit();
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    x[v] = map.has(v) ? logit_value<T>(src[map.expert(v)]) : closed_logit();
    top = fmaxf(top, x[v]);
  }
  peak = static_cast<double>(warp_max(top));
  sum = 1.0;
  if (p.bias == nullptr) return;
  sum = 0.0;
#pragma unroll 4   // that many exponentials side by side
  for (int v = 0; v < VPL; ++v) sum += x[v] != closed_logit() ? exp(static_cast<double>(x[v]) - peak) : 0.0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
}

// What a choice is compared by: its value, and the logit and the bias that gave it.
struct alignas(16) Ranked {
  float c, logit, bias;
  int32_t expert;
  __device__ __forceinline__ bool before(const Ranked& o) const { return c > o.c || (c == o.c && expert < o.expert); }
  // whether the values may be in another order than computed (this one before o)
  __device__ __forceinline__ bool near(const Ranked& o, bool sigmoid) const {
    const float gap = score_gap(sigmoid, fmaxf(c - bias, o.c - o.bias), fmaxf(fabsf(c), fabsf(o.c)));
    return !(c - o.c > gap) && !(logit == o.logit && bias == o.bias);
  }
};

// FP64 numbers as integers of the same order, and back: comparisons in integers, as one in FP64 takes an SM 16 cycles
// (131071 x 256 zeros in 4 of 8 groups, each row chosen here: 2.3 ms with those and an exponential per expert, 0.8 so).
__device__ __forceinline__ long long order64(double x) {
  const long long b = __double_as_longlong(x);
  return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);
}
__device__ __forceinline__ double value64(long long k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7FFFFFFFFFFFFFFFll)); }
constexpr long long kShut64 = static_cast<long long>(0x800FFFFFFFFFFFFFull);   // order64(-inf)

// Whether the lane's group stays, on FP64 values as defined, of which `need` has those of the lane that may be among its
// group's largest two.  Where all of them come of one logit and one bias, one exponential serves.  (Loops that are not
// unrolled: this runs for one row in thousands, and much of the time of such a row is that of fetching its code.)
template <typename T, int VPL>
__device__ __noinline__ bool choose_groups(const ScoreParams& p, const T* src, uint32_t need) {
  const int lane = threadIdx.x & 31;
  const ScoreMap<T, VPL> map(lane, p.lanes, p.size, p.groups);
  auto logit_at = [&](int v) { return logit_value<T>(src[map.expert(v)]); };
  auto bias_at = [&](int v) { return p.bias != nullptr ? p.bias[map.expert(v)] : 0.0f; };
  double peak = 0.0, sum = 1.0;
  if (!p.sigmoid) softmax_exact<T, VPL>(p, map, src, peak, sum);
  const int one = __ffs(__ballot_sync(kFullMask, need != 0u)) - 1;   // (an expert is open)
  const float x0 = __shfl_sync(kFullMask, need != 0u ? logit_at(__ffs(need) - 1) : 0.0f, one);
  const float b0 = __shfl_sync(kFullMask, need != 0u ? bias_at(__ffs(need) - 1) : 0.0f, one);
  bool same = true;
#pragma unroll 1
  for (uint32_t left = need; left != 0u; left &= left - 1u) same = same && logit_at(__ffs(left) - 1) == x0 && bias_at(__ffs(left) - 1) == b0;
  same = __all_sync(kFullMask, same);
  auto key = [&](float x, float bias) {
    const double s = score_exact(p.sigmoid, x, peak, sum);
    return order64(p.bias != nullptr ? s + static_cast<double>(bias) : s);
  };
  const long long all = same ? key(x0, b0) : 0;
  long long a = kShut64, b = kShut64;   // the largest two
#pragma unroll 1
  for (; __any_sync(kFullMask, need != 0u); need &= need - 1u) {
    long long c = kShut64;
    if (need != 0u) c = same ? all : key(logit_at(__ffs(need) - 1), bias_at(__ffs(need) - 1));
    b = max(b, min(a, c));
    a = max(a, c);
  }
#pragma unroll 1
  for (int d = p.lanes >> 1; d > 0; d >>= 1) {
    const long long oa = __shfl_xor_sync(kFullMask, a, d), ob = __shfl_xor_sync(kFullMask, b, d);
    b = max(min(a, oa), max(b, ob));
    a = max(a, oa);
  }
  const long long mine = p.best == 2 && b != kShut64 ? order64(value64(a) + value64(b)) : a;
  const int g = lane / p.lanes;
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < p.groups; ++i) {
    const long long o = __shfl_sync(kFullMask, mine, i * p.lanes);
    rank += o > mine || (o == mine && i < g) ? 1 : 0;
  }
  return rank < p.top_groups && mine != kShut64;
}

// The order of at most 32 listed experts (lane i holds the i-th) on FP64 values as defined: the lane's place.
template <typename T, int VPL>
__device__ __noinline__ int choose_listed(const ScoreParams& p, const T* src, int n, const Ranked& mine) {
  const int lane = threadIdx.x & 31;
  double peak = 0.0, sum = 1.0;
  if (!p.sigmoid) softmax_exact<T, VPL>(p, ScoreMap<T, VPL>(lane, p.lanes, p.size, p.groups), src, peak, sum);
  double s = score_exact(p.sigmoid, mine.logit, peak, sum);
  if (p.bias != nullptr) s += static_cast<double>(mine.bias);
  const long long c = order64(s);
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const long long o = __shfl_sync(kFullMask, c, i);
    const int at = __shfl_sync(kFullMask, mine.expert, i);
    rank += o > c || (o == c && at < mine.expert) ? 1 : 0;
  }
  return rank;
}

// A round per choice, and one more, over values c: for rows whose list would be too long.  Lane j gets the j-th, n of
// them in all; c is used up.
template <typename T, int VPL>
__device__ __noinline__ int choose_rounds(const ScoreMap<T, VPL>& map, const T* src, const float* bias, int k, float (&c)[VPL], Ranked& me) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int j = 0; j <= k; ++j) {
    float b = closed_logit();
    int at = 0xFFFF;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (c[v] > b) { b = c[v]; at = map.expert(v); }   // a lane's experts rise with v
    const float m = warp_max(b);
    if (m == closed_logit()) break;
    const int who = static_cast<int>(__reduce_min_sync(kFullMask, b == m ? static_cast<uint32_t>(at) : 0xFFFFu));
    if (lane == j) me = {m, logit_value<T>(src[who]), bias[who], who};
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (c[v] == m && map.expert(v) == who) c[v] = closed_logit();
    ++n;
  }
  return n;
}

// on ? a : b without a branch.  (Where lanes without a kept group took one, the compiler led them through all that
// follows apart from the others, up to each exchange: 131071 x 256 with 4 of 8 groups 302 us, without 190.)
__device__ __forceinline__ float select(bool on, float a, float b) {
  float r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\tselp.f32 %0, %1, %2, q;\n\t}"
               : "=f"(r)
               : "f"(a), "f"(b), "r"(static_cast<uint32_t>(on)));
  return r;
}

// *at = r where `on`, in shared memory, without a branch
__device__ __forceinline__ void put_ranked(bool on, Ranked* at, const Ranked& r) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t@q st.shared.v4.b32 [%1], {%2, %3, %4, %5};\n\t}"
               :
               : "r"(static_cast<uint32_t>(on)), "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "f"(r.c), "f"(r.logit),
                 "f"(r.bias), "r"(r.expert)
               : "memory");
}

// A row's choice out: lane j holds the j-th and its logit (-1 and -inf where there is none); sum and peak: softmax's of the row.
__device__ __forceinline__ void put_choice(const ScoreParams& p, uint32_t* bitmap, int words, int64_t t0, int r, int chosen, float logit,
                                           float sum, float peak) {
  const int lane = threadIdx.x & 31, k = p.r.top_k;
  float w = 0.0f;
  if (p.sigmoid) {
    w = chosen >= 0 ? fast_sigmoid(logit) : 0.0f;
    if (p.r.normalize) {
      const float z = warp_sum(w);
      if (z < kLeastSum) {   // (no choice: not written)
        const float top = warp_max_nan(logit);
        w = chosen < 0 ? 0.0f : shifted_sigmoid(logit, top);
        w = __fdividef(w, warp_sum(w));
      } else {
        w = __fdividef(w, z);
      }
    }
  } else if (p.r.normalize) {
    const float top = warp_max_nan(logit);
    w = chosen < 0 ? 0.0f : __expf(logit - top);
    w = __fdividef(w, warp_sum(w));
  } else if (chosen >= 0) {
    const RowExp ex(peak);
    w = __fdividef(ex.any(logit), sum);
  }
  if (chosen >= 0) atomicOr(&bitmap[chosen * words + (r >> 5)], 1u << (r & 31));
  if (lane < k) {
    p.r.expert[(t0 + r) * k + lane] = chosen;
    p.r.weight[(t0 + r) * k + lane] = chosen >= 0 ? w * p.weight_scale : 0.0f;
  }
}

// A row that the list left open, whose share of the sums is counted already: by the list again, by rounds where more
// are in reach than it holds, and by choose_exact where a NaN takes part or rounds do not tell.  Loops are not
// unrolled: of ordinary rows one in hundreds comes here, and its time is that of fetching the code.  All rows come where
//   - top_k is more than the lanes of the groups kept: the bound of their lanes' largest then bounds nothing (65536 x 512, 2
//     of 16 groups: k 4 131 us, k 6 532, k 10 648);
//   - sigmoids lie below 2^-18 without biases that hold them apart: gaps are those of scores up to 1 (131071 x 256, 4
//     of 8 groups: logits around -10 175 us, -12 342, -16 and less 5.4 ms).
// `kept`: the lanes whose groups stay, 0 where that is open.
template <typename T, int VPL>
__device__ __noinline__ void late_row(const ScoreParams& p, const float* bias, uint32_t* bitmap, int words, int64_t t0, int r, bool odd,
                                      uint32_t kept, Ranked* list) {
  const int lane = threadIdx.x & 31, k = p.r.top_k;
  const ScoreMap<T, VPL> map(lane, p.lanes, p.size, p.groups);
  const T* const src = static_cast<const T*>(p.r.logits) + (t0 + r) * p.r.ld;
  const bool sigmoid = p.sigmoid != 0;
  float c[VPL], sum = 0.0f, peak = closed_logit(), largest = 1.0f;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    c[v] = map.has(v) ? logit_value<T>(src[map.expert(v)]) : closed_logit();
    peak = max_nan(peak, c[v]);
  }
  peak = warp_max_nan(peak);   // (not -inf: an expert is open)
  const RowExp ex(peak);
  float own = closed_logit();
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const float s = c[v] == closed_logit() ? 0.0f : sigmoid ? fast_sigmoid(c[v]) : ex.any(c[v]);
    sum += s;
    c[v] = c[v] == closed_logit() ? closed_logit() : s;
  }
  sum = warp_sum(sum);
  const float inv = sigmoid ? 1.0f : __fdividef(1.0f, sum);
  if (!sigmoid) largest = fminf(1.0f, 1.1f * inv);
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    c[v] = __fadd_rn(__fmul_rn(c[v], inv), map.has(v) ? bias[map.expert(v)] : 0.0f);   // -inf stays
    own = fmaxf(own, c[v]);
  }
  Ranked me = {closed_logit(), closed_logit(), 0.0f, -1};   // lane j: the j-th
  int n = 0;
  bool exact = odd || sum != sum;
  if (!exact) {
    bool stays = (kept >> lane & 1u) != 0u;
    if (kept == 0u) {
      float a = closed_logit(), b = closed_logit();   // the group's largest two
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        b = fmaxf(b, fminf(a, c[v]));
        a = fmaxf(a, c[v]);
      }
#pragma unroll 1
      for (int d = p.lanes >> 1; d > 0; d >>= 1) {
        const float oa = __shfl_xor_sync(kFullMask, a, d), ob = __shfl_xor_sync(kFullMask, b, d);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
      }
      const float least = p.best == 2 && b != closed_logit() ? b : a;
      const float reach = fmaxf(least - 2.0f * score_gap(sigmoid, largest, least), kLowest);
      uint32_t need = 0u;
#pragma unroll
      for (int v = 0; v < VPL; ++v) need |= (c[v] >= reach ? 1u : 0u) << v;
      stays = choose_groups<T, VPL>(p, src, need);
    }
    if (!stays) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) c[v] = closed_logit();
      own = closed_logit();
    }
    float bound = warp_max(own);
#pragma unroll 1
    for (int j = 1; j < k; ++j) {
      own = own == bound ? closed_logit() : own;
      bound = warp_max(own);
    }
    bound = fmaxf(bound - 2.0f * score_gap(sigmoid, largest, bound), kLowest);
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool has = c[v] >= bound;
      const uint32_t who = __ballot_sync(kFullMask, has);
      const int slot = n + __popc(who & below);
      if (has && slot < kRouteCandidates) list[slot] = {c[v], 0.0f, 0.0f, map.expert(v)};
      n += __popc(who);
    }
    __syncwarp();
    if (n <= kRouteCandidates) {
      if (lane < n) {
        me = list[lane];
        me.logit = logit_value<T>(src[me.expert]);
        me.bias = bias[me.expert];
      }
      const int place = choose_listed<T, VPL>(p, src, n, me);
      __syncwarp();
      if (lane < n) list[place] = me;
      __syncwarp();
      if (lane < n) me = list[lane];
      __syncwarp();
    } else {
      n = choose_rounds<T, VPL>(map, src, bias, k, c, me);
      const Ranked after = {__shfl_down_sync(kFullMask, me.c, 1), __shfl_down_sync(kFullMask, me.logit, 1),
                            __shfl_down_sync(kFullMask, me.bias, 1), 0};
      bool unsure = lane < k && lane + 1 < n && (lane == 31 || me.near(after, sigmoid));   // 32 choices: the 33rd has no lane
      // what is left within reach of the last choice has to be of its logit and bias
      const float last = __shfl_sync(kFullMask, me.c, k - 1), last_logit = __shfl_sync(kFullMask, me.logit, k - 1);
      const float last_bias = __shfl_sync(kFullMask, me.bias, k - 1);
      const float reach = last - score_gap(sigmoid, largest, last);
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (n > k && c[v] >= reach && c[v] != closed_logit())
          unsure = unsure || logit_value<T>(src[map.expert(v)]) != last_logit || bias[map.expert(v)] != last_bias;
      exact = __any_sync(kFullMask, unsure);
    }
  }
  if (exact) {
    me.expert = choose_exact<T, VPL>(p, src, lane);
    me.logit = me.expert >= 0 ? logit_value<T>(src[me.expert]) : closed_logit();
    n = 32;
  }
  const bool mine = lane < k && lane < n && me.expert >= 0;
  put_choice(p, bitmap, words, t0, r, mine ? me.expert : -1, mine ? me.logit : closed_logit(), sum, peak);
}

// A warp per row, with the candidate list of route_rows_kernel on the values c.  Rows that it leaves open (values too
// close, more than the list holds, a NaN, and every row where a bias is a NaN or +inf) are marked, and chosen by
// late_row once all others are done: so the rows that come through carry no call (with calls between them, whose
// registers are then spilled around them, 30 us more of 150).  What bounds it is issue slots, as in route_rows_kernel:
// 131071 x 256 FP32, 4 of 8 groups, k 8, takes 147 us with the two launches after it, 138 of them here, in 861
// instructions a row at 0.74 of the slots; 220 rows are marked.
template <typename T, int VPL, bool VEC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS > 8 ? 1 : VPL <= 8 ? 4 : VPL == 16 ? 2 : 1)
    score_rows_kernel(const __grid_constant__ ScoreParams p) {
  using Map = ScoreMap<T, VPL>;
  extern __shared__ __align__(16) uint32_t route_smem[];
  __shared__ Ranked list[WARPS][kRouteCandidates + 1];   // and one place for what is too much
  __shared__ Ranked ranked[WARPS][kRouteCandidates];
  __shared__ alignas(16) float listed[WARPS][kRouteCandidates];
  __shared__ uint32_t open_rows[8], open_kept[256];      // a bit per row of the chunk; late_row's `kept`
  __shared__ int odd_bias;
  const int E = p.r.experts, k = p.r.top_k, words = p.r.chunk / 32;
  const RouteShared s(route_smem, E, words, WARPS);
  float* const bias = reinterpret_cast<float*>(route_smem + ((E * (words + WARPS + 1) + 1 + 3) & ~3));   // E
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.r.chunk;
  const int rows = static_cast<int>(p.r.tokens - t0 < p.r.chunk ? p.r.tokens - t0 : p.r.chunk);
  const Map map(lane, p.lanes, p.size, p.groups);
  const bool sigmoid = p.sigmoid != 0;

  if (threadIdx.x < 8) open_rows[threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    *s.live = 0;
    odd_bias = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E * words; i += 32 * WARPS) s.bitmap[i] = 0u;
  for (int i = threadIdx.x; i < E; i += 32 * WARPS) {
    const float b = p.bias ? p.bias[i] : 0.0f;
    bias[i] = b;
    if (!(b < __uint_as_float(0x7F800000u))) odd_bias = 1;
  }
  __syncthreads();
  const bool odd = odd_bias != 0;

  float acc[VPL], next[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;
  int live = 0;
  auto source = [&](int r) { return static_cast<const T*>(p.r.logits) + (t0 + r) * p.r.ld; };
  auto routed = [&](int r) { return p.r.mask == nullptr || p.r.mask[t0 + r] != 0; };
  if (warp < rows) map.template load<VEC>(source(warp), routed(warp), next);
  for (int r = warp; r < rows; r += WARPS) {
    float x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] = next[v];
    if (r + WARPS < rows)   // the next row's loads fly while this one is worked on
      map.template load<VEC>(source(r + WARPS), routed(r + WARPS), next);
    // scores, and their share of the row's
    float c[VPL], sum = 0.0f, largest = 1.0f, low = x[0], peak = 0.0f;   // no score is above `largest`; peak: softmax's top
    bool some = true;                                                    // an expert is open
    if (sigmoid) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        c[v] = fast_sigmoid(x[v]);   // 0 where closed
        sum += c[v];
      }
      sum = warp_sum(sum);
      if (sum < kLeastSum) {         // logits below -41 or closed: their shares as such
        float top = x[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) top = max_nan(top, x[v]);
        top = warp_max_nan(top);
        some = top != closed_logit();
        float part[VPL], all = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          part[v] = x[v] == closed_logit() ? 0.0f : shifted_sigmoid(x[v], top);
          all += part[v];
        }
        all = warp_sum(all);
        const float inv = some ? 1.0f / all : 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] = fmaf(part[v], inv, acc[v]);
      } else {
        const float inv = __fdividef(1.0f, sum);
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] = fmaf(c[v], inv, acc[v]);
      }
    } else {
      peak = x[0];
#pragma unroll
      for (int v = 1; v < VPL; ++v) peak = max_nan(peak, x[v]);
      peak = warp_max_nan(peak);
      some = peak != closed_logit();
      const RowExp ex(some ? peak : 0.0f);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        c[v] = x[v] == closed_logit() ? 0.0f : ex.any(x[v]);
        sum += c[v];
      }
      sum = warp_sum(sum);
      const float inv = some ? __fdividef(1.0f, sum) : 0.0f;   // sum <= 1075
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        c[v] = __fmul_rn(c[v], inv);   // not fused with the bias for some experts and not for others: one logit and bias
        acc[v] += c[v];                // have one value
      }
      largest = fminf(1.0f, 1.1f * inv);
    }
    if (!some) {
      put_choice(p, s.bitmap, words, t0, r, -1, closed_logit(), 1.0f, 0.0f);
      continue;
    }
    ++live;
    // the values that choose
    if (p.bias != nullptr) {
#pragma unroll
      for (int q = 0; q < VPL / Map::W; ++q) {
        struct alignas(VEC ? 4 * Map::W < 16 ? 4 * Map::W : 16 : 4) Biases { float v[Map::W]; };
        if (VEC) {
          if (map.has(q * Map::W)) {
            const Biases b = *reinterpret_cast<const Biases*>(bias + map.expert(q * Map::W));
#pragma unroll
            for (int i = 0; i < Map::W; ++i) c[q * Map::W + i] = __fadd_rn(c[q * Map::W + i], b.v[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < Map::W; ++i)
            if (map.has(q * Map::W + i)) c[q * Map::W + i] = __fadd_rn(c[q * Map::W + i], bias[map.expert(q * Map::W + i)]);
        }
      }
    }
#pragma unroll
    for (int v = 1; v < VPL; ++v) low = fminf(low, x[v]);
    if (__any_sync(kFullMask, low == closed_logit())) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) c[v] = x[v] == closed_logit() ? closed_logit() : c[v];
    }
    bool near = odd || sum != sum, kept = true, groups_near = false;
    float own = c[0];   // the lane's largest
    if (p.groups > 1) {
      float b = closed_logit();
      if (p.best == 2) {
#pragma unroll
        for (int v = 1; v < VPL; ++v) {
          b = fmaxf(b, fminf(own, c[v]));
          own = fmaxf(own, c[v]);
        }
      } else {
#pragma unroll
        for (int v = 1; v < VPL; ++v) own = fmaxf(own, c[v]);
      }
      float a = own;
      for (int d = p.lanes >> 1; d > 0; d >>= 1) {
        const float oa = __shfl_xor_sync(kFullMask, a, d);
        if (p.best == 2) b = fmaxf(fminf(a, oa), fmaxf(b, __shfl_xor_sync(kFullMask, b, d)));
        a = fmaxf(a, oa);
      }
      const float second = p.best == 2 ? select(b != closed_logit(), b, 0.0f) : 0.0f;
      // closed for a lane without a group; sums beyond FP32 equal its lowest value, as no open group is closed
      const float mine = fmaxf(a + second, fminf(a, kLowest));
      // what it may be off by goes with the summands, of which a sum of opposite signs keeps nothing: half of a pair's
      // distance for each of two scores, u (|a| + |b|) for the biases, and that again for the sum
      const float off = score_gap(sigmoid, largest, a) + score_gap(sigmoid, 0.0f, second);
      // the last value kept, by rounds; equal values are left to choose_groups
      float left = mine, last = warp_max(left);
      for (int j = 1; j < p.top_groups; ++j) {
        left = left == last ? closed_logit() : left;
        const float m = warp_max(left);
        if (m == closed_logit()) break;   // fewer groups are open
        last = m;
      }
      kept = mine >= last && mine != closed_logit();
      const float least = -warp_max(select(kept, off - mine, closed_logit()));   // of the kept, and the most of the others
      const float first = warp_max(select(kept || mine == closed_logit(), closed_logit(), mine + off));
      groups_near = __popc(__ballot_sync(kFullMask, kept)) > p.top_groups * p.lanes || (first != closed_logit() && !(least > first));
      near = near || groups_near;
      own = select(kept, own, closed_logit());
    } else {
#pragma unroll
      for (int v = 1; v < VPL; ++v) own = fmaxf(own, c[v]);
    }
    Ranked me = {closed_logit(), closed_logit(), 0.0f, -1};   // lane j: the j-th
    int n = 0;
    if (!near) {
      float bound = warp_max(own);
      for (int j = 1; j < k; ++j) {
        own = own == bound ? closed_logit() : own;
        bound = warp_max(own);
      }
      // what is listed: all that may reach the bound; a closed expert reaches none
      bound = fmaxf(bound - 2.0f * score_gap(sigmoid, largest, bound), kLowest);
      bound = select(kept, bound, __uint_as_float(0x7F800000u));   // (no value is +inf here)
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const bool has = c[v] >= bound;
        const uint32_t who = __ballot_sync(kFullMask, has);
        const int slot = n + __popc(who & below);
        put_ranked(has, &list[warp][slot < kRouteCandidates ? slot : kRouteCandidates], {c[v], x[v], 0.0f, map.expert(v)});
        n += __popc(who);
      }
      __syncwarp();
      near = n > kRouteCandidates;
      if (!near) {
        // each finds its rank by comparing itself with the others, two lanes to one when at most 16 are listed
        Ranked mine = list[warp][lane];
        listed[warp][lane] = lane < n ? mine.c : closed_logit();
        __syncwarp();
        const bool halves = n <= 16;
        const float value = halves ? __shfl_sync(kFullMask, mine.c, lane & 15) : mine.c;
        int rank = 0;
        for (int i = 0; i < n; i += halves ? 8 : 4) {
          const float4 o = *reinterpret_cast<const float4*>(&listed[warp][i + (halves ? lane >> 4 << 2 : 0)]);
          rank += static_cast<int>(o.x > value) + static_cast<int>(o.y > value) + static_cast<int>(o.z > value) + static_cast<int>(o.w > value);
        }
        if (halves) rank += __shfl_xor_sync(kFullMask, rank, 16);
        if (__popc(__reduce_or_sync(kFullMask, lane < n ? 1u << rank : 0u)) != n) {   // equal ones: the lower expert first
#pragma unroll 1
          for (int i = 0; i < n; ++i)
            rank += static_cast<int>(list[warp][i].c == mine.c) & static_cast<int>(list[warp][i].expert < mine.expert);
        }
        if (lane < n) {
          mine.bias = bias[mine.expert];
          ranked[warp][rank] = mine;
        }
        __syncwarp();
        if (lane < n) me = ranked[warp][lane];
        // neighbours behind the k-th too: one there may belong before several of one logit and bias
        near = __any_sync(kFullMask, lane + 1 < n && me.near(ranked[warp][lane + 1 < n ? lane + 1 : lane], sigmoid));
      }
      __syncwarp();
    }
    if (near) {
      const uint32_t who = __ballot_sync(kFullMask, kept);
      if (lane == 0) {
        open_kept[r] = groups_near ? 0u : who;
        atomicOr(&open_rows[r >> 5], 1u << (r & 31));
      }
      continue;
    }
    const bool mine = lane < k && lane < n;
    put_choice(p, s.bitmap, words, t0, r, mine ? me.expert : -1, mine ? me.logit : closed_logit(), sum, peak);
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (map.has(v)) s.prob[warp * E + map.expert(v)] = acc[v];
  if (lane == 0 && live > 0) atomicAdd(s.live, live);
  __syncthreads();
  int turn = 0;
  for (int i = 0; i < words; ++i)
    for (uint32_t left = open_rows[i]; left != 0u; left &= left - 1u)
      if (turn++ % WARPS == warp) {
        const int r = i * 32 + __ffs(left) - 1;
        late_row<T, VPL>(p, bias, s.bitmap, words, t0, r, odd, open_kept[r], list[warp]);
      }
  finish_chunk(p.r, s, words, WARPS, t0, rows);
}

// The gradient with the choice held fixed: with u_e = s_e dL/ds_e,
//   u_e = p_e (g_e - <p, g>), g_e = dL coef E c_e / (R n), and at the chosen experts
//   + f q_j (dw_j - <q, dw>), q = s / sum_S s   (normalized)   or   + f s_j dw_j,
//   sigmoid: d_l = u (1 - s);  softmax: d_l = u - p sum u.
// A warp per row; the chosen experts' parts pass through shared memory to the lanes that hold them.  The scores are
// computed twice, for the sums and for the gradient, which costs less than registers for them (spilled at 64).  Bound by
// issue slots, 504 instructions a row at 0.67 of them, then by its bytes: 65536 x 256 FP32 in 42 us in a graph, 0.48 of the
// copy rate (48 with the sums over the lanes one after another and the choice read when it was needed).
template <typename T, int VPL, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, VPL <= 8 ? 4 : VPL == 16 ? 2 : 1) score_grad_kernel(const ScoreGradParams p) {
  using Map = ScoreMap<T, VPL>;
  __shared__ alignas(16) float part_all[kRouteWarps][32 * VPL];
  const int E = p.r.experts, k = p.r.top_k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* part = part_all[warp];
  const Map map(lane, p.lanes, p.size, p.groups);
  const bool sigmoid = p.sigmoid != 0;
  const float scale = grad_scale(p.r);
  float g[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    g[v] = map.has(v) ? static_cast<float>(p.r.counts[map.expert(v)]) * scale : 0.0f;
    part[v * 32 + lane] = 0.0f;
  }
  __syncwarp();
  // where an expert's part lies: beside its lane's others
  auto place = [&](int e) {
    const int group = e / p.size, i = e - group * p.size, run = i / (p.lanes * Map::W), j = i - run * p.lanes * Map::W;
    return (run * 32 + group * p.lanes + j / Map::W) * Map::W + j % Map::W;
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps;
  auto routed = [&](int64_t t) { return p.r.mask == nullptr || p.r.mask[t] != 0; };
  auto row = [&](int64_t t) { return static_cast<const T*>(p.r.logits) + t * p.r.ld; };
  // row t's choice of this lane, and that expert's logit: read a row ahead
  auto choice = [&](int64_t t) {
    const int c = t < p.r.tokens && lane < k ? p.r.expert[t * k + lane] : -1;
    return c < E ? c : -1;
  };
  auto logit_of = [&](int64_t t, int c) { return c >= 0 ? logit_value<T>(row(t)[c]) : closed_logit(); };
  float next[VPL];
  int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  int chosen_next = choice(t);
  float logit_next = logit_of(t, chosen_next);
  if (t < p.r.tokens) map.template load<VEC>(row(t), routed(t), next);
  for (; t < p.r.tokens; t += step) {
    T* dst = static_cast<T*>(p.r.d_logits) + t * p.r.d_ld;
    float e[VPL], top = next[0];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      e[v] = next[v];
      top = max_nan(top, e[v]);
    }
    const int chosen = chosen_next;
    const float logit = logit_next;
    float dw = chosen >= 0 && p.r.d_weight != nullptr ? p.r.d_weight[t * k + lane] * p.weight_scale : 0.0f;
    chosen_next = choice(t + step);
    if (t + step < p.r.tokens) map.template load<VEC>(row(t + step), routed(t + step), next);
    top = warp_max_nan(top);
    if (top == closed_logit()) {   // nothing was routed: the row has no part in any output
#pragma unroll
      for (int v = 0; v < VPL; ++v) e[v] = 0.0f;
      map.template store<VEC>(dst, e);
      logit_next = logit_of(t + step, chosen_next);
      continue;
    }
    const RowExp ex(top);
    const float first = p.r.normalize ? warp_max_nan(logit) : 0.0f;   // of the chosen; -inf without any
    float own = 0.0f, sum = 0.0f, dot = 0.0f;   // the choice's score; the row's sums
    if (sigmoid) {
      if (chosen >= 0) own = p.r.normalize ? shifted_sigmoid(logit, first) : Sigmoid(logit).s;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const float s = fast_sigmoid(e[v]);   // 0 where closed
        sum += s;
        dot = fmaf(s, g[v], dot);
      }
    } else {
      if (chosen >= 0) own = p.r.normalize ? __expf(logit - first) : ex.any(logit);
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        e[v] = e[v] == closed_logit() ? 0.0f : ex.any(e[v]);
        sum += e[v];
        dot = fmaf(e[v], g[v], dot);
      }
    }
    // the sums that the row needs in one pass over the lanes, so that their latencies overlap
    float kept = own, kept_dot = own * dw;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      sum += __shfl_xor_sync(kFullMask, sum, m);
      dot += __shfl_xor_sync(kFullMask, dot, m);
      kept += __shfl_xor_sync(kFullMask, kept, m);
      kept_dot += __shfl_xor_sync(kFullMask, kept_dot, m);
    }
    bool small = false;
    if (sigmoid && sum < kLeastSum) {   // as in the forward pass: shares with a shift
      small = true;
      sum = dot = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        const float s = e[v] == closed_logit() ? 0.0f : shifted_sigmoid(e[v], top);
        sum += s;
        dot = fmaf(s, g[v], dot);
      }
      sum = warp_sum(sum);
      dot = warp_sum(dot);
    }
    const float inv = __fdividef(1.0f, sum);
    dot *= inv;
    // the weights' part of u at the chosen experts, and its sum
    float all = 0.0f;
    if (p.r.normalize) {
      const float over = kept > 0.0f || kept != kept ? __fdividef(1.0f, kept) : 0.0f;   // no choice: 0
      dw = own * over * (dw - kept_dot * over);
    } else {
      const float by = sigmoid ? 1.0f : inv;
      dw *= own * by;
      all = kept_dot * by;
    }
    const int at = chosen >= 0 ? place(chosen) : 0;
    if (chosen >= 0) part[at] = dw;
    logit_next = logit_of(t + step, chosen_next);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < VPL / Map::W; ++q) {
      struct alignas(4 * Map::W) Parts { float v[Map::W]; };
      const Parts add = *reinterpret_cast<const Parts*>(part + (q * 32 + lane) * Map::W);
#pragma unroll
      for (int i = 0; i < Map::W; ++i) {
        const int v = q * Map::W + i;
        if (sigmoid) {
          const Sigmoid s(e[v]);
          const float share = small ? e[v] == closed_logit() ? 0.0f : shifted_sigmoid(e[v], top) : s.s;
          const float u = fmaf(share * inv, g[v] - dot, add.v[i]);
          e[v] = e[v] == closed_logit() ? 0.0f : u * s.rest;
        } else {
          const float pe = e[v] * inv;
          e[v] = fmaf(pe, g[v] - dot, add.v[i]) - pe * all;
        }
      }
    }
    __syncwarp();
    if (chosen >= 0) part[at] = 0.0f;
    __syncwarp();
    map.template store<VEC>(dst, e);
  }
}

}  // namespace tst
