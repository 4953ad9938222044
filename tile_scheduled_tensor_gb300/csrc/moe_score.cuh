// Routing of a mixture of experts by scores: sigmoid or softmax, a bias for balance, expert groups,
// scaled weights; and the gradient of the logits.
//
//   s_te = 1 / (1 + e^-l_te),  or  e^l_te / sum_open e^l      over the open experts (-inf logits are closed)
//   c_te = s_te + b_e          as an FP64 value; a NaN counts as +inf; c = -inf is never chosen
//   group g = S adjacent experts, its value the sum of its 1 or 2 largest c; the top_groups groups of
//   the largest values stay (ties: the lower group)
//   S_t = the k largest c among them                          (ties: the lower expert)
//   w_tj = f s / sum_S s,  or  f s                            (the bias chooses, it does not weigh)
//   p_te = s_te / sum_open s_te,  L = coef E sum_e (c_e / R) (1 / n) sum_t p_te
//
// The choice is discontinuous, and rounded scores would make it depend on how a score was computed.  So
// it is defined on FP64 values, and computed in FP32 with a bound on the error: where two values that
// decide something (the choice, its order, the last group kept) lie within the bound of each other, and
// are not the same logit with the same bias, the row is chosen again in FP64 (choose_exact).
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

// 1 / (1 + e^-x) to a few units in the last place, for every x
struct Sigmoid {
  float s, rest;   // and 1 - s
  __device__ __forceinline__ explicit Sigmoid(float x) {
    const float t = RowExp::exp2_approx(-fabsf(x) * kLog2e), d = __fdividef(1.0f, 1.0f + t);
    s = x >= 0.0f ? d : t * d;
    rest = x >= 0.0f ? t * d : d;
  }
};
// e^-min(m, 0) / (1 + e^-x) for x <= m: scores of which the largest is at least 1/2, however far below 0 the logits are
__device__ __forceinline__ float shifted_sigmoid(float x, float m) {
  return x >= 0.0f ? Sigmoid(x).s : __fdividef(__expf(x - fminf(m, 0.0f)), 1.0f + __expf(x));
}
constexpr float kLeastSum = 8.6736174e-19f;   // 2^-60: sums of sigmoids below this are taken again with a shift

// Sums (not maxima) of a group: at least this far apart, two values computed in FP32 are in the order of
// their FP64 values.  With u = 2^-24: a score is computed with a relative error below 128 u (sigmoid:
// 1.5 |x| u from the exponent's argument, |x| < 80, and 8 u from ex2, the sum and the quotient; softmax:
// 2.4 |x - top| u and (12 + log2 E) u, and e^x that small is weighed by x), an absolute one below 8 u for
// a sigmoid (s (1 - s) |x| < 0.23), and the bias adds u |c|; twice that for a pair, below 2^-120 flushed.
__device__ __forceinline__ float score_gap(bool sigmoid, float s, float c) {
  const float mine = s * 1.52587890625e-5f;   // 2^-16
  return (sigmoid ? fminf(mine, 1.9073486e-6f) : mine) + fabsf(c) * 2.3841858e-7f + 1.5046328e-36f;   // 2^-19, 2^-22, 2^-119
}

// c as a value to compare: a NaN before everything
__device__ __forceinline__ float choice_value(float c) { return c != c ? __uint_as_float(0x7F800000u) : c; }

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

// What a choice is compared by: its value, and the logit and the bias that gave it.
struct alignas(16) Ranked {
  float c, logit, bias;
  int32_t expert;
  // whether the values may be in another order than computed (this one before o)
  __device__ __forceinline__ bool near(const Ranked& o, bool sigmoid) const {
    const float gap = score_gap(sigmoid, fmaxf(c - bias, o.c - o.bias), fmaxf(fabsf(c), fabsf(o.c)));
    return !(c - o.c > gap) && !(logit == o.logit && bias == o.bias);
  }
};

// A warp per row, as route_rows_kernel: the same candidate list, on c.
template <typename T, int VPL, bool VEC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS > 8 ? 1 : VPL <= 8 ? 3 : VPL == 16 ? 2 : 1) score_rows_kernel(const ScoreParams p) {
  using Map = ScoreMap<T, VPL>;
  extern __shared__ uint32_t route_smem[];
  __shared__ alignas(16) Candidate list[WARPS][kRouteCandidates];
  __shared__ Ranked ranked[WARPS][kRouteCandidates];
  const int E = p.r.experts, k = p.r.top_k, words = p.r.chunk / 32;
  const RouteShared s(route_smem, E, words, WARPS);
  float* const bias = reinterpret_cast<float*>(s.live + 1);   // E
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.r.chunk;
  const int rows = static_cast<int>(p.r.tokens - t0 < p.r.chunk ? p.r.tokens - t0 : p.r.chunk);
  const Map map(lane, p.lanes, p.size, p.groups);
  const bool sigmoid = p.sigmoid != 0;

  for (int i = threadIdx.x; i < E * words; i += 32 * WARPS) s.bitmap[i] = 0u;
  for (int i = threadIdx.x; i < E; i += 32 * WARPS) bias[i] = p.bias ? p.bias[i] : 0.0f;
  if (threadIdx.x == 0) *s.live = 0;
  __syncthreads();

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
    float best = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) best = max_nan(best, x[v]);
    const RowExp ex(warp_max_nan(best));
    int chosen = -1;
    float w = 0.0f;
    if (ex.top != closed_logit()) {
      ++live;
      // scores, and their share of the row's
      float e[VPL], sum = 0.0f, largest = 1.0f;   // no score is above `largest`
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        e[v] = x[v] == closed_logit() ? 0.0f : sigmoid ? Sigmoid(x[v]).s : ex.any(x[v]);
        sum += e[v];
      }
      sum = warp_sum(sum);
      if (sum < kLeastSum) {   // sigmoids of logits below -41: their shares as such
        float part[VPL], all = 0.0f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          part[v] = x[v] == closed_logit() ? 0.0f : shifted_sigmoid(x[v], ex.top);
          all += part[v];
        }
        const float inv = 1.0f / warp_sum(all);
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] = fmaf(part[v], inv, acc[v]);
      } else {
        const float inv = __fdividef(1.0f, sum);   // sum <= 1075
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          acc[v] = fmaf(e[v], inv, acc[v]);
          if (!sigmoid) e[v] *= inv;
        }
        if (!sigmoid) largest = fminf(1.0f, 1.1f * inv);
      }
      // the values that choose
      float c[VPL];
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        c[v] = x[v] == closed_logit() ? closed_logit() : choice_value(e[v] + (map.has(v) ? bias[map.expert(v)] : 0.0f));
      bool near = false;
      if (p.groups > 1) {
        float a = closed_logit(), b = closed_logit();
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          b = fmaxf(b, fminf(a, c[v]));
          a = fmaxf(a, c[v]);
        }
        for (int d = p.lanes >> 1; d > 0; d >>= 1) {
          const float oa = __shfl_xor_sync(kFullMask, a, d), ob = __shfl_xor_sync(kFullMask, b, d);
          b = fmaxf(fminf(a, oa), fmaxf(b, ob));
          a = fmaxf(a, oa);
        }
        const float mine = p.best == 2 && b != closed_logit() ? a + b : a;
        const int g = lane / p.lanes;
        int rank = 0;
        for (int i = 0; i < p.groups; ++i) {
          const float o = __shfl_sync(kFullMask, mine, i * p.lanes);
          rank += o > mine || (o == mine && i < g) ? 1 : 0;
        }
        const bool kept = rank < p.top_groups;
        // the last group kept and the first one not; the gap of a sum of two whose scores are 1 at most
        const float last = -warp_max(kept && g < p.groups ? -mine : closed_logit()), first = warp_max(kept || g >= p.groups ? closed_logit() : mine);
        const float most = fmaxf(fabsf(last), fabsf(first));
        near = first != closed_logit() && !(last - first > 2.0f * score_gap(sigmoid, largest, most));
        if (!kept) {
#pragma unroll
          for (int v = 0; v < VPL; ++v) c[v] = closed_logit();
        }
      }
      if (!near) {
        float own = c[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) own = fmaxf(own, c[v]);
        float bound = warp_max(own);
        for (int j = 1; j < k; ++j) {
          own = own == bound ? closed_logit() : own;
          bound = warp_max(own);
        }
        // what is listed: all that may reach the bound; a closed expert reaches none
        bound = fmaxf(bound - 2.0f * score_gap(sigmoid, largest, bound), -3.4028235e38f);
        int n = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const bool has = c[v] >= bound;
          const uint32_t who = __ballot_sync(kFullMask, has);
          const int slot = n + __popc(who & below);
          if (has && slot < kRouteCandidates) list[warp][slot] = {c[v], map.expert(v)};
          n += __popc(who);
        }
        __syncwarp();
        Ranked me = {};
        if (n <= kRouteCandidates) {
          // each finds its rank by comparing itself with the others
          Candidate mine = {closed_logit(), E};
          int rank = 0;
          if (lane < n) mine = list[warp][lane];
          for (int i = 0; i < n; ++i) rank += list[warp][i].before(mine) ? 1 : 0;
          if (lane < n) ranked[warp][rank] = {mine.logit, logit_value<T>(source(r)[mine.expert]), bias[mine.expert], mine.expert};
          __syncwarp();
          if (lane < n) me = ranked[warp][lane];
          near = lane < k && lane + 1 < n && me.near(ranked[warp][lane + 1], sigmoid);
          __syncwarp();
        } else {
          // more than the list holds (few lanes left by the groups, many equal values): a round per choice, and one more
          n = 0;
          for (int j = 0; j <= k; ++j) {
            float b = closed_logit();
            int at = E;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
              if (c[v] > b) { b = c[v]; at = map.expert(v); }   // a lane's experts rise with v
            const float m = warp_max(b);
            if (m == closed_logit()) break;
            const int who = static_cast<int>(__reduce_min_sync(kFullMask, b == m ? static_cast<uint32_t>(at) : 0xFFFFu));
            if (lane == j) me = {m, logit_value<T>(source(r)[who]), bias[who], who};
#pragma unroll
            for (int v = 0; v < VPL; ++v)
              if (c[v] == m && map.expert(v) == who) c[v] = closed_logit();
            ++n;
          }
          const Ranked after = {__shfl_down_sync(kFullMask, me.c, 1), __shfl_down_sync(kFullMask, me.logit, 1),
                                __shfl_down_sync(kFullMask, me.bias, 1), 0};
          near = lane < k && lane + 1 < n && (lane == 31 || me.near(after, sigmoid));   // 32 choices: the 33rd has no lane
        }
        near = __any_sync(kFullMask, near);
        if (lane < k && lane < n) chosen = me.expert;
      }
      if (near) chosen = choose_exact<T, VPL>(p, source(r), lane);   // (the whole warp)
      // the weights, from the chosen logits themselves
      const float logit = chosen >= 0 ? logit_value<T>(source(r)[chosen]) : closed_logit();
      if (p.r.normalize) {
        const float top = warp_max_nan(logit);
        w = chosen < 0 ? 0.0f : sigmoid ? shifted_sigmoid(logit, top) : __expf(logit - top);
        w = __fdividef(w, warp_sum(w)) * p.weight_scale;
      } else if (chosen >= 0) {
        w = (sigmoid ? Sigmoid(logit).s : __fdividef(ex.any(logit), sum)) * p.weight_scale;
      }
      if (chosen >= 0) atomicOr(&s.bitmap[chosen * words + (r >> 5)], 1u << (r & 31));
      else w = 0.0f;
    }
    if (lane < k) {
      p.r.expert[(t0 + r) * k + lane] = chosen;
      p.r.weight[(t0 + r) * k + lane] = w;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (map.has(v)) s.prob[warp * E + map.expert(v)] = acc[v];
  if (lane == 0 && live > 0) atomicAdd(s.live, live);
  finish_chunk(p.r, s, words, WARPS, t0, rows);
}

// The gradient with the choice held fixed: with u_e = s_e dL/ds_e,
//   u_e = p_e (g_e - <p, g>), g_e = dL coef E c_e / (R n), and at the chosen experts
//   + f q_j (dw_j - <q, dw>), q = s / sum_S s   (normalized)   or   + f s_j dw_j,
//   sigmoid: d_l = u (1 - s);  softmax: d_l = u - p sum u.
// A warp per row; the chosen experts' parts pass through shared memory to the lanes that hold them.
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
  float next[VPL];
  int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t < p.r.tokens) map.template load<VEC>(static_cast<const T*>(p.r.logits) + t * p.r.ld, routed(t), next);
  for (; t < p.r.tokens; t += step) {
    const T* src = static_cast<const T*>(p.r.logits) + t * p.r.ld;
    T* dst = static_cast<T*>(p.r.d_logits) + t * p.r.d_ld;
    float x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] = next[v];
    int chosen = lane < k ? p.r.expert[t * k + lane] : -1;
    if (chosen >= E) chosen = -1;
    float dw = chosen >= 0 && p.r.d_weight != nullptr ? p.r.d_weight[t * k + lane] * p.weight_scale : 0.0f;
    if (t + step < p.r.tokens)
      map.template load<VEC>(static_cast<const T*>(p.r.logits) + (t + step) * p.r.ld, routed(t + step), next);
    float best = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) best = max_nan(best, x[v]);
    const RowExp ex(warp_max_nan(best));
    if (ex.top == closed_logit()) {   // nothing was routed: the row has no part in any output
#pragma unroll
      for (int v = 0; v < VPL; ++v) x[v] = 0.0f;
      map.template store<VEC>(dst, x);
      continue;
    }
    float e[VPL], rest[VPL], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const bool on = x[v] != closed_logit();
      if (sigmoid) {
        const Sigmoid sg(x[v]);
        e[v] = on ? sg.s : 0.0f;
        rest[v] = on ? sg.rest : 0.0f;
      } else {
        e[v] = on ? ex.any(x[v]) : 0.0f;
        rest[v] = 0.0f;
      }
      sum += e[v];
      dot = fmaf(e[v], g[v], dot);
    }
    const float logit = chosen >= 0 ? logit_value<T>(src[chosen]) : closed_logit();
    sum = warp_sum(sum);
    if (sum < kLeastSum) {   // as in the forward pass
      sum = dot = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        e[v] = x[v] == closed_logit() ? 0.0f : shifted_sigmoid(x[v], ex.top);
        sum += e[v];
        dot = fmaf(e[v], g[v], dot);
      }
      sum = warp_sum(sum);
    }
    const float inv = 1.0f / sum;
    dot = warp_sum(dot) * inv;
    // the weights' part of u at the chosen experts
    float all = 0.0f;   // its sum (softmax without normalisation)
    if (p.r.normalize) {
      const float top = warp_max_nan(logit);
      float q = chosen < 0 ? 0.0f : sigmoid ? shifted_sigmoid(logit, top) : __expf(logit - top);
      const float z = warp_sum(q);
      q = z > 0.0f || z != z ? __fdividef(q, z) : 0.0f;   // no choice: 0
      dw = q * (dw - warp_sum(q * dw));
    } else {
      if (chosen >= 0) dw *= sigmoid ? Sigmoid(logit).s : ex.any(logit) * inv;
      all = warp_sum(dw);
    }
    const int at = chosen >= 0 ? place(chosen) : 0;
    if (chosen >= 0) part[at] = dw;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < VPL / Map::W; ++q) {
      struct alignas(4 * Map::W) Parts { float v[Map::W]; };
      const Parts add = *reinterpret_cast<const Parts*>(part + (q * 32 + lane) * Map::W);
#pragma unroll
      for (int i = 0; i < Map::W; ++i) {
        const int v = q * Map::W + i;
        const float pe = e[v] * inv;
        const float u = fmaf(pe, g[v] - dot, add.v[i]);
        e[v] = sigmoid ? u * rest[v] : u - pe * all;
      }
    }
    __syncwarp();
    if (chosen >= 0) part[at] = 0.0f;
    __syncwarp();
    map.template store<VEC>(dst, e);
  }
}

}  // namespace tst
