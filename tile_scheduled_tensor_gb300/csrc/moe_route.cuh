// Routing of a mixture of experts: the choice of each token's experts, the counts and row order
// that the grouped GEMM reads, the balance loss, and the gradient of the logits.
//
//   p_t = softmax(l_t)                        over the experts; -inf logits are closed experts
//   S_t = the k largest logits of row t       ties to the lower expert, NaN before everything,
//                                             a closed expert never
//   w_tj = p_t[S_tj], or p_t[S_tj] / sum_i p_t[S_ti]
//   c_e = #{(t, j): S_tj = e},  R = sum_e c_e,  n = rows with an open expert
//   L = coef E sum_e (c_e / R) (1 / n) sum_t p_te
//   row_tj = sum_{e' < S_tj} c_e' + #{t' < t: S_tj in S_t'}
//
// The logits are read once, by blocks of `chunk` tokens.  Each block leaves per expert the count
// and the probability sum of its tokens, and each choice's rank inside the chunk, from a bitmap
// (experts x tokens of the chunk) in shared memory: the population count of the bits before the
// token's, so the order does not depend on which warp got there first.  Then (moe_finish.cuh)
// route_scan_kernel turns the chunks' counts into prefix sums, a warp per expert, and
// route_place_kernel adds the experts' and the chunks' offsets to the ranks; few chunks are summed in
// route_sum_place_kernel's blocks, and a call of one chunk does all of it in its one block.  Every floating sum has a fixed order, so a call is repeatable
// bit for bit.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace tst {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteCandidates = 32;
constexpr int kRouteThreadRow = 32;   // up to this many experts a thread holds a whole row
constexpr uint32_t kFullMask = 0xFFFFFFFFu;

struct RouteParams {
  const void* logits;       // tokens x experts, FP32 or BF16, row stride ld
  int64_t ld;
  const uint8_t* mask;      // one byte per token, 0 = not routed; or null
  int32_t* expert;          // tokens x k
  float* weight;            // tokens x k
  int32_t* row;             // tokens x k
  int32_t* counts;          // experts
  int32_t* totals;          // {R, n}
  float* loss;              // 1
  int32_t* part_count;      // (experts + 1) x chunks: the chunks' counts (then prefix sums); last row: live rows
  float* part_prob;         // experts x chunks: the chunks' probability sums
  float* prob;              // experts: the probability sums
  int32_t tokens, experts, top_k, chunk, chunks;
  int32_t normalize;
  float coef;
};

struct RouteGradParams {
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  const int32_t* expert;    // tokens x k
  const int32_t* counts;
  const int32_t* totals;
  const float* d_weight;    // tokens x k, or null
  const float* d_loss;      // 1, or null
  void* d_logits;           // tokens x experts, type of the logits, row stride d_ld
  int64_t d_ld;
  int32_t tokens, experts, top_k;
  int32_t normalize;
  float coef;
};

// An unsigned integer with the order of x; both zeros alike, every NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (x != x) return 0xFFFFFFFFu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kKeyClosed = 0x007FFFFFu;   // order_key(-inf); lower keys stand for no expert
__device__ __forceinline__ float key_value(uint32_t k) {   // a NaN for the NaNs' key
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float closed_logit() { return __uint_as_float(0xFF800000u); }

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
  return v;
}

// e^(x - top).  For |top| below kPlainTop, 2^(x log2 e - top log2 e) with one fused step: the rounding
// of top log2 e, at most 2^-4 there (half a unit in the last place of what lies below 2^21), is a
// factor between 0.95 and 1.05 common to the row, which the division by the row's sum takes out, and
// the step's own rounding is |x - top| 2^-24 relative.  The bound keeps that factor near one: it is up
// to 2^(|top| log2 e 2^-24), which overflows FP32 or vanishes from |top| = 2^30 on.  Beyond, and for
// infinities and NaN: __expf of the difference, which is exact for logits within a factor of two of
// the top.
constexpr float kPlainTop = 1048576.0f;   // 2^20
constexpr float kLog2e = 1.44269504088896341f;
struct RowExp {
  float top, shift;
  bool plain;
  __device__ __forceinline__ explicit RowExp(float t) : top(t), shift(-t * kLog2e), plain(fabsf(t) < kPlainTop) {}
  __device__ __forceinline__ float fast(float x) const { return exp2_approx(fmaf(x, kLog2e, shift)); }
  __device__ __forceinline__ float any(float x) const { return plain ? fast(x) : __expf(x - top); }
  static __device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
  }
};

// A row in a warp's registers: lane l holds W adjacent logits in each run of 32 W, so that a lane's
// loads are up to 16 bytes.  VEC: rows and their starts are multiples of W elements.
template <typename T, int VPL>
struct RowMap {
  static constexpr int W = VPL < static_cast<int>(16 / sizeof(T)) ? VPL : static_cast<int>(16 / sizeof(T));
  struct alignas(W * sizeof(T)) Pack { T v[W]; };
  static __device__ __forceinline__ int expert(int v, int lane) { return (v / W) * 32 * W + lane * W + v % W; }
};

template <typename T>
__device__ __forceinline__ float logit_value(T v);
template <>
__device__ __forceinline__ float logit_value<float>(float v) { return v; }
template <>
__device__ __forceinline__ float logit_value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int VPL, bool VEC>
__device__ __forceinline__ void load_row(const T* src, int E, int lane, bool on, float (&x)[VPL]) {
  using Map = RowMap<T, VPL>;
#pragma unroll
  for (int q = 0; q < VPL / Map::W; ++q) {
    const int e0 = Map::expert(q * Map::W, lane);
    if (VEC) {
      typename Map::Pack pk;
      const bool in = on && e0 < E;
      if (in) pk = *reinterpret_cast<const typename Map::Pack*>(src + e0);
#pragma unroll
      for (int i = 0; i < Map::W; ++i) x[q * Map::W + i] = in ? logit_value<T>(pk.v[i]) : closed_logit();
    } else {
#pragma unroll
      for (int i = 0; i < Map::W; ++i)
        x[q * Map::W + i] = (on && e0 + i < E) ? logit_value<T>(src[e0 + i]) : closed_logit();
    }
  }
}

template <typename T, int VPL, bool VEC>
__device__ __forceinline__ void store_row(T* dst, int E, int lane, const float (&x)[VPL]) {
  using Map = RowMap<T, VPL>;
#pragma unroll
  for (int q = 0; q < VPL / Map::W; ++q) {
    const int e0 = Map::expert(q * Map::W, lane);
    if (VEC) {
      typename Map::Pack pk;
#pragma unroll
      for (int i = 0; i < Map::W; ++i) pk.v[i] = static_cast<T>(x[q * Map::W + i]);
      if (e0 < E) *reinterpret_cast<typename Map::Pack*>(dst + e0) = pk;
    } else {
#pragma unroll
      for (int i = 0; i < Map::W; ++i)
        if (e0 + i < E) dst[e0 + i] = static_cast<T>(x[q * Map::W + i]);
    }
  }
}

// A row of up to EM logits in one thread's registers, 16 bytes at a time where VEC (rows of whole,
// aligned 16-byte units).
template <typename T, int EM, bool VEC>
__device__ __forceinline__ void load_thread_row(const T* src, int E, bool on, float (&x)[EM]) {
  constexpr int V = 16 / sizeof(T) < EM ? 16 / sizeof(T) : EM;
  struct alignas(16) Pack { T v[16 / sizeof(T)]; };
#pragma unroll
  for (int q = 0; q < EM / V; ++q) {
    if (VEC) {
      Pack pk;
      const bool in = on && q * V < E;
      if (in) pk = *reinterpret_cast<const Pack*>(src + q * V);
#pragma unroll
      for (int i = 0; i < V; ++i) x[q * V + i] = in ? logit_value<T>(pk.v[i]) : closed_logit();
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x[q * V + i] = (on && q * V + i < E) ? logit_value<T>(src[q * V + i]) : closed_logit();
    }
  }
}

template <typename T, int EM, bool VEC>
__device__ __forceinline__ void store_thread_row(T* dst, int E, const float (&x)[EM]) {
  constexpr int V = 16 / sizeof(T) < EM ? 16 / sizeof(T) : EM;
  struct alignas(16) Pack { T v[16 / sizeof(T)]; };
#pragma unroll
  for (int q = 0; q < EM / V; ++q) {
    if (VEC) {
      Pack pk;
#pragma unroll
      for (int i = 0; i < V; ++i) pk.v[i] = static_cast<T>(x[q * V + i]);
      if (q * V < E) *reinterpret_cast<Pack*>(dst + q * V) = pk;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (q * V + i < E) dst[q * V + i] = static_cast<T>(x[q * V + i]);
    }
  }
}

// Shared memory of a routing block: the bitmap, each warp's probability sums, the experts' first
// rows (one-chunk calls), the count of live rows.
struct RouteShared {
  uint32_t* bitmap;   // E x words
  float* prob;        // warps x E
  int32_t* first;     // E
  int* live;          // 1
  __device__ __forceinline__ RouteShared(uint32_t* base, int E, int words, int warps) {
    bitmap = base;
    prob = reinterpret_cast<float*>(bitmap + E * words);
    first = reinterpret_cast<int32_t*>(prob + warps * E);
    live = first + E;
  }
};

// What a block does once its tokens' choices are in the bitmap (and in p.expert, written by this
// block): the chunk's counts and sums, and the ranks; or, alone, the final rows and totals.
__device__ __forceinline__ void finish_chunk(const RouteParams& p, const RouteShared& s, int words, int warps, int64_t t0,
                                             int rows) {
  const int E = p.experts, k = p.top_k;
  const bool alone = p.chunks == 1;
  __syncthreads();
  if (!alone) ptx::griddep_launch_dependents();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int c = 0;
    for (int i = 0; i < words; ++i) c += __popc(s.bitmap[e * words + i]);
    float sum = 0.0f;
    for (int i = 0; i < warps; ++i) sum += s.prob[i * E + e];
    if (alone) {
      s.first[e] = c;
      s.prob[e] = sum;   // this thread alone reads column e
      p.counts[e] = c;
    } else {
      p.part_count[static_cast<int64_t>(e) * p.chunks + blockIdx.x] = c;
      p.part_prob[static_cast<int64_t>(e) * p.chunks + blockIdx.x] = sum;
    }
  }
  if (!alone && threadIdx.x == 0) p.part_count[static_cast<int64_t>(E) * p.chunks + blockIdx.x] = *s.live;
  if (alone) {
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int32_t before = 0;
      float dot = 0.0f;
      for (int b = 0; b < E; b += 32) {
        const int e = b + lane;
        const int32_t c = e < E ? s.first[e] : 0;
        if (e < E) dot = fmaf(static_cast<float>(c), s.prob[e], dot);
        int32_t incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int32_t o = __shfl_up_sync(kFullMask, incl, d);
          if (lane >= d) incl += o;
        }
        if (e < E) s.first[e] = before + incl - c;
        before += __shfl_sync(kFullMask, incl, 31);
      }
      dot = warp_sum(dot);
      if (lane == 0) {
        const int live = *s.live;
        p.totals[0] = before;
        p.totals[1] = live;
        *p.loss = before > 0 ? p.coef * static_cast<float>(E) * (dot / static_cast<float>(before) / static_cast<float>(live))
                             : 0.0f;
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < rows * k; i += blockDim.x) {
    const int r = i / k;
    const int e = p.expert[t0 * k + i];
    int rank = -1;
    if (e >= 0) {
      rank = __popc(s.bitmap[e * words + (r >> 5)] & ((1u << (r & 31)) - 1u));
      for (int q = 0; q < (r >> 5); ++q) rank += __popc(s.bitmap[e * words + q]);
      if (alone) rank += s.first[e];
    }
    p.row[t0 * k + i] = rank;
  }
}

// The choice by k rounds of a warp maximum over integer keys: every value, any number of ties.
// The row is read again (it was just read).  Lane j gets the j-th choice.
template <typename T, int VPL, bool VEC>
__device__ __forceinline__ void choose_by_rounds(const T* src, int E, int k, int lane, bool on, int& chosen, float& value) {
  using Map = RowMap<T, VPL>;
  float x[VPL];
  load_row<T, VPL, VEC>(src, E, lane, on, x);
  uint32_t key[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) key[v] = Map::expert(v, lane) < E ? order_key(x[v]) : 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (key[v] > best) { best = key[v]; at = Map::expert(v, lane); }   // a lane's experts rise with v
    const uint32_t m = __reduce_max_sync(kFullMask, best);
    if (m <= kKeyClosed) break;
    const int who = static_cast<int>(__reduce_min_sync(kFullMask, best == m ? static_cast<uint32_t>(at) : 0xFFFFu));
    if (lane == j) { chosen = who; value = key_value(m); }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (Map::expert(v, lane) == who) key[v] = 0u;
  }
}

// A logit that may be among a row's k largest; none is NaN.
struct alignas(8) Candidate {
  float logit;
  int32_t expert;
  __device__ __forceinline__ bool before(const Candidate& c) const {
    return logit > c.logit || (logit == c.logit && expert < c.expert);
  }
};

// A warp per row, rows dealt to the block's warps in turn.  The choice: k - 1 rounds of a warp
// maximum over the lanes' own maxima leave a bound that at least k logits reach; those that do,
// seldom more than a few over k, go to a list in shared memory with their experts,
// and each finds its rank by comparing itself with the others.  Rounds over all logits remain for rows with
// more than 32 on the list, NaN, infinities or a top of 2^20 or more in magnitude.  What bounds it
// is issue slots, not the 1 KB that a row reads: 464 instructions for a row of 256 logits, 0.76 of the
// slots taken while a block runs, 0.68 over the launch, whose 586 blocks end unevenly.  131071 rows of
// 256, k = 8, in 83 us a call with the two launches after it, 235 by rounds alone, 156 where every top
// is at 2^20 or beyond; their bytes take 22 us.  Threads that hold whole or half rows of a tile in shared memory need 230
// to 300 instructions a row, but leave 5 to 10 warps on an SM and measured 128 and 99 us.
// WARPS: 8, or 32 for chunks of 32 tokens that do not fill the SMs: a row's chain of steps, about a
// microsecond, then passes once.
template <typename T, int VPL, bool VEC, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS > 8 ? 1 : VPL <= 8 ? 4 : VPL == 16 ? 2 : 1) route_rows_kernel(const RouteParams p) {
  using Map = RowMap<T, VPL>;
  extern __shared__ __align__(16) uint32_t route_smem[];
  __shared__ alignas(16) Candidate list[WARPS][kRouteCandidates + 4];   // and up to 4 that come last
  const int E = p.experts, k = p.top_k, words = p.chunk / 32;
  const RouteShared s(route_smem, E, words, WARPS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int rows = static_cast<int>(p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk);

  for (int i = threadIdx.x; i < E * words; i += 32 * WARPS) s.bitmap[i] = 0u;
  if (threadIdx.x == 0) *s.live = 0;
  __syncthreads();

  float acc[VPL], next[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;
  int live = 0;
  auto source = [&](int r) { return static_cast<const T*>(p.logits) + (t0 + r) * p.ld; };
  auto routed = [&](int r) { return p.mask == nullptr || p.mask[t0 + r] != 0; };
  if (warp < rows) load_row<T, VPL, VEC>(source(warp), E, lane, routed(warp), next);
  for (int r = warp; r < rows; r += WARPS) {
    float x[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) x[v] = next[v];
    if (r + WARPS < rows)   // the next row's loads fly while this one is worked on
      load_row<T, VPL, VEC>(source(r + WARPS), E, lane, routed(r + WARPS), next);
    float best = x[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) best = max_nan(best, x[v]);
    const RowExp ex(warp_max_nan(best));
    int chosen = -1, at = lane;   // this lane's choice and its place among the row's
    float w = 0.0f;
    if (ex.top != closed_logit()) {
      ++live;
      float e[VPL], sum = 0.0f;
      if (ex.plain) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) { e[v] = ex.fast(x[v]); sum += e[v]; }
      } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) { e[v] = ex.any(x[v]); sum += Map::expert(v, lane) < E ? e[v] : 0.0f; }
      }
      sum = warp_sum(sum);
      const float inv = __fdividef(1.0f, sum);   // 0.95 <= sum <= 1075 (RowExp), or NaN
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[v] = fmaf(e[v], inv, acc[v]);

      bool listed = ex.plain;
      if (listed) {
        float bound = ex.top, own = best;
        for (int j = 1; j < k; ++j) {
          own = own == bound ? closed_logit() : own;
          bound = warp_max(own);
        }
        bound = fmaxf(bound, -3.4028235e38f);   // a closed logit reaches no bound
        int n = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          const bool has = x[v] >= bound;
          const uint32_t who = __ballot_sync(kFullMask, has);
          const int slot = n + __popc(who & below);
          if (has && slot < kRouteCandidates)
            list[warp][slot] = {x[v], Map::expert(v, lane)};
          n += __popc(who);
        }
        listed = n <= kRouteCandidates;
        if (lane < 4 && listed) list[warp][n + lane] = {closed_logit(), E};
        __syncwarp();
        if (listed) {
          // two lanes per listed logit share the comparisons when at most 16 are listed
          const bool halves = n <= 16;
          const int mine = halves ? lane & 15 : lane;
          const Candidate c = list[warp][mine];   // from the n-th on: not used
          const int share = halves ? (n + 3) >> 2 : (n + 1) >> 1;   // pairs
          const int4* pair = reinterpret_cast<const int4*>(list[warp]) + (halves && lane >= 16 ? share : 0);
          int rank = 0;
          for (int i = 0; i < share; ++i) {
            const int4 two = pair[i];
            if (Candidate{__int_as_float(two.x), two.y}.before(c)) ++rank;
            if (Candidate{__int_as_float(two.z), two.w}.before(c)) ++rank;
          }
          if (halves) rank += __shfl_xor_sync(kFullMask, rank, 16);
          if (lane < n) {
            at = rank;   // from the k-th on: no place; the other lanes keep theirs, -1 where fewer than k are open
            if (rank < k) {
              chosen = c.expert;
              w = ex.fast(c.logit);
            }
          }
        }
        __syncwarp();
      }
      if (!listed) {
        float value = 0.0f;
        choose_by_rounds<T, VPL, VEC>(source(r), E, k, lane, true, chosen, value);
        if (chosen >= 0) w = ex.any(value);
      }
      const float over = p.normalize ? warp_sum(w) : sum;
      w = chosen >= 0 ? __fdividef(w, over) : 0.0f;   // 0.95 <= over <= 1075, or NaN
      if (chosen >= 0) atomicOr(&s.bitmap[chosen * words + (r >> 5)], 1u << (r & 31));
    }
    if (at < k) {
      p.expert[(t0 + r) * k + at] = chosen;
      p.weight[(t0 + r) * k + at] = w;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (Map::expert(v, lane) < E) s.prob[warp * E + Map::expert(v, lane)] = acc[v];
  if (lane == 0 && live > 0) atomicAdd(s.live, live);
  finish_chunk(p, s, words, WARPS, t0, rows);
}

// A thread per row, for up to 32 experts: the logits, their keys and the k rounds stay in one
// thread's registers, with no exchange between lanes but for the probability sums.  A block has a
// thread per token of its chunk; choices pass through shared memory so that they leave in order.
// 60000 x 32 in 22 us, 131071 x 8 in 14 us, the two launches after it included.
template <typename T, int EM, bool VEC>
__global__ void __launch_bounds__(kRouteThreads) route_rows_small_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint32_t route_smem[];
  const int E = p.experts, k = p.top_k, words = p.chunk / 32, warps = words;
  const RouteShared s(route_smem, E, words, warps);
  const int pitch = k | 1;   // odd: a warp's threads write distinct banks
  int32_t* out_expert = reinterpret_cast<int32_t*>(s.live + 1);
  float* out_weight = reinterpret_cast<float*>(out_expert + p.chunk * pitch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int rows = static_cast<int>(p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk);
  const int r = threadIdx.x;
  if (threadIdx.x == 0) *s.live = 0;
  __syncthreads();

  const bool on = r < rows && (p.mask == nullptr || p.mask[t0 + r] != 0);
  const T* src = static_cast<const T*>(p.logits) + (t0 + r) * p.ld;
  float x[EM];
  uint32_t key[EM], top_key = 0u;
  load_thread_row<T, EM, VEC>(src, E, on, x);
#pragma unroll
  for (int e = 0; e < EM; ++e) {
    key[e] = e < E ? order_key(x[e]) : 0u;
    top_key = key[e] > top_key ? key[e] : top_key;
  }
  const bool live = top_key > kKeyClosed;
  const RowExp ex(key_value(top_key));
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < EM; ++e) {
    x[e] = live && e < E ? ex.any(x[e]) : 0.0f;
    sum += x[e];
  }
  uint32_t taken = 0u;
  float chosen_sum = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = kKeyClosed;
    int at = -1;
#pragma unroll
    for (int e = 0; e < EM; ++e)
      if (key[e] > best) { best = key[e]; at = e; }
    float w = 0.0f;
#pragma unroll
    for (int e = 0; e < EM; ++e)
      if (e == at) { key[e] = 0u; w = x[e]; }
    if (at >= 0) taken |= 1u << at;
    chosen_sum += w;
    out_expert[r * pitch + j] = at;
    out_weight[r * pitch + j] = w;
  }
  const float inv = live ? 1.0f / sum : 0.0f;
  const float over = live ? 1.0f / (p.normalize ? chosen_sum : sum) : 0.0f;
  const uint32_t live_rows = __ballot_sync(kFullMask, live);
  if (lane == 0 && live_rows != 0u) atomicAdd(s.live, __popc(live_rows));
  for (int j = 0; j < k; ++j) out_weight[r * pitch + j] *= over;
#pragma unroll
  for (int e = 0; e < EM; ++e) {
    if (e < E) {
      const uint32_t bits = __ballot_sync(kFullMask, (taken >> e) & 1u);
      const float q = warp_sum(x[e] * inv);
      if (lane == 0) {
        s.bitmap[e * words + warp] = bits;
        s.prob[warp * E + e] = q;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * k; i += blockDim.x) {
    const int row = i / k, j = i - row * k;
    const int e = out_expert[row * pitch + j];
    p.expert[t0 * k + i] = e;
    p.weight[t0 * k + i] = e >= 0 ? out_weight[row * pitch + j] : 0.0f;
  }
  finish_chunk(p, s, words, warps, t0, rows);
}

// d_l = p (g - <p, g>) with g_e = dL coef E c_e / (R n), the counts held fixed, plus the weights'
// part: without normalisation dw joins g at the chosen experts; with it the weights are a softmax
// over the chosen logits alone, so w (dw - <w, dw>) is added there.  The probabilities are
// computed again from the logits, which costs less than reading them would.
__device__ __forceinline__ float grad_scale(const RouteGradParams& p) {
  if (p.d_loss == nullptr) return 0.0f;
  const float rows = static_cast<float>(p.totals[0] > 0 ? p.totals[0] : 1);
  const float live = static_cast<float>(p.totals[1] > 0 ? p.totals[1] : 1);
  return *p.d_loss * (p.coef * static_cast<float>(p.experts)) / (rows * live);
}

// A warp per row; the chosen experts' parts pass through a row of shared memory to the lanes that
// hold those experts.  Bound by memory, the logits in and the gradient out, with a row's chain of loads,
// exponentials and sums over the lanes hidden behind the other warps': 65536 x 256 float32 in 27.5 us in
// a graph, 0.74 of the copy rate, and 29 to 30 a call.  The sums over the lanes go together, one latency for all of them.
template <typename T, int VPL, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, VPL <= 8 ? 4 : VPL == 16 ? 2 : 1) route_grad_kernel(const RouteGradParams p) {
  using Map = RowMap<T, VPL>;
  __shared__ alignas(16) float part_all[kRouteWarps][32 * VPL];
  const int E = p.experts, k = p.top_k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* part = part_all[warp];
  const float scale = grad_scale(p);
  float g[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int e = Map::expert(v, lane);
    g[v] = e < E ? static_cast<float>(p.counts[e]) * scale : 0.0f;
    part[v * 32 + lane] = 0.0f;
  }
  __syncwarp();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps;
  auto routed = [&](int64_t t) { return p.mask == nullptr || p.mask[t] != 0; };
  // Row t's choice of this lane, and that expert's logit: read a row ahead, where the registers for it
  // are there (65536 x 256: in bf16 24.8 us with the spills it costs, 22.5 without; in float32 27.8 against
  // 29.1; 65536 x 512: 49 us against 65 in bf16, 52 against 57 in float32).
  constexpr bool kAhead = sizeof(T) == 4 || VPL != 8;
  auto choice = [&](int64_t t) { return t < p.tokens && lane < k ? p.expert[t * k + lane] : -1; };
  auto logit_of = [&](int64_t t, int c) {
    return c >= 0 && c < E ? logit_value<T>(static_cast<const T*>(p.logits)[t * p.ld + c]) : 0.0f;
  };
  float next[VPL];
  int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  int chosen_next = kAhead ? choice(t) : -1;
  float logit_next = logit_of(t, chosen_next);
  if (t < p.tokens) load_row<T, VPL, VEC>(static_cast<const T*>(p.logits) + t * p.ld, E, lane, routed(t), next);
  for (; t < p.tokens; t += step) {
    T* dst = static_cast<T*>(p.d_logits) + t * p.d_ld;
    float e[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) e[v] = next[v];
    int chosen = kAhead ? chosen_next : choice(t);
    const float logit = kAhead ? logit_next : logit_of(t, chosen);
    float dw = lane < k && p.d_weight != nullptr ? p.d_weight[t * k + lane] : 0.0f;
    if constexpr (kAhead) chosen_next = choice(t + step);
    if (t + step < p.tokens)
      load_row<T, VPL, VEC>(static_cast<const T*>(p.logits) + (t + step) * p.ld, E, lane, routed(t + step), next);
    float best = e[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v) best = max_nan(best, e[v]);
    const RowExp ex(warp_max_nan(best));
    if (ex.top == closed_logit()) {   // nothing was routed: the row has no part in any output
#pragma unroll
      for (int v = 0; v < VPL; ++v) e[v] = 0.0f;
      store_row<T, VPL, VEC>(dst, E, lane, e);
      if constexpr (kAhead) logit_next = logit_of(t + step, chosen_next);
      continue;
    }
    if (chosen >= E) chosen = -1;
    float ew = 0.0f;
    if (chosen >= 0) ew = ex.any(logit);
    else dw = 0.0f;
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      e[v] = ex.any(e[v]);
      if (!ex.plain && Map::expert(v, lane) >= E) e[v] = 0.0f;
      sum += e[v];
      dot = fmaf(e[v], g[v], dot);
    }
    // the sums that the row needs in one pass over the lanes, so that their latencies overlap
    float kept = ew, kept_dot = ew * dw;
    if (!p.normalize) dot += kept_dot;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      sum += __shfl_xor_sync(kFullMask, sum, m);
      dot += __shfl_xor_sync(kFullMask, dot, m);
      if (p.normalize) {
        kept += __shfl_xor_sync(kFullMask, kept, m);
        kept_dot += __shfl_xor_sync(kFullMask, kept_dot, m);
      }
    }
    const float inv = __fdividef(1.0f, sum);
    dot *= inv;
    if (p.normalize) {
      const float over = __fdividef(1.0f, kept);
      dw = ew * over * (dw - kept_dot * over);   // already the gradient of the chosen logits
    }
    if (chosen >= 0) part[chosen] = dw;
    if constexpr (kAhead) logit_next = logit_of(t + step, chosen_next);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < VPL / Map::W; ++q) {
      struct alignas(4 * Map::W) Parts { float v[Map::W]; };
      const Parts add = *reinterpret_cast<const Parts*>(part + Map::expert(q * Map::W, lane));
#pragma unroll
      for (int i = 0; i < Map::W; ++i) {
        const int v = q * Map::W + i;
        const float pe = e[v] * inv;
        e[v] = p.normalize ? fmaf(pe, g[v] - dot, add.v[i]) : pe * (g[v] + add.v[i] - dot);
      }
    }
    __syncwarp();
    if (chosen >= 0) part[chosen] = 0.0f;
    __syncwarp();
    store_row<T, VPL, VEC>(dst, E, lane, e);
  }
}

// A thread per row, for up to 32 experts: 60000 x 32 in 10.6 us, 131071 x 8 in 4.8 us.
template <typename T, int EM, bool VEC>
__global__ void __launch_bounds__(kRouteThreads) route_grad_small_kernel(const RouteGradParams p) {
  __shared__ float g[EM];
  const int E = p.experts, k = p.top_k;
  const float scale = grad_scale(p);
  for (int e = threadIdx.x; e < E; e += blockDim.x) g[e] = static_cast<float>(p.counts[e]) * scale;
  __syncthreads();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= p.tokens) return;
  const bool on = p.mask == nullptr || p.mask[t] != 0;
  const T* src = static_cast<const T*>(p.logits) + t * p.ld;
  T* dst = static_cast<T*>(p.d_logits) + t * p.d_ld;
  float x[EM];
  float top = closed_logit();
  load_thread_row<T, EM, VEC>(src, E, on, x);
#pragma unroll
  for (int e = 0; e < EM; ++e) top = max_nan(top, x[e]);
  const RowExp ex(top);
  const bool live = top != closed_logit();
  float sum = 0.0f, dot = 0.0f, chosen_sum = 0.0f, chosen_dot = 0.0f;
#pragma unroll
  for (int e = 0; e < EM; ++e) {
    x[e] = live && e < E ? ex.any(x[e]) : 0.0f;
    sum += x[e];
    dot = fmaf(x[e], e < E ? g[e] : 0.0f, dot);
  }
  // each chosen expert's dw where that expert's logit is
  float add[EM];
  uint32_t taken = 0u;
#pragma unroll
  for (int e = 0; e < EM; ++e) add[e] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int c = live ? p.expert[t * k + j] : -1;
    const float d = (c >= 0 && p.d_weight != nullptr) ? p.d_weight[t * k + j] : 0.0f;
    if (c >= 0 && c < EM) taken |= 1u << c;
#pragma unroll
    for (int e = 0; e < EM; ++e)
      if (e == c) {
        add[e] = d;
        chosen_sum += x[e];
        chosen_dot = fmaf(x[e], d, chosen_dot);
      }
  }
  const float inv = live ? 1.0f / sum : 0.0f;
  const float over = (live && taken != 0u) ? 1.0f / chosen_sum : 0.0f;
  dot = (p.normalize ? dot : dot + chosen_dot) * inv;
  chosen_dot *= over;
#pragma unroll
  for (int e = 0; e < EM; ++e) {
    if (e < E) {
      const float pe = x[e] * inv;
      float d = p.normalize ? pe * (g[e] - dot) : pe * (g[e] + add[e] - dot);
      if (p.normalize && ((taken >> e) & 1u)) d = fmaf(x[e] * over, add[e] - chosen_dot, d);
      x[e] = live ? d : 0.0f;
    }
  }
  store_thread_row<T, EM, VEC>(dst, E, x);
}

}  // namespace tst
