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
// Three launches.  route_rows_kernel reads the logits once: a warp holds a row's logits in
// registers, its maximum is the first chosen logit, and a block leaves per expert the count and
// the probability sum of its chunk of tokens, and each choice's rank inside the chunk.  Ranks come
// from a bitmap (experts x tokens of the chunk) in shared memory: the population count of the
// bits before the token's, so the order never depends on which warp got there first.
// route_scan_kernel turns the chunks' counts into prefix sums, a warp per expert.
// route_place_kernel adds the experts' and the chunk's offsets to the ranks.  Every floating
// sum has a fixed order, so a call is repeatable bit for bit.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace tst {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
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
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullMask, v, d);
  return v;
}

// __expf: its argument here is x - max <= 0; its relative error, 2^-22 and a term growing as
// |x| 2^-24, stays below 1e-6 for every term that a sum of at most 1024 of them can notice.
__device__ __forceinline__ float exp_shifted(float x, float top) { return __expf(x - top); }

// VPL: logits per lane; expert e of a row is slot e / 32 of lane e % 32.
template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_rows_kernel(const RouteParams p) {
  extern __shared__ uint32_t route_smem[];
  const int E = p.experts, k = p.top_k, words = p.chunk / 32;
  uint32_t* bitmap = route_smem;                                       // E x words
  float* prob = reinterpret_cast<float*>(bitmap + E * words);          // warps x E
  int* live_rows = reinterpret_cast<int*>(prob + kRouteWarps * E);     // 1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int rows = static_cast<int>(p.tokens - t0 < p.chunk ? p.tokens - t0 : p.chunk);

  for (int i = threadIdx.x; i < E * words; i += kRouteThreads) bitmap[i] = 0u;
  if (threadIdx.x == 0) *live_rows = 0;
  __syncthreads();

  float acc[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v] = 0.0f;
  for (int r = warp; r < rows; r += kRouteWarps) {
    const int64_t t = t0 + r;
    const bool on = p.mask == nullptr || p.mask[t] != 0;
    const T* src = static_cast<const T*>(p.logits) + t * p.ld;
    uint32_t key[VPL];
    float e[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int x = v * 32 + lane;
      e[v] = (on && x < E) ? load_logit(src + x) : __uint_as_float(0xFF800000u);
      key[v] = x < E ? order_key(e[v]) : 0u;
    }
    int chosen = -1;           // lane j: the j-th expert, its logit's key
    uint32_t chosen_key = 0u;
    uint32_t top_key = 0u;
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (key[v] > best) { best = key[v]; at = v; }
      const uint32_t m = __reduce_max_sync(kFullMask, best);
      if (j == 0) top_key = m;
      if (m <= kKeyClosed) break;
      const uint32_t who = __reduce_min_sync(kFullMask, best == m ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFu);
      if (lane == j) { chosen = static_cast<int>(who); chosen_key = m; }
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (static_cast<uint32_t>(v * 32 + lane) == who) key[v] = 0u;
    }
    const bool live = top_key > kKeyClosed;
    float w = 0.0f;
    if (live) {
      const float top = top_key == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : key_value(top_key);
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        e[v] = v * 32 + lane < E ? exp_shifted(e[v], top) : 0.0f;
        sum += e[v];
      }
      sum = warp_sum(sum);
      const float inv = 1.0f / sum;
#pragma unroll
      for (int v = 0; v < VPL; ++v) acc[v] = fmaf(e[v], inv, acc[v]);
      if (chosen >= 0)
        w = exp_shifted(chosen_key == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : key_value(chosen_key), top);
      const float over = p.normalize ? warp_sum(w) : sum;
      w = w / over;
      if (chosen < 0) w = 0.0f;
      if (lane == 0) atomicAdd(live_rows, 1);
      if (chosen >= 0) atomicOr(&bitmap[chosen * words + (r >> 5)], 1u << (r & 31));
    }
    if (lane < k) {
      p.expert[t * k + lane] = chosen;
      p.weight[t * k + lane] = w;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; ++v)
    if (v * 32 + lane < E) prob[warp * E + v * 32 + lane] = acc[v];
  __syncthreads();

  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    int c = 0;
    for (int i = 0; i < words; ++i) c += __popc(bitmap[e * words + i]);
    float s = 0.0f;
    for (int i = 0; i < kRouteWarps; ++i) s += prob[i * E + e];
    p.part_count[static_cast<int64_t>(e) * p.chunks + blockIdx.x] = c;
    p.part_prob[static_cast<int64_t>(e) * p.chunks + blockIdx.x] = s;
  }
  if (threadIdx.x == 0) p.part_count[static_cast<int64_t>(E) * p.chunks + blockIdx.x] = *live_rows;
  // this block's own writes of p.expert, read back after the barrier
  for (int i = threadIdx.x; i < rows * k; i += kRouteThreads) {
    const int r = i / k;
    const int e = p.expert[t0 * k + i];
    int rank = -1;
    if (e >= 0) {
      rank = __popc(bitmap[e * words + (r >> 5)] & ((1u << (r & 31)) - 1u));
      for (int q = 0; q < (r >> 5); ++q) rank += __popc(bitmap[e * words + q]);
    }
    p.row[t0 * k + i] = rank;
  }
}

// A warp per expert (and one for the live rows): the chunks' counts become exclusive prefix
// sums, their total counts[e]; the probability sums are added in a fixed order.
__global__ void __launch_bounds__(kRouteThreads) route_scan_kernel(const RouteParams p) {
  const int e = blockIdx.x * kRouteWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e > p.experts) return;
  int32_t* count = p.part_count + static_cast<int64_t>(e) * p.chunks;
  int32_t before = 0;
  float s = 0.0f;
  for (int b = 0; b < p.chunks; b += 32) {
    const bool in = b + lane < p.chunks;
    const int32_t c = in ? count[b + lane] : 0;
    if (e < p.experts && in) s += p.part_prob[static_cast<int64_t>(e) * p.chunks + b + lane];
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kFullMask, incl, d);
      if (lane >= d) incl += o;
    }
    if (in) count[b + lane] = before + incl - c;
    before += __shfl_sync(kFullMask, incl, 31);
  }
  s = warp_sum(s);
  if (lane == 0) {
    if (e < p.experts) {
      p.counts[e] = before;
      p.prob[e] = s;
    } else {
      p.totals[1] = before;
    }
  }
}

// Rows of a chunk's choices: the rank inside the chunk, the chunk's offset inside the expert and
// the expert's first row.  The last block writes R and the loss too.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const RouteParams p) {
  extern __shared__ uint32_t route_smem[];
  int32_t* first = reinterpret_cast<int32_t*>(route_smem);   // E: first row of each expert
  __shared__ int32_t warp_total[kRouteWarps];
  __shared__ float warp_loss[kRouteWarps];
  const int E = p.experts, k = p.top_k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t before = 0;
  for (int b = 0; b < E; b += kRouteThreads) {
    const int e = b + static_cast<int>(threadIdx.x);
    const int32_t c = e < E ? p.counts[e] : 0;
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kFullMask, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    int32_t add = before, all = 0;
    for (int w = 0; w < kRouteWarps; ++w) {
      if (w < warp) add += warp_total[w];
      all += warp_total[w];
    }
    if (e < E) first[e] = add + incl - c;
    before += all;
    __syncthreads();
  }
  if (blockIdx.x == gridDim.x - 1) {
    const int32_t live = p.totals[1];
    float s = 0.0f;
    for (int e = threadIdx.x; e < E; e += kRouteThreads)
      s += (static_cast<float>(p.counts[e]) / static_cast<float>(before > 0 ? before : 1)) *
           (p.prob[e] / static_cast<float>(live > 0 ? live : 1));
    s = warp_sum(s);
    if (lane == 0) warp_loss[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float all = 0.0f;
      for (int w = 0; w < kRouteWarps; ++w) all += warp_loss[w];
      p.totals[0] = before;
      *p.loss = p.coef * static_cast<float>(E) * all;
    }
  }
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int64_t left = static_cast<int64_t>(p.tokens) - t0;
  const int rows = static_cast<int>(left < p.chunk ? left : p.chunk);
  for (int i = threadIdx.x; i < rows * k; i += kRouteThreads) {
    const int e = p.expert[t0 * k + i];
    if (e >= 0) p.row[t0 * k + i] += first[e] + p.part_count[static_cast<int64_t>(e) * p.chunks + blockIdx.x];
  }
}

// d_l = p (g - <p, g>) with g_e = dL coef E c_e / (R n), the counts held fixed, plus the weights'
// part: without normalisation dw joins g at the chosen experts; with it the weights are a softmax
// over the chosen logits alone, so w (dw - <w, dw>) is added there.  A warp per row; the
// probabilities are computed again from the logits, which costs less than reading them would.
template <typename T, int VPL>
__global__ void __launch_bounds__(kRouteThreads) route_grad_kernel(const RouteGradParams p) {
  extern __shared__ uint32_t route_smem[];
  float* g_shared = reinterpret_cast<float*>(route_smem);
  const int E = p.experts, k = p.top_k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float rows_total = static_cast<float>(p.totals[0] > 0 ? p.totals[0] : 1);
  const float live_total = static_cast<float>(p.totals[1] > 0 ? p.totals[1] : 1);
  const float scale = p.d_loss ? *p.d_loss * (p.coef * static_cast<float>(E)) / (rows_total * live_total) : 0.0f;
  for (int e = threadIdx.x; e < E; e += kRouteThreads) g_shared[e] = static_cast<float>(p.counts[e]) * scale;
  __syncthreads();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp; t < p.tokens; t += step) {
    const bool on = p.mask == nullptr || p.mask[t] != 0;
    const T* src = static_cast<const T*>(p.logits) + t * p.ld;
    T* dst = static_cast<T*>(p.d_logits) + t * p.d_ld;
    float e[VPL];
    uint32_t key = 0u;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int x = v * 32 + lane;
      e[v] = (on && x < E) ? load_logit(src + x) : __uint_as_float(0xFF800000u);
      const uint32_t kv = order_key(e[v]);
      key = kv > key ? kv : key;
    }
    key = __reduce_max_sync(kFullMask, key);
    if (key <= kKeyClosed) {   // nothing was routed: the row has no part in any output
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (v * 32 + lane < E) dst[v * 32 + lane] = static_cast<T>(0.0f);
      continue;
    }
    const float top = key == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : key_value(key);
    int chosen = lane < k ? p.expert[t * k + lane] : -1;
    if (chosen >= E) chosen = -1;
    float dw = (chosen >= 0 && p.d_weight) ? p.d_weight[t * k + lane] : 0.0f;
    const float ew = chosen >= 0 ? exp_shifted(load_logit(src + chosen), top) : 0.0f;
    if (p.normalize) {
      const float w = ew / warp_sum(ew);
      dw = w * (dw - warp_sum(w * dw));   // already the gradient of the chosen logits
    }
    float sum = 0.0f, dot = 0.0f;
    float g[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int x = v * 32 + lane;
      e[v] = x < E ? exp_shifted(e[v], top) : 0.0f;
      g[v] = x < E ? g_shared[x] : 0.0f;
      sum += e[v];
      dot = fmaf(e[v], g[v], dot);
    }
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    if (!p.normalize) dot += warp_sum(ew * dw);
    const float inv = 1.0f / sum;
    dot *= inv;
#pragma unroll
    for (int v = 0; v < VPL; ++v) e[v] *= inv;
    float add[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v) add[v] = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int x = __shfl_sync(kFullMask, chosen, j);
      const float d = __shfl_sync(kFullMask, dw, j);
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (x == v * 32 + lane) add[v] = d;
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int x = v * 32 + lane;
      if (x < E)
        dst[x] = static_cast<T>(p.normalize ? fmaf(e[v], g[v] - dot, add[v]) : e[v] * (g[v] + add[v] - dot));
    }
  }
}

}  // namespace tst
