// The kernels that finish a routing call of several chunks (moe_route.cuh, moe_score.cuh): prefix sums
// of the chunks' counts, the rows of the choices, totals and the balance loss.
#pragma once
#include "moe_route.cuh"

namespace tst {

// A warp per expert (and one for the live rows): the chunks' counts become exclusive prefix
// sums, their total counts[e]; the probability sums are added in a fixed order.  A lane takes 8
// values, 32 apart, in flight at once.
__global__ void __launch_bounds__(kRouteThreads) route_scan_kernel(const RouteParams p) {
  constexpr int PER = 8;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int e = blockIdx.x * kRouteWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e > p.experts) return;
  int32_t* count = p.part_count + static_cast<int64_t>(e) * p.chunks;
  const float* part = p.part_prob + static_cast<int64_t>(e) * p.chunks;
  int32_t before = 0;
  float s = 0.0f;
  for (int b = 0; b < p.chunks; b += 32 * PER) {
    int32_t c[PER];
    float q[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = b + i * 32 + lane;
      c[i] = at < p.chunks ? count[at] : 0;
      q[i] = (at < p.chunks && e < p.experts) ? part[at] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = b + i * 32 + lane;
      s += q[i];
      int32_t incl = c[i];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(kFullMask, incl, d);
        if (lane >= d) incl += o;
      }
      if (at < p.chunks) count[at] = before + incl - c[i];
      before += __shfl_sync(kFullMask, incl, 31);
    }
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

// Exclusive sums of totals[0 .. E) added to first[0 .. E), by a whole block; returns their sum.
__device__ __forceinline__ int32_t add_first_rows(const int32_t* totals, int32_t* first, int E) {
  __shared__ int32_t warp_total[kRouteWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t before = 0;
  for (int b = 0; b < E; b += kRouteThreads) {
    const int e = b + static_cast<int>(threadIdx.x);
    const int32_t c = e < E ? totals[e] : 0;
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
    if (e < E) first[e] += add + incl - c;
    before += all;
    __syncthreads();
  }
  return before;
}

// R and the loss from the counts and the probability sums, by a whole block.
__device__ __forceinline__ void write_totals(const RouteParams& p, const int32_t* counts, const float* prob, int32_t rows,
                                             int32_t live) {
  __shared__ float warp_loss[kRouteWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float s = 0.0f;
  for (int e = threadIdx.x; e < p.experts; e += kRouteThreads) s = fmaf(static_cast<float>(counts[e]), prob[e], s);
  s = warp_sum(s);
  if (lane == 0) warp_loss[warp] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = 0.0f;
    for (int w = 0; w < kRouteWarps; ++w) all += warp_loss[w];
    p.totals[0] = rows;
    p.totals[1] = live;
    *p.loss = rows > 0 ? p.coef * static_cast<float>(p.experts) * (all / static_cast<float>(rows) / static_cast<float>(live)) : 0.0f;
  }
}

// Rows of a chunk's choices: the rank inside the chunk and first[e], the first row of the chunk's part of
// the expert.
__device__ __forceinline__ void place_chunk(const RouteParams& p, const int32_t* first) {
  const int k = p.top_k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int64_t left = static_cast<int64_t>(p.tokens) - t0;
  const int rows = static_cast<int>(left < p.chunk ? left : p.chunk);
  for (int i = threadIdx.x; i < rows * k; i += kRouteThreads) {
    const int e = p.expert[t0 * k + i];
    if (e >= 0) p.row[t0 * k + i] += first[e];
  }
}

// After route_scan_kernel.  The last block writes R and the loss too.  (No chunks: counts, totals and
// loss of no tokens.)
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint32_t route_smem[];
  int32_t* first = reinterpret_cast<int32_t*>(route_smem);   // E
  ptx::griddep_wait();
  for (int e = threadIdx.x; e < p.experts; e += kRouteThreads)
    first[e] = p.chunks > 0 ? p.part_count[static_cast<int64_t>(e) * p.chunks + blockIdx.x] : 0;
  const int32_t rows = add_first_rows(p.counts, first, p.experts);   // (a thread adds to what it wrote)
  if (blockIdx.x == gridDim.x - 1) write_totals(p, p.counts, p.prob, rows, p.totals[1]);
  place_chunk(p, first);
}

// Few chunks: every block sums the chunks' counts itself, a thread per expert, which costs less than a
// launch of its own for the prefix sums.
constexpr int kFewChunks = 16;
__global__ void __launch_bounds__(kRouteThreads) route_sum_place_kernel(const RouteParams p) {
  extern __shared__ __align__(16) uint32_t route_smem[];
  const int E = p.experts;
  int32_t* first = reinterpret_cast<int32_t*>(route_smem);            // E
  int32_t* total = first + E;                                         // E + 1: counts, live rows
  float* prob = reinterpret_cast<float*>(total + E + 1);              // E (the last block's)
  const bool last = blockIdx.x == gridDim.x - 1;
  ptx::griddep_wait();
  for (int e = threadIdx.x; e <= E; e += kRouteThreads) {
    const int32_t* count = p.part_count + static_cast<int64_t>(e) * p.chunks;
    const float* part = p.part_prob + static_cast<int64_t>(e) * p.chunks;
    int32_t before = 0, all = 0;
    float s = 0.0f;
#pragma unroll
    for (int b = 0; b < kFewChunks; ++b) {
      const bool in = b < p.chunks;
      const int32_t c = in ? count[b] : 0;
      all += c;
      if (b < static_cast<int>(blockIdx.x)) before += c;
      if (in && last && e < E) s += part[b];
    }
    total[e] = all;
    if (e < E) {
      first[e] = before;
      prob[e] = s;
      if (last) p.counts[e] = all;
    }
  }
  __syncthreads();
  const int32_t rows = add_first_rows(total, first, E);
  if (last) write_totals(p, total, prob, rows, total[E]);
  place_chunk(p, first);
}

}  // namespace tst
