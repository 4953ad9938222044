// The int8 GEMM for few tokens (gemm_int8.cuh: the same sums): weights straight from memory into integer dot
// products of four, without tiles, conversion or tensor core.  What bounds it is reading the weights once,
// and with few of them the latency of one trip to memory.
//
// A block of four warps has four channels (rows of B) and up to 16 tokens.  Each lane loads 16 bytes of each
// channel at once, a warp 512 of every 2048 of K; the tokens' bytes, the same for all blocks, come from the
// caches.  Sums of integers are exact, and the same in any order: over the lanes by the warp's reduction,
// over the warps through shared memory.  blockIdx.y: 16 tokens of a dense product, or a group, whose tokens
// the block takes 16 at a time.
#pragma once
#include "gemm_int8.cuh"

namespace tst {

constexpr int kInt8FewThreads = 128, kInt8FewColumns = 4, kInt8FewRows = 16;

template <int R, int OUT>
__device__ __forceinline__ void int8_few_rows(const KernelParams& p, const int8_t* a, const int8_t* b, int32_t group, int32_t row0, int32_t rows,
                                              int32_t col0, int32_t (*part)[kInt8FewRows * kInt8FewColumns]) {
  constexpr int C = kInt8FewColumns, WARPS = kInt8FewThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t sum[R][C];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) sum[r][c] = 0;
  const int8_t* w[C];
#pragma unroll
  for (int c = 0; c < C; ++c) w[c] = b + (static_cast<int64_t>(group) * p.N + (col0 + c < p.N ? col0 + c : p.N - 1)) * p.K;
  constexpr int U = R <= 4 ? 4 : R == 8 ? 2 : 1;   // steps of K in flight, as registers allow
  for (int32_t k0 = warp * 512 + lane * 16; k0 < p.K; k0 += U * WARPS * 512) {   // K is a multiple of 16
    int4 v[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < C; ++c)
        v[u][c] = k0 + u * WARPS * 512 < p.K ? __ldg(reinterpret_cast<const int4*>(w[c] + k0 + u * WARPS * 512)) : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int32_t k = k0 + u * WARPS * 512;
      if (k >= p.K) break;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int32_t row = row0 + (r < rows ? r : rows - 1);
        const int4 x = __ldg(reinterpret_cast<const int4*>(a + static_cast<int64_t>(row) * p.K + k));
#pragma unroll
        for (int c = 0; c < C; ++c)
          sum[r][c] = __dp4a(x.x, v[u][c].x, __dp4a(x.y, v[u][c].y, __dp4a(x.z, v[u][c].z, __dp4a(x.w, v[u][c].w, sum[r][c]))));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t s = __reduce_add_sync(0xFFFFFFFFu, sum[r][c]);
      if (lane == (r * C + c) % 32) part[warp][r * C + c] = s;
    }
  __syncthreads();
  const int r = static_cast<int>(threadIdx.x) / C, col = col0 + static_cast<int>(threadIdx.x) % C;
  if (r < rows && col < p.N) {
    int32_t s = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) s += part[i][threadIdx.x];
    const int64_t channel = static_cast<int64_t>(group) * p.N + col;
    const int32_t row = row0 + r;
    float z = fmaf(__int2float_rn(s) * __ldg(p.ext.row_scale + row), __ldg(p.ext.col_scale + channel), p.has_bias ? __ldg(p.bias + channel) : 0.0f);
    if (p.relu) z = relu_nan(z);
    static_cast<typename OutOf<OUT>::T*>(p.C)[static_cast<int64_t>(row) * p.N + col] = static_cast<typename OutOf<OUT>::T>(z);
  }
  __syncthreads();   // the parts are read before the next tokens' are written
}

template <int OUT>
__global__ void __launch_bounds__(kInt8FewThreads) int8_few_kernel(const __grid_constant__ KernelParams p, const int8_t* a, const int8_t* b) {
  __shared__ int32_t part[kInt8FewThreads / 32][kInt8FewRows * kInt8FewColumns];
  __shared__ long long first_row;
  const int32_t col0 = static_cast<int32_t>(blockIdx.x) * kInt8FewColumns;
  int32_t group = 0;
  int64_t row0 = static_cast<int64_t>(blockIdx.y) * kInt8FewRows, end = row0 + kInt8FewRows;
  if (p.sched.groups > 0) {
    group = static_cast<int32_t>(blockIdx.y);
    const int64_t mine = group_row_count(p.sched, group);
    if (mine == 0) return;
    if (threadIdx.x < 32) {
      int64_t before = 0;
      for (int32_t g = threadIdx.x; g < group; g += 32) before += group_row_count(p.sched, g);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
      if (threadIdx.x == 0) first_row = before;
    }
    __syncthreads();
    row0 = first_row;
    end = row0 + mine;
    if (end > p.M && threadIdx.x == 0) record_status(p, ST_DEVICE_CHECK, ROLE_PRODUCER);
  }
  if (end > p.M) end = p.M;
  for (; row0 < end; row0 += kInt8FewRows) {
    const int32_t left = static_cast<int32_t>(end - row0 < kInt8FewRows ? end - row0 : kInt8FewRows), at = static_cast<int32_t>(row0);
    if (left == 1) int8_few_rows<1, OUT>(p, a, b, group, at, left, col0, part);
    else if (left == 2) int8_few_rows<2, OUT>(p, a, b, group, at, left, col0, part);
    else if (left <= 4) int8_few_rows<4, OUT>(p, a, b, group, at, left, col0, part);
    else if (left <= 8) int8_few_rows<8, OUT>(p, a, b, group, at, left, col0, part);
    else int8_few_rows<16, OUT>(p, a, b, group, at, left, col0, part);
  }
}

}  // namespace tst
