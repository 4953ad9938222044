// Tokens into the experts' row order and back.
//
//   dispatch:  rows[row_tj] = x_t                                       (copied, or block-scaled e4m3)
//   combine:   out_t = sum_j w_tj rows[row_tj]
//   gradient:  d_rows[row_tj] = w_tj d_out_t,   d_w_tj = <d_out_t, rows[row_tj]>
//
// All are bound by memory: every token is read once, however many rows it goes to, and every row
// once.  row_tj = -1 is a choice without a row (skipped); a row past the matrix is skipped and
// recorded in the plan's status word, so a wrong index never leaves the buffers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace tst {

constexpr int kRowsThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 1.262177448e-29f;   // 2^-96: least magnitude a block's scale is taken from

struct RowsParams {
  const void* x;            // dispatch: tokens x hidden; gradient: d_out; row stride x_ld
  int64_t x_ld;
  const int32_t* row;       // tokens x k, or null: row t of token t
  const float* weight;      // tokens x k, or null: 1
  const void* rows;         // combine, gradient: n_rows x hidden
  void* out;                // dispatch, gradient: n_rows x hidden; combine: tokens x hidden, row stride out_ld
  int64_t out_ld;
  float* scales;            // e4m3: n_rows x blocks; gradient: d_weight
  uint32_t* status;
  int64_t tokens, n_rows;
  int32_t hidden, top_k, slices;
};

__device__ __forceinline__ bool row_ok(const RowsParams& p, int64_t r) {
  if (r >= 0 && r < p.n_rows) return true;
  if (r != -1) atomicOr(p.status, 1u);
  return false;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// N consecutive elements as FP32: 16-byte loads (VEC) or one by one.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[N]) {
  if constexpr (VEC) {
    constexpr int PER = 16 / sizeof(T);
    static_assert(N % PER == 0, "whole vectors");
#pragma unroll
    for (int q = 0; q < N / PER; ++q) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + q);
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < PER; ++i) v[q * PER + i] = to_f32<T>(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32<T>(p[i]);
  }
}

// e4m3 rows with one FP32 scale per 128 elements: scale = amax / 448, value = x (448 / amax)
// rounded to e4m3.  The largest magnitude is found on the absolute bits as integers, where NaN
// and infinity stand above every number, so a block that holds one gets a NaN scale or an infinite
// one and cannot pass for a number.  Eight lanes hold a block, sixteen elements each; a warp
// takes 512 elements of one token, 16 elements a lane, and writes it to every row that
// the token goes to.  Bound by those writes: 16384 tokens of 4096 BF16 to 8 rows each in 105 us, 0.97 of
// the copy rate.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kRowsThreads) dispatch_e4m3_kernel(const RowsParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / p.slices;
  const int h = static_cast<int>(item - t * p.slices) * 512 + lane * 16;
  if (t >= p.tokens) return;
  const bool in = h < p.hidden;   // hidden is a multiple of 16
  float v[16];
  uint32_t bits = 0u;
  if (in) {
    load_f32<T, 16, VEC>(static_cast<const T*>(p.x) + t * p.x_ld + h, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
      bits = a > bits ? a : bits;
    }
  }
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, bits, d);
    bits = o > bits ? o : bits;
  }
  if (!in) return;
  const uint32_t least = __float_as_uint(kScaleFloor);
  const float amax = __uint_as_float(bits > least ? bits : least);
  const float scale = amax / kE4m3Max, inv = kE4m3Max / amax;
  uint4 q;
  __nv_fp8x2_storage_t* q2 = reinterpret_cast<__nv_fp8x2_storage_t*>(&q);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    q2[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  const int blocks = (p.hidden + 127) / 128;
  const int k = p.row ? p.top_k : 1;
  for (int j = 0; j < k; ++j) {
    const int64_t r = p.row ? p.row[t * k + j] : t;
    if (!row_ok(p, r)) continue;
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + r * p.hidden + h) = q;
    if ((lane & 7) == 0) p.scales[r * blocks + h / 128] = scale;
  }
}

// int8 rows with one FP32 scale each: scale = amax / 127, value = x (127 / amax), rounded to FP32 and then to
// the nearest whole number, ties to even.  amax as above (a NaN or an infinity leaves its mark in the scale).
// TPT threads hold a token, U pieces of 16 elements each, TPT pieces apart; what a token has beyond them is
// read again for the values.  Adding 1.5 * 2^23 rounds a value of up to 127 and leaves its two's complement in
// the low byte.  Bound by memory: 16384 BF16 tokens of 4096 to 8 rows each in 101 us in a graph, 0.98 of the copy rate;
// 8190 FP32 rows of 1424 in 9.0, 0.96; 16 tokens to 8 rows each in 3.6.
constexpr float kInt8Max = 127.0f;
template <typename T, bool VEC, int TPT, int U>
__global__ void __launch_bounds__(TPT < 128 ? 128 : TPT) dispatch_int8_kernel(const RowsParams p) {
  constexpr int BLOCK = TPT < 128 ? 128 : TPT, WARPS = BLOCK / 32;
  __shared__ uint32_t part[WARPS];
  const int lane = threadIdx.x & 31, at = threadIdx.x % TPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (BLOCK / TPT) + threadIdx.x / TPT;
  const bool on = t < p.tokens;
  const T* const src = static_cast<const T*>(p.x) + (on ? t : 0) * p.x_ld;
  const int pieces = on ? p.hidden / 16 : 0;   // hidden is a multiple of 16
  float v[U][16];
  uint32_t bits = __float_as_uint(kScaleFloor);
  auto widen = [&](const float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      bits = a > bits ? a : bits;
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at + u * TPT < pieces) load_f32<T, 16, VEC>(src + static_cast<int64_t>(at + u * TPT) * 16, v[u]);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at + u * TPT < pieces) widen(v[u]);
  for (int q = at + U * TPT; q < pieces; q += TPT) {
    float x[16];
    load_f32<T, 16, VEC>(src + static_cast<int64_t>(q) * 16, x);
    widen(x);
  }
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if constexpr (TPT > 32) {
    if (lane == 0) part[threadIdx.x >> 5] = bits;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) bits = part[i] > bits ? part[i] : bits;
  }
  const float amax = __uint_as_float(bits);
  const float scale = amax / kInt8Max, inv = kInt8Max / amax;
  auto narrow = [&](const float (&x)[16]) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[4 * q + i], inv), 12582912.0f));
      w[q] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  uint4 q[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at + u * TPT < pieces) q[u] = narrow(v[u]);
  if (!on) return;
  const int k = p.row ? p.top_k : 1;
  for (int j = 0; j < k; ++j) {
    const int64_t r = p.row ? p.row[t * k + j] : t;
    if (!row_ok(p, r)) continue;
    uint4* const out = reinterpret_cast<uint4*>(static_cast<int8_t*>(p.out) + r * p.hidden);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at + u * TPT < pieces) out[at + u * TPT] = q[u];
    for (int i = at + U * TPT; i < pieces; i += TPT) {
      float x[16];
      load_f32<T, 16, VEC>(src + static_cast<int64_t>(i) * 16, x);
      out[i] = narrow(x);
    }
    if (at == 0) p.scales[r] = scale;
  }
}

// Rows copied unchanged, in units U of 16 bytes where the addresses allow, else of one element.
template <typename U>
__global__ void __launch_bounds__(kRowsThreads) dispatch_copy_kernel(const RowsParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = item / p.slices;
  const int h = static_cast<int>(item - t * p.slices) * 32 + lane;
  if (t >= p.tokens || h >= p.hidden) return;   // hidden, x_ld: in units
  const U v = static_cast<const U*>(p.x)[t * p.x_ld + h];
  const int k = p.row ? p.top_k : 1;
  for (int j = 0; j < k; ++j) {
    const int64_t r = p.row ? p.row[t * k + j] : t;
    if (row_ok(p, r)) static_cast<U*>(p.out)[r * p.hidden + h] = v;
  }
}

// N adjacent elements as they lie in memory: one load or store of up to 16 bytes when aligned for it.
template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Piece {
  T e[N];
};
template <typename T, int N>
__device__ __forceinline__ Piece<T, N> load_piece(const T* p) {
  Piece<T, N> v;
  if constexpr (N * sizeof(T) == 16) *reinterpret_cast<uint4*>(&v) = __ldg(reinterpret_cast<const uint4*>(p));
  else v = *reinterpret_cast<const Piece<T, N>*>(p);
  return v;
}

// A block has L threads for each of its 128 / L tokens; a thread sums U pieces of N elements over
// the token's rows in FP32, in the order of the choices.  The U pieces of one row are in flight
// together, L pieces apart, and stay as they came until they are added, which keeps the registers
// of many blocks free: rows of 8 KB, 8 per token, in 190 us where their bytes at the copy rate
// are 178 (207 with one piece per thread, 288 with pieces of four rows in flight).
constexpr int kTokenThreads = 128;
template <typename TI, typename TO, int N, int U, int L>
__global__ void __launch_bounds__(kTokenThreads) combine_kernel(const RowsParams p) {
  const int lane = threadIdx.x % L;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kTokenThreads / L) + threadIdx.x / L;
  const int64_t t = item / p.slices;
  if (t >= p.tokens) return;
  const int h0 = (static_cast<int>(item - t * p.slices) * L * U + lane) * N;   // then every L N elements
  float acc[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) acc[u][i] = 0.0f;
#pragma unroll 1
  for (int j = 0; j < p.top_k; ++j) {
    const int64_t r = p.row[t * p.top_k + j];
    if (!row_ok(p, r)) continue;
    const float w = p.weight ? p.weight[t * p.top_k + j] : 1.0f;
    const TI* const row = static_cast<const TI*>(p.rows) + r * p.hidden + h0;
    Piece<TI, N> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * L * N < p.hidden) v[u] = load_piece<TI, N>(row + u * L * N);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = fmaf(w, to_f32<TI>(v[u].e[i]), acc[u][i]);   // past the row: not stored
  }
  TO* const out = static_cast<TO*>(p.out) + t * p.out_ld + h0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (h0 + u * L * N < p.hidden) {
      Piece<TO, N> o;
#pragma unroll
      for (int i = 0; i < N; ++i) o.e[i] = static_cast<TO>(acc[u][i]);
      *reinterpret_cast<Piece<TO, N>*>(out + u * L * N) = o;
    }
}

// The same layout, with one token per block: d_out's pieces in registers, times each weight go to the
// rows, and the dot products with the rows are summed in FP32 by threads, lanes and warps, in a fixed
// order; the warps exchange theirs once, at the end.  8192 tokens and 65536 rows of 8 KB, read and written,
// in 182 us, 0.92 of the copy rate.
template <typename TI, typename TO, int N, int U>
__global__ void __launch_bounds__(kTokenThreads) combine_grad_kernel(const RowsParams p) {
  constexpr int WARPS = kTokenThreads / 32, STEP = kTokenThreads * N;
  __shared__ float part[WARPS][32];   // top_k <= 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  if (lane < p.top_k) part[warp][lane] = 0.0f;
  __syncwarp();
  for (int first = 0; first < p.hidden; first += U * STEP) {
    const int h0 = first + static_cast<int>(threadIdx.x) * N;
    const TO* const d_out = static_cast<const TO*>(p.x) + t * p.x_ld + h0;
    Piece<TO, N> d[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * STEP < p.hidden) d[u] = load_piece<TO, N>(d_out + u * STEP);
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
      const int64_t r = p.row[t * p.top_k + j];
      if (!row_ok(p, r)) continue;
      const float w = p.weight[t * p.top_k + j];
      const TI* const row = static_cast<const TI*>(p.rows) + r * p.hidden + h0;
      TI* const d_row = static_cast<TI*>(p.out) + r * p.hidden + h0;
      Piece<TI, N> v[U];
      float dot = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h0 + u * STEP < p.hidden) v[u] = load_piece<TI, N>(row + u * STEP);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h0 + u * STEP < p.hidden) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float x = to_f32<TO>(d[u].e[i]);
            dot = fmaf(x, to_f32<TI>(v[u].e[i]), dot);
            v[u].e[i] = static_cast<TI>(x * w);
          }
          *reinterpret_cast<Piece<TI, N>*>(d_row + u * STEP) = v[u];
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      if (lane == 0) part[warp][j] += dot;
    }
  }
  __syncthreads();
  if (threadIdx.x < p.top_k) {
    float s = 0.0f;
    for (int i = 0; i < WARPS; ++i) s += part[i][threadIdx.x];
    p.scales[t * p.top_k + threadIdx.x] = s;
  }
}

}  // namespace tst
