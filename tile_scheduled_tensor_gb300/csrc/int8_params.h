// The int8 GEMM's kernels and launches (gemm_int8.cu) and its tensor maps (api.cu), for its host side (int8.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernel_params.h"

// GEMM of 8-bit integers (gemm_int8.cu): `tokens` = 16, 32, 64 or 128 rows of A per 128-column tile of a CTA, or
// kInt8WideTokens per 256-column tile of a CTA pair; A is FP16, made by tst_int8_widen
constexpr int kInt8WideTokens = 192;
struct TstInt8Kernel {
  const void* kernel;
  int smem_bytes, threads;
};
TstInt8Kernel tst_int8_kernel(int tokens, int out_type);
// the same for few tokens, from A's and B's bytes: launched here
bool tst_int8_few(const tst::KernelParams& kp, const void* a, const void* b, int out_type, cudaStream_t stream);
// A's M x K bytes as FP16, those of the groups' rows alone (group_rows not null)
bool tst_int8_widen(const void* a, void* half, int64_t rows, int64_t K, const int32_t* group_rows, int32_t groups, int32_t num_sms,
                    cudaStream_t stream);

// A tensor map of rows x K bytes, K contiguous, in boxes of box_rows x 128 with the 128-byte swizzle
bool tst_encode_bytes(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int box_rows);
// ... of rows x K 16-bit elements, in boxes of box_rows x 64
bool tst_encode_halves(CUtensorMap* map, const void* ptr, int64_t rows, int64_t K, int box_rows);
