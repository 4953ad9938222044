// Instantiations of the block-scaled kernel with 128 x 256 tiles.
#include "gemm_bs_wide.cuh"

TstBsKernel tst_bs_wide(int out_type) {
  using namespace tst;
  const void* kernel = out_type == OUT_BF16  ? reinterpret_cast<const void*>(&gemm_bs_wide_kernel<OUT_BF16>)
                       : out_type == OUT_F32 ? reinterpret_cast<const void*>(&gemm_bs_wide_kernel<OUT_F32>)
                                             : nullptr;
  return {kernel, WideCfg::STAGES, WideCfg::SMEM_BYTES, kBsTileThreads};
}
