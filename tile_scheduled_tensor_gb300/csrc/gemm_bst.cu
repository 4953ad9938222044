// Instantiations of the block-scaled kernel for one scale of B per tile and k-block.
#include "gemm_bs_tile.cuh"

const void* tst_bs_tile_kernel(int out_type) {
  using namespace tst;
  if (out_type == OUT_BF16) return reinterpret_cast<const void*>(&gemm_bs_tile_kernel<OUT_BF16>);
  if (out_type == OUT_F32) return reinterpret_cast<const void*>(&gemm_bs_tile_kernel<OUT_F32>);
  return nullptr;
}
