// Instantiations of the block-scaled FP8 GEMM kernel (kind::f8f6f4 per k-block, FP32
// promotion in the epilogue warps): FP32 or BF16 output; one scale of B per 32-column
// chunk (block rows a multiple of 32) or one per column; one GEMM or grouped.
#include "gemm_blockscale.cuh"

namespace {
template <int OUT>
const void* kernel_of(bool per_col, bool grouped) {
  using namespace tst;
  if (grouped)
    return per_col ? reinterpret_cast<const void*>(&gemm_bs_kernel<DT_E4M3, OUT, true, true>)
                   : reinterpret_cast<const void*>(&gemm_bs_kernel<DT_E4M3, OUT, false, true>);
  return per_col ? reinterpret_cast<const void*>(&gemm_bs_kernel<DT_E4M3, OUT, true, false>)
                 : reinterpret_cast<const void*>(&gemm_bs_kernel<DT_E4M3, OUT, false, false>);
}
}  // namespace

const void* tst_bs_kernel(int out_type, bool per_col, bool grouped) {
  if (out_type == tst::OUT_BF16) return kernel_of<tst::OUT_BF16>(per_col, grouped);
  if (out_type == tst::OUT_F32) return kernel_of<tst::OUT_F32>(per_col, grouped);
  return nullptr;
}
