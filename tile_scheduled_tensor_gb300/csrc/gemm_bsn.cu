// Instantiations of the narrow block-scaled grouped kernel: 16 or 32 rows of a group per
// tile, FP32 or BF16 output, one scale of B per tile and k-block (shared) or one per column.
#include "gemm_bs_narrow.cuh"

namespace {
template <int NT>
const void* kernel_of(int out_type, bool shared) {
  using namespace tst;
  if (out_type == OUT_BF16)
    return shared ? reinterpret_cast<const void*>(&gemm_bs_narrow_kernel<NT, OUT_BF16, true>)
                  : reinterpret_cast<const void*>(&gemm_bs_narrow_kernel<NT, OUT_BF16, false>);
  if (out_type == OUT_F32)
    return shared ? reinterpret_cast<const void*>(&gemm_bs_narrow_kernel<NT, OUT_F32, true>)
                  : reinterpret_cast<const void*>(&gemm_bs_narrow_kernel<NT, OUT_F32, false>);
  return nullptr;
}
template <int NT>
TstBsKernel narrow_of(int out_type, bool shared) {
  using Cfg = tst::NarrowCfg<NT>;
  return {kernel_of<NT>(out_type, shared), Cfg::STAGES, Cfg::SMEM_BYTES, kBsNarrowThreads};
}
}  // namespace

TstBsKernel tst_bs_narrow(int rows, int out_type, bool shared) {
  return rows == 16 ? narrow_of<16>(out_type, shared) : narrow_of<32>(out_type, shared);
}
