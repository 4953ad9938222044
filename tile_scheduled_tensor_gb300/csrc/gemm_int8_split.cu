// Instantiations of the int8 GEMM kernel whose tiles are split along K over a cluster of CTAs.
#include "gemm_int8.cuh"

namespace {
template <int NT>
TstInt8Kernel kernel_of(int out_type) {
  using Cfg = tst::Int8Cfg<NT, true>;
  const void* f = out_type == tst::OUT_BF16 ? reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_BF16>)
                                            : reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_F32>);
  return {f, Cfg::SMEM_BYTES, Cfg::THREADS};
}
}  // namespace

TstInt8Kernel tst_int8_split_kernel(int tokens, int out_type) {
  return tokens == 16 ? kernel_of<16>(out_type) : tokens == 32 ? kernel_of<32>(out_type) : kernel_of<64>(out_type);
}
