// Instantiations of the int8 GEMM kernel: 16 to 128 tokens per tile, FP32 or BF16 output.
#include "gemm_int8.cuh"

namespace {
template <int NT>
TstInt8Kernel kernel_of(int out_type) {
  using Cfg = tst::Int8Cfg<NT>;
  const void* f = out_type == tst::OUT_BF16 ? reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_BF16>)
                                            : reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_F32>);
  return {f, Cfg::SMEM_BYTES, tst::kInt8Threads, Cfg::PER_SM};
}
}  // namespace

TstInt8Kernel tst_int8_kernel(int tokens, int out_type) {
  switch (tokens) {
    case 16: return kernel_of<16>(out_type);
    case 32: return kernel_of<32>(out_type);
    case 64: return kernel_of<64>(out_type);
    default: return kernel_of<128>(out_type);
  }
}
