// Instantiations of the int8 GEMM kernels: 16 to 128 tokens per tile of a CTA, 192 of a CTA pair; FP32 or
// BF16 output.
#include <algorithm>

#include "gemm_int8_wide.cuh"

TstInt8Kernel tst_int8_split_kernel(int tokens, int out_type);   // gemm_int8_split.cu

namespace {
template <int NT>
TstInt8Kernel kernel_of(int out_type) {
  using Cfg = tst::Int8Cfg<NT, false>;
  const void* f = out_type == tst::OUT_BF16 ? reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_BF16>)
                                            : reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_F32>);
  return {f, Cfg::SMEM_BYTES, Cfg::THREADS};
}
}  // namespace

TstInt8Kernel tst_int8_kernel(int tokens, int out_type, bool split) {
  if (split) return tst_int8_split_kernel(tokens, out_type);
  switch (tokens) {
    case 16: return kernel_of<16>(out_type);
    case 32: return kernel_of<32>(out_type);
    case 64: return kernel_of<64>(out_type);
    case 128: return kernel_of<128>(out_type);
    default: break;
  }
  using Cfg = tst::Int8WideCfg<kInt8WideTokens>;
  const void* f = out_type == tst::OUT_BF16 ? reinterpret_cast<const void*>(&tst::gemm_int8_wide_kernel<Cfg, tst::OUT_BF16>)
                                            : reinterpret_cast<const void*>(&tst::gemm_int8_wide_kernel<Cfg, tst::OUT_F32>);
  return {f, Cfg::SMEM_BYTES, tst::kInt8WideThreads};
}

bool tst_int8_widen(const void* a, void* half, int64_t rows, int64_t K, const int32_t* group_rows, int32_t groups, int32_t num_sms,
                    cudaStream_t stream) {
  tst::Int8WidenParams p{};
  p.a = static_cast<const int8_t*>(a);
  p.out = static_cast<uint32_t*>(half);
  p.group_rows = group_rows;
  p.units = rows * (K / 16);
  p.groups = groups;
  p.units_per_row = static_cast<int32_t>(K / 16);
  const int64_t blocks = (p.units + 4 * tst::kInt8WidenThreads - 1) / (4 * tst::kInt8WidenThreads);
  tst::int8_widen_kernel<<<static_cast<unsigned>(std::min<int64_t>(blocks, 8 * num_sms)), tst::kInt8WidenThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess;
}
