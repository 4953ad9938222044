// Instantiations of the int8 GEMM kernels: 16 to 128 tokens per tile of a CTA, 192 of a CTA pair, few tokens
// without tiles; FP32 or BF16 output.
#include <algorithm>

#include "gemm_int8_few.cuh"
#include "gemm_int8_wide.cuh"

namespace {
template <int NT>
TstInt8Kernel kernel_of(int out_type) {
  using Cfg = tst::Int8Cfg<NT>;
  const void* f = out_type == tst::OUT_BF16 ? reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_BF16>)
                                            : reinterpret_cast<const void*>(&tst::gemm_int8_kernel<Cfg, tst::OUT_F32>);
  return {f, Cfg::SMEM_BYTES, Cfg::THREADS};
}
}  // namespace

TstInt8Kernel tst_int8_kernel(int tokens, int out_type) {
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

bool tst_int8_few(const tst::KernelParams& kp, const void* a, const void* b, int out_type, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((kp.N + tst::kInt8FewColumns - 1) / tst::kInt8FewColumns),
                  static_cast<unsigned>(kp.sched.groups > 0 ? kp.sched.groups : (kp.M + tst::kInt8FewRows - 1) / tst::kInt8FewRows), 1);
  const int8_t *pa = static_cast<const int8_t*>(a), *pb = static_cast<const int8_t*>(b);
  if (out_type == tst::OUT_BF16) tst::int8_few_kernel<tst::OUT_BF16><<<grid, tst::kInt8FewThreads, 0, stream>>>(kp, pa, pb);
  else tst::int8_few_kernel<tst::OUT_F32><<<grid, tst::kInt8FewThreads, 0, stream>>>(kp, pa, pb);
  return cudaGetLastError() == cudaSuccess;
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
