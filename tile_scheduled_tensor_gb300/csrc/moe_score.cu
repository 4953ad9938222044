// Scored routing: the plan's creation and the instances of its kernels (moe_score.cuh).
#include "moe_plan.h"
#include "moe_score.cuh"

#define TST_OF(...) reinterpret_cast<const void*>(&tst::__VA_ARGS__)

namespace {
template <typename T, int VPL>
const void* rows_of(bool vec, int warps) {
  if constexpr (VPL <= 8)
    if (warps == 32) return TST_OF(score_rows_kernel<T, VPL, false, 32>);
  return vec ? TST_OF(score_rows_kernel<T, VPL, true, 8>) : TST_OF(score_rows_kernel<T, VPL, false, 8>);
}
template <typename T, int VPL>
const void* grad_of(bool vec, int) {
  return vec ? TST_OF(score_grad_kernel<T, VPL, true>) : TST_OF(score_grad_kernel<T, VPL, false>);
}
#define TST_BY_VPL(F)                        \
  switch (vpl) {                             \
    case 1: return F<T, 1>(vec, warps);      \
    case 2: return F<T, 2>(vec, warps);      \
    case 4: return F<T, 4>(vec, warps);      \
    case 8: return F<T, 8>(vec, warps);      \
    case 16: return F<T, 16>(vec, warps);    \
    default: return F<T, 32>(vec, warps);    \
  }
template <typename T>
const void* rows_kernel(int vpl, bool vec, int warps) { TST_BY_VPL(rows_of) }
template <typename T>
const void* grad_kernel(int vpl, bool vec, int warps) { TST_BY_VPL(grad_of) }

const void* score_rows(bool bf16, int vpl, bool vec, int warps) {
  return bf16 ? rows_kernel<__nv_bfloat16>(vpl, vec, warps) : rows_kernel<float>(vpl, vec, warps);
}
const void* score_grad(bool bf16, int vpl, bool vec) {
  return bf16 ? grad_kernel<__nv_bfloat16>(vpl, vec, 8) : grad_kernel<float>(vpl, vec, 8);
}
constexpr TstScoreKernels kScoreKernels = {score_rows, score_grad};
}  // namespace

extern "C" tst_status moe_plan_create_scored(tst_moe_plan** out, int64_t max_tokens, int32_t experts, int32_t top_k,
                                             const tst_moe_score_options* opts) {
  if (out == nullptr) return TST_ERR_INVALID_ARG;
  *out = nullptr;
  if (opts == nullptr) return TST_ERR_INVALID_ARG;
  tst_moe_options plain{};
  plain.normalize = opts->normalize;
  plain.balance_coef = opts->balance_coef;
  plain.host_only = opts->host_only;
  return tst_moe_create(out, max_tokens, experts, top_k, &plain, opts, &kScoreKernels);
}
