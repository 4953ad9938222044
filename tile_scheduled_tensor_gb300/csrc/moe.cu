// Host side of the mixture-of-experts calls declared in include/tstgemm.h: argument checks, the
// plan's workspace and the launches of the kernels in moe_route.cuh and moe_rows.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "moe_route.cuh"
#include "moe_rows.cuh"
#include "tstgemm.h"

struct tst_moe_plan {
  int64_t max_tokens = 0;
  int32_t experts = 0, top_k = 0, normalize = 0;
  float coef = 0.0f;
  bool host_only = false;
  int device = -1;
  int32_t num_sms = 0;
  void* dev_block = nullptr;   // [status | probability sums | chunk counts | chunk probability sums]
  size_t dev_bytes = 0;
  uint32_t* d_status = nullptr;
  float* d_prob = nullptr;
  int32_t* d_part_count = nullptr;
  float* d_part_prob = nullptr;
  cudaStream_t last_stream = nullptr;
  bool ran = false;
};

namespace {

using tst::RouteGradParams;
using tst::RouteParams;
using tst::RowsParams;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool float_type(int32_t t) { return t == TST_OUT_F32 || t == TST_OUT_BF16; }
int64_t type_bytes(int32_t t) { return t == TST_OUT_F32 ? 4 : t == TST_OUT_BF16 ? 2 : 1; }

// Tokens per block of the routing kernel: the fewest multiple of 32 that keeps to four blocks for each of
// the GPU's 152 SMs, up to 256 (whose bitmap is 8 words per expert).  Up to 256 experts these blocks are
// resident at once; registers leave room for two per SM up to 512 experts and one beyond, where they
// follow one another.
constexpr int64_t kResidentChunks = 4 * 152;
int32_t route_chunk(int64_t tokens) {
  const int64_t c = ceil_div(ceil_div(tokens, 32), kResidentChunks) * 32;
  return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(c, 32), 256));
}

// warps of a routing block: a warp per 32 threads' rows up to kRouteThreadRow experts; else 8, or 32 (a
// row each) where blocks of 32 tokens leave SMs idle and the registers allow it
int32_t route_warps(int32_t experts, int32_t chunk, int64_t chunks) {
  if (experts <= tst::kRouteThreadRow) return chunk / 32;
  return chunk == 32 && chunks <= 152 && experts <= 256 ? 32 : tst::kRouteWarps;
}

// shared memory of a routing block: RouteShared, and the small kernel's staged choices
size_t route_smem(int32_t experts, int32_t top_k, int32_t chunk, int32_t warps) {
  const size_t staged = experts <= tst::kRouteThreadRow ? 2 * static_cast<size_t>(chunk) * (top_k | 1) : 0;
  return (static_cast<size_t>(experts) * (chunk / 32 + warps + 1) + 1 + staged) * 4;
}

// Zero device memory before returning, on a stream of its own: cudaMemset is ordered with the default
// stream alone and may run after this returns, when a run on another stream has written there.
bool zero_now(void* p, size_t bytes) {
  cudaStream_t s;
  if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess) return false;
  const bool ok = cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
  return cudaStreamDestroy(s) == cudaSuccess && ok;
}

tst_status launched() {
  if (cudaGetLastError() != cudaSuccess) return TST_ERR_CUDA;
  return TST_OK;
}

// The kernels' instances by the number of experts: a thread's row of 8, 16 or 32 logits, or a
// warp's with 2 to 32 per lane.
#define TST_BY_EXPERTS(E, SMALL, WARP)   \
  do {                                   \
    if ((E) <= 8) { SMALL(8); }          \
    else if ((E) <= 16) { SMALL(16); }   \
    else if ((E) <= tst::kRouteThreadRow) { SMALL(32); } \
    else if ((E) <= 64) { WARP(2); }     \
    else if ((E) <= 128) { WARP(4); }    \
    else if ((E) <= 256) { WARP(8); }    \
    else if ((E) <= 512) { WARP(16); }   \
    else { WARP(32); }                   \
  } while (0)

// whether rows of `ld` elements at `p` can be read W elements at a time (moe_route.cuh's RowMap)
template <typename T, int VPL>
bool whole_packs(const void* p, int64_t ld, int32_t experts) {
  constexpr int W = tst::RowMap<T, VPL>::W;
  return aligned(p, W * sizeof(T)) && ld % W == 0 && experts % W == 0;
}

// the same, 16 bytes at a time
template <typename T>
bool whole_units(const void* p, int64_t ld, int32_t experts) {
  constexpr int V = 16 / sizeof(T);
  return aligned(p, 16) && ld % V == 0 && experts % V == 0;
}

template <typename T>
const void* route_kernel(const RouteParams& p, int32_t warps) {
  const void* f = nullptr;
#define TST_OF(...) reinterpret_cast<const void*>(&tst::__VA_ARGS__)
#define TST_SMALL(EM)                                                                             \
  f = whole_units<T>(p.logits, p.ld, p.experts) ? TST_OF(route_rows_small_kernel<T, EM, true>)    \
                                                : TST_OF(route_rows_small_kernel<T, EM, false>)
#define TST_WARP(V)                                                                                    \
  do {                                                                                                 \
    const bool vec = whole_packs<T, V>(p.logits, p.ld, p.experts);                                     \
    if constexpr (V <= 8) {                                                                            \
      if (warps == 32) {                                                                               \
        f = vec ? TST_OF(route_rows_kernel<T, V, true, 32>) : TST_OF(route_rows_kernel<T, V, false, 32>); \
        break;                                                                                         \
      }                                                                                                \
    }                                                                                                  \
    f = vec ? TST_OF(route_rows_kernel<T, V, true, 8>) : TST_OF(route_rows_kernel<T, V, false, 8>);    \
  } while (0)
  TST_BY_EXPERTS(p.experts, TST_SMALL, TST_WARP);
#undef TST_SMALL
#undef TST_WARP
  return f;
}

template <typename T>
const void* grad_kernel(const RouteGradParams& p) {
  const void* f = nullptr;
#define TST_SMALL(EM)                                                                                                   \
  f = whole_units<T>(p.logits, p.ld, p.experts) && whole_units<T>(p.d_logits, p.d_ld, p.experts)                        \
          ? TST_OF(route_grad_small_kernel<T, EM, true>)                                                                \
          : TST_OF(route_grad_small_kernel<T, EM, false>)
#define TST_WARP(V)                                                                                       \
  f = whole_packs<T, V>(p.logits, p.ld, p.experts) && whole_packs<T, V>(p.d_logits, p.d_ld, p.experts)    \
          ? TST_OF(route_grad_kernel<T, V, true>)                                                         \
          : TST_OF(route_grad_kernel<T, V, false>)
  TST_BY_EXPERTS(p.experts, TST_SMALL, TST_WARP);
#undef TST_SMALL
#undef TST_WARP
  return f;
}
#undef TST_OF

// Launch f(params); `after`: it may start while the kernel before it on the stream finishes, and
// waits for that kernel itself (griddepcontrol.wait).
template <typename P>
bool launch(const void* f, int64_t grid, int32_t threads, size_t smem, cudaStream_t s, P& params, bool after = false) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (after) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  void* args[] = {&params};
  return cudaLaunchKernelExC(&cfg, f, args) == cudaSuccess;
}

// What every run checks of its plan and token count; the plan's workspace, and the kernel attributes that
// its creation raised, are those of one GPU, which has to be the current one.
tst_status check_run(const tst_moe_plan* p, int64_t tokens, int64_t most) {
  if (p == nullptr || tokens < 0 || tokens > most) return TST_ERR_INVALID_ARG;
  if (p->host_only) return TST_OK;
  int now = -1;
  if (cudaGetDevice(&now) != cudaSuccess) {
    cudaGetLastError();
    return TST_ERR_CUDA;
  }
  return now == p->device ? TST_OK : TST_ERR_INVALID_ARG;
}

tst_status finish(tst_moe_plan* p, cudaStream_t s) {
  const tst_status st = launched();
  p->last_stream = s;
  p->ran = true;
  return st;
}

int32_t row_grid(int64_t items) { return static_cast<int32_t>(ceil_div(items, tst::kRowsThreads / 32)); }

// slices of a token's `units` per warp step; false when the launch would not fit a grid
bool slice(RowsParams& p, int64_t units, int64_t per_warp) {
  p.slices = static_cast<int32_t>(ceil_div(units, per_warp));
  return ceil_div(p.tokens * p.slices, tst::kRowsThreads / 32) < (int64_t(1) << 31);
}

}  // namespace

extern "C" {

tst_status moe_plan_create(tst_moe_plan** out, int64_t max_tokens, int32_t experts, int32_t top_k,
                           const tst_moe_options* opts) {
  if (out == nullptr) return TST_ERR_INVALID_ARG;
  *out = nullptr;
  if (opts == nullptr || max_tokens < 1 || experts < 1 || top_k < 1 || top_k > experts) return TST_ERR_INVALID_ARG;
  if (max_tokens * top_k >= (int64_t(1) << 31) || max_tokens >= (int64_t(1) << 31)) return TST_ERR_INVALID_ARG;
  if (!(opts->balance_coef == opts->balance_coef)) return TST_ERR_INVALID_ARG;
  if (experts > tst::kMoeMaxExperts || top_k > tst::kMoeMaxTopK) return TST_ERR_UNSUPPORTED;
  tst_moe_plan* p = new (std::nothrow) tst_moe_plan();
  if (p == nullptr) return TST_ERR_OOM;
  p->max_tokens = max_tokens;
  p->experts = experts;
  p->top_k = top_k;
  p->normalize = opts->normalize != 0;
  p->coef = opts->balance_coef;
  p->host_only = opts->host_only != 0;
  // the most chunks that any call of up to max_tokens tokens has
  const int64_t chunks = std::max(std::min(kResidentChunks, ceil_div(max_tokens, 32)), ceil_div(max_tokens, 256));
  const size_t prob = ((static_cast<size_t>(experts) * 4 + 255) / 256) * 256;
  const size_t part = ((static_cast<size_t>(experts + 1) * chunks * 4 + 255) / 256) * 256;
  p->dev_bytes = 256 + prob + 2 * part;
  if (!p->host_only) {
    int dev = 0, count = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDeviceCount(&count) != cudaSuccess || count == 0) {
      cudaGetLastError();
      delete p;
      return TST_ERR_NO_DEVICE;
    }
    if (cudaGetDevice(&dev) != cudaSuccess) { delete p; return TST_ERR_CUDA; }
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (major != 10 || minor != 3) { delete p; return TST_ERR_UNSUPPORTED; }  // built for sm_103a only
    p->device = dev;
    p->num_sms = sms;
    // each instance that a call of this plan may take, with and without whole packs
    RouteParams a{};
    a.experts = experts;
    for (int64_t ld : {int64_t(1024), int64_t(1025)})
      for (int32_t chunk : {32, 256}) {
        a.ld = ld;
        const int32_t warps = route_warps(experts, chunk, 1);
        const int smem = static_cast<int>(route_smem(experts, top_k, chunk, warps));
        for (const void* f : {route_kernel<float>(a, warps), route_kernel<__nv_bfloat16>(a, warps)}) {
          cudaFuncAttributes have;
          if (cudaFuncGetAttributes(&have, f) != cudaSuccess ||
              (have.maxDynamicSharedSizeBytes < smem &&
               cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)) {
            cudaGetLastError();
            delete p;
            return TST_ERR_CUDA;
          }
        }
      }
    if (cudaMalloc(&p->dev_block, p->dev_bytes) != cudaSuccess) {
      cudaGetLastError();
      delete p;
      return TST_ERR_OOM;
    }
    if (!zero_now(p->dev_block, 256)) {
      cudaGetLastError();
      cudaFree(p->dev_block);
      delete p;
      return TST_ERR_CUDA;
    }
    char* base = static_cast<char*>(p->dev_block);
    p->d_status = reinterpret_cast<uint32_t*>(base);
    p->d_prob = reinterpret_cast<float*>(base + 256);
    p->d_part_count = reinterpret_cast<int32_t*>(base + 256 + prob);
    p->d_part_prob = reinterpret_cast<float*>(base + 256 + prob + part);
  }
  *out = p;
  return TST_OK;
}

tst_status moe_plan_destroy(tst_moe_plan* p) {
  if (p == nullptr) return TST_OK;
  tst_status st = TST_OK;
  if (p->dev_block && cudaFree(p->dev_block) != cudaSuccess) st = TST_ERR_CUDA;
  delete p;
  return st;
}

tst_status moe_plan_get_info(const tst_moe_plan* p, tst_moe_plan_info* info) {
  if (p == nullptr || info == nullptr) return TST_ERR_INVALID_ARG;
  info->max_tokens = p->max_tokens;
  info->experts = p->experts;
  info->top_k = p->top_k;
  info->normalize = p->normalize;
  info->balance_coef = p->coef;
  info->workspace_bytes = static_cast<int64_t>(p->dev_bytes);
  return TST_OK;
}

tst_status moe_status_query(tst_moe_plan* p) {
  if (p == nullptr) return TST_ERR_INVALID_ARG;
  if (p->host_only) return TST_ERR_NO_DEVICE;
  if (!p->ran) return TST_OK;
  uint32_t word = 0;
  if (cudaStreamSynchronize(p->last_stream) != cudaSuccess ||
      cudaMemcpy(&word, p->d_status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
    return TST_ERR_CUDA;
  if (word != 0 && !zero_now(p->d_status, sizeof(word))) return TST_ERR_CUDA;   // before any later run
  return word == 0 ? TST_OK : TST_ERR_DEVICE_CHECK;
}

tst_status moe_route(tst_moe_plan* p, int64_t tokens, const void* logits, int32_t dtype, int64_t ld,
                     const uint8_t* mask, int32_t* expert, float* weight, int32_t* row, int32_t* counts,
                     int32_t* totals, float* loss, void* stream) {
  const tst_status st = check_run(p, tokens, p ? p->max_tokens : 0);
  if (st != TST_OK) return st;
  if (!float_type(dtype) || ld < p->experts || counts == nullptr || totals == nullptr || loss == nullptr)
    return TST_ERR_INVALID_ARG;
  if (tokens > 0 && (logits == nullptr || expert == nullptr || weight == nullptr || row == nullptr))
    return TST_ERR_INVALID_ARG;
  if (!aligned(logits, type_bytes(dtype)) || !aligned(expert, 4) || !aligned(weight, 4) || !aligned(row, 4) ||
      !aligned(counts, 4) || !aligned(totals, 4) || !aligned(loss, 4))
    return TST_ERR_ALIGNMENT;
  if (p->host_only) return TST_ERR_NO_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteParams a{};
  a.logits = logits;
  a.ld = ld;
  a.mask = mask;
  a.expert = expert;
  a.weight = weight;
  a.row = row;
  a.counts = counts;
  a.totals = totals;
  a.loss = loss;
  a.part_count = p->d_part_count;
  a.part_prob = p->d_part_prob;
  a.prob = p->d_prob;
  a.tokens = static_cast<int32_t>(tokens);
  a.experts = p->experts;
  a.top_k = p->top_k;
  a.chunk = route_chunk(tokens);
  a.chunks = static_cast<int32_t>(ceil_div(tokens, a.chunk));
  a.normalize = p->normalize;
  a.coef = p->coef;
  bool ok = true;
  if (tokens > 0) {
    const int32_t warps = route_warps(a.experts, a.chunk, a.chunks);
    const void* f = dtype == TST_OUT_F32 ? route_kernel<float>(a, warps) : route_kernel<__nv_bfloat16>(a, warps);
    ok = launch(f, a.chunks, 32 * warps, route_smem(a.experts, a.top_k, a.chunk, warps), s, a);
  }
  if (a.chunks == 1) {
    // it has finished by itself
  } else if (a.chunks > 1 && a.chunks <= tst::kFewChunks) {
    ok = ok && launch(reinterpret_cast<const void*>(&tst::route_sum_place_kernel), a.chunks, tst::kRouteThreads,
                      (3 * static_cast<size_t>(a.experts) + 1) * 4, s, a, true);
  } else {
    ok = ok &&
         launch(reinterpret_cast<const void*>(&tst::route_scan_kernel), ceil_div(a.experts + 1, tst::kRouteWarps),
                tst::kRouteThreads, 0, s, a, true) &&
         launch(reinterpret_cast<const void*>(&tst::route_place_kernel), std::max(a.chunks, 1), tst::kRouteThreads,
                static_cast<size_t>(a.experts) * 4, s, a, true);
  }
  if (!ok) {
    cudaGetLastError();
    return TST_ERR_CUDA;
  }
  return finish(p, s);
}

tst_status moe_route_backward(tst_moe_plan* p, int64_t tokens, const void* logits, int32_t dtype, int64_t ld,
                              const uint8_t* mask, const int32_t* expert, const int32_t* counts,
                              const int32_t* totals, const float* d_weight, const float* d_loss, void* d_logits,
                              int64_t d_ld, void* stream) {
  const tst_status st = check_run(p, tokens, p ? p->max_tokens : 0);
  if (st != TST_OK) return st;
  if (!float_type(dtype) || ld < p->experts || d_ld < p->experts || counts == nullptr || totals == nullptr)
    return TST_ERR_INVALID_ARG;
  if (tokens > 0 && (logits == nullptr || expert == nullptr || d_logits == nullptr)) return TST_ERR_INVALID_ARG;
  if (!aligned(logits, type_bytes(dtype)) || !aligned(d_logits, type_bytes(dtype)) || !aligned(expert, 4) ||
      !aligned(counts, 4) || !aligned(totals, 4) || !aligned(d_weight, 4) || !aligned(d_loss, 4))
    return TST_ERR_ALIGNMENT;
  if (p->host_only) return TST_ERR_NO_DEVICE;
  if (tokens == 0) return TST_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteGradParams a{};
  a.logits = logits;
  a.ld = ld;
  a.mask = mask;
  a.expert = expert;
  a.counts = counts;
  a.totals = totals;
  a.d_weight = d_weight;
  a.d_loss = d_loss;
  a.d_logits = d_logits;
  a.d_ld = d_ld;
  a.tokens = static_cast<int32_t>(tokens);
  a.experts = p->experts;
  a.top_k = p->top_k;
  a.normalize = p->normalize;
  a.coef = p->coef;
  const void* f = dtype == TST_OUT_F32 ? grad_kernel<float>(a) : grad_kernel<__nv_bfloat16>(a);
  const bool small = a.experts <= tst::kRouteThreadRow;
  // a thread per row, in blocks small enough to spread few rows; or warps, four blocks per SM's worth
  const int32_t threads = small ? (tokens <= 64 * p->num_sms ? 64 : tst::kRouteThreads) : tst::kRouteThreads;
  const int64_t grid = small ? ceil_div(tokens, threads)
                             : std::min<int64_t>(ceil_div(tokens, tst::kRouteWarps), 4 * p->num_sms);
  if (!launch(f, grid, threads, 0, s, a)) {
    cudaGetLastError();
    return TST_ERR_CUDA;
  }
  return finish(p, s);
}

tst_status moe_dispatch(tst_moe_plan* p, int64_t tokens, int64_t hidden, const void* x, int32_t x_dtype, int64_t x_ld,
                        const int32_t* row, void* rows, int32_t rows_dtype, int64_t n_rows, float* scales,
                        void* stream) {
  const tst_status st = check_run(p, tokens, p ? (row ? p->max_tokens : p->max_tokens * p->top_k) : 0);
  if (st != TST_OK) return st;
  const bool quantize = rows_dtype == TST_OUT_E4M3;
  if (hidden < 1 || hidden >= (int64_t(1) << 30) || n_rows < 0 || n_rows >= (int64_t(1) << 31) || x_ld < hidden ||
      !float_type(x_dtype))
    return TST_ERR_INVALID_ARG;
  if (!quantize && rows_dtype != x_dtype) return float_type(rows_dtype) ? TST_ERR_UNSUPPORTED : TST_ERR_INVALID_ARG;
  if (tokens > 0 && x == nullptr) return TST_ERR_INVALID_ARG;
  if (n_rows > 0 && (rows == nullptr || (quantize && scales == nullptr))) return TST_ERR_INVALID_ARG;
  if (row == nullptr && n_rows < tokens) return TST_ERR_INVALID_ARG;
  const int64_t elt = type_bytes(x_dtype);
  if (!aligned(x, elt) || !aligned(row, 4) || !aligned(scales, 4) || !aligned(rows, quantize ? 16 : elt))
    return TST_ERR_ALIGNMENT;
  if (quantize && hidden % 16 != 0) return TST_ERR_ALIGNMENT;   // the rows feed a TMA map, as K of a GEMM
  if (p->host_only) return TST_ERR_NO_DEVICE;
  if (tokens == 0) return TST_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowsParams a{};
  a.x = x;
  a.x_ld = x_ld;
  a.row = row;
  a.out = rows;
  a.scales = scales;
  a.status = p->d_status;
  a.tokens = tokens;
  a.n_rows = n_rows;
  a.hidden = static_cast<int32_t>(hidden);
  a.top_k = p->top_k;
  if (quantize) {
    if (!slice(a, hidden, 512)) return TST_ERR_UNSUPPORTED;
    const int32_t grid = row_grid(tokens * a.slices);
    const bool vec = aligned(x, 16) && (x_ld * elt) % 16 == 0;
    if (x_dtype == TST_OUT_F32) {
      if (vec) tst::dispatch_e4m3_kernel<float, true><<<grid, tst::kRowsThreads, 0, s>>>(a);
      else tst::dispatch_e4m3_kernel<float, false><<<grid, tst::kRowsThreads, 0, s>>>(a);
    } else {
      if (vec) tst::dispatch_e4m3_kernel<__nv_bfloat16, true><<<grid, tst::kRowsThreads, 0, s>>>(a);
      else tst::dispatch_e4m3_kernel<__nv_bfloat16, false><<<grid, tst::kRowsThreads, 0, s>>>(a);
    }
    return finish(p, s);
  }
  const bool vec = aligned(x, 16) && aligned(rows, 16) && (x_ld * elt) % 16 == 0 && (hidden * elt) % 16 == 0;
  const int64_t unit = vec ? 16 / elt : 1;
  a.hidden = static_cast<int32_t>(hidden / unit);
  a.x_ld = x_ld / unit;
  if (!slice(a, a.hidden, 32)) return TST_ERR_UNSUPPORTED;
  const int32_t grid = row_grid(tokens * a.slices);
  if (vec) tst::dispatch_copy_kernel<uint4><<<grid, tst::kRowsThreads, 0, s>>>(a);
  else if (elt == 4) tst::dispatch_copy_kernel<uint32_t><<<grid, tst::kRowsThreads, 0, s>>>(a);
  else tst::dispatch_copy_kernel<uint16_t><<<grid, tst::kRowsThreads, 0, s>>>(a);
  return finish(p, s);
}

}  // extern "C"

namespace {

// pieces of N elements per thread and, few of them, threads per token
template <typename TI, typename TO, int N>
tst_status launch_combine_of(RowsParams& a, cudaStream_t s) {
  const int64_t pieces = ceil_div(a.hidden, N);
#define TST_CALL(U, L)                                                                                       \
  do {                                                                                                       \
    a.slices = static_cast<int32_t>(ceil_div(pieces, (U) * (L)));                                            \
    const int64_t grid = ceil_div(a.tokens * a.slices, tst::kTokenThreads / (L));                            \
    if (grid >= (int64_t(1) << 31)) return TST_ERR_UNSUPPORTED;                                              \
    tst::combine_kernel<TI, TO, N, U, L><<<static_cast<unsigned>(grid), tst::kTokenThreads, 0, s>>>(a);      \
  } while (0)
  if (pieces <= 32) TST_CALL(1, 32);
  else if (pieces <= 128) TST_CALL(1, 128);
  else if (pieces <= 256) TST_CALL(2, 128);
  else TST_CALL(4, 128);
#undef TST_CALL
  return TST_OK;
}

// N: 16 bytes of the rows
template <typename TI, typename TO>
tst_status launch_combine(RowsParams& a, bool vec, cudaStream_t s) {
  return vec ? launch_combine_of<TI, TO, 16 / sizeof(TI)>(a, s) : launch_combine_of<TI, TO, 1>(a, s);
}

template <typename TI, typename TO, int N>
void launch_combine_grad_of(const RowsParams& a, cudaStream_t s) {
  const int64_t pieces = ceil_div(a.hidden, N);
  const unsigned grid = static_cast<unsigned>(a.tokens);
  if (pieces <= 128) tst::combine_grad_kernel<TI, TO, N, 1><<<grid, tst::kTokenThreads, 0, s>>>(a);
  else if (pieces <= 256) tst::combine_grad_kernel<TI, TO, N, 2><<<grid, tst::kTokenThreads, 0, s>>>(a);
  else tst::combine_grad_kernel<TI, TO, N, 4><<<grid, tst::kTokenThreads, 0, s>>>(a);
}

template <typename TI, typename TO>
tst_status launch_combine_grad(RowsParams& a, bool vec, cudaStream_t s) {
  if (vec) launch_combine_grad_of<TI, TO, 16 / sizeof(TI)>(a, s);
  else launch_combine_grad_of<TI, TO, 1>(a, s);
  return TST_OK;
}

}  // namespace

extern "C" {

tst_status moe_combine(tst_moe_plan* p, int64_t tokens, int64_t hidden, const void* rows, int32_t rows_dtype,
                       int64_t n_rows, const int32_t* row, const float* weight, void* out, int32_t out_dtype,
                       int64_t out_ld, void* stream) {
  tst_status st = check_run(p, tokens, p ? p->max_tokens : 0);
  if (st != TST_OK) return st;
  if (hidden < 1 || hidden >= (int64_t(1) << 30) || n_rows < 0 || n_rows >= (int64_t(1) << 31) || out_ld < hidden ||
      !float_type(rows_dtype) || !float_type(out_dtype))
    return TST_ERR_INVALID_ARG;
  if ((tokens > 0 && (row == nullptr || out == nullptr)) || (n_rows > 0 && rows == nullptr)) return TST_ERR_INVALID_ARG;
  const int64_t ei = type_bytes(rows_dtype), eo = type_bytes(out_dtype);
  if (!aligned(rows, ei) || !aligned(out, eo) || !aligned(row, 4) || !aligned(weight, 4)) return TST_ERR_ALIGNMENT;
  if (p->host_only) return TST_ERR_NO_DEVICE;
  if (tokens == 0) return TST_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowsParams a{};
  a.row = row;
  a.weight = weight;
  a.rows = rows;
  a.out = out;
  a.out_ld = out_ld;
  a.status = p->d_status;
  a.tokens = tokens;
  a.n_rows = n_rows;
  a.hidden = static_cast<int32_t>(hidden);
  a.top_k = p->top_k;
  const bool vec = hidden % 8 == 0 && aligned(rows, 16) && aligned(out, 16) && (out_ld * eo) % 16 == 0;
  using bf16 = __nv_bfloat16;
  if (rows_dtype == TST_OUT_F32)
    st = out_dtype == TST_OUT_F32 ? launch_combine<float, float>(a, vec, s) : launch_combine<float, bf16>(a, vec, s);
  else
    st = out_dtype == TST_OUT_F32 ? launch_combine<bf16, float>(a, vec, s) : launch_combine<bf16, bf16>(a, vec, s);
  return st != TST_OK ? st : finish(p, s);
}

tst_status moe_combine_backward(tst_moe_plan* p, int64_t tokens, int64_t hidden, const void* rows, int32_t rows_dtype,
                                int64_t n_rows, const int32_t* row, const float* weight, const void* d_out,
                                int32_t out_dtype, int64_t d_out_ld, void* d_rows, float* d_weight, void* stream) {
  tst_status st = check_run(p, tokens, p ? p->max_tokens : 0);
  if (st != TST_OK) return st;
  if (hidden < 1 || hidden >= (int64_t(1) << 30) || n_rows < 0 || n_rows >= (int64_t(1) << 31) || d_out_ld < hidden ||
      !float_type(rows_dtype) || !float_type(out_dtype))
    return TST_ERR_INVALID_ARG;
  if (tokens > 0 && (row == nullptr || weight == nullptr || d_out == nullptr || d_weight == nullptr))
    return TST_ERR_INVALID_ARG;
  if (n_rows > 0 && (rows == nullptr || d_rows == nullptr)) return TST_ERR_INVALID_ARG;
  const int64_t ei = type_bytes(rows_dtype), eo = type_bytes(out_dtype);
  if (!aligned(rows, ei) || !aligned(d_rows, ei) || !aligned(d_out, eo) || !aligned(row, 4) || !aligned(weight, 4) ||
      !aligned(d_weight, 4))
    return TST_ERR_ALIGNMENT;
  if (p->host_only) return TST_ERR_NO_DEVICE;
  if (tokens == 0) return TST_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowsParams a{};
  a.x = d_out;
  a.x_ld = d_out_ld;
  a.row = row;
  a.weight = weight;
  a.rows = rows;
  a.out = d_rows;
  a.scales = d_weight;
  a.status = p->d_status;
  a.tokens = tokens;
  a.n_rows = n_rows;
  a.hidden = static_cast<int32_t>(hidden);
  a.top_k = p->top_k;
  const bool vec = hidden % 8 == 0 && aligned(rows, 16) && aligned(d_rows, 16) && aligned(d_out, 16) &&
                   (d_out_ld * eo) % 16 == 0;
  using bf16 = __nv_bfloat16;
  if (rows_dtype == TST_OUT_F32)
    st = out_dtype == TST_OUT_F32 ? launch_combine_grad<float, float>(a, vec, s)
                                  : launch_combine_grad<float, bf16>(a, vec, s);
  else
    st = out_dtype == TST_OUT_F32 ? launch_combine_grad<bf16, float>(a, vec, s)
                                  : launch_combine_grad<bf16, bf16>(a, vec, s);
  return st != TST_OK ? st : finish(p, s);
}

}  // extern "C"
