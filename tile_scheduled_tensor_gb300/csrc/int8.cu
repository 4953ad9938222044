// Host side of the int8 GEMM calls declared in include/tstgemm.h: argument checks, the plan's tile
// and schedule, tensor maps and the launch of the kernel in gemm_int8.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "int8_params.h"
#include "tstgemm.h"

struct tst_int8_plan {
  int64_t M = 0, N = 0, K = 0;
  tst_int8_options opts{};
  int32_t tokens = 0;          // rows of A per tile; kFewTokens: no tiles
  int32_t num_sms = 0, device = -1;
  TstInt8Kernel kernel{};
  bool pairs = false;          // the wide form
  tst::Sched sched{};
  unsigned long long* d_status = nullptr;   // 256 bytes, then A in FP16
  size_t dev_bytes = 0;
  cudaStream_t last_stream = nullptr;
  bool ran = false;
};

namespace {

// The status word keeps what any run records until the query that reports it: every launch has the same tag.
constexpr uint32_t kStatusTag = 1;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;   // the last tile's rows and columns are 32-bit, past the matrix too
constexpr int64_t kMaxK = 131056;                        // 131071 products of up to 2^14 fit 32 bits; K is a multiple of 16

constexpr int32_t kFewTokens = 1;                        // tile_rows of the form without tiles
constexpr int64_t kMaxFewRows = 65535 * 16;              // 16 to a block, 65535 blocks in y

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Zero device memory before returning, on a stream of its own (cudaMemset is ordered with the default stream alone).
bool zero_now(void* p, size_t bytes) {
  cudaStream_t s;
  if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess) return false;
  const bool ok = cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
  return cudaStreamDestroy(s) == cudaSuccess && ok;
}

// Rows of A per tile for M rows of `groups` groups (0: one GEMM), `rows` to a group on average.
//
// Few rows go without tiles where that takes less time, estimated from measurements (us): without tiles
// 2.5, and the weights at 5 bytes per ps or the products at 36 per ps; with tiles 5, and 0.27 per k-block
// and wave, or the weights at 6.2 bytes per ps.  4096 x 4096: 1 row 4.2 and 12.8 with tiles, 16 rows 9.6
// and 12.8, 32 rows 16.5 and 12.9; 8192 x 8192: 1 row 13.4 and 22, 16 rows 32 and 22; 2 rows each for 32
// groups of 4096 x 4096 134 and 85.  (A group may hold all rows, 16 at a time: M is small then.)
//
// Tiles: pairs where they fill the SMs (2048 x 4096 x 4096 58 and 72 with 128 rows); else by a group's rows (32
// groups of 4096 x 4096: of 32 rows each 94 at 32 and 100 at 64, of 40 rows 128 and 101, of 64 rows 104 at 64
// and 135 at 128, of 96 rows 167 and 139), and narrower while one wave holds them (128 x 4096 x 4096: 15 at 32,
// 16 at 64, 21 at 128; 256 x 4096 x 4096: 23, 18 and 22).
int32_t tile_tokens(int64_t M, int64_t N, int64_t K, int64_t groups, int32_t num_sms) {
  const int64_t parts = std::max<int64_t>(groups, 1), rows = ceil_div(M, parts), kt = ceil_div(K, 128);
  const double weights = static_cast<double>(parts) * N * K;
  if (M <= 128) {
    int64_t r = 1;
    while (r < rows && r < 16) r *= 2;
    if (rows > 16) r = ceil_div(rows, 16) * 16;
    const double few = 2.5 + std::max(weights / 5e6, weights * r / 36e6);
    const double waves = static_cast<double>(ceil_div(parts * ceil_div(rows, 32) * ceil_div(N, 128), num_sms));
    const double tiled = 5.0 + std::max(0.27 * static_cast<double>(kt) * waves, weights / 6.2e6);
    if (few < tiled) return kFewTokens;
  }
  const int64_t wide = ceil_div(M, kInt8WideTokens) * ceil_div(N, 256);
  if (num_sms > 1 && rows > 96 && 2 * wide >= num_sms) return kInt8WideTokens;
  int32_t t = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  while (t > 16 && parts * ceil_div(rows, t / 2) * ceil_div(N, 128) <= num_sms) t /= 2;
  return t;
}

}  // namespace

extern "C" {

tst_status gemm_int8_plan_create(tst_int8_plan** out, int64_t M, int64_t N, int64_t K, const tst_int8_options* opts) {
  if (out == nullptr) return TST_ERR_INVALID_ARG;
  *out = nullptr;
  if (opts == nullptr || M < 1 || N < 1 || K < 1) return TST_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31)) return TST_ERR_INVALID_ARG;
  if (opts->groups < 0 || opts->num_sms < 0 || opts->timeout_ns < 0) return TST_ERR_INVALID_ARG;
  if (opts->out_dtype != TST_OUT_F32 && opts->out_dtype != TST_OUT_BF16) return TST_ERR_INVALID_ARG;
  if (opts->host_only && opts->num_sms == 0) return TST_ERR_INVALID_ARG;
  const int32_t tr = opts->tile_rows;
  if (tr < 0) return TST_ERR_INVALID_ARG;
  if ((tr != 0 && tr != kFewTokens && tr != 16 && tr != 32 && tr != 64 && tr != 128 && tr != kInt8WideTokens) ||
      (tr == kInt8WideTokens && opts->num_sms == 1) || (tr == kFewTokens && M > kMaxFewRows))
    return TST_ERR_UNSUPPORTED;
  if (K % 16 != 0) return TST_ERR_ALIGNMENT;   // a row of K bytes is a row of the tensor map
  const int64_t groups = opts->groups;
  if (M > kMaxRows || N > kMaxRows || std::max<int64_t>(groups, 1) * N > kMaxRows || K > kMaxK || groups > kBsWalkGroups)
    return TST_ERR_UNSUPPORTED;
  tst_int8_plan* p = new (std::nothrow) tst_int8_plan();
  if (p == nullptr) return TST_ERR_OOM;
  p->M = M;
  p->N = N;
  p->K = K;
  p->opts = *opts;
  p->num_sms = opts->num_sms;
  if (!opts->host_only) {
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
    p->num_sms = opts->num_sms > 0 ? std::min(opts->num_sms, sms) : sms;
  }
  const int32_t tokens = tr > 0 ? tr : tile_tokens(M, N, K, groups, p->num_sms);
  p->tokens = tokens;
  p->pairs = tokens == kInt8WideTokens;
  const bool pairs = p->pairs;
  const bool few = tokens == kFewTokens;
  const int32_t cols = few ? 0 : pairs ? 256 : 128;
  const int64_t mt = few ? 0 : ceil_div(M, tokens), nt = few ? 0 : ceil_div(N, cols);
  const int64_t tiles = (mt + groups) * nt;   // grouped: at most, whatever the split; none without tiles
  if (tiles >= (int64_t(1) << 30)) { delete p; return TST_ERR_UNSUPPORTED; }
  const int64_t kt = ceil_div(K, 128);
  if (!few) p->kernel = tst_int8_kernel(tokens, opts->out_dtype == TST_OUT_BF16 ? tst::OUT_BF16 : tst::OUT_F32);
  p->dev_bytes = 256 + (few ? 0 : 2 * static_cast<size_t>(M) * K);
  if (!opts->host_only) {
    if (!few && cudaFuncSetAttribute(p->kernel.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p->kernel.smem_bytes) != cudaSuccess) {
      cudaGetLastError();
      delete p;
      return TST_ERR_CUDA;
    }
    if (cudaMalloc(&p->d_status, p->dev_bytes) != cudaSuccess) {
      cudaGetLastError();
      delete p;
      return TST_ERR_OOM;
    }
    if (!zero_now(p->d_status, 256)) {
      cudaGetLastError();
      cudaFree(p->d_status);
      delete p;
      return TST_ERR_CUDA;
    }
  }
  tst::Sched& s = p->sched;
  s.mt = static_cast<int32_t>(mt);
  s.nt = static_cast<int32_t>(nt);
  s.kt = static_cast<int32_t>(kt);
  s.map_kind = tst::MAP_GROUPED_M;
  s.group = 8;
  s.dp_tiles = static_cast<int32_t>(mt * nt);
  s.grid = static_cast<int32_t>(std::min<int64_t>(p->num_sms / (pairs ? 2 : 1), tiles));
  if (!few && s.grid < 1) s.grid = 1;
  s.sk_groups = 1;
  s.rows = static_cast<int32_t>(M);
  s.bm = tokens;
  s.bn = cols;
  s.groups = static_cast<int32_t>(groups);
  s.group_b_rows = static_cast<int32_t>(N);
  s.cols = static_cast<int32_t>(N);
  s.bk = 128;
  *out = p;
  return TST_OK;
}

tst_status gemm_int8_plan_destroy(tst_int8_plan* p) {
  if (p == nullptr) return TST_OK;
  const tst_status st = p->d_status && cudaFree(p->d_status) != cudaSuccess ? TST_ERR_CUDA : TST_OK;
  delete p;
  return st;
}

tst_status gemm_int8_plan_get_info(const tst_int8_plan* p, tst_int8_plan_info* info) {
  if (p == nullptr || info == nullptr) return TST_ERR_INVALID_ARG;
  info->M = p->M;
  info->N = p->N;
  info->K = p->K;
  info->groups = p->sched.groups;
  info->tile_rows = p->tokens;
  info->tile_cols = p->sched.bn;
  info->grid = p->sched.grid * (p->pairs ? 2 : 1);
  info->smem_bytes = p->kernel.smem_bytes;
  info->workspace_bytes = static_cast<int64_t>(p->dev_bytes);
  return TST_OK;
}

tst_status gemm_int8_status_query(tst_int8_plan* p) {
  if (p == nullptr) return TST_ERR_INVALID_ARG;
  if (p->opts.host_only) return TST_ERR_NO_DEVICE;
  if (!p->ran) return TST_OK;
  unsigned long long word = 0;
  if (cudaStreamSynchronize(p->last_stream) != cudaSuccess ||
      cudaMemcpy(&word, p->d_status, sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess)
    return TST_ERR_CUDA;
  if (word == 0) return TST_OK;
  if (!zero_now(p->d_status, sizeof(word))) return TST_ERR_CUDA;   // before any later run
  return (word & 0xFFu) == tst::ST_TIMEOUT ? TST_ERR_TIMEOUT : TST_ERR_DEVICE_CHECK;
}

tst_status gemm_int8_run(tst_int8_plan* p, const int32_t* group_rows, const int8_t* A, const int8_t* B, void* D,
                         const float* row_scale, const float* col_scale, const float* bias, void* stream) {
  if (p == nullptr || A == nullptr || B == nullptr || D == nullptr || row_scale == nullptr || col_scale == nullptr)
    return TST_ERR_INVALID_ARG;
  if ((p->sched.groups > 0) != (group_rows != nullptr) || (p->opts.has_bias && bias == nullptr)) return TST_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, p->opts.out_dtype == TST_OUT_F32 ? 4 : 2) || !aligned(group_rows, 4) ||
      !aligned(row_scale, 4) || !aligned(col_scale, 4) || (p->opts.has_bias && !aligned(bias, 4)))
    return TST_ERR_ALIGNMENT;
  if (p->opts.host_only) return TST_ERR_NO_DEVICE;
  int now = -1;
  if (cudaGetDevice(&now) != cudaSuccess) {
    cudaGetLastError();
    return TST_ERR_CUDA;
  }
  if (now != p->device) return TST_ERR_INVALID_ARG;
  tst::KernelParams kp = {};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool pairs = p->pairs;
  void* const half = p->d_status + 32;
  kp.C = D;
  kp.bias = p->opts.has_bias ? bias : nullptr;
  kp.has_bias = p->opts.has_bias ? 1 : 0;
  kp.relu = p->opts.relu ? 1 : 0;
  kp.ext.row_scale = row_scale;
  kp.ext.col_scale = col_scale;
  kp.status = p->d_status;
  kp.run_id = kp.status_floor = kStatusTag;
  kp.M = static_cast<int32_t>(p->M);
  kp.N = static_cast<int32_t>(p->N);
  kp.K = static_cast<int32_t>(p->K);
  kp.sched = p->sched;
  kp.sched.group_rows = group_rows;
  kp.tma_store = aligned(D, 4) && p->N % 2 == 0;   // BF16 rows of whole words
  kp.timeout_ns = p->opts.timeout_ns > 0 ? static_cast<uint64_t>(p->opts.timeout_ns) : 10ull * 1000 * 1000 * 1000;
  p->last_stream = s;
  p->ran = true;
  if (p->tokens == kFewTokens)
    return tst_int8_few(kp, A, B, p->opts.out_dtype == TST_OUT_BF16 ? tst::OUT_BF16 : tst::OUT_F32, s) ? TST_OK : TST_ERR_CUDA;
  if (!tst_encode_halves(&kp.tmap_a, half, p->M, p->K, pairs ? p->tokens / 2 : p->tokens) ||
      !tst_encode_bytes(&kp.tmap_b, B, std::max<int64_t>(p->sched.groups, 1) * p->N, p->K, 128))
    return TST_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p->sched.grid * (pairs ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(p->kernel.threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(p->kernel.smem_bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned na = 0;
  if (pairs) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
  }
  // it may start while A is made FP16, and waits for that itself
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  cfg.attrs = attr;
  cfg.numAttrs = na;
  void* args[] = {&kp};
  if (!tst_int8_widen(A, half, p->M, p->K, group_rows, p->sched.groups, p->num_sms, s)) return TST_ERR_CUDA;
  if (cudaLaunchKernelExC(&cfg, p->kernel.kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return TST_ERR_CUDA;
  }
  return TST_OK;
}

}  // extern "C"
