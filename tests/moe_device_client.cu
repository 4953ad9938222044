// Runs of a mixture-of-experts plan while another GPU is current, with a fake of cudaGetDevice: the host
// side of csrc/moe.cu is compiled into this program, which needs no GPU.  Exit code: the number of calls
// that did not return what they should.
#include <cuda_runtime.h>
#include <cstdio>

static int g_current = 0;
static cudaError_t fake_get_device(int* device) {
  *device = g_current;
  return g_current < 0 ? cudaErrorUnknown : cudaSuccess;
}
#define cudaGetDevice fake_get_device
#include "moe.cu"

static int g_wrong = 0;
static void expect(const char* what, tst_status got, tst_status want) {
  if (got == want) return;
  std::printf("%s with GPU %d current: %d, not %d\n", what, g_current, got, want);
  ++g_wrong;
}

static void all_calls(tst_moe_plan* p, int64_t tokens, tst_status want) {
  alignas(16) static char b[4096];   // addresses that are only checked
  int32_t* i = reinterpret_cast<int32_t*>(b);
  float* f = reinterpret_cast<float*>(b);
  expect("moe_route", moe_route(p, tokens, b, TST_OUT_F32, 8, nullptr, i, f, i, i, i, f, nullptr), want);
  expect("moe_route_backward",
         moe_route_backward(p, tokens, b, TST_OUT_F32, 8, nullptr, i, i, i, f, f, b, 8, nullptr), want);
  expect("moe_dispatch", moe_dispatch(p, tokens, 16, b, TST_OUT_F32, 16, i, b, TST_OUT_F32, 8, nullptr, nullptr), want);
  expect("moe_combine", moe_combine(p, tokens, 16, b, TST_OUT_F32, 8, i, f, b, TST_OUT_F32, 16, nullptr), want);
  expect("moe_combine_backward",
         moe_combine_backward(p, tokens, 16, b, TST_OUT_F32, 8, i, f, b, TST_OUT_F32, 16, b, f, nullptr), want);
}

int main() {
  tst_moe_plan p;   // as if made while GPU 0 was current
  p.max_tokens = 4;
  p.experts = 8;
  p.top_k = 2;
  p.device = 0;
  for (int device : {1, 7}) {
    g_current = device;
    all_calls(&p, 4, TST_ERR_INVALID_ARG);
    all_calls(&p, 0, TST_ERR_INVALID_ARG);
  }
  g_current = -1;   // the query itself fails
  all_calls(&p, 4, TST_ERR_CUDA);
  g_current = 0;    // its own GPU: no tokens, nothing to launch
  alignas(16) static char b[64];
  int32_t* i = reinterpret_cast<int32_t*>(b);
  float* f = reinterpret_cast<float*>(b);
  expect("moe_dispatch", moe_dispatch(&p, 0, 16, b, TST_OUT_F32, 16, i, b, TST_OUT_F32, 8, nullptr, nullptr), TST_OK);
  expect("moe_combine", moe_combine(&p, 0, 16, b, TST_OUT_F32, 8, i, f, b, TST_OUT_F32, 16, nullptr), TST_OK);
  expect("moe_route_backward", moe_route_backward(&p, 0, b, TST_OUT_F32, 8, nullptr, i, i, i, f, f, b, 8, nullptr), TST_OK);
  p.host_only = true;
  p.device = -1;
  g_current = 3;    // a host-only plan has no GPU of its own
  all_calls(&p, 4, TST_ERR_NO_DEVICE);
  return g_wrong;
}
