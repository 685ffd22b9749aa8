// CPU-only checks of the host side of the 16-bit experts and the adapters
// (abi_dense.cpp and its share of plan.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer: launch failures reach the caller, refused calls
// launch nothing, and sizes up to the limits are planned without overflow.
#include <initializer_list>

#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "launch.h"
#include "moe_qexpert.h"
#include "stub_device.h"

namespace {
int failures = 0;
moe::Gemm16Args last;
int launched() {
  ++stub::launches;
  return stub::launch_error;
}
void* at(uintptr_t a) { return reinterpret_cast<void*>(a); }
template <class T>
T* as(uintptr_t a) { return static_cast<T*>(at(a)); }
}  // namespace

#define CHECK(cond)                                                            \
  do {                                                                         \
    if (!(cond)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                              \
    }                                                                          \
  } while (0)

namespace moe {
int launch_gemm16(const Gemm16Args& a, void*) {
  last = a;
  return launched();
}
int launch_gemm16_grad_rows(const Gemm16Args& a, void*) {
  last = a;
  return launched();
}
int launch_gemm16_grad_weights(const Gemm16Args& a, void*) {
  last = a;
  return launched();
}
int launch_combine_grad(const CombineGradArgs&, void*) { return launched(); }
int launch_adapter_add(const AdapterArgs&, void*) { return launched(); }
}  // namespace moe

static moe_status product(int E, int N, int K, int rows, int M, int epi, int kernel, const int32_t* gather = nullptr) {
  return moe_grouped_gemm(at(0x1000), MOE_DTYPE_BF16, E, N, K, at(0x2000), rows, gather, 2, as<int32_t>(0x3000), M, epi, kernel,
                          nullptr, at(0x4000), nullptr);
}
static moe_status weights(int E, int N, int K, int M, void* ws, size_t bytes) {
  return moe_grouped_gemm_grad_weights(at(0x1000), at(0x2000), MOE_DTYPE_F16, E, N, K, M, nullptr, 1, as<int32_t>(0x3000), M,
                                       MOE_EPI_NONE_F32, MOE_KERNEL_AUTO, at(0x4000), ws, bytes, nullptr);
}
static moe_status combine() {
  return moe_unpermute_combine_grad(as<uint16_t>(0x1000), at(0x2000), MOE_DTYPE_F16, as<int32_t>(0x3000), nullptr,
                                    as<float>(0x4000), nullptr, 4, 2, 64, 0, MOE_DTYPE_BF16, at(0x5000), as<float>(0x6000),
                                    nullptr, nullptr);
}
static moe_status adapters(int n, int r, int K, int N, int T) {
  return moe_adapter_add(at(0x1000), MOE_DTYPE_F32, at(0x2000), at(0x3000), at(0x4000), MOE_DTYPE_BF16, nullptr, n, r, K, N,
                         as<int32_t>(0x5000), as<int32_t>(0x6000), T, at(0x1000), nullptr);
}

int main() {
  // launches that fail
  stub::launch_error = 98;
  CHECK(product(4, 64, 64, 8, 8, MOE_EPI_NONE, 0) == MOE_ERR_HIP && strstr(moe_last_error_detail(), "grouped_gemm launch"));
  CHECK(weights(4, 64, 64, 8, nullptr, 0) == MOE_ERR_HIP && strstr(moe_last_error_detail(), "grad_weights"));
  CHECK(combine() == MOE_ERR_HIP && strstr(moe_last_error_detail(), "combine_grad"));
  CHECK(adapters(4, 16, 64, 64, 9) == MOE_ERR_HIP && strstr(moe_last_error_detail(), "adapter_add"));
  stub::launch_error = 0;
  CHECK(product(4, 64, 64, 8, 8, MOE_EPI_NONE, 0) == MOE_OK && moe_last_error_detail()[0] == '\0');
  stub::pending_error = 700;  // left by the caller
  CHECK(combine() == MOE_OK && stub::pending_error == 0);

  // refused calls launch nothing; an empty batch launches nothing, but its weights' gradient does (zeros)
  int n = stub::launches;
  CHECK(product(4, 64, 64, 7, 8, MOE_EPI_NONE, 0) == MOE_ERR_BAD_SHAPE);
  CHECK(product(INT_MAX, 64, 64, 8, 8, MOE_EPI_NONE, 0) == MOE_ERR_BAD_SHAPE);
  CHECK(product(4, INT_MAX - 7, INT_MAX - 7, 8, 8, MOE_EPI_NONE, 0) == MOE_ERR_UNSUPPORTED);
  CHECK(product(4, 64, 64, INT_MAX, INT_MAX, MOE_EPI_NONE, 0, as<int32_t>(0x7000)) == MOE_ERR_UNSUPPORTED);
  CHECK(product(4, 64, 64, INT_MAX, 1 << 30, MOE_EPI_NONE, 0) == MOE_ERR_UNSUPPORTED);
  CHECK(weights(4, 64, 64, 1 << 30, nullptr, 0) == MOE_ERR_UNSUPPORTED);
  CHECK(adapters(1024, 128, 1 << 30, 1 << 30, (1 << 24) - 1) == MOE_ERR_UNSUPPORTED);
  CHECK(adapters(INT_MAX, 128, 64, 64, 4) == MOE_ERR_BAD_SHAPE);
  CHECK(product(4, 64, 64, 0, 0, MOE_EPI_NONE, 0) == MOE_OK && adapters(4, 16, 64, 64, 0) == MOE_OK);
  CHECK(stub::launches == n);
  CHECK(weights(4, 64, 64, 0, nullptr, 0) == MOE_OK && stub::launches == n + 1 && last.M_total == 0);

  // the largest calls, without gather_pair past 4 GiB too
  CHECK(product(1024, 1 << 20, 2040, INT_MAX, (1 << 30) - 1, MOE_EPI_NONE_F32, 0) == MOE_OK);
  CHECK(product(1, 1 << 20, 2048, 8, 8, MOE_EPI_NONE_F32, 0) == MOE_ERR_UNSUPPORTED);  // 4 GiB of weights

  // plans at the limits
  for (int M : {0, 1, 64, 1000, 100000, INT_MAX})
    for (int E : {1, 8, 65, 1024})
      for (int N : {8, 264, 4096, 1 << 20})
        for (int K : {8, 264, 4096, 1 << 20})
          for (int kernel : {0, 1, 5, 9})
            for (int what : {0, 1, 2}) {
              const int path = moe::gemm16_path(what, E, N, K, M, kernel);
              CHECK(path == 0 || path == 128 || path == 256 || path == moe::kGemm16Deep);
              CHECK(what != 2 || path == 128 || path == 256);
              CHECK(kernel != 9 || path == 256);
              CHECK(kernel != 5 || path == 128 || path == moe::kGemm16Deep);
              if (what != 2 || kernel == 1) continue;
              const int parts = moe::gemm16_splits(E, N, K, M, kernel);
              const size_t bytes = moe::gemm16_grad_weights_workspace_bytes(E, N, K, M, kernel);
              CHECK(parts >= 1 && parts <= 512 && (parts == 1 || path == 128));
              CHECK(bytes == (parts > 1 ? (size_t)parts * E * N * K * 4 : 0));
              CHECK(parts == 1 || (int64_t)parts * 512 * E <= M);
              CHECK(bytes <= (size_t)512 * 128 * 128 * 4);  // 512 tiles of 128 x 128 at most
            }

  if (failures) return 1;
  printf("dense host layer checks passed\n");
  return 0;
}
