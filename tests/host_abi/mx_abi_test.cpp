// CPU-only checks of the host side of the scored routing and the MX path
// (abi_mx.cpp and its share of plan.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer: launch failures reach the caller, a layer stops at
// the launch that fails, refused calls launch nothing, and sizes up to the
// limits of the calls are planned without overflow.
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
int fail_at = -1;       // launches from now until one fails
bool start_groups = true;
moe::MxGemmArgs last_product;

int mx_launched() {
  ++stub::launches;
  if (fail_at > 0 && --fail_at == 0) return 719;
  return stub::launch_error;
}
void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }
template <class T>
T* at(uintptr_t a) { return static_cast<T*>(fake(a)); }
}  // namespace

#define CHECK(cond)                                                            \
  do {                                                                         \
    if (!(cond)) {                                                             \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                              \
    }                                                                          \
  } while (0)

namespace moe {
int launch_route_scored(const ScoredArgs&, void*) { return mx_launched(); }
int launch_mx_front(const ScoredArgs&, const FrontRows&, const FrontGroups&, bool* grouped, void*) {
  *grouped = start_groups;
  return mx_launched();
}
int launch_quantize_mx(const void*, int, int64_t, int, int, uint8_t*, uint8_t*, void*) { return mx_launched(); }
int launch_dequantize_mx(const uint8_t*, const uint8_t*, int64_t, int, int, int, void*, void*) { return mx_launched(); }
int launch_rmsnorm_mx(const NormArgs&, void*) { return mx_launched(); }
int launch_mx_repack(const uint8_t*, const uint8_t*, int, int, int, uint8_t*, uint8_t*, void*) { return mx_launched(); }
int launch_mxgemm(const MxGemmArgs& a, void*) {
  last_product = a;
  return mx_launched();
}
}  // namespace moe

static moe_mxdesc desc(int layout, int E, int N, int K, uintptr_t base) {
  moe_mxdesc d;
  memset(&d, 0, sizeof(d));
  d.abi_version = MOE_ABI_VERSION;
  d.layout = layout;
  d.E = E;
  d.N = N;
  d.K = K;
  d.codes = at<uint8_t>(base);
  d.scales = at<uint8_t>(base + 0x1000);
  return d;
}

static moe_status route(int T, int k) {
  return moe_route_scored(at<float>(0x1000), nullptr, T, 64, k, MOE_SCORE_SIGMOID, 1, 1, 1, 1, 1.0f, at<int32_t>(0x2000),
                          at<float>(0x3000), nullptr);
}

static moe_status layer(int T, size_t ws, const moe_mxdesc& gu, const moe_mxdesc& dn) {
  moe_mxlayer l;
  memset(&l, 0, sizeof(l));
  l.abi_version = MOE_ABI_VERSION;
  l.T = T;
  l.k = 2;
  l.x_dtype = MOE_DTYPE_BF16;
  l.x_fmt = l.h_fmt = MOE_MX_E4M3;
  l.y_dtype = MOE_DTYPE_F16;
  l.n_group = l.topk_group = l.group_top = l.renormalize = 1;
  l.scale = 1.0f;
  l.gate_up = &gu;
  l.down = &dn;
  uintptr_t p = 0x100000;
  const auto next = [&p] { return p += 0x1000; };
  l.x = fake(next());
  l.logits = at<float>(next());
  l.topk_ids = at<int32_t>(next());
  l.topk_w = at<float>(next());
  l.expert_counts = at<int32_t>(next());
  l.seg_offsets = at<int32_t>(next());
  l.sorted_pair = at<int32_t>(next());
  l.pair_pos = at<int32_t>(next());
  l.workspace = fake(next());
  l.workspace_bytes = ws;
  l.x_codes = at<uint8_t>(next());
  l.x_scales = at<uint8_t>(next());
  l.h_codes = at<uint8_t>(next());
  l.h_scales = at<uint8_t>(next());
  l.y = fake(next());
  l.out = at<uint16_t>(next());
  return moe_mx_layer(&l, nullptr);
}

int main() {
  // a launch that fails
  stub::launch_error = 98;
  CHECK(route(4, 2) == MOE_ERR_HIP);
  CHECK(strstr(moe_last_error_detail(), "route_scored") && strstr(moe_last_error_detail(), "stub device error"));
  CHECK(moe_quantize_mx(fake(0x1000), MOE_DTYPE_BF16, 4, 64, MOE_MX_E4M3, at<uint8_t>(0x2000), at<uint8_t>(0x3000),
                        nullptr) == MOE_ERR_HIP);
  CHECK(moe_rmsnorm_mx(fake(0x1000), nullptr, fake(0x2000), MOE_DTYPE_F16, 4, 64, 1e-5f, nullptr, fake(0x3000), 0, nullptr,
                       nullptr, nullptr) == MOE_ERR_HIP);
  stub::launch_error = 0;
  CHECK(route(4, 2) == MOE_OK && moe_last_error_detail()[0] == '\0');

  // an error that the caller left pending is not this call's
  stub::pending_error = 700;
  CHECK(route(4, 2) == MOE_OK && stub::pending_error == 0);

  // refused calls launch nothing
  int n = stub::launches;
  CHECK(route(-1, 2) == MOE_ERR_BAD_SHAPE && route(1 << 25, 1) == MOE_ERR_BAD_SHAPE && route(4, 65) == MOE_ERR_BAD_SHAPE);
  CHECK(moe_dequantize_mx(at<uint8_t>(0x1000), at<uint8_t>(0x2000), INT64_MAX, INT_MAX - 31, MOE_MX_E2M1, 0, fake(0x3000),
                          nullptr) == MOE_ERR_BAD_SHAPE);
  CHECK(moe_rmsnorm_mx(fake(0x1000), nullptr, fake(0x2000), 0, INT64_MAX, 64, 0.0f, nullptr, fake(0x3000), 0, nullptr,
                       nullptr, nullptr) == MOE_ERR_BAD_SHAPE);
  CHECK(stub::launches == n);

  // the largest calls
  CHECK(route((1 << 25) - 1, 63) == MOE_OK);
  CHECK(moe_quantize_mx(fake(0x1000), MOE_DTYPE_F32, ((int64_t)1 << 29) - 1, 32, MOE_MX_E2M1, at<uint8_t>(0x2000),
                        at<uint8_t>(0x3000), nullptr) == MOE_OK);

  // a layer: start, two products, combine; and the grouping where the start leaves it
  const moe_mxdesc gu = desc(MOE_LAYOUT_TILED, 64, 512, 128, 0x10000), dn = desc(MOE_LAYOUT_TILED, 64, 128, 256, 0x20000);
  const size_t ws = moe_mx_layer_workspace_size(100, 2, 64);
  n = stub::launches;
  CHECK(layer(100, ws, gu, dn) == MOE_OK && stub::launches == n + 4);
  CHECK(last_product.M_total == 200 && last_product.K == 256 && last_product.gather == nullptr &&
        last_product.epilogue == MOE_EPI_NONE_F16);
  start_groups = false;
  n = stub::launches;
  CHECK(layer(100, ws, gu, dn) == MOE_OK && stub::launches == n + 5);
  start_groups = true;
  n = stub::launches;
  CHECK(layer(100, ws - 1, gu, dn) == MOE_ERR_WORKSPACE_TOO_SMALL && layer(0, 0, gu, dn) == MOE_OK);
  CHECK(layer(100, ws, dn, gu) == MOE_ERR_BAD_SHAPE && stub::launches == n);
  for (int i = 1; i <= 3; ++i) {  // the launch that fails is the last
    n = stub::launches;
    fail_at = i;
    CHECK(layer(100, ws, gu, dn) == MOE_ERR_HIP && stub::launches == n + i);
    CHECK(strstr(moe_last_error_detail(), "mx_layer"));
  }
  fail_at = -1;

  // plans at the limits: workspaces, kernel paths
  const int most[] = {0, 1, 15, 16, 17, 8192, 1 << 20, (1 << 25) - 1};
  for (int T : most)
    for (int E : {1, 2, 63, 64, 65, 512, 513, 1024})
      for (int k : {1, 8, 63}) {
        if (k > E) continue;
        const size_t w = moe_mx_layer_workspace_size(T, k, E);
        const int tokens = moe::front_chunk_tokens(T, k, E);
        CHECK(w >= 256 && (tokens == 0 || w >= 256 + ((size_t)T + tokens - 1) / tokens * (E + 1) * 4));
        CHECK(tokens == 0 || tokens == moe::chunk_tokens(E <= 512 ? 1 : 16));
      }
  for (int M : {1, 64, 100000, INT_MAX})
    for (int E : {1, 8, 1024})
      for (int N : {32, 512, 1 << 20})
        for (int K : {128, 256, 512, 4096, 1 << 20})
          for (int kernel : {0, 1, 4, 5, 8}) {
            const bool e2m1 = kernel == 8 || (M & 1);
            const int path = moe::mxgemm_path(M, E, N, K, e2m1, kernel);
            CHECK(path == 0 || path == 64 || path == 128 || path == moe::kMxSplit);
            CHECK(path != moe::kMxSplit || (e2m1 && (K > 256 || kernel == 8)));
          }
  const moe_mxdesc wide = desc(MOE_LAYOUT_CANONICAL, 1024, 32, 384, 0x30000);
  CHECK(moe_mx_field_bytes(&wide, MOE_FIELD_CODES) == (size_t)1024 * 32 * 192);
  const moe_mxdesc tiled = desc(MOE_LAYOUT_TILED, 1024, 32, 384, 0x40000);
  CHECK(moe_mx_field_bytes(&tiled, MOE_FIELD_CODES) == (size_t)1024 * 32 * 256 &&
        moe_mx_field_bytes(&tiled, MOE_FIELD_SCALES) == (size_t)1024 * 32 * 16);
  CHECK(moe_mx_repack(&wide, &tiled, nullptr) == MOE_OK);

  if (failures) return 1;
  printf("MX host layer checks passed\n");
  return 0;
}
