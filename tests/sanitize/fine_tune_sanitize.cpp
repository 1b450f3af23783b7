// Host-side checks of the operators for fine-tuning a draft under
// AddressSanitizer and UndefinedBehaviorSanitizer: their argument validation,
// which answers before any HIP call, at the ends of its ranges.  Prints "ok"
// and exits 0 when every check holds.
#include <cfloat>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "specverify.h"

static int g_fail = 0;
#define CHECK(cond)                                                  \
  do {                                                               \
    if (!(cond)) {                                                   \
      std::printf("FAIL line %d: %s\n", __LINE__, #cond);            \
      ++g_fail;                                                      \
    }                                                                \
  } while (0)

// addresses a terabyte apart, never dereferenced
template <typename T>
static T* at(int i) {
  return reinterpret_cast<T*>((uintptr_t)(i + 1) << 40);
}

int main() {
  const int32_t big = std::numeric_limits<int32_t>::max(), small = std::numeric_limits<int32_t>::min();
  const float nan = std::numeric_limits<float>::quiet_NaN(), inf = std::numeric_limits<float>::infinity();

  auto layer = [&](int32_t rows, int32_t d, float eps, int32_t dt, int32_t odt, void* out, void* hres) {
    return sv_layer_norm(at<void>(0), at<void>(1), at<void>(2), at<void>(6), eps, out, at<float>(4), hres, rows, d, dt, odt,
                         nullptr);
  };
  void *o = at<void>(3), *h = at<void>(5);
  CHECK(layer(small, 64, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(layer(big, SV_MAX_NORM_D, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(layer(big, 1, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(layer(3, big, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(layer(3, small, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(layer(3, 64, nan, SV_BF16, SV_BF16, o, h) == SV_ERR_PARAM);
  CHECK(layer(3, 64, inf, SV_BF16, SV_BF16, o, h) == SV_ERR_PARAM);
  CHECK(layer(3, 64, 1e-6f, big, SV_BF16, o, h) == SV_ERR_DTYPE);
  CHECK(layer(3, 64, 1e-6f, SV_BF16, small, o, h) == SV_ERR_DTYPE);
  CHECK(layer(1 << 21, 512, 1e-6f, SV_F32, SV_BF16, at<void>(0), h) == SV_ERR_PARAM);
  CHECK(layer(0, 64, 1e-6f, SV_BF16, SV_BF16, nullptr, nullptr) == SV_OK);

  auto back = [&](int32_t rows, int32_t d, float eps, int32_t dt, void* dh, int64_t bytes) {
    const int a = sv_layer_norm_backward(at<void>(0), at<void>(1), at<void>(2), at<void>(3), eps, dh, at<float>(5),
                                         at<float>(6), at<void>(7), bytes, rows, d, dt, nullptr);
    const int b = sv_rms_norm_backward(at<void>(0), at<void>(1), at<void>(2), at<void>(3), eps, dh, at<float>(5), at<void>(7),
                                       bytes, rows, d, dt, nullptr);
    CHECK(a == b);
    return a;
  };
  void* dh = at<void>(4);
  CHECK(back(small, 64, 1e-6f, SV_BF16, dh, 1 << 30) == SV_ERR_SHAPE);
  CHECK(back(3, big, 1e-6f, SV_BF16, dh, 1 << 30) == SV_ERR_SHAPE);
  CHECK(back(3, small, 1e-6f, SV_BF16, dh, 1 << 30) == SV_ERR_SHAPE);
  CHECK(back(1 << 30, SV_MAX_NORM_D, 1e-6f, SV_F32, at<void>(2), std::numeric_limits<int64_t>::max()) == SV_ERR_PARAM);
  CHECK(back(300, 64, nan, SV_BF16, dh, 1 << 30) == SV_ERR_PARAM);
  CHECK(back(300, 64, 1e-6f, big, dh, 1 << 30) == SV_ERR_DTYPE);
  CHECK(back(300, 64, 1e-6f, SV_BF16, dh, 0) == SV_ERR_WORKSPACE);
  CHECK(back(300, 64, 1e-6f, SV_BF16, dh, std::numeric_limits<int64_t>::min()) == SV_ERR_WORKSPACE);
  CHECK(back(big, 1, 1e-6f, SV_BF16, dh, 1 << 30) == SV_ERR_SHAPE);
  CHECK(sv_norm_backward_workspace(1 << 30, SV_MAX_NORM_D) > 0);
  CHECK(sv_norm_backward_workspace(1 << 30, 1) > 0);
  CHECK(sv_norm_backward_workspace(big, 1) == SV_ERR_SHAPE);
  CHECK(sv_norm_backward_workspace(small, 64) == SV_ERR_SHAPE);
  CHECK(sv_norm_backward_workspace(64, big) == SV_ERR_SHAPE);
  CHECK(sv_norm_backward_workspace(0, 64) == 0);

  auto top = [&](int32_t rows, int32_t V, int32_t k, float T, int32_t dt, float* values) {
    return sv_top_logits(at<void>(0), k, T, values, at<int32_t>(2), at<float>(3), rows, V, dt, nullptr);
  };
  float* v = at<float>(1);
  CHECK(top(big, SV_MAX_V, 4, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(big, 1, 1, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(small, 64, 4, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(3, big, 4, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(3, small, 4, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(3, 64, big, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(3, 64, small, 1.0f, SV_F32, v) == SV_ERR_SHAPE);
  CHECK(top(3, SV_MAX_V, SV_MAX_TOP, 1.0f, SV_F32, at<float>(0)) == SV_ERR_PARAM);
  CHECK(top(3, SV_MAX_V, SV_MAX_TOP, nan, SV_F32, v) == SV_ERR_PARAM);
  CHECK(top(3, 64, 4, FLT_MIN / 2, SV_F32, v) == SV_ERR_PARAM);
  CHECK(top(3, 64, 4, 1.0f, small, v) == SV_ERR_DTYPE);
  CHECK(top(0, 64, 4, 1.0f, SV_F32, nullptr) == SV_OK);

  auto distill = [&](int32_t rows, int32_t V, int32_t k, float T, int32_t dt, float* loss, void* grad) {
    return sv_distill_loss(at<void>(0), at<int32_t>(1), at<float>(2), at<float>(3), at<float>(4), T, loss, grad, rows, V, k, dt,
                           nullptr);
  };
  float* l = at<float>(5);
  void* g = at<void>(6);
  CHECK(distill(big, SV_MAX_DISTILL_V, 4, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(big, 1, 1, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(small, 64, 4, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(3, big, 4, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(3, small, 4, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(3, 64, big, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(3, 64, small, 1.0f, SV_F32, l, g) == SV_ERR_SHAPE);
  CHECK(distill(3, SV_MAX_DISTILL_V, SV_MAX_TOP, inf, SV_F32, l, g) == SV_ERR_PARAM);
  CHECK(distill(1 << 20, SV_MAX_DISTILL_V, SV_MAX_TOP, 1.0f, SV_F32, l, at<void>(1)) == SV_ERR_PARAM);
  CHECK(distill(3, 64, 4, 1.0f, big, l, g) == SV_ERR_DTYPE);
  CHECK(distill(3, 64, 4, 1.0f, SV_BF16, nullptr, nullptr) == SV_ERR_NULL);
  CHECK(distill(0, 64, 4, 1.0f, SV_BF16, nullptr, nullptr) == SV_OK);

  if (g_fail == 0) std::printf("ok\n");
  return g_fail != 0;
}
