// Host-side checks of sv_rms_norm, sv_linear and sv_adjust_logits under
// AddressSanitizer and UndefinedBehaviorSanitizer: their argument validation,
// which answers before any HIP call, at the ends of its ranges.  Prints "ok"
// and exits 0 when every check holds.
#include <cmath>
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
  auto norm = [&](int32_t rows, int32_t d, float eps, int32_t dt, int32_t odt, void* out, void* hres) {
    return sv_rms_norm(at<void>(0), at<void>(1), at<void>(2), eps, out, at<float>(4), hres, rows, d, dt, odt, nullptr);
  };
  void *o = at<void>(3), *h = at<void>(5);
  CHECK(norm(small, 64, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(norm(big, SV_MAX_NORM_D, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(norm(3, big, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(norm(3, small, 1e-6f, SV_BF16, SV_BF16, o, h) == SV_ERR_SHAPE);
  CHECK(norm(3, 64, nan, SV_BF16, SV_BF16, o, h) == SV_ERR_PARAM);
  CHECK(norm(3, 64, inf, SV_BF16, SV_BF16, o, h) == SV_ERR_PARAM);
  CHECK(norm(3, 64, 1e-6f, big, SV_BF16, o, h) == SV_ERR_DTYPE);
  CHECK(norm(3, 64, 1e-6f, SV_BF16, small, o, h) == SV_ERR_DTYPE);
  CHECK(norm(1 << 21, 512, 1e-6f, SV_F32, SV_BF16, at<void>(0), h) == SV_ERR_PARAM);
  CHECK(norm(3, 64, 1e-6f, SV_BF16, SV_BF16, h, h) == SV_ERR_PARAM);
  CHECK(norm(0, 64, 1e-6f, SV_BF16, SV_BF16, nullptr, nullptr) == SV_OK);

  auto lin = [&](int32_t M, int32_t N, int32_t K, int32_t R, int32_t act, int32_t dt, int32_t odt, void* out) {
    return sv_linear(at<void>(0), at<void>(1), at<float>(2), at<float>(3), at<void>(4), at<void>(5), out, M, N, K, R, act,
                     dt, odt, nullptr);
  };
  void* lo = at<void>(6);
  CHECK(lin(big, big, 64, 1, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(small, 64, 64, 1, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, small, 64, 1, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, 64, small, 1, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, 64, big, 1, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, 64, 64, small, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, 64, 64, big, 0, SV_BF16, SV_F32, lo) == SV_ERR_SHAPE);
  CHECK(lin(1, 64, 64, 64, big, SV_BF16, SV_F32, lo) == SV_ERR_PARAM);
  CHECK(lin(1, 64, 64, 64, 0, SV_F32, SV_F32, lo) == SV_ERR_DTYPE);
  CHECK(lin(1 << 16, 1 << 20, 64, 64, 0, SV_E4M3, SV_F32, at<void>(0)) == SV_ERR_PARAM);
  CHECK(lin(0, 64, 64, 64, 0, SV_BF16, SV_F32, nullptr) == SV_OK);

  auto adj = [&](int32_t B, int32_t R, int32_t K, int32_t seen, int32_t cap, int32_t nb, int32_t mr, int32_t V, int32_t dt,
                 void* out) {
    return sv_adjust_logits(at<void>(0), out, at<int32_t>(2), at<int32_t>(3), at<int32_t>(4), at<int32_t>(5), at<float>(6),
                            at<float>(7), at<float>(8), at<int32_t>(9), at<int32_t>(10), at<float>(11), at<uint32_t>(12),
                            at<int32_t>(13), B, R, K, seen, cap, nb, mr, V, dt, nullptr);
  };
  void* ao = at<void>(1);
  CHECK(adj(big, big, 0, 0, 5, 4, 6, 100, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(big, 1, 0, 0, 5, 4, 6, SV_MAX_V, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(2, big, SV_MAX_K, big, 5, 4, 6, 100, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(2, 3, 2, 0, big, 4, 6, 100, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(2, 3, 2, 0, 5, small, 6, 100, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(2, 3, 2, 0, 5, 4, 6, big, SV_F32, ao) == SV_ERR_SHAPE);
  CHECK(adj(2, 3, 2, 0, 5, 4, 6, 100, big, ao) == SV_ERR_DTYPE);
  CHECK(adj(1 << 16, 9, 8, 0, SV_MAX_HISTORY, big, big, 1 << 17, SV_F32, at<void>(12)) == SV_ERR_PARAM);
  CHECK(adj(0, 3, 2, 0, 5, 4, 6, 100, SV_F32, nullptr) == SV_OK);
  auto rag = [&](int32_t B, int32_t N, int32_t max_k, int32_t bonus) {
    return sv_adjust_logits_ragged(at<void>(0), ao, at<int32_t>(2), at<int32_t>(3), at<int32_t>(4), at<int32_t>(5),
                                   at<int32_t>(14), at<float>(6), at<float>(7), at<float>(8), at<int32_t>(9),
                                   at<int32_t>(10), at<float>(11), at<uint32_t>(12), nullptr, B, N, max_k, bonus, 5, 4, 6,
                                   100, SV_F32, nullptr);
  };
  CHECK(rag(big, big, SV_MAX_K, 1) == SV_ERR_SHAPE);
  CHECK(rag(small, 0, 1, 1) == SV_ERR_SHAPE);
  CHECK(rag(3, big, SV_MAX_K, 1) == SV_ERR_SHAPE);
  CHECK(rag(3, 4, 2, small) == SV_ERR_PARAM);
  CHECK(rag(3, 4, 2, 1) == SV_ERR_SHAPE);  // 7 rows, 6 masks

  if (g_fail) return 1;
  std::printf("ok\n");
  return 0;
}
