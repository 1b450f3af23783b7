// Shared by the operators between a model's last layer and the verification
// (sv_norm.hip, sv_linear.hip, sv_adjust.hip): host-side argument helpers and
// conversions between float32 and the storage types.
#pragma once

#include "sv_common.hpp"

#include <cstddef>
#include <cstdint>

namespace sv {

enum OpType : int { T_F32 = 0, T_BF16 = 1, T_E4M3 = 2 };  // sv_dtype

// A launch must satisfy grid * threads < 2^32.
constexpr int64_t kGridThreads = (int64_t(1) << 32) - 1;

inline int type_bytes(int t) { return t == T_F32 ? 4 : t == T_BF16 ? 2 : 1; }
inline bool is_aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte (never for a NULL pointer
// or an empty range).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x && y && na && nb && x < y + nb && y < x + na;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two floats rounded to bfloat16 (nearest, ties to even; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float a) { return (uint16_t)pack_bf16(a, 0.0f); }

// Four floats rounded to e4m3 (nearest, ties to even), clamped to the largest
// magnitude 448 first (the conversion makes values past it NaN); NaN stays NaN.
__device__ __forceinline__ float clamp_e4m3(float v) {
  const float c = fminf(fmaxf(v, -448.0f), 448.0f);
  return v != v ? v : c;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(a), clamp_e4m3(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(c), clamp_e4m3(d), w, true);
}

}  // namespace sv
