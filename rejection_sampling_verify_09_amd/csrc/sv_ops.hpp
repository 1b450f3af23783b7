// Shared by the operators around a model's last layer (sv_norm.hip,
// sv_layer_norm.hip, sv_linear.hip, sv_adjust.hip, sv_top.hip,
// sv_distill.hip): host-side argument helpers, conversions between float32 and
// the storage types, and runs of elements in registers.
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

// Over the 16 lanes that hold a value for each of up to 16 waves.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp_mov<DPP_QP_1032>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mov<DPP_QP_2301>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mov<DPP_HALF_MIRROR>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_mov<DPP_MIRROR>(__float_as_uint(v))));
  return v;
}

__device__ __forceinline__ float row16_sum(float v) {
  v += __uint_as_float(dpp_mov<DPP_QP_1032>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<DPP_QP_2301>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<DPP_HALF_MIRROR>(__float_as_uint(v)));
  v += __uint_as_float(dpp_mov<DPP_MIRROR>(__float_as_uint(v)));
  return v;
}

// Element j of a row.
template <int T>
__device__ __forceinline__ float load1(const char* p, int j) {
  if (T == T_F32) return reinterpret_cast<const float*>(p)[j];
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[j] << 16);
}
template <int T>
__device__ __forceinline__ void store1(char* p, int j, float v) {
  if (T == T_F32)
    reinterpret_cast<float*>(p)[j] = v;
  else
    reinterpret_cast<uint16_t*>(p)[j] = to_bf16(v);
}

// Eight elements at p as floats, n of them (the others 0) where n < 8.  AL: p
// is 16-byte aligned; otherwise aligned to the element (the loads and stores
// are the same 16-byte ones, which the hardware splits where they cross).
template <int T, bool AL>
__device__ __forceinline__ void load8(const char* p, float (&f)[8], int n) {
  if (AL || n >= 8) {
    uint4 a, b;
    __builtin_memcpy(&a, AL ? __builtin_assume_aligned(p, 16) : p, 16);
    if (T == T_F32) {
      __builtin_memcpy(&b, AL ? __builtin_assume_aligned(p + 16, 16) : p + 16, 16);
      f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    } else {
      f[0] = bf16_lo(a.x), f[1] = bf16_hi(a.x), f[2] = bf16_lo(a.y), f[3] = bf16_hi(a.y);
      f[4] = bf16_lo(a.z), f[5] = bf16_hi(a.z), f[6] = bf16_lo(a.w), f[7] = bf16_hi(a.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = 0.0f;
      if (k < n)
        f[k] = T == T_F32 ? reinterpret_cast<const float*>(p)[k]
                          : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << 16);
    }
  }
}
template <int T, bool AL>
__device__ __forceinline__ void store8(char* p, const float (&f)[8], int n) {
  if (AL || n >= 8) {
    if (T == T_F32) {
      const float4 a = make_float4(f[0], f[1], f[2], f[3]), b = make_float4(f[4], f[5], f[6], f[7]);
      __builtin_memcpy(AL ? __builtin_assume_aligned(p, 16) : p, &a, 16);
      __builtin_memcpy(AL ? __builtin_assume_aligned(p + 16, 16) : p + 16, &b, 16);
    } else if (T == T_BF16) {
      const uint4 a = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
      __builtin_memcpy(AL ? __builtin_assume_aligned(p, 16) : p, &a, 16);
    } else {
      const uint2 a = make_uint2(pack_e4m3(f[0], f[1], f[2], f[3]), pack_e4m3(f[4], f[5], f[6], f[7]));
      __builtin_memcpy(AL ? __builtin_assume_aligned(p, 8) : p, &a, 8);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= n) continue;
      if (T == T_F32) reinterpret_cast<float*>(p)[k] = f[k];
      if (T == T_BF16) reinterpret_cast<uint16_t*>(p)[k] = to_bf16(f[k]);
      if (T == T_E4M3) reinterpret_cast<uint8_t*>(p)[k] = (uint8_t)pack_e4m3(f[k], f[k], f[k], f[k]);
    }
  }
}

}  // namespace sv
