// Rows of logits, 16 bytes a load, for the operators that take a row a workgroup
// (sv_top.hip, sv_distill.hip).
#pragma once

#include "sv_ops.hpp"

#include <cfloat>
#include <cmath>

namespace sv {

constexpr float LOG2E = 1.4426950408889634f;

// 16 bytes at any alignment of their elements, past the caches: nobody reads them
// before the row's end, and what is read a second time keeps its place there.
__device__ __forceinline__ void store_through(char* p, const uint32_t (&v)[4]) {
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(2)));
  const words w = {v[0], v[1], v[2], v[3]};
  __builtin_nontemporal_store(w, reinterpret_cast<words*>(p));
}

// E logits as they lie in memory.
template <int IN>
struct Run {
  static constexpr int E = IN == T_F32 ? 4 : 8, B = IN == T_F32 ? 4 : 2;
  static constexpr uint32_t NINF = IN == T_F32 ? 0xFF800000u : 0xFF80FF80u;
  uint32_t v[4];
  // the run that begins at column j >= 0 of a row of V >= E columns, whether it lies in the row or not
  __device__ __forceinline__ void load(const char* row, int j, int V) {
    __builtin_memcpy(v, row + (uint32_t)(min(j, V - E) * B), 16);  // a row is below 2^32 bytes
  }
  // a row of V < E columns (0: nothing)
  __device__ __forceinline__ void tiny(const char* row, int V) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = NINF;
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k < V) {
        const uint32_t u = __float_as_uint(load1<IN>(row, k));
        if (IN == T_F32)
          v[k] = u;
        else
          v[k / 2] = k & 1 ? (v[k / 2] & 0xFFFFu) | u : (v[k / 2] & 0xFFFF0000u) | (u >> 16);
      }
  }
  // takes what lies behind the row for -inf (after load)
  __device__ __forceinline__ void cut(int j, int V) {
    const int n = min(j - min(j, V - E), E) * B * 8;  // bits by which load began early
    uint64_t lo = ((uint64_t)(v[1] ^ NINF) << 32) | (v[0] ^ NINF), hi = ((uint64_t)(v[3] ^ NINF) << 32) | (v[2] ^ NINF);
    if (n >= 64) lo = hi, hi = 0;
    const int m = n & 63;
    if (n == 128) lo = 0;
    if (m) lo = (lo >> m) | (hi << (64 - m)), hi >>= m;
    v[0] = (uint32_t)lo ^ NINF, v[1] = (uint32_t)(lo >> 32) ^ NINF;
    v[2] = (uint32_t)hi ^ NINF, v[3] = (uint32_t)(hi >> 32) ^ NINF;
  }
  // something above -inf (or NaN) among the elements
  __device__ __forceinline__ bool any() const { return ((v[0] ^ NINF) | (v[1] ^ NINF) | (v[2] ^ NINF) | (v[3] ^ NINF)) != 0; }
  // element k to -inf for each bit k of mask
  __device__ __forceinline__ void drop(uint32_t mask) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (mask >> k & 1) {
        if (IN == T_F32)
          v[k] = NINF;
        else
          v[k / 2] = k & 1 ? (v[k / 2] & 0xFFFFu) | 0xFF800000u : (v[k / 2] & 0xFFFF0000u) | 0xFF80u;
      }
  }
  // as if loaded anew: what was formed from it before is formed again, not kept
  __device__ __forceinline__ void forget() { asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3])); }
  __device__ __forceinline__ float operator[](int k) const {
    return IN == T_F32 ? __uint_as_float(v[k]) : k & 1 ? bf16_hi(v[k / 2]) : bf16_lo(v[k / 2]);
  }
};

// A value that the compiler takes for a new one: what is formed from it is
// formed again, and not held in a register from one pass to the next.
__device__ __forceinline__ int fresh(int v) {
  asm("" : "+v"(v));
  return v;
}

// A sum of 2^(scale x - ref): one fused multiply-add and one exponential an
// element.  ref is not the maximum but a value that lies some powers of two below
// it (add: 8 at most, following the maximum in steps), which costs a float32 sum
// nothing.  It begins at LOW, up to whose magnitude half a step of a float32 is
// 64 at most, so that the exponential of a maximum's own rounding is finite.
// Values below LOW, as masks are, count as 0: a reference of their own would make
// their exponentials 0 or infinite, as the rounding falls, and then NaN of the
// ordinary ones' (448 x 128256 with the first half at -1e20: top_logits 221 us,
// 33 so; distill_loss 366, 74 so).  Where nothing lies above LOW, or scale x goes
// beyond its magnitude upwards, the sum comes out as 0, infinite or NaN, which its
// user has to look for.
struct RunSum {
  static constexpr float LOW = -0x1p31f;
  float ref = LOW, s = 0.0f;
  // formed by here: the compiler would put all of a row's sums behind the last of its loads (448 x 128256 bfloat16
  // without a gradient 42.9 us, 42.5 so)
  __device__ __forceinline__ void now() { asm volatile("" : "+v"(ref), "+v"(s)); }
  template <int IN>
  __device__ __forceinline__ float sum(const Run<IN>& r, float scale) const {
    constexpr int E = Run<IN>::E;
    float p[2];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(r[k], scale, -ref));
      p[k & 1] = k < 2 ? e : p[k & 1] + e;
    }
    return p[0] + p[1];
  }
  // mx: the running maximum (NaN apart)
  template <int IN>
  __device__ __forceinline__ void add(const Run<IN>& r, float scale, float& mx) {
    constexpr int E = Run<IN>::E;
#pragma unroll
    for (int k = 0; k < E; ++k) mx = fmaxf(mx, r[k]);
    const float y = mx * scale;
    if (__any(y > ref + 8.0f)) {  // few times a row
      const float n = y > ref + 8.0f ? y : ref;
      s *= __builtin_amdgcn_exp2f(ref - n);
      ref = n;
    }
    s += sum(r, scale);
  }
};

}  // namespace sv
