// Matrix product with its epilogue:
//   out[m, n] = act(sx[m] sw[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n mod R]
// on the matrix cores, for bfloat16 operands or e4m3 operands with a float32
// scale per row.  Products of two bfloat16 values are exact in float32 and are
// summed in float32 (v_mfma_f32_32x32x16_bf16); the epilogue is float32 too,
// rounded once.
//
// The 8-bit matrix instructions (v_mfma_f32_32x32x64_f8f6f4, twice the
// bfloat16 rate) keep their accumulators in float32 but form the sums of a
// few products with fewer bits: measured on normal values, 1.5e-5 of the
// result (2-norm), whatever the length of the sum and with every 8-bit form.
// That lies 100 times below the half step of a bfloat16 output (2^-9 of the
// value on average) and is used there; for a float32 output the operands are
// converted to bfloat16 (exactly: 4 significant bits) and multiplied as such,
// which measures 8e-8.
#include "sv_ops.hpp"
#include "specverify.h"

namespace sv {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;

enum Act : int { A_NONE = 0, A_RELU = 1, A_SILU = 2, A_GELU = 3, A_GELU_TANH = 4 };

struct LinArgs {
  const char* x;   // [M, K]
  const char* w;   // [N, K]
  const float* sx;  // [M], or null for bfloat16 operands
  const float* sw;  // [N]
  const void* bias;
  const void* res;  // [M, R]
  void* out;        // [M, N]
  int32_t M, N, K, R;
  int32_t act;
  int32_t mtiles, ntiles;
};

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case A_RELU: return v > 0.0f ? v : (v != v ? v : 0.0f);
    case A_SILU: return v / (1.0f + expf(-v));
    // forms without the cancellation of 1 + erf and 1 + tanh at negative v
    case A_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case A_GELU_TANH: return v / (1.0f + expf(-1.59576912160573071f * (v + 0.044715f * v * v * v)));
    default: return v;
  }
}

template <int OUT>
__device__ __forceinline__ float load_o(const void* p, size_t i) {
  if (OUT == T_F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// out[m, n] from its sum
template <int IN, int OUT>
__device__ __forceinline__ void put(const LinArgs& a, int m, int n, float v) {
  if (IN == T_E4M3) v = v * a.sx[m] * a.sw[n];
  if (a.bias) v += load_o<OUT>(a.bias, n);
  v = activate(v, a.act);
  if (a.res) v += load_o<OUT>(a.res, (size_t)m * a.R + n % a.R);
  const size_t at = (size_t)m * a.N + n;
  if (OUT == T_F32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<uint16_t*>(a.out)[at] = to_bf16(v);
}

// Eight e4m3 values as bfloat16 (exact).
__device__ __forceinline__ bf16x8 widen8(uint2 v) {
  bf16x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, false);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, true);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, false);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, true);
  return __builtin_bit_cast(bf16x8, p);
}

constexpr int LROW = 144;  // LDS bytes of a staged row: 128 of data, 16 of padding

// 64 x 64 tile, 4 waves of 32 x 32, k blocks of 128 bytes.
template <int IN, int OUT>
__global__ void __launch_bounds__(256) linear_kernel(LinArgs a) {
  __shared__ __attribute__((aligned(16))) char xs[64 * LROW];
  __shared__ __attribute__((aligned(16))) char ws[64 * LROW];
  const int nt = blockIdx.x / a.mtiles, mt = blockIdx.x - nt * a.mtiles;
  const int m0 = mt * 64, n0 = nt * 64;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, h = lane >> 5, l32 = lane & 31;
  const int kbytes = a.K * (IN == T_BF16 ? 2 : 1);
  f32x16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
  for (int k0 = 0; k0 < kbytes; k0 += 128) {
    const int nb = min(128, kbytes - k0);  // 128, or 64 in the last block of e4m3 operands
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 32 * i + (t >> 3), c = t & 7;
      if (16 * c < nb) {
        *reinterpret_cast<uint4*>(xs + r * LROW + 16 * c) =
            *reinterpret_cast<const uint4*>(a.x + (size_t)min(m0 + r, a.M - 1) * kbytes + k0 + 16 * c);
        *reinterpret_cast<uint4*>(ws + r * LROW + 16 * c) =
            *reinterpret_cast<const uint4*>(a.w + (size_t)min(n0 + r, a.N - 1) * kbytes + k0 + 16 * c);
      }
    }
    __syncthreads();
    const char* xa = xs + (32 * (w >> 1) + l32) * LROW;
    const char* wa = ws + (32 * (w & 1) + l32) * LROW;
    if (IN == T_BF16) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(xa + 32 * s + 16 * h),
                                                      *reinterpret_cast<const bf16x8*>(wa + 32 * s + 16 * h), acc, 0, 0, 0);
    } else if (OUT == T_F32) {
      for (int s = 0; s < nb / 16; ++s)
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8(*reinterpret_cast<const uint2*>(xa + 16 * s + 8 * h)),
                                                      widen8(*reinterpret_cast<const uint2*>(wa + 16 * s + 8 * h)), acc, 0, 0, 0);
    } else {
      for (int s = 0; s < nb / 64; ++s) {
        const i32x8 xf = *reinterpret_cast<const i32x8*>(xa + 64 * s + 32 * h);
        const i32x8 wf = *reinterpret_cast<const i32x8*>(wa + 64 * s + 32 * h);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xf, wf, acc, 0, 0, 0, 127, 0, 127);
      }
    }
    __syncthreads();
  }
  // lane (h, l32), accumulator r: row 8 (r / 4) + 4 h + r % 4, column l32
  const int n = n0 + 32 * (w & 1) + l32;
  if (n >= a.N) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int m = m0 + 32 * (w >> 1) + 8 * (r >> 2) + 4 * h + (r & 3);
    if (m < a.M) put<IN, OUT>(a, m, n, acc[r]);
  }
}

template <int IN, int OUT>
hipError_t launch_linear(LinArgs a, hipStream_t s) {
  a.mtiles = (a.M + 63) / 64;
  a.ntiles = (a.N + 63) / 64;
  hipLaunchKernelGGL((linear_kernel<IN, OUT>), dim3((unsigned)a.mtiles * (unsigned)a.ntiles), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_linear(const void* x, const void* weight, const float* x_scale, const float* weight_scale,
                         const void* bias, const void* residual, void* out, int32_t M, int32_t N, int32_t K,
                         int32_t residual_cols, int32_t activation, int32_t dtype, int32_t out_dtype, void* stream) {
  if (M < 0 || N < 1 || K < 64 || K > SV_MAX_LINEAR_K || K % 64 != 0) return SV_ERR_SHAPE;
  if (dtype != SV_BF16 && dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (out_dtype != SV_F32 && out_dtype != SV_BF16) return SV_ERR_DTYPE;
  if (activation < SV_ACT_NONE || activation > SV_ACT_GELU_TANH) return SV_ERR_PARAM;
  if (residual && (residual_cols < 1 || N % residual_cols != 0)) return SV_ERR_SHAPE;
  if ((((int64_t)M + 15) / 16) * (((int64_t)N + 15) / 16) * 64 > kGridThreads) return SV_ERR_SHAPE;
  if (M == 0) return SV_OK;
  const bool scaled = dtype == SV_E4M3;
  if (!x || !weight || !out || (scaled && (!x_scale || !weight_scale))) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), oe = (size_t)type_bytes(out_dtype);
  if (!is_aligned(x, 16) || !is_aligned(weight, 16) || !is_aligned(out, oe) || !is_aligned(bias, oe) ||
      !is_aligned(residual, oe) || (scaled && (!is_aligned(x_scale, 4) || !is_aligned(weight_scale, 4))))
    return SV_ERR_SHAPE;
  const size_t no = (size_t)M * (size_t)N * oe;
  const size_t nr = residual ? (size_t)M * (size_t)residual_cols * oe : 0;
  if (overlaps(out, no, x, (size_t)M * K * ie) || overlaps(out, no, weight, (size_t)N * K * ie) ||
      overlaps(out, no, bias, (size_t)N * oe) ||
      (scaled && (overlaps(out, no, x_scale, (size_t)M * 4) || overlaps(out, no, weight_scale, (size_t)N * 4))) ||
      (overlaps(out, no, residual, nr) && !(out == residual && residual_cols == N)))
    return SV_ERR_PARAM;
  LinArgs a;
  a.x = static_cast<const char*>(x);
  a.w = static_cast<const char*>(weight);
  a.sx = scaled ? x_scale : nullptr;
  a.sw = scaled ? weight_scale : nullptr;
  a.bias = bias;
  a.res = residual;
  a.out = out;
  a.M = M;
  a.N = N;
  a.K = K;
  a.R = residual ? residual_cols : 1;
  a.act = activation;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == SV_BF16
                           ? (out_dtype == SV_F32 ? launch_linear<T_BF16, T_F32>(a, s) : launch_linear<T_BF16, T_BF16>(a, s))
                           : (out_dtype == SV_F32 ? launch_linear<T_E4M3, T_F32>(a, s) : launch_linear<T_E4M3, T_BF16>(a, s));
  return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}
