// Root-mean-square norm with the residual's addition:
//   h = x + residual,  y_j = h_j w_j / sqrt(mean_j h_j^2 + eps)
// in float32, y rounded once to the output type; in 8 bits (e4m3) each row has
// its scale, max(max_j |y_j| / 448, FLT_MIN), and y_j / scale is stored.
//
// Memory bound: each element is read once (with its residual) and written
// once (with the new residual).  A row stays in registers between the sum of
// squares and the output, so nothing is read twice, whatever its width.
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* out;
  float* scale;
  void* out_res;
  int32_t rows, d;
  float eps;
};

constexpr int NORM_WG = 256;

__device__ __forceinline__ float block_sum(float v, float* part) {
  v = dpp_wave_fsum(v);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[w] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < (int)(blockDim.x >> 6); ++i) s += part[i];
  return s;
}
__device__ __forceinline__ float block_max(float v, float* part) {
  v = wave_fmax(v);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[w] = v;
  __syncthreads();
  float s = part[0];
  for (int i = 1; i < (int)(blockDim.x >> 6); ++i) s = fmaxf(s, part[i]);
  return s;
}

template <int T>
__device__ __forceinline__ float load_t(const void* p, size_t i) {
  if (T == T_F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}
template <int T>
__device__ __forceinline__ void store_t(void* p, size_t i, float v) {
  if (T == T_F32) static_cast<float*>(p)[i] = v;
  if (T == T_BF16) static_cast<uint16_t*>(p)[i] = to_bf16(v);
  if (T == T_E4M3) static_cast<uint8_t*>(p)[i] = (uint8_t)pack_e4m3(v, v, v, v);
}

// One workgroup per row, EPT elements a thread.
template <int IN, int OUT, int EPT>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormArgs a) {
  __shared__ float part[16];
  const int t = threadIdx.x, nt = blockDim.x;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.d;
    float h[EPT];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int j = t + i * nt;
      h[i] = 0.0f;
      if (j < a.d) {
        h[i] = load_t<IN>(a.x, base + j);
        if (a.res) h[i] += load_t<IN>(a.res, base + j);
      }
      ss += h[i] * h[i];
    }
    // a row whose sum is not finite comes out all NaN instead of as zeros
    const float ms = block_sum(ss, part) / (float)a.d + a.eps;
    const float r = ms < INFINITY ? rsqrtf(ms) : NAN;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int j = t + i * nt;
      if (j < a.d) {
        if (a.out_res) store_t<IN>(a.out_res, base + j, h[i]);
        h[i] = h[i] * r * load_t<IN>(a.w, j);
        if (OUT != T_E4M3) store_t<OUT>(a.out, base + j, h[i]);
        m = fmaxf(m, fabsf(h[i]));
      }
    }
    if (OUT == T_E4M3) {
      const float sc = r != r ? r : fmaxf(block_max(m, part) / 448.0f, FLT_MIN);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int j = t + i * nt;
        if (j < a.d) store_t<OUT>(a.out, base + j, h[i] / sc);
      }
      if (t == 0) a.scale[row] = sc;
    }
  }
}

template <int IN, int OUT>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)std::min(a.rows, 1 << 20);
  const int nt = a.d <= 16 * NORM_WG ? NORM_WG : 1024;
  const int ept = (a.d + nt - 1) / nt;
  if (ept <= 16)
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 16>), dim3(grid), dim3(nt), 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 64>), dim3(grid), dim3(nt), 0, s, a);
  return hipGetLastError();
}

template <int IN>
hipError_t launch_norm_out(const NormArgs& a, int out, hipStream_t s) {
  return out == T_F32 ? launch_norm<IN, T_F32>(a, s)
                      : out == T_BF16 ? launch_norm<IN, T_BF16>(a, s) : launch_norm<IN, T_E4M3>(a, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_rms_norm(const void* x, const void* residual, const void* weight, float eps, void* out,
                           float* out_scale, void* out_residual, int32_t rows, int32_t d, int32_t dtype,
                           int32_t out_dtype, void* stream) {
  if (rows < 0 || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (out_dtype != SV_F32 && out_dtype != SV_BF16 && out_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return SV_ERR_PARAM;
  if (rows == 0) return SV_OK;
  if (!x || !weight || !out || (out_dtype == SV_E4M3 && !out_scale) || (out_residual && !residual)) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), n = (size_t)rows * (size_t)d;
  const size_t nin = n * ie, nout = n * (size_t)type_bytes(out_dtype), nw = (size_t)d * ie;
  const size_t nsc = out_dtype == SV_E4M3 ? (size_t)rows * 4 : 0;
  if (!is_aligned(x, ie) || !is_aligned(residual, ie) || !is_aligned(weight, ie) || !is_aligned(out_residual, ie) ||
      !is_aligned(out, (size_t)type_bytes(out_dtype)) || (nsc && !is_aligned(out_scale, 4)))
    return SV_ERR_SHAPE;
  // an output may be an input of its own type, element for element; any other overlap is refused
  const bool same = dtype == out_dtype;
  if ((overlaps(out, nout, x, nin) && !(same && out == x)) ||
      (overlaps(out, nout, residual, nin) && !(same && out == residual)) ||
      (overlaps(out_residual, nin, x, nin) && out_residual != x) ||
      (overlaps(out_residual, nin, residual, nin) && out_residual != residual) ||
      overlaps(out, nout, out_residual, nin) || overlaps(out, nout, weight, nw) ||
      overlaps(out_residual, nin, weight, nw) || overlaps(out_scale, nsc, x, nin) ||
      overlaps(out_scale, nsc, residual, nin) || overlaps(out_scale, nsc, weight, nw) ||
      overlaps(out_scale, nsc, out, nout) || overlaps(out_scale, nsc, out_residual, nin))
    return SV_ERR_PARAM;
  NormArgs a;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.out = out;
  a.scale = out_scale;
  a.out_res = out_residual;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  const hipError_t e = dtype == SV_F32 ? launch_norm_out<T_F32>(a, out_dtype, (hipStream_t)stream)
                                       : launch_norm_out<T_BF16>(a, out_dtype, (hipStream_t)stream);
  return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}
