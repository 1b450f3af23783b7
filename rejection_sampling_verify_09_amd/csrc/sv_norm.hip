// Root-mean-square norm with the residual's addition:
//   h = x + residual,  y_j = h_j w_j / sqrt(mean_j h_j^2 + eps)
// in float32, y rounded once to the output type; in 8 bits (e4m3) each row has
// its scale, max(max_j |y_j| / 448, FLT_MIN), and y_j / scale is stored.
//
// Bound by memory: each element is read once (with its residual) and written
// once (with the new residual).  A row stays in registers between the sum of
// squares and the output, so nothing is read twice, whatever its width: 16384
// x 8192 bfloat16 rows with a residual take 177 us (6.1 TB/s; a large copy
// reaches 5.1), 8193 columns, whose rows start at any 2 bytes, 248 us (an
// element a load took 679).  Up to about 2000 rows of 4096 the launch is what
// counts.
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

// VPT runs of 8 elements a thread.  blockDim.x threads take a row (whole
// waves) and blockDim.y rows share a workgroup (only rows of one wave, which
// then need no barrier).  AL: 16-byte aligned rows of a multiple of 8.
template <int IN, int OUT, int VPT, bool AL>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormArgs a) {
  __shared__ float part[2][16];
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;  // blockDim.y > 1: no barrier follows
  constexpr int IB = IN == T_F32 ? 4 : 2, OB = OUT == T_F32 ? 4 : OUT == T_BF16 ? 2 : 1;
  const size_t base = (size_t)row * a.d;
  const char* x = static_cast<const char*>(a.x) + base * IB;
  const char* res = static_cast<const char*>(a.res) + base * IB;
  float h[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = 0.0f;
    if (j < a.d) load8<IN, AL>(x + (size_t)j * IB, h[i], a.d - j);
  }
  if (a.res) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int j = (t + i * nt) * 8;
      if (j < a.d) {
        float r[8];
        load8<IN, AL>(res + (size_t)j * IB, r, a.d - j);
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] += r[k];
      }
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += h[i][k] * h[i][k];
  ss = dpp_wave_fsum(ss);
  if (nw > 1) {
    if ((t & 63) == 0) part[0][t >> 6] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < nw; ++i) ss += part[0][i];
  }
  // a row whose sum is not finite comes out all NaN instead of as zeros
  const float ms = ss / (float)a.d + a.eps;
  const float r = ms < INFINITY ? rsqrtf(ms) : NAN;
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
    if (j < a.d) {
      if (a.out_res) store8<IN, AL>(static_cast<char*>(a.out_res) + (base + j) * IB, h[i], a.d - j);
      float w[8];
      load8<IN, AL>(static_cast<const char*>(a.w) + (size_t)j * IB, w, a.d - j);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] = h[i][k] * r * w[k];
        m = fmaxf(m, fabsf(h[i][k]));
      }
      if (OUT != T_E4M3) store8<OUT, AL>(static_cast<char*>(a.out) + (base + j) * OB, h[i], a.d - j);
    }
  }
  if (OUT == T_E4M3) {
    m = dpp_wave_fmax(m);
    if (nw > 1) {
      if ((t & 63) == 0) part[1][t >> 6] = m;
      __syncthreads();
      m = part[1][0];
      for (int i = 1; i < nw; ++i) m = fmaxf(m, part[1][i]);
    }
    const float sc = r != r ? r : fmaxf(m / 448.0f, FLT_MIN);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int j = (t + i * nt) * 8;
      if (j < a.d) {
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] /= sc;  // a product with 1 / sc rounds once more, and moves values across ties
        store8<OUT, AL>(static_cast<char*>(a.out) + base + j, h[i], a.d - j);
      }
    }
    if (t == 0) a.scale[row] = sc;
  }
}

// As many threads a row as it has runs of 8, up to 1024: on 16384 x 8192
// bfloat16 rows with a residual 1, 2, 4 and 8 runs a thread take 179, 183, 195
// and 212 us (the wider a workgroup, the sooner a row's loads are all in
// flight); rows up to 4096 do not tell them apart.  The rows of one wave go
// four to a workgroup.
struct NormLaunch {
  int nt, ny, vpt;  // threads a row, rows a workgroup, runs a thread
  int64_t wgs;
  NormLaunch(int64_t rows, int d) {
    const int nv = (d + 7) / 8;
    nt = std::min(1024, (nv + 63) / 64 * 64);
    ny = nt == 64 ? 4 : 1;
    vpt = (nv + nt - 1) / nt;
    wgs = (rows + ny - 1) / ny;
  }
};

template <int IN, int OUT, bool AL>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const NormLaunch l(a.rows, a.d);
  const int vpt = l.vpt;
  const dim3 grid((unsigned)l.wgs), wg((unsigned)l.nt, (unsigned)l.ny);
  if (vpt == 1)
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 1, AL>), grid, wg, 0, s, a);
  else if (vpt == 2)
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 2, AL>), grid, wg, 0, s, a);
  else if (vpt <= 4)
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 4, AL>), grid, wg, 0, s, a);
  else
    hipLaunchKernelGGL((rms_norm_kernel<IN, OUT, 8, AL>), grid, wg, 0, s, a);
  return hipGetLastError();
}

template <int IN, int OUT>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  const bool al = a.d % 8 == 0 && is_aligned(a.x, 16) && is_aligned(a.res, 16) && is_aligned(a.w, 16) &&
                  is_aligned(a.out, OUT == T_E4M3 ? 8 : 16) && is_aligned(a.out_res, 16);
  return al ? launch_norm<IN, OUT, true>(a, s) : launch_norm<IN, OUT, false>(a, s);
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
  const NormLaunch l(rows, d);
  if (l.wgs * l.nt * l.ny > kGridThreads) return SV_ERR_SHAPE;
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
