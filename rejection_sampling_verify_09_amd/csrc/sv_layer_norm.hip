// Layer norm with the residual's addition, and the gradients of layer norm and
// of the root-mean-square norm.
//
// Forward, of a row h = x + residual:
//   y_j = (h_j - mean h) / sqrt(mean (h - mean h)^2 + eps) * w_j + b_j
// Backward, of a row h with the gradient dy, g_j = dy_j w_j and
// n_j = (h_j - mean h) r (layer norm) or h_j r (root mean square), r the
// reciprocal root above:
//   dh_j = r (g_j - [mean g] - n_j mean(g n)) + dres_j
//   dw_j = sum over rows dy_j n_j,  db_j = sum over rows dy_j
// ([mean g]: layer norm only).  The row's statistics are formed again from h:
// the row has to be read in any case, and nothing else is kept from the
// forward pass.
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

struct LayerArgs {
  const void* x;
  const void* res;
  const void* w;
  const void* b;
  void* out;
  float* scale;
  void* out_res;
  int32_t rows, d;
  float eps;
};

// Sums of A values over the workgroup's nw waves, in a fixed order; part:
// [A * 16] floats that nothing else uses until the next barrier but one.
template <int A>
__device__ __forceinline__ void group_sum(float (&v)[A], float* part, int nw) {
#pragma unroll
  for (int i = 0; i < A; ++i) v[i] = dpp_wave_fsum(v[i]);
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < A; ++i) part[i * 16 + (threadIdx.x >> 6)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < A; ++i) {
    v[i] = 0.0f;
    for (int k = 0; k < nw; ++k) v[i] += part[i * 16 + k];
  }
}

// VPT runs of 8 elements a thread.  blockDim.x threads take a row (whole
// waves) and blockDim.y rows share a workgroup (only rows of one wave, which
// then need no barrier).  AL: 16-byte aligned rows of a multiple of 8.
//
// The mean is taken off in registers, and the mean of what is left once more
// with the sum of its squares: a row whose values are far from 0 and close to
// each other keeps the bits of their differences.
template <int IN, int OUT, int VPT, bool AL>
__global__ void __launch_bounds__(1024) layer_norm_kernel(LayerArgs a) {
  __shared__ float part[4][16];
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
  const float n = (float)a.d;
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[0] += h[i][k];
  group_sum(sum, part[0], nw);
  const float mean = sum[0] / n;
  float mom[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
    if (a.out_res && j < a.d) store8<IN, AL>(static_cast<char*>(a.out_res) + (base + j) * IB, h[i], a.d - j);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[i][k] = (AL ? j < a.d : j + k < a.d) ? h[i][k] - mean : 0.0f;
      mom[0] += h[i][k];
      mom[1] += h[i][k] * h[i][k];
    }
  }
  group_sum(mom, part[1], nw);
  const float left = mom[0] / n;
  // a row whose sum is not finite comes out all NaN instead of as zeros
  const float var = fmaxf(mom[1] / n - left * left, 0.0f) + a.eps;
  const float r = mom[1] < INFINITY && var < INFINITY ? rsqrtf(var) : NAN;
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
    if (j < a.d) {
      float w[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.0f, b[k] = 0.0f;
      if (a.w) load8<IN, AL>(static_cast<const char*>(a.w) + (size_t)j * IB, w, a.d - j);
      if (a.b) load8<IN, AL>(static_cast<const char*>(a.b) + (size_t)j * IB, b, a.d - j);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[i][k] = (h[i][k] - left) * r * w[k] + b[k];
        if (AL || j + k < a.d) m = fmaxf(m, fabsf(h[i][k]));
      }
      if (OUT != T_E4M3) store8<OUT, AL>(static_cast<char*>(a.out) + (base + j) * OB, h[i], a.d - j);
    }
  }
  if (OUT == T_E4M3) {
    m = dpp_wave_fmax(m);
    if (nw > 1) {
      if ((t & 63) == 0) part[3][t >> 6] = m;
      __syncthreads();
      m = part[3][0];
      for (int i = 1; i < nw; ++i) m = fmaxf(m, part[3][i]);
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

// As many threads a row as it has runs of 8, up to 1024; the rows of one wave
// go four to a workgroup.
struct LayerLaunch {
  int nt, ny, vpt;  // threads a row, rows a workgroup, runs a thread
  int64_t wgs;
  LayerLaunch(int64_t rows, int d) {
    const int nv = (d + 7) / 8;
    nt = std::min(1024, (nv + 63) / 64 * 64);
    ny = nt == 64 ? 4 : 1;
    vpt = (nv + nt - 1) / nt;
    wgs = (rows + ny - 1) / ny;
  }
};

template <int IN, int OUT, bool AL>
hipError_t launch_layer(const LayerArgs& a, hipStream_t s) {
  const LayerLaunch l(a.rows, a.d);
  const dim3 grid((unsigned)l.wgs), wg((unsigned)l.nt, (unsigned)l.ny);
  if (l.vpt == 1)
    hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, 1, AL>), grid, wg, 0, s, a);
  else if (l.vpt == 2)
    hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, 2, AL>), grid, wg, 0, s, a);
  else if (l.vpt <= 4)
    hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, 4, AL>), grid, wg, 0, s, a);
  else
    hipLaunchKernelGGL((layer_norm_kernel<IN, OUT, 8, AL>), grid, wg, 0, s, a);
  return hipGetLastError();
}

template <int IN, int OUT>
hipError_t launch_layer(const LayerArgs& a, hipStream_t s) {
  const bool al = a.d % 8 == 0 && is_aligned(a.x, 16) && is_aligned(a.res, 16) && is_aligned(a.w, 16) &&
                  is_aligned(a.b, 16) && is_aligned(a.out, OUT == T_E4M3 ? 8 : 16) && is_aligned(a.out_res, 16);
  return al ? launch_layer<IN, OUT, true>(a, s) : launch_layer<IN, OUT, false>(a, s);
}

template <int IN>
hipError_t launch_layer_out(const LayerArgs& a, int out, hipStream_t s) {
  return out == T_F32 ? launch_layer<IN, T_F32>(a, s)
                      : out == T_BF16 ? launch_layer<IN, T_BF16>(a, s) : launch_layer<IN, T_E4M3>(a, s);
}

// ------------------------------------------------------------- the gradients

struct BackArgs {
  const void* dy;
  const void* h;
  const void* w;
  const void* dres;
  void* dh;
  float* dw;  // [groups][d] sums over each workgroup's rows, or NULL
  float* db;
  int32_t rows, d;
  float eps;
};

// A workgroup takes rows blockIdx.x, blockIdx.x + gridDim.x, ..; its sums for
// the weights stand in its own part of the workspace.
template <int IN, bool CENTER>
__global__ void __launch_bounds__(1024) norm_backward_kernel(BackArgs a) {
  __shared__ float part[2][5][16];
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6;
  constexpr int IB = IN == T_F32 ? 4 : 2;
  const float n = (float)a.d;
  float* dw = a.dw ? a.dw + (size_t)blockIdx.x * a.d : nullptr;
  float* db = a.db ? a.db + (size_t)blockIdx.x * a.d : nullptr;
  int turn = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const size_t base = (size_t)row * a.d;
    const char* hp = static_cast<const char*>(a.h) + base * IB;
    const char* dyp = static_cast<const char*>(a.dy) + base * IB;
    float mean = 0.0f;
    if (CENTER) {
      float sum[1] = {0.0f};
      for (int j = t; j < a.d; j += nt) sum[0] += load1<IN>(hp, j);
      group_sum(sum, part[turn][0], nw);
      mean = sum[0] / n;
    }
    // sums of c, c^2, g and g c for c = h - mean
    float mom[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = t; j < a.d; j += nt) {
      const float c = load1<IN>(hp, j) - mean;
      const float g = load1<IN>(dyp, j) * (a.w ? load1<IN>(static_cast<const char*>(a.w), j) : 1.0f);
      mom[0] += c;
      mom[1] += c * c;
      mom[2] += g;
      mom[3] += g * c;
    }
    group_sum(mom, part[turn][1], nw);
    const float left = CENTER ? mom[0] / n : 0.0f;
    const float var = fmaxf(mom[1] / n - left * left, 0.0f) + a.eps;
    const float r = mom[1] < INFINITY && var < INFINITY ? rsqrtf(var) : NAN;
    const float gm = CENTER ? mom[2] / n : 0.0f;
    const float gn = (mom[3] / n - left * (mom[2] / n)) * r;
    for (int j = t; j < a.d; j += nt) {
      const float v = (load1<IN>(hp, j) - mean - left) * r;
      const float dy = load1<IN>(dyp, j);
      const float g = dy * (a.w ? load1<IN>(static_cast<const char*>(a.w), j) : 1.0f);
      float dh = r * (g - gm - v * gn);
      if (a.dres) dh += load1<IN>(static_cast<const char*>(a.dres) + base * IB, j);
      store1<IN>(static_cast<char*>(a.dh) + base * IB, j, dh);
      if (dw) dw[j] = (row < (int)gridDim.x ? 0.0f : dw[j]) + dy * v;
      if (db) db[j] = (row < (int)gridDim.x ? 0.0f : db[j]) + dy;
    }
  }
}

// Column sums of the workgroups' parts, in their order.
__global__ void __launch_bounds__(256) norm_backward_sum_kernel(const float* wp, const float* bp, float* dw, float* db,
                                                                int groups, int d) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= d) return;
  if (dw) {
    float s = 0.0f;
    for (int g = 0; g < groups; ++g) s += wp[(size_t)g * d + j];
    dw[j] = s;
  }
  if (db) {
    float s = 0.0f;
    for (int g = 0; g < groups; ++g) s += bp[(size_t)g * d + j];
    db[j] = s;
  }
}

// Workgroups of the backward pass: what the workspace holds a part for.
int back_groups(int rows) { return std::min(rows, 512); }

int norm_backward(bool center, const void* grad, const void* h, const void* weight, const void* grad_residual, float eps,
                  void* grad_h, float* grad_weight, float* grad_bias, void* workspace, int64_t workspace_bytes,
                  int32_t rows, int32_t d, int32_t dtype, hipStream_t s) {
  if (rows < 0 || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return SV_ERR_PARAM;
  const int groups = back_groups(rows);
  const size_t ie = (size_t)type_bytes(dtype), nin = (size_t)rows * (size_t)d * ie, nw = (size_t)d * ie;
  const size_t np = (size_t)d * 4, one = (size_t)groups * np;
  const size_t ws = groups > 1 ? one * ((grad_weight ? 1 : 0) + (grad_bias ? 1 : 0)) : 0;
  if (rows > 0 && (!grad || !h || !grad_h)) return SV_ERR_NULL;
  if (ws && !workspace) return SV_ERR_NULL;
  if (ws && workspace_bytes < (int64_t)ws) return SV_ERR_WORKSPACE;
  if (!is_aligned(grad, ie) || !is_aligned(h, ie) || !is_aligned(weight, ie) || !is_aligned(grad_residual, ie) ||
      !is_aligned(grad_h, ie) || !is_aligned(grad_weight, 4) || !is_aligned(grad_bias, 4) ||
      (ws && !is_aligned(workspace, 16)))
    return SV_ERR_SHAPE;
  // grad_h may be an input of its shape, element for element; any other overlap of what is written is refused
  struct Range {
    const void* p;
    size_t n;
  };
  const Range in[] = {{grad, nin}, {h, nin}, {grad_residual, nin}, {weight, nw}};
  const Range out[] = {{grad_h, nin}, {grad_weight, np}, {grad_bias, np}, {workspace, ws}};
  for (int i = 0; i < 4; ++i) {
    for (int k = 0; k < 4; ++k)
      if (overlaps(out[i].p, out[i].n, in[k].p, in[k].n) && !(i == 0 && k < 3 && in[k].p == grad_h)) return SV_ERR_PARAM;
    for (int k = 0; k < i; ++k)
      if (overlaps(out[i].p, out[i].n, out[k].p, out[k].n)) return SV_ERR_PARAM;
  }
  BackArgs a;
  a.dy = grad;
  a.h = h;
  a.w = weight;
  a.dres = grad_residual;
  a.dh = grad_h;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  char* part = static_cast<char*>(workspace);
  a.dw = !grad_weight ? nullptr : groups > 1 ? reinterpret_cast<float*>(part) : grad_weight;
  a.db = !grad_bias ? nullptr : groups > 1 ? reinterpret_cast<float*>(part + (grad_weight ? one : 0)) : grad_bias;
  if (rows > 0) {
    const dim3 grid((unsigned)groups), wg((unsigned)std::min(1024, (d + 63) / 64 * 64));
    if (center) {
      if (dtype == SV_F32)
        hipLaunchKernelGGL((norm_backward_kernel<T_F32, true>), grid, wg, 0, s, a);
      else
        hipLaunchKernelGGL((norm_backward_kernel<T_BF16, true>), grid, wg, 0, s, a);
    } else {
      if (dtype == SV_F32)
        hipLaunchKernelGGL((norm_backward_kernel<T_F32, false>), grid, wg, 0, s, a);
      else
        hipLaunchKernelGGL((norm_backward_kernel<T_BF16, false>), grid, wg, 0, s, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return SV_ERR_HIP;
  }
  if (groups != 1 && (grad_weight || grad_bias)) {
    hipLaunchKernelGGL(norm_backward_sum_kernel, dim3((unsigned)((d + 255) / 256)), dim3(256), 0, s, a.dw, a.db,
                       grad_weight, grad_bias, groups, d);
    if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  }
  return SV_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_layer_norm(const void* x, const void* residual, const void* weight, const void* bias, float eps,
                             void* out, float* out_scale, void* out_residual, int32_t rows, int32_t d, int32_t dtype,
                             int32_t out_dtype, void* stream) {
  if (rows < 0 || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (out_dtype != SV_F32 && out_dtype != SV_BF16 && out_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return SV_ERR_PARAM;
  const LayerLaunch l(rows, d);
  if (l.wgs * l.nt * l.ny > kGridThreads) return SV_ERR_SHAPE;
  if (rows == 0) return SV_OK;
  if (!x || !out || (out_dtype == SV_E4M3 && !out_scale) || (out_residual && !residual)) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), oe = (size_t)type_bytes(out_dtype);
  const size_t n = (size_t)rows * (size_t)d, nin = n * ie, nw = (size_t)d * ie;
  const size_t nsc = out_dtype == SV_E4M3 ? (size_t)rows * 4 : 0;
  if (!is_aligned(x, ie) || !is_aligned(residual, ie) || !is_aligned(weight, ie) || !is_aligned(bias, ie) ||
      !is_aligned(out_residual, ie) || !is_aligned(out, oe) || (nsc && !is_aligned(out_scale, 4)))
    return SV_ERR_SHAPE;
  // an output may be an input of its own type, element for element; any other overlap is refused
  const bool same = dtype == out_dtype;
  struct Range {
    const void* p;
    size_t n;
    bool type;  // of the inputs' type
  };
  const Range in[] = {{x, nin, true}, {residual, nin, true}, {weight, nw, false}, {bias, nw, false}};
  const Range outs[] = {{out, n * oe, same}, {out_residual, nin, true}, {out_scale, nsc, false}};
  for (int i = 0; i < 3; ++i) {
    for (int k = 0; k < 4; ++k)
      if (overlaps(outs[i].p, outs[i].n, in[k].p, in[k].n) && !(outs[i].type && in[k].type && outs[i].p == in[k].p))
        return SV_ERR_PARAM;
    for (int k = 0; k < i; ++k)
      if (overlaps(outs[i].p, outs[i].n, outs[k].p, outs[k].n)) return SV_ERR_PARAM;
  }
  LayerArgs a;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.b = bias;
  a.out = out;
  a.scale = out_scale;
  a.out_res = out_residual;
  a.rows = rows;
  a.d = d;
  a.eps = eps;
  const hipError_t e = dtype == SV_F32 ? launch_layer_out<T_F32>(a, out_dtype, (hipStream_t)stream)
                                       : launch_layer_out<T_BF16>(a, out_dtype, (hipStream_t)stream);
  return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int64_t sv_norm_backward_workspace(int32_t rows, int32_t d) {
  if (rows < 0 || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  const int groups = back_groups(rows);
  return groups > 1 ? (int64_t)groups * d * 8 : 0;
}

extern "C" int sv_layer_norm_backward(const void* grad, const void* h, const void* weight, const void* grad_residual,
                                      float eps, void* grad_h, float* grad_weight, float* grad_bias, void* workspace,
                                      int64_t workspace_bytes, int32_t rows, int32_t d, int32_t dtype, void* stream) {
  return norm_backward(true, grad, h, weight, grad_residual, eps, grad_h, grad_weight, grad_bias, workspace,
                       workspace_bytes, rows, d, dtype, (hipStream_t)stream);
}

extern "C" int sv_rms_norm_backward(const void* grad, const void* h, const void* weight, const void* grad_residual,
                                    float eps, void* grad_h, float* grad_weight, void* workspace,
                                    int64_t workspace_bytes, int32_t rows, int32_t d, int32_t dtype, void* stream) {
  return norm_backward(false, grad, h, weight, grad_residual, eps, grad_h, grad_weight, nullptr, workspace,
                       workspace_bytes, rows, d, dtype, (hipStream_t)stream);
}
