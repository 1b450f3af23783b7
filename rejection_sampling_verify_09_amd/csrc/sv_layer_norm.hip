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
//
// Bound by memory from a few MB on: 16384 x 8192 bfloat16 take 187 us a call and
// 196 traced alone forward with a residual (5.7 and 5.5 TB/s; a large copy
// reaches 5.0), 196 and 204 backward with a residual's gradient (5.5 and 5.3);
// below that by the launches and by a row's two reductions one after the other:
// one row of 4096 takes 2.5 us forward, 448 rows backward 9 to 10 + 3.6 us.  What
// holds the backward pass back elsewhere is instructions: at first 56 a column
// (separate products and sums, divisions, masks for columns past the row), 74% of
// the cycles, now with fused multiply-adds and the masks in the one wave that
// needs them about 30, and the same 16384 x 8192 went from 247 to 200 us in a
// graph.
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

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

// Sums of A values over the nw waves that share `part` (A * 16 floats, 16-byte
// aligned, which nothing else uses until the next barrier but one), in a fixed order, to all of
// their threads.  Waves first; then each lane takes one wave's sum and 16 lanes
// add theirs, instead of every lane adding all of them.
template <int A>
__device__ __forceinline__ void group_sum(float (&v)[A], float* part, int nw) {
#pragma unroll
  for (int i = 0; i < A; ++i) v[i] = dpp_wave_fsum(v[i]);
  if (nw == 1) return;
  const int lane = threadIdx.x & 63;
  if (lane == 0) __builtin_memcpy(__builtin_assume_aligned(part + (threadIdx.x >> 6) * A, 4 * A), v, sizeof(v));
  __syncthreads();
  const int w = lane & 15;
  float o[A];
  __builtin_memcpy(o, __builtin_assume_aligned(part + min(w, nw - 1) * A, 4 * A), sizeof(o));
#pragma unroll
  for (int i = 0; i < A; ++i) v[i] = row16_sum(w < nw ? o[i] : 0.0f);
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
  __shared__ __attribute__((aligned(16))) float part[4][16];
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
  const float inv = 1.0f / (float)a.d;
  float sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[0] += h[i][k];
  group_sum(sum, part[0], nw);
  const float mean = sum[0] * inv;
  float mom[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
    if (a.out_res && j < a.d) store8<IN, AL>(static_cast<char*>(a.out_res) + (base + j) * IB, h[i], a.d - j);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[i][k] = (AL ? j < a.d : j + k < a.d) ? h[i][k] - mean : 0.0f;
      mom[0] += h[i][k];
      mom[1] = __builtin_fmaf(h[i][k], h[i][k], mom[1]);
    }
  }
  group_sum(mom, part[1], nw);
  const float left = mom[0] * inv;
  // a row whose sum is not finite comes out all NaN instead of as zeros
  const float var = fmaxf(mom[1] * inv - left * left, 0.0f) + a.eps;
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
        h[i][k] = __builtin_fmaf((h[i][k] - left) * r, w[k], b[k]);
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

// A thread a run up to 4096 columns, two runs up to 16384: the waves share the
// two reductions' instructions out over more columns (16384 x 8192 bfloat16 with
// one, two and four runs a thread 204, 196 and 207 us, to e4m3 245, 198 and 196;
// one row of 8192 4.2, 4.6 and 5.7; x 4096 one and two 99 and 99).  The rows of
// one wave go four to a workgroup.
struct LayerLaunch {
  int nt, ny, vpt;  // threads a row, rows a workgroup, runs a thread
  int64_t wgs;
  LayerLaunch(int64_t rows, int d) {
    const int nv = (d + 7) / 8, runs = nv > 512 ? 2 : 1;
    nt = std::min(1024, ((nv + runs - 1) / runs + 63) / 64 * 64);
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
  float* dw;  // [groups][stride] sums over each workgroup's rows, or NULL
  float* db;
  int32_t rows, d, stride;
  size_t fold;  // wide rows: floats from a part to where it is folded
  float eps;
};

// Rows that are added to a sum one after another before it is set aside and
// begun anew: a workgroup's sum of n rows by itself is off by up to n 2^-24 of
// the magnitudes' sum (2^30 rows on 256 workgroups: by a fourth), folded by (1024
// + n / 1024) 2^-24.
constexpr int BACK_TURNS = 1024;

// What the sums over one row give: the factors of
// dh = r (g - gm - (c - left) r gn).
struct RowBack {
  float left, r, gm, gn;
  // mom: sums of c^2 and g c, and, with a mean, of c and g
  template <bool CENTER>
  __device__ __forceinline__ void set(const float (&mom)[CENTER ? 4 : 2], float inv, float eps) {
    left = CENTER ? mom[CENTER ? 2 : 0] * inv : 0.0f;
    gm = CENTER ? mom[CENTER ? 3 : 0] * inv : 0.0f;
    const float var = fmaxf(mom[0] * inv - left * left, 0.0f) + eps;
    r = mom[0] < INFINITY && var < INFINITY ? rsqrtf(var) : NAN;
    gn = (mom[1] * inv - left * gm) * r;
  }
  // n_j, and dh_j of it and of dy_j w_j
  __device__ __forceinline__ float unit(float c) const { return (c - left) * r; }
  __device__ __forceinline__ float grad(float g, float v) const { return r * __builtin_fmaf(-v, gn, g - gm); }
};

// Eight elements as they lie in memory, at any alignment: half the registers
// of floats for bfloat16, so that the next row can be on its way.
template <int IN>
struct Raw8 {
  uint4 v[IN == T_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* p) { __builtin_memcpy(v, p, sizeof(v)); }
  __device__ __forceinline__ void arrived() {
#pragma unroll
    for (uint4& q : v) asm volatile("" : "+v"(q.x), "+v"(q.y), "+v"(q.z), "+v"(q.w));
  }
  __device__ __forceinline__ void ones() {
    const uint32_t u = IN == T_F32 ? 0x3F800000u : 0x3F803F80u;
    v[0] = make_uint4(u, u, u, u);
    if (IN == T_F32) v[1] = v[0];
  }
  __device__ __forceinline__ float operator[](int k) const {
    uint32_t u[sizeof(v) / 4];
    __builtin_memcpy(u, v, sizeof(v));
    return IN == T_F32 ? __uint_as_float(u[k]) : k & 1 ? bf16_hi(u[k / 2]) : bf16_lo(u[k / 2]);
  }
};

// One pass over rows of 8 to 16384 columns: blockDim.x threads take a row, VPT
// runs of 8 columns each, and keep their columns' sums for the weights in
// registers over all of their rows; blockDim.y rows are under way in a
// workgroup, and their sums are joined at the end.  Rows (blockIdx.x + i
// gridDim.x) blockDim.y + threadIdx.y.
//
// The next row's loads are issued before this row's second reduction is used,
// and stay in flight over the stores: no load and no store stands in a branch,
// since at a branch's end the compiler has to wait for all of them.  So a run
// that would end past the row begins earlier: it reads, forms and writes some
// of its neighbour's columns once more, with the same result, and leaves them
// out of its sums.
//
// FOLD: a workgroup has more than BACK_TURNS turns.  In the other kernels it would
// cost registers (two runs a thread: 8192 x 16384 bfloat16 with a residual's
// gradient 236 us, 243 so); where it is needed, 270000 x 16384 takes 6.7 to 6.9 ms,
// 6.4 without, 1000000 x 1024 1.48 either way.
template <int IN, bool CENTER, int VPT, bool RES, bool FOLD>
__global__ void __launch_bounds__(1024) norm_backward_kernel(BackArgs a) {
  extern __shared__ __attribute__((aligned(16))) float smem[];
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6, ny = blockDim.y;
  float* part = smem + threadIdx.y * 160;  // [2][16 + 4 * 16]
  constexpr int IB = IN == T_F32 ? 4 : 2, S = CENTER ? 4 : 2;
  constexpr bool AHEAD = VPT == 1;  // two runs a thread have no registers for another row
  const float inv = 1.0f / (float)a.d;
  const char *hp = static_cast<const char*>(a.h), *dyp = static_cast<const char*>(a.dy),
             *rp = static_cast<const char*>(a.dres);
  Raw8<IN> w[VPT], h[VPT], dy[VPT], dr[RES ? VPT : 1];
  float sw[VPT][8], sb[VPT][8];
  int js[VPT], skip[VPT];  // the run's first column, and how many of its columns are the neighbour's
  bool edge = false;       // one of the wave's has some
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int j = (t + i * nt) * 8;
    js[i] = min(j, a.d - 8);
    skip[i] = min(j - js[i], 8);
    w[i].ones();
    if (a.w) w[i].load(static_cast<const char*>(a.w) + (size_t)js[i] * IB);
    edge |= __any(skip[i] != 0) != 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sw[i][k] = sb[i][k] = 0.0f;
  }
  auto fetch = [&](int row) {
    const size_t base = (size_t)min(row, a.rows - 1) * a.d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const size_t at = (base + js[i]) * IB;
      h[i].load(hp + at);
      dy[i].load(dyp + at);
      if (RES) dr[i].load(rp + at);
    }
  };
  int row = blockIdx.x * ny + threadIdx.y, turn = 0;
  const int step = gridDim.x * ny;
  // all: each of the workgroup's rows is there (mine: this one is)
  auto body = [&](auto all, bool mine) {
    if (!AHEAD) fetch(row);
    float c[VPT][8], mom[S];
    float mean = 0.0f;
    if (CENTER) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += h[i][k];
        if (edge) {
          v = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) v += k >= skip[i] ? h[i][k] : 0.0f;
        }
        sum[0] += v;
      }
      group_sum(sum, part + turn * 80, nw);
      mean = sum[0] * inv;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) mom[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float v[S];
      auto add = [&](float cc, float g) {
        v[0] = __builtin_fmaf(cc, cc, v[0]);
        v[1] = __builtin_fmaf(g, cc, v[1]);
        if (CENTER) v[S - 2] += cc, v[S - 1] += g;
      };
#pragma unroll
      for (int k = 0; k < S; ++k) v[k] = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[i][k] = h[i][k] - mean;
        add(c[i][k], dy[i][k] * w[i][k]);
      }
      if (edge) {
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) add(k >= skip[i] ? c[i][k] : 0.0f, k >= skip[i] ? dy[i][k] * w[i][k] : 0.0f);
      }
#pragma unroll
      for (int k = 0; k < S; ++k) mom[k] += v[k];
    }
    Raw8<IN> dyc[VPT], drc[RES ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      dyc[i] = dy[i];
      if (RES) {
        drc[i] = dr[i];
        drc[i].arrived();  // before the barrier behind which a neighbour may write over it (in place)
      }
    }
    if (AHEAD) fetch(row + step);
    group_sum(mom, part + turn * 80 + 16, nw);
    RowBack f;
    f.template set<CENTER>(mom, inv, a.eps);
    if (decltype(all)::value || mine) {
      const size_t base = (size_t)row * a.d;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = f.unit(c[i][k]), dyk = dyc[i][k];
          sw[i][k] = __builtin_fmaf(dyk, v, sw[i][k]);
          if (CENTER) sb[i][k] += dyk;
          o[k] = f.grad(dyk * w[i][k], v);
          if (RES) o[k] += drc[i][k];
        }
        store8<IN, false>(static_cast<char*>(a.dh) + (base + js[i]) * IB, o, 8);
      }
    }
    row += step;
    turn ^= 1;
  };
  int first = blockIdx.x * ny;
  if (AHEAD) {
    fetch(row);
    // all of it: in the loop each wait can then count on the store behind the loads
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  }
  if constexpr (FOLD) {
    // in LDS, where no load and no store of the rows has to be waited for; addresses anew each time, for their registers
    bool folded = false;
    auto each_sum = [&](auto&& f) {
      const int threads = blockDim.x * blockDim.y;
      float* fold = smem + blockDim.y * 160 + threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          f(sw[i][k], fold[(i * 8 + k) * threads]);
          if (CENTER) f(sb[i][k], fold[(VPT * 8 + i * 8 + k) * threads]);
        }
    };
    while (true) {
      for (int n = 0; n < BACK_TURNS && first + ny <= a.rows; ++n, first += step) body(std::true_type{}, true);
      if (first + ny > a.rows) break;
      each_sum([&](float& v, float& f) {
        f = folded ? f + v : v;
        v = 0.0f;
      });
      folded = true;
    }
    if (first < a.rows) body(std::false_type{}, row < a.rows);
    if (folded) each_sum([&](float& v, float& f) { v += f; });
  } else {
    for (; first + ny <= a.rows; first += step) body(std::true_type{}, true);
    if (first < a.rows) body(std::false_type{}, row < a.rows);
  }
  if (!a.dw && !a.db) return;
  // rows of the workgroup, then the workgroup's part of the workspace
  if (ny > 1) {
    float* join = smem + ny * 160 + (size_t)t * (VPT * 8);
    for (int y = 1; y < ny; ++y) {
      __syncthreads();
      if ((int)threadIdx.y == y)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            join[i * 8 + k] = sw[i][k];
            if (CENTER) join[(size_t)nt * VPT * 8 + i * 8 + k] = sb[i][k];
          }
      __syncthreads();
      if (threadIdx.y == 0)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sw[i][k] += join[i * 8 + k];
            if (CENTER) sb[i][k] += join[(size_t)nt * VPT * 8 + i * 8 + k];
          }
    }
    if (threadIdx.y != 0) return;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (skip[i] == 8) continue;
    const size_t at = (size_t)blockIdx.x * a.stride + js[i];
    if (a.dw) store8<T_F32, false>(reinterpret_cast<char*>(a.dw + at), sw[i], 8);
    if (CENTER && a.db) store8<T_F32, false>(reinterpret_cast<char*>(a.db + at), sb[i], 8);
  }
}

// Rows of other widths (up to 7, or above 16384 columns, whose sums the registers
// do not hold): a workgroup takes a row at a time, reads it again for each step,
// and keeps the sums for the weights in its part of the workspace (1024 x 40000
// bfloat16 199 us, with a residual's gradient 224, a fourth of the other kernel's rate).
template <int IN, bool CENTER>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(BackArgs a) {
  __shared__ __attribute__((aligned(16))) float part[2][80];
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6;
  constexpr int IB = IN == T_F32 ? 4 : 2;
  const float inv = 1.0f / (float)a.d;
  float* dw = a.dw ? a.dw + (size_t)blockIdx.x * a.stride : nullptr;
  float* db = a.db ? a.db + (size_t)blockIdx.x * a.stride : nullptr;
  // 8 columns' sums so far, added to what was set aside before; more: there is something
  auto set_aside = [&](int j, bool more) {
    for (float* p : {dw, db}) {
      if (!p) continue;
      float s[8], f[8];
      load8<T_F32, false>(reinterpret_cast<char*>(p + j), s, a.d - j);
      if (more) {
        load8<T_F32, false>(reinterpret_cast<char*>(p + a.fold + j), f, a.d - j);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] += f[k];
      }
      store8<T_F32, false>(reinterpret_cast<char*>(p + a.fold + j), s, a.d - j);
    }
  };
  int turn = 0, n = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1, ++n) {
    const size_t base = (size_t)row * a.d;
    const char* hp = static_cast<const char*>(a.h) + base * IB;
    const char* dyp = static_cast<const char*>(a.dy) + base * IB;
    const char* wp = static_cast<const char*>(a.w);
    float mean = 0.0f;
    if (CENTER) {
      float sum[1] = {0.0f};
      for (int j = t * 8; j < a.d; j += nt * 8) {
        float h[8];
        load8<IN, false>(hp + (size_t)j * IB, h, a.d - j);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[0] += h[k];
      }
      group_sum(sum, part[turn], nw);
      mean = sum[0] * inv;
    }
    constexpr int S = CENTER ? 4 : 2;
    float mom[S];
#pragma unroll
    for (int k = 0; k < S; ++k) mom[k] = 0.0f;
    float h[8], dy[8], w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    for (int j = t * 8; j < a.d; j += nt * 8) {
      load8<IN, false>(hp + (size_t)j * IB, h, a.d - j);
      load8<IN, false>(dyp + (size_t)j * IB, dy, a.d - j);
      if (wp) load8<IN, false>(wp + (size_t)j * IB, w, a.d - j);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float c = j + k < a.d ? h[k] - mean : 0.0f, g = dy[k] * w[k];
        mom[0] += c * c;
        mom[1] += g * c;
        if (CENTER) mom[S - 2] += c, mom[S - 1] += g;
      }
    }
    group_sum(mom, part[turn] + 16, nw);
    RowBack f;
    f.template set<CENTER>(mom, inv, a.eps);
    for (int j = t * 8; j < a.d; j += nt * 8) {
      float o[8], sw[8], sb[8];
      load8<IN, false>(hp + (size_t)j * IB, h, a.d - j);
      load8<IN, false>(dyp + (size_t)j * IB, dy, a.d - j);
      if (wp) load8<IN, false>(wp + (size_t)j * IB, w, a.d - j);
      if (a.dres) load8<IN, false>(static_cast<const char*>(a.dres) + (base + j) * IB, o, a.d - j);
      const bool begun = n % BACK_TURNS != 0;
      if (!begun && n > 0) set_aside(j, n > BACK_TURNS);
#pragma unroll
      for (int k = 0; k < 8; ++k) sw[k] = sb[k] = 0.0f;
      if (begun && dw) load8<T_F32, false>(reinterpret_cast<char*>(dw + j), sw, a.d - j);
      if (begun && db) load8<T_F32, false>(reinterpret_cast<char*>(db + j), sb, a.d - j);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = f.unit(h[k] - mean), dh = f.grad(dy[k] * w[k], v);
        o[k] = a.dres ? dh + o[k] : dh;
        sw[k] = __builtin_fmaf(dy[k], v, sw[k]);
        sb[k] += dy[k];
      }
      store8<IN, false>(static_cast<char*>(a.dh) + (base + j) * IB, o, a.d - j);
      if (dw) store8<T_F32, false>(reinterpret_cast<char*>(dw + j), sw, a.d - j);
      if (db) store8<T_F32, false>(reinterpret_cast<char*>(db + j), sb, a.d - j);
    }
  }
  if (n <= BACK_TURNS) return;
  for (int j = t * 8; j < a.d; j += nt * 8)
    for (float* p : {dw, db}) {
      if (!p) continue;
      float s[8], f[8];
      load8<T_F32, false>(reinterpret_cast<char*>(p + j), s, a.d - j);
      load8<T_F32, false>(reinterpret_cast<char*>(p + a.fold + j), f, a.d - j);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += f[k];
      store8<T_F32, false>(reinterpret_cast<char*>(p + j), s, a.d - j);
    }
}

// Column sums of the workgroups' parts: 64 columns a workgroup, 16 threads of 4
// columns side by side and 64 parts at a time, joined in a fixed order.
__global__ void __launch_bounds__(1024) norm_backward_sum_kernel(const float* wp, const float* bp, float* dw, float* db,
                                                                 int groups, int d, int stride) {
  __shared__ float4 join[16][16];
  const float* p = blockIdx.y ? bp : wp;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int q = threadIdx.x & 15, at = threadIdx.x >> 4, j = blockIdx.x * 64 + q * 4;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (j < d)
#pragma unroll 4
    for (int g = at; g < groups; g += 64) {
      const float4 v = *reinterpret_cast<const float4*>(p + (size_t)g * stride + j);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
#pragma unroll
  for (int o = 16; o < 64; o <<= 1)
    s.x += __shfl_xor(s.x, o), s.y += __shfl_xor(s.y, o), s.z += __shfl_xor(s.z, o), s.w += __shfl_xor(s.w, o);
  if ((threadIdx.x & 63) < 16) join[threadIdx.x >> 6][q] = s;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const int col = blockIdx.x * 64 + threadIdx.x;
  if (col >= d) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += reinterpret_cast<const float*>(join[i])[threadIdx.x];
  out[col] = v;
}

constexpr int BACK_LDS = (160 + 1024 * 2 * 16) * 4;  // two runs a thread
constexpr int BACK_ROWS = 1 << 30;  // a workgroup's next row stays within 32 bits

// A row's threads and runs, rows a workgroup, and workgroups: what the workspace
// holds a part for.  One compute unit a workgroup, with equal turns (16384 x 8192
// bfloat16 with 128, 224, 256, 384 and 512 workgroups 430, 215, 202, over 300 and
// 213 us; 448 x 4096, where the parts count, 13.1 with 112, 13.4 with 224, 16.3
// with 448), of at least 512 threads (16384 x 1024 with a residual's gradient
// with 256, 512 and 1024 threads 45, 34 and 35 us).  One workgroup without parts to join up to two turns (2 rows
// of 4096 5.7 us against 6.7, 4 rows 8.3 against 6.7).
struct BackPlan {
  int nt, ny, vpt, groups, stride;
  bool wide, fold;
  BackPlan(int rows, int d) {
    const int nv = (d + 7) / 8;
    wide = d < 8 || nv > 2048;
    vpt = nv > 1024 ? 2 : 1;
    nt = std::min(1024, ((nv + vpt - 1) / vpt + 63) / 64 * 64);
    ny = wide || nt >= 512 ? 1 : std::min(8, 512 / nt);
    const int turns = (rows + ny - 1) / ny;
    const int each = std::max(turns <= 2 ? turns : 1, (turns + 255) / 256);
    groups = turns == 0 ? 0 : (turns + each - 1) / each;
    stride = (d + 3) / 4 * 4;
    fold = each > BACK_TURNS;
  }
  // the reductions', and where sums are folded and, behind the last row, the workgroup's rows joined
  size_t lds() const { return ((size_t)ny * 160 + (fold ? (size_t)ny : ny > 1 ? 1 : 0) * nt * vpt * 16) * 4; }
  // floats of a sum's parts
  int64_t part() const { return groups > 1 ? (int64_t)groups * stride * (wide && fold ? 2 : 1) : 0; }
};

template <int IN, bool CENTER>
hipError_t launch_back(const BackArgs& a, const BackPlan& l, hipStream_t s) {
  const dim3 grid((unsigned)l.groups), wg((unsigned)l.nt, (unsigned)l.ny);
  if (l.wide) {
    hipLaunchKernelGGL((norm_backward_wide_kernel<IN, CENTER>), grid, wg, 0, s, a);
    return hipGetLastError();
  }
  hipError_t e = hipSuccess;
  auto go = [&](auto vpt, auto res, auto fold) {
    constexpr auto kernel = norm_backward_kernel<IN, CENTER, decltype(vpt)::value, decltype(res)::value, decltype(fold)::value>;
    if (l.fold) e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, BACK_LDS);
    if (e == hipSuccess) hipLaunchKernelGGL(kernel, grid, wg, l.lds(), s, a);
  };
  auto sums = [&](auto vpt, auto res) { l.fold ? go(vpt, res, std::true_type{}) : go(vpt, res, std::false_type{}); };
  auto width = [&](auto vpt) { a.dres ? sums(vpt, std::true_type{}) : sums(vpt, std::false_type{}); };
  l.vpt == 1 ? width(std::integral_constant<int, 1>{}) : width(std::integral_constant<int, 2>{});
  return e == hipSuccess ? hipGetLastError() : e;
}

int norm_backward(bool center, const void* grad, const void* h, const void* weight, const void* grad_residual, float eps,
                  void* grad_h, float* grad_weight, float* grad_bias, void* workspace, int64_t workspace_bytes,
                  int32_t rows, int32_t d, int32_t dtype, hipStream_t s) {
  if (rows < 0 || rows > BACK_ROWS || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return SV_ERR_PARAM;
  const BackPlan l(rows, d);
  const int groups = l.groups;
  const size_t ie = (size_t)type_bytes(dtype), nin = (size_t)rows * (size_t)d * ie, nw = (size_t)d * ie;
  const size_t np = (size_t)d * 4, one = (size_t)l.part() * 4;
  const size_t ws = one * ((grad_weight ? 1 : 0) + (grad_bias ? 1 : 0));
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
  a.stride = l.stride;
  a.fold = (size_t)groups * l.stride;
  if (rows > 0) {
    const hipError_t e = center ? (dtype == SV_F32 ? launch_back<T_F32, true>(a, l, s) : launch_back<T_BF16, true>(a, l, s))
                                : (dtype == SV_F32 ? launch_back<T_F32, false>(a, l, s) : launch_back<T_BF16, false>(a, l, s));
    if (e != hipSuccess) return SV_ERR_HIP;
  }
  if (groups != 1 && (grad_weight || grad_bias)) {
    hipLaunchKernelGGL(norm_backward_sum_kernel, dim3((unsigned)((d + 63) / 64), grad_bias ? 2 : 1), dim3(1024), 0, s, a.dw,
                       a.db, grad_weight, grad_bias, groups, d, l.stride);
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
  if (rows < 0 || rows > BACK_ROWS || d < 1 || d > SV_MAX_NORM_D) return SV_ERR_SHAPE;
  const BackPlan l(rows, d);
  return l.part() * 8;
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
