// Divergence of a draft's distribution from its target's top logits, and the
// gradient of the draft's logits.
//
// Teacher of a row: k entries (token i_j, logit t_j), entries outside [0, V)
// absent.  With the teacher's log-sum-exp L: p_j = exp(t_j / T - L), and what
// they leave, r = max(0, 1 - sum p), is the rest of the vocabulary as one more
// outcome; without: p = softmax of t_j / T over the list, r = 0.
// Student: q = softmax(s / T), R the mass of the tokens not listed.
//   loss   = w (sum_j p_j (log p_j - log q_{i_j}) + r (log r - log R))
//   grad_v = w / T (q_v - p_v)            v listed
//          = w / T (q_v / R) (R - r)      v not listed
//
// One workgroup takes a row.  The listed tokens are marked in a bitmap in LDS
// and the streaming passes see the others alone, so that R is a sum of its
// own and never a difference; q_v / R comes from the rest's own maximum and
// sum, which no list can underflow.  What is done once an entry is done in 64
// bits: there are few, and the loss is a difference of numbers close to each
// other.
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

struct DistillArgs {
  const void* x;
  const int32_t* index;
  const float* values;
  const float* top_lse;
  const float* weight;
  float* loss;
  void* grad;
  int32_t rows, V, k;
  float temperature;
};

// In LDS: probabilities, the student's logits and the tokens of the list, [k]
// each, and the bitmap [ceil(V / 32)].
inline size_t distill_lds(int V, int k) { return (size_t)k * 16 + (size_t)((V + 31) / 32) * 4; }

template <int IN>
__global__ void __launch_bounds__(1024) distill_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ float fmx[3][16];
  __shared__ double dsum[4][16];
  __shared__ int32_t repeated;
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x, V = a.V, k = a.k;
  constexpr int IB = IN == T_F32 ? 4 : 2;
  double* prob = reinterpret_cast<double*>(smem);          // [k] p_j, unnormalised
  float* student = reinterpret_cast<float*>(prob + k);     // [k] s_{i_j}
  int32_t* token = reinterpret_cast<int32_t*>(student + k);  // [k] i_j, -1 where absent
  uint32_t* marks = reinterpret_cast<uint32_t*>(token + k);
  const char* x = static_cast<const char*>(a.x) + (size_t)row * V * IB;
  char* grad = a.grad ? static_cast<char*>(a.grad) + (size_t)row * V * IB : nullptr;
  const float w = a.weight ? a.weight[row] : 1.0f;
  const float tl = a.top_lse ? a.top_lse[row] : 0.0f;
  bool none = w == 0.0f || tl == -INFINITY;  // nothing to learn from this row
  if (!none) {
    for (int i = t; i < (V + 31) / 32; i += nt) marks[i] = 0;
    if (t == 0) repeated = 0;
    float tm = -INFINITY, sm = -INFINITY;
    __syncthreads();
    for (int j = t; j < k; j += nt) {
      const int v = a.index[(size_t)row * k + j];
      const bool here = v >= 0 && v < V;
      token[j] = here ? v : -1;
      if (here) {
        const float s = load1<IN>(x, v), tv = a.values[(size_t)row * k + j];
        student[j] = s;
        sm = fmaxf(sm, s);
        tm = fmaxf(tm, tv);
        if (tv != tv) tm = INFINITY;  // fmaxf would lose it
        // the first of a token listed more than once stands for its q
        if (atomicOr(&marks[v >> 5], 1u << (v & 31)) >> (v & 31) & 1) {
          token[j] = v | 0x40000000;
          repeated = 1;
        }
      }
    }
    __syncthreads();
    float rm = -INFINITY;
    for (int j = t; j < V; j += nt)
      if (!(marks[j >> 5] >> (j & 31) & 1)) rm = fmaxf(rm, load1<IN>(x, j));
    rm = dpp_wave_fmax(rm), tm = dpp_wave_fmax(tm), sm = dpp_wave_fmax(sm);
    if (lane == 0) fmx[0][wave] = rm, fmx[1][wave] = tm, fmx[2][wave] = sm;
    __syncthreads();
    rm = fmx[0][0], tm = fmx[1][0], sm = fmx[2][0];
    for (int i = 1; i < nw; ++i) rm = fmaxf(rm, fmx[0][i]), tm = fmaxf(tm, fmx[1][i]), sm = fmaxf(sm, fmx[2][i]);
    none = !a.top_lse && tm == -INFINITY;
    if (!none) {
      const double invT = 1.0 / (double)a.temperature;
      const float scale = LOG2E / a.temperature;
      const float r0 = rm == -INFINITY ? 0.0f : rm;  // a rest that is all -inf adds exp(-inf)
      const double s0 = sm == -INFINITY ? 0.0 : (double)sm;
      double acc[4] = {0.0, 0.0, 0.0, 0.0};  // rest, listed, sum of p, sum of p (t - s) / T
      float sum = 0.0f;
      for (int j = t; j < V; j += nt)
        if (!(marks[j >> 5] >> (j & 31) & 1)) sum += __builtin_amdgcn_exp2f((load1<IN>(x, j) - r0) * scale);
      acc[0] = (double)sum;
      for (int j = t; j < k; j += nt) {
        if (token[j] < 0) continue;
        const double tv = (double)a.values[(size_t)row * k + j], s = (double)student[j];
        const double p = exp((tv - (a.top_lse ? 0.0 : (double)tm)) * invT - (a.top_lse ? (double)tl : 0.0));
        prob[j] = p;
        if (!(token[j] & 0x40000000)) acc[1] += exp((s - s0) * invT);
        acc[2] += p;
        if (p != 0.0) acc[3] += p * ((tv - s) * invT);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = dpp_wave_sum(acc[i]);
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) dsum[i][wave] = acc[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = dsum[i][0];
        for (int o = 1; o < nw; ++o) acc[i] += dsum[i][o];
      }
      const double total = acc[2], norm = a.top_lse ? 1.0 : 1.0 / total;
      // relative to the larger of the two maxima
      const double top = acc[0] == 0.0 ? s0 : acc[1] == 0.0 ? (double)r0 : fmax((double)r0, s0);
      const double A = acc[0] == 0.0 ? 0.0 : acc[0] * exp(((double)r0 - top) * invT);
      const double B = acc[1] == 0.0 ? 0.0 : acc[1] * exp((s0 - top) * invT);
      const double inv = A + B == 0.0 ? 0.0 : 1.0 / (A + B);
      const double left = a.top_lse && acc[0] != 0.0 ? fmax(0.0, 1.0 - total) : 0.0;
      const double gs = (double)w * invT;
      if (grad) {
        const float coef = acc[0] == 0.0 ? 0.0f : (float)(gs * (A * inv - left) / acc[0]);
        for (int j = t; j < V; j += nt) store1<IN>(grad, j, __builtin_amdgcn_exp2f((load1<IN>(x, j) - r0) * scale) * coef);
        __syncthreads();  // the listed tokens' own values come after
        for (int j = t; j < k; j += nt) {
          if (token[j] < 0) continue;
          const int v = token[j] & 0x3FFFFFFF;
          double p = prob[j];
          if (repeated) {
            p = 0.0;
            for (int o = 0; o < k; ++o)
              if (token[o] >= 0 && (token[o] & 0x3FFFFFFF) == v) p += prob[o];
          }
          const double q = exp(((double)student[j] - top) * invT) * inv;
          store1<IN>(grad, v, (float)(gs * ((student[j] == -INFINITY ? 0.0 : q) - p * norm)));
        }
      }
      if (a.loss && t == 0) {
        // log p_j - log q_j = (t_j - s_j) / T - log of the teacher's sum + log of the student's
        const double ls = top * invT + log(A + B);
        const double lt = a.top_lse ? (double)tl : (double)tm * invT + log(total);
        double loss = acc[3] * norm;
        if (total != 0.0 && loss != INFINITY) loss += total * norm * (ls - lt);
        if (left > 0.0) loss += left * (log(left) - (((double)r0 - top) * invT + log(acc[0]) - log(A + B)));
        a.loss[row] = (float)((double)w * loss);
      }
    }
  }
  if (none) {
    if (a.loss && t == 0) a.loss[row] = 0.0f;
    if (grad)
      for (int j = t; j < V; j += nt) store1<IN>(grad, j, 0.0f);
  }
}

template <int IN>
hipError_t launch_distill(const DistillArgs& a, int nt, hipStream_t s) {
  const size_t lds = distill_lds(a.V, a.k);
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)distill_kernel<IN>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((distill_kernel<IN>), dim3((unsigned)a.rows), dim3((unsigned)nt), lds, s, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_distill_loss(const void* logits, const int32_t* top_index, const float* top_values,
                               const float* top_lse, const float* weight, float temperature, float* out_loss,
                               void* out_grad, int32_t rows, int32_t V, int32_t k, int32_t dtype, void* stream) {
  if (rows < 0 || V < 1 || V > SV_MAX_DISTILL_V || k < 1 || k > SV_MAX_TOP) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!(temperature >= FLT_MIN) || !std::isfinite(temperature)) return SV_ERR_PARAM;
  const int e = dtype == SV_F32 ? 4 : 8, nt = std::min(1024, ((V + e - 1) / e + 63) / 64 * 64);
  if ((int64_t)rows * nt > kGridThreads) return SV_ERR_SHAPE;
  if (rows == 0) return SV_OK;
  if (!logits || !top_index || !top_values || (!out_loss && !out_grad)) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), nin = (size_t)rows * (size_t)V * ie, nk = (size_t)rows * (size_t)k * 4;
  const size_t nr = (size_t)rows * 4;
  if (!is_aligned(logits, ie) || !is_aligned(out_grad, ie) || !is_aligned(top_index, 4) || !is_aligned(top_values, 4) ||
      !is_aligned(top_lse, 4) || !is_aligned(weight, 4) || !is_aligned(out_loss, 4))
    return SV_ERR_SHAPE;
  // out_grad may be the logits, element for element; any other overlap of an output is refused
  struct Range {
    const void* p;
    size_t n;
  };
  if ((overlaps(out_grad, nin, logits, nin) && out_grad != logits) || overlaps(out_loss, nr, logits, nin) ||
      overlaps(out_grad, nin, out_loss, nr))
    return SV_ERR_PARAM;
  const Range lists[] = {{top_index, nk}, {top_values, nk}, {top_lse, nr}, {weight, nr}};
  for (const Range& i : lists)
    if (overlaps(out_grad, nin, i.p, i.n) || overlaps(out_loss, nr, i.p, i.n)) return SV_ERR_PARAM;
  const DistillArgs a{logits, top_index, top_values, top_lse, weight, out_loss, out_grad, rows, V, k, temperature};
  const hipError_t err = dtype == SV_F32 ? launch_distill<T_F32>(a, nt, (hipStream_t)stream)
                                         : launch_distill<T_BF16>(a, nt, (hipStream_t)stream);
  return err == hipSuccess ? SV_OK : SV_ERR_HIP;
}
