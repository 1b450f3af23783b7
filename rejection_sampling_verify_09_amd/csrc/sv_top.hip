// The k largest logits of each row, their tokens, and the row's log-sum-exp at
// a temperature.
//
// Order: larger value first, among equal ones (-0 equals +0) the lower token;
// NaN above +infinity.  One workgroup takes a row.  A lower bound of the k-th
// largest value comes from the threads' own maxima: of each wave's 64 maxima
// the ceil(k / waves)-th largest, and of those the smallest, has at least k
// maxima at or above it.  What is at or above it goes to an LDS list, and each
// entry's place is the number of entries before it in the order: all keys are
// unlike (value, then token), so no order of arrival shows.  Where the list is
// too short (rows in order of their tokens, many equal values), the k-th
// largest value itself is found by digits and the equal ones are taken in the
// order of their tokens.
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

constexpr int TOP_CAP = 2048;    // entries of the list; at least SV_MAX_TOP
constexpr int TOP_TURNS = 512;   // runs a thread, at most: SV_MAX_V / 4 runs on 1024 threads
constexpr float LOG2E = 1.4426950408889634f;

struct TopArgs {
  const void* x;
  float* values;
  int32_t* index;
  float* lse;
  int32_t rows, V, k;
  float temperature;
};

// ord_key with -0 as +0 and NaN above everything.
__device__ __forceinline__ uint32_t top_key(float x) {
  return x != x ? 0xFFFFFFFFu : ord_key(x + 0.0f);
}

// Largest first: a wave's 64 keys.
__device__ __forceinline__ uint32_t wave_sort_desc(uint32_t v) {
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int n = 2; n <= 64; n <<= 1)
#pragma unroll
    for (int j = n >> 1; j > 0; j >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)v, j);
      const bool up = ((l & n) == 0) == ((l & j) == 0);  // keeps the larger one
      v = up ? max(v, o) : min(v, o);
    }
  return v;
}

template <int IN>
struct TopRow {
  static constexpr int E = IN == T_F32 ? 4 : 8;  // elements of a 16-byte run
  const char* p;
  int V, nt;
  // f(key, token) for each element of this thread's run of turn i
  template <typename F>
  __device__ __forceinline__ void run(int i, F&& f) const {
    const int j = (threadIdx.x + i * nt) * E;
    for (int k = 0; k < E; ++k)
      if (j + k < V) f(top_key(load1<IN>(p, j + k)), j + k);
  }
};

template <int IN>
__global__ void __launch_bounds__(1024) top_kernel(TopArgs a) {
  constexpr int E = TopRow<IN>::E;
  __shared__ uint64_t list[TOP_CAP];
  __shared__ float fsum[16];
  __shared__ uint32_t bound[2][16];
  __shared__ int32_t count[TOP_TURNS];
  __shared__ int32_t hist[256];
  __shared__ int32_t wcount[16];
  __shared__ int32_t nlist, nabove, pick, need;
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x, V = a.V, k = a.k;
  const TopRow<IN> r{static_cast<const char*>(a.x) + (size_t)row * V * (IN == T_F32 ? 4 : 2), V, nt};
  const int turns = ((V + E - 1) / E + nt - 1) / nt;
  if (t == 0) nlist = 0, nabove = 0;

  uint32_t m = 0;
  for (int i = 0; i < turns; ++i) r.run(i, [&](uint32_t key, int) { m = max(m, key); });
  const uint32_t wm = dpp_wave_umax(m);
  const int c = (k + nw - 1) / nw;
  const uint32_t sorted = wave_sort_desc(m);
  // fewer maxima than k: no bound
  if (lane == 0) bound[0][wave] = wm;
  if (lane == min(c, 64) - 1) bound[1][wave] = c <= 64 ? sorted : 0;
  __syncthreads();
  uint32_t rowmax = 0, tau = 0xFFFFFFFFu;
  for (int i = 0; i < nw; ++i) {
    rowmax = max(rowmax, bound[0][i]);
    tau = min(tau, bound[1][i]);
  }

  // the list, how many lie above the bound, and the sum of exponentials
  const float mv = rowmax == KEY_NEG_INF ? 0.0f : key_val(rowmax), scale = LOG2E / a.temperature;
  float sum = 0.0f;
  int above = 0;
  for (int i = 0; i < turns; ++i)
    r.run(i, [&](uint32_t key, int token) {
      sum += __builtin_amdgcn_exp2f((key_val(key) - mv) * scale);
      if (key >= tau) {
        above += key > tau;
        const int at = atomicAdd(&nlist, 1);
        if (at < TOP_CAP) list[at] = ((uint64_t)key << 32) | (uint32_t)~token;
      }
    });
  sum = dpp_wave_fsum(sum);
  if (lane == 0) fsum[wave] = sum;
  if (above) atomicAdd(&nabove, above);
  __syncthreads();
  if (a.lse && t == 0) {
    double s = 0.0;
    for (int i = 0; i < nw; ++i) s += (double)fsum[i];
    float lse = (float)((double)mv / (double)a.temperature + log(s));
    if (rowmax == 0xFFFFFFFFu) lse = NAN;
    else if (mv == INFINITY) lse = INFINITY;
    a.lse[row] = lse;
  }
  int n = nlist;
  if (n > TOP_CAP) {
    // the k-th largest key: the bound itself, or by digits
    if (nabove >= k) {
      uint32_t known = 0;
      int left = k;  // the place of the key among those that begin with the known digits
      for (int s = 24; s >= 0; s -= 8) {
        __syncthreads();
        for (int i = t; i < 256; i += nt) hist[i] = 0;
        __syncthreads();
        for (int i = 0; i < turns; ++i)
          r.run(i, [&](uint32_t key, int) {
            if (key >= tau && (s == 24 || (key >> (s + 8)) == (known >> (s + 8)))) atomicAdd(&hist[(key >> s) & 255], 1);
          });
        __syncthreads();
        if (t == 0) {
          int d = 255, over = 0;
          while (d > 0 && over + hist[d] < left) over += hist[d--];
          pick = d;
          need = left - over;
        }
        __syncthreads();
        known |= (uint32_t)pick << s;
        left = need;
      }
      tau = known;
    }
    // what is above it, and as many of the equal ones as k leaves, by token
    __syncthreads();
    for (int i = t; i < turns; i += nt) count[i] = 0;
    if (t == 0) nlist = 0;
    __syncthreads();
    for (int i = 0; i < turns; ++i) {
      int eq = 0;
      r.run(i, [&](uint32_t key, int token) {
        if (key > tau) list[atomicAdd(&nlist, 1)] = ((uint64_t)key << 32) | (uint32_t)~token;
        eq += key == tau;
      });
      if (eq) atomicAdd(&count[i], eq);
    }
    __syncthreads();
    int left = k - nlist, last = 0;  // the turn in which the equal ones reach k
    while (left > count[last]) left -= count[last++];
    __syncthreads();
    for (int i = 0; i < last; ++i)
      r.run(i, [&](uint32_t key, int token) {
        if (key == tau) list[atomicAdd(&nlist, 1)] = ((uint64_t)key << 32) | (uint32_t)~token;
      });
    int eq = 0;
    r.run(last, [&](uint32_t key, int) { eq += key == tau; });
    const int before = (int)wave_scan_u32((uint32_t)eq) - eq;
    if (lane == 63) wcount[wave] = before + eq;
    __syncthreads();
    int at = before;
    for (int i = 0; i < wave; ++i) at += wcount[i];
    r.run(last, [&](uint32_t key, int token) {
      if (key == tau && at++ < left) list[atomicAdd(&nlist, 1)] = ((uint64_t)key << 32) | (uint32_t)~token;
    });
    __syncthreads();
    n = nlist;
  }
  for (int i = t; i < n; i += nt) {
    const uint64_t mine = list[i];
    int place = 0;
    for (int o = 0; o < n; ++o) place += list[o] > mine;
    if (place < k) {
      const int token = (int)~(uint32_t)mine;
      a.index[(size_t)row * k + place] = token;
      a.values[(size_t)row * k + place] = load1<IN>(r.p, token);
    }
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_top_logits(const void* logits, int32_t k, float temperature, float* out_values, int32_t* out_index,
                             float* out_lse, int32_t rows, int32_t V, int32_t dtype, void* stream) {
  if (rows < 0 || V < 1 || V > SV_MAX_V || k < 1 || k > SV_MAX_TOP || k > V) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!(temperature >= FLT_MIN) || !std::isfinite(temperature)) return SV_ERR_PARAM;
  // whole waves of threads that all have a run, where there are as many
  const int e = dtype == SV_F32 ? 4 : 8, nt = std::min(1024, std::max(64, (V + e - 1) / e / 64 * 64));
  if ((int64_t)rows * nt > kGridThreads) return SV_ERR_SHAPE;
  if (rows == 0) return SV_OK;
  if (!logits || !out_values || !out_index) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), nin = (size_t)rows * (size_t)V * ie, no = (size_t)rows * (size_t)k * 4;
  const size_t nl = (size_t)rows * 4;
  if (!is_aligned(logits, ie) || !is_aligned(out_values, 4) || !is_aligned(out_index, 4) || !is_aligned(out_lse, 4))
    return SV_ERR_SHAPE;
  if (overlaps(out_values, no, logits, nin) || overlaps(out_index, no, logits, nin) || overlaps(out_lse, nl, logits, nin) ||
      overlaps(out_values, no, out_index, no) || overlaps(out_values, no, out_lse, nl) || overlaps(out_index, no, out_lse, nl))
    return SV_ERR_PARAM;
  const TopArgs a{logits, out_values, out_index, out_lse, rows, V, k, temperature};
  const dim3 grid((unsigned)rows), wg((unsigned)nt);
  if (dtype == SV_F32)
    hipLaunchKernelGGL((top_kernel<T_F32>), grid, wg, 0, (hipStream_t)stream, a);
  else
    hipLaunchKernelGGL((top_kernel<T_BF16>), grid, wg, 0, (hipStream_t)stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
