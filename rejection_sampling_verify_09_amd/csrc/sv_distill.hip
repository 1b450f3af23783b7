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
// One workgroup takes a row and keeps it in registers, as it lies in memory,
// between the sums and the gradient: every logit is read once and written once
// (rows above 256 KiB: what lies behind that is read twice).  The listed tokens
// are marked in LDS and set to -inf in the registers, so that R is a sum of its
// own and never a difference, and q_v / R is formed from the rest alone, which
// no list can underflow.  The sums are formed as the loads arrive, relative to
// the largest logit of a thread's first run; what lies far above that (masked
// first runs, small temperatures) has the thread's wave form its sums once more.
// What is done once an entry is done in 64 bits: there are few, and the loss is
// a difference of numbers close to each other.
//
// 448 x 128256 bfloat16 with an eighth of the rows left out and lists of 64: 51 us
// (4.2 TB/s of what must be read and written; a large copy reaches 5.0), of
// which the vector units are busy for half: two exponentials a logit at a
// quarter of the rate, and the 256 compute units hold 256 rows at a time, in
// step, so that loads, sums, gradient and stores take turns.  2304 x 152064
// float32: 608 us (4.6 TB/s).  A single row takes 19 us, 12 of them instructions.
// What made the difference (448 x 128256): registers instead of three reads
// (185 -> 82 us); loads outside branches, at whose ends the compiler waits for
// all of them, and columns formed anew in each pass instead of being kept
// (82 -> 73); marks that a thread reads in one load (73 -> 71); the gradient
// stored past the caches (67 -> 60; 2304 x 152064 691 -> 614); one wave for what
// is done once a row (60 -> 57.5); a reference from the first run instead of a
// running maximum (57 -> 55).  Not kept: two rows a compute unit whose second
// pass reads them again (79 against 67, 2304 x 152064 925 against 692); a check
// of each run's sum instead of its maximum (61 against 57: a wait a run).
#include "sv_rows.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

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
// each, and the marks: a bit a token, in the order in which the threads take
// them.  A thread's runs in registers have theirs next to each other (a byte a
// run of 8, half a byte a run of 4), the runs behind them turn by turn.
struct Marks {
  int e, nt, nh, turns;  // columns a run, threads, runs a thread in registers and in all
  __host__ __device__ int of(int nruns) const { return e == 8 ? nruns : (nruns + 1) / 2; }
  __host__ __device__ int bytes() const { return (nt * (of(nh) + of(turns - nh)) + 15) & ~15; }
  // bit of the token
  __device__ __forceinline__ uint32_t bit(int token) const {
    const uint32_t run = (uint32_t)token / (uint32_t)e, i = run / (uint32_t)nt, t = run - i * nt;
    const uint32_t n = (uint32_t)nh, at = i < n ? i : i - n;
    const uint32_t byte = i < n ? t * of(nh) + (e == 8 ? at : at / 2) : nt * of(nh) + (e == 8 ? at : at / 2) * nt + t;
    return byte * 8 + (e == 8 ? 0 : at % 2 * 4) + (uint32_t)token % (uint32_t)e;
  }
};

// NH runs a thread in registers; MORE: rows that go on behind them; TINY: rows
// shorter than a run.
template <int IN, int NH, bool MORE, bool TINY>
__global__ void __launch_bounds__(1024) distill_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  __shared__ float4 fmx[16];
  __shared__ float fany[16];
  __shared__ double dsum[3][16];
  __shared__ int32_t repeated;
  struct Row {
    // mass: of the student's logits relative to top, inv its reciprocal; total: of the list, norm its reciprocal (1 with
    // the teacher's log-sum-exp); dot: sum of p (t - s) / T, s relative to the list's maximum and t too without the
    // teacher's log-sum-exp, so that what all of a row's logits have in common (1e20 in a row masked altogether) takes no
    // digits; base: the rest of log p - log q, but for the sums; left: the teacher's rest; coef: of the gradient there
    double mass, inv, top, total, norm, dot, base, left;
    float coef;
  };
  __shared__ Row fin;
  constexpr int E = Run<IN>::E, IB = Run<IN>::B;
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x, V = a.V, k = a.k;
  double* prob = reinterpret_cast<double*>(smem);          // [k] p_j, unnormalised
  float* student = reinterpret_cast<float*>(prob + k);     // [k] s_{i_j}
  int32_t* token = reinterpret_cast<int32_t*>(student + k);  // [k] i_j, -1 where absent
  uint32_t* marks = reinterpret_cast<uint32_t*>(token + k);
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(marks);
  constexpr int MB = E == 8 ? NH : (NH + 1) / 2;  // bytes of marks a thread for its runs in registers
  const char* x = static_cast<const char*>(a.x) + (size_t)row * V * IB;
  char* grad = a.grad ? static_cast<char*>(a.grad) + (size_t)row * V * IB : nullptr;
  const int turns = MORE ? ((V + E - 1) / E + nt - 1) / nt : NH;
  const Marks at{E, nt, NH, turns};
  const float w = a.weight ? a.weight[row] : 1.0f;
  const float tl = a.top_lse ? a.top_lse[row] : 0.0f;
  const float scale = LOG2E / a.temperature;
  bool none = w == 0.0f || tl == -INFINITY;  // nothing to learn from this row
  if (!none) {
    // The list's loads first: those of the row need not be waited for then.  None
    // stands in a branch, at whose end the compiler would wait for all of them,
    // and the student's logits, behind the row in the queue, are looked at last.
    const int32_t* ip = a.index + (size_t)row * k;
    const float* vp = a.values + (size_t)row * k;
    const int32_t iv = ip[min(t, k - 1)];
    const float tv = vp[min(t, k - 1)];
    Run<IN> r[NH];
    int j0 = t * E;  // this thread's column in turn 0
    if (TINY)
      r[0].tiny(x, t == 0 ? V : 0);
    else
#pragma unroll
      for (int i = 0; i < NH; ++i) r[i].load(x, j0 + i * (nt * E), V);
    for (int i = t; i < at.bytes() / 16; i += nt) reinterpret_cast<uint4*>(marks)[i] = make_uint4(0, 0, 0, 0);
    if (t == 0) repeated = 0;
    __syncthreads();
    // entry j's token, or -1
    auto mark = [&](int j, int v) {
      token[j] = v >= 0 && v < V ? v : -1;
      if (v >= 0 && v < V) {
        const uint32_t b = at.bit(v);
        if (atomicOr(&marks[b >> 5], 1u << (b & 31)) >> (b & 31) & 1) repeated = 1;
      }
    };
    const bool here = t < k && iv >= 0 && iv < V;
    const float sv = load1<IN>(x, here ? iv : 0);
    if (t < k) mark(t, iv);
    for (int j = t + nt; j < k; j += nt) mark(j, ip[j]);
    __syncthreads();
    const int twice = __builtin_amdgcn_readfirstlane(repeated);  // some token is listed more than once
    // the rest's maximum and sum
    auto take = [&](Run<IN>& v, int i, uint32_t mask) {
      const int j = j0 + i * (nt * E);
      if (!TINY && (i + 1) * nt * E > V) v.cut(j, V);  // some of this turn's runs
      if (mask) v.drop(mask);
    };
    uint32_t mk[(MB + 3) / 4];
    __builtin_memcpy(mk, __builtin_assume_aligned(bytes + t * MB, MB & -MB), MB);
    RunSum acc;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      j0 = fresh(j0);
      take(r[i], i, E == 8 ? mk[i / 4] >> (i % 4 * 8) & 255 : mk[i / 8] >> (i % 8 * 4) & 15);
      r[i].forget();
      if (i == 0) {
        float first = r[0][0];
#pragma unroll
        for (int e = 1; e < E; ++e) first = fmaxf(first, r[0][e]);
        acc.ref = fmaxf(first * scale, RunSum::LOW);
      }
      acc.s += acc.sum(r[i], scale);
      acc.now();
      __builtin_amdgcn_sched_barrier(0);  // one run at a time: more would not fit the registers
    }
    // the runs behind those in registers, four on their way at a time
    auto stream = [&](auto&& f) {
      constexpr int AHEAD = 4;
      Run<IN> o[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        o[u].load(x, j0 + (NH + u) * (nt * E), V);
        __builtin_amdgcn_sched_barrier(0);  // in the order of the loop, whose waits count on it
      }
      for (int i = NH; i < turns; i += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (i + u < turns) {
            const int n = i + u - NH;
            const uint32_t b = bytes[nt * MB + (E == 8 ? n : n / 2) * nt + t];
            take(o[u], i + u, E == 8 ? b : b >> (n % 2 * 4) & 15);
            f(o[u], i + u);
          }
          o[u].load(x, j0 + (i + u + AHEAD) * (nt * E), V);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    if (MORE) stream([&](const Run<IN>& v, int) { acc.s += acc.sum(v, scale); });
    if (__any(!(acc.s < 0x1p40f))) {
      // a thread whose first run lies far below its others (masked, for one): once more, with a reference that follows
      acc = RunSum();
      float mx = -INFINITY;
      for (int i = 0; i < turns; ++i) {
        Run<IN> o;
        if (TINY) {
          o.tiny(x, t == 0 ? V : 0);
        } else {
          o.load(x, j0 + i * (nt * E), V);
        }
        const int n = i < NH ? i : i - NH, b = E == 8 ? n : n / 2;
        const uint32_t m = bytes[i < NH ? t * MB + b : nt * MB + b * nt + t];
        take(o, i, E == 8 ? m : m >> (n % 2 * 4) & 15);
        acc.add(o, scale, mx);
      }
    }
    // the list's maxima
    float tm = -INFINITY, sm = -INFINITY;
    auto entry = [&](int j, float y, float s) {
      student[j] = s;
      sm = fmaxf(sm, s);
      tm = y != y ? INFINITY : fmaxf(tm, y);  // fmaxf would lose a NaN
    };
    if (here) entry(t, tv, sv);
    for (int j = t + nt; j < k; j += nt)
      if (token[j] >= 0) entry(j, vp[j], load1<IN>(x, token[j]));
    const float wr = dpp_wave_fmax(acc.ref);
    const float ws = dpp_wave_fsum(acc.s * __builtin_amdgcn_exp2f(acc.ref - wr));
    tm = dpp_wave_fmax(tm), sm = dpp_wave_fmax(sm);
    if (lane == 0) fmx[wave] = make_float4(wr, ws, tm, sm);
    __syncthreads();
    const int from = min(lane & 15, nw - 1);
    const float4 wv = fmx[from];
    const float ref = row16_max(wv.x);
    float rest = row16_sum((lane & 15) < nw ? wv.y * __builtin_amdgcn_exp2f(wv.x - ref) : 0.0f);
    tm = row16_max(wv.z), sm = row16_max(wv.w);
    none = !a.top_lse && tm == -INFINITY;
    if (!none) {
      const double invT = 1.0 / (double)a.temperature;
      const double s0 = sm == -INFINITY ? 0.0 : (double)sm;
      // the logit that the rest's sum is relative to: of ref as the float32 factor takes it there
      double rm = (double)ref / (double)scale;
      bool slow = !(rest > 0.0f && rest < INFINITY);
      if (rest == 0.0f) {
        // nothing, or all of the rest is -inf
        bool any = false;
#pragma unroll
        for (int i = 0; i < NH; ++i) any |= r[i].any();
        if (MORE) stream([&](const Run<IN>& v, int) { any |= v.any(); });
        if (lane == 0) fany[wave] = 0.0f;
        if (__any(any) && lane == 0) fany[wave] = 1.0f;
        __syncthreads();
        slow = row16_max(fany[from]) > 0.0f;
      }
      float far = 0.0f;
      if (slow) {
        // relative to the maximum itself, read again, an element at a time
        auto each = [&](auto&& f) {
          for (int j = t; j < V; j += nt) {
            const uint32_t b = at.bit(j);
            if (!(marks[b >> 5] >> (b & 31) & 1)) f(load1<IN>(x, j));
          }
        };
        float m = -INFINITY, e = 0.0f;
        each([&](float v) { m = fmaxf(m, v); });
        m = dpp_wave_fmax(m);
        __syncthreads();
        if (lane == 0) fmx[wave].x = m;
        __syncthreads();
        far = row16_max(fmx[from].x);
        each([&](float v) { e += __builtin_amdgcn_exp2f((v - far) * scale); });
        e = dpp_wave_fsum(e);
        if (lane == 0) fmx[wave].y = e;
        __syncthreads();
        rest = row16_sum((lane & 15) < nw ? fmx[from].y : 0.0f);
        rm = (double)far;
      }
      double sum[3] = {0.0, 0.0, 0.0};  // listed, sum of p, sum of p (t - s) / T
      for (int j = t; j < k; j += nt) {
        if (token[j] < 0) continue;
        const double y = (double)(j == t ? tv : vp[j]) - (a.top_lse ? 0.0 : (double)tm), d = (double)student[j] - s0;
        const double p = exp(y * invT - (a.top_lse ? (double)tl : 0.0));
        prob[j] = p;
        // the first of a token listed more than once stands for its q
        bool first = true;
        if (twice)
          for (int o = 0; o < j; ++o) first &= token[o] != token[j];
        if (first) sum[0] += exp(d * invT);
        sum[1] += p;
        if (p != 0.0) sum[2] += p * ((y - d) * invT);
      }
      const int lw = (min(k, nt) + 63) >> 6;  // waves that have entries
      if (wave < lw) {
#pragma unroll
        for (int i = 0; i < 3; ++i) sum[i] = dpp_wave_sum(sum[i]);
        if (lane == 0)
#pragma unroll
          for (int i = 0; i < 3; ++i) dsum[i][wave] = sum[i];
      }
      __syncthreads();
      // what the row comes to: formed by one wave
      if (wave == 0) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          sum[i] = dsum[i][0];
          for (int o = 1; o < lw; ++o) sum[i] += dsum[i][o];
        }
        const double R0 = (double)rest;
        Row f;
        f.total = sum[1];
        f.dot = sum[2];
        f.norm = a.top_lse ? 1.0 : 1.0 / sum[1];
        // relative to the larger of the two maxima; lane 0 for the rest, the others for the list
        f.top = R0 == 0.0 ? s0 : sum[0] == 0.0 ? rm : fmax(rm, s0);
        const double part = lane == 0 ? R0 : sum[0];
        const double AB = part == 0.0 ? 0.0 : part * exp(((lane == 0 ? rm : s0) - f.top) * invT);
        const double A = __shfl(AB, 0);
        f.mass = A + __shfl(AB, 1);
        f.inv = f.mass == 0.0 ? 0.0 : 1.0 / f.mass;
        f.base = (f.top - s0) * invT - (a.top_lse ? (double)tl : 0.0);
        f.left = a.top_lse && R0 != 0.0 ? fmax(0.0, 1.0 - sum[1]) : 0.0;
        const double R = A == f.mass ? 1.0 : A * f.inv;  // exactly 1, as left is, for a list without entries
        f.coef = R0 == 0.0 ? 0.0f : (float)((double)w * invT * (R - f.left) / R0);
        // NaN somewhere in the teacher or the student, which the maximum above and a rest of 0 would hide
        const double all = sum[1] + f.mass + (a.top_lse ? (double)tl : 0.0);
        if (all != all) f.norm = NAN, f.coef = NAN;
        if (lane == 0) fin = f;
      }
      __syncthreads();
      if (grad) {
        const float coef = fin.coef;
        if (slow)
          for (int j = t; j < V; j += nt)
            store1<IN>(grad, j, __builtin_amdgcn_exp2f((load1<IN>(x, j) - far) * scale) * coef);
        auto put = [&](const Run<IN>& v, int i) {
          const int j = j0 + i * (nt * E);
          float o[8];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], scale, -ref)) * coef;
          uint32_t u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = IN == T_F32 ? __float_as_uint(o[e]) : pack_bf16(o[(2 * e) % E], o[(2 * e + 1) % E]);
          if ((i + 1) * nt * E <= V || j + E <= V) {
            store_through(grad + (uint32_t)(j * IB), u);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (j + e < V) store1<IN>(grad, j + e, o[e]);
          }
        };
        if (!slow) {
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            j0 = fresh(j0);
            r[i].forget();
            put(r[i], i);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (MORE) stream(put);
        }
        __syncthreads();  // the listed tokens' own values come after
        for (int j = t; j < k; j += nt) {
          if (token[j] < 0) continue;
          const int v = token[j];
          double p = prob[j];
          if (twice) {
            p = 0.0;
            for (int o = 0; o < k; ++o)
              if (token[o] == v) p += prob[o];
          }
          const double q = exp(((double)student[j] - fin.top) * invT) * fin.inv;
          store1<IN>(grad, v, (float)((double)w * invT * ((student[j] == -INFINITY ? 0.0 : q) - p * fin.norm)));
        }
      }
      if (a.loss && wave == nw - 1) {
        // four logarithms at once, a lane each
        const double of = lane == 0 ? fin.mass : lane == 1 ? fin.total : lane == 2 ? fin.left : (double)rest;
        const double lg = log(of);
        const double lm = __shfl(lg, 0), lp = __shfl(lg, 1), lr = __shfl(lg, 2), lR = __shfl(lg, 3);
        // log p_j - log q_j = (t_j - s_j) / T - log of the teacher's sum + log of the student's
        double loss = fin.dot * fin.norm;
        if (fin.total != 0.0 && loss != INFINITY) loss += fin.total * fin.norm * (fin.base + lm - (a.top_lse ? 0.0 : lp));
        if (fin.left > 0.0) loss += fin.left * (lr - ((rm - fin.top) * invT + lR - lm));
        if (lane == 0) a.loss[row] = (float)((double)w * loss);
      }
    }
  }
  if (none) {
    if (a.loss && t == 0) a.loss[row] = 0.0f;
    if (grad)
      for (int j = t * E; j < V; j += nt * E) {
        if (j + E <= V) {
          const uint32_t u[4] = {0, 0, 0, 0};
          store_through(grad + (size_t)j * IB, u);
        } else {
          for (int e = j; e < V; ++e) store1<IN>(grad, e, 0.0f);
        }
      }
  }
}

// Runs a thread in registers, and whole waves of threads to go with them.  Few
// runs and many threads make a row quick, many runs and few threads let a
// compute unit hold more rows (2, 4, 8 and 16 runs, bfloat16, lists of 64: 16384 x
// 1000 35, 41, 53, 79 us; 8192 x 4096 47, 39, 36, 50; 4096 x 11000 76, 63, 45, 53;
// 2048 x 32000 from 4 on 83, 59, 59, float32 104 with 16, 118 with 8).
struct DistillLaunch {
  int nt, nh;
  bool more;
  DistillLaunch(int V, int dtype) {
    const int e = dtype == SV_F32 ? 4 : 8, runs = (V + e - 1) / e;
    nh = runs <= 256 ? 2 : runs <= 2048 ? 8 : 16;
    nt = std::min(1024, ((runs + nh - 1) / nh + 63) / 64 * 64);
    more = runs > nt * nh;
  }
};

// What a launch takes at most: the longest list and the longest row, a bit a token.  Calls of several threads set the same
// limit: one of their own could lower another's between its setting and its launch.
constexpr int DISTILL_LDS = SV_MAX_TOP * 16 + SV_MAX_DISTILL_V / 8;

template <int IN, int NH, bool MORE, bool TINY>
hipError_t launch_distill(const DistillArgs& a, const DistillLaunch& l, hipStream_t s) {
  const Marks at{Run<IN>::E, l.nt, NH, MORE ? ((a.V + Run<IN>::E - 1) / Run<IN>::E + l.nt - 1) / l.nt : NH};
  const size_t lds = (size_t)a.k * 16 + (size_t)at.bytes();
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)distill_kernel<IN, NH, MORE, TINY>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, DISTILL_LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((distill_kernel<IN, NH, MORE, TINY>), dim3((unsigned)a.rows), dim3((unsigned)l.nt), lds, s, a);
  return hipGetLastError();
}

template <int IN>
hipError_t launch_distill(const DistillArgs& a, const DistillLaunch& l, hipStream_t s) {
  if (a.V < Run<IN>::E) return launch_distill<IN, 1, false, true>(a, l, s);
  if (l.more) return launch_distill<IN, 16, true, false>(a, l, s);
  return l.nh == 2 ? launch_distill<IN, 2, false, false>(a, l, s)
                   : l.nh == 8 ? launch_distill<IN, 8, false, false>(a, l, s) : launch_distill<IN, 16, false, false>(a, l, s);
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
  const DistillLaunch l(V, dtype);
  if ((int64_t)rows * l.nt > kGridThreads) return SV_ERR_SHAPE;
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
  const hipError_t err = dtype == SV_F32 ? launch_distill<T_F32>(a, l, (hipStream_t)stream)
                                         : launch_distill<T_BF16>(a, l, (hipStream_t)stream);
  return err == hipSuccess ? SV_OK : SV_ERR_HIP;
}
