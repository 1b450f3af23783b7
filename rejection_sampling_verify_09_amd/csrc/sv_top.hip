// The k largest logits of each row, their tokens, and the row's log-sum-exp at
// a temperature.
//
// Order: larger value first, among equal ones (-0 equals +0) the lower token;
// NaN above +infinity.
//
// One workgroup takes a row, in one pass: the sum of exponentials with a running
// reference, and the maximum of each of a thread's slots (four runs of 16 bytes,
// or a multiple).  A lower bound of the k-th largest value comes from the
// threads' maxima: of each wave's 64 the ceil(k / waves)-th largest, and of those
// the smallest, has at least k maxima at or above it.  The slots that reach it
// are read again, a few hundred runs, and what is at or above it goes to a list
// in LDS, where each entry's place is the number of entries before it in the
// order: all keys are unlike (value, then token), so no order of arrival shows.
// Where more reach the bound than the lists hold, because many equal it, those
// above it and the first equal ones are enough, if these lie among the row's
// first tokens (masked rows); otherwise (rows in order of their tokens) the k-th
// largest value itself is found by digits, reading the row for each.
//
// 2304 x 152064 float32 with k = 256 take 278 us (5.0 TB/s, a large copy's rate);
// 448 x 128256 bfloat16 with k = 64 31 us (3.7 TB/s), where the vector units are
// busy for 55% of the cycles (the exponentials above all) and the rest is the
// steps after the sums, one after another; one row 16 us, of which 7 are
// instructions.  What made the difference (448 x 128256 with k = 64): slot maxima
// and reading a few slots again instead of the row (123 -> 38 us); the wave's
// maxima taken out one by one instead of sorted, and bins in steps of the value
// instead of comparing all with all or a sort (36 -> 33; with k = 256 55 -> 38,
// and 70 before the sort); with k = 1000 a second bound instead of digits (215 ->
// 60).  Rows held in registers were not quicker: the lists' code on eight runs
// spills (2048 x 32000 198 us against 42).
#include "sv_rows.hpp"
#include "specverify.h"

#include <algorithm>
#include <cfloat>
#include <cmath>

namespace sv {

namespace {

constexpr int TOP_CAP = 2048;   // entries of the list, at most; at least 2 SV_MAX_TOP
constexpr int TOP_HITS = 2048;  // slots read again, at most
constexpr int TOP_SLOTS = 16;   // slots a thread, at most
constexpr int TOP_TURNS = 512;  // runs a thread, at most: SV_MAX_V / 4 runs on 1024 threads
constexpr int TOP_BINS = 512;
// Up to here the wave's maxima are taken out one by one (at most 14 instructions each), beyond it they are sorted (about
// 250): with 0, 8 and 32 448 x 128256 with k = 64 (4 a wave) takes 33.9, 32.9 and 33.3 us, with k = 256 (16) 38.9, 38.5, 39.9.
constexpr int TOP_TAKE = 8;
// Lists up to sqrt(16 threads) entries are ranked one against all, longer ones by bins: 4, 16 and 64 take 32.9, 32.9 and
// 34.1 us at 448 x 128256 with k = 64, 59, 60 and 66 at 8192 x 4096.
constexpr int TOP_RANK = 16;

struct TopArgs {
  const void* x;
  float* values;
  int32_t* index;
  float* lse;
  int32_t rows, V, k, turns, each, cap, hits;
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

// A row's launch: threads, runs a thread, and runs a slot.
struct TopShape {
  int nt, turns, each;
  TopShape(int V, int k, int e) {
    // Eight runs a thread: with four, a compute unit holds fewer rows (2048 x 32000 bfloat16, k = 64: 56 us against 41),
    // with sixteen a row takes longer (64 x 32000 13.7 against 11.7); of short rows fewer.  More threads for long lists,
    // whose bound is the better the more maxima there are (8192 x 4096, k = 64: 121 us with 64 threads, 59 with 256, 81
    // with 512), but none without a run.
    const int runs = (V + e - 1) / e, full = std::max(64, runs / 64 * 64);
    nt = std::min({1024, full, std::max({(runs / 8 + 63) / 64 * 64, (4 * k + 63) / 64 * 64, 128})});
    nt = std::max(nt, 64);
    turns = (runs + nt - 1) / nt;
    each = ((turns + 3) / 4 + TOP_SLOTS - 1) / TOP_SLOTS * 4;
  }
  int slots() const { return (turns + each - 1) / each; }
  // entries that the list holds: several times k, which is more than what reaches the bound as a rule, and no more than a
  // row has
  int cap(int V, int k) const {
    int n = 64;
    while (n < V && n < TOP_CAP && (n < 512 || n < 16 * k)) n <<= 1;
    return n;
  }
  int hits(int V, int k) const { return std::max(std::min(TOP_HITS, slots() * nt), cap(V, k) / 2); }
  size_t lds(int V, int k) const { return (size_t)cap(V, k) * 8 + (size_t)(hits(V, k) + slots() * nt) * 4; }
};

// A key's bin, of TOP_BINS: rising with the key from tau to rowmax, in equal
// steps of the value where both are finite, else of the key.
struct TopBins {
  uint32_t tau;
  float lo, mul;
  int sh;
  // (lower keys are in the first bin)
  __device__ __forceinline__ TopBins(uint32_t tau, uint32_t rowmax) : tau(tau) {
    lo = key_val(tau);
    const float width = key_val(rowmax) - lo;
    mul = width > 0.0f && width < INFINITY ? (float)TOP_BINS / width : 0.0f;
    if (!(mul > 0.0f && mul < INFINITY)) mul = 0.0f;
    sh = 0;
    while (rowmax > tau && (rowmax - tau) >> sh >= TOP_BINS) ++sh;
  }
  __device__ __forceinline__ int operator()(uint32_t key) const {
    if (key == 0xFFFFFFFFu) return TOP_BINS - 1;  // NaN
    if (mul > 0.0f) return (int)fminf(fmaxf((key_val(key) - lo) * mul, 0.0f), (float)(TOP_BINS - 1));
    return key < tau ? 0 : (int)min((key - tau) >> sh, (uint32_t)TOP_BINS - 1);
  }
};

// Counts of bins into how many stand in the bins above.
__device__ __forceinline__ void bins_before(int32_t* hist) {
  const int t = threadIdx.x;
  if (t >= 64) return;
  constexpr int PER = TOP_BINS / 64;  // lane l: the bins below TOP_BINS - PER l
  int c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) sum += c[i] = hist[TOP_BINS - 1 - t * PER - i];
  int before = (int)wave_scan_u32((uint32_t)sum) - sum;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    hist[TOP_BINS - 1 - t * PER - i] = before;
    before += c[i];
  }
}

// TINY: rows shorter than a run.
template <int IN, bool TINY>
__global__ void __launch_bounds__(1024) top_kernel(TopArgs a) {
  constexpr int E = Run<IN>::E;
  extern __shared__ uint64_t list[];  // [cap]
  __shared__ uint32_t bound[2][16];
  __shared__ float2 fsum[16];
  __shared__ int32_t hist[TOP_BINS];
  __shared__ int32_t wcount[16];
  __shared__ int32_t nlist, nabove, nat, pick, need, nans;
  __shared__ uint32_t found;
  const int cap = a.cap, mhits = a.hits;
  // [mhits] slots above the bound, then those at it; later the list's order
  uint32_t* hits = reinterpret_cast<uint32_t*>(list + cap);
  uint32_t* slot = hits + mhits;                             // [slots][nt] the slot's largest key
  const int t = threadIdx.x, nt = blockDim.x, nw = nt >> 6, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x, V = a.V, k = a.k, turns = a.turns, each = a.each, nslots = (turns + each - 1) / each;
  const char* x = static_cast<const char*>(a.x) + (size_t)row * V * Run<IN>::B;
  const float scale = LOG2E / a.temperature;
  // thread `by`'s run of turn i: f(the run, its first token, how many of its elements are the row's)
  auto rerun = [&](int i, int by, auto&& f) {
    const int j = (by + i * nt) * E;
    if (j >= V) return;
    Run<IN> r;
    if (TINY) {
      r.tiny(x, V);
    } else {
      r.load(x, j, V);
      r.cut(j, V);
    }
    f(r, j, min(V - j, E));
  };
  // the same, f(logit, token) for each
  auto again = [&](int i, int by, auto&& f) {
    rerun(i, by, [&](const Run<IN>& r, int j, int len) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < len) f(r[e], j + e);
    });
  };
  if (t == 0) nlist = nabove = nat = nans = 0;

  // one pass, four runs ahead
  RunSum sum;
  float sm = -INFINITY, m = -INFINITY;
  Run<IN> r[4];
  auto fetch = [&](Run<IN>& o, int i) {
    if (!TINY) o.load(x, (t + i * nt) * E, V);
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    fetch(r[u], u);
    __builtin_amdgcn_sched_barrier(0);  // in the order of the loop, whose waits count on it
  }
  if (TINY) r[0].tiny(x, t == 0 ? V : 0);
  for (int i = 0; i < turns; i += 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u < turns) {
        if (!TINY && (i + u + 1) * nt * E > V) r[u].cut((t + (i + u) * nt) * E, V);
        sum.add(r[u], scale, sm);
      }
      fetch(r[u], i + 4 + u);
    }
    if ((i + 4) % each == 0 || i + 4 >= turns) {
      slot[i / each * nt + t] = top_key(sm);
      m = fmaxf(m, sm);
      sm = -INFINITY;
    }
  }
  // NaN (or an infinity, or a logit that is as good as one) somewhere: the maxima may know nothing of it, so all of the
  // thread's slots are marked, to be looked at
  if (sum.s != sum.s)
    for (int s = 0; s < nslots; ++s) slot[s * nt + t] = 0xFFFFFFFFu;

  // the bound
  const uint32_t mk = top_key(m), wm = dpp_wave_umax(mk);
  const int c = (k + nw - 1) / nw;
  // the c-th largest of the wave's 64: the larger ones taken out one by one, or all put in order
  uint32_t cth = mk;
  if (c <= TOP_TAKE) {
    uint32_t v = mk;
    for (int i = 1; i < c; ++i) {
      const uint64_t same = __ballot(v == dpp_wave_umax(v));
      if (lane == __ffsll((long long)same) - 1) v = 0;
    }
    cth = dpp_wave_umax(v);
  } else if (c <= 64 && c > 64 - TOP_TAKE) {
    uint32_t v = ~mk;  // from the other end
    for (int i = 64; i > c; --i) {
      const uint64_t same = __ballot(v == dpp_wave_umax(v));
      if (lane == __ffsll((long long)same) - 1) v = 0;
    }
    cth = ~dpp_wave_umax(v);
  } else {
    cth = __shfl(wave_sort_desc(mk), min(c, 64) - 1);
  }
  const float wr = dpp_wave_fmax(sum.ref);
  const float ws = dpp_wave_fsum(sum.s * __builtin_amdgcn_exp2f(sum.ref - wr));
  if (lane == 0) {
    bound[0][wave] = wm;
    bound[1][wave] = c <= 64 ? cth : KEY_NEG_INF;  // fewer maxima than k: no bound
    fsum[wave] = make_float2(wr, ws);
  }
  __syncthreads();
  uint32_t rowmax = 0, tau = 0xFFFFFFFFu;
  for (int i = 0; i < nw; ++i) {
    rowmax = max(rowmax, bound[0][i]);
    tau = min(tau, bound[1][i]);
  }
  const float2 fs = fsum[min(lane & 15, nw - 1)];
  const float ref = row16_max(fs.x);
  float total = row16_sum((lane & 15) < nw ? fs.y * __builtin_amdgcn_exp2f(fs.x - ref) : 0.0f);

  if (a.lse) {
    const float top = key_val(rowmax);
    double base = (double)ref / (double)scale;
    const bool slow = !(total > 0.0f && total < INFINITY) && !(rowmax == KEY_NEG_INF && total == 0.0f);
    if (slow) {
      // NaN, infinities, or logits next to the type's largest or lowest value: relative to the maximum itself
      float e = 0.0f;
      int nan = 0;
      for (int i = 0; i < turns; ++i)
        again(i, t, [&](float v, int) {
          e += __builtin_amdgcn_exp2f((v - top) * scale);
          nan |= v != v;
        });
      e = dpp_wave_fsum(e);
      if (nan) nans = 1;
      __syncthreads();
      if (lane == 0) fsum[wave].y = e;
      __syncthreads();
      total = row16_sum((lane & 15) < nw ? fsum[min(lane & 15, nw - 1)].y : 0.0f);
      base = (double)top;
    }
    if (t == nt - 1) {  // beside the others' search
      float lse = (float)(base / (double)a.temperature + log((double)total));
      if (rowmax == KEY_NEG_INF || top == INFINITY) lse = top;
      if (slow && nans) lse = NAN;
      a.lse[row] = lse;
    }
  }
  auto push = [&](uint32_t key, int token) {
    const int at = atomicAdd(&nlist, 1);
    if (at < cap) list[at] = ((uint64_t)key << 32) | (uint32_t)~token;
  };
  auto collect = [&](int n, uint32_t over) {  // logits above `over` in the first n hits
    for (int h = t; h < n * each; h += nt) {
      const int id = (int)hits[h / each], s = id / nt, i = s * each + h % each;
      if (i < turns)
        rerun(i, id - s * nt, [&](const Run<IN>& r, int j, int len) {
          uint32_t key[E];
          int mine = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            key[e] = e < len ? top_key(r[e]) : 0;
            mine += key[e] > over;
          }
          if (mine == 0) return;
          int at = atomicAdd(&nlist, mine);
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (key[e] > over) {
              if (at < cap) list[at] = ((uint64_t)key[e] << 32) | (uint32_t)~(j + e);
              ++at;
            }
        });
    }
    __syncthreads();
  };
  // the slots that reach tau, those above it first, and their logits that do: how many, or more than cap
  int above = 0;
  auto gather = [&]() {
    for (int s = 0; s < nslots; ++s)
      if (slot[s * nt + t] > tau) {
        const int at = atomicAdd(&nabove, 1);
        if (at < mhits) hits[at] = (uint32_t)(s * nt + t);
      }
    __syncthreads();
    above = nabove;
    for (int s = 0; s < nslots; ++s)
      if (slot[s * nt + t] == tau) {
        const int at = above + atomicAdd(&nat, 1);
        if (at < mhits) hits[at] = (uint32_t)(s * nt + t);
      }
    __syncthreads();
    const int reach = above + nat;
    if (reach > mhits) return cap + 1;
    collect(reach, tau - 1);  // no key is below that of -inf
    return (int)nlist;
  };
  int n = gather();
  const uint32_t sure = tau;  // which at least k logits reach, whatever becomes of tau
  if (n > cap && c <= 64) {
    // a better bound: k of the slots' maxima reach it too (as a rule: marked slots are left out, and if fewer than k
    // others reach sure, all of them are above it)
    const TopBins bin(tau, rowmax);
    auto each_slot = [&](auto&& f) {
      for (int s = 0; s < nslots; ++s) {
        const uint32_t key = slot[s * nt + t];
        if (key >= tau && key != 0xFFFFFFFFu) f(key);
      }
    };
    __syncthreads();
    if (t == 0) nlist = nabove = nat = 0, found = 0xFFFFFFFFu;
    for (int i = t; i < TOP_BINS; i += nt) hist[i] = 0;
    __syncthreads();
    each_slot([&](uint32_t key) { atomicAdd(&hist[bin(key)], 1); });
    __syncthreads();
    bins_before(hist);
    __syncthreads();
    // bins before which fewer than k stand: of the last one that is not empty, all of it
    each_slot([&](uint32_t key) {
      if (hist[bin(key)] < k) atomicMin(&found, key);
    });
    __syncthreads();
    if (found != 0xFFFFFFFFu) tau = found;
    n = gather();
    if (n < k) {
      // fewer than k logits reach this one
      tau = sure;
      n = cap + 1;
      above = mhits + 1;
    }
  }
  if (n > cap && above <= mhits) {
    __syncthreads();
    if (t == 0) nlist = 0;
    __syncthreads();
    collect(above, tau);
    n = nlist;
    if (n < k) {
      // and those at the bound, among the first tokens
      __syncthreads();
      for (int j = t; j < min(V, cap - n); j += nt)
        if (top_key(load1<IN>(x, j)) == tau) push(tau, j);
      __syncthreads();
      n = nlist < k ? cap + 1 : nlist;
    }
  }
  if (n > cap) {
    // The k-th largest key, by digits, of the keys that reach the first bound: the second one may be reached by fewer
    // than k (its list was never formed where there were too many marked slots).
    uint32_t known = 0;
    int left = k;  // its place among those that begin with the known digits
    for (int s = 24; s >= 0; s -= 8) {
      __syncthreads();
      for (int i = t; i < 256; i += nt) hist[i] = 0;
      __syncthreads();
      for (int i = 0; i < turns; ++i)
        again(i, t, [&](float v, int) {
          const uint32_t key = top_key(v);
          if (key >= sure && (s == 24 || (key >> (s + 8)) == (known >> (s + 8)))) atomicAdd(&hist[(key >> s) & 255], 1);
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
    // what is above it, and as many of the equal ones as k leaves, by token
    int32_t* count = reinterpret_cast<int32_t*>(slot);  // the equal ones of each turn: at most 4 slots of 64 threads
    static_assert(TOP_TURNS <= 64 * TOP_SLOTS, "a word for each turn");
    __syncthreads();
    for (int i = t; i < turns; i += nt) count[i] = 0;
    if (t == 0) nlist = 0;
    __syncthreads();
    for (int i = 0; i < turns; ++i) {
      int eq = 0;
      again(i, t, [&](float v, int token) {
        const uint32_t key = top_key(v);
        if (key > known) push(key, token);
        eq += key == known;
      });
      if (eq) atomicAdd(&count[i], eq);
    }
    __syncthreads();
    left = k - nlist;
    int last = 0;  // the turn in which the equal ones reach k
    while (left > count[last]) left -= count[last++];
    __syncthreads();
    for (int i = 0; i < last; ++i)
      again(i, t, [&](float v, int token) {
        if (top_key(v) == known) push(known, token);
      });
    int eq = 0;
    again(last, t, [&](float v, int) { eq += top_key(v) == known; });
    const int before = (int)wave_scan_u32((uint32_t)eq) - eq;
    if (lane == 63) wcount[wave] = before + eq;
    __syncthreads();
    int at = before;
    for (int i = 0; i < wave; ++i) at += wcount[i];
    again(last, t, [&](float v, int token) {
      if (top_key(v) == known && at++ < left) push(known, token);
    });
    __syncthreads();
    n = nlist;
  }
  auto put = [&](uint64_t entry, int place) {
    const int token = (int)~(uint32_t)entry;
    const uint32_t key = (uint32_t)(entry >> 32);
    a.index[(size_t)row * k + place] = token;
    // a key is its logit, but for the sign of 0 and what a NaN holds
    a.values[(size_t)row * k + place] = key == ord_key(0.0f) || key == 0xFFFFFFFFu ? load1<IN>(x, token) : key_val(key);
  };
  if (n * n <= TOP_RANK * nt) {
    // each entry's place, by as many lanes as there are for it
    int lg = 0;
    while (lg < 4 && (n << (lg + 1)) <= nt) ++lg;
    const int by = 1 << lg;
    for (int i = t >> lg; i < n; i += nt >> lg) {
      const uint64_t mine = list[i];
      int place = 0;
      for (int o = t & (by - 1); o < n; o += by) place += list[o] > mine;
      for (int o = 1; o < by; o <<= 1) place += __shfl_xor(place, o);
      if ((t & (by - 1)) == 0 && place < k) put(mine, place);
    }
  } else {
    // by bins, the largest values first: an entry's place is where its bin begins, and the place within
    uint16_t* order = reinterpret_cast<uint16_t*>(hits);  // [cap]
    __syncthreads();
    for (int i = t; i < TOP_BINS; i += nt) hist[i] = 0;
    if (t == 0) found = rowmax;
    __syncthreads();
    // from the smallest one above -inf
    uint32_t least = 0xFFFFFFFFu;
    for (int i = t; i < n; i += nt) {
      const uint32_t key = (uint32_t)(list[i] >> 32);
      if (key > KEY_NEG_INF) least = min(least, key);
    }
    least = ~dpp_wave_umax(~least);
    if (lane == 0) atomicMin(&found, least);
    __syncthreads();
    const TopBins bin(found, rowmax);
    for (int i = t; i < n; i += nt) atomicAdd(&hist[bin((uint32_t)(list[i] >> 32))], 1);
    __syncthreads();
    bins_before(hist);
    __syncthreads();
    for (int i = t; i < n; i += nt) order[atomicAdd(&hist[bin((uint32_t)(list[i] >> 32))], 1)] = (uint16_t)i;
    __syncthreads();
    // each bin's count has moved on to where it ends
    for (int i = t; i < n; i += nt) {
      const uint64_t mine = list[order[i]];
      const int b = bin((uint32_t)(mine >> 32)), from = b == TOP_BINS - 1 ? 0 : hist[b + 1], to = hist[b];
      if (from >= k) continue;
      int place = from;
      for (int o = from; o < to; ++o) place += list[order[o]] > mine;
      if (place < k) put(mine, place);
    }
  }
}

// What a launch takes at most.  Calls of several threads set the same limit: one of their own could lower another's
// between its setting and its launch.
constexpr int TOP_LDS = TOP_CAP * 8 + (TOP_HITS + TOP_SLOTS * 1024) * 4;

template <int IN, bool TINY>
hipError_t launch_top(const TopArgs& a, const TopShape& l, hipStream_t s) {
  const size_t lds = l.lds(a.V, a.k);
  if (lds > 32 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)top_kernel<IN, TINY>, hipFuncAttributeMaxDynamicSharedMemorySize, TOP_LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((top_kernel<IN, TINY>), dim3((unsigned)a.rows), dim3((unsigned)l.nt), lds, s, a);
  return hipGetLastError();
}

template <int IN>
hipError_t launch_top(const TopArgs& a, const TopShape& l, hipStream_t s) {
  return a.V < Run<IN>::E ? launch_top<IN, true>(a, l, s) : launch_top<IN, false>(a, l, s);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_top_logits(const void* logits, int32_t k, float temperature, float* out_values, int32_t* out_index,
                             float* out_lse, int32_t rows, int32_t V, int32_t dtype, void* stream) {
  if (rows < 0 || V < 1 || V > SV_MAX_V || k < 1 || k > SV_MAX_TOP || k > V) return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  if (!(temperature >= FLT_MIN) || !std::isfinite(temperature)) return SV_ERR_PARAM;
  const TopShape l(V, k, dtype == SV_F32 ? 4 : 8);
  if ((int64_t)rows * l.nt > kGridThreads) return SV_ERR_SHAPE;
  if (rows == 0) return SV_OK;
  if (!logits || !out_values || !out_index) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), nin = (size_t)rows * (size_t)V * ie, no = (size_t)rows * (size_t)k * 4;
  const size_t nl = (size_t)rows * 4;
  if (!is_aligned(logits, ie) || !is_aligned(out_values, 4) || !is_aligned(out_index, 4) || !is_aligned(out_lse, 4))
    return SV_ERR_SHAPE;
  if (overlaps(out_values, no, logits, nin) || overlaps(out_index, no, logits, nin) || overlaps(out_lse, nl, logits, nin) ||
      overlaps(out_values, no, out_index, no) || overlaps(out_values, no, out_lse, nl) || overlaps(out_index, no, out_lse, nl))
    return SV_ERR_PARAM;
  const TopArgs a{logits, out_values, out_index, out_lse, rows, V, k, l.turns, l.each, l.cap(V, k), l.hits(V, k), temperature};
  const hipError_t err =
      dtype == SV_F32 ? launch_top<T_F32>(a, l, (hipStream_t)stream) : launch_top<T_BF16>(a, l, (hipStream_t)stream);
  return err == hipSuccess ? SV_OK : SV_ERR_HIP;
}
