// Penalties, biases and grammar masks on logits, before the filters and the
// draw.  For token j at a position with c_j occurrences among the sequence's
// output tokens (its history behind the prompt, and the drafts that stand
// before the position):
//   l = logit_j
//   l = l / rep (l > 0) or l * rep        if c_j > 0 or j is in the prompt
//   l = l - (freq c_j + pres)             if c_j > 0
//   l = l + the sum of j's biases, which are added to each other in their order
//   l = -inf                              if the row's mask forbids j
// in float32, rounded once to the logits' type.
//
// Split: a workgroup owns a slice of the vocabulary of one sequence, counts
// the sequence's tokens that fall into it in an LDS table (integer atomics:
// no order changes a count), and then handles the slice of each of the
// sequence's rows.  The history is read once per slice, from the L2.
//
// Bound by memory.  Out of place every logit is read and written once, 16
// bytes a lane, four rows' loads in flight, the first of them under way while
// the table is built: 256 x 9 float32 rows of 152064 with histories of 8192
// and masks take 497 us (5.7 TB/s; a large copy reaches 5.1), 64 x 7 bfloat16
// rows of 128256 55 us (4.2 TB/s).  There the arithmetic shows: a branch per
// touched token, with a division in it, took 73 us, the branch-free form on 8
// tokens a lane 59, the drafted and biased ones alone one by one 55.  In place
// only what changes is touched: the list of the slice's tokens, and the runs of
// 8 that a mask cuts (the same 64 x 7 rows: 30 us, whose scattered logits lie in
// half of all lines; masks alone on 32 x 7 rows: 14.6 us, in which 38 MB are
// written and 30 read, 4.7 TB/s: a run that loses some of its tokens is read and
// written whole).
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>

namespace sv {

namespace {

struct AdjArgs {
  const void* in;
  void* out;
  const int32_t* hist;    // [B, cap]
  const int32_t* hlen;    // [B] or null (cap)
  const int32_t* plen;    // [B] or null (0)
  const int32_t* drafts;  // [B, K], or packed [N]
  const int32_t* cu;      // [B + 1] offsets of a ragged batch, or null
  const float *rep, *freq, *pres;  // [B] each or null
  const int32_t* cub;     // [B + 1] offsets of the biases, or null
  const int32_t* btok;
  const float* bval;
  const uint32_t* mask;   // [mask_rows, words], or null
  const int32_t* midx;    // [rows], or null (row r has mask r)
  int32_t B, R, K, seen, V, cap, nbias, mask_rows, words;
  int32_t N, max_k, bonus;  // ragged: drafts in all, the most of one sequence, rows past them (0 or 1)
  int32_t bcap;             // a slice's biases held in LDS (at most 16 a thread)
  int32_t nslices, rgroup;  // slices of the vocabulary; rows of a sequence per workgroup
};

// Table entry: occurrences in the low bits, and what else is known of the token.
constexpr uint32_t E_PROMPT = 1u << 31, E_DRAFT = 1u << 30, E_BIAS = 1u << 29, E_BIASES = 1u << 28;
constexpr int E_SHIFT = 22;  // six bits: of a drafted token, the first draft that is it
constexpr uint32_t E_COUNT = (1u << E_SHIFT) - 1;
static_assert(SV_MAX_HISTORY <= E_COUNT && MAX_K <= 64, "counts and drafts fit an entry");
constexpr uint16_t NONE = 0xFFFFu;
constexpr int ADJ_MAX_WG = 1024, ADJ_EPT = 8;  // a thread has 8 tokens of the slice

// What a sequence's c occurrences of a token take off its logit.
__device__ __forceinline__ float penalty(float c, float freq, float pres) { return c > 0.0f ? freq * c + pres : 0.0f; }

// One logit of a row: e its table entry, c further occurrences among the
// drafts; rinv = 1 / rep, which the positive logits are multiplied by (one
// rounding more than a division and a fifth of its instructions).
__device__ __forceinline__ float adjusted(float l, uint32_t e, float bias, float c, float rep, float rinv, float freq,
                                          float pres) {
  c += (float)(e & E_COUNT);
  if (c > 0.0f || (e & E_PROMPT)) l *= l > 0.0f ? rinv : rep;
  l -= penalty(c, freq, pres);
  if (e & E_BIAS) l += bias;
  return l;
}

// Eight logits as 32-bit words: one each (float32) or two in one (bfloat16).
template <int DT>
struct Eight {
  static constexpr int W = DT == T_F32 ? 8 : 4;
  uint32_t w[W];
  __device__ __forceinline__ float get(int k) const {
    return DT == T_F32 ? __uint_as_float(w[k]) : (k & 1) ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
  }
  // Element k, in a register that only run time knows: by masks (a choice
  // between the words would put them into memory).
  __device__ __forceinline__ float pick(int k) const {
    const int word = DT == T_F32 ? k : k >> 1;
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) v |= w[i] & (word == i ? ~0u : 0u);
    return DT == T_F32 ? __uint_as_float(v) : (k & 1) ? bf16_hi(v) : bf16_lo(v);
  }
  __device__ __forceinline__ void put(int k, float f) {
    const int word = DT == T_F32 ? k : k >> 1;
    const uint32_t b = DT == T_F32 ? __float_as_uint(f) : (uint32_t)to_bf16(f) << (k & 1 ? 16 : 0);
    const uint32_t part = DT == T_F32 ? ~0u : k & 1 ? 0xFFFF0000u : 0xFFFFu;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t on = word == i ? part : 0u;
      w[i] = (w[i] & ~on) | (b & on);
    }
  }
  // n < 8: the first n of them, the others 0.  Rows may start at any element
  // (the hardware splits a 16-byte access where it crosses a boundary).
  __device__ __forceinline__ void load(const char* p, int n) {
    if (n >= 8) {
      __builtin_memcpy(w, p, sizeof w);
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          if (DT == T_F32)
            w[k] = reinterpret_cast<const uint32_t*>(p)[k];
          else
            w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[k] << (k & 1 ? 16 : 0);
        }
    }
  }
  // -inf where m has a 0 bit
  __device__ __forceinline__ void forbid(uint32_t m) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t on = (uint32_t)((int32_t)(m << (31 - k)) >> 31);  // all ones where allowed
      if (DT == T_F32) {
        w[k] = (w[k] & on) | (0xFF800000u & ~on);
      } else {
        const uint32_t keep = on | ((k & 1) ? 0xFFFFu : 0xFFFF0000u);
        w[k / 2] = (w[k / 2] & keep) | (0xFF80FF80u & ~keep);
      }
    }
  }
  __device__ __forceinline__ void store(char* p, int n) const {
    if (n >= 8) {
      __builtin_memcpy(p, w, sizeof w);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          if (DT == T_F32)
            reinterpret_cast<uint32_t*>(p)[k] = w[k];
          else
            reinterpret_cast<uint16_t*>(p)[k] = (uint16_t)(w[k / 2] >> (k & 1 ? 16 : 0));
        }
    }
  }
};
template <int DT>
__device__ __forceinline__ void store1(char* p, int k, float v) {
  if (DT == T_F32)
    reinterpret_cast<float*>(p)[k] = v;
  else
    reinterpret_cast<uint16_t*>(p)[k] = to_bf16(v);
}
// The byte of row r's mask that holds token v0 + 8t .. + 7 (all ones where the
// row has no mask).
__device__ __forceinline__ const uint8_t* mask_row(const AdjArgs& a, size_t row) {
  if (!a.mask) return nullptr;
  const int64_t mi = a.midx ? (int64_t)a.midx[row] : (int64_t)row;
  if (mi < 0 || mi >= a.mask_rows) return nullptr;
  return reinterpret_cast<const uint8_t*>(a.mask + (size_t)mi * a.words);
}

// INPLACE: out is the input, and only logits that change are read or written.
template <int DT, bool INPLACE>
__global__ void __launch_bounds__(ADJ_MAX_WG) adjust_kernel(AdjArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t smem[];
  const int t = threadIdx.x, nt = blockDim.x, S = nt * ADJ_EPT;
  uint32_t* tab = smem;                                           // [S]
  uint32_t* bt = smem + S;                                        // [S] with biases: head of the token's chain, then the sum
  float* bvals = reinterpret_cast<float*>(smem + 2 * S);          // [bcap] with biases: values of the slice's,
  int32_t* bidx = reinterpret_cast<int32_t*>(bvals + a.bcap);     // [bcap] their indices,
  uint16_t* btoks = reinterpret_cast<uint16_t*>(bidx + a.bcap);   // [bcap] their tokens
  uint16_t* bnext = btoks + a.bcap;                               // [bcap] and another of the same token
  uint16_t* list = a.cub ? bnext + a.bcap : reinterpret_cast<uint16_t*>(smem + S);  // [S] in place: tokens of nonzero entries
  __shared__ int32_t xs[MAX_K];                                   // the sequence's drafts,
  __shared__ uint64_t same[MAX_K];                                // and which of them are the same token
  __shared__ int32_t nlist, nbiased, nordered;
  __shared__ int32_t wcount[ADJ_MAX_WG / 64];
  const int b = blockIdx.x / a.nslices, sl = blockIdx.x - b * a.nslices;
  const int v0 = sl * S, vn = min(S, a.V - v0);
  constexpr int EB = DT == T_F32 ? 4 : 2;

  // the sequence's rows and drafts
  int64_t row0, d0;
  int nr, nd;
  if (a.cu) {
    int bad = 0;
    for (int i = t; i <= a.B; i += nt) {
      const int c = a.cu[i];
      if (i == 0) bad |= c != 0;
      if (i == a.B) bad |= c != a.N;
      if (i > 0) {
        const int64_t k = (int64_t)c - a.cu[i - 1];
        bad |= k < 0 || k > a.max_k;
      }
    }
    if (__syncthreads_or(bad)) return;  // offsets that describe no packing: no row is written
    d0 = a.cu[b];
    nd = a.cu[b + 1] - a.cu[b];
    row0 = d0 + (int64_t)b * a.bonus;
    nr = nd + a.bonus;
    if ((int)(blockIdx.y * a.rgroup) >= nr) return;  // fewer groups of rows than the longest sequence has
  } else {
    d0 = (int64_t)b * a.K;
    nd = a.K;
    row0 = (int64_t)b * a.R;
    nr = a.R;
  }
  nd = min(nd, a.seen + nr - 1);  // drafts that some row has seen

  const bool counts = a.rep || a.freq || a.pres;
  const bool table = counts || a.cub;
  const int r0 = blockIdx.y * a.rgroup, r1 = min(nr, r0 + a.rgroup);
  const size_t pitch = (size_t)a.V * EB;

  // what the table takes, loaded ahead of the rows
  const float rep = a.rep ? a.rep[b] : 1.0f, freq = a.freq ? a.freq[b] : 0.0f, pres = a.pres ? a.pres[b] : 0.0f;
  const float rinv = 1.0f / rep;
  const int nh = !counts || !a.hist ? 0 : a.hlen ? min(max(a.hlen[b], 0), a.cap) : a.cap;
  const int np = nh && a.plen ? min(max(a.plen[b], 0), nh) : 0;
  const int32_t draft = counts && t < nd ? a.drafts[d0 + t] : -1;

  // Out of place: this thread's 8 tokens of every row, UN rows' loads in
  // flight; the first ones are under way while the table is built
  constexpr int UN = 4;
  const int n = min(8, vn - 8 * t), vt = v0 + 8 * t;
  uint32_t m[UN];
  Eight<DT> l[UN];
  auto masks = [&](uint32_t (&q)[UN], int r) {  // the rows' mask bytes of these tokens
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      q[u] = 0xFFu;
      if (a.mask && r + u < r1) {
        const uint8_t* mask = mask_row(a, (size_t)(row0 + r + u));
        if (mask) q[u] = mask[vt >> 3];
      }
    }
  };
  auto fetch = [&](int r) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (r + u < r1 && m[u])
        l[u].load(static_cast<const char*>(a.in) + (size_t)(row0 + r + u) * pitch + (size_t)vt * EB, n);
  };
  if (!INPLACE && n > 0) {
    masks(m, r0);
    fetch(r0);
  }
  // the sequence's ne biases, a thread's first in registers (positions are
  // unsigned: a few past the last one are formed, which 32 bits hold then)
  const int32_t* btl = nullptr;
  const float* bvl = nullptr;
  uint32_t ne = 0;
  int btok0 = 0;
  float bval0 = 0.0f;
  if (a.cub) {
    const int i0 = min(max(a.cub[b], 0), a.nbias);
    const int i1 = min(a.cub[b + 1], a.nbias);
    ne = (uint32_t)(max(i1, i0) - i0);
    btl = a.btok + i0;
    bvl = a.bval + i0;
    if ((uint32_t)t < ne) {
      btok0 = btl[t];
      bval0 = bvl[t];
    }
  }
  if (table) {
    for (int i = t; i < S / 4; i += nt) {
      reinterpret_cast<uint4*>(tab)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.cub) reinterpret_cast<uint4*>(bt)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    }
    if (t == 0) nlist = nbiased = nordered = 0;
    __syncthreads();
  }
  // every entry becomes nonzero once, by whichever operation comes first: that thread lists the token
  auto touch = [&](uint32_t j, uint32_t old) {
    if (INPLACE && old == 0) list[atomicAdd(&nlist, 1)] = (uint16_t)j;
  };
  if (counts) {
    if (a.hist) {
      const int32_t* h = a.hist + (size_t)b * a.cap;
      auto count = [&](int i, int32_t tok) {
        const uint32_t j = (uint32_t)tok - (uint32_t)v0;
        if (j < (uint32_t)vn) touch(j, i < np ? atomicOr(&tab[j], E_PROMPT) : atomicAdd(&tab[j], 1u));
      };
      // 16-byte loads, four in flight
      constexpr int HN = 4;
      for (int i = 4 * t; i < nh; i += 4 * HN * nt) {
        int32_t q[HN][4];
#pragma unroll
        for (int u = 0; u < HN; ++u) {
          const int p = i + 4 * u * nt;
          if (p + 4 <= nh) {
            __builtin_memcpy(q[u], h + p, 16);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) q[u][k] = p + k < nh ? h[p + k] : -1;
          }
        }
#pragma unroll
        for (int u = 0; u < HN; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) count(i + 4 * u * nt + k, q[u][k]);
      }
    }
    if (t < nd) xs[t] = draft;
    __syncthreads();
    if (t < nd) {
      uint64_t m = 0;
      for (int k = 0; k < nd; ++k) m |= (uint64_t)(xs[k] == xs[t]) << k;
      same[t] = m;
      const uint32_t j = (uint32_t)xs[t] - (uint32_t)v0;
      if (j < (uint32_t)vn && !(m & ((1ull << t) - 1))) touch(j, atomicOr(&tab[j], E_DRAFT | (uint32_t)t << E_SHIFT));
    }
  }
  if (a.cub) {
    // several biases of one token are added in the order they are listed, by
    // the thread that holds the first or, of a chain, its head; those of
    // E_BIASES tokens by a walk through the list
    for (uint32_t i = t; i < ne; i += nt) {
      const uint32_t j = (uint32_t)(i == (uint32_t)t ? btok0 : btl[i]) - (uint32_t)v0;
      if (j >= (uint32_t)vn) continue;
      const int p = atomicAdd(&nbiased, 1);
      if (p < a.bcap) {
        bidx[p] = (int32_t)i;
        btoks[p] = (uint16_t)j;
        bvals[p] = i == (uint32_t)t ? bval0 : bvl[i];
        bnext[p] = (uint16_t)atomicExch(&bt[j], (uint32_t)p);
      }
    }
    __syncthreads();
    const int nb = nbiased;
    if (nb <= a.bcap) {
      // the slice's biases in LDS, each token's chained, both in any order:
      // a chain's head takes the lowest index left until none is, or leaves a
      // long chain to the walk
      uint32_t head = 0;
      for (int p = t, c = 0; p < nb; p += nt, ++c)
        if (bt[btoks[p]] == (uint32_t)p) head |= 1u << c;
      __syncthreads();  // the sums take the heads' place
      for (int p = t, c = 0; p < nb; p += nt, ++c) {
        if (!((head >> c) & 1)) continue;
        const int j = btoks[p];
        float v = bvals[p];
        uint32_t bits = E_BIAS;
        if (bnext[p] != NONE) {
          constexpr int LONG = 17;
          int len = 0;
          for (int k = p; k != NONE && len < LONG; k = bnext[k]) ++len;
          bool any = false;
          if (len < LONG) {
            for (int q = 0, last = -1; q < len; ++q) {
              int low = INT32_MAX, at = p;
              for (int k = p; k != NONE; k = bnext[k])
                if (bidx[k] > last && bidx[k] < low) low = bidx[k], at = k;
              v = any ? v + bvals[at] : bvals[at];
              any = true;
              last = low;
            }
          } else {
            bits |= E_BIASES;
            nordered = 1;
          }
        }
        bt[j] = __float_as_uint(v);
        touch(j, atomicOr(&tab[j], bits));
      }
    } else {
      // too many: bt first takes the index of each token's first
      for (int i = t; i < S; i += nt) bt[i] = ~0u;
      __syncthreads();
      for (uint32_t i = t; i < ne; i += nt) {
        const uint32_t j = (uint32_t)btl[i] - (uint32_t)v0;
        if (j >= (uint32_t)vn) continue;
        atomicMin(&bt[j], i);
        touch(j, atomicOr(&tab[j], E_BIAS));
      }
      __syncthreads();
      for (uint32_t i = t; i < ne; i += nt) {
        const uint32_t j = (uint32_t)btl[i] - (uint32_t)v0;
        if (j < (uint32_t)vn && bt[j] != i) {
          atomicOr(&tab[j], E_BIASES);
          nordered = 1;
        }
      }
      __syncthreads();
      for (uint32_t i = t; i < ne; i += nt) {
        const uint32_t j = (uint32_t)btl[i] - (uint32_t)v0;
        if (j < (uint32_t)vn && !(tab[j] & E_BIASES)) bt[j] = __float_as_uint(bvl[i]);
      }
    }
    __syncthreads();
    if (nordered) {
      // The walk: of each piece of the list the E_BIASES tokens' entries are
      // brought together, in order, and every thread adds those of its 8
      // tokens.  Time grows with the list's length alone, however often a
      // token is in it.
      const int piece = min(nt, a.bcap);
      uint32_t begun = 0;  // which of the thread's tokens have a sum
      for (uint32_t base = 0; base < ne; base += piece) {
        const uint32_t i = base + t;
        uint32_t j = 0;
        bool mine = false;
        if (t < piece && i < ne) {
          j = (uint32_t)btl[i] - (uint32_t)v0;
          mine = j < (uint32_t)vn && (tab[j] & E_BIASES);
        }
        const uint64_t m = __ballot(mine);
        if ((t & 63) == 0) wcount[t >> 6] = __popcll(m);
        __syncthreads();
        int at = __popcll(m & ((1ull << (t & 63)) - 1)), total = 0;
        for (int w = 0; w < nt >> 6; ++w) {
          const int c = wcount[w];
          at += w < t >> 6 ? c : 0;
          total += c;
        }
        if (mine) {
          btoks[at] = (uint16_t)j;
          bvals[at] = bvl[i];
        }
        __syncthreads();
        for (int p = 0; p < total; ++p) {
          const int q = btoks[p];
          if (q / ADJ_EPT != t) continue;
          const uint32_t bit = 1u << q % ADJ_EPT;
          bt[q] = __float_as_uint(begun & bit ? __uint_as_float(bt[q]) + bvals[p] : bvals[p]);
          begun |= bit;
        }
        __syncthreads();  // the next piece takes its place
      }
    }
  } else if (table) {
    __syncthreads();
  }

  const bool biased = a.cub != nullptr;
  // a token's logit in a row that has seen the drafts in `seen`: table entry e, bias w
  auto fix = [&](float l, uint32_t e, uint32_t w, uint64_t seen) {
    const float c = e & E_DRAFT ? (float)__popcll(same[(e >> E_SHIFT) & 63] & seen) : 0.0f;
    return adjusted(l, e, __uint_as_float(w), c, rep, rinv, freq, pres);
  };
  auto seen_by = [&](int r) {
    const int k = a.seen + r;
    return k >= 64 ? ~0ull : (1ull << k) - 1;
  };

  if (INPLACE) {
    char* out = static_cast<char*>(a.out) + (size_t)row0 * pitch;
    if (a.mask) {
      // runs of 8 that lose some of their tokens are read and written whole,
      // those that lose all only written
      for (int r = r0; n > 0 && r < r1; r += UN) {
        char* p = out + (size_t)r * pitch + (size_t)vt * EB;
        masks(m, r);
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (m[u] != 0 && m[u] != 0xFFu) l[u].load(p + (size_t)u * pitch, n);
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (m[u] != 0xFFu) {
            l[u].forbid(m[u]);
            l[u].store(p + (size_t)u * pitch, n);
          }
      }
      if (table) __syncthreads();  // the list's logits lie in those runs
    }
    // P threads a row (a power of two that covers the list where it is short,
    // at most all of them), G rows at a time
    const int nl = table ? nlist : 0;
    int P = 1;
    while (P < nl && P < nt) P *= 2;
    P = min(P, nt);
    const int G = nt / P;
    for (int r = r0 + t / P; nl > 0 && t < G * P && r < r1; r += G) {
      const uint8_t* mask = mask_row(a, (size_t)(row0 + r));
      for (int q = t % P; q < nl; q += P) {
        const int j = list[q], v = v0 + j;
        if (mask && !((mask[v >> 3] >> (v & 7)) & 1)) continue;
        char* p = out + (size_t)r * pitch;
        const float x = DT == T_F32 ? reinterpret_cast<const float*>(p)[v]
                                    : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[v] << 16);
        store1<DT>(p, v, fix(x, tab[j], biased ? bt[j] : 0u, seen_by(r)));
      }
    }
    return;
  }

  if (n <= 0) return;
  // Per token once for all rows: what its count takes off (sub), and the bits
  // of the words it changes (sel).  Every wave of a sequence with a history
  // has such tokens, so the common ones are handled without a branch, and
  // then the drafted and biased ones (odd) one by one.
  float sub[8];
  uint32_t sel[Eight<DT>::W], odd = 0;
  bool any = false;
#pragma unroll
  for (int k = 0; k < Eight<DT>::W; ++k) sel[k] = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t e = table ? tab[8 * t + k] : 0u;
    const bool own = e & (E_DRAFT | E_BIAS), plain = e && !own;
    sub[k] = penalty((float)(e & E_COUNT), freq, pres);
    any |= plain;
    if (own) odd |= 1u << k;
    if (DT == T_F32)
      sel[k] = plain ? ~0u : 0u;
    else if (plain)
      sel[k / 2] |= (k & 1) ? 0xFFFF0000u : 0xFFFFu;
  }
  char* out = static_cast<char*>(a.out) + (size_t)row0 * pitch + (size_t)vt * EB;
  for (int r = r0; r < r1; r += UN) {
    if (r > r0) fetch(r);
    uint32_t next[UN];  // a load ahead: the logits' loads wait for them
    masks(next, r + UN);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (r + u >= r1) continue;
      if (any) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x = l[u].get(k);
          f[k] = x * (x > 0.0f ? rinv : rep) - sub[k];
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          if (DT == T_F32) {
            l[u].w[k] = (__float_as_uint(f[k]) & sel[k]) | (l[u].w[k] & ~sel[k]);
            l[u].w[k + 1] = (__float_as_uint(f[k + 1]) & sel[k + 1]) | (l[u].w[k + 1] & ~sel[k + 1]);
          } else {
            l[u].w[k / 2] = (pack_bf16(f[k], f[k + 1]) & sel[k / 2]) | (l[u].w[k / 2] & ~sel[k / 2]);
          }
        }
      }
      for (uint32_t q = odd; q; q &= q - 1) {
        const int k = __builtin_ctz(q);
        l[u].put(k, fix(l[u].pick(k), tab[8 * t + k], biased ? bt[8 * t + k] : 0u, seen_by(r + u)));
      }
      if (m[u] != 0xFFu) l[u].forbid(m[u]);
      l[u].store(out + (size_t)(r + u) * pitch, n);
    }
#pragma unroll
    for (int u = 0; u < UN; ++u) m[u] = next[u];
  }
}

template <int DT>
hipError_t launch_adjust(AdjArgs a, int32_t rows_per_seq, hipStream_t s) {
  const bool inplace = a.in == a.out;
  // Slices of 2048 tokens, smaller where the sequences are few.  Small slices
  // overlap one workgroup's table with the others' rows, large ones read the
  // history less often: 64 sequences of 7 bfloat16 rows of 128256 take 60, 56,
  // 60 and 66 us with 1024, 2048, 4096 and 8192 tokens a slice where the
  // histories are up to 4096 long, and 150, 106, 91 and 84 us at 65536.
  const int most = a.cap > 16384 ? ADJ_MAX_WG : 256;
  int nt = std::min(most, std::max(64, ((a.V + ADJ_EPT - 1) / ADJ_EPT + 63) / 64 * 64));
  auto slices = [&](int n) { return (a.V + n * ADJ_EPT - 1) / (n * ADJ_EPT); };
  while (a.cap <= 16384 && nt == 256 && (int64_t)a.B * slices(nt) < 512) nt = 128;
  a.nslices = slices(nt);
  const int64_t wgs = (int64_t)a.B * a.nslices;
  const int groups = (int)std::max<int64_t>(1, std::min<int64_t>(2048 / wgs, (rows_per_seq + 3) / 4));
  a.rgroup = (rows_per_seq + groups - 1) / groups;
  const dim3 grid((unsigned)wgs, (unsigned)((rows_per_seq + a.rgroup - 1) / a.rgroup));
  // Room for twice the biases that a slice has on average: less of it leaves
  // the compute unit room for more workgroups (128 x 11 bfloat16 rows of 24979
  // with 300 biases each: 45 us with room for 1024, 37 with 384).
  const int64_t biases = 2 * (int64_t)a.nbias / wgs;
  a.bcap = (int)std::min<int64_t>(1024, std::max<int64_t>(384, biases));
  const size_t S = (size_t)nt * ADJ_EPT;
  const bool table = a.rep || a.freq || a.pres || a.cub;
  const size_t lds = table ? S * 4 * (a.cub ? 2 : 1) + (a.cub ? (size_t)a.bcap * 12 : 0) + (inplace ? S * 2 : 0) : 0;
  if (inplace)
    hipLaunchKernelGGL((adjust_kernel<DT, true>), grid, dim3(nt), lds, s, a);
  else
    hipLaunchKernelGGL((adjust_kernel<DT, false>), grid, dim3(nt), lds, s, a);
  return hipGetLastError();
}

constexpr int64_t kMaxRows = int64_t(1) << 30;  // row numbers a few rows past the last are formed in 32 bits

size_t words_of(int32_t V) { return ((size_t)V + 31) / 32; }

int check_and_launch(AdjArgs& a, int64_t rows, int32_t dtype, void* stream) {
  const int32_t V = a.V;
  if (a.B < 0 || rows < 0 || V < 1 || V > MAX_V || a.cap < 0 || a.cap > SV_MAX_HISTORY || a.nbias < 0 ||
      a.mask_rows < 0)
    return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  // a thread for every 8 tokens, the last of a sequence's workgroups filled up
  if ((int64_t)a.B * (V / ADJ_EPT + ADJ_MAX_WG) > kGridThreads || rows > kMaxRows) return SV_ERR_SHAPE;
  const size_t oe = (size_t)type_bytes(dtype);
  if (!is_aligned(a.in, oe) || !is_aligned(a.out, oe) || !is_aligned(a.hist, 4) || !is_aligned(a.hlen, 4) ||
      !is_aligned(a.plen, 4) || !is_aligned(a.drafts, 4) || !is_aligned(a.cu, 4) || !is_aligned(a.rep, 4) ||
      !is_aligned(a.freq, 4) || !is_aligned(a.pres, 4) || !is_aligned(a.cub, 4) || !is_aligned(a.btok, 4) ||
      !is_aligned(a.bval, 4) || !is_aligned(a.mask, 4) || !is_aligned(a.midx, 4))
    return SV_ERR_SHAPE;
  if (a.B == 0 || rows == 0) return SV_OK;
  const int64_t drafts = a.cu ? a.N : (int64_t)a.B * a.K;
  const bool counts = a.rep || a.freq || a.pres;
  if (!a.in || !a.out) return SV_ERR_NULL;
  if (counts && a.cap > 0 && !a.hist) return SV_ERR_NULL;
  if (counts && drafts > 0 && !a.drafts) return SV_ERR_NULL;
  if (a.cub && a.nbias > 0 && (!a.btok || !a.bval)) return SV_ERR_NULL;
  if (a.mask && !a.midx && a.mask_rows != rows) return SV_ERR_SHAPE;
  // the logits may be adjusted in place; any other overlap of the output is refused
  const size_t no = (size_t)rows * (size_t)V * oe, B4 = (size_t)a.B * 4;
  if ((a.out != a.in && overlaps(a.out, no, a.in, no)) || overlaps(a.out, no, a.hist, B4 * a.cap) ||
      overlaps(a.out, no, a.hlen, B4) || overlaps(a.out, no, a.plen, B4) ||
      overlaps(a.out, no, a.drafts, (size_t)drafts * 4) || overlaps(a.out, no, a.cu, B4 + 4) ||
      overlaps(a.out, no, a.rep, B4) || overlaps(a.out, no, a.freq, B4) || overlaps(a.out, no, a.pres, B4) ||
      overlaps(a.out, no, a.cub, B4 + 4) || overlaps(a.out, no, a.btok, (size_t)a.nbias * 4) ||
      overlaps(a.out, no, a.bval, (size_t)a.nbias * 4) ||
      overlaps(a.out, no, a.mask, (size_t)a.mask_rows * words_of(V) * 4) ||
      overlaps(a.out, no, a.midx, (size_t)rows * 4))
    return SV_ERR_PARAM;
  a.words = (int32_t)words_of(V);
  if (a.cap == 0) a.hist = nullptr;
  if (a.nbias == 0) a.cub = nullptr;
  if (a.mask_rows == 0) a.mask = nullptr;
  if (a.in == a.out && !counts && !a.cub && !a.mask) return SV_OK;
  const int32_t rps = a.cu ? a.max_k + a.bonus : a.R;  // most rows of a sequence
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == SV_F32 ? launch_adjust<T_F32>(a, rps, s) : launch_adjust<T_BF16>(a, rps, s);
  return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

int sv_adjust_logits(const void* logits, void* out_logits, const int32_t* history, const int32_t* history_len,
                     const int32_t* prompt_len, const int32_t* draft_tokens, const float* repetition,
                     const float* frequency, const float* presence, const int32_t* cu_bias,
                     const int32_t* bias_tokens, const float* bias_values, const uint32_t* mask,
                     const int32_t* mask_index, int32_t B, int32_t R, int32_t K, int32_t drafts_seen,
                     int32_t history_cap, int32_t num_bias, int32_t mask_rows, int32_t V, int32_t dtype,
                     void* stream) {
  if (R < 0 || K < 0 || K > SV_MAX_K || drafts_seen < 0) return SV_ERR_SHAPE;
  if (K > 0 ? (int64_t)drafts_seen + R - 1 > K : drafts_seen > 0) return SV_ERR_SHAPE;
  AdjArgs a = {};
  a.in = logits;
  a.out = out_logits;
  a.hist = history;
  a.hlen = history_len;
  a.plen = prompt_len;
  a.drafts = draft_tokens;
  a.rep = repetition;
  a.freq = frequency;
  a.pres = presence;
  a.cub = cu_bias;
  a.btok = bias_tokens;
  a.bval = bias_values;
  a.mask = mask;
  a.midx = mask_index;
  a.B = B;
  a.R = R;
  a.K = K;
  a.seen = drafts_seen;
  a.V = V;
  a.cap = history_cap;
  a.nbias = num_bias;
  a.mask_rows = mask_rows;
  return check_and_launch(a, (int64_t)B * R, dtype, stream);
}

int sv_adjust_logits_ragged(const void* logits, void* out_logits, const int32_t* history, const int32_t* history_len,
                            const int32_t* prompt_len, const int32_t* draft_tokens, const int32_t* cu_num_draft,
                            const float* repetition, const float* frequency, const float* presence,
                            const int32_t* cu_bias, const int32_t* bias_tokens, const float* bias_values,
                            const uint32_t* mask, const int32_t* mask_index, int32_t B, int32_t total_draft,
                            int32_t max_k, int32_t bonus_rows, int32_t history_cap, int32_t num_bias,
                            int32_t mask_rows, int32_t V, int32_t dtype, void* stream) {
  if (B < 0 || total_draft < 0 || max_k < 0 || max_k > SV_MAX_K || (int64_t)total_draft > (int64_t)B * max_k)
    return SV_ERR_SHAPE;
  if (bonus_rows != 0 && bonus_rows != 1) return SV_ERR_PARAM;
  if (B > 0 && !cu_num_draft) return SV_ERR_NULL;
  AdjArgs a = {};
  a.in = logits;
  a.out = out_logits;
  a.hist = history;
  a.hlen = history_len;
  a.plen = prompt_len;
  a.drafts = draft_tokens;
  a.cu = cu_num_draft;
  a.rep = repetition;
  a.freq = frequency;
  a.pres = presence;
  a.cub = cu_bias;
  a.btok = bias_tokens;
  a.bval = bias_values;
  a.mask = mask;
  a.midx = mask_index;
  a.B = B;
  a.N = total_draft;
  a.max_k = max_k;
  a.bonus = bonus_rows;
  a.V = V;
  a.cap = history_cap;
  a.nbias = num_bias;
  a.mask_rows = mask_rows;
  return check_and_launch(a, (int64_t)total_draft + (int64_t)B * bonus_rows, dtype, stream);
}

}  // extern "C"
