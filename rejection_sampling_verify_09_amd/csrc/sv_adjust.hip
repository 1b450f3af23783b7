// Penalties, biases and grammar masks on logits, before the filters and the
// draw.  For token j at a position with c_j occurrences among the sequence's
// output tokens (its history behind the prompt, and the drafts that stand
// before the position):
//   l = logit_j
//   l = l / rep (l > 0) or l * rep        if c_j > 0 or j is in the prompt
//   l = l - freq c_j - pres [c_j > 0]
//   l = l + the sum of j's biases
//   l = -inf                              if the row's mask forbids j
// in float32, rounded once to the logits' type.
//
// Split: a workgroup owns a slice of the vocabulary of one sequence, counts
// the sequence's tokens that fall into it in an LDS table (integer atomics:
// no order changes a count), and then handles the slice of each of the
// sequence's rows.  The history is read once per slice, from the L2.
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
  int32_t nslices;
};

// Table entry: occurrences in the low bits, and what else is known of the token.
constexpr uint32_t E_PROMPT = 1u << 31, E_DRAFT = 1u << 30, E_BIAS = 1u << 29, E_BIASES = 1u << 28;
constexpr uint32_t E_COUNT = E_BIASES - 1;
constexpr int ADJ_MAX_WG = 1024, ADJ_EPT = 8;  // a thread has 8 tokens of the slice

// One logit of a row: e its table entry, c further occurrences among the drafts.
__device__ __forceinline__ float adjusted(float l, uint32_t e, float bias, float c, float rep, float freq, float pres) {
  c += (float)(e & E_COUNT);
  if (c > 0.0f || (e & E_PROMPT)) l = l > 0.0f ? l / rep : l * rep;
  if (c > 0.0f) l = l - freq * c - pres;
  if (e & E_BIAS) l += bias;
  return l;
}

template <int DT>
__device__ __forceinline__ float get(const void* p, size_t i) {
  if (DT == T_F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}
template <int DT>
__device__ __forceinline__ void set(void* p, size_t i, float v) {
  if (DT == T_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = to_bf16(v);
}

template <int DT>
__global__ void __launch_bounds__(ADJ_MAX_WG) adjust_kernel(AdjArgs a) {
  extern __shared__ uint32_t smem[];
  const int t = threadIdx.x, nt = blockDim.x, S = nt * ADJ_EPT;
  uint32_t* tab = smem;            // [S]
  uint32_t* bt = smem + S;         // [S]: index of the token's first bias, then the bias
  __shared__ int32_t xs[MAX_K];    // the sequence's drafts
  const int b = blockIdx.x / a.nslices, sl = blockIdx.x - b * a.nslices;
  const int v0 = sl * S, vn = min(S, a.V - v0);

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
  } else {
    d0 = (int64_t)b * a.K;
    nd = a.K;
    row0 = (int64_t)b * a.R;
    nr = a.R;
  }
  nd = min(nd, a.seen + nr - 1);  // drafts that some row has seen

  const bool counts = a.rep || a.freq || a.pres;
  for (int i = t; i < S; i += nt) {
    tab[i] = 0;
    if (a.cub) bt[i] = 0xFFFFFFFFu;
  }
  __syncthreads();
  if (counts) {
    if (a.hist) {
      const int32_t* h = a.hist + (size_t)b * a.cap;
      const int n = a.hlen ? min(max(a.hlen[b], 0), a.cap) : a.cap;
      const int np = a.plen ? min(max(a.plen[b], 0), n) : 0;
      for (int i = t; i < n; i += nt) {
        const uint32_t j = (uint32_t)h[i] - (uint32_t)v0;
        if (j < (uint32_t)vn) {
          if (i < np)
            atomicOr(&tab[j], E_PROMPT);
          else
            atomicAdd(&tab[j], 1u);
        }
      }
    }
    for (int i = t; i < nd; i += nt) {
      xs[i] = a.drafts[d0 + i];
      const uint32_t j = (uint32_t)xs[i] - (uint32_t)v0;
      if (j < (uint32_t)vn) atomicOr(&tab[j], E_DRAFT);
    }
  }
  if (a.cub) {
    // several biases of one token are added in the order they are listed:
    // the first one's thread adds them up
    const int i0 = min(max(a.cub[b], 0), a.nbias), i1 = min(a.cub[b + 1], a.nbias);
    for (int i = i0 + t; i < i1; i += nt) {
      const uint32_t j = (uint32_t)a.btok[i] - (uint32_t)v0;
      if (j < (uint32_t)vn) {
        atomicMin(&bt[j], (uint32_t)i);
        atomicOr(&tab[j], E_BIAS);
      }
    }
    __syncthreads();
    for (int i = i0 + t; i < i1; i += nt) {
      const uint32_t j = (uint32_t)a.btok[i] - (uint32_t)v0;
      if (j < (uint32_t)vn && bt[j] != (uint32_t)i) atomicOr(&tab[j], E_BIASES);
    }
    __syncthreads();
    for (int i = i0 + t; i < i1; i += nt) {
      const int32_t tok = a.btok[i];
      const uint32_t j = (uint32_t)tok - (uint32_t)v0;
      if (j >= (uint32_t)vn) continue;
      float v = a.bval[i];
      if (tab[j] & E_BIASES) {
        bool first = true;
        for (int k = i0; k < i && first; ++k) first = a.btok[k] != tok;
        if (!first) continue;
        for (int k = i + 1; k < i1; ++k)
          if (a.btok[k] == tok) v += a.bval[k];
      }
      bt[j] = __float_as_uint(v);  // its index is not looked at any more
    }
  }
  __syncthreads();

  const float rep = a.rep ? a.rep[b] : 1.0f, freq = a.freq ? a.freq[b] : 0.0f, pres = a.pres ? a.pres[b] : 0.0f;
  for (int r = 0; r < nr; ++r) {
    const size_t row = (size_t)(row0 + r);
    const int64_t mi = !a.mask ? -1 : a.midx ? (int64_t)a.midx[row] : (int64_t)row;
    const uint32_t* mask = mi >= 0 && mi < a.mask_rows ? a.mask + (size_t)mi * a.words : nullptr;
    const int nseen = min(nd, a.seen + r);
    for (int j = t; j < vn; j += nt) {
      const int v = v0 + j;
      float l;
      if (mask && !((mask[v >> 5] >> (v & 31)) & 1u)) {
        l = -INFINITY;
      } else {
        l = get<DT>(a.in, row * a.V + v);
        const uint32_t e = tab[j];
        if (e) {
          float c = 0.0f;
          if (e & E_DRAFT)
            for (int k = 0; k < nseen; ++k) c += xs[k] == v ? 1.0f : 0.0f;
          l = adjusted(l, e, __uint_as_float(a.cub ? bt[j] : 0u), c, rep, freq, pres);
        }
      }
      set<DT>(a.out, row * a.V + v, l);
    }
  }
}

template <int DT>
hipError_t launch_adjust(AdjArgs a, hipStream_t s) {
  // a thread for every 8 tokens, up to slices of 8192
  const int nt = std::min(ADJ_MAX_WG, std::max(64, ((a.V + ADJ_EPT - 1) / ADJ_EPT + 63) / 64 * 64));
  a.nslices = (a.V + nt * ADJ_EPT - 1) / (nt * ADJ_EPT);
  const size_t lds = (size_t)nt * ADJ_EPT * 4 * (a.cub ? 2 : 1);
  hipLaunchKernelGGL(adjust_kernel<DT>, dim3((unsigned)a.B * (unsigned)a.nslices), dim3(nt), lds, s, a);
  return hipGetLastError();
}

size_t words_of(int32_t V) { return ((size_t)V + 31) / 32; }

int check_and_launch(AdjArgs& a, int64_t rows, int32_t dtype, void* stream) {
  const int32_t V = a.V;
  if (a.B < 0 || rows < 0 || V < 1 || V > MAX_V || a.cap < 0 || a.cap > SV_MAX_HISTORY || a.nbias < 0 ||
      a.mask_rows < 0)
    return SV_ERR_SHAPE;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_DTYPE;
  // the smallest slices have 64 threads for 512 tokens
  if ((int64_t)a.B * (((int64_t)V + 511) / 512) * 64 > kGridThreads || rows > INT32_MAX) return SV_ERR_SHAPE;
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
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == SV_F32 ? launch_adjust<T_F32>(a, s) : launch_adjust<T_BF16>(a, s);
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
