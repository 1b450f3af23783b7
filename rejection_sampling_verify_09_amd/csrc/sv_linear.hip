// Matrix product with its epilogue:
//   out[m, n] = act(sx[m] sw[n] sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n mod R]
// on the matrix cores, for bfloat16 operands or e4m3 operands with a float32
// scale per row.  Products of two bfloat16 values are exact in float32 and are
// summed in float32 (v_mfma_f32_16x16x32_bf16); the epilogue is float32 too,
// rounded once.  e4m3 operands are read as such, converted to bfloat16 in
// registers (exactly: 4 significant bits) and multiplied so.
//
// The 8-bit matrix instructions (v_mfma_f32_16x16x128_f8f6f4, twice the
// bfloat16 rate) do not sum in float32: measured, of each run of eight
// products along k they cut every one off, towards zero, below 2^-13 of the
// largest one's power of two, and only then add to a float32 accumulator.  Next
// to 448 x 448 a product of 7 is lost altogether, also where the large ones
// cancel (2-norm of the error on normal values 1.5e-5 of the result, with
// outlier columns 6e-5; so converted, 8e-8).  They are not used, and the
// largest products take more than half again as long for it (448 x 128256 x 4096
// to bfloat16: 376 to 384 us, 235 with them).
//
// Two kernels: linear_rows_kernel for up to 16 rows, whose waves share k, and
// linear_tile_kernel for more, and for many columns; sv_linear_pick.hpp
// chooses.  In both the weight is the matrix instruction's first operand, so
// that a lane holds four consecutive columns of the output.
#include "sv_linear_pick.hpp"
#include "sv_ops.hpp"
#include "specverify.h"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace sv {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8;
typedef __attribute__((__vector_size__(8 * sizeof(int)))) int i32x8;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;

enum Act : int { A_NONE = 0, A_RELU = 1, A_SILU = 2, A_GELU = 3, A_GELU_TANH = 4 };

struct LinArgs {
  const char* x;   // [M, K]
  const char* w;   // [N, K]
  const float* sx;  // [M], or null for bfloat16 operands
  const float* sw;  // [N]
  const void* bias;
  const void* res;  // [M, R]
  void* out;        // [M, N]
  int32_t M, N, K, R;
  int32_t act;
  int32_t mtiles, ntiles;
  int32_t turn;  // workgroups begin at different parts of k
};

// v / (1 + exp(-z)), from a = exp(-|z|): v / (1 + a), or v a / (1 + a) for
// negative z.  a is 2^t (1 + d ln 2), d being what rounding t = -|z| log2(e)
// left out, so that the whole is good to 5 units in the last place; below 2^-64
// it is held 2^64 times larger, since v a may be a normal number where a is not.
// Where a is 0, d plays no part (and may be NaN).
__device__ __forceinline__ float gated(float v, float z) {
  const float x = fabsf(z), t = -1.44269504f * x;
  const float d = __builtin_fmaf(x, -1.92596299e-8f, __builtin_fmaf(x, -1.44269504f, -t));
  const bool small = t < -64.0f;
  const float a = __builtin_amdgcn_exp2f(small ? t + 64.0f : t) * (x < 128.0f ? __builtin_fmaf(d, 0.693147181f, 1.0f) : 1.0f);
  const float r = __builtin_amdgcn_rcpf(small ? 1.0f : 1.0f + a);
  return z >= 0.0f ? v * r : v * a * r * (small ? 0x1p-64f : 1.0f);
}

// The same for a bfloat16 output: what rounding t leaves out is at most |z| 2^-24
// of the result, and goes without (half the instructions).  All of it 2^8 times
// smaller, so that the reciprocal is a normal number where the result is.
__device__ __forceinline__ float gated_bf16(float v, float z) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, -1.44269504f, -8.0f));
  return v * 0x1p-8f * __builtin_amdgcn_rcpf(0x1p-8f + e);
}

// v erfc(-v / sqrt 2) / 2 without the cancellation of 1 + erf at negative v:
// erfc(z) = exp(-z^2) t P(t), t = 1 / (1 + 0.3 z), with the polynomial P of
// least relative error (2.0e-8) for z in [0, 10]; past it the result is 0 or v.
__device__ __forceinline__ float gelu(float v) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(fabsf(v), 0.3f * 0.707106781f, 1.0f));
  float p = -0.129522771f;
  p = __builtin_fmaf(p, t, 0.485562563f);
  p = __builtin_fmaf(p, t, -0.512276769f);
  p = __builtin_fmaf(p, t, 0.547718585f);
  p = __builtin_fmaf(p, t, -0.0946497396f);
  p = __builtin_fmaf(p, t, 0.214925647f);
  p = __builtin_fmaf(p, t, 0.148339272f);
  p = __builtin_fmaf(p, t, 0.170715213f);
  p = __builtin_fmaf(p, t, 0.169188008f);
  const float q = p * t * __builtin_amdgcn_exp2f(v * v * -0.721347520f);
  return 0.5f * v * (v < 0.0f ? q : 2.0f - q);
}

// Of n values at a time, so that their chains of instructions overlap.
template <int OUT, int n>
__device__ __forceinline__ void activate(f32x4 (&v)[n], int act) {
  auto gate = [](float v, float z) { return OUT == T_BF16 ? gated_bf16(v, z) : gated(v, z); };
  if (act == A_RELU) {
#pragma unroll
    for (int r = 0; r < 4 * n; ++r) {
      const float x = v[r / 4][r % 4];
      v[r / 4][r % 4] = x > 0.0f ? x : (x != x ? x : 0.0f);
    }
  } else if (act == A_SILU) {
#pragma unroll
    for (int r = 0; r < 4 * n; ++r) v[r / 4][r % 4] = gate(v[r / 4][r % 4], v[r / 4][r % 4]);
  } else if (act == A_GELU) {
#pragma unroll
    for (int r = 0; r < 4 * n; ++r) v[r / 4][r % 4] = gelu(v[r / 4][r % 4]);
  } else if (act == A_GELU_TANH) {
#pragma unroll
    for (int r = 0; r < 4 * n; ++r) {
      const float x = v[r / 4][r % 4];
      v[r / 4][r % 4] = gate(x, 1.59576912f * __builtin_fmaf(0.044715f * x * x, x, x));
    }
  }
}

template <int OUT>
__device__ __forceinline__ float load_o(const void* p, size_t i) {
  if (OUT == T_F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// Eight e4m3 values as bfloat16 (exact).
__device__ __forceinline__ bf16x8 widen8(uint2 v) {
  bf16x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, false);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.x, 1.0f, true);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, false);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v.y, 1.0f, true);
  return __builtin_bit_cast(bf16x8, p);
}

// The operands: bfloat16, or e4m3 widened to bfloat16.
enum Mode : int { L_BF16 = 0, L_F8 = 1 };

typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

// A 16-row fragment of 128 bytes of k: lane l holds row l % 16 and, of its 128
// bytes, the 16-byte chunks l / 16 and 4 + l / 16, in both operands.
typedef i32x8 Frag;
__device__ __forceinline__ Frag frag(const i32x4& a, const i32x4& b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
template <int I>
__device__ __forceinline__ i32x4 half(const Frag& f) {
  return __builtin_shufflevector(f, f, 4 * I, 4 * I + 1, 4 * I + 2, 4 * I + 3);
}

// Products of a (rows of the result) and NB fragments b (columns), added to c.
template <int MODE, int NB>
__device__ __forceinline__ void mma16(f32x4 (&c)[NB], const Frag& x, const Frag (&w)[NB]) {
  if (MODE == L_BF16) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
      c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, half<0>(w[j])), __builtin_bit_cast(bf16x8, half<0>(x)), c[j], 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NB; ++j)
      c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, half<1>(w[j])), __builtin_bit_cast(bf16x8, half<1>(x)), c[j], 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8 xv = widen8(make_uint2((uint32_t)x[2 * i], (uint32_t)x[2 * i + 1]));
#pragma unroll
      for (int j = 0; j < NB; ++j)
        c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(make_uint2((uint32_t)w[j][2 * i], (uint32_t)w[j][2 * i + 1])), xv, c[j], 0, 0, 0);
    }
  }
}

// A 16-byte buffer load, zeros where `in` is false (an offset past every buffer).
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, int off, int soff, bool in) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, in ? off : 0x7FFFFF00, in ? soff : 0, 0));
}

// The epilogue of four columns n .. n + 3 (n a multiple of 4), those below N:
// what depends on the columns alone is read once for all rows.
template <int IN, int OUT>
struct Cols {
  float sw[4], bias[4];
  int n, nv, rc;
  __device__ __forceinline__ Cols(const LinArgs& a, int n_) : n(n_), nv(min(4, a.N - n_)), rc(a.res ? n_ % a.R : 0) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      sw[r] = IN == T_E4M3 && r < nv ? a.sw[n + r] : 1.0f;
      bias[r] = a.bias && r < nv ? load_o<OUT>(a.bias, n + r) : 0.0f;
    }
  }
  // the residual's values of row m (0 without one)
  __device__ __forceinline__ f32x4 residual(const LinArgs& a, int m) const {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!a.res) return v;
    const size_t row = (size_t)m * a.R;
    if (nv == 4 && rc + 4 <= a.R) {
      if (OUT == T_F32) {
        __builtin_memcpy(&v, static_cast<const float*>(a.res) + row + rc, 16);
      } else {
        uint2 q;
        __builtin_memcpy(&q, static_cast<const uint16_t*>(a.res) + row + rc, 8);
        v = f32x4{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
      }
    } else {
      int c = rc;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r < nv) v[r] = load_o<OUT>(a.res, row + c);
        c = c + 1 == a.R ? 0 : c + 1;
      }
    }
    return v;
  }
  // the sums s with the scales and the bias
  __device__ __forceinline__ f32x4 value(const LinArgs& a, const f32x4& s, float sx) const {
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = IN == T_E4M3 ? s[r] * sx * sw[r] : s[r];
      if (a.bias) v[r] += bias[r];
    }
    return v;
  }
  // out[m, n .. n + 3]
  __device__ __forceinline__ void store(const LinArgs& a, int m, const f32x4& v) const {
    const size_t at = (size_t)m * a.N + n;
    if (nv == 4) {
      // rows may start at any element: the hardware splits a store where it crosses
      if (OUT == T_F32) {
        const float4 q = make_float4(v[0], v[1], v[2], v[3]);
        __builtin_memcpy(static_cast<float*>(a.out) + at, &q, 16);
      } else {
        const uint2 q = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        __builtin_memcpy(static_cast<uint16_t*>(a.out) + at, &q, 8);
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < nv) {
          if (OUT == T_F32)
            static_cast<float*>(a.out)[at + r] = v[r];
          else
            static_cast<uint16_t*>(a.out)[at + r] = to_bf16(v[r]);
        }
    }
  }
};

// Byte of chunk c (16 bytes), row r of a staged block of 128-byte rows: the 16
// rows that a fragment reads at once lie in 16 different 16-byte columns of
// the banks.
__device__ __forceinline__ int at(int r, int c) { return r * 128 + 16 * (c ^ ((r >> 1) & 7)); }

// The fragment of rows 16 i .. 16 i + 15 of a staged block.
__device__ __forceinline__ Frag read_frag(const char* block, int i) {
  const int l16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  return frag(*reinterpret_cast<const i32x4*>(block + at(16 * i + l16, g)),
              *reinterpret_cast<const i32x4*>(block + at(16 * i + l16, 4 + g)));
}

// Orders a wave's own LDS accesses across its lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The workgroups begin their rounds over k at different ones, each group of
// about 256 columns at its own: where they all begin at 0, they ask for the
// same bytes of every row at once, and rows a power of two apart keep only some
// of the memory's channels busy (64 x 24576 x 4096 bfloat16, the bare product
// with 64 x 128 tiles: 48.0 us from 0, 40.0 so; 16 x 32000 x 4096 e4m3: 29.6 and
// 25.4; rows of 4224 bytes: alike).  Where x is larger than an XCD's L2, all
// begin at 0, so that the column panels read the same part of x (2048 x 8192 x
// 8192 bfloat16: 258 us, 264 otherwise; five others of 1024 to 8192 rows: alike).
__device__ __forceinline__ int first_round(const LinArgs& a, int n0, int rounds) {
  return a.turn ? (n0 >> 8) % rounds : 0;
}
__device__ __forceinline__ int turned(int round, int first, int rounds) {
  return round + first - (round + first >= rounds ? rounds : 0);
}

// Few rows: a workgroup owns 16 MT rows and 16 NT columns of the output, its W
// waves take turns over the 128-byte steps of k, D of them in flight in
// registers; the waves' sums are added in LDS.  Loads take whole 128-byte
// lines, eight rows each (a fragment's own layout, 16 rows across neighbouring
// lanes, keeps the address unit four times as long, 64 against 16 cycles a
// load), and a wave brings them into fragments through LDS of its own (16 x
// 24576 x 4096 bfloat16 41 us, 50 with fragments loaded directly).  Bound by
// the weight's bytes on long weights: 1 x 128256 x 4096 takes 164 us in
// bfloat16 (6.4 TB/s) and 84 in e4m3 (6.2), 7 rows to float32 89; by the launch
// on short ones (1 x 4096 x 4096: 9.0 us).
template <int MODE, int OUT, int NT, int MT, int W, int D>
__global__ void __launch_bounds__(64 * W) linear_rows_kernel(LinArgs a) {
  constexpr int IN = MODE == L_BF16 ? T_BF16 : T_E4M3;
  extern __shared__ __attribute__((aligned(16))) char smem[];  // [W][16 (MT + NT)][128], then the sums
  f32x4* part = reinterpret_cast<f32x4*>(smem);  // [W][MT * NT * 64]
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int nt0 = blockIdx.x / a.mtiles, mt0 = blockIdx.x - nt0 * a.mtiles;
  const int m0 = mt0 * 16 * MT, n0 = nt0 * 16 * NT;
  const int kbytes = a.K * (IN == T_BF16 ? 2 : 1);
  const int steps = (kbytes + 127) / 128, first = first_round(a, n0, steps);
  // buffer loads that end at the last valid row: rows past it read as zeros,
  // and so does what lies past the end of k, without touching memory (every
  // load is issued on every path, so that the waits count exactly)
  const auto rx = wave_rsrc(a.x + (size_t)m0 * kbytes, min(16 * MT, a.M - m0) * kbytes);
  const auto rw = wave_rsrc(a.w + (size_t)n0 * kbytes, min(16 * NT, a.N - n0) * kbytes);
  const int row = lane >> 3, col = 16 * (lane & 7), off = row * kbytes + col;
  uint4 xr[D][2 * MT], wr[D][2 * NT];
  auto load = [&](uint4 (&x)[2 * MT], uint4 (&wt)[2 * NT], int step) {
    const int k0 = step < steps ? turned(step, first, steps) * 128 : kbytes;
    const bool in = k0 + col < kbytes;
#pragma unroll
    for (int l = 0; l < 2 * NT; ++l) wt[l] = __builtin_bit_cast(uint4, load16(rw, off + (8 * l * kbytes + k0), 0, in));
#pragma unroll
    for (int l = 0; l < 2 * MT; ++l) x[l] = __builtin_bit_cast(uint4, load16(rx, off + (8 * l * kbytes + k0), 0, in));
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < D; ++d) load(xr[d], wr[d], w + d * W);
  char* const xl = smem + w * (MT + NT) * 2048;
  char* const wl = xl + MT * 2048;
  for (int s = w; s < steps;) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      wave_sync();
#pragma unroll
      for (int l = 0; l < 2 * NT; ++l) *reinterpret_cast<uint4*>(wl + at(8 * l + row, lane & 7)) = wr[d][l];
#pragma unroll
      for (int l = 0; l < 2 * MT; ++l) *reinterpret_cast<uint4*>(xl + at(8 * l + row, lane & 7)) = xr[d][l];
      load(xr[d], wr[d], s + D * W);
      wave_sync();
      Frag wf[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) wf[j] = read_frag(wl, j);
#pragma unroll
      for (int i = 0; i < MT; ++i) mma16<MODE>(acc[i], read_frag(xl, i), wf);
      s += W;  // past the last step: zeros
    }
  }
  __syncthreads();  // the sums take the rows' place
  // lane l of block (i, j) holds row 16 i + l % 16, columns 16 j + 4 (l / 16) + 0 .. 3
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(w * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int q = t; q < MT * NT * 64; q += 64 * W) {
    // four threads along each 16-column block, its row's blocks next
    const int c = q & 3, j = (q >> 2) % NT, r = (q >> 2) / NT;
    const int m = m0 + r, n = n0 + 16 * j + 4 * c;
    if (m >= a.M || n >= a.N) continue;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < W; ++k) v += part[(k * MT * NT + (r >> 4) * NT + j) * 64 + 16 * c + (r & 15)];
    const Cols<IN, OUT> cols(a, n);
    f32x4 y[1] = {cols.value(a, v, IN == T_E4M3 ? a.sx[m] : 1.0f)};
    activate<OUT>(y, a.act);
    if (a.res) y[0] += cols.residual(a, m);
    cols.store(a, m, y[0]);
  }
}

template <int MODE, int OUT, int NT, int MT, int W, int D>
hipError_t launch_rows(LinArgs a, hipStream_t s) {
  a.mtiles = (a.M + 16 * MT - 1) / (16 * MT);
  a.ntiles = (a.N + 16 * NT - 1) / (16 * NT);
  constexpr size_t lds = std::max(W * (MT + NT) * 2048, W * MT * NT * 1024);
  hipLaunchKernelGGL((linear_rows_kernel<MODE, OUT, NT, MT, W, D>), dim3((unsigned)a.mtiles * (unsigned)a.ntiles),
                     dim3(64 * W), lds, s, a);
  return hipGetLastError();
}

constexpr int tile_eb(int mb, int wm) { return mb * wm < 4 ? mb : 4 / wm; }  // 16-row blocks per pass of the epilogue
constexpr int lcm2(int a, int b) { return a % b == 0 ? a : b % a == 0 ? b : a * b; }  // of such small numbers
constexpr int lcm3(int a, int b, int c) { return lcm2(lcm2(a, b), c); }
constexpr int LIN_XCD = 8;  // XCDs the workgroup ids are dealt over

// More rows: a workgroup owns TM = 16 MB WM rows and TN = 16 NB WN columns; WM
// x WN waves share it, 16 MB x 16 NB each, and WK such groups take turns over
// the 128-byte steps of k, WK steps a round (their sums are added in LDS).
// Both operands go through LDS, loaded as whole 128-byte lines, eight rows a
// load: a fragment's own layout, 16 rows across neighbouring lanes, keeps the
// address unit four times as long (64 against 16 cycles a load), which held
// an earlier form with the weight straight in registers at 243 us where this
// one took 233 (448 x 128256 x 4096, both on the 8-bit instructions), and at
// 23.5 us where this one takes 18 (333 x 5001 x 2112).
//
// What bounds the largest tile (224 x 256, k blocks of 128 bytes, 8 waves, one
// workgroup a compute unit): the matrix instructions, and in part beside them
// LDS traffic (112 KB of rows, 64 KB of weights read, 60 KB written a round)
// and, for e4m3, the conversions; by the counters the matrix units are busy 60%
// of the time there and LDS 22%.  At 448 x 128256 x 4096: e4m3 to bfloat16 376
// to 384 us (1.25 PFLOP/s), to float32 381 (1.24), bfloat16 422 (1.12); the
// library's product of bfloat16 operands takes 543, that of 8-bit ones, on the
// 8-bit instructions, 296.  The small tiles are bound by the latency of a round
// (loads, LDS, barrier: 0.7 us), of which 333 x 5001 x 2112 has 17 (17.4 us; the
// library 21 to 23).
template <int MODE, int OUT, int MB, int NB, int WM, int WN, int WK, int D>
__global__ void __launch_bounds__(64 * WM * WN * WK) linear_tile_kernel(LinArgs a) {
  constexpr int IN = MODE == L_BF16 ? T_BF16 : T_E4M3;
  constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN, NTH = 64 * WM * WN * WK;
  constexpr int CX = (WK * TM * 8 + NTH - 1) / NTH, CW = (WK * TN * 8 + NTH - 1) / NTH;  // 16-byte chunks a thread stages
  constexpr int EB = tile_eb(MB, WM), PITCH = TN + 4;
  extern __shared__ __attribute__((aligned(16))) char smem[];  // [3][WK][TM][128] of x, [2][WK][TN][128] of the weight; then the sums
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = w % WN, wm = w / WN % WM, wk = w / (WN * WM);
  const int l16 = lane & 15, g = lane >> 4;
  // the row tiles of one panel of columns are consecutive tiles of one XCD
  const int q = blockIdx.x % LIN_XCD * (gridDim.x / LIN_XCD) + blockIdx.x / LIN_XCD;
  if (q >= a.mtiles * a.ntiles) return;
  const int nt0 = q / a.mtiles, m0 = (q - nt0 * a.mtiles) * TM, n0 = nt0 * TN;
  const int kbytes = a.K * (IN == T_BF16 ? 2 : 1);
  const int steps = (kbytes + 127) / 128, rounds = (steps + WK - 1) / WK;
  const int first = first_round(a, n0, rounds);
  // buffer loads that end at the last valid row: rows past it read as zeros
  const auto rx = wave_rsrc(a.x + (size_t)m0 * kbytes, min(TM, a.M - m0) * kbytes);
  const auto rw = wave_rsrc(a.w + (size_t)n0 * kbytes, min(TN, a.N - n0) * kbytes);

  // A thread stages the 16-byte chunk t % 8 of rows t / 8 + 64 i (NTH = 512)
  // of the round's WK blocks of `rows` rows.  What the i-th adds to the first's
  // address is the same for all threads.  Past the end of k both operands read
  // as zeros; every load is issued on every path, so that the waits count
  // exactly.
  constexpr int RT = NTH / 8;
  const int trow = t >> 3, tch = 16 * (t & 7);
  struct Base {
    int off, col;
  };
  auto base_of = [&](int rows) {
    const int r = WK == 1 || rows >= RT ? trow : trow % rows, col = (WK == 1 ? 0 : trow / rows) * 128 + tch;
    return Base{r * kbytes + col, col};
  };
  auto load = [&](uint4& v, __amdgpu_buffer_rsrc_t rs, int rows, const Base& b, int i, int round) {
    const int dr = WK == 1 ? i * RT : rows >= RT ? i * RT % rows : 0;
    const int db = WK == 1 ? 0 : rows >= RT ? i * RT / rows : i * (RT / rows);
    const int k0 = (round < rounds ? turned(round, first, rounds) * WK * 128 : kbytes) + db * 128;
    v = __builtin_bit_cast(uint4, load16(rs, b.off + (dr * kbytes + k0), 0, b.col + k0 < kbytes));
  };
  auto store = [&](const uint4& v, char* stage, int rows, int n, int i) {
    if (n * NTH == WK * rows * 8 || trow + i * RT < WK * rows) *reinterpret_cast<uint4*>(stage + at(trow, t & 7) + i * RT * 128) = v;
  };
  static_assert(RT % 16 == 0 && (WK == 1 || ((TM >= RT ? TM % RT : RT % TM) == 0 && (TN >= RT ? TN % RT : RT % TN) == 0)),
                "the threads' rows fall alike into every block");
  const Base bx = base_of(TM), bw = base_of(TN);
  char* const ws = smem + 3 * WK * TM * 128;
  auto getx = [&](int stage, int i) { return read_frag(smem + (stage * WK + wk) * TM * 128 + wm * MB * 2048, i); };
  auto getw = [&](int stage, int j) { return read_frag(ws + (stage * WK + wk) * TN * 128 + wn * NB * 2048, j); };
  f32x4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Round r multiplies its stage while the next one is whole and the one after
  // is written, so the first fragments of a round are read before the barrier
  // that ends the one before, and no wave waits at its start.
  uint4 xr[CX], wr[D][CW];
  Frag wf[NB];
  // stages 0 and 1 of both; the registers then hold the rounds from 2 on
#pragma unroll
  for (int i = 0; i < CX; ++i) load(xr[i], rx, TM, bx, i, 0);
#pragma unroll
  for (int s = 0; s < D; ++s)
#pragma unroll
    for (int i = 0; i < CW; ++i) load(wr[s][i], rw, TN, bw, i, s);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int i = 0; i < CX; ++i) {
      store(xr[i], smem + s * WK * TM * 128, TM, CX, i);
      load(xr[i], rx, TM, bx, i, s + 1);
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      store(wr[s % D][i], ws + s * WK * TN * 128, TN, CW, i);
      load(wr[s % D][i], rw, TN, bw, i, s + D);
    }
  }
  __syncthreads();
  constexpr int AH = MB > 1 ? 2 : 1;  // fragments of x ahead of the one that is multiplied
  constexpr int UN = lcm3(2, D, MB % AH ? AH : 1);  // the rings close together
  Frag xf[AH];
#pragma unroll
  for (int k = 0; k < NB; ++k) wf[k] = getw(0, k);
#pragma unroll
  for (int i = 0; i < AH; ++i) xf[i] = getx(0, i);
  __syncthreads();  // round 0 writes the weight's stage 0
  int st = 0;  // the round's stage of x
  for (int r = 0;;) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int st1 = st == 2 ? 0 : st + 1, st2 = st == 0 ? 2 : st - 1;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int x = (u * MB + i) % AH;
        mma16<MODE>(acc[i], xf[x], wf);
        xf[x] = i + AH < MB ? getx(st, i + AH) : getx(st1, (i + AH) % MB);
        // spread over the round: the stages of the round after the next, and
        // the loads that follow them into the registers they leave
#pragma unroll
        for (int k = 0; k < CW; ++k)
          if (k * MB / CW == i) {
            store(wr[(u + 2) % D][k], ws + u % 2 * WK * TN * 128, TN, CW, k);
            load(wr[(u + 2) % D][k], rw, TN, bw, k, r + 2 + D);
          }
#pragma unroll
        for (int k = 0; k < CX; ++k)
          if ((2 * k + 1) * MB / (2 * CX) == i) {
            store(xr[k], smem + st2 * WK * TM * 128, TM, CX, k);
            load(xr[k], rx, TM, bx, k, r + 3);
          }
        if (MB > 4) __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) wf[k] = getw((u + 1) % 2, k);
      __syncthreads();
      st = st1;
      if (++r == rounds) goto done;
    }
  }
done:
  // Bfloat16: the whole tile at once, rounded before it goes through LDS to be
  // stored in whole rows.  A residual comes the same way, into its elements'
  // places.
  if constexpr (OUT == T_BF16 && WK == 1) {
    constexpr int P2 = 2 * TN + 16;  // bytes of a row, and a pad that keeps the lanes' rows in different banks
    constexpr int TR = TN / 8, NR = TM * TR / NTH;  // threads a row, eight columns each; rows a thread
    static_assert(TM * TR % NTH == 0, "whole rows");
    const int tr = t / TR, tc = t % TR * 8, nv = a.N - n0 - tc, mv = min(TM, a.M - m0);
    uint4 res[NR];
    if (a.res) {
      const int rc = (n0 + tc) % a.R;
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int m = min(m0 + tr + k * (NTH / TR), a.M - 1);
        const uint16_t* const r = static_cast<const uint16_t*>(a.res) + (size_t)m * a.R;
        if (nv >= 8 && rc + 8 <= a.R) {
          __builtin_memcpy(&res[k], r + rc, 16);
        } else {
          uint32_t q[4] = {0, 0, 0, 0};
          int c = rc;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e < nv) q[e / 2] |= (uint32_t)r[c] << (e & 1 ? 16 : 0);
            c = c + 1 == a.R ? 0 : c + 1;
          }
          res[k] = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
    }
    float sx[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) sx[i] = IN == T_E4M3 ? a.sx[min(m0 + wm * 16 * MB + 16 * i + l16, a.M - 1)] : 1.0f;
    f32x4 sw[NB], bias[NB];  // of the lane's columns
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const Cols<IN, OUT> cols(a, min(n0 + wn * 16 * NB + 16 * j + 4 * g, a.N - 1));
      sw[j] = f32x4{cols.sw[0], cols.sw[1], cols.sw[2], cols.sw[3]};
      bias[j] = f32x4{cols.bias[0], cols.bias[1], cols.bias[2], cols.bias[3]};
    }
    __syncthreads();  // the fragments read ahead
    char* const mine = smem + (wm * 16 * MB + l16) * P2 + 2 * (wn * 16 * NB + 4 * g);
    auto scaled = [&](const f32x4& s, int i, const f32x4& w, const f32x4& b) {
      const f32x4 v = IN == T_E4M3 ? s * sx[i] * w : s;
      return a.bias ? v + b : v;
    };
    auto put = [&](int i, int j, const f32x4& v) {  // 16 i rows and 16 j columns on
      *reinterpret_cast<uint2*>(mine + 16 * i * P2 + 32 * j) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    };
    if (!a.res && a.act == A_NONE) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) put(i, j, scaled(acc[i][j], i, sw[j], bias[j]));
    } else {
      if (a.res) {
#pragma unroll
        for (int k = 0; k < NR; ++k) *reinterpret_cast<uint4*>(smem + (tr + k * (NTH / TR)) * P2 + 2 * tc) = res[k];
        __syncthreads();
      }
#pragma unroll 1  // one copy of the activations' code
      for (int j = 0; j < NB; ++j) {
        f32x4 v[MB], w, q;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (b != 0 && j != b) continue;
          w = sw[b];
          q = bias[b];
#pragma unroll
          for (int i = 0; i < MB; ++i) v[i] = acc[i][b];
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) v[i] = scaled(v[i], i, w, q);
        activate<OUT>(v, a.act);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          if (a.res) {
            const uint2 r = *reinterpret_cast<const uint2*>(mine + 16 * i * P2 + 32 * j);
            v[i] += f32x4{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
          }
          put(i, j, v[i]);
        }
      }
    }
    __syncthreads();
    char* const out = static_cast<char*>(a.out) + 2 * ((size_t)m0 * a.N + n0 + tc);
#pragma unroll 4
    for (int m = tr; m < mv; m += NTH / TR) {
      const uint4 v = *reinterpret_cast<const uint4*>(smem + m * P2 + 2 * tc);
      char* const o = out + 2 * (size_t)m * a.N;
      if (nv >= 8) {
        __builtin_memcpy(o, &v, 16);
      } else {
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < nv) reinterpret_cast<uint16_t*>(o)[k] = (uint16_t)(q[k / 2] >> (k & 1 ? 16 : 0));
      }
    }
    return;
  }
  // Lane l of block (i, j) holds row 16 i + l % 16, columns 16 j + 4 (l / 16)
  // + 0 .. 3.  Through LDS, EB blocks of rows at a time: there the groups' sums
  // are added, in order, and the rows are stored whole, a thread having four
  // columns and every RS-th row.
  float* tile = reinterpret_cast<float*>(smem);
  float* sxs = tile + WM * 16 * EB * PITCH;  // the rows' scales
  constexpr int RS = NTH / (TN / 4);
  const int ncol = nt0 * TN + t % (TN / 4) * 4;
  const Cols<IN, OUT> cols(a, min(ncol, a.N - 1));
  __syncthreads();  // the fragments read ahead
  if (IN == T_E4M3)
    for (int i = t; i < min(TM, a.M - m0); i += NTH) sxs[i] = a.sx[m0 + i];
  float* mine = tile + (wm * 16 * EB + l16) * PITCH + wn * 16 * NB + 4 * g;
  static_assert(WM <= 2, "the rows of a pass lie in at most two parts");
#pragma unroll 1  // the code of a pass stays short: unrolled, its instructions miss their cache
  for (int ib = 0; ib < MB; ib += EB) {
    const int rows = 16 * min(EB, MB - ib);  // of each of the WM parts
#pragma unroll
    for (int k = 0; k < WK; ++k) {
      if (WK == 1 || wk == k) {
#pragma unroll
        for (int b = 0; b < MB; b += EB) {
          if (ib != b) continue;
#pragma unroll
          for (int i = b; i < b + EB && i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              f32x4* p = reinterpret_cast<f32x4*>(mine + 16 * (i - b) * PITCH + 16 * j);
              *p = k == 0 ? acc[i][j] : *p + acc[i][j];
            }
        }
      }
      __syncthreads();
    }
    if (ncol < a.N) {
      const int all = WM * rows, tc = t % (TN / 4) * 4;
      auto row_of = [&](int e) { return e < rows ? 16 * ib + e : 16 * (MB + ib) + e - rows; };  // of the tile
      auto sums = [&](int e) {
        return *reinterpret_cast<const f32x4*>(tile + (e < rows ? e : 16 * EB + e - rows) * PITCH + tc);
      };
      // four rows at a time, all loads before the stores; rows past the last
      // one are read as that one
      constexpr int RB = 4;
#pragma unroll 1
      for (int e0 = t / (TN / 4); e0 < all; e0 += RB * RS) {
        f32x4 v[RB], res[RB];
        float sx[RB];
        int m[RB];
#pragma unroll
        for (int k = 0; k < RB; ++k) {
          const int e = min(e0 + k * RS, all - 1);
          m[k] = row_of(e);
          v[k] = sums(e);
          sx[k] = IN == T_E4M3 ? sxs[m[k]] : 1.0f;
          m[k] += m0;
        }
        if (a.res) {
#pragma unroll
          for (int k = 0; k < RB; ++k) res[k] = cols.residual(a, min(m[k], a.M - 1));
        }
#pragma unroll
        for (int k = 0; k < RB; ++k) v[k] = cols.value(a, v[k], sx[k]);
        activate<OUT>(v, a.act);
        if (a.res) {
#pragma unroll
          for (int k = 0; k < RB; ++k) v[k] += res[k];
        }
#pragma unroll
        for (int k = 0; k < RB; ++k)
          if (e0 + k * RS < all && m[k] < a.M) cols.store(a, m[k], v[k]);
      }
    }
    __syncthreads();
  }
}

template <int MODE, int OUT, int MB, int NB, int WM, int WN, int WK, int D>
hipError_t launch_tile(LinArgs a, hipStream_t s) {
  constexpr int TM = 16 * MB * WM, TN = 16 * NB * WN;
  constexpr int lds = std::max(3 * WK * TM * 128 + 2 * WK * TN * 128, (16 * WM * tile_eb(MB, WM) * (TN + 4) + TM) * 4);
  static_assert(lds <= 160 * 1024, "LDS of a compute unit");
  static_assert(WK > 1 || TM * (2 * TN + 16) <= lds, "a bfloat16 tile goes through LDS at once");
  a.mtiles = (a.M + TM - 1) / TM;
  a.ntiles = (a.N + TN - 1) / TN;
  // the limit is raised once per device (twice from racing first calls is harmless)
  static std::atomic<bool> raised[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  if (!raised[dev].load(std::memory_order_acquire)) {
    const hipError_t e = hipFuncSetAttribute((const void*)linear_tile_kernel<MODE, OUT, MB, NB, WM, WN, WK, D>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    raised[dev].store(true, std::memory_order_release);
  }
  const unsigned grid = ((unsigned)a.mtiles * (unsigned)a.ntiles + LIN_XCD - 1) / LIN_XCD * LIN_XCD;
  hipLaunchKernelGGL((linear_tile_kernel<MODE, OUT, MB, NB, WM, WN, WK, D>), dim3(grid), dim3(64 * WM * WN * WK), lds, s, a);
  return hipGetLastError();
}

// Threads of the launch, or an upper bound (every workgroup has at most 512).
int64_t launch_threads(int kernel, int64_t M, int64_t N) {
  const int64_t tm = kernel >= 0 ? kTiles[kernel].tm : 16;
  const int64_t tn = kernel >= 0 ? kTiles[kernel].tn : kernel == ROWS_16 ? 16 : 32;
  return (((M + tm - 1) / tm) * ((N + tn - 1) / tn) + LIN_XCD) * 512;
}

template <int MODE, int OUT>
hipError_t launch_linear(const LinArgs& a, int kernel, hipStream_t s) {
  switch (kernel) {
    case ROWS_16: return launch_rows<MODE, OUT, 1, 1, 8, 2>(a, s);
    case ROWS_32: return launch_rows<MODE, OUT, 2, 1, 4, 2>(a, s);
    case 0: return launch_tile<MODE, OUT, 2, 1, 1, 2, 4, 2>(a, s);
    case 1: return launch_tile<MODE, OUT, 2, 2, 1, 2, 4, 2>(a, s);
    case 2: return launch_tile<MODE, OUT, 2, 2, 2, 2, 2, 2>(a, s);
    case 3: return launch_tile<MODE, OUT, 4, 2, 1, 4, 2, 2>(a, s);
    case 4: return launch_tile<MODE, OUT, 4, 4, 2, 2, 1, 2>(a, s);
    case 5: return launch_tile<MODE, OUT, 4, 4, 2, 4, 1, 2>(a, s);
    case 6: return launch_tile<MODE, OUT, 6, 4, 2, 4, 1, 2>(a, s);
    default: return launch_tile<MODE, OUT, 7, 4, 2, 4, 1, 1>(a, s);
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" int sv_linear(const void* x, const void* weight, const float* x_scale, const float* weight_scale,
                         const void* bias, const void* residual, void* out, int32_t M, int32_t N, int32_t K,
                         int32_t residual_cols, int32_t activation, int32_t dtype, int32_t out_dtype, void* stream) {
  if (M < 0 || N < 1 || K < 64 || K > SV_MAX_LINEAR_K || K % 64 != 0) return SV_ERR_SHAPE;
  if (dtype != SV_BF16 && dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (out_dtype != SV_F32 && out_dtype != SV_BF16) return SV_ERR_DTYPE;
  if (activation < SV_ACT_NONE || activation > SV_ACT_GELU_TANH) return SV_ERR_PARAM;
  if (residual && (residual_cols < 1 || N % residual_cols != 0)) return SV_ERR_SHAPE;
  if (M == 0) return SV_OK;
  const int kernel = pick_kernel(M, N, (int64_t)K * type_bytes(dtype));
  if (launch_threads(kernel, M, N) > kGridThreads) return SV_ERR_SHAPE;
  const bool scaled = dtype == SV_E4M3;
  if (!x || !weight || !out || (scaled && (!x_scale || !weight_scale))) return SV_ERR_NULL;
  const size_t ie = (size_t)type_bytes(dtype), oe = (size_t)type_bytes(out_dtype);
  if (!is_aligned(x, 16) || !is_aligned(weight, 16) || !is_aligned(out, oe) || !is_aligned(bias, oe) ||
      !is_aligned(residual, oe) || (scaled && (!is_aligned(x_scale, 4) || !is_aligned(weight_scale, 4))))
    return SV_ERR_SHAPE;
  const size_t no = (size_t)M * (size_t)N * oe;
  const size_t nr = residual ? (size_t)M * (size_t)residual_cols * oe : 0;
  if (overlaps(out, no, x, (size_t)M * K * ie) || overlaps(out, no, weight, (size_t)N * K * ie) ||
      overlaps(out, no, bias, (size_t)N * oe) ||
      (scaled && (overlaps(out, no, x_scale, (size_t)M * 4) || overlaps(out, no, weight_scale, (size_t)N * 4))) ||
      (overlaps(out, no, residual, nr) && !(out == residual && residual_cols == N)))
    return SV_ERR_PARAM;
  LinArgs a;
  a.x = static_cast<const char*>(x);
  a.w = static_cast<const char*>(weight);
  a.sx = scaled ? x_scale : nullptr;
  a.sw = scaled ? weight_scale : nullptr;
  a.bias = bias;
  a.res = residual;
  a.out = out;
  a.M = M;
  a.N = N;
  a.K = K;
  a.R = residual ? residual_cols : 1;
  a.act = activation;
  a.turn = (int64_t)M * K * (int64_t)ie <= (int64_t)4 << 20;
  hipStream_t s = (hipStream_t)stream;
  const hipError_t e = dtype == SV_BF16
                           ? (out_dtype == SV_F32 ? launch_linear<L_BF16, T_F32>(a, kernel, s) : launch_linear<L_BF16, T_BF16>(a, kernel, s))
                           : (out_dtype == SV_F32 ? launch_linear<L_F8, T_F32>(a, kernel, s) : launch_linear<L_F8, T_BF16>(a, kernel, s));
  return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}
