// Matrix-core operands for kernels that take bf16 or float32 tensors through one source: fragments of
// row-major LDS tiles, read along rows or transposed, and float32 values as bf16 terms.
#pragma once
#include "common.hpp"

namespace hla {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Nothing is scheduled across this point.  In a long unrolled loop the scheduler would otherwise move
// every LDS read to the front and spill.
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// The value, as one that the compiler knows nothing of: in a loop, what is computed from it is computed
// again each time and not kept in registers from before.
__device__ __forceinline__ int own(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ int own_s(int x) {  // of a uniform value
  asm volatile("" : "+s"(x));
  return x;
}

// Sums of N (16 or 32) values over the 32 lanes of a half wave, lane c receiving that of v[c % N]: at every
// step a lane hands its partner the values that the partner keeps.  (A half-row mirror pairs lane i with
// i ^ 7; the two steps behind it add what that leaves in the quad.)
template <int N>
__device__ __forceinline__ float rows_to_lanes(const float (&v)[N], int lane) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (N == 32) {
      const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v[i]), __builtin_bit_cast(unsigned, v[i + 16]),
                                                      false, false);
      x[i] = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
    } else {
      x[i] = v[i];
    }
  }
  const bool b3 = lane & 8, b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (b3 ? x[i + 8] : x[i]) + dpp_f<0x128>(b3 ? x[i] : x[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (b2 ? x[i + 4] : x[i]) + dpp_f<0x141>(b2 ? x[i] : x[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = (b1 ? x[i + 2] : x[i]) + dpp_f<0x4E>(b1 ? x[i] : x[i + 2]);
  x[0] = (b0 ? x[1] : x[0]) + dpp_f<0xB1>(b0 ? x[0] : x[1]);
  return N == 32 ? x[0] : swap16_sum(x[0]);
}

// The operands of a product over K: `Frag` is what a lane holds of KG consecutive k.
// bf16: one 32x32x16 instruction, 8 values a lane.  float32: four 32x32x2, slot e of the group is
// k = 4 h + e, which is also the order in which an accumulator holds its rows.
template <class T> struct La;

template <> struct La<bf16> {
  static constexpr int P = 64, KG = 16, TERMS = 3;
  using Frag = bf16x8;
  // An LDS tile of W columns: rows of 16-byte chunks, permuted by the row so that the row reads (16
  // rows, one chunk) and the transposing reads (4 rows, 4 chunks) both meet every bank once.
  template <int W> __device__ __forceinline__ static int at(int row, int col) {
    const int s = W == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    return row * W + (((col >> 3) ^ s) << 3) + (col & 7);
  }
  template <int W> static constexpr int rs() { return W; }  // elements of an LDS row
  template <int W> static constexpr int size() { return P * W; }
  // Decayed scores as two terms, each the 32 x 32 tiles 0: (0, 0), 1: (1, 0), 2: (1, 1) of a 64 x 64 lower
  // triangle: rows of four 16-byte chunks, permuted by the row so that 16 rows' reads meet every bank once.
  static constexpr int SCORE_TERMS = 2, SCORE_TERM = 3 * 1024, SCORES = SCORE_TERMS * SCORE_TERM;
  __device__ __forceinline__ static int score_at(int tile, int c, int q, int h) {  // row c, columns 8 q + 4 h ..
    return tile * 1024 + c * 32 + ((q ^ ((c >> 2) & 3)) << 3) + h * 4;
  }
  __device__ __forceinline__ static Frag score_row(const bf16* sc, int I, int c, int g, int h, int term) {
    const int tile = I ? (g >= 2 ? 2 : 1) : 0;
    return *reinterpret_cast<const bf16x8*>(sc + term * SCORE_TERM + tile * 1024 + c * 32 + (((2 * (g & 1) + h) ^ ((c >> 2) & 3)) << 3));
  }
  __device__ __forceinline__ static f32x16 mma(Frag a, Frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // Element offsets that a lane's reads start from; the chunk permutation makes every further read an
  // exclusive or of a constant.  `own` (see there) keeps these few in registers, not the reads' own.
  template <int W> __device__ __forceinline__ static int row_base(int lane) { return at<W>(lane & 31, (lane >> 5) * 8); }
  template <int W> __device__ __forceinline__ static int rowc_base(int lane) { return at<W>(lane & 31, (lane >> 5) * 4); }
  template <int W> __device__ __forceinline__ static int col_base(int lane) {
    return at<W>((lane >> 5) * 8 + ((lane >> 2) & 3), ((lane >> 4) & 1) * 16 + (lane & 3) * 4);
  }
  // row r0 + lane % 32 (r0 a multiple of 16): k = 16 g + 8 h + e
  __device__ __forceinline__ static Frag plain(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }
  template <int W> __device__ __forceinline__ static Frag row(const bf16* t, int base, int r0, int g) {
    return plain(t + r0 * W + (base ^ (g << 4)));
  }
  // the same row, k = 16 g + 8 (e / 4) + 4 h + e % 4: the accumulators' order
  template <int W> __device__ __forceinline__ static Frag rowc(const bf16* t, int base, int r0, int g) {
    const bf16x4 lo = *reinterpret_cast<const bf16x4*>(t + r0 * W + (base ^ (g << 4)));
    const bf16x4 hi = *reinterpret_cast<const bf16x4*>(t + r0 * W + (base ^ (g << 4) ^ 8));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  // column 32 m + lane % 32, rows k = 16 g + 8 h + e: the transposing LDS read hands lane i of 16 the
  // i-th column of the four rows that its 16 lanes address (4 lanes a row, 4 columns each)
  template <int W> __device__ __forceinline__ static Frag col(const bf16* t, int base, int m, int g) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const bf16* p = t + g * 16 * W;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + (base ^ (m << 5))));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * W + (base ^ (m << 5) ^ 8)));
    return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  // element (row 32 I + acc_row(e, h), column col): the tile in the accumulators' layout
  template <int W> __device__ __forceinline__ static int acc_base(int lane, int col) { return at<W>(4 * (lane >> 5), col); }
  template <int W> __device__ __forceinline__ static float acc_el(const bf16* t, int base, int I, int e) {
    const int q = e >> 2, r = e & 3, x = (W == 128 ? r << 2 : (r >> 1) << 2) | ((2 * q) & 2);
    return (float)t[(32 * I + 8 * q + r) * W + (base ^ (x << 3))];
  }
  __device__ __forceinline__ static int col_k(int g, int h) { return g * 16 + h * 8; }  // first of 8 k
  static constexpr int FN = 8;
  typedef float Vals __attribute__((ext_vector_type(8)));
  // the first N bf16 terms of 8 float32 values (pairs: one conversion packs two)
  template <int N> __device__ __forceinline__ static void split(Vals x, Frag (&f)[N]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int t = 0; t < N; ++t) {
      unsigned u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{x[2 * e], x[2 * e + 1]}, bf16x2));
        if (t + 1 < N) {
          x[2 * e] -= __builtin_bit_cast(float, u[e] << 16);
          x[2 * e + 1] -= __builtin_bit_cast(float, u[e] & 0xffff0000u);
        }
      }
      f[t] = __builtin_bit_cast(Frag, u32x4{u[0], u[1], u[2], u[3]});
    }
  }
};

template <> struct La<float> {
  static constexpr int P = 32, KG = 8, TERMS = 1;
  using Frag = f32x4;
  template <int W> __device__ __forceinline__ static int at(int row, int col) { return row * (W + 8) + col; }
  template <int W> static constexpr int rs() { return W + 8; }
  template <int W> static constexpr int size() { return P * (W + 8); }
  static constexpr int SCORE_TERMS = 1, SCORE_TERM = P * (P + 8), SCORES = SCORE_TERM;
  __device__ __forceinline__ static int score_at(int, int c, int q, int h) { return c * (P + 8) + q * 8 + h * 4; }
  __device__ __forceinline__ static Frag score_row(const float* sc, int, int c, int g, int h, int) {
    return *reinterpret_cast<const f32x4*>(sc + c * (P + 8) + g * 8 + h * 4);
  }
  __device__ __forceinline__ static f32x16 mma(Frag a, Frag b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  template <int W> __device__ __forceinline__ static int row_base(int lane) { return at<W>(lane & 31, (lane >> 5) * 4); }
  template <int W> __device__ __forceinline__ static int rowc_base(int lane) { return row_base<W>(lane); }
  template <int W> __device__ __forceinline__ static int col_base(int lane) { return at<W>((lane >> 5) * 4, lane & 31); }
  __device__ __forceinline__ static Frag plain(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
  template <int W> __device__ __forceinline__ static Frag row(const float* t, int base, int r0, int g) {
    return plain(t + base + r0 * (W + 8) + g * 8);
  }
  template <int W> __device__ __forceinline__ static Frag rowc(const float* t, int base, int r0, int g) {
    return row<W>(t, base, r0, g);
  }
  template <int W> __device__ __forceinline__ static Frag col(const float* t, int base, int m, int g) {
    Frag f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = t[base + (g * 8 + e) * (W + 8) + 32 * m];
    return f;
  }
  template <int W> __device__ __forceinline__ static int acc_base(int lane, int col) { return at<W>(4 * (lane >> 5), col); }
  template <int W> __device__ __forceinline__ static float acc_el(const float* t, int base, int I, int e) {
    return t[base + (32 * I + acc_row(e, 0)) * (W + 8)];
  }
  __device__ __forceinline__ static int col_k(int g, int h) { return g * 8 + h * 4; }
  static constexpr int FN = 4;
  typedef f32x4 Vals;
  template <int N> __device__ __forceinline__ static void split(Vals x, Frag (&f)[N]) { f[0] = x; }
};

// The same for 16 x 16 tiles: rows (or columns) lane % 16, with G = lane / 16 four quarters of k; the
// accumulator is rows 4 G + e, column lane % 16.
template <class T> struct La16;

template <> struct La16<bf16> {  // one 16x16x32, 8 values a lane: k = 32 g + 8 G + e
  static constexpr int KG = 32, TERMS = 3;
  using O = La<bf16>;
  using Frag = bf16x8;
  __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  template <int W> __device__ __forceinline__ static int row_base(int lane) { return O::at<W>(lane & 15, (lane >> 4) * 8); }
  template <int W> __device__ __forceinline__ static Frag row(const bf16* t, int base, int r0, int g) {
    return O::plain(t + r0 * W + (base ^ (g << 5)));
  }
  template <int W> __device__ __forceinline__ static int col_base(int lane) {
    return O::at<W>((lane >> 4) * 8 + ((lane >> 2) & 3), (lane & 3) * 4);
  }
  // column 16 m + lane % 16, rows k
  template <int W> __device__ __forceinline__ static Frag col(const bf16* t, int base, int m, int g) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const bf16* p = t + g * 32 * W;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + (base ^ (m << 4))));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * W + (base ^ (m << 4) ^ 8)));
    return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

template <> struct La16<float> {  // four 16x16x4, 4 values a lane: k = 16 g + 4 G + e
  static constexpr int KG = 16, TERMS = 1;
  using O = La<float>;
  using Frag = f32x4;
  __device__ __forceinline__ static f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
  }
  template <int W> __device__ __forceinline__ static int row_base(int lane) { return O::at<W>(lane & 15, (lane >> 4) * 4); }
  template <int W> __device__ __forceinline__ static Frag row(const float* t, int base, int r0, int g) {
    return O::plain(t + base + r0 * (W + 8) + g * 16);
  }
};

}  // namespace hla
