// Linear attention with a decay for each head: M_t = exp(g_t) M_{t-1} + k_t v_t^T, o_t = M_t^T q_t.
//
// A piece of P tokens from state M_0, with lg the inclusive sums of g over it (float64, in units of
// log 2) and D_ij = 2^(lg_i - lg_j) for j <= i:
//     o_i = 2^lg_i M_0^T q_i + sum_{j<=i} D_ij (q_i . k_j) v_j
//     M_P = 2^lg_P M_0 + sum_j 2^(lg_P - lg_j) k_j v_j^T
// so a piece is four matrix products: scores K Q^T, Q M, (D o scores) V and K^T (decayed V).
// The gradients are the same recurrence with the roles changed.  With G_t = dL/dM_t (o_t included),
// G_t = exp(g_{t+1}) G_{t+1} + q_t do_t^T, and
//     dq_t = M_t do_t       roles (do, v, k), state M^T, forward
//     dk_t = G_t v_t        roles (v, do, q), state G^T, reversed
//     dv_t = G_t^T k_t      roles (k, q, do), state G, reversed, with dk in one kernel
//     exp(g_t) dL/d(exp g_t) = exp(g_t) <G_t, M_{t-1}>, see la_decay_kernel.
//
// The state lives in the accumulators of the matrix cores: wave w owns columns [32 w, 32 w + 32) and
// all dk rows, and an accumulator tile is the B operand of the next product without leaving its lane.
// float32 tensors run on the float32 matrix instructions.  bf16 tensors enter exactly; what is float32
// enters as bf16 terms, each of which takes 8 bits.  Three of them (24 bits) where the result comes out
// as float32: the decayed values, which enter the states, and the state where the decays' gradient is
// formed from it.  Two (2^-16 at most) where it reaches bf16 outputs only: the state that outputs read and
// the decayed scores.
#include "../../include/hla.h"

#include "operands.hpp"
#include "la.hpp"
#include "kernels.hpp"

namespace hla {

namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr float kLgFloor = -1.0e4f;  // stands for -inf: 2^-14427 is zero in every type used here

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
// exp(g) by way of log 2 in float64; a NaN stays, and below 2^-126 the instruction gives zero
__device__ __forceinline__ float decay_of(float g) {
  return exp2_((float)((double)(g < kLgFloor ? kLgFloor : g) * kLog2e));
}

// The sums lg of one piece and what follows from them, in LDS.
template <int P> struct Decays {
  double lg[P];   // inclusive sums of g, in log 2
  float gam[P];   // 2^lg: what is left of the piece's start
  float w[P];     // 2^(lg_last - lg): what the piece's end has left of each row
  float total;    // 2^lg_last
};

template <int P>
__device__ __forceinline__ void decays(float g, int lane, Decays<P>& d, double* sum) {
  g = g < kLgFloor ? kLgFloor : g;  // NaN stays
  double x = lane < P ? (double)g * kLog2e : 0.0;
#pragma unroll
  for (int o = 1; o < P; o <<= 1) {
    const double y = __shfl_up(x, o, 64);
    if (lane >= o) x += y;
  }
  const double last = __shfl(x, P - 1, 64);
  if (lane < P) {
    d.lg[lane] = x;
    d.gam[lane] = exp2_((float)x);
    d.w[lane] = exp2_((float)(last - x));
  }
  if (lane == 0) d.total = exp2_((float)last);
  *sum += last;
}

template <class T, int DK, int DV, bool OUT, bool EXTRA> struct LaShared {
  using O = La<T>;
  alignas(16) T x1[OUT ? O::template size<DK>() : 8];
  alignas(16) T x2[O::template size<DK>()];
  alignas(16) T x3[O::template size<DV>()];
  alignas(16) T x4[EXTRA ? O::template size<DV>() : 8];
  alignas(16) T sc[OUT ? O::SCORES : 8];
  Decays<O::P> d[2];
  float dot[EXTRA ? DV / 32 : 1][O::P];
};

// s += rows [a0, a0 + 32) of `a` times rows [b0, b0 + 32) of `b`, W columns; eight reads ahead of their four products.
template <int W, class T>
__device__ __forceinline__ void score(f32x16& s, const T* a, const T* b, int base, int a0, int b0) {
  using O = La<T>;
  constexpr int GN = W / O::KG, ST = 4;
#pragma unroll
  for (int g0 = 0; g0 < GN; g0 += ST) {
    typename O::Frag x[ST], y[ST];
#pragma unroll
    for (int g = 0; g < ST; ++g) {
      x[g] = O::template row<W>(a, base, a0, g0 + g);
      y[g] = O::template row<W>(b, base, b0, g0 + g);
    }
    sched_fence();
#pragma unroll
    for (int g = 0; g < ST; ++g) s = O::mma(x[g], y[g], s);
    sched_fence();
  }
}

// A 32 x 32 tile of scores, transposed -- rows j = 32 J + acc_row(e, h), column i = 32 I + c -- so that a
// lane writes runs of one row.  Tile 0: I = J = 0, 1: I = 1, J = 0, 2: I = J = 1.
__device__ __forceinline__ int tile_i(int tile) { return tile ? 1 : 0; }
__device__ __forceinline__ int tile_j(int tile) { return tile == 2 ? 1 : 0; }

// D_ij.  Selects and no branches: every sum is read, and what lies behind i becomes 2^-inf.
template <int P>
__device__ __forceinline__ void tile_decays(float (&D)[16], const Decays<P>& d, int tile, int c, int h) {
  const int ii = 32 * tile_i(tile) + c, last = ii - 32 * tile_j(tile) - 4 * h;
  const double lgi = d.lg[ii];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float x = (float)(lgi - d.lg[32 * tile_j(tile) + acc_row(e, h)]);
    D[e] = exp2_(acc_row(e, 0) <= last ? x : -INFINITY);
  }
}

// s D into the piece's scores (rows i, columns j); what lies behind i is zero whatever s is.
template <class T>
__device__ __forceinline__ void put_scores(T* sc, const f32x16& s, const float (&D)[16], int tile, int c, int h) {
  const int last = 32 * tile_i(tile) + c - 32 * tile_j(tile) - 4 * h;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = acc_row(4 * q + e, 0) <= last ? s[4 * q + e] * D[4 * q + e] : 0.f;
    T* to = sc + La<T>::score_at(tile, c, q, h);
#pragma unroll
    for (int t = 0; t < La<T>::SCORE_TERMS; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const T y = (T)x[e];
        to[t * La<T>::SCORE_TERM + e] = y;
        x[e] -= (float)y;
      }
  }
}

// What the piece's start gives: acc = X1 M (the first MT tiles of M), the rows scaled by what is left of
// it.  The rows of a step (ST groups) are asked for a step ahead.
template <int W, int TERMS, int ST, class T, int NM, int IT>
__device__ __forceinline__ void inter(f32x16 (&acc)[IT], const f32x16 (&M)[NM], const T* x1, const Decays<La<T>::P>& d,
                                      int base, int h) {
  using O = La<T>;
  constexpr int GT = 32 / O::KG, STEPS = W / O::KG / ST;
#pragma unroll
  for (int I = 0; I < IT; ++I) acc[I] = zero16();
  typename O::Frag q[2][IT][ST];
  auto ask = [&](int step) {
#pragma unroll
    for (int I = 0; I < IT; ++I)
#pragma unroll
      for (int g = 0; g < ST; ++g) q[step & 1][I][g] = O::template rowc<W>(x1, base, 32 * I, step * ST + g);
  };
  ask(0);
#pragma unroll
  for (int step = 0; step < STEPS; ++step) {
    if (step + 1 < STEPS) ask(step + 1);
    sched_fence();
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      const int g = step * ST + k;
      typename O::Vals x;
      typename O::Frag f[TERMS];
#pragma unroll
      for (int e = 0; e < O::FN; ++e) x[e] = M[g / GT][O::FN * (g % GT) + e];
      O::split(x, f);
#pragma unroll
      for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
        for (int I = 0; I < IT; ++I) acc[I] = O::mma(q[step & 1][I][k], f[t], acc[I]);
    }
    sched_fence();
  }
#pragma unroll
  for (int I = 0; I < IT; ++I)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[I][e] *= d.gam[32 * I + acc_row(e, h)];
}

template <int IT> __device__ __forceinline__ void clear(f32x16 (&acc)[IT]) {
#pragma unroll
  for (int I = 0; I < IT; ++I) acc[I] = zero16();
}

// to[row] = sum over the wave's 32 columns of acc times the tile x4, for every row of the piece.
template <int W, class T, int IT>
__device__ __forceinline__ void row_dots(const f32x16 (&acc)[IT], const T* x4, float* to, int base, int lane, int c, int h) {
  float x[16 * IT];
#pragma unroll
  for (int I = 0; I < IT; ++I) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[16 * I + e] = acc[I][e] * La<T>::template acc_el<W>(x4, base, I, e);
    sched_fence();
  }
  const float dot = rows_to_lanes(x, lane);
  if (c < 16 * IT) to[32 * (c >> 4) + acc_row(c & 15, h)] = dot;
}

// The piece joins the state: M = total M + X2^T (w o X3), and with OUT the scores meet the values, acc +=
// scores X3, for columns [32 w, 32 w + 32) of X3.  The values are asked for a step ahead, the keys in
// front of the conversions.
template <int WK, int WV, bool OUT, class T, int NM, int IT>
__device__ __forceinline__ void absorb(f32x16 (&M)[NM], f32x16 (&acc)[IT], const T* x2, const T* x3, const T* scores,
                                       const Decays<La<T>::P>& d, int ck, int cv, int w, int c, int h) {
  using O = La<T>;
  using Frag = typename O::Frag;
  constexpr int GN = O::P / O::KG, MT = WK / 32;
  const float total = d.total;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 16; ++e) M[m][e] *= total;
  Frag v = O::template col<WV>(x3, cv, w, 0);
#pragma unroll
  for (int g = 0; g < GN; ++g) {
    typename O::Vals x;
    Frag f[O::TERMS], k[MT], vn = v;
    const int k0 = O::col_k(g, h);
#pragma unroll
    for (int e = 0; e < O::FN; ++e) x[e] = d.w[k0 + e];
#pragma unroll
    for (int m = 0; m < MT; ++m) k[m] = O::template col<WK>(x2, ck, m, g);
    if (g + 1 < GN) vn = O::template col<WV>(x3, cv, w, g + 1);
    sched_fence();
#pragma unroll
    for (int e = 0; e < O::FN; ++e) x[e] *= (float)v[e];
    O::split(x, f);
#pragma unroll
    for (int t = O::TERMS - 1; t >= 0; --t)
#pragma unroll
      for (int m = 0; m < MT; ++m) M[m] = O::mma(k[m], f[t], M[m]);
    if constexpr (OUT) {
      sched_fence();  // the scores take the keys' registers
#pragma unroll
      for (int I = 0; I < IT; ++I)
        if (g * O::KG < 32 * (I + 1)) {
          Frag sc[O::SCORE_TERMS];
#pragma unroll
          for (int t = 0; t < O::SCORE_TERMS; ++t) sc[t] = O::score_row(scores, I, c, g, h, t);
#pragma unroll
          for (int t = O::SCORE_TERMS - 1; t >= 0; --t) acc[I] = O::mma(sc[t], v, acc[I]);
        }
    }
    v = vn;
    sched_fence();
  }
}

// A piece's outputs, columns W wide, 32 of them a wave.  `out`: the piece's first token of this head;
// `rows` tokens lie in the tensor and `live` in the sequence (the rest are zero).  Rows 32 I + 8 q + 4 h + e:
// the lane's offset holds 4 h, a uniform pointer walks the rest.
template <bool REV, int P, class T, int IT>
__device__ __forceinline__ void put_out(f32x16 (&acc)[IT], void* out, bool f32, int stride, int rows, int live, int col, int h) {
  // whether row 32 I + acc_row(e, h) is one of the first n tokens, by one bound a lane
  auto among = [](int n, int h) { return REV ? P - 4 * h - n : n - 4 * h; };
  auto in = [](int I, int e, int bound) { return REV ? 32 * I + acc_row(e, 0) >= bound : 32 * I + acc_row(e, 0) < bound; };
  const unsigned off = (unsigned)((REV ? 4 - 4 * h : 4 * h) * stride + col);
  if (live < P) {
    const int bound = among(live, h);
#pragma unroll
    for (int I = 0; I < IT; ++I)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[I][e] = in(I, e, bound) ? acc[I][e] : 0.f;
  }
  const int bound = among(rows, h);
  auto put = [&](auto* to, auto whole) {
    using TO = std::remove_pointer_t<decltype(to)>;
    TO* at = to + (REV ? (int64_t)(P - 5) * stride : 0);
#pragma unroll
    for (int I = 0; I < IT; ++I)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (decltype(whole)::value || in(I, e, bound)) at[off] = (TO)acc[I][e];
        const int step = e % 4 == 3 ? 5 : 1;
        at += REV ? -(step * stride) : step * stride;
      }
  };
  if (rows == P) {
    if (f32) put(static_cast<float*>(out), std::true_type{});
    else put(static_cast<T*>(out), std::true_type{});
  } else {
    if (f32) put(static_cast<float*>(out), std::false_type{});
    else put(static_cast<T*>(out), std::false_type{});
  }
}

// 16-byte pieces that a thread of NT moves of a P x W tile.  It moves the same columns of every RS-th row,
// so its addresses are one 32-bit offset (64 rows of heads * width elements stay below 2^31 bytes: the host
// checks) from uniform pointers.
template <int NT, int P, int W, bool REV, class T> struct Mover {
  static constexpr int V = 16 / (int)sizeof(T), CPR = W / V, RS = NT / CPR, ALL = P * CPR, N = (ALL + NT - 1) / NT;
  static_assert(NT % CPR == 0, "a thread keeps its columns");
  __device__ __forceinline__ static void load(const T* base, int heads, int64_t p, int64_t Tb, int tid, u32x4* regs) {
    const int stride = own_s(heads * W);
    const int r0 = own(tid) / CPR, t0 = REV ? P - 1 - r0 : r0;
    const unsigned col = (unsigned)(tid % CPR * V);
    const T* at = base + p * P * stride;
    const int64_t left = Tb - p * P;
    if (left >= P) {
      const unsigned off = (unsigned)(t0 * stride) + col;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const T* u = REV ? at : at + (int64_t)(RS * i) * stride;
        const unsigned o = REV ? off - (unsigned)(RS * i * stride) : off;
        if (ALL % NT == 0 || i + 1 < N || r0 + RS * i < P) regs[i] = *reinterpret_cast<const u32x4*>(u + o);
      }
    } else {  // the last piece: rows behind the sequence are read from its first token and become zero
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int t = REV ? t0 - RS * i : t0 + RS * i;
        const bool in = t >= 0 && t < left;
        const u32x4 x = *reinterpret_cast<const u32x4*>(at + (unsigned)((in ? t : 0) * stride) + col);
        regs[i] = in ? x : u32x4{0, 0, 0, 0};
      }
    }
  }
  __device__ __forceinline__ static void store(T* tile, int tid, const u32x4* regs) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = i * NT + tid;
      if (ALL % NT == 0 || id < ALL) *reinterpret_cast<u32x4*>(tile + La<T>::template at<W>(id / CPR, id % CPR * V)) = regs[i];
    }
  }
};

// Columns `col` of a state of MT tiles of 32 rows, W columns wide, from memory: as it is, or turned (stored
// [W, 32 MT]: a lane's rows come in runs of four).
template <int MT, int W, int NM>
__device__ __forceinline__ void load_state(f32x16 (&M)[NM], const float* s0, bool turned, int col, int h) {
  if (turned) {
    const float* at = s0 + col * (32 * MT) + 4 * h;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(at + 32 * m + 8 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) M[m][4 * q + e] = x[e];
      }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) M[m][e] = s0[(32 * m + acc_row(e, h)) * W + col];
  }
}

template <int IT> constexpr int kTiles = IT == 2 ? 3 : 1;  // score tiles on and below the diagonal

// One workgroup of DV / 32 waves runs one segment of one row.  OUT: outputs from the state in front
// of the segment; else the segment's state (from init, or zero).  EXTRA: the products with x4 that
// the decays' gradient takes (`dot`).
//
// The next piece's tiles are asked for as this one's registers are stored to LDS, so a workgroup always has a
// piece in flight; two workgroups a compute unit (their LDS) cover each other's barriers.  65536 tokens of 16
// heads of 128 x 128 (bf16, 32 segments a row): the states 132 us for 540 MB (4.1 TB/s, matrix cores 40%
// busy), the outputs 317 us for 1.1 GB (3.5 TB/s, 34%) as the profiler has them (285 and 124 in a stream of
// calls); the loads and stores of the latter alone took 234, so memory bounds both, and the state pass is what
// cutting the rows costs.  13 x 1531 tokens of 12 heads of 64 x 128 (float32, lengths 1 to 1531) 42 and 104
// us: the float32 instructions have a sixteenth of bf16's rate.  What carries it: no branch in the scores
// (504 -> 466 us in all), reads a step ahead of their products, addresses formed again in every piece instead
// of kept (before that the registers spilled: 1640 us).
template <class T, int DK, int DV, bool OUT, bool REV, bool EXTRA>
__global__ __launch_bounds__(DV * 2, DK == 128 && DV == 64 ? 1 : 2) void la_sweep_kernel(LaSweep a) {
  static_assert(!(OUT && REV), "outputs are made forward; la_reverse_kernel makes the reversed ones");
  using O = La<T>;
  constexpr int P = O::P, NT = DV * 2, NW = DV / 32, MT = DK / 32, IT = P / 32;
  __shared__ LaShared<T, DK, DV, OUT, EXTRA> sh;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, h0 = lane >> 5, c0 = lane & 31;
  const int64_t row = blockIdx.x / a.nseg;
  const int seg = blockIdx.x % a.nseg;
  if (!OUT && a.loc && !a.whole && seg == (REV ? 0 : a.nseg - 1)) return;  // no segment starts behind it
  const int64_t b = row / a.H;
  const int head = (int)(row % a.H);
  int64_t Tb = a.T;
  if (a.lens) {
    Tb = a.lens[b];
    Tb = Tb < 0 ? 0 : (Tb > a.T ? a.T : Tb);
  }
  const int64_t first = (int64_t)seg * a.seg_pieces;            // this segment's pieces
  int64_t end = first + a.seg_pieces;
  const int64_t all = (a.T + P - 1) / P, live = (Tb + P - 1) / P;
  end = end < all ? end : all;
  const int64_t last = end < live ? end : live;                 // [first, last) hold tokens
  const int64_t n = last > first ? last - first : 0;

  const int G1 = (int)(a.H / (a.x1.heads ? a.x1.heads : 1)), G2 = (int)(a.H / a.x2.heads), G3 = (int)(a.H / a.x3.heads);
  const T* p1 = OUT ? (const T*)a.x1.p + (b * a.x1.ld * a.x1.heads + head / G1) * DK : nullptr;
  const T* p2 = (const T*)a.x2.p + (b * a.x2.ld * a.x2.heads + head / G2) * DK;
  const T* p3 = (const T*)a.x3.p + (b * a.x3.ld * a.x3.heads + head / G3) * DV;
  const T* p4 = nullptr;
  if constexpr (EXTRA) p4 = (const T*)a.x4.p + (b * a.x4.ld * a.x4.heads + head / (int)(a.H / a.x4.heads)) * DV;
  const float* gp = a.per_head ? a.g + head : a.g + b * a.ld_g * a.H + head;

  // row r of piece p is token P p + r, or (reversed) counted from the piece's end, with the decay behind it
  auto load_g = [&](int64_t p) -> float {
    if (lane >= P) return 0.f;
    const int64_t t = p * P + (REV ? P - lane : lane);
    return t < Tb ? (a.per_head ? gp[0] : gp[t * a.H]) : 0.f;
  };
  using ML1 = Mover<NT, P, DK, REV, T>;
  using ML3 = Mover<NT, P, DV, REV, T>;
  u32x4 r1[OUT ? ML1::N : 1], r2[ML1::N], r3[ML3::N], r4[EXTRA ? ML3::N : 1];
  // x1 and x4 are done with sooner than the others; their next tiles are asked for then (back), since
  // registers are short until then
  auto load = [&](int64_t p, bool front, bool back) {
    if constexpr (OUT) if (back) ML1::load(p1, a.x1.heads, p, Tb, tid, r1);
    if (front) ML1::load(p2, a.x2.heads, p, Tb, tid, r2);
    if (front) ML3::load(p3, a.x3.heads, p, Tb, tid, r3);
    if constexpr (EXTRA) if (back) ML3::load(p4, a.x4.heads, p, Tb, tid, r4);
  };
  auto store = [&]() {
    if constexpr (OUT) ML1::store(sh.x1, tid, r1);
    ML1::store(sh.x2, tid, r2);
    ML3::store(sh.x3, tid, r3);
    if constexpr (EXTRA) ML3::store(sh.x4, tid, r4);
  };
  auto piece = [&](int64_t i) { return REV ? last - 1 - i : first + i; };

  f32x16 M[MT];
  const int col = 32 * w + c0;
  if (a.init) {
    load_state<MT, DV>(M, a.init + row * a.init_row + (int64_t)seg * DK * DV, a.init_t, col, h0);
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m) M[m] = zero16();
  }

  const int rk0 = O::template row_base<DK>(lane);
  const int rc0 = O::template rowc_base<DK>(lane), ck0 = O::template col_base<DK>(lane), cv0 = O::template col_base<DV>(lane),
            xa0 = O::template acc_base<DV>(lane, col);
  (void)rk0; (void)rc0;
  double decay = 0.0;
  float gnext = 0.f;  // two pieces ahead and in front of the tiles: memory answers in order, and the sums
  if (n) {            // of the next piece must not wait for its tiles
    float g0 = 0.f;
    if (w == NW - 1) {
      g0 = load_g(piece(0));
      if (n > 1) gnext = load_g(piece(1));
    }
    load(piece(0), true, true);
    if (w == NW - 1) decays<P>(g0, lane, sh.d[0], &decay);
  }
  for (int64_t i = 0; i < n; ++i) {
    const int64_t p = piece(i);
    const Decays<P>& d = sh.d[i & 1];
    const int h = own(h0), c = own(c0);  // row indices are formed again in every piece, not kept
    const int rk = own(rk0), rc = own(rc0), ck = own(ck0), cv = own(cv0), xa = own(xa0);
    (void)rk; (void)rc; (void)xa;
    store();
    __syncthreads();
    float gnow;  // a copy made here, where the tiles have arrived anyway, frees gnext for the next load
    asm volatile("v_mov_b32 %0, %1" : "=v"(gnow) : "v"(gnext));
    if (i + 2 < n && w == NW - 1) gnext = load_g(piece(i + 2));
    if (i + 1 < n) load(piece(i + 1), true, false);
    f32x16 acc[IT];
    if constexpr (OUT) {
      for (int tile = w; tile < kTiles<IT>; tile += NW) {
        f32x16 s = zero16();
        float D[16];
        score<DK>(s, sh.x2, sh.x1, rk, 32 * tile_j(tile), 32 * tile_i(tile));
        tile_decays(D, d, tile, c, h);
        put_scores(sh.sc, s, D, tile, c, h);
      }
      if (a.init || i) inter<DK, EXTRA || O::TERMS < 2 ? O::TERMS : 2, 1>(acc, M, sh.x1, d, rc, h);
      else clear(acc);  // the state is zero
      if constexpr (EXTRA) row_dots<DV>(acc, sh.x4, sh.dot[w], xa, lane, c, h);
    }
    if (i + 1 < n && w == NW - 1) decays<P>(gnow, lane, sh.d[(i + 1) & 1], &decay);
    if constexpr (OUT) __syncthreads();
    if (OUT && i + 1 < n) load(piece(i + 1), false, true);
    absorb<DK, DV, OUT>(M, acc, sh.x2, sh.x3, sh.sc, d, ck, cv, w, c, h);
    if constexpr (OUT) {
      const int rows = (int)(a.T - p * P < P ? a.T - p * P : P), live_rows = (int)(Tb - p * P < P ? Tb - p * P : P);
      const int64_t o0 = ((b * a.T + p * P) * a.H + head) * DV;
      void* to = a.out_f32 ? (void*)(static_cast<float*>(a.out) + o0) : (void*)(static_cast<T*>(a.out) + o0);
      put_out<false, P, T>(acc, to, a.out_f32, own_s((int)a.H * DV), rows, live_rows, col, h);
      if constexpr (EXTRA) {
        if (tid < P) {
          const int64_t t = p * P + tid;
          if (t < a.T) {
            float x = 0.f;
            for (int q = 0; q < NW; ++q) x += sh.dot[q][tid];
            a.dot[row * a.T + t] = t < Tb ? x : 0.f;
          }
        }
      }
    }
    __syncthreads();
  }
  if constexpr (OUT) {  // tokens behind the row's length
    const int64_t t0 = (last > first ? last : first) * P, t1 = end * P < a.T ? end * P : a.T;
    for (int64_t t = t0 + tid / DV; t < t1; t += NT / DV) {
      const int64_t at = ((b * a.T + t) * a.H + head) * DV + tid % DV;
      if (a.out_f32) static_cast<float*>(a.out)[at] = 0.f;
      else static_cast<T*>(a.out)[at] = (T)0.f;
    }
    if constexpr (EXTRA)
      for (int64_t t = t0 + tid; t < t1; t += NT) a.dot[row * a.T + t] = 0.f;
  }
  float* to = nullptr;  // a reversed pass has `loc`
  if (REV || a.loc) to = a.loc + row * a.loc_row + (int64_t)seg * DK * DV;
  else if (a.fin && seg == a.nseg - 1) to = a.fin + row * a.fin_row;
  if (to) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) to[(32 * m + acc_row(e, h0)) * DV + col] = M[m][e];
  }
  if (a.decay && tid == NT - 64) a.decay[row * a.nseg + seg] = decay;
}

// The reversed sweep of both gradients that meet behind a token: dk_t = G_t v_t and dv_t = G_t^T k_t.  The
// first DK / 32 waves hold G^T [DV, DK] and give dk (32 columns each), the others G [DK, DV] and give dv; the
// four tiles are read once for both, and with both tiles of scores at hand, E and its sums too (see
// la_decay_kernel).  One workgroup of (DK + DV) / 32 waves a segment.
//
// 4 x 4096 tokens of 16 heads of 128 x 128 (bf16): 183 us for 430 MB (2.3 TB/s), matrix cores 29% busy: eight
// waves of 256 registers fill a compute unit, so nothing covers the two barriers and the score phase, in which
// three of the eight waves work.  It stands for two sweeps that each read all four tiles (a training step 715
// us with them, 563 with it).
template <class T, int DK, int DV> struct LaReverseShared {
  using O = La<T>;
  alignas(16) T q[O::template size<DK>()];
  alignas(16) T k[O::template size<DK>()];
  alignas(16) T v[O::template size<DV>()];
  alignas(16) T o[O::template size<DV>()];
  alignas(16) T sk[O::SCORES];  // scores of dk: v_i . do_j
  alignas(16) T sv[O::SCORES];  // of dv: k_i . q_j
  Decays<O::P> d[2];
  float dot[DK / 32][O::P];
  float erow[3][32], ecol[3][32];
};

template <class T, int DK, int DV>
__global__ __launch_bounds__((DK + DV) * 2, 2) void la_reverse_kernel(LaReverse a) {
  using O = La<T>;
  constexpr int P = O::P, NT = (DK + DV) * 2, NW = NT / 64, KW = DK / 32, IT = P / 32, NM = (DK > DV ? DK : DV) / 32;
  using MK = Mover<NT, P, DK, true, T>;
  using MV = Mover<NT, P, DV, true, T>;
  __shared__ LaReverseShared<T, DK, DV> sh;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, h0 = lane >> 5, c0 = lane & 31;
  const int64_t row = blockIdx.x / a.nseg;
  const int seg = blockIdx.x % a.nseg;
  const int64_t b = row / a.H;
  const int head = (int)(row % a.H), hk = head / (int)(a.H / a.Hk);
  int64_t Tb = a.T;
  if (a.lens) {
    Tb = a.lens[b];
    Tb = Tb < 0 ? 0 : (Tb > a.T ? a.T : Tb);
  }
  const int64_t all = (a.T + P - 1) / P, live = (Tb + P - 1) / P, first = (int64_t)seg * a.seg_pieces;
  const int64_t end = first + a.seg_pieces < all ? first + a.seg_pieces : all, last = end < live ? end : live;
  const int64_t n = last > first ? last - first : 0;
  const T* pq = (const T*)a.q + (b * a.ld_T * a.Hk + hk) * DK;
  const T* pk = (const T*)a.k + (b * a.ld_T * a.Hk + hk) * DK;
  const T* pv = (const T*)a.v + (b * a.ld_T * a.H + head) * DV;
  const T* po = (const T*)a.dO + (b * a.T * a.H + head) * DV;
  const float* gp = a.per_head ? a.g + head : a.g + b * a.ld_T * a.H + head;
  auto load_g = [&](int64_t p) -> float {  // row r is token P - 1 - r of the piece and takes the decay behind it
    if (lane >= P) return 0.f;
    const int64_t t = p * P + P - lane;
    return t < Tb ? (a.per_head ? gp[0] : gp[t * a.H]) : 0.f;
  };
  u32x4 rq[MK::N], rk[MK::N], rv[MV::N], ro[MV::N];
  auto load = [&](int64_t p) {
    MV::load(pv, (int)a.H, p, Tb, tid, rv);
    MV::load(po, (int)a.H, p, Tb, tid, ro);
    MK::load(pq, (int)a.Hk, p, Tb, tid, rq);
    MK::load(pk, (int)a.Hk, p, Tb, tid, rk);
  };
  const bool is_k = w < KW;
  const int wc = is_k ? w : w - KW, col = 32 * wc + c0;
  f32x16 M[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) M[m] = zero16();
  if (a.init) {
    const float* s0 = a.init + row * a.init_row + (int64_t)seg * DK * DV;
    const bool turned = is_k == (a.init_t != 0);  // stored [DV, DK], or [DK, DV] with init_t
    if (is_k) load_state<DV / 32, DK>(M, s0, turned, col, h0);
    else load_state<KW, DV>(M, s0, turned, col, h0);
  }
  const int fk0 = O::template row_base<DK>(lane), fv0 = O::template row_base<DV>(lane);
  const int rk0 = O::template rowc_base<DK>(lane), rv0 = O::template rowc_base<DV>(lane);
  const int ck0 = O::template col_base<DK>(lane), cv0 = O::template col_base<DV>(lane);
  const int xa0 = O::template acc_base<DK>(lane, is_k ? col : c0);
  double decay = 0.0;
  float gnext = 0.f;
  if (n) {
    float g0 = 0.f;
    if (w == NW - 1) {
      g0 = load_g(last - 1);
      if (n > 1) gnext = load_g(last - 2);
    }
    load(last - 1);
    if (w == NW - 1) decays<P>(g0, lane, sh.d[0], &decay);
  }
  for (int64_t i = 0; i < n; ++i) {
    const int64_t p = last - 1 - i;
    const Decays<P>& d = sh.d[i & 1];
    const int h = own(h0), c = own(c0);
    const int ck = own(ck0), cv = own(cv0);
    MV::store(sh.v, tid, rv);
    MV::store(sh.o, tid, ro);
    MK::store(sh.q, tid, rq);
    MK::store(sh.k, tid, rk);
    __syncthreads();
    float gnow;
    asm volatile("v_mov_b32 %0, %1" : "=v"(gnow) : "v"(gnext));
    if (i + 2 < n && w == NW - 1) gnext = load_g(p - 2);
    if (i + 1 < n) load(p - 1);
    for (int tile = w; tile < kTiles<IT>; tile += NW) {
      const int I = tile_i(tile), J = tile_j(tile);
      f32x16 s = zero16(), u = zero16();
      float D[16], x[16], rs = 0.f;
      score<DV>(s, sh.o, sh.v, own(fv0), 32 * J, 32 * I);
      score<DK>(u, sh.q, sh.k, own(fk0), 32 * J, 32 * I);
      tile_decays(D, d, tile, c, h);
      put_scores(sh.sk, s, D, tile, c, h);
      put_scores(sh.sv, u, D, tile, c, h);
      const int before = 32 * I + c - 32 * J - 4 * h;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        x[e] = acc_row(e, 0) < before ? s[e] * D[e] * u[e] : 0.f;
        rs += x[e];
      }
      rs = swap32_sum(rs);
      const float cs = rows_to_lanes(x, lane);
      if (c < 16) sh.ecol[tile][acc_row(c, h)] = cs;
      if (h == 0) sh.erow[tile][c] = rs;
    }
    f32x16 acc[IT];
    if (is_k) {
      if (a.init || i) inter<DV, O::TERMS, 1>(acc, M, sh.v, d, own(rv0), h);
      else clear(acc);
      row_dots<DK>(acc, sh.k, sh.dot[w], own(xa0), lane, c, h);
    } else {
      if (a.init || i) inter<DK, O::TERMS < 2 ? 1 : 2, 1>(acc, M, sh.k, d, own(rk0), h);
      else clear(acc);
    }
    if (i + 1 < n && w == NW - 1) decays<P>(gnow, lane, sh.d[(i + 1) & 1], &decay);
    __syncthreads();
    const int rows = (int)(a.T - p * P < P ? a.T - p * P : P), live_rows = (int)(Tb - p * P < P ? Tb - p * P : P);
    if (is_k) {
      absorb<DV, DK, true>(M, acc, sh.o, sh.q, sh.sk, d, cv, ck, wc, c, h);
      const int heads = a.k_f32 ? (int)a.H : (int)a.Hk;
      const int64_t o0 = ((b * a.T + p * P) * heads + (a.k_f32 ? head : hk)) * DK;
      void* to = a.k_f32 ? (void*)(static_cast<float*>(a.dk) + o0) : (void*)(static_cast<T*>(a.dk) + o0);
      put_out<true, P, T>(acc, to, a.k_f32, own_s(heads * DK), rows, live_rows, col, h);
    } else {
      absorb<DK, DV, true>(M, acc, sh.q, sh.o, sh.sv, d, ck, cv, wc, c, h);
      put_out<true, P, T>(acc, static_cast<T*>(a.dv) + ((b * a.T + p * P) * a.H + head) * DV, false, own_s((int)a.H * DV), rows,
                          live_rows, col, h);
    }
    if (tid < P) {
      const int64_t t = p * P + P - 1 - tid;
      if (t < a.T) {
        float x = 0.f;
        for (int k = 0; k < KW; ++k) x += sh.dot[k][tid];
        const int i5 = tid & 31;
        float y;  // a row of E here is the earlier token's, a column the later one's
        if (IT == 1) y = sh.ecol[0][i5] - sh.erow[0][i5];
        else if (tid < 32) y = sh.ecol[0][i5] + sh.ecol[1][i5] - sh.erow[0][i5];
        else y = sh.ecol[2][i5] - sh.erow[1][i5] - sh.erow[2][i5];
        a.dot[row * a.T + t] = t < Tb ? x : 0.f;
        a.esum[row * a.T + t] = t < Tb ? y : 0.f;
      }
    }
    __syncthreads();
  }
  // tokens behind the row's length
  for (int64_t t = (last > first ? last : first) * P + tid / 64; t < end * P && t < a.T; t += NW) {
    const int64_t at = (b * a.T + t) * (a.k_f32 ? a.H : a.Hk) + (a.k_f32 ? head : hk);
    for (int e = lane; e < DK; e += 64) {
      if (a.k_f32) static_cast<float*>(a.dk)[at * DK + e] = 0.f;
      else static_cast<T*>(a.dk)[at * DK + e] = (T)0.f;
    }
    for (int e = lane; e < DV; e += 64) static_cast<T*>(a.dv)[((b * a.T + t) * a.H + head) * DV + e] = (T)0.f;
    if (lane == 0) {
      a.dot[row * a.T + t] = 0.f;
      a.esum[row * a.T + t] = 0.f;
    }
  }
  if (!is_k && a.dS0 && seg == 0) {
    const float f = Tb > 0 ? decay_of(gp[0]) : 1.f;
#pragma unroll
    for (int m = 0; m < KW; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) a.dS0[row * DK * DV + (32 * m + acc_row(e, h0)) * DV + col] = M[m][e] * f;
  }
}

// The states in front of every segment from the segments' states from zero, in place.  A thread a value,
// eight segments' loads ahead of the chain.  32 segments of 16 rows of 128 x 128: 17 us for 33 MB read and as
// much written (3.9 TB/s).
__global__ __launch_bounds__(256) void la_scan_kernel(LaScan a) {
  const int n = a.dk * a.dv;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / n;
  if (row >= a.rows) return;
  const int i = (int)(id % n);
  float cur = 0.f;
  if (a.init) cur = a.init[row * n + (a.init_t ? (i % a.dv) * a.dk + i / a.dv : i)];
  const int64_t dir = a.reverse ? -(int64_t)n : n;
  float* p = a.state + row * a.state_row + (a.reverse ? (int64_t)(a.nseg - 1) * n : 0) + i;
  const double* d = a.decay + row * a.nseg;
  const int count = a.fin ? a.nseg : a.nseg - 1;  // nothing starts behind the last one
  for (int s0 = 0; s0 < a.nseg; s0 += 8) {
    float own[8], f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < count) {
        own[k] = p[(s0 + k) * dir];
        f[k] = exp2_((float)d[a.reverse ? a.nseg - 1 - s0 - k : s0 + k]);
      }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < a.nseg) {
        p[(s0 + k) * dir] = cur;
        if (s0 + k < count) cur = cur * f[k] + own[k];
      }
  }
  if (a.fin) a.fin[row * a.fin_row + i] = cur;
}

// dL/dg_t = exp(g_t) <G_t, M_{t-1}>.  In a piece with M_0 in front, dM the gradient of its last state
// and gamma the decay of all its tokens, that is
//     gamma <dM, M_0> + sum_{j<t} b_j + sum_{i>=t} c_i + sum_{i>=t>j} E_ij
// (b_j = k_j . the part of dk_j that comes from behind the piece, c_i = q_i . the part of dq_i from in
// front of it, E_ij the score pairs): the double sum is, with e_s row s's sum less column s's, that of -e_s
// over s < t.  With B and C the piece's sums of b and c, the first term X is known from either side,
//     X = <dM, M_P> - B = <gamma dM + ..., M_0> - C,
// and X + C and X + B are the next pieces' whole products in either direction; at both ends of the segment they are
// products of whole states.  Such a chain carries the roundings of all it has summed, where the true X shrinks
// with every decay, and a number that is not finite, so X is taken from the chain that has summed less: m, the
// magnitudes summed so far, stands for its error.  (From the end alone, 540 rows of 900 tokens with a loss on the
// last 40 and decays of 0.1 to 0.3: tokens far in front had roundings of the last ones for values that are below
// float32's range.)  Where
// gamma < 2^-24 and the end's difference is below its roundings X is zero; so it is in the piece that starts from a
// zero state.  A decay that clears the state has gradient 0, one that is NaN a NaN.  One workgroup
// runs one segment, a wave a piece; only the chains are one thread's.  33 us in the step of 4 x 4096 tokens named
// above, most of it the two products of whole states (124 MiB; 23.6 us with the end's alone).
struct Whole { double x, m; };  // a product of whole states, and its magnitudes
template <int P>
__global__ __launch_bounds__(256) void la_decay_kernel(LaDecay a) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x / a.nseg;
  const int seg = blockIdx.x % a.nseg;
  const int64_t b = row / a.H;
  const int head = (int)(row % a.H);
  int64_t Tb = a.T;
  if (a.lens) {
    Tb = a.lens[b];
    Tb = Tb < 0 ? 0 : (Tb > a.T ? a.T : Tb);
  }
  auto g_at = [&](int64_t t) -> float {
    const float g = a.per_head ? a.g[head] : a.g[(b * a.ld_g + t) * a.H + head];
    return g < kLgFloor ? kLgFloor : g;
  };
  auto out = [&](int64_t t) -> float* { return a.dg + (a.per_head ? row * a.T + t : (b * a.T + t) * a.H + head); };
  const int64_t all = (a.T + P - 1) / P, live = (Tb + P - 1) / P, first = (int64_t)seg * a.seg_pieces;
  const int64_t end = first + a.seg_pieces < all ? first + a.seg_pieces : all, last = end < live ? end : live;
  __shared__ Whole part[2][4];
  auto add = [](Whole& s, float u, float v) {
    const double x = (double)u * v;
    s.x += x;
    s.m += fabs(x);
  };
  auto plain = [&](Whole& s, const float* m, const float* r) {  // 4096 divides every dk dv
    for (int i0 = tid; i0 < a.n; i0 += 256 * 16) {
      float u[16], v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        u[e] = m[i0 + 256 * e];
        v[e] = r[i0 + 256 * e];
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) add(s, u[e], v[e]);
    }
  };
  auto turned = [&](Whole& s, const float* m, const float* r) {  // r [dk, dv], m [dv, dk]: 16 x 16 tiles, a lane four values of a row of r
    const int w = a.w, tall = a.n / w, tiles = a.n / 256, k = lane & 15, c = (lane >> 4) * 4;
    for (int t0 = wave; t0 < tiles; t0 += 16) {  // 16 divides the number of tiles
      float4 v[4];
      float u[4][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + 4 * e, k0 = t % (w / 16) * 16 + k, c0 = t / (w / 16) * 16 + c;
        v[e] = *reinterpret_cast<const float4*>(r + k0 * tall + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q) u[e][q] = m[(c0 + q) * w + k0];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        add(s, u[e][0], v[e].x); add(s, u[e][1], v[e].y); add(s, u[e][2], v[e].z); add(s, u[e][3], v[e].w);
      }
    }
  };
  if (first < last) {  // <dM, M> behind the segment, and in front of it
    Whole s[2] = {{0.0, 0.0}, {0.0, 0.0}};
    const float *fwd = a.fwd + (row * (a.nseg + 1) + seg) * (int64_t)a.n, *rev = a.rev + (row * a.nseg + seg) * (int64_t)a.n;
    if (seg + 1 < a.nseg) plain(s[0], fwd + a.n, rev);
    else if (a.dS) turned(s[0], fwd + a.n, a.dS + row * a.n);
    if (seg) plain(s[1], fwd, rev - a.n);
    else if (a.S0) plain(s[1], a.S0 + row * a.n, a.dS0 + row * a.n);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) {
        s[i].x += __shfl_xor(s[i].x, o, 64);
        s[i].m += __shfl_xor(s[i].m, o, 64);
      }
      if (lane == 0) part[i][wave] = s[i];
    }
  }
  // every piece's sums, then the two chains over the pieces, then the pieces' outputs
  __shared__ double sum_b[kLaChain], sum_c[kLaChain], X[kLaChain], X_m[kLaChain];  // the segment's pieces
  __shared__ float mag_b[kLaChain], mag_c[kLaChain], gamma[kLaChain];
  auto take = [&](int64_t p, float& bb, float& cc, float& ee, float& g) {
    const int64_t t = p * P + lane;
    const bool on = lane < P && t < Tb;
    bb = on ? a.b[row * a.T + t] : 0.f;
    cc = on ? a.c[row * a.T + t] : 0.f;
    ee = on ? a.e[row * a.T + t] : 0.f;
    g = on ? g_at(t) : 0.f;
    return on;
  };
  auto whole = [&](int i, int64_t t) {  // the product at a boundary, as the token t behind it leaves it (its decay)
    const double f = t < 0 || t >= Tb ? 1.0 : (double)decay_of(g_at(t));
    Whole s{0.0, 0.0};
    for (int w = 0; w < 4; ++w) {
      s.x += part[i][w].x * f;
      s.m += part[i][w].m * f;
    }
    return s;
  };
  for (int64_t p = first + wave; p < last; p += 4) {
    float bb, cc, ee, g;
    take(p, bb, cc, ee, g);
    double sb = bb, sc = cc, lg = g;
    float mb = fabsf(bb), mc = fabsf(cc);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      sb += __shfl_xor(sb, o, 64);
      sc += __shfl_xor(sc, o, 64);
      lg += __shfl_xor(lg, o, 64);
      mb += __shfl_xor(mb, o, 64);
      mc += __shfl_xor(mc, o, 64);
    }
    if (lane == 0) {
      sum_b[p - first] = sb;
      sum_c[p - first] = sc;
      mag_b[p - first] = mb;
      mag_c[p - first] = mc;
      gamma[p - first] = exp2_((float)(lg * kLog2e));
    }
  }
  __syncthreads();
  if (tid == 0 && first < last) {
    const int n = (int)(last - first);
    const bool zero = first == 0 && !a.S0;  // the first piece starts from a zero state
    Whole s = whole(0, last * P);
#pragma unroll 4
    for (int i = n - 1; i >= 0; --i) {
      const double m = s.m + mag_b[i];
      s.x -= sum_b[i];
      if (zero && i == 0) {
        s = {0.0, 0.0};
      } else if (gamma[i] < 0x1p-24f && fabs(s.x) <= 0x1p-24 * m) {
        s.x = 0.0;
        s.m *= gamma[i] * 0x1p24;
      } else {
        s.m = m;
      }
      X[i] = s.x;
      X_m[i] = s.m;
      s.x += sum_c[i];
      s.m += mag_c[i];
    }
    s = whole(1, seg ? first * P : -1);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      s.x -= sum_c[i];
      s.m += mag_c[i];
      if ((zero && i == 0) || (X_m[i] < (double)INFINITY && !(s.m < X_m[i]))) s = {X[i], X_m[i]};
      else X[i] = s.x;
      s.x += sum_b[i];
      s.m += mag_b[i];
    }
  }
  __syncthreads();
  for (int64_t p = first + wave; p < last; p += 4) {
    float bb, cc, ee, g;
    const bool on = take(p, bb, cc, ee, g);
    const double own_before = (double)bb - ee;
    double before = own_before, behind = cc;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double y = __shfl_up(before, o, 64), z = __shfl_down(behind, o, 64);
      if (lane >= o) before += y;
      if (lane + o < 64) behind += z;
    }
    const int64_t t = p * P + lane;
    if (lane < P && t < a.T) *out(t) = on && decay_of(g) != 0.f ? (float)(X[p - first] + (before - own_before) + behind) : 0.f;
  }
  for (int64_t t = (last > first ? last : first) * P + tid; t < end * P && t < a.T; t += 256) *out(t) = 0.f;
}

// The gradient of one decay for each head: the sum over its rows' tokens, in a fixed order.  One workgroup a head
// walks the batch's rows one behind another, so short rows cost it most: 4096 rows of 8 tokens of 2 heads make the
// backward call 302 us with a decay for each token and 1051 with one a head, 1024 x 64 of 16 heads 584 and 858, 32 x 4096
// of 16 heads 1174 and 1163.
__global__ __launch_bounds__(1024) void la_head_sum_kernel(const float* x, float* y, int64_t B, int64_t H, int64_t T) {
  double s = 0.0;
  for (int64_t b = 0; b < B; ++b)
    for (int64_t t = threadIdx.x; t < T; t += 1024) s += x[(b * H + blockIdx.x) * T + t];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  __shared__ double part[16];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) s += part[i];
    y[blockIdx.x] = (float)s;
  }
}

// Gradients of shared heads: the sum over each group of the heads' float32 gradients.
template <class T>
__global__ __launch_bounds__(256) void la_group_sum_kernel(LaGroup a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = (int64_t)a.heads * a.width / 4;
  if (id >= a.tokens * per) return;
  const int64_t t = id / per;
  const int e = (int)(id % per) * 4, head = e / a.width, i = e % a.width;
  const float* p = a.x + (t * a.heads * a.group + (int64_t)head * a.group) * a.width + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int g = 0; g < a.group; ++g) {
    const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)g * a.width);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  T* y = static_cast<T*>(a.y) + t * a.heads * a.width + e;
  y[0] = (T)s.x; y[1] = (T)s.y; y[2] = (T)s.z; y[3] = (T)s.w;
}

// One token of every row: the state is read, updated and written in one pass.  A thread's loads of the state
// (16 bytes each) are all in flight before the first product.  256 sequences of 16 heads of 128 x 128: 80 us
// for 540 MB (6.7 TB/s), at the memory's rate; one sequence 5.1 us, of which a launch is most.
template <class T, int DK, int DV>
__global__ __launch_bounds__(256) void la_step_kernel(LaStep a) {
  constexpr int CPR = DV / 4, RPP = 256 / CPR, NP = DK / RPP;
  const int tid = threadIdx.x, col = (tid % CPR) * 4, r0 = tid / CPR;
  const int64_t row = blockIdx.x;
  const int head = (int)(row % a.H);
  const int64_t krow = row / a.H * (a.H / a.group) + head / a.group;
  const T* q = static_cast<const T*>(a.q) + krow * DK;
  const T* k = static_cast<const T*>(a.k) + krow * DK;
  const T* v = static_cast<const T*>(a.v) + row * DV + col;
  float* S = a.S + row * DK * DV + col;
  const float decay = decay_of(a.per_head ? a.g[head] : a.g[row]);
  const float4 vv = make_float4((float)v[0], (float)v[1], (float)v[2], (float)v[3]);
  float4 m[NP], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int p = 0; p < NP; ++p) m[p] = *reinterpret_cast<const float4*>(S + (p * RPP + r0) * DV);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = p * RPP + r0;
    const float kr = (float)k[r], qr = (float)q[r];
    m[p].x = decay * m[p].x + kr * vv.x; m[p].y = decay * m[p].y + kr * vv.y;
    m[p].z = decay * m[p].z + kr * vv.z; m[p].w = decay * m[p].w + kr * vv.w;
    o.x += qr * m[p].x; o.y += qr * m[p].y; o.z += qr * m[p].z; o.w += qr * m[p].w;
    *reinterpret_cast<float4*>(S + r * DV) = m[p];
  }
  __shared__ float4 red[RPP][CPR];
  red[r0][tid % CPR] = o;
  __syncthreads();
  if (tid < DV) {
    float s = 0.f;
    for (int r = 0; r < RPP; ++r) s += reinterpret_cast<const float*>(red[r])[tid];
    static_cast<T*>(a.o)[row * DV + tid] = (T)s;
  }
}

template <class T, int DK, int DV, bool OUT, bool REV, bool EXTRA>
hipError_t sweep(const LaSweep& a, hipStream_t s) {
  static_assert(2 * sizeof(LaShared<T, DK, DV, OUT, EXTRA>) <= 160 * 1024, "two workgroups share a compute unit's LDS");
  hipLaunchKernelGGL((la_sweep_kernel<T, DK, DV, OUT, REV, EXTRA>), dim3((unsigned)(a.B * a.H * a.nseg)), dim3(DV * 2), 0, s, a);
  return hipGetLastError();
}

// the sweeps that there are: states of segments in both directions; outputs, and outputs with dots, forward
template <class T, int DK, int DV>
hipError_t sweep_d(const LaSweep& a, bool state_only, bool reverse, hipStream_t s) {
  if (state_only) return reverse ? sweep<T, DK, DV, false, true, false>(a, s) : sweep<T, DK, DV, false, false, false>(a, s);
  return a.dot ? sweep<T, DK, DV, true, false, true>(a, s) : sweep<T, DK, DV, true, false, false>(a, s);
}

template <class T, int DK, int DV>
hipError_t reverse_d(const LaReverse& a, hipStream_t s) {
  hipLaunchKernelGGL((la_reverse_kernel<T, DK, DV>), dim3((unsigned)(a.B * a.H * a.nseg)), dim3((DK + DV) * 2), 0, s, a);
  return hipGetLastError();
}

template <class T>
hipError_t reverse_t(const LaReverse& a, int dk, int dv, hipStream_t s) {
  if (dk == 64) return dv == 64 ? reverse_d<T, 64, 64>(a, s) : reverse_d<T, 64, 128>(a, s);
  return dv == 64 ? reverse_d<T, 128, 64>(a, s) : reverse_d<T, 128, 128>(a, s);
}

template <class T>
hipError_t sweep_t(const LaSweep& a, int dk, int dv, bool state_only, bool reverse, hipStream_t s) {
  if (dk == 64) return dv == 64 ? sweep_d<T, 64, 64>(a, state_only, reverse, s) : sweep_d<T, 64, 128>(a, state_only, reverse, s);
  return dv == 64 ? sweep_d<T, 128, 64>(a, state_only, reverse, s) : sweep_d<T, 128, 128>(a, state_only, reverse, s);
}

template <class T>
hipError_t step_t(const LaStep& a, int dk, int dv, hipStream_t s) {
  const dim3 grid((unsigned)(a.Bs * a.H)), block(256);
  if (dk == 64 && dv == 64) hipLaunchKernelGGL((la_step_kernel<T, 64, 64>), grid, block, 0, s, a);
  else if (dk == 64) hipLaunchKernelGGL((la_step_kernel<T, 64, 128>), grid, block, 0, s, a);
  else if (dv == 64) hipLaunchKernelGGL((la_step_kernel<T, 128, 64>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((la_step_kernel<T, 128, 128>), grid, block, 0, s, a);
  return hipGetLastError();
}

unsigned blocks(int64_t n, int per) { return (unsigned)((n + per - 1) / per); }

}  // namespace

int la_piece(int dtype) { return dtype == HLA_BF16 ? La<bf16>::P : La<float>::P; }

hipError_t launch_la_sweep(const LaSweep& a, int dtype, int dk, int dv, bool state_only, bool reverse, hipStream_t s) {
  return dtype == HLA_BF16 ? sweep_t<bf16>(a, dk, dv, state_only, reverse, s) : sweep_t<float>(a, dk, dv, state_only, reverse, s);
}

hipError_t launch_la_reverse(const LaReverse& a, int dtype, int dk, int dv, hipStream_t s) {
  return dtype == HLA_BF16 ? reverse_t<bf16>(a, dk, dv, s) : reverse_t<float>(a, dk, dv, s);
}

hipError_t launch_la_scan(const LaScan& a, hipStream_t s) {
  hipLaunchKernelGGL(la_scan_kernel, dim3(blocks(a.rows * a.dk * a.dv, 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_decay(const LaDecay& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * a.H * a.nseg));
  if (a.piece == 64) hipLaunchKernelGGL(la_decay_kernel<64>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(la_decay_kernel<32>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_head_sum(const float* x, float* y, int64_t B, int64_t H, int64_t T, hipStream_t s) {
  hipLaunchKernelGGL(la_head_sum_kernel, dim3((unsigned)H), dim3(1024), 0, s, x, y, B, H, T);
  return hipGetLastError();
}

hipError_t launch_la_group_sum(const LaGroup& a, int dtype, hipStream_t s) {
  const dim3 grid(blocks(a.tokens * a.heads * a.width / 4, 256));
  if (dtype == HLA_BF16) hipLaunchKernelGGL(la_group_sum_kernel<bf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(la_group_sum_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_la_step(const LaStep& a, int dtype, int dk, int dv, hipStream_t s) {
  return dtype == HLA_BF16 ? step_t<bf16>(a, dk, dv, s) : step_t<float>(a, dk, dv, s);
}

}  // namespace hla
