// Single-token decode over the 8-bit chunk cache.
//
// Per (sequence, head), with the live chunk (At_cur, M_cur) and n cached chunks whose maps are
// held as E_j = A_j - I and B_j (math orientation, 8 bits, one scale each) in time order:
//   M_cur  <- diag(a) M_cur - e (k^T diag(a) M_cur) + k w^T      At_cur likewise, without k w^T
//             (Gated DeltaNet: a = alpha, e = beta k, w = beta v; Gated DeltaNet-2: a, e = b o k,
//             w = w o v)
//   g_j    = sigmoid(log-mean-exp_r(q . r sR_j / sqrt(dk))),  ghat_j = g_j [g_j >= tau]
//   z <- At_cur^T q,  o <- M_cur^T q;  for j = n-1 .. 0:  x = z,
//       o += ghat_j sB_j (B_j x),   z = x + ghat_j sA_j (E_j x),   weight_j += ghat_j
// Chunks with ghat_j = 0 are not read.  (The composition of states, [dv, dk] a chunk, is never
// formed: read backwards, only the vector z passes from chunk to chunk.)
// Many rows: bound by HBM.  256 x 16 rows of 64 chunks (dk = dv = 128, int8, 64 representatives)
// take 1.92 ms: 8.59 GB of maps, 2.15 of representatives and 1.07 of live matrices, read and
// written, are 11.8 GB at 6.2 TB/s (counters: 11.56 GB fetched, 0.54 written).  Few rows: bound by the chain's latency, 0.65 us a chunk at dk = 128 and 0.5 at 64 (LDS
// reads, the product, the sums, the new terms and a barrier, one after the other).
#include <hip/hip_runtime.h>

#include "cache8.hpp"
#include "kernels.hpp"
#include "timing.hpp"

namespace hla {
namespace {

constexpr int kMaxCache = 1024;

// Loads and stores of what a step touches once and the cache hierarchy cannot hold (ordinary loads
// of the maps: 2027 us where these take 1925).
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
// (The vector type matters for an ordinary load too: one of uint4's own components is copied, and so
// waited for, where it is held across a loop.)
__device__ __forceinline__ uint4 load_keep(const uint8_t* p) {
  const u32x4 v = *reinterpret_cast<const u32x4*>(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ float4 load_once(const float* p) {
  const f32x4v v = __builtin_nontemporal_load(reinterpret_cast<const f32x4v*>(p));
  return make_float4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store_once(float* p, float4 x) {
  const f32x4v v = {x.x, x.y, x.z, x.w};
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4v*>(p));
}

// One read + write pass over a live [DK][W] matrix: mat <- diag(a) mat - e u^T + k w^T with
// u = (a o k)^T mat, and out = q^T mat (after) = (a o q)^T mat - (q . e) u + (q . k) w.
// LDS rows: ka = a o k, qa = a o q, a, e, k, and dot = (q . k, q . e); w null for the transition.
// The columns go their own ways, so the matrix may be W columns of a wider one (rows ld apart).  A
// thread holds four columns of every RPP-th row; the sums over rows go across the lanes of a wave,
// then over the waves through LDS (`red`, NT / 64 x 2 W floats).
struct LiveRows {
  const float* ka;
  const float* qa;
  const float* a;
  const float* e;
  const float* k;
  const float* dot;
};
template <int DK, int W, int NT> struct Live {
  static constexpr int CPR = W / 4, RPP = NT / CPR, NP = DK / RPP, NW = NT / 64;
  float4 m[NP];
  __device__ __forceinline__ static int col() { return (threadIdx.x % CPR) * 4; }
  __device__ __forceinline__ static int row0() { return threadIdx.x / CPR; }
  __device__ __forceinline__ void load(const float* mat, int ld) {
#pragma unroll
    for (int p = 0; p < NP; ++p) m[p] = load_once(mat + (p * RPP + row0()) * ld + col());
  }
  __device__ __forceinline__ void sums(const LiveRows& r, float* red) const {
    float u[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const float kr = r.ka[p * RPP + row0()], qr = r.qa[p * RPP + row0()];
      const float x[4] = {m[p].x, m[p].y, m[p].z, m[p].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) { u[i] += kr * x[i]; z[i] += qr * x[i]; }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) { u[i] = stride_sum<CPR>(u[i]); z[i] = stride_sum<CPR>(z[i]); }
    if (lane_id() < CPR) {
      float* at = red + (threadIdx.x >> 6) * 2 * W + col();
      *reinterpret_cast<float4*>(at) = make_float4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<float4*>(at + W) = make_float4(z[0], z[1], z[2], z[3]);
    }
  }
  // column c by one thread: u into red's first row, out
  __device__ __forceinline__ static float finish(const LiveRows& r, const float* w, float* red, int c) {
    float u = 0.f, z = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) { u += red[i * 2 * W + c]; z += red[i * 2 * W + W + c]; }
    red[c] = u;
    return z - r.dot[1] * u + (w ? r.dot[0] * w[c] : 0.f);
  }
  __device__ __forceinline__ void store(float* mat, int ld, const LiveRows& r, const float* w, const float* red) const {
    const float4 uu = *reinterpret_cast<const float4*>(red + col());
    const float4 ww = w ? *reinterpret_cast<const float4*>(w + col()) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = p * RPP + row0();
      const float ar = r.a[i], er = r.e[i], kr = r.k[i];
      float4 n;
      n.x = ar * m[p].x - er * uu.x + kr * ww.x;
      n.y = ar * m[p].y - er * uu.y + kr * ww.y;
      n.z = ar * m[p].z - er * uu.z + kr * ww.z;
      n.w = ar * m[p].w - er * uu.w + kr * ww.w;
      store_once(mat + i * ld + col(), n);
    }
  }
};

// ---- products of stored rows with a float32 vector on the matrix cores
//
// The vector is written as four terms that stand in four columns of the B operand; a 16-row
// product gives every column's sum, and the four sums are added at the end.  The vector units
// would spend a conversion, a multiply-add and a share of a cross-lane sum on every stored
// number; here they see only the sums.
//   int8: the vector as 32-bit fixed point, x = F 2^(e-30) with |x| <= 2^e, and F's four signed
//         bytes as terms.  The stored bytes enter the int8 product as they are, and its int32
//         sums are exact; what is rounded is x, to 2^-30 of 2^e.
//   e4m3: three bf16 terms (and 0), each the leading eight bits of what the ones before left, which
//         hold a float32 exactly; stored numbers converted to bf16 exactly, float32 sums.
// In the product's layout lane l holds row l % 16 and the 16 stored bytes from 64 p + 16 (l / 16)
// on for each p; column l % 16 is term l % 4, and element i of the sums is row 4 (l / 16) + i.
// Loaded like that, 16 neighbouring lanes would touch 16 cache lines (measured: 27 GB/s a CU).
// So a wave loads its 16 rows as they lie, 1 KiB an instruction, and turns them in its own piece
// of LDS, whose 16-byte pieces are swizzled by row so that neither side has bank conflicts.
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4;
typedef __attribute__((__vector_size__(4 * sizeof(int)))) int i32x4;

template <int FMT, int DK> struct Operand;
template <int DK> struct Operand<kI8, DK> {
  static constexpr bool kFixed = true;
  uint8_t t[4][DK + 16];  // 16 bytes of padding: the four terms start in different banks
  using Frag = i32x4;
  // factor of the lane's term in the sums
  __device__ __forceinline__ static float term_unit() {
    return __builtin_bit_cast(float, (unsigned)(127 + 8 * (lane_id() & 3)) << 23);
  }
  // Rows row0 + 4 g .. of x, the same in all 16 lanes of group g; enc = 2^(30-e).
  __device__ __forceinline__ void put(int row0, const float (&x)[4], float enc) {
    unsigned f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // F's bytes b_3 (signed) and b_2 .. b_0, less 128 each: F = sum b_i 256^i
      f[i] = (unsigned)(int)(x[i] * enc) + 0x00808080u;
    const unsigned term = lane_id() & 3, sel = (4u + term) << 8 | term;  // byte `term` of two words
    const unsigned lo = __builtin_amdgcn_perm(f[1], f[0], sel), hi = __builtin_amdgcn_perm(f[3], f[2], sel);
    // four lanes of a group have the same term and write the same word
    *reinterpret_cast<unsigned*>(&t[term][row0 + (lane_id() >> 4) * 4]) =
        __builtin_amdgcn_perm(hi, lo, 0x05040100u) ^ (term == 3 ? 0u : 0x80808080u);
  }
  __device__ __forceinline__ Frag get(int p) const {
    return *reinterpret_cast<const i32x4*>(&t[lane_id() & 3][p * 64 + (lane_id() >> 4) * 16]);
  }
  using Acc = i32x4;
  __device__ __forceinline__ static Acc step(const uint4& raw, const Frag& x, Acc acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, raw), x, acc, 0, 0, 0);
  }
};
template <int DK> struct Operand<kE4M3, DK> {
  static constexpr bool kFixed = false;
  bf16 t[4][DK + 8];
  struct Frag { bf16x8 lo, hi; };
  __device__ __forceinline__ static float term_unit() { return 1.f; }
  __device__ __forceinline__ void put(int row0, const float (&x)[4], float) {
    const int term = lane_id() & 3;
    unsigned v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r1 = x[i] - cut(x[i]), r2 = r1 - cut(r1);  // (exact)
      v[i] = __builtin_bit_cast(unsigned, term == 0 ? x[i] : term == 1 ? r1 : term == 2 ? r2 : 0.f);
    }
    *reinterpret_cast<uint2*>(&t[term][row0 + (lane_id() >> 4) * 4]) =  // (the same from four lanes)
        make_uint2(__builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u));
  }
  __device__ __forceinline__ static float cut(float x) {
    return __builtin_bit_cast(float, __builtin_bit_cast(unsigned, x) & 0xffff0000u);
  }
  __device__ __forceinline__ Frag get(int p) const {
    const bf16* at = &t[lane_id() & 3][p * 64 + (lane_id() >> 4) * 16];
    return {*reinterpret_cast<const bf16x8*>(at), *reinterpret_cast<const bf16x8*>(at + 8)};
  }
  using Acc = f32x4;
  __device__ __forceinline__ static Acc step(const uint4& raw, const Frag& x, Acc acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_frag(raw.x, raw.y), x.lo, acc, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_frag(raw.z, raw.w), x.hi, acc, 0, 0, 0);
  }
};

// Sum of the four terms' shares a * unit.  The product is rounded on its own: fused into one of
// the additions it would leave the four lanes with different last bits, and terms split from
// different sums do not add up.
__device__ __forceinline__ float terms_sum(float a, float unit) {
#pragma clang fp contract(off)
  const float x = a * unit;
  return group_sum<4>(x);
}

template <int DK> struct Turn {
  static constexpr int KP = DK / 64, PPR = DK / 16;  // 16-byte pieces to a row
  uint4 t[16 * PPR];
  __device__ __forceinline__ static int piece(int row, int c) { return row * PPR + (c ^ (KP == 2 ? row & 7 : row >> 1 & 3)); }
  // raw[i]: piece l % PPR of row i 64 / PPR + l / PPR; frag[p] as the product takes it
  __device__ __forceinline__ void turn(const uint4 (&raw)[KP], uint4 (&frag)[KP]) {
    const int l = lane_id();
#pragma unroll
    for (int i = 0; i < KP; ++i) t[piece(i * (64 / PPR) + l / PPR, l % PPR)] = raw[i];
    __builtin_amdgcn_wave_barrier();  // the LDS serves a wave's requests in order
#pragma unroll
    for (int p = 0; p < KP; ++p) frag[p] = t[piece(l & 15, 4 * p + (l >> 4))];
    __builtin_amdgcn_wave_barrier();
  }
};

// 2^(30-e) for the least e in reach with bound < 2^e, and its counterpart 2^(e-30) = 1 / enc.
struct Fixed { float enc, dec; };
__device__ __forceinline__ Fixed fixed_for(float bound) {
  int b = (int)(__builtin_bit_cast(unsigned, bound) >> 23) & 0xff;
  b = b < 30 ? 30 : (b > 253 ? 253 : b);
  return {__builtin_bit_cast(float, (unsigned)(283 - b) << 23), __builtin_bit_cast(float, (unsigned)(b - 29) << 23)};
}
// Magnitudes compare as their bits, and what is not finite is above every number.  Fixed point ends
// at 2^127: from there on it makes NaN, as of what is not finite.
constexpr unsigned kFixedEnd = 0x7f000000u;
// Largest over the lanes 16, 32 and 48 apart (the lanes of one 16-lane row hold the same value).
__device__ __forceinline__ unsigned rows_max(unsigned x) {
  auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max_u(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max_u(r[0], r[1]);
}

// A vector that all NW waves can see becomes an operand; returns the factor of its sums (NaN where
// fixed point cannot hold a value).
template <class Op, int DK, int NW> __device__ __forceinline__ float encode(Op& op, const float* src) {
  const int lane = lane_id(), w = threadIdx.x >> 6;
  float m = 0.f, bad = 0.f;
  for (int i = lane; i < DK; i += 64) {
    m = fmaxf(m, fabsf(src[i]));
    bad += Op::kFixed && mag(src[i]) >= kFixedEnd ? __builtin_nanf("") : src[i] * 0.f;
  }
  const Fixed fx = fixed_for(wave_max_valu(m));
  for (int r0 = 16 * w; r0 < DK; r0 += 16 * NW) {
    const float4 x = *reinterpret_cast<const float4*>(src + r0 + (lane >> 4) * 4);
    const float v[4] = {x.x, x.y, x.z, x.w};
    op.put(r0, v, fx.enc);
  }
  return (Op::kFixed ? fx.dec : 1.f) + wave_sum_valu(bad);
}

// The token as the live update takes it, in LDS: thread i fetches element i of everything first
// (no more elements than threads), so that other loads can be asked for before these are waited for.
template <class T, int DK, int DV> struct Token {
  float q[DK], k[DK], a[DK], e[DK], ka[DK], qa[DK], w[DV], dot[2];
  struct Regs { float q, k, dec, erase, w; };
  __device__ __forceinline__ static Regs fetch(const Decode8Args& in, int64_t row) {
    const int i = threadIdx.x;
    Regs r{0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < DK) {
      r.q = to_f<T>(reinterpret_cast<const T*>(in.q)[row * DK + i]);
      r.k = to_f<T>(reinterpret_cast<const T*>(in.k)[row * DK + i]);
      r.dec = in.ga ? in.ga[row * DK + i] : in.alpha[row];
      r.erase = in.ga ? in.gb[row * DK + i] : in.beta[row];
    }
    if (i < DV) r.w = (in.ga ? in.gw[row * DV + i] : in.beta[row]) * to_f<T>(reinterpret_cast<const T*>(in.v)[row * DV + i]);
    return r;
  }
  // (ends before the dots are written: the live update's barrier is theirs too)
  __device__ __forceinline__ LiveRows store(const Regs& r) {
    const int i = threadIdx.x;
    if (i < DK) {
      q[i] = r.q;
      k[i] = r.k;
      a[i] = r.dec;
      ka[i] = r.dec * r.k;
      qa[i] = r.dec * r.q;
      e[i] = r.erase * r.k;
    }
    if (i < DV) w[i] = r.w;
    __syncthreads();
    if (i < 128) {
      const float* s = i < 64 ? k : e;
      float x = 0.f;
      for (int j = lane_id(); j < DK; j += 64) x += q[j] * s[j];
      x = wave_sum_valu(x);
      if (lane_id() == 0) dot[i >> 6] = x;
    }
    return {ka, qa, a, e, k, dot};
  }
};

// A gate counts: skipped below tau, reported, added to its chunk's weight.
__device__ __forceinline__ float take_gate(const Decode8Args& a, int64_t row, int j, float x) {
  const float gh = x >= a.tau ? x : 0.f;
  if (a.gates_out) a.gates_out[row * a.c.n_cap + j] = x;
  if (a.c.weight) a.c.weight[row * a.c.n_cap + j] += gate_mass(gh);
  return gh;
}

// Gates of the positions [lo, hi) whose slots and representatives' scales are slot[j - lo] and
// g[j - lo], which becomes the gate.  The block works through them kScores scores at a time: 16
// representatives a product, then the log-mean-exp by eight lanes a chunk, or a wave where a chunk
// has more than 32 representatives (64 of them by eight lanes took as long as their products).
constexpr int kScores = 1024;  // n_rep <= 256: at least four chunks
template <int FMT, int DK, int NW>
__device__ __forceinline__ void chunk_gates(const Decode8Args& a, int64_t row, int lo, int hi, const int* slot, float* g,
                                            const Operand<FMT, DK>& q, float q_unit, Turn<DK>& turn, float* s_score) {
  using Op = Operand<FMT, DK>;
  constexpr int KP = DK / 64, PPR = DK / 16, NT = NW * 64;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, n_rep = a.c.n_rep;
  typename Op::Frag qf[KP];
#pragma unroll
  for (int p = 0; p < KP; ++p) qf[p] = q.get(p);
  const float qu = q_unit * Op::term_unit();
  const int per = kScores / n_rep;  // chunks a block of scores holds
  const unsigned inv = ((1u << 20) + n_rep - 1) / n_rep;  // r / n_rep = r inv >> 20 for r < 1024, n_rep <= 256
  const uint8_t* reps = a.c.reps + row * a.c.n_cap * (int64_t)n_rep * DK;
  const float unit = 1.f / sqrtf((float)DK);
  for (int j0 = 0; j0 < hi - lo; j0 += per) {
    const int nj = hi - lo - j0 < per ? hi - lo - j0 : per, rows = nj * n_rep;
    // a piece is 16 rows; four of a wave's are on their way, past the end the last row again
    constexpr int AHEAD = 4;
    uint4 ring[AHEAD][KP];
    auto ask = [&](uint4 (&t)[KP], int r0) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        // (the row's representatives span at most 2^25 bytes; every factor fits 24 bits)
        const int at = r0 + i * 8 + lane / PPR, r = at < rows ? at : rows - 1;
        const int jj = (int)(__umul24(r, inv) >> 20);
        t[i] = load_keep(reps + ((unsigned)(__mul24(slot[j0 + jj] - jj, n_rep) + r) * DK + lane % PPR * 16));
      }
    };
    if (w * 16 < rows) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) ask(ring[i], (w + i * NW) * 16);
    }
    for (int base = w * 16; base < rows; base += NW * 16 * AHEAD)
      static_for<0, AHEAD>([&](auto I) __attribute__((always_inline)) {
        const int r0 = base + I * NW * 16;
        uint4 frag[KP];
        turn.turn(ring[I], frag);
        ask(ring[I], r0 + NW * 16 * AHEAD);
        if (r0 < rows) {
          typename Op::Acc acc = {0, 0, 0, 0};
#pragma unroll
          for (int p = 0; p < KP; ++p) acc = Op::step(frag[p], qf[p], acc);
          float s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = terms_sum((float)acc[i], qu);
          if ((lane & 15) == 0)
            *reinterpret_cast<float4*>(s_score + r0 + (lane >> 4) * 4) = make_float4(s[0], s[1], s[2], s[3]);
        }
      });
    __syncthreads();
    auto gates_of = [&](auto lanes) __attribute__((always_inline)) {  // that many lanes a chunk
      constexpr int G = lanes;
      for (int jj = tid / G; jj < nj; jj += NT / G) {
        const float sc = g[j0 + jj] * unit;
        const float* score = s_score + jj * n_rep;
        float m = -INFINITY, sum = 0.f;
        for (int r = tid % G; r < n_rep; r += G) m = fmaxf(m, score[r] * sc);
        if constexpr (G == 64) {
          m = wave_max_valu(m);
        } else {
          m = fmaxf(m, dpp_f<0xB1>(m));
          m = fmaxf(m, dpp_f<0x4E>(m));
          m = fmaxf(m, dpp_f<0x141>(m));
        }
        // (the fast exponential's error is that of the argument's product with log2 e, |x| 2^-24
        // of e^x: for x <= 0 less than 2^-25 of the largest term)
        for (int r = tid % G; r < n_rep; r += G) sum += __expf(score[r] * sc - m);
        sum = lane_group_sum<G>(sum);
        if (tid % G == 0)
          g[j0 + jj] = take_gate(a, row, lo + j0 + jj, 1.f / (1.f + expf(-(m + logf(sum / (float)n_rep)))));
      }
    };
    if (n_rep > 32) gates_of(std::integral_constant<int, 64>{});
    else gates_of(std::integral_constant<int, 8>{});
    __syncthreads();
  }
}

// One workgroup per (sequence, head), a wave for every 16 rows of a chunk's record: dk / 16 waves
// own z with E's rows, dv / 16 own o with B's.  First the live update, the gates (16
// representatives a product, their scores through LDS in blocks of whole chunks), then the chain:
// every wave multiplies its 16 rows with z, and a chunk's new z becomes terms in the other of two
// LDS buffers, so one barrier a chunk is enough.  The raw bytes of the next P chunks are on their
// way to registers meanwhile.  Only z's waves are on the path from one chunk to the next (with both
// parts in the same waves decode_skip took 40 us instead of 34; giving z's waves priority changed nothing).
// int8 needs a bound of |z| before z is known to every wave.  The largest |z| is exchanged with
// the terms, and the next z is at most (1 + |ghat sA| 128 dk) times that; where this factor is
// over 2^7 (a term would then hold fewer than 23 bits of the largest |z|), the waves exchange the
// new maximum first, at the price of a second barrier.
// PART: the chain over one segment of a row's positions for the split form below: gates, live part
// and the z that enters come from the workspace, and o's share goes there.
template <int FMT, class T, int DK, int DV, bool PART>
__global__ __launch_bounds__((DK + DV) * 4) void decode8_kernel(Decode8Args a) {
  using Op = Operand<FMT, DK>;
  constexpr int NZ = DK / 16, NW = NZ + DV / 16, NT = NW * 64, P = 4, KP = DK / 64;
  constexpr int LT = 512;  // threads of the live update, at most NT
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4;
  const int64_t row = PART ? blockIdx.x / a.segs : blockIdx.x;
  constexpr int kRed = 2 * (LT / 64) * (DK + DV);  // the live update's sums, later the chain's lists
  __shared__ __align__(16) float s_o[DV], s_z[DK];
  __shared__ __align__(16) float s_red[kRed > 3 * kMaxCache ? kRed : 3 * kMaxCache];
  __shared__ __align__(16) unsigned s_max[2][NZ];
  __shared__ __align__(16) Op s_x[2];
  // by position: slot, scale of A - I and B, and the scale of the representatives, then the gate
  __shared__ int s_slot[kMaxCache];
  __shared__ float s_sa[kMaxCache], s_sb[kMaxCache], s_g[kMaxCache];
  __shared__ unsigned long long s_on[kMaxCache / 64];
  __shared__ __align__(16) Turn<DK> s_turn[NW];  // each wave's own

  // what depends on nothing is asked for first
  typename Token<T, DK, DV>::Regs token{};
  Live<DK, DV, LT> live_s;
  Live<DK, DK, LT> live_a;
  if constexpr (!PART) {
    token = Token<T, DK, DV>::fetch(a, row);
    if (tid < LT) {
      live_s.load(a.S_cur + row * DK * DV, DV);
      live_a.load(a.At_cur + row * DK * DK, DK);
    }
  }
  const int held = cache8_count(a.c, row), n_cap = a.c.n_cap;
  const int segs = PART ? split_segments(a, held) : 1, seg = PART ? (int)(blockIdx.x % a.segs) : 0;
  if (seg >= segs) return;
  const int lo = seg * a.seg_len, n = segs == 1 ? held : (held - lo < a.seg_len ? held - lo : a.seg_len);
  for (int j = tid; j < n; j += NT) {
    const int slot = cache8_slot(a.c, row, lo + j);
    const float4 sc = a.c.scale[row * n_cap + slot];
    s_slot[j] = slot;
    s_sa[j] = sc.x;
    s_sb[j] = sc.y;
    s_g[j] = PART ? a.ws.gate[row * n_cap + lo + j] : sc.z;
  }
  if constexpr (PART) {
    const float* from = segs == 1 ? a.ws.y + row * DK : a.ws.z + (row * a.segs + seg) * DK;
    if (tid < DK) s_z[tid] = from[tid];
    if (tid < DV) s_o[tid] = segs == 1 ? a.ws.o[row * DV + tid] : 0.f;
  } else {
    __shared__ __align__(16) Token<T, DK, DV> s_token;
    __shared__ __align__(16) float s_score[kScores];
    const LiveRows lr = s_token.store(token);
    const float q_unit = encode<Op, DK, NW>(s_x[1], s_token.q);
    float *red_s = s_red, *red_a = s_red + 2 * (LT / 64) * DV;
    if (tid < LT) {
      live_s.sums(lr, red_s);
      live_a.sums(lr, red_a);
    }
    __syncthreads();
    for (int c = tid; c < DV + DK; c += NT) {
      if (c < DV) s_o[c] = live_s.finish(lr, s_token.w, red_s, c);
      else s_z[c - DV] = live_a.finish(lr, nullptr, red_a, c - DV);
    }
    __syncthreads();
    if (tid < LT) {
      live_s.store(a.S_cur + row * DK * DV, DV, lr, s_token.w, red_s);
      live_a.store(a.At_cur + row * DK * DK, DK, lr, nullptr, red_a);
    }
    if (a.gates_in) {
      for (int j = tid; j < n; j += NT) s_g[j] = take_gate(a, row, j, a.gates_in[row * n_cap + j]);
    } else {
      chunk_gates<FMT, DK, NW>(a, row, 0, n, s_slot, s_g, s_x[1], q_unit, s_turn[w], s_score);
    }
    if (a.gates_out)
      for (int j = n + tid; j < n_cap; j += NT) a.gates_out[row * n_cap + j] = 0.f;
  }
  __syncthreads();
  for (int i = w; i < (n + 63) / 64; i += NW) {
    const int j = 64 * i + lane;
    const unsigned long long on = __ballot(j < n && s_g[j] != 0.f);
    if (lane == 0) s_on[i] = on;
  }
  float unit = encode<Op, DK, NW>(s_x[0], s_z);  // 2^(e-30) of the operand in use
  float acc[4];  // the lane's rows of z, or its terms' shares of its rows of o
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = w < NZ ? s_z[16 * w + g * 4 + i] : 0.f;
  auto share_max = [&](int buf) {
    const unsigned m = rows_max(max_u(max_u(mag(acc[0]), mag(acc[1])), max_u(mag(acc[2]), mag(acc[3]))));
    s_max[buf][w] = m;  // the same from every lane
  };
  auto read_max = [&](int buf) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < NZ; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(&s_max[buf][i]);
      m = max_u(max_u(m, max_u(x.x, x.y)), max_u(x.z, x.w));
    }
    return m;
  };
  if (Op::kFixed && w < NZ) share_max(0);
  __syncthreads();
  // the chunks in use, newest first: slot, ghat sA, ghat sB (in the live update's LDS)
  int* l_slot = reinterpret_cast<int*>(s_red);
  float *l_ca = s_red + kMaxCache, *l_cb = l_ca + kMaxCache;
  int used = 0;
  for (int i = 0; i < (n + 63) / 64; ++i) used += __builtin_popcountll(s_on[i]);
  used = __builtin_amdgcn_readfirstlane(used);
  for (int j = tid; j < n; j += NT) {
    const unsigned long long on = s_on[j >> 6];
    if (!(on >> (j & 63) & 1)) continue;
    int at = __builtin_popcountll(on >> (j & 63)) - 1;
    for (int i = (j >> 6) + 1; i < (n + 63) / 64; ++i) at += __builtin_popcountll(s_on[i]);
    l_slot[at] = s_slot[j];
    l_ca[at] = s_g[j] * s_sa[j];
    l_cb[at] = s_g[j] * s_sb[j];
  }
  __syncthreads();

  // ---- chain
  struct Raw { uint4 t[KP]; };
  const uint8_t* base = a.c.maps + row * n_cap * (int64_t)((DK + DV) * DK);
  const unsigned at = w * 16 * DK + lane * 16;
  auto load = [&](Raw& r, int slot) __attribute__((always_inline)) {
    const uint8_t* m = base + (int64_t)__builtin_amdgcn_readfirstlane(slot) * ((DK + DV) * DK);
#pragma unroll
    for (int p = 0; p < KP; ++p) r.t[p] = load_once(m + (at + p * 1024));
  };
  const float tu = Op::term_unit();
  Raw frag;  // the chunk in work, in the products' layout
  int buf = 0;
  // Chunk `it`.  The product comes first; then the chunk behind (`ring`) is turned and the one P
  // behind that asked for, and the LDS and memory work on those while z is brought up to date.
  auto process = [&](int it, Raw& ring) __attribute__((always_inline)) {
    const bool live = it < used;
    const float ca = live ? l_ca[it] : 0.f, cb = live ? l_cb[it] : 0.f;
    const int slot = l_slot[it + 1 + P < used ? it + 1 + P : used - 1];
    typename Op::Acc sums = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < KP; ++p) sums = Op::step(frag.t[p], s_x[buf].get(p), sums);
    float us = unit * tu;
    Fixed fx{1.f, 1.f};
    bool measure = false;  // (the same in every thread)
    if constexpr (Op::kFixed) {
      const unsigned m = read_max(buf);
      us = m >= kFixedEnd ? __builtin_nanf("") : us;  // and of everything behind it
      const float factor = 1.f + fabsf(ca) * (128.f * DK);
      measure = !(factor <= 128.f);
      fx = fixed_for(__builtin_bit_cast(float, m) * factor);
    }
    buf ^= 1;
    s_turn[w].turn(ring.t, frag.t);
    load(ring, slot);
    if (w < NZ) {
      const float cz = ca * us;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += terms_sum((float)sums[i], cz);
      if (Op::kFixed) share_max(buf);
    } else if (live) {  // each lane keeps its own term's share until the end
      const float co = cb * us;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += co * (float)sums[i];
    }
    if (measure) {
      __syncthreads();
      fx = fixed_for(__builtin_bit_cast(float, read_max(buf)));
    }
    if (w < NZ) s_x[buf].put(16 * w, acc, fx.enc);
    if constexpr (Op::kFixed) unit = fx.dec;
    __syncthreads();
  };
  if (used > 0) {
    Raw ring[P];
    load(frag, l_slot[0]);
#pragma unroll
    for (int i = 0; i < P; ++i) load(ring[i], l_slot[i + 1 < used ? i + 1 : used - 1]);
    {
      const Raw first = frag;
      s_turn[w].turn(first.t, frag.t);
    }
    // Past the end the last chunk is loaded again, and composed with gate 0: a load under a
    // condition would make every wait for a load one for all of them.
    for (int it = 0; it < used; it += P) static_for<0, P>([&](auto I) { process(it + I, ring[I]); });
  }
  if (w >= NZ) {  // o: the live part and the chain's
    const int c = (w - NZ) * 16 + g * 4;
    float* out = (segs == 1 ? a.o + row * DV : a.ws.part + (row * a.segs + seg) * DV) + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sum = group_sum<4>(acc[i]);
      if ((lane & 15) == 0) out[i] = s_o[c + i] + sum;
    }
  }
}

// ---- the split form, for few rows
//
// A chain is a sequence of dependent products on one CU (0.65 us a chunk at dk = 128; the CU draws
// some 50 GB/s), so with few rows most of the card would wait.  The positions are cut into segments of
// seg_len.  For every segment but the oldest all workgroups at once compose the linear parts,
//   Phi_s = product over its chunks, newest first, of (I + ghat sA E),
// a matrix product a chunk instead of a vector's; then one workgroup a row takes z through the
// segments (z <- Phi_s z), and with every segment's z known all segments' chains run at once, their
// shares of o added in a fixed order.
//
// First: the live update by 32-column slices, and the gates by blocks of positions.
template <int FMT, class T, int DK, int DV>
__global__ __launch_bounds__(256) void split_gates_kernel(Decode8Args a) {
  using Op = Operand<FMT, DK>;
  constexpr int NT = 256, LB = (DK + DV) / 32;
  const int blocks = LB + a.gate_blocks, tid = threadIdx.x;
  const int64_t row = blockIdx.x / blocks;
  const int b = (int)(blockIdx.x % blocks);
  __shared__ __align__(16) Token<T, DK, DV> s_token;
  if (b < LB) {
    __shared__ __align__(16) float s_red[NT / 64 * 64];
    const bool state = b < DV / 32;
    const int c0 = (state ? b : b - DV / 32) * 32, ld = state ? DV : DK;
    float* mat = (state ? a.S_cur + row * DK * DV : a.At_cur + row * DK * DK) + c0;
    const typename Token<T, DK, DV>::Regs token = Token<T, DK, DV>::fetch(a, row);
    Live<DK, 32, NT> live;
    live.load(mat, ld);
    const LiveRows lr = s_token.store(token);
    const float* w = state ? s_token.w + c0 : nullptr;
    live.sums(lr, s_red);
    __syncthreads();
    if (tid < 32) (state ? a.ws.o + row * DV : a.ws.y + row * DK)[c0 + tid] = live.finish(lr, w, s_red, tid);
    __syncthreads();
    live.store(mat, ld, lr, w, s_red);
    return;
  }
  const int n = cache8_count(a.c, row), n_cap = a.c.n_cap;
  const int lo = (b - LB) * a.gate_len;
  const int end = lo + a.gate_len < n_cap ? lo + a.gate_len : n_cap, hi = end < n ? end : n;
  if (a.gates_out)
    for (int j = (lo < n ? n : lo) + tid; j < end; j += NT) a.gates_out[row * n_cap + j] = 0.f;
  if (lo >= hi) return;
  if (a.gates_in) {
    for (int j = lo + tid; j < hi; j += NT)
      a.ws.gate[row * n_cap + j] = take_gate(a, row, j, a.gates_in[row * n_cap + j]);
    return;
  }
  __shared__ __align__(16) Op s_x;
  __shared__ __align__(16) Turn<DK> s_turn[NT / 64];
  __shared__ __align__(16) float s_score[kScores];
  __shared__ int s_slot[kMaxCache];
  __shared__ float s_g[kMaxCache];
  for (int j = lo + tid; j < hi; j += NT) {
    const int slot = cache8_slot(a.c, row, j);
    s_slot[j - lo] = slot;
    s_g[j - lo] = a.c.scale[row * n_cap + slot].z;
  }
  for (int i = tid; i < DK; i += NT) s_token.q[i] = to_f<T>(reinterpret_cast<const T*>(a.q)[row * DK + i]);
  __syncthreads();
  const float q_unit = encode<Op, DK, NT / 64>(s_x, s_token.q);
  __syncthreads();
  chunk_gates<FMT, DK, NT / 64>(a, row, lo, hi, s_slot, s_g, s_x, q_unit, s_turn[tid >> 6], s_score);
  for (int j = lo + tid; j < hi; j += NT) a.ws.gate[row * n_cap + j] = s_g[j - lo];
}

// Phi of one segment.  The matrix P (float32, in the accumulators of the 32 x 32 products) starts as
// the identity; a chunk does P <- P + c E P, with E's stored numbers exact in bf16 and P as three
// bf16 terms (24 bits: float32).  Wave w owns P's columns 32 w .., for which an accumulator tile
// is, register for register, the next product's B operand; so P never leaves the wave, and the
// waves share only E, which they bring to LDS as A fragments, a chunk ahead, in two buffers.
// Bound by the products, 3 x 2 dk^3 flops a chunk: 16 rows of 1024 chunks (dk = 128, 0.2 Tflop) take
// 190 us, 1.06 Pflop/s, where a large library product of bf16 matrices reaches 1.21 on this card.
template <int FMT, int DK>
__global__ __launch_bounds__(DK * 2, 2) void split_compose_kernel(Decode8Args a, int rec) {
  constexpr int NT = DK * 2, RT = DK / 32, KS = DK / 16, PER = DK * DK / 16 / NT, FR = 1024 + 16;
  __shared__ __align__(16) uint8_t s_e[2][RT * KS * FR];
  __shared__ int l_slot[kMaxSegment];
  __shared__ float l_ca[kMaxSegment];
  __shared__ int s_used;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, h = lane >> 5;
  const int64_t row = blockIdx.x / (a.segs - 1);
  const int seg = (int)(blockIdx.x % (a.segs - 1)) + 1, n_cap = a.c.n_cap;
  const int held = cache8_count(a.c, row), lo = seg * a.seg_len;
  if (seg >= split_segments(a, held)) return;
  const int n = held - lo < a.seg_len ? held - lo : a.seg_len;
  if (w == 0) {  // chunks in use, newest first (n <= 64)
    const int j = lo + n - 1 - lane;
    const float gh = lane < n ? a.ws.gate[row * n_cap + j] : 0.f;
    const unsigned long long on = __ballot(lane < n && gh != 0.f);
    if (lane < n && gh != 0.f) {
      const int at = __popcll(on & ((1ull << lane) - 1)), slot = cache8_slot(a.c, row, j);
      l_slot[at] = slot;
      l_ca[at] = gh * a.c.scale[row * n_cap + slot].x;
    }
    if (lane == 0) s_used = __popcll(on);
  }
  __syncthreads();
  const int used = __builtin_amdgcn_readfirstlane(s_used);

  f32x16 P[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) P[t][i] = 32 * t + acc_row(i, h) == 32 * w + (lane & 31) ? 1.f : 0.f;

  const uint8_t* base = a.c.maps + row * n_cap * (int64_t)rec;
  uint4 ring[PER];
  auto load = [&](uint4 (&r)[PER], int it) __attribute__((always_inline)) {
    const int slot = __builtin_amdgcn_readfirstlane(l_slot[it < used ? it : used - 1]);
    const uint8_t* m = base + (int64_t)slot * rec;
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = load_once(m + (unsigned)(tid * 16 + i * NT * 16));
  };
  // 16 stored numbers of row r are two lanes' fragments: slot e of lane half h is
  // k = 16 ks + 8 (e / 4) + 4 h + e % 4 (the order in which an accumulator tile holds its rows)
  auto stage = [&](const uint4 (&r)[PER], int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = i * NT + tid, er = u / KS, ks = u % KS;
      uint8_t* at = &s_e[buf][((er >> 5) * KS + ks) * FR + (er & 31) * 16];
      *reinterpret_cast<bf16x8*>(at) = stored_frag<FMT>(r[i].x, r[i].z);
      *reinterpret_cast<bf16x8*>(at + 512) = stored_frag<FMT>(r[i].y, r[i].w);
    }
  };
  auto compose = [&](int it, int buf) __attribute__((always_inline)) {  // (P stays in registers)
    const float ca = l_ca[it];
    bf16x8 b[3][KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint4 pack[3];
      unsigned* word[3] = {&pack[0].x, &pack[1].x, &pack[2].x};
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // terms by cutting off, 8 bits of the significand each: and + subtract
        float x[2] = {P[ks >> 1][(ks & 1) * 8 + 2 * e], P[ks >> 1][(ks & 1) * 8 + 2 * e + 1]};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const unsigned u0 = __builtin_bit_cast(unsigned, x[0]), u1 = __builtin_bit_cast(unsigned, x[1]);
          word[i][e] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);
          x[0] -= __builtin_bit_cast(float, u0 & 0xffff0000u);
          x[1] -= __builtin_bit_cast(float, u1 & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) b[i][ks] = __builtin_bit_cast(bf16x8, pack[i]);
    }
    constexpr int AHEAD = 4;  // fragments on their way from LDS
    bf16x8 f[AHEAD];
    auto get = [&](int i) __attribute__((always_inline)) {
      return *reinterpret_cast<const bf16x8*>(&s_e[buf][i * FR + lane * 16]);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) f[i] = get(i);
    f32x16 d;
    static_for<0, RT * KS>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = I, t = i / KS, ks = i % KS;
      if constexpr (ks == 0) d = zero16();
#pragma unroll
      for (int x = 0; x < 3; ++x) d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % AHEAD], b[x][ks], d, 0, 0, 0);
      if constexpr (i + AHEAD < RT * KS) f[i % AHEAD] = get(i + AHEAD);
      if constexpr (ks == KS - 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) P[t][e] += ca * d[e];
      }
    });
  };
  if (used > 0) {
    load(ring, 0);
    stage(ring, 0);
    load(ring, 1);
    __syncthreads();
    for (int it = 0; it < used; it += 2)
      static_for<0, 2>([&](auto I) __attribute__((always_inline)) {
        if (it + I < used) compose(it + I, I);
        stage(ring, I ^ 1);
        load(ring, it + I + 2);
        __syncthreads();
      });
  }
  float* out = a.ws.phi + ((row * a.segs + seg) * DK + 32 * w + (lane & 31)) * DK + 4 * h;  // column by column
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(out + 32 * t + 8 * i) = make_float4(P[t][4 * i], P[t][4 * i + 1], P[t][4 * i + 2], P[t][4 * i + 3]);
}

// z through a row's segments, newest first: 16 groups of threads take DK / 16 columns of Phi each.
template <int DK>
__global__ __launch_bounds__(DK * 4) void split_join_kernel(Decode8Args a) {
  constexpr int M4 = DK / 4, G = 16, PER = DK / G;
  __shared__ __align__(16) float s_z[DK], s_red[G][DK];
  const int tid = threadIdx.x, m = (tid % M4) * 4, grp = tid / M4;
  const int64_t row = blockIdx.x;
  const int segs = split_segments(a, cache8_count(a.c, row));
  if (segs == 1) return;
  float4 cur[PER], ahead[PER];
  auto load = [&](float4 (&x)[PER], int seg) {
    const float* phi = a.ws.phi + ((row * a.segs + seg) * DK + grp * PER) * DK + m;
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = *reinterpret_cast<const float4*>(phi + i * DK);
  };
  load(ahead, segs - 1);
  if (tid < DK) s_z[tid] = a.ws.y[row * DK + tid];
  __syncthreads();
  for (int seg = segs - 1; seg > 0; --seg) {
#pragma unroll
    for (int i = 0; i < PER; ++i) cur[i] = ahead[i];
    load(ahead, seg > 1 ? seg - 1 : 1);
    if (tid < DK) a.ws.z[(row * a.segs + seg) * DK + tid] = s_z[tid];
    float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float x = s_z[grp * PER + i];
      p.x += x * cur[i].x; p.y += x * cur[i].y; p.z += x * cur[i].z; p.w += x * cur[i].w;
    }
    *reinterpret_cast<float4*>(&s_red[grp][m]) = p;
    __syncthreads();
    if (tid < DK) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) z += s_red[i][tid];
      s_z[tid] = z;
    }
    __syncthreads();
  }
  if (tid < DK) a.ws.z[row * a.segs * DK + tid] = s_z[tid];
}

// o = the live part + every segment's share, newest first.
__global__ __launch_bounds__(128) void split_sum_kernel(Decode8Args a, int dv) {
  const int64_t row = blockIdx.x;
  const int segs = split_segments(a, cache8_count(a.c, row)), c = threadIdx.x;
  if (segs == 1 || c >= dv) return;
  float o = a.ws.o[row * dv + c];
#pragma unroll 8
  for (int s = segs - 1; s >= 0; --s) o += a.ws.part[(row * a.segs + s) * dv + c];
  a.o[row * dv + c] = o;
}

template <int FMT, class T, int DK, int DV>
hipError_t run_decode8(const Decode8Args& a, hipStream_t s) {
  TimedLaunch tl(HLA_KERNEL_DECODE, s);
  const unsigned rows = (unsigned)a.c.rows;
  if (a.segs == 0) {
    hipLaunchKernelGGL((decode8_kernel<FMT, T, DK, DV, false>), dim3(rows), dim3((DK + DV) * 4), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((split_gates_kernel<FMT, T, DK, DV>), dim3(rows * ((DK + DV) / 32 + a.gate_blocks)), dim3(256), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((split_compose_kernel<FMT, DK>), dim3(rows * (a.segs - 1)), dim3(DK * 2), 0, s, a, (DK + DV) * DK);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((split_join_kernel<DK>), dim3(rows), dim3(DK * 4), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((decode8_kernel<FMT, T, DK, DV, true>), dim3(rows * a.segs), dim3((DK + DV) * 4), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(split_sum_kernel, dim3(rows), dim3(128), 0, s, a, DV);
  return hipGetLastError();
}
template <int FMT, class T>
hipError_t pick_decode8(const Decode8Args& a, int dk, int dv, hipStream_t s) {
  if (dk == 64) return dv == 64 ? run_decode8<FMT, T, 64, 64>(a, s) : run_decode8<FMT, T, 64, 128>(a, s);
  return dv == 64 ? run_decode8<FMT, T, 128, 64>(a, s) : run_decode8<FMT, T, 128, 128>(a, s);
}

}  // namespace

// Which form a call takes, from its sizes and whether it scores representatives (n_rep = 0 here where
// the gates are given).  In microseconds, fitted to both forms' times (dk = 128 / 64, n = n_cap
// chunks): one workgroup a row takes (0.65 + 0.0055 n_rep) n / (0.47 + 0.0025 n_rep) n, whatever the
// number of rows up to the CUs'; the split form 42 + 0.1 n / 26 + 0.06 n for its launches and the walk
// over the segments, and 0.0145 n / 0.0033 n for every row (the composition's matrix products, and the
// maps read a second time).  Measured, split and not: dk = 128, n_rep = 2: n = 1024: 1 row 136 and 665,
// 16 rows 346 and 675, 48 rows 808 and 683; n = 128: 8 rows 67 and 94, 32 rows 115 and 97; n = 64: 8
// rows 54 and 51.  n_rep = 64, n = 64, 16 rows: 62 and 71.  dk = 64: n = 512: 64 rows 147 and 265, 128
// rows 270 and 267.  With the gates given: dk = 128, n = 1024: 50 rows 809 and 670, 100 rows 1523 and
// 697; n = 64, 16 rows: 58 and 52; dk = 64, n = 512, 160 rows: 279 and 242.
static bool split_pays(int64_t rows, int n, int n_rep, int dk) {
  const float whole = dk == 128 ? 0.65f + 0.0055f * n_rep : 0.47f + 0.0025f * n_rep;
  const float fixed = dk == 128 ? 42.f + 0.1f * n : 26.f + 0.06f * n, each = dk == 128 ? 0.0145f : 0.0033f;
  return n >= kSplitFrom && rows < 256 && fixed + each * rows * n < whole * n;
}

int64_t plan_decode8(Decode8Args& a, int dk, int dv, void* ws) {
  const int64_t rows = a.c.rows;
  const int n_cap = a.c.n_cap;
  a.segs = 0;
  if (!split_pays(rows, n_cap, a.gates_in ? 0 : a.c.n_rep, dk)) return 0;
  // a segment's composition and its chain take turns with the walk over the segments, at about
  // sqrt(n / 2) of each; and, as far as the longest segment allows, no more than four workgroups of
  // the composition for each CU (up to 64 rows of 1024 chunks; above that they take turns)
  int len = (int)(sqrtf(n_cap / 2.f) + 0.5f);
  const int busy = (int)((rows * n_cap + 1023) / 1024);
  if (len < busy) len = busy;
  a.seg_len = len < 8 ? 8 : (len > kMaxSegment ? kMaxSegment : len);
  a.segs = (n_cap + a.seg_len - 1) / a.seg_len;
  a.gate_len = a.c.n_rep ? 512 / a.c.n_rep : 64;
  a.gate_len = a.gate_len < 1 ? 1 : (a.gate_len > 64 ? 64 : a.gate_len);
  a.gate_blocks = (n_cap + a.gate_len - 1) / a.gate_len;
  int64_t used = 0;
  auto take = [&](int64_t floats) {
    float* p = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + used) : nullptr;
    used += (floats * 4 + 255) / 256 * 256;
    return p;
  };
  a.ws.gate = take(rows * n_cap);
  a.ws.y = take(rows * dk);
  a.ws.o = take(rows * dv);
  a.ws.z = take(rows * a.segs * dk);
  a.ws.part = take(rows * a.segs * dv);
  a.ws.phi = take(rows * a.segs * dk * dk);
  return used;
}

hipError_t launch_decode8(const Decode8Args& a, int fmt, int dtype, int dk, int dv, hipStream_t s) {
  if (fmt == kI8) return dtype == 1 ? pick_decode8<kI8, bf16>(a, dk, dv, s) : pick_decode8<kI8, float>(a, dk, dv, s);
  return dtype == 1 ? pick_decode8<kE4M3, bf16>(a, dk, dv, s) : pick_decode8<kE4M3, float>(a, dk, dv, s);
}

}  // namespace hla
