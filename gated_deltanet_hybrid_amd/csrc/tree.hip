// Trees of drafted tokens over the decode state of a gated delta rule and its cached chunk maps.
//
// Node i with parent p continues p's state (the live state M_0 for p = -1):
//     M_i = alpha_i (I - beta_i k_i k_i^T) M_p + beta_i k_i v_i^T
// With D_ij the product of alpha over the path below ancestor j down to i (1 for j = i), gamma_i the one
// from the live state and L_jl = beta_j D_jl (k_j . k_l) for the strict ancestors l of j, the updates that
// the nodes make solve (I + L) U = diag(beta) V and (I + L) W = diag(beta gamma) K -- parents come before
// their children, so L is strictly lower -- and with P_ij = D_ij (q_i . k_j) over i's ancestors and itself
//     r_i = gamma_i q_i - sum_j P_ij w_j,    o_i = sum_j P_ij u_j + M_0^T r_i,    z_i = At_cur^T r_i.
// The z_i then meet the cached chunks, newest first, with every node's own gates:
//     o_i += g_ij Bc_j^T z_i;   z_i <- z_i + g_ij (At_j^T z_i - z_i)
// so the live matrices and every chunk's maps and representatives are read once for all nodes.
#include "../../include/hla.h"

#include "tree.hpp"
#include "kernels.hpp"
#include "operands.hpp"

namespace hla {

namespace {

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// A lane's node: its ancestors and itself as bits (0 where the node is absent: a parent out of range, or
// an absent ancestor), and the sum of `lg` over them.  Six rounds of pointer doubling by the whole wave.
struct Path { unsigned long long mask; double lg; };
__device__ __forceinline__ Path tree_path(const int32_t* parent, int n, int lane, double lg) {
  int p = lane < n ? parent[lane] : -2;
  int bad = p < -1 || p >= lane;
  p = bad ? -1 : p;
  unsigned long long m = 1ull << lane;
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const int from = p < 0 ? lane : p;
    const unsigned long long pm = __shfl(m, from, 64);
    const double pl = __shfl(lg, from, 64);
    const int pb = __shfl(bad, from, 64), pp = __shfl(p, from, 64);
    if (p >= 0) {
      m |= pm;
      lg += pl;
      bad |= pb;
      p = pp;
    }
  }
  return {bad ? 0ull : m, lg};
}

template <class T, int DK, int DV, int N> struct LiveShared {
  using O = La<T>;
  static constexpr int RD = DK + 4, OD = DV + 4;
  union {
    struct {
      alignas(16) T k[N * O::template rs<DK>()];
      alignas(16) T q[N * O::template rs<DK>()];
    } in;
    struct {
      alignas(16) float r[N * RD];
      alignas(16) float o[N * OD];
    } out;
  };
  alignas(16) float L[N][N + 4], P[N][N + 4];
  double lg[N];
  unsigned long long mask[N];
  float gamma[N], beta[N];
};

// The live part of every node: r, then o = P U + M_0^T r and z = At_cur^T r.  One workgroup a row.
// The solve runs one thread a column (dk of W, dv of U), its values in registers; the live matrices come
// straight from memory, every value to the one lane that multiplies it.  1024 rows of 16 nodes of 128 x 128
// (bf16): 48 us for 170 MB (3.5 TB/s), matrix cores 29% busy; 105 rows of 33 nodes of 64 x 128 (float32) 34 us,
// most of it the solve, whose 64 steps follow one another.
template <class T, int DK, int DV, int N>
__device__ __forceinline__ void live_part(const TreeArgs& a, LiveShared<T, DK, DV, N>& sh, int64_t row) {
  using O = La<T>;
  using S = LiveShared<T, DK, DV, N>;
  constexpr int V = 16 / (int)sizeof(T), NT = (N + 31) / 32, TW = (DK + DV + 127) / 128;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, h = lane >> 5, c = lane & 31;
  const int64_t b = row / a.H;
  const int head = (int)(row % a.H), n = a.n;
  // 32 columns of a live matrix a tile
  const int tiles = DV / 32 + (a.At_cur ? DK / 32 : 0);
  if (w == 0) {
    double lg = 0.0;
    float beta = 0.f;
    if (lane < n) {
      const int64_t at = (b * n + lane) * a.H + head;
      const float l = __log2f(a.alpha[at]);
      lg = l < -1.0e4f ? -1.0e4 : (double)l;  // alpha = 0 clears; NaN stays
      beta = a.beta[at];
    }
    const Path p = tree_path(a.parent + b * n, n, lane, lg);
    if (lane < N) {
      sh.lg[lane] = p.lg;
      sh.mask[lane] = p.mask;
      sh.gamma[lane] = p.mask ? exp2_((float)p.lg) : 0.f;
      sh.beta[lane] = p.mask ? beta : 0.f;
    }
  }
  __syncthreads();
  for (int id = tid; id < N * DK / V; id += 256) {  // absent nodes enter as zeros
    const int i = id / (DK / V), e = id % (DK / V) * V;
    uint4 kk = make_uint4(0, 0, 0, 0), qq = kk;
    if (sh.mask[i]) {
      const int64_t at = ((b * n + i) * a.H + head) * DK + e;
      kk = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + at);
      qq = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + at);
    }
    *reinterpret_cast<uint4*>(sh.in.k + O::template at<DK>(i, e)) = kk;
    *reinterpret_cast<uint4*>(sh.in.q + O::template at<DK>(i, e)) = qq;
  }
  __syncthreads();
  // L and P by 32 x 32 tiles, transposed: rows j, column i
  for (int job = w; job < 2 * NT * NT; job += 4) {
    const int which = job & 1, I = (job >> 1) / NT, J = (job >> 1) % NT;
    if (J > I) continue;
    const int i = (32 * I + c) % N, rb = O::template row_base<DK>(lane % 32 % N + (lane & 32));
    f32x16 s = zero16();
    const T* other = which ? sh.in.q : sh.in.k;
#pragma unroll
    for (int g = 0; g < DK / O::KG; ++g)
      s = O::mma(O::template row<DK>(sh.in.k, rb, 32 * J, g), O::template row<DK>(other, rb, 32 * I, g), s);
    if (32 * I + c < N) {
      const unsigned long long m = sh.mask[i];
      const double lgi = sh.lg[i];
      const float bi = sh.beta[i];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = 32 * J + acc_row(e, h);
        if (j >= N) continue;
        float x = 0.f;
        if ((m >> j) & 1) x = s[e] * exp2_((float)(lgi - sh.lg[j]));
        if (which) sh.P[i][j] = x;
        else sh.L[i][j] = j == i ? 0.f : x * bi;
      }
    }
  }
  __syncthreads();
  float x[N];
  if (tid < DK + DV) {
    const bool is_k = tid < DK;
    const int col = is_k ? tid : tid - DK;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
      if (is_k) s = sh.gamma[i] * (float)sh.in.k[O::template at<DK>(i, col)];
      else if (sh.mask[i]) s = (float)static_cast<const T*>(a.v)[((b * n + i) * a.H + head) * DV + col];
      x[i] = s * sh.beta[i];
    }
    // An update that is not finite belongs to its node and the nodes below it and to no other: it is kept
    // out of the sums, where a zero of L or P would spread it, and put into their results at the end.
    unsigned long long lost = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= n) continue;
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const f32x4 l = *reinterpret_cast<const f32x4*>(&sh.L[i][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < i) x[i] -= l[e] * x[j + e];
      }
      if (!(fabsf(x[i]) < INFINITY)) {
        x[i] = 0.f;
        lost |= 1ull << i;
      }
      sched_fence();
    }
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
      if (i >= n) continue;
      float s = 0.f;
#pragma unroll
      for (int j = 0; j <= i; j += 4) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(&sh.P[i][j]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e <= i) s += p[e] * x[j + e];
      }
      x[i] = (lost & sh.mask[i]) ? __builtin_nanf("") : s;
      sched_fence();
    }
    if (is_k) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = sh.gamma[i] * (float)sh.in.q[O::template at<DK>(i, col)] - x[i];
    }
  }
  __syncthreads();
  if (tid < DK) {
#pragma unroll
    for (int i = 0; i < N; ++i) sh.out.r[i * S::RD + tid] = x[i];
  } else if (tid < DK + DV) {
#pragma unroll
    for (int i = 0; i < N; ++i) sh.out.o[i * S::OD + tid - DK] = x[i];
  }
  __syncthreads();
  // M^T r on the float32 matrix cores
#pragma unroll
  for (int tw = 0; tw < TW; ++tw) {
    const int t = w + 4 * tw;
    if (t >= tiles) continue;
    const bool state = t < DV / 32;
    const int n0 = state ? 32 * t : 32 * t - DV, W = state ? DV : DK;
    const float* M = (state ? a.S_cur + row * DK * DV : a.At_cur + row * DK * DK) + n0 + c;
    f32x16 acc[NT];
#pragma unroll
    for (int I = 0; I < NT; ++I) acc[I] = zero16();
#pragma unroll
    for (int g0 = 0; g0 < DK / 8; g0 += 8) {  // 32 loads a lane at a time
      float m[8][4];
#pragma unroll
      for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[g][e] = M[((g0 + g) * 8 + h * 4 + e) * W];
#pragma unroll
      for (int g = 0; g < 8; ++g) {
#pragma unroll
        for (int I = 0; I < NT; ++I) {
          const f32x4 r = *reinterpret_cast<const f32x4*>(sh.out.r + ((32 * I + c) % N) * S::RD + (g0 + g) * 8 + h * 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[I] = __builtin_amdgcn_mfma_f32_32x32x2f32(m[g][e], r[e], acc[I], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int i = 32 * I + c;
      if (i >= n) continue;
      const bool here = sh.mask[i] != 0;  // an absent node's r is zero, a live value need not be finite
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = n0 + q * 8 + h * 4;
        f32x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = here ? acc[I][4 * q + e] : 0.f;
        if (state) {
          const f32x4 u = *reinterpret_cast<const f32x4*>(sh.out.o + i * S::OD + at);
          *reinterpret_cast<f32x4*>(a.o + ((b * n + i) * a.H + head) * DV + at) = y + u;
        } else {
          *reinterpret_cast<f32x4*>(a.z + (row * n + i) * DK + at) = y;
        }
      }
    }
  }
}

// Gates of every node for the held chunks, a wave a chunk: sigmoid of the log-mean-exp of the node's scores
// over the chunk's representatives, 16 of them (rows) and 16 nodes (columns) a tile.  Exponents are to base
// 2; the next 16 representatives are asked for while these are exponentiated.  1024 rows of 16 nodes, 64 chunks
// of 64 representatives of 128 (bf16): 213 us for 1.07 GB (5.0 TB/s), bound by memory.
template <class T, int DK, int NT>
__device__ __forceinline__ void gates_part(const TreeArgs& a, int64_t row, int part, int per_block) {
  using O = La16<T>;
  using Frag = typename O::Frag;
  constexpr int GN = DK / O::KG, E = O::KG / 4;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, G = lane >> 4, c = lane & 15;
  const int64_t b = row / a.H;
  const int head = (int)(row % a.H), n = a.n;
  int nc = a.n_cache[b];
  nc = nc < 0 ? 0 : (nc > a.n_cap ? a.n_cap : nc);
  const unsigned long long here = __ballot(tree_path(a.parent + b * n, n, lane, 0.0).mask != 0);
  Frag q[NT][GN];
  if (!a.gates_in) {
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int i = 16 * I + c < n ? 16 * I + c : n - 1;
#pragma unroll
      for (int g = 0; g < GN; ++g)
        q[I][g] = O::O::plain(static_cast<const T*>(a.q) + ((b * n + i) * a.H + head) * DK + g * O::KG + G * E);
    }
  }
  const float scale = (float)(1.4426950408889634 / sqrt((double)DK));
  const int end = (part + 1) * per_block < a.n_cap ? (part + 1) * per_block : a.n_cap;
  for (int j = part * per_block + w; j < end; j += 4) {
    float m[NT], sum[NT];
#pragma unroll
    for (int I = 0; I < NT; ++I) { m[I] = -INFINITY; sum[I] = 0.f; }
    if (j < nc && !a.gates_in) {
      const T* reps = static_cast<const T*>(a.reps_cache) + (row * a.n_cap + j) * (int64_t)a.n_rep * DK + G * E;
      Frag k[GN];
      auto ask = [&](int r0) {
        const int r = r0 + c < a.n_rep ? r0 + c : a.n_rep - 1;
#pragma unroll
        for (int g = 0; g < GN; ++g) k[g] = O::O::plain(reps + (int64_t)r * DK + g * O::KG);
      };
      ask(0);
      for (int r0 = 0; r0 < a.n_rep; r0 += 16) {
        f32x4 s[NT];
#pragma unroll
        for (int I = 0; I < NT; ++I) {
          s[I] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int g = 0; g < GN; ++g) s[I] = O::mma(k[g], q[I][g], s[I]);
        }
        if (r0 + 16 < a.n_rep) ask(r0 + 16);
        const int left = a.n_rep - r0 - 4 * G;
#pragma unroll
        for (int I = 0; I < NT; ++I) {
          float top = m[I];
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, e < left ? s[I][e] * scale : -INFINITY);
          float add = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) add += e < left ? exp2_(__builtin_fmaf(s[I][e], scale, -top)) : 0.f;
          sum[I] = sum[I] * (m[I] > -INFINITY ? exp2_(m[I] - top) : 0.f) + add;  // a NaN stays
          m[I] = top;
        }
      }
    }
    unsigned any = 0;
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int i = 16 * I + c;
      float g = 0.f;
      if (j < nc) {
        if (a.gates_in) {
          if (i < n) g = a.gates_in[((b * n + i) * a.H + head) * a.n_cap + j];
        } else {
          float top = m[I], all = sum[I];
#pragma unroll
          for (int o = 16; o <= 32; o <<= 1) {
            const float m2 = __shfl_xor(top, o, 64), s2 = __shfl_xor(all, o, 64), t = fmaxf(top, m2);
            all = all * (top > -INFINITY ? exp2_(top - t) : 0.f) + s2 * (m2 > -INFINITY ? exp2_(m2 - t) : 0.f);
            top = t;
          }
          // 1 / (1 + e^-l) with e^l = 2^top all / n_rep
          const float l2 = top + log2f(all / (float)a.n_rep);
          g = 1.f / (1.f + exp2f(-l2));
          if (all != all) g = all;  // fmaxf drops a NaN score; its sum does not
        }
      }
      const bool on = (here >> i) & 1;
      if (!on) g = 0.f;
      const bool keep = j < nc && on && g >= a.tau;
      if (__any(keep)) any |= 1u << I;
      if (G == 0 && i < n) {
        if (a.gates_out) a.gates_out[((b * n + i) * a.H + head) * a.n_cap + j] = g;
        if (j < nc) a.gate[(row * a.n_cap + j) * n + i] = keep ? g : 0.f;
      }
    }
    if (lane == 0 && j < nc) a.active[row * a.n_cap + j] = (int)any;
  }
}

template <class T, int DK, int NT>
__global__ __launch_bounds__(256) void tree_gates_kernel(TreeArgs a, int per_block) {
  gates_part<T, DK, NT>(a, blockIdx.x, blockIdx.y, per_block);
}

// The two parts need nothing of each other: `parts` workgroups a row, the first the live part's and the
// others (in a launch of few workgroups, which saves one) the gates'.
template <class T, int DK, int DV, int N>
__global__ __launch_bounds__(256) void tree_front_kernel(TreeArgs a, int parts, int per_block) {
  __shared__ LiveShared<T, DK, DV, N> sh;
  const int64_t row = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  if (part == 0) live_part<T, DK, DV, N>(a, sh, row);
  else gates_part<T, DK, N / 16>(a, row, part - 1, per_block);
}

// The chain over the cached chunks, for NT tiles of 16 nodes of a row.  Each of the 8 waves owns tiles of 16
// columns of At (their z, as accumulators: rows the columns, column the node) or of Bc (their o).  bf16 maps
// go through LDS, which hands them out transposed, and z enters as three bf16 terms, float32 to its last
// bit; float32 maps come straight from memory, every value to the one lane that multiplies it.  The chunk
// that is AHEAD read chunks away is asked for while this one is worked on.
//
// 1024 rows of 16 nodes over 64 chunks of 128 x 128 (bf16): 640 us for 4.3 GB (6.7 TB/s), bound by memory.
// 16 rows of 7 nodes over 8 chunks 14.7 us, 1.8 us a chunk: maps and z go through LDS and a barrier, which
// nothing else of a lone workgroup covers.  105 rows of 33 nodes over up to 100 chunks of 64 x 128 (float32) 156 us, the longest row's chain.
template <class T, int DK, int DV, int NT, int AHEAD>
__global__ __launch_bounds__(512, NT == 1 && AHEAD == 1 && sizeof(T) == 2 ? 4 : 2) void tree_chain_kernel(TreeArgs a, int groups) {
  using O = La16<T>;
  using Frag = typename O::Frag;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int N = 16 * NT, TILES = (DK + DV) / 16, AT = DK / 16, TW = (TILES + 7) / 8, GN = DK / O::KG;
  constexpr int RZ = La<T>::template rs<DK>(), LD = BF ? DK * (DK + DV) / 8 / 512 : 1;
  // two buffers in turn where LDS has room for them: no barrier between a wave's reads and its writes of z
  // (7 nodes of 16 rows over 8 chunks, whole call 29.6 -> 28.9 us)
  constexpr int BUF = !BF || AHEAD == 2 ? 2 : 1;
  __shared__ alignas(16) T at_[BF ? BUF * DK * DK : 8], bt_[BF ? BUF * DK * DV : 8];
  __shared__ alignas(16) T zs_[BUF][O::TERMS][N * RZ];
  __shared__ unsigned char act[kTreeSlots];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, G = lane >> 4, c = lane & 15;
  const int64_t row = blockIdx.x / groups, b = row / a.H;
  const int head = (int)(row % a.H), n = a.n, n0 = (int)(blockIdx.x % groups) * N;
  int nc = a.n_cache[b];
  nc = nc < 0 ? 0 : (nc > a.n_cap ? a.n_cap : nc);
  const unsigned mine = ((1u << NT) - 1) << (n0 / 16);
  for (int j = tid; j < nc; j += 512) act[j] = (unsigned char)((a.active[row * a.n_cap + j] & mine) >> (n0 / 16));
  __syncthreads();
  auto next = [&](int j) {
    --j;
    while (j >= 0 && !act[j]) --j;
    return j;
  };
  int j = next(nc);
  if (j < 0) return;  // no node here reads a chunk: o is the live part
  const T* Ac = static_cast<const T*>(a.At_cache) + row * a.n_cap * DK * DK;
  const T* Bc = static_cast<const T*>(a.Bc_cache) + row * a.n_cap * DK * DV;
  u32x4 raw[AHEAD][LD];
  Frag m[AHEAD][BF ? 1 : TW][GN];
  float gn[AHEAD][NT];
  auto load_map = [&](int j, u32x4 (&raw)[LD]) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int id = i * 512 + tid;
      const T* p = id < DK * DK / 8 ? Ac + (int64_t)j * DK * DK + id * 8 : Bc + (int64_t)j * DK * DV + (id - DK * DK / 8) * 8;
      raw[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    }
  };
  auto load_tile = [&](int j, int i, Frag (&m)[GN]) {
    const int t = w + 8 * i;
    if (t >= TILES) return;
    const int W = t < AT ? DK : DV;
    const T* p = t < AT ? Ac + (int64_t)j * DK * DK + 16 * t + c : Bc + (int64_t)j * DK * DV + 16 * (t - AT) + c;
#pragma unroll
    for (int g = 0; g < GN; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) m[g][e] = p[(16 * g + 4 * G + e) * W];
  };
  auto load_gates = [&](int j, float (&gn)[NT]) {
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int node = n0 + 16 * I + c;
      gn[I] = node < n ? a.gate[(row * a.n_cap + j) * n + node] : 0.f;
    }
  };
  int jb[AHEAD + 1] = {j};  // the chunks in hand, and the one to ask for next
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    if (jb[k] >= 0) {
      load_gates(jb[k], gn[k]);
      if constexpr (BF) load_map(jb[k], raw[k]);
      else
#pragma unroll
        for (int i = 0; i < TW; ++i) load_tile(jb[k], i, m[k][i]);
    }
    jb[k + 1] = jb[k] >= 0 ? next(jb[k]) : -1;
  }
  f32x4 v[TW][NT];  // z of this wave's columns of At, or o of its columns of Bc
  int turn = 0;
  auto put_z = [&](int t, int I, f32x4 r) {
#pragma unroll
    for (int s = 0; s < O::TERMS; ++s) {
      T* to = zs_[turn][s] + La<T>::template at<DK>(16 * I + c, 16 * t + 4 * G);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const T x = (T)r[e];
        to[e] = x;
        r[e] -= (float)x;
      }
    }
  };
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const int t = w + 8 * i;
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int node = n0 + 16 * I + c;
      v[i][I] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (t >= TILES) continue;
      if (node < n)
        v[i][I] = t < AT ? *reinterpret_cast<const f32x4*>(a.z + (row * n + node) * DK + 16 * t + 4 * G)
                         : *reinterpret_cast<const f32x4*>(a.o + ((b * n + node) * a.H + head) * DV + 16 * (t - AT) + 4 * G);
    }
  }
#pragma unroll
  for (int i = 0; i < TW; ++i)
    if (w + 8 * i < AT)
#pragma unroll
      for (int I = 0; I < NT; ++I) put_z(w + 8 * i, I, v[i][I]);
  const int rz0 = O::template row_base<DK>(lane);
  auto step = [&](auto buf) {  // the chunk jb[0], whose values are in buffer `buf`
    constexpr int B = decltype(buf)::value;
    const int j = jb[0], ja = jb[AHEAD];
    float g[NT];
#pragma unroll
    for (int I = 0; I < NT; ++I) g[I] = gn[B][I];
    const unsigned read = act[j];
    T *at = at_ + (BF ? turn * DK * DK : 0), *bt = bt_ + (BF ? turn * DK * DV : 0);
    const auto& zs = zs_[turn];
    if constexpr (BF) {
#pragma unroll
      for (int i = 0; i < LD; ++i) {
        const int id = i * 512 + tid;
        if (id < DK * DK / 8) {
          *reinterpret_cast<u32x4*>(at + La<T>::template at<DK>(id / (DK / 8), id % (DK / 8) * 8)) = raw[B][i];
        } else {
          const int k = id - DK * DK / 8;
          *reinterpret_cast<u32x4*>(bt + La<T>::template at<DV>(k / (DV / 8), k % (DV / 8) * 8)) = raw[B][i];
        }
      }
    }
    __syncthreads();
    const int rz = own(rz0);
    if (ja >= 0) {
      load_gates(ja, gn[B]);
      if constexpr (BF) load_map(ja, raw[B]);
    }
    // one chain of products a term where registers allow: a chain waits for each of its products
    constexpr int CH = NT == 1 ? O::TERMS : 1;
    f32x4 acc[TW][NT];
    Frag f[TW][GN];
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const int t = w + 8 * i;
      if (t >= TILES) continue;
#pragma unroll
      for (int k = 0; k < GN; ++k) {
        if constexpr (BF) f[i][k] = t < AT ? O::template col<DK>(at, O::template col_base<DK>(lane), t, k)
                                           : O::template col<DV>(bt, O::template col_base<DV>(lane), t - AT, k);
        else f[i][k] = m[B][i][k];
      }
    }
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      f32x4 part[TW][CH];
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int s = 0; s < CH; ++s) part[i][s] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (NT == 1 || ((read >> I) & 1)) {  // else no node of this tile reads the chunk
#pragma unroll
        for (int k = 0; k < GN; ++k)
#pragma unroll
          for (int s = O::TERMS - 1; s >= 0; --s) {
            const Frag z = O::template row<DK>(zs[s], rz, 16 * I, k);
#pragma unroll
            for (int i = 0; i < TW; ++i)
              if (i == 0 || TILES % 8 == 0 || w + 8 * i < TILES) part[i][s % CH] = O::mma(f[i][k], z, part[i][s % CH]);
          }
      }
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        acc[i][I] = part[i][CH - 1];
#pragma unroll
        for (int s = CH - 2; s >= 0; --s) acc[i][I] += part[i][s];
      }
    }
    if constexpr (!BF) {
      if (ja >= 0) {
#pragma unroll
        for (int i = 0; i < TW; ++i) load_tile(ja, i, m[B][i]);
      }
    }
    if constexpr (BUF == 1) __syncthreads();
    else turn ^= 1;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const int t = w + 8 * i;
      if (t >= TILES) continue;
      const bool isA = t < AT;
#pragma unroll
      for (int I = 0; I < NT; ++I) {
        if (g[I] != 0.f) {  // a node that skips the chunk keeps its values, whatever the chunk holds
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][I][e] += g[I] * (acc[i][I][e] - (isA ? v[i][I][e] : 0.f));
        }
        if (isA) put_z(t, I, v[i][I]);
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) jb[k] = jb[k + 1];
    jb[AHEAD] = ja >= 0 ? next(ja) : -1;
  };
  while (true) {
    step(std::integral_constant<int, 0>{});
    if (jb[0] < 0) break;
    if constexpr (AHEAD > 1) {
      step(std::integral_constant<int, 1>{});
      if (jb[0] < 0) break;
    }
  }
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const int t = w + 8 * i;
    if (t < AT || t >= TILES) continue;
#pragma unroll
    for (int I = 0; I < NT; ++I) {
      const int node = n0 + 16 * I + c;
      if (node < n) *reinterpret_cast<f32x4*>(a.o + ((b * n + node) * a.H + head) * DV + 16 * (t - AT) + 4 * G) = v[i][I];
    }
  }
}

// The accepted path enters the live matrices: a thread holds a whole column (its dk values), so the
// tokens of the path follow one another without any exchange; the matrices are read and written once.  1024
// rows of 128 x 128, paths of up to 16 tokens, a quarter committed: 49 us for 290 MB (5.9 TB/s), bound by
// memory; one sequence 7.9 us, the path's chain.
template <class T, int DK, int DV>
__global__ __launch_bounds__(DK + DV) void tree_accept_kernel(TreeAccept a) {
  __shared__ alignas(16) float ks[kTreeNodes][DK];
  __shared__ float al[kTreeNodes], be[kTreeNodes];
  __shared__ int idx[kTreeNodes];
  __shared__ int len_;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t row = blockIdx.x, b = row / a.H;
  const int head = (int)(row % a.H), n = a.n;
  if (tid < 64) {
    const unsigned long long m = tree_path(a.parent + b * n, n, lane, 0.0).mask;
    const int node = a.node[b];
    const unsigned long long path = __shfl(m, node < 0 || node >= n ? 0 : node, 64);
    const unsigned long long on = node < 0 || node >= n ? 0ull : path;
    if ((on >> lane) & 1) {
      const int at = __popcll(on & ((1ull << lane) - 1));
      idx[at] = lane;
      al[at] = a.alpha[(b * n + lane) * a.H + head];
      be[at] = a.beta[(b * n + lane) * a.H + head];
    }
    if (lane == 0) len_ = __popcll(on);
  }
  __syncthreads();
  const int len = len_;
  bool commit = false;
  int slot = 0;
  if (a.commit && a.commit[b] != 0) {
    slot = a.n_cache[b];
    commit = slot >= 0 && slot < a.n_cap;
  }
  if (!len && !commit) return;
  for (int id = tid; id < len * DK; id += DK + DV)
    ks[id / DK][id % DK] = (float)static_cast<const T*>(a.k)[((b * n + idx[id / DK]) * a.H + head) * DK + id % DK];
  const bool state = tid < DV;
  const int col = state ? tid : tid - DV, W = state ? DV : DK;
  float* p = state ? a.S_cur + row * DK * DV + col : a.At_cur ? a.At_cur + row * DK * DK + col : nullptr;
  float x[DK];
  if (p) {
#pragma unroll
    for (int r = 0; r < DK; ++r) x[r] = p[r * W];
  }
  __syncthreads();
  if (!p) return;
  for (int i = 0; i < len; ++i) {
    const float alpha = al[i], beta = be[i];
    const float v = state ? (float)static_cast<const T*>(a.v)[((b * n + idx[i]) * a.H + head) * DV + col] : 0.f;
    float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < DK; r += 4) {
      const f32x4 k = *reinterpret_cast<const f32x4*>(&ks[i][r]);
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] += k[e] * x[r + e];
    }
    const float add = beta * (v - alpha * ((u[0] + u[1]) + (u[2] + u[3])));
#pragma unroll
    for (int r = 0; r < DK; r += 4) {
      const f32x4 k = *reinterpret_cast<const f32x4*>(&ks[i][r]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[r + e] = alpha * x[r + e] + k[e] * add;
    }
  }
  if (commit) {
    T* to = state ? static_cast<T*>(a.Bc_cache) + (row * a.n_cap + slot) * DK * DV + col
                  : static_cast<T*>(a.At_cache) + (row * a.n_cap + slot) * DK * DK + col;
#pragma unroll
    for (int r = 0; r < DK; ++r) {
      to[r * W] = (T)x[r];
      x[r] = !state && r == col ? 1.f : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < DK; ++r) p[r * W] = x[r];
}

__global__ void tree_advance_kernel(int32_t* n_cache, const int32_t* commit, int32_t n_cap, int64_t Bs) {
  const int64_t b = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (b < Bs && commit[b] != 0 && n_cache[b] >= 0 && n_cache[b] < n_cap) n_cache[b] += 1;
}

template <class T, int DK, int DV, int N>
hipError_t decode_n(const TreeArgs& a, hipStream_t s) {
  const unsigned rows = (unsigned)(a.Bs * a.H);
  // The gates' workgroups take up to 64 chunks of a row, 16 a wave (each starts with the tree's and the
  // queries' loads), and fewer, down to one a wave, as long as there are fewer than 1024 of them: 105 rows of
  // 100 chunks, whole call with 64 a workgroup 228 us, with 16 214, with 4 218.
  int per = 64;
  while (per > 4 && (int64_t)rows * ((a.n_cap + per - 1) / per) < 1024) per /= 2;
  const int gate_parts = a.At_cur ? (a.n_cap + per - 1) / per : 0;
  // Where all fit the chip at once, both are one launch (the live part's registers and LDS would cost the
  // gates of a large batch their place on the compute units): 16 rows, whole call with one launch 30 us, with
  // two 35; 1024 rows 934 and 891.
  const bool together = (int64_t)rows * (1 + gate_parts) <= 256;
  const int parts = together ? 1 + gate_parts : 1;
  hipLaunchKernelGGL((tree_front_kernel<T, DK, DV, N>), dim3(rows * parts), dim3(256), 0, s, a, parts, per);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.At_cur) return e;
  if (!together) {
    hipLaunchKernelGGL((tree_gates_kernel<T, DK, N / 16>), dim3(rows, gate_parts), dim3(256), 0, s, a, per);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // A workgroup takes 1, 2 or 4 tiles of 16 nodes, as few as give each compute unit a workgroup (16 nodes), so
  // that more units work, each reading the maps; many rows: all, so that maps are read once.  40 bf16 maps of
  // 128 x 128, us with 1, 2 and 4 tiles: 100 rows of 32 nodes 132, 144, 100 of 48 226, 180, 206, 200 of 48
  // 351, 298, 221.  Where sequences hold 0 to 40 maps, less is lost: 100 of 32 124, 142, 100 of 48 190, 177,
  // 205, 200 of 48 243, 256, 218.
  const int tiles = (a.n + 15) / 16;
  int per_wg = 1;
  if (tiles > 1 && (int64_t)rows * a.n > 16 * 256) per_wg = 2;
  if (tiles > 2 && (int64_t)rows * ((tiles + 1) / 2) > 256) per_wg = 4;
  const int groups = (tiles + per_wg - 1) / per_wg;
  const dim3 grid(rows * groups);
  // Two chunks ahead where a compute unit has one workgroup at most, whose chain waits for memory; else the
  // registers are better spent on a second workgroup.  10 rows of 437 float32 maps: 452 us one ahead, 432 two;
  // 300 workgroups of 40 bf16 maps 226 and 248.
  if (per_wg == 1 && grid.x <= 256) hipLaunchKernelGGL((tree_chain_kernel<T, DK, DV, 1, 2>), grid, dim3(512), 0, s, a, groups);
  else if (per_wg == 1) hipLaunchKernelGGL((tree_chain_kernel<T, DK, DV, 1, 1>), grid, dim3(512), 0, s, a, groups);
  else if (per_wg == 2) hipLaunchKernelGGL((tree_chain_kernel<T, DK, DV, 2, 1>), grid, dim3(512), 0, s, a, groups);
  else hipLaunchKernelGGL((tree_chain_kernel<T, DK, DV, 4, 1>), grid, dim3(512), 0, s, a, groups);
  return hipGetLastError();
}

template <class T, int DK, int DV>
hipError_t decode_d(const TreeArgs& a, hipStream_t s) {
  if (a.n <= 16) return decode_n<T, DK, DV, 16>(a, s);
  if (a.n <= 32) return decode_n<T, DK, DV, 32>(a, s);
  return decode_n<T, DK, DV, 64>(a, s);
}

template <class T>
hipError_t decode_t(const TreeArgs& a, int dk, int dv, hipStream_t s) {
  if (dk == 64) return dv == 64 ? decode_d<T, 64, 64>(a, s) : decode_d<T, 64, 128>(a, s);
  return dv == 64 ? decode_d<T, 128, 64>(a, s) : decode_d<T, 128, 128>(a, s);
}

template <class T>
void accept_t(const TreeAccept& a, int dk, int dv, hipStream_t s) {
  const dim3 grid((unsigned)(a.Bs * a.H));
  if (dk == 64 && dv == 64) hipLaunchKernelGGL((tree_accept_kernel<T, 64, 64>), grid, dim3(128), 0, s, a);
  else if (dk == 64) hipLaunchKernelGGL((tree_accept_kernel<T, 64, 128>), grid, dim3(192), 0, s, a);
  else if (dv == 64) hipLaunchKernelGGL((tree_accept_kernel<T, 128, 64>), grid, dim3(192), 0, s, a);
  else hipLaunchKernelGGL((tree_accept_kernel<T, 128, 128>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_tree_decode(const TreeArgs& a, int dtype, int dk, int dv, hipStream_t s) {
  return dtype == HLA_BF16 ? decode_t<bf16>(a, dk, dv, s) : decode_t<float>(a, dk, dv, s);
}

hipError_t launch_tree_accept(const TreeAccept& a, int dtype, int dk, int dv, hipStream_t s) {
  if (dtype == HLA_BF16) accept_t<bf16>(a, dk, dv, s);
  else accept_t<float>(a, dk, dv, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.commit) return e;
  hipLaunchKernelGGL(tree_advance_kernel, dim3((unsigned)((a.Bs + 255) / 256)), dim3(256), 0, s, a.n_cache, a.commit,
                     a.n_cap, a.Bs);
  return hipGetLastError();
}

}  // namespace hla
