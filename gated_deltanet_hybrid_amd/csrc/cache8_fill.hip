// What goes into the 8-bit chunk cache and what leaves it: quantise-and-append, the weights a
// prefill's gates give its chunks, and eviction by weight.
#include <hip/hip_runtime.h>

#include "cache8.hpp"
#include "kernels.hpp"

namespace hla {
namespace {

// ------------------------------------------------------------------------------ append
// Chunks appended to a row: what the caller asks for, cut to the room that is left.
__device__ __forceinline__ int append_count(const Append8Args& a, int64_t row, int held) {
  const int want = a.n_new ? a.n_new[row] : a.n_src;
  const int lim = a.n_src < a.c.n_cap - held ? a.n_src : a.c.n_cap - held;
  return want < 0 ? 0 : (want > lim ? lim : want);
}

template <class T> __device__ __forceinline__ void unpack16(const uint4& raw, float (&f)[16 / sizeof(T)]) {
  const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) f[i] = to_f<T>(e[i]);
}

// Largest magnitude (as bits) over the block, on every thread.
template <int NT>
__device__ __forceinline__ unsigned block_max(unsigned x, unsigned* red) {
#pragma unroll
  for (int off = 32; off > 0; off /= 2) x = max_u(x, __shfl_xor(x, off, 64));
  __syncthreads();  // red may still be read from the call before
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  unsigned m = red[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) m = max_u(m, red[i]);
  return m;
}

// One source map [DK][W] (state orientation) held in registers by the block as units of four
// rows x 16 bytes, so that four consecutive k of one output row are in one thread's hands and
// the transposed image is written to LDS a word at a time.
template <class T, int DK, int W, int NT> struct MapRegs {
  static constexpr int E = 16 / sizeof(T), CPR = W / E, UNITS = (DK / 4) * CPR, PER = (UNITS + NT - 1) / NT;
  uint4 raw[PER][4];
  __device__ __forceinline__ void load(const T* m) {
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = p * NT + threadIdx.x;
      if (UNITS % NT != 0 && u >= UNITS) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        raw[p][i] = *reinterpret_cast<const uint4*>(m + ((u / CPR) * 4 + i) * W + (u % CPR) * E);
    }
  }
  // f(p, i, e, value) with the identity taken off where SUB
  template <bool SUB> __device__ __forceinline__ float value(int p, int i, int e) const {
    const int u = p * NT + threadIdx.x;
    float f[E];
    unpack16<T>(raw[p][i], f);
    return f[e] - (SUB && (u / CPR) * 4 + i == (u % CPR) * E + e ? 1.f : 0.f);
  }
  template <bool SUB> __device__ __forceinline__ unsigned largest() const {
    unsigned m = 0;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      if (UNITS % NT != 0 && p * NT + (int)threadIdx.x >= UNITS) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) m = max_u(m, mag(value<SUB>(p, i, e)));
    }
    return m;
  }
  template <bool SUB, int FMT, int LD> __device__ __forceinline__ void store(uint8_t* img, unsigned m) const {
    const float inv = to_stored<FMT>(m);
    const unsigned mask = stored_mask(m);
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int u = p * NT + threadIdx.x;
      if (UNITS % NT != 0 && u >= UNITS) continue;
#pragma unroll
      for (int e = 0; e < E; ++e)
        *reinterpret_cast<unsigned*>(img + ((u % CPR) * E + e) * LD + (u / CPR) * 4) =
            Stored<FMT>::pack(value<SUB>(p, 0, e) * inv, value<SUB>(p, 1, e) * inv, value<SUB>(p, 2, e) * inv,
                              value<SUB>(p, 3, e) * inv) & mask;
    }
  }
};

template <class T, int W, int NT>
__device__ __forceinline__ void reset_map(T* m, int rows, bool identity) {
  for (int i = threadIdx.x; i < rows * W; i += NT) m[i] = from_f<T>(identity && i / W == i % W ? 1.f : 0.f);
}

// A row's bookkeeping by one wave once its chunks are stored: count, and the new positions'
// weights; a cache that starts empty also gets its order (position p in slot p).
__device__ __forceinline__ void append_finish(const Append8Args& a, int64_t row, int held, int add) {
  const int lane = threadIdx.x & 63, n_cap = a.c.n_cap;
  const int p0 = a.reset ? 0 : held, p1 = a.reset ? n_cap : held + add;
  for (int p = p0 + lane; p < p1; p += 64) {
    if (a.reset) a.c.order[row * n_cap + p] = p;
    const int i = p - held;
    if (a.c.weight) a.c.weight[row * n_cap + p] = i < add && a.weight_in ? a.weight_in[row * a.ld_src + i] : 0.f;
  }
  if (lane == 0) a.c.count[row] = held + add;
}

// One workgroup per (row, appended chunk): the maps are read once into registers, their largest
// magnitudes found, and the quantised transposes go through LDS to 16-byte stores.  Bound by HBM:
// 512 chunks of 16 heads (dk = dv = 128, bf16, 64 representatives, 1.01 GB read and written) take
// 191 us, 5.3 TB/s, where a large copy moves 4.8; a batch's 1024 live chunks (float32, set back to
// the identity, 303 MB) 40 us from the caches' reach and about 65 from HBM.
template <int FMT, class T, int DK, int DV, int NT>
__global__ __launch_bounds__(NT) void append8_kernel(Append8Args a) {
  constexpr int LD = DK + 4;  // image row: one word of padding spreads the transposed writes over the banks
  __shared__ __align__(16) uint8_t s_img[(DK + DV) * LD];
  __shared__ unsigned s_red[NT / 64];
  const int64_t row = blockIdx.x / a.n_src;
  const int i = (int)(blockIdx.x % a.n_src), tid = threadIdx.x;
  const int held = a.reset ? 0 : cache8_count(a.c, row), add = append_count(a, row, held);
  if (a.n_src == 1) {  // the row's only workgroup does its bookkeeping too
    __syncthreads();   // every thread has read the count
    if (tid < 64) append_finish(a, row, held, add);
  }
  if (i >= add) return;
  int from = i;
  if (a.src) {
    from = a.src[row * a.ld_src + i];
    from = from < 0 ? 0 : (from >= a.n_src ? a.n_src - 1 : from);
  }
  const int64_t slot = row * a.c.n_cap + (a.reset ? i : cache8_slot(a.c, row, held + i));
  T* At = reinterpret_cast<T*>(a.At) + (row * a.ld_src + from) * DK * DK;
  T* Bc = reinterpret_cast<T*>(a.Bc) + (row * a.ld_src + from) * DK * DV;

  MapRegs<T, DK, DK, NT> ra;
  MapRegs<T, DK, DV, NT> rb;
  ra.load(At);
  rb.load(Bc);
  const unsigned ma = block_max<NT>(ra.template largest<true>(), s_red);
  const unsigned mb = block_max<NT>(rb.template largest<false>(), s_red);
  ra.template store<true, FMT, LD>(s_img, ma);
  rb.template store<false, FMT, LD>(s_img + DK * LD, mb);

  // representatives: rows of one head, H dk elements apart
  unsigned mr = 0;
  constexpr int E = 16 / sizeof(T), CPR = DK / E;
  if (a.c.n_rep) {
    const T* rep = reinterpret_cast<const T*>(a.reps) +
                   ((row / a.H * a.ld_R + (int64_t)from * a.c.n_rep) * a.H + row % a.H) * DK;
    for (int u = tid; u < a.c.n_rep * CPR; u += NT) {
      const uint4 raw = *reinterpret_cast<const uint4*>(rep + (int64_t)(u / CPR) * a.H * DK + (u % CPR) * E);
      float f[E];
      unpack16<T>(raw, f);
#pragma unroll
      for (int e = 0; e < E; ++e) mr = max_u(mr, mag(f[e]));
    }
    mr = block_max<NT>(mr, s_red);
    const float ir = to_stored<FMT>(mr);
    const unsigned mask = stored_mask(mr);
    uint8_t* out = a.c.reps + slot * a.c.n_rep * DK;
    for (int u = tid; u < a.c.n_rep * CPR; u += NT) {
      const uint4 raw = *reinterpret_cast<const uint4*>(rep + (int64_t)(u / CPR) * a.H * DK + (u % CPR) * E);
      float f[E];
      unpack16<T>(raw, f);
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<unsigned*>(out + u * E + e) =
            Stored<FMT>::pack(f[e] * ir, f[e + 1] * ir, f[e + 2] * ir, f[e + 3] * ir) & mask;
    }
  }
  __syncthreads();
  uint4* maps = reinterpret_cast<uint4*>(a.c.maps + slot * (DK + DV) * DK);
  for (int u = tid; u < (DK + DV) * DK / 16; u += NT) {
    const unsigned* p = reinterpret_cast<const unsigned*>(s_img + (u / (DK / 16)) * LD + (u % (DK / 16)) * 16);
    maps[u] = make_uint4(p[0], p[1], p[2], p[3]);
  }
  if (tid == 0)
    a.c.scale[slot] = make_float4(from_stored<FMT>(ma), from_stored<FMT>(mb), from_stored<FMT>(mr), 0.f);
  if (a.reset_live) {
    reset_map<T, DK, NT>(At, DK, true);
    reset_map<T, DV, NT>(Bc, DK, false);
  }
}

__global__ __launch_bounds__(256) void append8_finish_kernel(Append8Args a) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.c.rows) return;
  const int held = a.reset ? 0 : cache8_count(a.c, row);
  append_finish(a, row, held, append_count(a, row, held));
}

template <int FMT, class T, int DK, int DV>
hipError_t run_append8(const Append8Args& a, hipStream_t s) {
  constexpr int NT = sizeof(T) == 2 ? 256 : 512;  // 16 or 32 KiB of a 128 x 128 map in 64 registers a thread
  if (a.n_src > 0) {
    hipLaunchKernelGGL((append8_kernel<FMT, T, DK, DV, NT>), dim3((unsigned)(a.c.rows * a.n_src)), dim3(NT), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.n_src == 1) return e;
  }
  hipLaunchKernelGGL(append8_finish_kernel, dim3((unsigned)((a.c.rows + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int FMT, class T>
hipError_t pick_append8(const Append8Args& a, int dk, int dv, hipStream_t s) {
  if (dk == 64) return dv == 64 ? run_append8<FMT, T, 64, 64>(a, s) : run_append8<FMT, T, 64, 128>(a, s);
  return dv == 64 ? run_append8<FMT, T, 128, 64>(a, s) : run_append8<FMT, T, 128, 128>(a, s);
}

// ------------------------------------------------------------------------ gate weights
// w_j = sum over query chunks i > j (below n_b) of the gates that reach tau.  One workgroup per
// (row, 32 columns): V columns to a lane, 32 / V lanes to a row of the matrix, so that a wave's
// load is whole 128-byte lines, eight loads on their way.  The lanes' sums are added across the
// wave and then over the four waves, always in that order.  Reads n (n - 1) / 2 floats a head, and
// the half lines on the diagonal: 16 heads of 1024 chunks, 33.6 MB, in 7.4 us (4.5 TB/s; 13 us with
// each load under its own condition, 83 us with one load at a time).
typedef float f32x4v __attribute__((ext_vector_type(4)));
template <int V>
__global__ __launch_bounds__(256) void gate_weights_kernel(GateWeightsArgs a) {
  constexpr int LPR = 32 / V, RPP = 256 / LPR, U = 8;
  __shared__ float s_sum[4][32];
  const int blocks = (a.N + 31) / 32, tid = threadIdx.x;
  const int64_t row = blockIdx.x / blocks;
  const int j0 = (int)(blockIdx.x % blocks) * 32, j = j0 + tid % LPR * V;
  int n = a.N;
  if (a.n_chunks) {
    n = a.n_chunks[row / a.H];
    n = n < 0 ? 0 : (n > a.N ? a.N : n);
  }
  // a lane past the last column, or a row past the last chunk, reads the last one and counts for nothing:
  // a load under a condition would be waited for on its own
  const float* g = a.gates + row * a.N * (int64_t)a.N + (j < a.N ? j : a.N - V);
  float sum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum[v] = 0.f;
  for (int i0 = j0 + 1; i0 < n; i0 += RPP * U) {
    float x[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPP + tid / LPR;
      const float* p = g + (int64_t)(i < n ? i : n - 1) * a.N;
      if constexpr (V == 4) {
        const f32x4v f = *reinterpret_cast<const f32x4v*>(p);
        x[u][0] = f.x; x[u][1] = f.y; x[u][2] = f.z; x[u][3] = f.w;
      } else {
        x[u][0] = *p;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPP + tid / LPR;
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += i < n && j + v < i && x[u][v] >= a.tau ? gate_mass(x[u][v]) : 0.f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int off = LPR; off < 64; off *= 2) sum[v] += __shfl_xor(sum[v], off, 64);
    if ((tid & 63) < LPR) s_sum[tid >> 6][(tid & 63) * V + v] = sum[v];
  }
  __syncthreads();
  if (tid < 32 && j0 + tid < a.N)
    a.weight[row * a.N + j0 + tid] = s_sum[0][tid] + s_sum[1][tid] + s_sum[2][tid] + s_sum[3][tid];
}

// ------------------------------------------------------------------------------- evict
// float order as unsigned order: NaN below everything, -0 as +0.
__device__ __forceinline__ unsigned order_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __builtin_bit_cast(unsigned, x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// NW waves per row, wave v holding the 64 NI positions from 64 NI v on (position 64 (NI v + i) +
// lane in register i).  The m lightest of the positions [0, n - n_recent) leave: the threshold
// key (the m-th smallest) is found bit by bit from the top by counting ballots, every key below
// it leaves, and of the equal ones the first in time.  All of a row is read before any of it is
// written, so outputs may be the inputs.  Latency: 32 rounds of ballots, 9 us for 128 rows of 1024
// by four waves a row (19 by one, whose 16 ballots a round follow one another), 4 us for 64
// positions, 25 us for 512 rows of 4096 and 43 us for 128 rows of 16384 (16 positions a lane).
// Up to 256 positions one wave needs at most four ballots a round and no barrier.
template <int NI, int NW>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void evict_kernel(EvictArgs a) {
  constexpr int RPB = NW == 1 ? 4 : 1;  // rows per workgroup
  const int lane = threadIdx.x & 63, v = NW == 1 ? 0 : threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPB + (NW == 1 ? threadIdx.x >> 6 : 0);
  if (row >= a.rows) return;
  __shared__ int s_part[2][NW];
  // sum over the row's waves; `before`: over the waves in front of this one
  int turn = 0;
  auto row_sum = [&](int x, int& before) {
    before = 0;
    if constexpr (NW == 1) return x;
    turn ^= 1;  // two buffers, so one barrier a call
    if (lane == 0) s_part[turn][v] = x;
    __syncthreads();
    int sum = 0;
    for (int i = 0; i < NW; ++i) {
      if (i < v) before += s_part[turn][i];
      sum += s_part[turn][i];
    }
    return sum;
  };
  const int64_t base = row * a.n;
  int held = a.count[row];
  held = held < 0 ? 0 : (held > a.n ? a.n : held);
  const int m = held > a.budget ? held - a.budget : 0;
  const int cand = m > 0 ? held - a.n_recent : 0;  // positions below it may leave (m <= cand, as n_recent <= budget)
  float w[NI];
  int ord[NI];
  unsigned key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = 64 * (NI * v + i) + lane;
    w[i] = p < a.n ? a.weight[base + p] : 0.f;
    ord[i] = p < a.n ? (a.order ? a.order[base + p] : p) : 0;
    key[i] = order_key(w[i]);
  }
  // t: the largest key with fewer than m candidates below it, the m-th smallest candidate
  unsigned t = 0;
  int below = 0, unused;
  if (m > 0) {
    for (int b = 31; b >= 0; --b) {
      const unsigned top = t | (1u << b);
      int c = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) c += __popcll(__ballot(64 * (NI * v + i) + lane < cand && key[i] < top));
      c = row_sum(c, unused);
      if (c < m) { t = top; below = c; }
    }
  }
  // of the keys equal to t, the first m - below in time leave
  const unsigned long long before = (1ull << lane) - 1;
  int eq_seen = 0, go_seen = 0, keep_seen = 0;
  if constexpr (NW > 1) {
    int n_eq = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) n_eq += __popcll(__ballot(64 * (NI * v + i) + lane < cand && key[i] == t));
    row_sum(n_eq, eq_seen);
  }
  bool go[NI];
  int n_go = 0, n_keep = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = 64 * (NI * v + i) + lane;
    const bool eq = p < cand && key[i] == t;
    const unsigned long long be = __ballot(eq);
    go[i] = p < cand && (key[i] < t || (eq && eq_seen + __popcll(be & before) < m - below));
    eq_seen += __popcll(be);
    n_go += __popcll(__ballot(go[i]));
    n_keep += __popcll(__ballot(p < held && !go[i]));
  }
  row_sum(n_go, go_seen);
  row_sum(n_keep, keep_seen);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = 64 * (NI * v + i) + lane;
    const bool keep = p < held && !go[i];
    const unsigned long long bg = __ballot(go[i]), bk = __ballot(keep);
    if (p < a.n) {
      int to = p;  // free slots stay where they are
      if (go[i]) to = held - m + go_seen + __popcll(bg & before);
      else if (keep) to = keep_seen + __popcll(bk & before);
      a.order_out[base + to] = ord[i];
      a.weight_out[base + to] = keep ? w[i] : 0.f;
    }
    go_seen += __popcll(bg);
    keep_seen += __popcll(bk);
  }
  if (lane == 0 && v == 0) a.count_out[row] = held - m;
}

}  // namespace

hipError_t launch_append8(const Append8Args& a, int fmt, int dtype, int dk, int dv, hipStream_t s) {
  if (fmt == kI8) return dtype == 1 ? pick_append8<kI8, bf16>(a, dk, dv, s) : pick_append8<kI8, float>(a, dk, dv, s);
  return dtype == 1 ? pick_append8<kE4M3, bf16>(a, dk, dv, s) : pick_append8<kE4M3, float>(a, dk, dv, s);
}

hipError_t launch_gate_weights(const GateWeightsArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * a.H * ((a.N + 31) / 32)));
  // 16-byte loads where every row of the matrix is 16-byte aligned
  if (a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.gates) & 15) == 0)
    hipLaunchKernelGGL((gate_weights_kernel<4>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((gate_weights_kernel<1>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_evict(const EvictArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 3) / 4)), block(256), wide((unsigned)a.rows);
  if (a.n <= 64) hipLaunchKernelGGL((evict_kernel<1, 1>), grid, block, 0, s, a);
  else if (a.n <= 256) hipLaunchKernelGGL((evict_kernel<4, 1>), grid, block, 0, s, a);
  else if (a.n <= 1024) hipLaunchKernelGGL((evict_kernel<4, 4>), wide, block, 0, s, a);
  else if (a.n <= 4096) hipLaunchKernelGGL((evict_kernel<16, 4>), wide, block, 0, s, a);
  else hipLaunchKernelGGL((evict_kernel<16, 16>), wide, dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace hla
