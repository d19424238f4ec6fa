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
// Chunks with ghat_j = 0 are not read.
#include <hip/hip_runtime.h>

#include "cache8.hpp"
#include "kernels.hpp"
#include "timing.hpp"

namespace hla {
namespace {

constexpr int kMaxCache = 1024;

// One read + write pass over a live [DK][W] matrix: mat <- diag(a) mat - e u^T + k w^T with
// u = (a o k)^T mat, and out = q^T mat (after) = (a o q)^T mat - (q . e) u + (q . k) w.
// LDS rows: ka = a o k, qa = a o q, a, e, k; w null for the transition.
struct LiveRows {
  const float* ka;
  const float* qa;
  const float* a;
  const float* e;
  const float* k;
  float qe, qk;
};
template <int DK, int W, int NT>
__device__ __forceinline__ void live_update(float* mat, const LiveRows& r, const float* w, float* red0, float* red1,
                                            float* s_u, float* out) {
  constexpr int CPR = W / 4, RPP = NT / CPR, NP = DK / RPP;
  const int tid = threadIdx.x, col = (tid % CPR) * 4, r0 = tid / CPR;
  float4 m[NP], pu = make_float4(0.f, 0.f, 0.f, 0.f), pz = pu;
#pragma unroll
  for (int p = 0; p < NP; ++p) m[p] = *reinterpret_cast<const float4*>(mat + (p * RPP + r0) * W + col);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const float kr = r.ka[p * RPP + r0], qr = r.qa[p * RPP + r0];
    pu.x += kr * m[p].x; pu.y += kr * m[p].y; pu.z += kr * m[p].z; pu.w += kr * m[p].w;
    pz.x += qr * m[p].x; pz.y += qr * m[p].y; pz.z += qr * m[p].z; pz.w += qr * m[p].w;
  }
  *reinterpret_cast<float4*>(red0 + r0 * W + col) = pu;
  *reinterpret_cast<float4*>(red1 + r0 * W + col) = pz;
  __syncthreads();
  if (tid < W) {
    float u = 0.f, z = 0.f;
    for (int g = 0; g < RPP; ++g) { u += red0[g * W + tid]; z += red1[g * W + tid]; }
    s_u[tid] = u;
    out[tid] = z - r.qe * u + (w ? r.qk * w[tid] : 0.f);
  }
  __syncthreads();
  const float4 uu = *reinterpret_cast<const float4*>(s_u + col);
  const float4 ww = w ? *reinterpret_cast<const float4*>(w + col) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = p * RPP + r0;
    const float ar = r.a[i], er = r.e[i], kr = r.k[i];
    float4 n;
    n.x = ar * m[p].x - er * uu.x + kr * ww.x;
    n.y = ar * m[p].y - er * uu.y + kr * ww.y;
    n.z = ar * m[p].z - er * uu.z + kr * ww.z;
    n.w = ar * m[p].w - er * uu.w + kr * ww.w;
    *reinterpret_cast<float4*>(mat + i * W + col) = n;
  }
  __syncthreads();
}

// Dot product of a stored row of DK bytes with DK floats in LDS.
template <int FMT, int DK>
__device__ __forceinline__ float row_dot(const uint8_t* row, const float* s_x) {
  float acc = 0.f;
#pragma unroll
  for (int c = 0; c < DK / 16; ++c) {
    const uint4 raw = *reinterpret_cast<const uint4*>(row + 16 * c);
    const unsigned w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      Stored<FMT>::unpack(w[i], f);
      const float4 x = *reinterpret_cast<const float4*>(s_x + 16 * c + 4 * i);
      acc += f[0] * x.x + f[1] * x.y + f[2] * x.z + f[3] * x.w;
    }
  }
  return acc;
}

template <int FMT, class T, int DK, int DV>
__global__ __launch_bounds__(256) void decode8_kernel(Decode8Args a) {
  constexpr int NT = 256, WMAX = DV > DK ? DV : DK;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t row = blockIdx.x;
  __shared__ float s_q[DK], s_k[DK], s_a[DK], s_e[DK], s_ka[DK], s_qa[DK], s_w[DV];
  __shared__ float s_u[WMAX], s_o[DV], s_z[DK], s_red[2][NT * 4];
  __shared__ float s_dot[2], s_g[kMaxCache];

  if (tid < DK) {
    const float qv = to_f<T>(reinterpret_cast<const T*>(a.q)[row * DK + tid]);
    const float kv = to_f<T>(reinterpret_cast<const T*>(a.k)[row * DK + tid]);
    const float dec = a.ga ? a.ga[row * DK + tid] : a.alpha[row];
    s_q[tid] = qv;
    s_k[tid] = kv;
    s_a[tid] = dec;
    s_ka[tid] = dec * kv;
    s_qa[tid] = dec * qv;
    s_e[tid] = (a.ga ? a.gb[row * DK + tid] : a.beta[row]) * kv;
  }
  if (tid < DV) s_w[tid] = (a.ga ? a.gw[row * DV + tid] : a.beta[row]) * to_f<T>(reinterpret_cast<const T*>(a.v)[row * DV + tid]);
  __syncthreads();
  if (w < 2) {
    const float* s = w ? s_e : s_k;
    float x = 0.f;
    for (int i = lane; i < DK; i += 64) x += s_q[i] * s[i];
    x = wave_sum(x);
    if (lane == 0) s_dot[w] = x;
  }
  __syncthreads();
  const LiveRows lr{s_ka, s_qa, s_a, s_e, s_k, s_dot[1], s_dot[0]};
  live_update<DK, DV, NT>(a.S_cur + row * DK * DV, lr, s_w, s_red[0], s_red[1], s_u, s_o);
  live_update<DK, DK, NT>(a.At_cur + row * DK * DK, lr, nullptr, s_red[0], s_red[1], s_u, s_z);

  const int n = cache8_count(a.c, row), n_cap = a.c.n_cap, n_rep = a.c.n_rep;
  for (int j = w; j < n; j += NT / 64) {
    float g;
    if (a.gates_in) {
      g = a.gates_in[row * n_cap + j];
    } else {
      const int64_t slot = row * n_cap + cache8_slot(a.c, row, j);
      const float sc = a.c.scale[slot].z / sqrtf((float)DK);
      float m = -INFINITY, sum = 0.f;
      for (int r = lane; r < n_rep; r += 64) {
        const float s = row_dot<FMT, DK>(a.c.reps + (slot * n_rep + r) * DK, s_q) * sc;
        const float mn = fmaxf(m, s);
        sum = (m > -INFINITY ? sum * expf(m - mn) : 0.f) + expf(s - mn);
        m = mn;
      }
      const float top = wave_max(m);
      sum = wave_sum(m > -INFINITY ? sum * expf(m - top) : 0.f);
      g = 1.f / (1.f + expf(-(top + logf(sum / (float)n_rep))));
    }
    if (lane == 0) {
      const float gh = g >= a.tau ? g : 0.f;
      s_g[j] = gh;
      if (a.gates_out) a.gates_out[row * n_cap + j] = g;
      if (a.c.weight) a.c.weight[row * n_cap + j] += gate_mass(gh);
    }
  }
  if (a.gates_out)
    for (int j = n + tid; j < n_cap; j += NT) a.gates_out[row * n_cap + j] = 0.f;
  __syncthreads();

  for (int j = n - 1; j >= 0; --j) {
    const float g = s_g[j];
    if (g == 0.f) continue;
    const int64_t slot = row * n_cap + cache8_slot(a.c, row, j);
    const float4 sc = a.c.scale[slot];
    float d = 0.f;
    if (tid < DK + DV) d = row_dot<FMT, DK>(a.c.maps + (slot * (DK + DV) + tid) * DK, s_z);
    __syncthreads();
    if (tid < DK) s_z[tid] += g * sc.x * d;
    else if (tid < DK + DV) s_o[tid - DK] += g * sc.y * d;
    __syncthreads();
  }
  if (tid < DV) a.o[row * DV + tid] = s_o[tid];
}

template <int FMT, class T, int DK, int DV>
hipError_t run_decode8(const Decode8Args& a, hipStream_t s) {
  TimedLaunch tl(HLA_KERNEL_DECODE, s);
  hipLaunchKernelGGL((decode8_kernel<FMT, T, DK, DV>), dim3((unsigned)a.c.rows), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <int FMT, class T>
hipError_t pick_decode8(const Decode8Args& a, int dk, int dv, hipStream_t s) {
  if (dk == 64) return dv == 64 ? run_decode8<FMT, T, 64, 64>(a, s) : run_decode8<FMT, T, 64, 128>(a, s);
  return dv == 64 ? run_decode8<FMT, T, 128, 64>(a, s) : run_decode8<FMT, T, 128, 128>(a, s);
}

}  // namespace

hipError_t launch_decode8(const Decode8Args& a, int fmt, int dtype, int dk, int dv, hipStream_t s) {
  if (fmt == kI8) return dtype == 1 ? pick_decode8<kI8, bf16>(a, dk, dv, s) : pick_decode8<kI8, float>(a, dk, dv, s);
  return dtype == 1 ? pick_decode8<kE4M3, bf16>(a, dk, dv, s) : pick_decode8<kE4M3, float>(a, dk, dv, s);
}

}  // namespace hla
