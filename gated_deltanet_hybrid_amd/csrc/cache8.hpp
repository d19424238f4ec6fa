// The 8-bit chunk cache: its device view, the two stored formats, and the launchers.
#pragma once
#include "common.hpp"

namespace hla {

// hla_cache8_t as the kernels take it (include/hla.h describes the arrays).
struct Cache8View {
  uint8_t* maps;    // [Bs,H,n_cap,dk+dv,dk]
  uint8_t* reps;    // [Bs,H,n_cap,n_rep,dk]
  float4* scale;    // [Bs,H,n_cap]: of A - I, of B, of the representatives, 0
  int32_t* order;   // [Bs,H,n_cap]
  int32_t* count;   // [Bs,H]
  float* weight;    // [Bs,H,n_cap] or null
  int64_t rows;     // Bs H
  int32_t n_cap, n_rep;
};

// What the caller's memory holds is clamped before it becomes an address: a count to the
// capacity, a slot to the cache.
__device__ __forceinline__ int cache8_count(const Cache8View& c, int64_t row) {
  const int n = c.count[row];
  return n < 0 ? 0 : (n > c.n_cap ? c.n_cap : n);
}
__device__ __forceinline__ int cache8_slot(const Cache8View& c, int64_t row, int pos) {
  const unsigned s = (unsigned)c.order[row * c.n_cap + pos];
  return s < (unsigned)c.n_cap ? (int)s : c.n_cap - 1;
}

// The stored formats.  A block with largest magnitude m is multiplied by (1 / m) top and rounded
// to the nearest stored value, ties to even, so that m lands on `top`; the scale is m (1 / top).
// Each of the two factors is rounded twice, as written: what is stored depends on the last bit.
// m < 2^-100 stores zeros with scale 0, since 1 / m would overflow.  A block with a number that is
// not finite stores zeros with scale NaN, so that every decode that reads it shows it.
// m is held as its bits: magnitudes compare as those, and what is not finite is above every number
// (fmaxf would drop a NaN).
constexpr int kI8 = 0, kE4M3 = 1;
constexpr unsigned kCache8Tiny = (127u - 100u) << 23, kNotFinite = 0x7f800000u;
__device__ __forceinline__ unsigned mag(float x) { return __builtin_bit_cast(unsigned, x) & 0x7fffffffu; }
__device__ __forceinline__ unsigned max_u(unsigned a, unsigned b) { return a > b ? a : b; }
template <int FMT> struct Stored;
template <> struct Stored<kI8> {
  static constexpr float top = 127.f;
  __device__ __forceinline__ static unsigned pack(float a, float b, float c, float d) {
    auto q = [](float x) { return (unsigned)(int)fminf(fmaxf(rintf(x), -127.f), 127.f) & 0xffu; };
    return q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
  }
};
template <> struct Stored<kE4M3> {
  static constexpr float top = 448.f;
  __device__ __forceinline__ static unsigned pack(float a, float b, float c, float d) {
    // rounding may leave x (top / max) one step above top: clamped, it stores top
    auto cl = [](float x) { return fminf(fmaxf(x, -448.f), 448.f); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(cl(a), cl(b), 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(cl(c), cl(d), w, true);
  }
};

// Eight stored numbers (two words) as bf16, exactly.
__device__ __forceinline__ bf16x8 e4m3_frag(unsigned w0, unsigned w1) {
  return __builtin_bit_cast(
      bf16x8, make_uint4(__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, false)),
                         __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, true)),
                         __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, false)),
                         __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, true))));
}

template <int FMT> __device__ __forceinline__ bf16x8 stored_frag(unsigned w0, unsigned w1) {
  if constexpr (FMT == kE4M3) return e4m3_frag(w0, w1);
  auto two = [](unsigned w, int at) {  // 8-bit integers: the low halves of their float32 images are zero
    const float x = (float)(int8_t)(w >> at), y = (float)(int8_t)(w >> (at + 8));
    return __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, y), __builtin_bit_cast(unsigned, x), 0x07060302u);
  };
  return __builtin_bit_cast(bf16x8, make_uint4(two(w0, 0), two(w0, 16), two(w1, 0), two(w1, 16)));
}

template <int FMT> __device__ __forceinline__ float to_stored(unsigned m) {
  return m >= kCache8Tiny && m < kNotFinite ? (1.f / __builtin_bit_cast(float, m)) * Stored<FMT>::top : 0.f;
}
template <int FMT> __device__ __forceinline__ float from_stored(unsigned m) {
  if (m >= kNotFinite) return __builtin_nanf("");
  return m >= kCache8Tiny ? __builtin_bit_cast(float, m) * (1.f / Stored<FMT>::top) : 0.f;
}
// the packed words of a block are taken through this: none of one that is not finite
__device__ __forceinline__ unsigned stored_mask(unsigned m) { return m < kNotFinite ? ~0u : 0u; }

struct Decode8Args {
  Cache8View c;
  const void* q;          // [Bs,H,dk] (dtype)
  const void* k;
  const void* v;          // [Bs,H,dv]
  const float* beta;      // [Bs,H], Gated DeltaNet
  const float* alpha;
  const float* ga;        // [Bs,H,dk], Gated DeltaNet-2 (ga set): decay, erase gate
  const float* gb;
  const float* gw;        // [Bs,H,dv]: write gate
  float* S_cur;           // [Bs,H,dk,dv]
  float* At_cur;          // [Bs,H,dk,dk]
  const float* gates_in;  // [Bs,H,n_cap] or null
  float* o;               // [Bs,H,dv]
  float* gates_out;       // [Bs,H,n_cap] or null
  float tau;
  // The split form (segs = 0: one workgroup a row does everything): at most `segs` segments of
  // seg_len positions a row, the gates in gate_blocks blocks of gate_len.
  int32_t segs, seg_len, gate_blocks, gate_len;
  struct Work {
    float* gate;  // [rows,n_cap]: gates after the threshold
    float* y;     // [rows,dk]: At_cur^T q
    float* o;     // [rows,dv]: the live part of o
    float* z;     // [rows,segs,dk]: z as it enters each segment
    float* part;  // [rows,segs,dv]: each segment's share of o
    float* phi;   // [rows,segs,dk,dk]: column by column
  } ws;
};
constexpr int kMaxSegment = 64;
constexpr int kSplitFrom = 64;  // a row that holds fewer chunks is one segment
__device__ __forceinline__ int split_segments(const Decode8Args& a, int held) {
  return held < kSplitFrom ? 1 : (held + a.seg_len - 1) / a.seg_len;
}
// Sets the form of a call and its workspace (offsets from `ws`, which may be null); returns the
// workspace's bytes.  Without gates_in it is the most that a call on the cache takes.
int64_t plan_decode8(Decode8Args& a, int dk, int dv, void* ws);
hipError_t launch_decode8(const Decode8Args& a, int fmt, int dtype, int dk, int dv, hipStream_t s);

struct Append8Args {
  Cache8View c;
  void* At;               // [Bs,H,ld_src,dk,dk] (dtype), state orientation
  void* Bc;               // [Bs,H,ld_src,dk,dv]
  const void* reps;       // [Bs,ld_R,H,dk]: source chunk i's rows are [i n_rep, (i+1) n_rep)
  int64_t H, ld_R;
  const int32_t* src;     // [Bs,H,ld_src] source chunk of each appended one, or null (i)
  const int32_t* n_new;   // [Bs,H] or null (n_src)
  const float* weight_in; // [Bs,H,ld_src] or null (0)
  int32_t n_src, ld_src;
  int32_t reset, reset_live;
};
hipError_t launch_append8(const Append8Args& a, int fmt, int dtype, int dk, int dv, hipStream_t s);

struct GateWeightsArgs {
  const float* gates;       // [B,H,N,N]
  const int32_t* n_chunks;  // [B] or null (N)
  float* weight;            // [B,H,N]
  int64_t B, H;
  int32_t N;
  float tau;
};
hipError_t launch_gate_weights(const GateWeightsArgs& a, hipStream_t s);

struct EvictArgs {
  const float* weight;     // [rows,n]
  const int32_t* order;    // [rows,n] or null (identity)
  const int32_t* count;    // [rows]
  int32_t* order_out;
  float* weight_out;
  int32_t* count_out;
  int64_t rows;
  int32_t n, budget, n_recent;
};
hipError_t launch_evict(const EvictArgs& a, hipStream_t s);

// Gate of one chunk as it counts for its weight.
__device__ __forceinline__ float gate_mass(float g) { return fminf(fmaxf(g, 0.f), 1.f); }

}  // namespace hla
