// C ABI of the 8-bit chunk cache (decode, append, weights, eviction): argument checks and
// dispatch, as in abi.cpp -- an invalid call returns its status with the stream untouched.
#include "../../include/hla.h"

#include <cmath>
#include <cstdint>

#include "cache8.hpp"

namespace {

// A launch counts its workgroups in 31 bits and its threads in 32.
bool launchable(double blocks, double threads) { return blocks <= 2147483647.0 && blocks * threads <= 4294967295.0; }
constexpr int32_t kMaxSlots = 1024, kMaxRep = 256, kMaxEvict = 16384;

template <int A, class... P>
bool aligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & (A - 1)) == 0) && ...);
}

hla_status_t check_cache(const hla_cache8_t* c) {
  if (!c) return HLA_ERR_NULL_ARG;
  if (c->format != HLA_CACHE_I8 && c->format != HLA_CACHE_E4M3) return HLA_ERR_BAD_DTYPE;
  if (c->Bs < 1 || c->H < 1 || (c->dk != 64 && c->dk != 128) || (c->dv != 64 && c->dv != 128)) return HLA_ERR_BAD_SHAPE;
  if (c->n_cap < 1 || c->n_cap > kMaxSlots || c->n_rep < 0 || c->n_rep > kMaxRep) return HLA_ERR_BAD_SHAPE;
  if (!launchable((double)c->Bs * (double)c->H, (c->dk + c->dv) * 4.0)) return HLA_ERR_BAD_SHAPE;
  if (!c->maps || !c->scale || !c->order || !c->count || (c->n_rep && !c->reps)) return HLA_ERR_NULL_ARG;
  if (!aligned<16>(c->maps, c->reps, c->scale) || !aligned<4>(c->order, c->count, c->weight)) return HLA_ERR_ALIGN;
  return HLA_OK;
}

hla::Cache8View view(const hla_cache8_t* c) {
  hla::Cache8View v{};
  v.maps = static_cast<uint8_t*>(c->maps);
  v.reps = static_cast<uint8_t*>(c->reps);
  v.scale = reinterpret_cast<float4*>(c->scale);
  v.order = c->order;
  v.count = c->count;
  v.weight = c->weight;
  v.rows = c->Bs * c->H;
  v.n_cap = c->n_cap;
  v.n_rep = c->n_rep;
  return v;
}

hla_status_t status(hipError_t e) { return e == hipSuccess ? HLA_OK : HLA_ERR_HIP; }

// Checks shared by the two decode calls, and their common arguments.
hla_status_t decode8(const hla_cache8_t* c, int32_t dtype, hla::Decode8Args& a, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  if (std::isnan(a.tau)) return HLA_ERR_BAD_SHAPE;
  if (!a.q || !a.k || !a.v || !a.S_cur || !a.At_cur || !a.o || (!a.gates_in && c->n_rep == 0)) return HLA_ERR_NULL_ARG;
  if (!aligned<16>(a.S_cur, a.At_cur, ws) || !aligned<4>(a.q, a.k, a.v, a.gates_in, a.o, a.gates_out))
    return HLA_ERR_ALIGN;
  a.c = view(c);
  const size_t need = (size_t)hla::plan_decode8(a, c->dk, c->dv, ws);
  if (need && (!ws || ws_bytes < need)) return HLA_ERR_WORKSPACE;
  return status(hla::launch_decode8(a, c->format, dtype, c->dk, c->dv, stream));
}

}  // namespace

extern "C" {

hla_status_t hla_decode8_workspace_bytes(const hla_cache8_t* c, size_t* out) {
  if (!out) return HLA_ERR_NULL_ARG;
  *out = 0;
  const hla_status_t st = check_cache(c);
  if (st != HLA_OK) return st;
  hla::Decode8Args a{};
  a.c = view(c);
  *out = (size_t)hla::plan_decode8(a, c->dk, c->dv, nullptr);
  return HLA_OK;
}

hla_status_t hla_gdn_decode8(const hla_cache8_t* c, int32_t dtype, const void* q, const void* k, const void* v,
                             const float* beta, const float* alpha, float* S_cur, float* At_cur,
                             const float* gates_in, float tau, float* o, float* gates_out, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
  const hla_status_t st = check_cache(c);
  if (st != HLA_OK) return st;
  if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_BAD_DTYPE;
  if (!beta || !alpha) return HLA_ERR_NULL_ARG;
  if (!aligned<4>(beta, alpha)) return HLA_ERR_ALIGN;
  hla::Decode8Args a{};
  a.q = q; a.k = k; a.v = v; a.beta = beta; a.alpha = alpha; a.S_cur = S_cur; a.At_cur = At_cur;
  a.gates_in = gates_in; a.tau = tau; a.o = o; a.gates_out = gates_out;
  return decode8(c, dtype, a, ws, ws_bytes, stream);
}

hla_status_t hla_gdn2_decode8(const hla_cache8_t* c, int32_t dtype, const void* q, const void* k, const void* v,
                              const float* a_decay, const float* b_erase, const float* w_write, float* S_cur,
                              float* At_cur, const float* gates_in, float tau, float* o, float* gates_out,
                              void* ws, size_t ws_bytes, hipStream_t stream) {
  const hla_status_t st = check_cache(c);
  if (st != HLA_OK) return st;
  if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_BAD_DTYPE;
  if (!a_decay || !b_erase || !w_write) return HLA_ERR_NULL_ARG;
  if (!aligned<4>(a_decay, b_erase, w_write)) return HLA_ERR_ALIGN;
  hla::Decode8Args a{};
  a.q = q; a.k = k; a.v = v; a.ga = a_decay; a.gb = b_erase; a.gw = w_write; a.S_cur = S_cur; a.At_cur = At_cur;
  a.gates_in = gates_in; a.tau = tau; a.o = o; a.gates_out = gates_out;
  return decode8(c, dtype, a, ws, ws_bytes, stream);
}

hla_status_t hla_cache8_append(const hla_cache8_t* c, int32_t dtype, int32_t n_src, int32_t ld_src, void* At, void* Bc,
                               const void* reps, int64_t ld_R, const int32_t* src, const int32_t* n_new,
                               const float* weight_in, int32_t reset, int32_t reset_live, hipStream_t stream) {
  const hla_status_t st = check_cache(c);
  if (st != HLA_OK) return st;
  if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_BAD_DTYPE;
  if (n_src < 0 || ld_src < n_src || ld_src < 1 || (reset != 0 && reset != 1) || (reset_live != 0 && reset_live != 1)) return HLA_ERR_BAD_SHAPE;
  if (!launchable((double)c->Bs * (double)c->H * (double)ld_src, 512.0)) return HLA_ERR_BAD_SHAPE;
  if (!At || !Bc || (c->n_rep && !reps)) return HLA_ERR_NULL_ARG;
  if (c->n_rep && ld_R < (int64_t)n_src * c->n_rep) return HLA_ERR_BAD_SHAPE;
  if (c->n_rep && (double)c->Bs * (double)ld_R * (double)c->H * c->dk > 4.0e18) return HLA_ERR_BAD_SHAPE;
  if (reset_live && (src || dtype != HLA_F32)) return HLA_ERR_UNSUPPORTED;
  if (!aligned<16>(At, Bc, reps) || !aligned<4>(src, n_new, weight_in)) return HLA_ERR_ALIGN;
  hla::Append8Args a{};
  a.c = view(c);
  a.At = At; a.Bc = Bc; a.reps = reps; a.H = c->H; a.ld_R = ld_R; a.src = src; a.n_new = n_new;
  a.weight_in = weight_in; a.n_src = n_src; a.ld_src = ld_src; a.reset = reset; a.reset_live = reset_live;
  return status(hla::launch_append8(a, c->format, dtype, c->dk, c->dv, stream));
}

hla_status_t hla_gate_weights(int64_t B, int64_t H, int32_t N, const float* gates, const int32_t* n_chunks,
                              float tau, float* weight, hipStream_t stream) {
  if (B < 1 || H < 1 || N < 1 || std::isnan(tau)) return HLA_ERR_BAD_SHAPE;
  if (!launchable((double)B * (double)H * ((N + 31.0) / 32.0), 256.0) ||
      (double)B * (double)H * (double)N * (double)N > 4.0e18)
    return HLA_ERR_BAD_SHAPE;
  if (!gates || !weight) return HLA_ERR_NULL_ARG;
  if (!aligned<4>(gates, n_chunks, weight)) return HLA_ERR_ALIGN;
  hla::GateWeightsArgs a{gates, n_chunks, weight, B, H, N, tau};
  return status(hla::launch_gate_weights(a, stream));
}

hla_status_t hla_evict_chunks(int64_t Bs, int64_t H, int32_t n, const float* weight, const int32_t* order,
                              const int32_t* count, int32_t budget, int32_t n_recent, int32_t* order_out,
                              float* weight_out, int32_t* count_out, hipStream_t stream) {
  if (Bs < 1 || H < 1 || n < 1 || n > kMaxEvict) return HLA_ERR_BAD_SHAPE;
  if (!launchable((double)Bs * (double)H, n <= 256 ? 64.0 : n <= 4096 ? 256.0 : 1024.0)) return HLA_ERR_BAD_SHAPE;
  if (budget < 0 || n_recent < 0 || n_recent > budget) return HLA_ERR_BAD_SHAPE;
  if (!weight || !count || !order_out || !weight_out || !count_out) return HLA_ERR_NULL_ARG;
  if (!aligned<4>(weight, order, count, order_out, weight_out, count_out)) return HLA_ERR_ALIGN;
  hla::EvictArgs a{weight, order, count, order_out, weight_out, count_out, Bs * H, n, budget, n_recent};
  return status(hla::launch_evict(a, stream));
}

}  // extern "C"
