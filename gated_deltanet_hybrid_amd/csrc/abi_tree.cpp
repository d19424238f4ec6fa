// C ABI of trees of drafted tokens over a decode state: argument checks, workspace layout and
// dispatch, as in abi.cpp -- an invalid call returns its status with the stream untouched.
#include "../../include/hla.h"

#include <cmath>
#include <cstdint>

#include "timing.hpp"
#include "tree.hpp"

namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 23) - 1;  // a launch counts its threads (512 a row) in 32 bits

template <int A, class... P>
bool aligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & (A - 1)) == 0) && ...);
}

hla_status_t status(hipError_t e) { return e == hipSuccess ? HLA_OK : HLA_ERR_HIP; }

hla_status_t check_sizes(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t dtype) {
  if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_BAD_DTYPE;
  if (Bs < 1 || H < 1 || n < 1 || n > hla::kTreeNodes) return HLA_ERR_BAD_SHAPE;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return HLA_ERR_BAD_SHAPE;
  if ((double)Bs * (double)H > (double)kMaxRows) return HLA_ERR_BAD_SHAPE;
  return HLA_OK;
}

// z, gates after the threshold, and whether any node reads a chunk
struct Layout { size_t gate, active, total; };
Layout layout(int64_t rows, int32_t n, int32_t dk, int32_t n_cap) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Layout l{};
  l.gate = up((size_t)rows * n * dk * 4);
  l.active = l.gate + up((size_t)rows * n_cap * n * 4);
  l.total = l.active + up((size_t)rows * n_cap * 4);
  return l;
}

}  // namespace

extern "C" {

hla_status_t hla_gdn_tree_workspace_bytes(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t n_cap,
                                          size_t* out) {
  if (!out) return HLA_ERR_NULL_ARG;
  *out = 0;
  const hla_status_t st = check_sizes(Bs, H, n, dk, dv, HLA_F32);
  if (st != HLA_OK) return st;
  if (n_cap < 0 || n_cap > hla::kTreeSlots) return HLA_ERR_BAD_SHAPE;
  if (n_cap) *out = layout(Bs * H, n, dk, n_cap).total;
  return HLA_OK;
}

hla_status_t hla_gdn_tree_decode(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t dtype,
                                 const void* q, const void* k, const void* v, const float* beta, const float* alpha,
                                 const int32_t* parent, const float* S_cur, const float* At_cur, const void* At_cache,
                                 const void* Bc_cache, const void* reps_cache, int32_t n_rep, const int32_t* n_cache,
                                 int32_t n_cap, const float* gates_in, float tau, float* o, float* gates_out,
                                 void* ws, size_t ws_bytes, hipStream_t stream) {
  const hla_status_t st = check_sizes(Bs, H, n, dk, dv, dtype);
  if (st != HLA_OK) return st;
  if (!q || !k || !v || !beta || !alpha || !parent || !S_cur || !o) return HLA_ERR_NULL_ARG;
  if (!At_cur && gates_out) return HLA_ERR_NULL_ARG;  // without a cache there are no gates to write
  if (!aligned<16>(q, k, v, S_cur, At_cur, At_cache, Bc_cache, reps_cache, o, ws) ||
      !aligned<4>(beta, alpha, parent, n_cache, gates_in, gates_out))
    return HLA_ERR_ALIGN;
  hla::TreeArgs a{};
  if (At_cur) {
    if (!At_cache || !Bc_cache || !n_cache || (!gates_in && !reps_cache)) return HLA_ERR_NULL_ARG;
    if (n_cap < 1 || n_cap > hla::kTreeSlots || n_rep < 0 || (!gates_in && n_rep < 1) || std::isnan(tau))
      return HLA_ERR_BAD_SHAPE;
    const Layout l = layout(Bs * H, n, dk, n_cap);
    if (!ws || ws_bytes < l.total) return HLA_ERR_WORKSPACE;
    char* w = static_cast<char*>(ws);
    a.z = reinterpret_cast<float*>(w);
    a.gate = reinterpret_cast<float*>(w + l.gate);
    a.active = reinterpret_cast<int32_t*>(w + l.active);
  }
  const hla::TimedLaunch tl(HLA_KERNEL_TREE, stream);
  a.q = q; a.k = k; a.v = v; a.beta = beta; a.alpha = alpha; a.parent = parent;
  a.S_cur = S_cur; a.At_cur = At_cur; a.At_cache = At_cache; a.Bc_cache = Bc_cache; a.reps_cache = reps_cache;
  a.n_cache = n_cache; a.gates_in = gates_in; a.o = o; a.gates_out = gates_out;
  a.Bs = Bs; a.H = H; a.n = n; a.n_cap = n_cap; a.n_rep = n_rep; a.tau = tau;
  return status(hla::launch_tree_decode(a, dtype, dk, dv, stream));
}

hla_status_t hla_gdn_tree_accept(int64_t Bs, int64_t H, int32_t n, int32_t dk, int32_t dv, int32_t dtype,
                                 const void* k, const void* v, const float* beta, const float* alpha,
                                 const int32_t* parent, const int32_t* node, float* S_cur, float* At_cur,
                                 void* At_cache, void* Bc_cache, int32_t* n_cache, int32_t n_cap,
                                 const int32_t* commit, hipStream_t stream) {
  const hla_status_t st = check_sizes(Bs, H, n, dk, dv, dtype);
  if (st != HLA_OK) return st;
  if (!k || !v || !beta || !alpha || !parent || !node || !S_cur) return HLA_ERR_NULL_ARG;
  if (commit && (!At_cur || !At_cache || !Bc_cache || !n_cache)) return HLA_ERR_NULL_ARG;
  if (commit && (n_cap < 1 || n_cap > hla::kTreeSlots)) return HLA_ERR_BAD_SHAPE;
  if (!aligned<16>(k, v, S_cur, At_cur, At_cache, Bc_cache) || !aligned<4>(beta, alpha, parent, node, n_cache, commit))
    return HLA_ERR_ALIGN;
  const hla::TimedLaunch tl(HLA_KERNEL_TREE, stream);
  hla::TreeAccept a{};
  a.k = k; a.v = v; a.beta = beta; a.alpha = alpha; a.parent = parent; a.node = node;
  a.S_cur = S_cur; a.At_cur = At_cur; a.At_cache = At_cache; a.Bc_cache = Bc_cache;
  a.n_cache = n_cache; a.commit = commit;
  a.Bs = Bs; a.H = H; a.n = n; a.n_cap = n_cap;
  return status(hla::launch_tree_accept(a, dtype, dk, dv, stream));
}

}  // extern "C"
