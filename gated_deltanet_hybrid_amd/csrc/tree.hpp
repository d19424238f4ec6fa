// Trees of drafted tokens over a decode state: what the kernels take, and their launchers.
#pragma once
#include "common.hpp"

namespace hla {

constexpr int kTreeNodes = 64;    // most nodes of a tree
constexpr int kTreeSlots = 1024;  // largest n_cap

struct TreeArgs {
  const void *q, *k, *v;        // [Bs, n, H, dk], [Bs, n, H, dk], [Bs, n, H, dv]
  const float *beta, *alpha;    // [Bs, n, H]
  const int32_t* parent;        // [Bs, n]
  const float *S_cur, *At_cur;  // [Bs, H, dk, dv], [Bs, H, dk, dk] or null
  const void *At_cache, *Bc_cache, *reps_cache;
  const int32_t* n_cache;       // [Bs]
  const float* gates_in;        // [Bs, n, H, n_cap] or null
  float *o, *gates_out;         // [Bs, n, H, dv]; [Bs, n, H, n_cap] or null
  float* z;                     // workspace [rows, n, dk]: the nodes' queries as the newest chunk meets them
  float* gate;                  // workspace [rows, n_cap, n]: gates after the threshold
  int32_t* active;              // workspace [rows, n_cap]: a bit for each 16 nodes of which any reads the chunk
  int64_t Bs, H;
  int32_t n, n_cap, n_rep;
  float tau;
};

struct TreeAccept {
  const void *k, *v;
  const float *beta, *alpha;
  const int32_t *parent, *node;  // [Bs, n], [Bs]
  float *S_cur, *At_cur;
  void *At_cache, *Bc_cache;
  int32_t* n_cache;
  const int32_t* commit;         // [Bs] or null
  int64_t Bs, H;
  int32_t n, n_cap;
};

hipError_t launch_tree_decode(const TreeArgs& a, int dtype, int dk, int dv, hipStream_t s);
hipError_t launch_tree_accept(const TreeAccept& a, int dtype, int dk, int dv, hipStream_t s);

}  // namespace hla
