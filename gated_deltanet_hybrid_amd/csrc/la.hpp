// Linear attention with a decay for each head: what the kernels take, and their launchers.
#pragma once
#include "common.hpp"

namespace hla {

constexpr int kLaSlots = 128;  // most segments of a row, unless its segments of kLaChain pieces are more (backward)
constexpr int kLaChain = 64;   // most pieces of a segment of the backward call: la_decay_kernel holds them

// One token tensor in a role of the recurrence: [B, ld, heads, width] of the call's dtype; heads
// divides the call's heads, and neighbouring heads share.
struct LaRole {
  const void* p;
  int64_t ld;
  int32_t heads;
};

// One sweep of the recurrence M_t = exp(g_t) M_{t-1} + x2_t x3_t^T, out_t = M_t^T x1_t over the
// tokens of every row (b, h), cut into nseg segments of seg_pieces pieces.  Reversed sweeps (states only) run from
// the last token to the first and take the decay of the token behind (x1, x2, x3 at t; g at t + 1).
struct LaSweep {
  LaRole x1, x2, x3, x4;
  const float* g;        // [B, ld_g, H], or [H] (per_head)
  int64_t ld_g;
  const int32_t* lens;   // [B] or null
  const float* init;     // state in front of segment s of row r: init + r init_row + s dk dv, or null
  int64_t init_row;
  int32_t init_t;        // the initial state is stored transposed
  float* loc;            // state pass: where every segment's state from zero goes, as init
  int64_t loc_row;
  double* decay;         // [rows, nseg]: sum of g over each segment (state pass)
  float* fin;            // state behind the last token: fin + r fin_row, or null
  int64_t fin_row;
  void* out;             // [B, T, H, width of x3], the call's dtype or float32
  float* dot;            // [rows, T]: x4_t . (the part of out_t that comes from the piece's start), or null
  int64_t B, T, H;
  int32_t per_head, nseg, seg_pieces, out_f32;
  int32_t whole;         // state pass: the last segment's state is asked for too
};

// dk_t = G_t v_t and dv_t = G_t^T k_t, reversed.
struct LaReverse {
  const void *q, *k, *v, *dO;
  const float* g;
  const int32_t* lens;
  const float* init;     // the gradient that enters segment s of row r from behind: init + r init_row + s dk dv, or null
  int64_t init_row;
  int32_t init_t;        // stored [dk, dv], else [dv, dk]
  void* dk;              // [B, T, Hk, dk] of the call's dtype, or (k_f32) [B, T, H, dk] float32: every head's part
  void* dv;              // [B, T, H, dv]
  float* dS0;            // [rows, dk, dv] or null
  float *dot, *esum;     // [rows, T]: see la_decay_kernel
  int64_t B, T, H, Hk, ld_T;
  int32_t per_head, nseg, seg_pieces, k_f32;
};

struct LaScan {
  const float* init;     // [rows, n] or null; init_t: stored transposed, [dv, dk] read as [dk, dv]
  float* state;          // in: segments' states from zero; out: the state in front of each segment
  const double* decay;   // [rows, nseg]
  float* fin;            // state behind the last segment: fin + r fin_row, or null
  int64_t rows, state_row, fin_row;
  int32_t nseg, dk, dv, reverse, init_t;
};

struct LaDecay {         // the gradient of g from the sweeps' dot products
  const float* g;
  int64_t ld_g;
  const int32_t* lens;
  const float *b, *c, *e;     // [rows, T]
  const float* fwd;           // [rows, nseg + 1, n]: states in front of each segment, and behind the last
  const float* rev;           // [rows, nseg, n]: the gradient that enters each segment from behind (but the last's)
  const float* dS;            // [rows, n transposed] or null: the final state's gradient
  const float *S0, *dS0;      // [rows, n transposed]: the initial state and its gradient; S0 null: zero
  float* dg;                  // [B, T, H], or [rows, T] (per_head)
  int64_t B, T, H;
  int32_t per_head, nseg, seg_pieces, n, piece, w;  // n = dk dv; w: the row width of fwd and rev
};

struct LaGroup { const float* x; void* y; int64_t tokens; int32_t group, width, heads; };

struct LaStep {
  const void *q, *k, *v;
  const float* g;
  float* S;
  void* o;
  int64_t Bs, H;
  int32_t group, per_head;
};

int la_piece(int dtype);                       // tokens of a piece
hipError_t launch_la_sweep(const LaSweep& a, int dtype, int dk, int dv, bool state_only, bool reverse, hipStream_t s);
hipError_t launch_la_reverse(const LaReverse& a, int dtype, int dk, int dv, hipStream_t s);
hipError_t launch_la_scan(const LaScan& a, hipStream_t s);
hipError_t launch_la_decay(const LaDecay& a, hipStream_t s);
hipError_t launch_la_head_sum(const float* x, float* y, int64_t B, int64_t H, int64_t T, hipStream_t s);
hipError_t launch_la_group_sum(const LaGroup& a, int dtype, hipStream_t s);
hipError_t launch_la_step(const LaStep& a, int dtype, int dk, int dv, hipStream_t s);

}  // namespace hla
