// C ABI of linear attention with a decay for each head: argument checks, workspace plan and
// dispatch, as in abi.cpp -- an invalid call returns its status with the stream untouched.
#include "../../include/hla.h"

#include <cstdint>

#include "la.hpp"
#include "timing.hpp"

namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 23) - 1;    // rows times segments: a launch counts its threads in 32 bits
constexpr int64_t kMaxTokens = (int64_t)1 << 35;  // a segment's pieces (32 tokens and more) are counted in 32 bits

template <int A, class... P>
bool aligned(P... p) {
  return (((reinterpret_cast<uintptr_t>(p) & (A - 1)) == 0) && ...);
}

hla_status_t status(hipError_t e) { return e == hipSuccess ? HLA_OK : HLA_ERR_HIP; }

// How a row's pieces are cut into segments that run side by side, and what the workspace holds.
struct Plan {
  int64_t rows, n;
  int32_t nseg, seg_pieces;
  size_t fwd, rev, dec_f, dec_r, dS0, b, c, e, dg, dq, dk, total;  // offsets
};

hla_status_t check_dims(const hla_la_dims_t* d) {
  if (!d) return HLA_ERR_NULL_ARG;
  if (d->dtype != HLA_F32 && d->dtype != HLA_BF16) return HLA_ERR_BAD_DTYPE;
  if (d->B < 1 || d->T < 1 || d->H < 1 || d->Hk < 1 || d->ld_T < d->T || d->H % d->Hk) return HLA_ERR_BAD_SHAPE;
  if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128)) return HLA_ERR_BAD_SHAPE;
  if (d->decay_per_head != 0 && d->decay_per_head != 1) return HLA_ERR_BAD_SHAPE;
  if (d->H > 65536 || (double)d->B * (double)d->H > (double)kMaxRows || d->T > kMaxTokens) return HLA_ERR_BAD_SHAPE;
  if ((double)d->B * (double)d->ld_T * (double)d->H * 128.0 > 4.0e18) return HLA_ERR_BAD_SHAPE;
  return HLA_OK;
}

// The number of segments that costs least, in the time that a piece takes a workgroup.  A row that is not
// cut is one pass over its pieces.  One that is cut pays a pass for the segments' states too (about half a
// piece's time a piece), the start of two passes, the states' traffic and the scan's chain; in return as
// many workgroups as the chip runs side by side (two a compute unit; of 64 x 64 states more, by their LDS)
// share the pieces, in rounds, and one that has its compute unit to itself takes three quarters of the time
// (but not the forward call's over 128 x 64 states: its two waves leave half of the unit idle either way).
// The constants are fitted to measured times of 4 to 512 rows of 3 to 160 pieces in all types and widths:
// within 2 per cent of the best number of segments on (geometric) average.  The plain rule before it, as
// many segments of two pieces and more as fill the chip, was 10 per cent behind the best on average and up
// to 90 per cent: 360 rows of 6 pieces (128 x 64, bf16) 96 us in two segments and 50 us uncut; 200 rows
// of 48 (64 x 64) 154 us in three and 121 us in five.
int64_t segments(double rows, int64_t pieces, int64_t least, int dk, int dv, bool backward) {
  const double room = dk + dv > 128 ? 512.0 : backward ? 768.0 : 1024.0, start = backward ? 1.0 : 1.5;
  const double alone = dk > dv && !backward ? 1.0 : 0.75;
  const int64_t most = pieces < hla::kLaSlots ? pieces : hla::kLaSlots;
  int64_t best = 1;
  double cost = 0.0;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t each = (pieces + s - 1) / s;
    if ((pieces + each - 1) / each != s) continue;
    const double all = rows * (double)s, full = all / room;
    if (s > least && full > 4.0) break;
    double x = s > 1 ? 1.5 * (double)each + 2.0 * start : (double)each + start;
    x *= full > 2.0 ? full + 0.5 : full > 1.0 ? 2.0 : all > 256.0 ? 1.0 : alone;
    if (s > 1) x += all / 512.0 + 0.04 * (double)s;
    if (s <= least || x < cost) {
      best = s;
      cost = x;
    }
  }
  return best;
}

hla_status_t plan(const hla_la_dims_t* d, bool backward, bool lens, Plan* p) {
  const int64_t rows = d->B * d->H, piece = hla::la_piece(d->dtype), pieces = (d->T + piece - 1) / piece;
  // The backward call's segments are 32 pieces at most, since the decays' gradient runs differences of sums
  // through a segment; where that makes more than kLaSlots of them, they grow up to kLaChain pieces.  The segments
  // behind a row's length end at once: given lengths count as 0.6 of the rows (lengths drawn from 1 to T, 22 sizes:
  // 0.6 of the rows 2 per cent faster than all of them, and 13 x 1531 tokens of 12 heads of 64 x 128, float32,
  // 196 -> 169 us).  Where lengths are given and all of them are T that costs: over 12 sizes 8 per cent of a prompt and 10
  // of the gradients against a call without lengths on average, at most 20 and 28 (4 x 4096 tokens of 16 heads of
  // 128 x 128, bf16, 133 and 152 us, gradients 420 and 533).
  const int64_t few = (pieces + hla::kLaSlots - 1) / hla::kLaSlots, long_each = few < hla::kLaChain ? few : hla::kLaChain;
  const int64_t nseg = backward && few > 32
      ? (pieces + long_each - 1) / long_each
      : segments((lens ? 0.6 : 1.0) * (double)rows, pieces, backward ? (pieces + 31) / 32 : 1, d->dk, d->dv, backward);
  const int64_t each = (pieces + nseg - 1) / nseg;
  p->rows = rows;
  p->n = (int64_t)d->dk * d->dv;
  p->nseg = (int32_t)nseg;
  p->seg_pieces = (int32_t)each;
  if (rows * nseg > kMaxRows || (nseg > 1 && rows * p->n > 4294967295ll)) return HLA_ERR_BAD_SHAPE;
  if (backward && d->Hk != d->H && (double)d->B * (double)d->T * (double)d->Hk * (d->dk / 4) > 4294967040.0)
    return HLA_ERR_BAD_SHAPE;  // the sum over shared heads
  size_t at = 0;
  auto take = [&at](int64_t bytes) {
    const size_t r = at;
    at += ((size_t)bytes + 255) & ~(size_t)255;
    return r;
  };
  const int64_t state = rows * p->n * 4, tokens = rows * d->T * 4;
  if (!backward) {
    if (nseg > 1) {
      p->fwd = take(state * nseg);
      p->dec_f = take(rows * nseg * 8);
    }
  } else {
    p->fwd = take(state * (nseg + 1));
    if (nseg > 1) {
      p->rev = take(state * nseg);
      p->dec_f = take(rows * nseg * 8);
      p->dec_r = take(rows * nseg * 8);
    }
    p->dS0 = take(state);
    p->b = take(tokens);
    p->c = take(tokens);
    p->e = take(tokens);
    if (d->decay_per_head) p->dg = take(tokens);
    if (d->Hk != d->H) {
      p->dq = take(tokens * d->dk);
      p->dk = take(tokens * d->dk);
    }
  }
  p->total = at;
  return HLA_OK;
}

hla::LaSweep common(const hla_la_dims_t* d, const Plan& p, const float* g, const int32_t* lens) {
  hla::LaSweep a{};
  a.g = g;
  a.ld_g = d->ld_T;
  a.lens = lens;
  a.B = d->B; a.T = d->T; a.H = d->H;
  a.per_head = d->decay_per_head;
  a.nseg = p.nseg;
  a.seg_pieces = p.seg_pieces;
  return a;
}

}  // namespace

extern "C" {

hla_status_t hla_la_workspace_bytes(int32_t fn, const hla_la_dims_t* d, size_t* out) {
  if (!out) return HLA_ERR_NULL_ARG;
  *out = 0;
  if (fn != HLA_LA_PREFILL && fn != HLA_LA_PREFILL_BACKWARD) return HLA_ERR_UNSUPPORTED;
  hla_status_t st = check_dims(d);
  if (st != HLA_OK) return st;
  size_t most = 0;  // enough with lens and without
  for (int lens = 0; lens < 2; ++lens) {
    Plan p{};
    if ((st = plan(d, fn == HLA_LA_PREFILL_BACKWARD, lens, &p)) != HLA_OK) return st;
    if (p.total > most) most = p.total;
  }
  *out = most;
  return HLA_OK;
}

hla_status_t hla_la_prefill(const hla_la_dims_t* d, const void* q, const void* k, const void* v,
                            const float* log_decay, const int32_t* lens, const float* S0, void* o, float* S_final,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  hla_status_t st = check_dims(d);
  if (st != HLA_OK) return st;
  if (!k || !v || !log_decay || (!o && !S_final) || (o && !q)) return HLA_ERR_NULL_ARG;
  if (!aligned<16>(q, k, v, S0, o, S_final, ws) || !aligned<4>(log_decay, lens)) return HLA_ERR_ALIGN;
  Plan p{};
  st = plan(d, false, lens != nullptr, &p);
  if (st != HLA_OK) return st;
  if (p.total && (!ws || ws_bytes < p.total)) return HLA_ERR_WORKSPACE;
  const hla::TimedLaunch tl(HLA_KERNEL_LA, stream);
  char* w = static_cast<char*>(ws);
  float* states = reinterpret_cast<float*>(w + p.fwd);
  hla::LaSweep a = common(d, p, log_decay, lens);
  a.x1 = {q, d->ld_T, (int32_t)d->Hk};
  a.x2 = {k, d->ld_T, (int32_t)d->Hk};
  a.x3 = {v, d->ld_T, (int32_t)d->H};
  hipError_t e;
  if (p.nseg > 1) {
    hla::LaSweep s = a;
    s.loc = states;
    s.loc_row = p.nseg * p.n;
    s.decay = reinterpret_cast<double*>(w + p.dec_f);
    s.whole = o == nullptr;
    if ((e = hla::launch_la_sweep(s, d->dtype, d->dk, d->dv, true, false, stream)) != hipSuccess) return status(e);
    hla::LaScan c{};
    c.init = S0;
    c.state = states;
    c.decay = s.decay;
    c.rows = p.rows;
    c.state_row = p.nseg * p.n;
    c.nseg = p.nseg;
    c.dk = d->dk; c.dv = d->dv;
    if (!o) {
      c.fin = S_final;
      c.fin_row = p.n;
    }
    e = hla::launch_la_scan(c, stream);
    if (e != hipSuccess || !o) return status(e);
    a.init = states;
    a.init_row = p.nseg * p.n;
  } else {
    a.init = S0;
    a.init_row = p.n;
  }
  a.fin = S_final;
  a.fin_row = p.n;
  a.out = o;
  return status(hla::launch_la_sweep(a, d->dtype, d->dk, d->dv, o == nullptr, false, stream));
}

hla_status_t hla_la_prefill_backward(const hla_la_dims_t* d, const void* q, const void* k, const void* v,
                                     const float* log_decay, const int32_t* lens, const float* S0, const void* dO,
                                     const float* dS_final, void* dq, void* dk, void* dv, float* dlog_decay,
                                     float* dS0, void* ws, size_t ws_bytes, hipStream_t stream) {
  hla_status_t st = check_dims(d);
  if (st != HLA_OK) return st;
  if (!q || !k || !v || !log_decay || !dO || !dq || !dk || !dv || !dlog_decay) return HLA_ERR_NULL_ARG;
  if (!aligned<16>(q, k, v, S0, dO, dS_final, dq, dk, dv, dS0, ws) || !aligned<4>(log_decay, lens, dlog_decay))
    return HLA_ERR_ALIGN;
  Plan p{};
  st = plan(d, true, lens != nullptr, &p);
  if (st != HLA_OK) return st;
  if (!ws || ws_bytes < p.total) return HLA_ERR_WORKSPACE;
  const hla::TimedLaunch tl(HLA_KERNEL_BWD_LA, stream);
  char* w = static_cast<char*>(ws);
  auto f = [w](size_t at) { return reinterpret_cast<float*>(w + at); };
  const hla::LaRole rq{q, d->ld_T, (int32_t)d->Hk}, rk{k, d->ld_T, (int32_t)d->Hk}, rv{v, d->ld_T, (int32_t)d->H},
      rdo{dO, d->T, (int32_t)d->H};
  const bool many = p.nseg > 1, shared = d->Hk != d->H;
  const int64_t fwd_row = (p.nseg + 1) * p.n, rev_row = p.nseg * p.n;
  float *fwd = f(p.fwd), *rev = f(p.rev);
  const hla::LaSweep base = common(d, p, log_decay, lens);
  hipError_t e;
  if (many) {  // the states M^T in front of every segment, and the gradients G^T that enter from behind
    for (int r = 0; r < 2; ++r) {
      hla::LaSweep s = base;
      s.x2 = r ? rdo : rv;
      s.x3 = r ? rq : rk;
      s.loc = r ? rev : fwd;
      s.loc_row = r ? rev_row : fwd_row;
      s.decay = reinterpret_cast<double*>(w + (r ? p.dec_r : p.dec_f));
      if ((e = hla::launch_la_sweep(s, d->dtype, d->dv, d->dk, true, r == 1, stream)) != hipSuccess) return status(e);
      hla::LaScan c{};
      c.init = r ? dS_final : S0;
      c.init_t = 1;
      c.state = s.loc;
      c.state_row = s.loc_row;
      c.decay = s.decay;
      c.rows = p.rows;
      c.nseg = p.nseg;
      c.dk = d->dv; c.dv = d->dk;
      c.reverse = r;
      if ((e = hla::launch_la_scan(c, stream)) != hipSuccess) return status(e);
    }
  }
  {  // dq_t = M_t do_t
    hla::LaSweep s = base;
    s.x1 = rdo; s.x2 = rv; s.x3 = rk; s.x4 = rq;
    s.init = many ? fwd : S0;
    s.init_row = many ? fwd_row : p.n;
    s.init_t = !many;
    s.fin = fwd + p.nseg * p.n;
    s.fin_row = fwd_row;
    s.out = shared ? f(p.dq) : dq;
    s.out_f32 = shared;
    s.dot = f(p.c);
    if ((e = hla::launch_la_sweep(s, d->dtype, d->dv, d->dk, false, false, stream)) != hipSuccess) return status(e);
  }
  {  // dk_t = G_t v_t, dv_t = G_t^T k_t
    hla::LaReverse r{};
    r.q = q; r.k = k; r.v = v; r.dO = dO;
    r.g = log_decay;
    r.lens = lens;
    r.init = many ? rev : dS_final;
    r.init_row = many ? rev_row : p.n;
    r.init_t = !many;
    r.dk = shared ? f(p.dk) : dk;
    r.dv = dv;
    r.dS0 = dS0 ? dS0 : S0 ? f(p.dS0) : nullptr;  // the decays' gradient needs it
    r.dot = f(p.b);
    r.esum = f(p.e);
    r.B = d->B; r.T = d->T; r.H = d->H; r.Hk = d->Hk; r.ld_T = d->ld_T;
    r.per_head = d->decay_per_head;
    r.nseg = p.nseg;
    r.seg_pieces = p.seg_pieces;
    r.k_f32 = shared;
    if ((e = hla::launch_la_reverse(r, d->dtype, d->dk, d->dv, stream)) != hipSuccess) return status(e);
  }
  hla::LaDecay c{};
  c.g = log_decay;
  c.ld_g = d->ld_T;
  c.lens = lens;
  c.b = f(p.b); c.c = f(p.c); c.e = f(p.e);
  c.fwd = fwd;
  c.rev = rev;
  c.dS = dS_final;
  c.dg = d->decay_per_head ? f(p.dg) : dlog_decay;
  c.B = d->B; c.T = d->T; c.H = d->H;
  c.per_head = d->decay_per_head;
  c.nseg = p.nseg;
  c.seg_pieces = p.seg_pieces;
  c.n = (int32_t)p.n;
  c.piece = hla::la_piece(d->dtype);
  c.w = d->dk;
  c.S0 = S0;
  c.dS0 = dS0 ? dS0 : f(p.dS0);
  if ((e = hla::launch_la_decay(c, stream)) != hipSuccess) return status(e);
  if (d->decay_per_head && (e = hla::launch_la_head_sum(c.dg, dlog_decay, d->B, d->H, d->T, stream)) != hipSuccess)
    return status(e);
  if (shared) {
    for (int r = 0; r < 2; ++r) {
      const hla::LaGroup s{f(r ? p.dk : p.dq), r ? dk : dq, d->B * d->T, (int32_t)(d->H / d->Hk), d->dk, (int32_t)d->Hk};
      if ((e = hla::launch_la_group_sum(s, d->dtype, stream)) != hipSuccess) return status(e);
    }
  }
  return HLA_OK;
}

hla_status_t hla_la_decode(int64_t Bs, int64_t H, int64_t Hk, int32_t dk, int32_t dv, int32_t dtype, const void* q,
                           const void* k, const void* v, const float* log_decay, int32_t decay_per_head, float* S,
                           void* o, hipStream_t stream) {
  const hla_la_dims_t d{Bs, 1, H, Hk, 1, dk, dv, dtype, decay_per_head};
  const hla_status_t st = check_dims(&d);
  if (st != HLA_OK) return st;
  if (!q || !k || !v || !log_decay || !S || !o) return HLA_ERR_NULL_ARG;
  if (!aligned<16>(S) || !aligned<4>(q, k, v, log_decay, o)) return HLA_ERR_ALIGN;
  const hla::TimedLaunch tl(HLA_KERNEL_LA, stream);
  hla::LaStep a{};
  a.q = q; a.k = k; a.v = v; a.g = log_decay; a.S = S; a.o = o;
  a.Bs = Bs; a.H = H;
  a.group = (int32_t)(H / Hk);
  a.per_head = decay_per_head;
  return status(hla::launch_la_step(a, dtype, dk, dv, stream));
}

}  // extern "C"
