// C ABI of the operators around the read step: argument validation and dispatch (the contract is
// in include/ccq.h).  Nothing here allocates, keeps state between calls or synchronises.
#include <hip/hip_runtime.h>
#include <math.h>

#include "ccq.h"
#include "ccq_internal.hpp"

namespace {

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool bad_dtype(int dtype) { return dtype != CCQ_DTYPE_F32 && dtype != CCQ_DTYPE_BF16; }
size_t esize(int dtype) { return dtype == CCQ_DTYPE_BF16 ? 2 : 4; }

// The bytes a call may touch behind a pointer, from its first to its last.
struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
// Whether a written range meets any other one.  The first `written` of the n ranges are written.
bool written_overlaps(const Range* r, int n, int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(r[i], r[j])) return true;
  return false;
}
template <int N>
bool any_misaligned(const Range (&r)[N]) {
  for (const Range& x : r)
    if (misaligned(x.p)) return true;
  return false;
}

bool bad_stride(int64_t s, size_t E) { return ((uint64_t)s * E & 15u) != 0; }
constexpr int64_t kMaxSpan = (int64_t)1 << 46;  // elements a stride may span; keeps byte offsets inside 64 bits

// Bytes from the first to the last element of [n0, n1, n2, inner] with these strides.
size_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t inner, size_t E) {
  return (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + inner) * E;
}
bool stride_in_range(int64_t n, int64_t s) { return s >= 0 && s <= kMaxSpan && (n <= 1 || s <= kMaxSpan / (n - 1)); }
bool strides_in_range(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
  return stride_in_range(n0, s0) && stride_in_range(n1, s1) && stride_in_range(n2, s2);
}

// ---------------------------------------------------------------- queries and keys

int qk_sizes(const ccq_qk_params& p) {
  if (bad_dtype(p.dtype)) return CCQ_ERR_INVALID_ARG;
  if (p.B <= 0 || p.T <= 0 || p.H_q < 0 || p.H_k < 0 || p.H_q + (long long)p.H_k <= 0 || p.d <= 0) return CCQ_ERR_INVALID_ARG;
  if (p.q_norm < CCQ_NORM_NONE || p.q_norm > CCQ_NORM_L2 || p.k_norm < CCQ_NORM_NONE || p.k_norm > CCQ_NORM_L2)
    return CCQ_ERR_INVALID_ARG;
  if ((p.interleaved | p.expand_keys) & ~1) return CCQ_ERR_INVALID_ARG;
  if (!(p.eps >= 0.f) || isinf(p.eps)) return CCQ_ERR_INVALID_ARG;
  if (p.rot < 0 || p.rot > p.d) return CCQ_ERR_INVALID_ARG;
  if (p.expand_keys && (p.H_k == 0 || p.H_q == 0 || p.H_q % p.H_k != 0)) return CCQ_ERR_INVALID_ARG;
  if ((p.d != 64 && p.d != 128) || p.rot % 16 != 0) return CCQ_ERR_UNSUPPORTED;
  if ((long long)p.B * p.T > (1LL << 30) || p.H_q > 4096 || p.H_k > 4096) return CCQ_ERR_UNSUPPORTED;
  if ((p.H_q > 0) != (p.q != nullptr) || (p.H_k > 0) != (p.k != nullptr)) return CCQ_ERR_INVALID_ARG;
  if ((p.rot > 0) != (p.inv_freq != nullptr)) return CCQ_ERR_INVALID_ARG;
  if ((p.q_weight && !p.q) || (p.k_weight && !p.k)) return CCQ_ERR_INVALID_ARG;
  if (!strides_in_range(p.B, p.q_stride_b, p.T, p.q_stride_t, p.H_q, p.q_stride_h) ||
      !strides_in_range(p.B, p.k_stride_b, p.T, p.k_stride_t, p.H_k, p.k_stride_h))
    return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p.dtype);
  for (int64_t s : {p.q_stride_b, p.q_stride_t, p.q_stride_h, p.k_stride_b, p.k_stride_t, p.k_stride_h})
    if (bad_stride(s, E)) return CCQ_ERR_MISALIGNED;
  return CCQ_OK;
}

// Extents of one side, dense head-major (out) and strided token-major (in).
size_t qk_dense(const ccq_qk_params& p, int heads, size_t E) { return (size_t)p.B * heads * p.T * p.d * E; }
size_t qk_q_extent(const ccq_qk_params& p) {
  return p.H_q ? extent(p.B, p.q_stride_b, p.T, p.q_stride_t, p.H_q, p.q_stride_h, p.d, esize(p.dtype)) : 0;
}
size_t qk_k_extent(const ccq_qk_params& p) {
  return p.H_k ? extent(p.B, p.k_stride_b, p.T, p.k_stride_t, p.H_k, p.k_stride_h, p.d, esize(p.dtype)) : 0;
}

int validate_qk(const ccq_qk_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const int st = qk_sizes(*p);
  if (st != CCQ_OK) return st;
  if (!ccq::qk_grid_fits(*p)) return CCQ_ERR_UNSUPPORTED;
  if ((p->H_q > 0) != (p->q_out != nullptr) || (p->H_k > 0) != (p->k_out != nullptr)) return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p->dtype);
  const Range r[] = {{p->q_out, qk_dense(*p, p->H_q, E)},
                     {p->k_out, qk_dense(*p, p->expand_keys ? p->H_q : p->H_k, E)},
                     {p->q, qk_q_extent(*p)},
                     {p->k, qk_k_extent(*p)},
                     {p->positions, (size_t)p->B * p->T * 8},
                     {p->inv_freq, (size_t)p->rot * 2},
                     {p->q_weight, (size_t)p->d * 4},
                     {p->k_weight, (size_t)p->d * 4}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 8, 2)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

// Whether rows of `inner` elements at these strides are all apart: sorted by stride, every dimension
// steps over what the smaller ones span.
bool rows_apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t inner) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
  int64_t span = inner;
  bool used[3] = {n[0] <= 1, n[1] <= 1, n[2] <= 1};
  for (int round = 0; round < 3; ++round) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (best < 0 || s[i] < s[best])) best = i;
    if (best < 0) break;
    if (s[best] < span) return false;
    span += (n[best] - 1) * s[best];
    used[best] = true;
  }
  return true;
}

int validate_qk_backward(const ccq_qk_bwd_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const ccq_qk_params& f = p->fwd;
  const int st = qk_sizes(f);
  if (st != CCQ_OK) return st;
  if ((f.H_q > 0) != (p->dq_out != nullptr) || (f.H_q > 0) != (p->dq != nullptr) ||
      (f.H_k > 0) != (p->dk_out != nullptr) || (f.H_k > 0) != (p->dk != nullptr))
    return CCQ_ERR_INVALID_ARG;
  if ((f.q_weight != nullptr) != (p->dq_weight != nullptr) || (f.k_weight != nullptr) != (p->dk_weight != nullptr))
    return CCQ_ERR_INVALID_ARG;
  if (!strides_in_range(f.B, p->dq_stride_b, f.T, p->dq_stride_t, f.H_q, p->dq_stride_h) ||
      !strides_in_range(f.B, p->dk_stride_b, f.T, p->dk_stride_t, f.H_k, p->dk_stride_h))
    return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(f.dtype);
  for (int64_t s : {p->dq_stride_b, p->dq_stride_t, p->dq_stride_h, p->dk_stride_b, p->dk_stride_t, p->dk_stride_h})
    if (bad_stride(s, E)) return CCQ_ERR_MISALIGNED;
  if (f.H_q && !rows_apart(f.B, p->dq_stride_b, f.T, p->dq_stride_t, f.H_q, p->dq_stride_h, f.d)) return CCQ_ERR_INVALID_ARG;
  if (f.H_k && !rows_apart(f.B, p->dk_stride_b, f.T, p->dk_stride_t, f.H_k, p->dk_stride_h, f.d)) return CCQ_ERR_INVALID_ARG;
  const size_t dq_extent = f.H_q ? extent(f.B, p->dq_stride_b, f.T, p->dq_stride_t, f.H_q, p->dq_stride_h, f.d, E) : 0;
  const size_t dk_extent = f.H_k ? extent(f.B, p->dk_stride_b, f.T, p->dk_stride_t, f.H_k, p->dk_stride_h, f.d, E) : 0;
  const Range r[] = {{p->dq_weight, (size_t)f.d * 4},
                     {p->dk_weight, (size_t)f.d * 4},
                     {p->dq, dq_extent},
                     {p->workspace, ccq::qk_backward_workspace_bytes(*p)},
                     {p->dk, dk_extent},
                     {p->dq_out, qk_dense(f, f.H_q, 4)},
                     {p->dk_out, qk_dense(f, f.expand_keys ? f.H_q : f.H_k, 4)},
                     {f.q, qk_q_extent(f)},
                     {f.k, qk_k_extent(f)},
                     {f.positions, (size_t)f.B * f.T * 8},
                     {f.inv_freq, (size_t)f.rot * 2},
                     {f.q_weight, (size_t)f.d * 4},
                     {f.k_weight, (size_t)f.d * 4}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  // dq and dk are commonly the two parts of one packed gradient: their extents interleave, their
  // rows do not.  Where not even their first rows are apart the call is refused; for the others the
  // caller answers.
  if (overlap({p->dq, (size_t)f.d * E}, {p->dk, (size_t)f.d * E})) return CCQ_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 13; ++j)
      if (!(i == 2 && j == 4) && overlap(r[i], r[j])) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

// ---------------------------------------------------------------- gated linear recurrence

int scan_sizes(int dtype, int B, int T, int D, int complement) {
  if (bad_dtype(dtype) || B <= 0 || T <= 0 || D <= 0 || (complement & ~1)) return CCQ_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > (1 << 24) || (long long)B * T > (1LL << 30) || (long long)B * D > 0x7fffffffLL) return CCQ_ERR_UNSUPPORTED;
  return CCQ_OK;
}
size_t scan_carry_bytes(int B, int T, int D) { return (size_t)B * ((T + 63) / 64) * D * 4; }

int validate_scan(const ccq_scan_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const int st = scan_sizes(p->dtype, p->B, p->T, p->D, p->complement);
  if (st != CCQ_OK) return st;
  if (!ccq::scan_grid_fits(p->dtype, p->B, p->T, p->D)) return CCQ_ERR_UNSUPPORTED;
  if (!p->x || !p->log_alpha || !p->y) return CCQ_ERR_INVALID_ARG;
  if (!strides_in_range(p->B, p->x_stride_b, p->T, p->x_stride_t, 1, 0) ||
      !strides_in_range(p->B, p->la_stride_b, p->T, p->la_stride_t, 1, 0))
    return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p->dtype), state = (size_t)p->B * p->D * 4;
  for (int64_t s : {p->x_stride_b, p->x_stride_t, p->la_stride_b, p->la_stride_t})
    if (bad_stride(s, E)) return CCQ_ERR_MISALIGNED;
  const Range r[] = {{p->y, (size_t)p->B * p->T * p->D * E},
                     {p->chunk_carry, scan_carry_bytes(p->B, p->T, p->D)},
                     {p->workspace, ccq::scan_workspace_bytes(*p)},
                     {p->h_out, state},
                     {p->x, extent(p->B, p->x_stride_b, p->T, p->x_stride_t, 1, 0, p->D, E)},
                     {p->log_alpha, extent(p->B, p->la_stride_b, p->T, p->la_stride_t, 1, 0, p->D, E)},
                     {p->lengths, (size_t)p->B * 4},
                     {p->h_out == p->h0 ? nullptr : p->h0, state}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 8, 4)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

int validate_scan_backward(const ccq_scan_bwd_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const int st = scan_sizes(p->dtype, p->B, p->T, p->D, p->complement);
  if (st != CCQ_OK) return st;
  if (!ccq::scan_backward_grid_fits(*p)) return CCQ_ERR_UNSUPPORTED;
  if (!p->x || !p->log_alpha || !p->dy || !p->dx || !p->dlog_alpha) return CCQ_ERR_INVALID_ARG;
  if (!strides_in_range(p->B, p->x_stride_b, p->T, p->x_stride_t, p->B, p->dy_stride_b) ||
      !strides_in_range(p->B, p->la_stride_b, p->T, p->la_stride_t, p->T, p->dy_stride_t))
    return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p->dtype), state = (size_t)p->B * p->D * 4, all = (size_t)p->B * p->T * p->D * E;
  for (int64_t s : {p->x_stride_b, p->x_stride_t, p->la_stride_b, p->la_stride_t, p->dy_stride_b, p->dy_stride_t})
    if (bad_stride(s, E)) return CCQ_ERR_MISALIGNED;
  const Range r[] = {{p->dx, all},
                     {p->dlog_alpha, all},
                     {p->workspace, ccq::scan_backward_workspace_bytes(*p)},
                     {p->dh0, state},
                     {p->x, extent(p->B, p->x_stride_b, p->T, p->x_stride_t, 1, 0, p->D, E)},
                     {p->log_alpha, extent(p->B, p->la_stride_b, p->T, p->la_stride_t, 1, 0, p->D, E)},
                     {p->dy, extent(p->B, p->dy_stride_b, p->T, p->dy_stride_t, 1, 0, p->D, E)},
                     {p->lengths, (size_t)p->B * 4},
                     {p->h0, state},
                     {p->chunk_carry, scan_carry_bytes(p->B, p->T, p->D)},
                     {p->dh0 == p->dh_out ? nullptr : p->dh_out, state}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 11, 4)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

// ---------------------------------------------------------------- beams

int validate_beam(const ccq_beam_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  if (bad_dtype(p->dtype) || p->N <= 0 || p->K <= 0 || p->V <= 0 || p->M <= 0) return CCQ_ERR_INVALID_ARG;
  if ((long long)p->M > (long long)p->K * p->V) return CCQ_ERR_INVALID_ARG;
  if (p->logits_stride < p->V || p->logits_stride > ((int64_t)1 << 36)) return CCQ_ERR_INVALID_ARG;
  if (p->pad_token < 0 || p->pad_token >= p->V) return CCQ_ERR_INVALID_ARG;
  const long long chunks = ((long long)p->V + ccq::kBeamMaxChunk - 1) / ccq::kBeamMaxChunk;
  if (p->K > ccq::kBeamMaxBeams || p->M > ccq::kBeamMaxPicks || (long long)p->K * p->V > 0x7fffffffLL ||
      p->K * chunks > ccq::kBeamMaxLists || !ccq::beam_grid_fits(*p))
    return CCQ_ERR_UNSUPPORTED;
  if (!p->logits || !p->scores || !p->token || !p->parent || !p->score) return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p->dtype), rows = (size_t)p->N * p->K, picks = (size_t)p->N * p->M * 4;
  const Range r[] = {{p->token, picks},
                     {p->parent, picks},
                     {p->score, picks},
                     {p->workspace, ccq::beam_workspace_bytes(*p)},
                     {p->logits, ((rows - 1) * (size_t)p->logits_stride + p->V) * E},
                     {p->scores, rows * 4},
                     {p->finished, rows}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 7, 4)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

// ---------------------------------------------------------------- linear attention

// A tensor of a call: [B, T, heads, d], or [rows, heads, d] packed, at these strides.
struct Layout {
  const void* p;
  int64_t b, t, h;
  int heads, d;
};
struct Tokens {
  int64_t nb, nt;  // sequences and tokens as the strides count them
  explicit Tokens(const ccq_linear_attn_params& p) : nb(p.offsets ? 1 : p.B), nt(p.offsets ? p.rows : p.T) {}
};
size_t extent_of(const Layout& l, const Tokens& n, size_t E) {
  return extent(n.nb, n.nb > 1 ? l.b : 0, n.nt, l.t, l.heads, l.h, l.d, E);
}
int check_layout(const Layout& l, const Tokens& n, size_t E, bool written) {
  const int64_t b = n.nb > 1 ? l.b : 0;
  if (!strides_in_range(n.nb, b, n.nt, l.t, l.heads, l.h)) return CCQ_ERR_INVALID_ARG;
  if (bad_stride(b, E) || bad_stride(l.t, E) || bad_stride(l.h, E)) return CCQ_ERR_MISALIGNED;
  if (n.nt > 1 && l.t >= (1 << 24)) return CCQ_ERR_UNSUPPORTED;  // a chunk's rows are told apart by 32-bit offsets
  if (written && !rows_apart(n.nb, b, n.nt, l.t, l.heads, l.h, l.d)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}
Layout la_q(const ccq_linear_attn_params& p) { return {p.q, p.q_stride_b, p.q_stride_t, p.q_stride_h, p.H_q, p.d_k}; }
Layout la_k(const ccq_linear_attn_params& p) { return {p.k, p.k_stride_b, p.k_stride_t, p.k_stride_h, p.H_k, p.d_k}; }
Layout la_v(const ccq_linear_attn_params& p) { return {p.v, p.v_stride_b, p.v_stride_t, p.v_stride_h, p.H_v, p.d_v}; }

// What the forward and the gradient have in common.
int la_inputs(const ccq_linear_attn_params& p) {
  if (bad_dtype(p.dtype) || bad_dtype(p.gate_dtype)) return CCQ_ERR_INVALID_ARG;
  if (p.B <= 0 || p.T <= 0 || p.H <= 0 || p.H_q <= 0 || p.H_k <= 0 || p.H_v <= 0 || p.d_k <= 0 || p.d_v <= 0) return CCQ_ERR_INVALID_ARG;
  if (p.H % p.H_q != 0 || p.H % p.H_k != 0 || p.H % p.H_v != 0) return CCQ_ERR_INVALID_ARG;
  if (!isfinite(p.scale)) return CCQ_ERR_INVALID_ARG;
  if ((p.d_k != 64 && p.d_k != 128) || (p.d_v != 64 && p.d_v != 128)) return CCQ_ERR_UNSUPPORTED;
  if ((long long)p.B * p.H > (1LL << 20) || (long long)p.B * p.T > (1LL << 30) || p.rows >= (1LL << 31)) return CCQ_ERR_UNSUPPORTED;
  if (!p.q || !p.k || !p.v) return CCQ_ERR_INVALID_ARG;
  if ((p.lengths && p.offsets) || (p.offsets ? p.rows <= 0 : p.rows != 0)) return CCQ_ERR_INVALID_ARG;
  const Tokens n(p);
  const size_t E = esize(p.dtype);
  for (const Layout& l : {la_q(p), la_k(p), la_v(p)}) {
    const int st = check_layout(l, n, E, false);
    if (st != CCQ_OK) return st;
  }
  // gates are read one by one: a slice of another tensor will do
  if (reinterpret_cast<uintptr_t>(p.log_alpha) % esize(p.gate_dtype) != 0) return CCQ_ERR_MISALIGNED;
  if (p.log_alpha && !strides_in_range(n.nb, n.nb > 1 ? p.la_stride_b : 0, n.nt, p.la_stride_t, p.H, p.la_stride_h))
    return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}
size_t la_gate_extent(const ccq_linear_attn_params& p, const Tokens& n) {
  return extent(n.nb, n.nb > 1 ? p.la_stride_b : 0, n.nt, p.la_stride_t, p.H, p.la_stride_h, 1, esize(p.gate_dtype));
}
size_t la_state(const ccq_linear_attn_params& p) { return (size_t)p.B * p.H * p.d_k * p.d_v * 4; }

int validate_la(const ccq_linear_attn_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  int st = la_inputs(*p);
  if (st != CCQ_OK) return st;
  if (!p->o) return CCQ_ERR_INVALID_ARG;
  const Tokens n(*p);
  const size_t E = esize(p->dtype);
  const Layout o{p->o, p->o_stride_b, p->o_stride_t, p->o_stride_h, p->H, p->d_v};
  st = check_layout(o, n, E, true);
  if (st != CCQ_OK) return st;
  const Range r[] = {{p->o, extent_of(o, n, E)},
                     {p->S_out, la_state(*p)},
                     {p->workspace, ccq::linear_attn_workspace_bytes(*p)},
                     {p->q, extent_of(la_q(*p), n, E)},
                     {p->k, extent_of(la_k(*p), n, E)},
                     {p->v, extent_of(la_v(*p), n, E)},
                     {p->lengths, (size_t)p->B * 4},
                     {p->offsets, (size_t)p->B * 4 + 4},
                     {p->S0 == p->S_out ? nullptr : p->S0, la_state(*p)}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 9, 3)) return CCQ_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (overlap(r[i], {p->log_alpha, la_gate_extent(*p, n)})) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

int validate_la_backward(const ccq_linear_attn_bwd_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const ccq_linear_attn_params& f = p->fwd;
  int st = la_inputs(f);
  if (st != CCQ_OK) return st;
  if (bad_dtype(p->grad_dtype) || (f.dtype == CCQ_DTYPE_F32 && p->grad_dtype != CCQ_DTYPE_F32)) return CCQ_ERR_INVALID_ARG;
  if (!p->d_o || !p->dq || !p->dk || !p->dv || (p->dlog_alpha && !f.log_alpha)) return CCQ_ERR_INVALID_ARG;
  const Tokens n(f);
  const size_t E = esize(f.dtype), GE = esize(p->grad_dtype);
  const Layout d_o{p->d_o, p->do_stride_b, p->do_stride_t, p->do_stride_h, f.H, f.d_v};
  const Layout g[3] = {{p->dq, p->dq_stride_b, p->dq_stride_t, p->dq_stride_h, f.H_q, f.d_k},
                       {p->dk, p->dk_stride_b, p->dk_stride_t, p->dk_stride_h, f.H_k, f.d_k},
                       {p->dv, p->dv_stride_b, p->dv_stride_t, p->dv_stride_h, f.H_v, f.d_v}};
  st = check_layout(d_o, n, E, false);
  if (st != CCQ_OK) return st;
  for (const Layout& l : g) {
    st = check_layout(l, n, GE, true);
    if (st != CCQ_OK) return st;
  }
  const Range r[] = {{p->dq, extent_of(g[0], n, GE)},
                     {p->dk, extent_of(g[1], n, GE)},
                     {p->dv, extent_of(g[2], n, GE)},
                     {p->dlog_alpha, (size_t)(n.nb * n.nt) * f.H * esize(f.gate_dtype)},
                     {p->dS0, la_state(f)},
                     {p->workspace, ccq::linear_attn_backward_workspace_bytes(*p)},
                     {p->d_o, extent_of(d_o, n, E)},
                     {f.q, extent_of(la_q(f), n, E)},
                     {f.k, extent_of(la_k(f), n, E)},
                     {f.v, extent_of(la_v(f), n, E)},
                     {f.lengths, (size_t)f.B * 4},
                     {f.offsets, (size_t)f.B * 4 + 4},
                     {f.S0, la_state(f)},
                     {p->dS_out, la_state(f)}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  // dq, dk and dv are commonly parts of one packed gradient, whose extents interleave: their first rows must
  // be apart, for the others the caller answers.
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (overlap({g[i].p, g[i].d * GE}, {g[j].p, g[j].d * GE})) return CCQ_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i) {
    for (int j = i < 3 ? 3 : i + 1; j < 14; ++j)
      if (overlap(r[i], r[j])) return CCQ_ERR_INVALID_ARG;
    if (overlap(r[i], {f.log_alpha, la_gate_extent(f, n)})) return CCQ_ERR_INVALID_ARG;
  }
  return CCQ_OK;
}

// ---------------------------------------------------------------- group norm

int norm_tensor(int64_t sb, int64_t st, int64_t sh, const ccq_group_norm_params& p, bool written) {
  if (!strides_in_range(p.B, sb, p.T, st, p.G, sh)) return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p.dtype);
  if (bad_stride(sb, E) || bad_stride(st, E) || bad_stride(sh, E)) return CCQ_ERR_MISALIGNED;
  if (written && !rows_apart(p.B, sb, p.T, st, p.G, sh, p.d)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}
size_t norm_extent(int64_t sb, int64_t st, int64_t sh, const ccq_group_norm_params& p) {
  return extent(p.B, sb, p.T, st, p.G, sh, p.d, esize(p.dtype));
}
int norm_inputs(const ccq_group_norm_params& p) {
  if (bad_dtype(p.dtype) || p.B <= 0 || p.T <= 0 || p.G <= 0 || p.d <= 0) return CCQ_ERR_INVALID_ARG;
  if (((p.center | p.affine_shared) & ~1) || p.activation < CCQ_ACT_NONE || p.activation > CCQ_ACT_SIGMOID) return CCQ_ERR_INVALID_ARG;
  if (!(p.eps >= 0.f) || isinf(p.eps)) return CCQ_ERR_INVALID_ARG;
  if (p.d % 8 != 0 || p.d > 1024 || p.G > 65535 || (long long)p.B * p.T > 0x7fffffffLL / p.G) return CCQ_ERR_UNSUPPORTED;
  if (!p.x) return CCQ_ERR_INVALID_ARG;
  int st = norm_tensor(p.x_stride_b, p.x_stride_t, p.x_stride_h, p, false);
  if (st == CCQ_OK && p.gate) st = norm_tensor(p.gate_stride_b, p.gate_stride_t, p.gate_stride_h, p, false);
  return st;
}
size_t norm_affine(const ccq_group_norm_params& p) { return (size_t)p.d * (p.affine_shared ? 1 : p.G) * 4; }

int validate_norm(const ccq_group_norm_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  int st = norm_inputs(*p);
  if (st != CCQ_OK) return st;
  if (!p->y) return CCQ_ERR_INVALID_ARG;
  st = norm_tensor(p->y_stride_b, p->y_stride_t, p->y_stride_h, *p, true);
  if (st != CCQ_OK) return st;
  auto same = [&](const void* q, int64_t b, int64_t t, int64_t h) {
    return q == p->y && b == p->y_stride_b && t == p->y_stride_t && h == p->y_stride_h;
  };
  const Range r[] = {{p->y, norm_extent(p->y_stride_b, p->y_stride_t, p->y_stride_h, *p)},
                     {same(p->x, p->x_stride_b, p->x_stride_t, p->x_stride_h) ? nullptr : p->x,
                      norm_extent(p->x_stride_b, p->x_stride_t, p->x_stride_h, *p)},
                     {same(p->gate, p->gate_stride_b, p->gate_stride_t, p->gate_stride_h) ? nullptr : p->gate,
                      p->gate ? norm_extent(p->gate_stride_b, p->gate_stride_t, p->gate_stride_h, *p) : 0},
                     {p->weight, norm_affine(*p)},
                     {p->bias, norm_affine(*p)}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 5, 1)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

int validate_norm_backward(const ccq_group_norm_bwd_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  const ccq_group_norm_params& f = p->fwd;
  int st = norm_inputs(f);
  if (st != CCQ_OK) return st;
  if (!p->dy || !p->dx || (f.gate != nullptr) != (p->dgate != nullptr) || (f.weight != nullptr) != (p->dweight != nullptr) ||
      (f.bias != nullptr) != (p->dbias != nullptr))
    return CCQ_ERR_INVALID_ARG;
  st = norm_tensor(p->dy_stride_b, p->dy_stride_t, p->dy_stride_h, f, false);
  if (st == CCQ_OK) st = norm_tensor(p->dx_stride_b, p->dx_stride_t, p->dx_stride_h, f, true);
  if (st == CCQ_OK && p->dgate) st = norm_tensor(p->dgate_stride_b, p->dgate_stride_t, p->dgate_stride_h, f, true);
  if (st != CCQ_OK) return st;
  const bool in_dy = p->dx == p->dy && p->dx_stride_b == p->dy_stride_b && p->dx_stride_t == p->dy_stride_t && p->dx_stride_h == p->dy_stride_h;
  const bool in_gate = p->dgate == f.gate && p->dgate_stride_b == f.gate_stride_b && p->dgate_stride_t == f.gate_stride_t &&
                       p->dgate_stride_h == f.gate_stride_h;
  const Range r[] = {{p->dx, norm_extent(p->dx_stride_b, p->dx_stride_t, p->dx_stride_h, f)},
                     {p->dgate, p->dgate ? norm_extent(p->dgate_stride_b, p->dgate_stride_t, p->dgate_stride_h, f) : 0},
                     {p->dweight, norm_affine(f)},
                     {p->dbias, norm_affine(f)},
                     {p->workspace, ccq::group_norm_backward_workspace_bytes(*p)},
                     {in_dy ? nullptr : p->dy, norm_extent(p->dy_stride_b, p->dy_stride_t, p->dy_stride_h, f)},
                     {f.x, norm_extent(f.x_stride_b, f.x_stride_t, f.x_stride_h, f)},
                     {in_gate ? nullptr : f.gate, f.gate ? norm_extent(f.gate_stride_b, f.gate_stride_t, f.gate_stride_h, f) : 0},
                     {f.weight, norm_affine(f)},
                     {f.bias, norm_affine(f)}};
  if (any_misaligned(r)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 10, 5)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

// ---------------------------------------------------------------- logits

int validate_adjust(const ccq_logits_adjust_params* p) {
  if (!p) return CCQ_ERR_INVALID_ARG;
  if (bad_dtype(p->dtype) || p->R <= 0 || p->V <= 0 || p->L < 0 || p->n_bias < 0) return CCQ_ERR_INVALID_ARG;
  if (p->logits_stride < p->V || p->out_stride < p->V || p->logits_stride > ((int64_t)1 << 36) || p->out_stride > ((int64_t)1 << 36))
    return CCQ_ERR_INVALID_ARG;
  if ((p->L > 0) != (p->history != nullptr) || (p->n_bias > 0) != (p->bias_token != nullptr) ||
      (p->n_bias > 0) != (p->bias_value != nullptr) || (p->L == 0 && (p->lengths || p->prompt_lengths)))
    return CCQ_ERR_INVALID_ARG;
  if (!(p->repetition > 0.f) || isinf(p->repetition) || !isfinite(p->presence) || !isfinite(p->frequency)) return CCQ_ERR_INVALID_ARG;
  if (p->n_bias > 1024 || p->V > (1 << 24) || p->L > (1 << 24) || !ccq::logits_adjust_grid_fits(*p)) return CCQ_ERR_UNSUPPORTED;
  if (!p->logits || !p->out) return CCQ_ERR_INVALID_ARG;
  const size_t E = esize(p->dtype), rows = (size_t)p->R;
  const bool in_place = p->out == p->logits && p->out_stride == p->logits_stride;
  const Range r[] = {{p->out, ((rows - 1) * (size_t)p->out_stride + p->V) * E},
                     {in_place ? nullptr : p->logits, ((rows - 1) * (size_t)p->logits_stride + p->V) * E},
                     {p->history, rows * p->L * 4},
                     {p->lengths, rows * 4},
                     {p->prompt_lengths, rows * 4},
                     {p->repetition_rows, rows * 4},
                     {p->presence_rows, rows * 4},
                     {p->frequency_rows, rows * 4},
                     {p->bias_token, rows * p->n_bias * 4},
                     {p->bias_value, rows * p->n_bias * 4},
                     {p->allowed, rows * (((size_t)p->V + 31) / 32) * 4}};
  // rows may stand anywhere, so each tensor needs its elements' alignment only
  if (((reinterpret_cast<uintptr_t>(p->logits) | reinterpret_cast<uintptr_t>(p->out)) & (E - 1)) != 0) return CCQ_ERR_MISALIGNED;
  for (size_t i = 2; i < sizeof(r) / sizeof(r[0]); ++i)
    if ((reinterpret_cast<uintptr_t>(r[i].p) & 3u) != 0) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, 11, 1)) return CCQ_ERR_INVALID_ARG;
  return CCQ_OK;
}

int status_of(hipError_t e) { return e == hipSuccess ? CCQ_OK : CCQ_ERR_LAUNCH; }

bool short_of(const void* workspace, size_t bytes, size_t need) {
  return need > 0 && (workspace == nullptr || bytes < need);
}

}  // namespace

extern "C" {

int ccq_qk_norm_rope(const ccq_qk_params* p, void* hip_stream) {
  const int st = validate_qk(p);
  return st != CCQ_OK ? st : status_of(ccq::launch_qk(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_qk_backward_workspace_bytes(const ccq_qk_bwd_params* p) {
  return validate_qk_backward(p) == CCQ_OK ? ccq::qk_backward_workspace_bytes(*p) : 0;
}

int ccq_qk_norm_rope_backward(const ccq_qk_bwd_params* p, void* hip_stream) {
  const int st = validate_qk_backward(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::qk_backward_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_qk_backward(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_scan_workspace_bytes(const ccq_scan_params* p) {
  return validate_scan(p) == CCQ_OK ? ccq::scan_workspace_bytes(*p) : 0;
}

int ccq_scan(const ccq_scan_params* p, void* hip_stream) {
  const int st = validate_scan(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::scan_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_scan(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_scan_backward_workspace_bytes(const ccq_scan_bwd_params* p) {
  return validate_scan_backward(p) == CCQ_OK ? ccq::scan_backward_workspace_bytes(*p) : 0;
}

int ccq_scan_backward(const ccq_scan_bwd_params* p, void* hip_stream) {
  const int st = validate_scan_backward(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::scan_backward_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_scan_backward(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_beam_select_workspace_bytes(const ccq_beam_params* p) {
  return validate_beam(p) == CCQ_OK ? ccq::beam_workspace_bytes(*p) : 0;
}

int ccq_beam_select(const ccq_beam_params* p, void* hip_stream) {
  const int st = validate_beam(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::beam_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_beam_select(*p, static_cast<hipStream_t>(hip_stream)));
}

int ccq_beam_reorder(int32_t n_states, void* const* states, const size_t* row_bytes, int32_t N, int32_t K,
                     const int32_t* parent, void* hip_stream) {
  if (n_states <= 0 || n_states > CCQ_MAX_REORDER_STATES || !states || !row_bytes || N <= 0 || K <= 0 || !parent)
    return CCQ_ERR_INVALID_ARG;
  if (K > ccq::kBeamMaxBeams || (long long)N * K > (1LL << 24)) return CCQ_ERR_UNSUPPORTED;
  Range r[CCQ_MAX_REORDER_STATES + 1];
  for (int i = 0; i < n_states; ++i) {
    if (!states[i] || row_bytes[i] == 0 || row_bytes[i] % 4 != 0) return CCQ_ERR_INVALID_ARG;
    if (row_bytes[i] > ((size_t)1 << 36)) return CCQ_ERR_UNSUPPORTED;
    r[i] = {states[i], row_bytes[i] * (size_t)N * K};
  }
  if (!ccq::beam_reorder_grid_fits(n_states, row_bytes, N, K)) return CCQ_ERR_UNSUPPORTED;
  r[n_states] = {parent, (size_t)N * K * 4};
  for (int i = 0; i <= n_states; ++i)
    if (misaligned(r[i].p)) return CCQ_ERR_MISALIGNED;
  if (written_overlaps(r, n_states + 1, n_states)) return CCQ_ERR_INVALID_ARG;
  return status_of(ccq::launch_beam_reorder(n_states, states, row_bytes, N, K, parent,
                                            static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_linear_attn_workspace_bytes(const ccq_linear_attn_params* p) {
  return validate_la(p) == CCQ_OK ? ccq::linear_attn_workspace_bytes(*p) : 0;
}

int ccq_linear_attn(const ccq_linear_attn_params* p, void* hip_stream) {
  const int st = validate_la(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::linear_attn_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_linear_attn(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_linear_attn_backward_workspace_bytes(const ccq_linear_attn_bwd_params* p) {
  return validate_la_backward(p) == CCQ_OK ? ccq::linear_attn_backward_workspace_bytes(*p) : 0;
}

int ccq_linear_attn_backward(const ccq_linear_attn_bwd_params* p, void* hip_stream) {
  const int st = validate_la_backward(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::linear_attn_backward_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_linear_attn_backward(*p, static_cast<hipStream_t>(hip_stream)));
}

int ccq_group_norm(const ccq_group_norm_params* p, void* hip_stream) {
  const int st = validate_norm(p);
  return st != CCQ_OK ? st : status_of(ccq::launch_group_norm(*p, static_cast<hipStream_t>(hip_stream)));
}

size_t ccq_group_norm_backward_workspace_bytes(const ccq_group_norm_bwd_params* p) {
  return validate_norm_backward(p) == CCQ_OK ? ccq::group_norm_backward_workspace_bytes(*p) : 0;
}

int ccq_group_norm_backward(const ccq_group_norm_bwd_params* p, void* hip_stream) {
  const int st = validate_norm_backward(p);
  if (st != CCQ_OK) return st;
  if (short_of(p->workspace, p->workspace_bytes, ccq::group_norm_backward_workspace_bytes(*p))) return CCQ_ERR_WORKSPACE;
  return status_of(ccq::launch_group_norm_backward(*p, static_cast<hipStream_t>(hip_stream)));
}

int ccq_logits_adjust(const ccq_logits_adjust_params* p, void* hip_stream) {
  const int st = validate_adjust(p);
  return st != CCQ_OK ? st : status_of(ccq::launch_logits_adjust(*p, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
