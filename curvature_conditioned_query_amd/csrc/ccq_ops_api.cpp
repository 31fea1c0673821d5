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

}  // extern "C"
