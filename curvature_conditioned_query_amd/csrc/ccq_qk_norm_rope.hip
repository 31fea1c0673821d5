// Queries and keys of a projection, normalised per head, rotated by their position and laid out
// head-major for the read step; and the gradient.
//
// For a row x of d entries: y = x r w, then entries i < rot turn in pairs by position * inv_freq.
// Everything is a few operations an element, so both directions are bound by memory: a row is read
// once and written once.  A row lies on d / 8 lanes, eight entries (16 bytes of bf16) a lane; 256
// threads hold 256 / (d / 8) tokens, each thread the same eight entries of one token, and walk over
// that token's heads.  The angles depend on token and entry alone, so a thread forms its eight
// cosines and sines once, in registers, for all heads it visits.  Consecutive tokens of a workgroup
// are consecutive rows of the head-major side, consecutive heads are consecutive rows of the
// projection, so both sides move whole cache lines.
#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr float kL2Floor = 1e-12f;

// Eight consecutive entries of a row.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a[e];
    x[4 + e] = b[e];
  }
}
__device__ __forceinline__ void load8(const __bf16* p, float (&x)[8]) {
  const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}
__device__ __forceinline__ void store8(__bf16* p, const float (&x)[8]) {
  bf16x8 a;
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = (__bf16)x[e];
  *reinterpret_cast<bf16x8*>(p) = a;
}

// The rotation of a thread's eight entries: out_e = x_e c_e + partner_e s_e, s_e carrying the sign.
struct Turn {
  float c[8], s[8];
  int partner;  // lane that holds the partners (split halves)
};

// The angle is formed in 64 bits and in turns, reduced to [-1/2, 1/2] there, so a far position loses
// nothing; sine and cosine of the remainder are fp32.
__device__ __forceinline__ void turn_sincos(double position, float inv_freq, float* sn, float* cs) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double t = position * ((double)inv_freq * kInvTwoPi);
  const float r = (float)(t - rint(t));
  sincospif(2.f * r, sn, cs);
}

__device__ __forceinline__ Turn make_turn(const ccq_qk_params& p, int lane, int row_lane, int64_t position) {
  Turn u;
  u.partner = lane;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u.c[e] = 1.f;
    u.s[e] = 0.f;
  }
  const int i0 = 8 * row_lane, half = p.rot / 2;
  if (i0 < p.rot) {
    const double pos = (double)position;
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        turn_sincos(pos, p.inv_freq[(i0 + e) >> 1], &u.s[e + 1], &u.c[e]);
        u.c[e + 1] = u.c[e];
        u.s[e] = -u.s[e + 1];
      }
    } else {
      const bool low = i0 < half;
      u.partner = low ? lane + half / 8 : lane - half / 8;
      const float* f = p.inv_freq + (low ? i0 : i0 - half);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        turn_sincos(pos, f[e], &u.s[e], &u.c[e]);
        if (low) u.s[e] = -u.s[e];
      }
    }
  }
  return u;
}

// x turned by u, or back (the transpose, which is the inverse).  Every lane of a row takes part.
template <bool BACK>
__device__ __forceinline__ void turn(float (&x)[8], const Turn& u, const ccq_qk_params& p) {
  if (p.rot == 0) return;
  float y[8];
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __shfl(x[e], u.partner, 64);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = BACK ? x[e] * u.c[e] - y[e] * u.s[e] : x[e] * u.c[e] + y[e] * u.s[e];
}

// 1 / norm of a row from its sum of squares.
__device__ __forceinline__ float row_scale(float sumsq, int kind, float inv_d, float eps) {
  if (kind == CCQ_NORM_RMS) return 1.f / sqrtf(sumsq * inv_d + eps);
  if (kind == CCQ_NORM_L2) return 1.f / fmaxf(sqrtf(sumsq), kL2Floor);
  return 1.f;
}

// The heads of one workgroup: `per` heads of the queries, or of the keys behind them.
struct HeadRange {
  int begin, end;
  bool keys;
};
__device__ __forceinline__ HeadRange head_range(const ccq_qk_params& p, int part, int per) {
  const int parts_q = (p.H_q + per - 1) / per;
  HeadRange h;
  h.keys = part >= parts_q;
  h.begin = (h.keys ? part - parts_q : part) * per;
  h.end = min(h.begin + per, h.keys ? p.H_k : p.H_q);
  return h;
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void qk_forward_kernel(ccq_qk_params p, int per) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR;
  const int lane = threadIdx.x & 63, rl = threadIdx.x % LPR;
  const int tokens = p.B * p.T;
  const int tok = blockIdx.x * TOK + threadIdx.x / LPR;
  const bool live = tok < tokens;
  const int bt = live ? tok : tokens - 1;
  const int b = bt / p.T, t = bt - b * p.T;
  const HeadRange hr = head_range(p, blockIdx.y, per);
  const int64_t position = p.positions ? p.positions[bt] : p.position0 + t;
  const Turn u = make_turn(p, lane, rl, position);

  const T* in = static_cast<const T*>(hr.keys ? p.k : p.q) + 8 * rl;
  in += hr.keys ? b * p.k_stride_b + t * p.k_stride_t : b * p.q_stride_b + t * p.q_stride_t;
  const int64_t step = hr.keys ? p.k_stride_h : p.q_stride_h;
  const float* w = hr.keys ? p.k_weight : p.q_weight;
  const int kind = hr.keys ? p.k_norm : p.q_norm;
  const int copies = hr.keys && p.expand_keys ? p.H_q / p.H_k : 1;
  const int heads_out = hr.keys ? p.H_k * copies : p.H_q;
  T* out = static_cast<T*>(hr.keys ? p.k_out : p.q_out) + 8 * rl;

  float wt[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wt[e] = 1.f;
  if (w) load8(w + 8 * rl, wt);

  for (int h = hr.begin; h < hr.end; ++h) {
    float x[8];
    load8(in + h * step, x);
    if (kind != CCQ_NORM_NONE) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
      const float r = row_scale(group_sum<LPR>(ss), kind, 1.f / D, p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= wt[e];
    turn<false>(x, u, p);
    if (live) {
      for (int c = 0; c < copies; ++c)
        store8(out + (((int64_t)b * heads_out + h * copies + c) * p.T + t) * D, x);
    }
  }
}

// Gradient.  With z the gradient of the row turned back and summed over the heads that share it,
//   dx = w z r - x r^3 (sum w z x) / (d or 1),  dw = sum of z x r over rows,
// the second term of dx absent without a norm and where an L2 norm is at its floor.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void qk_backward_kernel(ccq_qk_bwd_params q, int per, float* partial) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR;
  const ccq_qk_params& p = q.fwd;
  const int lane = threadIdx.x & 63, rl = threadIdx.x % LPR;
  const int tokens = p.B * p.T;
  const HeadRange hr = head_range(p, blockIdx.y, per);
  const T* in0 = static_cast<const T*>(hr.keys ? p.k : p.q) + 8 * rl;
  const float* g0 = (hr.keys ? q.dk_out : q.dq_out) + 8 * rl;
  T* out0 = static_cast<T*>(hr.keys ? q.dk : q.dq) + 8 * rl;
  const int64_t sb = hr.keys ? p.k_stride_b : p.q_stride_b, st = hr.keys ? p.k_stride_t : p.q_stride_t,
                sh = hr.keys ? p.k_stride_h : p.q_stride_h;
  const int64_t ob = hr.keys ? q.dk_stride_b : q.dq_stride_b, ot = hr.keys ? q.dk_stride_t : q.dq_stride_t,
                oh = hr.keys ? q.dk_stride_h : q.dq_stride_h;
  const float* w = hr.keys ? p.k_weight : p.q_weight;
  const int kind = hr.keys ? p.k_norm : p.q_norm;
  const int copies = hr.keys && p.expand_keys ? p.H_q / p.H_k : 1;
  const int heads_out = hr.keys ? p.H_k * copies : p.H_q;

  float wt[8], dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wt[e] = 1.f;
    dw[e] = 0.f;
  }
  if (w) load8(w + 8 * rl, wt);

  for (int tile = blockIdx.x; tile * TOK < tokens; tile += gridDim.x) {
    const int tok = tile * TOK + threadIdx.x / LPR;
    const bool live = tok < tokens;
    const int bt = live ? tok : tokens - 1;
    const int b = bt / p.T, t = bt - b * p.T;
    const int64_t position = p.positions ? p.positions[bt] : p.position0 + t;
    const Turn u = make_turn(p, lane, rl, position);
    for (int h = hr.begin; h < hr.end; ++h) {
      float x[8], z[8];
      load8(in0 + b * sb + t * st + h * sh, x);
      load8(g0 + (((int64_t)b * heads_out + h * copies) * p.T + t) * D, z);
      for (int c = 1; c < copies; ++c) {
        float more[8];
        load8(g0 + (((int64_t)b * heads_out + h * copies + c) * p.T + t) * D, more);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += more[e];
      }
      turn<true>(z, u, p);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss += x[e] * x[e];
        dot += wt[e] * z[e] * x[e];
      }
      float r = 1.f, pull = 0.f;
      if (kind != CCQ_NORM_NONE) {
        ss = group_sum<LPR>(ss);
        dot = group_sum<LPR>(dot);
        r = row_scale(ss, kind, 1.f / D, p.eps);
        if (kind == CCQ_NORM_RMS) pull = r * r * r * dot * (1.f / D);
        else if (sqrtf(ss) > kL2Floor) pull = r * r * r * dot;
      }
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] += z[e] * x[e] * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = wt[e] * z[e] * r - x[e] * pull;
        store8(out0 + b * ob + t * ot + h * oh, x);
      }
    }
  }
  if (!w) return;
  // the workgroup's part of the weight gradient, summed over its tokens in a fixed order
  __shared__ float red[TOK][D];
#pragma unroll
  for (int e = 0; e < 8; ++e) red[threadIdx.x / LPR][8 * rl + e] = dw[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int i = 0; i < TOK; ++i) s += red[i][threadIdx.x];
    partial[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
  }
}

// dq_weight (blockIdx.y 0) and dk_weight (1): sums of the workgroups' parts, 32 columns a workgroup.
__global__ __launch_bounds__(kThreads) void qk_weight_kernel(const float* partial, int d, int parts_q, int parts_k,
                                                             float* dq_weight, float* dk_weight) {
  const bool keys = blockIdx.y != 0;
  float* out = keys ? dk_weight : dq_weight;
  if (out == nullptr) return;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const float* src = partial + (keys ? (size_t)parts_q * d : 0);
  const int n = keys ? parts_k : parts_q;
  float s = 0.f;
  for (int i = row; i < n; i += kThreads / 32) s += src[(size_t)i * d + col];
  __shared__ float red[kThreads / 32][32];
  red[row][threadIdx.x & 31] = s;
  __syncthreads();
  if (row == 0) {
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) s += red[i][threadIdx.x];
    out[col] = s;
  }
}

// How many heads a workgroup walks over: all of a token's heads share its angles, but the chip wants
// about 2048 workgroups.
int heads_per_group(const ccq_qk_params& p, int tiles) {
  const int most = p.H_q > p.H_k ? p.H_q : p.H_k;
  int per = most;
  while (per > 1 && (long long)tiles * ((p.H_q + per - 1) / per + (p.H_k + per - 1) / per) < 2048) per = (per + 1) / 2;
  return per;
}
int tokens_per_tile(const ccq_qk_params& p) { return kThreads / (p.d / 8); }
int tiles_of(const ccq_qk_params& p) { return (p.B * p.T - 1) / tokens_per_tile(p) + 1; }

struct BackwardGrid {
  int per, x, parts_q, parts_k;
};
BackwardGrid backward_grid(const ccq_qk_params& p) {
  BackwardGrid g;
  const int tiles = tiles_of(p);
  g.per = heads_per_group(p, tiles);
  g.parts_q = (p.H_q + g.per - 1) / g.per;
  g.parts_k = (p.H_k + g.per - 1) / g.per;
  g.x = tiles < 1024 ? tiles : 1024;
  return g;
}

}  // namespace

hipError_t launch_qk(const ccq_qk_params& p, hipStream_t stream) {
  const int tiles = tiles_of(p), per = heads_per_group(p, tiles);
  const dim3 grid(tiles, (p.H_q + per - 1) / per + (p.H_k + per - 1) / per);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.d == 128) qk_forward_kernel<__bf16, 128><<<grid, kThreads, 0, stream>>>(p, per);
    else qk_forward_kernel<__bf16, 64><<<grid, kThreads, 0, stream>>>(p, per);
  } else {
    if (p.d == 128) qk_forward_kernel<float, 128><<<grid, kThreads, 0, stream>>>(p, per);
    else qk_forward_kernel<float, 64><<<grid, kThreads, 0, stream>>>(p, per);
  }
  return hipGetLastError();
}

size_t qk_backward_workspace_bytes(const ccq_qk_bwd_params& q) {
  const ccq_qk_params& p = q.fwd;
  if (!p.q_weight && !p.k_weight) return 0;
  const BackwardGrid g = backward_grid(p);
  return (size_t)g.x * (g.parts_q + g.parts_k) * p.d * 4;
}

hipError_t launch_qk_backward(const ccq_qk_bwd_params& q, hipStream_t stream) {
  const ccq_qk_params& p = q.fwd;
  const BackwardGrid g = backward_grid(p);
  const dim3 grid(g.x, g.parts_q + g.parts_k);
  float* part = static_cast<float*>(q.workspace);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.d == 128) qk_backward_kernel<__bf16, 128><<<grid, kThreads, 0, stream>>>(q, g.per, part);
    else qk_backward_kernel<__bf16, 64><<<grid, kThreads, 0, stream>>>(q, g.per, part);
  } else {
    if (p.d == 128) qk_backward_kernel<float, 128><<<grid, kThreads, 0, stream>>>(q, g.per, part);
    else qk_backward_kernel<float, 64><<<grid, kThreads, 0, stream>>>(q, g.per, part);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.q_weight && !p.k_weight)) return e;
  qk_weight_kernel<<<dim3(p.d / 32, 2), kThreads, 0, stream>>>(part, p.d, g.x * g.parts_q, g.x * g.parts_k, q.dq_weight,
                                                              q.dk_weight);
  return hipGetLastError();
}

}  // namespace ccq
