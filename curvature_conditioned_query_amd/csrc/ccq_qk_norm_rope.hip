// Queries and keys of a projection, normalised per head, rotated by their position and laid out
// head-major for the read step; and the gradient.
//
// For a row x of d entries: y = x r w, then entries i < rot turn in pairs by position * inv_freq.
// Everything is a few operations an element, so both directions are bound by memory: a row is read
// once and written once.  A row lies on d / 8 lanes, eight entries (16 bytes of bf16) a lane; 256
// threads hold 256 / (d / 8) tokens, each thread the same eight entries of one token, and walk over
// that token's heads, queries and then keys, several rows' loads under way: as many as there are heads left,
// not more (loading the last head again in their place: 50 against 40 us for fp32 rows of 4 + 2 heads).  The
// angles depend on token and entry alone: a workgroup forms each cosine and sine once, in LDS, and a thread
// takes its eight into registers for all heads it visits (formed by every thread for itself and for queries
// and keys apart they were about 5 of 56 us of the prefill).  Consecutive tokens of a workgroup are consecutive rows of
// the head-major side, consecutive heads are consecutive rows of the projection, so both sides move
// whole cache lines.
//
// Measured: B4 T4096 16 + 16 heads of 128, bf16: 51 us for the 268 MB it reads and writes, 5.3 TB/s, against
// 6.0 of a plain stream past the caches; the gradient (16 + 4 heads, expanded; 436 MB with the fp32 gradients
// it reads) 91 us and the sum of the weights' parts 4.6, 4.6 TB/s over both.  A decode step's 64 tokens take
// 4.2 us, the launch's and one load's latency.
#include <type_traits>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
// Rows a thread loads at a time: 128 bytes (fp32, 4 + 2 heads of 128, 23,361 tokens: 37.5 us; eight rows 40).
template <typename T>
constexpr int kAhead = 16 / (int)sizeof(T);
constexpr int kBackAhead = 4;  // and of the gradient, whose rows are three times as wide
constexpr float kL2Floor = 1e-12f;

// Rows are read past the caches, being read once.  The gradient, whose rows leave as they came, is also
// written past them (101 against 108 us at B4 T4096, with twice the workgroups it has now); the forward, whose
// rows part by head, is not: its caches gather the rows of a head (53 against 59 us).
// Eight entries as they are stored, so that several rows' loads are under way at a time.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = a[e];
      x[4 + e] = b[e];
    }
  }
};
template <>
struct Raw8<__bf16> {
  bf16x8 a;
  __device__ __forceinline__ void load(const __bf16* p) { a = __builtin_nontemporal_load(reinterpret_cast<const bf16x8*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
  }
};

// STREAM: past the caches.
template <bool STREAM, typename V>
__device__ __forceinline__ void store_vec(V v, V* p) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool STREAM>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  store_vec<STREAM>(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p));
  store_vec<STREAM>(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4*>(p + 4));
}
template <bool STREAM>
__device__ __forceinline__ void store8(__bf16* p, const float (&x)[8]) {
  bf16x8 a;
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = (__bf16)x[e];
  store_vec<STREAM>(a, reinterpret_cast<bf16x8*>(p));
}

// The rotation of a thread's eight entries: out_e = x_e c_e + partner_e s_e, s_e carrying the sign.
struct Turn {
  float c[8], s[8];
  int partner;  // lane that holds the partners (split halves)
  bool on;      // whether the entries are rotated at all
};

// The angle is formed in 64 bits and in turns, reduced to [-1/2, 1/2] there, so a far position loses
// nothing; sine and cosine of the remainder are fp32.
__device__ __forceinline__ float2 turn_sincos(double position, float inv_freq) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double t = position * ((double)inv_freq * kInvTwoPi);
  float2 r;
  sincospif(2.f * (float)(t - rint(t)), &r.y, &r.x);
  return r;
}

// Cosine (x) and sine (y) of every pair of the workgroup's tokens.
template <int D>
struct Angles {
  static constexpr int TOK = kThreads / (D / 8), PAIRS = D / 2;
  float2 a[TOK][PAIRS];

  // All threads; tokens from `first` on, those past the last as the last.
  __device__ __forceinline__ void form(const ccq_qk_params& p, int first, int tokens) {
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < TOK * PAIRS; i += kThreads) {
      const int tok = i / PAIRS, k = i % PAIRS;
      if (k < pairs) {
        const int bt = min(first + tok, tokens - 1);
        const int64_t position = p.positions ? p.positions[bt] : p.position0 + bt % p.T;
        a[tok][k] = turn_sincos((double)position, p.inv_freq[k]);
      }
    }
  }
  __device__ __forceinline__ Turn take(const ccq_qk_params& p, int tok, int row_lane, int lane) const {
    Turn u;
    u.partner = lane;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u.c[e] = 1.f;
      u.s[e] = 0.f;
    }
    const int i0 = 8 * row_lane, half = p.rot / 2;
    u.on = i0 < p.rot;
    if (u.on) {
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 v = a[tok][(i0 + e) >> 1];
          u.c[e] = u.c[e + 1] = v.x;
          u.s[e] = -v.y;
          u.s[e + 1] = v.y;
        }
      } else {
        const bool low = i0 < half;
        u.partner = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = a[tok][(low ? i0 : i0 - half) + e];
          u.c[e] = v.x;
          u.s[e] = low ? -v.y : v.y;
        }
      }
    }
    return u;
  }
};

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
  // an entry behind the rotated part is not multiplied by 1 and its neighbour by 0: infinities would make NaN
  if (u.on) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = BACK ? x[e] * u.c[e] - y[e] * u.s[e] : x[e] * u.c[e] + y[e] * u.s[e];
  }
}

// 1 / norm of a row from its sum of squares.
__device__ __forceinline__ float row_scale(float sumsq, int kind, float inv_d, float eps) {
  if (kind == CCQ_NORM_RMS) return 1.f / sqrtf(sumsq * inv_d + eps);
  if (kind == CCQ_NORM_L2) {
    const float n = sqrtf(sumsq);
    return 1.f / (n < kL2Floor ? kL2Floor : n);  // NaN stays
  }
  return 1.f;
}

// One side of a call: queries or keys.
struct Side {
  const void* in;
  int64_t sb, st, sh;
  const float* w;
  void* out;
  int norm, copies, heads_out;
};
__device__ __forceinline__ Side side_of(const ccq_qk_params& p, bool keys) {
  Side s;
  s.in = keys ? p.k : p.q;
  s.sb = keys ? p.k_stride_b : p.q_stride_b;
  s.st = keys ? p.k_stride_t : p.q_stride_t;
  s.sh = keys ? p.k_stride_h : p.q_stride_h;
  s.w = keys ? p.k_weight : p.q_weight;
  s.out = keys ? p.k_out : p.q_out;
  s.norm = keys ? p.k_norm : p.q_norm;
  s.copies = keys && p.expand_keys ? p.H_q / p.H_k : 1;
  s.heads_out = keys ? p.H_k * s.copies : p.H_q;
  return s;
}
__device__ __forceinline__ void load_weight(const float* w, int row_lane, float (&wt)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) wt[e] = 1.f;
  if (w) {
    Raw8<float> raw;
    raw.load(w + 8 * row_lane);
    raw.get(wt);
  }
}

// A workgroup's heads: `per` of the queries' and keys' together, from blockIdx.y per on.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void qk_forward_kernel(ccq_qk_params p, int per) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR;
  __shared__ Angles<D> angles;
  const int lane = threadIdx.x & 63, rl = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int tokens = p.B * p.T, first = blockIdx.x * TOK;
  const bool live = first + row < tokens;
  const int bt = live ? first + row : tokens - 1;
  const int b = bt / p.T, t = bt - b * p.T;
  if (p.rot) angles.form(p, first, tokens);
  __syncthreads();
  const Turn u = angles.take(p, row, rl, lane);

  const int from = blockIdx.y * per, to = min(from + per, p.H_q + p.H_k);
  for (int side = 0; side < 2; ++side) {
    const int begin = side ? max(from - p.H_q, 0) : from, end = side ? to - p.H_q : min(to, p.H_q);
    if (begin >= end) continue;
    const Side s = side_of(p, side != 0);
    const T* in = static_cast<const T*>(s.in) + b * s.sb + t * s.st + 8 * rl;
    T* out = static_cast<T*>(s.out) + (((int64_t)b * s.heads_out) * p.T + t) * D + 8 * rl;
    const int64_t out_step = (int64_t)p.T * D;
    float wt[8];
    load_weight(s.w, rl, wt);
    // rows h0 .. h0 + n - 1, all loads under way
    auto rows = [&](auto n, int h0) {
      constexpr int N = decltype(n)::value;
      Raw8<T> raw[N];
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i].load(in + (h0 + i) * s.sh);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int h = h0 + i;
        float x[8];
        raw[i].get(x);
        if (s.norm != CCQ_NORM_NONE) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
          const float r = row_scale(group_sum<LPR>(ss), s.norm, 1.f / D, p.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= r;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= wt[e];
        turn<false>(x, u, p);
        if (live) {
          for (int c = 0; c < s.copies; ++c) store8<false>(out + (h * s.copies + c) * out_step, x);
        }
      }
      return h0 + N;
    };
    int h = begin;
    while (h + kAhead<T> <= end) h = rows(std::integral_constant<int, kAhead<T>>{}, h);
    if (sizeof(T) == 2 && h + 4 <= end) h = rows(std::integral_constant<int, 4>{}, h);
    if (h + 2 <= end) h = rows(std::integral_constant<int, 2>{}, h);
    if (h < end) rows(std::integral_constant<int, 1>{}, h);
  }
}

// Gradient.  With z the gradient of the row turned back and summed over the heads that share it,
//   dx = w z r - x r^3 (sum w z x) / (d or 1),  dw = sum of z x r over rows,
// the second term of dx absent without a norm and where an L2 norm is at its floor.  The weights'
// gradients gather in registers over a workgroup's rows; workgroups go on from tile to tile, so that
// few parts are left to be summed.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void qk_backward_kernel(ccq_qk_bwd_params q, int per, float* partial) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR;
  __shared__ union {
    Angles<D> angles;
    float red[TOK][D];
  } lds;
  const ccq_qk_params& p = q.fwd;
  const int lane = threadIdx.x & 63, rl = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int tokens = p.B * p.T;
  const int from = blockIdx.y * per, to = min(from + per, p.H_q + p.H_k);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;

  for (int first = blockIdx.x * TOK; first < tokens; first += gridDim.x * TOK) {
    const bool live = first + row < tokens;
    const int bt = live ? first + row : tokens - 1;
    const int b = bt / p.T, t = bt - b * p.T;
    __syncthreads();
    if (p.rot) lds.angles.form(p, first, tokens);
    __syncthreads();
    const Turn u = lds.angles.take(p, row, rl, lane);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int begin = side ? max(from - p.H_q, 0) : from, end = side ? to - p.H_q : min(to, p.H_q);
      if (begin >= end) continue;
      const Side s = side_of(p, side != 0);
      const T* in = static_cast<const T*>(s.in) + b * s.sb + t * s.st + 8 * rl;
      const float* grad = (side ? q.dk_out : q.dq_out) + (((int64_t)b * s.heads_out) * p.T + t) * D + 8 * rl;
      const int64_t grad_step = (int64_t)p.T * D;
      T* out = static_cast<T*>(side ? q.dk : q.dq) + b * (side ? q.dk_stride_b : q.dq_stride_b) +
               t * (side ? q.dk_stride_t : q.dq_stride_t) + 8 * rl;
      const int64_t oh = side ? q.dk_stride_h : q.dq_stride_h;
      float wt[8];
      load_weight(s.w, rl, wt);
      auto gradient = [&](const Raw8<T>& x_raw, float (&z)[8], int h) {
        float x[8];
        x_raw.get(x);
        turn<true>(z, u, p);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss += x[e] * x[e];
          dot += wt[e] * z[e] * x[e];
        }
        float r = 1.f, pull = 0.f;
        if (s.norm != CCQ_NORM_NONE) {
          ss = group_sum<LPR>(ss);
          dot = group_sum<LPR>(dot);
          r = row_scale(ss, s.norm, 1.f / D, p.eps);
          if (s.norm == CCQ_NORM_RMS) pull = r * r * r * dot * (1.f / D);
          else if (sqrtf(ss) > kL2Floor) pull = r * r * r * dot;
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dw[side][e] += z[e] * x[e] * r;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = wt[e] * z[e] * r - (s.norm != CCQ_NORM_NONE ? x[e] * pull : 0.f);
          store8<true>(out + h * oh, x);
        }
      };
      if (s.copies == 1) {
        auto rows = [&](auto n, int h0) {
          constexpr int N = decltype(n)::value;
          Raw8<T> x_raw[N];
          Raw8<float> z_raw[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x_raw[i].load(in + (h0 + i) * s.sh);
            z_raw[i].load(grad + (h0 + i) * grad_step);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float z[8];
            z_raw[i].get(z);
            gradient(x_raw[i], z, h0 + i);
          }
          return h0 + N;
        };
        int h = begin;
        while (h + kBackAhead <= end) h = rows(std::integral_constant<int, kBackAhead>{}, h);
        if (h + 2 <= end) h = rows(std::integral_constant<int, 2>{}, h);
        if (h < end) rows(std::integral_constant<int, 1>{}, h);
      } else {
        for (int h = begin; h < end; ++h) {
          Raw8<T> x_raw;
          x_raw.load(in + h * s.sh);
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = 0.f;
          for (int c0 = 0; c0 < s.copies; c0 += kBackAhead) {
            Raw8<float> z_raw[kBackAhead];
#pragma unroll
            for (int i = 0; i < kBackAhead; ++i) z_raw[i].load(grad + (h * s.copies + min(c0 + i, s.copies - 1)) * grad_step);
#pragma unroll
            for (int i = 0; i < kBackAhead; ++i) {
              if (c0 + i >= s.copies) break;
              float more[8];
              z_raw[i].get(more);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] += more[e];
            }
          }
          gradient(x_raw, z, h);
        }
      }
    }
  }
  // the workgroup's part of the weight gradients, summed over its tokens in a fixed order
  const int parts = gridDim.x * gridDim.y, part = blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (!(side ? p.k_weight : p.q_weight)) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) lds.red[row][8 * rl + e] = dw[side][e];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
      for (int i = 0; i < TOK; ++i) s += lds.red[i][threadIdx.x];
      partial[((size_t)side * parts + part) * D + threadIdx.x] = s;
    }
  }
}

// dq_weight (blockIdx.y 0) and dk_weight (1): sums of the workgroups' parts, 16 columns a workgroup, 64
// rows at a time, so that a thread adds few parts, in a fixed order, with their loads under way together.
constexpr int kWeightThreads = 1024, kWeightCols = 16, kWeightRows = kWeightThreads / kWeightCols;
__global__ __launch_bounds__(kWeightThreads) void qk_weight_kernel(const float* partial, int d, int parts, float* dq_weight,
                                                                   float* dk_weight) {
  const bool keys = blockIdx.y != 0;
  float* out = keys ? dk_weight : dq_weight;
  if (out == nullptr) return;
  const int col = threadIdx.x % kWeightCols, row = threadIdx.x / kWeightCols;
  const float* src = partial + (keys ? (size_t)parts * d : 0) + blockIdx.x * kWeightCols + col;
  float s = 0.f;
#pragma unroll 8
  for (int i = row; i < parts; i += kWeightRows) s += src[(size_t)i * d];
  __shared__ float red[kWeightRows][kWeightCols];
  red[row][col] = s;
  __syncthreads();
  if (row == 0) {
    for (int i = 1; i < kWeightRows; ++i) s += red[i][col];
    out[blockIdx.x * kWeightCols + col] = s;
  }
}

int tokens_per_tile(const ccq_qk_params& p) { return kThreads / (p.d / 8); }
int tiles_of(const ccq_qk_params& p) { return (p.B * p.T - 1) / tokens_per_tile(p) + 1; }

// Heads that a workgroup walks over: all, sharing the angles, where that leaves 1024 workgroups, four for
// each CU; else fewer.
int heads_per_group(const ccq_qk_params& p, int tiles) {
  const int all = p.H_q + p.H_k;
  int per = all;
  while (per > 1 && (long long)tiles * ((all + per - 1) / per) < 1024) per = (per + 1) / 2;
  return per;
}

dim3 grid_of(const ccq_qk_params& p, int per, int most) {
  const int tiles = tiles_of(p);
  return dim3(tiles < most ? tiles : most, (p.H_q + p.H_k + per - 1) / per);
}
// The gradient's workgroups along the tokens: two for each CU, going on from tile to tile (92 us at the
// prefill's size; with 1024, of which 768 run at a time, 101).
constexpr int kBackGroups = 512;

}  // namespace

bool qk_grid_fits(const ccq_qk_params& p) { return grid_fits(tiles_of(p), kThreads); }

hipError_t launch_qk(const ccq_qk_params& p, hipStream_t stream) {
  const int per = heads_per_group(p, tiles_of(p));
  const dim3 grid = grid_of(p, per, 0x7fffffff);
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
  const dim3 grid = grid_of(p, heads_per_group(p, tiles_of(p)), kBackGroups);
  return (size_t)grid.x * grid.y * 2 * p.d * 4;
}

hipError_t launch_qk_backward(const ccq_qk_bwd_params& q, hipStream_t stream) {
  const ccq_qk_params& p = q.fwd;
  const int per = heads_per_group(p, tiles_of(p));
  const dim3 grid = grid_of(p, per, kBackGroups);
  float* part = static_cast<float*>(q.workspace);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.d == 128) qk_backward_kernel<__bf16, 128><<<grid, kThreads, 0, stream>>>(q, per, part);
    else qk_backward_kernel<__bf16, 64><<<grid, kThreads, 0, stream>>>(q, per, part);
  } else {
    if (p.d == 128) qk_backward_kernel<float, 128><<<grid, kThreads, 0, stream>>>(q, per, part);
    else qk_backward_kernel<float, 64><<<grid, kThreads, 0, stream>>>(q, per, part);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.q_weight && !p.k_weight)) return e;
  qk_weight_kernel<<<dim3(p.d / kWeightCols, 2), kWeightThreads, 0, stream>>>(part, p.d, (int)(grid.x * grid.y),
                                                                             q.dq_weight, q.dk_weight);
  return hipGetLastError();
}

}  // namespace ccq
