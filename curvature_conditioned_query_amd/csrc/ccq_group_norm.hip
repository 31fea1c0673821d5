// Group norm of every token by itself, channels last, with an activation or a gate; and the gradient.
//
// z = (x - mu) r w + b over a group's d channels, y = act(z) or z act(gate).  A few operations an element: bound by
// memory, each row read once and written once.  A row lies on LANES lanes, eight channels (16 bytes of bf16) a
// lane, twice that where d > 512.  A thread keeps its group and channels while it walks over tokens, so the weights
// stay in registers and the weights' gradients gather there; consecutive rows of a workgroup are `groups` groups of a
// token and then the next token.
// 16,384 tokens of 16 groups of 128 in bf16, gated: 37 us, 5.5 TB/s (45 with twice the workgroups, whose weights are
// loaded as often, and one row of 256 bytes a workgroup; 46 with two rows of a thread in flight, which fewer waves then
// fit); in fp32 90 us, 4.5 TB/s.  Gradient of 6,141 tokens of 12 groups of 80 in fp32: 23 us with the sum of the weights' gradients;
// of the 16,384 tokens, gated, 68 us in bf16 and 152 in fp32 (5.0 and 4.4 TB/s), a weight for all groups alike.
#include <type_traits>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kSumThreads = 1024, kSumCols = 16, kSumRows = kSumThreads / kSumCols;

// Eight channels as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
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
  u32x4 a;
  __device__ __forceinline__ void load(const __bf16* p) { a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)); }
  __device__ __forceinline__ void zero() { a = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const bf16x8 v = __builtin_bit_cast(bf16x8, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
  }
};
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4*>(p + 4));
}
__device__ __forceinline__ void store8(__bf16* p, const float (&x)[8]) {
  bf16x8 a;
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] = (__bf16)x[e];
  __builtin_nontemporal_store(a, reinterpret_cast<bf16x8*>(p));
}

// right to 2^-23 (1 + |x|); the divide's own sequence costs as much as the rest of an element
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }
__device__ __forceinline__ float act(float x, int kind) {
  if (kind == CCQ_ACT_NONE) return x;
  const float s = sigmoid(x);
  return kind == CCQ_ACT_SILU ? x * s : s;
}
// its value and slope
__device__ __forceinline__ float act_slope(float x, int kind, float& value) {
  if (kind == CCQ_ACT_NONE) {
    value = x;
    return 1.f;
  }
  const float s = sigmoid(x);
  value = kind == CCQ_ACT_SILU ? x * s : s;
  return kind == CCQ_ACT_SILU ? s * (1.f + x * (1.f - s)) : s * (1.f - s);
}

// How a launch's threads share the rows.
struct Shape {
  int groups;        // groups of a workgroup, a power of two
  int tokens;        // tokens of a workgroup at a time
  int64_t all;       // B T
};

// A thread's place: its group, its first channel, and its token among the workgroup's.
template <int LANES, int NU>
struct Place {
  int lane, g, token, units;
  bool live;
  __device__ __forceinline__ Place(const ccq_group_norm_params& p, const Shape& s) {
    lane = threadIdx.x % LANES;
    const int row = threadIdx.x / LANES;
    g = blockIdx.y * s.groups + row % s.groups;
    token = row / s.groups;
    live = g < p.G;
    units = p.d / 8;
  }
  __device__ __forceinline__ bool has(int i) const { return live && lane + LANES * i < units; }
};
// The tokens that a thread walks over, the launch's stride apart.
struct Walk {
  int64_t bt, b, t, all, step, step_b, step_t, T;
  __device__ __forceinline__ Walk(const ccq_group_norm_params& p, const Shape& s, int token) {
    bt = (int64_t)blockIdx.x * s.tokens + token;
    all = s.all;
    step = (int64_t)gridDim.x * s.tokens;
    T = p.T;
    b = (unsigned)bt / (unsigned)p.T;  // B T G < 2^31
    t = bt - b * T;
    step_b = (unsigned)step / (unsigned)p.T;
    step_t = step - step_b * T;
  }
  __device__ __forceinline__ bool on() const { return bt < all; }
  __device__ __forceinline__ void next() {
    bt += step;
    b += step_b;
    t += step_t;
    if (t >= T) {
      t -= T;
      ++b;
    }
  }
};

template <int NU>
__device__ __forceinline__ void load_affine(const float* w, const ccq_group_norm_params& p, int g, int lane, int lanes,
                                            float fill, float (&out)[NU][8]) {
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = lane + lanes * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[i][e] = fill;
    if (w && g < p.G && u < p.d / 8) {
      const float* q = w + (p.affine_shared ? 0 : (size_t)g * p.d) + 8 * u;
      const f32x4 a = *reinterpret_cast<const f32x4*>(q), b = *reinterpret_cast<const f32x4*>(q + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        out[i][e] = a[e];
        out[i][4 + e] = b[e];
      }
    }
  }
}

// n = (x - mu) r in place; returns r.
template <int LANES, int NU>
__device__ __forceinline__ float normalise(float (&x)[NU][8], const Place<LANES, NU>& at, const ccq_group_norm_params& p) {
  const float inv_d = 1.f / (float)p.d;
  if (p.center) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[i][e];
    const float mu = group_sum<LANES>(s) * inv_d;
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = at.has(i) ? x[i][e] - mu : 0.f;
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x[i][e] * x[i][e];
  const float r = 1.f / sqrtf(group_sum<LANES>(ss) * inv_d + p.eps);
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] *= r;
  return r;
}

template <typename T, int LANES, int NU>
__global__ __launch_bounds__(kThreads) void group_norm_kernel(ccq_group_norm_params p, Shape s) {
  const Place<LANES, NU> at(p, s);
  float w[NU][8], bias[NU][8];
  load_affine<NU>(p.weight, p, at.g, at.lane, LANES, 1.f, w);
  load_affine<NU>(p.bias, p, at.g, at.lane, LANES, 0.f, bias);
  Walk at_token(p, s, at.token);
  for (int64_t first = (int64_t)blockIdx.x * s.tokens; first < s.all; first += at_token.step, at_token.next()) {
    const bool on = at_token.on();
    const int64_t b = at_token.b, t = at_token.t;
    Raw8<T> xr[NU], gr[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int c = 8 * (at.lane + LANES * i);
      xr[i].zero();
      gr[i].zero();
      if (on && at.has(i)) {
        xr[i].load(static_cast<const T*>(p.x) + b * p.x_stride_b + t * p.x_stride_t + at.g * p.x_stride_h + c);
        if (p.gate) gr[i].load(static_cast<const T*>(p.gate) + b * p.gate_stride_b + t * p.gate_stride_t + at.g * p.gate_stride_h + c);
      }
    }
    float x[NU][8];
#pragma unroll
    for (int i = 0; i < NU; ++i) xr[i].get(x[i]);
    normalise<LANES, NU>(x, at, p);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float g[8];
      gr[i].get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = x[i][e] * w[i][e] + bias[i][e];
        x[i][e] = p.gate ? z * act(g[e], p.activation) : act(z, p.activation);
      }
      if (on && at.has(i))
        store8(static_cast<T*>(p.y) + b * p.y_stride_b + t * p.y_stride_t + at.g * p.y_stride_h + 8 * (at.lane + LANES * i), x[i]);
    }
  }
}

// Gradient.  With dz = dy act'(z), or dy act(gate): dn = dz w, dx = r (dn - [center] mean(dn) - n mean(dn n)),
// dgate = dy z act'(gate), dw = sum of dz n, db = sum of dz.
template <typename T, int LANES, int NU>
__global__ __launch_bounds__(kThreads) void group_norm_backward_kernel(ccq_group_norm_bwd_params q, Shape s, float* part_w, float* part_b) {
  const ccq_group_norm_params& p = q.fwd;
  const Place<LANES, NU> at(p, s);
  float w[NU][8], bias[NU][8], dw[NU][8], db[NU][8];
  load_affine<NU>(p.weight, p, at.g, at.lane, LANES, 1.f, w);
  load_affine<NU>(p.bias, p, at.g, at.lane, LANES, 0.f, bias);
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = db[i][e] = 0.f;
  const float inv_d = 1.f / (float)p.d;
  Walk at_token(p, s, at.token);
  for (int64_t first = (int64_t)blockIdx.x * s.tokens; first < s.all; first += at_token.step, at_token.next()) {
    const bool on = at_token.on();
    const int64_t b = at_token.b, t = at_token.t;
    Raw8<T> xr[NU], yr[NU], gr[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int c = 8 * (at.lane + LANES * i);
      xr[i].zero();
      yr[i].zero();
      gr[i].zero();
      if (on && at.has(i)) {
        xr[i].load(static_cast<const T*>(p.x) + b * p.x_stride_b + t * p.x_stride_t + at.g * p.x_stride_h + c);
        yr[i].load(static_cast<const T*>(q.dy) + b * q.dy_stride_b + t * q.dy_stride_t + at.g * q.dy_stride_h + c);
        if (p.gate) gr[i].load(static_cast<const T*>(p.gate) + b * p.gate_stride_b + t * p.gate_stride_t + at.g * p.gate_stride_h + c);
      }
    }
    float n[NU][8], dn[NU][8];
#pragma unroll
    for (int i = 0; i < NU; ++i) xr[i].get(n[i]);
    const float r = normalise<LANES, NU>(n, at, p);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float dy[8], g[8];
      yr[i].get(dy);
      gr[i].get(g);
      const bool mine = on && at.has(i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = n[i][e] * w[i][e] + bias[i][e];
        float value, dz;
        if (p.gate) {
          const float slope = act_slope(g[e], p.activation, value);
          dz = dy[e] * value;
          g[e] = dy[e] * z * slope;
        } else {
          dz = dy[e] * act_slope(z, p.activation, value);
        }
        if (mine) {
          dw[i][e] += dz * n[i][e];
          db[i][e] += dz;
        }
        dn[i][e] = mine ? dz * w[i][e] : 0.f;
        s1 += dn[i][e];
        s2 += dn[i][e] * n[i][e];
      }
      if (p.gate && mine)
        store8(static_cast<T*>(q.dgate) + b * q.dgate_stride_b + t * q.dgate_stride_t + at.g * q.dgate_stride_h + 8 * (at.lane + LANES * i), g);
    }
    s1 = p.center ? group_sum<LANES>(s1) * inv_d : 0.f;
    s2 = group_sum<LANES>(s2) * inv_d;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) dn[i][e] = r * (dn[i][e] - s1 - n[i][e] * s2);
      if (on && at.has(i))
        store8(static_cast<T*>(q.dx) + b * q.dx_stride_b + t * q.dx_stride_t + at.g * q.dx_stride_h + 8 * (at.lane + LANES * i), dn[i]);
    }
  }
  // the workgroup's part of the weights' gradients, summed over its tokens in a fixed order
  __shared__ float red[kThreads / LANES][LANES * NU * 8];
  const int row = threadIdx.x / LANES;
  for (int k = 0; k < 2; ++k) {
    float* part = k ? part_b : part_w;
    if (!part) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) red[row][8 * (at.lane + LANES * i) + e] = k ? db[i][e] : dw[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < s.groups * p.d; c += kThreads) {
      const int gl = c / p.d, ch = c - gl * p.d, g = blockIdx.y * s.groups + gl;
      float sum = 0.f;
      for (int i = gl; i < kThreads / LANES; i += s.groups) sum += red[i][ch];
      if (g < p.G) part[((size_t)blockIdx.x * p.G + g) * p.d + ch] = sum;
    }
  }
}

// out[c] = sum over the parts' rows of part[row][c], 16 columns a workgroup, 64 rows at a time.
__global__ __launch_bounds__(kSumThreads) void group_norm_sum_kernel(const float* part_w, const float* part_b, int cols, int64_t rows,
                                                                     float* dweight, float* dbias) {
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, c = blockIdx.x * kSumCols + col;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t i = row; i < rows; i += kSumRows) s += part[(size_t)i * cols + c];
  }
  __shared__ float red[kSumRows][kSumCols];
  red[row][col] = s;
  __syncthreads();
  if (row == 0 && c < cols) {
    for (int i = 1; i < kSumRows; ++i) s += red[i][col];
    out[c] = s;
  }
}

int lanes_of(int d) {
  const int units = d / 8;
  int n = 4;
  while (n < units && n < 64) n *= 2;
  return n;
}

// `most`: workgroups that a launch shall have.
Shape shape_of(const ccq_group_norm_params& p, int most, dim3* grid) {
  Shape s;
  const int rows = kThreads / lanes_of(p.d), bytes = p.d * (p.dtype == CCQ_DTYPE_BF16 ? 2 : 4);
  s.groups = 1;  // whole cache lines, four of them, where the rows allow it (one row of 320 bytes: 26 against 25 us)
  while (s.groups < rows && s.groups < p.G && (s.groups * bytes < 512 || s.groups * bytes % 128)) s.groups *= 2;
  s.tokens = rows / s.groups;
  s.all = (int64_t)p.B * p.T;
  const int64_t gy = (p.G + s.groups - 1) / s.groups, tiles = (s.all - 1) / s.tokens + 1;
  int64_t gx = most / gy < 1 ? 1 : most / gy;
  if (gx > tiles) gx = tiles;
  *grid = dim3((unsigned)gx, (unsigned)gy);
  return s;
}
constexpr int kForwardGroups = 2048, kBackwardGroups = 1024;

template <typename F>
void by_lanes(int d, F f) {
  const int n = lanes_of(d);
  if (d > 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (n == 64) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (n == 32) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  else if (n == 16) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (n == 8) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
}

size_t part_floats(const ccq_group_norm_params& p) {
  dim3 grid;
  shape_of(p, kBackwardGroups, &grid);
  return (size_t)grid.x * p.G * p.d;
}

}  // namespace

hipError_t launch_group_norm(const ccq_group_norm_params& p, hipStream_t stream) {
  dim3 grid;
  const Shape s = shape_of(p, kForwardGroups, &grid);
  by_lanes(p.d, [&](auto lanes, auto nu) {
    if (p.dtype == CCQ_DTYPE_BF16) group_norm_kernel<__bf16, decltype(lanes)::value, decltype(nu)::value><<<grid, kThreads, 0, stream>>>(p, s);
    else group_norm_kernel<float, decltype(lanes)::value, decltype(nu)::value><<<grid, kThreads, 0, stream>>>(p, s);
  });
  return hipGetLastError();
}

size_t group_norm_backward_workspace_bytes(const ccq_group_norm_bwd_params& q) {
  return ((q.dweight != nullptr) + (q.dbias != nullptr)) * part_floats(q.fwd) * 4;
}

hipError_t launch_group_norm_backward(const ccq_group_norm_bwd_params& q, hipStream_t stream) {
  const ccq_group_norm_params& p = q.fwd;
  dim3 grid;
  const Shape s = shape_of(p, kBackwardGroups, &grid);
  float* part_w = q.dweight ? static_cast<float*>(q.workspace) : nullptr;
  float* part_b = q.dbias ? static_cast<float*>(q.workspace) + (q.dweight ? part_floats(p) : 0) : nullptr;
  by_lanes(p.d, [&](auto lanes, auto nu) {
    constexpr int L = decltype(lanes)::value, N = decltype(nu)::value;
    if (p.dtype == CCQ_DTYPE_BF16) group_norm_backward_kernel<__bf16, L, N><<<grid, kThreads, 0, stream>>>(q, s, part_w, part_b);
    else group_norm_backward_kernel<float, L, N><<<grid, kThreads, 0, stream>>>(q, s, part_w, part_b);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!part_w && !part_b)) return e;
  const int cols = p.affine_shared ? p.d : p.G * p.d;
  const int64_t rows = (int64_t)grid.x * (p.affine_shared ? p.G : 1);
  group_norm_sum_kernel<<<dim3((cols + kSumCols - 1) / kSumCols, 2), kSumThreads, 0, stream>>>(part_w, part_b, cols, rows, q.dweight, q.dbias);
  return hipGetLastError();
}

}  // namespace ccq
