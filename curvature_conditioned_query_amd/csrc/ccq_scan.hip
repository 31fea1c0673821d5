// Gated linear recurrence h_t = alpha_t h_{t-1} + s_t x_t, channel by channel, and its gradient.
#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 64;

__device__ __forceinline__ int sequence_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// 1 - exp(g), exact to rounding also where exp(g) is near 1.
__device__ __forceinline__ float one_minus_exp(float g) { return -expm1f(g); }

// One thread a channel, token by token.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_kernel(ccq_scan_params p) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)p.B * p.D) return;
  const int b = (int)(i / p.D), c = (int)(i - (int64_t)b * p.D);
  const int n = sequence_length(p.lengths, b, p.T), chunks = (p.T + kChunk - 1) / kChunk;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c;
  const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c;
  T* y = static_cast<T*>(p.y) + (int64_t)b * p.T * p.D + c;
  float h = p.h0 ? p.h0[i] : 0.f;
  for (int t = 0; t < n; ++t) {
    if (p.chunk_carry && t % kChunk == 0) p.chunk_carry[((int64_t)b * chunks + t / kChunk) * p.D + c] = h;
    const float gt = to_f32(g[t * p.la_stride_t]), a = expf(gt);
    float xt = to_f32(x[t * p.x_stride_t]);
    if (p.complement) xt *= one_minus_exp(gt);
    h = a == 0.f ? xt : a * h + xt;
    y[(int64_t)t * p.D] = from_f32<T>(h);
  }
  if (p.h_out) p.h_out[i] = h;
}

// One thread a channel, chunk by chunk from the end; a chunk's states are formed again in LDS.
template <typename T>
__global__ __launch_bounds__(64) void scan_backward_kernel(ccq_scan_bwd_params p, const float* carry) {
  __shared__ float before[kChunk][64];
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= (int64_t)p.B * p.D) return;
  const int b = (int)(i / p.D), c = (int)(i - (int64_t)b * p.D);
  const int n = sequence_length(p.lengths, b, p.T), chunks = (p.T + kChunk - 1) / kChunk;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c;
  const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c;
  const T* dy = static_cast<const T*>(p.dy) + b * p.dy_stride_b + c;
  T* dx = static_cast<T*>(p.dx) + (int64_t)b * p.T * p.D + c;
  T* dg = static_cast<T*>(p.dlog_alpha) + (int64_t)b * p.T * p.D + c;
  for (int t = n; t < p.T; ++t) {
    dx[(int64_t)t * p.D] = from_f32<T>(0.f);
    dg[(int64_t)t * p.D] = from_f32<T>(0.f);
  }
  float d = p.dh_out ? p.dh_out[i] : 0.f;  // the part of the adjoint that comes from later tokens
  for (int k = (n + kChunk - 1) / kChunk - 1; k >= 0; --k) {
    const int t0 = k * kChunk, t1 = min(n, t0 + kChunk);
    float h = carry[((int64_t)b * chunks + k) * p.D + c];
    for (int t = t0; t < t1; ++t) {
      before[t - t0][threadIdx.x] = h;
      const float gt = to_f32(g[t * p.la_stride_t]), a = expf(gt);
      float xt = to_f32(x[t * p.x_stride_t]);
      if (p.complement) xt *= one_minus_exp(gt);
      h = a == 0.f ? xt : a * h + xt;
    }
    for (int t = t1 - 1; t >= t0; --t) {
      const float gt = to_f32(g[t * p.la_stride_t]), a = expf(gt);
      d += to_f32(dy[t * p.dy_stride_t]);
      float back = before[t - t0][threadIdx.x], s = 1.f;
      if (p.complement) {
        back -= to_f32(x[t * p.x_stride_t]);
        s = one_minus_exp(gt);
      }
      dx[(int64_t)t * p.D] = from_f32<T>(s * d);
      dg[(int64_t)t * p.D] = from_f32<T>(a == 0.f ? 0.f : a * d * back);
      d = a == 0.f ? 0.f : a * d;
    }
  }
  if (p.dh0) p.dh0[i] = d;
}

// The states before every chunk, where the caller has not kept the forward's.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_carry_kernel(ccq_scan_bwd_params p, float* carry) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)p.B * p.D) return;
  const int b = (int)(i / p.D), c = (int)(i - (int64_t)b * p.D);
  const int n = sequence_length(p.lengths, b, p.T), chunks = (p.T + kChunk - 1) / kChunk;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c;
  const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c;
  float h = p.h0 ? p.h0[i] : 0.f;
  for (int t = 0; t < n; ++t) {
    if (t % kChunk == 0) carry[((int64_t)b * chunks + t / kChunk) * p.D + c] = h;
    const float gt = to_f32(g[t * p.la_stride_t]), a = expf(gt);
    float xt = to_f32(x[t * p.x_stride_t]);
    if (p.complement) xt *= one_minus_exp(gt);
    h = a == 0.f ? xt : a * h + xt;
  }
}

}  // namespace

size_t scan_workspace_bytes(const ccq_scan_params&) { return 0; }

hipError_t launch_scan(const ccq_scan_params& p, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)p.B * p.D + kThreads - 1) / kThreads);
  if (p.dtype == CCQ_DTYPE_BF16) scan_kernel<__bf16><<<grid, kThreads, 0, stream>>>(p);
  else scan_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

size_t scan_backward_workspace_bytes(const ccq_scan_bwd_params& p) {
  return p.chunk_carry ? 0 : (size_t)p.B * ((p.T + kChunk - 1) / kChunk) * p.D * 4;
}

hipError_t launch_scan_backward(const ccq_scan_bwd_params& p, hipStream_t stream) {
  const int64_t channels = (int64_t)p.B * p.D;
  const unsigned all = (unsigned)((channels + kThreads - 1) / kThreads), one = (unsigned)((channels + 63) / 64);
  const float* carry = p.chunk_carry;
  if (!carry) {
    float* ws = static_cast<float*>(p.workspace);
    if (p.dtype == CCQ_DTYPE_BF16) scan_carry_kernel<__bf16><<<all, kThreads, 0, stream>>>(p, ws);
    else scan_carry_kernel<float><<<all, kThreads, 0, stream>>>(p, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    carry = ws;
  }
  if (p.dtype == CCQ_DTYPE_BF16) scan_backward_kernel<__bf16><<<one, 64, 0, stream>>>(p, carry);
  else scan_backward_kernel<float><<<one, 64, 0, stream>>>(p, carry);
  return hipGetLastError();
}

}  // namespace ccq
