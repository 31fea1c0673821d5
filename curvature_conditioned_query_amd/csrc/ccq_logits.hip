// Penalties for tokens seen, biases and grammar masks on logits.
//
// A workgroup owns a stretch of one row's vocabulary.  It counts the row's history into a table in LDS (integer
// atomics: their order changes nothing), then goes over its logits once, 16 bytes a thread at a time.  The few
// tokens with a bias are formed apart, by one thread each, from the logits as they came, and written last.
#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kStretch = 8192;           // tokens of a workgroup: 32 KB of table
constexpr int kBiasRounds = 1024 / kThreads;
constexpr unsigned kSeen = 0x80000000u;  // a token of the prompt; the counts are below

typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <typename T>
struct Any;
template <>
struct Any<__bf16> {
  typedef bf16x8_any type;
};
template <>
struct Any<float> {
  typedef f32x4_any type;
};

struct Penalty {
  float repetition, presence, frequency;
};

__device__ __forceinline__ float penalised(float x, unsigned word, const Penalty& k) {
  if (word == 0) return x;
  x = x > 0.f ? x / k.repetition : x * k.repetition;
  const unsigned c = word & ~kSeen;
  return c ? x - k.frequency * (float)c - k.presence : x;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void logits_adjust_kernel(ccq_logits_adjust_params p) {
  constexpr int VE = 16 / (int)sizeof(T);
  typedef typename Any<T>::type V;
  __shared__ unsigned table[kStretch];
  __shared__ int listed[1024];
  const int stretches = (p.V - 1) / kStretch + 1, r = blockIdx.x / stretches, base = (blockIdx.x - r * stretches) * kStretch, end = min(p.V, base + kStretch), tid = threadIdx.x;
  const T* src = static_cast<const T*>(p.logits) + (int64_t)r * p.logits_stride;
  T* dst = static_cast<T*>(p.out) + (int64_t)r * p.out_stride;
  const uint32_t* bits = p.allowed ? p.allowed + (int64_t)r * ((p.V + 31) / 32) : nullptr;
  Penalty k;
  k.repetition = p.repetition_rows ? p.repetition_rows[r] : p.repetition;
  k.presence = p.presence_rows ? p.presence_rows[r] : p.presence;
  k.frequency = p.frequency_rows ? p.frequency_rows[r] : p.frequency;
  int n = p.L;
  if (p.lengths) n = max(0, min(p.lengths[r], p.L));
  int prompt = 0;
  if (p.prompt_lengths) prompt = max(0, min(p.prompt_lengths[r], n));

  if (n > 0) {
    for (int i = tid; i < kStretch; i += kThreads) table[i] = 0;
    __syncthreads();
    const int32_t* hist = p.history + (int64_t)r * p.L;
    for (int i = tid; i < n; i += kThreads) {
      const int at = hist[i] - base;
      if (at >= 0 && at < end - base) {
        if (i < prompt) atomicOr(&table[at], kSeen);
        else atomicAdd(&table[at], 1u);
      }
    }
  }
  // the owner of a biased token is its first place in the list
  int own[kBiasRounds];
  float own_x[kBiasRounds];
  if (p.n_bias) {
    const int32_t* at = p.bias_token + (int64_t)r * p.n_bias;
    for (int i = tid; i < p.n_bias; i += kThreads) listed[i] = at[i];
  }
  __syncthreads();
  if (p.n_bias) {
    const float* value = p.bias_value + (int64_t)r * p.n_bias;
#pragma unroll
    for (int q = 0; q < kBiasRounds; ++q) {
      own[q] = -1;
      own_x[q] = 0.f;
      const int i = tid + q * kThreads;
      if (i >= p.n_bias) continue;
      const int v = listed[i];
      if (v < base || v >= end) continue;
      bool first = true;
      for (int j = 0; j < i; ++j) first = first && listed[j] != v;
      if (!first) continue;
      float sum = value[i];
      for (int j = i + 1; j < p.n_bias; ++j)
        if (listed[j] == v) sum += value[j];
      own[q] = v;
      own_x[q] = penalised(to_f32(src[v]), n > 0 ? table[v - base] : 0u, k) + sum;
    }
    __syncthreads();
  }
  for (int v0 = base + tid * VE; v0 < end; v0 += kThreads * VE) {
    V x;
    const bool whole = v0 + VE <= end;
    if (whole) x = *reinterpret_cast<const V*>(src + v0);
    else
      for (int e = 0; e < VE; ++e) x[e] = src[min(v0 + e, end - 1)];
    unsigned word[VE];
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < VE; ++e) word[e] = table[v0 - base + e];
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (word[e]) x[e] = from_f32<T>(penalised(to_f32((T)x[e]), word[e], k));
    }
    if (bits) {
      const unsigned m = bits[v0 / 32] >> (v0 % 32);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (!((m >> e) & 1u)) x[e] = from_f32<T>(-INFINITY);
    }
    if (whole) *reinterpret_cast<V*>(dst + v0) = x;
    else
      for (int e = 0; e < VE && v0 + e < end; ++e) dst[v0 + e] = x[e];
  }
  if (p.n_bias) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kBiasRounds; ++q) {
      if (own[q] < 0) continue;
      const bool on = !bits || ((bits[own[q] / 32] >> (own[q] % 32)) & 1u);
      dst[own[q]] = from_f32<T>(on ? own_x[q] : -INFINITY);
    }
  }
}

}  // namespace

bool logits_adjust_grid_fits(const ccq_logits_adjust_params& p) {
  return grid_fits((uint64_t)p.R * (p.V / 4096 + 1), kThreads);
}

hipError_t launch_logits_adjust(const ccq_logits_adjust_params& p, hipStream_t stream) {
  const unsigned grid = (unsigned)p.R * ((p.V - 1) / kStretch + 1);
  if (p.dtype == CCQ_DTYPE_BF16) logits_adjust_kernel<__bf16><<<grid, kThreads, 0, stream>>>(p);
  else logits_adjust_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace ccq
