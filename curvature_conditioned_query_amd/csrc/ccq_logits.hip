// Penalties for tokens seen, biases and grammar masks on logits.
//
// A workgroup owns a stretch of one row's vocabulary.  Its logits, mask and the start of the history are loaded at once;
// the history is counted into a table in LDS (integer atomics: their order changes nothing), the few tokens with a bias
// are formed by one thread each and left in the table, and the logits are then finished in registers and written.
// Bound by memory, and by the chain of loads, counts and stores of a workgroup: 256 rows of 131,071 bf16 logits with up to
// 4096 tokens seen take 41 us, 3.4 TB/s (where this took 42, stretches of 4096 tokens took 44, of 16,384 tokens 44 to 49).
#include <type_traits>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 512;
constexpr int kStretch = 8192;           // tokens of a workgroup: 32 KB of table, four workgroups a CU
constexpr int kMostBias = 1024;
constexpr unsigned kGridX = 1u << 22;   // workgroups along x; a launch has less than 2^32 threads along it
constexpr unsigned kSeen = 0x80000000u;  // a token of the prompt; the counts are below

typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(4)));
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
  float repetition, inverse, presence, frequency;
};

// Branch-free: among 64 lanes' tokens one is nearly always a seen one.  A bf16 logit is divided by a product with the
// inverse, off by 2^-23 where its own rounding is 2^-8.
template <typename T>
__device__ __forceinline__ float penalised(float x, unsigned word, const Penalty& k) {
  const float y = sizeof(T) == 2 ? x * (x > 0.f ? k.inverse : k.repetition) : x > 0.f ? x / k.repetition : x * k.repetition;
  const float c = (float)(word & ~kSeen), z = y - k.frequency * c - k.presence * fminf(c, 1.f);
  return word ? z : x;
}

// x where mask's bit is set, else -inf
template <typename T>
__device__ __forceinline__ typename Any<T>::type allowed_only(typename Any<T>::type x, unsigned mask) {
  if constexpr (sizeof(T) == 2) {
    u32x4 v = __builtin_bit_cast(u32x4, (bf16x8)x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned low = (unsigned)((int)(mask << (31 - 2 * i)) >> 31), high = (unsigned)((int)(mask << (30 - 2 * i)) >> 31);
      const unsigned on = (low & 0xffffu) | (high & 0xffff0000u);
      v[i] = (v[i] & on) | (0xff80ff80u & ~on);
    }
    return __builtin_bit_cast(bf16x8, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!((mask >> e) & 1u)) x[e] = -INFINITY;
    return x;
  }
}

// What a bias needs: tokens of the list inside the stretch, in the list's order, 64 places a block.
struct BiasList {
  float value[kMostBias];
  unsigned short at[kMostBias];
  int kept[kMostBias / 64];
  unsigned char flags[kStretch / 8];  // tokens whose table entry holds the finished logit
};
struct NoBias {};

template <typename T, bool BIAS>
__global__ __launch_bounds__(kThreads) void logits_adjust_kernel(ccq_logits_adjust_params p) {
  constexpr int VE = 16 / (int)sizeof(T), NV = kStretch / (kThreads * VE), kRounds = kMostBias / kThreads;
  typedef typename Any<T>::type V;
  __shared__ __attribute__((aligned(16))) unsigned table[kStretch];
  __shared__ __attribute__((aligned(16))) typename std::conditional<BIAS, BiasList, NoBias>::type list;
  const int stretches = (p.V - 1) / kStretch + 1, group = blockIdx.y * kGridX + blockIdx.x, r = group / stretches, base = (group - r * stretches) * kStretch;
  if (r >= p.R) return;
  const int end = min(p.V, base + kStretch), tid = threadIdx.x, lane = tid & 63;
  const T* src = static_cast<const T*>(p.logits) + (int64_t)r * p.logits_stride;
  T* dst = static_cast<T*>(p.out) + (int64_t)r * p.out_stride;
  const uint32_t* bits = p.allowed ? p.allowed + (int64_t)r * ((p.V + 31) / 32) : nullptr;

  // all that does not hang on something else
  const int32_t* hist = p.history + (int64_t)r * p.L;
  const int h0 = 4 * tid;
  i32x4 seen = {-1, -1, -1, -1};
  if (h0 + 4 <= p.L) seen = *reinterpret_cast<const i32x4_any*>(hist + h0);
  else
    for (int e = 0; e < 4; ++e)
      if (h0 + e < p.L) seen[e] = hist[h0 + e];
  V x[NV];
  unsigned mask[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int v0 = base + (q * kThreads + tid) * VE;
    mask[q] = ~0u;
    if (v0 + VE <= end) x[q] = *reinterpret_cast<const V*>(src + v0);
    else
      for (int e = 0; e < VE; ++e) x[q][e] = src[min(v0 + e, end - 1)];
    if (bits && v0 < end) mask[q] = bits[v0 / 32] >> (v0 % 32);
  }
  Penalty k;
  k.repetition = p.repetition_rows ? p.repetition_rows[r] : p.repetition;
  k.presence = p.presence_rows ? p.presence_rows[r] : p.presence;
  k.frequency = p.frequency_rows ? p.frequency_rows[r] : p.frequency;
  k.inverse = 1.f / k.repetition;
  int n = p.L;
  if (p.lengths) n = max(0, min(p.lengths[r], p.L));
  int prompt = 0;
  if (p.prompt_lengths) prompt = max(0, min(p.prompt_lengths[r], n));
  int place[kRounds], token[kRounds];
  float value[kRounds], own_x[kRounds];
  if constexpr (BIAS) {
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      const int i = tid + q * kThreads;
      token[q] = -1;
      value[q] = own_x[q] = 0.f;
      if (i < p.n_bias) {
        token[q] = p.bias_token[(int64_t)r * p.n_bias + i];
        value[q] = p.bias_value[(int64_t)r * p.n_bias + i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kStretch / (4 * kThreads); ++i) *reinterpret_cast<u32x4*>(&table[4 * (tid + i * kThreads)]) = u32x4{0u, 0u, 0u, 0u};
  if constexpr (BIAS) {
    for (int i = tid; i < (int)sizeof(list.flags) / 4; i += kThreads) reinterpret_cast<unsigned*>(list.flags)[i] = 0u;
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      const bool mine = token[q] >= base && token[q] < end;
      const uint64_t those = __ballot(mine);
      const int block = (tid + q * kThreads) / 64;
      place[q] = -1;
      if (lane == 0) list.kept[block] = __popcll(those);
      if (mine) {
        place[q] = 64 * block + __popcll(those & ((1ull << lane) - 1));
        list.at[place[q]] = (unsigned short)(token[q] - base);
        list.value[place[q]] = value[q];
        own_x[q] = to_f32(src[token[q]]);
      }
    }
  }
  __syncthreads();
  auto count = [&](int i, int v) {
    if (i >= n || v < base || v >= end) return;
    const int at = v - base;
    if (i < prompt) atomicOr(&table[at], kSeen);
    else atomicAdd(&table[at], 1u);
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) count(h0 + e, seen[e]);
  for (int i = h0 + 4 * kThreads; i < n; i += 4 * kThreads) {
    if (i + 4 <= p.L) {
      const i32x4 t = *reinterpret_cast<const i32x4_any*>(hist + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) count(i + e, t[e]);
    } else {
      for (int e = 0; e < 4 && i + e < n; ++e) count(i + e, hist[i + e]);
    }
  }
  __syncthreads();
  if constexpr (BIAS) {
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
      if (place[q] < 0) continue;
      const int at = token[q] - base;
      float sum = 0.f;
      bool owner = true;  // its first place in the list
      for (int b = 0; b <= (p.n_bias - 1) / 64; ++b)
        for (int i = 64 * b; i < 64 * b + list.kept[b]; ++i) {
          const bool same = list.at[i] == at;
          owner = owner && !(same && i < place[q]);
          sum += same ? list.value[i] : 0.f;
        }
      if (!owner) continue;
      table[at] = __builtin_bit_cast(unsigned, penalised<T>(own_x[q], table[at], k) + sum);
      atomicOr(reinterpret_cast<unsigned*>(list.flags) + at / 32, 1u << (at % 32));
    }
    __syncthreads();
  }
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int at = (q * kThreads + tid) * VE, v0 = base + at;
    unsigned word[VE], any = 0;
#pragma unroll
    for (int e = 0; e < VE; e += 4) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(&table[at + e]);
#pragma unroll
      for (int i = 0; i < 4; ++i) any |= word[e + i] = w[i];
    }
    unsigned done = 0;
    if constexpr (BIAS) done = list.flags[at / 8] >> (at % 8) & ((1u << VE) - 1);
    if (any) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float y = penalised<T>(to_f32((T)x[q][e]), word[e], k);
        x[q][e] = from_f32<T>(y);
      }
    }
    if constexpr (BIAS) {
      if (done) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if ((done >> e) & 1u) x[q][e] = from_f32<T>(__builtin_bit_cast(float, word[e]));
      }
    }
    if (bits) x[q] = allowed_only<T>(x[q], mask[q]);
    if (v0 + VE <= end) *reinterpret_cast<V*>(dst + v0) = x[q];
    else
      for (int e = 0; e < VE && v0 + e < end; ++e) dst[v0 + e] = x[q][e];
  }
}

}  // namespace

// The header's limit, which counts stretches half as long as these: a launch could take twice as many.
bool logits_adjust_grid_fits(const ccq_logits_adjust_params& p) {
  return (uint64_t)p.R * (p.V / 4096 + 1) < 1u << 24;
}

hipError_t launch_logits_adjust(const ccq_logits_adjust_params& p, hipStream_t stream) {
  const unsigned groups = (unsigned)p.R * ((p.V - 1) / kStretch + 1);
  const dim3 grid(groups < kGridX ? groups : kGridX, (groups - 1) / kGridX + 1);
  auto run = [&](auto t, auto bias) {
    logits_adjust_kernel<decltype(t), decltype(bias)::value><<<grid, kThreads, 0, stream>>>(p);
  };
  auto typed = [&](auto t) {
    if (p.n_bias) run(t, std::true_type{});
    else run(t, std::false_type{});
  };
  if (p.dtype == CCQ_DTYPE_BF16) typed(__bf16{});
  else typed(float{});
  return hipGetLastError();
}

}  // namespace ccq
