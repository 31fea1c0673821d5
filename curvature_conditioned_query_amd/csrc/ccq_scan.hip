// Gated linear recurrence h_t = alpha_t h_{t-1} + s_t x_t, channel by channel, and its gradient.
//
// A few operations an element: memory is the bound, so every input is read once.  A run of tokens acts
// on the state as h -> P h + q (P the product of its gates, q what the run adds), and runs compose:
// (P1, q1) then (P2, q2) is (P1 P2, P2 q1 + q2).  A workgroup takes a tile of 128 tokens by 128 channels
// into registers (a thread: four tokens of eight channels, one 16-byte load each in bf16), folds its
// tokens, joins the threads' pairs in LDS, and publishes the tile's pair; the state before the tile is
// the fold of the pairs of the tiles before it, and the tile's tokens are then walked again, from
// registers, to their outputs.  So a sequence is spread over as many workgroups as it has tiles and
// still read once: about 1/2 of the traffic of a pass that sums up the pieces before the pass that
// writes them would be spent on reading twice.
//
// A row of a tile is 256 bytes (bf16): read two, write one of that shape reaches 5.3 TB/s, where rows of
// 128 bytes reach 4.8; past the caches (non-temporal), which a single use has no use for, 6.0 and 5.4.
//
// Measured.  B4 T4096 D2048 bf16: 49 us for 201 MB, 4.1 TB/s (43 without the waiting, and 2 for the clearing of
// the pairs), 55 with the complement, whose 1 - alpha is formed for the fold and again for the walk; the gradient
// of a padded batch of that size with the complement, lengths 1/2 to 1, 70 us for 287 MB, 4.1 TB/s (63 without the
// waiting; 79 with the rows behind the sequences read, too): two workgroups fit a CU and the vector units are busy
// for half of it, so loads and arithmetic overlap in part only.  B1 T20480 D1024 fp32: 70 us for 251 MB, 3.6 TB/s
// (54 to 60 without the waiting): eight columns of 160 tiles one behind the other, 1,280 tiles on 512 places, so
// the third round is half empty.  Farther from their floor: the fp32 gradient, whose runs are two tokens and its
// tiles 64 (B1 T6798 D1464: 71 us for 200 MB), and lengths a little above a multiple of 128 (the gradient of B93
// T262 D1264: 105 us for 312 MB, its third tile holding 6 tokens).  Not kept: workgroups that stay and load their
// next tile ahead (98 us against 59: fewer share a CU, and the waiting shows); 64-token tiles (56; of 256 threads
// 53, with the fp32 sequence at 68 and the gradient at 80 against 79); seven or eight waves a SIMD (53 and 63:
// spills); groups of 8 or 32 tiles.
//
// Waiting.  A tile's pair depends on its own inputs alone and is published before its workgroup waits
// for any other, and each column's tiles are handed out by a counter in the order of the recurrence, so
// whatever a workgroup waits for is already being worked on by one that waits for nothing first.  The folds go
// in a fixed order (16 tiles make a group, whose last tile publishes the group's pair), so two
// calls give the same bits.  A wait gives up after about a second and leaves NaN: only a workspace
// that another call is writing can bring that about.
//
// A gate of 0 drops the state before it, even an infinite one or NaN.  A run that holds such a gate has
// P = -0: the sign tells it from a product that has only become too small, which still passes an
// infinity or NaN on.
#include <float.h>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 512;      // of a tile
constexpr int kStepThreads = 256;  // of the kernels without tiles
constexpr int kChunk = 64;         // tokens between kept states
constexpr int kCols = 128;         // channels of a tile
constexpr int kOct = kCols / 8;    // threads side by side: eight channels each
constexpr int kRuns = kThreads / kOct;  // runs of a tile, one behind the other
constexpr int kParts = kThreads / kCols;  // threads that share a channel where pairs are joined
constexpr int kPartRuns = kRuns / kParts;
constexpr int kGroup = 16;  // tiles of a group
// Tokens of a thread: 32 to 64 registers of inputs.
template <typename T, bool BACK>
struct Run {
  static constexpr int n = sizeof(T) == 4 && BACK ? 2 : 4;
  static constexpr int tile = n * kRuns;  // tokens of a tile
  static_assert(tile % kChunk == 0, "tiles start at a kept state");
};
inline int tile_tokens(int dtype, bool back) {
  return dtype == CCQ_DTYPE_BF16 ? (back ? Run<__bf16, true>::tile : Run<__bf16, false>::tile)
                                 : (back ? Run<float, true>::tile : Run<float, false>::tile);
}

__device__ __forceinline__ int sequence_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// ---------------------------------------------------------------- gates

// alpha = exp(g); 0 below about -87.  The hardware's 2^p takes the rounded product p = g log2(e), whose
// rounding is worth up to |g| 2^-24 of the result.  For fp32 inputs it is made good to first order, which
// leaves about 2 units in the last place; bf16 inputs stand for values 2^-9 |g| apart, and go without.
template <typename T>
__device__ __forceinline__ float gate(float g) {
  constexpr float hi = 1.44269502162933349609f, lo = 1.92596299112661746887e-8f, ln2 = 0.693147180559945f;
  const float p = g * hi;
  const float a = __builtin_amdgcn_exp2f(p);
  if constexpr (sizeof(T) == 2) return a;
  const float rest = fmaf(g, lo, fmaf(g, hi, -p));
  return fabsf(p) < 127.f ? fmaf(a, rest * ln2, a) : a;  // beyond: 0, infinity or NaN
}

// 1 - alpha, good to a few units in the last place also where alpha is near 1: the series of 1 - exp(g)
// to the sixth power there (its next term is below 2^-24 of the sum for |g| < 1/4).
__device__ __forceinline__ float one_minus(float g, float alpha) {
  float s = 1.f / 720.f;
  s = fmaf(s, g, 1.f / 120.f);
  s = fmaf(s, g, 1.f / 24.f);
  s = fmaf(s, g, 1.f / 6.f);
  s = fmaf(s, g, 0.5f);
  s = fmaf(s, g, 1.f);
  return fabsf(g) < 0.25f ? -g * s : 1.f - alpha;
}

// The same within 2^-19 of itself, for what is stored in bf16 a few tokens on (all of the series there: 56 against 55 us
// at B4 T4096 D2048, 84 against 82 for the gradient).
__device__ __forceinline__ float one_minus_short(float g, float alpha) {
  return fabsf(g) < 1.f / 32.f ? -g * fmaf(fmaf(1.f / 6.f, g, 0.5f), g, 1.f) : 1.f - alpha;
}
template <bool SHORT>
__device__ __forceinline__ float complement_of(float g, float alpha) {
  return SHORT ? one_minus_short(g, alpha) : one_minus(g, alpha);
}

// alpha h, and alpha h + u; with RESETS 0 h = 0 for every h.  Where no gate of a wave is 0, as is the
// rule, its walks go without that test, a third of their operations.
template <bool RESETS>
__device__ __forceinline__ float gated(float alpha, float h) {
  return RESETS && alpha == 0.f ? 0.f : alpha * h;
}
template <bool RESETS>
__device__ __forceinline__ float step(float alpha, float h, float u) {
  return RESETS && alpha == 0.f ? u : fmaf(alpha, h, u);
}
// The state behind a token.  With the complement scale, alpha h + (1 - alpha) x, from 1 - alpha formed for itself:
// x + alpha (h - x), which spares some operations, rounds at the size of x, and behind gates next to 1 the state is
// far smaller.
template <bool RESETS, bool COMPLEMENT, bool SHORT>
__device__ __forceinline__ float advance(float alpha, float g, float h, float x) {
  return step<RESETS>(alpha, h, COMPLEMENT ? x * complement_of<SHORT>(g, alpha) : x);
}

__device__ __forceinline__ bool drops(float P) { return __float_as_int(P) < 0; }

// The product of a run's gates, one more of them.  Once it drops the state it stays so, whatever gates follow.
template <bool RESETS>
__device__ __forceinline__ float gates_product(float P, float alpha) {
  return RESETS && (alpha == 0.f || drops(P)) ? -0.f : P * alpha;
}

// Whether a run's product of gates leaves open that one of them is 0: NaN, too, is 0 times an infinity or NaN.
__device__ __forceinline__ bool may_drop(float P) { return !(P > 0.f); }

// ---------------------------------------------------------------- runs

struct Pair {
  float P, q;
};

// The state behind a run that found `h`.  A product of gates that has left the range of fp32 counts as its least or
// its largest number: an infinity or NaN passes the one, and no state, 0, is left alone by the other.
__device__ __forceinline__ float through(float h, const Pair& r) {
  return drops(r.P) ? r.q : fmaf(__builtin_amdgcn_fmed3f(r.P, FLT_MIN, FLT_MAX), h, r.q);
}
__device__ __forceinline__ Pair then(const Pair& a, const Pair& b) {
  Pair c;
  c.q = through(a.q, b);
  c.P = (__float_as_int(a.P) | __float_as_int(b.P)) < 0 ? -0.f : a.P * b.P;
  return c;
}

// ---------------------------------------------------------------- eight channels of a token

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

// The stored form, so that a thread's loads are all under way before the first is waited for: eight
// channels in words of kPer.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <typename T>
struct Raw8 {
  static constexpr int kPer = 4 / (int)sizeof(T), kWords = 8 / kPer;
  unsigned w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + i * kPer));
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i + j] = v[j];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      __builtin_nontemporal_store(u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]}, reinterpret_cast<u32x4*>(p + i * kPer));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // channel e of word i
  __device__ __forceinline__ float get(int i, int e) const {
    if constexpr (kPer == 1) return __uint_as_float(w[i]);
    return __uint_as_float(e ? w[i] & 0xffff0000u : w[i] << 16);
  }
  __device__ __forceinline__ void set(int i, const float (&x)[kPer]) {
    if constexpr (kPer == 1) w[i] = __float_as_uint(x[0]);
    else w[i] = __builtin_bit_cast(unsigned, bf16x2{(__bf16)x[0], (__bf16)x[1]});
  }
};

// Behind the end of a sequence: gates of 1 and inputs of 0, so nothing changes.
template <typename R, int N>
__device__ __forceinline__ void clear_from(R (&raw)[N], int live) {
#pragma unroll
  for (int r = 0; r < N; ++r)
    if (r >= live) raw[r].clear();
}

// Makes word i of a run new to the compiler once `done` is known: without this it forms all of a run's
// gates before it folds the first, or keeps them for the walk, and neither fits the registers.
template <typename R, int N>
__device__ __forceinline__ void in_turn(R (&raw)[N], int i, float done) {
#pragma unroll
  for (int r = 0; r < N; ++r) asm volatile("" : "+v"(raw[r].w[i]) : "v"(done));
}

// A thread's run of one input: token t0 on, eight channels from c0 on.  Every load is made, at a row and
// column inside the tensor (behind the sequence: its last, read once for all); what lies outside is cleared later.
template <typename T, int RUN>
__device__ __forceinline__ void load_run(Raw8<T> (&raw)[RUN], const void* base, int64_t stride_b, int64_t stride_t, int b,
                                         int t0, int c0, int n, int D) {
  const T* p = static_cast<const T*>(base) + b * stride_b + min(c0, D - 8);
#pragma unroll
  for (int r = 0; r < RUN; ++r) raw[r].load(p + (int64_t)max(min(t0 + r, n - 1), 0) * stride_t);
}

// ---------------------------------------------------------------- tiles

// The tiles of a call: (sequence, 128 channels) columns of `segments` tiles.  Counter k hands out the
// tiles of columns k, k + kCounters, ... in the order of the recurrence: all of the first tokens, then of
// the next.  One counter for all took 4.4 ns a tile, 18 of 78 us at B4 T4096 D2048 with 4096 tiles.  The
// workspace holds the counters, a pair for every tile and channel, and one for every group of tiles.
constexpr int kCounters = 16;
constexpr int kCounterStride = 32;  // words: a cache line each
struct Tiles {
  int columns;   // B ceil(D / 128)
  int per_row;   // ceil(D / 128)
  int segments;  // ceil(T / tile)
  unsigned* counters;
  uint64_t* pairs;   // [segments][columns][128]
  uint64_t* groups;  // [segments / kGroup][columns][128]
};
constexpr size_t kCounterBytes = kCounters * kCounterStride * 4;

// No pair: all ones; the half of P is then a NaN that is never published.

__device__ __forceinline__ void publish(uint64_t* at, Pair r) {
  if (r.P != r.P) r.P = __int_as_float(0x7fc00000);
  const uint64_t word = ((uint64_t)__float_as_uint(r.q) << 32) | __float_as_uint(r.P);
  __hip_atomic_store(at, word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Pair unpack(uint64_t word) {
  return Pair{__uint_as_float((unsigned)word), __uint_as_float((unsigned)(word >> 32))};
}

__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool is_empty(uint64_t word) { return (unsigned)word == 0xffffffffu; }

// The fold of n published pairs, `stride` words apart.  The wave waits as one: where a pair is missing, one
// lane for each pair watches its first word, so that waiting costs the memory little.
template <int BATCH>
__device__ __forceinline__ Pair fold_published(const uint64_t* from, int lane, int n, size_t stride) {
  Pair acc{1.f, 0.f};
  int polls = 0;
  for (int i = 0; i < n; i += BATCH) {
    uint64_t w[BATCH];
    for (;;) {
      bool empty = false;
#pragma unroll
      for (int j = 0; j < BATCH; ++j) w[j] = peek(from + (size_t)min(i + j, n - 1) * stride + lane);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) empty |= is_empty(w[j]);
      if (!__any(empty)) break;
      do {
        if (++polls > (1 << 19)) return Pair{-0.f, __int_as_float(0x7fc00000)};
        __builtin_amdgcn_s_sleep(4);
      } while (__any(lane < BATCH && is_empty(peek(from + (size_t)min(i + lane, n - 1) * stride))));
    }
#pragma unroll
    for (int j = 0; j < BATCH; ++j)
      if (i + j < n) acc = then(acc, unpack(w[j]));
  }
  return acc;
}

// Pairs of a channel, a part a thread.
typedef Pair Parts[kParts][kCols];
__device__ __forceinline__ Pair fold_parts(const Parts& parts, int ch) {
  Pair all = parts[0][ch];
#pragma unroll
  for (int i = 1; i < kParts; ++i) all = then(all, parts[i][ch]);
  return all;
}

// The state before segment s > 0 of a column, for channel ch: the threads that share the channel (part 0 ..
// kParts - 1) fold a part of the pairs each.  own: the segment's pair, which part 0 has published; the
// last segment of a group publishes the group's.  All threads take part.
__device__ __forceinline__ float state_before(const Tiles& t, int s, int column, int part, int half, int lane,
                                              const Parts& own, Parts& parts) {
  const size_t stride = (size_t)t.columns * kCols, at = (size_t)column * kCols + 64 * half;
  const int ch = 64 * half + lane, g = s / kGroup, first = g * kGroup, inside = s - first;
  Pair here{1.f, 0.f};
  if (inside > 0) {
    constexpr int share = kGroup / kParts;
    const int from = part * share;
    parts[part][ch] =
        fold_published<share>(t.pairs + (size_t)(first + from) * stride + at, lane, min(share, inside - from), stride);
    __syncthreads();
    here = fold_parts(parts, ch);
  }
  if (inside == kGroup - 1 && part == 0) publish(t.groups + (size_t)g * stride + at + lane, then(here, fold_parts(own, ch)));
  if (g == 0) return here.q;  // segment 0's pair holds the state before it and drops what it is given
  const int share = (g + kParts - 1) / kParts, from = part * share;
  if (inside > 0) __syncthreads();
  parts[part][ch] = fold_published<4>(t.groups + (size_t)from * stride + at, lane, min(share, g - from), stride);
  __syncthreads();
  return through(fold_parts(parts, ch).q, here);
}

// A tile behind the sequence, the order-th of its column, lets the state pass.  It need not wait for it, and
// there is nothing else to do, unless it is the column's first or last or ends a group.
__device__ __forceinline__ bool passes_on(const Tiles& t, int order, int column, int part, int ch) {
  if (order == 0 || order == t.segments - 1 || order % kGroup == kGroup - 1) return false;
  if (part == 0) publish(t.pairs + ((size_t)order * t.columns + column) * kCols + ch, Pair{1.f, 0.f});
  return true;
}

__global__ __launch_bounds__(kStepThreads) void scan_clear_kernel(Tiles t, size_t words) {
  if (blockIdx.x == 0 && threadIdx.x < kCounters) t.counters[threadIdx.x * kCounterStride] = 0;
  // words come 128 at a time
  for (size_t i = ((size_t)blockIdx.x * kStepThreads + threadIdx.x) * 2; i < words; i += (size_t)gridDim.x * kStepThreads * 2)
    *reinterpret_cast<u32x4*>(t.pairs + i) = u32x4{~0u, ~0u, ~0u, ~0u};
}

// A thread's run of tokens, from the stored inputs: folded to its pairs, and walked from the state before
// it.  Folding tells whether a gate is 0 (or the product too small to tell): then it is done again with
// that in mind.  The gates are formed each time: keeping them would take 64 registers, and the registers decide how
// many loads a CU has under way.
template <bool RESETS, bool COMPLEMENT, typename T, int RUN>
__device__ __forceinline__ bool fold_run(Raw8<T> (&g_raw)[RUN], Raw8<T> (&x_raw)[RUN], Pair (&out)[8]) {
  constexpr int PER = Raw8<T>::kPer;
  bool zero = false;
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) {
    in_turn(g_raw, i, i ? out[i * PER - 1].q : 0.f);
    in_turn(x_raw, i, i ? out[i * PER - 1].q : 0.f);
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      Pair r{1.f, 0.f};
#pragma unroll
      for (int t = 0; t < RUN; ++t) {
        const float g = g_raw[t].get(i, e), x = x_raw[t].get(i, e), a = gate<T>(g);
        r.q = advance<RESETS, COMPLEMENT, false>(a, g, r.q, x);
        r.P = t == 0 && !RESETS ? a : gates_product<RESETS>(r.P, a);
      }
      zero |= may_drop(r.P);
      out[i * PER + e] = r;
    }
  }
  return zero;
}
// From the states before the run to the stored states, in the place of the inputs.
template <bool RESETS, bool COMPLEMENT, typename T, int RUN>
__device__ __forceinline__ void walk_run(Raw8<T> (&g_raw)[RUN], Raw8<T> (&x_raw)[RUN], const Pair* starts) {
  constexpr int PER = Raw8<T>::kPer;
  float done = 0.f;
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) {
    in_turn(g_raw, i, done);
    in_turn(x_raw, i, done);
    float h[RUN][PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float state = starts[i * PER + e].P;
#pragma unroll
      for (int t = 0; t < RUN; ++t) {
        const float g = g_raw[t].get(i, e), x = x_raw[t].get(i, e), a = gate<T>(g);
        h[t][e] = state = advance<RESETS, COMPLEMENT, sizeof(T) == 2>(a, g, state, x);
      }
      done = state;
    }
#pragma unroll
    for (int t = 0; t < RUN; ++t) x_raw[t].set(i, h[t]);
  }
}

// This workgroup's tile: its place in the order of the recurrence and its column.
struct Place {
  int order, column;
};
__device__ __forceinline__ Place next_tile(const Tiles& t, unsigned* shared) {
  if (t.segments == 1) return Place{0, (int)blockIdx.x};
  const unsigned k = (blockIdx.x % (unsigned)t.columns) % kCounters;
  const unsigned share = ((unsigned)t.columns - k + kCounters - 1) / kCounters;  // the counter's columns
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(t.counters + k * kCounterStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const unsigned i = __builtin_amdgcn_readfirstlane(*shared), order = i / share;
  return Place{(int)order, (int)(k + kCounters * (i - order * share))};
}

template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : COMPLEMENT ? 4 : 6) void scan_tile_kernel(ccq_scan_params p, Tiles tiles) {
  constexpr int RUN = Run<T, false>::n, TILE = Run<T, false>::tile;
  // 40 KB: four workgroups fit a CU
  __shared__ __align__(16) Pair runs[kRuns][kCols];  // every run's pair, and then the state before it
  __shared__ Parts own, parts;
  const Place place = next_tile(tiles, reinterpret_cast<unsigned*>(&parts));
  const int s = place.order, column = place.column;
  const int b = column / tiles.per_row, c_tile = (column - b * tiles.per_row) * kCols;
  const int n = sequence_length(p.lengths, b, p.T);
  // where tokens are held: run and eight channels
  const int run = threadIdx.x / kOct, oct = threadIdx.x % kOct;
  const int t0 = s * TILE + run * RUN, c0 = c_tile + 8 * oct;
  // where pairs are joined: part and channel
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int part = wave / (kCols / 64), half = wave % (kCols / 64), ch = 64 * half + lane, c = c_tile + ch;

  if (s * TILE >= n && passes_on(tiles, s, column, part, ch)) return;
  Raw8<T> g_raw[RUN], x_raw[RUN];
  load_run(g_raw, p.log_alpha, p.la_stride_b, p.la_stride_t, b, t0, c0, n, p.D);
  load_run(x_raw, p.x, p.x_stride_b, p.x_stride_t, b, t0, c0, n, p.D);
  if ((s + 1) * TILE > n) {
    clear_from(g_raw, n - t0);
    clear_from(x_raw, n - t0);
  }
  Pair mine[8];
  const bool resets = __any(fold_run<false, COMPLEMENT>(g_raw, x_raw, mine));
  if (resets) fold_run<true, COMPLEMENT>(g_raw, x_raw, mine);
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    *reinterpret_cast<f32x4*>(&runs[run][8 * oct + e]) = f32x4{mine[e].P, mine[e].q, mine[e + 1].P, mine[e + 1].q};
  __syncthreads();
  Pair sum{1.f, 0.f};
#pragma unroll
  for (int r = 0; r < kPartRuns; ++r) sum = then(sum, runs[part * kPartRuns + r][ch]);
  float start = 0.f;
  if (s == 0) {
    start = p.h0 && c < p.D ? p.h0[(size_t)b * p.D + c] : 0.f;
    if (part == 0) sum = Pair{-0.f, through(start, sum)};  // holds the state before it
  }
  own[part][ch] = sum;
  __syncthreads();
  if (part == 0 && tiles.segments > 1)
    publish(tiles.pairs + ((size_t)s * tiles.columns + column) * kCols + ch, fold_parts(own, ch));
  if (s > 0) start = state_before(tiles, s, column, part, half, lane, own, parts);
  float h = start;
  for (int i = 0; i < part; ++i) h = through(h, own[i][ch]);
#pragma unroll
  for (int r = 0; r < kPartRuns; ++r) {
    const Pair pair = runs[part * kPartRuns + r][ch];
    runs[part * kPartRuns + r][ch].P = h;
    const int t = s * TILE + (part * kPartRuns + r) * RUN;
    if (p.chunk_carry && t % kChunk == 0 && t < n && c < p.D)
      p.chunk_carry[((size_t)b * ((p.T + kChunk - 1) / kChunk) + t / kChunk) * p.D + c] = h;
    h = through(h, pair);
  }
  if (p.h_out && s == tiles.segments - 1 && part == kParts - 1 && c < p.D) p.h_out[(size_t)b * p.D + c] = h;
  __syncthreads();
  if (p.y == nullptr || c0 >= p.D) return;
  if (resets) walk_run<true, COMPLEMENT>(g_raw, x_raw, &runs[run][8 * oct]);
  else walk_run<false, COMPLEMENT>(g_raw, x_raw, &runs[run][8 * oct]);
  T* y = static_cast<T*>(p.y) + ((size_t)b * p.T + t0) * p.D + c0;
#pragma unroll
  for (int r = 0; r < RUN; ++r)
    if (t0 + r < n) x_raw[r].store(y + (size_t)r * p.D);
}

// A thread's run for the gradient: the state's pair and the adjoint's q; then both walked.
template <bool RESETS, bool COMPLEMENT, typename T, int RUN>
__device__ __forceinline__ bool fold_run_back(Raw8<T> (&g_raw)[RUN], Raw8<T> (&x_raw)[RUN],
                                              Raw8<T> (&d_raw)[RUN], Pair (&out)[8], float (&q)[8]) {
  constexpr int PER = Raw8<T>::kPer;
  bool zero = false;
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) {
    in_turn(g_raw, i, i ? q[i * PER - 1] : 0.f);
    in_turn(x_raw, i, i ? q[i * PER - 1] : 0.f);
    in_turn(d_raw, i, i ? q[i * PER - 1] : 0.f);
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float a[RUN], adj = 0.f;
      Pair r{1.f, 0.f};
#pragma unroll
      for (int t = 0; t < RUN; ++t) {
        const float g = g_raw[t].get(i, e), x = x_raw[t].get(i, e);
        a[t] = gate<T>(g);
        r.q = advance<RESETS, COMPLEMENT, sizeof(T) == 2>(a[t], g, r.q, x);
        r.P = t == 0 && !RESETS ? a[t] : gates_product<RESETS>(r.P, a[t]);
      }
      // the scaled inputs first: the adjoint's gradients taken up among them, registers spill (94 against 82 us at
      // B4 T4096 D2048)
      if constexpr (COMPLEMENT && sizeof(T) == 2) in_turn(d_raw, i, r.q);
#pragma unroll
      for (int t = RUN - 1; t >= 0; --t) adj = gated<RESETS>(a[t], adj + d_raw[t].get(i, e));
      zero |= may_drop(r.P);
      out[i * PER + e] = r;
      q[i * PER + e] = adj;
    }
  }
  return zero;
}
// From the states before the run and the adjoints behind it (P, q of `ends`) to the stored gradients: the
// input's in the place of x_raw, log_alpha's in the place of g_raw.
template <bool RESETS, bool COMPLEMENT, typename T, int RUN>
__device__ __forceinline__ void walk_run_back(Raw8<T> (&g_raw)[RUN], Raw8<T> (&x_raw)[RUN],
                                              Raw8<T> (&d_raw)[RUN], const Pair* ends) {
  constexpr int PER = Raw8<T>::kPer;
  float done = 0.f;
#pragma unroll
  for (int i = 0; i < Raw8<T>::kWords; ++i) {
    in_turn(g_raw, i, done);
    in_turn(x_raw, i, done);
    in_turn(d_raw, i, done);
    float ox[RUN][PER], og[RUN][PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float h = ends[i * PER + e].P, adj = ends[i * PER + e].q;
      float a[RUN], s[RUN], of[RUN];  // of: what log_alpha's gradient takes: the state before, less the input
#pragma unroll
      for (int t = 0; t < RUN; ++t) {
        const float g = g_raw[t].get(i, e), x = x_raw[t].get(i, e);
        a[t] = gate<T>(g);
        of[t] = COMPLEMENT ? h - x : h;
        s[t] = COMPLEMENT ? complement_of<sizeof(T) == 2>(g, a[t]) : 1.f;
        h = step<RESETS>(a[t], h, COMPLEMENT ? s[t] * x : x);
      }
#pragma unroll
      for (int t = RUN - 1; t >= 0; --t) {
        const float full = adj + d_raw[t].get(i, e);
        adj = gated<RESETS>(a[t], full);
        ox[t][e] = COMPLEMENT ? s[t] * full : full;
        og[t][e] = RESETS ? gated<RESETS>(a[t], full * of[t]) : adj * of[t];
      }
      done = adj;
    }
#pragma unroll
    for (int t = 0; t < RUN; ++t) {
      x_raw[t].set(i, ox[t]);
      g_raw[t].set(i, og[t]);
    }
  }
}

template <typename T, int RUN>
__device__ __forceinline__ void store_runs(const ccq_scan_bwd_params& p, const Raw8<T> (&x_raw)[RUN], const Raw8<T> (&g_raw)[RUN],
                                           int b, int t0, int c0) {
  if (c0 >= p.D) return;
  const size_t at = ((size_t)b * p.T + t0) * p.D + c0;
  T *dx = static_cast<T*>(p.dx) + at, *dg = static_cast<T*>(p.dlog_alpha) + at;
#pragma unroll
  for (int r = 0; r < RUN; ++r) {
    if (t0 + r < p.T) {
      x_raw[r].store(dx + (size_t)r * p.D);
      g_raw[r].store(dg + (size_t)r * p.D);
    }
  }
}

// The gradient: the same tiles from the end.  The adjoint that reaches a token from behind, d, becomes
// alpha (d + dy) in front of it, so a run acts on it as d -> P d + q with the run's own product of gates.
// The states are walked forward again, from the state kept before the tile.
template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads, 4) void scan_backward_tile_kernel(ccq_scan_bwd_params p, const float* carry,
                                                                         Tiles tiles) {
  constexpr int RUN = Run<T, true>::n, TILE = Run<T, true>::tile;
  __shared__ __align__(16) Pair runs[kRuns][kCols];   // every run's pair; then state before it, adjoint behind it
  __shared__ __align__(16) float back[kRuns][kCols];  // q of every run for the adjoint
  __shared__ Parts ahead, own, parts;                 // own: for the adjoint, the tile's last part first
  const Place place = next_tile(tiles, reinterpret_cast<unsigned*>(&parts));
  const int order = place.order, column = place.column, s = tiles.segments - 1 - order;
  const int b = column / tiles.per_row, c_tile = (column - b * tiles.per_row) * kCols;
  const int n = sequence_length(p.lengths, b, p.T);
  const int run = threadIdx.x / kOct, oct = threadIdx.x % kOct;
  const int t0 = s * TILE + run * RUN, c0 = c_tile + 8 * oct;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int part = wave / (kCols / 64), half = wave % (kCols / 64), ch = 64 * half + lane, c = c_tile + ch;

  Raw8<T> g_raw[RUN], x_raw[RUN], d_raw[RUN];
  if (s * TILE >= n && passes_on(tiles, order, column, part, ch)) {
    clear_from(g_raw, 0);
    clear_from(x_raw, 0);
    store_runs(p, x_raw, g_raw, b, t0, c0);
    return;
  }
  load_run(g_raw, p.log_alpha, p.la_stride_b, p.la_stride_t, b, t0, c0, n, p.D);
  load_run(x_raw, p.x, p.x_stride_b, p.x_stride_t, b, t0, c0, n, p.D);
  load_run(d_raw, p.dy, p.dy_stride_b, p.dy_stride_t, b, t0, c0, n, p.D);
  float h = 0.f;  // state before the tile
  if (carry && s * TILE < n && c < p.D)
    h = carry[((size_t)b * ((p.T + kChunk - 1) / kChunk) + s * (TILE / kChunk)) * p.D + c];
  if ((s + 1) * TILE > n) {
    clear_from(g_raw, n - t0);
    clear_from(x_raw, n - t0);
    clear_from(d_raw, n - t0);
  }
  bool resets;
  {
    Pair mine[8];
    float q[8];
    resets = __any(fold_run_back<false, COMPLEMENT>(g_raw, x_raw, d_raw, mine, q));
    if (resets) fold_run_back<true, COMPLEMENT>(g_raw, x_raw, d_raw, mine, q);
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      *reinterpret_cast<f32x4*>(&runs[run][8 * oct + e]) = f32x4{mine[e].P, mine[e].q, mine[e + 1].P, mine[e + 1].q};
    store8(&back[run][8 * oct], q);
  }
  __syncthreads();
  Pair sum{1.f, 0.f}, rsum{1.f, 0.f};
#pragma unroll
  for (int r = 0; r < kPartRuns; ++r) sum = then(sum, runs[part * kPartRuns + r][ch]);
#pragma unroll
  for (int r = kPartRuns - 1; r >= 0; --r)
    rsum = then(rsum, Pair{runs[part * kPartRuns + r][ch].P, back[part * kPartRuns + r][ch]});
  float end = 0.f;
  if (order == 0) {
    end = p.dh_out && c < p.D ? p.dh_out[(size_t)b * p.D + c] : 0.f;
    if (part == kParts - 1) rsum = Pair{-0.f, through(end, rsum)};
  }
  ahead[part][ch] = sum;
  own[kParts - 1 - part][ch] = rsum;
  __syncthreads();
  if (part == 0 && tiles.segments > 1)
    publish(tiles.pairs + ((size_t)order * tiles.columns + column) * kCols + ch, fold_parts(own, ch));
  if (order > 0) end = state_before(tiles, order, column, part, half, lane, own, parts);
  float d = end;
  for (int i = 0; i < kParts - 1 - part; ++i) d = through(d, own[i][ch]);
  for (int i = 0; i < part; ++i) h = through(h, ahead[i][ch]);
#pragma unroll
  for (int r = kPartRuns - 1; r >= 0; --r) {
    float& q = back[part * kPartRuns + r][ch];
    const float next = through(d, Pair{runs[part * kPartRuns + r][ch].P, q});
    q = d;
    d = next;
  }
  if (p.dh0 && s == 0 && part == 0 && c < p.D) p.dh0[(size_t)b * p.D + c] = d;
#pragma unroll
  for (int r = 0; r < kPartRuns; ++r) {
    const Pair pair = runs[part * kPartRuns + r][ch];
    runs[part * kPartRuns + r][ch] = Pair{h, back[part * kPartRuns + r][ch]};
    h = through(h, pair);
  }
  __syncthreads();
  const Pair* ends = &runs[run][8 * oct];
  if (resets) walk_run_back<true, COMPLEMENT>(g_raw, x_raw, d_raw, ends);
  else walk_run_back<false, COMPLEMENT>(g_raw, x_raw, d_raw, ends);
  if ((s + 1) * TILE > n) {
    clear_from(g_raw, n - t0);
    clear_from(x_raw, n - t0);
  }
  store_runs(p, x_raw, g_raw, b, t0, c0);
}

// ---------------------------------------------------------------- short sequences

// Up to kChunk tokens: the runs of a workgroup are dealt out to several sequences, `each` (a power of two) a
// sequence, on the same channels.  A thread folds its sequence's other runs for itself, and nothing is waited
// for.  (131 sequences of up to 11 tokens, 2992 channels, bf16: 49 us in tiles, whose runs stood empty.)
struct Seat {
  int b, n, t0, c0;      // sequence, its length, the run's first token, the first of eight channels
  int first, run, last;  // runs of the sequence
  bool live;             // inside the tensor; else b is the last sequence
};
template <int RUN>
__device__ __forceinline__ Seat take_seat(const int32_t* lengths, int B, int T, int D, int per_row, int each) {
  Seat a;
  const int group = blockIdx.x / per_row;
  a.run = threadIdx.x / kOct;
  a.first = a.run & ~(each - 1);
  a.last = a.first + each - 1;
  a.c0 = (blockIdx.x - group * per_row) * kCols + 8 * (threadIdx.x % kOct);
  a.t0 = (a.run - a.first) * RUN;
  const int b = group * (kRuns / each) + a.run / each;
  a.live = b < B && a.c0 < D;
  a.b = min(b, B - 1);
  a.n = sequence_length(lengths, a.b, T);
  return a;
}

template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads, 4) void scan_short_kernel(ccq_scan_params p, int per_row, int each) {
  constexpr int RUN = Run<T, false>::n;
  __shared__ __align__(16) Pair runs[kRuns][kCols];
  const Seat a = take_seat<RUN>(p.lengths, p.B, p.T, p.D, per_row, each);
  const int ch = 8 * (threadIdx.x % kOct);
  const size_t at = (size_t)a.b * p.D + min(a.c0, p.D - 8);
  Raw8<T> g_raw[RUN], x_raw[RUN];
  load_run(g_raw, p.log_alpha, p.la_stride_b, p.la_stride_t, a.b, a.t0, a.c0, a.n, p.D);
  load_run(x_raw, p.x, p.x_stride_b, p.x_stride_t, a.b, a.t0, a.c0, a.n, p.D);
  float h[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.h0) load8(p.h0 + at, h);  // before anyone writes h_out, which may be h0
  clear_from(g_raw, a.n - a.t0);
  clear_from(x_raw, a.n - a.t0);
  Pair mine[8];
  const bool resets = __any(fold_run<false, COMPLEMENT>(g_raw, x_raw, mine));
  if (resets) fold_run<true, COMPLEMENT>(g_raw, x_raw, mine);
#pragma unroll
  for (int e = 0; e < 8; ++e) runs[a.run][ch + e] = mine[e];
  __syncthreads();
  if (!a.live) return;
  if (p.chunk_carry && a.run == a.first && a.n > 0) store8(p.chunk_carry + at, h);
  for (int r = a.first; r < a.run; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = through(h[e], runs[r][ch + e]);
  }
  if (p.h_out && a.run == a.last) {
    float end[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) end[e] = through(h[e], mine[e]);
    store8(p.h_out + at, end);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e].P = h[e];
  if (resets) walk_run<true, COMPLEMENT>(g_raw, x_raw, mine);
  else walk_run<false, COMPLEMENT>(g_raw, x_raw, mine);
  T* y = static_cast<T*>(p.y) + ((size_t)a.b * p.T + a.t0) * p.D + a.c0;
#pragma unroll
  for (int r = 0; r < RUN; ++r)
    if (a.t0 + r < a.n) x_raw[r].store(y + (size_t)r * p.D);
}

// states: before the only chunk, [B, D], or null.
template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads, 4) void scan_short_backward_kernel(ccq_scan_bwd_params p, const float* states,
                                                                          int per_row, int each) {
  constexpr int RUN = Run<T, true>::n;
  __shared__ __align__(16) Pair runs[kRuns][kCols];
  __shared__ __align__(16) float back[kRuns][kCols];
  const Seat a = take_seat<RUN>(p.lengths, p.B, p.T, p.D, per_row, each);
  const int ch = 8 * (threadIdx.x % kOct);
  const size_t at = (size_t)a.b * p.D + min(a.c0, p.D - 8);
  Raw8<T> g_raw[RUN], x_raw[RUN], d_raw[RUN];
  load_run(g_raw, p.log_alpha, p.la_stride_b, p.la_stride_t, a.b, a.t0, a.c0, a.n, p.D);
  load_run(x_raw, p.x, p.x_stride_b, p.x_stride_t, a.b, a.t0, a.c0, a.n, p.D);
  load_run(d_raw, p.dy, p.dy_stride_b, p.dy_stride_t, a.b, a.t0, a.c0, a.n, p.D);
  float h[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  auto load_ends = [&] {  // before anyone writes dh0, which may be dh_out
    if (states && a.n > 0) load8(states + at, h);
    if (p.dh_out) load8(p.dh_out + at, d);
  };
  // with bf16 and the complement the fold needs their registers (18.2 against 17 us for 131 sequences of up to 11 tokens)
  constexpr bool LATE = COMPLEMENT && sizeof(T) == 2;
  if constexpr (!LATE) load_ends();
  clear_from(g_raw, a.n - a.t0);
  clear_from(x_raw, a.n - a.t0);
  clear_from(d_raw, a.n - a.t0);
  Pair mine[8];
  float q[8];
  const bool resets = __any(fold_run_back<false, COMPLEMENT>(g_raw, x_raw, d_raw, mine, q));
  if (resets) fold_run_back<true, COMPLEMENT>(g_raw, x_raw, d_raw, mine, q);
  if constexpr (LATE) load_ends();
#pragma unroll
  for (int e = 0; e < 8; ++e) runs[a.run][ch + e] = mine[e];
  store8(&back[a.run][ch], q);
  __syncthreads();
  if (!a.live) return;
  for (int r = a.first; r < a.run; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = through(h[e], runs[r][ch + e]);
  }
  for (int r = a.last; r > a.run; --r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] = through(d[e], Pair{runs[r][ch + e].P, back[r][ch + e]});
  }
  if (p.dh0 && a.run == a.first) {
    float front[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) front[e] = through(d[e], Pair{mine[e].P, q[e]});
    store8(p.dh0 + at, front);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = Pair{h[e], d[e]};
  if (resets) walk_run_back<true, COMPLEMENT>(g_raw, x_raw, d_raw, mine);
  else walk_run_back<false, COMPLEMENT>(g_raw, x_raw, d_raw, mine);
  clear_from(g_raw, a.n - a.t0);
  clear_from(x_raw, a.n - a.t0);
  store_runs(p, x_raw, g_raw, a.b, a.t0, a.c0);
}

// A few tokens: eight channels a thread, one token behind the other.
template <typename T>
__global__ __launch_bounds__(kStepThreads) void scan_step_kernel(ccq_scan_params p) {
  const int per_row = p.D / 8;
  const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  if (i >= (int64_t)p.B * per_row) return;
  const int b = (int)(i / per_row), c = 8 * (int)(i - (int64_t)b * per_row);
  const int n = sequence_length(p.lengths, b, p.T);
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c;
  const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c;
  T* y = static_cast<T*>(p.y) + (int64_t)b * p.T * p.D + c;
  float h[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.h0) load8(p.h0 + (int64_t)b * p.D + c, h);
  if (p.chunk_carry && n > 0) store8(p.chunk_carry + (int64_t)b * p.D + c, h);  // one chunk: T <= 64
  for (int t = 0; t < n; ++t) {
    float gt[8], xt[8];
    load8(g + t * p.la_stride_t, gt);
    load8(x + t * p.x_stride_t, xt);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float alpha = gate<T>(gt[e]);
      h[e] = step<true>(alpha, h[e], p.complement ? xt[e] * one_minus(gt[e], alpha) : xt[e]);
    }
    store8(y + (int64_t)t * p.D, h);
  }
  if (p.h_out) store8(p.h_out + (int64_t)b * p.D + c, h);
}

// ---------------------------------------------------------------- launches

Tiles tiles_of(int dtype, bool back, int B, int T, int D, void* workspace) {
  Tiles t{};
  t.per_row = (D + kCols - 1) / kCols;
  t.columns = B * t.per_row;
  t.segments = (T - 1) / tile_tokens(dtype, back) + 1;
  t.counters = static_cast<unsigned*>(workspace);
  t.pairs = reinterpret_cast<uint64_t*>(static_cast<unsigned char*>(workspace) + kCounterBytes);
  t.groups = t.pairs + (size_t)t.segments * t.columns * kCols;
  return t;
}
size_t tile_words(int dtype, bool back, int B, int T, int D) {
  const size_t segments = (size_t)((T - 1) / tile_tokens(dtype, back) + 1);
  if (segments == 1) return 0;
  return (segments + segments / kGroup) * B * ((D + kCols - 1) / kCols) * kCols;
}
size_t tile_bytes(int dtype, bool back, int B, int T, int D) {
  const size_t words = tile_words(dtype, back, B, T, D);
  return words ? kCounterBytes + words * sizeof(uint64_t) : 0;
}

hipError_t clear_tiles(const Tiles& t, size_t words, hipStream_t stream) {
  if (words == 0) return hipSuccess;
  const size_t blocks = (words + kStepThreads * 4 - 1) / (kStepThreads * 4);
  scan_clear_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), kStepThreads, 0, stream>>>(t, words);
  return hipGetLastError();
}

// Up to this many tokens go one behind the other in a thread.
constexpr int kMostSteps = 8;

// Runs of a short sequence, which every thread of it goes through, and the workgroups that hold all sequences.
// With 32 a sequence (the fp32 gradient of 64 tokens) the tiles' own way is faster, 35 against 58 us at B64
// D2048; with 16 it is not (30 tokens 23.6 against 22.9; the bf16 forward of 64 14.8 against 13.5).
constexpr int kMostRuns = 16;
int runs_each(int T, int run) {
  int each = 1;
  while (each <= kMostRuns && each * run < T) each *= 2;
  return each;
}
uint64_t short_grid(int B, int D, int each) {
  const int sequences = kRuns / each;
  return ((uint64_t)B + sequences - 1) / sequences * ((D + kCols - 1) / kCols);
}
uint64_t tile_grid(int dtype, bool back, int B, int T, int D) {
  return (uint64_t)B * ((D + kCols - 1) / kCols) * ((T - 1) / tile_tokens(dtype, back) + 1);
}
int run_tokens(int dtype, bool back) { return tile_tokens(dtype, back) / kRuns; }

hipError_t launch_tiles(const ccq_scan_params& p, void* workspace, hipStream_t stream) {
  const Tiles t = tiles_of(p.dtype, false, p.B, p.T, p.D, workspace);
  const hipError_t e = clear_tiles(t, tile_words(p.dtype, false, p.B, p.T, p.D), stream);
  if (e != hipSuccess) return e;
  const unsigned grid = (unsigned)tile_grid(p.dtype, false, p.B, p.T, p.D);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.complement) scan_tile_kernel<__bf16, true><<<grid, kThreads, 0, stream>>>(p, t);
    else scan_tile_kernel<__bf16, false><<<grid, kThreads, 0, stream>>>(p, t);
  } else {
    if (p.complement) scan_tile_kernel<float, true><<<grid, kThreads, 0, stream>>>(p, t);
    else scan_tile_kernel<float, false><<<grid, kThreads, 0, stream>>>(p, t);
  }
  return hipGetLastError();
}

// Whether the gradient forms the states again: not if they were kept, or where h0 is the only one.
bool forms_states(const ccq_scan_bwd_params& p) { return p.chunk_carry == nullptr && p.T > kChunk; }

// The gradient's tiles and, where the states are formed again, the forward's before them.
size_t tile_space(const ccq_scan_bwd_params& p) {
  const size_t back = tile_bytes(p.dtype, true, p.B, p.T, p.D);
  const size_t ahead = forms_states(p) ? tile_bytes(p.dtype, false, p.B, p.T, p.D) : 0;
  return back > ahead ? back : ahead;
}
size_t carry_bytes(int B, int T, int D) {
  return ((size_t)B * ((T + kChunk - 1) / kChunk) * D * 4 + 255) / 256 * 256;
}

}  // namespace

bool scan_grid_fits(int dtype, int B, int T, int D) {
  if (T <= kMostSteps) return true;  // at most 2^28 threads
  return grid_fits(T <= kChunk ? short_grid(B, D, runs_each(T, run_tokens(dtype, false))) : tile_grid(dtype, false, B, T, D), kThreads);
}

bool scan_backward_grid_fits(const ccq_scan_bwd_params& p) {
  const int each = runs_each(p.T, run_tokens(p.dtype, true));
  if (p.T <= kChunk && each <= kMostRuns) return grid_fits(short_grid(p.B, p.D, each), kThreads);
  return grid_fits(tile_grid(p.dtype, true, p.B, p.T, p.D), kThreads) &&
         (!forms_states(p) || grid_fits(tile_grid(p.dtype, false, p.B, p.T, p.D), kThreads));
}

size_t scan_workspace_bytes(const ccq_scan_params& p) { return p.T <= kMostSteps ? 0 : tile_bytes(p.dtype, false, p.B, p.T, p.D); }

hipError_t launch_scan(const ccq_scan_params& p, hipStream_t stream) {
  if (p.T > kMostSteps && p.T <= kChunk) {
    static_assert(kChunk <= kMostRuns * Run<__bf16, false>::n && kChunk <= kMostRuns * Run<float, false>::n, "short");
    const int per_row = (p.D + kCols - 1) / kCols;
    const int each = runs_each(p.T, run_tokens(p.dtype, false));
    const unsigned grid = (unsigned)short_grid(p.B, p.D, each);
    if (p.dtype == CCQ_DTYPE_BF16) {
      if (p.complement) scan_short_kernel<__bf16, true><<<grid, kThreads, 0, stream>>>(p, per_row, each);
      else scan_short_kernel<__bf16, false><<<grid, kThreads, 0, stream>>>(p, per_row, each);
    } else {
      if (p.complement) scan_short_kernel<float, true><<<grid, kThreads, 0, stream>>>(p, per_row, each);
      else scan_short_kernel<float, false><<<grid, kThreads, 0, stream>>>(p, per_row, each);
    }
    return hipGetLastError();
  }
  if (p.T > kMostSteps) return launch_tiles(p, p.workspace, stream);
  const unsigned grid = (unsigned)(((int64_t)p.B * (p.D / 8) + kStepThreads - 1) / kStepThreads);
  if (p.dtype == CCQ_DTYPE_BF16) scan_step_kernel<__bf16><<<grid, kStepThreads, 0, stream>>>(p);
  else scan_step_kernel<float><<<grid, kStepThreads, 0, stream>>>(p);
  return hipGetLastError();
}

size_t scan_backward_workspace_bytes(const ccq_scan_bwd_params& p) {
  return tile_space(p) + (forms_states(p) ? carry_bytes(p.B, p.T, p.D) : 0);
}

hipError_t launch_scan_backward(const ccq_scan_bwd_params& p, hipStream_t stream) {
  const float* carry = p.chunk_carry ? p.chunk_carry : p.h0;
  const int each = runs_each(p.T, run_tokens(p.dtype, true));
  if (p.T <= kChunk && each <= kMostRuns) {
    const int per_row = (p.D + kCols - 1) / kCols;
    const unsigned grid = (unsigned)short_grid(p.B, p.D, each);
    if (p.dtype == CCQ_DTYPE_BF16) {
      if (p.complement) scan_short_backward_kernel<__bf16, true><<<grid, kThreads, 0, stream>>>(p, carry, per_row, each);
      else scan_short_backward_kernel<__bf16, false><<<grid, kThreads, 0, stream>>>(p, carry, per_row, each);
    } else {
      if (p.complement) scan_short_backward_kernel<float, true><<<grid, kThreads, 0, stream>>>(p, carry, per_row, each);
      else scan_short_backward_kernel<float, false><<<grid, kThreads, 0, stream>>>(p, carry, per_row, each);
    }
    return hipGetLastError();
  }
  if (forms_states(p)) {
    // the forward once more, for its kept states alone
    float* kept = reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + tile_space(p));
    ccq_scan_params f{};
    f.dtype = p.dtype;
    f.B = p.B;
    f.T = p.T;
    f.D = p.D;
    f.complement = p.complement;
    f.x = p.x;
    f.log_alpha = p.log_alpha;
    f.x_stride_b = p.x_stride_b;
    f.x_stride_t = p.x_stride_t;
    f.la_stride_b = p.la_stride_b;
    f.la_stride_t = p.la_stride_t;
    f.lengths = p.lengths;
    f.h0 = p.h0;
    f.chunk_carry = kept;
    const hipError_t e = launch_tiles(f, p.workspace, stream);
    if (e != hipSuccess) return e;
    carry = kept;
  }
  const Tiles t = tiles_of(p.dtype, true, p.B, p.T, p.D, p.workspace);
  const hipError_t e = clear_tiles(t, tile_words(p.dtype, true, p.B, p.T, p.D), stream);
  if (e != hipSuccess) return e;
  const unsigned grid = (unsigned)tile_grid(p.dtype, true, p.B, p.T, p.D);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.complement) scan_backward_tile_kernel<__bf16, true><<<grid, kThreads, 0, stream>>>(p, carry, t);
    else scan_backward_tile_kernel<__bf16, false><<<grid, kThreads, 0, stream>>>(p, carry, t);
  } else {
    if (p.complement) scan_backward_tile_kernel<float, true><<<grid, kThreads, 0, stream>>>(p, carry, t);
    else scan_backward_tile_kernel<float, false><<<grid, kThreads, 0, stream>>>(p, carry, t);
  }
  return hipGetLastError();
}

}  // namespace ccq
