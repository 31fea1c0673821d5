// Gated linear recurrence h_t = alpha_t h_{t-1} + s_t x_t, channel by channel, and its gradient.
//
// A few operations an element: memory is the bound, so every input is read once.  A run of tokens acts
// on the state as h -> P h + q (P the product of its gates, q what the run adds), and runs compose:
// (P1, q1) then (P2, q2) is (P1 P2, P2 q1 + q2).  A workgroup takes a tile of 128 tokens by 64 channels
// into registers (a thread: four tokens of eight channels, one 16-byte load each in bf16), folds its
// tokens, joins the threads' pairs in LDS, and publishes the tile's pair; the state before the tile is
// the fold of the pairs of the tiles before it, and the tile's tokens are then walked again, from
// registers, to their outputs.  So a sequence is spread over as many workgroups as it has tiles and
// still read once: about 1/2 of the traffic of a pass that sums up the pieces before the pass that
// writes them would be spent on reading twice.
//
// Waiting.  A tile's pair depends on its own inputs alone and is published before its workgroup waits
// for any other, and tiles are handed out by a counter in the order of the recurrence, so whatever a
// workgroup waits for is already being worked on by one that waits for nothing first.  The folds go
// in a fixed order (16 or 64 tiles make a group, whose last tile publishes the group's pair), so two
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

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kChunk = 64;              // tokens between kept states
constexpr int kCols = 64;               // channels of a tile: one lane each where pairs are joined
constexpr int kRun = 4;                 // tokens of a thread
constexpr int kRuns = 8;                // runs of a wave, one behind the other
constexpr int kTile = kRun * kRuns * kWaves;  // tokens of a tile
static_assert(kTile % kChunk == 0, "tiles start at a kept state");

__device__ __forceinline__ int sequence_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// ---------------------------------------------------------------- gates

// alpha = exp(g) to about 2 units in the last place; 0 below about -87.  The hardware's 2^p takes the
// rounded product p = g log2(e), whose rounding, up to |p| / 2 units of the result, is made good to first
// order.
__device__ __forceinline__ float gate(float g) {
  constexpr float hi = 1.44269502162933349609f, lo = 1.92596299112661746887e-8f, ln2 = 0.693147180559945f;
  const float p = g * hi;
  const float rest = fmaf(g, lo, fmaf(g, hi, -p));
  const float a = __builtin_amdgcn_exp2f(p);
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

// alpha h, and alpha h + u, with 0 h = 0 for every h.
__device__ __forceinline__ float gated(float alpha, float h) { return alpha == 0.f ? 0.f : alpha * h; }
__device__ __forceinline__ float step(float alpha, float h, float u) { return alpha == 0.f ? u : fmaf(alpha, h, u); }

// The product of a run's gates, one more of them.
__device__ __forceinline__ float gates_product(float P, float alpha) { return alpha == 0.f ? -0.f : P * alpha; }

// ---------------------------------------------------------------- runs

struct Pair {
  float P, q;
};
__device__ __forceinline__ bool drops(float P) { return __float_as_int(P) < 0; }

// The state behind a run that found `h`.
__device__ __forceinline__ float through(float h, const Pair& r) {
  return drops(r.P) ? r.q : fmaf(fmaxf(r.P, FLT_MIN), h, r.q);
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

// ---------------------------------------------------------------- tiles

// The tiles of a call, in the order of the recurrence: all (sequence, 64 channels) columns of the first
// tokens, then of the next.  The workspace holds a counter, a pair for every tile and channel, and one
// for every group of tiles.
struct Tiles {
  int columns;   // B ceil(D / 64)
  int per_row;   // ceil(D / 64)
  int segments;  // ceil(T / kTile)
  int group;     // segments of a group
  unsigned* counter;
  uint64_t* pairs;   // [segments][columns][64]
  uint64_t* groups;  // [segments / group][columns][64]
};
constexpr size_t kCounterBytes = 256;

__host__ __device__ inline int group_of(int segments) { return segments <= 256 ? 16 : 64; }

constexpr uint64_t kEmpty = ~(uint64_t)0;  // no pair: the half of P is a NaN that is never published

__device__ __forceinline__ void publish(uint64_t* at, Pair r) {
  if (r.P != r.P) r.P = __int_as_float(0x7fc00000);
  const uint64_t word = ((uint64_t)__float_as_uint(r.q) << 32) | __float_as_uint(r.P);
  __hip_atomic_store(at, word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Pair unpack(uint64_t word) {
  return Pair{__uint_as_float((unsigned)word), __uint_as_float((unsigned)(word >> 32))};
}

// The fold of n published pairs, `stride` words apart.  Every lane of the wave waits with the others.
__device__ Pair fold_published(const uint64_t* from, int n, size_t stride) {
  Pair acc{1.f, 0.f};
  int polls = 0;
  for (int i = 0; i < n; i += 8) {
    uint64_t w[8];
    bool empty;
    do {
      empty = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = __hip_atomic_load(from + (size_t)min(i + j, n - 1) * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int j = 0; j < 8; ++j) empty |= (unsigned)w[j] == 0xffffffffu;
      if (__any(empty)) {
        if (++polls > (1 << 19)) return Pair{-0.f, __int_as_float(0x7fc00000)};
        __builtin_amdgcn_s_sleep(1);
      }
    } while (__any(empty));
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) acc = then(acc, unpack(w[j]));
  }
  return acc;
}

// The state before segment s of a column (lane = channel), from the pairs published so far; own: the
// segment's pair, which has been published; the last segment of a group publishes the group's.
__device__ float state_before(const Tiles& t, int s, int column, int lane, const Pair& own) {
  const size_t stride = (size_t)t.columns * kCols, at = (size_t)column * kCols + lane;
  const int g = s / t.group, first = g * t.group;
  const Pair here = fold_published(t.pairs + (size_t)first * stride + at, s - first, stride);
  if (s == first + t.group - 1) publish(t.groups + (size_t)g * stride + at, then(here, own));
  const Pair earlier = fold_published(t.groups + at, g, stride);
  return through(earlier.q, here);  // segment 0's pair holds the state before it and drops what it is given
}

__global__ __launch_bounds__(kThreads) void scan_clear_kernel(Tiles t, size_t words) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *t.counter = 0;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (size_t)gridDim.x * kThreads)
    t.pairs[i] = kEmpty;
}

// This workgroup's tile: by the counter where workgroups wait for one another.
__device__ __forceinline__ unsigned next_tile(const Tiles& t, unsigned* shared) {
  if (t.segments == 1) return blockIdx.x;
  if (threadIdx.x == 0) *shared = __hip_atomic_fetch_add(t.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return *shared;
}

template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads) void scan_tile_kernel(ccq_scan_params p, Tiles tiles) {
  __shared__ unsigned ticket;
  __shared__ __align__(16) Pair runs[kWaves][kRuns][kCols];   // every run's pair
  __shared__ __align__(16) float starts[kWaves][kRuns][kCols];  // the state before every run
  __shared__ Pair wave_pair[kWaves][kCols];
  __shared__ float tile_start[kCols];
  const unsigned tile = next_tile(tiles, &ticket);
  const int s = (int)(tile / (unsigned)tiles.columns), column = (int)(tile - (unsigned)s * tiles.columns);
  const int b = column / tiles.per_row, c_tile = (column - b * tiles.per_row) * kCols;
  const int n = sequence_length(p.lengths, b, p.T);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, oct = lane & 7, run = lane >> 3;
  const int t_wave = s * kTile + wave * kRun * kRuns, t0 = t_wave + run * kRun, c0 = c_tile + 8 * oct;

  float a[kRun][8], u[kRun][8];
  {
    const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c0;
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c0;
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      if (t0 + r < n && c0 < p.D) {
        load8(g + (int64_t)(t0 + r) * p.la_stride_t, a[r]);
        load8(x + (int64_t)(t0 + r) * p.x_stride_t, u[r]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[r][e] = u[r][e] = 0.f;  // the state stays as it is
      }
    }
  }
  Pair mine[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) mine[e] = Pair{1.f, 0.f};
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = a[r][e], alpha = gate(g);
      if constexpr (COMPLEMENT) u[r][e] *= one_minus(g, alpha);
      a[r][e] = alpha;
      mine[e].q = step(alpha, mine[e].q, u[r][e]);
      mine[e].P = gates_product(mine[e].P, alpha);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    *reinterpret_cast<f32x4*>(&runs[wave][run][8 * oct + e]) = f32x4{mine[e].P, mine[e].q, mine[e + 1].P, mine[e + 1].q};
  __syncthreads();
  // a lane takes a channel: the pairs in front of each of its wave's runs
  Pair before[kRuns], sum{1.f, 0.f};
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    before[r] = sum;
    sum = then(sum, runs[wave][r][lane]);
  }
  wave_pair[wave][lane] = sum;
  __syncthreads();
  const int c = c_tile + lane;
  if (wave == 0) {
    Pair all = wave_pair[0][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) all = then(all, wave_pair[w][lane]);
    float start = 0.f;
    if (s == 0) {
      start = p.h0 && c < p.D ? p.h0[(size_t)b * p.D + c] : 0.f;
      all = Pair{-0.f, through(start, all)};
    }
    if (tiles.segments > 1) {
      publish(tiles.pairs + ((size_t)s * tiles.columns + column) * kCols + lane, all);
      if (s > 0) start = state_before(tiles, s, column, lane, all);
    }
    tile_start[lane] = start;
    if (p.h_out && s == tiles.segments - 1 && c < p.D) p.h_out[(size_t)b * p.D + c] = through(start, all);
  }
  __syncthreads();
  float h = tile_start[lane];
  for (int w = 0; w < wave; ++w) h = through(h, wave_pair[w][lane]);
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const float start = through(h, before[r]);
    starts[wave][r][lane] = start;
    const int t = t_wave + r * kRun;
    if (p.chunk_carry && t % kChunk == 0 && t < n && c < p.D)
      p.chunk_carry[((size_t)b * ((p.T + kChunk - 1) / kChunk) + t / kChunk) * p.D + c] = start;
  }
  __syncthreads();
  if (p.y == nullptr || c0 >= p.D) return;
  float state[8];
  load8(&starts[wave][run][8 * oct], state);
  T* y = static_cast<T*>(p.y) + ((size_t)b * p.T + t0) * p.D + c0;
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) state[e] = step(a[r][e], state[e], u[r][e]);
    if (t0 + r < n) store8(y + (size_t)r * p.D, state);
  }
}

// The gradient: the same tiles from the end.  The adjoint that reaches a token from behind, d, becomes
// alpha (d + dy) in front of it, so a run acts on it as d -> P d + q with the run's own product of gates.
// The states are walked forward again, from the state kept before the tile.
template <typename T, bool COMPLEMENT>
__global__ __launch_bounds__(kThreads) void scan_backward_tile_kernel(ccq_scan_bwd_params p, const float* carry,
                                                                      Tiles tiles) {
  __shared__ unsigned ticket;
  __shared__ __align__(16) Pair runs[kWaves][kRuns][kCols];
  __shared__ __align__(16) float back[kWaves][kRuns][kCols];  // q of every run for the adjoint
  __shared__ Pair wave_pair[kWaves][kCols];
  __shared__ float wave_back[kWaves][kCols];
  __shared__ float tile_end[kCols];  // adjoint behind the tile
  const unsigned tile = next_tile(tiles, &ticket);
  const int order = (int)(tile / (unsigned)tiles.columns), column = (int)(tile - (unsigned)order * tiles.columns);
  const int s = tiles.segments - 1 - order;
  const int b = column / tiles.per_row, c_tile = (column - b * tiles.per_row) * kCols;
  const int n = sequence_length(p.lengths, b, p.T);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, oct = lane & 7, run = lane >> 3;
  const int t0 = s * kTile + wave * kRun * kRuns + run * kRun, c0 = c_tile + 8 * oct, c = c_tile + lane;

  float a[kRun][8], u[kRun][8], dy[kRun][8], sc[COMPLEMENT ? kRun : 1][8];
  {
    const T* g = static_cast<const T*>(p.log_alpha) + b * p.la_stride_b + c0;
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride_b + c0;
    const T* d = static_cast<const T*>(p.dy) + b * p.dy_stride_b + c0;
#pragma unroll
    for (int r = 0; r < kRun; ++r) {
      if (t0 + r < n && c0 < p.D) {
        load8(g + (int64_t)(t0 + r) * p.la_stride_t, a[r]);
        load8(x + (int64_t)(t0 + r) * p.x_stride_t, u[r]);
        load8(d + (int64_t)(t0 + r) * p.dy_stride_t, dy[r]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[r][e] = u[r][e] = dy[r][e] = 0.f;
      }
    }
  }
  float h_tile = 0.f;  // state before the tile
  if (s * kTile < n && c < p.D)
    h_tile = carry[((size_t)b * ((p.T + kChunk - 1) / kChunk) + s * (kTile / kChunk)) * p.D + c];

  Pair mine[8];
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mine[e] = Pair{1.f, 0.f};
    q[e] = 0.f;
  }
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = a[r][e], alpha = gate(g);
      a[r][e] = alpha;
      float in = u[r][e];
      if constexpr (COMPLEMENT) {
        sc[r][e] = one_minus(g, alpha);
        in *= sc[r][e];
      }
      mine[e].q = step(alpha, mine[e].q, in);
      mine[e].P = gates_product(mine[e].P, alpha);
    }
  }
#pragma unroll
  for (int r = kRun - 1; r >= 0; --r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = gated(a[r][e], q[e] + dy[r][e]);
  }
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    *reinterpret_cast<f32x4*>(&runs[wave][run][8 * oct + e]) = f32x4{mine[e].P, mine[e].q, mine[e + 1].P, mine[e + 1].q};
  store8(&back[wave][run][8 * oct], q);
  __syncthreads();
  // a lane takes a channel: the pairs in front of each of its wave's runs, and behind each for the adjoint
  Pair before[kRuns], behind[kRuns], sum{1.f, 0.f}, rsum{1.f, 0.f};
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    before[r] = sum;
    sum = then(sum, runs[wave][r][lane]);
  }
#pragma unroll
  for (int r = kRuns - 1; r >= 0; --r) {
    behind[r] = rsum;
    rsum = then(rsum, Pair{runs[wave][r][lane].P, back[wave][r][lane]});
  }
  wave_pair[wave][lane] = sum;
  wave_back[wave][lane] = rsum.q;
  __syncthreads();
  if (wave == 0) {
    Pair all{1.f, 0.f};
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w) all = then(all, Pair{wave_pair[w][lane].P, wave_back[w][lane]});
    float end = 0.f;
    if (order == 0) {
      end = p.dh_out && c < p.D ? p.dh_out[(size_t)b * p.D + c] : 0.f;
      all = Pair{-0.f, through(end, all)};
    }
    if (tiles.segments > 1) {
      publish(tiles.pairs + ((size_t)order * tiles.columns + column) * kCols + lane, all);
      if (order > 0) end = state_before(tiles, order, column, lane, all);
    }
    tile_end[lane] = end;
    if (p.dh0 && s == 0 && c < p.D) p.dh0[(size_t)b * p.D + c] = through(end, all);
  }
  __syncthreads();
  float h = h_tile, d = tile_end[lane];
  for (int w = 0; w < wave; ++w) h = through(h, wave_pair[w][lane]);
  for (int w = kWaves - 1; w > wave; --w) d = through(d, Pair{wave_pair[w][lane].P, wave_back[w][lane]});
  // every run's state in front of it and adjoint behind it, where its pair stood
#pragma unroll
  for (int r = 0; r < kRuns; ++r) runs[wave][r][lane] = Pair{through(h, before[r]), through(d, behind[r])};
  __syncthreads();
  if (c0 >= p.D) return;
  float state[8], adj[8];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(&runs[wave][run][8 * oct + e]);
    state[e] = v[0];
    adj[e] = v[1];
    state[e + 1] = v[2];
    adj[e + 1] = v[3];
  }
  // u becomes what log_alpha's gradient takes from each token: the state before it, less the input
#pragma unroll
  for (int r = 0; r < kRun; ++r) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = u[r][e];
      u[r][e] = COMPLEMENT ? state[e] - x : state[e];
      state[e] = step(a[r][e], state[e], COMPLEMENT ? sc[r][e] * x : x);
    }
  }
  const size_t at = ((size_t)b * p.T + t0) * p.D + c0;
  T* dx = static_cast<T*>(p.dx) + at;
  T* dg = static_cast<T*>(p.dlog_alpha) + at;
#pragma unroll
  for (int r = kRun - 1; r >= 0; --r) {
    const bool live = t0 + r < n;
    float ox[8], og[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float full = adj[e] + dy[r][e];
      ox[e] = live ? (COMPLEMENT ? sc[r][e] * full : full) : 0.f;
      adj[e] = gated(a[r][e], full);
      og[e] = live ? gated(a[r][e], full * u[r][e]) : 0.f;
    }
    if (t0 + r < p.T) {
      store8(dx + (size_t)r * p.D, ox);
      store8(dg + (size_t)r * p.D, og);
    }
  }
}

// A few tokens: eight channels a thread, one token behind the other.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ccq_scan_params p) {
  const int per_row = p.D / 8;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
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
      const float alpha = gate(gt[e]);
      h[e] = step(alpha, h[e], p.complement ? xt[e] * one_minus(gt[e], alpha) : xt[e]);
    }
    store8(y + (int64_t)t * p.D, h);
  }
  if (p.h_out) store8(p.h_out + (int64_t)b * p.D + c, h);
}

// ---------------------------------------------------------------- launches

Tiles tiles_of(int B, int T, int D, void* workspace) {
  Tiles t{};
  t.per_row = (D + kCols - 1) / kCols;
  t.columns = B * t.per_row;
  t.segments = (T + kTile - 1) / kTile;
  t.group = group_of(t.segments);
  t.counter = static_cast<unsigned*>(workspace);
  t.pairs = reinterpret_cast<uint64_t*>(static_cast<unsigned char*>(workspace) + kCounterBytes);
  t.groups = t.pairs + (size_t)t.segments * t.columns * kCols;
  return t;
}
size_t tile_words(int B, int T, int D) {
  const size_t segments = (size_t)((T + kTile - 1) / kTile);
  if (segments == 1) return 0;
  return (segments + segments / group_of((int)segments)) * B * ((D + kCols - 1) / kCols) * kCols;
}
size_t tile_bytes(int B, int T, int D) {
  const size_t words = tile_words(B, T, D);
  return words ? kCounterBytes + words * sizeof(uint64_t) : 0;
}

hipError_t clear_tiles(const Tiles& t, size_t words, hipStream_t stream) {
  if (words == 0) return hipSuccess;
  const size_t blocks = (words + kThreads * 4 - 1) / (kThreads * 4);
  scan_clear_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), kThreads, 0, stream>>>(t, words);
  return hipGetLastError();
}

// Up to this many tokens go one behind the other in a thread.
constexpr int kMostSteps = 8;

hipError_t launch_tiles(const ccq_scan_params& p, void* workspace, hipStream_t stream) {
  const Tiles t = tiles_of(p.B, p.T, p.D, workspace);
  const hipError_t e = clear_tiles(t, tile_words(p.B, p.T, p.D), stream);
  if (e != hipSuccess) return e;
  const unsigned grid = (unsigned)((int64_t)t.columns * t.segments);
  if (p.dtype == CCQ_DTYPE_BF16) {
    if (p.complement) scan_tile_kernel<__bf16, true><<<grid, kThreads, 0, stream>>>(p, t);
    else scan_tile_kernel<__bf16, false><<<grid, kThreads, 0, stream>>>(p, t);
  } else {
    if (p.complement) scan_tile_kernel<float, true><<<grid, kThreads, 0, stream>>>(p, t);
    else scan_tile_kernel<float, false><<<grid, kThreads, 0, stream>>>(p, t);
  }
  return hipGetLastError();
}

size_t carry_bytes(int B, int T, int D) {
  return ((size_t)B * ((T + kChunk - 1) / kChunk) * D * 4 + 255) / 256 * 256;
}

}  // namespace

size_t scan_workspace_bytes(const ccq_scan_params& p) { return p.T <= kMostSteps ? 0 : tile_bytes(p.B, p.T, p.D); }

hipError_t launch_scan(const ccq_scan_params& p, hipStream_t stream) {
  if (p.T > kMostSteps) return launch_tiles(p, p.workspace, stream);
  const unsigned grid = (unsigned)(((int64_t)p.B * (p.D / 8) + kThreads - 1) / kThreads);
  if (p.dtype == CCQ_DTYPE_BF16) scan_step_kernel<__bf16><<<grid, kThreads, 0, stream>>>(p);
  else scan_step_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

size_t scan_backward_workspace_bytes(const ccq_scan_bwd_params& p) {
  return tile_bytes(p.B, p.T, p.D) + (p.chunk_carry ? 0 : carry_bytes(p.B, p.T, p.D));
}

hipError_t launch_scan_backward(const ccq_scan_bwd_params& p, hipStream_t stream) {
  const float* carry = p.chunk_carry;
  const size_t tile_space = tile_bytes(p.B, p.T, p.D);
  if (carry == nullptr) {
    // the forward once more, for its kept states alone
    float* kept = reinterpret_cast<float*>(static_cast<unsigned char*>(p.workspace) + tile_space);
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
  const Tiles t = tiles_of(p.B, p.T, p.D, p.workspace);
  const hipError_t e = clear_tiles(t, tile_words(p.B, p.T, p.D), stream);
  if (e != hipSuccess) return e;
  const unsigned grid = (unsigned)((int64_t)t.columns * t.segments);
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
