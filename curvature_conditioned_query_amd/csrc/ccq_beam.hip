// Beam search: the best continuations of every request over its beams and the vocabulary, and the
// reordering of the states that the beams carry.
//
// Selection reads the logits once.  beam_rows_kernel gives a workgroup a stretch of one beam's row: it
// leaves the stretch's M best logits, in order, and its part of the normaliser sum exp(x - top).
// beam_join_kernel, one workgroup a request, joins the parts into each beam's normaliser and picks the M
// best continuations out of the stretches' lists.
//
// Picking M of many needs no sort.  A workgroup goes through its stretch in pieces held in registers (32
// logits a thread, 8 where there are few rows).  In the first, the (M + 1)-th best of the threads' maxima, the
// bound, is found bit by bit; at least M logits reach it, and few lie above it.  Those, and in the later pieces
// whatever lies above the bound, go into a list of their wave's own, in no order, without a word between the
// waves; a list that fills up (a row that rises, a mask over the first tokens) is thinned to its M best, which
// raise the wave's bound.  Should fewer than M logits lie above the bound, as in a row of few values or under
// a mask that leaves few tokens, the lowest tokens at the bound itself are looked up at the end.  The lists are
// put in order by counting, for each candidate, the greater ones; that is quadratic, so longer lists are
// thinned first.  A stretch of one piece takes its bound from the waves' own maxima, sorted and joined more
// loosely: 7.9 against 8.8 us for four rows of 32,000, where for 256 rows of 131,071, in stretches of four
// pieces, it is 28.5 against 26.3.
//
// Measured, 32 requests of 8 beams over 131,071 tokens, M = 16, bf16: 26 us for the rows (67 MB, 2.6 TB/s: the
// vector units are busy for half of it, and with one batch of workgroups of four pieces each the first loads, the
// bound and the last ranking stand alone) and 6 for the join.  464 rows of 23,341 in fp32, M = 8: 21 us for 43 MB and 5,
// for the same reasons with stretches of one piece.  Four rows of 32,000 in fp32: 7 and 5 us, latencies throughout.
//
// Scores of different beams meet in the comparison, so the normaliser has to be good to more than
// fp32: the candidates, which carry most of a peaked distribution, are left out of the fp32 sum and added
// in 64 bits, and the threads' sums of the rest, 2^((x - top) log2(e)), are joined in 64 bits.  The difference
// comes first, so that a term's error goes by its distance from the top and not by the logits' size, and what lies
// far below is 0 (x log2(e) - top log2(e) as one fused operation saves an instruction a logit, and is wrong by the
// product's rounding: 0.01 % for logits at 10^4, everything from 10^9 on).
#include <float.h>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The workspace: a part of the normaliser and a list of M logits for every (row, stretch).
struct Part {
  double sum;  // sum of exp(x - top) over the stretch
  float top;   // its largest logit
  int pad;
};
struct Pick {
  float logit;
  int token;  // -1: the stretch has no more
};

struct BeamWork {
  Part* parts;
  Pick* picks;
};
__host__ __device__ inline size_t parts_bytes(size_t lists) { return lists * sizeof(Part); }

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
  return x;
}

// A logit as it counts: NaN as -inf (the maximum with a NaN is the other operand), +inf as the largest
// finite number.
__device__ __forceinline__ float as_counted(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

constexpr float kLog2e = 1.44269502162933349609f;

// A row's beam: 0 goes on, 1 finished, 2 dead (its score is -inf or NaN, finished or not: all its continuations are
// at -inf, the pad token's too).  Both loads are made, so that neither waits for the other.
__device__ __forceinline__ int beam_kind(const ccq_beam_params& p, int row, float& score) {
  score = p.scores[row];
  const bool finished = p.finished && p.finished[row];
  return score > -INFINITY ? (finished ? 1 : 0) : 2;
}

// 16 bytes from any element on: a row starts where the one before ends, at an odd address for an odd
// vocabulary.  Which thread holds a token must not depend on that address: beams with equal logits have
// to get equal normalisers to the last bit, or their ties would fall either way.
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

// A thread's logits of a piece as they are stored: vectors of 16 bytes, 256 vectors apart.
template <typename T, int NV>
struct Raw {
  static constexpr int VE = 16 / sizeof(T);
  typedef typename Any<T>::type V;
  V v[NV];
  // From token `first` on, of the piece that begins at token `at`.
  __device__ __forceinline__ void load(const T* src, int first, int at, int V_all) {
    if (at + kThreads * VE * NV <= V_all) {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = __builtin_nontemporal_load(reinterpret_cast<const V*>(src + first + j * (kThreads * VE)));
      return;
    }
    // the row ends in this piece: vectors inside it, then the one across its end
    if (V_all >= VE) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        v[j] = *reinterpret_cast<const V*>(src + min(first + j * (kThreads * VE), V_all - VE));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v0 = first + j * (kThreads * VE);
      if (v0 < V_all && v0 + VE > V_all) {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[j][e] = src[min(v0 + e, V_all - 1)];
      }
    }
  }
  // Logits g .. g + 7 of the thread; -inf behind the row.
  __device__ __forceinline__ void get(float (&x)[8], int g, int first, bool whole, int V_all) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[(g + i) / VE][(g + i) % VE];
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (first + (g + i) / VE * (kThreads * VE) + (g + i) % VE >= V_all) x[i] = -INFINITY;
    }
  }
};

// Sorts 64 lanes' values, the largest first.
__device__ __forceinline__ float sort_lanes(float v, int lane) {
#pragma unroll
  for (int size = 2; size <= 64; size *= 2) {
#pragma unroll
    for (int gap = size / 2; gap > 0; gap /= 2) {
      const float o = __shfl_xor(v, gap, 64);
      const bool larger = ((lane & gap) == 0) == ((lane & size) == 0 || size == 64);
      v = larger ? fmaxf(v, o) : fminf(v, o);
    }
  }
  return v;
}

// Whether logit a at token va comes before b at vb.
__device__ __forceinline__ bool before(float a, int va, float b, int vb) { return a > b || (a == b && va < vb); }

// The part and the picks of a stretch with NaN or +inf among its logits, which count as as_counted() says: one
// pass through memory for each pick, all of the sum in 64 bits.  shared: room for 8 words.
template <typename T>
__device__ __attribute__((noinline)) void careful_stretch(const T* src, int begin, int end, int M, Pick* picks, Part* part,
                                                          float* shared) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int* tokens = reinterpret_cast<int*>(shared) + kWaves;
  float x0 = INFINITY, top = -INFINITY;  // the pick before: everything comes after +inf
  int v0 = -1;
  for (int m = 0; m < M; ++m) {
    float x = -INFINITY;
    int v = 0x7fffffff;
    for (int i = begin + (int)threadIdx.x; i < end; i += kThreads) {
      const float o = as_counted(to_f32(src[i]));
      if (before(x0, v0, o, i) && before(o, i, x, v)) {
        x = o;
        v = i;
      }
    }
    for (int off = 32; off > 0; off >>= 1) {
      const float ox = __shfl_xor(x, off, 64);
      const int ov = __shfl_xor(v, off, 64);
      if (before(ox, ov, x, v)) {
        x = ox;
        v = ov;
      }
    }
    __syncthreads();
    if (lane == 0) {
      shared[wave] = x;
      tokens[wave] = v;
    }
    __syncthreads();
    x = shared[0];
    v = tokens[0];
    for (int w = 1; w < kWaves; ++w)
      if (before(shared[w], tokens[w], x, v)) {
        x = shared[w];
        v = tokens[w];
      }
    if (m == 0) top = x;
    if (threadIdx.x == 0) picks[m] = v == 0x7fffffff ? Pick{-INFINITY, -1} : Pick{x, v};
    x0 = x;
    v0 = v;
  }
  double s = 0.0;
  if (top > -INFINITY)
    for (int i = begin + (int)threadIdx.x; i < end; i += kThreads) s += exp((double)as_counted(to_f32(src[i])) - (double)top);
  s = wave_sum(s);
  double* sums = reinterpret_cast<double*>(shared);
  __syncthreads();
  if (lane == 0) sums[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) *part = Part{(sums[0] + sums[1]) + (sums[2] + sums[3]), top, 0};
}

// Picks n .. M - 1: the lowest tokens at `value`.
template <typename T>
__device__ __attribute__((noinline)) void fill_picks(const T* src, int begin, int end, float value, int n, int M, Pick* picks,
                                                     int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int at = begin; at < end && n < M; at += kThreads) {
    const int i = at + (int)threadIdx.x;
    const bool is = i < end && to_f32(src[i]) == value;
    const uint64_t all = __ballot(is);
    if (lane == 0) counts[wave] = __popcll(all);
    __syncthreads();
    int to = n + __popcll(all & ((1ull << lane) - 1));
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) to += counts[w];
      n += counts[w];
    }
    if (is && to < M) picks[to] = Pick{value, i};
    __syncthreads();
  }
  for (int i = n + (int)threadIdx.x; i < M; i += kThreads) picks[i] = Pick{-INFINITY, -1};
}

// A logit as a number of the same order, and back; with its token as one number, the greater comes first.
__device__ __forceinline__ unsigned to_word(float x) {
  const unsigned b = __float_as_uint(x + 0.f);  // -0 ties with 0
  return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float word_logit(unsigned b) { return __uint_as_float((int)b < 0 ? b & 0x7fffffffu : ~b); }
__device__ __forceinline__ uint64_t to_key(float x, int token) { return (uint64_t)to_word(x) << 32 | (unsigned)~token; }
__device__ __forceinline__ float key_logit(uint64_t key) { return word_logit((unsigned)(key >> 32)); }
__device__ __forceinline__ int key_token(uint64_t key) { return (int)~(unsigned)key; }

// How many of n keys are greater; behind them stand seven that are 0, the least there is.
__device__ __forceinline__ int count_greater(const uint64_t* keys, int n, uint64_t mine) {
  int r = 0;
  for (int j = 0; j < n; j += 8) {
    uint64_t k[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = keys[j + i];
#pragma unroll
    for (int i = 0; i < 8; ++i) r += k[i] > mine ? 1 : 0;
  }
  return r;
}

// A number that `count` of the threads' words reach and, unless words are equal, no more do; words that differ
// in their BITS highest bits at most.
template <int BITS>
__device__ __forceinline__ unsigned reached_by(const unsigned (&words)[kThreads], int count) {
  unsigned w[kWaves], reached = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) w[i] = words[(threadIdx.x & 63) + 64 * i];
  for (int bit = 30; bit >= 32 - BITS; bit -= 2) {
    int n[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
#pragma unroll
      for (unsigned d = 1; d < 4; ++d) n[d] += __popcll(__builtin_amdgcn_ballot_w64(w[i] >= (reached | d << bit)));
    const int digit = n[3] >= count ? 3 : n[2] >= count ? 2 : n[1] >= count ? 1 : 0;
    reached |= (unsigned)digit << bit;
    if (digit && (digit == 3 ? n[3] : digit == 2 ? n[2] : n[1]) == count) break;
  }
  // the bits that none differs in are ones in the word of a negative number: without them the number would lie
  // just below the one it stands for, and a row of one negative value would be all candidates
  if (BITS < 32 && reached < 0x80000000u) reached |= (1u << (32 - BITS)) - 1;
  return reached;
}

// How many of the lanes in `mask` stand before this one.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
}

// A wave's candidates in LDS, in the order they were found.  Before a group of eight logits a lane is looked
// at, there is room for all of them.
constexpr int kGroup = 8;
constexpr int kHeld = 64 * kGroup + 128;
struct Held {
  uint64_t key[(kHeld + 8 + 255) / 256 * 256];
};
__device__ __forceinline__ void wave_fence() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// Thins a wave's n >= M candidates to the M best, in the order they stand; returns the least of their logits.
// The others are added to gone, which counts from ref.  All keys differ, so some number is reached by M of
// them alone: its bits are found from the highest down.
// The keys are read again for every bit: held in registers they would cost the kernel a workgroup a CU.
__device__ __forceinline__ float thin(Held& held, int n, int M, double& gone, float& ref) {
  const int lane = threadIdx.x & 63, padded = (n + 255) & ~255;
  for (int i = n + lane; i < padded; i += 64) held.key[i] = 0;
  wave_fence();
  float highest = -INFINITY, lowest = INFINITY;
  for (int i = lane; i < n; i += 64) {
    const float logit = key_logit(held.key[i]);
    highest = fmaxf(highest, logit);
    lowest = fminf(lowest, logit);
  }
  highest = wave_max(highest);
  lowest = -wave_max(-lowest);
  if (ref > -INFINITY) gone *= exp((double)ref - (double)highest);
  ref = highest;
  // the highest bits are those that all logits share
  const uint64_t ends = to_key(highest, -1) ^ to_key(lowest, 0);
  int bit = 63 - __clzll((long long)ends);
  uint64_t reached = to_key(lowest, 0) >> bit >> 1 << bit << 1;
  for (; bit >= 0; --bit) {
    const uint64_t higher = reached | 1ull << bit;
    int count = 0;
    for (int i = lane; i < padded; i += 256) {
      uint64_t key[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) key[j] = held.key[i + 64 * j];
#pragma unroll
      for (int j = 0; j < 4; ++j) count += __popcll(__builtin_amdgcn_ballot_w64(key[j] >= higher));
    }
    if (count >= M) reached = higher;
    if (count == M) break;
  }
  int to = 0;
  float least = INFINITY;
  for (int i = 0; i < n; i += 64) {
    const bool is = i + lane < n;
    const uint64_t key = held.key[min(i + lane, n - 1)];
    const float logit = key_logit(key);
    const bool stays = is && key >= reached;
    const uint64_t all = __builtin_amdgcn_ballot_w64(stays);
    wave_fence();  // read before it is written: places behind these 64 stay
    if (stays) {
      held.key[to + lanes_below(all)] = key;
      least = fminf(least, logit);
    } else if (is) {
      gone += exp((double)logit - (double)highest);
    }
    to += __popcll(all);
  }
  wave_fence();
  return -wave_max(-least);
}

// Tokens of a piece: 256 threads hold E each, in vectors of VE, vector j from token (j 256 + tid) VE of the
// piece on.  The logits are taken as they come: a NaN shows in the sum and +inf among the candidates, and a
// stretch that has one is left to careful_stretch.
// ONE: a stretch is one piece.
template <typename T, int E, bool ONE>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 1) void beam_rows_kernel(ccq_beam_params p, int stretches, int pieces, BeamWork work) {
  constexpr int VE = 16 / sizeof(T), NV = E / VE, G = kGroup;  // a group of logits has a maximum of its own
  constexpr int PIECE = kThreads * E;
  __shared__ __align__(16) Held held[kWaves];
  __shared__ __align__(16) float few[8];
  __shared__ unsigned words[kThreads];
  __shared__ float bounds[kWaves], tops[kWaves], froms[kWaves];
  __shared__ int counts[kWaves];
  __shared__ double sums[kWaves];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), M = p.M;
  const int row = blockIdx.x / stretches, stretch = blockIdx.x - row * stretches;
  const size_t list = blockIdx.x;
  Pick* picks = work.picks + list * M;

  const T* src = static_cast<const T*>(p.logits) + (int64_t)row * p.logits_stride;
  const int begin = stretch * pieces * PIECE, end = min(p.V, begin + pieces * PIECE);
  Raw<T, NV> ahead;
  ahead.load(src, begin + tid * VE, begin, p.V);  // under way while the beam's kind is found
  float score;
  const int kind = beam_kind(p, row, score);
  if (kind != 0) {
    // a finished beam's one continuation and then, as a dead beam's, tokens in order at -inf
    for (int i = tid; i < M; i += kThreads) {
      Pick k{-INFINITY, -1};
      if (stretch == 0) {
        if (kind == 2) k.token = i;
        else if (i == 0) k = Pick{0.f, p.pad_token};
        else k.token = i - 1 < p.pad_token ? i - 1 : i;
        if (k.token >= p.V) k.token = -1;
      }
      picks[i] = k;
    }
    if (tid == 0) work.parts[list] = Part{0.0, -INFINITY, 0};
    return;
  }

  float bound = -INFINITY;  // candidates lie above it
  float top = -INFINITY;    // the sum of the others counts from here: no logit of theirs lies above it
  double part = 0.0;        // a thread's 32 logits of a piece go into it together, summed in fp32
  double gone = 0.0;        // of candidates that were thinned out, counted from ref; and of part before top moved
  float ref = -INFINITY;
  int n = 0;                // candidates of the wave

  for (int at = begin; at < end; at += PIECE) {
    const int first = at + tid * VE;  // token of the thread's first logit: the rest follow by constants
    const bool whole = at + PIECE <= p.V;
    const Raw<T, NV> raw = ahead;
    if (at + PIECE < end) ahead.load(src, first + PIECE, at + PIECE, p.V);
    if (at == begin) {
      float mine = -INFINITY;
#pragma unroll
      for (int g = 0; g < E; g += G) {
        float x[G];
        raw.get(x, g, first, whole, p.V);
#pragma unroll
        for (int i = 0; i < G; ++i) mine = fmaxf(mine, x[i]);
      }
      if constexpr (ONE) {
        // no later piece that a tighter bound would spare candidates: the least of the waves' own (M / 4 + 1)-th best, of a short stretch of those
        // whose every thread holds logits
        const int full = max(1, min(kWaves, (end - begin) / (64 * VE)));
        const float sorted = sort_lanes(mine, lane);
        if (lane == 0) tops[wave] = sorted;
        if (lane == min((M + full - 1) / full, 63)) bounds[wave] = sorted;
        __syncthreads();
        bound = bounds[0];
        for (int w = 1; w < full; ++w) bound = fminf(bound, bounds[w]);
      } else {
        words[tid] = to_word(mine);
        mine = wave_max(mine);
        if (lane == 0) tops[wave] = mine;
        __syncthreads();
        bound = word_logit(max(reached_by<sizeof(T) * 8>(words, M + 1), to_word(-INFINITY)));
      }
      top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    }
    float higher = bound;  // for the pieces to come: this one's later groups hold tokens on either side of a tie
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < E; g += G) {
      float x[G];
      raw.get(x, g, first, whole, p.V);
      float most = x[0];
#pragma unroll
      for (int i = 1; i < G; ++i) most = fmaxf(most, x[i]);
      if (__builtin_amdgcn_ballot_w64(most > bound)) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const uint64_t all = __builtin_amdgcn_ballot_w64(x[i] > bound);
          if (all == 0) continue;
          if (x[i] > bound) {
            const int to = n + lanes_below(all);
            held[wave].key[to] = to_key(x[i], first + (g + i) / VE * (kThreads * VE) + (g + i) % VE);
            x[i] = -INFINITY;  // not in the fp32 sum
          }
          n += __popcll(all);
        }
        if (n > kHeld - 64 * G) {
          higher = thin(held[wave], n, M, gone, ref);
          n = M;
          if (!ONE && higher > top) {
            // logits up to here are no candidates from now on, and may lie far above the first piece's top: what
            // was summed goes to the thinned ones' sum, and the fp32 sum begins anew
            gone += (part + (double)((sum[0] + sum[1]) + (sum[2] + sum[3]))) * exp((double)top - (double)ref);
            part = 0.0;
            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
            top = higher;
          }
        }
      }
      if (top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < G; ++i) sum[i & 3] += __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
      } else {
        // nothing above -inf in the first piece, and no sum to show a NaN
#pragma unroll
        for (int i = 0; i < G; ++i) sum[0] = x[i] != x[i] ? x[i] : sum[0];
      }
    }
    part += (double)((sum[0] + sum[1]) + (sum[2] + sum[3]));
    bound = higher;
  }
  bool careful = part != part || gone != gone || top == INFINITY;
  if (n > 128) {
    thin(held[wave], n, M, gone, ref);
    n = M;
  }
  if (lane < 8) held[wave].key[n + lane] = 0;
  wave_fence();
  float most = -INFINITY;  // of the wave's candidates
  for (int i = lane; i < n; i += 64) most = fmaxf(most, key_logit(held[wave].key[i]));
  most = wave_max(most);
  careful |= most == INFINITY;
  // the wave's part of the normaliser, from the greater of the two on
  const float from = fmaxf(top, most);
  double sum = 0.0;
  if (from > -INFINITY) {
    if (top > -INFINITY) sum = part * exp((double)top - (double)from);
    for (int i = lane; i < n; i += 64) sum += exp((double)key_logit(held[wave].key[i]) - (double)from);
    if (ref > -INFINITY) sum += gone * exp((double)ref - (double)from);
  }
  sum = wave_sum(sum);
  if (lane == 0) {
    sums[wave] = sum;
    froms[wave] = from;
    counts[wave] = n;
  }
  if (__syncthreads_or(careful)) {
    careful_stretch(src, begin, end, M, picks, work.parts + list, few);
    return;
  }
  // all waves' candidates in order: a thread's against every other
  const int m = counts[0] + counts[1] + counts[2] + counts[3];
  for (int i = tid; i < m; i += kThreads) {
    int w = 0, at = i;
    while (at >= counts[w]) at -= counts[w++];
    const uint64_t key = held[w].key[at];
    int r = 0;
    for (int o = 0; o < kWaves; ++o) r += count_greater(held[o].key, counts[o], key);
    if (r < M) picks[r] = Pick{key_logit(key), key_token(key)};
  }
  if (tid < kWaves) {
    const float highest = fmaxf(fmaxf(froms[0], froms[1]), fmaxf(froms[2], froms[3]));
    double s = froms[tid] > -INFINITY ? sums[tid] * exp((double)froms[tid] - (double)highest) : 0.0;
    s += __shfl_xor(s, 1, 64);
    s += __shfl_xor(s, 2, 64);
    if (tid == 0) work.parts[list] = Part{s, highest, 0};
  }
  if (m < M) {
    __syncthreads();
    fill_picks(src, begin, end, bound, m, M, picks, counts);
  }
}

// A beam's part of its continuations' scores: score - log sum exp(x - top), and top.  The logit meets
// top before anything else does, so large logits cancel exactly.
struct BeamBase {
  double rest, top;
  int kind;
};
__device__ __forceinline__ double pick_total(const Pick& k, const BeamBase& b) {
  if (b.kind == 2 || !(k.logit > -INFINITY)) return -INFINITY;
  return b.rest + ((double)k.logit - b.top) + 0.0;  // never -0, which orders below 0
}

// A total as an unsigned number of the same order.
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return (int64_t)b < 0 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ double key_order(uint64_t key) {
  return __longlong_as_double((long long)((int64_t)key < 0 ? key & 0x7fffffffffffffffull : ~key));
}

// Picks M of a request's lists.  Of the lists' entries at one depth, the best M / depth give a bound that M
// continuations reach and few others do; the depth is such that one list in eight speaks for it, beams being
// unlike (8 beams of 4 lists, M = 16: 20 to 70 reach it, 6.5 us; with half of the lists, their heads, 70 to 140,
// 10 us).  Where many reach it all the same, as at M = 64 of 32 lists (24 us, 21 without the attempt):
// eight bits at a time of the total and then of the place, the continuations that agree with the M-th best so
// far are counted by their next digit, until few enough are left with those above them to be ranked by counting.
constexpr int kRanked = 128;
constexpr int kHeads = 256;  // most lists of a request
__global__ __launch_bounds__(kThreads) void beam_join_kernel(ccq_beam_params p, int stretches, BeamWork work) {
  __shared__ BeamBase base[kBeamMaxBeams];
  __shared__ int bins[256];
  __shared__ int digit, above, inside, found;
  __shared__ unsigned long long least;
  __shared__ __align__(16) uint64_t heads[kHeads + 8];
  __shared__ uint64_t keys[kRanked + 4];
  __shared__ unsigned places[kRanked + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = blockIdx.x, K = p.K, M = p.M;
  const int lists = K * stretches, entries = lists * M;
  const Part* parts = work.parts + (size_t)n * lists;
  const Pick* picks = work.picks + (size_t)n * lists * M;

  // as many lanes a beam as it has stretches: the exponentials and logarithms in 64 bits, 2 us a time, are then
  // formed for many beams at once (12 beams of one stretch: 10.8 us with a wave a beam, 7.6)
  int width = 1;
  while (width < stretches && width < 64) width *= 2;
  for (int k = tid / width; k < (K + kThreads / width - 1) / (kThreads / width) * (kThreads / width); k += kThreads / width) {
    const int mine = tid & (width - 1), row = n * K + min(k, K - 1);
    const Part* at = parts + min(k, K - 1) * stretches;
    const Part first = at[min(mine, stretches - 1)];
    float score;
    int kind = beam_kind(p, row, score);
    if (k >= K) kind = 2;
    BeamBase b{score, 0.0, kind};
    float top = -INFINITY;
    if (kind == 0) {
      if (mine < stretches) top = first.top;
      for (int c = mine + width; c < stretches; c += width) top = fmaxf(top, at[c].top);
    }
    for (int off = width / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    double s = 0.0;
    if (top > -INFINITY) {
      if (mine < stretches && first.top > -INFINITY) s = first.sum * exp((double)first.top - (double)top);
      for (int c = mine + width; c < stretches; c += width) {
        const Part q = at[c];
        if (q.top > -INFINITY) s += q.sum * exp((double)q.top - (double)top);
      }
    }
    for (int off = width / 2; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
    if (top > -INFINITY) {
      b.rest -= log(s);
      b.top = top;
    }
    if (mine == 0 && k < K) base[k] = b;
  }
  if (tid == 0) {
    found = 0;
    least = ~0ull;
  }
  __syncthreads();

  auto value = [&](int i, const Pick& q, double& total, unsigned& place) {
    const int k = i / (M * stretches);
    total = pick_total(q, base[k]);
    place = (unsigned)k * (unsigned)p.V + (unsigned)q.token;
    return q.token >= 0;
  };
  auto entry = [&](int i, double& total, unsigned& place) { return value(i, picks[i], total, place); };
  bool few = false;  // those that reach the bound
  if (M <= 32 || lists > M) {
    const int deep = min(M, (8 * M + lists - 1) / lists), enough = (M + deep - 1) / deep;
    double total;
    unsigned place;
    const uint64_t head = tid < lists && entry(tid * M + deep - 1, total, place) ? order_key(total) : 0;
    heads[tid] = head;
    if (tid < 8) heads[kHeads + tid] = 0;
    __syncthreads();
    if (head != 0 && count_greater(heads, lists, head) < enough) atomicMin(&least, (unsigned long long)head);
    __syncthreads();
    const uint64_t bound = least;
    for (int i = tid; i < entries; i += 4 * kThreads) {
      Pick q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = picks[min(i + j * kThreads, entries - 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j * kThreads >= entries || !value(i + j * kThreads, q[j], total, place)) continue;
        const uint64_t key = order_key(total);
        if (key >= bound) {
          const int at = atomicAdd(&found, 1);
          if (at < kRanked) {
            keys[at] = key;
            places[at] = place;
          }
        }
      }
    }
    __syncthreads();
    few = found >= M && found <= kRanked;
    __syncthreads();
    if (!few && tid == 0) found = 0;
    __syncthreads();  // what is counted below may follow at once
  }
  uint64_t high = 0;  // the digits of the M-th best known so far: of the total, and of the place's complement
  unsigned low = 0;
  int step = 0, more = 0, left = entries;  // digits known, continuations above them, those that agree
  while (!few && more + left > kRanked) {
    bins[tid] = 0;
    __syncthreads();
    for (int i = tid; i < entries; i += kThreads) {
      double total;
      unsigned place;
      if (!entry(i, total, place)) continue;
      const uint64_t key = order_key(total);
      int d = -1;
      if (step < 8) {
        if (step == 0 || (key >> (64 - 8 * step)) == (high >> (64 - 8 * step))) d = (int)(key >> (56 - 8 * step)) & 255;
      } else if (key == high) {
        const unsigned at = ~place;
        if (step == 8 || (at >> (96 - 8 * step)) == (low >> (96 - 8 * step))) d = (int)(at >> (88 - 8 * step)) & 255;
      }
      if (d >= 0) atomicAdd(&bins[d], 1);
    }
    __syncthreads();
    if (wave == 0) {
      // lane 0 holds the four highest bins
      int four = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) four += bins[255 - 4 * lane - j];
      int sum = four;
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(sum, off, 64);
        if (lane >= off) sum += o;
      }
      const int want = M - more, before_me = sum - four;
      if (before_me < want && sum >= want) {
        int up = before_me, j = 0;
        for (; j < 3 && up + bins[255 - 4 * lane - j] < want; ++j) up += bins[255 - 4 * lane - j];
        digit = 255 - 4 * lane - j;
        above = up;
        inside = bins[255 - 4 * lane - j];
      }
    }
    __syncthreads();
    if (step < 8) high |= (uint64_t)digit << (56 - 8 * step);
    else low |= (unsigned)digit << (88 - 8 * step);
    more += above;
    left = inside;
    ++step;
    __syncthreads();
  }

  if (!few)
    for (int i = tid; i < entries; i += kThreads) {
      double total;
      unsigned place;
      if (!entry(i, total, place)) continue;
      const uint64_t key = order_key(total);
      bool in = true;
      if (step > 0) {
        const int bits = step < 8 ? 64 - 8 * step : 0;
        in = (key >> bits) >= (high >> bits);
        if (step > 8 && key == high) in = (~place >> (96 - 8 * step)) >= (low >> (96 - 8 * step));
      }
      if (in) {
        const int at = atomicAdd(&found, 1);
        keys[at] = key;
        places[at] = place;
      }
    }
  __syncthreads();
  const int c = found;
  if (tid < 4) keys[c + tid] = 0;  // the least there is
  __syncthreads();
  if (tid < c) {
    const uint64_t key = keys[tid];
    const unsigned place = places[tid];
    int r = 0;
    for (int j = 0; j < c; j += 4) {
      uint64_t k[4];
      unsigned at[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        k[i] = keys[j + i];
        at[i] = places[j + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) r += (int)(k[i] > key) | ((int)(k[i] == key) & (int)(at[i] < place));
    }
    if (r < M) {
      const size_t at = (size_t)n * M + r;
      p.parent[at] = (int)(place / (unsigned)p.V);
      p.token[at] = (int)(place % (unsigned)p.V);
      p.score[at] = (float)key_order(key);
    }
  }
}

struct BeamShape {
  int per_thread, pieces, stretches;  // logits a thread holds, pieces of a stretch, stretches of a row
};

// 32 logits a thread and as many stretches a row as make 1024 workgroups, four for each CU; with few rows,
// where the time is the latency of one workgroup, 8 logits a thread.  A request has no more lists than the
// join has threads (one of 16 beams, 41,115 tokens, bf16: 19 us; with 336 lists
// 43; one of 64, 131,072 tokens, fp32, M = 64: 108 and 400).
BeamShape beam_shape(const ccq_beam_params& p) {
  const long long rows = (long long)p.N * p.K;
  BeamShape s;
  const long long quarter = (p.V + kThreads * 32 - 1) / (kThreads * 32);
  s.per_thread = rows * quarter < 256 ? 8 : 32;
  const long long whole = (p.V + (long long)kThreads * s.per_thread - 1) / (kThreads * s.per_thread);  // pieces of a row
  long long want = (1024 + rows - 1) / rows;
  if (want > whole) want = whole;
  if (want * p.K > kHeads) want = kHeads / p.K;
  s.pieces = (int)((whole + want - 1) / want);
  s.stretches = (int)((whole + s.pieces - 1) / s.pieces);
  return s;
}

template <typename T, int E, bool ONE>
void launch_rows(const ccq_beam_params& p, const BeamShape& s, BeamWork w, hipStream_t stream) {
  beam_rows_kernel<T, E, ONE><<<(unsigned)(p.N * p.K * s.stretches), kThreads, 0, stream>>>(p, s.stretches, s.pieces, w);
}

template <typename T>
void launch_rows_of(const ccq_beam_params& p, const BeamShape& s, BeamWork w, hipStream_t stream) {
  if (s.per_thread == 8 && s.pieces == 1) launch_rows<T, 8, true>(p, s, w, stream);
  else if (s.per_thread == 8) launch_rows<T, 8, false>(p, s, w, stream);
  else if (s.pieces == 1) launch_rows<T, 32, true>(p, s, w, stream);
  else launch_rows<T, 32, false>(p, s, w, stream);
}

// ---------------------------------------------------------------- reordering

struct ReorderArgs {
  unsigned char* state[CCQ_MAX_REORDER_STATES];
  size_t row_bytes[CCQ_MAX_REORDER_STATES];
  unsigned first_block[CCQ_MAX_REORDER_STATES + 1];  // of a request's blocks, where each state's begin
  int n_states, K;
  const int32_t* parent;
};

// One thread owns the same W bytes of all K beams of a request, reads what moves and then writes it:
// no other thread touches those bytes, so the move is in place, whatever the parents are, and only
// rows that move are touched.  STREAM: past the caches.
// Measured: 64 requests of 4 beams, the carries of 16 heads of 128 (718 MB moved): 130 us, 5.5 TB/s past the
// caches, 141 through them; 8 requests' (67 MB of states): 17.2 and 14.9.  More than 16 beams, four bytes a thread:
// 16 requests of 17 (895 MB) 216 us, 8 of 32 (860 MB) 163, 4 of 64 (870 MB) 189: 4.1, 5.3 and 4.6 TB/s.
template <typename W, int KMAX, bool STREAM>
__device__ __forceinline__ void move_columns(unsigned char* base, size_t row, size_t off, const int (&par)[KMAX], int K) {
  W v[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j < K && par[j] != j) {
      const W* from = reinterpret_cast<const W*>(base + (size_t)par[j] * row + off);
      if constexpr (STREAM) v[j] = __builtin_nontemporal_load(from);
      else v[j] = *from;
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    if (j < K && par[j] != j) {
      W* to = reinterpret_cast<W*>(base + (size_t)j * row + off);
      if constexpr (STREAM) __builtin_nontemporal_store(v[j], to);
      else *to = v[j];
    }
  }
}

template <int KMAX, bool STREAM>
__global__ __launch_bounds__(kThreads) void beam_reorder_kernel(ReorderArgs a, unsigned blocks_per_request) {
  const unsigned n = blockIdx.x / blocks_per_request, blk = blockIdx.x - n * blocks_per_request;
  int s = 0;
  while (s + 1 < a.n_states && blk >= a.first_block[s + 1]) ++s;
  int par[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    par[j] = j;
    if (j < a.K) {
      const int q = a.parent[(size_t)n * a.K + j];
      if (q >= 0 && q < a.K) par[j] = q;
    }
  }
  const size_t row = a.row_bytes[s];
  unsigned char* base = a.state[s] + (size_t)n * a.K * row;
  const size_t i = (size_t)(blk - a.first_block[s]) * kThreads + threadIdx.x;
  if constexpr (KMAX <= 16) {
    if (row % 16 == 0) {
      if (i * 16 < row) move_columns<u32x4, KMAX, STREAM>(base, row, i * 16, par, a.K);
      return;
    }
  }
  if (i * 4 < row) move_columns<unsigned, KMAX, STREAM>(base, row, i * 4, par, a.K);
}

}  // namespace

bool beam_grid_fits(const ccq_beam_params& p) {
  return (long long)p.N * p.K < (1LL << 24) && grid_fits((uint64_t)p.N * p.K * beam_shape(p).stretches, kThreads);
}

size_t beam_workspace_bytes(const ccq_beam_params& p) {
  const size_t lists = (size_t)p.N * p.K * beam_shape(p).stretches;
  return parts_bytes(lists) + lists * p.M * sizeof(Pick);
}

hipError_t launch_beam_select(const ccq_beam_params& p, hipStream_t stream) {
  const BeamShape s = beam_shape(p);
  const size_t lists = (size_t)p.N * p.K * s.stretches;
  unsigned char* ws = static_cast<unsigned char*>(p.workspace);
  const BeamWork w{reinterpret_cast<Part*>(ws), reinterpret_cast<Pick*>(ws + parts_bytes(lists))};
  if (p.dtype == CCQ_DTYPE_BF16) launch_rows_of<__bf16>(p, s, w, stream);
  else launch_rows_of<float>(p, s, w, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  beam_join_kernel<<<p.N, kThreads, 0, stream>>>(p, s.stretches, w);
  return hipGetLastError();
}

// Room for 4, 16 or 64 beams.  (Room for 8 takes 222 registers, two waves a SIMD, where 16 takes 66: 223 requests
// of 8 beams, 468 MB of states, 214 us against 135.)
template <bool STREAM>
static void launch_reorder(const ReorderArgs& a, unsigned grid, unsigned blocks, hipStream_t stream) {
  if (a.K <= 4) beam_reorder_kernel<4, STREAM><<<grid, kThreads, 0, stream>>>(a, blocks);
  else if (a.K <= 16) beam_reorder_kernel<16, STREAM><<<grid, kThreads, 0, stream>>>(a, blocks);
  else beam_reorder_kernel<64, STREAM><<<grid, kThreads, 0, stream>>>(a, blocks);
}

// States of up to half the 256 MB cache find themselves in it from call to call.  (134 MB of them: 31 us past the
// caches, 27 through them if they were there, 34.6 against 33.4 if not.)
static constexpr uint64_t kCached = 128 << 20;

// Workgroups that go along a request's rows of one state.
static uint64_t reorder_blocks(size_t row_bytes, int K) {
  const size_t width = K <= 16 && row_bytes % 16 == 0 ? 16 : 4;
  return (row_bytes / width + kThreads - 1) / kThreads;
}
bool beam_reorder_grid_fits(int n_states, const size_t* row_bytes, int N, int K) {
  uint64_t blocks = 0;
  for (int i = 0; i < n_states; ++i) blocks += reorder_blocks(row_bytes[i], K);
  return grid_fits(blocks * N, kThreads);
}

hipError_t launch_beam_reorder(int n_states, void* const* states, const size_t* row_bytes, int N, int K,
                               const int32_t* parent, hipStream_t stream) {
  ReorderArgs a{};
  a.n_states = n_states;
  a.K = K;
  a.parent = parent;
  uint64_t blocks = 0, bytes = 0;
  for (int i = 0; i < n_states; ++i) {
    bytes += (uint64_t)row_bytes[i] * N * K;
    a.state[i] = static_cast<unsigned char*>(states[i]);
    a.row_bytes[i] = row_bytes[i];
    a.first_block[i] = (unsigned)blocks;
    blocks += reorder_blocks(row_bytes[i], K);
  }
  a.first_block[n_states] = (unsigned)blocks;
  const unsigned grid = (unsigned)(blocks * N);
  if (bytes > kCached) launch_reorder<true>(a, grid, (unsigned)blocks, stream);
  else launch_reorder<false>(a, grid, (unsigned)blocks, stream);
  return hipGetLastError();
}

}  // namespace ccq
