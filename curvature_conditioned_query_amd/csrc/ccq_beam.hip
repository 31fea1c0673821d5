// Beam search: the best continuations of every request over its beams and the vocabulary, and the
// reordering of the states that the beams carry.
//
// Selection reads the logits once.  beam_rows_kernel gives a workgroup one chunk of one beam's row,
// held in registers (up to 64 logits a thread): it leaves the chunk's M best logits, in order, and its
// part of the normaliser sum exp(x - m).  beam_join_kernel, one workgroup a request, joins the parts
// into each beam's normaliser and picks the M best continuations out of the chunks' lists.
//
// Picking M of 16384 needs no sort: with every thread's own maximum known, the M-th best of those
// maxima is a bound that at least M logits reach, and a logit that reaches it lies on one of the M
// threads whose maximum does, so at most 64 M logits are left to be ranked (a few more than M in
// earnest).  Ties go to the lowest token throughout: the bound is a pair (logit, token).
//
// Scores of different beams meet in the comparison, so the normaliser has to be good to more than
// fp32: the logits that reach the bound, which carry most of a peaked distribution, are left out of the
// fp32 sum and added in 64 bits, and the threads' sums of the rest are joined in 64 bits.
#include <float.h>

#include "ccq_device.hpp"
#include "ccq_internal.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// The workspace: a part of the normaliser and a list of M logits for every (row, chunk).
struct Part {
  double sum;  // sum of exp(x - top) over the chunk
  float top;   // its largest logit
  int pad;
};
struct Pick {
  float logit;
  int token;  // -1: the chunk has no more
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

// exp(d) for d <= 0, fp32, with the product by log2(e) good to more than its rounding.
__device__ __forceinline__ float exp_tail(float d) {
  constexpr float hi = 1.44269502162933349609f, lo = 1.92596299112661746887e-8f;  // log2(e) in two parts
  return __builtin_amdgcn_exp2f(__builtin_fmaf(d, hi, d * lo));
}

// A row's beam: 0 goes on, 1 finished, 2 dead (its score is -inf or NaN).
__device__ __forceinline__ int beam_kind(const ccq_beam_params& p, int row) {
  if (p.finished && p.finished[row]) return 1;
  const float s = p.scores[row];
  return s > -INFINITY ? 0 : 2;
}

// 16 bytes from any element on: a row starts where the one before ends, at an odd address for an odd
// vocabulary.  Which thread holds a token must not depend on that address: beams with equal logits have
// to get equal normalisers to the last bit, or their ties would fall either way.
typedef bf16x8 bf16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// Elements of the chunk that thread `tid` holds: E of them, in vectors of VE, vector j from token
// (j 256 + tid) VE of the chunk on.
template <typename T, int E>
__global__ __launch_bounds__(kThreads) void beam_rows_kernel(ccq_beam_params p, int chunks, BeamWork work) {
  constexpr int VE = 16 / sizeof(T), NV = E / VE;
  extern __shared__ __align__(16) unsigned char dyn[];  // candidates: M E logits, M E tokens, M E logits in order
  __shared__ __align__(16) float best[kWaves][64];
  __shared__ float bound_value;
  __shared__ unsigned bound_token;
  __shared__ int above[kWaves], equal[kWaves], found;
  __shared__ double sums[kWaves];
  __shared__ unsigned firsts[kThreads];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, M = p.M;
  const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
  const size_t list = blockIdx.x;
  Pick* picks = work.picks + list * M;

  const int kind = beam_kind(p, row);
  if (kind != 0) {
    // a finished beam's one continuation and then, as a dead beam's, tokens in order at -inf
    for (int i = tid; i < M; i += kThreads) {
      Pick k{-INFINITY, -1};
      if (chunk == 0) {
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

  const T* src = static_cast<const T*>(p.logits) + (int64_t)row * p.logits_stride;
  // token of the thread's first element: the rest follow by constants
  const int first = chunk * (kThreads * E) + tid * VE;
  float x[E];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v0 = first + j * (kThreads * VE);
    if (v0 + VE <= p.V) {
      if constexpr (sizeof(T) == 2) {
        const bf16x8 a = *reinterpret_cast<const bf16x8_any*>(src + v0);
#pragma unroll
        for (int e = 0; e < VE; ++e) x[j * VE + e] = as_counted((float)a[e]);
      } else {
        const f32x4 a = *reinterpret_cast<const f32x4_any*>(src + v0);
#pragma unroll
        for (int e = 0; e < VE; ++e) x[j * VE + e] = as_counted(a[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        x[j * VE + e] = v0 + e < p.V ? as_counted(to_f32(src[v0 + e])) : -INFINITY;
    }
  }
  float mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < E; ++i) mine = fmaxf(mine, x[i]);

  // the M best thread maxima of each wave, in order
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < 64; ++i) {
    const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), i));
    rank += (o > mine || (o == mine && i < lane)) ? 1 : 0;
  }
  best[wave][rank] = mine;
  if (tid == 0) found = 0;
  __syncthreads();
  // the M-th best of all: every wave's lists, an entry a thread
  const float top = fmaxf(fmaxf(best[0][0], best[1][0]), fmaxf(best[2][0], best[3][0]));
  if (lane < M) {
    const float v = best[wave][lane];
    int r = lane;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) continue;
      for (int i = 0; i < M; ++i) {
        const float o = best[w][i];
        r += (o > v || (o == v && w < wave)) ? 1 : 0;
      }
    }
    if (r == M - 1) bound_value = v;
  }
  __syncthreads();
  const float bound = bound_value;
  const uint64_t gt = __ballot(mine > bound), eq = __ballot(mine == bound);
  if (lane == 0) {
    above[wave] = __popcll(gt);
    equal[wave] = __popcll(eq);
  }
  __syncthreads();
  const int want = M - (above[0] + above[1] + above[2] + above[3]);  // threads at the bound that are needed
  unsigned last = 0xffffffffu;
  if (equal[0] + equal[1] + equal[2] + equal[3] > want) {
    // more threads sit at the bound than are needed: those whose first such token is lowest
    unsigned f = 0xffffffffu;
    if (mine == bound) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int v = first + (i / VE) * (kThreads * VE) + i % VE;
        if (x[i] == bound && v < p.V) f = min(f, (unsigned)v);
      }
    }
    firsts[tid] = f;
    if (tid == 0) bound_token = 0xffffffffu;
    __syncthreads();
    if (f != 0xffffffffu) {
      int r = 0;
      for (int i = 0; i < kThreads; ++i) r += firsts[i] < f ? 1 : 0;
      if (r == want - 1) bound_token = f;
    }
    __syncthreads();
    last = bound_token;
  }

  float* cand_x = reinterpret_cast<float*>(dyn);
  int* cand_v = reinterpret_cast<int*>(cand_x + M * E);
  float* in_order = reinterpret_cast<float*>(cand_v + M * E);
  if (mine >= bound) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int v = first + (i / VE) * (kThreads * VE) + i % VE;
      if (v < p.V && (x[i] > bound || (x[i] == bound && (unsigned)v <= last))) {
        const int at = atomicAdd(&found, 1);
        cand_x[at] = x[i];
        cand_v[at] = v;
        x[i] = -INFINITY;  // not in the fp32 sum
      }
    }
  }
  float part = 0.f;
  if (top > -INFINITY) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E; ++i) s[i & 3] += exp_tail(x[i] - top);
    part = (s[0] + s[1]) + (s[2] + s[3]);
  }
  const double total = wave_sum((double)part);
  if (lane == 0) sums[wave] = total;
  __syncthreads();

  const int n = found;
  for (int i = tid; i < n; i += kThreads) {
    const float v = cand_x[i];
    const int token = cand_v[i];
    int r = 0;
    for (int j = 0; j < n; ++j) {
      const float o = cand_x[j];
      r += (o > v || (o == v && cand_v[j] < token)) ? 1 : 0;
    }
    in_order[r] = v;
    if (r < M) picks[r] = Pick{v, token};
  }
  for (int i = n + tid; i < M; i += kThreads) picks[i] = Pick{-INFINITY, -1};
  __syncthreads();
  if (wave == 0) {
    double s = 0.0;
    if (top > -INFINITY)
      for (int i = lane; i < n; i += 64) s += exp((double)in_order[i] - (double)top);
    s = wave_sum(s);
    if (lane == 0) work.parts[list] = Part{s + ((sums[0] + sums[1]) + (sums[2] + sums[3])), top, 0};
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
  return b.rest + ((double)k.logit - b.top);
}

__global__ __launch_bounds__(kThreads) void beam_join_kernel(ccq_beam_params p, int chunks, BeamWork work) {
  extern __shared__ __align__(16) unsigned char dyn[];  // heads' totals, then candidates: totals and places
  __shared__ BeamBase base[kBeamMaxBeams];
  __shared__ double bound_total;
  __shared__ int bound_list, found;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = blockIdx.x, K = p.K, M = p.M;
  const int lists = K * chunks;
  const Part* parts = work.parts + (size_t)n * lists;
  const Pick* picks = work.picks + (size_t)n * lists * M;

  for (int k = wave; k < K; k += kWaves) {
    const int kind = beam_kind(p, n * K + k);
    const float score = p.scores[n * K + k];
    BeamBase b{score > -INFINITY ? score : -INFINITY, 0.0, kind};  // NaN counts as -inf
    if (kind == 0) {
      float top = -INFINITY;
      for (int c = lane; c < chunks; c += 64) top = fmaxf(top, parts[k * chunks + c].top);
      top = wave_max(top);
      double s = 0.0;
      if (top > -INFINITY)
        for (int c = lane; c < chunks; c += 64) {
          const Part q = parts[k * chunks + c];
          if (q.top > -INFINITY) s += q.sum * exp((double)q.top - (double)top);
        }
      s = wave_sum(s);
      if (top > -INFINITY) {
        b.rest -= log(s);
        b.top = top;
      }
    }
    if (lane == 0) base[k] = b;
  }
  if (tid == 0) {
    found = 0;
    bound_total = -INFINITY;
    bound_list = lists;  // every list, unless there are more than M
  }
  __syncthreads();

  if (lists > M) {
    double* heads = reinterpret_cast<double*>(dyn);
    for (int i = tid; i < lists; i += kThreads) {
      const Pick k = picks[(size_t)i * M];
      heads[i] = k.token < 0 ? -INFINITY : pick_total(k, base[i / chunks]);
    }
    __syncthreads();
    double bt = 0.0;
    int bl = -1;
    for (int i = tid; i < lists; i += kThreads) {
      const double v = heads[i];
      int r = 0;
      for (int j = 0; j < lists; ++j) {
        const double o = heads[j];
        r += (o > v || (o == v && j < i)) ? 1 : 0;
      }
      if (r == M - 1) {
        bt = v;
        bl = i;
      }
    }
    if (bl >= 0) {
      bound_total = bt;
      bound_list = bl;
    }
    __syncthreads();
  }

  // the lists' entries that reach the bound: those of at most M lists
  const double bt = bound_total;
  const int bl = bound_list;
  double* totals = reinterpret_cast<double*>(dyn);
  unsigned* places = reinterpret_cast<unsigned*>(totals + M * M);
  for (int i = tid; i < lists * M; i += kThreads) {
    const int list = i / M, k = list / chunks;
    const Pick q = picks[i];
    if (q.token < 0) continue;
    const double v = pick_total(q, base[k]);
    if (v > bt || (v == bt && list <= bl)) {
      const int at = atomicAdd(&found, 1);
      totals[at] = v;
      places[at] = (unsigned)k * (unsigned)p.V + (unsigned)q.token;
    }
  }
  __syncthreads();
  const int c = found;
  for (int i = tid; i < c; i += kThreads) {
    const double v = totals[i];
    const unsigned place = places[i];
    int r = 0;
    for (int j = 0; j < c; ++j) {
      const double o = totals[j];
      r += (o > v || (o == v && places[j] < place)) ? 1 : 0;
    }
    if (r < M) {
      const size_t at = (size_t)n * M + r;
      p.parent[at] = (int)(place / (unsigned)p.V);
      p.token[at] = (int)(place % (unsigned)p.V);
      p.score[at] = (float)v;
    }
  }
}

struct BeamShape {
  int per_thread, chunks;
};

// Logits a thread holds: 64 where that leaves 512 workgroups, fewer for few rows, where the time is
// the latency of one workgroup.
BeamShape beam_shape(const ccq_beam_params& p) {
  BeamShape s{64, 0};
  for (;; s.per_thread /= 2) {
    const long long chunk = (long long)kThreads * s.per_thread;
    s.chunks = (int)((p.V + chunk - 1) / chunk);
    if (s.per_thread == 8 || (long long)p.N * p.K * s.chunks >= 512 || p.K * (long long)s.chunks * 2 > kBeamMaxLists)
      return s;
  }
}

template <typename T, int E>
void launch_rows(const ccq_beam_params& p, const BeamShape& s, BeamWork w, hipStream_t stream) {
  beam_rows_kernel<T, E><<<(unsigned)(p.N * p.K * s.chunks), kThreads, (size_t)p.M * E * 12, stream>>>(p, s.chunks, w);
}

template <typename T>
void launch_rows_of(const ccq_beam_params& p, const BeamShape& s, BeamWork w, hipStream_t stream) {
  if (s.per_thread == 64) launch_rows<T, 64>(p, s, w, stream);
  else if (s.per_thread == 32) launch_rows<T, 32>(p, s, w, stream);
  else if (s.per_thread == 16) launch_rows<T, 16>(p, s, w, stream);
  else launch_rows<T, 8>(p, s, w, stream);
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
// rows that move are touched.
template <typename W, int KMAX>
__device__ __forceinline__ void move_columns(unsigned char* base, size_t row, size_t off, const int (&par)[KMAX], int K) {
  W v[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && par[j] != j) v[j] = __builtin_nontemporal_load(reinterpret_cast<const W*>(base + (size_t)par[j] * row + off));
#pragma unroll
  for (int j = 0; j < KMAX; ++j)
    if (j < K && par[j] != j) __builtin_nontemporal_store(v[j], reinterpret_cast<W*>(base + (size_t)j * row + off));
}

template <int KMAX>
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
      if (i * 16 < row) move_columns<u32x4, KMAX>(base, row, i * 16, par, a.K);
      return;
    }
  }
  if (i * 4 < row) move_columns<unsigned, KMAX>(base, row, i * 4, par, a.K);
}

}  // namespace

size_t beam_workspace_bytes(const ccq_beam_params& p) {
  const size_t lists = (size_t)p.N * p.K * beam_shape(p).chunks;
  return parts_bytes(lists) + lists * p.M * sizeof(Pick);
}

hipError_t launch_beam_select(const ccq_beam_params& p, hipStream_t stream) {
  const BeamShape s = beam_shape(p);
  const size_t lists = (size_t)p.N * p.K * s.chunks;
  unsigned char* ws = static_cast<unsigned char*>(p.workspace);
  const BeamWork w{reinterpret_cast<Part*>(ws), reinterpret_cast<Pick*>(ws + parts_bytes(lists))};
  if (p.dtype == CCQ_DTYPE_BF16) launch_rows_of<__bf16>(p, s, w, stream);
  else launch_rows_of<float>(p, s, w, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t heads = p.K * s.chunks > p.M ? (size_t)p.K * s.chunks * 8 : 0, cands = (size_t)p.M * p.M * 12;
  beam_join_kernel<<<p.N, kThreads, heads > cands ? heads : cands, stream>>>(p, s.chunks, w);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(int n_states, void* const* states, const size_t* row_bytes, int N, int K,
                               const int32_t* parent, hipStream_t stream) {
  ReorderArgs a{};
  a.n_states = n_states;
  a.K = K;
  a.parent = parent;
  uint64_t blocks = 0;
  for (int i = 0; i < n_states; ++i) {
    a.state[i] = static_cast<unsigned char*>(states[i]);
    a.row_bytes[i] = row_bytes[i];
    a.first_block[i] = (unsigned)blocks;
    const size_t width = K <= 16 && row_bytes[i] % 16 == 0 ? 16 : 4;
    blocks += (row_bytes[i] / width + kThreads - 1) / kThreads;
    if (blocks * N > 0x7fffffffu) return hipErrorInvalidValue;
  }
  a.first_block[n_states] = (unsigned)blocks;
  const unsigned grid = (unsigned)(blocks * N);
  if (K <= 4) beam_reorder_kernel<4><<<grid, kThreads, 0, stream>>>(a, (unsigned)blocks);
  else if (K <= 8) beam_reorder_kernel<8><<<grid, kThreads, 0, stream>>>(a, (unsigned)blocks);
  else if (K <= 16) beam_reorder_kernel<16><<<grid, kThreads, 0, stream>>>(a, (unsigned)blocks);
  else beam_reorder_kernel<64><<<grid, kThreads, 0, stream>>>(a, (unsigned)blocks);
  return hipGetLastError();
}

}  // namespace ccq
