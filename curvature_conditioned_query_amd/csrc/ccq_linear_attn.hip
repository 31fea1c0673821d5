// Linear attention with one decay for each head, S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, and
// its gradient.
//
// Everything is one form, out_i = e^{B_i} S x_i + sum_{j <= i} e^{B_i - B_j} (x_i . y_j) z_j with B the running
// sum of the log decays and S the state before the first token, S' = e^{B_L} S + sum_j e^{B_L - B_j} z_j y_j^T
// behind the last:
//   o  = (x, y, z) = (q, k, v);
//   dq = (d_o, v, k), whose state is S transposed;
//   dk = (v, d_o, q) and dv = (k, q, d_o) over the sequence from its end (j >= i, e^{B_j - B_i}), whose state is the
//        adjoint of S (transposed for dk);
// so one kernel, the walk, computes a "role" (x, y, z, direction), and the gradient is three roles in one launch.
//
// The walk.  A workgroup owns one chain (sequence and head) and a slice of 32 columns of z, keeps its 32 x d_x part of
// the state in MFMA accumulators, and goes over the chain's 64-token chunks, one barrier a chunk:
//   two waves issue the rows' loads, straight into LDS, two chunks ahead;
//   one forms the next chunk's decays;
//   four form outputs, wave w the tokens 16 w .. 16 w + 15:
//     scores   Y X^T by 16 x 16 tiles, against the tokens its direction allows; weighted by e^{B_i - B_j} they are the
//              B operand of
//     near     out^T += Z^T P^T as they lie in the registers;
//     far      out^T += a_i St X^T with the state's copy St in LDS, in the inputs' type;
//   four hold the state, wave w a quarter of d_x:
//     update   S^T = e^{B_L} S^T + Y^T (b z), b z as a sum of three bf16 where the inputs have 16 bits: what enters a
//              state, which later tokens and calls build on, is right to 2^-24; and the copy St for the next chunk.
// What bounds it: nothing alone.  B4 T4096, 16 heads of 128 takes 94 to 99 us; without the rows' loads 84, without the outputs 78,
// without the state 86, the loads and decays alone 69 (36 KB a chunk and workgroup, 604 MB, 8.8 TB/s from the L2s), the decays and
// barriers alone 24.  A chunk is a chain of LDS reads, products and a barrier for one workgroup of 11 waves a CU, each of which
// waits for a part of it.  A slice of 64 columns would halve the reading and share the scores; laid out as now its tiles need 174 KB
// of LDS (about 149 with two tiles of x and outputs staged in 16 bits, which was not tried).
// Weights of pairs, not e^{B_i} e^{-B_j}: nothing leaves fp32's range whatever the decay.  Running sums are
// formed in 64 bits and kept as two floats, in units of log 2.
#include <type_traits>

#include "ccq_prefill_common.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256;
constexpr int kSlice = 32;             // columns of z that a workgroup owns
constexpr int kStepRows = 32;          // rows of a state that a workgroup owns in a step of single tokens
constexpr double kLog2e = 1.4426950408889634074;
constexpr double kReset = -126.0;      // log2 of a decay below which it is 0, fp32's least normal number: a reset
constexpr double kGateFloor = -1.5e4;  // and what it counts as in sums, so that growth behind it brings nothing back: 2^-15000 is 0,
                                       // sums of 64 stay exact enough

struct Strides {
  int64_t b, t, h;
};

// One walk over (x, y, z).
struct Role {
  const void *x, *y, *z;
  Strides xs, ys, zs;
  int x_share, y_share, z_share;  // heads that read one row
  void* out;                      // [B, T, H, 32 slices]
  Strides os;
  int out_f32;
  int zero_idle;                  // rows of no token are set to 0
  const void* w;                  // gradient: rows of the slice's columns, whose products with the outputs are summed
  Strides ws;
  int w_share;
  float* r;                       // [slices][chains][T], or null
  const float* s_in;              // state before, or null; entry (dz, dx) at dz s_i + dx s_j of the chain's
  int s_i, s_j;
  float* s_out;                   // state behind, [dz][dx] rows, or null
  const float* dot;               // matrix whose product with the state behind is summed (strides s_i, s_j), or null
  float* dot_out;                 // [chains][slices][4]
  float in_scale, out_scale;
  int reverse, slices, dz;
  float* slots;                   // summaries of segments, or null with one segment
  double* slot_log;               // [chains][segments] their log decays, in units of log 2; -inf with a reset among them
};

struct Args {
  int B, T, H, chains, segments, chunks_per_segment, roles, slots_per_group, snapshot;
  const void* la;
  Strides ls;
  int gate_bf16;
  const int32_t *lengths, *offsets;
  int64_t rows;
  Role role[3];
};

// Tokens of sequence b, and its first row.
struct Span {
  int len;
  int64_t row0;
};
__device__ __forceinline__ Span span_of(const int32_t* lengths, const int32_t* offsets, int64_t rows, int T, int b) {
  Span s{T, 0};
  if (offsets) {
    const int64_t from = offsets[b], to = offsets[b + 1];
    s.row0 = from < 0 ? 0 : (from > rows ? rows : from);
    int64_t n = to - s.row0;
    if (n > rows - s.row0) n = rows - s.row0;
    s.len = (int)(n < 0 ? 0 : (n > T ? T : n));
  } else if (lengths) {
    const int n = lengths[b];
    s.len = n < 0 ? 0 : (n > T ? T : n);
  }
  return s;
}
__device__ __forceinline__ Span span_of(const Args& a, int b) { return span_of(a.lengths, a.offsets, a.rows, a.T, b); }

// Rows of no token that sequence b answers for, 0 .. front - 1 and from .. to - 1: those behind its end, counted from its own first
// row; packed, those up to the next sequence's first row, and before the first sequence, counted over all rows.
struct Idle {
  int64_t front, from, to;
};
__device__ __forceinline__ Idle idle_of(const Args& a, const Span& s, int b) {
  if (a.offsets == nullptr) return Idle{0, s.len, a.T};
  const int64_t next = b + 1 < a.B ? (int64_t)a.offsets[b + 1] : a.rows;
  return Idle{b == 0 ? s.row0 : 0, s.row0 + s.len, next < a.rows ? next : a.rows};
}

template <typename T>
__device__ __forceinline__ T* rows_of(const void* p, const Strides& s, int share, const Args& a, const Span& sp, int b, int h) {
  return const_cast<T*>(static_cast<const T*>(p)) + (a.offsets ? sp.row0 * s.t : b * s.b) + (h / share) * s.h;
}

// log2 of the decay of one token, from its bits as stored: a load that is not waited for until its value is needed.
__device__ __forceinline__ unsigned gate_bits(const Args& a, int64_t at) {
  if (a.la == nullptr) return 0u;
  if (a.gate_bf16) return static_cast<const uint16_t*>(a.la)[at];
  return static_cast<const uint32_t*>(a.la)[at];
}
__device__ __forceinline__ double gate_value(const Args& a, unsigned bits) {
  const double g = (double)__builtin_bit_cast(float, a.gate_bf16 ? bits << 16 : bits) * kLog2e;
  return g < kReset ? kGateFloor : g;  // NaN stays
}
__device__ __forceinline__ double gate_of(const Args& a, int64_t at) { return gate_value(a, gate_bits(a, at)); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Four entries of a row, whatever it holds.
template <typename T>
__device__ __forceinline__ void store_out(void* p, int64_t at, const f32x4& v, int f32) {
  if (sizeof(T) == 4 || f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
  else *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p) + at) = to_bf16x4(v);
}

template <typename T, int DX, bool SPLIT, bool SUMMARY>
struct Smem {
  // bf16 rows of x, y and the state's copy lie without padding, 16-byte slot s of row r at slot s ^ swizzle(r): rows and
  // columns are read at the rate of consecutive addresses (4.75 to 5.25 clocks a wave; with padding 8), and four neighbouring lanes
  // of a load still take 64 bytes that belong together (with padded rows a load took 44 clocks for 16).  fp32 rows are padded.
  static constexpr int ZS = kSlice;
  static constexpr bool SW = sizeof(T) == 2;
  static constexpr int PY = DX + (SW ? 0 : 4), PS = PY, PZ = ZS + (SW ? 0 : 4);
  static constexpr int AHEAD = sizeof(T) == 2 ? 2 : 1;          // chunks between a load and its use
  static constexpr int NB = AHEAD + 1;                          // tiles held of y and z
  static constexpr int NH = sizeof(T) == 2 ? 3 : 1;             // parts of b z
  static constexpr int NS = sizeof(T) == 2 && SPLIT ? 2 : 1;    // parts of the state's copy
  T Y[NB][kL][PY];
  T Z[NB][kL][PZ];
  T St[SUMMARY ? 1 : 2][NS][SUMMARY ? 1 : ZS][PS];
  static constexpr bool XL = sizeof(T) == 2;  // fp32 rows of x do not fit: they are loaded into registers
  static constexpr int PO = ZS + 4;
  T X[SUMMARY || !XL ? 1 : NB][SUMMARY || !XL ? 1 : kL][PY];
  float out[SUMMARY ? 1 : 4][16][PO];  // each wave's outputs of a chunk on their way to memory
  // Of each token: its running sum as two floats, the weight of the state before the chunk for it, its weight in
  // the state behind, and e^(its sum to the end of its 16 tokens), or from their beginning.
  float bh[2][kL], bl[2][kL], aw[2][kL], bw[2][kL], cf[2][kL];
  float dec[2];
  int first[2], last[2];       // the chunk's first and last token whose decay is 0: kL and -1 if there is none
  uint32_t raw[NB + 1][kL];    // gates as stored
};

// A wave's running sum of 64-bit values, in registers alone.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xf, true);
  const unsigned hi = (unsigned)__builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xf, true);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_running(double x) {
  x = dpp_add<0x111, 0xf>(x);  // by 1, 2, 4 and 8 within 16 lanes
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // lane 15 to the next 16, then lane 31 to the upper half
  return dpp_add<0x143, 0xc>(x);
}

// The weights of a chunk's 64 tokens into buffer `buf`; one wave, lane t token t, g its log2 decay (0 behind the
// end).  Returns the chunk's log2 decay, -inf with a reset.  What a reset cuts off from the state has a weight of 0 whatever stands
// among the other decays, NaN too: sums to the chunk's end begin behind the last reset.
template <bool REV, typename SM>
__device__ __forceinline__ double form_gates(SM& sm, int buf, double g, bool live, float in_scale, int lane) {
  const double s = wave_running(g), all = __shfl(s, 63, 64), near = __shfl(s, REV ? lane & 48 : lane | 15, 64);
  const uint64_t resets = __ballot(g < kReset);
  const int first = resets ? __builtin_ctzll(resets) : kL, last = 63 - __builtin_clzll(resets | 1) - (resets == 0);
  double rest = all - s;
  if (resets) {
    const double r = wave_running(lane > last ? g : 0.0);
    rest = __shfl(r, 63, 64) - r;
  }
  const float hi = (float)s;
  sm.bh[buf][lane] = hi;
  sm.bl[buf][lane] = (float)(s - (double)hi);
  const float up = exp2_fast((float)s), down = exp2_fast((float)rest);
  sm.aw[buf][lane] = REV ? down : up;
  sm.bw[buf][lane] = live && (REV ? lane < first : lane >= last) ? (REV ? up : down) * in_scale : 0.f;
  sm.cf[buf][lane] = live ? exp2_fast((float)(REV ? s - near : near - s)) * in_scale : 0.f;
  if (lane == 0) {
    sm.dec[buf] = exp2_fast((float)all);
    sm.first[buf] = first;
    sm.last[buf] = last;
  }
  return resets ? -INFINITY : all;
}

// An address that is the same in all lanes, in scalar registers, and vectors at byte offsets from it.  (Made of an
// integer, a plain pointer would be a generic one, whose loads count as LDS accesses too.)
#define CCQ_GLOBAL __attribute__((address_space(1)))
typedef CCQ_GLOBAL char* UniformPtr;
__device__ __forceinline__ UniformPtr uniform_ptr(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<UniformPtr>((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32 |
                                      (unsigned)__builtin_amdgcn_readfirstlane((int)u));
}
template <typename V>
__device__ __forceinline__ V load_at(UniformPtr p, unsigned off) {
  return *reinterpret_cast<CCQ_GLOBAL const V*>(p + off);
}
template <typename V>
__device__ __forceinline__ void store_at(UniformPtr p, unsigned off, const V& v) {
  *reinterpret_cast<CCQ_GLOBAL V*>(p + off) = v;
}

// Which slot of 16 bytes of row r of D bf16 the row's first is.
template <int D>
__device__ __forceinline__ int swizzle(int r) { return D == 128 ? r & 15 : (r >> 1) & 7; }

// A chunk's rows of COLS entries straight into an LDS tile of pitch P by one wave, rows behind the sequence's end as
// row 0 (their weights are 0).  Each lane's places are worked out once.  The U loads are not the compiler's: the caller
// waits, and the s_nop is the wait state that a load into LDS needs behind a write of M0.
template <typename T, int COLS, int P, bool SWIZZLED>
struct RowLoads {
  static constexpr int U = P * (int)sizeof(T) / 16, DU = COLS * (int)sizeof(T) / 16;
  unsigned off[U];
  __device__ __forceinline__ RowLoads(int lane, int64_t step) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int u = 64 * j + lane, row = u / U, slot = u - row * U;
      off[j] = slot < DU ? (unsigned)row * (unsigned)(step * (int)sizeof(T)) + 16u * (SWIZZLED ? slot ^ swizzle<COLS>(row) : slot) : 0u;
    }
  }
  __device__ __forceinline__ void load(void* dst, UniformPtr src, int live, int lane) const {
    const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)dst;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      unsigned o = off[j];
      if (live < kL) o = (64 * j + lane) / U < live ? o : 0u;
      const unsigned m0 = __builtin_amdgcn_readfirstlane(base + 1024u * (unsigned)j);
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0), "v"(o), "s"(src) : "memory", "m0");
    }
  }
};

template <int N>
__device__ __forceinline__ void vm_wait() {
  static_assert(N < 64, "the counter of loads under way has six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Columns of a row-major LDS tile as an MFMA operand in the order of an accumulator pair (tr_frag_acc), from the
// lane's own place in the tile: what is added to it is known at compile time.
template <typename T>
__device__ __forceinline__ int tr_place(int pitch, int lane) {
  const int g = lane >> 4, i = lane & 15;
  return sizeof(T) == 2 ? (4 * g + (i >> 2)) * pitch + 4 * (i & 3) : 4 * g * pitch + i;
}
// As tr_place for columns 16 x .. 16 x + 15 of swizzled rows of D.
template <typename T, int D, int PITCH>
__device__ __forceinline__ int tr_place_swizzled(int x, int lane) {
  if (sizeof(T) == 4) return tr_place<T>(PITCH, lane) + 16 * x;
  const int g = lane >> 4, i = lane & 15, row = 4 * g + (i >> 2);
  return row * PITCH + 8 * ((2 * x + ((i & 3) >> 1)) ^ swizzle<D>(row)) + 4 * (i & 1);
}
template <typename T, int PITCH>
__device__ __forceinline__ Frag<T> tr_at(const T* p) {
  Frag<T> f;
  if constexpr (sizeof(T) == 2) {
    const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p));
    const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 16 * PITCH));
    f.v = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[(16 * (e >> 2) + (e & 3)) * PITCH];
  }
  return f;
}
// Rows alike (lds_frag in order): lane (g, l) row l, entries 8 g .. 8 g + 7 of every 32: the lane's place for the kk-th of them.
template <typename T, int D, int PITCH>
__device__ __forceinline__ int row_place(int kk, int lane) {
  const int l = lane & 15, slot = 4 * kk + (lane >> 4);
  return sizeof(T) == 2 ? l * PITCH + 8 * (slot ^ swizzle<D>(l)) : l * PITCH + 8 * slot;
}
template <typename T>
__device__ __forceinline__ Frag<T> row_at(const T* p) {
  Frag<T> f;
  if constexpr (sizeof(T) == 2) {
    f.v = *reinterpret_cast<const bf16x8*>(p);
  } else {
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f.v[e] = lo[e];
      f.v[4 + e] = hi[e];
    }
  }
  return f;
}

// A row as MFMA operands: lane (g, l) entries 8 g .. of every 32 of its row, which begins (with 8 g) at `off`.
template <typename T, int DX>
__device__ __forceinline__ void load_x(Frag<T> (&f)[DX / 32], UniformPtr p, unsigned off) {
#pragma unroll
  for (int kk = 0; kk < DX / 32; ++kk) {
    if constexpr (sizeof(T) == 2) {
      f[kk].v = load_at<bf16x8>(p, off + 64 * kk);
    } else {
      const f32x4 lo = load_at<f32x4>(p, off + 128 * kk), hi = load_at<f32x4>(p, off + 128 * kk + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[kk].v[e] = lo[e];
        f[kk].v[4 + e] = hi[e];
      }
    }
  }
}

// The gates of a walk's chunks, by one wave: formed a chunk ahead, from what a wave of the state has loaded into the LDS.
template <bool REV, typename SM>
struct Gates {
  const Args& a;
  SM& sm;
  int len, c_lo, c_hi, lane, at;
  float in_scale;
  double total;
  bool reset;
  __device__ __forceinline__ Gates(const Args& a, const Role& ro, SM& sm, const Span& sp, int c_lo, int c_hi, int lane)
      : a(a), sm(sm), len(sp.len), c_lo(c_lo), c_hi(c_hi), lane(lane), at(0), in_scale(ro.in_scale), total(0.0), reset(false) {}
  // chunk it, into buffer BUF
  template <int BUF>
  __device__ __forceinline__ void form(int it) {
    if (it < c_hi - c_lo) {
      const bool live = (REV ? c_hi - 1 - it : c_lo + it) * kL + lane < len;
      const double one = form_gates<REV>(sm, BUF, live && a.la ? gate_value(a, sm.raw[at][lane]) : 0.0, live, in_scale, lane);
      total += one;
      reset = reset || one == -INFINITY;
    }
    at = at == SM::NB ? 0 : at + 1;
  }
};
// Loads a chunk's gates into the LDS, one a lane, tokens behind the end as the chunk's first.  The caller waits.
__device__ __forceinline__ void load_gates(const Args& a, uint32_t* dst, int64_t at, int live, int lane) {
  if (a.la == nullptr) return;
  const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint32_t*)dst;
  const unsigned m0 = __builtin_amdgcn_readfirstlane(base);
  const int64_t own = at + (lane < live ? lane * a.ls.t : 0);
  if (a.gate_bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.la) + own;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off" ::"s"(m0), "v"(p) : "memory", "m0");
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(a.la) + own;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(m0), "v"(p) : "memory", "m0");
  }
}

// Wave W of a walk's outputs: queries 16 W .. 16 W + 15 of every chunk.
template <typename T, int DX, bool SPLIT, bool REV, int W>
__device__ __forceinline__ void walk_outputs(const Args& a, const Role& ro, int chain, int slice, const Span& sp, int c_lo, int c_hi, int lane,
                                             Smem<T, DX, SPLIT, false>& sm) {
  using SM = Smem<T, DX, SPLIT, false>;
  constexpr int ZS = SM::ZS, NZ = ZS / 16, NK = DX / 32, T0 = REV ? W : 0, T1 = REV ? 3 : W;
  const int g = lane >> 4, l = lane & 15, n = c_hi - c_lo;
  const int b = chain / a.H, h = chain - b * a.H;
  auto chunk_at = [&](int it) { return REV ? c_hi - 1 - it : c_lo + it; };
  const UniformPtr xb = uniform_ptr(rows_of<T>(ro.x, ro.xs, ro.x_share, a, sp, b, h));
  const UniformPtr wb = uniform_ptr(ro.r ? rows_of<T>(ro.w, ro.ws, ro.w_share, a, sp, b, h) + slice * ZS : nullptr);
  const int64_t ob = (a.offsets ? sp.row0 * ro.os.t : b * ro.os.b) + h * ro.os.h + slice * ZS;
  const int oe = sizeof(T) == 4 || ro.out_f32 ? 4 : 2;
  const UniformPtr outb = uniform_ptr(static_cast<char*>(ro.out) + ob * oe);
  constexpr unsigned kElem = sizeof(T);
  const unsigned own = 16 * W + l;
  const unsigned x_off = own * (unsigned)(ro.xs.t * (int)sizeof(T)) + 8 * g * kElem;
  // outputs leave, and what they are multiplied by comes, eight columns a lane: neighbouring lanes on neighbouring columns
  // (of the accumulators' rows each lane's 8 bytes were a request of their own: a fifth of the kernel's time)
  constexpr int LPO = ZS / 8;
  const int o_row = lane / LPO, o_col = 8 * (lane % LPO);
  const unsigned o_own = 16 * W + o_row;
  const unsigned w_off = o_own * (unsigned)(ro.ws.t * (int)sizeof(T)) + o_col * kElem;
  const unsigned o_off = o_own * (unsigned)(ro.os.t * oe) + o_col * oe;
  Frag<T> X[NK], weights[2];
  // fp32: the wave's own rows of a chunk, the chunk's first where the sequence has ended
  auto load_own = [&](int it) {
    const int c = chunk_at(it);
    load_x<T, DX>(X, xb + (int64_t)c * kL * ro.xs.t * kElem, (int)own < sp.len - c * kL ? x_off : 8u * g * kElem);
  };
  // what a chunk's outputs are multiplied by, as they leave
  auto load_w = [&](Frag<T>& f, int it) {
    const int c = chunk_at(min(it, n - 1));
    const UniformPtr p = wb + (int64_t)c * kL * ro.ws.t * kElem;
    const unsigned off = (int)o_own < sp.len - c * kL ? w_off : (unsigned)o_col * kElem;
    if constexpr (SM::XL) {
      f.v = load_at<bf16x8>(p, off);
    } else {
      const f32x4 lo = load_at<f32x4>(p, off), hi = load_at<f32x4>(p, off + 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f.v[e] = lo[e];
        f.v[4 + e] = hi[e];
      }
    }
  };
  // A chunk's outputs, in the accumulators' order when they were put down, as rows to memory: a chunk later, so that neither
  // the LDS nor the stores are waited for.
  auto store_rows = [&](const Frag<T>& w, int it) {
    const int c = chunk_at(it);
    const f32x4 lo = *reinterpret_cast<const f32x4*>(&sm.out[W][o_row][o_col]), hi = *reinterpret_cast<const f32x4*>(&sm.out[W][o_row][o_col + 4]);
    const bool on = (int)o_own < sp.len - c * kL;
    const UniformPtr p = outb + (int64_t)c * kL * ro.os.t * oe;
    if (on) {
      if (sizeof(T) == 4 || ro.out_f32) {
        store_at<f32x4>(p, o_off, lo);
        store_at<f32x4>(p, o_off + 16, hi);
      } else {
        store_at<bf16x8>(p, o_off, bf16x8{(__bf16)lo[0], (__bf16)lo[1], (__bf16)lo[2], (__bf16)lo[3], (__bf16)hi[0], (__bf16)hi[1],
                                          (__bf16)hi[2], (__bf16)hi[3]});
      }
    }
    if (ro.r) {
      float r = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) r += lo[e] * (float)w.v[e];
#pragma unroll
      for (int e = 0; e < 4; ++e) r += hi[e] * (float)w.v[4 + e];
      r = group_sum<LPO>(r);
      if (on && o_col == 0) ro.r[((size_t)slice * a.chains + chain) * a.T + c * kL + o_own] = r;
    }
  };
  int place[NK];  // of rows of x, y and the state's copy alike
#pragma unroll
  for (int kk = 0; kk < NK; ++kk) place[kk] = row_place<T, DX, SM::PY>(kk, lane);
  const int z_place = tr_place<T>(SM::PZ, lane);
  // a chunk's scores, weighted: chunk it, gates in buffer gb
  auto scores = [&](f32x4 (&P)[4], const Frag<T> (&x)[NK], int it, int at, int gb) {
    const T* y0 = &sm.Y[at][0][0];
#pragma unroll
    for (int t = 0; t < 4; ++t) P[t] = zero4();
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
      for (int t = T0; t <= T1; ++t) mma(P[t], row_at<T>(y0 + place[kk] + 16 * t * SM::PY), x[kk]);
    const float bh = sm.bh[gb][own], bl = sm.bl[gb][own];
#pragma unroll
    for (int t = T0; t <= T1; ++t) {
      if (t == W) {
        const f32x4 kh = *reinterpret_cast<const f32x4*>(&sm.bh[gb][16 * t + 4 * g]);
        const f32x4 kl = *reinterpret_cast<const f32x4*>(&sm.bl[gb][16 * t + 4 * g]);
        const int live = sp.len - chunk_at(it) * kL - 16 * t;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 4 * g + r;
          const float d = REV ? (kh[r] - bh) + (kl[r] - bl) : (bh - kh[r]) + (bl - kl[r]);
          P[t][r] = (REV ? j >= l && j < live : j <= l) ? P[t][r] * (exp2_fast(d) * ro.in_scale) : 0.f;
        }
      } else {
        // e^(B_i - B_j) in two parts, from the query to the tile's edge and on to the key: both below 1 for decays
        const int edge = REV ? 16 * t : 16 * t + 15;
        const float eh = sm.bh[gb][edge], el = sm.bl[gb][edge];
        const float row = exp2_fast(REV ? (eh - bh) + (el - bl) : (bh - eh) + (bl - el));
        const f32x4 cf = *reinterpret_cast<const f32x4*>(&sm.cf[gb][16 * t + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) P[t][r] *= row * cf[r];
      }
    }
  };
  if constexpr (!SM::XL) load_own(0);
  if (ro.r) load_w(weights[0], 0);
  lds_barrier();
  lds_barrier();
  {
    int at = 0;  // it modulo NB
    // one chunk, whose parity GB is
    auto step = [&](auto parity, int it) {
      constexpr int GB = decltype(parity)::value;
      if constexpr (SM::XL) {
        const T* x = &sm.X[at][16 * W][0];
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) X[kk] = row_at<T>(x + place[kk]);
      }
      if (it > 0) store_rows(weights[1 - GB], it - 1);
      if (ro.r) load_w(weights[1 - GB], it + 1);
      const T* st = &sm.St[GB][0][0][0];
      const T* z0 = &sm.Z[at][0][0] + z_place;
      const float aw = sm.aw[GB][own];
      const int edge = REV ? sm.last[GB] : sm.first[GB];
      // far: the state before the chunk
      f32x4 acc[NZ], P[4];
#pragma unroll
      for (int z = 0; z < NZ; ++z) acc[z] = zero4();
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int z = 0; z < NZ; ++z)
#pragma unroll
          for (int s = 0; s < SM::NS; ++s) mma(acc[z], row_at<T>(st + place[kk] + (s * ZS + 16 * z) * SM::PS), X[kk]);
      scores(P, X, it, at, GB);
      if constexpr (!SM::XL) {
        if (it + 1 < n) load_own(it + 1);
      }
      // (one loop with a select made the scheduler's block longer and the gradient 440 us for 360)
      if (REV ? edge >= 0 : edge < kL) {  // a reset stands between the state and some tokens, whatever the state holds
        const bool cut = REV ? (int)own < edge : (int)own >= edge;
#pragma unroll
        for (int z = 0; z < NZ; ++z)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[z][r] = cut ? 0.f : acc[z][r] * aw;
      } else {
#pragma unroll
        for (int z = 0; z < NZ; ++z)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[z][r] *= aw;
      }
      // near
#pragma unroll
      for (int kk = T0 / 2; kk <= T1 / 2; ++kk) {
        const Frag<T> p = acc_frag<T>(P[2 * kk], P[2 * kk + 1]);
        Frag<T> q;
        if constexpr (SM::NS == 2) {
          f32x4 lo[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) lo[u][r] = P[2 * kk + u][r] - (float)(__bf16)P[2 * kk + u][r];
          q = acc_frag<T>(lo[0], lo[1]);
        }
#pragma unroll
        for (int z = 0; z < NZ; ++z) {
          const Frag<T> v = tr_at<T, SM::PZ>(z0 + 32 * kk * SM::PZ + 16 * z);
          mma(acc[z], v, p);
          if constexpr (SM::NS == 2) mma(acc[z], v, q);
        }
      }
#pragma unroll
      for (int z = 0; z < NZ; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[z][r] *= ro.out_scale;
#pragma unroll
      for (int z = 0; z < NZ; ++z) *reinterpret_cast<f32x4*>(&sm.out[W][l][16 * z + 4 * g]) = acc[z];
      at = at + 1 == SM::NB ? 0 : at + 1;
      lds_barrier();
    };
    for (int it = 0; it < n; it += 2) {
      step(std::integral_constant<int, 0>{}, it);
      if (it + 1 < n) step(std::integral_constant<int, 1>{}, it + 1);
    }
  }
  if (n & 1) store_rows(weights[0], n - 1);
  else store_rows(weights[1], n - 1);
}

constexpr int walk_threads(bool summary) { return summary ? 448 : 704; }

// One chain, slice and segment.  Waves 0 .. 3 form the outputs (SUMMARY: one wave, for the gates alone), the four
// behind them carry the state, one forms the gates, two load (where the other waves issued the loads, 36 KB a chunk, they stood
// still for a third of their time), and a chunk has one barrier.  SUMMARY: the state alone, from zeros, into
// the segment's slot.
template <typename T, int DX, bool SPLIT, bool REV, bool SUMMARY>
__device__ __forceinline__ void walk(const Args& a, const Role& ro, int chain, int slice, int seg, Smem<T, DX, SPLIT, SUMMARY>& sm) {
  using SM = Smem<T, DX, SPLIT, SUMMARY>;
  constexpr int NO = SUMMARY ? 1 : 4, ZS = SM::ZS, NZ = ZS / 16, NX = DX / 16 * NZ / 4, AH = SM::AHEAD;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool carries = wave >= NO && wave < NO + 4;
  const int b = chain / a.H, h = chain - b * a.H;
  Span sp = span_of(a, b);
  sp.len = __builtin_amdgcn_readfirstlane(sp.len);
  const int nc = (sp.len + kL - 1) / kL;
  const int c_lo = seg * a.chunks_per_segment, c_hi = min(nc, c_lo + a.chunks_per_segment), n = c_hi - c_lo;
  const size_t mat = (size_t)ro.dz * DX;
  auto chunk_at = [&](int it) { return REV ? c_hi - 1 - it : c_lo + it; };
  // a state's place in the accumulators' order: 16 bytes a lane
  const int sw = wave - NO, zt = sw % NZ, xt = sw / NZ * NX;
  auto slot_of = [&](int s) {
    return ro.slots + (((size_t)chain * a.segments + s) * ro.slices + slice) * (ZS * DX) + (size_t)sw * NX * 256 + lane * 4;
  };

  if constexpr (!SUMMARY) {
    if (ro.zero_idle) {
      const Idle idle = idle_of(a, sp, b);
      const int64_t ob = (a.offsets ? 0 : b * ro.os.b) + h * ro.os.h + slice * ZS + 4 * (tid % (ZS / 4));
      constexpr int kRows = walk_threads(false) / (ZS / 4);
      const int64_t own = (int64_t)seg * kRows + tid / (ZS / 4), step = (int64_t)a.segments * kRows;
      for (int64_t t = own; t < idle.front; t += step) store_out<T>(ro.out, ob + t * ro.os.t, zero4(), ro.out_f32);
      for (int64_t t = idle.from + own; t < idle.to; t += step) store_out<T>(ro.out, ob + t * ro.os.t, zero4(), ro.out_f32);
    }
  }

  if (carries) {
    // ---------------------------------------------------------------- the state
    f32x4 S[NX];  // rows 16 (xt + x) + 4 g + r of x, column 16 zt + l of z
    auto take_in = [&]() {
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        S[x] = zero4();
        if (ro.s_in) {
          const float* p = ro.s_in + chain * mat + (size_t)(slice * ZS + 16 * zt + l) * ro.s_i + (size_t)(16 * (xt + x) + 4 * g) * ro.s_j;
          if (ro.s_j == 1) S[x] = *reinterpret_cast<const f32x4*>(p);
          else
#pragma unroll
            for (int r = 0; r < 4; ++r) S[x][r] = p[(size_t)r * ro.s_j];
        }
      }
    };
    auto store_slot = [&](int s) {
      float* p = slot_of(s);
#pragma unroll
      for (int x = 0; x < NX; ++x) *reinterpret_cast<f32x4*>(p + x * 256) = S[x];
    };
    auto decay_by = [&](float d, bool reset) {
      if (reset) {  // whatever the state holds
#pragma unroll
        for (int x = 0; x < NX; ++x) S[x] = zero4();
      } else {
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[x][r] *= d;
      }
    };
    if constexpr (SUMMARY) {
      if (a.snapshot && seg == 0) {  // the state before, which the last segment may write over
        take_in();
        store_slot(a.segments - 1);
      }
#pragma unroll
      for (int x = 0; x < NX; ++x) S[x] = zero4();
    } else {
      // the state before the segment: the one before the sequence, then the segments between
      const int nseg = (nc + a.chunks_per_segment - 1) / a.chunks_per_segment;
      if (a.snapshot) {
        const float* p = slot_of(a.segments - 1);
#pragma unroll
        for (int x = 0; x < NX; ++x) S[x] = *reinterpret_cast<const f32x4*>(p + x * 256);
      } else {
        take_in();
      }
      for (int i = REV ? nseg - 1 : 0; REV ? i > seg : i < seg; i += REV ? -1 : 1) {
        const double d = ro.slot_log[(size_t)chain * a.segments + i];
        decay_by(exp2_fast((float)d), d == -INFINITY);
        const float* p = slot_of(i);
#pragma unroll
        for (int x = 0; x < NX; ++x) S[x] += *reinterpret_cast<const f32x4*>(p + x * 256);
      }
    }
    if (n > 0) {
      auto store_copy = [&](int it) {
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          const int slot = 2 * (xt + x) + (g >> 1), at = SM::SW ? 8 * (slot ^ swizzle<DX>(l)) + 4 * (g & 1) : 16 * (xt + x) + 4 * g;
          st4<T>(&sm.St[it & 1][0][16 * zt + l][at], S[x]);
          if constexpr (SM::NS == 2) {
            f32x4 lo;
#pragma unroll
            for (int r = 0; r < 4; ++r) lo[r] = S[x][r] - (float)(__bf16)S[x][r];
            st4<T>(&sm.St[it & 1][1][16 * zt + l][at], lo);
          }
        }
      };
      lds_barrier();
      if constexpr (!SUMMARY) store_copy(0);
      lds_barrier();
      int y_place[NX];
#pragma unroll
      for (int x = 0; x < NX; ++x) y_place[x] = tr_place_swizzled<T, DX, SM::PY>(xt + x, lane);
      const int z_place = tr_place<T>(SM::PZ, lane) + 16 * zt;
      int at = 0;  // it modulo NB
      for (int it = 0; it < n; ++it) {
        const T* y0 = &sm.Y[at][0][0];
        const T* z0 = &sm.Z[at][0][0] + z_place;
        const float dec = sm.dec[it & 1];
        const int first = sm.first[it & 1];
        // b z: the lane's eight tokens of every 32, as tr_at has them
        Frag<T> y[2][NX], zf[2][SM::NH];
        Frag<T> z[2];
        f32x4 bw[2][2];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          z[kk] = tr_at<T, SM::PZ>(z0 + 32 * kk * SM::PZ);
          bw[kk][0] = *reinterpret_cast<const f32x4*>(&sm.bw[it & 1][32 * kk + 4 * g]);
          bw[kk][1] = *reinterpret_cast<const f32x4*>(&sm.bw[it & 1][32 * kk + 16 + 4 * g]);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
          for (int x = 0; x < NX; ++x) y[kk][x] = tr_at<T, SM::PY>(y0 + y_place[x] + 32 * kk * SM::PY);
        at = at + 1 == SM::NB ? 0 : at + 1;
        auto update = [&](bool reset) {
          if (reset) {
            // rows that the reset cuts off may hold anything, and so may the chunk's first, which rows behind the end repeat
            const int lo = REV ? 0 : sm.last[it & 1], hi = min(REV ? first : kL, sp.len - chunk_at(it) * kL);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int j = 32 * kk + 16 * (e >> 2) + 4 * g + (e & 3);
                if (j >= lo && j < hi) continue;
                z[kk].v[e] = (T)0.f;
#pragma unroll
                for (int x = 0; x < NX; ++x) y[kk][x].v[e] = (T)0.f;
              }
          }
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)z[kk].v[e] * bw[kk][e >> 2][e & 3];
#pragma unroll
            for (int p = 0; p < SM::NH; ++p)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                zf[kk][p].v[e] = (T)v[e];
                if (p + 1 < SM::NH) v[e] -= (float)zf[kk][p].v[e];
              }
          }
          decay_by(dec, reset);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int p = 0; p < SM::NH; ++p)
#pragma unroll
              for (int x = 0; x < NX; ++x) mma(S[x], y[kk][x], zf[kk][p]);
        };
        // chunks without a reset have code of their own, which a summary does not gain from (20,480 tokens: 172 against 184 us)
        if (SUMMARY) update(first < kL);
        else if (first < kL) update(true);
        else update(false);
        if constexpr (!SUMMARY) store_copy(it + 1);
        lds_barrier();
      }
    }
    if constexpr (SUMMARY) {
      if (n > 0) store_slot(seg);
      return;
    } else {
      const bool ends = REV ? seg == 0 : (nc == 0 ? seg == 0 : n > 0 && c_hi == nc);  // the walk's last chunk is here
      if (!ends) return;
      float d = 0.f;
#pragma unroll
      for (int x = 0; x < NX; ++x) {
        const int i = slice * ZS + 16 * zt + l, j = 16 * (xt + x) + 4 * g;
        if (ro.s_out) *reinterpret_cast<f32x4*>(ro.s_out + chain * mat + (size_t)i * DX + j) = S[x];
        if (ro.dot)
#pragma unroll
          for (int r = 0; r < 4; ++r) d += S[x][r] * ro.dot[chain * mat + (size_t)i * ro.s_i + (size_t)(j + r) * ro.s_j];
      }
      if (ro.dot) {
        d = group_sum<64>(d);
        if (lane == 0) ro.dot_out[((size_t)chain * ro.slices + slice) * 4 + sw] = d;
      }
      return;
    }
  }

  if (n <= 0) return;
  if (wave >= NO + 4 && wave < NO + 6) {
    // ---------------------------------------------------------------- the loads
    // the first wave y and the gates, the second z and x
    auto load_chunks = [&](auto issue, auto count) {
      for (int i = 0; i < AH && i < n; ++i) issue(i);
      vm_wait<0>();
      lds_barrier();
      for (int it = 0; it < n; ++it) {
        if (it + AH < n) {
          issue(it + AH);
          // what has been issued just now may be under way, what was before must have landed
          if (AH == 1) vm_wait<0>();
          else vm_wait<decltype(count)::value>();
        } else {
          vm_wait<0>();
        }
        lds_barrier();
      }
    };
    if (wave == NO + 4) {
      const UniformPtr yb = uniform_ptr(rows_of<T>(ro.y, ro.ys, ro.y_share, a, sp, b, h));
      const RowLoads<T, DX, SM::PY, SM::SW> yl(lane, ro.ys.t);
      const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
      auto gates = [&](int it) {
        const int c = chunk_at(it);
        load_gates(a, sm.raw[it % (SM::NB + 1)], la0 + (int64_t)c * kL * a.ls.t, sp.len - c * kL, lane);
      };
      gates(0);
      vm_wait<0>();
      lds_barrier();
      // a chunk's gates come a chunk before its rows
      load_chunks(
          [&](int it) {
            const int c = chunk_at(it);
            gates(min(it + 1, n - 1));
            yl.load(sm.Y[it % SM::NB], yb + (int64_t)c * kL * ro.ys.t * (int)sizeof(T), sp.len - c * kL, lane);
          },
          std::integral_constant<int, RowLoads<T, DX, SM::PY, SM::SW>::U>{});
    } else {
      const UniformPtr zb = uniform_ptr(rows_of<T>(ro.z, ro.zs, ro.z_share, a, sp, b, h) + slice * ZS);
      const RowLoads<T, ZS, SM::PZ, false> zl(lane, ro.zs.t);
      lds_barrier();
      if constexpr (!SUMMARY && SM::XL) {
        const UniformPtr xb = uniform_ptr(rows_of<T>(ro.x, ro.xs, ro.x_share, a, sp, b, h));
        const RowLoads<T, DX, SM::PY, SM::SW> xl(lane, ro.xs.t);
        load_chunks(
            [&](int it) {
              const int c = chunk_at(it);
              zl.load(sm.Z[it % SM::NB], zb + (int64_t)c * kL * ro.zs.t * (int)sizeof(T), sp.len - c * kL, lane);
              xl.load(sm.X[it % SM::NB], xb + (int64_t)c * kL * ro.xs.t * (int)sizeof(T), sp.len - c * kL, lane);
            },
            std::integral_constant<int, RowLoads<T, ZS, SM::PZ, false>::U + RowLoads<T, DX, SM::PY, SM::SW>::U>{});
      } else {
        load_chunks(
            [&](int it) {
              const int c = chunk_at(it);
              zl.load(sm.Z[it % SM::NB], zb + (int64_t)c * kL * ro.zs.t * (int)sizeof(T), sp.len - c * kL, lane);
            },
            std::integral_constant<int, RowLoads<T, ZS, SM::PZ, false>::U>{});
      }
    }
    return;
  }
  // ---------------------------------------------------------------- the outputs, and the gates
  if (SUMMARY || wave == NO + 6) {
    Gates<REV, SM> gates(a, ro, sm, sp, c_lo, c_hi, lane);
    lds_barrier();
    gates.template form<0>(0);
    lds_barrier();
    for (int it = 0; it < n; it += 2) {
      gates.template form<1>(it + 1);
      lds_barrier();
      if (it + 1 < n) {
        gates.template form<0>(it + 2);
        lds_barrier();
      }
    }
    if (SUMMARY && slice == 0 && lane == 0) ro.slot_log[(size_t)chain * a.segments + seg] = gates.reset ? -INFINITY : gates.total;
    return;
  }
  if constexpr (!SUMMARY) {
    if (wave == 0) walk_outputs<T, DX, SPLIT, REV, 0>(a, ro, chain, slice, sp, c_lo, c_hi, lane, sm);
    else if (wave == 1) walk_outputs<T, DX, SPLIT, REV, 1>(a, ro, chain, slice, sp, c_lo, c_hi, lane, sm);
    else if (wave == 2) walk_outputs<T, DX, SPLIT, REV, 2>(a, ro, chain, slice, sp, c_lo, c_hi, lane, sm);
    else walk_outputs<T, DX, SPLIT, REV, 3>(a, ro, chain, slice, sp, c_lo, c_hi, lane, sm);
  }
}

constexpr unsigned kGridX = 1u << 22;  // a launch has less than 2^32 threads along x; what is more lies along z

// Workgroups of a launch: along x, eight chains at a time, one on each XCD, with the roles and slices of a chain next to
// each other, so that rows which they share come into one L2 once; along y the segments.  An XCD takes an eighth of the
// chains in order.
template <typename T, int DX, bool SPLIT, bool SUMMARY>
__global__ __launch_bounds__(walk_threads(SUMMARY)) void la_walk_kernel(Args a) {
  __shared__ __align__(16) Smem<T, DX, SPLIT, SUMMARY> sm;
  const int block = blockIdx.z * kGridX + blockIdx.x, at = block / 8, group = at / a.slots_per_group;
  int k = at - group * a.slots_per_group, role = 0;
  const int each = (a.chains + 7) / 8, chain = block % 8 * each + group;
  if (group >= each || chain >= a.chains) return;
  while (role + 1 < a.roles && k >= a.role[role].slices) k -= a.role[role++].slices;
  const Role& ro = a.role[role];
  const bool rev = ro.reverse != 0;
  const int seg = (int)blockIdx.y + (SUMMARY && rev ? 1 : 0);
  if (rev) {
    if constexpr (SPLIT || SUMMARY) walk<T, DX, SPLIT, true, SUMMARY>(a, ro, chain, k, seg, sm);
  } else {
    walk<T, DX, SPLIT, false, SUMMARY>(a, ro, chain, k, seg, sm);
  }
}

// A few tokens, one after the other: 32 rows of a state a workgroup, each row on DX / 4 lanes, read once and
// written once.
template <typename T, int DX>
__global__ __launch_bounds__(kThreads) void la_step_kernel(Args a) {
  constexpr int LPR = DX / 4, RPP = kThreads / LPR, NP = kStepRows / RPP;
  const Role& ro = a.role[0];
  const int slices = ro.dz / kStepRows, chain = blockIdx.x / slices, slice = blockIdx.x - chain * slices;
  const int b = chain / a.H, h = chain - b * a.H;
  const int col = 4 * (threadIdx.x % LPR), row = threadIdx.x / LPR;
  const Span sp = span_of(a, b);
  const size_t mat = (size_t)ro.dz * DX;
  const T* xb = rows_of<T>(ro.x, ro.xs, ro.x_share, a, sp, b, h) + col;
  const T* yb = rows_of<T>(ro.y, ro.ys, ro.y_share, a, sp, b, h) + col;
  const T* zb = rows_of<T>(ro.z, ro.zs, ro.z_share, a, sp, b, h) + slice * kStepRows + row;
  T* ob = rows_of<T>(ro.out, ro.os, 1, a, sp, b, h) + slice * kStepRows + row;
  const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
  const size_t s0 = chain * mat + (size_t)(slice * kStepRows + row) * DX + col;
  f32x4 S[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    S[i] = zero4();
    if (ro.s_in) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(ro.s_in + s0 + (size_t)i * RPP * DX));
  }
  for (int t = 0; t < sp.len; ++t) {
    const f32x4 x = ld4(xb + t * ro.xs.t), y = ld4(yb + t * ro.ys.t);
    const double gate = gate_of(a, la0 + (int64_t)t * a.ls.t);
    const bool reset = gate < kReset;
    const float d = exp2_fast((float)gate);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float z = to_f32(zb[t * ro.zs.t + i * RPP]);
      float o = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[i][e] = (reset ? 0.f : S[i][e] * d) + z * y[e];
        o += S[i][e] * x[e];
      }
      o = group_sum<LPR>(o);
      if (col == 0) ob[t * ro.os.t + i * RPP] = from_f32<T>(o * ro.out_scale);
    }
  }
  if (ro.s_out)
#pragma unroll
    for (int i = 0; i < NP; ++i) __builtin_nontemporal_store(S[i], reinterpret_cast<f32x4*>(ro.s_out + s0 + (size_t)i * RPP * DX));
}

// Gradient rows that several heads share: the sum of their parts, in order.  Parts are [H][rows][d] fp32: the walk tells a chunk's
// rows apart by 32-bit offsets, which H d between them would pass with many heads.
struct Shared {
  const float* part;
  void* out;
  Strides os;
  int heads, share, d, f32;
};
struct SumArgs {
  int64_t rows, T;  // of all sequences, and of one (packed: as if of one sequence)
  Shared side[3];
};
__global__ __launch_bounds__(kThreads) void la_sum_kernel(SumArgs a) {
  const Shared& s = a.side[blockIdx.y];
  const int quads = s.d / 4;
  const int64_t per = (int64_t)s.heads * quads, all = per * a.rows;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < all; at += (int64_t)gridDim.x * kThreads) {
    const int64_t row = at / per, b = row / a.T, t = row - b * a.T;
    const int rest = (int)(at - row * per), hh = rest / quads, c = 4 * (rest - hh * quads);
    const float* p = s.part + ((int64_t)hh * s.share * a.rows + row) * s.d + c;
    f32x4 v = zero4();
    for (int i = 0; i < s.share; ++i) v += *reinterpret_cast<const f32x4*>(p + i * a.rows * s.d);
    store_out<__bf16>(s.out, b * s.os.b + t * s.os.t + hh * s.os.h + c, v, s.f32);
  }
}

// dlog alpha of one chain: the sums from the end of rq - rk (over the slices), plus the state's product, in 64 bits.  They
// begin anew at a reset: what stands behind it sums up to 0, but for its roundings and for what is infinite or NaN.  A
// thread takes four tokens that follow each other, so that a few thousand tokens are one round of loads and one scan
// (one token a thread: 24 us for 64 chains of 4096, now 17).
constexpr int kGateThreads = 1024, kGateRun = 4;
typedef f32x4 f32x4_any __attribute__((aligned(4)));
struct GateArgs {
  Args a;
  const float *rq, *rk, *dot;  // [slices][chains][T], the same, [chains][dot_slices] or null
  int q_slices, k_slices, dot_slices;
  void* out;
};
__global__ __launch_bounds__(kGateThreads) void la_gate_kernel(GateArgs q) {
  const Args& a = q.a;
  const int chain = blockIdx.x, b = chain / a.H, h = chain - b * a.H;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const Span sp = span_of(a, b);
  __shared__ double tops[kGateThreads / 64];
  __shared__ int cut[kGateThreads / 64];  // a reset among a wave's tokens
  __shared__ double behind;
  const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
  const int64_t row0 = a.offsets ? 0 : (int64_t)b * a.T;
  auto store = [&](int64_t row, float v) {
    const int64_t at = row * a.H + h;
    if (a.gate_bf16) static_cast<__bf16*>(q.out)[at] = (__bf16)v;
    else static_cast<float*>(q.out)[at] = v;
  };
  if (tid == 0) {
    double s = 0.0;
    if (q.dot)
      for (int i = 0; i < q.dot_slices; ++i) s += (double)q.dot[(size_t)chain * q.dot_slices + i];
    behind = s;
  }
  __syncthreads();
  for (int last = sp.len; last > 0; last -= kGateThreads * kGateRun) {  // thread 0 the last tokens of the stretch
    const int t0 = last - kGateRun * (tid + 1);                          // may be below 0
    unsigned bits[kGateRun];
#pragma unroll
    for (int i = 0; i < kGateRun; ++i) bits[i] = t0 + i >= 0 ? gate_bits(a, la0 + (int64_t)(t0 + i) * a.ls.t) : 0u;
    double r[kGateRun] = {0.0, 0.0, 0.0, 0.0};
    auto add = [&](const float* p, int slices, double sign) {
      for (int s = 0; s < slices; ++s, p += (size_t)a.chains * a.T) {
        if (t0 >= 0) {
          const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p + t0);
#pragma unroll
          for (int i = 0; i < kGateRun; ++i) r[i] += sign * (double)v[i];
        } else {
#pragma unroll
          for (int i = 0; i < kGateRun; ++i)
            if (t0 + i >= 0) r[i] += sign * (double)p[t0 + i];
        }
      }
    };
    add(q.rq + (size_t)chain * a.T, q.q_slices, 1.0);
    add(q.rk + (size_t)chain * a.T, q.k_slices, -1.0);
    bool reset[kGateRun], any = false;
#pragma unroll
    for (int i = 0; i < kGateRun; ++i) {
      reset[i] = gate_value(a, bits[i]) < kReset;
      any = any || reset[i];
    }
#pragma unroll
    for (int i = kGateRun - 2; i >= 0; --i) r[i] += reset[i + 1] ? 0.0 : r[i + 1];
    // over the lanes, whose tokens come before those of the lanes below: each lane's sum since the last reset
    const double own = reset[0] ? 0.0 : r[0];
    const uint64_t resets = __ballot(any);
    const bool cut_before = (resets & ((1ull << lane) - 1)) != 0;
    double sum = own;
    if (resets == 0) {
      sum = wave_running(own);
    } else {
      const int since = cut_before || any ? 63 - __builtin_clzll(resets & (~0ull >> (63 - lane))) : 0;  // the sum's first lane
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double o = __shfl_up(sum, d, 64);
        if (lane - d >= since) sum += o;
      }
    }
    const double up = __shfl_up(sum, 1, 64);
    if (lane == 63) {
      tops[w] = sum;
      cut[w] = resets != 0;
    }
    __syncthreads();
    double base = behind;
    for (int i = 0; i < w; ++i) base = (cut[i] ? 0.0 : base) + tops[i];
    if (cut_before) base = 0.0;
    if (lane > 0) base += up;
#pragma unroll
    for (int i = kGateRun - 1; i >= 0; --i) {
      if (t0 + i >= 0) store(row0 + sp.row0 + t0 + i, reset[i] ? 0.f : (float)(r[i] + base));
      if (reset[i]) base = 0.0;
    }
    __syncthreads();
    if (tid == kGateThreads - 1) behind = base + own;
    __syncthreads();
  }
  const Idle idle = idle_of(a, sp, b);
  for (int64_t t = tid; t < idle.front; t += kGateThreads) store(row0 + t, 0.f);
  for (int64_t t = idle.from + tid; t < idle.to; t += kGateThreads) store(row0 + t, 0.f);
}

// ---------------------------------------------------------------- host

// Where a call's parts of the workspace lie; base null: sizes alone.
struct Space {
  char* at;
  explicit Space(void* p) : at(static_cast<char*>(p)) {}
  template <typename U>
  U* take(size_t n) {
    U* r = reinterpret_cast<U*>(at);
    at += (n * sizeof(U) + 255) / 256 * 256;
    return r;
  }
};

constexpr int kStepTokens = 8;

// Segments of a sequence.  A workgroup has a CU to itself, so `groups` of them (chains, roles and slices) take
// ceil(groups / 256) turns of all its chunks; cut in P they take turns of a P-th, behind a summary, which takes about
// half as long for a chunk, two to a CU, and a launch that costs some six chunks.  The P with the least of these.  (One sequence of
// 20,480 tokens, 16 heads of 128: 8 segments, 172 us; 4 take the same, 2 316, the whole 385.  42 chains of up to 777 tokens in fp32: 45 whole,
// 59 with 2.  One of 4096 tokens, 16 heads: 8 segments, 50 us, though 4 would take 44.)
void split_of(const ccq_linear_attn_params& p, int groups, int* segments, int* per) {
  const int nc = (p.T - 1) / kL + 1;
  *segments = 1;
  *per = nc;
  int64_t least = 0;
  for (int s = 1; s <= 32 && s <= nc; ++s) {
    const int each = (nc + s - 1) / s;
    if (s > 1 && (s - 1) * each >= nc) continue;  // the last one would be empty
    int64_t cost = 2 * (((int64_t)groups * s + 255) / 256) * each;
    if (s > 1) cost += 12 + (((int64_t)groups * (s - 1) + 511) / 512) * each * 2 + s;
    if (s == 1 || cost < least) {
      least = cost;
      *segments = s;
      *per = each;
    }
  }
}

Args base_of(const ccq_linear_attn_params& p) {
  Args a{};
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.chains = p.B * p.H;
  a.la = p.log_alpha;
  a.ls = Strides{p.la_stride_b, p.la_stride_t, p.la_stride_h};
  a.gate_bf16 = p.gate_dtype == CCQ_DTYPE_BF16;
  a.lengths = p.lengths;
  a.offsets = p.offsets;
  a.rows = p.rows;
  a.segments = 1;
  return a;
}

void space_for_segments(Args& a, int dx, Space& sp) {
  if (a.segments <= 1) return;
  for (int i = 0; i < a.roles; ++i) {
    Role& r = a.role[i];
    r.slots = sp.take<float>((size_t)a.chains * a.segments * r.dz * dx);
    r.slot_log = sp.take<double>((size_t)a.chains * a.segments);
  }
}

// The forward's role and launch; returns the workspace's end.
char* plan_forward(const ccq_linear_attn_params& p, Args& a, void* workspace) {
  a = base_of(p);
  Role& r = a.role[0];
  r.x = p.q;
  r.y = p.k;
  r.z = p.v;
  r.xs = Strides{p.q_stride_b, p.q_stride_t, p.q_stride_h};
  r.ys = Strides{p.k_stride_b, p.k_stride_t, p.k_stride_h};
  r.zs = Strides{p.v_stride_b, p.v_stride_t, p.v_stride_h};
  r.x_share = p.H / p.H_q;
  r.y_share = p.H / p.H_k;
  r.z_share = p.H / p.H_v;
  r.out = p.o;
  r.os = Strides{p.o_stride_b, p.o_stride_t, p.o_stride_h};
  r.out_f32 = p.dtype == CCQ_DTYPE_F32;
  r.s_in = p.S0;
  r.s_i = p.d_k;
  r.s_j = 1;
  r.s_out = p.S_out;
  r.in_scale = 1.f;
  r.out_scale = p.scale;
  r.dz = p.d_v;
  r.slices = p.d_v / kSlice;
  a.roles = 1;
  a.slots_per_group = r.slices;
  Space sp(workspace);
  if (p.T > kStepTokens) {
    split_of(p, a.chains * r.slices, &a.segments, &a.chunks_per_segment);
    a.snapshot = a.segments > 1 && p.S0 != nullptr && p.S0 == p.S_out;
    space_for_segments(a, p.d_k, sp);
  }
  return sp.at;
}

template <typename T, int DX, bool SPLIT>
hipError_t run_walk(const Args& a, hipStream_t stream) {
  const unsigned groups = (unsigned)((a.chains + 7) / 8 * 8) * a.slots_per_group;
  const unsigned x = groups < kGridX ? groups : kGridX, z = (groups - 1) / kGridX + 1;
  if (a.segments > 1) la_walk_kernel<T, DX, false, true><<<dim3(x, a.segments - 1, z), walk_threads(true), 0, stream>>>(a);
  la_walk_kernel<T, DX, SPLIT, false><<<dim3(x, a.segments, z), walk_threads(false), 0, stream>>>(a);
  return hipGetLastError();
}

template <bool SPLIT>
hipError_t run_walk(const Args& a, int dtype, int dx, hipStream_t stream) {
  if (dtype == CCQ_DTYPE_BF16) return dx == 128 ? run_walk<__bf16, 128, SPLIT>(a, stream) : run_walk<__bf16, 64, SPLIT>(a, stream);
  return dx == 128 ? run_walk<float, 128, SPLIT>(a, stream) : run_walk<float, 64, SPLIT>(a, stream);
}

// The gradient's roles: dq and dk contract over d_v, dv over d_k: one launch where these are the same, else two.
struct BackPlan {
  Args a[2];
  int dx[2], launches;
  SumArgs sum;
  int sums, most;
  GateArgs gate;
  char* end;
};
BackPlan plan_backward(const ccq_linear_attn_bwd_params& q) {
  const ccq_linear_attn_params& p = q.fwd;
  BackPlan bp{};
  Space sp(q.workspace);
  const Strides xs[3] = {{p.q_stride_b, p.q_stride_t, p.q_stride_h}, {p.k_stride_b, p.k_stride_t, p.k_stride_h},
                         {p.v_stride_b, p.v_stride_t, p.v_stride_h}};
  const Strides gs[3] = {{q.dq_stride_b, q.dq_stride_t, q.dq_stride_h}, {q.dk_stride_b, q.dk_stride_t, q.dk_stride_h},
                         {q.dv_stride_b, q.dv_stride_t, q.dv_stride_h}};
  const Strides ds{q.do_stride_b, q.do_stride_t, q.do_stride_h};
  const void* in[3] = {p.q, p.k, p.v};
  void* out[3] = {q.dq, q.dk, q.dv};
  const int share[3] = {p.H / p.H_q, p.H / p.H_k, p.H / p.H_v}, dim[3] = {p.d_k, p.d_k, p.d_v};
  const bool grad_f32 = q.grad_dtype == CCQ_DTYPE_F32;
  const size_t rows = p.offsets ? (size_t)p.rows : (size_t)p.B * p.T, chains = (size_t)p.B * p.H;
  Role role[3] = {};
  // operands of the three roles among q (0), k (1), v (2) and d_o (3)
  const int ops[3][3] = {{3, 2, 1}, {2, 3, 0}, {1, 0, 3}};
  for (int i = 0; i < 3; ++i) {
    Role& r = role[i];
    const void** ptr[3] = {&r.x, &r.y, &r.z};
    Strides* st[3] = {&r.xs, &r.ys, &r.zs};
    int* sh[3] = {&r.x_share, &r.y_share, &r.z_share};
    for (int o = 0; o < 3; ++o) {
      const int k = ops[i][o];
      *ptr[o] = k == 3 ? q.d_o : in[k];
      *st[o] = k == 3 ? ds : xs[k];
      *sh[o] = k == 3 ? 1 : share[k];
    }
    r.dz = dim[i];
    r.slices = dim[i] / kSlice;
    r.reverse = i > 0;
    r.in_scale = i > 0 ? p.scale : 1.f;
    r.out_scale = i > 0 ? 1.f : p.scale;
    r.s_in = i == 0 ? p.S0 : q.dS_out;
    r.s_i = i < 2 ? 1 : p.d_k;  // the states of dq and dk are transposed
    r.s_j = i < 2 ? p.d_k : 1;
    if (share[i] > 1) {
      float* part = sp.take<float>(rows * p.H * dim[i]);
      r.out = part;
      r.os = Strides{(int64_t)p.T * dim[i], dim[i], (int64_t)rows * dim[i]};
      r.out_f32 = 1;
      Shared& s = bp.sum.side[bp.sums++];
      s = Shared{part, out[i], gs[i], p.H / share[i], share[i], dim[i], grad_f32};
      const int quads = s.heads * dim[i] / 4;
      if (quads > bp.most) bp.most = quads;
    } else {
      r.out = out[i];
      r.os = gs[i];
      r.out_f32 = grad_f32;
    }
    r.zero_idle = 1;
    if (q.dlog_alpha && i < 2) {
      r.w = in[i];
      r.ws = xs[i];
      r.w_share = share[i];
      r.r = sp.take<float>((size_t)r.slices * chains * p.T);
    }
  }
  if (q.dlog_alpha && q.dS_out) {
    role[0].dot = q.dS_out;
    role[0].dot_out = sp.take<float>(chains * role[0].slices * 4);
  }
  role[2].s_out = q.dS0;
  const bool one = p.d_k == p.d_v;
  bp.launches = one ? 1 : 2;
  for (int i = 0; i < bp.launches; ++i) {
    Args& a = bp.a[i];
    a = base_of(p);
    bp.dx[i] = i == 0 ? p.d_v : p.d_k;
    const int from = i == 0 ? 0 : 2, to = one || i == 1 ? 3 : 2;
    for (int k = from; k < to; ++k) {
      a.slots_per_group += role[k].slices;
      a.role[a.roles++] = role[k];
    }
    split_of(p, a.chains * a.slots_per_group, &a.segments, &a.chunks_per_segment);
    space_for_segments(a, bp.dx[i], sp);
  }
  bp.sum.rows = (int64_t)rows;
  bp.sum.T = p.offsets ? p.rows : p.T;
  bp.gate.a = base_of(p);
  bp.gate.rq = role[0].r;
  bp.gate.rk = role[1].r;
  bp.gate.dot = role[0].dot_out;
  bp.gate.q_slices = role[0].slices;
  bp.gate.k_slices = role[1].slices;
  bp.gate.dot_slices = role[0].slices * 4;
  bp.gate.out = q.dlog_alpha;
  bp.end = sp.at;
  return bp;
}

// Workgroups of the sum over shared heads.
unsigned sum_blocks(const BackPlan& bp) {
  const uint64_t n = ((uint64_t)bp.most * bp.sum.rows + kThreads - 1) / kThreads;
  return (unsigned)(n < 8192 ? n : 8192);
}

}  // namespace

size_t linear_attn_workspace_bytes(const ccq_linear_attn_params& p) {
  Args a;
  return (size_t)(plan_forward(p, a, nullptr) - static_cast<char*>(nullptr));
}

hipError_t launch_linear_attn(const ccq_linear_attn_params& p, hipStream_t stream) {
  Args a;
  plan_forward(p, a, p.workspace);
  if (p.T <= kStepTokens) {
    const unsigned grid = (unsigned)a.chains * (a.role[0].dz / kStepRows);
    if (p.dtype == CCQ_DTYPE_BF16) {
      if (p.d_k == 128) la_step_kernel<__bf16, 128><<<grid, kThreads, 0, stream>>>(a);
      else la_step_kernel<__bf16, 64><<<grid, kThreads, 0, stream>>>(a);
    } else {
      if (p.d_k == 128) la_step_kernel<float, 128><<<grid, kThreads, 0, stream>>>(a);
      else la_step_kernel<float, 64><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
  }
  // 16-bit inputs: scores and the state's copy in one part of 2^-8 each on the way to o, which is rounded to 2^-8 itself; the state stays fp32.
  // o is 2.35e-3 off (relative, over all of it) where its own rounding alone is 1.66e-3; two parts, as in the gradient, leave just that
  // and take 112 us for 99, and 190 for 172 over 20,480 tokens.
  return run_walk<false>(a, p.dtype, p.d_k, stream);
}

size_t linear_attn_backward_workspace_bytes(const ccq_linear_attn_bwd_params& q) {
  ccq_linear_attn_bwd_params none = q;
  none.workspace = nullptr;
  return (size_t)(plan_backward(none).end - static_cast<char*>(nullptr));
}

hipError_t launch_linear_attn_backward(const ccq_linear_attn_bwd_params& q, hipStream_t stream) {
  const BackPlan bp = plan_backward(q);
  for (int i = 0; i < bp.launches; ++i) {
    const hipError_t e = run_walk<true>(bp.a[i], q.fwd.dtype, bp.dx[i], stream);
    if (e != hipSuccess) return e;
  }
  if (bp.sums) la_sum_kernel<<<dim3(sum_blocks(bp), bp.sums), kThreads, 0, stream>>>(bp.sum);
  if (q.dlog_alpha) la_gate_kernel<<<bp.gate.a.chains, kGateThreads, 0, stream>>>(bp.gate);
  return hipGetLastError();
}

}  // namespace ccq
