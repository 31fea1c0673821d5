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
// The walk.  A workgroup of four waves owns one chain (sequence and head) and a slice of 32 columns of z, keeps
// its 32 x d_x part of the state in MFMA accumulators, and goes over the chain's 64-token chunks:
//   scores   K X^T by 16 x 16 tiles, wave w the queries 16 w .. 16 w + 15, against the keys its direction allows;
//            the tiles, weighted by e^{B_i - B_j} element by element, are the B operand of
//   near     out^T += Z^T P^T as they lie in the registers;
//   far      out^T += a_i St X^T with the state's copy St in LDS, in the inputs' type;
//   update   S^T = e^{B_L} S^T + Y^T (b z), b z as a sum of three bf16 where the inputs have 16 bits: what enters a
//            state, which later tokens and calls build on, is right to 2^-24.
// Weights of pairs, not e^{B_i} e^{-B_j}: nothing leaves fp32's range whatever the decay.  Running sums are
// formed in 64 bits and kept as two floats, in units of log 2.
#include "ccq_prefill_common.hpp"

namespace ccq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kSlice = 32;             // columns of z that a workgroup owns
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kGateFloor = -1.0e4f;  // log decays below count as this: e^-10000 is 0, sums of 64 stay exact enough

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
  int zero_tail;                  // rows behind a sequence's end are set to 0
  const void* w;                  // gradient: rows of the slice's columns, whose products with the outputs are summed
  Strides ws;
  int w_share;
  float* r;                       // [slices][chains][T], or null
  const float* s_in;              // state before, or null; entry (dz, dx) at dz s_i + dx s_j of the chain's
  int s_i, s_j;
  float* s_out;                   // state behind, [dz][dx] rows, or null
  const float* dot;               // matrix whose product with the state behind is summed (strides s_i, s_j), or null
  float* dot_out;                 // [chains][slices]
  float in_scale, out_scale;
  int reverse, slices, dz;
  float* slots;                   // summaries of segments, or null with one segment
  double* slot_log;               // [chains][segments] their log decays, in units of log 2
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

template <typename T>
__device__ __forceinline__ T* rows_of(const void* p, const Strides& s, int share, const Args& a, const Span& sp, int b, int h) {
  return const_cast<T*>(static_cast<const T*>(p)) + (a.offsets ? sp.row0 * s.t : b * s.b) + (h / share) * s.h;
}

// log2 of the decay of one token.
__device__ __forceinline__ double gate_of(const Args& a, int64_t at) {
  if (a.la == nullptr) return 0.0;
  float g = a.gate_bf16 ? (float)static_cast<const __bf16*>(a.la)[at] : static_cast<const float*>(a.la)[at];
  g = g < kGateFloor ? kGateFloor : g;  // NaN stays
  return (double)g * kLog2e;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Four entries of a row, whatever it holds.
template <typename T>
__device__ __forceinline__ void store_out(void* p, int64_t at, const f32x4& v, int f32) {
  if (sizeof(T) == 4 || f32) *reinterpret_cast<f32x4*>(static_cast<float*>(p) + at) = v;
  else *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(p) + at) = to_bf16x4(v);
}

template <typename T, int DX, bool SPLIT>
struct Smem {
  static constexpr int PY = DX + 16 / (int)sizeof(T), PZ = kSlice + 16 / (int)sizeof(T);
  static constexpr int NH = sizeof(T) == 2 ? 3 : 1;             // parts of b z
  static constexpr int NS = sizeof(T) == 2 && SPLIT ? 2 : 1;    // parts of the state's copy
  T Y[2][kL][PY];
  T Z[2][kL][PZ];
  T Zw[NH][kL][PZ];
  T St[NS][kSlice][PY];
  float bh[2][kL], bl[2][kL];  // running sums, as two floats
  float aw[2][kL], bw[2][kL];  // weights of the state for each query, of each key in the state
  float dec[2];
  float red[kWaves];
};

template <typename T, int DX>
__device__ __forceinline__ void load_x(Frag<T> (&f)[DX / 32], const T* p) {
#pragma unroll
  for (int kk = 0; kk < DX / 32; ++kk) {
    if constexpr (sizeof(T) == 2) {
      f[kk].v = *reinterpret_cast<const bf16x8*>(p + 32 * kk);
    } else {
      const f32x4 lo = *reinterpret_cast<const f32x4*>(p + 32 * kk), hi = *reinterpret_cast<const f32x4*>(p + 32 * kk + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[kk].v[e] = lo[e];
        f[kk].v[4 + e] = hi[e];
      }
    }
  }
}

// Rows 0 .. n - 1 (COLS entries every `step`) of a chunk straight into an LDS tile of pitch P, rows n .. 63 as row 0
// (their weights are 0).  The caller waits.
template <typename T, int COLS, int P>
__device__ __forceinline__ void load_rows(T (*dst)[P], const T* src, int64_t step, int n, int w, int lane) {
  constexpr int U = P * (int)sizeof(T) / 16, DU = COLS * (int)sizeof(T) / 16, EPU = 16 / (int)sizeof(T);
  const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) T*)&dst[0][0];
#pragma unroll
  for (int m = 0; m < (U + kWaves - 1) / kWaves; ++m) {
    const int j = w + kWaves * m;
    if (j >= U) break;
    const int u = 64 * j + lane, row = u / U, slot = u - row * U;
    const T* p = src + (slot < DU && row < n ? row * step + slot * EPU : 0);
    const unsigned m0 = __builtin_amdgcn_readfirstlane(base + 1024u * (unsigned)j);
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(m0), "v"(p) : "memory", "m0");
  }
}

// The weights of a chunk's 64 tokens into buffer `buf`; one wave, lane t token t, g its log2 decay (0 behind the end).
template <bool REV, typename SM>
__device__ __forceinline__ double form_gates(SM& sm, int buf, double g, bool live, float in_scale, int lane) {
  double s = g;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double up = __shfl_up(s, off, 64);
    if (lane >= off) s += up;
  }
  const double all = __shfl(s, 63, 64);
  const float hi = (float)s;
  sm.bh[buf][lane] = hi;
  sm.bl[buf][lane] = (float)(s - (double)hi);
  const float up = exp2_fast((float)s), down = exp2_fast((float)(all - s));
  sm.aw[buf][lane] = REV ? down : up;
  sm.bw[buf][lane] = live ? (REV ? up : down) * in_scale : 0.f;
  if (lane == 0) sm.dec[buf] = exp2_fast((float)all);
  return all;
}

// One chain, slice and segment.  SUMMARY: the state alone, from zeros, into the segment's slot.
template <typename T, int DX, bool SPLIT, bool REV, bool SUMMARY>
__device__ __forceinline__ void walk(const Args& a, const Role& ro, int chain, int slice, int seg, Smem<T, DX, SPLIT>& sm) {
  using SM = Smem<T, DX, SPLIT>;
  constexpr int NX = DX / 16 / kWaves, NZ = kSlice / 16, NK = DX / 32;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = chain / a.H, h = chain - b * a.H;
  const Span sp = span_of(a, b);
  const int nc = (sp.len + kL - 1) / kL;
  const int c_lo = seg * a.chunks_per_segment, c_hi = min(nc, c_lo + a.chunks_per_segment), n = c_hi - c_lo;
  constexpr int kGateWave = REV ? kWaves - 1 : 0;  // the wave with the fewest score tiles
  const size_t mat = (size_t)ro.dz * DX;

  const T* xb = rows_of<T>(ro.x, ro.xs, ro.x_share, a, sp, b, h);
  const T* yb = rows_of<T>(ro.y, ro.ys, ro.y_share, a, sp, b, h);
  const T* zb = rows_of<T>(ro.z, ro.zs, ro.z_share, a, sp, b, h) + slice * kSlice;
  const T* wb = ro.r ? rows_of<T>(ro.w, ro.ws, ro.w_share, a, sp, b, h) + slice * kSlice : nullptr;
  const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
  const int64_t ob = (a.offsets ? sp.row0 * ro.os.t : b * ro.os.b) + h * ro.os.h + slice * kSlice;

  // a state's place in the accumulators' order: 16 bytes a lane
  auto slot_of = [&](int s) {
    return ro.slots + (((size_t)chain * a.segments + s) * ro.slices + slice) * (kSlice * DX) + (size_t)w * NX * NZ * 256 + lane * 4;
  };
  f32x4 S[NX][NZ];
  auto take_in = [&]() {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
        S[x][z] = zero4();
        if (ro.s_in) {
          const float* p = ro.s_in + chain * mat + (size_t)(slice * kSlice + 16 * z + l) * ro.s_i +
                           (size_t)(16 * (w * NX + x) + 4 * g) * ro.s_j;
          if (ro.s_j == 1) S[x][z] = *reinterpret_cast<const f32x4*>(p);
          else
#pragma unroll
            for (int r = 0; r < 4; ++r) S[x][z][r] = p[(size_t)r * ro.s_j];
        }
      }
  };
  auto store_slot = [&](int s) {
    float* p = slot_of(s);
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int z = 0; z < NZ; ++z) *reinterpret_cast<f32x4*>(p + (x * NZ + z) * 256) = S[x][z];
  };
  auto decay_by = [&](float d) {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int z = 0; z < NZ; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[x][z][r] = d == 0.f ? 0.f : S[x][z][r] * d;
  };

  if constexpr (SUMMARY) {
    if (a.snapshot && seg == 0) {  // the state before, which the last segment may write over
      take_in();
      store_slot(a.segments - 1);
    }
    if (n <= 0) return;
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int z = 0; z < NZ; ++z) S[x][z] = zero4();
  } else {
    if (ro.zero_tail && a.offsets == nullptr) {  // rows of no token
      const int last = seg == a.segments - 1 ? a.T : min(a.T, (c_lo + a.chunks_per_segment) * kL);
      for (int t = max(sp.len, c_lo * kL) + (tid >> 3); t < last; t += kThreads / 8)
        store_out<T>(ro.out, ob + (int64_t)t * ro.os.t + 4 * (tid & 7), zero4(), ro.out_f32);
    }
    if (n <= 0 && !(nc == 0 && seg == 0)) return;
    // the state before the segment: the one before the sequence, then the segments between
    const int nseg = (nc + a.chunks_per_segment - 1) / a.chunks_per_segment;
    if (a.snapshot) {
      const float* p = slot_of(a.segments - 1);
#pragma unroll
      for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int z = 0; z < NZ; ++z) S[x][z] = *reinterpret_cast<const f32x4*>(p + (x * NZ + z) * 256);
    } else {
      take_in();
    }
    for (int i = REV ? nseg - 1 : 0; REV ? i > seg : i < seg; i += REV ? -1 : 1) {
      decay_by(exp2_fast((float)ro.slot_log[(size_t)chain * a.segments + i]));
      const float* p = slot_of(i);
#pragma unroll
      for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int z = 0; z < NZ; ++z) S[x][z] += *reinterpret_cast<const f32x4*>(p + (x * NZ + z) * 256);
    }
  }

  auto store_copy = [&]() {
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
      for (int z = 0; z < NZ; ++z) {
        st4<T>(&sm.St[0][16 * z + l][16 * (w * NX + x) + 4 * g], S[x][z]);
        if constexpr (SM::NS == 2) {
          f32x4 lo;
#pragma unroll
          for (int r = 0; r < 4; ++r) lo[r] = S[x][z][r] - (float)(__bf16)S[x][z][r];
          st4<T>(&sm.St[SM::NS - 1][16 * z + l][16 * (w * NX + x) + 4 * g], lo);
        }
      }
  };
  auto chunk_at = [&](int it) { return REV ? c_hi - 1 - it : c_lo + it; };
  auto issue = [&](int it) {
    const int c = chunk_at(it), live = min(kL, sp.len - c * kL);
    load_rows<T, DX, SM::PY>(sm.Y[it & 1], yb + (int64_t)c * kL * ro.ys.t, ro.ys.t, live, w, lane);
    load_rows<T, kSlice, SM::PZ>(sm.Z[it & 1], zb + (int64_t)c * kL * ro.zs.t, ro.zs.t, live, w, lane);
  };
  // the wave's own row of a chunk, its first where the sequence has ended
  auto own_row = [&](int it) {
    const int t = chunk_at(it) * kL + 16 * w + l;
    return (int64_t)(t < sp.len ? t : chunk_at(it) * kL);
  };
  auto gate_at = [&](int it) {
    const int t = chunk_at(it) * kL + lane;
    return it < n && t < sp.len ? gate_of(a, la0 + (int64_t)t * a.ls.t) : 0.0;
  };
  double total = 0.0, g_next = 0.0;
  Frag<T> X[NK], Xn[NK];
  f32x4 wn[NZ], out[NZ];
  float r_out = 0.f;
  int out_chunk = -1;
  auto load_own = [&](int it) {
    if constexpr (!SUMMARY) {
      const int64_t t = own_row(it);
      load_x<T, DX>(Xn, xb + t * ro.xs.t + 8 * g);
      if (ro.r) {
#pragma unroll
        for (int z = 0; z < NZ; ++z) wn[z] = ld4(wb + t * ro.ws.t + 16 * z + 4 * g);
      }
    }
  };
  auto flush = [&]() {  // the outputs of the chunk before: its stores have a chunk's time
    const int t = out_chunk * kL + 16 * w + l;
    if (out_chunk >= 0 && t < sp.len) {
#pragma unroll
      for (int z = 0; z < NZ; ++z) store_out<T>(ro.out, ob + (int64_t)t * ro.os.t + 16 * z + 4 * g, out[z], ro.out_f32);
      if (ro.r && g == 0) ro.r[((size_t)slice * a.chains + chain) * a.T + t] = r_out;
    }
  };

  if (n > 0) {
    issue(0);
    load_own(0);
    if (w == kGateWave) {
      total += form_gates<REV>(sm, 0, gate_at(0), chunk_at(0) * kL + lane < sp.len, ro.in_scale, lane);
      g_next = gate_at(1);
    }
    if constexpr (!SUMMARY) store_copy();
  }
  for (int it = 0; it < n; ++it) {
    const int buf = it & 1;
    vm_wait_all();
    lds_barrier();
#pragma unroll
    for (int kk = 0; kk < NK; ++kk) X[kk] = Xn[kk];
    f32x4 wr[NZ];
#pragma unroll
    for (int z = 0; z < NZ; ++z) wr[z] = wn[z];
    double g_now = g_next;
    if constexpr (!SUMMARY) flush();
    if (w == kGateWave) g_next = gate_at(it + 2);
    if (it + 1 < n) {
      issue(it + 1);
      load_own(it + 1);
    }

    {  // b z, 8 entries a thread
      const int row = tid / (kSlice / 8), col = 8 * (tid % (kSlice / 8));
      const float bw = sm.bw[buf][row];
      float z[8];
      if constexpr (sizeof(T) == 2) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(&sm.Z[buf][row][col]);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = bw == 0.f ? 0.f : (float)v[e] * bw;
#pragma unroll
        for (int p = 0; p < SM::NH; ++p) {
          bf16x8 part;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            part[e] = (__bf16)z[e];
            z[e] -= (float)part[e];
          }
          *reinterpret_cast<bf16x8*>(&sm.Zw[p][row][col]) = part;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          f32x4 v = *reinterpret_cast<const f32x4*>(&sm.Z[buf][row][col + 4 * q]);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = bw == 0.f ? 0.f : v[e] * bw;
          *reinterpret_cast<f32x4*>(&sm.Zw[0][row][col + 4 * q]) = v;
        }
      }
    }
    f32x4 acc[NZ], P[kWaves];
    if constexpr (!SUMMARY) {
      // far: the state before the chunk
#pragma unroll
      for (int z = 0; z < NZ; ++z) acc[z] = zero4();
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int z = 0; z < NZ; ++z)
#pragma unroll
          for (int s = 0; s < SM::NS; ++s)
            mma(acc[z], lds_frag<T, KORD_CONTIG>(&sm.St[s][0][0], SM::PY, 16 * z, 32 * kk, lane), X[kk]);
      const float aw = sm.aw[buf][16 * w + l];
#pragma unroll
      for (int z = 0; z < NZ; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[z][r] = aw == 0.f ? 0.f : acc[z][r] * aw;
      // scores
      const float bh = sm.bh[buf][16 * w + l], bl = sm.bl[buf][16 * w + l];
      const int live = min(kL, sp.len - chunk_at(it) * kL);
#pragma unroll
      for (int t = 0; t < kWaves; ++t) {
        P[t] = zero4();
        if (REV ? t < w : t > w) continue;
        f32x4 s = zero4();
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) mma(s, lds_frag<T, KORD_CONTIG>(&sm.Y[buf][0][0], SM::PY, 16 * t, 32 * kk, lane), X[kk]);
        const f32x4 kh = *reinterpret_cast<const f32x4*>(&sm.bh[buf][16 * t + 4 * g]);
        const f32x4 kl = *reinterpret_cast<const f32x4*>(&sm.bl[buf][16 * t + 4 * g]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * t + 4 * g + r, i = 16 * w + l;
          const float d = REV ? (kh[r] - bh) + (kl[r] - bl) : (bh - kh[r]) + (bl - kl[r]);
          const float e = exp2_fast(d) * ro.in_scale;
          const bool on = (REV ? j >= i : j <= i) && j < live && e != 0.f;
          P[t][r] = on ? s[r] * e : 0.f;
        }
      }
    }
    lds_barrier();
    if constexpr (!SUMMARY) {
      // near
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        if (REV ? 2 * kk + 1 < w : 2 * kk > w) continue;
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
          const Frag<T> v = tr_frag_acc<T>(&sm.Z[buf][0][0], SM::PZ, 32 * kk, 16 * z, lane);
          mma(acc[z], v, p);
          if constexpr (SM::NS == 2) mma(acc[z], v, q);
        }
      }
      float rs = 0.f;
#pragma unroll
      for (int z = 0; z < NZ; ++z)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          out[z][r] = acc[z][r] * ro.out_scale;
          rs += out[z][r] * wr[z][r];
        }
      if (ro.r) {
        rs += __shfl_xor(rs, 16, 64);
        r_out = rs + __shfl_xor(rs, 32, 64);
      }
      out_chunk = chunk_at(it);
    }
    // update
    decay_by(sm.dec[buf]);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      Frag<T> y[NX];
#pragma unroll
      for (int x = 0; x < NX; ++x) y[x] = tr_frag<T>(&sm.Y[buf][0][0], SM::PY, 32 * kk, 16 * (w * NX + x), lane);
#pragma unroll
      for (int z = 0; z < NZ; ++z)
#pragma unroll
        for (int p = 0; p < SM::NH; ++p) {
          const Frag<T> v = tr_frag<T>(&sm.Zw[p][0][0], SM::PZ, 32 * kk, 16 * z, lane);
#pragma unroll
          for (int x = 0; x < NX; ++x) mma(S[x][z], y[x], v);
        }
    }
    if constexpr (!SUMMARY) {
      if (it + 1 < n) store_copy();
    }
    if (w == kGateWave && it + 1 < n)
      total += form_gates<REV>(sm, buf ^ 1, g_now, chunk_at(it + 1) * kL + lane < sp.len, ro.in_scale, lane);
  }
  if constexpr (SUMMARY) {
    store_slot(seg);
    if (slice == 0 && w == kGateWave && lane == 0) ro.slot_log[(size_t)chain * a.segments + seg] = total;
    return;
  }
  flush();
  const bool ends = REV ? seg == 0 : (nc == 0 || c_hi == nc);  // this segment has the walk's last chunk
  if (!ends) return;
  float d = 0.f;
#pragma unroll
  for (int x = 0; x < NX; ++x)
#pragma unroll
    for (int z = 0; z < NZ; ++z) {
      const int i = slice * kSlice + 16 * z + l, j = 16 * (w * NX + x) + 4 * g;
      if (ro.s_out) *reinterpret_cast<f32x4*>(ro.s_out + chain * mat + (size_t)i * DX + j) = S[x][z];
      if (ro.dot)
#pragma unroll
        for (int r = 0; r < 4; ++r) d += S[x][z][r] * ro.dot[chain * mat + (size_t)i * ro.s_i + (size_t)(j + r) * ro.s_j];
    }
  if (ro.dot) {
    d = group_sum<64>(d);
    if (lane == 0) sm.red[w] = d;
    lds_barrier();
    if (tid == 0) ro.dot_out[(size_t)chain * ro.slices + slice] = (sm.red[0] + sm.red[1]) + (sm.red[2] + sm.red[3]);
  }
}

// Workgroups of a launch: along x, eight chains at a time, each on an XCD of its own, with the roles and slices of
// a chain (which share its rows) next to each other; along y the segments.
template <typename T, int DX, bool SPLIT, bool SUMMARY>
__global__ __launch_bounds__(kThreads) void la_walk_kernel(Args a) {
  __shared__ __align__(16) Smem<T, DX, SPLIT> sm;
  const int at = blockIdx.x / 8, group = at / a.slots_per_group;
  int k = at - group * a.slots_per_group, role = 0;
  const int chain = 8 * group + (int)(blockIdx.x % 8);
  if (chain >= a.chains) return;
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
  constexpr int LPR = DX / 4, RPP = kThreads / LPR, NP = kSlice / RPP;
  const Role& ro = a.role[0];
  const int chain = blockIdx.x / ro.slices, slice = blockIdx.x - chain * ro.slices;
  const int b = chain / a.H, h = chain - b * a.H;
  const int col = 4 * (threadIdx.x % LPR), row = threadIdx.x / LPR;
  const Span sp = span_of(a, b);
  const size_t mat = (size_t)ro.dz * DX;
  const T* xb = rows_of<T>(ro.x, ro.xs, ro.x_share, a, sp, b, h) + col;
  const T* yb = rows_of<T>(ro.y, ro.ys, ro.y_share, a, sp, b, h) + col;
  const T* zb = rows_of<T>(ro.z, ro.zs, ro.z_share, a, sp, b, h) + slice * kSlice + row;
  T* ob = rows_of<T>(ro.out, ro.os, 1, a, sp, b, h) + slice * kSlice + row;
  const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
  const size_t s0 = chain * mat + (size_t)(slice * kSlice + row) * DX + col;
  f32x4 S[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    S[i] = zero4();
    if (ro.s_in) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(ro.s_in + s0 + (size_t)i * RPP * DX));
  }
  for (int t = 0; t < sp.len; ++t) {
    const f32x4 x = ld4(xb + t * ro.xs.t), y = ld4(yb + t * ro.ys.t);
    const float d = exp2_fast((float)gate_of(a, la0 + (int64_t)t * a.ls.t));
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float z = to_f32(zb[t * ro.zs.t + i * RPP]);
      float o = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        S[i][e] = (d == 0.f ? 0.f : S[i][e] * d) + z * y[e];
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

// Gradient rows that several heads share: the sum of their parts, in order.  Parts are [rows][H][d] fp32.
struct Shared {
  const float* part;
  void* out;
  Strides os;
  int heads, share, d, f32;
};
struct SumArgs {
  int B, T, H;
  const int32_t *lengths, *offsets;
  int64_t rows;
  Shared side[3];
};
__global__ __launch_bounds__(kThreads) void la_sum_kernel(SumArgs a) {
  const Shared& s = a.side[blockIdx.y];
  const int quads = s.d / 4;
  const int64_t per = (int64_t)s.heads * quads, all = per * a.B * a.T;
  for (int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x; at < all; at += (int64_t)gridDim.x * kThreads) {
    const int64_t bt = at / per;
    const int rest = (int)(at - bt * per), hh = rest / quads, c = 4 * (rest - hh * quads);
    const int b = (int)(bt / a.T), t = (int)(bt - (int64_t)b * a.T);
    const Span sp = span_of(a.lengths, a.offsets, a.rows, a.T, b);
    if (t >= sp.len && a.offsets) continue;
    f32x4 v = zero4();
    if (t < sp.len) {
      const float* p = s.part + ((a.offsets ? sp.row0 + t : bt) * a.H + (int64_t)hh * s.share) * s.d + c;
      for (int i = 0; i < s.share; ++i) v += *reinterpret_cast<const f32x4*>(p + (size_t)i * s.d);
    }
    const int64_t o = (a.offsets ? (sp.row0 + t) * s.os.t : b * s.os.b + t * s.os.t) + hh * s.os.h + c;
    store_out<__bf16>(s.out, o, v, s.f32);
  }
}

// dlog alpha of one chain: the sums from the end of rq - rk (over the slices), plus the state's product, in 64 bits.
constexpr int kGateThreads = 1024;
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
  __shared__ double behind;
  const int64_t la0 = (a.offsets ? sp.row0 * a.ls.t : b * a.ls.b) + h * a.ls.h;
  auto store = [&](int t, float v) {
    const int64_t at = ((a.offsets ? sp.row0 : (int64_t)b * a.T) + t) * a.H + h;
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
  for (int last = sp.len; last > 0; last -= kGateThreads) {  // thread 0 the last token of the stretch
    const int t = last - 1 - tid;
    double r = 0.0;
    if (t >= 0) {
      for (int s = 0; s < q.q_slices; ++s) r += (double)q.rq[((size_t)s * a.chains + chain) * a.T + t];
      for (int s = 0; s < q.k_slices; ++s) r -= (double)q.rk[((size_t)s * a.chains + chain) * a.T + t];
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double up = __shfl_up(r, off, 64);
      if (lane >= off) r += up;
    }
    if (lane == 63) tops[w] = r;
    __syncthreads();
    for (int i = 0; i < w; ++i) r += tops[i];
    const double sum = r + behind;
    if (t >= 0) {
      const bool dropped = exp2_fast((float)gate_of(a, la0 + (int64_t)t * a.ls.t)) == 0.f;
      store(t, dropped ? 0.f : (float)sum);
    }
    __syncthreads();
    if (tid == kGateThreads - 1) behind = sum;
    __syncthreads();
  }
  if (a.offsets == nullptr)
    for (int t = sp.len + tid; t < a.T; t += kGateThreads) store(t, 0.f);
}

// ---------------------------------------------------------------- host

Strides dense(int64_t T, int64_t H, int64_t d) { return Strides{T * H * d, H * d, d}; }

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

// Segments: enough workgroups for the card, of at least four chunks each.
void split_of(const ccq_linear_attn_params& p, int groups, int* segments, int* per) {
  const int nc = (p.T - 1) / kL + 1;
  int want = (512 + groups - 1) / groups;
  want = want < 1 ? 1 : (want > 32 ? 32 : want);
  if (want > nc / 4) want = nc / 4 < 1 ? 1 : nc / 4;
  *per = (nc + want - 1) / want;
  *segments = (nc + *per - 1) / *per;
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
    r.slots = sp.take<float>((size_t)a.chains * a.segments * r.slices * kSlice * dx);
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
  if (a.segments > 1) la_walk_kernel<T, DX, false, true><<<dim3(groups, a.segments - 1), kThreads, 0, stream>>>(a);
  la_walk_kernel<T, DX, SPLIT, false><<<dim3(groups, a.segments), kThreads, 0, stream>>>(a);
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
      r.os = dense(p.T, p.H, dim[i]);
      r.out_f32 = 1;
      Shared& s = bp.sum.side[bp.sums++];
      s = Shared{part, out[i], gs[i], p.H / share[i], share[i], dim[i], grad_f32};
      const int quads = s.heads * dim[i] / 4;
      if (quads > bp.most) bp.most = quads;
    } else {
      r.out = out[i];
      r.os = gs[i];
      r.out_f32 = grad_f32;
      r.zero_tail = 1;
    }
    if (q.dlog_alpha && i < 2) {
      r.w = in[i];
      r.ws = xs[i];
      r.w_share = share[i];
      r.r = sp.take<float>((size_t)r.slices * chains * p.T);
    }
  }
  if (q.dlog_alpha && q.dS_out) {
    role[0].dot = q.dS_out;
    role[0].dot_out = sp.take<float>(chains * role[0].slices);
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
  bp.sum.B = p.B;
  bp.sum.T = p.T;
  bp.sum.H = p.H;
  bp.sum.lengths = p.lengths;
  bp.sum.offsets = p.offsets;
  bp.sum.rows = p.rows;
  bp.gate.a = base_of(p);
  bp.gate.rq = role[0].r;
  bp.gate.rk = role[1].r;
  bp.gate.dot = role[0].dot_out;
  bp.gate.q_slices = role[0].slices;
  bp.gate.k_slices = role[1].slices;
  bp.gate.dot_slices = role[0].slices;
  bp.gate.out = q.dlog_alpha;
  bp.end = sp.at;
  return bp;
}

// Workgroups of the sum over shared heads.
unsigned sum_blocks(const BackPlan& bp) {
  const uint64_t n = ((uint64_t)bp.most * bp.sum.B * bp.sum.T + kThreads - 1) / kThreads;
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
    const unsigned grid = (unsigned)a.chains * a.role[0].slices;
    if (p.dtype == CCQ_DTYPE_BF16) {
      if (p.d_k == 128) la_step_kernel<__bf16, 128><<<grid, kThreads, 0, stream>>>(a);
      else la_step_kernel<__bf16, 64><<<grid, kThreads, 0, stream>>>(a);
    } else {
      if (p.d_k == 128) la_step_kernel<float, 128><<<grid, kThreads, 0, stream>>>(a);
      else la_step_kernel<float, 64><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
  }
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
