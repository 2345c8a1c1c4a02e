// Gated delta rule for gfx950: the backward.  With the notation of
// delta_common.h, S and D the state and its gradient at a step's two ends,
// dU, dR as in the reverse walk, dP = dY U^T (j <= i) and dT = -dR U^T (j < i):
//   dQ    = scale 2^c (dY S^T) + Pm K                 Pm = scale E dP
//   dK    = -beta 2^c (dR S^T) + 2^(c_end-c) (U D^T) + Pm^T Q + (Xm + Xm^T) K
//                                                     Xm = beta E dT
//   dbeta_i = dR_i.V_i - 2^c_i k_i.(dR S^T)_i + sum_j dT_ij E_ij k_i.k_j
//   dg_t  = the sum of what passes from before token t to token t and behind:
//           sum_{i >= t} A_i + sum_{j < t} F_j + sum_{i >= t > j} Z_ij + 2^c_end <S, D>
//           A_i = scale 2^c_i q_i.(dY S^T)_i - beta_i 2^c_i k_i.(dR S^T)_i
//           F_j = 2^(c_end-c_j) k_j.(U D^T)_j,  Z_ij = Pm_ij q_i.k_j + Xm_ij k_i.k_j
// dg_t is added up from those pairs, not as a difference of sums: where decays
// are strong it is far smaller than what passes within a token.
//
// Four launches: every step's matrices (delta_bwd_prep_kernel), the walk of the
// states, which keeps each step's starting state and U (delta_keep_kernel), the
// walk of the state's gradient (delta_reverse_kernel), and the gradients of
// every step (delta_grads_kernel), whose work-group takes the heads of a group
// one after another and adds up the shared q's and k's gradients in registers.
#include "delta_common.h"
#include "delta_pair.h"
#include "delta_prep.h"
#include "delta_walk.h"

namespace {

using namespace delta;

// Times here: 4 x 4096 tokens, 16 groups of two heads of 128 x 128, bf16.  96 us, as
// delta_prep_kernel, with 0.3 GB written.
template <class T, int NB>
__global__ __launch_bounds__(kPrepWaves * 64, prep_per_cu(sizeof(T), NB * 32)) void delta_bwd_prep_kernel(DeltaArgs a) {
  __shared__ PrepLds<T, NB> s;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const PrepWork w = prep_work(a);
  const Unit u = locate(a.seqs, w.step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  make_steps<T, NB, true>(s, a, u, w.step, w.first, w.heads, a.pt, [&](long cell) {
    put_pieces<false>(a.m + cell * kPieces * kPiece, s.sq.m, wave, lane);
    put_pieces<true>(a.mt + cell * kPieces * kPiece, s.sq.m, wave, lane);
  });
}

// 234 us, 3.7 a step; 0.8 GB written (3.4 TB/s).
template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_keep_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairFwdLds<NB, kKept> s;
    pair_forward<NB, kKept>(a, s);
  } else {
    __shared__ FwdLds<T, NB, kKept> s;
    walk_forward<T, NB, kKept>(a, s);
  }
}

// 402 us, 6.3 a step: two triangular products on its chain, and LDS has room for one
// step's operands only.  LDS is busy for 40% of it, the vector pipes for 31%, the matrix
// pipes for 24%.  With all but K put into LDS before the walkers are done, the same.
template <class T, int NB, bool SUMMARY>
__global__ __launch_bounds__(walk_threads<T>) void delta_reverse_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairRevLds<NB> s;
    pair_reverse<NB, SUMMARY>(a, s);
  } else {
    __shared__ RevLds<T, NB> s;
    walk_reverse<T, NB, SUMMARY>(a, s);
  }
}

// ------------------------------------------------------- a step's gradients
template <class T>
constexpr int kPart = sizeof(T) == 2 ? 128 : 64;  // columns of a head that LDS holds at a time

// Eight waves share a step's 2 NB tiles of 16 states by four tiles of 16 tokens:
// one by NB of them a wave, so that each state is loaded and split once.
// 674 us, 2.0 GB read; with two by two tiles a wave 750, and 690 with what is kept in
// rows.  LDS holds one work-group on a CU, whose phases take turns: of its cycles the
// vector pipes are busy for 36%, the matrix pipes for 24%, LDS for 36%, and HBM could
// have moved the bytes in 420 us.  Sixteen waves, and work-groups that stay for several
// steps and load the next one's operands ahead, spilled registers: 960 and 747 us; the
// next head's states loaded ahead with its rows took 713 (S) and 761 us (S and D), as
// the loads are issued in order and those needed first wait behind them.
constexpr int kGradWaves = 8;

template <class T, int NB>
struct GradLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  static constexpr int ldv = stride_of<T>(kPart<T>);
  static constexpr int ldm = stride_of<T>(kTok);
  static constexpr int kAcross = 2 * NB;
  alignas(16) T k[kTok * ldn];
  alignas(16) T q[kTok * ldn];
  union {
    struct {
      T y[kTok * ldv];
      T r[kExact<T>][kTok * ldv];  // dR
      T u[kExact<T>][kTok * ldv];  // U
    } in;
    struct {
      T pm[kTwo<T>][kTok * ldm];   // Pm
      T xm[kTwo<T>][kTok * ldm];   // Xm
      float z[kTok * kSq];         // Z
      float qs[kAcross][kTok], ks[kAcross][kTok], kd[kAcross][kTok];  // some states' part of A_i's two terms, without their factors, and F_j's
    } sq;
  };
  alignas(16) Coef coef;
  float c_hi[kTok], c_lo[kTok];
  float rv[kTok];                                  // dR_i.V_i
  float bt[4][kTok];                               // a column tile's part of sum_j dT_ij E_ij k_i.k_j
  float sd[kAcross];                               // some states' part of <S, D>
  float a_i[kTok], f_j[kTok];
};

// The thread's number, as a value that the compiler knows nothing of: what is
// computed from it is computed where it is used, and not kept in registers over
// the whole loop (143 of them spilled).
__device__ __forceinline__ int thread_here() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// acc[i + j] += a b[j] in parts, small products first, over all tiles in turn.
template <class T, int I, int J, int B>
__device__ __forceinline__ void mma_row(v4f (&acc)[I], int i, const Split<T, kExact<T>>& a, const Frag<T> (&b)[J][B]) {
  constexpr int kMost = kExact<T>;
#pragma unroll
  for (int m = kMost - 1; m >= 0; --m)
#pragma unroll
    for (int z = 0; z <= m; ++z)
      if (m - z < B) {
#pragma unroll
        for (int j = 0; j < J; ++j) mma(acc[i + j], a.f[z], b[j][m - z]);
      }
}

// Eight values to an LDS row in PARTS parts, `plane` elements apart.
template <class T, int PARTS>
__device__ __forceinline__ void put8(T* p, int plane, const float (&v)[8]) {
  const Split<T, PARTS> f = split_of<T, PARTS>(v);
#pragma unroll
  for (int z = 0; z < PARTS; ++z) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<v8bf*>(p + z * plane) = f.f[z].v;
    } else {
      v4f* r = reinterpret_cast<v4f*>(p + z * plane);
      r[0] = f.f[z].v[0];
      r[1] = f.f[z].v[1];
    }
  }
}

// Eight values of T as they were loaded.
template <class T>
struct Eight {
  v4i v[sizeof(T) / 2];
  __device__ __forceinline__ void load(Rsrc rs, unsigned off) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16 * i, 0, 0);
  }
  __device__ __forceinline__ void load_kept(Rsrc rs, unsigned off) {  // of what the walks keep
    static_assert(sizeof(T) == 4, "in fp32");
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, off + 1024 * i, 0, 0);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const v8bf b = __builtin_bit_cast(v8bf, v[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = static_cast<float>(b[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_bit_cast(v4f, v[j >> 2])[j & 3];
    }
  }
  __device__ __forceinline__ void put(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<v4i*>(p)[i] = v[i];
  }
};

// The sums of I values over the four lanes with the same l & 15: value
// g / (4 / I) in the lanes of group g.  Where a lane has several values, they
// share the swaps.
template <int I>
__device__ __forceinline__ float sums_of_groups(const float (&v)[I]) {
  if constexpr (I == 1) {
    return sum_groups(v[0]);
  } else {
    float half[I / 2];
#pragma unroll
    for (int i = 0; i < I / 2; ++i) {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + I / 2]), false, false);
      half[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(half[0]), __float_as_uint(half[I / 2 - 1]), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
}

// A group's heads are split over several work-groups where there are few steps;
// their parts of the shared gradients then meet in delta_sum_kernel.  3 x 333
// tokens, 10 heads of 24 x 40 in 2 groups, fp32: 54 us with all five heads of a
// group in one work-group, 16 and 6 us with one each.
__host__ __device__ inline int grad_parts(const DeltaArgs& a) { return (a.ratio + a.grad_heads - 1) / a.grad_heads; }
__host__ __device__ inline long grad_part_at(const DeltaArgs& a, long i) { return i * 2 * kTok * a.states; }

template <class T, int NB>
__global__ __launch_bounds__(kGradWaves * 64) void delta_grads_kernel(DeltaArgs a) {
  typedef GradLds<T, NB> L;
  __shared__ L s;
  constexpr int kW = kGradWaves, kThreads = kW * 64;
  constexpr int kI = NB, kJ = NB < 2 ? 1 : 2;      // a wave's tiles of tokens, and those of them at a time
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int groups = a.heads / a.ratio, parts = grad_parts(a);
  const int step = work / (groups * parts), at = work % (groups * parts), group = at / parts, part = at % parts;
  const int first = group * a.ratio + part * a.grad_heads, behind_h = min(first + a.grad_heads, (group + 1) * a.ratio);
  const Unit u = locate(a.seqs, step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  const bool packed = a.seqs.offsets != nullptr;
  const int rows = min(u.len - u.t0, kTok);
  const long bytes = kept_bytes(a.states, a.width), slab = kept_bytes(kTok, a.width);
  constexpr int kAcross = 2 * NB;                  // waves side by side over the states
  const int s0 = wave % kAcross;                   // this wave's tile of states
  const int i0 = wave / kAcross * kI;              // and the first of tokens

  // A part of a head's columns on their way to LDS: a thread has eight columns of
  // every 32 of one row, of dR and V (the first four waves) or of U and dY.
  constexpr int kEights = kPart<T> / 32;
  Eight<float> flat[kEights];
  Eight<T> token[kEights];
  const bool second = __builtin_amdgcn_readfirstlane(tid >= 256);
  const long my_stride = second ? a.d_y.row_stride : a.v.row_stride;
  const T* my_p = second ? seq_ptr<const T>(a.d_y, u.seq, u.row0, packed) + u.t0 * a.d_y.row_stride
                         : seq_ptr<const T>(a.v, u.seq, u.row0, packed) + u.t0 * a.v.row_stride;
  const auto fetch = [&](int h, int c0) {  // behind the last head nothing, by the same loads
    const long cell = static_cast<long>(step) * a.heads + h;
    const bool any = h < behind_h;
    const Rsrc rf = make_rsrc((second ? a.u : a.d_r) + cell * (slab / 4), any ? static_cast<unsigned>(slab) : 0);
    const Rsrc rt = rows_rsrc(my_p + h * a.width, my_stride, any ? rows : 0, a.width);
    const int t = thread_here() & 255, row = (t >> 6) * 16 + (t & 15), col = c0 + 8 * (t >> 4 & 3);
    const unsigned off = static_cast<unsigned>((t >> 6) * kept_strip(a.width) + kept_at(0, c0) + 16 * (t & 63));
    const unsigned tok = static_cast<unsigned>(row * static_cast<int>(my_stride) + col) * sizeof(T);
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const bool in = col + 32 * i < a.width;
      flat[i].load_kept(rf, in ? off + 2048 * i : kOutside);
      token[i].load(rt, in ? tok + 32 * sizeof(T) * i : kOutside);
    }
  };
  float rv = 0.0f;
  const auto put = [&] {
    const int t = thread_here() & 255, at0 = ((t >> 6) * 16 + (t & 15)) * L::ldv + 8 * (t >> 4 & 3);
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const int at = at0 + 32 * i;
      float f[8];
      flat[i].get(f);
      put8<T, kExact<T>>((second ? s.in.u[0] : s.in.r[0]) + at, kTok * L::ldv, f);
      if (second) {
        token[i].put(s.in.y + at);
      } else {
        float t[8];
        token[i].get(t);
#pragma unroll
        for (int j = 0; j < 8; ++j) rv = fmaf(f[j], t[j], rv);
      }
    }
  };
  // This lane's rows of a kept state, columns 8 g .. of 32; rows and columns outside are zero.
  const auto load_state = [&](Eight<float>& e, const float* kept, long cell, int c0) {
    const Rsrc rs = make_rsrc(kept + cell * (bytes / 4), static_cast<unsigned>(bytes));
    const int t = thread_here() & 63;
    const bool in = 16 * s0 + (t & 15) < a.states && c0 + 8 * (t >> 4) < a.width;
    const unsigned off = in ? static_cast<unsigned>(s0 * kept_strip(a.width) + kept_at(0, c0) + 16 * t) : kOutside;
    e.load_kept(rs, off);
  };
  float g_raw = 0.0f;
  v4f coef_raw = {0, 0, 0, 0};
  const auto fetch_gates = [&](int h) {
    if (wave == kW - 1) g_raw = load_gate(a.g, a.gate_bf16, u, packed, u.t0, rows, h, a.heads);
    else if (tid < static_cast<int>(sizeof(Coef) / 16))
      coef_raw = reinterpret_cast<const v4f*>(a.coef + static_cast<long>(step) * a.heads + h)[tid];
  };
  {
    Tile<T, kTok, NB * 32, kThreads> tk, tq;
    tk.init(a.k.row_stride, a.states, tid);
    tq.init(a.q.row_stride, a.states, tid);
    const int j = group * a.states;
    tk.load(rows_rsrc(seq_ptr<const T>(a.k, u.seq, u.row0, packed) + u.t0 * a.k.row_stride + j, a.k.row_stride, rows, a.states));
    tq.load(rows_rsrc(seq_ptr<const T>(a.q, u.seq, u.row0, packed) + u.t0 * a.q.row_stride + j, a.q.row_stride, rows, a.states));
    fetch_gates(first);
    fetch(first, 0);
    tk.store(s.k, L::ldn, tid);
    tq.store(s.q, L::ldn, tid);
  }
  // A wave's share of the ten score tiles (row ti, column tj <= ti): of the rows
  // that it has products of.
  constexpr int kMine = 2;
  int mine[kMine], row_of[kMine], col_of[kMine];
#pragma unroll
  for (int n = 0; n < kMine; ++n) {
    const int at = i0 * (i0 + 1) / 2 + s0 + n * kAcross;
    mine[n] = at < (i0 + kI) * (i0 + kI + 1) / 2;
    row_of[n] = at < 1 ? 0 : at < 3 ? 1 : at < 6 ? 2 : 3;
    col_of[n] = at - row_of[n] * (row_of[n] + 1) / 2;
  }
  // the gradients of q and k, transposed: token l15 of a tile, states 4 g .. of another
  v4f dq[kI], dk[kI];
#pragma unroll
  for (int i = 0; i < kI; ++i) dq[i] = dk[i] = v4f{0, 0, 0, 0};
  for (int h = first; h < behind_h; ++h) {
    const int tid = thread_here(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
    __syncthreads();  // the last head's matrices are read
    if (wave == kW - 1) {
      const double c = scan64(gate_log(g_raw));
      s.c_hi[lane] = static_cast<float>(c);
      s.c_lo[lane] = static_cast<float>(c - static_cast<float>(c));
    } else if (tid < static_cast<int>(sizeof(Coef) / 16)) {
      reinterpret_cast<v4f*>(&s.coef)[tid] = coef_raw;
    }
    rv = 0.0f;
    const long cell = static_cast<long>(step) * a.heads + h;
    float sd = 0.0f, sq[kI] = {}, sk[kI] = {}, sf[kI] = {};
    v4f dp[kMine], dt[kMine];  // this wave's tiles of dP^T and -dT^T
#pragma unroll
    for (int i = 0; i < kMine; ++i) dp[i] = dt[i] = v4f{0, 0, 0, 0};
    constexpr bool kWhole = kPart<T> >= kMaxDim;  // LDS holds every head's columns at once
    for (int c0 = 0; c0 < (kWhole ? 1 : a.width); c0 += kPart<T>) {
      if (!kWhole && c0 > 0) {
        __syncthreads();
        fetch(h, c0);
      }
      const int behind = min(a.width - c0, kPart<T>);
      // all of a part's columns of S and D are on their way before they are needed
      Eight<float> state[kEights], grad[kEights];
#pragma unroll
      for (int e = 0; e < kEights; ++e) load_state(state[e], a.keep, cell, c0 + 32 * e);
#pragma unroll
      for (int e = 0; e < kEights; ++e) load_state(grad[e], a.d_keep, cell, c0 + 32 * e);
      put();
      __syncthreads();
      {  // products over the columns with S, transposed: S dY^T, S dR^T; and the score tiles
        v4f ys[kI], rs[kI];
#pragma unroll
        for (int i = 0; i < kI; ++i) ys[i] = rs[i] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kEights; ++e) {
          const int c = 32 * e;
          if (c >= behind) break;
          float f[8];
          state[e].get(f);
          const Split<T, kExact<T>> part = split_of<T, kExact<T>>(f);
#pragma unroll
          for (int i = 0; i < kI; i += kJ) {
            Frag<T> yf[kJ][1], rf[kJ][kExact<T>];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
              yf[j][0] = frag_row(s.in.y, L::ldv, 16 * (i0 + i + j), c, lane);
#pragma unroll
              for (int z = 0; z < kExact<T>; ++z) rf[j][z] = frag_row(s.in.r[z], L::ldv, 16 * (i0 + i + j), c, lane);
            }
            keep_reads_here();
            mma_row<T>(ys, i, part, yf);
            mma_row<T>(rs, i, part, rf);
#pragma unroll
            for (int n = 0; n < kMine; ++n)
#pragma unroll
              for (int j = 0; j < kJ; ++j)
                if (mine[n] && row_of[n] == i0 + i + j) {
                  Frag<T> uf[kExact<T>];
#pragma unroll
                  for (int z = 0; z < kExact<T>; ++z) uf[z] = frag_row(s.in.u[z], L::ldv, 16 * col_of[n], c, lane);
                  mma_parts<T>(dp[n], uf, yf[j]);
                  mma_parts<T>(dt[n], uf, rf[j]);
                }
          }
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          const int t = 16 * (i0 + i) + l15, at = t * L::ldn + 16 * s0 + 4 * g;
          const float from = s.coef.from[t], beta = s.coef.beta[t];
          const v4f pq = quad_get(s.q + at) * ys[i], pk = quad_get(s.k + at) * rs[i];
          sq[i] += (pq[0] + pq[1]) + (pq[2] + pq[3]);
          sk[i] += (pk[0] + pk[1]) + (pk[2] + pk[3]);
          dq[i] += (a.scale * from) * ys[i];
          dk[i] -= (beta * from) * rs[i];
        }
      }
      {  // with D: D U^T
        v4f ud[kI];
#pragma unroll
        for (int i = 0; i < kI; ++i) ud[i] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kEights; ++e) {
          const int c = 32 * e;
          if (c >= behind) break;
          float d[8], f[8];
          grad[e].get(d);
          state[e].get(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) sd = fmaf(f[j], d[j], sd);
          const Split<T, kExact<T>> part = split_of<T, kExact<T>>(d);
#pragma unroll
          for (int i = 0; i < kI; i += kJ) {
            Frag<T> uf[kJ][kExact<T>];
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
              for (int z = 0; z < kExact<T>; ++z) uf[j][z] = frag_row(s.in.u[z], L::ldv, 16 * (i0 + i + j), c, lane);
            keep_reads_here();
            mma_row<T>(ud, i, part, uf);
          }
        }
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          const int t = 16 * (i0 + i) + l15;
          const v4f pd = quad_get(s.k + t * L::ldn + 16 * s0 + 4 * g) * ud[i];
          sf[i] += (pd[0] + pd[1]) + (pd[2] + pd[3]);
          dk[i] += s.coef.to[t] * ud[i];
        }
      }
    }
    rv = sum_groups(rv);
    if (!second && g == 0) s.rv[wave * 16 + l15] = rv;
    __syncthreads();  // the columns give way to the matrices
    fetch_gates(h + 1 < behind_h ? h + 1 : h);  // the next head's

    sd = sum64(sd);
    if (lane == 0 && i0 == 0) s.sd[s0] = sd;
    {
      const float tq = sums_of_groups(sq), tk = sums_of_groups(sk), tf = sums_of_groups(sf);
      const int t = 16 * (i0 + g * kI / 4) + l15;
      if (g * kI % 4 == 0) {
        s.sq.qs[s0][t] = tq;
        s.sq.ks[s0][t] = tk;
        s.sq.kd[s0][t] = tf;
      }
    }
    // the matrices of the step: this lane's row of a tile, columns 4 g ..
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      if (mine[n]) {
        const int ti = row_of[n], tj = col_of[n];
        v4f kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          const Frag<T> b = frag_row(s.k, L::ldn, 16 * tj, 32 * m, lane);
          mma(kk, b, frag_row(s.k, L::ldn, 16 * ti, 32 * m, lane));
          mma(qk, b, frag_row(s.q, L::ldn, 16 * ti, 32 * m, lane));
        }
        const int row = 16 * ti + l15, col = 16 * tj + 4 * g;
        const float ch = s.c_hi[row], cl = s.c_lo[row], beta = s.coef.beta[row];
        const v4f hi = rows_of(s.c_hi, tj, g), lo = rows_of(s.c_lo, tj, g);
        v4f pm, et;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = exp2_of((ch - hi[r]) + (cl - lo[r]));
          pm[r] = col + r <= row ? a.scale * (e * dp[n][r]) : 0.0f;
          et[r] = col + r < row ? -e * dt[n][r] : 0.0f;
        }
        const v4f xm = beta * et, ek = et * kk;
        quad_put_parts<kTwo<T>>(&s.sq.pm[0][row * L::ldm + col], kTok * L::ldm, pm);
        quad_put_parts<kTwo<T>>(&s.sq.xm[0][row * L::ldm + col], kTok * L::ldm, xm);
        quad_put(&s.sq.z[row * kSq + col], pm * qk + xm * kk);
        const float bt = sum_groups((ek[0] + ek[1]) + (ek[2] + ek[3]));
        if (g == 0) s.bt[tj][row] = bt;
      }
    }
    // zeros above the diagonal where a product of 32 columns reaches
    if (tid < 128) {
      const int z = tid >> 6, row = 32 * z + (tid >> 2 & 15), col = 32 * z + 16 + 4 * (tid & 3);
      quad_put_parts<kTwo<T>>(&s.sq.pm[0][row * L::ldm + col], kTok * L::ldm, v4f{0, 0, 0, 0});
      quad_put_parts<kTwo<T>>(&s.sq.xm[0][row * L::ldm + col], kTok * L::ldm, v4f{0, 0, 0, 0});
    }
    __syncthreads();
    // dQ^T += K^T Pm^T, dK^T += Q^T Pm + K^T (Xm + Xm^T)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const Frag<T> kf[1] = {frag_col(s.k, L::ldn, 32 * j, 16 * s0, lane)};
      const Frag<T> qf[1] = {frag_col(s.q, L::ldn, 32 * j, 16 * s0, lane)};
#pragma unroll
      for (int m = 0; m < kI; ++m) {
        const int i = i0 + m;
        Frag<T> pf[kTwo<T>], xf[kTwo<T>];
        if (j <= i / 2) {
#pragma unroll
          for (int z = 0; z < kTwo<T>; ++z) {
            pf[z] = frag_row(s.sq.pm[z], L::ldm, 16 * i, 32 * j, lane);
            xf[z] = frag_row(s.sq.xm[z], L::ldm, 16 * i, 32 * j, lane);
          }
          mma_parts<T>(dq[m], kf, pf);
          mma_parts<T>(dk[m], kf, xf);
        }
        if (j >= i / 2) {
#pragma unroll
          for (int z = 0; z < kTwo<T>; ++z) {
            pf[z] = frag_col(s.sq.pm[z], L::ldm, 32 * j, 16 * i, lane);
            xf[z] = frag_col(s.sq.xm[z], L::ldm, 32 * j, 16 * i, lane);
          }
          mma_parts<T>(dk[m], qf, pf);
          mma_parts<T>(dk[m], kf, xf);
        }
      }
    }
    keep_all_here();
    fetch(h + 1, 0);  // no earlier: the matrices' products need the registers
    // the gates' gradients: A_i and F_j by the wave with the fewest Z to add up
    if (wave == kW - 1) {
      float tq = 0.0f, tk = 0.0f, tf = 0.0f;
#pragma unroll
      for (int w = 0; w < kAcross; ++w) {
        tq += s.sq.qs[w][lane];
        tk += s.sq.ks[w][lane];
        tf += s.sq.kd[w][lane];
      }
      const float from = s.coef.from[lane], beta = s.coef.beta[lane];
      s.a_i[lane] = a.scale * (from * tq) - beta * (from * tk);
      s.f_j[lane] = s.coef.to[lane] * tf;
      float bt = 0.0f;
      for (int c = 0; c <= lane / 16; ++c) bt += s.bt[c][lane];
      const float db = s.rv[lane] - from * tk + bt;
      if (lane < rows) {
        const long e = static_cast<long>(u.t0 + lane) * a.d_beta.row_stride + h;
        if (a.gate_bf16) seq_ptr<bf16>(a.d_beta, u.seq, u.row0, packed)[e] = static_cast<bf16>(db);
        else seq_ptr<float>(a.d_beta, u.seq, u.row0, packed)[e] = db;
      }
    }
    constexpr int kEach = kTok / kW;  // tokens of a wave
    static_assert(kEach == 8, "two values of each group");
    const int t0 = wave * kEach;
    float z = 0.0f;                   // lane j: sum of Z_ij over i >= t
    for (int i = kTok - 8; i >= t0 + kEach; i -= 8) {
      float zs[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) zs[e] = s.sq.z[(i + e) * kSq + lane];
#pragma unroll
      for (int e = 7; e >= 0; --e) z += lane <= i + e ? zs[e] : 0.0f;
    }
    float zs[kEach], dg[2][4];
#pragma unroll
    for (int e = 0; e < kEach; ++e) zs[e] = s.sq.z[(t0 + e) * kSq + lane];
    __syncthreads();
    float ends = 0.0f;
#pragma unroll
    for (int w = 0; w < kAcross; ++w) ends += s.sd[w];
    ends *= s.coef.total;
    const float fj = s.f_j[lane], ai = s.a_i[lane];
#pragma unroll
    for (int e = kEach - 1; e >= 0; --e) {
      const int t = t0 + e;
      z += lane <= t ? zs[e] : 0.0f;
      dg[e >> 2][e & 3] = (lane < t ? z + fj : 0.0f) + (lane >= t ? ai : 0.0f);
    }
    // token 4 n + g of the wave's in the lanes n of group g
    const float low = sum16(sums_of_groups(dg[0])), high = sum16(sums_of_groups(dg[1]));
    const float sum = (l15 == 0 ? low : high) + ends;
    const int t = t0 + 4 * l15 + g;
    if (l15 < 2 && t < rows) {
      const long at = static_cast<long>(u.t0 + t) * a.d_g.row_stride + h;
      if (a.gate_bf16) seq_ptr<bf16>(a.d_g, u.seq, u.row0, packed)[at] = static_cast<bf16>(sum);
      else seq_ptr<float>(a.d_g, u.seq, u.row0, packed)[at] = sum;
    }
  }
  if (parts > 1) {  // added up by delta_sum_kernel
    float* p = a.grad_part + grad_part_at(a, (static_cast<long>(step) * groups + group) * parts + part);
    const unsigned bytes = static_cast<unsigned>(kTok * a.states * 4);
    const Rsrc rq = make_rsrc(p, bytes), rk = make_rsrc(p + kTok * a.states, bytes);
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      const int row = 16 * (i0 + i) + l15, col = 16 * s0 + 4 * g;
      const unsigned off = col < a.states ? static_cast<unsigned>((row * a.states + col) * 4) : kOutside;
      Quad<float>::store(rq, off, dq[i]);
      Quad<float>::store(rk, off, dk[i]);
    }
    return;
  }
  const Rsrc rq = rows_rsrc(seq_ptr<const T>(a.d_q, u.seq, u.row0, packed) + u.t0 * a.d_q.row_stride + group * a.states,
                            a.d_q.row_stride, rows, a.states);
  const Rsrc rk = rows_rsrc(seq_ptr<const T>(a.d_k, u.seq, u.row0, packed) + u.t0 * a.d_k.row_stride + group * a.states,
                            a.d_k.row_stride, rows, a.states);
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const int row = 16 * (i0 + i) + l15, col = 16 * s0 + 4 * g;
    Quad<T>::store(rq, col < a.states ? static_cast<unsigned>((row * static_cast<int>(a.d_q.row_stride) + col) * sizeof(T)) : kOutside, dq[i]);
    Quad<T>::store(rk, col < a.states ? static_cast<unsigned>((row * static_cast<int>(a.d_k.row_stride) + col) * sizeof(T)) : kOutside, dk[i]);
  }
}

// Adds up the parts of a step's and group's shared gradients, in order.
template <class T>
__global__ __launch_bounds__(256) void delta_sum_kernel(DeltaArgs a) {
  const int groups = a.heads / a.ratio, parts = grad_parts(a);
  const int step = blockIdx.x / groups, group = blockIdx.x % groups;
  const Unit u = locate(a.seqs, step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  const bool packed = a.seqs.offsets != nullptr;
  const int rows = min(u.len - u.t0, kTok), quads = a.states / 4;
  const float* p = a.grad_part + grad_part_at(a, static_cast<long>(blockIdx.x) * parts);
  for (int e = threadIdx.x; e < 2 * rows * quads; e += 256) {
    const int which = e >= rows * quads, i = e - which * rows * quads, row = i / quads, col = i % quads * 4;
    const float* src = p + (which * kTok + row) * a.states + col;
    v4f sum = *reinterpret_cast<const v4f*>(src);
    for (int n = 1; n < parts; ++n) sum += *reinterpret_cast<const v4f*>(src + grad_part_at(a, n));
    const mamba2_rows& out = which ? a.d_k : a.d_q;
    T* dst = seq_ptr<T>(out, u.seq, u.row0, packed) + (u.t0 + row) * out.row_stride + group * a.states + col;
    quad_put(dst, sum);
  }
}

// ---------------------------------------------------------------- host side
template <class T, int NB>
int launch_bwd(const DeltaArgs& a, unsigned steps, int type, hipStream_t s) {
  if (steps > 0) {
    delta_bwd_prep_kernel<T, NB><<<prep_blocks(a, steps), kPrepWaves * 64, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    int st = start_segments(a, type, s);
    if (st != MAMBA2_SCAN_OK) return st;
    delta_keep_kernel<T, NB><<<walk_blocks(a), walk_threads<T>, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    if (a.seg_grad != nullptr) {
      delta_reverse_kernel<T, NB, true><<<walk_blocks(a), walk_threads<T>, 0, s>>>(a);
      if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
      if ((st = carry_gradients(a, s)) != MAMBA2_SCAN_OK) return st;
    }
  }
  delta_reverse_kernel<T, NB, false><<<walk_blocks(a), walk_threads<T>, 0, s>>>(a);
  if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  if (steps > 0) {
    const unsigned shared = steps / a.ratio;
    delta_grads_kernel<T, NB><<<shared * grad_parts(a), kGradWaves * 64, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    if (grad_parts(a) > 1) delta_sum_kernel<T><<<shared, 256, 0, s>>>(a);
  }
  return launch_status();
}
template <class T>
int launch_bwd_states(const DeltaArgs& a, unsigned steps, int type, hipStream_t s) {
  if (a.states <= 32) return launch_bwd<T, 1>(a, steps, type, s);
  if (a.states <= 64) return launch_bwd<T, 2>(a, steps, type, s);
  return launch_bwd<T, 4>(a, steps, type, s);
}

// Heads of a group that one work-group takes: all of them, unless that leaves CUs
// without one (there is one on a CU).
int grad_heads(const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const long ratio = d.heads / d.groups, cells = static_cast<long>(unit_count(q, kTok)) * d.heads, each = cells / kCUs;
  return static_cast<int>(each < 1 ? 1 : each < ratio ? each : ratio);
}
size_t grad_part_bytes(const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const int ratio = d.heads / d.groups, each = grad_heads(q, d), parts = (ratio + each - 1) / each;
  if (parts == 1) return 0;
  return static_cast<size_t>(unit_count(q, kTok)) * d.groups * parts * 2 * kTok * d.states * sizeof(float);
}

// The workspace's parts: bytes for each step of each head.
struct BwdCell {
  size_t m, state, rows, all;
};
BwdCell bwd_cell(const mamba2_delta_dims& d) {
  BwdCell c;
  c.m = kPieces * kPiece * sizeof(float);
  c.state = static_cast<size_t>(kept_bytes(d.states, d.width));
  c.rows = static_cast<size_t>(kept_bytes(kTok, d.width));
  c.all = 3 * c.m + 2 * c.state + 2 * c.rows + sizeof(Coef);
  return c;
}

}  // namespace

extern "C" {

size_t mamba2_delta_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims d) {
  if (check_delta(seqs, d) != MAMBA2_SCAN_OK) return 0;
  return static_cast<size_t>(unit_count(seqs, kTok)) * d.heads * bwd_cell(d).all + grad_part_bytes(seqs, d) +
         segment_bytes(seqs, d, true);
}

int mamba2_delta_bwd(mamba2_seqs seqs, mamba2_delta_dims d, mamba2_rows q, mamba2_rows k, mamba2_rows v, mamba2_rows g,
                     mamba2_rows beta, const float* initial_state, mamba2_rows d_y, const float* d_final_state,
                     mamba2_rows d_q, mamba2_rows d_k, mamba2_rows d_v, mamba2_rows d_g, mamba2_rows d_beta,
                     float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  DeltaArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.d_y = d_y;
  a.d_q = d_q;
  a.d_k = d_k;
  a.d_v = d_v;
  a.d_g = d_g;
  a.d_beta = d_beta;
  int st = check_delta(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  mamba2_rows* const keys[] = {&a.q, &a.k, &a.d_q, &a.d_k};
  mamba2_rows* const values[] = {&a.v, &a.d_y, &a.d_v};
  mamba2_rows* const gates[] = {&a.g, &a.beta, &a.d_g, &a.d_beta};
  for (mamba2_rows* r : keys)
    if ((st = check_keys(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  for (mamba2_rows* r : values)
    if ((st = check_values(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  for (mamba2_rows* r : gates)
    if ((st = check_gates(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  if (!aligned_to(initial_state, 16) || !aligned_to(d_final_state, 16) || !aligned_to(d_initial_state, 16))
    return MAMBA2_SCAN_EALIGN;
  if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
  if (workspace_bytes < mamba2_delta_bwd_workspace_bytes(seqs, d)) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  if (seqs.length == 0 && d_initial_state == nullptr) return MAMBA2_SCAN_OK;
  a.initial = initial_state;
  a.d_final = d_final_state;
  a.d_initial = d_initial_state;
  set_dims(&a, seqs, d, true);
  const long cells = static_cast<long>(unit_count(seqs, kTok)) * d.heads;
  const BwdCell c = bwd_cell(d);
  char* at = static_cast<char*>(workspace);
  const auto take = [&](size_t bytes) {
    char* p = at;
    at += cells * bytes;
    return p;
  };
  a.m = reinterpret_cast<float*>(take(c.m));
  a.mt = reinterpret_cast<float*>(take(c.m));
  a.pt = reinterpret_cast<float*>(take(c.m));
  a.keep = reinterpret_cast<float*>(take(c.state));
  a.d_keep = reinterpret_cast<float*>(take(c.state));
  a.u = reinterpret_cast<float*>(take(c.rows));
  a.d_r = reinterpret_cast<float*>(take(c.rows));
  a.coef = reinterpret_cast<Coef*>(take(sizeof(Coef)));
  const unsigned steps = seqs.length == 0 ? 0 : static_cast<unsigned>(cells);
  a.grad_heads = grad_heads(seqs, d);
  a.grad_part = reinterpret_cast<float*>(at);
  set_segments(&a, at + grad_part_bytes(seqs, d), true);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return d.type == MAMBA2_BF16 ? launch_bwd_states<bf16>(a, steps, d.type, s) : launch_bwd_states<float>(a, steps, d.type, s);
}

}  // extern "C"
