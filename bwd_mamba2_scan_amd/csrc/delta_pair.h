// The walks of the gated delta rule for bf16 tensors: eight waves of two roles.
//
// A walk is a chain: a step's state needs the last one's.  Four waves walk, 16
// columns of the state each, and do nothing that the chain does not need; a
// helper wave beside each loads the next step, computes what does not depend on
// the chain and moves results to memory.  Walkers and helpers share a SIMD in
// pairs and meet three times a step.  With four waves that did everything, a
// step of 128 states took 10000 cycles, half of them loads, results and waits.
#pragma once

#include "delta_walk.h"

namespace delta {

constexpr int kPairThreads = 2 * kWaves * 64;
constexpr int kHelpers = kWaves * 64;
// Threads of a walk: fp32's tiles leave no LDS for what walkers and helpers exchange.
template <class T>
constexpr int walk_threads = sizeof(T) == 2 ? kPairThreads : kWaves * 64;

// A 16 x 16 fp32 tile that a walker hands to its helper or back: lane l's four
// values at 4 (l + l / 16), so that reading four columns of a row takes distinct banks.
constexpr int kSwapTile = 68 * 4;
__device__ __forceinline__ void swap_put(float* p, int lane, v4f v) {
  *reinterpret_cast<v4f*>(p + 4 * (lane + (lane >> 4))) = v;
}
__device__ __forceinline__ v4f swap_get(const float* p, int lane) {
  return *reinterpret_cast<const v4f*>(p + 4 * (lane + (lane >> 4)));
}
// Row lane / 4 of a tile, columns 4 (lane % 4) ..
__device__ __forceinline__ v4f swap_row(const float* p, int lane) {
  const int row = lane >> 2, at = 4 * (17 * (row >> 2) + 4 * (lane & 3)) + (row & 3);
  return v4f{p[at], p[at + 4], p[at + 8], p[at + 12]};
}
// The tiles of a wave's 16 columns of `rows` rows, kept.
template <int TILES>
__device__ __forceinline__ void swap_keep(float* out, int rows, int width, int col0, const float* p, int lane) {
  const Rsrc rs = make_rsrc(out, static_cast<unsigned>(kept_bytes(rows, width)));
  const int c = col0 + 4 * (lane & 3), strip = kept_strip(width);
  const unsigned off = c < width ? static_cast<unsigned>(kept_at(lane >> 2, c)) : kOutside;
#pragma unroll
  for (int n = 0; n < TILES; ++n)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, swap_row(p + n * kSwapTile, lane)), rs, off + n * strip, 0, 0);
}

// A matrix's fp32 pieces on their way to LDS, where they lie in three bf16 parts that
// add up to them.  In memory they would be half as long again.
struct Pieces {
  static constexpr int kN = kPieces * kPiece / 4 / kHelpers;
  v4f v[kN];
  __device__ __forceinline__ void load(const float* p, long cell, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = reinterpret_cast<const v4f*>(p + cell * kPieces * kPiece)[tid + i * kHelpers];
  }
  __device__ __forceinline__ void store(bf16* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) quad_put_parts<3>(lds + 4 * (tid + i * kHelpers), kPieces * kPiece, v[i]);
  }
};

// What the walkers read of a step.
template <int NB>
struct PairStep {
  static constexpr int ldn = stride_of<bf16>(NB * 32);
  alignas(16) bf16 k[kTok * ldn];
  alignas(16) bf16 m[3 * kPieces * kPiece];
  alignas(16) Coef coef;
};

__device__ __forceinline__ void read_pieces(Frag<bf16> (&f)[3][kPieces], const bf16* p, int lane) {
#pragma unroll
  for (int z = 0; z < 3; ++z)
#pragma unroll
    for (int i = 0; i < kPieces; ++i) f[z][i] = piece_get(p + (z * kPieces + i) * kPiece, lane);
}


template <int NB, Walked MODE>
struct PairFwdLds {
  static constexpr int ldn = stride_of<bf16>(NB * 32);
  static constexpr int ldv = stride_of<bf16>(kCols);
  PairStep<NB> step[2];
  alignas(16) bf16 v[2][kTok * ldv];
  union {
    struct {
      bf16 q[kTok * ldn];
      bf16 s[kWaves][NB][2][kPiece];   // a walker's state, in two parts
      bf16 u[kWaves][2][2][kPiece];    // its U
    } out;
    struct {
      float s[kWaves][2 * NB * kSwapTile];
      float u[kWaves][4 * kSwapTile];
    } keep;
  };
};

// As walk_forward.
template <int NB, Walked MODE>
__device__ __forceinline__ void pair_forward(const DeltaArgs& a, PairFwdLds<NB, MODE>& s) {
  typedef PairFwdLds<NB, MODE> L;
  constexpr int kP = 2 * kPieces * kPiece;
  const int wave = wave_id(), lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  const int strip = wave & (kWaves - 1);
  const Columns cl = columns_of<MODE>(a);
  if (cl.unit < 0) return;
  const Unit u = locate(a.seqs, cl.unit, a.seg);
  if (!u.live || !wanted<MODE>(a, cl, u)) return;
  const int h = cl.h, p0 = cl.p0;
  const bool packed = a.seqs.offsets != nullptr;
  const long kept = kept_bytes(a.states, a.width) / 4, slab = kept_bytes(kTok, a.width) / 4;
  const long cell0 = static_cast<long>(unit_base(a.seqs, u.seq, kTok)) * a.heads + h;  // of the sequence's first step
  const int end = min(u.t0 + a.seg, u.len);

  if (wave >= kWaves) {  // a helper
    const int tid = threadIdx.x - kHelpers;
    const bf16* kp = seq_ptr<const bf16>(a.k, u.seq, u.row0, packed) + h / a.ratio * a.states;
    const bf16* qp = seq_ptr<const bf16>(a.q, u.seq, u.row0, packed) + h / a.ratio * a.states;
    const bf16* vp = seq_ptr<const bf16>(a.v, u.seq, u.row0, packed) + h * a.width + p0;
    bf16* yp = seq_ptr<bf16>(a.y, u.seq, u.row0, packed) + h * a.width;
    Tile<bf16, kTok, NB * 32, kHelpers> tk, tq;
    Tile<bf16, kTok, kCols, kHelpers> tv;
    Pieces tm;
    Flat<sizeof(Coef), kHelpers> tc;
    Frag<bf16> pf[2][kPieces];
    const int cols = cl.cols;
    tk.init(a.k.row_stride, a.states, tid);
    tq.init(a.q.row_stride, a.states, tid);
    tv.init(a.v.row_stride, cols, tid);
    const int quad = p0 + strip * 16 + 4 * g;
    const unsigned y_off = quad < a.width ? static_cast<unsigned>((l15 * static_cast<int>(a.y.row_stride) + quad) * 2) : kOutside;
    const int y16 = static_cast<int>(32 * a.y.row_stride);
    const auto fetch = [&](int t) {
      const int rows = min(end - t, kTok);
      const long at = cell0 + static_cast<long>(t / kTok) * a.heads;
      tk.load(rows_rsrc(kp + t * a.k.row_stride, a.k.row_stride, rows, a.states));
      tm.load(a.m, at, tid);
      tc.load(a.coef + at, tid);
      tv.load(rows_rsrc(vp + t * a.v.row_stride, a.v.row_stride, rows, cols));
      if (MODE == kResults) tq.load(rows_rsrc(qp + t * a.q.row_stride, a.q.row_stride, rows, a.states));
    };
    const auto put = [&](int b) {
      tk.store(s.step[b].k, L::ldn, tid);
      tm.store(s.step[b].m, tid);
      tc.store(&s.step[b].coef, tid);
      tv.store(s.v[b], L::ldv, tid);
      if (MODE == kResults) tq.store(s.out.q, L::ldn, tid);
    };
    const auto fetch_p = [&](int t) {
      const bf16* p = static_cast<const bf16*>(a.p) + (cell0 + static_cast<long>(t / kTok) * a.heads) * kP;
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) pf[z][i] = piece_get(p + (z * kPieces + i) * kPiece, lane);
    };
    // the step behind the one at t; behind the last one, it again: a branch here would
    // make the waits for these loads wait for what is issued after them, too
    const auto behind = [&](int t) { return t + kTok < end ? t + kTok : t; };
    if (u.t0 < end) {
      fetch(u.t0);
      if (MODE == kResults) fetch_p(u.t0);
      put(0);
      if (MODE == kSummary) fetch(behind(u.t0));
    }
    int b = 0;
    for (int t = u.t0; t < end; t += kTok, b ^= 1) {
      __syncthreads();
      const int next = behind(t);
      if (MODE == kSummary) {  // with nothing else to do, loaded a step ahead
        put(b ^ 1);
        fetch(behind(next));
        continue;
      }
      fetch(next);
      __syncthreads();  // the state is in LDS
      const long cell = cell0 + static_cast<long>(t / kTok) * a.heads;
      v4f y[4];
      if (MODE == kKept) {
        swap_keep<2 * NB>(a.keep + cell * kept, a.states, a.width, p0 + strip * 16, s.keep.s[strip], lane);
      } else {  // (Q S)^T
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const Frag<bf16> s0 = piece_get(s.out.s[strip][n][0], lane), s1 = piece_get(s.out.s[strip][n][1], lane);
          Frag<bf16> qf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[i] = frag_row_result(s.out.q, L::ldn, 16 * i, 32 * n);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma(y[i], s1, qf[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) mma(y[i], s0, qf[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = y[i] * (a.scale * s.step[b].coef.from[16 * i + l15]);
      }
      __syncthreads();  // U is in LDS
      if (MODE == kKept) {
        swap_keep<4>(a.u + cell * slab, kTok, a.width, p0 + strip * 16, s.keep.u[strip], lane);
      } else {
        Split<bf16, 2> us[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int z = 0; z < 2; ++z) us[j].f[z] = piece_get(s.out.u[strip][j][z], lane);
        mma_lower<bf16, 2, 2, true>(y, pf, us);
        fetch_p(next);
        const Rsrc ry = rows_rsrc(yp + t * a.y.row_stride, a.y.row_stride, min(end - t, kTok), a.width);
#pragma unroll
        for (int i = 0; i < 4; ++i) Quad<bf16>::store(ry, y_off + i * y16, y[i]);
      }
      // Here, where walkers have little to do: put beside their first product, a step
      // ahead, the walk of delta_fwd_kernel's figures took 294 us for 275, and with P U
      // and the results there 289.
      put(b ^ 1);
    }
    return;
  }

  State<NB, true> st;
  first_state<MODE>(st, a, cl, u, strip);
  int b = 0;
  for (int t = u.t0; t < end; t += kTok, b ^= 1) {
    __syncthreads();
    const PairStep<NB>& p = s.step[b];
    Frag<bf16> kf[2][4];
    const auto read_rows = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[n & 1][i] = frag_row_result(p.k, L::ldn, 16 * i, 32 * n);
    };
    read_rows(0);
    if (MODE == kKept) {
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n) swap_put(s.keep.s[strip] + n * kSwapTile, lane, st.st[n]);
    }
    v4f ks[4], x[4];
    Frag<bf16> mf[3][kPieces];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n + 1 < NB) {
        read_rows(n + 1);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = tile_col(s.v[b], L::ldv, i, strip * 16, lane);
        read_pieces(mf, p.m, lane);
      }
      keep_reads_here();
      const Split<bf16, 3> sp = split_pair<bf16, 3>(st.st[2 * n], st.st[2 * n + 1]);
      if (MODE == kResults) {
        piece_put(s.out.s[strip][n][0], lane, sp.f[0]);
        piece_put(s.out.s[strip][n][1], lane, sp.f[1]);
      }
#pragma unroll
      for (int z = 2; z >= 0; --z)
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(ks[i], kf[n & 1][i], sp.f[z]);
    }
    if (MODE != kSummary) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = rows_of(p.coef.beta, i, g) * (x[i] - rows_of(p.coef.from, i, g) * ks[i]);
    const Split<bf16, 3> xs[2] = {split_pair<bf16, 3>(x[0], x[1]), split_pair<bf16, 3>(x[2], x[3])};
    v4f w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v4f{0, 0, 0, 0};
    mma_lower<bf16, 3, 3>(w, mf, xs);
    constexpr int kTiles = 2 * NB < 4 ? 2 * NB : 4;
    Frag<bf16> cf[2][kTiles];
    const auto read_cols = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) cf[j][i] = frag_col_result(p.k, L::ldn, 32 * j, 16 * (n + i));
    };
    v4f to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = rows_of(p.coef.to, i, g);
    read_cols(0);
    const float total = p.coef.total;
    keep_reads_here();
    if (MODE == kKept) {
#pragma unroll
      for (int i = 0; i < 4; ++i) swap_put(s.keep.u[strip] + i * kSwapTile, lane, w[i]);
    } else if (MODE == kResults) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Split<bf16, 2> us = split_pair<bf16, 2>(w[2 * j], w[2 * j + 1]);
        piece_put(s.out.u[strip][j][0], lane, us.f[0]);
        piece_put(s.out.u[strip][j][1], lane, us.f[1]);
      }
    }
    if (MODE != kSummary) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * to[i];
    const Split<bf16, 3> us[2] = {split_pair<bf16, 3>(w[0], w[1]), split_pair<bf16, 3>(w[2], w[3])};
#pragma unroll
    for (int n = 0; n < 2 * NB; n += kTiles) {
      v4f add[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) add[i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int z = 2; z >= 0; --z)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) mma(add[i], cf[j][i], us[j].f[z]);
      if (n + kTiles < 2 * NB) read_cols(n + kTiles);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) st.st[n + i] = st.st[n + i] * total + add[i];
    }
  }
  last_state<MODE>(st, a, cl, u, strip);
}

template <int NB>
struct PairRevLds {
  static constexpr int ldn = stride_of<bf16>(NB * 32);
  static constexpr int ldv = stride_of<bf16>(kCols);
  PairStep<NB> step;                                // m: M^T
  alignas(16) bf16 pt[3 * kPieces * kPiece];
  alignas(16) bf16 y[kTok * ldv];
  alignas(16) bf16 q[kTok * ldn];
  alignas(16) float r[kWaves][4 * kSwapTile];       // a walker's dR
  alignas(16) float d[kWaves][2 * NB * kSwapTile];  // its D, then scale Q^T (2^c dY) for it
};

// As walk_reverse.  LDS holds one step here: the helpers keep the next one in
// registers until the walkers are done with this one's operands.
template <int NB, bool SUMMARY>
__device__ __forceinline__ void pair_reverse(const DeltaArgs& a, PairRevLds<NB>& s) {
  typedef PairRevLds<NB> L;
  constexpr int kTiles = 2 * NB < 4 ? 2 * NB : 4;
  const int wave = wave_id(), lane = threadIdx.x & 63, g = lane >> 4;
  const int strip = wave & (kWaves - 1);
  const WalkWork wk = walk_work(a, a.slices);
  if (wk.unit < 0) return;
  const Unit u = locate(a.seqs, wk.unit, a.seg);
  if (!u.live || (SUMMARY && u.index == 0)) return;
  const int h = wk.h, slice = wk.slice;
  const bool packed = a.seqs.offsets != nullptr;
  const int p0 = slice * kCols;
  const long kept = kept_bytes(a.states, a.width) / 4, slab = kept_bytes(kTok, a.width) / 4;
  const long cell0 = static_cast<long>(unit_base(a.seqs, u.seq, kTok)) * a.heads + h;
  const int end = min(u.t0 + a.seg, u.len);
  const int last = end > u.t0 ? u.t0 + (end - 1 - u.t0) / kTok * kTok : u.t0 - kTok;
  const Coef& coef = s.step.coef;

  if (wave >= kWaves) {  // a helper
    const int tid = threadIdx.x - kHelpers;
    const bf16* kp = seq_ptr<const bf16>(a.k, u.seq, u.row0, packed) + h / a.ratio * a.states;
    const bf16* qp = seq_ptr<const bf16>(a.q, u.seq, u.row0, packed) + h / a.ratio * a.states;
    const bf16* yp = seq_ptr<const bf16>(a.d_y, u.seq, u.row0, packed) + h * a.width + p0;
    bf16* vp = seq_ptr<bf16>(a.d_v, u.seq, u.row0, packed) + h * a.width;
    Tile<bf16, kTok, NB * 32, kHelpers> tk, tq;
    Tile<bf16, kTok, kCols, kHelpers> ty;
    Pieces tm, tp;
    Flat<sizeof(Coef), kHelpers> tc;
    const int cols = min(a.width - p0, kCols);
    tk.init(a.k.row_stride, a.states, tid);
    tq.init(a.q.row_stride, a.states, tid);
    ty.init(a.d_y.row_stride, cols, tid);
    // dV: row lane / 4 of each tile, four columns
    const int quad = p0 + strip * 16 + 4 * (lane & 3);
    const unsigned v_off = quad < a.width ? static_cast<unsigned>(((lane >> 2) * static_cast<int>(a.d_v.row_stride) + quad) * 2) : kOutside;
    const int v16 = static_cast<int>(32 * a.d_v.row_stride);
    const auto fetch = [&](int t) {
      const int rows = min(end - t, kTok);
      const long at = cell0 + static_cast<long>(t / kTok) * a.heads;
      tk.load(rows_rsrc(kp + t * a.k.row_stride, a.k.row_stride, rows, a.states));
      tq.load(rows_rsrc(qp + t * a.q.row_stride, a.q.row_stride, rows, a.states));
      ty.load(rows_rsrc(yp + t * a.d_y.row_stride, a.d_y.row_stride, rows, cols));
      tm.load(a.mt, at, tid);
      tp.load(a.pt, at, tid);
      tc.load(a.coef + at, tid);
    };
    const auto put = [&] {
      tk.store(s.step.k, L::ldn, tid);
      tq.store(s.q, L::ldn, tid);
      ty.store(s.y, L::ldv, tid);
      tm.store(s.step.m, tid);
      tp.store(s.pt, tid);
      tc.store(&s.step.coef, tid);
    };
    if (last >= u.t0) fetch(last);
    for (int t = last; t >= u.t0; t -= kTok) {
      put();
      __syncthreads();  // the step's operands are in LDS
      const int next = t > u.t0 ? t - kTok : t;  // as in the forward walk
      fetch(next);
      float beta[4];
      v4f add[2 * NB];
      {  // scale Q^T (2^c dY)
        v4f dy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          beta[i] = coef.beta[16 * i + (lane >> 2)];
          dy[i] = a.scale * (rows_of(coef.from, i, g) * tile_col(s.y, L::ldv, i, strip * 16, lane));
        }
        const Split<bf16, 3> ss[2] = {split_pair<bf16, 3>(dy[0], dy[1]), split_pair<bf16, 3>(dy[2], dy[3])};
#pragma unroll
        for (int n = 0; n < 2 * NB; n += kTiles) {
          Frag<bf16> qf[2][kTiles];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < kTiles; ++i) qf[j][i] = frag_col_result(s.q, L::ldn, 32 * j, 16 * (n + i));
#pragma unroll
          for (int i = 0; i < kTiles; ++i) add[n + i] = v4f{0, 0, 0, 0};
#pragma unroll
          for (int z = 2; z >= 0; --z)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < kTiles; ++i) mma(add[n + i], qf[j][i], ss[j].f[z]);
        }
      }
      __syncthreads();  // D and dR are in LDS
      const long cell = cell0 + static_cast<long>(t / kTok) * a.heads;
      if (!SUMMARY) swap_keep<2 * NB>(a.d_keep + cell * kept, a.states, a.width, p0 + strip * 16, s.d[strip], lane);
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n) swap_put(s.d[strip] + n * kSwapTile, lane, add[n]);
      __syncthreads();  // the walkers are done with the operands but for what was put last
      if (SUMMARY) continue;
      swap_keep<4>(a.d_r + cell * slab, kTok, a.width, p0 + strip * 16, s.r[strip], lane);
      const Rsrc rv = rows_rsrc(vp + t * a.d_v.row_stride, a.d_v.row_stride, min(end - t, kTok), a.width);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        Quad<bf16>::store(rv, v_off + i * v16, swap_row(s.r[strip] + i * kSwapTile, lane) * beta[i]);
    }
    return;
  }

  State<NB, true> st;
  st.init(a.width, p0, strip);
  first_gradient<SUMMARY>(st, a, wk, u);
  for (int t = last; t >= u.t0; t -= kTok) {
    __syncthreads();
    const PairStep<NB>& p = s.step;
    Frag<bf16> kf[2][4];
    const auto read_rows = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[n & 1][i] = frag_row_result(p.k, L::ldn, 16 * i, 32 * n);
    };
    read_rows(0);
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n)
      if (!SUMMARY) swap_put(s.d[strip] + n * kSwapTile, lane, st.st[n]);
    v4f w[4], dy[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v4f{0, 0, 0, 0};
    Frag<bf16> mf[3][kPieces];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n + 1 < NB) {
        read_rows(n + 1);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) dy[i] = tile_col(s.y, L::ldv, i, strip * 16, lane);
        read_pieces(mf, s.pt, lane);
      }
      keep_reads_here();
      const Split<bf16, 3> sp = split_pair<bf16, 3>(st.st[2 * n], st.st[2 * n + 1]);
#pragma unroll
      for (int z = 2; z >= 0; --z)
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(w[i], kf[n & 1][i], sp.f[z]);
    }
    // dU, then dR
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * rows_of(p.coef.to, i, g);
    {
      const Split<bf16, 1> ys[2] = {split_pair<bf16, 1>(dy[0], dy[1]), split_pair<bf16, 1>(dy[2], dy[3])};
      mma_upper<bf16, 3, 1>(w, mf, ys);
    }
    keep_reads_here();
    read_pieces(mf, p.m, lane);
    v4f coefs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) coefs[i] = rows_of(p.coef.beta, i, g) * rows_of(p.coef.from, i, g);
    const float total = p.coef.total;
    keep_reads_here();
    const Split<bf16, 3> us[2] = {split_pair<bf16, 3>(w[0], w[1]), split_pair<bf16, 3>(w[2], w[3])};
    v4f dr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dr[i] = v4f{0, 0, 0, 0};
    mma_upper<bf16, 3, 3>(dr, mf, us);
    Frag<bf16> cf[2][kTiles];
    const auto read_cols = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) cf[j][i] = frag_col_result(p.k, L::ldn, 32 * j, 16 * (n + i));
    };
    read_cols(0);
    keep_reads_here();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!SUMMARY) swap_put(s.r[strip] + i * kSwapTile, lane, dr[i]);
    __syncthreads();
    // D = 2^c_end D - K^T (beta 2^c dR) + what the helper has
#pragma unroll
    for (int i = 0; i < 4; ++i) dr[i] = -coefs[i] * dr[i];
    const Split<bf16, 3> rs[2] = {split_pair<bf16, 3>(dr[0], dr[1]), split_pair<bf16, 3>(dr[2], dr[3])};
    v4f add[2 * NB];
#pragma unroll
    for (int n = 0; n < 2 * NB; n += kTiles) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i) add[n + i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int z = 2; z >= 0; --z)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) mma(add[n + i], cf[j][i], rs[j].f[z]);
      if (n + kTiles < 2 * NB) read_cols(n + kTiles);
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n)
      st.st[n] = st.st[n] * total + (add[n] + swap_get(s.d[strip] + n * kSwapTile, lane));
  }
  last_gradient<SUMMARY>(st, a, wk, u);
}

}  // namespace delta
