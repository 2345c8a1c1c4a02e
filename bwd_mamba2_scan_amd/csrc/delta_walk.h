// The walks of the gated delta rule's states over the tokens.
#pragma once

#include "delta_common.h"

namespace delta {

constexpr int kWaves = 4;  // of a walk: 64 columns

// Contiguous memory to LDS, in 16-byte vectors by THREADS threads.
template <int BYTES, int THREADS>
struct Flat {
  static constexpr int kAll = BYTES / 16, kN = (kAll + THREADS - 1) / THREADS;
  v4u v[kN];
  __device__ __forceinline__ void load(const void* p, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = min(tid + i * THREADS, kAll - 1);
      v[i] = static_cast<const v4u*>(p)[e];
    }
  }
  __device__ __forceinline__ void store(void* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = tid + i * THREADS;
      if (kAll % THREADS == 0 || e < kAll) static_cast<v4u*>(lds)[e] = v[i];
    }
  }
};

constexpr int kCols = kWaves * 16;

// A wave's columns of `rows` rows, kept.
template <int N>
__device__ __forceinline__ void save_kept(float* p, int rows, int width, int col, int g, const v4f (&w)[N]) {
  const Rsrc rs = make_rsrc(p, static_cast<unsigned>(kept_bytes(rows, width)));
  const int strip = kept_strip(width);
  const unsigned off = col < width ? static_cast<unsigned>(kept_at(4 * g, col)) : kOutside;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) store_elem<float>(rs, off + n * strip + 16 * i, w[n][i]);
}

// Four rows 4 g .. of column l15 of tile i of an LDS tile of tokens.
__device__ __forceinline__ v4f tile_col(const bf16* p, int ld, int i, int col, int lane) {
  const v4s r = read_tr(p + (16 * i + 4 * (lane >> 4) + ((lane & 15) >> 2)) * ld + col + 4 * (lane & 3));
  v4f v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(static_cast<unsigned>(static_cast<unsigned short>(r[j])) << 16);
  return v;
}
__device__ __forceinline__ v4f tile_col(const float* p, int ld, int i, int col, int lane) {
  const float* r = p + (16 * i + 4 * (lane >> 4)) * ld + col + (lane & 15);
  return v4f{r[0], r[ld], r[2 * ld], r[3 * ld]};
}

// A walk's columns: of the head's values, or in a summary behind those of the
// state itself.
struct Columns {
  int unit, h, p0, width, cols;  // cols: of V
  bool trans;
};
template <Walked MODE>
__device__ __forceinline__ Columns columns_of(const DeltaArgs& a) {
  const int ks = MODE == kSummary ? (a.states + kCols - 1) / kCols : 0;
  const WalkWork w = walk_work(a, a.slices + ks);
  const bool trans = MODE == kSummary && w.slice >= a.slices;
  const int p0 = (trans ? w.slice - a.slices : w.slice) * kCols;
  return {w.unit, w.h, p0, trans ? a.states : a.width, trans ? 0 : min(a.width - p0, kCols), trans};
}
__device__ __forceinline__ bool last_unit(const DeltaArgs& a, const Unit& u) {
  return u.t0 + static_cast<long>(a.seg) >= u.len;
}
// A summary is of use to a segment behind, and in the backward, where the gradient
// passes through the transposed transitions, of a segment before.
template <Walked MODE>
__device__ __forceinline__ bool wanted(const DeltaArgs& a, const Columns& c, const Unit& u) {
  if (MODE != kSummary) return true;
  const bool last = last_unit(a, u);
  if (c.trans) return last ? a.seg_grad != nullptr && u.index > 0 : true;
  return !last;
}
template <Walked MODE, int NB>
__device__ __forceinline__ void first_state(State<NB, true>& st, const DeltaArgs& a, const Columns& c, const Unit& u, int strip) {
  const long head = static_cast<long>(a.states) * a.width;
  st.init(c.width, c.p0, strip);
  if (MODE == kSummary) {
    const int lane = threadIdx.x & 63, col = c.p0 + strip * 16 + (lane & 15), row = 4 * (lane >> 4);
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) st.st[n][i] = c.trans && 16 * n + row + i == col ? 1.0f : 0.0f;
  } else if (u.index > 0) {
    st.load(a.seg_state + (static_cast<long>(c.unit) * a.heads + c.h) * head, a.width, a.states);
  } else {
    st.load(a.initial == nullptr ? nullptr : a.initial + (static_cast<long>(u.seq) * a.heads + c.h) * head, a.width, a.states);
  }
}
template <Walked MODE, int NB>
__device__ __forceinline__ void last_state(const State<NB, true>& st, const DeltaArgs& a, const Columns& c, const Unit& u, int strip) {
  const long at = static_cast<long>(c.unit) * a.heads + c.h;
  if (MODE == kSummary) {
    if (c.trans) {
      const long square = static_cast<long>(a.states) * a.states;
      st.save(a.seg_trans + at * square, a.states, a.states);
      if (a.seg_trans_t != nullptr) {  // its transpose: this lane's column is a row, 4 g .. of each tile
        const int lane = threadIdx.x & 63, row = c.p0 + strip * 16 + (lane & 15), col = 4 * (lane >> 4);
        const Rsrc rs = make_rsrc(a.seg_trans_t + at * square, static_cast<unsigned>(square * 4));
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n)
          Quad<float>::store(rs, row < a.states && 16 * n + col < a.states ? static_cast<unsigned>((row * a.states + 16 * n + col) * 4) : kOutside, st.st[n]);
      }
    } else st.save(a.seg_state + (at + a.heads) * a.states * a.width, a.width, a.states);  // the next one's place
  } else if (MODE == kResults && a.final_state != nullptr && last_unit(a, u)) {
    st.save(a.final_state + (static_cast<long>(u.seq) * a.heads + c.h) * a.states * a.width, a.width, a.states);
  }
}

template <class T, int NB, Walked MODE>
struct FwdLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  static constexpr int ldv = stride_of<T>(kCols);
  alignas(16) T k[kTok * ldn];
  alignas(16) T m[kExact<T> * kPieces * kPiece];
  alignas(16) Coef coef;
  alignas(16) T v[kTok * ldv];
  alignas(16) T q[MODE != kResults ? 8 : kTok * ldn];
  alignas(16) T p[MODE != kResults ? 8 : kTwo<T> * kPieces * kPiece];
};

// The walk of 64 columns of a head over a segment.
template <class T, int NB, Walked MODE>
__device__ __forceinline__ void walk_forward(const DeltaArgs& a, FwdLds<T, NB, MODE>& s) {
  typedef FwdLds<T, NB, MODE> L;
  constexpr int kThreads = kWaves * 64;
  constexpr int kM = kExact<T> * kPieces * kPiece, kP = kTwo<T> * kPieces * kPiece;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const Columns cl = columns_of<MODE>(a);
  if (cl.unit < 0) return;
  const Unit u = locate(a.seqs, cl.unit, a.seg);
  if (!u.live || !wanted<MODE>(a, cl, u)) return;
  const int h = cl.h, p0 = cl.p0;
  const bool packed = a.seqs.offsets != nullptr;
  const int col = p0 + wave * 16 + l15;
  const T* kp = seq_ptr<const T>(a.k, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* qp = seq_ptr<const T>(a.q, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* vp = seq_ptr<const T>(a.v, u.seq, u.row0, packed) + h * a.width + p0;
  T* yp = seq_ptr<T>(a.y, u.seq, u.row0, packed) + h * a.width;

  State<NB, true> st;
  first_state<MODE>(st, a, cl, u, wave);

  const int end = min(u.t0 + a.seg, u.len);
  const long cell0 = static_cast<long>(unit_base(a.seqs, u.seq, kTok)) * a.heads + h;  // of the sequence's first step
  Tile<T, kTok, NB * 32, kThreads> tk, tq;
  tk.init(a.k.row_stride, a.states, tid);
  tq.init(a.q.row_stride, a.states, tid);
  Flat<kM * sizeof(T), kThreads> tm;
  Flat<kP * sizeof(T), kThreads> tp;
  Flat<sizeof(Coef), kThreads> tc;
  Tile<T, kTok, kCols, kThreads> tv;
  tv.init(a.v.row_stride, cl.cols, tid);
  // y^T: this lane's token of each tile, four columns
  const int quad = p0 + wave * 16 + 4 * g;
  const unsigned y_off = quad < a.width ? static_cast<unsigned>((l15 * static_cast<int>(a.y.row_stride) + quad) * sizeof(T)) : kOutside;
  const int y16 = static_cast<int>(16 * a.y.row_stride * sizeof(T));
  const auto fetch = [&](int t) {
    const int rows = min(end - t, kTok);
    const long at = cell0 + static_cast<long>(t / kTok) * a.heads;
    tk.load(rows_rsrc(kp + t * a.k.row_stride, a.k.row_stride, rows, a.states));
    if (MODE == kResults) tq.load(rows_rsrc(qp + t * a.q.row_stride, a.q.row_stride, rows, a.states));
    tm.load(a.m + at * kPieces * kPiece, tid);
    if (MODE == kResults) tp.load(static_cast<const T*>(a.p) + at * kP, tid);
    tc.load(a.coef + at, tid);
    tv.load(rows_rsrc(vp + t * a.v.row_stride, a.v.row_stride, rows, cl.cols));
  };
  if (u.t0 < end) fetch(u.t0);
  for (int t = u.t0; t < end; t += kTok) {
    __syncthreads();
    tk.store(s.k, L::ldn, tid);
    if (MODE == kResults) tq.store(s.q, L::ldn, tid);
    tm.store(s.m, tid);
    if (MODE == kResults) tp.store(s.p, tid);
    tc.store(&s.coef, tid);
    tv.store(s.v, L::ldv, tid);
    __syncthreads();
    if (t + kTok < end) fetch(t + kTok);

    const long cell = cell0 + static_cast<long>(t / kTok) * a.heads;
    if (MODE == kKept) save_kept(a.keep + cell * (kept_bytes(a.states, a.width) / 4), a.states, a.width, col, g, st.st);
    // K S and (Q S)^T.  The operands of a part are read from LDS while the part
    // before it is multiplied: one wave a SIMD hides no latency by itself.
    constexpr int kBuf = NB > 1 ? 2 : 1;
    Frag<T> kf[kBuf][4], qf[kBuf][4];
    Frag<T> mf[kExact<T>][kPieces];
    const auto read_rows = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kf[n % kBuf][i] = frag_row_result(s.k, L::ldn, 16 * i, 32 * n);
        if (MODE == kResults) qf[n % kBuf][i] = frag_row_result(s.q, L::ldn, 16 * i, 32 * n);
      }
    };
    v4f ks[4], qs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = v4f{0, 0, 0, 0};
    read_rows(0);
    v4f from[4], beta[4], to[4], x[4];
    float mine[4];  // scale 2^c of this lane's token of each tile
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n + 1 < NB) {
        read_rows(n + 1);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          beta[i] = rows_of(s.coef.beta, i, g);
          from[i] = rows_of(s.coef.from, i, g);
          x[i] = tile_col(s.v, L::ldv, i, wave * 16, lane);
        }
#pragma unroll
        for (int z = 0; z < kExact<T>; ++z)
#pragma unroll
          for (int i = 0; i < kPieces; ++i) mf[z][i] = piece_get(s.m + (z * kPieces + i) * kPiece, lane);
      }
      keep_reads_here();
      const Split<T, kExact<T>> sp = split_pair<T, kExact<T>>(st.st[2 * n], st.st[2 * n + 1]);
#pragma unroll
      for (int z = kExact<T> - 1; z >= 0; --z) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(ks[i], kf[n % kBuf][i], sp.f[z]);
        if (MODE == kResults && z < kTwo<T>) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mma(qs[i], sp.f[z], qf[n % kBuf][i]);
        }
      }
    }
    // beta (V - 2^c K S), then U = M that
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = beta[i] * (x[i] - from[i] * ks[i]);
    const Split<T, kExact<T>> xs[2] = {split_pair<T, kExact<T>>(x[0], x[1]), split_pair<T, kExact<T>>(x[2], x[3])};
    Frag<T> pf[kTwo<T>][kPieces];
    if (MODE == kResults) {
#pragma unroll
      for (int z = 0; z < kTwo<T>; ++z)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) pf[z][i] = piece_get(s.p + (z * kPieces + i) * kPiece, lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      to[i] = rows_of(s.coef.to, i, g);
      if (MODE == kResults) mine[i] = a.scale * s.coef.from[16 * i + l15];
    }
    keep_reads_here();
    v4f w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v4f{0, 0, 0, 0};
    mma_lower<T, kExact<T>, kExact<T>>(w, mf, xs);
    // the left operands of the state's products, four tiles at a time
    constexpr int kTiles = 2 * NB < 4 ? 2 * NB : 4;
    Frag<T> cf[2][kTiles];
    const auto read_cols = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) cf[j][i] = frag_col_result(s.k, L::ldn, 32 * j, 16 * (n + i));
    };
    read_cols(0);
    keep_reads_here();
    if (MODE == kKept) {
      save_kept(a.u + cell * (kept_bytes(kTok, a.width) / 4), kTok, a.width, col, g, w);
    } else if (MODE == kResults) {  // Y^T = (scale 2^c Q S)^T + U^T P^T
      const Split<T, kTwo<T>> us[2] = {split_pair<T, kTwo<T>>(w[0], w[1]), split_pair<T, kTwo<T>>(w[2], w[3])};
      const Rsrc ry = rows_rsrc(yp + t * a.y.row_stride, a.y.row_stride, min(end - t, kTok), a.width);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[i] = qs[i] * mine[i];
      mma_lower<T, kTwo<T>, kTwo<T>, true>(qs, pf, us);
#pragma unroll
      for (int i = 0; i < 4; ++i) Quad<T>::store(ry, y_off + i * y16, qs[i]);
    }
    // S = 2^c_end S + K^T (2^(c_end - c) U); a step's products are added up by
    // themselves: on top of the state, each would round at the state's size
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * to[i];
    const Split<T, kExact<T>> us[2] = {split_pair<T, kExact<T>>(w[0], w[1]), split_pair<T, kExact<T>>(w[2], w[3])};
    const float total = s.coef.total;
#pragma unroll
    for (int n = 0; n < 2 * NB; n += kTiles) {
      v4f add[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) add[i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int z = kExact<T> - 1; z >= 0; --z)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) mma(add[i], cf[j][i], us[j].f[z]);
      if (n + kTiles < 2 * NB) read_cols(n + kTiles);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) st.st[n + i] = st.st[n + i] * total + add[i];
    }
  }
  last_state<MODE>(st, a, cl, u, wave);
}

template <class T, int NB>
struct RevLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  alignas(16) T k[kTok * ldn];
  alignas(16) T q[kTok * ldn];
  alignas(16) T mt[kExact<T> * kPieces * kPiece];
  alignas(16) T pt[kExact<T> * kPieces * kPiece];
  alignas(16) T y[kTok * stride_of<T>(kCols)];
  alignas(16) Coef coef;
  static constexpr int ldv = stride_of<T>(kCols);
};

// The gradient of the state that a segment ends with, and what its walk leaves.
template <bool SUMMARY, int NB>
__device__ __forceinline__ void first_gradient(State<NB, true>& st, const DeltaArgs& a, const WalkWork& w, const Unit& u) {
  const long head = static_cast<long>(a.states) * a.width;
  if (SUMMARY) st.zero();
  else if (!last_unit(a, u)) st.load(a.seg_grad + (static_cast<long>(w.unit) * a.heads + w.h) * head, a.width, a.states);
  else st.load(a.d_final == nullptr ? nullptr : a.d_final + (static_cast<long>(u.seq) * a.heads + w.h) * head, a.width, a.states);
}
template <bool SUMMARY, int NB>
__device__ __forceinline__ void last_gradient(const State<NB, true>& st, const DeltaArgs& a, const WalkWork& w, const Unit& u) {
  const long head = static_cast<long>(a.states) * a.width;
  if (SUMMARY)  // the place of the segment before
    st.save(a.seg_grad + (static_cast<long>(w.unit - 1) * a.heads + w.h) * head, a.width, a.states);
  else if (a.d_initial != nullptr && u.index == 0)
    st.save(a.d_initial + (static_cast<long>(u.seq) * a.heads + w.h) * head, a.width, a.states);
}

// The walk of the state's gradient D, from the last step to the first:
//   dU = P^T dY + 2^(c_end - c) K D,   dR = M^T dU,   dV = beta dR
//   D  = 2^c_end D + scale Q^T (2^c dY) - K^T (beta 2^c dR)
// It leaves every step's D (of the state the step ends with) and dR; SUMMARY: only
// the segment's own contribution to the gradient before it.
template <class T, int NB, bool SUMMARY>
__device__ __forceinline__ void walk_reverse(const DeltaArgs& a, RevLds<T, NB>& s) {
  typedef RevLds<T, NB> L;
  constexpr int kThreads = kWaves * 64;
  constexpr int kM = kExact<T> * kPieces * kPiece;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const WalkWork wk = walk_work(a, a.slices);
  if (wk.unit < 0) return;
  const Unit u = locate(a.seqs, wk.unit, a.seg);
  if (!u.live || (SUMMARY && u.index == 0)) return;
  const int h = wk.h, slice = wk.slice;
  const bool packed = a.seqs.offsets != nullptr;
  const int p0 = slice * kThreads / 4;
  const int col = p0 + wave * 16 + l15;
  const T* kp = seq_ptr<const T>(a.k, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* qp = seq_ptr<const T>(a.q, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* yp = seq_ptr<const T>(a.d_y, u.seq, u.row0, packed) + h * a.width + p0;
  T* vp = seq_ptr<T>(a.d_v, u.seq, u.row0, packed) + h * a.width;

  State<NB, true> st;
  st.init(a.width, p0, wave);
  first_gradient<SUMMARY>(st, a, wk, u);

  const int end = min(u.t0 + a.seg, u.len);
  const long cell0 = static_cast<long>(unit_base(a.seqs, u.seq, kTok)) * a.heads + h;  // of the sequence's first step
  Tile<T, kTok, NB * 32, kThreads> tk, tq;
  tk.init(a.k.row_stride, a.states, tid);
  tq.init(a.q.row_stride, a.states, tid);
  Flat<kM * sizeof(T), kThreads> tm, tp;
  Flat<sizeof(Coef), kThreads> tc;
  Tile<T, kTok, kCols, kThreads> ty;
  ty.init(a.d_y.row_stride, min(a.width - p0, kCols), tid);
  const unsigned v_off = col < a.width ? static_cast<unsigned>((4 * g * static_cast<int>(a.d_v.row_stride) + col) * sizeof(T)) : kOutside;
  const int v_row = static_cast<int>(a.d_v.row_stride * sizeof(T));
  const auto fetch = [&](int t) {
    const int rows = min(end - t, kTok);
    const long at = cell0 + static_cast<long>(t / kTok) * a.heads;
    tk.load(rows_rsrc(kp + t * a.k.row_stride, a.k.row_stride, rows, a.states));
    tq.load(rows_rsrc(qp + t * a.q.row_stride, a.q.row_stride, rows, a.states));
    tm.load(a.mt + at * kPieces * kPiece, tid);
    tp.load(a.pt + at * kPieces * kPiece, tid);
    tc.load(a.coef + at, tid);
    ty.load(rows_rsrc(yp + t * a.d_y.row_stride, a.d_y.row_stride, rows, min(a.width - p0, kCols)));
  };
  const int last = end > u.t0 ? u.t0 + (end - 1 - u.t0) / kTok * kTok : u.t0 - kTok;
  if (last >= u.t0) fetch(last);
  for (int t = last; t >= u.t0; t -= kTok) {
    __syncthreads();
    tk.store(s.k, L::ldn, tid);
    tq.store(s.q, L::ldn, tid);
    tm.store(s.mt, tid);
    tp.store(s.pt, tid);
    tc.store(&s.coef, tid);
    ty.store(s.y, L::ldv, tid);
    __syncthreads();
    if (t > u.t0) fetch(t - kTok);

    const long cell = cell0 + static_cast<long>(t / kTok) * a.heads;
    if (!SUMMARY) save_kept(a.d_keep + cell * (kept_bytes(a.states, a.width) / 4), a.states, a.width, col, g, st.st);
    // dU
    constexpr int kBuf = NB > 1 ? 2 : 1;
    Frag<T> kf[kBuf][4];
    Frag<T> mf[kExact<T>][kPieces];
    const auto read_rows = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[n % kBuf][i] = frag_row_result(s.k, L::ldn, 16 * i, 32 * n);
    };
    const auto read_pieces = [&](const T* p) {
#pragma unroll
      for (int z = 0; z < kExact<T>; ++z)
#pragma unroll
        for (int i = 0; i < kPieces; ++i) mf[z][i] = piece_get(p + (z * kPieces + i) * kPiece, lane);
    };
    v4f w[4], to[4], from[4], beta[4], dy[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v4f{0, 0, 0, 0};
    read_rows(0);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n + 1 < NB) {
        read_rows(n + 1);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          to[i] = rows_of(s.coef.to, i, g);
          dy[i] = tile_col(s.y, L::ldv, i, wave * 16, lane);
        }
        read_pieces(s.pt);
      }
      keep_reads_here();
      const Split<T, kExact<T>> sp = split_pair<T, kExact<T>>(st.st[2 * n], st.st[2 * n + 1]);
#pragma unroll
      for (int z = kExact<T> - 1; z >= 0; --z)
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(w[i], kf[n % kBuf][i], sp.f[z]);
    }
    const Split<T, 1> ys[2] = {split_pair<T, 1>(dy[0], dy[1]), split_pair<T, 1>(dy[2], dy[3])};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * to[i];
    mma_upper<T, kExact<T>, 1>(w, mf, ys);
    keep_reads_here();
    read_pieces(s.mt);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      from[i] = rows_of(s.coef.from, i, g);
      beta[i] = rows_of(s.coef.beta, i, g);
    }
    keep_reads_here();
    // dR
    const Split<T, kExact<T>> us[2] = {split_pair<T, kExact<T>>(w[0], w[1]), split_pair<T, kExact<T>>(w[2], w[3])};
    v4f dr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dr[i] = v4f{0, 0, 0, 0};
    mma_upper<T, kExact<T>, kExact<T>>(dr, mf, us);
    constexpr int kTiles = 2 * NB < 4 ? 2 * NB : 4;
    Frag<T> cf[2][kTiles], df[2][kTiles];
    const auto read_cols = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          df[j][i] = frag_col_result(s.q, L::ldn, 32 * j, 16 * (n + i));
          cf[j][i] = frag_col_result(s.k, L::ldn, 32 * j, 16 * (n + i));
        }
    };
    read_cols(0);
    keep_reads_here();
    if (!SUMMARY) save_kept(a.d_r + cell * (kept_bytes(kTok, a.width) / 4), kTok, a.width, col, g, dr);
    const Rsrc rv = rows_rsrc(vp + t * a.d_v.row_stride, a.d_v.row_stride, min(end - t, kTok), a.width);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dr[i] = dr[i] * beta[i];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!SUMMARY) store_elem<T>(rv, v_off + (16 * i + r) * v_row, dr[i][r]);
      dr[i] = -from[i] * dr[i];
      dy[i] = a.scale * (from[i] * dy[i]);
    }
    // D
    const Split<T, kExact<T>> rs[2] = {split_pair<T, kExact<T>>(dr[0], dr[1]), split_pair<T, kExact<T>>(dr[2], dr[3])};
    const Split<T, kExact<T>> ss[2] = {split_pair<T, kExact<T>>(dy[0], dy[1]), split_pair<T, kExact<T>>(dy[2], dy[3])};
    const float total = s.coef.total;
#pragma unroll
    for (int n = 0; n < 2 * NB; n += kTiles) {
      v4f add[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) add[i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int z = kExact<T> - 1; z >= 0; --z)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int i = 0; i < kTiles; ++i) mma(add[i], df[j][i], ss[j].f[z]);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) mma(add[i], cf[j][i], rs[j].f[z]);
        }
      if (n + kTiles < 2 * NB) read_cols(n + kTiles);
#pragma unroll
      for (int i = 0; i < kTiles; ++i) st.st[n + i] = st.st[n + i] * total + add[i];
    }
  }
  last_gradient<SUMMARY>(st, a, wk, u);
}

}  // namespace delta
