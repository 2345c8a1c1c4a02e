// The matrices of the gated delta rule's steps: M = (1 + T)^-1 and P, for one
// step of one head, as the left operands that the walks read.
#pragma once

#include "delta_common.h"

namespace delta {

constexpr int kPrepWaves = 4;
// Work-groups of the matrices' kernels that a CU's LDS holds: of 35 KB each, fp32 with
// over 64 states 68.
__host__ __device__ constexpr int prep_per_cu(size_t elem, int states) { return elem == 2 || states <= 64 ? 4 : 2; }
constexpr int kSq = kTok + 4;  // row stride of a 64 x 64 fp32 matrix in LDS

template <class T, int NB>
struct PrepLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  union {
    struct {
      T k[kTok * ldn];
      T q[kTok * ldn];
    } in;
    struct {
      float t[kTok * kSq];
      float m[kTok * kSq];
    } sq;
  };
  alignas(16) float hi[kTok], lo[kTok], beta[kTok];  // c_t in two floats
};

// acc += A B over 16: A row-major at a, B in the order of a result: register r
// holds row 4 g + r.
__device__ __forceinline__ void mul16(v4f& acc, const float* a, const v4f& b, int l15, int g) {
  const v4f x = *reinterpret_cast<const v4f*>(a + l15 * kSq + 4 * g);
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], b[r], acc, 0, 0, 0);
}
__device__ __forceinline__ v4f block_get(const float* a, int l15, int g) {
  v4f v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = a[(4 * g + r) * kSq + l15];
  return v;
}
__device__ __forceinline__ void block_put(float* a, v4f v, int l15, int g) {
#pragma unroll
  for (int r = 0; r < 4; ++r) a[(4 * g + r) * kSq + l15] = v[r];
}

// The inverse of 1 + t (t strictly lower, 64 x 64) into m, by all four waves:
// each inverts a 16 x 16 block of the diagonal row by row, a lane a column;
// then the blocks below the diagonal by halves,
//   [[A, 0], [B, C]]^-1 = [[A^-1, 0], [-C^-1 B A^-1, C^-1]].
// fp32 products throughout: the inverse's entries multiply every correction.
__device__ __forceinline__ void invert(float* m, const float* t, int wave, int lane) {
  const int l15 = lane & 15, g = lane >> 4;
  const auto at = [](int i, int j) { return 16 * i * kSq + 16 * j; };
  {
    const float* d = t + at(wave, wave);
    float col[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == l15 ? 1.0f : 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-d[i * kSq + j], col[j], s);
      col[i] = s;
    }
    if (g == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m[at(wave, wave) + i * kSq + l15] = col[i];
    }
    if (wave < 2) block_put(m + at(2 * wave, 2 * wave + 1), v4f{0, 0, 0, 0}, l15, g);
  }
  __syncthreads();
  if (wave < 2) {
    const int i = 2 * wave;
    v4f x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    mul16(x, t + at(i + 1, i), block_get(m + at(i, i), l15, g), l15, g);
    mul16(y, m + at(i + 1, i + 1), x, l15, g);
    block_put(m + at(i + 1, i), -y, l15, g);
  }
  __syncthreads();
  const int rb = wave >> 1, cb = wave & 1;  // a block of the lower left quarter each
  v4f y = {0, 0, 0, 0};
  for (int r = 0; r <= rb; ++r) {
    v4f x = {0, 0, 0, 0};
    for (int j = cb; j < 2; ++j) mul16(x, t + at(2 + r, j), block_get(m + at(j, cb), l15, g), l15, g);
    mul16(y, m + at(2 + rb, 2 + r), x, l15, g);
  }
  block_put(m + at(2 + rb, cb), -y, l15, g);
  __syncthreads();
}

// Writes the pieces of a 64 x 64 matrix (transposed: of its transpose) in fp32, a
// wave's share of them.
template <bool TRANSPOSED>
__device__ __forceinline__ void put_pieces(float* out, const float* m, int wave, int lane) {
  const int l15 = lane & 15, g = lane >> 4;
  for (int n = wave; n < kPieces; n += kPrepWaves) {
    int i, s;  // the piece's tile row and k-step
    if (TRANSPOSED) {
      i = n < 4 ? n >> 1 : n - 2;
      s = n < 4 ? n & 1 : 1;
    } else {
      i = n < 2 ? n : (n + 2) >> 1;
      s = n < 2 ? 0 : n & 1;
    }
    Frag<float> f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int row = 16 * i + l15, k = 32 * s + (j >> 2) * 16 + 4 * g + (j & 3);
      f.v[j >> 2][j & 3] = TRANSPOSED ? m[k * kSq + row] : m[row * kSq + k];
    }
    piece_put(out + n * kPiece, lane, f);
  }
}

// P's pieces: two parts of T, as the forward multiplies them; the backward's in fp32.
template <class T, bool BWD>
struct PiecesOf {
  typedef T type;
};
template <class T>
struct PiecesOf<T, true> {
  typedef float type;
};

// Work-groups per step: each has up to prep_heads heads of one group.
__host__ __device__ inline int prep_parts(const DeltaArgs& a) { return (a.ratio + a.prep_heads - 1) / a.prep_heads; }
inline unsigned prep_blocks(const DeltaArgs& a, unsigned cells) {
  return cells / a.heads * (a.heads / a.ratio) * prep_parts(a);
}
struct PrepWork {
  int step, first, heads;
};
__device__ __forceinline__ PrepWork prep_work(const DeltaArgs& a) {
  const int work = xcd_contiguous(blockIdx.x, gridDim.x), parts = prep_parts(a);
  const int per = a.heads / a.ratio * parts, step = work / per, at = work % per;
  const int part = at % parts, skip = part * a.prep_heads;
  return {step, at / parts * a.ratio + skip, min(a.prep_heads, a.ratio - skip)};
}

// One step of `heads` heads of a group, one after the other, the products of their
// shared q and k formed once: writes P's pieces (BWD: those of its transpose) and
// the gates, and calls done(cell) with M in s.sq.m.
//
// A product's result that has a matrix's row in a lane and 4 g .. of its columns is
// a piece of that matrix as it lies in the registers: so K Q^T gives P's pieces and
// Q K^T those of P^T, without a way through LDS.
template <class T, int NB, bool BWD, class Done>
__device__ __forceinline__ void make_steps(PrepLds<T, NB>& s, const DeltaArgs& a, const Unit& u, int step, int first, int heads,
                                           typename PiecesOf<T, BWD>::type* pieces, Done done) {
  typedef PrepLds<T, NB> L;
  typedef typename PiecesOf<T, BWD>::type P;
  constexpr int kThreads = kPrepWaves * 64;
  constexpr int kParts = kTwo<P>;
  const bool packed = a.seqs.offsets != nullptr;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int rows = min(u.len - u.t0, kTok);
  const int j = first / a.ratio * a.states;
  float g_raw = 0.0f, beta_raw = 0.0f;
  const auto fetch_gates = [&](int h) {
    if (wave != kPrepWaves - 1) return;
    g_raw = load_gate(a.g, a.gate_bf16, u, packed, u.t0, rows, h, a.heads);
    beta_raw = load_gate(a.beta, a.gate_bf16, u, packed, u.t0, rows, h, a.heads);
  };
  fetch_gates(first);
  // a wave's sixteen rows of K K^T up to the diagonal, transposed: row l15, columns 4 g ..
  v4f kk[4], qk[4];
  {
    Tile<T, kTok, NB * 32, kThreads> tk, tq;
    tk.init(a.k.row_stride, a.states, tid);
    tq.init(a.q.row_stride, a.states, tid);
    tk.load(rows_rsrc(seq_ptr<const T>(a.k, u.seq, u.row0, packed) + u.t0 * a.k.row_stride + j, a.k.row_stride, rows,
                      a.states));
    tq.load(rows_rsrc(seq_ptr<const T>(a.q, u.seq, u.row0, packed) + u.t0 * a.q.row_stride + j, a.q.row_stride, rows,
                      a.states));
    tk.store(s.in.k, L::ldn, tid);
    tq.store(s.in.q, L::ldn, tid);
    __syncthreads();
    Frag<T> kf[NB], of[NB];  // of: this wave's rows of Q; BWD: of K, for P's columns
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      kf[n] = frag_row(s.in.k, L::ldn, wave * 16, n * 32);
      of[n] = BWD ? kf[n] : frag_row(s.in.q, L::ldn, wave * 16, n * 32);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      kk[c] = qk[c] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (c <= wave) {
          const Frag<T> b = frag_row(s.in.k, L::ldn, c * 16, n * 32);
          mma(kk[c], b, kf[n]);
          if (!BWD) mma(qk[c], b, of[n]);
        }
        if (BWD && c >= wave) mma(qk[c], frag_row(s.in.q, L::ldn, c * 16, n * 32), of[n]);
      }
    }
  }
  const int mine = wave * 16 + l15;
  for (int h = first; h < first + heads; ++h) {
    const long cell = static_cast<long>(step) * a.heads + h;
    __syncthreads();  // k and q, or the last head's matrices, give way to T and M
    if (wave == kPrepWaves - 1) {
      const double c = scan64(gate_log(g_raw));
      const long bits = __builtin_bit_cast(long, c);
      const double end = __builtin_bit_cast(
          double, (static_cast<long>(__builtin_amdgcn_readlane(static_cast<int>(bits >> 32), 63)) << 32) |
                      static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(bits), 63)));
      s.hi[lane] = static_cast<float>(c);
      s.lo[lane] = static_cast<float>(c - static_cast<float>(c));
      s.beta[lane] = beta_raw;
      Coef& coef = a.coef[cell];
      coef.from[lane] = exp2_of(c);
      coef.to[lane] = exp2_of(end - c);
      coef.beta[lane] = beta_raw;
      if (lane == 0) coef.total = exp2_of(end);
      fetch_gates(h + 1 < first + heads ? h + 1 : h);
    }
    __syncthreads();
    const float ch = s.hi[mine], cl = s.lo[mine], beta = s.beta[mine];
    v4f pq[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const v4f hi = rows_of(s.hi, c, g), lo = rows_of(s.lo, c, g);
      v4f t;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int other = c * 16 + 4 * g + r;
        const float d = (ch - hi[r]) + (cl - lo[r]);  // c_mine - c_other
        const float e = exp2_of(BWD && c > wave ? -d : d);
        t[r] = other < mine ? beta * (e * kk[c][r]) : 0.0f;
        if (BWD) {
          const float w = c == wave ? exp2_of(-d) : e;
          pq[c][r] = other >= mine ? a.scale * (w * qk[c][r]) : 0.0f;
        } else {
          pq[c][r] = other <= mine ? a.scale * (e * qk[c][r]) : 0.0f;
        }
      }
      if (c <= wave) *reinterpret_cast<v4f*>(&s.sq.t[mine * kSq + c * 16 + 4 * g]) = t;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (BWD ? k < wave / 2 : k > wave / 2) continue;
      const Split<P, kParts> f = split_pair<P, kParts>(pq[2 * k], pq[2 * k + 1]);
      const int n = BWD ? piece_of_t(wave, k) : piece_of(wave, k);
#pragma unroll
      for (int z = 0; z < kParts; ++z) piece_put(pieces + ((cell * kParts + z) * kPieces + n) * kPiece, lane, f.f[z]);
    }
    __syncthreads();
    invert(s.sq.m, s.sq.t, wave, lane);
    done(cell);
  }
}

}  // namespace delta
