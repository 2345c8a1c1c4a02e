// Shared by the gated delta rule's kernels: the call's arguments, the matrices
// of a step, and the walk of a state over the tokens.
//
// The rule is computed in steps of 64 tokens.  With c_t the sum of log2(e) g
// over the step up to t, S the state before the step, E_ij = 2^(c_i - c_j) and
//   T_ij = beta_i E_ij k_i.k_j  (j < i),   M = (1 + T)^-1,
//   P_ij = scale E_ij q_i.k_j   (j <= i),
// the step's corrections U [64][width] solve a triangular system,
//   U     = M (beta (V - 2^c K S))
//   Y     = scale 2^c Q S + P U
//   S_end = 2^c_end S + K^T (2^(c_end - c) U)
// so everything but M is a matrix product, and the columns of V, U, Y and S do
// not meet: they are what the work is split over.
#pragma once

#include "mamba2_delta.h"
#include "ssm_common.h"

namespace delta {

using namespace ssm;

// A 64 x 64 lower triangular matrix as the left operand of a product: six
// 16 x 32 pieces (tile row i, k-step s: s = 0 for i < 2, both for i >= 2) in
// result order, lane by lane.
constexpr int kPieces = 6;
constexpr int kPiece = 512;  // elements
__host__ __device__ constexpr int piece_of(int i, int s) { return i < 2 ? i : 2 * i - 2 + s; }
// The transpose's pieces: both k-steps for i < 2, s = 1 for i >= 2.
__host__ __device__ constexpr int piece_of_t(int i, int s) { return i < 2 ? 2 * i + s : i + 2; }

// Parts that hold 16 bits of a value: for operands of results that are rounded to
// bf16 and go nowhere else (S, U and P in y, Pm and Xm in d_q and d_k).  Against
// operands that are whole this moves 0.3% of those results (d_q, d_k 0.2%) to the
// neighbouring bf16 value, and their distance from 64 bits, 1.658e-3 of the 2-norm,
// by less than 1e-8.  What reaches a state, a kept value or a gate's gradient is whole.
template <class T>
constexpr int kTwo = sizeof(T) == 2 ? 2 : 1;

// What the walks need of a step's gates.  64 floats each; behind the last token
// from = to = those of the last one, beta = 0.
struct Coef {
  float from[kTok];  // 2^c_t
  float to[kTok];    // 2^(c_end - c_t)
  float beta[kTok];
  float total;       // 2^c_end
  float pad[3];
};

struct DeltaArgs {
  mamba2_seqs seqs;
  mamba2_rows q, k, v, g, beta, y;
  const float* initial;    // [batch][heads][states][width]
  float* final_state;
  float scale;
  int heads, width, ratio, states;
  int slices;              // work-groups per head: slices of its width
  int prep_heads;          // heads of a group that one work-group makes the matrices of
  int gate_bf16;
  int seg;                 // tokens per segment (a multiple of kTok)
  int units;               // segments of the call
  float* seg_state;        // [units][heads][states][width]: the state a segment starts from
  float* seg_trans;        // [units][heads][states][states]: what a segment makes of it
  float* seg_trans_t;      // the same, transposed (the backward)
  float* seg_grad;         // [units][heads][states][width]: the gradient of the state a segment ends with
  float* m;                // [steps][heads][kPieces][kPiece]: M
  void* p;                 // [steps][heads][kTwo][kPieces][kPiece]: P
  Coef* coef;              // [steps][heads]
  // the backward's
  mamba2_rows d_y, d_q, d_k, d_v, d_g, d_beta;
  const float* d_final;
  float* d_initial;
  float* mt;               // as m: the transpose of M
  float* pt;               // as m: the transpose of P
  float* keep;             // [steps][heads], kept_bytes each: the state each step starts from
  float* d_keep;           // the same: the gradient of the state each step ends with
  float* u;                // the same for kTok rows: U
  float* d_r;              // and the gradient of beta (V - 2^c K S)
  int grad_heads;          // heads of a group that one work-group takes the gradients of
  float* grad_part;        // [steps][groups][parts][2][kTok][states]: their parts of d_q and d_k
};

// What the walks keep lies as delta_grads_kernel reads it, a kilobyte at a time: tiles of
// 16 rows by 32 columns, of which lane l has row l & 15 and columns 8 (l >> 4) .., four
// columns of all lanes and then the other four.  Bytes of 16 rows, of all of them, and of
// an element from its 16 rows' start.
__host__ __device__ inline int kept_strip(int width) { return (width + 31) / 32 * 2048; }
__host__ __device__ inline long kept_bytes(int rows, int width) { return static_cast<long>((rows + 15) / 16) * kept_strip(width); }
__device__ __forceinline__ int kept_at(int row, int col) {
  return (col >> 5) * 2048 + (col >> 2 & 1) * 1024 + (col >> 3 & 3) * 256 + row * 16 + (col & 3) * 4;
}

// An element as it was loaded, and its value.  Values are formed where they are
// used: forming one waits for its load.
template <class T>
struct Raw {
  int v;
};
template <>
struct Raw<bf16> {
  short v;
};
// What a walk over a segment is for: the results, each step's starting state and U
// (for the backward), or a summary for the segments behind: with columns of V
// the segment's own contribution to the state, and with columns of the unit
// matrix in place of the state and no V what it makes of the state before it.
enum Walked { kResults, kKept, kSummary };

// A walk's place in the call.
struct WalkWork {
  int unit, h, slice;
};
// The unit of a packed call's r-th longest sequence, none of them cut.  Called by
// whole waves; batch <= 64, a lane a sequence.
__device__ __forceinline__ int longest_unit(const DeltaArgs& a, int r) {
  const int lane = threadIdx.x & 63, batch = a.seqs.batch;
  long row0;
  int len = -1, rank = 0;
  if (lane < batch) seq_rows(a.seqs, lane, &row0, &len);
  for (int j = 0; j < batch; ++j) {
    const int other = __builtin_amdgcn_readlane(len, j);
    rank += other > len || (other == len && j < lane) ? 1 : 0;
  }
  const unsigned long long m = __ballot(lane < batch && rank == r);
  const int seq = m == 0 ? 0 : __builtin_ctzll(m);
  return r < batch ? unit_base(a.seqs, seq, a.seg) : -1;
}
// Every XCD gets all sequences of some heads, whose unequal lengths would else
// leave some XCDs with more, and the longest of them first: nine prompts of 1 to
// 2048 tokens, 32 heads of 128 x 128: with neighbouring sequences on an XCD 257 us,
// all of them 174 us, the longest first 132 us.
__device__ __forceinline__ WalkWork walk_work(const DeltaArgs& a, int slices) {
  const int per = a.heads * slices;
  const bool sorted = a.seqs.offsets != nullptr && a.seqs.batch > 1 && a.seqs.batch <= 64 && a.seg >= a.seqs.length;
  if (sorted && per % 8 == 0) {
    const int each = per / 8, k = blockIdx.x >> 3, hs = (blockIdx.x & 7) * each + k % each;
    return {longest_unit(a, k / each), hs / slices, hs % slices};
  }
  const int i = xcd_contiguous(blockIdx.x, gridDim.x);
  const int hs = i / a.units, unit = i - hs * a.units;
  return {sorted ? longest_unit(a, unit) : unit, hs / slices, hs % slices};
}

template <class T>
__device__ __forceinline__ Raw<T> load_raw_elem(Rsrc rs, unsigned off) {
  if constexpr (sizeof(T) == 2) return {static_cast<short>(__builtin_amdgcn_raw_buffer_load_b16(rs, off, 0, 0))};
  else return {static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0))};
}
__device__ __forceinline__ float value_of(Raw<bf16> r) {
  return __uint_as_float(static_cast<unsigned>(static_cast<unsigned short>(r.v)) << 16);
}
__device__ __forceinline__ float value_of(Raw<float> r) { return __int_as_float(r.v); }
template <class T>
__device__ __forceinline__ float load_elem(Rsrc rs, unsigned off) {
  return value_of(load_raw_elem<T>(rs, off));
}
template <class T>
__device__ __forceinline__ void store_elem(Rsrc rs, unsigned off, float v) {
  if constexpr (sizeof(T) == 2)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, static_cast<bf16>(v)), rs, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), rs, off, 0, 0);
}

// Lane t's gate of token t of a step with `rows` tokens; 0 behind the last.
__device__ __forceinline__ float load_gate(const mamba2_rows& r, int is_bf16, const Unit& u, bool packed, int t,
                                           int rows, int h, int heads) {
  const unsigned e = static_cast<unsigned>((threadIdx.x & 63) * static_cast<int>(r.row_stride) + h);
  if (is_bf16)
    return load_elem<bf16>(rows_rsrc(seq_ptr<const bf16>(r, u.seq, u.row0, packed) + t * r.row_stride, r.row_stride,
                                     rows, heads), e * 2);
  return load_elem<float>(rows_rsrc(seq_ptr<const float>(r, u.seq, u.row0, packed) + t * r.row_stride, r.row_stride,
                                    rows, heads), e * 4);
}

// log2 of a token's decay.  One that underflows any fp32 is held at 2^-1100, so
// that later differences keep their bits; a NaN stays one.
__device__ __forceinline__ double gate_log(float g) {
  const double l = static_cast<double>(g) * 1.4426950408889634074;
  return l < -1100.0 ? -1100.0 : l;
}

// Eight elements of a piece as its lane holds them.
template <class T>
__device__ __forceinline__ Frag<T> piece_get(const T* p, int lane) {
  if constexpr (sizeof(T) == 2) {
    return {*reinterpret_cast<const v8bf*>(p + lane * 8)};
  } else {
    const v4f* r = reinterpret_cast<const v4f*>(p + lane * 8);
    return {{r[0], r[1]}};
  }
}
template <class T>
__device__ __forceinline__ void piece_put(T* p, int lane, const Frag<T>& f) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<v8bf*>(p + lane * 8) = f.v;
  } else {
    v4f* r = reinterpret_cast<v4f*>(p + lane * 8);
    r[0] = f.v[0];
    r[1] = f.v[1];
  }
}

// acc += a b for operands in parts, small products first; what is dropped is
// below 2^-24 (three parts each), 2^-16 (two) of the product.
template <class T, int A, int B>
__device__ __forceinline__ void mma_parts(v4f& acc, const Frag<T> (&a)[A], const Frag<T> (&b)[B]) {
  constexpr int kMost = A > B ? A : B;
#pragma unroll
  for (int n = kMost - 1; n >= 0; --n)
#pragma unroll
    for (int i = 0; i <= n; ++i)
      if (i < A && n - i < B) mma(acc, a[i], b[n - i]);
}

// acc += A b for a 64 x 64 lower triangular A in pieces and a b of 64 rows, in
// parts, small products first; neighbouring products are on different tiles, as
// one waits for the last one on its own.  TRANSPOSED: acc += (A b)^T.
template <class T, int A, int B, bool TRANSPOSED = false>
__device__ __forceinline__ void mma_lower(v4f (&acc)[4], const Frag<T> (&a)[A][kPieces], const Split<T, B> (&b)[2]) {
  constexpr int kMost = A > B ? A : B;
#pragma unroll
  for (int n = kMost - 1; n >= 0; --n)
#pragma unroll
    for (int z = 0; z <= n; ++z)
      if (z < A && n - z < B) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 2 * s; i < 4; ++i) {
            if (TRANSPOSED) mma(acc[i], b[s].f[n - z], a[z][piece_of(i, s)]);
            else mma(acc[i], a[z][piece_of(i, s)], b[s].f[n - z]);
          }
      }
}
// The same for an upper triangular A (a transpose's pieces).
template <class T, int A, int B>
__device__ __forceinline__ void mma_upper(v4f (&acc)[4], const Frag<T> (&a)[A][kPieces], const Split<T, B> (&b)[2]) {
  constexpr int kMost = A > B ? A : B;
#pragma unroll
  for (int n = kMost - 1; n >= 0; --n)
#pragma unroll
    for (int z = 0; z <= n; ++z)
      if (z < A && n - z < B) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int i = 0; i < 2 * s + 2; ++i) mma(acc[i], a[z][piece_of_t(i, s)], b[s].f[n - z]);
      }
}

// Reads of LDS stay on their side of this; everything else may be moved over it.
__device__ __forceinline__ void keep_reads_here() { __builtin_amdgcn_sched_barrier(0x7f); }
// Nothing is moved over this.
__device__ __forceinline__ void keep_all_here() { __builtin_amdgcn_sched_barrier(0); }

// Four values of rows 4 g .. of tile i, of an array by token.
__device__ __forceinline__ v4f rows_of(const float* p, int i, int g) {
  return *reinterpret_cast<const v4f*>(p + 16 * i + 4 * g);
}

// Two stacked results as an operand over their rows.
template <class T, int TERMS>
__device__ __forceinline__ Split<T, TERMS> split_pair(v4f a, v4f b) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split_of<T, TERMS>(v);
}

// Host side, in delta.hip.  check_keys, check_values, check_gates: a tensor of
// the call, whose unused strides they replace.
int check_delta(const mamba2_seqs& q, const mamba2_delta_dims& d);
int check_keys(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d);
int check_values(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d);
int check_gates(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d);
int segment_tokens(const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd);
size_t segment_bytes(const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd);
void set_dims(DeltaArgs* a, const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd);
void set_segments(DeltaArgs* a, char* at, bool bwd);  // the segments' part of the workspace
// The states that the segments start from, where there are several; for the
// backward also their transitions, with which carry_gradients finishes the gradients.
int start_segments(const DeltaArgs& a, int type, hipStream_t s);
int carry_gradients(const DeltaArgs& a, hipStream_t s);
unsigned walk_blocks(const DeltaArgs& a);

}  // namespace delta
