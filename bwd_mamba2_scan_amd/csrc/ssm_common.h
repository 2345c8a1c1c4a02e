// Shared by the selective scan's kernels: matrix fragments of both element
// types, LDS tiles, the decays of a step, and the call's arguments.
//
// The scan is computed in steps of 64 tokens.  With l_t = d_t A log2(e) and c_t the sum of
// l over the step up to t, and S the state before the step,
//   y_t   = 2^c_t S^T C_t + sum_{s <= t} (C_t . B_s) 2^(c_t - c_s) d_s x_s
//   S_end = 2^c_end S + sum_s 2^(c_end - c_s) d_s B_s x_s^T
// so everything but the elementwise decays is a matrix product.
#pragma once

#include "layer_common.h"

namespace ssm {

using namespace layer;

constexpr int kTok = 64;        // tokens per step of a kernel: one lane each in the decay scan
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxDim = 128;    // largest width and number of states

struct SsmArgs {
  mamba2_seqs q;
  mamba2_rows x, dt, B, C, y;
  const float* A;
  const float* D;
  const float* bias;
  const float* initial;    // [batch][heads][states][width]
  float* final_state;
  int heads, width, ratio, states;
  int slices;              // work-groups per head: slices of its width
  int softplus, dt_bf16;
  int seg;                 // tokens per segment (a multiple of kTok)
  int units;
  int fold;                // a segment adds up the states before it itself; no carry pass
};

// A 16 x 32 (or 32 x 16) matrix operand: lane l holds row (column) l & 15 and
// eight of the 32 k positions.  Which position of the sum sits in which slot
// does not matter as long as both operands agree, so there are two orders:
//   natural: slot j of lane group g = l >> 4 is k = 8 g + j
//   result:  slot j is k = 4 g + j (j < 4) and 16 + 4 g + j - 4: the order in
//            which two stacked 16 x 16 results hold their rows, so a result
//            becomes an operand without leaving its lane.
template <class T>
struct Frag;
template <>
struct Frag<bf16> {
  v8bf v;
};
template <>
struct Frag<float> {
  v4f v[2];
};

// acc[m][n] += sum_k a[m][k] b[k][n]; lane l gets column l & 15, rows 4 g + i.
// bf16: one matrix instruction over the 32 k positions.  fp32: eight over 4.
__device__ __forceinline__ void mma(v4f& acc, const Frag<bf16>& a, const Frag<bf16>& b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(v4f& acc, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h][j], b.v[h][j], acc, 0, 0, 0);
}

typedef short v4s __attribute__((ext_vector_type(4)));

// LDS row stride of `n` columns: 16 bytes of padding spread neighbouring rows
// over the banks and keep them 16-byte aligned.
template <class T>
constexpr int stride_of(int n) {
  return n + 16 / static_cast<int>(sizeof(T));
}

// Operand whose row (column) index is an LDS row, k along the row: natural order.
__device__ __forceinline__ Frag<bf16> frag_row(const bf16* p, int ld, int row, int k0,
                                               int l = threadIdx.x & 63) {
  return {*reinterpret_cast<const v8bf*>(p + (row + (l & 15)) * ld + k0 + 8 * (l >> 4))};
}
__device__ __forceinline__ Frag<float> frag_row(const float* p, int ld, int row, int k0,
                                               int l = threadIdx.x & 63) {
  const v4f* r = reinterpret_cast<const v4f*>(p + (row + (l & 15)) * ld + k0 + 8 * (l >> 4));
  return {{r[0], r[1]}};
}
// The same in result order.
__device__ __forceinline__ Frag<bf16> frag_row_result(const bf16* p, int ld, int row, int k0,
                                               int l = threadIdx.x & 63) {
  const bf16* r = p + (row + (l & 15)) * ld + k0 + 4 * (l >> 4);
  const v4bf a = *reinterpret_cast<const v4bf*>(r);
  const v4bf b = *reinterpret_cast<const v4bf*>(r + 16);
  return {__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7)};
}
__device__ __forceinline__ Frag<float> frag_row_result(const float* p, int ld, int row, int k0,
                                               int l = threadIdx.x & 63) {
  const float* r = p + (row + (l & 15)) * ld + k0 + 4 * (l >> 4);
  return {{*reinterpret_cast<const v4f*>(r), *reinterpret_cast<const v4f*>(r + 16)}};
}
// Operand whose k runs over LDS rows and whose row (column) index is an LDS
// column: natural order.  bf16: the transposing LDS read hands lane i of 16
// lanes column i of the 4 x 16 block whose rows the lanes address in fours.
__device__ __forceinline__ v4s read_tr(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(const_cast<bf16*>(p)));
}
__device__ __forceinline__ Frag<bf16> frag_join(v4s a, v4s b) {
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return {__builtin_bit_cast(v8bf, v)};
}
__device__ __forceinline__ Frag<bf16> frag_col(const bf16* p, int ld, int k0, int col,
                                               int l = threadIdx.x & 63) {
  const bf16* r = p + (k0 + 8 * (l >> 4) + ((l & 15) >> 2)) * ld + col + 4 * (l & 3);
  return frag_join(read_tr(r), read_tr(r + 4 * ld));
}
__device__ __forceinline__ Frag<float> frag_col(const float* p, int ld, int k0, int col,
                                               int l = threadIdx.x & 63) {
  const float* r = p + (k0 + 8 * (l >> 4)) * ld + col + (l & 15);
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j >> 2][j & 3] = r[j * ld];
  return f;
}
// The same in result order.
__device__ __forceinline__ Frag<bf16> frag_col_result(const bf16* p, int ld, int k0, int col,
                                               int l = threadIdx.x & 63) {
  const bf16* r = p + (k0 + 4 * (l >> 4) + ((l & 15) >> 2)) * ld + col + 4 * (l & 3);
  return frag_join(read_tr(r), read_tr(r + 16 * ld));
}
__device__ __forceinline__ Frag<float> frag_col_result(const float* p, int ld, int k0, int col,
                                               int l = threadIdx.x & 63) {
  const float* r = p + (k0 + 4 * (l >> 4)) * ld + col + (l & 15);
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j >> 2][j & 3] = r[((j >> 2) * 16 + (j & 3)) * ld];
  return f;
}

// Eight fp32 values as an operand in TERMS parts that add up to it: with bf16
// each part holds 8 more bits (3 parts: all 24), fp32 needs one.
template <class T, int TERMS>
struct Split {
  Frag<T> f[TERMS];
};
// Two floats rounded to bf16 in one word, and the floats of such a word.
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_convertvector((v2f){a, b}, v2bf));
}
__device__ __forceinline__ float low_of(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(unsigned w) { return __uint_as_float(w & 0xffff0000u); }

template <class T, int TERMS>
__device__ __forceinline__ Split<T, TERMS> split_of(const float (&v)[8]) {
  Split<T, TERMS> s;
  if constexpr (sizeof(T) == 4) {
    s.f[0] = {{{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}}};
  } else {
    v4u w[TERMS];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = v[2 * j], b = v[2 * j + 1];
#pragma unroll
      for (int t = 0; t < TERMS; ++t) {
        const unsigned p = pack_bf16(a, b);
        w[t][j] = p;
        a -= low_of(p);
        b -= high_of(p);
      }
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t) s.f[t].v = __builtin_bit_cast(v8bf, w[t]);
  }
  return s;
}
template <class T>
__device__ __forceinline__ Frag<T> frag_of(const float (&v)[8]) {
  return split_of<T, 1>(v).f[0];
}
__device__ __forceinline__ float frag_get(const Frag<bf16>& f, int j) { return static_cast<float>(f.v[j]); }
__device__ __forceinline__ float frag_get(const Frag<float>& f, int j) { return f.v[j >> 2][j & 3]; }
// The bf16 matrix instruction's sums are a little low: what it drops of each
// product leaves a result below the exact sum more often than above it.  Sums
// over thousands of tokens (d_A, d_dt_bias) show that where their terms have a
// mean, 2e-6 of d_A at 4 x 4096 tokens.  So every other row of such a product
// is computed with the opposite sign, and the rows' errors cancel in the sum.
__device__ __forceinline__ Frag<float> flip_odd(const Frag<float>& f, int) { return f; }
__device__ __forceinline__ Frag<bf16> flip_odd(const Frag<bf16>& f, int row) {
  const unsigned m = (row & 1) != 0 ? 0x80008000u : 0u;
  return {__builtin_bit_cast(v8bf, __builtin_bit_cast(v4u, f.v) ^ v4u{m, m, m, m})};
}
template <class T>
constexpr bool kFlips = sizeof(T) == 2;
template <class T>
constexpr int kExact = sizeof(T) == 2 ? 3 : 1;  // parts that hold an fp32 value whole

// ------------------------------------------------------------------- tiles
// Tiles are moved through buffer resources that end with the last valid row:
// loads behind it give zero and stores are dropped, so a step's ragged end
// needs no branches.  A column outside the tensor gets an offset outside any
// resource.  Offsets within a step's 64 rows fit 31 bits (check_vec_rows).
typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
constexpr unsigned kOutside = 0x80000000u;

__device__ __forceinline__ Rsrc make_rsrc(const void* p, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}
// `rows` rows of `width` elements, `stride` elements apart.
template <class T>
__device__ __forceinline__ Rsrc rows_rsrc(const T* p, long stride, int rows, int width) {
  return make_rsrc(p, rows > 0 ? static_cast<unsigned>(((rows - 1) * stride + width) * sizeof(T)) : 0u);
}

// R rows (tokens) by C columns of a token-major tensor, moved by THREADS
// threads in 16-byte vectors; `cols` of the columns exist.
template <class T, int R, int C, int THREADS>
struct Tile {
  static constexpr int kVec = Vec<T>::n;
  static constexpr int kPerRow = C / kVec;
  static constexpr int kN = (R * kPerRow + THREADS - 1) / THREADS;
  v4i v[kN];
  unsigned off[kN];

  __device__ __forceinline__ void init(long stride, int cols, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = tid + i * THREADS, r = e / kPerRow, c = e % kPerRow * kVec;
      off[i] = (c < cols && r < R) ? static_cast<unsigned>((r * static_cast<int>(stride) + c) * sizeof(T)) : kOutside;
    }
  }
  __device__ __forceinline__ void load(Rsrc rs) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, off[i], 0, 0);
  }
  __device__ __forceinline__ void store(T* lds, int ld, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = tid + i * THREADS, r = e / kPerRow, c = e % kPerRow * kVec;
      if (R * kPerRow % THREADS == 0 || r < R) *reinterpret_cast<v4i*>(lds + r * ld + c) = v[i];
    }
  }
};

// Four consecutive elements of type T.
template <class T>
struct Quad;
template <>
struct Quad<bf16> {
  typedef v4bf type;
  static __device__ __forceinline__ void store(Rsrc rs, unsigned off, v4f v) {
    const v2u r = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2i, r), rs, off, 0, 0);
  }
};
template <>
struct Quad<float> {
  typedef v4f type;
  static __device__ __forceinline__ void store(Rsrc rs, unsigned off, v4f v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, v), rs, off, 0, 0);
  }
};
template <class T>
__device__ __forceinline__ v4f quad_get(const T* p) {
  const typename Quad<T>::type r = *reinterpret_cast<const typename Quad<T>::type*>(p);
  return v4f{static_cast<float>(r[0]), static_cast<float>(r[1]), static_cast<float>(r[2]), static_cast<float>(r[3])};
}
__device__ __forceinline__ void quad_put(float* p, v4f v) { *reinterpret_cast<v4f*>(p) = v; }
__device__ __forceinline__ void quad_put(bf16* p, v4f v) {
  *reinterpret_cast<v2u*>(p) = v2u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// The parts of split_of, one `plane` elements behind the other.
template <int TERMS>
__device__ __forceinline__ void quad_put_parts(bf16* p, int plane, v4f v) {
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    const unsigned a = pack_bf16(v[0], v[1]), b = pack_bf16(v[2], v[3]);
    *reinterpret_cast<v2u*>(p + t * plane) = v2u{a, b};
    v = v4f{v[0] - low_of(a), v[1] - high_of(a), v[2] - low_of(b), v[3] - high_of(b)};
  }
}
template <int TERMS>
__device__ __forceinline__ void quad_put_parts(float* p, int, v4f v) {
  static_assert(TERMS == 1, "fp32 is whole in one part");
  quad_put(p, v);
}

// ------------------------------------------------------------------ decays
// v + the lane's DPP neighbour, where the DPP control reaches one (else v).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const long b = __builtin_bit_cast(long, v);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, (static_cast<long>(hi) << 32) | static_cast<unsigned>(lo));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  const int n = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(float, n);
}
// The sum over each 16 lanes, in all of them.
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0x128, 0xf>(v);  // row_ror:8
  v = dpp_add<0x124, 0xf>(v);  // row_ror:4
  v = dpp_add<0x122, 0xf>(v);  // row_ror:2
  return dpp_add<0x121, 0xf>(v);
}
// A value of this lane's 16 and of the three other 16s.  permlane16_swap
// hands back (rows 0, 0, 2, 2) and (rows 1, 1, 3, 3) of a register swapped
// with itself, permlane32_swap the lower and the upper half.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair swap16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Pair swap32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}
// The sum over the four lanes with the same l & 15.
__device__ __forceinline__ float sum_groups(float v) {
  const Pair p = swap16(v);
  const Pair q = swap32(p.a + p.b);
  return q.a + q.b;
}
__device__ __forceinline__ float sum64(float v) { return sum_groups(sum16(v)); }
// The wave's number, known to be the same in all its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
// Inclusive prefix sum over the 64 lanes.
template <class F>
__device__ __forceinline__ F scan64(F v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr:1
  v = dpp_add<0x112, 0xf>(v);  // row_shr:2
  v = dpp_add<0x114, 0xf>(v);  // row_shr:4
  v = dpp_add<0x118, 0xf>(v);  // row_shr:8
  v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }

// 2^v for a 64-bit v: the whole part is an exact scaling, so the result has
// fp32's full precision however large |v| is.
__device__ __forceinline__ float exp2_of(double v) {
  const double r = rint(v);
  return exp2_of(static_cast<float>(v - r)) * exp2_of(static_cast<float>(r));
}

// The raw step sizes of a step's tokens; token behind the last give zero.
__device__ __forceinline__ Rsrc step_rsrc(const SsmArgs& a, const Unit& u, bool packed, int t, int rows) {
  if (a.dt_bf16) return rows_rsrc(seq_ptr<const bf16>(a.dt, u.seq, u.row0, packed) + t * a.dt.row_stride,
                                  a.dt.row_stride, rows, a.heads);
  return rows_rsrc(seq_ptr<const float>(a.dt, u.seq, u.row0, packed) + t * a.dt.row_stride, a.dt.row_stride, rows,
                   a.heads);
}
__device__ __forceinline__ float load_raw(const SsmArgs& a, Rsrc rs, int h) {
  const int e = static_cast<int>(threadIdx.x & 63) * static_cast<int>(a.dt.row_stride) + h;
  if (a.dt_bf16)
    return __builtin_bit_cast(float, static_cast<unsigned>(
               static_cast<unsigned short>(__builtin_amdgcn_raw_buffer_load_b16(rs, e * 2, 0, 0))) << 16);
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, e * 4, 0, 0));
}
// softplus(v) = log(1 + e^v) to fp32's last bits.  e^v: the product with
// log2(e) in two terms.  log(1 + t): log(w) t / (w - 1) with w = 1 + t rounded
// cancels that rounding (Kahan); below 2^-6, where w - 1 keeps few bits of t,
// the series.
__device__ __forceinline__ float step_of(const SsmArgs& a, float raw, float bias) {
  const float v = raw + bias;
  if (!a.softplus) return v;
  const float p = v * kLog2e;
  const float rest = fmaf(v, 1.925963033500e-8f, fmaf(v, kLog2e, -p));  // log2(e) - kLog2e, and p's rounding
  float t = exp2_of(p);
  t = fmaf(t, 0.69314718056f * rest, t);
  const float w = 1.0f + t;
  const float kahan = __builtin_amdgcn_logf(w) * 0.69314718056f * (t * __builtin_amdgcn_rcpf(w - 1.0f));
  const float series = t * fmaf(t, fmaf(t, fmaf(t, -0.25f, 0.33333333f), -0.5f), 1.0f);
  const float s = t < 0.015625f ? series : kahan;
  return v > 20.0f ? v : v < -80.0f ? expf(v) : s;
}

// The decays of a step of kTok tokens.  Sums of log2 decays are formed in 64
// bits and kept as two floats: a difference of two of them is needed to
// about 1e-7, and they reach into the thousands.
template <bool LEFT>
struct DecaysOf {
  float hi[kTok], lo[kTok];   // c_t
  float d[kTok];              // d_t; 0 behind the last token
  float from[kTok];           // 2^c_t
  float to[kTok];             // 2^(c_end - c_t) d_t
  float left[LEFT ? kTok : 4];  // 2^(c_end - c_t), where the backward needs it
  float total;                // 2^c_end
  double end;                 // c_end
};
typedef DecaysOf<false> Decays;

// log2(e) A, finite, so that a step of 0 decays nothing even where A is infinite;
// a NaN stays one.
__device__ __forceinline__ double decay_rate(float A) {
  const double r = static_cast<double>(A) * 1.4426950408889634074;
  return A == A ? fmin(fmax(r, -1e300), 1e300) : r;
}
// log2 of a token's decay.  One that underflows any fp32 (2^-1100) is held there,
// so that later differences keep their bits; a NaN stays one.
__device__ __forceinline__ double log_decay(float d, double rate) {
  const double l = static_cast<double>(d) * rate;
  return l < -1100.0 ? -1100.0 : l;
}

// One wave; lane t has token t.
template <bool LEFT>
__device__ __forceinline__ void make_decays(DecaysOf<LEFT>& dc, float d, double rate) {
  const int t = threadIdx.x & 63;
  const double c = scan64(log_decay(d, rate));
  const long cbits = __builtin_bit_cast(long, c);
  const double end = __builtin_bit_cast(
      double, (static_cast<long>(__builtin_amdgcn_readlane(static_cast<int>(cbits >> 32), 63)) << 32) |
                  static_cast<unsigned>(__builtin_amdgcn_readlane(static_cast<int>(cbits), 63)));
  const float hi = static_cast<float>(c);
  dc.hi[t] = hi;
  dc.lo[t] = static_cast<float>(c - hi);
  dc.d[t] = d;
  dc.from[t] = exp2_of(c);
  const float left = exp2_of(end - c);
  if (LEFT) dc.left[LEFT ? t : 0] = left;
  dc.to[t] = left * d;
  if (t == 63) {
    dc.total = exp2_of(c);
    dc.end = c;
  }
}

// Dispatch is round-robin over the 8 XCDs: gives each XCD a contiguous range
// of the work, so that the heads that share B and C share an L2.
__device__ __forceinline__ int xcd_contiguous(int block, int total) {
  const int xcd = block & 7, k = block >> 3, q = total >> 3, r = total & 7;
  return xcd * q + min(xcd, r) + k;
}

// ------------------------------------------------------------------- walk
// One pass of a state over the tokens: forward,
//   S <- 2^c_end S + sum_s 2^(c_end - c_s) d_s B_s x_s^T      per step,
// or in reverse, for the gradient G of the state,
//   G <- 2^c_end G + sum_t 2^c_t C_t d_y_t^T.
struct Walk {
  mamba2_rows v, m;        // x and B, or d_y and C
  const float* first;      // the state the pass starts from, per sequence (NULL: 0)
  float* last;             // where it ends, per sequence (NULL: not kept)
  float* seg_state;        // [units][heads][states][width]: the state each segment starts from
  float* seg_decay;        // [units][heads]: each segment's decay
  float* keep;             // the state each step starts from; see kept_at
  int rev;
};

// A wave's 16 columns of a state [states][width], as fp32 results.  COLS true:
// lane l has column l & 15, rows 4 g + i (the order an operand needs); false:
// lane l has row l & 15 of each 16, columns 4 g + i (16-byte accesses).
template <int NB, bool COLS>
struct State {
  v4f st[2 * NB];
  unsigned off;    // bytes, of the lane's first element; kOutside for a column that does not exist

  __device__ __forceinline__ void init(int width, int col0, int wave) {
    const int l = threadIdx.x & 63, l15 = l & 15, g = l >> 4;
    const int c = col0 + wave * 16 + (COLS ? l15 : 4 * g), r = COLS ? 4 * g : l15;
    off = c < width ? static_cast<unsigned>((r * width + c) * 4) : kOutside;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) st[n] = v4f{0, 0, 0, 0};
  }
  static __device__ __forceinline__ Rsrc rsrc(const float* p, int width, int states) {
    return make_rsrc(p, static_cast<unsigned>(states * width * 4));
  }
  __device__ __forceinline__ void load(const float* p, int width, int states) {
    if (p == nullptr) {
      zero();
      return;
    }
    const Rsrc rs = rsrc(p, width, states);
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
      const unsigned o = off + n * 64 * width;
      if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st[n][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, o + i * 4 * width, 0, 0));
      } else {
        st[n] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0));
      }
    }
  }
  __device__ __forceinline__ void save(float* p, int width, int states) const {
    const Rsrc rs = rsrc(p, width, states);
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
      const unsigned o = off + n * 64 * width;
      if constexpr (COLS) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(st[n][i]), rs, o + i * 4 * width, 0, 0);
      } else {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, st[n]), rs, o, 0, 0);
      }
    }
  }
  // The columns of odd numbers with the opposite sign (COLS false).
  __device__ __forceinline__ static v4f flipped(v4f v) { return v4f{v[0], -v[1], v[2], -v[3]}; }
  __device__ __forceinline__ void flip() {
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) st[n] = flipped(st[n]);
  }
  // S = total S + M^T (coef_s v_s); vf holds v.  With bf16 the scaled v goes
  // in whole, in three parts: M is exact, so the state keeps fp32's precision.
  // A step's products are added up by themselves: on top of the state, each
  // would round, or drop bits, at the state's size.
  template <class T>
  __device__ __forceinline__ void advance(float total, const float* coef, const T* m, int ldn,
                                          const Frag<T> (&vf)[2]) {
    const int g = (threadIdx.x & 63) >> 4;
    Split<T, kExact<T>> parts[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[8];
      const v4f* c = reinterpret_cast<const v4f*>(coef + k * 32 + 8 * g);
      const v4f c0 = c[0], c1 = c[1];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = frag_get(vf[k], j) * (j < 4 ? c0[j & 3] : c1[j & 3]);
      parts[k] = split_of<T, kExact<T>>(v);
    }
    // four tiles at a time: a product waits for the last one on the same tile
    constexpr int kTiles = 2 * NB < 4 ? 2 * NB : 4;
#pragma unroll
    for (int n = 0; n < 2 * NB; n += kTiles) {
      v4f add[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) add[i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Frag<T> mf[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) mf[i] = frag_col(m, ldn, k * 32, (n + i) * 16);
#pragma unroll
        for (int z = 0; z < kExact<T>; ++z)
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            if constexpr (COLS) mma(add[i], mf[i], parts[k].f[z]); else mma(add[i], parts[k].f[z], mf[i]);
          }
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i) st[n + i] = st[n + i] * total + add[i];
    }
  }
};

// The kept states lie as a wave holds them, so that they are written and read
// a kilobyte at a time: [steps][heads][width / 16][states / 16] tiles (counts
// rounded up) of [64 lanes][4], lane l with row l & 15 and columns 4 (l >> 4) ..
// of its tile.  What a tile has beyond the state is zero.
constexpr int kKeptTile = 256;  // floats
constexpr int kNonTemporal = 2; // read and written once: past the lines that the heads share (188 against 173 us)
__host__ __device__ inline int tiles_of(int n) { return (n + 15) / 16; }
__host__ __device__ inline long kept_size(int width, int states) {
  return static_cast<long>(tiles_of(width)) * tiles_of(states) * kKeptTile;
}

template <class T, int NB, int NW>
struct WalkLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  static constexpr int ldp = stride_of<T>(NW * 16);
  alignas(16) T m[kTok * ldn];
  alignas(16) T v[kTok * ldp];
  alignas(16) Decays dc[2];
};

// Waves on a SIMD that registers are allotted for: as many as LDS holds of a CU's
// four, up to `most`.
constexpr int simd_waves(size_t lds, int nw, int most) {
  const int n = (160 * 1024 / static_cast<int>(lds) * nw + 3) / 4;
  return n < most ? n : most;
}

// The state a segment starts from: the sequence's first one, brought through
// the segments before it (in the pass's direction), whose own contributions
// lie in the place of the segment behind each.  With few segments every one
// does that itself; the carry pass leaves the sum in their places otherwise.
template <int NB, bool COLS>
__device__ __forceinline__ void start_state(State<NB, COLS>& st, const SsmArgs& a, const Walk& w, const Unit& u, int unit,
                                            int h) {
  const long head = static_cast<long>(a.states) * a.width;
  const int d = w.rev ? -1 : 1;
  const int before = w.rev ? units_of(u.len, a.seg) - 1 - u.index : u.index;
  if (before > 0 && !a.fold) {
    st.load(w.seg_state + (static_cast<long>(unit) * a.heads + h) * head, a.width, a.states);
    return;
  }
  st.load(w.first == nullptr ? nullptr : w.first + (static_cast<long>(u.seq) * a.heads + h) * head, a.width, a.states);
  for (int i = before - 1; i >= 0; --i) {
    const long at = (static_cast<long>(unit) - d * i) * a.heads + h;
    State<NB, COLS> own;
    own.off = st.off;
    own.load(w.seg_state + at * head, a.width, a.states);
    const float decay = w.seg_decay[at - d * a.heads];
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) st.st[n] = st.st[n] * decay + own.st[n];
  }
}

// KEEP false: the summary of a segment that another follows, from a zero
// state, into that segment's place.  KEEP true: the walk itself, from the
// states the carry left, writing every step's starting state.
template <class T, int NB, int NW, bool KEEP>
__device__ __forceinline__ void walk(const SsmArgs& a, const Walk& w, WalkLds<T, NB, NW>& s) {
  typedef WalkLds<T, NB, NW> L;
  constexpr int kThreads = NW * 64;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int per = a.heads * a.slices;
  const int unit = work / per;
  const int h = work % per / a.slices;
  const int slice = work % a.slices;
  const Unit u = locate(a.q, unit, a.seg);
  if (!u.live) return;
  const bool last = w.rev ? u.index == 0 : u.t0 + static_cast<long>(a.seg) >= u.len;
  if (!KEEP && last) return;
  const bool packed = a.q.offsets != nullptr;
  const int p0 = slice * NW * 16;
  const int cols = min(a.width - p0, NW * 16);
  const long head = static_cast<long>(a.states) * a.width;
  const T* vp = seq_ptr<const T>(w.v, u.seq, u.row0, packed) + h * a.width + p0;
  const T* mp = seq_ptr<const T>(w.m, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const double rate = decay_rate(a.A[h]);
  const float bias = a.bias != nullptr ? a.bias[h] : 0.0f;
  const long at = static_cast<long>(unit) * a.heads + h;
  const long of_seq = (static_cast<long>(u.seq) * a.heads + h) * head;
  State<NB, false> st;
  st.init(a.width, p0, wave);
  if (KEEP) {
    start_state(st, a, w, u, unit, h);
    if (kFlips<T>) st.flip();
  } else {
    st.zero();
  }
  double decay = 0.0;
  Tile<T, kTok, NB * 32, kThreads> tm;
  Tile<T, kTok, NW * 16, kThreads> tv;
  tm.init(w.m.row_stride, a.states, tid);
  tv.init(w.v.row_stride, cols, tid);
  const int end = min(u.t0 + a.seg, u.len);
  const int steps = (end - u.t0 + kTok - 1) / kTok;
  const auto token = [&](int i) { return u.t0 + (w.rev ? steps - 1 - i : i) * kTok; };
  const auto fetch = [&](int t) {
    const int rows = min(end - t, kTok);
    tm.load(rows_rsrc(mp + t * w.m.row_stride, w.m.row_stride, rows, a.states));
    tv.load(rows_rsrc(vp + t * w.v.row_stride, w.v.row_stride, rows, cols));
  };
  // The last wave prepares the next step's decays while the others multiply;
  // the raw step sizes are loaded a step before that.
  const bool decays = wave == NW - 1;
  float raw = 0.0f;
  const auto fetch_raw = [&](int t) { raw = load_raw(a, step_rsrc(a, u, packed, t, min(end - t, kTok)), h); };
  const auto prepare = [&](Decays& dc, int t) {
    make_decays(dc, lane < end - t ? step_of(a, raw, bias) : 0.0f, rate);
  };
  if (steps > 0) {
    fetch(token(0));
    if (decays) {
      fetch_raw(token(0));
      prepare(s.dc[0], token(0));
      if (steps > 1) fetch_raw(token(1));
    }
  }
  for (int i = 0; i < steps; ++i) {
    const int t = token(i);
    const Decays& dc = s.dc[i & 1];
    __syncthreads();
    tm.store(s.m, L::ldn, tid);
    tv.store(s.v, L::ldp, tid);
    __syncthreads();
    if (i + 1 < steps) {
      fetch(token(i + 1));
      if (decays) {
        prepare(s.dc[(i + 1) & 1], token(i + 1));
        if (i + 2 < steps) fetch_raw(token(i + 2));
      }
    }
    if (KEEP) {
      const long step = static_cast<long>(unit_base(a.q, u.seq, kTok)) + t / kTok;
      const int strip = slice * NW + wave, tiles = tiles_of(a.states);
      const Rsrc rs = make_rsrc(w.keep + (step * a.heads + h) * kept_size(a.width, a.states) +
                                    static_cast<long>(strip) * tiles * kKeptTile,
                                strip < tiles_of(a.width) ? tiles * kKeptTile * 4u : 0u);
#pragma unroll
      for (int n = 0; n < 2 * NB; ++n)
        __builtin_amdgcn_raw_buffer_store_b128(
            __builtin_bit_cast(v4i, kFlips<T> ? st.flipped(st.st[n]) : st.st[n]), rs, (n * 64 + lane) * 16, 0,
            kNonTemporal);
    }
    Frag<T> vf[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) vf[k] = flip_odd(frag_col(s.v, L::ldp, k * 32, wave * 16), lane);
    st.template advance<T>(dc.total, w.rev ? dc.from : dc.to, s.m, L::ldn, vf);
    if (!KEEP) decay += dc.end;
  }
  if (kFlips<T>) st.flip();
  if (KEEP) {
    if (last && w.last != nullptr) st.save(w.last + of_seq, a.width, a.states);
  } else {
    const long next = at + (w.rev ? -a.heads : a.heads);
    st.save(w.seg_state + next * head, a.width, a.states);
    if (tid == 0 && slice == 0) w.seg_decay[at] = exp2_of(decay);
  }
}

// 8 us for 32 segments of 24 heads of 64 x 64, the chain's length (24 MB).
// Carry: turns the segments' own contributions into the state each segment
// starts from.  One thread per four elements of a sequence's head.
__device__ __forceinline__ void carry(const SsmArgs& a, const Walk& w, int seq, int block) {
  const long head = static_cast<long>(a.states) * a.width;
  const long e = (static_cast<long>(block) * blockDim.x + threadIdx.x) * 4;
  if (e >= head) return;
  const int h = blockIdx.y;
  long row0;
  int len;
  seq_rows(a.q, seq, &row0, &len);
  const int n = units_of(len, a.seg);
  const long base = unit_base(a.q, seq, a.seg);
  v4f run = {0, 0, 0, 0};
  if (w.first != nullptr)
    run = *reinterpret_cast<const v4f*>(w.first + (static_cast<long>(seq) * a.heads + h) * head + e);
  const int d = w.rev ? -1 : 1;
  constexpr int kAhead = 8;  // segments whose states are in flight together
  for (int i = w.rev ? n - 2 : 1; i >= 0 && i < n; i += d * kAhead) {
    v4f own[kAhead];
    float decay[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = i + d * j;
      if (k >= 0 && k < n) {
        const long at = (base + k) * a.heads + h;
        own[j] = *reinterpret_cast<const v4f*>(w.seg_state + at * head + e);
        decay[j] = w.seg_decay[at - d * a.heads];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = i + d * j;
      if (k >= 0 && k < n) {
        run = run * decay[j] + own[j];
        *reinterpret_cast<v4f*>(w.seg_state + ((base + k) * a.heads + h) * head + e) = run;
      }
    }
  }
}

// Host side, in ssm.hip.
int check_dims(const mamba2_seqs& q, const mamba2_ssm_dims& d);
int check_scan(const mamba2_seqs& q, const mamba2_ssm_dims& d, bool bwd);
int check_vec_rows(const mamba2_rows& r, const mamba2_seqs& q, long long width, size_t elem);
int check_step_rows(const mamba2_rows& r, const mamba2_seqs& q, const mamba2_ssm_dims& d);
int waves_of(int width);
int segment_tokens(const mamba2_seqs& q, const mamba2_ssm_dims& d, bool bwd);
int fold_segments(const mamba2_seqs& q, const mamba2_ssm_dims& d, int seg);

}  // namespace ssm
