// Shared by the selective layer's kernels: element types, vector access, and
// the mapping of units of work onto dense or packed sequences.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "mamba2_layer.h"

namespace layer {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef __bf16 bf16;
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kCUs = 256;

template <class T>
struct Vec;  // the 16-byte vector of T
template <>
struct Vec<float> {
  static constexpr int n = 4;
  typedef v4f type;
};
template <>
struct Vec<bf16> {
  static constexpr int n = 8;
  typedef v8bf type;
};

// V consecutive elements as floats: one 16-byte access when V fills it,
// element accesses otherwise.
template <class T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  if constexpr (V == Vec<T>::n) {
    const typename Vec<T>::type r = *reinterpret_cast<const typename Vec<T>::type*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = static_cast<float>(r[i]);
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    const v4bf r = *reinterpret_cast<const v4bf*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = static_cast<float>(r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = static_cast<float>(p[i]);
  }
}
template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (V == Vec<T>::n) {
    typename Vec<T>::type r;
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = static_cast<T>(v[i]);
    *reinterpret_cast<typename Vec<T>::type*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = static_cast<T>(v[i]);
  }
}

// One unit of `run` tokens of one sequence.
struct Unit {
  int seq;     // sequence
  int index;   // number of the unit within its sequence
  long row0;   // row of the sequence's first token (packed), 0 (dense)
  int len;     // tokens of the sequence
  int t0;      // first token of the unit; t0 >= len: no tokens
  bool live;   // the unit is one of its sequence's (an empty sequence has one)
};

// Dense sequences have ceil(length / run) units each, one when they are empty.
// Packed sequences: sequence s starts at unit off[s] / run + s.  That leaves
// every sequence at least ceil(len / run) units, needs no scan over the
// lengths, and bounds the units of a call by length / run + batch, which the
// host knows.  A few units stay empty.
__host__ __device__ inline int units_of(int len, int run) { return len > run ? (len + run - 1) / run : 1; }

__host__ __device__ inline long unit_count(const mamba2_seqs& q, int run) {
  if (q.offsets != nullptr) return static_cast<long>(q.length / run) + q.batch;
  return static_cast<long>(units_of(q.length, run)) * q.batch;
}

__device__ __forceinline__ int clamp_row(int v, int length) { return min(max(v, 0), length); }

__device__ __forceinline__ int unit_base(const mamba2_seqs& q, int s, int run) {
  if (q.offsets == nullptr) return s * units_of(q.length, run);
  return clamp_row(q.offsets[s], q.length) / run + s;
}

__device__ __forceinline__ void seq_rows(const mamba2_seqs& q, int s, long* row0, int* len) {
  if (q.offsets == nullptr) {
    *row0 = 0;
    *len = q.length;
    return;
  }
  const int b = clamp_row(q.offsets[s], q.length);
  *row0 = b;
  *len = max(clamp_row(q.offsets[s + 1], q.length) - b, 0);
}

// Called by whole waves.  A packed call's sequence is found with one load per
// lane once 64 candidates are left (a search step costs a trip to the cache).
__device__ __forceinline__ Unit locate(const mamba2_seqs& q, int unit, int run) {
  Unit u;
  if (q.offsets == nullptr) {
    const int per = units_of(q.length, run);
    u.seq = unit / per;
    u.index = unit - u.seq * per;
  } else {
    int lo = 0, hi = q.batch;  // the last s with unit_base(s) <= unit
    while (hi - lo > 64) {
      const int mid = (lo + hi) >> 1;
      if (unit_base(q, mid, run) <= unit) lo = mid; else hi = mid;
    }
    const int s = lo + static_cast<int>(threadIdx.x & 63);
    const bool before = s < hi && unit_base(q, s, run) <= unit;
    const unsigned long long m = __ballot(before);
    u.seq = lo + (m == 0 ? 0 : 63 - __builtin_clzll(m));
    u.index = unit - unit_base(q, u.seq, run);
  }
  long row0;
  int len;
  seq_rows(q, u.seq, &row0, &len);
  // known to be the same in all lanes
  u.seq = __builtin_amdgcn_readfirstlane(u.seq);
  u.index = __builtin_amdgcn_readfirstlane(u.index);
  u.row0 = __builtin_amdgcn_readfirstlane(static_cast<int>(row0));
  u.len = __builtin_amdgcn_readfirstlane(len);
  const long t = static_cast<long>(u.index) * run;
  u.live = u.index >= 0 && t < max(u.len, 1);
  u.t0 = u.live ? static_cast<int>(t) : u.len;
  return u;
}

// Address of a sequence's first token; token t is t * row_stride further on.
template <class T>
__device__ __forceinline__ T* seq_ptr(const mamba2_rows& r, int seq, long row0, bool packed) {
  return static_cast<T*>(r.data) + (packed ? row0 * r.row_stride : seq * r.batch_stride);
}

// ------------------------------------------------------------- host checks
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t type_size(int type) { return type == MAMBA2_BF16 ? 2 : 4; }
inline bool type_ok(int type) { return type == MAMBA2_F32 || type == MAMBA2_BF16; }

inline int check_seqs(const mamba2_seqs& q) {
  if (q.batch < 1 || q.length < 0) return MAMBA2_SCAN_EBADDIM;
  const long long rows = static_cast<long long>(q.length) * (q.offsets != nullptr ? 1 : q.batch);
  if (rows + q.batch > 2147483647LL - 65536) return MAMBA2_SCAN_EBADDIM;
  if (!aligned_to(q.offsets, 4)) return MAMBA2_SCAN_EALIGN;
  return MAMBA2_SCAN_OK;
}

// A tensor with the strides that its addresses need: a single row's stride and a
// single sequence's (or packed rows') may be anything, and the kernels form the
// addresses of rows behind the last, which have to lie behind the tensor's end.
inline mamba2_rows used_strides(mamba2_rows r, const mamba2_seqs& q, long long width) {
  if (q.length <= 1) r.row_stride = width;
  if (q.offsets != nullptr || q.batch == 1) r.batch_stride = 0;
  return r;
}

// A token-major tensor of `width` elements per row.
inline int check_rows(const mamba2_rows& r, const mamba2_seqs& q, long long width, size_t elem) {
  if (q.length == 0) return MAMBA2_SCAN_OK;
  if (r.data == nullptr) return MAMBA2_SCAN_ENULL;
  if (!aligned_to(r.data, elem)) return MAMBA2_SCAN_EALIGN;
  if (q.length > 1 && r.row_stride < width) return MAMBA2_SCAN_EBADDIM;
  if (q.offsets == nullptr && q.batch > 1 && r.batch_stride < width) return MAMBA2_SCAN_EBADDIM;
  return MAMBA2_SCAN_OK;
}

// May rows be accessed in 16-byte vectors?
inline bool rows_vec(const mamba2_rows& r, size_t elem) {
  const long long n = static_cast<long long>(16 / elem);
  return aligned_to(r.data, 16) && r.row_stride % n == 0 && r.batch_stride % n == 0;
}

// The memory of a tensor: rows of `width` bytes, `stride` bytes apart (0: one row).
struct Region {
  uintptr_t lo, hi;
  long long stride, width;
};
inline Region region(const void* p, long long bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return p == nullptr ? Region{0, 0, 0, 0} : Region{lo, lo + bytes, 0, bytes};
}
inline Region token_region(const mamba2_rows& r, int batch, long long width, size_t elem) {
  const long long bytes = width * static_cast<long long>(elem);
  if (batch == 1) return region(r.data, bytes);
  const long long stride = r.batch_stride * static_cast<long long>(elem);
  Region v = region(r.data, (batch - 1) * stride + bytes);
  v.stride = stride;
  v.width = bytes;
  return v;
}
// Slices of one wide row-major tensor interleave without overlapping.
inline bool overlap(const Region& a, const Region& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  const long long d = static_cast<long long>(b.lo - a.lo) % a.stride, gap = d < 0 ? d + a.stride : d;
  return a.width > gap || gap + b.width > a.stride;
}
// Of the first n regions, the outputs, none may overlap another one or an input.
inline bool apart(const Region* v, int n, int count) {
  for (int i = 0; i < n; ++i)
    for (int k = i + 1; k < count; ++k)
      if (overlap(v[i], v[k])) return false;
  return true;
}

// A launch counts its threads in 32 bits.
inline bool grid_ok(long long blocks, int threads) { return blocks <= 0xffffffffLL / threads; }

inline int launch_status() { return hipGetLastError() == hipSuccess ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EHIP; }

}  // namespace layer
