// Group norm with an activation, channels last, for gfx950: forward and
// backward.  Per token and group of `width` channels
//   h = x (or x silu(z)),  r = (mean((h - mean)^2) + eps)^-1/2,  n = (h - mean) r,
//   o = n w + b,  y = o, silu(o) or o silu(z);
// backward, with d = dL/do, d_n = d w:
//   d_w = sum d n,  d_b = sum d,  d_h = r (d_n - n mean(d_n n) - mean(d_n)).
//
// Memory is what bounds it: every tensor is read or written once, a group is
// held in the registers of the lanes that share it between its statistics and
// its results, and the backward recomputes the statistics.  A group has L lanes
// (a power of two up to 64, or the whole block) of R vectors; a thread keeps its
// channels from row to row, so weights are loaded once and the weights' gradients
// add up in registers.
//
// 16384 tokens, 32 groups of 128 channels, bf16, gated, a weight for all groups:
// forward 76 us, 0.40 GB, 5.3 TB/s; backward 128 us, 0.67 GB, 5.2 TB/s, and 5 us for
// the sums over its blocks.  3063 tokens, 8 groups of 97 channels, fp32, element by
// element: forward 10 us, backward 16 and 5.
#include "layer_common.h"
#include "mamba2_delta.h"
#include "ssm_common.h"

namespace {

using namespace layer;
using ssm::dpp_add;
using ssm::Pair;
using ssm::sum64;
using ssm::swap16;
using ssm::swap32;

struct NormArgs {
  mamba2_seqs q;
  mamba2_rows x, gate, y, d_y, d_x, d_gate;
  const float* weight;
  const float* bias;
  float* partial;        // [slices][2][n]: the weights' gradients, then the biases'; a slice for each run of rows
                         // (shared: for each block)
  int groups, width, shared, centered;
  int lanes;             // L: lanes of a group
  int across;            // neighbouring groups of a block
  int columns;           // blocks that a row takes
  int run;               // rows of a block
  int n;                 // elements of weight: width (shared) or channels
  int flat;              // row r is r * row_stride from the start
  float eps, inv_width;
};

// 1 / (1 + e^-v), to fp32's last bits; the exponent's product in two terms.  The
// second one's share is added where 2^p is finite: from 2^128 on it is infinite, and
// infinity times a negative rest would make a NaN of a sigmoid that is 0.
__device__ __forceinline__ float sigmoid_of(float v) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float p = -v * kLog2e;
  const float rest = fmaf(-v, 1.925963033500e-8f, fmaf(-v, kLog2e, -p));
  float t = __builtin_amdgcn_exp2f(p);
  t = fabsf(p) < 128.0f ? fmaf(t, 0.69314718056f * rest, t) : t;
  return __builtin_amdgcn_rcpf(1.0f + t);
}

// The sum over a group's lanes, in all of them.  Up to a wave: lanes that differ
// in one bit after the other.  WIDE: the block, through `part`, of which a block
// uses two halves in turn.
template <bool WIDE>
struct GroupSum {
  int lanes;
  float* part;
  int turn;
  __device__ __forceinline__ float operator()(float v) {
    if constexpr (WIDE) {
      const int waves = blockDim.x >> 6;
      v = sum64(v);
      float* p = part + turn * 16;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) p[threadIdx.x >> 6] = v;
      __syncthreads();
      v = 0.0f;
      for (int i = 0; i < waves; ++i) v += p[i];
      return v;
    } else {
      if (lanes > 1) v = dpp_add<0xb1, 0xf>(v);   // quad_perm 1 0 3 2
      if (lanes > 2) v = dpp_add<0x4e, 0xf>(v);   // quad_perm 2 3 0 1
      if (lanes > 4) v = dpp_add<0x141, 0xf>(v);  // row_half_mirror
      if (lanes > 8) v = dpp_add<0x140, 0xf>(v);  // row_mirror
      if (lanes > 16) {
        const Pair p = swap16(v);
        v = p.a + p.b;
      }
      if (lanes > 32) {
        const Pair p = swap32(v);
        v = p.a + p.b;
      }
      return v;
    }
  }
};

// What a thread works on: its group, its channels, its rows.
struct Place {
  bool live;        // has a group
  int channel;      // of its first vector in a row; vector i is i * lanes * V further on
  int in_group;     // the same within its group
  int group;        // of the block's groups
  int row, step;    // first row (of the block's), distance to its next
};
template <int V>
__device__ __forceinline__ Place place_of(const NormArgs& a, int column) {
  Place p;
  const int item = threadIdx.x / a.lanes, lane = threadIdx.x - item * a.lanes;
  p.group = item & (a.across - 1);
  p.row = item / a.across;
  p.step = blockDim.x / a.lanes / a.across;
  const int group = column * a.across + p.group;
  p.live = group < a.groups;
  p.in_group = lane * V;
  p.channel = group * a.width + p.in_group;
  return p;
}

template <class T>
__device__ __forceinline__ T* row_ptr(const mamba2_rows& r, const NormArgs& a, int row) {
  T* p = static_cast<T*>(r.data);
  if (a.flat) return p + row * r.row_stride;
  const int b = row / a.q.length;
  return p + b * r.batch_stride + (row - b * a.q.length) * r.row_stride;
}

// The call's rows: those of the sequences.
__device__ __forceinline__ void rows_range(const NormArgs& a, int* first, int* behind) {
  if (a.q.offsets == nullptr) {
    *first = 0;
    *behind = a.q.batch * a.q.length;
  } else {
    *first = clamp_row(a.q.offsets[0], a.q.length);
    *behind = clamp_row(a.q.offsets[a.q.batch], a.q.length);
  }
}

// V neighbouring elements as they were loaded.
template <class T, int V>
struct Piece {
  typename Vec<T>::type v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const typename Vec<T>::type*>(p); }
  __device__ __forceinline__ float operator[](int j) const { return static_cast<float>(v[j]); }
};
template <class T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ float operator[](int) const { return static_cast<float>(v); }
};
// A thread's pieces of a row.  AHEAD: one that its group does not have is the group's
// first one, so that all are loaded, none behind a branch, which would make a wait for
// these loads a wait for what is issued after them, too.  Else it is 0, and the offsets
// are formed where they are used: formed before the branch, all are kept over the rows
// (2048 rows of 16384 elements, fp32, backward: 213 us, 138 so).
template <class T, int V, int R, bool AHEAD>
struct Pieces {
  Piece<T, V> p[R];
  __device__ __forceinline__ void load(const mamba2_rows& r, const NormArgs& a, const Place& w, int row) {
    const T* base = row_ptr<const T>(r, a, row);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = w.in_group + i * a.lanes * V < a.width;
      if (AHEAD) p[i].load(base + (in ? w.channel + i * a.lanes * V : w.channel - w.in_group));
      else if (in) p[i].load(base + w.channel + i * a.lanes * V);
      else p[i] = {};
    }
  }
};
template <class T, int V>
__device__ __forceinline__ void store_piece(T* p, const Place& w, const NormArgs& a, int i, const float (&v)[V]) {
  if (w.in_group + i * a.lanes * V < a.width) store_vec<T, V>(p + w.channel + i * a.lanes * V, v);
}
// A parameter's values of a thread's channels.
template <int V, int R>
__device__ __forceinline__ void load_parameter(const float* p, const Place& w, const NormArgs& a, float without,
                                               float (&v)[R][V]) {
  const int c = a.shared ? w.in_group : w.channel;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j)
      v[i][j] = p != nullptr && w.live && w.in_group + i * a.lanes * V < a.width ? p[c + i * a.lanes * V + j] : without;
}

// h of the loaded x and gate (in place) to n; returns r.
template <int V, int R, class Sum>
__device__ __forceinline__ float normalise(float (&h)[R][V], const Place& w, const NormArgs& a, Sum& sum) {
  if (a.centered) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) m += h[i][j];
    m = sum(m) * a.inv_width;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] = w.in_group + i * a.lanes * V < a.width ? h[i][j] - m : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s = fmaf(h[i][j], h[i][j], s);
  const float r = rsqrtf(fmaf(sum(s), a.inv_width, a.eps));
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) h[i][j] *= r;
  return r;
}

// A block's rows, the call's `first` .. `behind` - 1.
__device__ __forceinline__ long rows_of_block(const NormArgs& a, int chunk, int* end) {
  int first, behind;
  rows_range(a, &first, &behind);
  const long row0 = static_cast<long>(first) + static_cast<long>(chunk) * a.run;
  *end = static_cast<int>(min(row0 + a.run, static_cast<long>(behind)));
  return row0;
}

// The next row is loaded while one is worked on, where a thread has the registers.
// Backward, gated, bf16: 16384 rows of 4096 channels 164 us without, 155 with it; 65536
// of 1024, 152 and 146; 65536 of 8 groups of 97, element by element, 425 and 205 (3063 of
// them 24 and 23, plain 19 and 21: the last row is loaded twice).  fp32 elements are left
// out: 3063 rows of 8 groups of 97, plain, 19 and 21; 32768 of them 94 and 81.  Nor do
// wide blocks' forwards of whole vectors gain, of which more are on a CU (8192 rows of
// 8192, gated: 84 us without, 97 with it; by elements, 16384 of 4096, 315 and 136).
template <class T, int V, int R, bool WIDE, bool BWD>
constexpr bool kAhead = !WIDE ? V > 1 || sizeof(T) == 2 : BWD ? R * V * static_cast<int>(sizeof(T)) <= 16 : V == 1 && R < 16;
// The gate's gradients are stored at once, before the group's sums, which frees their
// registers.  Groups taken by elements in a wave have those and lose by it (65536 rows
// of 8 groups of 97, bf16: 220 us, 205 behind the sums).
template <int V, bool WIDE>
constexpr bool kGateAtOnce = WIDE || V > 1;
// The backward of a block of 1024 threads reads its parameters again for each row where
// it has two vectors of bf16 or four of fp32: held, it spills.  4096 rows of 12288, bf16,
// held and not: gate first 372 and 322 us, 512 rows 93 and 81; fp32, SiLU 196 and 187;
// the other side is the gate behind, 242 and 268.
template <int V, int R, bool WIDE>
constexpr bool kHold = !WIDE || V == 1 || R * V <= 8;

template <class T, int V, int R, int FORM, bool WIDE>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void norm_fwd_kernel(NormArgs a) {
  __shared__ float part[32];
  constexpr bool kGate = FORM == MAMBA2_NORM_GATED || FORM == MAMBA2_NORM_GATE_FIRST;
  const int column = blockIdx.x % a.columns, chunk = blockIdx.x / a.columns;
  const Place w = place_of<V>(a, column);
  GroupSum<WIDE> sum{a.lanes, part, 0};
  int end;
  long row = rows_of_block(a, chunk, &end) + w.row;
  float weight[R][V], bias[R][V];
  load_parameter<V, R>(a.weight, w, a, 1.0f, weight);
  load_parameter<V, R>(a.bias, w, a, 0.0f, bias);
  if (!w.live || row >= end) return;  // a wide block has one group and one row at a time
  constexpr bool kNext = kAhead<T, V, R, WIDE, false>;
  Pieces<T, V, R, kNext> x, gate;
  const auto fetch = [&](long r) {
    x.load(a.x, a, w, r);
    if constexpr (kGate) gate.load(a.gate, a, w, r);
  };
  if constexpr (kNext) fetch(row);
  for (; row < end; row += w.step) {
    if constexpr (!kNext) fetch(row);
    const Pieces<T, V, R, kNext> hx = x, hz = gate;
    if constexpr (kNext) fetch(row + w.step < end ? row + w.step : row);  // the last one again
    float h[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v = hx.p[i][j];
        if constexpr (FORM == MAMBA2_NORM_GATE_FIRST) v *= hz.p[i][j] * sigmoid_of(hz.p[i][j]);
        h[i][j] = !kNext || w.in_group + i * a.lanes * V < a.width ? v : 0.0f;
      }
    normalise<V, R>(h, w, a, sum);
    T* y = row_ptr<T>(a.y, a, row);
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float o = fmaf(h[i][j], weight[i][j], bias[i][j]);
        if constexpr (FORM == MAMBA2_NORM_SILU) o *= sigmoid_of(o);
        if constexpr (FORM == MAMBA2_NORM_GATED) o *= hz.p[i][j] * sigmoid_of(hz.p[i][j]);
        h[i][j] = o;
      }
      store_piece<T, V>(y, w, a, i, h[i]);
    }
  }
}

template <class T, int V, int R, int FORM, bool WIDE>
__global__ __launch_bounds__(WIDE ? 1024 : 256) void norm_bwd_kernel(NormArgs a) {
  __shared__ float part[32];
  constexpr int kSums = 2 * R * V;  // sums that a thread holds
  __shared__ float sums[WIDE ? 1 : 256][kSums + 1];
  constexpr bool kGate = FORM == MAMBA2_NORM_GATED || FORM == MAMBA2_NORM_GATE_FIRST;
  const int column = blockIdx.x % a.columns, chunk = blockIdx.x / a.columns;
  const Place w = place_of<V>(a, column);
  GroupSum<WIDE> sum{a.lanes, part, 0};
  int end;
  long row = rows_of_block(a, chunk, &end) + w.row;
  float weight[R][V], bias[R][V], d_w[R][V], d_b[R][V];
  const auto parameters = [&] {
    load_parameter<V, R>(a.weight, w, a, 1.0f, weight);
    if constexpr (FORM == MAMBA2_NORM_SILU || FORM == MAMBA2_NORM_GATED) load_parameter<V, R>(a.bias, w, a, 0.0f, bias);
  };
  if constexpr (kHold<V, R, WIDE>) parameters();
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) d_w[i][j] = d_b[i][j] = 0.0f;
  constexpr bool kNext = kAhead<T, V, R, WIDE, true>;
  Pieces<T, V, R, kNext> x, gate, d_y;
  const auto fetch = [&](long r) {
    x.load(a.x, a, w, r);
    if constexpr (kGate) gate.load(a.gate, a, w, r);
    d_y.load(a.d_y, a, w, r);
  };
  const bool any = w.live && row < end;
  if (kNext && any) fetch(row);
  for (; any && row < end; row += w.step) {
    if constexpr (!kNext) fetch(row);
    const Pieces<T, V, R, kNext> hx = x, hz = gate, hd = d_y;
    if constexpr (kNext) fetch(row + w.step < end ? row + w.step : row);
    float h[R][V], d[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v = hx.p[i][j];
        if constexpr (FORM == MAMBA2_NORM_GATE_FIRST) v *= hz.p[i][j] * sigmoid_of(hz.p[i][j]);
        h[i][j] = !kNext || w.in_group + i * a.lanes * V < a.width ? v : 0.0f;
      }
    const float r = normalise<V, R>(h, w, a, sum);
    if constexpr (!kHold<V, R, WIDE>) parameters();
    T* const d_gate = kGate ? row_ptr<T>(a.d_gate, a, row) : nullptr;
    const bool put_gate = a.d_gate.data != nullptr;
    float dn = 0.0f, dnn = 0.0f;
    float dz[R][V];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = !kNext || w.in_group + i * a.lanes * V < a.width;  // else 0 was loaded
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = h[i][j];
        float e = in ? hd.p[i][j] : 0.0f;
        if constexpr (FORM == MAMBA2_NORM_SILU) {
          const float o = fmaf(n, weight[i][j], bias[i][j]), so = sigmoid_of(o);
          e *= so * fmaf(o, 1.0f - so, 1.0f);
        }
        if constexpr (FORM == MAMBA2_NORM_GATED) {
          const float z = in ? hz.p[i][j] : 0.0f, g = sigmoid_of(z), o = fmaf(n, weight[i][j], bias[i][j]);
          dz[i][j] = e * o * (g * fmaf(z, 1.0f - g, 1.0f));
          e *= z * g;
        }
        d_w[i][j] = fmaf(e, n, d_w[i][j]);
        d_b[i][j] += e;
        e *= weight[i][j];
        dn += e;
        dnn = fmaf(e, n, dnn);
        d[i][j] = e;
      }
      if constexpr (FORM == MAMBA2_NORM_GATED && kGateAtOnce<V, WIDE>) {
        if (put_gate) store_piece<T, V>(d_gate, w, a, i, dz[i]);
      }
    }
    dnn = sum(dnn) * a.inv_width;
    dn = a.centered ? sum(dn) * a.inv_width : 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float dh = r * (fmaf(-h[i][j], dnn, d[i][j]) - dn);
        if constexpr (FORM == MAMBA2_NORM_GATE_FIRST) {
          const float z = hz.p[i][j], g = sigmoid_of(z);
          dz[i][j] = dh * hx.p[i][j] * (g * fmaf(z, 1.0f - g, 1.0f));
          dh *= z * g;
        }
        d[i][j] = dh;
      }
    }
    // stores behind all of it: among it, 4096 rows of 16384, bf16, the gate in front, took
    // 438 us, 404 so; the other side is fp32 by elements, 2048 rows of them 326 and 344
    if (a.d_x.data != nullptr) {
      T* const d_x = row_ptr<T>(a.d_x, a, row);
#pragma unroll
      for (int i = 0; i < R; ++i) store_piece<T, V>(d_x, w, a, i, d[i]);
    }
    if constexpr (FORM == MAMBA2_NORM_GATE_FIRST || (FORM == MAMBA2_NORM_GATED && !kGateAtOnce<V, WIDE>)) {
      if (put_gate) {
#pragma unroll
        for (int i = 0; i < R; ++i) store_piece<T, V>(d_gate, w, a, i, dz[i]);
      }
    }
  }
  if (a.partial == nullptr) return;
  if constexpr (WIDE) {
    float* p = a.partial + (a.shared ? static_cast<long>(chunk) * a.columns + column : chunk) * 2 * a.n +
               (a.shared ? w.in_group : w.channel);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (w.in_group + i * a.lanes * V < a.width) {
          p[i * a.lanes * V + j] = d_w[i][j];
          p[a.n + i * a.lanes * V + j] = d_b[i][j];
        }
  } else {
    // the block's items with the same parameters: those of a group, or with shared
    // parameters all
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sums[threadIdx.x][i * V + j] = d_w[i][j];
        sums[threadIdx.x][R * V + i * V + j] = d_b[i][j];
      }
    __syncthreads();
    const int keys = a.shared ? 1 : a.across, items = 256 / a.lanes;
    float* p = a.partial + (a.shared ? static_cast<long>(chunk) * a.columns + column : chunk) * 2 * a.n;
    for (int o = threadIdx.x; o < keys * kSums * a.lanes; o += 256) {
      const int lane = o % a.lanes, e = o / a.lanes % kSums, key = o / a.lanes / kSums;
      const int v = e < R * V ? e : e - R * V;
      const int in_group = (v / V * a.lanes + lane) * V + v % V, group = column * a.across + key;
      if (in_group >= a.width || group >= a.groups) continue;
      float s = 0.0f;
      for (int i = key; i < items; i += keys) s += sums[i * a.lanes + lane][e];
      p[(e < R * V ? 0 : a.n) + (a.shared ? 0 : group * a.width) + in_group] = s;
    }
  }
}

// Sums [slices][2][n] over the slices: 32 columns a block, 32 runs of slices, in a
// fixed order.  Latency bounds it, so kSumAhead loads are on their way at a time:
// 1024 slices of 256 columns 4.9 us, one load after the other 11.7.
constexpr int kSumCols = 32, kSumRuns = 32, kSumAhead = 8;
struct SumArgs {
  const float* partial;
  float* d_weight;
  float* d_bias;
  long slices;
  int n;
};
__global__ __launch_bounds__(kSumCols * kSumRuns) void norm_sum_kernel(SumArgs a) {
  __shared__ float part[kSumRuns][kSumCols + 1];
  const int c = threadIdx.x % kSumCols, run = threadIdx.x / kSumCols;
  const long col = static_cast<long>(blockIdx.x) * kSumCols + c;  // of 2 n
  float s = 0.0f;
  if (col < 2 * a.n) {
    long i = run;
    for (; i + (kSumAhead - 1) * kSumRuns < a.slices; i += kSumAhead * kSumRuns) {
      float v[kSumAhead];
#pragma unroll
      for (int j = 0; j < kSumAhead; ++j) v[j] = a.partial[(i + j * kSumRuns) * 2 * a.n + col];
#pragma unroll
      for (int j = 0; j < kSumAhead; ++j) s += v[j];
    }
    for (; i < a.slices; i += kSumRuns) s += a.partial[i * 2 * a.n + col];
  }
  part[run][c] = s;
  __syncthreads();
  if (run == 0 && col < 2 * a.n) {
    for (int i = 1; i < kSumRuns; ++i) s += part[i][c];
    if (col < a.n) {
      if (a.d_weight != nullptr) a.d_weight[col] = s;
    } else if (a.d_bias != nullptr) {
      a.d_bias[col - a.n] = s;
    }
  }
}

// ---------------------------------------------------------------- host side
constexpr int kMaxWidth = 16384;

long long rows_of(const mamba2_seqs& q) {
  return static_cast<long long>(q.length) * (q.offsets != nullptr ? 1 : q.batch);
}

// How a call's rows and groups lie on blocks and lanes.
struct Shape {
  int vec, r, lanes, threads, across, columns, run;
  bool wide;
  long chunks, slices;
};
int pow2_from(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}
Shape shape_of(const mamba2_seqs& q, const mamba2_norm_dims& d, bool vec, bool bwd) {
  Shape s;
  s.vec = vec ? (d.type == MAMBA2_BF16 ? 8 : 4) : 1;
  const int vectors = (d.width + s.vec - 1) / s.vec;
  s.wide = vectors > 128;
  s.threads = vectors > 512 ? 1024 : vectors > 256 ? 512 : 256;
  s.lanes = s.wide ? s.threads : pow2_from(vectors) < 64 ? pow2_from(vectors) : 64;
  const int each = (vectors + s.lanes - 1) / s.lanes;
  s.r = each <= 1 ? 1 : each <= 2 ? 2 : each <= 4 ? 4 : 16;
  // neighbouring groups of a block: as many as leave the fewest lanes without one
  const int items = s.threads / s.lanes;
  s.across = 1;
  for (int n = 2; n <= items; n *= 2)
    if ((d.groups + n - 1) / n * n <= (d.groups + s.across - 1) / s.across * s.across) s.across = n;
  s.columns = (d.groups + s.across - 1) / s.across;
  const int at_once = items / s.across;
  const long long rows = rows_of(q);
  // rows of a block: blocks for the chip first, then longer runs
  const long long want = (bwd ? 4LL : 16LL) * kCUs;
  const long long per = (rows * s.columns + want - 1) / want;
  long long run = (per + at_once - 1) / at_once * at_once;
  if (run < at_once) run = at_once;
  s.run = static_cast<int>(run);
  s.chunks = static_cast<long>((rows + run - 1) / run);
  s.slices = s.chunks * (d.shared ? s.columns : 1);
  return s;
}

template <class T, int V, int R, bool WIDE>
void launch_form(bool bwd, int form, const NormArgs& a, const Shape& s, hipStream_t st) {
  const unsigned blocks = static_cast<unsigned>(s.chunks * s.columns);
  switch (form) {
#define NORM_CASE(F)                                                                       \
  case F:                                                                                  \
    if (bwd) norm_bwd_kernel<T, V, R, F, WIDE><<<blocks, s.threads, 0, st>>>(a);           \
    else norm_fwd_kernel<T, V, R, F, WIDE><<<blocks, s.threads, 0, st>>>(a);               \
    break;
    NORM_CASE(MAMBA2_NORM_PLAIN)
    NORM_CASE(MAMBA2_NORM_SILU)
    NORM_CASE(MAMBA2_NORM_GATED)
    NORM_CASE(MAMBA2_NORM_GATE_FIRST)
#undef NORM_CASE
  }
}
// Up to 128 vectors a group has one wave's lanes, so R is 1 or 2 there.
template <class T, int V>
void launch_r(bool bwd, int form, const NormArgs& a, const Shape& s, hipStream_t st) {
  if (!s.wide) {
    if (s.r == 1) launch_form<T, V, 1, false>(bwd, form, a, s, st);
    else launch_form<T, V, 2, false>(bwd, form, a, s, st);
  } else if (s.r == 1) {
    launch_form<T, V, 1, true>(bwd, form, a, s, st);
  } else if (s.r == 2) {
    launch_form<T, V, 2, true>(bwd, form, a, s, st);
  } else if constexpr (V < 8) {  // 1024 lanes of two 8-element vectors hold any group
    if (V > 1 || s.r == 4) launch_form<T, V, 4, true>(bwd, form, a, s, st);
    else launch_form<T, 1, 16, true>(bwd, form, a, s, st);
  }
}
void launch_norm(bool bwd, const mamba2_norm_dims& d, const NormArgs& a, const Shape& s, hipStream_t st) {
  if (d.type == MAMBA2_BF16) {
    if (s.vec > 1) launch_r<bf16, 8>(bwd, d.form, a, s, st);
    else launch_r<bf16, 1>(bwd, d.form, a, s, st);
  } else {
    if (s.vec > 1) launch_r<float, 4>(bwd, d.form, a, s, st);
    else launch_r<float, 1>(bwd, d.form, a, s, st);
  }
}

bool gated(const mamba2_norm_dims& d) { return d.form == MAMBA2_NORM_GATED || d.form == MAMBA2_NORM_GATE_FIRST; }

int check_norm(const mamba2_seqs& q, const mamba2_norm_dims& d) {
  if (!type_ok(d.type) || d.form < MAMBA2_NORM_PLAIN || d.form > MAMBA2_NORM_GATE_FIRST) return MAMBA2_SCAN_EUNSUPPORTED;
  const int st = check_seqs(q);
  if (st != MAMBA2_SCAN_OK) return st;
  if (d.groups < 1 || d.width < 1 || !(d.eps >= 1.17549435e-38f && d.eps < INFINITY)) return MAMBA2_SCAN_EBADDIM;
  if (d.groups > 65535 || d.width > kMaxWidth || static_cast<long long>(d.groups) * d.width > (1 << 22))
    return MAMBA2_SCAN_EUNSUPPORTED;
  for (const bool bwd : {false, true}) {
    const Shape s = shape_of(q, d, false, bwd);
    if (!grid_ok(s.chunks * s.columns, s.threads)) return MAMBA2_SCAN_EBADDIM;
  }
  return MAMBA2_SCAN_OK;
}

// One tensor of a call: checked, its unused strides replaced; vec and flat stay
// true as long as every tensor allows them.
struct Tensors {
  const mamba2_seqs& q;
  long long channels;
  size_t elem;
  bool vec, flat;
  int add(mamba2_rows* r) {
    *r = used_strides(*r, q, channels);
    const int st = check_rows(*r, q, channels, elem);
    if (st != MAMBA2_SCAN_OK) return st;
    vec = vec && rows_vec(*r, elem);
    flat = flat && (q.offsets != nullptr || q.batch == 1 || r->batch_stride == q.length * r->row_stride);
    return MAMBA2_SCAN_OK;
  }
};

NormArgs args_of(const mamba2_seqs& q, const mamba2_norm_dims& d, const Shape& s, bool flat) {
  NormArgs a = {};
  a.q = q;
  a.groups = d.groups;
  a.width = d.width;
  a.shared = d.shared != 0;
  a.centered = d.centered;
  a.lanes = s.lanes;
  a.across = s.across;
  a.columns = s.columns;
  a.run = s.run;
  a.n = d.shared ? d.width : d.groups * d.width;
  a.flat = flat;
  a.eps = d.eps;
  a.inv_width = 1.0f / static_cast<float>(d.width);
  return a;
}

}  // namespace

extern "C" {

int mamba2_norm_fwd(mamba2_seqs seqs, mamba2_norm_dims d, mamba2_rows x, const float* weight, const float* bias,
                    mamba2_rows gate, mamba2_rows y, void* stream) {
  int st = check_norm(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(d.type);
  Tensors t = {seqs, static_cast<long long>(d.groups) * d.width, e, d.width % (16 / static_cast<int>(e)) == 0, true};
  if ((st = t.add(&x)) != MAMBA2_SCAN_OK || (gated(d) && (st = t.add(&gate)) != MAMBA2_SCAN_OK) ||
      (st = t.add(&y)) != MAMBA2_SCAN_OK)
    return st;
  if (bias != nullptr && weight == nullptr) return MAMBA2_SCAN_ENULL;
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4)) return MAMBA2_SCAN_EALIGN;
  if (seqs.length == 0) return MAMBA2_SCAN_OK;
  const Shape s = shape_of(seqs, d, t.vec, false);
  NormArgs a = args_of(seqs, d, s, t.flat);
  a.x = x;
  a.gate = gate;
  a.y = y;
  a.weight = weight;
  a.bias = bias;
  launch_norm(false, d, a, s, static_cast<hipStream_t>(stream));
  return launch_status();
}

size_t mamba2_norm_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_norm_dims d) {
  if (check_norm(seqs, d) != MAMBA2_SCAN_OK) return 0;
  const long long n = d.shared ? d.width : static_cast<long long>(d.groups) * d.width;
  const long a = shape_of(seqs, d, false, true).slices;
  const long b = d.width % (d.type == MAMBA2_BF16 ? 8 : 4) == 0 ? shape_of(seqs, d, true, true).slices : 0;
  const long most = a > b ? a : b;
  return (static_cast<size_t>(most > 0 ? most : 1) * 2 * n * sizeof(float) + 15) / 16 * 16;
}

int mamba2_norm_bwd(mamba2_seqs seqs, mamba2_norm_dims d, mamba2_rows x, const float* weight, const float* bias,
                    mamba2_rows gate, mamba2_rows d_y, mamba2_rows d_x, float* d_weight, float* d_bias,
                    mamba2_rows d_gate, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_norm(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(d.type);
  Tensors t = {seqs, static_cast<long long>(d.groups) * d.width, e, d.width % (16 / static_cast<int>(e)) == 0, true};
  if ((st = t.add(&x)) != MAMBA2_SCAN_OK || (gated(d) && (st = t.add(&gate)) != MAMBA2_SCAN_OK) ||
      (st = t.add(&d_y)) != MAMBA2_SCAN_OK || (d_x.data != nullptr && (st = t.add(&d_x)) != MAMBA2_SCAN_OK) ||
      (gated(d) && d_gate.data != nullptr && (st = t.add(&d_gate)) != MAMBA2_SCAN_OK))
    return st;
  if ((bias != nullptr && weight == nullptr) || (d_weight != nullptr && weight == nullptr) ||
      (d_bias != nullptr && bias == nullptr) ||
      (seqs.length > 0 && d_x.data == nullptr && d_weight == nullptr && d_bias == nullptr &&
       (!gated(d) || d_gate.data == nullptr)))  // a tensor of no rows may have no address
    return MAMBA2_SCAN_ENULL;
  if (!gated(d) && d_gate.data != nullptr) return MAMBA2_SCAN_EUNSUPPORTED;
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(d_weight, 4) || !aligned_to(d_bias, 4))
    return MAMBA2_SCAN_EALIGN;
  const bool sums = d_weight != nullptr || d_bias != nullptr;
  if (sums) {
    if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
    if (workspace_bytes < mamba2_norm_bwd_workspace_bytes(seqs, d)) return MAMBA2_SCAN_ESIZE;
    if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  }
  if (seqs.length == 0 && !sums) return MAMBA2_SCAN_OK;
  const Shape s = shape_of(seqs, d, t.vec, true);
  hipStream_t hs = static_cast<hipStream_t>(stream);
  NormArgs a = args_of(seqs, d, s, t.flat);
  a.x = x;
  a.gate = gate;
  a.d_y = d_y;
  a.d_x = d_x;
  a.d_gate = d_gate;
  a.weight = weight;
  a.bias = bias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  if (s.chunks > 0) {
    launch_norm(true, d, a, s, hs);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  }
  if (sums) {
    const SumArgs sa = {a.partial, d_weight, d_bias, s.slices, a.n};
    norm_sum_kernel<<<(2 * a.n + kSumCols - 1) / kSumCols, kSumCols * kSumRuns, 0, hs>>>(sa);
  }
  return launch_status();
}

}  // extern "C"
