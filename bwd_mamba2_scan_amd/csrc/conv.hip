// Short causal depthwise convolution with SiLU: forward, backward and the
// single-token form, for gfx950.
//
//   pre_t = bias + sum_k w[k] x_{t-W+1+k},  y_t = f(pre_t)
//   dp_t  = d_y_t f'(pre_t)
//   d_x_u = sum_k w[k] dp_{u+W-1-k},  d_w[k] = sum_t dp_t x_{t-W+1+k},  d_bias = sum_t dp_t
//
// A few operations per element against two (forward) or three (backward)
// streamed tensors: bound by HBM, the backward nearly as much by arithmetic.
// A lane owns 16 bytes of channels (8 in the backward with bf16) and walks a
// run of tokens with the last W - 1 inputs (and W pre-activation gradients) in
// registers, so x and d_y are read once but for the W - 1 tokens where runs
// meet.  The next tokens' loads are in flight while the last ones are computed.
// At 4 x 4096 tokens of 4352 bf16 channels, 4 taps: forward 56 us, 285 MB at
// 5.1 TB/s, what a large copy reaches; backward 95 us, 428 MB at 4.5 TB/s, the
// vector units busy nearly as long: some 35 instructions an element, among them
// an exponential and a reciprocal.
#include "layer_common.h"

namespace {

using namespace layer;

constexpr int kLanes = 64;      // lanes over channels
constexpr int kAhead = 4;       // tokens that are loaded while as many are computed
constexpr int kBwdWaves = 4;    // waves of a backward work-group, along the tokens
constexpr int kMaxTaps = 4;
constexpr int kLeastRun = 8;

struct ConvArgs {
  mamba2_seqs q;
  int channels;
  int run;       // tokens of a unit (forward) or of a wave (backward)
  int units;
  int cblocks;   // blocks of kLanes channel vectors
  mamba2_rows x, y, d_y, d_x;
  const float* weight;
  const float* bias;
  const void* initial;   // [batch][taps - 1][channels]
  const void* d_final;
  void* final_state;
  void* d_initial;
  float* partial;        // [units][taps + 1][channels]
};

template <class T>
__device__ __forceinline__ float exp_of(float v) {
  if constexpr (sizeof(T) == 4) return expf(v);
  return __expf(v);  // a bf16 result keeps 8 bits
}

// 1 / (1 + e^-v); 0 for v = -inf.
template <class T>
__device__ __forceinline__ float sigmoid_of(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp_of<T>(-v));
}

template <int V, int W>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c0, float (&w)[W][V], float (&b)[V]) {
  // a lane's V * W weights lie in a row
  const float* p = a.weight + static_cast<long>(c0) * W;
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = p[i * W + k];
    b[i] = a.bias != nullptr ? a.bias[c0 + i] : 0.0f;
  }
}

// Input `p` of a sequence for p < len, from the initial state for p < 0.
template <class T, int V, int W>
__device__ __forceinline__ void load_input(const ConvArgs& a, const T* xs, int seq, int p, int c0, float (&v)[V]) {
  if (p >= 0) {
    load_vec<T, V>(xs + p * a.x.row_stride + c0, v);
  } else if (a.initial != nullptr) {
    load_vec<T, V>(static_cast<const T*>(a.initial) +
                       (static_cast<long>(seq) * (W - 1) + (W - 1 + p)) * a.channels + c0, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
  }
}

// V elements as they lie in memory, loaded through a buffer resource that
// starts at a run's first row: the lane's channel is one offset register, the
// token a scalar one, so a row costs one instruction.
template <class T, int V>
struct Raw {
  typedef typename Vec<T>::type vec;
  vec v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int lane_off, int row_off) {
    v = __builtin_bit_cast(vec, __builtin_amdgcn_raw_buffer_load_b128(rs, lane_off, row_off, 0));
  }
  __device__ __forceinline__ float get(int i) const { return static_cast<float>(v[i]); }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int lane_off, int row_off) {
    v = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, lane_off, row_off, 0));
  }
  __device__ __forceinline__ float get(int) const { return v; }
};
template <>
struct Raw<bf16, 4> {
  v4bf v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int lane_off, int row_off) {
    v = __builtin_bit_cast(v4bf, __builtin_amdgcn_raw_buffer_load_b64(rs, lane_off, row_off, 0));
  }
  __device__ __forceinline__ float get(int i) const { return static_cast<float>(v[i]); }
};
template <>
struct Raw<bf16, 1> {
  unsigned short v;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int lane_off, int row_off) {
    v = static_cast<unsigned short>(__builtin_amdgcn_raw_buffer_load_b16(rs, lane_off, row_off, 0));
  }
  __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<unsigned>(v) << 16); }
};
// The rows of a run are only ever addressed inside the tensor, so the
// resource needs no end.
template <class T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t run_rsrc(const T* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(static_cast<const void*>(p)), 0, 0x7fffffff, 0x00020000);
}
// A store's row goes into the lane's offset, not into a scalar one: a 16-byte
// store that takes a scalar offset reads its data registers late, the compiler
// counts on it not to, and an instruction right behind that writes them changed
// the first 8 bytes that lanes 12 .. 15 of every 16 stored, now and then, when
// the memory was busy.  Without one the compiler keeps the distance.  One
// addition per row, which no measurement shows.
template <class T, int V>
__device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t rs, int lane_off, int row_off, const float (&v)[V]) {
  const int off = lane_off + row_off;
  if constexpr (V == 1) {
    const T t = static_cast<T>(v[0]);
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, t), rs, off, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(t), rs, off, 0, 0);
  } else if constexpr (V != Vec<T>::n) {
    v4bf r;
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = static_cast<T>(v[i]);
    typedef int v2i __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2i, r), rs, off, 0, 0);
  } else {
    typename Vec<T>::type r;
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = static_cast<T>(v[i]);
    typedef int v4i __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4i, r), rs, off, 0, 0);
  }
}

// The window of the last W inputs moves on by one token.
template <class T, int V, int W>
__device__ __forceinline__ void shift(float (&win)[W][V], const Raw<T, V>& next) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
    win[W - 1][i] = next.get(i);
  }
}

// Bound by HBM in long calls and by the number of waves in short ones (9
// prompts of 5515 tokens, 2304 channels: 16 us).  A lane has a run's whole
// window, so no LDS and no exchange between lanes are needed.
// Blocks 0 .. units * cblocks - 1 each compute a run of tokens; the blocks
// behind them copy the sequences' last W - 1 inputs to final_state.
template <class T, int V, int W, bool SILU>
__global__ __launch_bounds__(kLanes) void conv_fwd_kernel(ConvArgs a) {
  const int cb = blockIdx.x % a.cblocks;
  const int unit = blockIdx.x / a.cblocks;
  const int c0 = (cb * kLanes + threadIdx.x) * V;
  const bool packed = a.q.offsets != nullptr;
  if (unit >= a.units) {
    if (c0 >= a.channels) return;
    const int s = unit - a.units;
    long row0;
    int len;
    seq_rows(a.q, s, &row0, &len);
    const T* xs = seq_ptr<const T>(a.x, s, row0, packed);
    T* out = static_cast<T*>(a.final_state) + static_cast<long>(s) * (W - 1) * a.channels + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      load_input<T, V, W>(a, xs, s, len - (W - 1) + j, c0, v);
      store_vec<T, V>(out + static_cast<long>(j) * a.channels, v);
    }
    return;
  }
  const Unit u = locate(a.q, unit, a.run);
  if (u.t0 >= u.len || c0 >= a.channels) return;
  const T* xs = seq_ptr<const T>(a.x, u.seq, u.row0, packed);
  const int rows = min(a.run, u.len - u.t0);
  const auto rx = run_rsrc(xs + u.t0 * a.x.row_stride);
  const auto ry = run_rsrc(seq_ptr<T>(a.y, u.seq, u.row0, packed) + u.t0 * a.y.row_stride);
  const int lane_off = c0 * static_cast<int>(sizeof(T));
  const int sx = static_cast<int>(a.x.row_stride * sizeof(T)), sy = static_cast<int>(a.y.row_stride * sizeof(T));
  Raw<T, V> now[kAhead], next[kAhead];
  const auto fetch = [&](Raw<T, V> (&r)[kAhead], int t) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (t + j < rows) r[j].load(rx, lane_off, (t + j) * sx);
  };
  fetch(now, 0);
  float w[W][V], b[V], win[W][V];
  load_weights<V, W>(a, c0, w, b);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_input<T, V, W>(a, xs, u.seq, u.t0 - (W - 1) + j, c0, win[j + 1]);
  for (int t = 0; t < rows; t += kAhead) {
    if (t + kAhead < rows) fetch(next, t + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (t + j < rows) {
        float y[V];
        shift<T, V, W>(win, now[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float s = b[i];
#pragma unroll
          for (int k = 0; k < W; ++k) s = fmaf(w[k][i], win[k][i], s);
          y[i] = SILU ? s * sigmoid_of<T>(s) : s;
        }
        put<T, V>(ry, lane_off, (t + j) * sy, y);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) now[j] = next[j];
  }
}

// dp_t for one token: win holds the inputs t - W + 1 .. t.
template <class T, int V, int W, bool SILU>
__device__ __forceinline__ void pre_grad(const float (&w)[W][V], const float (&b)[V], const float (&win)[W][V],
                                         const float (&dy)[V], float (&dp)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (SILU) {
      float s = b[i];
#pragma unroll
      for (int k = 0; k < W; ++k) s = fmaf(w[k][i], win[k][i], s);
      const float g = sigmoid_of<T>(s);
      dp[i] = dy[i] * (g * fmaf(s, 1.0f - g, 1.0f));
    } else {
      dp[i] = dy[i];
    }
  }
}

// A work-group's waves take neighbouring runs of one unit, and their sums of
// the weights' gradients meet in LDS, so that a unit leaves one partial per
// channel and tap; the blocks behind the units compute d_initial_state.  The
// pre-activation is recomputed from x: a saved one would be another tensor to
// read.  W - 1 tokens behind the run are loaded and differentiated again, 3 in
// 36 at the size above.
template <class T, int V, int W, bool SILU>
__global__ __launch_bounds__(kLanes * kBwdWaves, sizeof(T) == 2 ? 4 : 2) void conv_bwd_kernel(ConvArgs a) {
  __shared__ float lds[kBwdWaves][kLanes * V];
  const int lane = threadIdx.x % kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int cb = blockIdx.x % a.cblocks;
  const int unit = blockIdx.x / a.cblocks;
  const int c0 = (cb * kLanes + lane) * V;
  const bool live = c0 < a.channels;
  const bool packed = a.q.offsets != nullptr;

  if (unit >= a.units) {
    if (!live || wave != 0) return;
    const int s = unit - a.units;
    long row0;
    int len;
    seq_rows(a.q, s, &row0, &len);
    const T* xs = seq_ptr<const T>(a.x, s, row0, packed);
    const T* gs = seq_ptr<const T>(a.d_y, s, row0, packed) + c0;
    float w[W][V], b[V], win[W][V], dp[W - 1][V];
    load_weights<V, W>(a, c0, w, b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_input<T, V, W>(a, xs, s, j - (W - 1), c0, win[j + 1]);
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
#pragma unroll
      for (int i = 0; i < V; ++i) dp[t][i] = 0.0f;
      if (t < len) {
        float dy[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int k = 0; k < W - 1; ++k) win[k][i] = win[k + 1][i];
        load_input<T, V, W>(a, xs, s, t, c0, win[W - 1]);
        load_vec<T, V>(gs + t * a.d_y.row_stride, dy);
        pre_grad<T, V, W, SILU>(w, b, win, dy, dp[t]);
      }
    }
    T* out = static_cast<T*>(a.d_initial) + static_cast<long>(s) * (W - 1) * a.channels + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {  // input u = j - (W - 1) < 0
      float v[V];
      const int f = j - len;  // its place in final_state, if it is still among the last W - 1
      if (a.d_final != nullptr && f >= 0) {
        load_vec<T, V>(static_cast<const T*>(a.d_final) + (static_cast<long>(s) * (W - 1) + f) * a.channels + c0, v);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k <= j; ++k)  // output t = j - k >= 0
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaf(w[k][i], dp[j - k][i], v[i]);
      store_vec<T, V>(out + static_cast<long>(j) * a.channels, v);
    }
    return;
  }

  float dw[W][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][i] = 0.0f;
  }
  const Unit u = locate(a.q, unit, a.run * kBwdWaves);
  const int first = u.t0 + wave * a.run;
  if (live && first < u.len) {
    const T* xs = seq_ptr<const T>(a.x, u.seq, u.row0, packed);
    const int rows = min(a.run, u.len - first);              // the weights' gradients take these tokens,
    const int last = min(rows + W - 1, u.len - first);       // d_x the W - 1 behind them too
    const auto rx = run_rsrc(xs + first * a.x.row_stride);
    const auto rg = run_rsrc(seq_ptr<const T>(a.d_y, u.seq, u.row0, packed) + first * a.d_y.row_stride);
    const auto ro = run_rsrc(seq_ptr<T>(a.d_x, u.seq, u.row0, packed) + first * a.d_x.row_stride);
    const int lane_off = c0 * static_cast<int>(sizeof(T));
    const int sx = static_cast<int>(a.x.row_stride * sizeof(T)), sg = static_cast<int>(a.d_y.row_stride * sizeof(T)),
              so = static_cast<int>(a.d_x.row_stride * sizeof(T));
    Raw<T, V> nx[kAhead], ng[kAhead], mx[kAhead], mg[kAhead];
    const auto fetch = [&](Raw<T, V> (&x)[kAhead], Raw<T, V> (&gr)[kAhead], int t) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (t + j < last) {
          x[j].load(rx, lane_off, (t + j) * sx);
          gr[j].load(rg, lane_off, (t + j) * sg);
        }
      }
    };
    fetch(nx, ng, 0);
    float w[W][V], b[V], win[W][V], dpw[W][V];
    load_weights<V, W>(a, c0, w, b);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_input<T, V, W>(a, xs, u.seq, first - (W - 1) + j, c0, win[j + 1]);
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) dpw[k][i] = 0.0f;
    for (int t = 0; t < rows + W - 1; t += kAhead) {
      fetch(mx, mg, t + kAhead);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int tt = t + j;
        if (tt < rows + W - 1) {
          float dp[V];
          if (tt < last) {
            float dy[V];
            shift<T, V, W>(win, nx[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) dy[i] = ng[j].get(i);
            pre_grad<T, V, W, SILU>(w, b, win, dy, dp);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) dp[i] = 0.0f;
          }
          if (tt < rows) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              db[i] += dp[i];
#pragma unroll
              for (int k = 0; k < W; ++k) dw[k][i] = fmaf(dp[i], win[k][i], dw[k][i]);
            }
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {  // dpw[k] = dp of token tt - k
#pragma unroll
            for (int k = W - 1; k > 0; --k) dpw[k][i] = dpw[k - 1][i];
            dpw[0][i] = dp[i];
          }
          const int o = tt - (W - 1);
          if (o >= 0 && a.d_x.data != nullptr) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.0f;
            const int f = first + o - u.len + (W - 1);
            if (a.d_final != nullptr && f >= 0)
              load_vec<T, V>(static_cast<const T*>(a.d_final) +
                                 (static_cast<long>(u.seq) * (W - 1) + f) * a.channels + c0, v);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
              for (int k = 0; k < W; ++k) v[i] = fmaf(w[k][i], dpw[k][i], v[i]);
            put<T, V>(ro, lane_off, o * so, v);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        nx[j] = mx[j];
        ng[j] = mg[j];
      }
    }
  }
  if (a.partial == nullptr) return;
  // The waves' sums meet in LDS, one quantity at a time, in a fixed order.
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) lds[wave][lane * V + i] = k < W ? dw[k < W ? k : 0][i] : db[i];
    __syncthreads();
    for (int i = threadIdx.x; i < kLanes * V; i += kLanes * kBwdWaves) {
      const int c = cb * kLanes * V + i;
      if (c < a.channels) {
        float s = lds[0][i];
#pragma unroll
        for (int v = 1; v < kBwdWaves; ++v) s += lds[v][i];
        a.partial[(static_cast<long>(unit) * (W + 1) + k) * a.channels + c] = s;
      }
    }
  }
}

// 5.9 us for 116 units of 4352 channels and 5 sums each (10 MB), most of it the
// launch.  Sums the units' partials of one (tap or bias, channel) in a fixed order:
// lanes over channels, four waves over the units.
__global__ __launch_bounds__(256) void conv_reduce_kernel(const float* partial, int units, int channels, int taps,
                                                          float* d_weight, float* d_bias) {
  __shared__ float lds[4][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int c = blockIdx.x * 64 + lane;
  const int k = blockIdx.y;
  float s = 0.0f;
  if (c < channels) {
    const float* p = partial + static_cast<long>(k) * channels + c;
    const long step = static_cast<long>(taps + 1) * channels;
#pragma unroll 8
    for (int u = wave; u < units; u += 4) s += p[u * step];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= channels) return;
  s = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
  if (k < taps) {
    if (d_weight != nullptr) d_weight[static_cast<long>(c) * taps + k] = s;
  } else if (d_bias != nullptr) {
    d_bias[c] = s;
  }
}

// One token: bound by the launch (16 sequences of 2304 channels, 0.6 MB: 3 us).
// The window is read before it is written, so new_state may be state itself.
template <class T, int V, int W, bool SILU>
__global__ __launch_bounds__(kLanes) void conv_step_kernel(ConvArgs a) {
  const int c0 = (blockIdx.x * kLanes + threadIdx.x) * V;
  if (c0 >= a.channels) return;
  const int s = blockIdx.y;
  float w[W][V], b[V], win[W][V], y[V];
  const T* old = static_cast<const T*>(a.initial) + static_cast<long>(s) * (W - 1) * a.channels + c0;
  T* now = static_cast<T*>(a.final_state) + static_cast<long>(s) * (W - 1) * a.channels + c0;
  load_vec<T, V>(static_cast<const T*>(a.x.data) + s * a.x.batch_stride + c0, win[W - 1]);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<T, V>(old + static_cast<long>(j) * a.channels, win[j]);
  load_weights<V, W>(a, c0, w, b);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = b[i];
#pragma unroll
    for (int k = 0; k < W; ++k) v = fmaf(w[k][i], win[k][i], v);
    y[i] = SILU ? v * sigmoid_of<T>(v) : v;
  }
  store_vec<T, V>(static_cast<T*>(a.y.data) + s * a.y.batch_stride + c0, y);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<T, V>(now + static_cast<long>(j) * a.channels, win[j + 1]);
}

// --------------------------------------------------------------------- host
enum Which { kFwd, kBwd, kStep };

// Channels of a backward lane.  The windows, weights and sums of eight take 254
// registers, two waves on a SIMD; four with 8-byte accesses take 128, four waves:
// 94 us against 113 (4 x 4096 tokens of 4352 channels).
constexpr int bwd_vec(int v) { return v > 4 ? 4 : v; }

template <class T, int V, int W, bool SILU>
void launch(Which which, const ConvArgs& a, dim3 grid, hipStream_t s) {
  switch (which) {
    case kFwd: conv_fwd_kernel<T, V, W, SILU><<<grid, kLanes, 0, s>>>(a); break;
    case kBwd: conv_bwd_kernel<T, bwd_vec(V), W, SILU><<<grid, kLanes * kBwdWaves, 0, s>>>(a); break;
    case kStep: conv_step_kernel<T, V, W, SILU><<<grid, kLanes, 0, s>>>(a); break;
  }
}

template <class T, int V, int W>
void launch_act(Which which, int silu, const ConvArgs& a, dim3 grid, hipStream_t s) {
  if (silu) launch<T, V, W, true>(which, a, grid, s); else launch<T, V, W, false>(which, a, grid, s);
}

template <class T, int V>
void launch_taps(Which which, int taps, int silu, const ConvArgs& a, dim3 grid, hipStream_t s) {
  switch (taps) {
    case 2: launch_act<T, V, 2>(which, silu, a, grid, s); break;
    case 3: launch_act<T, V, 3>(which, silu, a, grid, s); break;
    default: launch_act<T, V, 4>(which, silu, a, grid, s); break;
  }
}

void launch_conv(Which which, int type, bool vec, int taps, int silu, const ConvArgs& a, dim3 grid, hipStream_t s) {
  if (type == MAMBA2_F32) {
    if (vec) launch_taps<float, 4>(which, taps, silu, a, grid, s);
    else launch_taps<float, 1>(which, taps, silu, a, grid, s);
  } else {
    if (vec) launch_taps<bf16, 8>(which, taps, silu, a, grid, s);
    else launch_taps<bf16, 1>(which, taps, silu, a, grid, s);
  }
}

int check_conv(int type, const mamba2_seqs& q, int channels, int taps) {
  if (!type_ok(type)) return MAMBA2_SCAN_EUNSUPPORTED;
  const int st = check_seqs(q);
  if (st != MAMBA2_SCAN_OK) return st;
  if (channels < 1 || channels > (1 << 22)) return MAMBA2_SCAN_EBADDIM;
  if (taps < 2 || taps > kMaxTaps) return MAMBA2_SCAN_EUNSUPPORTED;
  return MAMBA2_SCAN_OK;
}

// A run's rows are addressed with 31-bit offsets from its first.
bool strides_ok(const mamba2_rows& r) { return r.row_stride <= (1 << 22); }

long long total_rows(const mamba2_seqs& q) {
  return static_cast<long long>(q.length) * (q.offsets != nullptr ? 1 : q.batch);
}

// Tokens per run: enough waves to fill the chip first, then longer runs, which
// re-read fewer meeting tokens.  Measured at 4 x 4096 tokens of 4352 channels:
// forward runs of 64 tokens 55 us, of 32 60 us; backward runs of 36 94 us, of 32
// 96 us; of 8 twice that (more partial sums).
int run_tokens(const mamba2_seqs& q, int channels, int waves_per_cu, int most) {
  const long long tokens = total_rows(q) * ((channels + 511) / 512);
  const long long r = (tokens / (kCUs * waves_per_cu) + kAhead - 1) / kAhead * kAhead;
  return static_cast<int>(r < kLeastRun ? kLeastRun : r > most ? most : r);
}
int fwd_run(const mamba2_seqs& q, int channels) { return run_tokens(q, channels, 8, 64); }
int bwd_run(const mamba2_seqs& q, int channels) { return run_tokens(q, channels, 16, 64); }

int cblocks_of(Which which, int type, bool vec, int channels) {
  const int v = vec ? (type == MAMBA2_BF16 ? 8 : 4) : 1, per = kLanes * (which == kBwd ? bwd_vec(v) : v);
  return (channels + per - 1) / per;
}

bool state_vec(const void* p) { return aligned_to(p, 16); }

}  // namespace

extern "C" {

int mamba2_conv_fwd(int type, mamba2_seqs q, int channels, int taps, int silu, mamba2_rows x, const float* weight,
                    const float* bias, const void* initial_state, mamba2_rows y, void* final_state, void* stream) {
  int st = check_conv(type, q, channels, taps);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(type);
  if (weight == nullptr) return MAMBA2_SCAN_ENULL;
  x = used_strides(x, q, channels);
  y = used_strides(y, q, channels);
  if ((st = check_rows(x, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if ((st = check_rows(y, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(initial_state, e) || !aligned_to(final_state, e))
    return MAMBA2_SCAN_EALIGN;
  if (!strides_ok(x) || !strides_ok(y)) return MAMBA2_SCAN_EUNSUPPORTED;
  const bool vec = channels % (16 / static_cast<int>(e)) == 0 && rows_vec(x, e) && rows_vec(y, e) &&
                   state_vec(initial_state) && state_vec(final_state);
  ConvArgs a = {};
  a.q = q;
  a.channels = channels;
  a.run = fwd_run(q, channels);
  a.units = static_cast<int>(unit_count(q, a.run));
  a.cblocks = cblocks_of(kFwd, type, vec, channels);
  a.x = x;
  a.y = y;
  a.weight = weight;
  a.bias = bias;
  a.initial = initial_state;
  a.final_state = final_state;
  const long long blocks = (static_cast<long long>(a.units) + (final_state != nullptr ? q.batch : 0)) * a.cblocks;
  if (blocks == 0) return MAMBA2_SCAN_OK;
  if (!grid_ok(blocks, kLanes)) return MAMBA2_SCAN_EBADDIM;
  launch_conv(kFwd, type, vec, taps, silu, a, dim3(static_cast<unsigned>(blocks)), static_cast<hipStream_t>(stream));
  return launch_status();
}

size_t mamba2_conv_bwd_workspace_bytes(mamba2_seqs q, int channels, int taps) {
  if (check_conv(MAMBA2_F32, q, channels, taps) != MAMBA2_SCAN_OK) return 0;
  const long units = unit_count(q, bwd_run(q, channels) * kBwdWaves);
  const size_t n = static_cast<size_t>(units > 0 ? units : 1) * (taps + 1) * channels * sizeof(float);
  return (n + 15) / 16 * 16;
}

int mamba2_conv_bwd(int type, mamba2_seqs q, int channels, int taps, int silu, mamba2_rows x, const float* weight,
                    const float* bias, const void* initial_state, mamba2_rows d_y, const void* d_final_state,
                    mamba2_rows d_x, float* d_weight, float* d_bias, void* d_initial_state, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = check_conv(type, q, channels, taps);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(type);
  const bool sums = d_weight != nullptr || d_bias != nullptr;
  if (weight == nullptr) return MAMBA2_SCAN_ENULL;
  if (d_x.data == nullptr && !sums && d_initial_state == nullptr) return MAMBA2_SCAN_ENULL;
  x = used_strides(x, q, channels);
  d_y = used_strides(d_y, q, channels);
  d_x = used_strides(d_x, q, channels);
  if ((st = check_rows(x, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if ((st = check_rows(d_y, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if (d_x.data != nullptr && (st = check_rows(d_x, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if (sums) {
    if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
    if (workspace_bytes < mamba2_conv_bwd_workspace_bytes(q, channels, taps)) return MAMBA2_SCAN_ESIZE;
    if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  }
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(d_weight, 4) || !aligned_to(d_bias, 4) ||
      !aligned_to(initial_state, e) || !aligned_to(d_final_state, e) || !aligned_to(d_initial_state, e))
    return MAMBA2_SCAN_EALIGN;
  if (!strides_ok(x) || !strides_ok(d_y) || (d_x.data != nullptr && !strides_ok(d_x))) return MAMBA2_SCAN_EUNSUPPORTED;
  const bool vec = channels % (16 / static_cast<int>(e)) == 0 && rows_vec(x, e) && rows_vec(d_y, e) &&
                   (d_x.data == nullptr || rows_vec(d_x, e)) && state_vec(initial_state) && state_vec(d_final_state) &&
                   state_vec(d_initial_state);
  hipStream_t s = static_cast<hipStream_t>(stream);
  ConvArgs a = {};
  a.q = q;
  a.channels = channels;
  a.run = bwd_run(q, channels);
  a.units = static_cast<int>(unit_count(q, a.run * kBwdWaves));
  a.cblocks = cblocks_of(kBwd, type, vec, channels);
  a.x = x;
  a.d_y = d_y;
  a.d_x = d_x;
  a.weight = weight;
  a.bias = bias;
  a.initial = initial_state;
  a.d_final = d_final_state;
  a.d_initial = d_initial_state;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  const long long blocks = (static_cast<long long>(a.units) + (d_initial_state != nullptr ? q.batch : 0)) * a.cblocks;
  if (!grid_ok(blocks, kLanes * kBwdWaves)) return MAMBA2_SCAN_EBADDIM;
  if (blocks > 0) {
    launch_conv(kBwd, type, vec, taps, silu, a, dim3(static_cast<unsigned>(blocks)), s);
    if ((st = launch_status()) != MAMBA2_SCAN_OK) return st;
  }
  if (sums) {
    conv_reduce_kernel<<<dim3((channels + 63) / 64, taps + 1), 256, 0, s>>>(a.partial, a.units, channels, taps,
                                                                           d_weight, d_bias);
    st = launch_status();
  }
  return st;
}

int mamba2_conv_step(int type, int batch, int channels, int taps, int silu, mamba2_rows x, const float* weight,
                     const float* bias, const void* state, mamba2_rows y, void* new_state, void* stream) {
  const mamba2_seqs q = {batch, 1, nullptr};
  int st = check_conv(type, q, channels, taps);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(type);
  if (weight == nullptr || state == nullptr || new_state == nullptr) return MAMBA2_SCAN_ENULL;
  if (batch > 65535) return MAMBA2_SCAN_EBADDIM;
  x.row_stride = y.row_stride = 0;
  if ((st = check_rows(x, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if ((st = check_rows(y, q, channels, e)) != MAMBA2_SCAN_OK) return st;
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(state, e) || !aligned_to(new_state, e))
    return MAMBA2_SCAN_EALIGN;
  const long long row = static_cast<long long>(channels) * static_cast<long long>(e), tail = batch * (taps - 1) * row;
  const Region mem[] = {token_region(y, batch, channels, e), region(new_state, tail), token_region(x, batch, channels, e),
                        region(weight, 4LL * channels * taps), region(bias, 4LL * channels),
                        region(state != new_state ? state : nullptr, tail)};
  if (!apart(mem, 2, 6)) return MAMBA2_SCAN_EOVERLAP;
  const bool vec = channels % (16 / static_cast<int>(e)) == 0 && rows_vec(x, e) && rows_vec(y, e) &&
                   state_vec(state) && state_vec(new_state);
  ConvArgs a = {};
  a.channels = channels;
  a.cblocks = cblocks_of(kStep, type, vec, channels);
  a.x = x;
  a.y = y;
  a.weight = weight;
  a.bias = bias;
  a.initial = state;
  a.final_state = new_state;
  launch_conv(kStep, type, vec, taps, silu, a, dim3(a.cblocks, batch), static_cast<hipStream_t>(stream));
  return launch_status();
}

}  // extern "C"
