// The global 2-norm of many gradient tensors, and clipping by it, for gfx950.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g min(1, max_norm / (norm + 1e-6))
//
// Bound by HBM: every gradient is read for the norm and read again to be
// scaled (the factor is known only after the last square), and written once.
// Two launches per table of tensors: each block sums the squares of its piece
// of one tensor into one partial; each block of the second launch adds up all
// partials itself, in a fixed order, instead of waiting for a third launch.
// 60 tensors of 617 MB in all: squares 102 us (6.0 TB/s: the last call's tail is in
// the cache), scaling 230 us (5.4 TB/s); a large copy reaches 5.1.  Small calls
// take two launches' time, 4 and 5 us.
// The number of blocks is held near kBlocks so that those partials stay few.
// The second pass walks the pieces backwards: what the first pass read last
// is still in the 256 MB cache.
#include <stdlib.h>

#include <algorithm>

#include "layer_common.h"

namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kTable = 96;              // tensors per launch: the table travels as kernel arguments (< 4 KB)
constexpr int kFew = 16;                // up to so many take a smaller table: 1.1 us less of a call's host time (1 tensor
                                        // 10.2 us against 11.3, 14 tensors 20.5 against 21.6; on the GPU the same)
constexpr long long kPiece = 8192;      // smallest piece of a tensor given to one block
constexpr long long kBlocks = 4096;     // blocks to aim for (1024: 376 us for 617 MB of gradients, 2048: 336, 4096: 322)

struct Entry {
  const void* grad;
  void* out;
  long long numel;
  int type;
  int first;  // first block of the tensor within the launch
};

template <int N>
struct Table {
  Entry e[N];
  int count;
  int blocks;
  long long piece;  // elements per block
};
static_assert(sizeof(Table<kTable>) <= 4000, "the table travels as kernel arguments");

template <int N>
__device__ __forceinline__ int entry_of(const Table<N>& t, int block) {
  int lo = 0, hi = t.count;  // the last entry with first <= block (empty tensors have no block)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first <= block) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
  __syncthreads();
  double s = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s += lds[w];
  return s;
}

// f(i) for single elements, g(i, v) for the 16-byte vector v at element i of
// [lo, hi), relative to a pointer that is only element-aligned.  kAhead
// vectors of a thread are loaded before the first is used.
constexpr int kAhead = 8;
template <class T, class F, class G>
__device__ __forceinline__ void for_span(const T* p, long lo, long hi, F f, G g) {
  typedef typename Vec<T>::type vec;
  constexpr int n = Vec<T>::n;
  constexpr long step = static_cast<long>(kThreads) * n;
  const long head = min<long>(hi, lo + ((16 - (reinterpret_cast<uintptr_t>(p + lo) & 15)) & 15) / sizeof(T));
  for (long i = lo + threadIdx.x; i < head; i += kThreads) f(i);
  const long body = head + (hi - head) / n * n;
  long i = head + static_cast<long>(threadIdx.x) * n;
  for (; i + (kAhead - 1) * step < body; i += kAhead * step) {
    vec v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) v[j] = *reinterpret_cast<const vec*>(p + i + j * step);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) g(i + j * step, v[j]);
  }
  for (; i < body; i += step) g(i, *reinterpret_cast<const vec*>(p + i));
  for (i = body + threadIdx.x; i < hi; i += kThreads) f(i);
}

template <class T>
__device__ __forceinline__ double squares(const void* grad, long lo, long hi) {
  const T* p = static_cast<const T*>(grad);
  // 64-bit sums: no square of a finite fp32 overflows, and the sum of any
  // number of them is right to fp32's last bit
  double s = 0.0, t[4] = {0.0, 0.0, 0.0, 0.0};
  for_span<T>(p, lo, hi,
              [&](long i) {
                const double v = static_cast<float>(p[i]);
                s = fma(v, v, s);
              },
              [&](long, typename Vec<T>::type v) {
#pragma unroll
                for (int j = 0; j < Vec<T>::n; ++j) {
                  const double d = static_cast<float>(v[j]);
                  t[j & 3] = fma(d, d, t[j & 3]);
                }
              });
  return ((t[0] + t[1]) + (t[2] + t[3])) + s;
}

template <int N>
__global__ __launch_bounds__(kThreads) void grad_squares_kernel(Table<N> t, double* partial) {
  __shared__ double lds[kThreads / 64];
  const Entry& e = t.e[entry_of(t, blockIdx.x)];
  const long lo = (blockIdx.x - e.first) * t.piece;
  const long hi = min(lo + t.piece, e.numel);
  const double s = e.type == MAMBA2_BF16 ? squares<bf16>(e.grad, lo, hi) : squares<float>(e.grad, lo, hi);
  const double all = block_sum(s, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = all;
}

__device__ __forceinline__ double total(const double* partial, int n, double* lds) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  return block_sum(s, lds);
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* partial, int n, float* norm) {
  __shared__ double lds[kThreads / 64];
  const double s = total(partial, n, lds);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

template <class T>
__device__ __forceinline__ void scale(const Entry& e, long lo, long hi, float f) {
  const T* p = static_cast<const T*>(e.grad);
  T* o = static_cast<T*>(e.out);
  constexpr int n = Vec<T>::n;
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    for_span<T>(p, lo, hi, [&](long i) { o[i] = static_cast<T>(static_cast<float>(p[i]) * f); },
                [&](long i, typename Vec<T>::type v) {
                  typename Vec<T>::type r;
#pragma unroll
                  for (int j = 0; j < n; ++j) r[j] = static_cast<T>(static_cast<float>(v[j]) * f);
                  __builtin_nontemporal_store(r, reinterpret_cast<typename Vec<T>::type*>(o + i));
                });
  } else {  // grad and out cannot both be accessed in vectors
    for (long i = lo + threadIdx.x; i < hi; i += kThreads) o[i] = static_cast<T>(static_cast<float>(p[i]) * f);
  }
}

template <int N>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Table<N> t, const double* partial, int n, float max_norm,
                                                              float* norm) {
  __shared__ double lds[kThreads / 64];
  const double r = sqrt(total(partial, n, lds));
  const int block = t.blocks - 1 - static_cast<int>(blockIdx.x);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(r);
  // the factor stays right where norm overflows fp32; NaN passes through the comparison
  const double q = static_cast<double>(max_norm) / (r + 1e-6);
  const float f = q >= 1.0 || (isinf(max_norm) && r == r) ? 1.0f : static_cast<float>(q);
  const Entry& e = t.e[entry_of(t, block)];
  if (f == 1.0f && e.out == e.grad) return;  // in place, nothing to clip
  const long lo = (block - e.first) * t.piece;
  const long hi = min(lo + t.piece, e.numel);
  if (e.type == MAMBA2_BF16) scale<bf16>(e, lo, hi, f); else scale<float>(e, lo, hi, f);
}

// --------------------------------------------------------------------- host
struct Sizes {
  long long piece;
  long long blocks;
};

int check_grads(const mamba2_grad* g, int count, bool clip, Sizes* out) {
  if (count < 1) return MAMBA2_SCAN_EBADDIM;
  if (g == nullptr) return MAMBA2_SCAN_ENULL;
  long long sum = 0;
  for (int i = 0; i < count; ++i) {
    if (!type_ok(g[i].type)) return MAMBA2_SCAN_EUNSUPPORTED;
    if (g[i].numel < 0 || g[i].numel >= (1LL << 46) || (sum += g[i].numel) >= (1LL << 46)) return MAMBA2_SCAN_EBADDIM;
  }
  for (int i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    if (g[i].grad == nullptr || (clip && g[i].out == nullptr)) return MAMBA2_SCAN_ENULL;
    if (!aligned_to(g[i].grad, type_size(g[i].type)) || (clip && !aligned_to(g[i].out, type_size(g[i].type))))
      return MAMBA2_SCAN_EALIGN;
  }
  long long piece = (sum + kBlocks - 1) / kBlocks;
  piece = (piece + kPiece - 1) / kPiece * kPiece;
  if (piece < kPiece) piece = kPiece;
  out->piece = piece;
  out->blocks = 0;
  for (int i = 0; i < count; ++i) out->blocks += (g[i].numel + piece - 1) / piece;
  if (out->blocks > 2147483647LL) return MAMBA2_SCAN_EBADDIM;
  return MAMBA2_SCAN_OK;
}

struct Span {
  uintptr_t lo, hi;
};

// Does the norm or the workspace overlap the other or a gradient?  (Gradients
// that are only read may overlap.)
int check_norm_apart(const mamba2_grad* g, int count, const float* norm, const void* workspace, size_t workspace_bytes) {
  const Region r = region(norm, sizeof(float)), w = region(workspace, static_cast<long long>(workspace_bytes));
  bool apart = !overlap(r, w);
  for (int i = 0; i < count; ++i) {
    const Region v = region(g[i].grad, g[i].numel * static_cast<long long>(type_size(g[i].type)));
    apart = apart && (g[i].numel == 0 || (!overlap(v, r) && !overlap(v, w)));
  }
  return apart ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EOVERLAP;
}

// Does any gradient or output overlap another?  The second pass writes while
// the first one's other tensors are still to be scaled, so each must be apart.
int check_apart(const mamba2_grad* g, int count, const float* norm, const void* workspace, size_t workspace_bytes) {
  const size_t most = 2 * static_cast<size_t>(count) + 2;
  Span few[256];
  Span* spans = few;
  if (most > 256) {
    spans = static_cast<Span*>(malloc(most * sizeof(Span)));
    if (spans == nullptr) return MAMBA2_SCAN_EHIP;
  }
  const uintptr_t pn = reinterpret_cast<uintptr_t>(norm), pw = reinterpret_cast<uintptr_t>(workspace);
  spans[0] = {pn, pn + sizeof(float)};
  spans[1] = {pw, pw + workspace_bytes};
  size_t n = 2;
  for (int i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    const size_t bytes = static_cast<size_t>(g[i].numel) * type_size(g[i].type);
    const uintptr_t p = reinterpret_cast<uintptr_t>(g[i].grad), o = reinterpret_cast<uintptr_t>(g[i].out);
    spans[n++] = {p, p + bytes};
    if (o != p) spans[n++] = {o, o + bytes};
  }
  std::sort(spans, spans + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  bool apart = true;
  for (size_t i = 1; i < n; ++i) apart = apart && spans[i - 1].hi <= spans[i].lo;
  if (spans != few) free(spans);
  return apart ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EOVERLAP;
}

// Calls f(table, first block of the table) for each table of the list.
template <int N, class F>
int for_tables(const mamba2_grad* g, int count, const Sizes& sz, F f) {
  Table<N> t;
  t.count = 0;
  t.blocks = 0;
  t.piece = sz.piece;
  int before = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].numel != 0) {
      t.e[t.count++] = {g[i].grad, g[i].out, g[i].numel, g[i].type, t.blocks};
      t.blocks += static_cast<int>((g[i].numel + sz.piece - 1) / sz.piece);
    }
    if (t.count > 0 && (t.count == N || i == count - 1)) {
      f(t, before);
      const int st = launch_status();
      if (st != MAMBA2_SCAN_OK) return st;
      before += t.blocks;
      t.count = t.blocks = 0;
    }
  }
  return MAMBA2_SCAN_OK;
}

template <int N>
int run_squares(const mamba2_grad* g, int count, const Sizes& sz, void* workspace, hipStream_t s) {
  double* partial = static_cast<double*>(workspace);
  return for_tables<N>(g, count, sz, [&](const Table<N>& t, int before) {
    grad_squares_kernel<N><<<t.blocks, kThreads, 0, s>>>(t, partial + before);
  });
}

template <int N>
int run_clip(const mamba2_grad* g, int count, const Sizes& sz, float max_norm, float* norm, void* workspace,
             hipStream_t s) {
  const int st = run_squares<N>(g, count, sz, workspace, s);
  if (st != MAMBA2_SCAN_OK) return st;
  const double* partial = static_cast<const double*>(workspace);
  const int n = static_cast<int>(sz.blocks);
  if (n == 0) {  // every tensor is empty
    grad_norm_kernel<<<1, kThreads, 0, s>>>(partial, 0, norm);
    return launch_status();
  }
  return for_tables<N>(g, count, sz, [&](const Table<N>& t, int before) {
    grad_scale_kernel<N><<<t.blocks, kThreads, 0, s>>>(t, partial, n, max_norm, before == 0 ? norm : nullptr);
  });
}

int check_call(const mamba2_grad* g, int count, bool clip, const float* norm, const void* workspace,
               size_t workspace_bytes, Sizes* sz) {
  const int st = check_grads(g, count, clip, sz);
  if (st != MAMBA2_SCAN_OK) return st;
  if (norm == nullptr || workspace == nullptr) return MAMBA2_SCAN_ENULL;
  if (workspace_bytes < mamba2_grad_workspace_bytes(g, count)) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(norm, 4) || !aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  return MAMBA2_SCAN_OK;
}

}  // namespace

extern "C" {

size_t mamba2_grad_workspace_bytes(const mamba2_grad* grads, int count) {
  Sizes sz;
  if (check_grads(grads, count, false, &sz) != MAMBA2_SCAN_OK) return 0;
  return (static_cast<size_t>(sz.blocks) * sizeof(double) + 31) / 16 * 16;
}

int mamba2_grad_norm(const mamba2_grad* grads, int count, float* norm, void* workspace, size_t workspace_bytes,
                     void* stream) {
  Sizes sz;
  int st = check_call(grads, count, false, norm, workspace, workspace_bytes, &sz);
  if (st != MAMBA2_SCAN_OK) return st;
  if ((st = check_norm_apart(grads, count, norm, workspace, workspace_bytes)) != MAMBA2_SCAN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  st = count <= kFew ? run_squares<kFew>(grads, count, sz, workspace, s) : run_squares<kTable>(grads, count, sz, workspace, s);
  if (st != MAMBA2_SCAN_OK) return st;
  grad_norm_kernel<<<1, kThreads, 0, s>>>(static_cast<const double*>(workspace), static_cast<int>(sz.blocks), norm);
  return launch_status();
}

int mamba2_clip_grads(const mamba2_grad* grads, int count, float max_norm, float* norm, void* workspace,
                      size_t workspace_bytes, void* stream) {
  Sizes sz;
  if (!(max_norm >= 0.0f)) return MAMBA2_SCAN_EBADDIM;
  int st = check_call(grads, count, true, norm, workspace, workspace_bytes, &sz);
  if (st != MAMBA2_SCAN_OK) return st;
  if ((st = check_apart(grads, count, norm, workspace, workspace_bytes)) != MAMBA2_SCAN_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return count <= kFew ? run_clip<kFew>(grads, count, sz, max_norm, norm, workspace, s)
                       : run_clip<kTable>(grads, count, sz, max_norm, norm, workspace, s);
}

}  // extern "C"
