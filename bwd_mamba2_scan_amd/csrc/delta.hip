// Gated delta rule for gfx950: the forward over prompts and the single-token
// form.  The mathematics of a step is in delta_common.h.
//
// delta_prep_kernel: one work-group per step and group of heads writes the step's M
// and P as operands.  delta_fwd_kernel: a wave owns 16 columns of a head's state, S
// [states][16], in registers in fp32 as a matrix result, and walks the tokens
// in steps of 64; every product's result is the next one's right operand
// without leaving its lane, so waves meet only where they share the loads of a
// step's left operands (K, Q, M, P) through LDS.
#include "delta_common.h"
#include "delta_pair.h"
#include "delta_prep.h"
#include "delta_walk.h"

namespace {

using namespace delta;

// A work-group's time is mostly its chain: 16 rows of substitution, one behind the
// other, and the barriers between the inverse's halves; four work-groups on a CU hide
// one another's.  4 x 4096 tokens, 16 groups of two heads, 128 states, bf16: 79 us,
// 0.2 GB written (2.6 TB/s), the matrix pipes busy for 15% of it.  With every head's
// products of q and k formed anew 91 us.
template <class T, int NB>
__global__ __launch_bounds__(kPrepWaves * 64, prep_per_cu(sizeof(T), NB * 32)) void delta_prep_kernel(DeltaArgs a) {
  __shared__ PrepLds<T, NB> s;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const PrepWork w = prep_work(a);
  const Unit u = locate(a.seqs, w.step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  make_steps<T, NB, false>(s, a, u, w.step, w.first, w.heads, static_cast<T*>(a.p), [&](long cell) {
    put_pieces<false>(a.m + cell * kPieces * kPiece, s.sq.m, wave, lane);
  });
}

// A chain of steps: 4 x 4096 tokens, 32 heads of 128 x 128, bf16, a work-group on every
// CU: 278 us, 4.3 a step, LDS busy for 48% of it, the vector pipes for 38%, the matrix
// pipes for 33%.  fp32 (simple walks, 3 x 333 tokens, 10 heads of 24 x 40):
// 28 us, 4.7 a step.
template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_fwd_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairFwdLds<NB, kResults> s;
    pair_forward<NB, kResults>(a, s);
  } else {
    __shared__ FwdLds<T, NB, kResults> s;
    walk_forward<T, NB, kResults>(a, s);
  }
}

// What segments make of the states before them: a step costs 0.7 of delta_fwd_kernel's.
// One sequence of 32768 tokens, 24 heads of 64 x 64, ten segments: 192 us, beside 182
// of the walk itself and 12 of the carry.
template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_summary_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairFwdLds<NB, kSummary> s;
    pair_forward<NB, kSummary>(a, s);
  } else {
    __shared__ FwdLds<T, NB, kSummary> s;
    walk_forward<T, NB, kSummary>(a, s);
  }
}

// Turns the segments' own contributions into the states they start from, one
// segment of a sequence after the other: S = Phi S + own.  REVERSE: the gradients
// they end with, by the transposed Phi, from the last.  fp32 products throughout.
//
// A work-group has 16 columns, a wave 16 rows of them; the segments follow one
// another, so a wave's rows of the next one's Phi are loaded while this one is
// multiplied, and the waves meet once a segment, in LDS.  With a wave for all rows
// of 16 columns, 128 states took 13 us a segment, with this 1.
template <int NB, bool REVERSE>
__global__ __launch_bounds__(2 * NB * 64) void delta_carry_kernel(DeltaArgs a) {
  __shared__ v4f state[2][2 * NB][64];
  const int wave = wave_id(), lane = threadIdx.x & 63, l15 = lane & 15, g = lane >> 4;
  const int h = blockIdx.y, seq = blockIdx.z;
  long row0;
  int len;
  seq_rows(a.seqs, seq, &row0, &len);
  const int n = units_of(len, a.seg);
  if (n < 2) return;
  const long base = unit_base(a.seqs, seq, a.seg);
  const long head = static_cast<long>(a.states) * a.width, square = static_cast<long>(a.states) * a.states;
  const float* first = REVERSE ? a.d_final : a.initial;
  const float* phi = REVERSE ? a.seg_trans_t : a.seg_trans;
  float* places = REVERSE ? a.seg_grad : a.seg_state;
  // this lane's part of the wave's tile: column l15, rows 4 g ..
  const int col = blockIdx.x * 16 + l15, row = wave * 16 + 4 * g;
  const unsigned off = col < a.width ? static_cast<unsigned>((row * a.width + col) * 4) : kOutside;
  const unsigned bytes = static_cast<unsigned>(head * 4);
  const auto load = [&](const float* p) {
    const Rsrc rs = make_rsrc(p, bytes);
    v4f v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load_elem<float>(rs, off + i * 4 * a.width);
    return v;
  };
  Frag<float> f[NB];
  v4f own;
  const auto fetch = [&](int i) {  // the place that segment step i fills, and the Phi it takes
    const long at = base + (REVERSE ? n - 1 - i : i), by = REVERSE ? at + 1 : at - 1;
    own = load(places + (at * a.heads + h) * head);
    const Rsrc rs = make_rsrc(phi + (by * a.heads + h) * square, static_cast<unsigned>(square * 4));
    const int r = wave * 16 + l15;  // rows behind the states are outside
#pragma unroll
    for (int k = 0; k < NB; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = 32 * k + 16 * j + 4 * g;
        f[k].v[j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
            rs, c < a.states ? static_cast<unsigned>((r * a.states + c) * 4) : kOutside, 0, 0));
      }
  };
  fetch(1);
  v4f mine = {0, 0, 0, 0};
  if (first != nullptr) mine = load(first + (static_cast<long>(seq) * a.heads + h) * head);
  for (int i = 1; i < n; ++i) {
    v4f (&s)[2 * NB][64] = state[i & 1];
    s[wave][lane] = mine;
    __syncthreads();
    mine = own;
    Frag<float> now[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) now[k] = f[k];
    if (i + 1 < n) fetch(i + 1);
#pragma unroll
    for (int k = 0; k < NB; ++k) mma(mine, now[k], split_pair<float, 1>(s[2 * k][lane], s[2 * k + 1][lane]).f[0]);
    const Rsrc rs = make_rsrc(places + ((base + (REVERSE ? n - 1 - i : i)) * a.heads + h) * head, bytes);
#pragma unroll
    for (int j = 0; j < 4; ++j) store_elem<float>(rs, off + j * 4 * a.width, mine[j]);
  }
}

// ------------------------------------------------------------ single tokens
// One token of one sequence's head: S' = a S, u = beta (v - S'^T k),
// S = S' + k u^T, y = scale S^T q.  With w = S^T k and z = S^T q of the old
// state, u = beta (v - a w) and y = scale (a z + (q.k) u): the state is read
// once, kept in registers and written once.  A thread has 4 columns and every
// eighth row.  The state's traffic bounds it: 256 sequences of 32 heads of 128 x 64,
// 0.54 GB: 97 us, 5.5 TB/s.
struct StepArgs {
  mamba2_rows q, k, v, g, beta, y;
  const float* state;
  float* new_state;
  float scale;
  int heads, width, ratio, states, gate_bf16;
};

constexpr int kStepThreads = 256;
constexpr int kStepRows = 16;  // rows of the state that a thread holds at most

template <class T>
__global__ __launch_bounds__(kStepThreads) void delta_step_kernel(StepArgs a) {
  __shared__ float sk[kMaxDim], sq[kMaxDim];
  __shared__ alignas(16) float part[2][kStepThreads / 64][kMaxDim];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x, b = blockIdx.y, j = h / a.ratio;
  const long of_seq = (static_cast<long>(b) * a.heads + h) * (static_cast<long>(a.states) * a.width);
  const int quad = (tid & 31) * 4, row = tid >> 5;
  const bool mine = quad < a.width;
  v4f st[kStepRows];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = row + 8 * i;
    st[i] = mine && r < a.states ? *reinterpret_cast<const v4f*>(a.state + of_seq + r * a.width + quad) : v4f{0, 0, 0, 0};
  }
  const auto gate = [&](const mamba2_rows& r) {
    const long e = b * r.batch_stride + h;
    return a.gate_bf16 ? static_cast<float>(static_cast<const bf16*>(r.data)[e]) : static_cast<const float*>(r.data)[e];
  };
  if (tid < kMaxDim) {
    const bool in = tid < a.states;
    sk[tid] = in ? static_cast<float>(static_cast<const T*>(a.k.data)[b * a.k.batch_stride + j * a.states + tid]) : 0.0f;
    sq[tid] = in ? static_cast<float>(static_cast<const T*>(a.q.data)[b * a.q.batch_stride + j * a.states + tid]) : 0.0f;
  }
  const float decay = exp2_of(gate_log(gate(a.g))), beta = gate(a.beta);
  v4f v = {0, 0, 0, 0};
  if (mine) {
    const T* vp = static_cast<const T*>(a.v.data) + b * a.v.batch_stride + static_cast<long>(h) * a.width + quad;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(vp[i]);
  }
  __syncthreads();
  v4f w = {0, 0, 0, 0}, z = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    w += st[i] * sk[row + 8 * i];
    z += st[i] * sq[row + 8 * i];
  }
  // rows of the two halves of a wave, then of the waves
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Pair p = swap32(w[i]), r = swap32(z[i]);
    w[i] = p.a + p.b;
    z[i] = r.a + r.b;
  }
  if (lane < 32) {
    *reinterpret_cast<v4f*>(&part[0][wave][quad]) = w;
    *reinterpret_cast<v4f*>(&part[1][wave][quad]) = z;
  }
  const float qk = sum64(sk[lane] * sq[lane] + sk[lane + 64] * sq[lane + 64]);
  __syncthreads();
  w = z = v4f{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kStepThreads / 64; ++i) {
    w += *reinterpret_cast<const v4f*>(&part[0][i][quad]);
    z += *reinterpret_cast<const v4f*>(&part[1][i][quad]);
  }
  const v4f u = beta * (v - decay * w);
  if (!mine) return;
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = row + 8 * i;
    if (r < a.states) *reinterpret_cast<v4f*>(a.new_state + of_seq + r * a.width + quad) = decay * st[i] + sk[r] * u;
  }
  if (row == 0) {
    const v4f y = a.scale * (decay * z + qk * u);
    T* yp = static_cast<T*>(a.y.data) + b * a.y.batch_stride + static_cast<long>(h) * a.width + quad;
#pragma unroll
    for (int i = 0; i < 4; ++i) yp[i] = static_cast<T>(y[i]);
  }
}

// ---------------------------------------------------------------- host side
template <class T, int NB>
int launch_summary(const DeltaArgs& a, hipStream_t s) {
  const int slices = a.slices + (a.states + kCols - 1) / kCols;
  delta_summary_kernel<T, NB><<<static_cast<unsigned>(a.units) * a.heads * slices, walk_threads<T>, 0, s>>>(a);
  if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  delta_carry_kernel<NB, false><<<dim3((a.width + 15) / 16, a.heads, a.seqs.batch), 2 * NB * 64, 0, s>>>(a);
  return launch_status();
}
template <class T>
int launch_summary_states(const DeltaArgs& a, hipStream_t s) {
  if (a.states <= 32) return launch_summary<T, 1>(a, s);
  if (a.states <= 64) return launch_summary<T, 2>(a, s);
  return launch_summary<T, 4>(a, s);
}

template <class T, int NB>
int launch_fwd(const DeltaArgs& a, unsigned steps, int type, hipStream_t s) {
  if (steps > 0) {
    delta_prep_kernel<T, NB><<<prep_blocks(a, steps), kPrepWaves * 64, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    const int st = start_segments(a, type, s);
    if (st != MAMBA2_SCAN_OK) return st;
  }
  delta_fwd_kernel<T, NB><<<walk_blocks(a), walk_threads<T>, 0, s>>>(a);
  return launch_status();
}
template <class T>
int launch_fwd_states(const DeltaArgs& a, unsigned steps, int type, hipStream_t s) {
  if (a.states <= 32) return launch_fwd<T, 1>(a, steps, type, s);
  if (a.states <= 64) return launch_fwd<T, 2>(a, steps, type, s);
  return launch_fwd<T, 4>(a, steps, type, s);
}

long steps_of(const mamba2_seqs& q) { return unit_count(q, kTok); }
constexpr size_t kMBytes = kPieces * kPiece * sizeof(float);
size_t p_bytes(int type) { return (type == MAMBA2_BF16 ? 2 * 2 : 4) * kPieces * kPiece; }

}  // namespace

namespace delta {

namespace {
mamba2_ssm_dims scan_dims(const mamba2_delta_dims& d) {
  return {d.type, d.gate_type, d.heads, d.width, d.groups, d.states, 0};
}
}  // namespace

int check_delta(const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const int st = check_dims(q, scan_dims(d));
  if (st != MAMBA2_SCAN_OK) return st;
  if (!(d.scale - d.scale == 0.0f)) return MAMBA2_SCAN_EBADDIM;
  // the largest launches: 512 threads for every step and head, and for every segment,
  // head and 64 columns, in summaries of the values and of the state
  for (const bool bwd : {false, true}) {
    const long long units = unit_count(q, segment_tokens(q, d, bwd)) * ((d.width + kCols - 1) / kCols + (d.states + kCols - 1) / kCols);
    if (!grid_ok(units * d.heads, 512)) return MAMBA2_SCAN_EBADDIM;
  }
  return grid_ok(static_cast<long long>(steps_of(q)) * d.heads, 512) ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EBADDIM;
}
int check_keys(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const long long n = static_cast<long long>(d.groups) * d.states;
  *r = used_strides(*r, q, n);
  return check_vec_rows(*r, q, n, type_size(d.type));
}
int check_values(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const long long n = static_cast<long long>(d.heads) * d.width;
  *r = used_strides(*r, q, n);
  return check_vec_rows(*r, q, n, type_size(d.type));
}
int check_gates(mamba2_rows* r, const mamba2_seqs& q, const mamba2_delta_dims& d) {
  *r = used_strides(*r, q, d.heads);
  return check_step_rows(*r, q, scan_dims(d));
}
// Tokens per segment.  A head's columns are walked by work-groups of which a CU
// holds one; with fewer of them than CUs the tokens are cut into segments.  That
// costs the summary, a walk of the state's columns beside the values' that is 0.7
// of one with results, and the carry, whose segments follow one another (0.3 of a
// step each); two steps pass before a walk's first.  The fewest such steps are
// taken, rounds of work-groups counted whole.  Forward, us a call, bf16, one sequence:
//                                       whole   cut by the rule   best of the cuts tried
//   32768 tokens, 24 heads of 64 x 64   1557    434 (10)          434 (10)
//   8192 tokens, 8 heads of 128 x 128    463    132 (16)          132 (16)
//   4096 tokens, 32 heads of 128 x 128   247    174 (4)           174 (4)
//   1024 tokens, 8 heads of 128 x 128     68     52 (8)            52 (4 to 12)
// and forward and backward, 4096 tokens, 8 heads of 128 x 128: 742, 328 (16), 308 (8).
int segment_tokens(const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd) {
  const bool packed = q.offsets != nullptr;
  // how a packed call's rows are shared out is not known here
  const long seqs = packed ? (q.batch < 4 ? q.batch : 4) : q.batch;
  const long steps = ((packed ? q.length / seqs : q.length) + kTok - 1) / kTok;
  const long slices = (d.width + kCols - 1) / kCols, more = (d.states + kCols - 1) / kCols;
  const long lanes = seqs * d.heads * slices, summary = seqs * d.heads * (slices + more);
  const auto rounds = [](long n) { return static_cast<float>((n + kCUs - 1) / kCUs); };
  float best = 0.0f;
  long cut = 1;
  // A packed call of many sequences is not cut, though one of them may be long: each
  // has a place for a segment's state and transition, and the carry its work-groups.
  if (lanes < kCUs && q.batch * d.heads * slices < 16 * kCUs) {
    for (long n = 1; n <= 64 && n <= steps; ++n) {
      const float walk = static_cast<float>((steps + n - 1) / n + 2);
      float cost = rounds(lanes * n) * walk * (bwd ? 2.35f : 1.0f);
      if (n > 1) {
        cost += rounds(summary * n) * walk * 0.7f + 0.3f * n + 2.0f;
        if (bwd) cost += rounds(lanes * n) * walk * 1.1f + 0.3f * n + 2.0f;
      }
      if (n == 1 || cost < best) {
        best = cost;
        cut = n;
      }
    }
  }
  const long rows = packed ? q.length / seqs : q.length;
  long seg = cut > 1 ? (rows + cut - 1) / cut : q.length;
  seg = (seg + kTok - 1) / kTok * kTok;
  return static_cast<int>(seg < kTok ? kTok : seg);
}

int start_segments(const DeltaArgs& a, int type, hipStream_t s) {
  if (a.seqs.length <= a.seg) return MAMBA2_SCAN_OK;
  return type == MAMBA2_BF16 ? launch_summary_states<bf16>(a, s) : launch_summary_states<float>(a, s);
}
int carry_gradients(const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((a.width + 15) / 16, a.heads, a.seqs.batch);
  if (a.states <= 32) delta_carry_kernel<1, true><<<grid, 128, 0, s>>>(a);
  else if (a.states <= 64) delta_carry_kernel<2, true><<<grid, 256, 0, s>>>(a);
  else delta_carry_kernel<4, true><<<grid, 512, 0, s>>>(a);
  return launch_status();
}
unsigned walk_blocks(const DeltaArgs& a) { return static_cast<unsigned>(a.units) * a.heads * a.slices; }

size_t segment_bytes(const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd) {
  const int seg = segment_tokens(q, d, bwd);
  if (q.length <= seg) return 0;
  const size_t head = (bwd ? 2 : 1) * static_cast<size_t>(d.states) * (d.width + d.states);
  return static_cast<size_t>(unit_count(q, seg)) * d.heads * head * sizeof(float);
}
void set_segments(DeltaArgs* a, char* at, bool bwd) {
  if (a->seqs.length <= a->seg) return;
  const long cells = static_cast<long>(a->units) * a->heads, head = static_cast<long>(a->states) * a->width;
  a->seg_state = reinterpret_cast<float*>(at);
  a->seg_trans = a->seg_state + cells * head;
  if (!bwd) return;
  a->seg_trans_t = a->seg_trans + cells * a->states * a->states;
  a->seg_grad = a->seg_trans_t + cells * a->states * a->states;
}

void set_dims(DeltaArgs* a, const mamba2_seqs& q, const mamba2_delta_dims& d, bool bwd) {
  a->seqs = q;
  a->scale = d.scale;
  a->heads = d.heads;
  a->width = d.width;
  a->ratio = d.heads / d.groups;
  a->states = d.states;
  a->slices = (d.width + kWaves * 16 - 1) / (kWaves * 16);
  a->gate_bf16 = d.gate_type == MAMBA2_BF16;
  // the matrices: heads that share a q and k one after the other, once the chip is full.
  // Counted for 4, 3 and 2 work-groups on a CU, us: 2 x 4096 tokens, 32 heads of 64
  // states in 4 groups, bf16, 29, 33, 36; fp32 with 128 states 56, 61, 45.
  const long full = steps_of(q) * d.heads / (prep_per_cu(type_size(d.type), d.states) * kCUs);
  a->prep_heads = full < 1 ? 1 : full < a->ratio ? static_cast<int>(full) : a->ratio;
  a->seg = segment_tokens(q, d, bwd);
  a->units = static_cast<int>(unit_count(q, a->seg));
}

}  // namespace delta

extern "C" {

size_t mamba2_delta_fwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims d) {
  if (check_delta(seqs, d) != MAMBA2_SCAN_OK) return 0;
  return static_cast<size_t>(steps_of(seqs)) * d.heads * (kMBytes + p_bytes(d.type) + sizeof(Coef)) +
         segment_bytes(seqs, d, false);
}

int mamba2_delta_fwd(mamba2_seqs seqs, mamba2_delta_dims d, mamba2_rows q, mamba2_rows k, mamba2_rows v, mamba2_rows g,
                     mamba2_rows beta, const float* initial_state, mamba2_rows y, float* final_state, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int st = check_delta(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  DeltaArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.y = y;
  if ((st = check_keys(&a.q, seqs, d)) != MAMBA2_SCAN_OK || (st = check_keys(&a.k, seqs, d)) != MAMBA2_SCAN_OK ||
      (st = check_values(&a.v, seqs, d)) != MAMBA2_SCAN_OK || (st = check_values(&a.y, seqs, d)) != MAMBA2_SCAN_OK ||
      (st = check_gates(&a.g, seqs, d)) != MAMBA2_SCAN_OK || (st = check_gates(&a.beta, seqs, d)) != MAMBA2_SCAN_OK)
    return st;
  if (!aligned_to(initial_state, 16) || !aligned_to(final_state, 16)) return MAMBA2_SCAN_EALIGN;
  if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
  if (workspace_bytes < mamba2_delta_fwd_workspace_bytes(seqs, d)) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  if (seqs.length == 0 && final_state == nullptr) return MAMBA2_SCAN_OK;
  a.initial = initial_state;
  a.final_state = final_state;
  set_dims(&a, seqs, d, false);
  const long cells = steps_of(seqs) * d.heads;
  char* at = static_cast<char*>(workspace);
  a.m = reinterpret_cast<float*>(at);
  a.p = at + cells * kMBytes;
  a.coef = reinterpret_cast<Coef*>(at + cells * (kMBytes + p_bytes(d.type)));
  const unsigned steps = seqs.length == 0 ? 0 : static_cast<unsigned>(cells);
  set_segments(&a, reinterpret_cast<char*>(a.coef + cells), false);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return d.type == MAMBA2_BF16 ? launch_fwd_states<bf16>(a, steps, d.type, s) : launch_fwd_states<float>(a, steps, d.type, s);
}

int mamba2_delta_step(int batch, mamba2_delta_dims d, mamba2_rows q, mamba2_rows k, mamba2_rows v, mamba2_rows g,
                      mamba2_rows beta, const float* state, mamba2_rows y, float* new_state, void* stream) {
  const mamba2_seqs seqs = {batch, 1, nullptr};
  int st = check_delta(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  if (state == nullptr || new_state == nullptr) return MAMBA2_SCAN_ENULL;
  const size_t e = type_size(d.type), eg = type_size(d.gate_type);
  const long long vw = static_cast<long long>(d.heads) * d.width, kw = static_cast<long long>(d.groups) * d.states;
  q.row_stride = k.row_stride = v.row_stride = g.row_stride = beta.row_stride = y.row_stride = 0;
  if ((st = check_keys(&q, seqs, d)) != MAMBA2_SCAN_OK || (st = check_keys(&k, seqs, d)) != MAMBA2_SCAN_OK ||
      (st = check_values(&v, seqs, d)) != MAMBA2_SCAN_OK || (st = check_values(&y, seqs, d)) != MAMBA2_SCAN_OK ||
      (st = check_gates(&g, seqs, d)) != MAMBA2_SCAN_OK || (st = check_gates(&beta, seqs, d)) != MAMBA2_SCAN_OK)
    return st;
  if (!aligned_to(state, 16) || !aligned_to(new_state, 16)) return MAMBA2_SCAN_EALIGN;
  const long long states = static_cast<long long>(batch) * d.heads * d.states * d.width * 4;
  const Region mem[] = {token_region(y, batch, vw, e),    region(new_state, states),
                        token_region(q, batch, kw, e),    token_region(k, batch, kw, e),
                        token_region(v, batch, vw, e),    token_region(g, batch, d.heads, eg),
                        token_region(beta, batch, d.heads, eg), region(state != new_state ? state : nullptr, states)};
  if (!apart(mem, 2, 8)) return MAMBA2_SCAN_EOVERLAP;
  const StepArgs a = {q, k, v, g, beta, y, state, new_state, d.scale, d.heads, d.width, d.heads / d.groups, d.states,
                      d.gate_type == MAMBA2_BF16};
  const dim3 grid(d.heads, batch);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (d.type == MAMBA2_BF16) delta_step_kernel<bf16><<<grid, kStepThreads, 0, s>>>(a);
  else delta_step_kernel<float><<<grid, kStepThreads, 0, s>>>(a);
  return launch_status();
}

}  // extern "C"
