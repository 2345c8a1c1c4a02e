// Gated delta rule for gfx950: the forward over prompts and the single-token
// form.  The mathematics of a step is in delta_common.h.
//
// delta_prep_kernel: one work-group per step and head writes the step's M and P
// as operands.  delta_fwd_kernel: a wave owns 16 columns of a head's state, S
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

template <class T, int NB>
__global__ __launch_bounds__(kPrepWaves * 64) void delta_prep_kernel(DeltaArgs a) {
  __shared__ PrepLds<T, NB> s;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int step = work / a.heads, h = work % a.heads;
  const Unit u = locate(a.seqs, step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  make_step<T, NB>(s, a, u, h, a.seqs.offsets != nullptr);
  const long at = static_cast<long>(step) * a.heads + h;
  put_pieces<T, kExact<T>, false>(static_cast<T*>(a.m) + at * kExact<T> * kPieces * kPiece, s.m, wave, lane);
  put_pieces<T, kTwo<T>, false>(static_cast<T*>(a.p) + at * kTwo<T> * kPieces * kPiece, s.sq.p, wave, lane);
  if (threadIdx.x < sizeof(Coef) / 16)
    reinterpret_cast<v4f*>(a.coef + at)[threadIdx.x] = reinterpret_cast<const v4f*>(&s.coef)[threadIdx.x];
}

template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_fwd_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairFwdLds<NB, false> s;
    pair_forward<NB, false>(a, s);
  } else {
    __shared__ FwdLds<T, NB, false> s;
    walk_forward<T, NB, false>(a, s);
  }
}

// ------------------------------------------------------------ single tokens
// One token of one sequence's head: S' = a S, u = beta (v - S'^T k),
// S = S' + k u^T, y = scale S^T q.  With w = S^T k and z = S^T q of the old
// state, u = beta (v - a w) and y = scale (a z + (q.k) u): the state is read
// once, kept in registers and written once.  A thread has 4 columns and every
// eighth row.
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
int launch_fwd(const DeltaArgs& a, unsigned steps, unsigned blocks, hipStream_t s) {
  if (steps > 0) {
    delta_prep_kernel<T, NB><<<steps, kPrepWaves * 64, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  }
  delta_fwd_kernel<T, NB><<<blocks, walk_threads<T>, 0, s>>>(a);
  return launch_status();
}
template <class T>
int launch_fwd_states(const DeltaArgs& a, unsigned steps, unsigned blocks, hipStream_t s) {
  if (a.states <= 32) return launch_fwd<T, 1>(a, steps, blocks, s);
  if (a.states <= 64) return launch_fwd<T, 2>(a, steps, blocks, s);
  return launch_fwd<T, 4>(a, steps, blocks, s);
}

long steps_of(const mamba2_seqs& q) { return unit_count(q, kTok); }
size_t m_bytes(int type) { return (type == MAMBA2_BF16 ? 3 * 2 : 4) * kPieces * kPiece; }
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
  // the largest launches: up to 512 threads for every step and head, and 256 for every
  // sequence (packed: one more), head and 64 columns
  const long long most = steps_of(q) > q.batch + 1LL ? steps_of(q) : q.batch + 1LL;
  return grid_ok(most * d.heads, 512) ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EBADDIM;
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
void set_dims(DeltaArgs* a, const mamba2_seqs& q, const mamba2_delta_dims& d) {
  a->seqs = q;
  a->scale = d.scale;
  a->heads = d.heads;
  a->width = d.width;
  a->ratio = d.heads / d.groups;
  a->states = d.states;
  a->slices = (d.width + kWaves * 16 - 1) / (kWaves * 16);
  a->gate_bf16 = d.gate_type == MAMBA2_BF16;
  a->seg = q.length > kTok ? (q.length + kTok - 1) / kTok * kTok : kTok;
}

}  // namespace delta

extern "C" {

size_t mamba2_delta_fwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims d) {
  if (check_delta(seqs, d) != MAMBA2_SCAN_OK) return 0;
  return static_cast<size_t>(steps_of(seqs)) * d.heads * (m_bytes(d.type) + p_bytes(d.type) + sizeof(Coef));
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
  set_dims(&a, seqs, d);
  const long cells = steps_of(seqs) * d.heads;
  char* at = static_cast<char*>(workspace);
  a.m = at;
  a.p = at + cells * m_bytes(d.type);
  a.coef = reinterpret_cast<Coef*>(at + cells * (m_bytes(d.type) + p_bytes(d.type)));
  const unsigned steps = seqs.length == 0 ? 0 : static_cast<unsigned>(cells);
  const unsigned blocks = static_cast<unsigned>(unit_count(seqs, a.seg) * d.heads * a.slices);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return d.type == MAMBA2_BF16 ? launch_fwd_states<bf16>(a, steps, blocks, s) : launch_fwd_states<float>(a, steps, blocks, s);
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
