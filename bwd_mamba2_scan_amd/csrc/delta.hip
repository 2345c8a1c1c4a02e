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
#include "delta_prep.h"

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

template <class T, int NB>
struct FwdLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  alignas(16) T k[kTok * ldn];
  alignas(16) T q[kTok * ldn];
  alignas(16) T m[kExact<T> * kPieces * kPiece];
  alignas(16) T p[kTwo<T> * kPieces * kPiece];
  alignas(16) Coef coef;
};

template <class T, int NB>
__global__ __launch_bounds__(kWaves * 64, 1) void delta_fwd_kernel(DeltaArgs a) {
  typedef FwdLds<T, NB> L;
  __shared__ L s;
  constexpr int kThreads = kWaves * 64;
  constexpr int kM = kExact<T> * kPieces * kPiece, kP = kTwo<T> * kPieces * kPiece;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int per = a.heads * a.slices;
  const int unit = work / per, h = work % per / a.slices, slice = work % a.slices;
  const Unit u = locate(a.seqs, unit, a.seg);
  if (!u.live) return;
  const bool packed = a.seqs.offsets != nullptr;
  const int p0 = slice * kThreads / 4;
  const int col = p0 + wave * 16 + l15;
  const long of_seq = (static_cast<long>(u.seq) * a.heads + h) * (static_cast<long>(a.states) * a.width);
  const T* kp = seq_ptr<const T>(a.k, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* qp = seq_ptr<const T>(a.q, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* vp = seq_ptr<const T>(a.v, u.seq, u.row0, packed) + h * a.width;
  T* yp = seq_ptr<T>(a.y, u.seq, u.row0, packed) + h * a.width;

  State<NB, true> st;
  st.init(a.width, p0, wave);
  st.load(a.initial == nullptr ? nullptr : a.initial + of_seq, a.width, a.states);

  const int end = u.len;
  Tile<T, kTok, NB * 32, kThreads> tk, tq;
  tk.init(a.k.row_stride, a.states, tid);
  tq.init(a.q.row_stride, a.states, tid);
  Flat<kM * sizeof(T), kThreads> tm;
  Flat<kP * sizeof(T), kThreads> tp;
  Flat<sizeof(Coef), kThreads> tc;
  float v[4][4];
  const unsigned v_off = col < a.width ? static_cast<unsigned>((4 * g * static_cast<int>(a.v.row_stride) + col) * sizeof(T)) : kOutside;
  const unsigned y_off = col < a.width ? static_cast<unsigned>((4 * g * static_cast<int>(a.y.row_stride) + col) * sizeof(T)) : kOutside;
  const int v_row = static_cast<int>(a.v.row_stride * sizeof(T)), y_row = static_cast<int>(a.y.row_stride * sizeof(T));
  const auto fetch = [&](int t) {
    const int rows = min(end - t, kTok);
    const long at = step_at(a.seqs, u.seq, t) * a.heads + h;
    tk.load(rows_rsrc(kp + t * a.k.row_stride, a.k.row_stride, rows, a.states));
    tq.load(rows_rsrc(qp + t * a.q.row_stride, a.q.row_stride, rows, a.states));
    tm.load(static_cast<const T*>(a.m) + at * kM, tid);
    tp.load(static_cast<const T*>(a.p) + at * kP, tid);
    tc.load(a.coef + at, tid);
    const Rsrc rv = rows_rsrc(vp + t * a.v.row_stride, a.v.row_stride, rows, a.width);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[i][r] = load_elem<T>(rv, v_off + (16 * i + r) * v_row);
  };
  if (u.t0 < end) fetch(u.t0);
  for (int t = u.t0; t < end; t += kTok) {
    __syncthreads();
    tk.store(s.k, L::ldn, tid);
    tq.store(s.q, L::ldn, tid);
    tm.store(s.m, tid);
    tp.store(s.p, tid);
    tc.store(&s.coef, tid);
    v4f x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v4f{v[i][0], v[i][1], v[i][2], v[i][3]};
    __syncthreads();
    if (t + kTok < end) fetch(t + kTok);

    // K S and Q S
    v4f ks[4], qs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i] = qs[i] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const Split<T, kExact<T>> sp = split_pair<T, kExact<T>>(st.st[2 * n], st.st[2 * n + 1]);
      Frag<T> two[kTwo<T>];
#pragma unroll
      for (int z = 0; z < kTwo<T>; ++z) two[z] = sp.f[z];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Frag<T> kf[1] = {frag_row_result(s.k, L::ldn, 16 * i, 32 * n)};
        const Frag<T> qf[1] = {frag_row_result(s.q, L::ldn, 16 * i, 32 * n)};
        mma_parts<T>(ks[i], kf, sp.f);
        mma_parts<T>(qs[i], qf, two);
      }
    }
    // beta (V - 2^c K S), then U = M that
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = rows_of(s.coef.beta, i, g) * (x[i] - rows_of(s.coef.from, i, g) * ks[i]);
    const Split<T, kExact<T>> xs[2] = {split_pair<T, kExact<T>>(x[0], x[1]), split_pair<T, kExact<T>>(x[2], x[3])};
    v4f w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n <= i / 2; ++n) {
        Frag<T> mf[kExact<T>];
#pragma unroll
        for (int z = 0; z < kExact<T>; ++z) mf[z] = piece_get(s.m + (z * kPieces + piece_of(i, n)) * kPiece, lane);
        mma_parts<T>(w[i], mf, xs[n].f);
      }
    }
    // Y = scale 2^c Q S + P U
    {
      const Split<T, kTwo<T>> us[2] = {split_pair<T, kTwo<T>>(w[0], w[1]), split_pair<T, kTwo<T>>(w[2], w[3])};
      const Rsrc ry = rows_rsrc(yp + t * a.y.row_stride, a.y.row_stride, min(end - t, kTok), a.width);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v4f y = qs[i] * rows_of(s.coef.from, i, g) * a.scale;
#pragma unroll
        for (int n = 0; n <= i / 2; ++n) {
          Frag<T> pf[kTwo<T>];
#pragma unroll
          for (int z = 0; z < kTwo<T>; ++z) pf[z] = piece_get(s.p + (z * kPieces + piece_of(i, n)) * kPiece, lane);
          mma_parts<T>(y, pf, us[n].f);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) store_elem<T>(ry, y_off + (16 * i + r) * y_row, y[r]);
      }
    }
    // S = 2^c_end S + K^T (2^(c_end - c) U); a step's products are added up by
    // themselves: on top of the state, each would round at the state's size
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = w[i] * rows_of(s.coef.to, i, g);
    const Split<T, kExact<T>> us[2] = {split_pair<T, kExact<T>>(w[0], w[1]), split_pair<T, kExact<T>>(w[2], w[3])};
    const float total = s.coef.total;
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
      v4f add = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Frag<T> kf[1] = {frag_col_result(s.k, L::ldn, 32 * j, 16 * n)};
        mma_parts<T>(add, kf, us[j].f);
      }
      st.st[n] = st.st[n] * total + add;
    }
  }
  if (a.final_state != nullptr) st.save(a.final_state + of_seq, a.width, a.states);
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
  delta_fwd_kernel<T, NB><<<blocks, kWaves * 64, 0, s>>>(a);
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

int check_delta(const mamba2_seqs& q, const mamba2_delta_dims& d) {
  const mamba2_ssm_dims like = {d.type, d.gate_type, d.heads, d.width, d.groups, d.states, 0};
  const int st = check_dims(q, like);
  if (st != MAMBA2_SCAN_OK) return st;
  if (!(d.scale - d.scale == 0.0f)) return MAMBA2_SCAN_EBADDIM;
  // a step's work-group of four waves for every step and head, and for every sequence, head and 64 columns
  const long long most = steps_of(q) > 2LL * q.batch ? steps_of(q) : 2LL * q.batch;
  return grid_ok(most * d.heads, kPrepWaves * 64) ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EBADDIM;
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
  const size_t e = type_size(d.type);
  const long long vw = static_cast<long long>(d.heads) * d.width, kw = static_cast<long long>(d.groups) * d.states;
  const mamba2_ssm_dims like = {d.type, d.gate_type, d.heads, d.width, d.groups, d.states, 0};
  DeltaArgs a = {};
  a.seqs = seqs;
  a.q = used_strides(q, seqs, kw);
  a.k = used_strides(k, seqs, kw);
  a.v = used_strides(v, seqs, vw);
  a.y = used_strides(y, seqs, vw);
  a.g = used_strides(g, seqs, d.heads);
  a.beta = used_strides(beta, seqs, d.heads);
  if ((st = check_vec_rows(a.q, seqs, kw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(a.k, seqs, kw, e)) != MAMBA2_SCAN_OK ||
      (st = check_vec_rows(a.v, seqs, vw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(a.y, seqs, vw, e)) != MAMBA2_SCAN_OK ||
      (st = check_step_rows(a.g, seqs, like)) != MAMBA2_SCAN_OK || (st = check_step_rows(a.beta, seqs, like)) != MAMBA2_SCAN_OK)
    return st;
  if (!aligned_to(initial_state, 16) || !aligned_to(final_state, 16)) return MAMBA2_SCAN_EALIGN;
  const size_t need = mamba2_delta_fwd_workspace_bytes(seqs, d);
  if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
  if (workspace_bytes < need) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  if (seqs.length == 0 && final_state == nullptr) return MAMBA2_SCAN_OK;
  a.initial = initial_state;
  a.final_state = final_state;
  a.scale = d.scale;
  a.heads = d.heads;
  a.width = d.width;
  a.ratio = d.heads / d.groups;
  a.states = d.states;
  a.slices = (d.width + kWaves * 16 - 1) / (kWaves * 16);
  a.gate_bf16 = d.gate_type == MAMBA2_BF16;
  a.seg = (seqs.length + kTok - 1) / kTok * kTok;
  if (a.seg == 0) a.seg = kTok;
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
  const mamba2_ssm_dims like = {d.type, d.gate_type, d.heads, d.width, d.groups, d.states, 0};
  q.row_stride = k.row_stride = v.row_stride = g.row_stride = beta.row_stride = y.row_stride = 0;
  if ((st = check_vec_rows(q, seqs, kw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(k, seqs, kw, e)) != MAMBA2_SCAN_OK ||
      (st = check_vec_rows(v, seqs, vw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(y, seqs, vw, e)) != MAMBA2_SCAN_OK ||
      (st = check_step_rows(g, seqs, like)) != MAMBA2_SCAN_OK || (st = check_step_rows(beta, seqs, like)) != MAMBA2_SCAN_OK)
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
