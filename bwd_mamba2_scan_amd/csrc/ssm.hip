// Selective state space scan for gfx950: the forward over prompts and the
// single-token form.
//
// ssm_fwd_kernel: a work-group owns one head (or 64 of its columns), its NW
// waves 16 columns each, and walks the tokens in steps of 64.  A wave keeps
// its columns of the state, S [states][16], in registers in fp32 as a matrix
// result; result order makes that register file directly the operand of
// S^T C.  Per step:
//   scores   W[t][s] = (C_t . B_s) 2^(c_t - c_s) d_s (s <= t): the ten 16 x 16
//            tiles on and below the diagonal, dealt to the waves, to LDS
//   y        2^c_t (C_t . S) + W x + D x, 64 x 16 per wave
//   S        2^c_end S + B^T (2^(c_end - c_s) d_s x_s)
// B, C, x of the next step are loaded while this one is computed.
//
// Long sequences with few heads are cut into segments that run in parallel:
// a summary pass (ssm_summary_kernel: each segment's own contribution to
// the state), the carry across segments (ssm_carry_kernel), and the forward from
// the states so found.  Few segments carry by themselves (start_state).
//
// Measured at 4 x 4096 tokens, 32 heads of 64 columns, one group of 128 states,
// bf16: summary 46 us, forward 100 us.  The forward's bytes (165 MB) would take
// 32 us at a large copy's rate and its products keep the matrix cores busy 29 % of
// the time; what bounds both kernels is LDS, whose pipes are busy 62 % of the
// forward's time, and the barriers of a step, which two work-groups on a CU hide
// for each other.
#include "ssm_common.h"

namespace {

using namespace ssm;

// Tile i of the ten with s <= t: row tile (t) and column tile (s).
__device__ __forceinline__ void lower_tile(int i, int* ti, int* si) {
  *ti = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
  *si = i - (*ti * (*ti + 1)) / 2;
}

template <class T, int NB, int NW>
struct FwdLds {
  static constexpr int kN = NB * 32;          // states, padded
  static constexpr int kP = NW * 16;          // columns of the head in this work-group
  static constexpr int ldn = stride_of<T>(kN);
  static constexpr int ldp = stride_of<T>(kP);
  static constexpr int ldw = stride_of<T>(kTok);
  // The scores and the state are operands in two bf16 parts: with one, y's terms
  // lost what cancels between them (1.87e-3 of y against 1.66e-3, its own
  // rounding), for 4 us of 116 at 4 x 4096 tokens, 32 heads of 64, 128 states.
  static constexpr int kParts = sizeof(T) == 2 ? 2 : 1;
  alignas(16) T b[kTok * ldn];
  alignas(16) T c[kTok * ldn];
  alignas(16) T x[kTok * ldp];
  alignas(16) T w[kParts][kTok * ldw];
  alignas(16) Decays dc[2];
};

// Up to 64 states three waves fit a SIMD (24 heads of 64, 64 states, 32768 tokens:
// 127 us a call, with two waves 160); of 128 states three would spill.
template <class T, int NB, int NW>
__global__ __launch_bounds__(NW * 64, simd_waves(sizeof(FwdLds<T, NB, NW>), NW, NB < 4 ? 3 : 2)) void ssm_fwd_kernel(SsmArgs a, Walk w) {
  typedef FwdLds<T, NB, NW> L;
  __shared__ L s;
  constexpr int kThreads = NW * 64;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int per = a.heads * a.slices;
  const int unit = work / per;
  const int h = work % per / a.slices;
  const int slice = work % a.slices;
  const Unit u = locate(a.q, unit, a.seg);
  if (!u.live) return;
  const bool packed = a.q.offsets != nullptr;
  const int p0 = slice * L::kP;                          // first column of the work-group
  const int cols = min(a.width - p0, L::kP);
  const int quad = wave * 16 + 4 * g;                    // this lane's four columns of y
  const long head = static_cast<long>(a.states) * a.width;
  const long of_seq = (static_cast<long>(u.seq) * a.heads + h) * head;

  const T* xp = seq_ptr<const T>(a.x, u.seq, u.row0, packed) + h * a.width + p0;
  const T* bp = seq_ptr<const T>(a.B, u.seq, u.row0, packed) + h / a.ratio * a.states;
  const T* cp = seq_ptr<const T>(a.C, u.seq, u.row0, packed) + h / a.ratio * a.states;
  T* yp = seq_ptr<T>(a.y, u.seq, u.row0, packed) + h * a.width + p0;
  const double rate = decay_rate(a.A[h]);
  const float bias = a.bias != nullptr ? a.bias[h] : 0.0f, D = a.D != nullptr ? a.D[h] : 0.0f;

  State<NB, true> st;
  st.init(a.width, p0, wave);
  start_state(st, a, w, u, unit, h);
  // tiles above the diagonal that a 32-wide product step touches stay zero
  constexpr int kQuads = sizeof(s.w) / sizeof(v4u);
  for (int i = tid; i < kQuads; i += kThreads) reinterpret_cast<v4u*>(s.w[0])[i] = v4u{0, 0, 0, 0};

  const int end = min(u.t0 + a.seg, u.len);
  Tile<T, kTok, L::kN, kThreads> tb, tc;
  Tile<T, kTok, L::kP, kThreads> tx;
  tb.init(a.B.row_stride, a.states, tid);
  tc.init(a.C.row_stride, a.states, tid);
  tx.init(a.x.row_stride, cols, tid);
  const auto fetch = [&](int t) {
    const int rows = min(end - t, kTok);
    tb.load(rows_rsrc(bp + t * a.B.row_stride, a.B.row_stride, rows, a.states));
    tc.load(rows_rsrc(cp + t * a.C.row_stride, a.C.row_stride, rows, a.states));
    tx.load(rows_rsrc(xp + t * a.x.row_stride, a.x.row_stride, rows, cols));
  };
  // The last wave, which has the fewest score tiles, prepares the next step's
  // decays; the raw step sizes are loaded a step before that.
  const bool decays = wave == NW - 1;
  float raw = 0.0f;
  const auto fetch_raw = [&](int t) { raw = load_raw(a, step_rsrc(a, u, packed, t, min(end - t, kTok)), h); };
  const auto prepare = [&](Decays& dc, int t) {
    make_decays(dc, lane < end - t ? step_of(a, raw, bias) : 0.0f, rate);
  };
  if (u.t0 < end) {
    fetch(u.t0);
    if (decays) {
      fetch_raw(u.t0);
      prepare(s.dc[0], u.t0);
      if (u.t0 + kTok < end) fetch_raw(u.t0 + kTok);
    }
  }
  const int y16 = static_cast<int>(16 * a.y.row_stride * sizeof(T));  // sixteen rows of y
  const unsigned yoff =
      quad < cols ? static_cast<unsigned>((l15 * static_cast<int>(a.y.row_stride) + quad) * sizeof(T)) : kOutside;
  int turn = 0;
  for (int t = u.t0; t < end; t += kTok, turn ^= 1) {
    const Decays& dc = s.dc[turn];
    __syncthreads();  // the last step's readers are done
    tb.store(s.b, L::ldn, tid);
    tc.store(s.c, L::ldn, tid);
    tx.store(s.x, L::ldp, tid);
    __syncthreads();
    if (t + kTok < end) {
      fetch(t + kTok);
      if (decays) {
        prepare(s.dc[turn ^ 1], t + kTok);
        if (t + 2 * kTok < end) fetch_raw(t + 2 * kTok);
      }
    }

    // scores, transposed as a result: lane has t = l15, s = 4 g + i
#pragma unroll
    for (int i0 = 0; i0 < 10; i0 += NW) {
      if (i0 + wave >= 10) continue;
      int ti, si;
      lower_tile(i0 + wave, &ti, &si);
      v4f w = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < NB; ++k)
        mma(w, frag_row(s.b, L::ldn, si * 16, k * 32), frag_row(s.c, L::ldn, ti * 16, k * 32));
      const int tt = ti * 16 + l15, ss = si * 16 + 4 * g;
      const float ch = dc.hi[tt], cl = dc.lo[tt];
      const v4f hi = *reinterpret_cast<const v4f*>(&dc.hi[ss]), lo = *reinterpret_cast<const v4f*>(&dc.lo[ss]);
      const v4f d = *reinterpret_cast<const v4f*>(&dc.d[ss]);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] *= exp2_of((ch - hi[j]) + (cl - lo[j])) * d[j];
      if (ti == si) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * g + j > l15) w[j] = 0.0f;
      }
      // the scores become an operand, with bf16 in two parts
      quad_put_parts<L::kParts>(&s.w[0][tt * L::ldw + ss], kTok * L::ldw, w);
    }
    // y transposed (lane: t = l15, columns 4 g + i), from the state before the
    // step, as an operand in as many parts.
    v4f y[4];
    {
#pragma unroll
      for (int ti = 0; ti < 4; ++ti) y[ti] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = st.st[2 * k + (j >> 2)][j & 3];
        const auto sf = split_of<T, L::kParts>(v);
        Frag<T> cf[4];
#pragma unroll
        for (int ti = 0; ti < 4; ++ti) cf[ti] = frag_row_result(s.c, L::ldn, ti * 16, k * 32);
#pragma unroll
        for (int z = 0; z < L::kParts; ++z)
#pragma unroll
          for (int ti = 0; ti < 4; ++ti) mma(y[ti], sf.f[z], cf[ti]);
      }
#pragma unroll
      for (int ti = 0; ti < 4; ++ti) y[ti] *= dc.from[ti * 16 + l15];
    }
    Frag<T> xf[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) xf[k] = frag_col(s.x, L::ldp, k * 32, wave * 16);
    st.template advance<T>(dc.total, dc.to, s.b, L::ldn, xf);
    __syncthreads();
    const Rsrc ry = rows_rsrc(yp + t * a.y.row_stride, a.y.row_stride, min(end - t, kTok), cols);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int z = 0; z < L::kParts; ++z)
#pragma unroll
        for (int ti = 2 * k; ti < 4; ++ti) mma(y[ti], xf[k], frag_row(s.w[z], L::ldw, ti * 16, k * 32));
#pragma unroll
    for (int ti = 0; ti < 4; ++ti) {
      y[ti] += D * quad_get(&s.x[(ti * 16 + l15) * L::ldp + quad]);
      Quad<T>::store(ry, yoff + ti * y16, y[ti]);
    }
  }
  if (a.final_state != nullptr && u.t0 + static_cast<long>(a.seg) >= u.len)
    st.save(a.final_state + of_seq, a.width, a.states);
}

// Summary pass of the segments; see walk().  46 us where the forward takes 100:
// it reads x and B (54 MB) and has no scores to compute.
template <class T, int NB, int NW>
__global__ __launch_bounds__(NW * 64, simd_waves(sizeof(WalkLds<T, NB, NW>), NW, 2)) void ssm_summary_kernel(SsmArgs a, Walk w) {
  __shared__ WalkLds<T, NB, NW> s;
  walk<T, NB, NW, false>(a, w, s);
}

__global__ __launch_bounds__(256) void ssm_carry_kernel(SsmArgs a, Walk w) { carry(a, w, blockIdx.z, blockIdx.x); }

// ------------------------------------------------------------- single token
// A work-group per sequence and head; a thread holds four neighbouring
// columns and walks the state's rows, so a row is read and written as 16-byte
// accesses and y needs no sum across the lanes of a row.  Bound by HBM, the
// fp32 state read and written once: 256 sequences of 32 heads, 128 x 64, 539 MB
// in 98 us, 5.5 TB/s.  Two sequences of 24 heads take 4 us, a launch's time.
constexpr int kStepThreads = 256;

struct StepArgs {
  SsmArgs a;
  const float* state;
  float* new_state;
};

template <class T>
__global__ __launch_bounds__(kStepThreads) void ssm_step_kernel(StepArgs sa) {
  const SsmArgs& a = sa.a;
  __shared__ float lds[kStepThreads * 4];
  __shared__ float sb[kMaxDim], sc[kMaxDim];
  const int h = blockIdx.x, seq = blockIdx.y, tid = threadIdx.x;
  const int quads = a.width / 4;
  const int rows = kStepThreads / quads;  // state rows per pass
  const int q = tid % quads, r0 = tid / quads;
  const long base = (static_cast<long>(seq) * a.heads + h) * a.states * a.width;
  constexpr int kAhead = 8;
  v4f s[kAhead];
  const bool live = r0 < rows;
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int n = r0 + j * rows;
    if (live && n < a.states) s[j] = *reinterpret_cast<const v4f*>(sa.state + base + static_cast<long>(n) * a.width + 4 * q);
  }
  const int gr = h / a.ratio * a.states;
  if (tid < a.states) sb[tid] = static_cast<float>((static_cast<const T*>(a.B.data) + seq * a.B.batch_stride)[gr + tid]);
  else if (tid >= kMaxDim && tid - kMaxDim < a.states)
    sc[tid - kMaxDim] = static_cast<float>((static_cast<const T*>(a.C.data) + seq * a.C.batch_stride)[gr + tid - kMaxDim]);
  const long di = seq * a.dt.batch_stride + h;
  const float raw = a.dt_bf16 ? static_cast<float>(static_cast<const bf16*>(a.dt.data)[di])
                              : static_cast<const float*>(a.dt.data)[di];
  const float d = step_of(a, raw, a.bias != nullptr ? a.bias[h] : 0.0f);
  const float decay = exp2_of(log_decay(d, decay_rate(a.A[h])));
  const T* xp = static_cast<const T*>(a.x.data) + seq * a.x.batch_stride + h * a.width + 4 * q;
  float x[4], xd[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = static_cast<float>(xp[i]);
    xd[i] = x[i] * d;
  }
  __syncthreads();
  v4f y = {0, 0, 0, 0};
  for (int j0 = 0; j0 * rows < a.states; j0 += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int n = r0 + (j0 + j) * rows;
      if (live && n < a.states) {
        const long at = base + static_cast<long>(n) * a.width + 4 * q;
        v4f v = j0 == 0 ? s[j] : *reinterpret_cast<const v4f*>(sa.state + at);
        const float b = sb[n], c = sc[n];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = fmaf(decay, v[i], b * xd[i]);
          y[i] = fmaf(c, v[i], y[i]);
        }
        *reinterpret_cast<v4f*>(sa.new_state + at) = v;
      }
    }
  }
  if (live) *reinterpret_cast<v4f*>(&lds[(r0 * quads + q) * 4]) = y;
  __syncthreads();
  if (tid < a.width) {
    float v = 0.0f;
    for (int r = 0; r < rows; ++r) v += lds[r * a.width + tid];
    const float xv = static_cast<float>((static_cast<const T*>(a.x.data) + seq * a.x.batch_stride)[h * a.width + tid]);
    if (a.D != nullptr) v = fmaf(a.D[h], xv, v);
    (static_cast<T*>(a.y.data) + seq * a.y.batch_stride)[h * a.width + tid] = static_cast<T>(v);
  }
}

// --------------------------------------------------------------------- host
template <class T, int NB, int NW>
int launch_fwd(const SsmArgs& a, const Walk& w, bool segments, unsigned blocks, hipStream_t s) {
  if (segments) {
    ssm_summary_kernel<T, NB, NW><<<blocks, NW * 64, 0, s>>>(a, w);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    if (!a.fold) {
      const unsigned quads = static_cast<unsigned>((a.states * a.width + 1023) / 1024);
      ssm_carry_kernel<<<dim3(quads, a.heads, a.q.batch), 256, 0, s>>>(a, w);
      if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    }
  }
  ssm_fwd_kernel<T, NB, NW><<<blocks, NW * 64, 0, s>>>(a, w);
  return launch_status();
}

template <class T, int NB>
int launch_fwd_width(const SsmArgs& a, const Walk& w, bool segments, unsigned blocks, int nw,
                     hipStream_t s) {
  switch (nw) {
    case 1: return launch_fwd<T, NB, 1>(a, w, segments, blocks, s);
    case 2: return launch_fwd<T, NB, 2>(a, w, segments, blocks, s);
    default: return launch_fwd<T, NB, 4>(a, w, segments, blocks, s);
  }
}

template <class T>
int launch_fwd_states(const SsmArgs& a, const Walk& w, bool segments, unsigned blocks, int nw,
                     hipStream_t s) {
  if (a.states <= 32) return launch_fwd_width<T, 1>(a, w, segments, blocks, nw, s);
  if (a.states <= 64) return launch_fwd_width<T, 2>(a, w, segments, blocks, nw, s);
  return launch_fwd_width<T, 4>(a, w, segments, blocks, nw, s);
}

}  // namespace

namespace ssm {

int check_dims(const mamba2_seqs& q, const mamba2_ssm_dims& d) {
  if (!type_ok(d.type) || !type_ok(d.dt_type)) return MAMBA2_SCAN_EUNSUPPORTED;
  const int st = check_seqs(q);
  if (st != MAMBA2_SCAN_OK) return st;
  if (d.heads < 1 || d.groups < 1 || d.width < 1 || d.states < 1 || d.heads % d.groups != 0) return MAMBA2_SCAN_EBADDIM;
  if (d.width % 8 != 0 || d.states % 8 != 0 || d.width > kMaxDim || d.states > kMaxDim || d.heads > 65535 ||
      q.batch > 65535)
    return MAMBA2_SCAN_EUNSUPPORTED;
  return MAMBA2_SCAN_OK;
}

// Rows that are accessed in 16-byte vectors.
int check_vec_rows(const mamba2_rows& r, const mamba2_seqs& q, long long width, size_t elem) {
  const int st = check_rows(r, q, width, elem);
  if (st != MAMBA2_SCAN_OK || q.length == 0) return st;
  const long long n = 8;
  if (!aligned_to(r.data, 16)) return MAMBA2_SCAN_EALIGN;
  // a step's 64 rows of either type are addressed with 31-bit offsets
  if (q.length > 1 && r.row_stride > (1LL << 29) / (kTok + 1)) return MAMBA2_SCAN_EUNSUPPORTED;
  if ((q.length > 1 && r.row_stride % n != 0) || (q.offsets == nullptr && q.batch > 1 && r.batch_stride % n != 0))
    return MAMBA2_SCAN_EALIGN;
  return MAMBA2_SCAN_OK;
}

// dt: any stride that the same offsets reach.
int check_step_rows(const mamba2_rows& r, const mamba2_seqs& q, const mamba2_ssm_dims& d) {
  const int st = check_rows(r, q, d.heads, type_size(d.dt_type));
  if (st != MAMBA2_SCAN_OK) return st;
  return q.length > 1 && r.row_stride > (1LL << 29) / (kTok + 1) ? MAMBA2_SCAN_EUNSUPPORTED : MAMBA2_SCAN_OK;
}

int waves_of(int width) { return width <= 16 ? 1 : width <= 32 ? 2 : 4; }

// Tokens per segment.  A work-group walks its tokens one step after another,
// so short of one or two rounds of work-groups the tokens are cut into
// segments.  Each costs a second reading of x and B and a state, and all of
// them one launch or two, so no more than needed, and none where a few steps do:
// six in the forward (8 heads of 64, 128 states, bf16, GPU time: 4 steps 17.5 us,
// cut 18.7; 6 steps 22.6, cut 19.5; 10 steps 35.7, cut 21.6; but a launch more
// costs the host 4 us: 6 steps and their backward, called from Python, 56 us, cut
// 60, 7 steps 62, cut 60), ten in the backward, where the walk is a part of the
// time (8 steps 47.6 us, cut 47.8; 10 steps 51.9, cut 50.3; 16 heads of 128: 67.5,
// cut 70.4; 13 steps, 24 heads, 64 states: 59.9, cut 58.2).  The lengths of packed
// sequences are not known here: up to ten steps of rows are taken to be shared out
// evenly (10 of 64 tokens: 9.9 us, cut 12.1).
// A CU holds two work-groups with up to 128 states (LDS) and three with up to 64
// (registers); one work-group more than the rounds hold costs a round (24 heads,
// 64 states: 1032 work-groups 109 us, 768 89 us).  Packed sequences' ends add units
// by themselves: half as many segments again, for their unequal lengths, took
// 0.93 to 1.28 times as long over seven mixes of 1 to 32 prompts.
int segment_tokens(const mamba2_seqs& q, const mamba2_ssm_dims& d, bool bwd) {
  constexpr int kFewSteps = 6, kFewStepsBwd = 10;
  const bool packed = q.offsets != nullptr;
  const long work = static_cast<long>(kCUs) * (d.states > 64 ? 2 : 3);
  const long slices = (d.width + waves_of(d.width) * 16 - 1) / (waves_of(d.width) * 16);
  const long lanes = static_cast<long>(d.heads) * slices * (packed ? 1 : q.batch);
  const long want = work / lanes > 1 ? work / lanes : 1;  // segments, over all rows of a packed call
  long seg = (q.length + want - 1) / want;
  const long few = (bwd ? kFewStepsBwd : packed ? min(static_cast<long>(kFewSteps) * q.batch, 10L) : kFewSteps) * kTok;
  if (q.length <= few) seg = q.length;
  seg = (seg + kTok - 1) / kTok * kTok;
  return static_cast<int>(seg < 2 * kTok ? 2 * kTok : seg);
}

// Few segments add up the states before them themselves: i of them read
// i (i - 1) / 2 states where the carry pass reads and writes 2 (i - 1) in a launch
// of its own.  Forwards of 256 tokens a segment that fill the chip, us, added up
// and carried: 128 states 4 segments 49.8 and 50.7, 6 segments 50.2 and 48.2, 16
// segments 58 and 50; 64 states 46.3 and 48.0, 46.5 and 46.1, 51.8 and 48.6.
// How a packed call's rows are shared out is not known here; with several
// sequences each is taken to have a part of them (128 states, forwards, 3 alike
// with 12 segments 60.8 and 63.8, 6 with 16 segments 61.5 and 67.3; 3 of which one
// has nine tenths, 12 segments: 73 and 65).
int fold_segments(const mamba2_seqs& q, const mamba2_ssm_dims& d, int seg) {
  return units_of(q.length, seg) <= (d.states > 64 ? 4 : 6) * (q.offsets != nullptr ? min(q.batch, 4) : 1);
}

// check_dims, and that the passes over the segments can be launched.
int check_scan(const mamba2_seqs& q, const mamba2_ssm_dims& d, bool bwd) {
  const int st = check_dims(q, d);
  if (st != MAMBA2_SCAN_OK) return st;
  const int nw = waves_of(d.width), slices = (d.width + nw * 16 - 1) / (nw * 16);
  const long long units = unit_count(q, segment_tokens(q, d, bwd));
  return grid_ok(units * d.heads * slices, nw * 64) ? MAMBA2_SCAN_OK : MAMBA2_SCAN_EBADDIM;
}

}  // namespace ssm

extern "C" {

const char* mamba2_layer_strerror(int status) {
  switch (status) {
    case MAMBA2_SCAN_OK: return "success";
    case MAMBA2_SCAN_EBADDIM: return "invalid dimension or stride (sizes positive, strides not shorter than a row)";
    case MAMBA2_SCAN_EUNSUPPORTED: return "unsupported type or size (taps 2-4; width and states multiples of 8 up to 128)";
    case MAMBA2_SCAN_ENULL: return "a required pointer is NULL";
    case MAMBA2_SCAN_ESIZE: return "workspace is smaller than required";
    case MAMBA2_SCAN_EALIGN: return "a pointer or stride is not aligned as required (the scan: 16 bytes, strides 8 elements)";
    case MAMBA2_SCAN_EHIP: return "HIP runtime error while enqueuing a kernel";
    case MAMBA2_SCAN_EOVERLAP: return "tensors that must be apart overlap";
    default: return "unknown status";
  }
}

size_t mamba2_ssm_fwd_workspace_bytes(mamba2_seqs q, mamba2_ssm_dims d) {
  if (check_scan(q, d, false) != MAMBA2_SCAN_OK) return 0;
  const int seg = segment_tokens(q, d, false);
  if (q.length <= seg) return 0;
  const size_t n = static_cast<size_t>(unit_count(q, seg)) * d.heads * (static_cast<size_t>(d.states) * d.width + 1);
  return (n * sizeof(float) + 15) / 16 * 16;
}

int mamba2_ssm_fwd(mamba2_seqs q, mamba2_ssm_dims d, mamba2_rows x, mamba2_rows dt, const float* A, mamba2_rows B,
                   mamba2_rows C, const float* D, const float* dt_bias, const float* initial_state, mamba2_rows y,
                   float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_scan(q, d, false);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(d.type);
  const long long xw = static_cast<long long>(d.heads) * d.width, bw = static_cast<long long>(d.groups) * d.states;
  if (A == nullptr) return MAMBA2_SCAN_ENULL;
  x = used_strides(x, q, xw);
  y = used_strides(y, q, xw);
  B = used_strides(B, q, bw);
  C = used_strides(C, q, bw);
  dt = used_strides(dt, q, d.heads);
  if ((st = check_vec_rows(x, q, xw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(B, q, bw, e)) != MAMBA2_SCAN_OK ||
      (st = check_vec_rows(C, q, bw, e)) != MAMBA2_SCAN_OK || (st = check_vec_rows(y, q, xw, e)) != MAMBA2_SCAN_OK ||
      (st = check_step_rows(dt, q, d)) != MAMBA2_SCAN_OK)
    return st;
  if (!aligned_to(A, 4) || !aligned_to(D, 4) || !aligned_to(dt_bias, 4) || !aligned_to(initial_state, 16) ||
      !aligned_to(final_state, 16))
    return MAMBA2_SCAN_EALIGN;
  const size_t need = mamba2_ssm_fwd_workspace_bytes(q, d);
  if (need > 0) {
    if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
    if (workspace_bytes < need) return MAMBA2_SCAN_ESIZE;
    if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  }
  if (q.length == 0 && final_state == nullptr) return MAMBA2_SCAN_OK;
  SsmArgs a = {};
  a.q = q;
  a.x = x;
  a.dt = dt;
  a.B = B;
  a.C = C;
  a.y = y;
  a.A = A;
  a.D = D;
  a.bias = dt_bias;
  a.initial = initial_state;
  a.final_state = final_state;
  a.heads = d.heads;
  a.width = d.width;
  a.ratio = d.heads / d.groups;
  a.states = d.states;
  a.softplus = d.softplus;
  a.dt_bf16 = d.dt_type == MAMBA2_BF16;
  const int nw = waves_of(d.width);
  a.slices = (d.width + nw * 16 - 1) / (nw * 16);
  a.seg = segment_tokens(q, d, false);
  a.units = static_cast<int>(unit_count(q, a.seg));
  a.fold = fold_segments(q, d, a.seg);
  Walk w = {};
  w.v = x;
  w.m = B;
  w.first = initial_state;
  w.seg_state = static_cast<float*>(workspace);
  w.seg_decay = need > 0 ? w.seg_state + static_cast<size_t>(a.units) * d.heads * d.states * d.width : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned n = static_cast<unsigned>(a.units) * a.heads * a.slices;
  return d.type == MAMBA2_BF16 ? launch_fwd_states<bf16>(a, w, need > 0, n, nw, s)
                               : launch_fwd_states<float>(a, w, need > 0, n, nw, s);
}

int mamba2_ssm_step(int batch, mamba2_ssm_dims d, mamba2_rows x, mamba2_rows dt, const float* A, mamba2_rows B,
                    mamba2_rows C, const float* D, const float* dt_bias, const float* state, mamba2_rows y,
                    float* new_state, void* stream) {
  const mamba2_seqs q = {batch, 1, nullptr};
  int st = check_dims(q, d);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(d.type);
  const long long xw = static_cast<long long>(d.heads) * d.width, bw = static_cast<long long>(d.groups) * d.states;
  if (A == nullptr || state == nullptr || new_state == nullptr) return MAMBA2_SCAN_ENULL;
  if ((st = check_rows(x, q, xw, e)) != MAMBA2_SCAN_OK || (st = check_rows(B, q, bw, e)) != MAMBA2_SCAN_OK ||
      (st = check_rows(C, q, bw, e)) != MAMBA2_SCAN_OK || (st = check_rows(y, q, xw, e)) != MAMBA2_SCAN_OK ||
      (st = check_rows(dt, q, d.heads, type_size(d.dt_type))) != MAMBA2_SCAN_OK)
    return st;
  if (!aligned_to(A, 4) || !aligned_to(D, 4) || !aligned_to(dt_bias, 4) || !aligned_to(state, 16) ||
      !aligned_to(new_state, 16))
    return MAMBA2_SCAN_EALIGN;
  const long long all = 4LL * batch * xw * d.states, vec = 4LL * d.heads;
  const Region mem[] = {token_region(y, batch, xw, e), region(new_state, all), token_region(x, batch, xw, e),
                        token_region(dt, batch, d.heads, type_size(d.dt_type)), token_region(B, batch, bw, e),
                        token_region(C, batch, bw, e), region(A, vec), region(D, vec), region(dt_bias, vec),
                        region(state != new_state ? state : nullptr, all)};
  if (!apart(mem, 2, 10)) return MAMBA2_SCAN_EOVERLAP;
  StepArgs sa = {};
  SsmArgs& a = sa.a;
  a.x = x;
  a.dt = dt;
  a.B = B;
  a.C = C;
  a.y = y;
  a.A = A;
  a.D = D;
  a.bias = dt_bias;
  a.heads = d.heads;
  a.width = d.width;
  a.ratio = d.heads / d.groups;
  a.states = d.states;
  a.softplus = d.softplus;
  a.dt_bf16 = d.dt_type == MAMBA2_BF16;
  sa.state = state;
  sa.new_state = new_state;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(d.heads, batch);
  if (d.type == MAMBA2_BF16) ssm_step_kernel<bf16><<<grid, kStepThreads, 0, s>>>(sa);
  else ssm_step_kernel<float><<<grid, kStepThreads, 0, s>>>(sa);
  return launch_status();
}

}  // extern "C"
