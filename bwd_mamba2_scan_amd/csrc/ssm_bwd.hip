// Backward of the selective state space scan for gfx950.
//
// With G_t the gradient of the state S_t (G_t = C_t d_y_t^T + e^(d A)_{t+1} G_{t+1}):
//   d_x_t = d_t G_t^T B_t + D d_y_t          d_B_t = sum_heads G_t (d_t x_t)
//   d_C_t = sum_heads S_t d_y_t              d_S_0 = e^(d A)_1 G_1
//   d_d_t = x_t . (G_t^T B_t) + A m_t        d_A = sum_t d_t m_t,  m_t = <G_t, e^(d A)_t S_{t-1}>
// where m_t is the gradient of token t's log decay: everything that flows
// from before t to t or behind it.
//
// Two passes.  The walk (ssm_walk_kernel) recomputes the state forward and its
// gradient in reverse, side by side, and writes both at every step of 64
// tokens.  ssm_bwd_kernel then takes all steps in parallel: a work-group owns
// the 64 tokens of one step and a run of the heads that share B and C, so d_B
// and d_C are summed over heads in registers, in a fixed order.  In a step,
// per head, with E[t][s] = 2^(c_t - c_s) (s <= t):
//   P = (C B^T) o E,  Q = (d_y x^T) o E o d
//   d_x = d o (P^T d_y + 2^(c_end-c) o (B G))        + D d_y
//   d_B = Q^T C + 2^(c_end-c) d o (x G^T)
//   d_C = Q B   + 2^c o (d_y S^T)
// m_t is a sum of terms that are all of its own kind: pairs s < t <= t' of
// P o d_y x^T, the step's starting state into rows at or behind t, rows before t
// into what follows the step, and the starting state through the whole step.
// Nothing is obtained as a difference of larger sums.
#include "ssm_common.h"

#include <initializer_list>

namespace {

using namespace ssm;

struct BwdArgs {
  SsmArgs a;
  mamba2_rows d_y, d_x, d_dt, d_B, d_C;
  const float* keep_s;     // the walk's kept states
  const float* keep_g;
  float* part;             // [steps][heads][4]: d_A, d_D, d_dt_bias of the step
  float* part_b;           // [splits][rows][groups][states]: d_B of a run of heads
  float* part_c;
  long rows;
  int steps;
  int groups;
  int splits;              // runs of heads per group
  int run;                 // heads per run
};

// The walk is bound by HBM: it writes the kept states, 537 MB, and reads 179 MB in
// 126 us, 5.7 TB/s.  Its summaries take 63 us.
struct Walks {  // forward, reverse: side by side in one launch
  Walk w[2];
};

template <class T, int NB, int NW>
__global__ __launch_bounds__(NW * 64, simd_waves(sizeof(WalkLds<T, NB, NW>), NW, 2)) void ssm_walk_kernel(SsmArgs a, Walks ws) {
  __shared__ WalkLds<T, NB, NW> s;
  walk<T, NB, NW, true>(a, ws.w[blockIdx.y], s);
}
template <class T, int NB, int NW>
__global__ __launch_bounds__(NW * 64, simd_waves(sizeof(WalkLds<T, NB, NW>), NW, 2)) void ssm_walk_summary_kernel(SsmArgs a, Walks ws) {
  __shared__ WalkLds<T, NB, NW> s;
  walk<T, NB, NW, false>(a, ws.w[blockIdx.y], s);
}
__global__ __launch_bounds__(256) void ssm_walk_carry_kernel(SsmArgs a, Walks ws) {
  carry(a, ws.w[blockIdx.x & 1], blockIdx.z, blockIdx.x >> 1);
}

constexpr int kBwdThreads = 512;

// A state in LDS.  bf16: strips of 16 columns, each with its rows one after
// the other (32 bytes a row), so that a tile is written, and an operand read by
// rows or by columns, from neighbouring banks without padding; three parts of
// both states fit that way.  fp32: rows of LD.
template <class T, int ROWS, int COLS, int LD>
struct StateLds {
  static constexpr bool kStrips = sizeof(T) == 2;
  static constexpr int kSize = ROWS * (kStrips ? COLS : LD);
  static __device__ __forceinline__ int at(int row, int col) {
    return kStrips ? (col >> 4) * (ROWS * 16) + row * 16 + (col & 15) : row * LD + col;
  }
  static __device__ __forceinline__ Frag<T> by_row(const T* p, int row, int k0, int l) {
    if constexpr (kStrips)
      return {*reinterpret_cast<const v8bf*>(p + (k0 >> 4) * (ROWS * 16) + (l >> 5) * (ROWS * 16) +
                                             (row + (l & 15)) * 16 + (l >> 4 & 1) * 8)};
    else
      return frag_row(p, LD, row, k0, l);
  }
  static __device__ __forceinline__ Frag<T> by_col(const T* p, int k0, int col, int l) {
    if constexpr (kStrips) return frag_col(p + (col >> 4) * (ROWS * 16), 16, k0, 0, l);
    else return frag_col(p, LD, k0, col, l);
  }
};

template <class T, int NB, int PT>
struct BwdLds {
  static constexpr int kN = NB * 32;
  static constexpr int kP = PT * 16 < 32 ? 32 : PT * 16;  // a product over the columns takes 32 at a time
  static constexpr int kTerms = sizeof(T) == 2 ? 3 : 1;
  // Parts of P and Q, and of the gradient's state in d_B: with one, Q's rounding
  // shows in d_B and d_C (2.4e-3 against 1.66e-3, their own rounding), P's in d_x
  // (1.89e-3), the state's in d_B (1.71e-3).
  static constexpr int kParts = sizeof(T) == 2 ? 2 : 1;
  static constexpr int kRows = sizeof(T) == 2 || kN < 64 ? kN : 64;  // state rows staged at a time
  // b and c are read by rows and, in fours of neighbouring ones, by columns:
  // 32 bytes of padding put four rows of 128 bf16 into different banks
  static constexpr int ldn = stride_of<T>(kN) + (sizeof(T) == 2 && kN == 128 ? 8 : 0);
  static constexpr int ldp = stride_of<T>(kP);
  alignas(16) T b[kTok * ldn];
  alignas(16) T c[kTok * ldn];
  alignas(16) T x[kTok * ldp];
  alignas(16) T dy[kTok * ldp];
  typedef StateLds<T, kRows, kP, ldp> State;
  alignas(16) T st[2][kTerms][State::kSize];  // rows of the starting state and of the gradient behind the step
  alignas(16) DecaysOf<true> dc[3];  // of the head before (its gradients are put together), this one and the next
  float slope[3][kTok];      // d d_t / d dt_t
  struct Sums {              // of a head and the one before
    float inner[4][kTok];    // m_t: pairs within the step, per wave's columns
    float after[kTok];       // starting state into row t
    float before[kTok];      // row t into what follows (without d)
    float direct[kTok];      // x . P^T d_y
    float whole[8];          // starting state through the step, per wave
    float skip[4];           // sum d_y . x, per wave
  } sums[2];
};

// Rows of a [states][width] fp32 matrix slice in registers, then LDS, where a
// bf16 product finds them whole, in three parts.  d_x and d_C would do with
// two, but d_A and d_dt_bias, fp32 sums of terms of both signs, show the third:
// 2e-7 of them against 7e-7, and 1.5e-6 over short sequences (for 40 us at
// 4 x 4096 tokens, 32 heads of 64 columns, 128 states).
template <class T, int NB, int PT>
struct StateTile {
  typedef BwdLds<T, NB, PT> L;
  static constexpr int kTiles = L::kRows / 16;                // of a strip of 16 columns
  static constexpr int kAll = kTiles * (L::kP / 16);          // a tile per wave and turn
  static constexpr int kWaves = kBwdThreads / 64;
  static constexpr int kN = (kAll + kWaves - 1) / kWaves;
  v4f v[kN];
  // From strip0 and tile0 on; what the state does not have is zero.
  __device__ __forceinline__ void load(const float* kept, int width, int states, int strip0, int tile0) {
    const int strips = tiles_of(width), tiles = tiles_of(states), lane = threadIdx.x & 63;
    const Rsrc rs = make_rsrc(kept, static_cast<unsigned>(strips * tiles * kKeptTile * 4));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int t = wave_id() + i * kWaves, strip = strip0 + t / kTiles, tile = tile0 + t % kTiles;
      const bool in = t < kAll && strip < strips && tile < tiles;
      v[i] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
                                         rs, (in ? (strip * tiles + tile) * kKeptTile * 4u : kOutside) + lane * 16, 0,
                                         kNonTemporal));
    }
  }
  __device__ __forceinline__ void store(T (&st)[L::kTerms][L::State::kSize]) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int t = wave_id() + i * kWaves;
      if (kAll % kWaves != 0 && t >= kAll) continue;
      quad_put_parts<L::kTerms>(&st[0][L::State::at(t % kTiles * 16 + (lane & 15), t / kTiles * 16 + 4 * (lane >> 4))],
                                L::State::kSize, v[i]);
    }
  }
};

// Two result tiles stacked along k as one operand.
template <class T, int TERMS>
__device__ __forceinline__ Split<T, TERMS> split_tiles(const v4f& a, const v4f& b) {
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split_of<T, TERMS>(v);
}

// The lane's number, as if it could change: what is computed from it stays in
// its round.  Kept across rounds, the addresses would cost more registers than
// there are (and a spilled register's reload waits for the loads in flight).
__device__ __forceinline__ int lane_anew() {
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));
  return l;
}

// A quad of columns from column c of a result's row: stored where it exists.
template <class T>
__device__ __forceinline__ void put_quad(Rsrc rs, int row_off, int c, int cols, v4f v) {
  Quad<T>::store(rs, c < cols ? static_cast<unsigned>((row_off + c) * static_cast<int>(sizeof(T))) : kOutside, v);
}

// At 4 x 4096 tokens, 32 heads of 64 columns, 128 states, bf16: 317 us (301 at
// best) for 681 MB read (the kept states 537 MB, in fp32) and 103 MB written.  The
// bytes would take 154 us; LDS is busy 43 % of the time, the matrix cores 16 %,
// and half of the waves' time is waiting: for a head's states, which
// are loaded one head ahead (the registers hold no more), and at the two barriers
// of a head.  The staging alone, without the products, takes 188 us.
// Eight waves: the first four own 16 rows each of d_x and d_B (rows s), the
// others 16 rows each of d_C (rows t), so that they work on the gradient
// behind the step and on the starting state at the same time.  Wave w of the
// one kind and of the other share a SIMD; their shares of the triangle, 4 - w
// and w + 1 tiles, add up to the same for all.
// Results lie so that a lane has one row (token) and four neighbouring
// columns: a row's factor is one value, and results go out as they are.
template <class T, int NB, int PT>
__global__ __launch_bounds__(kBwdThreads, 2) void ssm_bwd_kernel(BwdArgs ba) {
  typedef BwdLds<T, NB, PT> L;
  typedef StateTile<T, NB, PT> ST;
  __shared__ L s;
  const SsmArgs& a = ba.a;
  constexpr int kKp = L::kP / 32;   // 32-wide product steps over the columns
  constexpr int kPt = L::kP / 16;
  constexpr int kPhases = L::kN / L::kRows;
  constexpr int kNt = L::kRows / 16;  // 16-row tiles of the state per phase
  constexpr int kBatch = 2 * NB < 4 ? 2 * NB : 4;
  constexpr int kSide = kNt < 4 ? kNt : 4;
  const int tid = threadIdx.x, id = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const bool for_x = id < 4;
  const int wave = id & 3;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int split = work % ba.splits;
  const int gr = work / ba.splits % ba.groups;
  const int step = work / ba.splits / ba.groups;
  const Unit u = locate(a.q, step, kTok);
  const bool packed = a.q.offsets != nullptr;
  const int rows = min(u.len - u.t0, kTok);
  const int h0 = gr * a.ratio + split * ba.run;
  const int h1 = min(h0 + ba.run, (gr + 1) * a.ratio);
  if (rows <= 0) {  // a step without tokens adds nothing
    for (int i = tid; i < (h1 - h0) * 4; i += kBwdThreads) ba.part[(static_cast<long>(step) * a.heads + h0) * 4 + i] = 0.0f;
    return;
  }
  const int row = wave * 16;                // this wave's rows
  const int mine = row + l15;               // this lane's row
  const int slices = (a.width + L::kP - 1) / L::kP;

  const T* xp = seq_ptr<const T>(a.x, u.seq, u.row0, packed) + u.t0 * a.x.row_stride;
  const T* gp = seq_ptr<const T>(ba.d_y, u.seq, u.row0, packed) + u.t0 * ba.d_y.row_stride;
  T* op = seq_ptr<T>(ba.d_x, u.seq, u.row0, packed) + u.t0 * ba.d_x.row_stride;
  const Rsrc rdt = step_rsrc(a, u, packed, u.t0, rows);
  {
    Tile<T, kTok, L::kN, kBwdThreads> tb, tc;
    tb.init(a.B.row_stride, a.states, tid);
    tc.init(a.C.row_stride, a.states, tid);
    tb.load(rows_rsrc(seq_ptr<const T>(a.B, u.seq, u.row0, packed) + u.t0 * a.B.row_stride + gr * a.states,
                      a.B.row_stride, rows, a.states));
    tc.load(rows_rsrc(seq_ptr<const T>(a.C, u.seq, u.row0, packed) + u.t0 * a.C.row_stride + gr * a.states,
                      a.C.row_stride, rows, a.states));
    tb.store(s.b, L::ldn, tid);
    tc.store(s.c, L::ldn, tid);
    s.sums[id >> 2].inner[wave][lane] = 0.0f;  // rows before a wave's columns stay zero
  }

  Tile<T, kTok, L::kP, kBwdThreads> tx, ty;
  ST ts, tg;
  const auto fetch_rows = [&](int h, int p0) {
    const int cols = min(a.width - p0, L::kP);
    tx.init(a.x.row_stride, cols, tid);
    ty.init(ba.d_y.row_stride, cols, tid);
    tx.load(rows_rsrc(xp + h * a.width + p0, a.x.row_stride, rows, cols));
    ty.load(rows_rsrc(gp + h * a.width + p0, ba.d_y.row_stride, rows, cols));
  };
  const auto fetch_states = [&](int h, int p0, int phase) {
    const long at = (static_cast<long>(step) * a.heads + h) * kept_size(a.width, a.states);
    ts.load(ba.keep_s + at, a.width, a.states, p0 / 16, phase * ST::kTiles);
    tg.load(ba.keep_g + at, a.width, a.states, p0 / 16, phase * ST::kTiles);
  };
  // Two of the waves with less to multiply prepare the next head's decays
  // and put the last head's gradients together meanwhile.
  const bool decays = id == 5, finishes = id == 4;
  float raw = 0.0f;
  const auto prepare = [&](int h, int k) {
    const int lane = lane_anew();
    const float bias = a.bias != nullptr ? a.bias[h] : 0.0f;
    make_decays(s.dc[k], lane < rows ? step_of(a, raw, bias) : 0.0f, decay_rate(a.A[h]));
    s.slope[k][lane] = a.softplus ? __builtin_amdgcn_rcpf(1.0f + expf(-(raw + bias))) : 1.0f;
  };
  // The step sizes' gradients of a head whose sums are complete: a token per lane.
  const auto finish = [&](int h, int k, int par) {
    const int lane = lane_anew();
    const auto& sum = s.sums[par];
    const DecaysOf<true>& dc = s.dc[k];
    const float A = a.A[h], d = dc.d[lane];
    const float after = __shfl(scan64(sum.after[63 - lane]), 63 - lane);
    float upto = __shfl_up(scan64(d * sum.before[lane]), 1);
    if (lane == 0) upto = 0.0f;
    const float whole = (((sum.whole[0] + sum.whole[1]) + (sum.whole[2] + sum.whole[3])) +
                         ((sum.whole[4] + sum.whole[5]) + (sum.whole[6] + sum.whole[7]))) * dc.total;
    const float inner = (sum.inner[0][lane] + sum.inner[1][lane]) + (sum.inner[2][lane] + sum.inner[3][lane]);
    const float m = inner + after + upto + whole;
    float dd = (sum.direct[lane] + sum.before[lane] + A * m) * s.slope[k][lane];
    float dA = d * m;
    if (lane < rows) {
      const long i = (u.t0 + lane) * ba.d_dt.row_stride + h;
      if (a.dt_bf16) seq_ptr<bf16>(ba.d_dt, u.seq, u.row0, packed)[i] = static_cast<bf16>(dd);
      else seq_ptr<float>(ba.d_dt, u.seq, u.row0, packed)[i] = dd;
    } else {
      dd = dA = 0.0f;
    }
    dA = sum64(dA);
    dd = sum64(dd);
    if (lane == 0) {
      float* p = ba.part + (static_cast<long>(step) * a.heads + h) * 4;
      p[0] = dA;
      p[1] = (sum.skip[0] + sum.skip[1]) + (sum.skip[2] + sum.skip[3]);
      p[2] = dd;
      p[3] = 0.0f;
    }
  };

  fetch_rows(h0, 0);
  fetch_states(h0, 0, 0);
  if (decays) {
    raw = load_raw(a, rdt, h0);
    prepare(h0, 0);
    if (h0 + 1 < h1) raw = load_raw(a, rdt, h0 + 1);
  }
  v4f acc[2 * NB];  // d_B or d_C
#pragma unroll
  for (int n = 0; n < 2 * NB; ++n) acc[n] = v4f{0, 0, 0, 0};
  v4f cb[4];  // (C B^T)[t][s], column s = mine, rows t = 16 ti + 4 g + i
  __syncthreads();
#pragma unroll
  for (int ti = 0; ti < 4; ++ti) {
    cb[ti] = v4f{0, 0, 0, 0};
    if (for_x && ti >= wave) {
#pragma unroll
      for (int k = 0; k < NB; ++k) mma(cb[ti], frag_row(s.c, L::ldn, ti * 16, k * 32), frag_row(s.b, L::ldn, row, k * 32));
    }
  }

  int cur = 0, par = 0;
  for (int h = h0; h < h1; ++h) {
    const float D = a.D != nullptr ? a.D[h] : 0.0f;
    const int next = cur == 2 ? 0 : cur + 1, last = cur == 0 ? 2 : cur - 1;
    const DecaysOf<true>& dc = s.dc[cur];
    auto& sum = s.sums[par];
    for (int slice = 0; slice < slices; ++slice) {
      const int p0 = slice * L::kP, cols = min(a.width - p0, L::kP);
      const int ln = lane_anew();
      const int l15 = ln & 15, g = ln >> 4, mine = row + l15;
      const bool more = slice + 1 < slices || h + 1 < h1;  // a round follows this one, of:
      const int hn = slice + 1 < slices ? h : h + 1, pn = slice + 1 < slices ? p0 + L::kP : 0;
      v4f dx[kPt];
      float whole = 0.0f, edge = 0.0f;  // edge: x . (what follows), or C . (starting state)
#pragma unroll
      for (int p = 0; p < kPt; ++p) dx[p] = v4f{0, 0, 0, 0};
      for (int ph = 0; ph < kPhases; ++ph) {
#pragma unroll
        for (int i = 0; i < ST::kN; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) whole = fmaf(ts.v[i][j], tg.v[i][j], whole);
        __syncthreads();  // the last round's readers are done
        if (ph == 0) {
          tx.store(s.x, L::ldp, tid);
          ty.store(s.dy, L::ldp, tid);
        }
        ts.store(s.st[0]);
        tg.store(s.st[1]);
        __syncthreads();
        if (ph + 1 < kPhases) {
          fetch_states(h, p0, ph + 1);
        } else if (more) {
          fetch_rows(hn, pn);
          fetch_states(hn, pn, 0);
        }
        if (ph == 0 && slice == 0) {
          if (finishes && h > h0) finish(h - 1, last, par ^ 1);
          if (decays && h + 1 < h1) {
            prepare(h + 1, next);
            if (h + 2 < h1) raw = load_raw(a, rdt, h + 2);
          }
        }
        if (for_x) {
          if (ph == 0) {
            // ---- within the step, column s = mine
            const float ch = dc.hi[mine], cl = dc.lo[mine], d = dc.d[mine];
            v4f pw[4], qw[4];
            float direct = 0.0f, skip = 0.0f, behind = 0.0f;
#pragma unroll
            for (int ti = 3; ti >= 0; --ti) {
              pw[ti] = qw[ti] = v4f{0, 0, 0, 0};
              if (ti < wave) continue;
              v4f yx = {0, 0, 0, 0};
#pragma unroll
              for (int k = 0; k < kKp; ++k)
                mma(yx, frag_row(s.dy, L::ldp, ti * 16, k * 32, ln), frag_row(s.x, L::ldp, row, k * 32, ln));
              const int t0 = ti * 16 + 4 * g;
              const v4f hi = *reinterpret_cast<const v4f*>(&dc.hi[t0]), lo = *reinterpret_cast<const v4f*>(&dc.lo[t0]);
              v4f pair;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float e = exp2_of((hi[i] - ch) + (lo[i] - cl));
                if (ti == wave) e = 4 * g + i >= l15 ? e : 0.0f;
                pw[ti][i] = cb[ti][i] * e;
                qw[ti][i] = yx[i] * (e * d);
                pair[i] = pw[ti][i] * yx[i];
                direct += pair[i];
                if (ti == wave) {
                  if (4 * g + i == l15) skip = yx[i];
                  pair[i] = 4 * g + i > l15 ? pair[i] : 0.0f;
                }
              }
              // the column's pairs at rows >= t: in the lane, over the lane
              // groups behind, and over the tiles behind
              pair[2] += pair[3];
              pair[1] += pair[2];
              pair[0] += pair[1];
              const Pair two = swap16(pair[0]);          // groups 0 and 1, or 2 and 3
              const Pair all = swap32(two.a + two.b);    // the first two, the last two
              const float rest = behind + ((g & 1) == 0 ? two.b : 0.0f) + (g < 2 ? all.b : 0.0f);
              v4f v;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[i] = (pair[i] + rest) * d;
                if (ti == wave) v[i] = l15 < 4 * g + i ? v[i] : 0.0f;
                v[i] = sum16(v[i]);
              }
              if (l15 == 0) {
                v4f* o = reinterpret_cast<v4f*>(&sum.inner[wave][t0]);
                *o = slice == 0 ? v : *o + v;
              }
              behind += all.a + all.b;
            }
            direct = sum_groups(direct);
            if (g == 0) sum.direct[mine] = slice == 0 ? direct : sum.direct[mine] + direct;
            skip = sum64(skip);
            if (lane == 0) sum.skip[wave] = slice == 0 ? skip : sum.skip[wave] + skip;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (2 * k + 1 < wave) continue;
              const auto pf = split_tiles<T, L::kParts>(pw[2 * k], pw[2 * k + 1]);
              const auto qf = split_tiles<T, L::kParts>(qw[2 * k], qw[2 * k + 1]);
#pragma unroll
              for (int p = 0; p < kPt; ++p) {
                const Frag<T> yf = frag_col_result(s.dy, L::ldp, k * 32, p * 16, ln);
#pragma unroll
                for (int z = 0; z < L::kParts; ++z) mma(dx[p], yf, pf.f[z]);
              }
#pragma unroll
              for (int n0 = 0; n0 < 2 * NB; n0 += kBatch) {
                Frag<T> cf[kBatch];
#pragma unroll
                for (int n = 0; n < kBatch; ++n) cf[n] = frag_col_result(s.c, L::ldn, k * 32, (n0 + n) * 16, ln);
#pragma unroll
                for (int z = 0; z < L::kParts; ++z)
#pragma unroll
                  for (int n = 0; n < kBatch; ++n) mma(acc[n0 + n], cf[n], qf.f[z]);
              }
            }
          }
          // ---- this lane's row into what follows the step
          const float to = dc.to[mine];
          const float left = kFlips<T> && (l15 & 1) != 0 ? -dc.left[mine] : dc.left[mine];
          Frag<T> bf[L::kRows / 32];
#pragma unroll
          for (int k = 0; k < L::kRows / 32; ++k)
            bf[k] = flip_odd(frag_row(s.b, L::ldn, row, ph * L::kRows + k * 32, ln), l15);
          v4f o[4];  // four tiles at a time: a product waits for the last one on the same tile
#pragma unroll
          for (int p = 0; p < kPt; ++p) o[p] = v4f{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < L::kRows / 32; ++k)
#pragma unroll
            for (int z = 0; z < L::kTerms; ++z)
#pragma unroll
              for (int p = 0; p < kPt; ++p) mma(o[p], L::State::by_col(s.st[1][z], k * 32, p * 16, ln), bf[k]);
#pragma unroll
          for (int p = 0; p < kPt; ++p) {
            const v4f x = quad_get(&s.x[mine * L::ldp + p * 16 + 4 * g]);
            o[p] *= left;
            dx[p] += o[p];
            o[p] *= x;
            edge += (o[p][0] + o[p][1]) + (o[p][2] + o[p][3]);
          }
          Frag<T> xf[kKp];
#pragma unroll
          for (int k = 0; k < kKp; ++k) xf[k] = frag_row(s.x, L::ldp, row, k * 32, ln);
#pragma unroll
          for (int n0 = 0; n0 < kNt; n0 += kSide) {
#pragma unroll
            for (int n = 0; n < kSide; ++n) o[n] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kKp; ++k)
#pragma unroll
              for (int z = 0; z < L::kParts; ++z)
#pragma unroll
                for (int n = 0; n < kSide; ++n) mma(o[n], L::State::by_row(s.st[1][z], (n0 + n) * 16, k * 32, ln), xf[k]);
#pragma unroll
            for (int n = 0; n < kSide; ++n)
#pragma unroll
              for (int q = 0; q < kPhases; ++q)
                if (q == ph) acc[q * kNt + n0 + n] += to * o[n];
          }
        } else {
          if (ph == 0) {
            // ---- within the step, row t = mine
            const float ch = dc.hi[mine], cl = dc.lo[mine];
            v4f qw[4];
#pragma unroll
            for (int si = 0; si < 4; ++si) {
              qw[si] = v4f{0, 0, 0, 0};
              if (si > wave) continue;
              v4f yx = {0, 0, 0, 0};
#pragma unroll
              for (int k = 0; k < kKp; ++k)
                mma(yx, frag_row(s.x, L::ldp, si * 16, k * 32, ln), frag_row(s.dy, L::ldp, row, k * 32, ln));
              const int s0 = si * 16 + 4 * g;
              const v4f hi = *reinterpret_cast<const v4f*>(&dc.hi[s0]), lo = *reinterpret_cast<const v4f*>(&dc.lo[s0]);
              const v4f d = *reinterpret_cast<const v4f*>(&dc.d[s0]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float e = exp2_of((ch - hi[i]) + (cl - lo[i])) * d[i];
                if (si == wave) e = l15 >= 4 * g + i ? e : 0.0f;
                qw[si][i] = yx[i] * e;
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (2 * k > wave) continue;
              const auto qf = split_tiles<T, L::kParts>(qw[2 * k], qw[2 * k + 1]);
#pragma unroll
              for (int n0 = 0; n0 < 2 * NB; n0 += kBatch) {
                Frag<T> cf[kBatch];
#pragma unroll
                for (int n = 0; n < kBatch; ++n) cf[n] = frag_col_result(s.b, L::ldn, k * 32, (n0 + n) * 16, ln);
#pragma unroll
                for (int z = 0; z < L::kParts; ++z)
#pragma unroll
                  for (int n = 0; n < kBatch; ++n) mma(acc[n0 + n], cf[n], qf.f[z]);
              }
            }
          }
          // ---- the starting state into this lane's row
          Frag<T> yf[kKp];
#pragma unroll
          for (int k = 0; k < kKp; ++k) yf[k] = flip_odd(frag_row(s.dy, L::ldp, row, k * 32, ln), l15);
          const float from = kFlips<T> && (l15 & 1) != 0 ? -dc.from[mine] : dc.from[mine];
#pragma unroll
          for (int n0 = 0; n0 < kNt; n0 += kSide) {
            v4f o[kSide];
#pragma unroll
            for (int n = 0; n < kSide; ++n) o[n] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kKp; ++k)
#pragma unroll
              for (int z = 0; z < L::kTerms; ++z)
#pragma unroll
                for (int n = 0; n < kSide; ++n) mma(o[n], L::State::by_row(s.st[0][z], (n0 + n) * 16, k * 32, ln), yf[k]);
#pragma unroll
            for (int n = 0; n < kSide; ++n) {
              const v4f c = quad_get(&s.c[mine * L::ldn + ph * L::kRows + (n0 + n) * 16 + 4 * g]);
              o[n] *= from;
#pragma unroll
              for (int q = 0; q < kPhases; ++q)
                if (q == ph) acc[q * kNt + n0 + n] += o[n];
              o[n] *= c;
              edge += (o[n][0] + o[n][1]) + (o[n][2] + o[n][3]);
            }
          }
        }
      }
      edge = sum_groups(edge);
      whole = sum64(whole);
      float* edges = for_x ? sum.before : sum.after;
      if (g == 0) edges[mine] = slice == 0 ? edge : edges[mine] + edge;
      if (lane == 0) sum.whole[id] = slice == 0 ? whole : sum.whole[id] + whole;
      if (for_x) {
        const Rsrc ro = rows_rsrc(op + h * a.width + p0, ba.d_x.row_stride, rows, cols);
        const int at = mine * static_cast<int>(ba.d_x.row_stride);
        const float d = dc.d[mine];
#pragma unroll
        for (int p = 0; p < kPt; ++p) {
          const int c = p * 16 + 4 * g;
          put_quad<T>(ro, at, c, cols, d * dx[p] + D * quad_get(&s.dy[mine * L::ldp + c]));
        }
      }
    }
    if (h + 1 == h1) {
      __syncthreads();
      if (finishes) finish(h, cur, par);
    }
    cur = next;
    par ^= 1;
  }

  // ---- d_B or d_C
  if (ba.splits > 1) {
    const long r0 = (packed ? u.row0 : static_cast<long>(u.seq) * a.q.length) + u.t0;
    const long at = ((split * ba.rows + r0) * ba.groups + gr) * a.states;
    const int stride = ba.groups * a.states;
    const Rsrc rs = rows_rsrc((for_x ? ba.part_b : ba.part_c) + at, stride, rows, a.states);
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) put_quad<float>(rs, mine * stride, n * 16 + 4 * g, a.states, acc[n]);
    return;
  }
  const mamba2_rows& out = for_x ? ba.d_B : ba.d_C;
  const Rsrc rs = rows_rsrc(seq_ptr<T>(out, u.seq, u.row0, packed) + u.t0 * out.row_stride + gr * a.states,
                            out.row_stride, rows, a.states);
#pragma unroll
  for (int n = 0; n < 2 * NB; ++n)
    put_quad<T>(rs, mine * static_cast<int>(out.row_stride), n * 16 + 4 * g, a.states, acc[n]);
}

// 12 us at the size above (35 MB read).  What is left to add up, in a fixed order: the first blocks take a step's
// rows of d_B and d_C each (over the runs of heads, where there are several),
// the last ones a head's d_A, d_D and d_dt_bias (over the steps).
template <class T>
__global__ __launch_bounds__(256) void ssm_bwd_sums_kernel(BwdArgs ba, int joins, float* d_A, float* d_D,
                                                           float* d_bias) {
  const SsmArgs& a = ba.a;
  const int block = blockIdx.x;
  if (block < joins) {
    const Unit u = locate(a.q, block >> 1, kTok);
    if (u.t0 >= u.len) return;
    const bool packed = a.q.offsets != nullptr;
    const int rows = min(u.len - u.t0, kTok), wide = ba.groups * a.states, quads = wide / 4;
    const long r0 = (packed ? u.row0 : static_cast<long>(u.seq) * a.q.length) + u.t0;
    const float* part = (block & 1) == 0 ? ba.part_b : ba.part_c;
    const mamba2_rows& out = (block & 1) == 0 ? ba.d_B : ba.d_C;
    T* op = seq_ptr<T>(out, u.seq, u.row0, packed) + u.t0 * out.row_stride;
    const long next = ba.rows * wide;
    for (int e = threadIdx.x; e < rows * quads; e += 256) {
      const int r = e / quads, c = e % quads * 4;
      const float* p = part + (r0 + r) * wide + c;
      v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll 4
      for (int k = 1; k < ba.splits; ++k) v += *reinterpret_cast<const v4f*>(p + k * next);
      quad_put(op + r * out.row_stride + c, v);
    }
    return;
  }
  __shared__ float lds[3][4];
  const int h = block - joins;
  float v[3] = {0, 0, 0};
#pragma unroll 4
  for (int i = threadIdx.x; i < ba.steps; i += 256) {
    const v4f p = *reinterpret_cast<const v4f*>(ba.part + (static_cast<long>(i) * a.heads + h) * 4);
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] += p[k];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v[k] = sum64(v[k]);
    if ((threadIdx.x & 63) == 0) lds[k][threadIdx.x >> 6] = v[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    const int k = threadIdx.x;
    float* out = k == 0 ? d_A : k == 1 ? d_D : d_bias;
    if (out != nullptr) out[h] = (lds[k][0] + lds[k][1]) + (lds[k][2] + lds[k][3]);
  }
}

// --------------------------------------------------------------------- host
struct Plan {
  int seg, units, steps, slices, nw;
  int splits, run;
  long rows;
  bool segments;
  size_t keep, seg_state, seg_decay, part, part_bc, total;  // floats
};

size_t pad4(size_t n) { return (n + 3) / 4 * 4; }

int make_plan(const mamba2_seqs& q, const mamba2_ssm_dims& d, Plan* p) {
  const int st = check_scan(q, d, true);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t head = static_cast<size_t>(d.states) * d.width;
  p->nw = waves_of(d.width);
  p->slices = (d.width + p->nw * 16 - 1) / (p->nw * 16);
  p->seg = segment_tokens(q, d, true);
  p->units = static_cast<int>(unit_count(q, p->seg));
  p->steps = static_cast<int>(unit_count(q, kTok));
  p->segments = q.length > p->seg;
  p->rows = static_cast<long>(q.length) * (q.offsets != nullptr ? 1 : q.batch);
  // heads that share B and C stay together as long as the work-groups fill the chip
  const int ratio = d.heads / d.groups;
  const long groups = static_cast<long>(p->steps) * d.groups;
  long splits = (2 * kCUs + groups - 1) / groups;
  if (splits > ratio) splits = ratio;
  p->run = static_cast<int>((ratio + splits - 1) / splits);
  p->splits = (ratio + p->run - 1) / p->run;
  if (!grid_ok(static_cast<long long>(p->steps) * d.groups * p->splits, kBwdThreads)) return MAMBA2_SCAN_EBADDIM;
  p->keep = static_cast<size_t>(p->steps) * d.heads * kept_size(d.width, d.states);
  p->seg_state = p->segments ? pad4(static_cast<size_t>(p->units) * d.heads * head) : 0;
  p->seg_decay = p->segments ? pad4(static_cast<size_t>(p->units) * d.heads) : 0;
  p->part = pad4(static_cast<size_t>(p->steps) * d.heads * 4);
  p->part_bc = p->splits > 1 ? pad4(static_cast<size_t>(p->splits) * p->rows * d.groups * d.states) : 0;
  p->total = 2 * (p->keep + p->seg_state + p->seg_decay + p->part_bc) + p->part;
  return MAMBA2_SCAN_OK;
}

struct Call {
  BwdArgs ba;
  Walks w;
  Plan p;
  float *d_A, *d_D, *d_bias;
  hipStream_t s;
};

template <class T, int NB, int NW>
int launch_bwd(const Call& c) {
  const SsmArgs& a = c.ba.a;
  const dim3 grid(static_cast<unsigned>(static_cast<long>(c.p.units) * a.heads * c.p.slices), 2);
  if (c.p.segments) {
    ssm_walk_summary_kernel<T, NB, NW><<<grid, NW * 64, 0, c.s>>>(a, c.w);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    if (!a.fold) {
      const unsigned quads = static_cast<unsigned>((a.states * a.width + 1023) / 1024);
      ssm_walk_carry_kernel<<<dim3(2 * quads, a.heads, a.q.batch), 256, 0, c.s>>>(a, c.w);
      if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    }
  }
  ssm_walk_kernel<T, NB, NW><<<grid, NW * 64, 0, c.s>>>(a, c.w);
  if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  const unsigned blocks = static_cast<unsigned>(static_cast<long>(c.p.steps) * c.ba.groups * c.p.splits);
  ssm_bwd_kernel<T, NB, NW><<<blocks, kBwdThreads, 0, c.s>>>(c.ba);
  if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  const int joins = c.p.splits > 1 ? 2 * c.p.steps : 0;
  ssm_bwd_sums_kernel<T><<<joins + a.heads, 256, 0, c.s>>>(c.ba, joins, c.d_A, c.d_D, c.d_bias);
  return launch_status();
}

template <class T, int NB>
int launch_bwd_width(const Call& c) {
  switch (c.p.nw) {
    case 1: return launch_bwd<T, NB, 1>(c);
    case 2: return launch_bwd<T, NB, 2>(c);
    default: return launch_bwd<T, NB, 4>(c);
  }
}

template <class T>
int launch_bwd_states(const Call& c) {
  if (c.ba.a.states <= 32) return launch_bwd_width<T, 1>(c);
  if (c.ba.a.states <= 64) return launch_bwd_width<T, 2>(c);
  return launch_bwd_width<T, 4>(c);
}

}  // namespace

extern "C" {

size_t mamba2_ssm_bwd_workspace_bytes(mamba2_seqs q, mamba2_ssm_dims d) {
  Plan p;
  if (make_plan(q, d, &p) != MAMBA2_SCAN_OK) return 0;
  return p.total * sizeof(float);
}

int mamba2_ssm_bwd(mamba2_seqs q, mamba2_ssm_dims d, mamba2_rows x, mamba2_rows dt, const float* A, mamba2_rows B,
                   mamba2_rows C, const float* D, const float* dt_bias, const float* initial_state, mamba2_rows d_y,
                   const float* d_final_state, mamba2_rows d_x, mamba2_rows d_dt, float* d_A, mamba2_rows d_B,
                   mamba2_rows d_C, float* d_D, float* d_dt_bias, float* d_initial_state, void* workspace,
                   size_t workspace_bytes, void* stream) {
  Call c = {};
  int st = make_plan(q, d, &c.p);
  if (st != MAMBA2_SCAN_OK) return st;
  const size_t e = type_size(d.type);
  const long long xw = static_cast<long long>(d.heads) * d.width, bw = static_cast<long long>(d.groups) * d.states;
  if (A == nullptr || d_A == nullptr || workspace == nullptr) return MAMBA2_SCAN_ENULL;
  for (mamba2_rows* r : {&x, &d_y, &d_x}) {
    *r = used_strides(*r, q, xw);
    if ((st = check_vec_rows(*r, q, xw, e)) != MAMBA2_SCAN_OK) return st;
  }
  for (mamba2_rows* r : {&B, &C, &d_B, &d_C}) {
    *r = used_strides(*r, q, bw);
    if ((st = check_vec_rows(*r, q, bw, e)) != MAMBA2_SCAN_OK) return st;
  }
  dt = used_strides(dt, q, d.heads);
  d_dt = used_strides(d_dt, q, d.heads);
  if ((st = check_step_rows(dt, q, d)) != MAMBA2_SCAN_OK || (st = check_step_rows(d_dt, q, d)) != MAMBA2_SCAN_OK)
    return st;
  if (workspace_bytes < c.p.total * sizeof(float)) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(A, 4) || !aligned_to(D, 4) || !aligned_to(dt_bias, 4) || !aligned_to(initial_state, 16) ||
      !aligned_to(d_final_state, 16) || !aligned_to(d_initial_state, 16) || !aligned_to(workspace, 16) ||
      !aligned_to(d_A, 4) || !aligned_to(d_D, 4) || !aligned_to(d_dt_bias, 4))
    return MAMBA2_SCAN_EALIGN;

  SsmArgs& a = c.ba.a;
  a.q = q;
  a.x = x;
  a.dt = dt;
  a.B = B;
  a.C = C;
  a.A = A;
  a.D = D;
  a.bias = dt_bias;
  a.heads = d.heads;
  a.width = d.width;
  a.ratio = d.heads / d.groups;
  a.states = d.states;
  a.softplus = d.softplus;
  a.dt_bf16 = d.dt_type == MAMBA2_BF16;
  a.slices = c.p.slices;
  a.seg = c.p.seg;
  a.units = c.p.units;
  a.fold = fold_segments(q, d, a.seg);

  float* w = static_cast<float*>(workspace);
  const auto take = [&w](size_t n) {
    float* p = n > 0 ? w : nullptr;
    w += n;
    return p;
  };
  Walk &f = c.w.w[0], &r = c.w.w[1];
  f.v = x;
  f.m = B;
  f.first = initial_state;
  f.keep = take(c.p.keep);
  f.seg_state = take(c.p.seg_state);
  f.seg_decay = take(c.p.seg_decay);
  r.v = d_y;
  r.m = C;
  r.first = d_final_state;
  r.last = d_initial_state;
  r.keep = take(c.p.keep);
  r.seg_state = take(c.p.seg_state);
  r.seg_decay = take(c.p.seg_decay);
  r.rev = 1;
  c.ba.part_b = take(c.p.part_bc);
  c.ba.part_c = take(c.p.part_bc);
  c.ba.part = take(c.p.part);
  c.ba.d_y = d_y;
  c.ba.d_x = d_x;
  c.ba.d_dt = d_dt;
  c.ba.d_B = d_B;
  c.ba.d_C = d_C;
  c.ba.keep_s = f.keep;
  c.ba.keep_g = r.keep;
  c.ba.rows = c.p.rows;
  c.ba.steps = c.p.steps;
  c.ba.groups = d.groups;
  c.ba.splits = c.p.splits;
  c.ba.run = c.p.run;
  c.d_A = d_A;
  c.d_D = d_D;
  c.d_bias = d_dt_bias;
  c.s = static_cast<hipStream_t>(stream);
  return d.type == MAMBA2_BF16 ? launch_bwd_states<bf16>(c) : launch_bwd_states<float>(c);
}

}  // extern "C"
