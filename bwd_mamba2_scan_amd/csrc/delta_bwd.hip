// Gated delta rule for gfx950: the backward.  With the notation of
// delta_common.h, S and D the state and its gradient at a step's two ends,
// dU, dR as in the reverse walk, dP = dY U^T (j <= i) and dT = -dR U^T (j < i):
//   dQ    = scale 2^c (dY S^T) + Pm K                 Pm = scale E dP
//   dK    = -beta 2^c (dR S^T) + 2^(c_end-c) (U D^T) + Pm^T Q + (Xm + Xm^T) K
//                                                     Xm = beta E dT
//   dbeta_i = dR_i.V_i - 2^c_i k_i.(dR S^T)_i + sum_j dT_ij E_ij k_i.k_j
//   dg_t  = the sum of what passes from before token t to token t and behind:
//           sum_{i >= t} A_i + sum_{j < t} F_j + sum_{i >= t > j} Z_ij + 2^c_end <S, D>
//           A_i = scale 2^c_i q_i.(dY S^T)_i - beta_i 2^c_i k_i.(dR S^T)_i
//           F_j = 2^(c_end-c_j) k_j.(U D^T)_j,  Z_ij = Pm_ij q_i.k_j + Xm_ij k_i.k_j
// dg_t is added up from those pairs, not as a difference of sums: where decays
// are strong it is far smaller than what passes within a token.
//
// Four launches: every step's matrices (delta_bwd_prep_kernel), the walk of the
// states, which keeps each step's starting state and U (delta_keep_kernel), the
// walk of the state's gradient (delta_reverse_kernel), and the gradients of
// every step (delta_grads_kernel), whose work-group takes the heads of a group
// one after another and adds up the shared q's and k's gradients in registers.
#include "delta_common.h"
#include "delta_pair.h"
#include "delta_prep.h"
#include "delta_walk.h"

namespace {

using namespace delta;

template <class T, int NB>
__global__ __launch_bounds__(kPrepWaves * 64) void delta_bwd_prep_kernel(DeltaArgs a) {
  __shared__ PrepLds<T, NB> s;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int step = work / a.heads, h = work % a.heads;
  const Unit u = locate(a.seqs, step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  make_step<T, NB>(s, a, u, h, a.seqs.offsets != nullptr);
  const long at = static_cast<long>(step) * a.heads + h;
  constexpr int kM = kExact<T> * kPieces * kPiece;
  put_pieces<T, kExact<T>, false>(static_cast<T*>(a.m) + at * kM, s.m, wave, lane);
  put_pieces<T, kExact<T>, true>(static_cast<T*>(a.mt) + at * kM, s.m, wave, lane);
  put_pieces<T, kExact<T>, true>(static_cast<T*>(a.pt) + at * kM, s.sq.p, wave, lane);
  if (threadIdx.x < sizeof(Coef) / 16)
    reinterpret_cast<v4f*>(a.coef + at)[threadIdx.x] = reinterpret_cast<const v4f*>(&s.coef)[threadIdx.x];
}

template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_keep_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairFwdLds<NB, true> s;
    pair_forward<NB, true>(a, s);
  } else {
    __shared__ FwdLds<T, NB, true> s;
    walk_forward<T, NB, true>(a, s);
  }
}

template <class T, int NB>
__global__ __launch_bounds__(walk_threads<T>) void delta_reverse_kernel(DeltaArgs a) {
  if constexpr (sizeof(T) == 2) {
    __shared__ PairRevLds<NB> s;
    pair_reverse<NB>(a, s);
  } else {
    __shared__ RevLds<T, NB> s;
    walk_reverse<T, NB>(a, s);
  }
}

// ------------------------------------------------------- a step's gradients
constexpr int kPart = 64;   // columns of a head that are staged at a time

template <int NB>
constexpr int kGradWaves = NB < 2 ? 4 : 2 * NB;  // 16 rows of the states each

template <class T, int NB>
struct GradLds {
  static constexpr int ldn = stride_of<T>(NB * 32);
  static constexpr int ldv = stride_of<T>(kPart);
  static constexpr int ldm = stride_of<T>(kTok);
  static constexpr int kW = kGradWaves<NB>;
  alignas(16) T k[kTok * ldn];
  alignas(16) T q[kTok * ldn];
  union {
    struct {
      T y[kTok * ldv];
      T r[kExact<T>][kTok * ldv];  // dR
      T u[kExact<T>][kTok * ldv];  // U
    } in;
    struct {
      T pm[kTwo<T>][kTok * ldm];   // Pm
      T xm[kTwo<T>][kTok * ldm];   // Xm + Xm^T
      float z[kTok * kSq];         // Z
    } sq;
  };
  alignas(16) Coef coef;
  float c_hi[kTok], c_lo[kTok];
  float qs[kW][kTok], ks[kW][kTok], kd[kW][kTok];  // a wave's states of A_i's two terms, without their factors, and F_j's
  float rv[kTok];                                  // dR_i.V_i
  float bt[4][kTok];                               // a column tile's part of sum_j dT_ij E_ij k_i.k_j
  float sd[kW];                                    // a wave's part of <S, D>
  float a_i[kTok], f_j[kTok];
};

// Eight floats of a row of the kept state, columns c ..; zero outside.
__device__ __forceinline__ void load8(Rsrc rs, unsigned off, float (&v)[8]) {
  const v4f a = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  const v4f b = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, off + 16, 0, 0));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[j + 4] = b[j];
  }
}

// Eight values of T from global memory as floats; zero outside.
template <class T>
__device__ __forceinline__ void load8_as(Rsrc rs, unsigned off, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const v8bf a = __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<float>(a[j]);
  } else {
    load8(rs, off, v);
  }
}

// Eight values to an LDS row in PARTS parts, `plane` elements apart.
template <class T, int PARTS>
__device__ __forceinline__ void put8(T* p, int plane, const float (&v)[8]) {
  const Split<T, PARTS> f = split_of<T, PARTS>(v);
#pragma unroll
  for (int z = 0; z < PARTS; ++z) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<v8bf*>(p + z * plane) = f.f[z].v;
    } else {
      v4f* r = reinterpret_cast<v4f*>(p + z * plane);
      r[0] = f.f[z].v[0];
      r[1] = f.f[z].v[1];
    }
  }
}

template <class T, int PARTS>
__device__ __forceinline__ void put1(T* p, int plane, float v) {
#pragma unroll
  for (int z = 0; z < PARTS; ++z) {
    const T t = static_cast<T>(v);
    p[z * plane] = t;
    v -= static_cast<float>(t);
  }
}

template <class T, int NB>
__global__ __launch_bounds__(kGradWaves<NB> * 64) void delta_grads_kernel(DeltaArgs a) {
  typedef GradLds<T, NB> L;
  __shared__ L s;
  constexpr int kW = kGradWaves<NB>, kThreads = kW * 64;
  const int tid = threadIdx.x, wave = wave_id(), lane = tid & 63, l15 = lane & 15, g = lane >> 4;
  const int work = xcd_contiguous(blockIdx.x, gridDim.x);
  const int groups = a.heads / a.ratio;
  const int step = work / groups, group = work % groups;
  const Unit u = locate(a.seqs, step, kTok);
  if (!u.live || u.t0 >= u.len) return;
  const bool packed = a.seqs.offsets != nullptr;
  const int rows = min(u.len - u.t0, kTok);
  const long head = static_cast<long>(a.states) * a.width, slab = kTok * static_cast<long>(a.width);
  {
    Tile<T, kTok, NB * 32, kThreads> tk, tq;
    tk.init(a.k.row_stride, a.states, tid);
    tq.init(a.q.row_stride, a.states, tid);
    const int j = group * a.states;
    tk.load(rows_rsrc(seq_ptr<const T>(a.k, u.seq, u.row0, packed) + u.t0 * a.k.row_stride + j, a.k.row_stride, rows, a.states));
    tq.load(rows_rsrc(seq_ptr<const T>(a.q, u.seq, u.row0, packed) + u.t0 * a.q.row_stride + j, a.q.row_stride, rows, a.states));
    tk.store(s.k, L::ldn, tid);
    tq.store(s.q, L::ldn, tid);
  }
  const bool states = wave < 2 * NB;   // has a tile of the states
  const int n0 = 16 * wave;            // its first
  v4f dq[4], dk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dq[i] = dk[i] = v4f{0, 0, 0, 0};

  for (int hh = 0; hh < a.ratio; ++hh) {
    const int h = group * a.ratio + hh;
    const long cell = static_cast<long>(step) * a.heads + h;
    __syncthreads();  // the last head's matrices are read
    if (wave == kW - 1) {
      const double c = scan64(gate_log(load_gate(a.g, a.gate_bf16, u, packed, u.t0, rows, h, a.heads)));
      s.c_hi[lane] = static_cast<float>(c);
      s.c_lo[lane] = static_cast<float>(c - static_cast<float>(c));
    } else if (tid < static_cast<int>(sizeof(Coef) / 16)) {
      reinterpret_cast<v4f*>(&s.coef)[tid] = reinterpret_cast<const v4f*>(a.coef + cell)[tid];
    }
    if (tid < kTok) s.rv[tid] = 0.0f;

    // products over the columns
    v4f ys[4], rs[4], ud[4];  // dY S^T, dR S^T, U D^T: 64 tokens by this wave's states
#pragma unroll
    for (int i = 0; i < 4; ++i) ys[i] = rs[i] = ud[i] = v4f{0, 0, 0, 0};
    constexpr int kMine = (10 + kW - 1) / kW;
    v4f dp[kMine], dt[kMine];  // this wave's tiles of dP and -dT
#pragma unroll
    for (int i = 0; i < kMine; ++i) dp[i] = dt[i] = v4f{0, 0, 0, 0};
    float sd = 0.0f;
    const Rsrc rS = make_rsrc(a.keep + cell * head, static_cast<unsigned>(head * 4));
    const Rsrc rD = make_rsrc(a.d_keep + cell * head, static_cast<unsigned>(head * 4));
    const Rsrc rU = make_rsrc(a.u + cell * slab, static_cast<unsigned>(slab * 4));
    const Rsrc rR = make_rsrc(a.d_r + cell * slab, static_cast<unsigned>(slab * 4));
    const Rsrc rY = rows_rsrc(seq_ptr<const T>(a.d_y, u.seq, u.row0, packed) + u.t0 * a.d_y.row_stride + h * a.width,
                              a.d_y.row_stride, rows, a.width);
    const Rsrc rV = rows_rsrc(seq_ptr<const T>(a.v, u.seq, u.row0, packed) + u.t0 * a.v.row_stride + h * a.width,
                              a.v.row_stride, rows, a.width);
    for (int c0 = 0; c0 < a.width; c0 += kPart) {
      __syncthreads();
      for (int e = tid; e < kTok * kPart / 8; e += kThreads) {
        const int row = e >> 3, c = c0 + (e & 7) * 8;
        const bool in = c < a.width;
        float y[8], v[8], r[8], w[8];
        load8_as<T>(rY, in ? static_cast<unsigned>((row * static_cast<int>(a.d_y.row_stride) + c) * sizeof(T)) : kOutside, y);
        load8_as<T>(rV, in ? static_cast<unsigned>((row * static_cast<int>(a.v.row_stride) + c) * sizeof(T)) : kOutside, v);
        load8(rR, in ? static_cast<unsigned>((row * a.width + c) * 4) : kOutside, r);
        load8(rU, in ? static_cast<unsigned>((row * a.width + c) * 4) : kOutside, w);
        const int at = row * L::ldv + (e & 7) * 8;
        put8<T, 1>(s.in.y + at, 0, y);
        put8<T, kExact<T>>(s.in.r[0] + at, kTok * L::ldv, r);
        put8<T, kExact<T>>(s.in.u[0] + at, kTok * L::ldv, w);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(r[j], v[j], sum);
        sum += __shfl_xor(sum, 1);
        sum += __shfl_xor(sum, 2);
        sum += __shfl_xor(sum, 4);
        if ((e & 7) == 0) s.rv[row] += sum;
      }
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < kPart / 32; ++ks) {
        if (c0 + ks * 32 >= a.width) break;
        if (states) {
          // the lane's row of the states, eight columns; rows and columns outside are zero
          float f[8], d[8];
          const int c = c0 + ks * 32 + 8 * g;
          const unsigned off = c < a.width ? static_cast<unsigned>(((n0 + l15) * a.width + c) * 4) : kOutside;
          load8(rS, off, f);
          load8(rD, off, d);
#pragma unroll
          for (int j = 0; j < 8; ++j) sd = fmaf(f[j], d[j], sd);
          const Split<T, kExact<T>> fs = split_of<T, kExact<T>>(f), ds = split_of<T, kExact<T>>(d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Frag<T> yf[1] = {frag_row(s.in.y, L::ldv, 16 * i, 32 * ks)};
            Frag<T> rf[kExact<T>], uf[kExact<T>];
#pragma unroll
            for (int z = 0; z < kExact<T>; ++z) {
              rf[z] = frag_row(s.in.r[z], L::ldv, 16 * i, 32 * ks);
              uf[z] = frag_row(s.in.u[z], L::ldv, 16 * i, 32 * ks);
            }
            mma_parts<T>(ys[i], yf, fs.f);
            mma_parts<T>(rs[i], rf, fs.f);
            mma_parts<T>(ud[i], uf, ds.f);
          }
        }
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          const int tile = wave + n * kW;
          if (tile < 10) {
            const int ti = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, tj = tile - ti * (ti + 1) / 2;
            const Frag<T> yf[1] = {frag_row(s.in.y, L::ldv, 16 * ti, 32 * ks)};
            Frag<T> rf[kExact<T>], uf[kExact<T>];
#pragma unroll
            for (int z = 0; z < kExact<T>; ++z) {
              rf[z] = frag_row(s.in.r[z], L::ldv, 16 * ti, 32 * ks);
              uf[z] = frag_row(s.in.u[z], L::ldv, 16 * tj, 32 * ks);
            }
            mma_parts<T>(dp[n], yf, uf);
            mma_parts<T>(dt[n], rf, uf);
          }
        }
      }
    }
    __syncthreads();  // the columns' tiles give way to the matrices

    // what the states give: the shared gradients, and the sums over the states
    sd = sum64(sd);
    if (lane == 0) s.sd[wave] = sd;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f from = rows_of(s.coef.from, i, g), to = rows_of(s.coef.to, i, g), beta = rows_of(s.coef.beta, i, g);
      v4f sq, sk, sf;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g + r;
        const float qe = states ? static_cast<float>(s.q[row * L::ldn + n0 + l15]) : 0.0f;
        const float ke = states ? static_cast<float>(s.k[row * L::ldn + n0 + l15]) : 0.0f;
        sq[r] = sum16(qe * ys[i][r]);
        sk[r] = sum16(ke * rs[i][r]);
        sf[r] = sum16(ke * ud[i][r]);
      }
      if (l15 == 0) {
        *reinterpret_cast<v4f*>(&s.qs[wave][16 * i + 4 * g]) = sq;
        *reinterpret_cast<v4f*>(&s.ks[wave][16 * i + 4 * g]) = sk;
        *reinterpret_cast<v4f*>(&s.kd[wave][16 * i + 4 * g]) = sf;
      }
      dq[i] += a.scale * (from * ys[i]);
      dk[i] += to * ud[i] - beta * (from * rs[i]);
    }
    // the matrices of the step
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      const int tile = wave + n * kW;
      if (tile < 10) {
        const int ti = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, tj = tile - ti * (ti + 1) / 2;
        v4f kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < NB; ++m) {
          const Frag<T> b = frag_row(s.k, L::ldn, 16 * tj, 32 * m);
          mma(kk, frag_row(s.k, L::ldn, 16 * ti, 32 * m), b);
          mma(qk, frag_row(s.q, L::ldn, 16 * ti, 32 * m), b);
        }
        const int col = 16 * tj + l15;
        const float ch = s.c_hi[col], cl = s.c_lo[col];
        v4f bt;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * ti + 4 * g + r;
          const float e = exp2_of((s.c_hi[row] - ch) + (s.c_lo[row] - cl));
          const float pm = col <= row ? a.scale * (e * dp[n][r]) : 0.0f;
          const float et = col < row ? -e * dt[n][r] : 0.0f;
          const float xm = s.coef.beta[row] * et;
          put1<T, kTwo<T>>(&s.sq.pm[0][row * L::ldm + col], kTok * L::ldm, pm);
          // the symmetric sum, each element written once (the diagonal of Xm is zero)
          if (ti != tj || col <= row) put1<T, kTwo<T>>(&s.sq.xm[0][row * L::ldm + col], kTok * L::ldm, xm);
          if (ti != tj || col < row) put1<T, kTwo<T>>(&s.sq.xm[0][col * L::ldm + row], kTok * L::ldm, xm);
          s.sq.z[row * kSq + col] = pm * qk[r] + xm * kk[r];
          bt[r] = sum16(et * kk[r]);
        }
        if (l15 == 0) *reinterpret_cast<v4f*>(&s.bt[tj][16 * ti + 4 * g]) = bt;
      }
    }
    // Pm is zero above the diagonal where a product of 32 columns reaches
    for (int e = tid; e < 2 * 16 * 16; e += kThreads) {
      const int b = e >> 8, row = 32 * b + (e >> 4 & 15), col = 32 * b + 16 + (e & 15);
      put1<T, kTwo<T>>(&s.sq.pm[0][row * L::ldm + col], kTok * L::ldm, 0.0f);
    }
    __syncthreads();
    if (states) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Frag<T> kf[1] = {frag_col(s.k, L::ldn, 32 * j, n0)}, qf[1] = {frag_col(s.q, L::ldn, 32 * j, n0)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Frag<T> pf[kTwo<T>], tf[kTwo<T>], xf[kTwo<T>];
#pragma unroll
          for (int z = 0; z < kTwo<T>; ++z) {
            xf[z] = frag_row(s.sq.xm[z], L::ldm, 16 * i, 32 * j);
            if (j <= i / 2) pf[z] = frag_row(s.sq.pm[z], L::ldm, 16 * i, 32 * j);
            if (j >= i / 2) tf[z] = frag_col(s.sq.pm[z], L::ldm, 32 * j, 16 * i);
          }
          mma_parts<T>(dk[i], xf, kf);
          if (j <= i / 2) mma_parts<T>(dq[i], pf, kf);
          if (j >= i / 2) mma_parts<T>(dk[i], tf, qf);
        }
      }
    }
    // the gates' gradients: A_i and F_j first
    if (tid < kTok) {
      float sq = 0.0f, sk = 0.0f, sf = 0.0f;
#pragma unroll
      for (int w = 0; w < 2 * NB; ++w) {
        sq += s.qs[w][tid];
        sk += s.ks[w][tid];
        sf += s.kd[w][tid];
      }
      const float from = s.coef.from[tid], beta = s.coef.beta[tid];
      s.a_i[tid] = a.scale * (from * sq) - beta * (from * sk);
      s.f_j[tid] = s.coef.to[tid] * sf;
      float bt = 0.0f;
      for (int c = 0; c <= tid / 16; ++c) bt += s.bt[c][tid];
      const float db = s.rv[tid] - from * sk + bt;
      if (tid < rows) {
        const long e = static_cast<long>(u.t0 + tid) * a.d_beta.row_stride + h;
        if (a.gate_bf16) seq_ptr<bf16>(a.d_beta, u.seq, u.row0, packed)[e] = static_cast<bf16>(db);
        else seq_ptr<float>(a.d_beta, u.seq, u.row0, packed)[e] = db;
      }
    }
    __syncthreads();
    {
      float ends = 0.0f;
#pragma unroll
      for (int w = 0; w < 2 * NB; ++w) ends += s.sd[w];
      ends *= s.coef.total;
      constexpr int kEach = kTok / kW;  // tokens of a wave
      const int first = wave * kEach;
      float z = 0.0f;                   // lane j: sum of Z_ij over i >= t
      for (int i = kTok - 1; i >= first + kEach; --i) z += lane <= i ? s.sq.z[i * kSq + lane] : 0.0f;
      for (int t = first + kEach - 1; t >= first; --t) {
        z += lane <= t ? s.sq.z[t * kSq + lane] : 0.0f;
        const float part = (lane < t ? z + s.f_j[lane] : 0.0f) + (lane >= t ? s.a_i[lane] : 0.0f);
        const float dg = sum64(part) + ends;
        if (lane == 0 && t < rows) {
          const long e = static_cast<long>(u.t0 + t) * a.d_g.row_stride + h;
          if (a.gate_bf16) seq_ptr<bf16>(a.d_g, u.seq, u.row0, packed)[e] = static_cast<bf16>(dg);
          else seq_ptr<float>(a.d_g, u.seq, u.row0, packed)[e] = dg;
        }
      }
    }
  }
  if (states) {
    const Rsrc rq = rows_rsrc(seq_ptr<const T>(a.d_q, u.seq, u.row0, packed) + u.t0 * a.d_q.row_stride + group * a.states,
                              a.d_q.row_stride, rows, a.states);
    const Rsrc rk = rows_rsrc(seq_ptr<const T>(a.d_k, u.seq, u.row0, packed) + u.t0 * a.d_k.row_stride + group * a.states,
                              a.d_k.row_stride, rows, a.states);
    const int col = n0 + l15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g + r;
        store_elem<T>(rq, col < a.states ? static_cast<unsigned>((row * static_cast<int>(a.d_q.row_stride) + col) * sizeof(T)) : kOutside, dq[i][r]);
        store_elem<T>(rk, col < a.states ? static_cast<unsigned>((row * static_cast<int>(a.d_k.row_stride) + col) * sizeof(T)) : kOutside, dk[i][r]);
      }
  }
}

// ---------------------------------------------------------------- host side
template <class T, int NB>
int launch_bwd(const DeltaArgs& a, unsigned steps, unsigned blocks, hipStream_t s) {
  if (steps > 0) {
    delta_bwd_prep_kernel<T, NB><<<steps, kPrepWaves * 64, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
    delta_keep_kernel<T, NB><<<blocks, walk_threads<T>, 0, s>>>(a);
    if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  }
  delta_reverse_kernel<T, NB><<<blocks, walk_threads<T>, 0, s>>>(a);
  if (launch_status() != MAMBA2_SCAN_OK) return MAMBA2_SCAN_EHIP;
  if (steps > 0) delta_grads_kernel<T, NB><<<steps / a.ratio, kGradWaves<NB> * 64, 0, s>>>(a);
  return launch_status();
}
template <class T>
int launch_bwd_states(const DeltaArgs& a, unsigned steps, unsigned blocks, hipStream_t s) {
  if (a.states <= 32) return launch_bwd<T, 1>(a, steps, blocks, s);
  if (a.states <= 64) return launch_bwd<T, 2>(a, steps, blocks, s);
  return launch_bwd<T, 4>(a, steps, blocks, s);
}

// The workspace's parts: bytes for each step of each head.
struct BwdCell {
  size_t m, state, rows, all;
};
BwdCell bwd_cell(const mamba2_delta_dims& d) {
  BwdCell c;
  c.m = (d.type == MAMBA2_BF16 ? 3 * 2 : 4) * kPieces * kPiece;
  c.state = static_cast<size_t>(d.states) * d.width * 4;
  c.rows = static_cast<size_t>(kTok) * d.width * 4;
  c.all = 3 * c.m + 2 * c.state + 2 * c.rows + sizeof(Coef);
  return c;
}

}  // namespace

extern "C" {

size_t mamba2_delta_bwd_workspace_bytes(mamba2_seqs seqs, mamba2_delta_dims d) {
  if (check_delta(seqs, d) != MAMBA2_SCAN_OK) return 0;
  return static_cast<size_t>(unit_count(seqs, kTok)) * d.heads * bwd_cell(d).all;
}

int mamba2_delta_bwd(mamba2_seqs seqs, mamba2_delta_dims d, mamba2_rows q, mamba2_rows k, mamba2_rows v, mamba2_rows g,
                     mamba2_rows beta, const float* initial_state, mamba2_rows d_y, const float* d_final_state,
                     mamba2_rows d_q, mamba2_rows d_k, mamba2_rows d_v, mamba2_rows d_g, mamba2_rows d_beta,
                     float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  DeltaArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.d_y = d_y;
  a.d_q = d_q;
  a.d_k = d_k;
  a.d_v = d_v;
  a.d_g = d_g;
  a.d_beta = d_beta;
  int st = check_delta(seqs, d);
  if (st != MAMBA2_SCAN_OK) return st;
  mamba2_rows* const keys[] = {&a.q, &a.k, &a.d_q, &a.d_k};
  mamba2_rows* const values[] = {&a.v, &a.d_y, &a.d_v};
  mamba2_rows* const gates[] = {&a.g, &a.beta, &a.d_g, &a.d_beta};
  for (mamba2_rows* r : keys)
    if ((st = check_keys(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  for (mamba2_rows* r : values)
    if ((st = check_values(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  for (mamba2_rows* r : gates)
    if ((st = check_gates(r, seqs, d)) != MAMBA2_SCAN_OK) return st;
  if (!aligned_to(initial_state, 16) || !aligned_to(d_final_state, 16) || !aligned_to(d_initial_state, 16))
    return MAMBA2_SCAN_EALIGN;
  if (workspace == nullptr) return MAMBA2_SCAN_ENULL;
  if (workspace_bytes < mamba2_delta_bwd_workspace_bytes(seqs, d)) return MAMBA2_SCAN_ESIZE;
  if (!aligned_to(workspace, 16)) return MAMBA2_SCAN_EALIGN;
  if (seqs.length == 0 && d_initial_state == nullptr) return MAMBA2_SCAN_OK;
  a.initial = initial_state;
  a.d_final = d_final_state;
  a.d_initial = d_initial_state;
  set_dims(&a, seqs, d);
  const long cells = static_cast<long>(unit_count(seqs, kTok)) * d.heads;
  const BwdCell c = bwd_cell(d);
  char* at = static_cast<char*>(workspace);
  const auto take = [&](size_t bytes) {
    char* p = at;
    at += cells * bytes;
    return p;
  };
  a.m = take(c.m);
  a.mt = take(c.m);
  a.pt = take(c.m);
  a.keep = reinterpret_cast<float*>(take(c.state));
  a.d_keep = reinterpret_cast<float*>(take(c.state));
  a.u = reinterpret_cast<float*>(take(c.rows));
  a.d_r = reinterpret_cast<float*>(take(c.rows));
  a.coef = reinterpret_cast<Coef*>(take(sizeof(Coef)));
  const unsigned steps = seqs.length == 0 ? 0 : static_cast<unsigned>(cells);
  const unsigned blocks = static_cast<unsigned>(unit_count(seqs, a.seg) * d.heads * a.slices);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return d.type == MAMBA2_BF16 ? launch_bwd_states<bf16>(a, steps, blocks, s) : launch_bwd_states<float>(a, steps, blocks, s);
}

}  // extern "C"
