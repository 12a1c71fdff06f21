// The gradients of the head scan on the matrix cores (bfloat16 io), in two kernels; at the end of the file the decays'
// gradients of the token-by-token backward, from the same sums.
//
// k_heads_states walks the states: h forward, and from the last token to the first their adjoint
//   Gam <- e^{c_last} Gam + sum_i e^{c_i} dy_i C_i^T          (the gradient of the state before a block)
// and stores h at the start and Gam at the end of every 64-token block.  The blocks are those of the packed
// stream (segment rows of length 64), so that
// k_heads_grads can take every block by itself: a workgroup takes a block and some heads of a group, one after
// another.  With M_ij = (C_i . B_j) d_ij, W_ij = dy_i . x_j, d_ij = e^{c_i - c_j}, w_j = e^{c_last - c_j} delta_j:
//   dx_j = delta_j sum_{i>=j} M_ij dy_i + w_j Gam B_j + D dy_j
//   dB_j = sum_{i>=j} delta_j W_ij d_ij C_i + w_j Gam^T x_j              (summed over the heads in registers)
//   dC_i = sum_{j<=i} delta_j W_ij d_ij B_j + e^{c_i} h^T dy_i           (likewise)
//   r_j  = sum_{i>=j} M_ij W_ij + e^{c_last - c_j} x_j . (Gam B_j)       (= dL/d(delta_j x_j) . x_j)
//   dl_t = sum_{i>=t>j} delta_j M_ij W_ij + sum_{i>=t} e^{c_i} dy_i . (h C_i) + sum_{j<t} w_j x_j . (Gam B_j)
//          + e^{c_last} <Gam, h>                                         (l = log a)
//   ddelta = r + A dl
// Each term of dl joins something before t to something from t on, and the first sum is put together from those of whole
// 16 x 16 tiles, parts of tiles' row and column sums and the diagonal's tile, all of pairs that belong to it: nothing cancels.
// (As row sums minus column sums from the block's end, which is one scan, dA_log and ddt_bias were off by 1.2e-6 where float32
// arithmetic throughout gives 2e-7.)
//
// Precision: dx, dB and dC leave in bfloat16.  Of their computed operands delta M (dx, whose own rounding hides it) and the
// states h and Gam (dC, dB) are rounded to bfloat16 once; delta W d, the better part of dB, is taken in two parts.  dx and dB are
// then off by their own rounding, 1.66e-3 to 1.7e-3 of their norm, dC, where the states weigh, by up to 2.3e-3 (the states in two
// parts would be three more barriers a head; delta W d in one left dB at 2.3e-3 too, the call at 371 instead of 383 us).
// dl, r and what is summed from them (dA_log, ddt_bias: float32 results) use float32 products of the exact
// scores, and h and Gam in three bfloat16 parts (24 bits).
#pragma once

#include "mm_heads_mma.h"

namespace mm {

struct StateArgs {
  Tok<uint16_t> u[2], v[2];   // forward x, B; reverse dy, C
  int P, N, G, npb;
  int slices;                 // of the state's columns, 32 NK each, a workgroup for each
  int64_t Ls;
  int whole;                  // Ls > T
  const float* init[2];       // [S] states, or NULL: zeros
  float* carry[2];            // [rows] states: written by local runs, else read where a sequence has several segments
  float* decay[2];            // [rows, H] log2 of a segment's decay, written by local runs
  // [rows64, H npb] states at the blocks' starts / ends (not by local runs): element (p, n) of a 64-channel block at
  // ((p / 16) NP + n / 4 * 4) 16 + (p % 16) 4 + n % 4, the order of the accumulators
  float* store[2];
  float* fin[2];              // [S] final states, or NULL
  int all;                    // local runs: every segment, not only those that another one follows
  int64_t even;               // not 0: only if a sequence is longer
};

template <int NK>
struct StateGeo {
  static constexpr int NP = NK * 32, PC = NP / 8;
  static constexpr int B = 0, X = kMmaTok * NP * 2, F = X + kMmaTok * kMmaTok * 2, bytes = F + 2 * (kMmaTok + 4) * 4;
};

// grid: (row, 64-channel block, slice) x direction; a wave takes 16 of the channels
// The storing walks are bound by their stores: 8 x 2048 tokens, 24 heads 64 x 128, both directions, write 403 MB of
// states in 157 us (traced mean, inputs of successive calls in different memory; 536 MB in all, 3.4 TB/s).  States pass the
// caches by, on the way out and in: the whole backward 382 us where plain accesses took 397 (4 x 2048 tokens 227 and
// 262).  The local walks of 16384 tokens, 64 heads, take 95 us: VALU issue 32%, MFMA 22%, the rest waits in the chain of a
// block (load, LDS, weights, product); shorter stretches would add carries.
// LOCAL: what a segment adds to a zero state; else the whole walk, which stores.
// (The two are told apart at compile time so that the stores' place among the outstanding accesses is known: a wait
// for the tile loads then leaves the stores in flight.)
template <int NK, bool VEC, bool LOCAL>
__global__ __launch_bounds__(kMmaThreads, 4) void k_heads_states(StateArgs q, HeadPar hp) {
  typedef StateGeo<NK> G;
  constexpr int NT = 2 * NK, PC = G::PC;
  extern __shared__ __align__(16) char lds[];
  char *const sB = lds + G::B, *const sX = lds + G::X;
  float* const sF = reinterpret_cast<float*>(lds + G::F);  // two sets of [block][64] weights and [block] last decays

  if (q.even > 0 && !longer_than(hp.cu, hp.S, q.even)) return;
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int dir = blockIdx.y;
  const int wg = xcd_unit(blockIdx.x, gridDim.x, hp.H / q.G * q.npb * q.slices);
  const int n0 = wg % q.slices * G::NP, vh = wg / q.slices % (hp.H * q.npb);
  SegmentWalk walk(hp.cu, hp.S, wg / q.slices / (hp.H * q.npb), q.Ls, q.whole != 0);
  const Tok<uint16_t> tu = q.u[dir], tv = q.v[dir];

  const int h = vh / q.npb, p0 = (vh % q.npb) * 64, group = h / (hp.H / q.G);
  const int pw = q.P - p0 < 64 ? q.P - p0 : 64;
  const int p = 16 * wave + li;  // the lane's channel in the block
  const int64_t PN = static_cast<int64_t>(q.P) * q.N, set = hp.H * PN;

  Segment sg;
  int64_t rho;
  while (walk.next(sg, rho)) {
  const bool many = sg.many(q.Ls);
  if (LOCAL && !q.all && (!many || (dir ? sg.first() : sg.last()))) continue;
  hf4 st[NT];  // [n = 16 nt + 4g + r][channel p]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) st[nt] = hf4{0, 0, 0, 0};
  if (!LOCAL) {
    const float* from = many ? q.carry[dir] + rho * set : (q.init[dir] ? q.init[dir] + sg.s * set : nullptr);
    if (from != nullptr && p < pw)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int n = n0 + 16 * nt + 4 * g;
        const float* a = from + h * PN + static_cast<int64_t>(p0 + p) * q.N + n;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < q.N) st[nt][r] = a[r];
      }
  }

  const int brow = tid / PC, bcol = (tid % PC) * 8;
  constexpr int bstep = kMmaThreads / PC;
  const int xrow = tid >> 3, xcol = (tid & 7) * 8, xn = pw - xcol, bn = q.N - n0 - bcol;
  const int dH = hp.H * q.P, gn = (hp.H / tv.div) * q.N;
  const int b_off = (brow * static_cast<int>(tv.ts) + group * q.N + n0 + bcol) * 2;
  const int x_off = (xrow * static_cast<int>(tu.ts) + h * q.P + p0 + xcol) * 2;
  hu4 rB[NK], rX[2];
  const auto load = [&](int64_t tb, int cnt) {
    const hbuf bB = token_rows(tv.p, tb, tv.ts, cnt, gn), bX = token_rows(tu.p, tb, tu.ts, cnt, dH);
#pragma unroll
    for (int i = 0; i < NK; ++i) rB[i] = load8<VEC>(bB, b_off + i * bstep * static_cast<int>(tv.ts) * 2, bn);
#pragma unroll
    for (int i = 0; i < 2; ++i) rX[i] = load8<VEC>(bX, x_off + i * 32 * static_cast<int>(tu.ts) * 2, xn);
  };
  // wave 0 makes the tokens' weights, a chunk ahead
  const float A2 = head_A2(hp, h), bias = hp.dt != nullptr ? hp.dt_bias[h] : 0.0f;
  uint32_t rdt = 0;
  double dsum = 0.0;
  const auto load_dt = [&](int64_t tb, int cnt) {
    if (wave == 0 && hp.dt != nullptr && lane < cnt)
      rdt = static_cast<const uint16_t*>(hp.dt)[(tb + lane) * hp.dt_ts + h];
  };
  const auto factors = [&](int cnt, int fs) {
    if (wave != 0) return;
    const float del = lane >= cnt ? 0.0f : hp.dt == nullptr ? 1.0f : head_softplus(io_value<uint16_t>(rdt) + bias);
    const double c = lane_scan(exponent(del, A2));
    const double last = last_lane(c);
    float* f = sF + fs * (kMmaTok + 4);
    f[lane] = dir ? exp2_hw(static_cast<float>(c)) : exp2_hw(static_cast<float>(last - c)) * del;
    if (lane == 0) f[kMmaTok] = exp2_hw(static_cast<float>(last));
    dsum += last;
  };
  // the segment's blocks of the packed stream, in the direction's order
  const int64_t b0 = sg.t0 / kMmaTok, nb = sg.t0 < sg.t1 ? (sg.t1 - 1) / kMmaTok - b0 + 1 : 0;
  const auto block = [&](int64_t k, int64_t& tb, int& cnt) {
    const int64_t b = b0 + (dir ? nb - 1 - k : k);
    tb = b * kMmaTok > sg.t0 ? b * kMmaTok : sg.t0;
    const int64_t te = (b + 1) * kMmaTok < sg.t1 ? (b + 1) * kMmaTok : sg.t1;
    cnt = k < nb ? static_cast<int>(te - tb) : 0;
    return b;
  };
  int64_t tb, tn;
  int cnt, cn;
  block(0, tb, cnt);
  if (nb > 0) {
    load_dt(tb, cnt);
    if (VEC) load(tb, cnt);
    factors(cnt, 0);
    block(1, tn, cn);
    load_dt(tn, cn);
  }
  int aT = tile_at<PC>(4 * g + (li >> 2), 4 * (li & 3));
  int xT = tile_at<kMmaMP>(4 * g + (li >> 2), 16 * wave + 4 * (li & 3));
  constexpr int R16 = 16 * PC * 16, X16 = 16 * kMmaMP * 16;
  for (int64_t k = 0; k < nb; ++k) {
    const int64_t b = block(k, tb, cnt);
    asm volatile("" : "+v"(aT), "+v"(xT));
    if (!VEC) load(tb, cnt);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NK; ++i) *reinterpret_cast<hu4*>(sB + tile_at<PC>(brow + i * bstep, bcol)) = rB[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<hu4*>(sX + tile_at<kMmaMP>(xrow + 32 * i, xcol)) = rX[i];
    __syncthreads();
    const float* const f = sF + (k & 1) * (kMmaTok + 4);
    const float el = f[kMmaTok];
    block(k + 1, tn, cn);
    if (VEC && k + 1 < nb) load(tn, cn);
    factors(cn, (k + 1) & 1);
    {
      int64_t t2;
      int c2;
      block(k + 2, t2, c2);
      load_dt(t2, c2);
    }
    if (!LOCAL) {  // as it lies in the registers, 1024 contiguous bytes a tile; read once, by the next kernel: past the caches
      const int np16 = q.slices * (16 * G::NP);  // of 16 channels
      float* o = q.store[dir] + ((sg.s + b) * hp.H * q.npb + vh) * (4 * np16) + wave * np16 + 16 * n0 + lane * 4;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) nt_store(st[nt], reinterpret_cast<hf4*>(o + 256 * nt));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) st[nt] *= el;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const hf4 w0 = *reinterpret_cast<const hf4*>(f + 32 * ks + 4 * g);
      const hf4 w1 = *reinterpret_cast<const hf4*>(f + 32 * ks + 16 + 4 * g);
      const char* a = sX + 2 * ks * X16 + xT;
      hb8 part[3];
      weighted_parts(join(tr_read(a), tr_read(a + X16)), w0, w1, part);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const char* a = sB + 2 * ks * R16 + (aT ^ (nt << 5));
        const hb8 bt = join(tr_read(a), tr_read(a + R16));
#pragma unroll
        for (int u = 0; u < 3; ++u) st[nt] = mfma(bt, part[u], st[nt]);
      }
    }
  }
  float* to = LOCAL ? q.carry[dir] + rho * set
                      : ((dir ? sg.first() : sg.last()) && q.fin[dir] != nullptr ? q.fin[dir] + sg.s * set : nullptr);
  if (to != nullptr && p < pw)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = n0 + 16 * nt + 4 * g;
      float* a = to + h * PN + static_cast<int64_t>(p0 + p) * q.N + n;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < q.N) a[r] = st[nt][r];
    }
  if (LOCAL && wave == 0 && lane == 0 && p0 == 0 && n0 == 0) q.decay[dir][rho * hp.H + h] = static_cast<float>(dsum);
  __syncthreads();  // the last chunk's weights are read until here
  }
}

// Sums within the lane's row of 16: of the lanes from it on, and of those before it; and lane `l`'s value, to all
__device__ __forceinline__ float row_from(float v) {
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x101, 0xF, 0xF, true);  // row_shl:1
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x102, 0xF, 0xF, true);  // row_shl:2
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x104, 0xF, 0xF, true);  // row_shl:4
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x108, 0xF, 0xF, true);  // row_shl:8
  return v;
}
__device__ __forceinline__ float row_before(float v) {
  v = __builtin_amdgcn_update_dpp(0.0f, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x111, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x112, 0xF, 0xF, true);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x114, 0xF, 0xF, true);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0.0f, v, 0x118, 0xF, 0xF, true);  // row_shr:8
  return v;
}
__device__ __forceinline__ float lane_of(float v, int l) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}

// The sums of products z_ij = delta_j M_ij W_ij that the gradients of the decays need, from 16 x 16 tiles (rows j, columns i
// in the accumulators: lane (g, li) has j = 4g .. 4g+3 of i = li).
struct DecaySums {
  float* at;  // in LDS
  static constexpr int floats = 18 * kMmaTok + 8;
  __device__ float* rq() const { return at; }                 // row sums of z, by column tile left of the diagonal's [3][64]
  __device__ float* rt() const { return at + 3 * kMmaTok; }   // sums over i >= t > j in the diagonal's tiles [64]
  __device__ float* rp() const { return at + 4 * kMmaTok; }   // column sums of M W without the diagonal, by row tile [4][64]
  __device__ float* ri() const { return at + 8 * kMmaTok; }   // dy . (h C), by channel tile [4][64]
  __device__ float* rj() const { return at + 12 * kMmaTok; }  // x . (Gam B), likewise
  __device__ float* rd() const { return at + 16 * kMmaTok; }  // M_tt W_tt, then W_tt [2][64]
  __device__ float* re() const { return at + 18 * kMmaTok; }  // <Gam, h> by channel tile [4], e^{c_last}
  // tile (it, jt): tt = M W, w = W, del = the rows' delta; add(place, value) writes or adds
  template <typename Add>
  __device__ __forceinline__ void tile(int it, int jt, hf4 tt, hf4 w, hf4 del, int lane, int li, int g, Add add) const {
    const int i = 16 * it + li, j = 16 * jt + 4 * g;
    if (it == jt && li >> 2 == g) {
      const int r = li & 3;
      add(rd() + i, r == 0 ? tt[0] : r == 1 ? tt[1] : r == 2 ? tt[2] : tt[3]);
      add(rd() + kMmaTok + i, r == 0 ? w[0] : r == 1 ? w[1] : r == 2 ? w[2] : w[3]);
    }
    hf4 z;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (it == jt && 4 * g + r == li) tt[r] = 0.0f;
      z[r] = tt[r] * del[r];
      tt[r] = row_sum16(tt[r]);
    }
    if (li < 4) add(rp() + it * kMmaTok + j + li, li == 0 ? tt[0] : li == 1 ? tt[1] : li == 2 ? tt[2] : tt[3]);
    // sums over j up to each of the lane's: within the lane, then those of the lanes before it
    z[1] += z[0];
    z[2] += z[1];
    z[3] += z[2];
    const float o16 = __shfl_xor(z[3], 16), two = z[3] + o16, o32 = __shfl_xor(two, 32);
    if (it != jt) {
      if (g == 0) add(rq() + jt * kMmaTok + i, two + o32);
    } else {
      const float before = (g & 1 ? o16 : 0.0f) + (g & 2 ? o32 : 0.0f);
#pragma unroll
      for (int r = 0; r < 4; ++r) z[r] = row_sum16(li > 4 * g + r ? before + z[r] : 0.0f);  // of the rows below: t = j + 1
      if (li < 4 && 4 * g + li < 15) add(rt() + j + li + 1, li == 0 ? z[0] : li == 1 ? z[1] : li == 2 ? z[2] : z[3]);
      if (lane == 0) rt()[j] = 0.0f;
    }
  }
  // one wave, a token t a lane: dl_t and r_t from them; e and ew: e^{c_t}, e^{c_last - c_t}
  __device__ __forceinline__ void decay(float del, float e, float ew, int lane, int g, float& dl, float& r) const {
    float qi = 0.0f, pi = 0.0f, below = 0.0f;  // below: column sums of the row tiles below the token's own
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t > g) below += rp()[t * kMmaTok + lane];
      qi += ri()[t * kMmaTok + lane];
      pi += rj()[t * kMmaTok + lane];
    }
    const float q0 = g > 0 ? rq()[lane] : 0.0f, q1 = g > 1 ? rq()[kMmaTok + lane] : 0.0f;
    const float q2 = g > 2 ? rq()[2 * kMmaTok + lane] : 0.0f;
    qi *= e;
    pi *= ew;
    r = below + rp()[g * kMmaTok + lane] + rd()[lane] + pi;
    // sum over i >= t > j of z, with t in tile g: whole tiles below and left of it, columns j < t of the tiles below it,
    // rows i >= t of the tiles left of it, and the diagonal's tile
    const float t0 = row_sum16(q0), t1 = row_sum16(q1);
    const float far1 = lane_of(t0, 32) + lane_of(t0, 48), far2 = lane_of(t0, 48) + lane_of(t1, 48);
    const float in = ((g == 1 ? far1 : g == 2 ? far2 : 0.0f) + row_before(below * del)) + (row_from(q0 + q1 + q2) + rt()[lane]);
    // dy . (h C) of i >= t, delta x . (Gam B) of j < t
    const float qs = row_from(qi), qt1 = lane_of(qs, 16), qt2 = lane_of(qs, 32), qt3 = lane_of(qs, 48);
    const float pd = del * pi, ps = row_sum16(pd), pt0 = lane_of(ps, 0), pt1 = lane_of(ps, 16), pt2 = lane_of(ps, 32);
    const float from = qs + (g == 0 ? qt1 + qt2 + qt3 : g == 1 ? qt2 + qt3 : g == 2 ? qt3 : 0.0f);
    const float before = row_before(pd) + (g == 3 ? pt0 + pt1 + pt2 : g == 2 ? pt0 + pt1 : g == 1 ? pt0 : 0.0f);
    dl = ((in + from) + before) + re()[4] * ((re()[0] + re()[1]) + (re()[2] + re()[3]));
  }
};
// ddt of the wave's tokens, and the block's shares of dA_log, ddt_bias and dD
template <typename IO>
__device__ __forceinline__ void step_gradients(const HeadPar& hp, const DecaySums& ds, float del, float e, float ew, int64_t tb,
                                               int cnt, int64_t rho, int h, int lane, int g, IO* ddt, int64_t ddt_ts,
                                               float* __restrict__ sums) {
  float dl, r, wd = ds.rd()[kMmaTok + lane];
  ds.decay(del, e, ew, lane, g, dl, r);
  const float A = -exp2_hw(hp.A_log[h] * kLog2e);
  float dA = 0.0f, db = 0.0f;
  if (lane < cnt) {
    dA = del * dl * A;
    if (hp.dt != nullptr) {
      const float v = ld_io(static_cast<const IO*>(hp.dt) + (tb + lane) * hp.dt_ts, h) + hp.dt_bias[h];
      db = __builtin_fmaf(A, dl, r) * rcp_hw(1.0f + exp2_hw(-v * kLog2e));
      st_io(ddt, (tb + lane) * ddt_ts + h, db);
    }
  }
  for (int k = 32; k > 0; k /= 2) {
    dA += __shfl_xor(dA, k);
    db += __shfl_xor(db, k);
    wd += __shfl_xor(wd, k);
  }
  if (lane == 0) {
    float* o = sums + (rho * hp.H + h) * 3;
    o[0] = dA;
    o[1] = db;
    o[2] = wd;
  }
}

struct GradArgs {
  Tok<uint16_t> x, dy, B, C;
  int P, N, npb, G, splits;
  const float *hs, *gs;   // the states at the blocks' starts, their adjoints at the ends
  uint16_t* dx;
  int64_t dx_ts;
  float *pB, *pC;         // [splits, T, G N] sums over a workgroup's heads
  uint16_t* ddt;
  int64_t ddt_ts;
  float* sums;            // [rows64, H, 3]: the block's shares of dA_log, ddt_bias and dD
};

enum { kGci, kGcf, kGdel, kGe, kGew, kGv16, kGe16, kGn = kGe16 + 3 };
template <int NK>
struct GradGeo {
  static constexpr int NP = NK * 32, PC = NP / 8, T2 = kMmaTok * kMmaTok * 2;
  static constexpr int B = 0, C = B + kMmaTok * NP * 2, X = C + kMmaTok * NP * 2, Y = X + T2, S = Y + T2,
                       M = S + 64 * NP * 2, F = M + T2, R = F + kGn * kMmaTok * 4, bytes = R + (DecaySums::floats + 8) * 4;
};

// grid: (block, group, share of its heads)
// B, C and the scores C . B stay for all heads of the workgroup, x, dy and the two states of the next head are loaded
// under this one's products.  8 x 2048 tokens, 24 heads: 228 us (traced mean), of which its traffic (0.73 GB, the
// states mostly) would be 120 at the copy's rate.  A head is a chain of products between barriers, and two workgroups
// (256 registers, 28 more spilled; 81 KB of LDS) cover it in part: waves wait 62% of their cycles, VALU issue 32%, MFMA
// 14%.
// Values that are not finite: masked zeros of M and of delta W d must not meet them in dy, C or B, so blocks that hold one
// take those products token by token.  (x needs no such care: its products are masked before they are used.)
template <int NK, bool VEC>
__global__ __launch_bounds__(kMmaThreads, 2) void k_heads_grads(GradArgs q, HeadPar hp) {
  typedef GradGeo<NK> G;
  constexpr int NT = 2 * NK, PC = G::PC, NTW = (NT + 3) / 4;  // column tiles of dB and dC per wave
  extern __shared__ __align__(16) char lds[];
  char *const sB = lds + G::B, *const sC = lds + G::C, *const sX = lds + G::X, *const sY = lds + G::Y;
  char *const sS = lds + G::S, *const sM = lds + G::M;
  float* const f = reinterpret_cast<float*>(lds + G::F);
  const DecaySums ds{reinterpret_cast<float*>(lds + G::R)};
  int* const odd = reinterpret_cast<int*>(ds.re() + 8);         // by wave: not all finite in its pieces of dy [4], of B and C [4]

  const int tid = threadIdx.x;
  int lane = tid & 63, li = lane & 15, g = lane >> 4;
  int wv = tid >> 6, wave = __builtin_amdgcn_readfirstlane(wv);
  const int split = blockIdx.x % q.splits;
  const int group = (blockIdx.x / q.splits) % q.G;
  const int64_t rho = blockIdx.x / q.splits / q.G;
  const Segment sg = segment_of(hp.cu, hp.S, rho, kMmaTok);
  const int hg = hp.H / q.G;
  const int h0 = group * hg + split * hg / q.splits, h1 = group * hg + (split + 1) * hg / q.splits;
  if (sg.t0 >= sg.t1) {
    for (int i = tid; i < (h1 - h0) * 3; i += kMmaThreads) q.sums[(rho * hp.H + h0) * 3 + i] = 0.0f;
    return;
  }
  const int64_t tb = sg.t0;
  const int cnt = static_cast<int>(sg.t1 - tb);

  // LDS offsets of a lane's operands (natural order, four columns, transposed) in tiles of PC and of 8 pieces;
  // opaque for each head, since their sums with the tiles' constants would not fit the registers
  int aN = tile_at<PC>(li, 8 * g), aT = tile_at<PC>(4 * g + (li >> 2), 4 * (li & 3));
  int mN = tile_at<kMmaMP>(li, 8 * g), mK = tile_at<kMmaMP>(li, 4 * g), mT = tile_at<kMmaMP>(4 * g + (li >> 2), 4 * (li & 3));
  constexpr int R16 = 16 * PC * 16, M16 = 16 * kMmaMP * 16;

  // B and C of the block, for all heads
  const int dH = hp.H * q.P, gn = q.G * q.N;
  {
    const int brow = tid / PC, bcol = (tid % PC) * 8;
    constexpr int bstep = kMmaThreads / PC;
    const hbuf bB = token_rows(q.B.p, tb, q.B.ts, cnt, gn), bC = token_rows(q.C.p, tb, q.C.ts, cnt, gn);
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int row = brow + i * bstep, col = group * q.N + bcol;
      const hu4 b = load8<VEC>(bB, (row * static_cast<int>(q.B.ts) + col) * 2, q.N - bcol);
      const hu4 c = load8<VEC>(bC, (row * static_cast<int>(q.C.ts) + col) * 2, q.N - bcol);
      *reinterpret_cast<hu4*>(sB + tile_at<PC>(row, bcol)) = b;
      *reinterpret_cast<hu4*>(sC + tile_at<PC>(row, bcol)) = c;
      bad |= not_finite(b) | not_finite(c);
    }
    const int any = __any(bad != 0);
    if (lane == 0) odd[4 + wave] = any;
  }
  const hbuf bX = token_rows(q.x.p, tb, q.x.ts, cnt, dH), bY = token_rows(q.dy.p, tb, q.dy.ts, cnt, dH);
  const hbuf bO = token_rows(q.dx, tb, q.dx_ts, cnt, dH);
  const int xrow = tid >> 3, xcol = (tid & 7) * 8;
  hu4 rX[2], rY[2];
  const auto load = [&](int h, int pb) {
    const int n = q.P - 64 * pb - xcol, at = h * q.P + 64 * pb + xcol;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      rX[i] = load8<VEC>(bX, ((xrow + 32 * i) * static_cast<int>(q.x.ts) + at) * 2, n);
      rY[i] = load8<VEC>(bY, ((xrow + 32 * i) * static_cast<int>(q.dy.ts) + at) * 2, n);
    }
  };
  load(h0, 0);
  __syncthreads();
  const bool odd_bc = __builtin_amdgcn_readfirstlane(odd[4] | odd[5] | odd[6] | odd[7]) != 0;

  // the wave's score tiles (it, jt <= it): C_i . B_j, rows j and columns i, the same for every head
  const auto tile_i = [&](int u) { return u < 2 ? (wave < 2 ? 3 : wave == 2 ? 2 : 1) : (wave == 2 ? 2 : 0); };
  const auto tile_j = [&](int u) { return u < 2 ? (wave == 1 ? 2 + u : u) : (wave == 2 ? 2 : 0); };
  hf4 cb[3];
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    cb[u] = hf4{0, 0, 0, 0};
    if (u == 2 && wave < 2) continue;
#pragma unroll
    for (int k = 0; k < NK; ++k)
      cb[u] = mfma(lds8(sB + tile_j(u) * R16 + (aN ^ (k << 6))), lds8(sC + tile_i(u) * R16 + (aN ^ (k << 6))), cb[u]);
  }
  hf4 dB[4][NTW], dC[4][NTW];  // [token 16 t + 4g + r][n = 16 nt + li]
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int n = 0; n < NTW; ++n) dB[t][n] = dC[t][n] = hf4{0, 0, 0, 0};

  const hb4 none = to_bf4(hf4{0, 0, 0, 0});
  for (int h = h0; h < h1; ++h)
    for (int pb = 0; pb < q.npb; ++pb) {
      // a token's sums over the channel blocks of a head gather where they lie: the same lane adds to a place each time
      const auto add = [&](float* at, float v) { *at = pb > 0 ? *at + v : v; };
      asm volatile("" : "+v"(aN), "+v"(aT), "+v"(mN), "+v"(mK), "+v"(mT), "+v"(lane), "+v"(li), "+v"(g), "+v"(wv));
      wave = __builtin_amdgcn_readfirstlane(wv);
      // the state and its adjoint: rows p = 16 wave + li, columns 32 k + 8 g ..
      const int64_t srow = ((rho * hp.H + h) * q.npb + pb) * (64 * G::NP) + wave * (16 * G::NP) + (g >> 1) * 256 + (g & 1) * 128 + li * 4;
      hf4 s[NK][2];
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        s[k][0] = nt_load(reinterpret_cast<const hf4*>(q.hs + srow + 512 * k));
        s[k][1] = nt_load(reinterpret_cast<const hf4*>(q.hs + srow + 512 * k + 64));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<hu4*>(sX + tile_at<kMmaMP>(xrow + 32 * i, xcol)) = rX[i];
        *reinterpret_cast<hu4*>(sY + tile_at<kMmaMP>(xrow + 32 * i, xcol)) = rY[i];
      }
      const int any = __any((not_finite(rY[0]) | not_finite(rY[1])) != 0);
      if (lane == 0) odd[wave] = any;
      if (wave == 3 && pb == 0) {
        float del = 0.0f;
        if (lane < cnt) del = head_delta<uint16_t>(hp, tb + lane, h);
        const double c = lane_scan(exponent(del, head_A2(hp, h)));
        const double last = last_lane(c);
        const double whole = floor(c);
        const float ci = static_cast<float>(whole), cf = static_cast<float>(c - whole);
        f[kGci * kMmaTok + lane] = ci;
        f[kGcf * kMmaTok + lane] = cf;
        f[kGdel * kMmaTok + lane] = del;
        f[kGe * kMmaTok + lane] = exp2_hw(static_cast<float>(c));
        f[kGew * kMmaTok + lane] = exp2_hw(static_cast<float>(last - c));
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const float ti = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ci), 16 * t + 15));
          const float tf = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cf), 16 * t + 15));
          const float d = (ci - ti) + (cf - tf);
          f[(kGe16 + t) * kMmaTok + lane] = exp2_hw(d);
          if (lane >> 4 == t) f[kGv16 * kMmaTok + lane] = exp2_hw(-d);
        }
        if (lane == 0) ds.re()[4] = exp2_hw(static_cast<float>(last));
      }
      __syncthreads();
      // scores dy_i . x_j; the tiles of delta M (for dx) now, those of delta W d (for dB, dC) later
      hb4 m2[3], m2l[3];
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        m2[u] = m2l[u] = none;
        if (u == 2 && wave < 2) continue;
        const int it = tile_i(u), jt = tile_j(u), i = 16 * it + li, j = 16 * jt + 4 * g;
        hf4 w = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 2; ++k)
          w = mfma(lds8(sX + jt * M16 + (mN ^ (k << 6))), lds8(sY + it * M16 + (mN ^ (k << 6))), w);
        const hf4 del = *reinterpret_cast<const hf4*>(f + kGdel * kMmaTok + j);
        hf4 d;
        if (it != jt) {
          d = f[(kGe16 + jt) * kMmaTok + i] * *reinterpret_cast<const hf4*>(f + kGv16 * kMmaTok + j);
        } else {
          const float ci = f[kGci * kMmaTok + i], cf = f[kGcf * kMmaTok + i];
          const hf4 cj = *reinterpret_cast<const hf4*>(f + kGci * kMmaTok + j), fj = *reinterpret_cast<const hf4*>(f + kGcf * kMmaTok + j);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float v = exp2_hw((ci - cj[r]) + (cf - fj[r]));
            d[r] = 4 * g + r <= li ? v : 0.0f;
          }
        }
        // a value that is not finite times a masked zero would be NaN: the mask selects
        hf4 m1, w2, tt;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool on = it != jt || 4 * g + r <= li;
          const float md = on ? cb[u][r] * d[r] : 0.0f;
          m1[r] = md * del[r];
          w2[r] = on ? w[r] * d[r] * del[r] : 0.0f;
          tt[r] = on ? md * w[r] : 0.0f;
        }
        ds.tile(it, jt, tt, w, del, lane, li, g, add);
        *reinterpret_cast<hb4*>(sM + it * M16 + (mK ^ (jt << 5))) = to_bf4(m1);
        m2[u] = to_bf4(w2);
        m2l[u] = to_bf4(w2 - to_f4(m2[u]));
      }
      __builtin_amdgcn_sched_barrier(0);
      // h C for q, in three parts; h's first part to LDS for dC
      hf4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = hf4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        hb8 part[3];
        bf_parts(s[k][0], s[k][1], part);
        *reinterpret_cast<hb8*>(sS + wave * R16 + (aN ^ (k << 6))) = part[0];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const hb8 c = lds8(sC + t * R16 + (aN ^ (k << 6)));
#pragma unroll
          for (int u = 0; u < 3; ++u) acc[t] = mfma(part[u], c, acc[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const hf4 y = to_f4(lds4(sY + t * M16 + (mK ^ (wave << 5))));
        float v = (acc[t][0] * y[0] + acc[t][1] * y[1]) + (acc[t][2] * y[2] + acc[t][3] * y[3]);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (g == 0) add(ds.ri() + wave * kMmaTok + 16 * t + li, v);
      }
      __syncthreads();
      // the adjoint's loads, in flight over the products of the state
      hf4 a[NK][2];
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        a[k][0] = nt_load(reinterpret_cast<const hf4*>(q.gs + srow + 512 * k));
        a[k][1] = nt_load(reinterpret_cast<const hf4*>(q.gs + srow + 512 * k + 64));
      }
      __builtin_amdgcn_sched_barrier(0);
      // dx within the block: rows p = 16 wave + 4g + r, columns j = 16 jt + li
      hf4 dx[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) dx[t] = hf4{0, 0, 0, 0};
      if (__builtin_amdgcn_readfirstlane(odd[0] | odd[1] | odd[2] | odd[3]) == 0) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const char* ya = sY + 2 * ks * M16 + (mT ^ (wave << 5));
        const hb8 yt = join(tr_read(ya), tr_read(ya + M16));
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
          if (ks == 0 && jt > 1) continue;
          const char* ma = sM + 2 * ks * M16 + (mT ^ (jt << 5));
          // tiles above the diagonal's were not written: zeros
          const hb8 m = join((jt & 1) && jt / 2 == ks ? none : tr_read(ma), tr_read(ma + M16));
          dx[jt] = mfma(yt, m, dx[jt]);
        }
      }
      } else {  // a value that is not finite must not meet the zeros of later tokens: token by token
#pragma unroll 1
        for (int i = 0; i < cnt; ++i) {
          const hf4 y = to_f4(lds4(sY + tile_at<kMmaMP>(i, 16 * wave + 4 * g)));
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (16 * t + li <= i)
              dx[t] += y * io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sM + tile_at<kMmaMP>(i, 16 * t + li)));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // dC from the state
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const int nt = wave * NTW + n;
        if (nt >= NT) continue;
        hb8 sT[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const char* sa = sS + 2 * ks * R16 + (aT ^ (nt << 5));
          sT[ks] = join(tr_read(sa), tr_read(sa + R16));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          hf4 v = {0, 0, 0, 0};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            v = mfma(join(lds4(sY + t * M16 + (mK ^ (ks << 6))), lds4(sY + t * M16 + (mK ^ (ks << 6) ^ 32))), sT[ks], v);
          dC[t][n] += v * *reinterpret_cast<const hf4*>(f + kGe * kMmaTok + 16 * t + 4 * g);
        }
      }
      __syncthreads();
      // Gam B in three parts, <Gam, h>; the tiles of delta W d and Gam's first part to LDS
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (u == 2 && wave < 2) continue;
        *reinterpret_cast<hb4*>(sM + tile_i(u) * M16 + (mK ^ (tile_j(u) << 5))) = m2[u];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = hf4{0, 0, 0, 0};
      float dot = 0.0f;
#pragma unroll
      for (int k = 0; k < NK; ++k) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dot = __builtin_fmaf(s[k][0][r], a[k][0][r], dot);
          dot = __builtin_fmaf(s[k][1][r], a[k][1][r], dot);
        }
        hb8 part[3];
        bf_parts(a[k][0], a[k][1], part);
        *reinterpret_cast<hb8*>(sS + wave * R16 + (aN ^ (k << 6))) = part[0];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const hb8 b = lds8(sB + t * R16 + (aN ^ (k << 6)));
#pragma unroll
          for (int u = 0; u < 3; ++u) acc[t] = mfma(part[u], b, acc[t]);
        }
      }
      dot = row_sum16(dot);
      dot += __shfl_xor(dot, 16);
      dot += __shfl_xor(dot, 32);
      if (lane == 0) add(ds.re() + wave, dot);
      __builtin_amdgcn_sched_barrier(0);
      const float Dh = hp.D != nullptr ? hp.D[h] : 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int j = 16 * t + li, p = 16 * wave + 4 * g;
        const hf4 x = to_f4(lds4(sX + t * M16 + (mK ^ (wave << 5))));
        const hf4 y = to_f4(lds4(sY + t * M16 + (mK ^ (wave << 5))));
        float v = (acc[t][0] * x[0] + acc[t][1] * x[1]) + (acc[t][2] * x[2] + acc[t][3] * x[3]);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (g == 0) add(ds.rj() + wave * kMmaTok + j, v);
        const hf4 o = dx[t] + acc[t] * (f[kGew * kMmaTok + j] * f[kGdel * kMmaTok + j]) + y * Dh;
        const hu2 ob = __builtin_bit_cast(hu2, to_bf4(o));
        const int off = (j * static_cast<int>(q.dx_ts) + h * q.P + 64 * pb + p) * 2, n = q.P - 64 * pb - p;
        if (VEC) {
          typedef uint32_t u2 __attribute__((ext_vector_type(2)));
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, ob), bO, n > 0 ? off : kMmaPastEnd, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(ob[e / 2] >> (16 * (e % 2))), bO,
                                                  e < n ? off + 2 * e : kMmaPastEnd, 0, 0);
        }
      }
      __syncthreads();
      // delta W d's second part in dy's place, which is not needed any more
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (u == 2 && wave < 2) continue;
        *reinterpret_cast<hb4*>(sY + tile_i(u) * M16 + (mK ^ (tile_j(u) << 5))) = m2l[u];
      }
      {  // the next tiles' loads, now that the adjoint has left its registers
        const int hn = pb + 1 < q.npb ? h : h + 1, pn = pb + 1 < q.npb ? pb + 1 : 0;
        if (hn < h1) load(hn, pn);
      }
      // dB from the adjoint
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const int nt = wave * NTW + n;
        if (nt >= NT) continue;
        hb8 gT[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const int o = 2 * ks * R16 + (aT ^ (nt << 5));
          gT[ks] = join(tr_read(sS + o), tr_read(sS + o + R16));
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          hf4 v = {0, 0, 0, 0};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            v = mfma(join(lds4(sX + t * M16 + (mK ^ (ks << 6))), lds4(sX + t * M16 + (mK ^ (ks << 6) ^ 32))), gT[ks], v);
          dB[t][n] += v * (*reinterpret_cast<const hf4*>(f + kGew * kMmaTok + 16 * t + 4 * g) *
                           *reinterpret_cast<const hf4*>(f + kGdel * kMmaTok + 16 * t + 4 * g));
        }
      }
      __syncthreads();
      // dB and dC within the block
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const int nt = wave * NTW + n;
        if (nt >= NT) continue;
        if (!odd_bc) {
          hb8 cT[2], bT[2];
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const int o = 2 * ks * R16 + (aT ^ (nt << 5));
            cT[ks] = join(tr_read(sC + o), tr_read(sC + o + R16));
            bT[ks] = join(tr_read(sB + o), tr_read(sB + o + R16));
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const char* const sm = part ? sY : sM;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                if (!(ks == 0 && t > 1)) {  // i >= j: rows j = 16 t ..
                  const char* ma = sm + 2 * ks * M16 + (mT ^ (t << 5));
                  dB[t][n] = mfma(join((t & 1) && t / 2 == ks ? none : tr_read(ma), tr_read(ma + M16)), cT[ks], dB[t][n]);
                }
                if (!(ks == 1 && t < 2)) {  // j <= i: rows i = 16 t ..
                  const char* ma = sm + t * M16;
                  dC[t][n] = mfma(join(lds4(ma + (mK ^ (ks << 6))), (t & 1) == 0 && t / 2 == ks ? none : lds4(ma + (mK ^ (ks << 6) ^ 32))),
                                  bT[ks], dC[t][n]);
                }
              }
          }
        }
        if (odd_bc) {  // as for dx: C of earlier and B of later tokens have no part in a sum
          const int col = 16 * nt + li;
#pragma unroll 1
          for (int u = 0; u < cnt; ++u) {
            const float c = io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sC + tile_at<PC>(u, col)));
            const float b = io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sB + tile_at<PC>(u, col)));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int at = tile_at<kMmaMP>(u, 16 * t + 4 * g);
              const hf4 m = to_f4(lds4(sM + at)) + to_f4(lds4(sY + at));
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int row = 16 * t + 4 * g + r;
                if (row <= u) dB[t][n][r] = __builtin_fmaf(m[r], c, dB[t][n][r]);
                if (row >= u) {
                  const int one = tile_at<kMmaMP>(row, u);
                  dC[t][n][r] = __builtin_fmaf(io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sM + one)) +
                                                   io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sY + one)),
                                               b, dC[t][n][r]);
                }
              }
            }
          }
        }
      }
      if (wave == 0 && pb == q.npb - 1)
        step_gradients(hp, ds, f[kGdel * kMmaTok + lane], f[kGe * kMmaTok + lane], f[kGew * kMmaTok + lane], tb, cnt, rho, h, lane, g,
                       q.ddt, q.ddt_ts, q.sums);
      __syncthreads();
    }
#pragma unroll
  for (int n = 0; n < NTW; ++n) {
    const int col = 16 * (wave * NTW + n) + li;
    if (wave * NTW + n < NT && col < q.N)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * t + 4 * g + r;
          if (row < cnt) {
            const int64_t o = (static_cast<int64_t>(split) * hp.T + tb + row) * gn + group * q.N + col;
            q.pB[o] = dB[t][n][r];
            q.pC[o] = dC[t][n][r];
          }
        }
  }
}

// dB and dC: the sums of the workgroups' shares, in order
__global__ __launch_bounds__(256) void k_heads_shares(const float* __restrict__ pB, const float* __restrict__ pC,
                                                      uint16_t* __restrict__ dB, uint16_t* __restrict__ dC, int64_t db_ts,
                                                      int64_t dc_ts, int64_t T, int gn, int splits) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= T * gn) return;
  float b = 0.0f, c = 0.0f;
  for (int k = 0; k < splits; ++k) {
    b += pB[k * T * gn + i];
    c += pC[k * T * gn + i];
  }
  const int64_t t = i / gn;
  const int n = static_cast<int>(i % gn);
  st_io(dB, t * db_ts + n, b);
  st_io(dC, t * dc_ts + n, c);
}

// The same sums for the token-by-token backward, in float32 products on the matrix cores (v_mfma_f32_16x16x4_f32): dl and r of
// a 64-token block from its scores and from the states that the walks stored at its start (hs) and end (gs).  One
// workgroup per (block, head).  It stages 64 columns at a time of B and C, then of x and dy, the next ones loaded under
// this one's products; for each 64 channels the states' columns go from memory to the wave that takes their 16 channels.
// Lane l supplies row (or column) l % 16, and of 16 K indices 4g .. 4g+3, one to each of four products.
// 8 x 2048 float32 tokens, 24 heads 64 x 128: 303 us of the call's 5080 (0.4 GB of states read, 19 GFLOP; 212 registers,
// two workgroups a CU); 389 ragged tokens, 6 heads 40 x 24: 11 us of 58.  The sums of C . dC - B . dB from the block's end,
// which need no scores, took 150 and 9 with errors of 1e-6 where these have 2e-7.
// Four elements of a row, of which n exist (the others read as zeros); rows may start anywhere.  WIDE: rows have four at
// least, so that a row's last ones can be loaded with those before them.
template <bool WIDE, typename IO>
__device__ __forceinline__ hf4 ld4(const IO* p, int n) {
  hf4 v = {0, 0, 0, 0};
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = ld_io(p, i);
  } else if (n > 0) {
    typedef IO vec __attribute__((ext_vector_type(4), aligned(sizeof(IO))));
    const vec u = *reinterpret_cast<const vec*>(p - (n < 4 ? 4 - n : 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(IO) == 4) v[i] = u[i];
      else v[i] = io_value<IO>(u[i]);
    }
    if (n < 4) v = n == 3 ? hf4{v[1], v[2], v[3], 0} : n == 2 ? hf4{v[2], v[3], 0, 0} : hf4{v[3], 0, 0, 0};
  }
  return v;
}
__device__ __forceinline__ hf4 lds_f4(const float* p) { return *reinterpret_cast<const hf4*>(p); }
__device__ __forceinline__ hf4 mfma4(hf4 a, hf4 b, hf4 c) {
#pragma unroll
  for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[k], b[k], c, 0, 0, 0);
  return c;
}
template <typename IO, bool WIDE>
__global__ __launch_bounds__(kMmaThreads) void k_heads_ddt(Tok<IO> x, Tok<IO> dy, Tok<IO> B, Tok<IO> C, HeadPar hp,
                                                           const float* __restrict__ hs, const float* __restrict__ gs, int P,
                                                           int N, float* __restrict__ delta, IO* __restrict__ ddt,
                                                           int64_t ddt_ts, float* __restrict__ sums) {
  __shared__ float sf[5][kMmaTok], ss[DecaySums::floats];
  __shared__ __align__(16) float sa[kMmaTok][64 + 4], sb[kMmaTok][64 + 4];  // (B, C) or (x, dy)
  auto &sci = sf[0], &scf = sf[1], &sdel = sf[2], &se = sf[3], &sew = sf[4];
  const DecaySums ds{ss};
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = blockIdx.x % hp.H;
  const int64_t rho = blockIdx.x / hp.H;
  const Segment sg = segment_of(hp.cu, hp.S, rho, kHeadsBlock);
  if (sg.t0 >= sg.t1) {
    if (tid < 3) sums[(rho * hp.H + h) * 3 + tid] = 0.0f;
    return;
  }
  const int64_t tb = sg.t0;
  const int cnt = static_cast<int>(sg.t1 - tb);
  hf4 ra[4], rb[4], hv[4], gv[4];  // as loaded: the staged pair's, and the states' columns
  const int srow = tid >> 2, scol = (tid & 3) * 4, p = 16 * wave + li;
  const int nchunks = (N + 63) / 64, per = nchunks + 1, steps = per * ((P + 63) / 64);
  // step s: B and C (and the states of the step's channels), or x and dy
  const auto load = [&](int s) {
    const bool bc = s % per < nchunks;
    const int c0 = bc ? s % per * 64 : s / per * 64, width = (bc ? N : P) - c0;
    const int64_t t = tb + (srow < cnt ? srow : 0);
    const IO *u = (bc ? B : x).at(t, h) + c0, *v = (bc ? C : dy).at(t, h) + c0;
    const int pc = s / per * 64 + p;
    const int64_t at = ((rho * hp.H + h) * P + (pc < P ? pc : 0)) * static_cast<int64_t>(N) + c0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = srow < cnt ? width - scol - 16 * k : 0;
      ra[k] = ld4<WIDE>(u + scol + 16 * k, n);
      rb[k] = ld4<WIDE>(v + scol + 16 * k, n);
      const int m = bc && pc < P ? width - 4 * g - 16 * k : 0;
      hv[k] = ld4<WIDE>(hs + at + 4 * g + 16 * k, m);
      gv[k] = ld4<WIDE>(gs + at + 4 * g + 16 * k, m);
    }
  };
  load(0);
  if (wave == 0) {
    float del = 0.0f;
    if (lane < cnt) {
      del = head_delta<IO>(hp, tb + lane, h);
      delta[(tb + lane) * hp.H + h] = del;
    }
    const double c = lane_scan(exponent(del, head_A2(hp, h))), last = last_lane(c), whole = floor(c);
    sci[lane] = static_cast<float>(whole);
    scf[lane] = static_cast<float>(c - whole);
    sdel[lane] = del;
    se[lane] = exp2_hw(static_cast<float>(c));
    sew[lane] = exp2_hw(static_cast<float>(last - c));
    if (lane == 0) ds.re()[4] = exp2_hw(static_cast<float>(last));
  }
  // the scores' tiles (it, jt <= it) over the waves
  const auto tile_i = [&](int u) { return u < 2 ? (wave < 2 ? 3 : wave == 2 ? 2 : 1) : (wave == 2 ? 2 : 0); };
  const auto tile_j = [&](int u) { return u < 2 ? (wave == 1 ? 2 + u : u) : (wave == 2 ? 2 : 0); };
  hf4 cb[3], w[3], hc[4], gb[4];  // C . B and dy . x of the tiles; h C and Gam B of the wave's 16 channels
#pragma unroll
  for (int u = 0; u < 3; ++u) cb[u] = w[u] = hf4{0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < 4; ++t) hc[t] = gb[t] = hf4{0, 0, 0, 0};
  float qi[4] = {0, 0, 0, 0}, pi[4] = {0, 0, 0, 0}, dot = 0.0f;
  for (int s = 0; s < steps; ++s) {
    const bool bc = s % per < nchunks;
    const int left = bc ? N - s % per * 64 : P - s / per * 64;  // columns
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      *reinterpret_cast<hf4*>(&sa[srow][scol + 16 * k]) = ra[k];
      *reinterpret_cast<hf4*>(&sb[srow][scol + 16 * k]) = rb[k];
    }
    __syncthreads();
    if (bc) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (16 * k >= left) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) dot = __builtin_fmaf(hv[k][r], gv[k][r], dot);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          hc[t] = mfma4(hv[k], lds_f4(&sb[16 * t + li][16 * k + 4 * g]), hc[t]);
          gb[t] = mfma4(gv[k], lds_f4(&sa[16 * t + li][16 * k + 4 * g]), gb[t]);
        }
      }
    }
    if (s + 1 < steps) load(s + 1);
    if (!bc || s < nchunks) {  // C . B once, dy . x of all channels
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (u == 2 && wave < 2) break;
        hf4 acc = bc ? cb[u] : w[u];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (16 * k >= left) break;
          acc = mfma4(lds_f4(&sa[16 * tile_j(u) + li][16 * k + 4 * g]), lds_f4(&sb[16 * tile_i(u) + li][16 * k + 4 * g]), acc);
        }
        (bc ? cb[u] : w[u]) = acc;
      }
    }
    if (!bc) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const hf4 xv = lds_f4(&sa[16 * t + li][16 * wave + 4 * g]), yv = lds_f4(&sb[16 * t + li][16 * wave + 4 * g]);
        qi[t] += (hc[t][0] * yv[0] + hc[t][1] * yv[1]) + (hc[t][2] * yv[2] + hc[t][3] * yv[3]);
        pi[t] += (gb[t][0] * xv[0] + gb[t][1] * xv[1]) + (gb[t][2] * xv[2] + gb[t][3] * xv[3]);
        hc[t] = gb[t] = hf4{0, 0, 0, 0};
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    if (u == 2 && wave < 2) break;
    const int it = tile_i(u), jt = tile_j(u), i = 16 * it + li, j = 16 * jt + 4 * g;
    hf4 tt, del;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float d = exp2_hw((sci[i] - sci[j + r]) + (scf[i] - scf[j + r]));
      del[r] = sdel[j + r];
      tt[r] = j + r <= i ? cb[u][r] * d * w[u][r] : 0.0f;
    }
    ds.tile(it, jt, tt, w[u], del, lane, li, g, [](float* at, float v) { *at = v; });
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    qi[t] += __shfl_xor(qi[t], 16);
    qi[t] += __shfl_xor(qi[t], 32);
    pi[t] += __shfl_xor(pi[t], 16);
    pi[t] += __shfl_xor(pi[t], 32);
    if (g == 0) {
      ds.ri()[wave * kMmaTok + 16 * t + li] = qi[t];
      ds.rj()[wave * kMmaTok + 16 * t + li] = pi[t];
    }
  }
  dot = row_sum16(dot);
  dot += __shfl_xor(dot, 16);
  dot += __shfl_xor(dot, 32);
  if (lane == 0) ds.re()[wave] = dot;
  __syncthreads();
  if (wave == 0) step_gradients(hp, ds, sdel[lane], se[lane], sew[lane], tb, cnt, rho, h, lane, g, ddt, ddt_ts, sums);
}

}  // namespace mm
