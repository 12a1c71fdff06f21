// The head scan: linear attention with one decay per head, over packed sequences.
//
//   delta = softplus(dt + dt_bias)          (1 when no dt is given: a fixed decay for each head)
//   h_t   = a_t h_{t-1} + delta_t x_t B_t^T,   a_t = exp(-exp(A_log) delta_t)     [P, N] per head
//   y_t   = h_t C_t + D x_t                    head h reads group h / (H / G) of B and C
//
// Segments.  A sequence is cut where the packed token index is a multiple of Ls (the segment
// length), so the segment with tokens [b Ls, (b + 1) Ls) of sequence s has the row s + b in every
// per-segment array: the rows of the sequences follow one another without overlap, no plan has to
// be computed, and there are at most T / Ls + S of them.  With Ls > T every sequence is one segment.
// With shorter segments three launches replace one: the state each segment adds from zero
// (LOCAL), the states the segments start from (k_heads_carry), and the outputs.
//
// The kernels here take the recurrence token by token in float32 and serve every type, size and
// stride.  (The gradients of their decays come from k_heads_ddt, by blocks of 64 tokens.)
#pragma once

#include "mm_device.h"

namespace mm {

constexpr int kHeadsMaxN = 256;  // columns of the state (N, and P in the backward's transposed runs)
constexpr int kHeadsMaxP = 256;
constexpr int kSeqThreads = 256;
constexpr int kSeqRows = 16;     // state rows per workgroup: one per 16-lane row
constexpr int kSeqTok = 16;      // tokens staged at a time
constexpr int kHeadsBlock = 64;  // tokens per block of the backward's inner products

// row rho of a per-segment array: its sequence, and its tokens [t0, t1) (none: t0 >= t1)
struct Segment {
  int s;
  int64_t t0, t1;
  int64_t seq0, seq1;  // the sequence's tokens
  __device__ bool first() const { return t0 <= seq0; }
  __device__ bool last() const { return t1 >= seq1; }
  // whether the sequence has several segments, and whether this row is one (or an empty sequence's only one)
  __device__ bool many(int64_t L) const {
    return seq1 > seq0 && static_cast<uint32_t>(seq1 - 1) / static_cast<uint32_t>(L) >
                              static_cast<uint32_t>(seq0) / static_cast<uint32_t>(L);
  }
  __device__ bool none(int64_t rho, int64_t L) const {
    return t0 >= t1 && !(seq0 == seq1 && rho == s + static_cast<uint32_t>(seq0) / static_cast<uint32_t>(L));
  }
};
// the largest s with s + cu[s] / L <= rho
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ cu, int S, int64_t rho, int64_t L) {
  int lo = 0, hi = S - 1;
  const uint32_t L32 = static_cast<uint32_t>(L);
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mid + static_cast<int64_t>(static_cast<uint32_t>(cu[mid]) / L32) <= rho) lo = mid; else hi = mid - 1;
  }
  Segment g;
  g.s = lo;
  g.seq0 = cu[lo];
  g.seq1 = cu[lo + 1];
  const int64_t b = rho - lo;
  g.t0 = b * L > g.seq0 ? b * L : g.seq0;
  g.t1 = (b + 1) * L < g.seq1 ? (b + 1) * L : g.seq1;
  return g;
}
// The segments that a workgroup of the matrix-core kernels walks: with `whole`, sequence `row` (Ls > T); else all
// segments of the packed stream's tokens [row Ls, (row + 1) Ls), whatever sequences they belong to, so that every
// workgroup has the same number of tokens.
struct SegmentWalk {
  const int32_t* cu;
  int S, s;
  int64_t row, L;
  bool whole;
  __device__ SegmentWalk(const int32_t* cu_, int S_, int64_t row_, int64_t L_, bool whole_)
      : cu(cu_), S(S_), s(whole_ ? static_cast<int>(row_) : seq_of(cu_, S_, row_ * L_)), row(row_), L(L_), whole(whole_) {}
  // the next segment and its row of the per-segment arrays; false: none
  __device__ bool next(Segment& g, int64_t& rho) {
    const int64_t lo = whole ? 0 : row * L, hi = whole ? INT32_MAX : (row + 1) * L;
    while (s < S) {
      g.s = s;
      g.seq0 = cu[s];
      g.seq1 = cu[s + 1];
      if (g.seq0 >= hi) return false;
      s = whole ? S : s + 1;
      g.t0 = g.seq0 > lo ? g.seq0 : lo;
      g.t1 = g.seq1 < hi ? g.seq1 : hi;
      rho = g.s + (whole ? 0 : row);
      if (whole || g.t0 < g.t1) return true;
    }
    return false;
  }
};
// whether a sequence has more than `limit` tokens: the choice between two ways that the host, which does not know the
// lengths, leaves to the kernels of both; every wave finds it by itself
__device__ __forceinline__ bool longer_than(const int32_t* __restrict__ cu, int S, int64_t limit) {
  int any = 0;
  for (int s = threadIdx.x & 63; s < S; s += kWave) any |= static_cast<int64_t>(cu[s + 1]) - cu[s] > limit;
  return __any(any) != 0;
}
// rows of a per-segment array for S sequences and T tokens
inline int64_t segment_rows(int64_t S, int64_t T, int64_t L) { return S + T / L; }

// a token tensor [T, ., W]: element (t, h, i) at t * ts + (h / div) * W + i
template <typename IO>
struct Tok {
  const IO* p;
  int64_t ts;
  int W, div;
  __device__ const IO* at(int64_t t, int h) const { return p + t * ts + static_cast<int64_t>(h / div) * W; }
};

struct HeadPar {
  const void* dt;        // [T, H] io, or NULL
  int64_t dt_ts;
  const float* A_log;    // [H]
  const float* dt_bias;  // [H] (NULL without dt)
  const float* D;        // [H] or NULL
  const int32_t* cu;
  int S, H;
  int64_t T;
};
// softplus with a minimum and a maximum that keep a NaN
__device__ __forceinline__ float head_softplus(float v) {
  const float e = exp2_hw(__builtin_elementwise_minimum(v, 20.0f) * kLog2e);
  const float u = 1.0f + e;
  const float d = e - (u - 1.0f);
  return __builtin_elementwise_maximum(v, __builtin_fmaf(log2_hw(u), kLn2, d));
}
template <typename IO>
__device__ __forceinline__ float head_delta(const HeadPar& hp, int64_t t, int h) {
  if (hp.dt == nullptr) return 1.0f;
  return head_softplus(ld_io(static_cast<const IO*>(hp.dt) + t * hp.dt_ts, h) + hp.dt_bias[h]);
}
// A log2(e), finite (or NaN): a place without a token has delta = 0, and must have the exponent 0
__device__ __forceinline__ float head_A2(const HeadPar& hp, int h) {
  return __builtin_elementwise_maximum(-exp2_hw(hp.A_log[h] * kLog2e) * kLog2e, -3e38f);
}

// One run of the recurrence on a state of R rows and K columns (element (r, k) of a stored state at
// r sr + k sk):
//   forward   h = a_t h + w_t u_t[r] v_t[k],   out_t[r] = sum_k h s_t[k]          w = delta
//   reverse   h = h + u_t[r] v_t[k],           out_t[r] = sum_k h s_t[k],  then h = a_t h
// (the reverse run is the adjoint's recurrence from the last token to the first).  The four
// products of the scan and its gradients are such runs:
//   y   forward, u = x (R = P), v = B, s = C          dx   reverse, u = dy (R = P), v = C, s = B
//   dC  forward, u = B (R = N), v = x, s = dy         dB   reverse, u = C (R = N), v = dy, s = x
template <typename IO>
struct SeqRun {
  Tok<IO> u, v, s;
  int R, K;
  int64_t sr, sk, sh;         // strides of a stored state: rows, columns, heads
  const float* init;          // [S] states, or NULL for zeros
  float* fin;                 // [S] states out, or NULL
  float* carry;               // [rows] states: written by LOCAL runs, else read where a sequence has several segments
  float* decay;               // [rows, H] log2 of a segment's decay, written by LOCAL runs
  int64_t Ls;
  IO* out;                    // [T, H, R], rows out_ts apart, or NULL
  int64_t out_ts;
  float* out32;               // [T, H, R] contiguous in float32, or NULL
  int out_delta;              // multiply the output by delta
  int add_D;                  // add D u
  float* store;               // [rows64] the states at the starts of 64-token blocks, reverse at their ends, or NULL
};

// A workgroup walks its segment in groups of 16 tokens of the packed stream, the next one loaded while this one is
// computed.  Places of a group that are not the segment's hold zeros and delta = 0, which leave the state as it is.
// 16 lanes share a state row, whose readout is then one DPP sum.  Bound by the chain from token to token; 777 ragged
// float32 tokens, 6 heads of 40 x 24: prefill 23 us in three launches, the backward 55 (without the loads ahead and
// with its two runs one after the other 30 and 102).
template <int KV>
struct SeqLds {
  float v[kSeqTok][16 * KV], s[kSeqTok][16 * KV], u[kSeqTok][kSeqRows], o[kSeqTok][kSeqRows + 1];
  float del[kSeqTok], dec[kSeqTok];
};
// STORE: the blocks' states may be wanted (the backward's runs)
template <typename IO, int KV, bool REV, bool LOCAL, bool STORE>
__device__ __forceinline__ void heads_seq(const SeqRun<IO>& q, const HeadPar& hp, int64_t item, SeqLds<KV>& lds) {
  constexpr int KP = 16 * KV;
  auto &sv = lds.v, &ss = lds.s;
  auto& su = lds.u;
  auto& so = lds.o;
  auto &sdel = lds.del, &sdec = lds.dec;
  const int tid = threadIdx.x, lane = tid & 15, row = tid >> 4;
  const int nrb = (q.R + kSeqRows - 1) / kSeqRows;
  const int rb = static_cast<int>(item % nrb);
  const int h = static_cast<int>(item / nrb % hp.H);
  const int64_t rho = item / nrb / hp.H;
  const Segment g = segment_of(hp.cu, hp.S, rho, q.Ls);
  const int r = rb * kSeqRows + row;
  const bool many = g.many(q.Ls);
  if (g.none(rho, q.Ls)) return;
  if (LOCAL && (!many || (REV ? g.first() : g.last()))) return;
  const int64_t soff = h * q.sh + static_cast<int64_t>(r) * q.sr;
  const int64_t sset = static_cast<int64_t>(hp.H) * q.sh;
  const float A2 = head_A2(hp, h);
  const float bias = hp.dt != nullptr ? hp.dt_bias[h] : 0.0f;
  const float Dh = (q.add_D && hp.D != nullptr) ? hp.D[h] : 0.0f;
  float st[KV];
#pragma unroll
  for (int i = 0; i < KV; ++i) st[i] = 0.0f;
  if (!LOCAL) {
    const float* from = many ? q.carry + rho * sset : (q.init ? q.init + g.s * sset : nullptr);
    if (from != nullptr && r < q.R)
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int k = lane * KV + i;
        if (k < q.K) st[i] = from[soff + k * q.sk];
      }
  }
  float dsum = 0.0f;
  const int64_t b0 = g.t0 / kSeqTok, nb = g.t0 < g.t1 ? (g.t1 - 1) / kSeqTok - b0 + 1 : 0;
  uint32_t rv[KV], rs[KV], ru = 0, rdt = 0;  // as loaded
  bool din = false;
  const auto load = [&](int64_t ib) {
    const int64_t tb = (b0 + (REV ? nb - 1 - ib : ib)) * kSeqTok;
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      const int e = tid + i * kSeqThreads, t = e / KP, k = e % KP;
      const bool in = tb + t >= g.t0 && tb + t < g.t1 && k < q.K;
      rv[i] = in ? ld_io_raw(q.v.at(tb + t, h), k) : 0u;
      if (!LOCAL) rs[i] = in ? ld_io_raw(q.s.at(tb + t, h), k) : 0u;
    }
    const int64_t tu = tb + (tid >> 4);
    const int rr = rb * kSeqRows + (tid & 15);
    ru = tu >= g.t0 && tu < g.t1 && rr < q.R ? ld_io_raw(q.u.at(tu, h), rr) : 0u;
    if (tid < kSeqTok) {
      din = tb + tid >= g.t0 && tb + tid < g.t1;
      if (din && hp.dt != nullptr) rdt = ld_io_raw(static_cast<const IO*>(hp.dt) + (tb + tid) * hp.dt_ts, h);
    }
  };
  if (nb > 0) load(0);
  for (int64_t ib = 0; ib < nb; ++ib) {
    const int64_t b = b0 + (REV ? nb - 1 - ib : ib), tb = b * kSeqTok;
    const int lo = g.t0 > tb ? static_cast<int>(g.t0 - tb) : 0;
    const int hi = g.t1 - tb < kSeqTok ? static_cast<int>(g.t1 - tb) : kSeqTok;
    // where the walk enters a 64-token block: from its start, or from its end
    const bool edge = REV ? (b + 1) % (kHeadsBlock / kSeqTok) == 0 || tb + hi == g.seq1
                          : b % (kHeadsBlock / kSeqTok) == 0 || tb + lo == g.seq0;
    const int64_t at64 = (g.s + tb / kHeadsBlock) * sset + soff;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      const int e = tid + i * kSeqThreads, t = e / KP, k = e % KP;
      sv[t][k] = io_value<IO>(rv[i]);
      if (!LOCAL) ss[t][k] = io_value<IO>(rs[i]);
    }
    su[tid >> 4][tid & 15] = io_value<IO>(ru);
    if (tid < kSeqTok) {
      const float d = !din ? 0.0f : hp.dt == nullptr ? 1.0f : head_softplus(io_value<IO>(rdt) + bias);
      sdel[tid] = d;
      sdec[tid] = d * A2;
    }
    __syncthreads();
    if (ib + 1 < nb) load(ib + 1);
    if (STORE && !LOCAL && q.store != nullptr && edge && r < q.R)
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int k = lane * KV + i;
        if (k < q.K) q.store[at64 + k * q.sk] = st[i];
      }
#pragma unroll
    for (int j = 0; j < kSeqTok; ++j) {
      const int t = REV ? kSeqTok - 1 - j : j;
      const float a = exp2_hw(sdec[t]);
      dsum += sdec[t];
      const float uu = su[t][row] * (REV ? 1.0f : sdel[t]);
      float o = 0.0f;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const int k = lane * KV + i;
        st[i] = REV ? __builtin_fmaf(uu, sv[t][k], st[i]) : __builtin_fmaf(a, st[i], uu * sv[t][k]);
        if (!LOCAL) o = __builtin_fmaf(st[i], ss[t][k], o);
        if (REV) st[i] *= a;
      }
      if (!LOCAL) {
        o = row_sum16(o);
        if (lane == 0) so[t][row] = (q.out_delta ? sdel[t] * o : o) + Dh * su[t][row];
      }
    }
    if (!LOCAL && (q.out != nullptr || q.out32 != nullptr)) {
      __syncthreads();
      const int t = tid >> 4, rr = rb * kSeqRows + (tid & 15);
      if (t >= lo && t < hi && rr < q.R) {
        const int64_t at = static_cast<int64_t>(h) * q.R + rr;
        if (q.out != nullptr) st_io(q.out, (tb + t) * q.out_ts + at, so[t][tid & 15]);
        if (q.out32 != nullptr) q.out32[(tb + t) * hp.H * q.R + at] = so[t][tid & 15];
      }
    }
  }
  float* to = LOCAL ? q.carry + rho * sset : ((REV ? g.first() : g.last()) && q.fin ? q.fin + g.s * sset : nullptr);
  if (to != nullptr && r < q.R)
#pragma unroll
    for (int i = 0; i < KV; ++i) {
      const int k = lane * KV + i;
      if (k < q.K) to[soff + k * q.sk] = st[i];
    }
  if (LOCAL && rb == 0 && tid == 0) q.decay[rho * hp.H + h] = dsum;
}
template <typename IO, int KV, bool REV, bool LOCAL>
__global__ __launch_bounds__(kSeqThreads) void k_heads_seq(SeqRun<IO> q, HeadPar hp) {
  __shared__ SeqLds<KV> lds;
  heads_seq<IO, KV, REV, LOCAL, REV>(q, hp, blockIdx.x, lds);
}
// a forward and a reverse run that do not need one another
template <typename IO, int KV, bool LOCAL>
__global__ __launch_bounds__(kSeqThreads) void k_heads_seq_both(SeqRun<IO> fwd, SeqRun<IO> rev, HeadPar hp) {
  __shared__ SeqLds<KV> lds;
  if (blockIdx.y == 0) heads_seq<IO, KV, false, LOCAL, true>(fwd, hp, blockIdx.x, lds);
  else heads_seq<IO, KV, true, LOCAL, false>(rev, hp, blockIdx.x, lds);
}

// The states that the segments of a sequence start from, in place of what they add: one thread per
// state element of a sequence, segment after segment (four loads ahead).  reverse: from the last.
// all == 0: the sequences with several segments, whose last segment added nothing, and fin (if not NULL) only of
// empty sequences; else all sequences, all of whose segments added, and the final states of all.  fin may be init.
// blockIdx.z: the forward states and the adjoints.
// Bound by the carries' traffic, read and written once: 23 rows of 64 heads x 64 x 128 (122 MB) 25 to 30 us.
struct Carry {
  float* carry[2];
  const float *decay[2], *init[2];
  float* fin[2];
  int64_t even;  // not 0: only if a sequence is longer
};
__global__ __launch_bounds__(256) void k_heads_carry(Carry c, const int32_t* __restrict__ cu, int H, int64_t PN,
                                                     int64_t Ls, int all, int S) {
  if (c.even > 0 && !longer_than(cu, S, c.even)) return;
  const int reverse = blockIdx.z;
  float* const carry = c.carry[reverse];
  const float *const decay = c.decay[reverse], *const init = c.init[reverse];
  float* const fin = c.fin[reverse];
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t set = H * PN;
  if (e >= set) return;
  for (int s = blockIdx.y; s < S; s += gridDim.y) {
  const uint32_t L = static_cast<uint32_t>(Ls), seq0 = cu[s], seq1 = cu[s + 1];
  const int n = seq1 > seq0 ? static_cast<int>((seq1 - 1) / L - seq0 / L) + 1 : 0;
  if (!all && n == 0 && fin != nullptr) fin[s * set + e] = init != nullptr ? init[s * set + e] : 0.0f;
  if (!all && n < 2) continue;
  const int h = static_cast<int>(e / PN);
  const int64_t r0 = s + static_cast<int64_t>(seq0 / L), step = reverse ? -1 : 1;
  int64_t rho = reverse ? r0 + n - 1 : r0;
  float cur = init != nullptr ? init[s * set + e] : 0.0f;
  const int added = all ? n : n - 1;  // segments whose shares are there
  for (int i = 0; i < n; i += 4) {
    float local[4], a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      local[k] = a[k] = 0.0f;
      if (i + k < added) {
        local[k] = carry[(rho + k * step) * set + e];
        a[k] = decay[(rho + k * step) * H + h];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) {
        carry[rho * set + e] = cur;
        rho += step;
        cur = __builtin_fmaf(exp2_hw(a[k]), cur, local[k]);
      }
  }
  if (all) fin[s * set + e] = cur;
  }
}

// ------------------------------------------------------------------------------------ decode
// One token for each row of a batch: state rows p over 16-lane rows as in the sequential kernel.
template <typename IO, int KV>
__global__ __launch_bounds__(kSeqThreads) void k_heads_decode_any(Tok<IO> x, Tok<IO> B, Tok<IO> C, HeadPar hp,
                                                                  const float* state_in, float* state_out,
                                                                  IO* __restrict__ y, int P, int N) {
  const int tid = threadIdx.x, lane = tid & 15, row = tid >> 4;
  const int nrb = (P + kSeqRows - 1) / kSeqRows;
  const int rb = blockIdx.x % nrb;
  const int h = (blockIdx.x / nrb) % hp.H;
  const int64_t b = blockIdx.x / nrb / hp.H;
  const int p = rb * kSeqRows + row;
  if (p >= P) return;
  const float delta = head_delta<IO>(hp, b, h);
  const float a = exp2_hw(delta * head_A2(hp, h));
  const float xv = ld_io(x.at(b, h), p);
  const float dx = delta * xv;
  const int64_t off = ((b * hp.H + h) * P + p) * static_cast<int64_t>(N);
  const IO *Bp = B.at(b, h), *Cp = C.at(b, h);
  float o = 0.0f;
#pragma unroll
  for (int i = 0; i < KV; ++i) {
    const int n = i * 16 + lane;
    if (n < N) {
      const float v = __builtin_fmaf(a, state_in ? state_in[off + n] : 0.0f, dx * ld_io(Bp, n));
      state_out[off + n] = v;
      o = __builtin_fmaf(v, ld_io(Cp, n), o);
    }
  }
  o = row_sum16(o);
  if (lane == 0) st_io(y, (b * hp.H + h) * P + p, o + (hp.D ? hp.D[h] * xv : 0.0f));
}

// The same for N a multiple of 4 with every row on 16 bytes: RL lanes take a state row, 4 entries each, and a
// thread two rows, so that a workgroup's accesses are contiguous.  Bound by the states' traffic, 8 P N bytes a
// head, which passes the caches by (nontemporal).  256 rows, d 8192, state 64 x 128 (2.15 GB): 351 us, 6.2 TB/s
// (traced mean; a plain copy reaches 6.2); when it was 363, one row per thread took 481, four 364, eight 611 (204
// registers), plain accesses 392.
constexpr int kDecodeRows = 2;
template <typename IO, int RL>
__global__ __launch_bounds__(kSeqThreads) void k_heads_decode(Tok<IO> x, Tok<IO> B, Tok<IO> C, HeadPar hp,
                                                              const float* state_in, float* state_out,
                                                              IO* __restrict__ y, int P, int N, int blocks) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  constexpr int RG = kSeqThreads / RL;  // row groups
  constexpr int U = kDecodeRows;
  const int lane = threadIdx.x % RL, rg = threadIdx.x / RL;
  const int blk = blockIdx.x % blocks;
  const int h = (blockIdx.x / blocks) % hp.H;
  const int64_t b = blockIdx.x / blocks / hp.H;
  const int p0 = blk * RG * U + rg, n = 4 * lane;
  const bool in = n < N;
  const int64_t off = ((b * hp.H + h) * P + p0) * static_cast<int64_t>(N) + n;
  f4 s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = f4{0, 0, 0, 0};
    if (state_in != nullptr && in && p0 + RG * u < P) s[u] = nt_load(reinterpret_cast<const f4*>(state_in + off + RG * u * N));
  }
  const IO *Bp = B.at(b, h), *Cp = C.at(b, h), *xp = x.at(b, h);
  f4 bv = {0, 0, 0, 0}, cv = {0, 0, 0, 0};
  if (in)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bv[i] = ld_io(Bp, n + i);
      cv[i] = ld_io(Cp, n + i);
    }
  float xv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) xv[u] = p0 + RG * u < P ? ld_io(xp, p0 + RG * u) : 0.0f;
  const float delta = head_delta<IO>(hp, b, h);
  const float a = exp2_hw(delta * head_A2(hp, h));
  const float Dh = hp.D != nullptr ? hp.D[h] : 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float dx = delta * xv[u];
    float o = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[u][i] = __builtin_fmaf(a, s[u][i], dx * bv[i]);
      o = __builtin_fmaf(s[u][i], cv[i], o);
    }
    if (in && p0 + RG * u < P) nt_store(s[u], reinterpret_cast<f4*>(state_out + off + RG * u * N));
    // the row's sum
    if (RL >= 2) o += __builtin_amdgcn_update_dpp(0.0f, o, 0xB1, 0xF, 0xF, true);   // quad_perm 1,0,3,2
    if (RL >= 4) o += __builtin_amdgcn_update_dpp(0.0f, o, 0x4E, 0xF, 0xF, true);   // quad_perm 2,3,0,1
    if (RL >= 8) o += __builtin_amdgcn_update_dpp(0.0f, o, 0x141, 0xF, 0xF, true);  // row_half_mirror
    if (RL >= 16) o += __builtin_amdgcn_update_dpp(0.0f, o, 0x140, 0xF, 0xF, true); // row_mirror
    if (RL >= 32) o += __shfl_xor(o, 16);
    if (RL >= 64) o += __shfl_xor(o, 32);
    o = __builtin_fmaf(Dh, xv[u], o);
    if (lane == 0 && p0 + RG * u < P) st_io(y, (b * hp.H + h) * P + p0 + RG * u, o);
  }
}

// ------------------------------------------------------------------------------------ backward
// dB and dC of a group: the sums of its heads' shares (dB's times delta)
template <typename IO>
__global__ __launch_bounds__(256) void k_heads_group(const float* __restrict__ dBh, const float* __restrict__ dCh,
                                                     const float* __restrict__ delta, IO* __restrict__ dB,
                                                     IO* __restrict__ dC, int64_t db_ts, int64_t dc_ts, int64_t T, int H,
                                                     int G, int N) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= T * G * N) return;
  const int n = static_cast<int>(i % N);
  const int g = static_cast<int>(i / N % G);
  const int64_t t = i / N / G;
  const int hg = H / G;
  float b = 0.0f, c = 0.0f;
  for (int h = g * hg; h < (g + 1) * hg; ++h) {
    const int64_t o = (t * H + h) * N + n;
    b = __builtin_fmaf(delta[t * H + h], dBh[o], b);
    c += dCh[o];
  }
  st_io(dB, t * db_ts + static_cast<int64_t>(g) * N + n, b);
  st_io(dC, t * dc_ts + static_cast<int64_t>(g) * N + n, c);
}

// dA_log, ddt_bias and dD: the sums of the blocks' parts, one workgroup per head, in a fixed order
__global__ __launch_bounds__(256) void k_heads_params(const float* __restrict__ sums, int64_t rows, int H,
                                                      float* __restrict__ dA_log, float* __restrict__ ddt_bias,
                                                      float* __restrict__ dD) {
  __shared__ float s[3][256];
  const int h = blockIdx.x, tid = threadIdx.x;
  float v[3] = {0.0f, 0.0f, 0.0f};
  for (int64_t i = tid; i < rows; i += 256)
    for (int k = 0; k < 3; ++k) v[k] += sums[(i * H + h) * 3 + k];
  for (int k = 0; k < 3; ++k) s[k][tid] = v[k];
  for (int w = 128; w > 0; w /= 2) {
    __syncthreads();
    if (tid < w)
      for (int k = 0; k < 3; ++k) s[k][tid] += s[k][tid + w];
  }
  if (tid == 0) {
    dA_log[h] = s[0][0];
    if (ddt_bias != nullptr) ddt_bias[h] = s[1][0];
    if (dD != nullptr) dD[h] = s[2][0];
  }
}

}  // namespace mm
