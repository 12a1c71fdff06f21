// The head scan and the norms around a mixer block: argument checks, plans and launches of the
// entry points declared in include/mambamix.h.  The kernels are in mm_heads.h
// (token by token, decode), mm_heads_mma.h, mm_heads_grad.h (matrix cores) and mm_norm.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include <stdint.h>


#include "mambamix.h"
#include "mm_device.h"
#include "mm_heads.h"
#include "mm_heads_grad.h"
#include "mm_heads_mma.h"
#include "mm_host.h"
#include "mm_norm.h"

namespace mm {
namespace {

constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;  // of one launch
constexpr int64_t kCUs = 256;

int launched() { return hipGetLastError() == hipSuccess ? MM_OK : MM_ERR_HIP; }

// ---------------------------------------------------------------- the head scan: plans

struct HeadsPlan {
  int64_t Ls;      // tokens per segment
  bool mma;        // the matrix-core kernels
  bool whole;      // every sequence is one segment
  int64_t rows;    // segments at most
  int64_t walks;   // matrix-core kernels: sequences, or stretches of Ls tokens
  int64_t even;    // not 0: both ways are launched, and the whole sequences run if none is longer than this
  int64_t rows64;  // 64-token blocks at most (backward)
  int nrp, nrn;    // 16-row blocks of P and N
  size_t off_carry, off_decay, off_carry2, off_decay2, off_hb, off_gs, off_dB, off_dC, off_delta, off_sums, total;
  int npb, nk, splits;  // matrix-core backward: 64-channel blocks per head, 32-column steps of N, shares of a group's heads
};

// A workgroup of the sequential kernels walks one segment token by token, so few long sequences are cut until some four
// workgroups are on every CU, down to 64 tokens (777 tokens in 8 sequences, 6 heads: segments of 256 tokens took 87 us
// where those of 64 took 30).
constexpr int64_t kSeqWorkgroups = 1024;

// The matrix-core kernels take bfloat16 io and N <= 128.  Their workgroups take two 64-channel blocks of
// a group; two workgroups fit on a CU.
constexpr int kMmaMaxN = 128;
constexpr int64_t kMmaWorkgroups = 512;
// Prefill: up to so many sequences the device chooses between whole sequences and stretches, by the longest one.  Beyond,
// whole sequences run unasked: with 24 heads 1000 sequences of 16 tokens take 360 us (494 when both ways are launched),
// 300 of 90 180 (201), with 64 heads in 8 groups 913 (1294) and 418 (459).  One long sequence among many pays for it where
// the heads are few: 299 of 50 tokens and one of 12000, 24 heads 1075 us, in stretches 678; 64 heads 1247 and 1532.
constexpr int64_t kMmaMaxEven = 256;

int plan_heads(HeadsPlan& p, int64_t S, int64_t T, int H, int P, int G, int N, int io, bool backward, int64_t max_stride) {
  p = HeadsPlan{};
  p.mma = io == MM_IO_BF16 && N <= kMmaMaxN && max_stride <= kMmaMaxStride &&
          static_cast<int64_t>(H) * P <= kMmaMaxStride;
  p.nrp = static_cast<int>(cdiv(P, kSeqRows));
  p.nrn = static_cast<int>(cdiv(N, kSeqRows));
  const int64_t per = static_cast<int64_t>(H) * (backward ? std::min(p.nrp, p.nrn) : p.nrp);
  const int64_t want = cdiv(kSeqWorkgroups, std::max<int64_t>(per, 1));
  p.Ls = std::max<int64_t>(kHeadsBlock, cdiv(cdiv(T, std::max<int64_t>(want, 1)), kHeadsBlock) * kHeadsBlock);
  if (want <= S || p.Ls >= T) p.Ls = (T / kHeadsBlock + 1) * kHeadsBlock;
  if (p.mma) {
    // Prefill: whole sequences where they alone give the GPU its workgroups and none is longer than two stretches, which
    // the kernels of both ways find out (16 x 1024 tokens, 64 heads in 8 groups: whole 158 us, cut 254; 24 x 100 54 and
    // 167; but one long sequence among short ones would be one long chain).  The backward, whose two walks store every
    // block's state, takes them with one workgroup per CU, whatever their lengths: its stretches walk everything twice.
    // 8 x 2044 tokens, 24 heads, whole 474 us, cut 608; seven of 425 to 4011 tokens, 24 heads 536 and 596, 64 heads 1307
    // and 1484; 2 x 8192, 64 heads, 963 and 1075.  One long sequence alone among short ones loses: 16000 and 384 tokens, 64
    // heads, 1237 and 1178; 16000 and seven of 50, 24 heads, 898 and 659.  Else
    // stretches of equal length, as many as the GPU runs workgroups at once (two walks per CU, of two 64-channel
    // blocks, or four state walks of one), so that all end together.  Short calls have fewer: a walk's time grows with
    // its length L, the carries' with the T / L states of every pair of blocks, and sqrt(T pairs / 2) is near the least sum
    // (64 heads in 8 groups, N 128: 1024 tokens 67 us in stretches of 512, 47 of 256, 44 of 128; 2048 tokens 69, 60,
    // 67; 4096 84, 87, 87).  The backward, with three times the carries, gains nothing below 512 (512 tokens 72 us,
    // cut to 256 87; 4096 tokens 337 and 373).
    const int64_t pairs = H > 0 ? G * cdiv(H / G * cdiv(P, 64), 2) : 1;
    const int64_t walks = std::max<int64_t>(1, 2 * kCUs / pairs);
    const bool enough = backward ? S * H * cdiv(P, 64) * 2 >= kCUs : S * pairs >= kMmaWorkgroups;
    const bool whole = enough && (backward || S > kMmaMaxEven);
    const int64_t least = backward ? 512 : static_cast<int64_t>(std::sqrt(0.5 * T * pairs));
    p.Ls = std::max<int64_t>(1, cdiv(std::max(least, cdiv(T, walks)), kMmaTok)) * kMmaTok;
    if (whole || p.Ls >= T) p.Ls = (T / kMmaTok + 1) * kMmaTok;
    else if (enough && !backward) p.even = 2 * p.Ls;
  }
  p.whole = p.Ls > T;
  p.npb = static_cast<int>(cdiv(P, 64));
  p.nk = N <= 32 ? 1 : N <= 64 ? 2 : 4;
  // Two workgroups of the gradient kernel per CU, or one for each head.  (The count is that of full blocks; a few more
  // than fit at once make a round of their own: 8 x 2048 tokens, 24 heads, 384 us, 8 x 2044 about 480.)
  p.splits = H > 0 ? static_cast<int>(std::max<int64_t>(
                 1, std::min<int64_t>(H / G, cdiv(2 * kCUs, std::max<int64_t>(segment_rows(S, T, kHeadsBlock) * G, 1))))) : 1;
  p.rows = segment_rows(S, T, p.Ls);
  p.walks = p.whole ? S : cdiv(T, p.Ls);
  p.rows64 = segment_rows(S, T, kHeadsBlock);
  const size_t set = static_cast<size_t>(H) * P * N * 4;
  const size_t th = static_cast<size_t>(T) * H;
  size_t off = 0;
  const auto take = [&off](size_t& at, size_t n) { at = off; off += align256(n); };
  if (!p.whole) {
    take(p.off_carry, p.rows * set);
    take(p.off_decay, static_cast<size_t>(p.rows) * H * 4);
  }
  if (backward) {
    if (!p.whole) {
      take(p.off_carry2, p.rows * set);
      take(p.off_decay2, static_cast<size_t>(p.rows) * H * 4);
    }
  }
  if (backward && p.mma) {
    const size_t blocks = static_cast<size_t>(p.rows64) * H * p.npb * 64 * (32 * p.nk) * 4;
    const size_t part = static_cast<size_t>(p.splits) * T * G * N * 4;
    take(p.off_hb, blocks);
    take(p.off_gs, blocks);
    take(p.off_dB, part);
    take(p.off_dC, part);
    take(p.off_sums, static_cast<size_t>(p.rows64) * H * 3 * 4);
  } else if (backward) {
    take(p.off_hb, p.rows64 * set);
    take(p.off_gs, p.rows64 * set);
    take(p.off_dB, th * N * 4);
    take(p.off_dC, th * N * 4);
    take(p.off_delta, th * 4);
    take(p.off_sums, static_cast<size_t>(p.rows64) * H * 3 * 4);
  }
  p.total = off;
  // the threads of each launch of the path taken (whole sequences run beside stretches: S of them)
  const int64_t tgn = T * G * N, seq = p.rows * H * (backward ? std::max(p.nrp, p.nrn) : p.nrp) * kSeqThreads;
  int64_t most = static_cast<int64_t>(H) * std::max(P * N, kSeqThreads);
  if (p.mma) {
    most = std::max(most, std::max(p.walks, S) * H * p.npb * kMmaThreads);
    if (backward) most = std::max({most, p.rows64 * G * p.splits * kMmaThreads, tgn});
  } else {
    most = std::max(most, seq);
    if (backward) most = std::max({most, p.rows64 * H * kMmaThreads, tgn});
  }
  return most > kMaxThreads ? MM_ERR_DIM : MM_OK;
}

int check_heads_sizes(int64_t S, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N, int32_t io) {
  if (S < 0 || T < 0 || H < 0 || P < 0 || G < 0 || N < 0 || T > INT32_MAX || S > INT32_MAX) return MM_ERR_DIM;
  if (io != MM_IO_F32 && io != MM_IO_BF16) return MM_ERR_UNSUPPORTED;
  if (P < 1 || P > MM_HEADS_MAX_P || N < 1 || N > MM_HEADS_MAX_N) return MM_ERR_UNSUPPORTED;
  if (S == 0 && T > 0) return MM_ERR_DIM;
  if (H > 0 && (G < 1 || H % G != 0)) return MM_ERR_DIM;
  const uint64_t d = static_cast<uint64_t>(H) * P;
  if (d > 0 && (static_cast<uint64_t>(T) > MM_MAX_ROWS_X_D / d || static_cast<uint64_t>(S) > MM_MAX_ROWS_X_D / d))
    return MM_ERR_DIM;
  return MM_OK;
}

template <typename IO>
Tok<IO> tok(const void* p, int64_t ts, int W, int div) {
  return Tok<IO>{static_cast<const IO*>(p), ts, W, div};
}

template <typename IO, bool REV, bool LOCAL>
void launch_seq(const SeqRun<IO>& q, const HeadPar& hp, int64_t rows, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(rows * hp.H * cdiv(q.R, kSeqRows))), block(kSeqThreads);
  if (grid.x == 0) return;
  if (q.K <= 16) hipLaunchKernelGGL((k_heads_seq<IO, 1, REV, LOCAL>), grid, block, 0, st, q, hp);
  else if (q.K <= 32) hipLaunchKernelGGL((k_heads_seq<IO, 2, REV, LOCAL>), grid, block, 0, st, q, hp);
  else if (q.K <= 64) hipLaunchKernelGGL((k_heads_seq<IO, 4, REV, LOCAL>), grid, block, 0, st, q, hp);
  else if (q.K <= 128) hipLaunchKernelGGL((k_heads_seq<IO, 8, REV, LOCAL>), grid, block, 0, st, q, hp);
  else hipLaunchKernelGGL((k_heads_seq<IO, 16, REV, LOCAL>), grid, block, 0, st, q, hp);
}

// a forward and a reverse run of the same sizes in one launch
template <typename IO, bool LOCAL>
void launch_seq_both(const SeqRun<IO>& f, const SeqRun<IO>& r, const HeadPar& hp, int64_t rows, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(rows * hp.H * cdiv(f.R, kSeqRows)), 2), block(kSeqThreads);
  if (grid.x == 0) return;
  if (f.K <= 16) hipLaunchKernelGGL((k_heads_seq_both<IO, 1, LOCAL>), grid, block, 0, st, f, r, hp);
  else if (f.K <= 32) hipLaunchKernelGGL((k_heads_seq_both<IO, 2, LOCAL>), grid, block, 0, st, f, r, hp);
  else if (f.K <= 64) hipLaunchKernelGGL((k_heads_seq_both<IO, 4, LOCAL>), grid, block, 0, st, f, r, hp);
  else if (f.K <= 128) hipLaunchKernelGGL((k_heads_seq_both<IO, 8, LOCAL>), grid, block, 0, st, f, r, hp);
  else hipLaunchKernelGGL((k_heads_seq_both<IO, 16, LOCAL>), grid, block, 0, st, f, r, hp);
}

// dirs: 1, the forward states, or 2, the adjoints too
void launch_carry(const Carry& c, const HeadPar& hp, int64_t PN, int64_t Ls, int dirs, bool all, hipStream_t st) {
  hipLaunchKernelGGL(k_heads_carry, dim3(static_cast<unsigned>(cdiv(hp.H * PN, 256)),
                                         static_cast<unsigned>(std::min(hp.S, 8)), static_cast<unsigned>(dirs)),
                     dim3(256), 0, st, c, hp.cu, hp.H, PN, Ls, all ? 1 : 0, hp.S);
}

struct HeadsArgs {
  const void *x, *B, *C;
  int64_t x_ts, b_ts, c_ts;
  int P, G, N;
  HeadPar hp;
};

// 16-byte pieces of rows and states: every row starts on one.  Where one does not, all tiles are loaded element by
// element: the prefill of 16384 packed tokens of 10 heads takes 187 us with rows of 1546 columns, 81 with 1552.
bool heads_vec(const HeadsArgs& a, std::initializer_list<const void*> more) {
  if (a.P % 8 != 0 || a.N % 8 != 0 || a.x_ts % 8 != 0 || a.b_ts % 8 != 0 || a.c_ts % 8 != 0) return false;
  for (const void* p : {a.x, a.B, a.C})
    if (!aligned(p, 16)) return false;
  for (const void* p : more)
    if (!aligned(p, 16)) return false;
  return true;
}

template <typename K>
int allow_lds(K kernel, size_t bytes) {
  if (bytes > 64 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bytes)) != hipSuccess)
    return MM_ERR_HIP;
  return MM_OK;
}

template <typename F>
int by_steps(int nk, bool vec, F f) {
  const auto go = [&](auto k) { return vec ? f(k, std::true_type{}) : f(k, std::false_type{}); };
  if (nk == 1) return go(std::integral_constant<int, 1>{});
  if (nk == 2) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 4>{});
}

template <bool LOCAL>
int launch_states(StateArgs q, const HeadPar& hp, int64_t rows, int nk, int dirs, bool vec, hipStream_t st) {
  // Two slices of the columns where the walks alone are at most two per CU: a block's chain is then shorter and more
  // chains overlap, but x is read and weighted twice.  Backward of 512 tokens of 64 heads 72 us whole, 64 in slices, of
  // four sequences of 5100 474 and 449; with four walks per CU (4096 tokens) 327 and 330, with eight 613 and 629.
  q.slices = nk == 4 && rows * hp.H * q.npb * dirs <= 2 * kCUs ? 2 : 1;
  return by_steps(nk / q.slices, vec, [&](auto k, auto v) -> int {
    constexpr int NK = decltype(k)::value;
    constexpr bool VEC = decltype(v)::value;
    const dim3 grid(static_cast<unsigned>(rows * hp.H * q.npb * q.slices), static_cast<unsigned>(dirs));
    if (grid.x > 0)
      hipLaunchKernelGGL((k_heads_states<NK, VEC, LOCAL>), grid, dim3(kMmaThreads), StateGeo<NK>::bytes, st, q, hp);
    return MM_OK;
  });
}

template <int PARTS>
int launch_mma(const MmaArgs& q, const HeadPar& hp, int64_t rows, int nk, bool vec, hipStream_t st) {
  return by_steps(nk, vec, [&](auto k, auto v) -> int {
    constexpr int NK = decltype(k)::value;
    constexpr bool VEC = decltype(v)::value;
    const int rc = allow_lds(&k_heads_mma<NK, PARTS, VEC>, MmaGeo<NK>::bytes);
    if (rc != MM_OK) return rc;
    const dim3 grid(static_cast<unsigned>(rows * q.pairs));
    if (grid.x > 0)
      hipLaunchKernelGGL((k_heads_mma<NK, PARTS, VEC>), grid, dim3(kMmaThreads), MmaGeo<NK>::bytes, st, q, hp);
    return MM_OK;
  });
}

int launch_prefill_mma(const HeadsPlan& p, const HeadsArgs& a, const float* state_in, float* state_out, void* y,
                       char* ws, hipStream_t st) {
  const int div = a.hp.H / a.G;
  MmaArgs q{};
  q.x = tok<uint16_t>(a.x, a.x_ts, a.P, 1);
  q.B = tok<uint16_t>(a.B, a.b_ts, a.N, div);
  q.C = tok<uint16_t>(a.C, a.c_ts, a.N, div);
  q.P = a.P;
  q.N = a.N;
  q.npb = static_cast<int>(cdiv(a.P, 64));
  q.vper = div * q.npb;
  q.ppg = static_cast<int>(cdiv(q.vper, 2));
  q.pairs = q.ppg * a.G;
  q.Ls = p.Ls;
  q.state_in = state_in;
  q.state_out = state_out;
  q.y = static_cast<uint16_t*>(y);
  const bool vec = heads_vec(a, {state_in, state_out, y});
  if (p.whole) {
    const int rc = launch_mma<3>(q, a.hp, p.walks, p.nk, vec, st);
    return rc != MM_OK ? rc : launched();
  }
  q.even = p.even;
  if (p.even > 0) {
    MmaArgs w = q;
    w.Ls = a.hp.T + 1;
    const int rc = launch_mma<3>(w, a.hp, a.hp.S, p.nk, vec, st);
    if (rc != MM_OK) return rc;
  }
  StateArgs s{};
  s.even = p.even;
  s.u[0] = q.x;
  s.v[0] = q.B;
  s.P = q.P;
  s.N = q.N;
  s.G = a.G;
  s.npb = q.npb;
  s.Ls = q.Ls;
  s.carry[0] = reinterpret_cast<float*>(ws + p.off_carry);
  s.decay[0] = reinterpret_cast<float*>(ws + p.off_decay);
  s.all = 1;
  q.carry = s.carry[0];
  int rc = launch_states<true>(s, a.hp, p.walks, p.nk, 1, vec, st);
  if (rc != MM_OK) return rc;
  launch_carry({{s.carry[0]}, {s.decay[0]}, {state_in}, {state_out}, p.even}, a.hp, static_cast<int64_t>(a.P) * a.N, p.Ls, 1, true, st);
  rc = launch_mma<1>(q, a.hp, p.walks, p.nk, vec, st);
  return rc != MM_OK ? rc : launched();
}

template <typename IO>
int launch_prefill(const HeadsPlan& p, const HeadsArgs& a, const float* state_in, float* state_out, void* y, char* ws,
                   hipStream_t st) {
  const int div = a.hp.H / a.G;
  SeqRun<IO> q{};
  q.u = tok<IO>(a.x, a.x_ts, a.P, 1);
  q.v = tok<IO>(a.B, a.b_ts, a.N, div);
  q.s = tok<IO>(a.C, a.c_ts, a.N, div);
  q.R = a.P;
  q.K = a.N;
  q.sr = a.N;
  q.sk = 1;
  q.sh = static_cast<int64_t>(a.P) * a.N;
  q.init = state_in;
  q.fin = state_out;
  q.Ls = p.Ls;
  q.out = static_cast<IO*>(y);
  q.out_ts = static_cast<int64_t>(a.hp.H) * a.P;
  q.add_D = 1;
  if (!p.whole) {
    q.carry = reinterpret_cast<float*>(ws + p.off_carry);
    q.decay = reinterpret_cast<float*>(ws + p.off_decay);
    launch_seq<IO, false, true>(q, a.hp, p.rows, st);
    launch_carry({{q.carry}, {q.decay}, {state_in}, {nullptr}}, a.hp, q.sh, p.Ls, 1, false, st);
  }
  launch_seq<IO, false, false>(q, a.hp, p.rows, st);
  return launched();
}

struct HeadsGrads {
  const void* dy;
  const float *state_in, *dstate_out;
  void *dx, *ddt, *dB, *dC;
  int64_t dx_ts, ddt_ts, db_ts, dc_ts;
  float *dA_log, *dD, *ddt_bias, *dstate_in;
};

int launch_backward_mma(const HeadsPlan& p, const HeadsArgs& a, const HeadsGrads& o, char* ws, hipStream_t st) {
  const int H = a.hp.H, div = H / a.G;
  const int64_t T = a.hp.T, PN = static_cast<int64_t>(a.P) * a.N;
  const Tok<uint16_t> x = tok<uint16_t>(a.x, a.x_ts, a.P, 1);
  const Tok<uint16_t> dy = tok<uint16_t>(o.dy, static_cast<int64_t>(H) * a.P, a.P, 1);
  const Tok<uint16_t> B = tok<uint16_t>(a.B, a.b_ts, a.N, div), C = tok<uint16_t>(a.C, a.c_ts, a.N, div);
  const bool vec = heads_vec(a, {o.dy, o.dx}) && o.dx_ts % 8 == 0;
  const auto at = [ws](size_t off) { return reinterpret_cast<float*>(ws + off); };
  StateArgs s{};
  s.u[0] = x;
  s.v[0] = B;
  s.u[1] = dy;
  s.v[1] = C;
  s.P = a.P;
  s.N = a.N;
  s.G = a.G;
  s.npb = p.npb;
  s.Ls = p.Ls;
  s.whole = p.whole ? 1 : 0;
  s.init[0] = o.state_in;
  s.init[1] = o.dstate_out;
  if (!p.whole) {
    s.carry[0] = at(p.off_carry);
    s.decay[0] = at(p.off_decay);
    s.carry[1] = at(p.off_carry2);
    s.decay[1] = at(p.off_decay2);
    const int rc = launch_states<true>(s, a.hp, p.walks, p.nk, 2, vec, st);
    if (rc != MM_OK) return rc;
    launch_carry({{s.carry[0], s.carry[1]}, {s.decay[0], s.decay[1]}, {s.init[0], s.init[1]}, {nullptr, o.dstate_in}}, a.hp,
                 PN, p.Ls, 2, false, st);
  }
  s.store[0] = at(p.off_hb);
  s.store[1] = at(p.off_gs);
  s.fin[1] = o.dstate_in;
  int rc = launch_states<false>(s, a.hp, p.walks, p.nk, 2, vec, st);
  if (rc != MM_OK) return rc;
  if (T > 0) {
    const GradArgs g{x, dy, B, C, a.P, a.N, p.npb, a.G, p.splits, s.store[0], s.store[1], static_cast<uint16_t*>(o.dx),
                     o.dx_ts, at(p.off_dB), at(p.off_dC), static_cast<uint16_t*>(o.ddt), o.ddt_ts, at(p.off_sums)};
    rc = by_steps(p.nk, vec, [&](auto k, auto v) -> int {
      constexpr int NK = decltype(k)::value;
      constexpr bool VEC = decltype(v)::value;
      const int r = allow_lds(&k_heads_grads<NK, VEC>, GradGeo<NK>::bytes);
      if (r != MM_OK) return r;
      hipLaunchKernelGGL((k_heads_grads<NK, VEC>), dim3(static_cast<unsigned>(p.rows64 * a.G * p.splits)), dim3(kMmaThreads),
                         GradGeo<NK>::bytes, st, g, a.hp);
      return MM_OK;
    });
    if (rc != MM_OK) return rc;
    hipLaunchKernelGGL(k_heads_shares, dim3(static_cast<unsigned>(cdiv(T * a.G * a.N, 256))), dim3(256), 0, st, g.pB, g.pC,
                       static_cast<uint16_t*>(o.dB), static_cast<uint16_t*>(o.dC), o.db_ts, o.dc_ts, T, a.G * a.N, p.splits);
  }
  hipLaunchKernelGGL(k_heads_params, dim3(static_cast<unsigned>(H)), dim3(256), 0, st, at(p.off_sums), T > 0 ? p.rows64 : 0, H,
                     o.dA_log, o.ddt_bias, o.dD);
  return launched();
}

template <typename IO>
int launch_backward(const HeadsPlan& p, const HeadsArgs& a, const HeadsGrads& o, char* ws, hipStream_t st) {
  const int H = a.hp.H, div = H / a.G;
  const int64_t T = a.hp.T, set = static_cast<int64_t>(a.P) * a.N;
  const Tok<IO> x = tok<IO>(a.x, a.x_ts, a.P, 1), dy = tok<IO>(o.dy, static_cast<int64_t>(H) * a.P, a.P, 1);
  const Tok<IO> B = tok<IO>(a.B, a.b_ts, a.N, div), C = tok<IO>(a.C, a.c_ts, a.N, div);
  const auto at = [ws](size_t off) { return reinterpret_cast<float*>(ws + off); };
  // dC and the states at the blocks' starts: forward, the state transposed (rows N)
  SeqRun<IO> c{};
  c.u = B;
  c.v = x;
  c.s = dy;
  c.R = a.N;
  c.K = a.P;
  c.sr = 1;
  c.sk = a.N;
  c.sh = set;
  c.init = o.state_in;
  c.Ls = p.Ls;
  c.out32 = at(p.off_dC);
  c.store = at(p.off_hb);
  // dB: reverse, the state transposed
  SeqRun<IO> b = c;
  b.u = C;
  b.v = dy;
  b.s = x;
  b.init = o.dstate_out;
  b.out32 = at(p.off_dB);
  b.store = nullptr;
  // dx, dstate_in and the adjoints at the blocks' ends: reverse (rows P)
  SeqRun<IO> d = b;
  d.u = dy;
  d.v = C;
  d.s = B;
  d.R = a.P;
  d.K = a.N;
  d.sr = a.N;
  d.sk = 1;
  d.fin = o.dstate_in;
  d.out32 = nullptr;
  d.out = static_cast<IO*>(o.dx);
  d.out_ts = o.dx_ts;
  d.out_delta = 1;
  d.add_D = 1;
  d.store = at(p.off_gs);
  if (!p.whole) {
    c.carry = reinterpret_cast<float*>(ws + p.off_carry);
    c.decay = reinterpret_cast<float*>(ws + p.off_decay);
    b.carry = d.carry = reinterpret_cast<float*>(ws + p.off_carry2);
    b.decay = d.decay = reinterpret_cast<float*>(ws + p.off_decay2);
    SeqRun<IO> f = d;  // the forward states' shares with the state as it is stored (rows P), as the adjoints'
    f.u = x;
    f.v = B;
    f.carry = c.carry;
    f.decay = c.decay;
    launch_seq_both<IO, true>(f, d, a.hp, p.rows, st);
    launch_carry({{c.carry, d.carry}, {c.decay, d.decay}, {o.state_in, o.dstate_out}, {nullptr, nullptr}}, a.hp, set, p.Ls, 2,
                 false, st);
  }
  if (T > 0) launch_seq_both<IO, false>(c, b, a.hp, p.rows, st);
  launch_seq<IO, true, false>(d, a.hp, p.rows, st);
  if (T > 0) {
    const auto steps = [&](auto wide) {
      hipLaunchKernelGGL((k_heads_ddt<IO, decltype(wide)::value>), dim3(static_cast<unsigned>(p.rows64 * H)), dim3(kMmaThreads), 0,
                         st, x, dy, B, C, a.hp, at(p.off_hb), at(p.off_gs), a.P, a.N, at(p.off_delta), static_cast<IO*>(o.ddt),
                         o.ddt_ts, at(p.off_sums));
    };
    if (a.P >= 4 && a.N >= 4) steps(std::true_type{}); else steps(std::false_type{});
    hipLaunchKernelGGL((k_heads_group<IO>), dim3(static_cast<unsigned>(cdiv(T * a.G * a.N, 256))), dim3(256), 0, st,
                       at(p.off_dB), at(p.off_dC), at(p.off_delta), static_cast<IO*>(o.dB), static_cast<IO*>(o.dC), o.db_ts,
                       o.dc_ts, T, H, a.G, a.N);
  }
  hipLaunchKernelGGL(k_heads_params, dim3(static_cast<unsigned>(H)), dim3(256), 0, st, at(p.off_sums), T > 0 ? p.rows64 : 0, H,
                     o.dA_log, o.ddt_bias, o.dD);
  return launched();
}

// ---------------------------------------------------------------- the head scan: checks

Rows rows(const void* p, int64_t n, int64_t width, int64_t stride, size_t es) {
  return Rows{p, n, static_cast<size_t>(width) * es, static_cast<size_t>(stride) * es};
}
Rows flat(const void* p, size_t bytes) { return Rows{p, 1, bytes, bytes}; }

// arrays of zero bytes may be NULL; `es`: the element size they are aligned to
struct Array {
  Rows r;
  size_t es;
  bool optional;  // NULL allowed
};
int check_arrays(const Array* a, int n) {
  for (int i = 0; i < n; ++i)
    if (a[i].r.p == nullptr && !a[i].optional && a[i].r.extent() > 0) return MM_ERR_NULL;
  for (int i = 0; i < n; ++i)
    if (!aligned(a[i].r.p, a[i].es)) return MM_ERR_ALIGN;
  return MM_OK;
}
// an output that may be an input itself (in place), by their places in the call's lists
struct InPlace {
  int out, in;
};
// no output on an input or another output, but an output at the very address of the input it may replace
int check_overlap(const Array* in, int ni, const Array* out, int no, InPlace same = {-1, -1}) {
  for (int i = 0; i < no; ++i) {
    if (out[i].r.p == nullptr) continue;
    for (int k = 0; k < ni; ++k) {
      if (in[k].r.p == nullptr || (i == same.out && k == same.in && out[i].r.p == in[k].r.p)) continue;
      if (overlap(out[i].r, in[k].r)) return MM_ERR_ALIAS;
    }
    for (int k = i + 1; k < no; ++k)
      if (out[k].r.p != nullptr && overlap(out[i].r, out[k].r)) return MM_ERR_ALIAS;
  }
  return MM_OK;
}

// the workspace of a call of these sizes, of rows up to kMmaMaxStride elements apart
size_t heads_workspace(int64_t S, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N, int32_t io, bool backward) {
  HeadsPlan p;
  if (check_heads_sizes(S, T, H, P, G, N, io) != MM_OK || H == 0) return 0;
  return plan_heads(p, S, T, H, P, G, N, io, backward, 0) == MM_OK ? p.total : 0;
}

size_t esize(int32_t io) { return io == MM_IO_BF16 ? 2 : 4; }

// ---------------------------------------------------------------- norms: checks

int check_norm_sizes(int64_t rows, int32_t d, float eps, int32_t io) {
  if (rows < 0 || d < 0 || !(eps >= 0.0f)) return MM_ERR_DIM;
  if (io != MM_IO_F32 && io != MM_IO_BF16) return MM_ERR_UNSUPPORTED;
  if (rows > INT32_MAX || (d > 0 && static_cast<uint64_t>(rows) > MM_MAX_ROWS_X_D / static_cast<uint64_t>(d))) return MM_ERR_DIM;
  return MM_OK;
}
int check_gate_sizes(int64_t rows, int32_t d, int32_t groups, float eps, int32_t io) {
  const int rc = check_norm_sizes(rows, d, eps, io);
  if (rc != MM_OK) return rc;
  if (groups < 1 || d % groups != 0) return MM_ERR_DIM;
  if (d / groups > kNormUnit && rows * groups * kWideThreads > kMaxThreads) return MM_ERR_DIM;
  return MM_OK;
}
int check_residual_sizes(int64_t rows, int32_t d, float eps, int32_t io, int32_t res) {
  const int rc = check_norm_sizes(rows, d, eps, io);
  if (rc != MM_OK) return rc;
  if (d > kNormUnit && rows * kWideThreads > kMaxThreads) return MM_ERR_DIM;
  if (d > MM_NORM_MAX_D || (res != MM_IO_F32 && res != io)) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}

// the io and residual types of a call, as template arguments of f
template <typename F>
int by_types(int32_t io, int32_t res, F f) {
  if (io == MM_IO_F32) return f(float{}, float{});
  if (res == MM_IO_F32) return f(uint16_t{}, float{});
  return f(uint16_t{}, uint16_t{});
}

// How a row (or its group) of n columns is spread: NV pieces of E columns for each thread.  With float32 arrays E = 4
// (16 bytes).  With bfloat16 alone 8 (gate_norm of 16384 x 4096: 75.5 us, with 4 78.0), or 4 where that leaves fewer
// lanes idle (groups of 640 columns: 8 leaves 38% idle, 4 17%; the backward of 8192 x 5120 92.2 against 93.3 us).
struct NormShape {
  int e, threads, nv;
};
NormShape norm_shape(int n, bool f32) {
  const auto of = [n](int e) {
    const int pieces = static_cast<int>(cdiv(n, e)), nv = pieces > kNormMaxThreads ? 2 : 1;
    return NormShape{e, static_cast<int>(cdiv(cdiv(pieces, nv), kWave) * kWave), nv};
  };
  const NormShape four = of(4), eight = of(8);
  return f32 || (four.nv == 1 && four.threads * 4 < eight.threads * 8) ? four : eight;
}
// Workgroups for every group of columns; rows beyond this many wait their turn, the next one's loads ahead.
// Backward: what is resident together (24 waves per CU), because each workgroup adds a row of partial sums: gate_norm
// 8192 x 5120 in 8 groups 92.2 us, with 20 waves 97.4, with 28 (the last ones a round of their own) 120; residual_norm
// 8191 x 2560 89.0 us, 10 waves 88.4.  Forward: several rounds even out the ends: gate_norm 16384 x 4096 75.0 us with
// 16 workgroups per CU, with 4 to 8 77 to 79.
int64_t norm_slots(int64_t rows, int n, int groups, bool backward) {
  const int t = norm_shape(n, true).threads;
  const int64_t wgs = kCUs * (backward ? std::max(1, 24 * kWave / t) : std::max(16, 8192 / t));
  return std::max<int64_t>(1, std::min<int64_t>(rows, cdiv(wgs, groups)));
}
// gate_norm's other launches: a workgroup for each group at least, and 16 threads for each column of the weights' sums
int check_gate_launch(int64_t rows, int d, int groups, bool backward) {
  const int n = d / groups;
  if (n <= kNormUnit && norm_slots(rows, n, groups, backward) * groups * norm_shape(n, true).threads > kMaxThreads)
    return MM_ERR_DIM;
  return backward && int64_t{d} * 16 > kMaxThreads ? MM_ERR_DIM : MM_OK;
}
// f(E, NV) of a shape
template <bool BF16, typename F>
void by_pieces(const NormShape& sh, F f) {
  constexpr auto one = std::integral_constant<int, 1>{};
  constexpr auto four = std::integral_constant<int, 4>{};
  if constexpr (BF16) {
    if (sh.e == 8) f(std::integral_constant<int, 8>{}, one);
    else f(four, one);
  } else {
    if (sh.nv == 1) f(four, one);
    else f(four, std::integral_constant<int, 2>{});
  }
}

// workspace of a backward call: partial sums of K weights, for wide rows behind the rows' factors
size_t norm_workspace(int64_t rows, int d, int groups, int K) {
  if (d == 0) return 0;
  if (d / groups > kNormUnit)
    return align256(static_cast<size_t>(rows) * groups * K * 4) + align256(static_cast<size_t>(kWideParts) * K * d * 4);
  return align256(static_cast<size_t>(norm_slots(rows, d / groups, groups, true)) * K * d * 4);
}

}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mamba_mixer_heads_prefill_workspace_bytes(int32_t S, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N,
                                                 int32_t io_dtype) {
  return heads_workspace(S, T, H, P, G, N, io_dtype, false);
}

int mamba_mixer_heads_prefill(const void* x, const void* dt, const void* B, const void* C, const float* A_log,
                              const float* D, const float* dt_bias, const int32_t* cu_seqlens, const float* state_in,
                              float* state_out, void* y, int32_t S, int64_t T, int32_t H, int32_t P, int32_t G,
                              int32_t N, int32_t io_dtype, int64_t x_stride, int64_t dt_stride, int64_t b_stride,
                              int64_t c_stride, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_heads_sizes(S, T, H, P, G, N, io_dtype);
  if (rc != MM_OK) return rc;
  if (H == 0 || S == 0) return MM_OK;
  const int64_t d = static_cast<int64_t>(H) * P, gn = static_cast<int64_t>(G) * N;
  if (x_stride < d || b_stride < gn || c_stride < gn || (dt != nullptr && dt_stride < H)) return MM_ERR_DIM;
  const size_t es = esize(io_dtype), nh = static_cast<size_t>(H) * 4, ns = static_cast<size_t>(S) * d * N * 4;
  const Array in[] = {{rows(x, T, d, x_stride, es), es, false}, {rows(dt, T, H, dt_stride, es), es, true},
                      {rows(B, T, gn, b_stride, es), es, false}, {rows(C, T, gn, c_stride, es), es, false},
                      {flat(A_log, nh), 4, false}, {flat(D, nh), 4, true},
                      {flat(dt_bias, dt != nullptr ? nh : 0), 4, false},
                      {flat(cu_seqlens, (static_cast<size_t>(S) + 1) * 4), 4, false}, {flat(state_in, ns), 4, true}};
  const Array out[] = {{flat(y, static_cast<size_t>(T) * d * es), es, false}, {flat(state_out, ns), 4, false}};
  if ((rc = check_arrays(in, 9)) != MM_OK || (rc = check_arrays(out, 2)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 9, out, 2, {1, 8})) != MM_OK) return rc;
  HeadsPlan p;
  if ((rc = plan_heads(p, S, T, H, P, G, N, io_dtype, false, std::max({x_stride, b_stride, c_stride}))) != MM_OK) return rc;
  if (p.total > 0 && (workspace == nullptr || workspace_bytes < p.total)) return MM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MM_ERR_ALIGN;
  const HeadsArgs a{x, B, C, x_stride, b_stride, c_stride, P, G, N,
                    {dt, dt_stride, A_log, dt_bias, D, cu_seqlens, S, H, T}};
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p.mma) return launch_prefill_mma(p, a, state_in, state_out, y, ws, st);
  if (io_dtype == MM_IO_BF16) return launch_prefill<uint16_t>(p, a, state_in, state_out, y, ws, st);
  return launch_prefill<float>(p, a, state_in, state_out, y, ws, st);
}

int mamba_mixer_heads_decode(const void* x, const void* dt, const void* B, const void* C, const float* A_log,
                             const float* D, const float* dt_bias, const float* state_in, float* state_out, void* y,
                             int32_t Bs, int32_t H, int32_t P, int32_t G, int32_t N, int32_t io_dtype,
                             int64_t x_stride, int64_t dt_stride, int64_t b_stride, int64_t c_stride, void* stream) {
  int rc = check_heads_sizes(Bs, Bs, H, P, G, N, io_dtype);
  if (rc != MM_OK) return rc;
  if (H == 0 || Bs == 0) return MM_OK;
  const int64_t d = static_cast<int64_t>(H) * P, gn = static_cast<int64_t>(G) * N;
  if (x_stride < d || b_stride < gn || c_stride < gn || (dt != nullptr && dt_stride < H)) return MM_ERR_DIM;
  const size_t es = esize(io_dtype), nh = static_cast<size_t>(H) * 4, ns = static_cast<size_t>(Bs) * d * N * 4;
  const Array in[] = {{rows(x, Bs, d, x_stride, es), es, false}, {rows(dt, Bs, H, dt_stride, es), es, true},
                      {rows(B, Bs, gn, b_stride, es), es, false}, {rows(C, Bs, gn, c_stride, es), es, false},
                      {flat(A_log, nh), 4, false}, {flat(D, nh), 4, true},
                      {flat(dt_bias, dt != nullptr ? nh : 0), 4, false}, {flat(state_in, ns), 4, true}};
  const Array out[] = {{flat(y, static_cast<size_t>(Bs) * d * es), es, false}, {flat(state_out, ns), 4, false}};
  if ((rc = check_arrays(in, 8)) != MM_OK || (rc = check_arrays(out, 2)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 8, out, 2, {1, 7})) != MM_OK) return rc;
  const HeadPar hp{dt, dt_stride, A_log, dt_bias, D, nullptr, Bs, H, Bs};
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool vec = N % 4 == 0 && aligned(state_in, 16) && aligned(state_out, 16);
  const auto go = [&](auto io) -> int {
    using IO = decltype(io);
    const Tok<IO> xt = tok<IO>(x, x_stride, P, 1), bt = tok<IO>(B, b_stride, N, H / G), ct = tok<IO>(C, c_stride, N, H / G);
    IO* yo = static_cast<IO*>(y);
    const int64_t heads = static_cast<int64_t>(Bs) * H;
    if (!vec) {
      const int64_t blocks = heads * cdiv(P, kSeqRows);
      if (blocks * kSeqThreads > kMaxThreads) return MM_ERR_DIM;
      const dim3 grid(static_cast<unsigned>(blocks)), block(kSeqThreads);
      if (N <= 64)
        hipLaunchKernelGGL((k_heads_decode_any<IO, 4>), grid, block, 0, st, xt, bt, ct, hp, state_in, state_out, yo, P, N);
      else
        hipLaunchKernelGGL((k_heads_decode_any<IO, 16>), grid, block, 0, st, xt, bt, ct, hp, state_in, state_out, yo, P, N);
      return launched();
    }
    const auto run = [&](auto rl) -> int {
      constexpr int RL = decltype(rl)::value;
      const int64_t per = cdiv(P, kSeqThreads / RL * kDecodeRows);
      if (heads * per * kSeqThreads > kMaxThreads) return MM_ERR_DIM;
      hipLaunchKernelGGL((k_heads_decode<IO, RL>), dim3(static_cast<unsigned>(heads * per)), dim3(kSeqThreads), 0, st, xt, bt,
                         ct, hp, state_in, state_out, yo, P, N, static_cast<int>(per));
      return launched();
    };
    if (N <= 16) return run(std::integral_constant<int, 4>{});
    if (N <= 32) return run(std::integral_constant<int, 8>{});
    if (N <= 64) return run(std::integral_constant<int, 16>{});
    if (N <= 128) return run(std::integral_constant<int, 32>{});
    return run(std::integral_constant<int, 64>{});
  };
  return io_dtype == MM_IO_BF16 ? go(uint16_t{}) : go(float{});
}

size_t mamba_mixer_heads_backward_workspace_bytes(int32_t S, int64_t T, int32_t H, int32_t P, int32_t G, int32_t N,
                                                  int32_t io_dtype) {
  return heads_workspace(S, T, H, P, G, N, io_dtype, true);
}

int mamba_mixer_heads_backward(const void* x, const void* dt, const void* B, const void* C, const float* A_log,
                               const float* D, const float* dt_bias, const int32_t* cu_seqlens, const float* state_in,
                               const void* dy, const float* dstate_out, void* dx, void* ddt, void* dB, void* dC,
                               float* dA_log, float* dD, float* ddt_bias, float* dstate_in, int32_t S, int64_t T,
                               int32_t H, int32_t P, int32_t G, int32_t N, int32_t io_dtype, int64_t x_stride,
                               int64_t dt_stride, int64_t b_stride, int64_t c_stride, int64_t dx_stride,
                               int64_t ddt_stride, int64_t db_stride, int64_t dc_stride, void* workspace,
                               size_t workspace_bytes, void* stream) {
  int rc = check_heads_sizes(S, T, H, P, G, N, io_dtype);
  if (rc != MM_OK) return rc;
  if (H == 0) return MM_OK;
  const int64_t d = static_cast<int64_t>(H) * P, gn = static_cast<int64_t>(G) * N;
  if (x_stride < d || b_stride < gn || c_stride < gn || dx_stride < d || db_stride < gn || dc_stride < gn ||
      (dt != nullptr && (dt_stride < H || ddt_stride < H)))
    return MM_ERR_DIM;
  const size_t es = esize(io_dtype), nh = static_cast<size_t>(H) * 4, ns = static_cast<size_t>(S) * d * N * 4;
  const size_t ndt = dt != nullptr ? nh : 0;
  const Array in[] = {{rows(x, T, d, x_stride, es), es, false}, {rows(dt, T, H, dt_stride, es), es, true},
                      {rows(B, T, gn, b_stride, es), es, false}, {rows(C, T, gn, c_stride, es), es, false},
                      {flat(dy, static_cast<size_t>(T) * d * es), es, false}, {flat(A_log, nh), 4, false},
                      {flat(D, nh), 4, true}, {flat(dt_bias, ndt), 4, false},
                      {flat(cu_seqlens, S > 0 ? (static_cast<size_t>(S) + 1) * 4 : 0), 4, false},
                      {flat(state_in, ns), 4, true}, {flat(dstate_out, ns), 4, true}};
  const Array out[] = {{rows(dx, T, d, dx_stride, es), es, false}, {rows(ddt, dt != nullptr ? T : 0, H, ddt_stride, es), es, false},
                       {rows(dB, T, gn, db_stride, es), es, false}, {rows(dC, T, gn, dc_stride, es), es, false},
                       {flat(dA_log, nh), 4, false}, {flat(dD, D != nullptr ? nh : 0), 4, false},
                       {flat(ddt_bias, ndt), 4, false}, {flat(dstate_in, ns), 4, true}};
  if ((rc = check_arrays(in, 11)) != MM_OK || (rc = check_arrays(out, 8)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 11, out, 8)) != MM_OK) return rc;
  HeadsPlan p;
  if ((rc = plan_heads(p, S, T, H, P, G, N, io_dtype, true, std::max({x_stride, b_stride, c_stride, dx_stride}))) != MM_OK) return rc;
  if (p.total > 0 && (workspace == nullptr || workspace_bytes < p.total)) return MM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MM_ERR_ALIGN;
  const HeadsArgs a{x, B, C, x_stride, b_stride, c_stride, P, G, N,
                    {dt, dt_stride, A_log, dt_bias, D, cu_seqlens, S, H, T}};
  const HeadsGrads o{dy, state_in, dstate_out, dx, ddt, dB, dC, dx_stride, ddt_stride, db_stride, dc_stride,
                     dA_log, D != nullptr ? dD : nullptr, dt != nullptr ? ddt_bias : nullptr, dstate_in};
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p.mma) return launch_backward_mma(p, a, o, ws, st);
  if (io_dtype == MM_IO_BF16) return launch_backward<uint16_t>(p, a, o, ws, st);
  return launch_backward<float>(p, a, o, ws, st);
}

// ---------------------------------------------------------------- norms

int mamba_mixer_gate_norm(const void* y, const void* z, const float* weight, void* out, int64_t nrows, int32_t d,
                          int32_t groups, float eps, int32_t gate_first, int32_t io_dtype, int64_t y_stride,
                          int64_t z_stride, void* stream) {
  int rc = check_gate_sizes(nrows, d, groups, eps, io_dtype);
  if (rc != MM_OK) return rc;
  if (nrows == 0 || d == 0) return MM_OK;
  if ((rc = check_gate_launch(nrows, d, groups, false)) != MM_OK) return rc;
  if (y_stride < d || z_stride < d) return MM_ERR_DIM;
  const size_t es = esize(io_dtype);
  const Array in[] = {{rows(y, nrows, d, y_stride, es), es, false}, {rows(z, nrows, d, z_stride, es), es, false},
                      {flat(weight, static_cast<size_t>(d) * 4), 4, false}};
  const Array o[] = {{flat(out, static_cast<size_t>(nrows) * d * es), es, false}};
  if ((rc = check_arrays(in, 3)) != MM_OK || (rc = check_arrays(o, 1)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 3, o, 1, y_stride == d ? InPlace{0, 0} : InPlace{-1, -1})) != MM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const auto go = [&](auto io) {
    using IO = decltype(io);
    const GateArgs<IO> a{static_cast<const IO*>(y), static_cast<const IO*>(z), nullptr, y_stride, z_stride, weight,
                         nrows, d, groups, eps, gate_first != 0 ? 1 : 0};
    if (d / groups > kNormUnit) {
      hipLaunchKernelGGL((k_wide_gate_norm<IO>), dim3(static_cast<unsigned>(nrows * groups)), dim3(kWideThreads), 0, st, a,
                         static_cast<IO*>(out));
      return;
    }
    const NormShape sh = norm_shape(d / groups, io_dtype == MM_IO_F32);
    const dim3 grid(static_cast<unsigned>(norm_slots(nrows, d / groups, groups, false) * groups));
    by_pieces<sizeof(IO) == 2>(sh, [&](auto e, auto nv) {
      constexpr int E = decltype(e)::value, NV = decltype(nv)::value;
      const dim3 block(sh.threads);
      IO* o = static_cast<IO*>(out);
      if (gate_first != 0) hipLaunchKernelGGL((k_gate_norm<IO, E, NV, true>), grid, block, 0, st, a, o);
      else hipLaunchKernelGGL((k_gate_norm<IO, E, NV, false>), grid, block, 0, st, a, o);
    });
  };
  if (io_dtype == MM_IO_BF16) go(uint16_t{}); else go(float{});
  return launched();
}

size_t mamba_mixer_gate_norm_backward_workspace_bytes(int64_t nrows, int32_t d, int32_t groups) {
  if (check_gate_sizes(nrows, d, groups, 0.0f, MM_IO_F32) != MM_OK || d == 0) return 0;
  return check_gate_launch(nrows, d, groups, true) == MM_OK ? norm_workspace(nrows, d, groups, 1) : 0;
}

int mamba_mixer_gate_norm_backward(const void* dout, const void* y, const void* z, const float* weight, void* dy,
                                   void* dz, float* dweight, int64_t nrows, int32_t d, int32_t groups, float eps,
                                   int32_t gate_first, int32_t io_dtype, int64_t y_stride, int64_t z_stride,
                                   int64_t dy_stride, int64_t dz_stride, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  int rc = check_gate_sizes(nrows, d, groups, eps, io_dtype);
  if (rc != MM_OK) return rc;
  if (d == 0) return MM_OK;
  if ((rc = check_gate_launch(nrows, d, groups, true)) != MM_OK) return rc;
  if (y_stride < d || z_stride < d || dy_stride < d || dz_stride < d) return MM_ERR_DIM;
  const size_t es = esize(io_dtype), nd = static_cast<size_t>(d) * 4;
  const Array in[] = {{flat(dout, static_cast<size_t>(nrows) * d * es), es, false},
                      {rows(y, nrows, d, y_stride, es), es, false}, {rows(z, nrows, d, z_stride, es), es, false},
                      {flat(weight, nd), 4, false}};
  const Array o[] = {{rows(dy, nrows, d, dy_stride, es), es, false}, {rows(dz, nrows, d, dz_stride, es), es, false},
                     {flat(dweight, nd), 4, false}};
  if ((rc = check_arrays(in, 4)) != MM_OK || (rc = check_arrays(o, 3)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 4, o, 3)) != MM_OK) return rc;
  const size_t need = mamba_mixer_gate_norm_backward_workspace_bytes(nrows, d, groups);
  if (workspace == nullptr || workspace_bytes < need) return MM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MM_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const int n = d / groups;
  const bool wide = n > kNormUnit;
  const int64_t slots = wide ? std::min<int64_t>(kWideParts, nrows) : norm_slots(nrows, n, groups, true);
  float* const stats = part;
  if (wide) part += align256(static_cast<size_t>(nrows) * groups * 4) / 4;
  const auto go = [&](auto io) {
    using IO = decltype(io);
    const GateArgs<IO> a{static_cast<const IO*>(y), static_cast<const IO*>(z), static_cast<const IO*>(dout), y_stride,
                         z_stride, weight, nrows, d, groups, eps, gate_first != 0 ? 1 : 0};
    if (wide) {
      const dim3 block(kWideThreads), cols(static_cast<unsigned>(cdiv(d, kWideThreads)), static_cast<unsigned>(slots));
      hipLaunchKernelGGL((k_wide_gate_norm_bwd<IO>), dim3(static_cast<unsigned>(nrows * groups)), block, 0, st, a,
                         static_cast<IO*>(dy), static_cast<IO*>(dz), dy_stride, dz_stride, stats);
      hipLaunchKernelGGL((k_wide_gate_norm_dw<IO>), cols, block, 0, st, a, stats, part, cdiv(nrows, slots));
      return;
    }
    const NormShape sh = norm_shape(n, io_dtype == MM_IO_F32);
    by_pieces<sizeof(IO) == 2>(sh, [&](auto e, auto nv) {
      constexpr int E = decltype(e)::value, NV = decltype(nv)::value;
      const dim3 grid(static_cast<unsigned>(slots * groups)), block(sh.threads);
      IO *oy = static_cast<IO*>(dy), *oz = static_cast<IO*>(dz);
      if (gate_first != 0)
        hipLaunchKernelGGL((k_gate_norm_bwd<IO, E, NV, true>), grid, block, 0, st, a, oy, oz, dy_stride, dz_stride, part);
      else
        hipLaunchKernelGGL((k_gate_norm_bwd<IO, E, NV, false>), grid, block, 0, st, a, oy, oz, dy_stride, dz_stride, part);
    });
  };
  if (nrows > 0) { if (io_dtype == MM_IO_BF16) go(uint16_t{}); else go(float{}); }
  const NormParts np{{part, nullptr, nullptr}, {dweight, nullptr, nullptr}};
  hipLaunchKernelGGL(k_norm_parts, dim3(static_cast<unsigned>(cdiv(d, 16))), dim3(256), 0, st, np,
                     static_cast<int>(nrows > 0 ? slots : 0), static_cast<int64_t>(d), d);
  return launched();
}

int mamba_mixer_residual_norm(const void* h, const void* residual, const float* weight, const float* post_weight,
                              const float* scale_vec, float scale, void* residual_out, void* out, int64_t nrows,
                              int32_t d, float eps, int32_t io_dtype, int32_t res_dtype, void* stream) {
  int rc = check_residual_sizes(nrows, d, eps, io_dtype, res_dtype);
  if (rc != MM_OK) return rc;
  if (nrows == 0 || d == 0) return MM_OK;
  const size_t es = esize(io_dtype), rs = esize(res_dtype), n = static_cast<size_t>(nrows) * d, nd = static_cast<size_t>(d) * 4;
  const Array in[] = {{flat(h, n * es), es, false}, {flat(residual, n * rs), rs, true}, {flat(weight, nd), 4, false},
                      {flat(post_weight, nd), 4, true}, {flat(scale_vec, nd), 4, true}};
  const Array o[] = {{flat(residual_out, n * rs), rs, false}, {flat(out, n * es), es, false}};
  if ((rc = check_arrays(in, 5)) != MM_OK || (rc = check_arrays(o, 2)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 5, o, 2, {0, 1})) != MM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_types(io_dtype, res_dtype, [&](auto io, auto rt) {
    using IO = decltype(io);
    using RES = decltype(rt);
    const ResArgs<IO, RES> a{static_cast<const IO*>(h), static_cast<const RES*>(residual), weight, post_weight,
                             scale_vec, scale, eps, nrows, d};
    if (d > kNormUnit) {
      const int r = allow_lds(&k_wide_residual_norm<IO, RES>, nd);
      if (r != MM_OK) return r;
      hipLaunchKernelGGL((k_wide_residual_norm<IO, RES>), dim3(static_cast<unsigned>(nrows)), dim3(kWideThreads), nd, st, a,
                         static_cast<RES*>(residual_out), static_cast<IO*>(out));
      return launched();
    }
    const NormShape sh = norm_shape(d, res_dtype == MM_IO_F32);
    by_pieces<sizeof(RES) == 2>(sh, [&](auto e, auto nv) {
      hipLaunchKernelGGL((k_residual_norm<IO, RES, decltype(e)::value, decltype(nv)::value>),
                         dim3(static_cast<unsigned>(norm_slots(nrows, d, 1, false))), dim3(sh.threads), 0, st, a,
                         static_cast<RES*>(residual_out), static_cast<IO*>(out));
    });
    return launched();
  });
}

size_t mamba_mixer_residual_norm_backward_workspace_bytes(int64_t nrows, int32_t d) {
  if (check_residual_sizes(nrows, d, 0.0f, MM_IO_F32, MM_IO_F32) != MM_OK) return 0;
  return norm_workspace(nrows, d, 1, 3);
}

int mamba_mixer_residual_norm_backward(const void* dout, const void* dresidual_out, const void* h,
                                       const void* residual_out, const float* weight, const float* post_weight,
                                       const float* scale_vec, float scale, void* dresidual, void* dh, float* dweight,
                                       float* dpost_weight, float* dscale_vec, int64_t nrows, int32_t d, float eps,
                                       int32_t io_dtype, int32_t res_dtype, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  int rc = check_residual_sizes(nrows, d, eps, io_dtype, res_dtype);
  if (rc != MM_OK) return rc;
  if (d == 0) return MM_OK;
  const size_t es = esize(io_dtype), rs = esize(res_dtype), n = static_cast<size_t>(nrows) * d, nd = static_cast<size_t>(d) * 4;
  const Array in[] = {{flat(dout, n * es), es, false}, {flat(dresidual_out, n * rs), rs, true}, {flat(h, n * es), es, false},
                      {flat(residual_out, n * rs), rs, false}, {flat(weight, nd), 4, false},
                      {flat(post_weight, nd), 4, true}, {flat(scale_vec, nd), 4, true}};
  const Array o[] = {{flat(dresidual, n * rs), rs, false}, {flat(dh, n * es), es, false}, {flat(dweight, nd), 4, false},
                     {flat(dpost_weight, post_weight != nullptr ? nd : 0), 4, false},
                     {flat(dscale_vec, scale_vec != nullptr ? nd : 0), 4, false}};
  if ((rc = check_arrays(in, 7)) != MM_OK || (rc = check_arrays(o, 5)) != MM_OK) return rc;
  if ((rc = check_overlap(in, 7, o, 5, {0, 1})) != MM_OK) return rc;
  const size_t need = mamba_mixer_residual_norm_backward_workspace_bytes(nrows, d);
  if (workspace == nullptr || workspace_bytes < need) return MM_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MM_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const bool wide = d > kNormUnit;
  const int64_t slots = wide ? std::min<int64_t>(kWideParts, nrows) : norm_slots(nrows, d, 1, true);
  float* const stats = part;
  if (wide) part += align256(static_cast<size_t>(nrows) * 3 * 4) / 4;
  if (nrows > 0) {
    rc = by_types(io_dtype, res_dtype, [&](auto io, auto rt) {
      using IO = decltype(io);
      using RES = decltype(rt);
      const ResArgs<IO, RES> a{static_cast<const IO*>(h), static_cast<const RES*>(residual_out), weight, post_weight,
                               scale_vec, scale, eps, nrows, d};
      if (wide) {
        const int r = allow_lds(&k_wide_residual_norm_bwd<IO, RES>, nd);
        if (r != MM_OK) return r;
        const IO* go = static_cast<const IO*>(dout);
        const RES* gr = static_cast<const RES*>(dresidual_out);
        const dim3 grid(static_cast<unsigned>(nrows)), block(kWideThreads);
        const dim3 cols(static_cast<unsigned>(cdiv(d, kWideThreads)), static_cast<unsigned>(slots));
        // the rows' factors and the weights' sums before the gradients: dresidual may be written over dresidual_out
        hipLaunchKernelGGL((k_wide_residual_norm_bwd<IO, RES>), grid, block, nd, st, a, go, gr, static_cast<RES*>(nullptr),
                           static_cast<IO*>(nullptr), stats);
        hipLaunchKernelGGL((k_wide_residual_norm_dw<IO, RES>), cols, block, 0, st, a, go, gr, stats, part,
                           cdiv(nrows, slots));
        hipLaunchKernelGGL((k_wide_residual_norm_bwd<IO, RES>), grid, block, nd, st, a, go, gr,
                           static_cast<RES*>(dresidual), static_cast<IO*>(dh), stats);
        return launched();
      }
      const NormShape sh = norm_shape(d, res_dtype == MM_IO_F32);
      by_pieces<sizeof(RES) == 2>(sh, [&](auto e, auto nv) {
        hipLaunchKernelGGL((k_residual_norm_bwd<IO, RES, decltype(e)::value, decltype(nv)::value>), dim3(static_cast<unsigned>(slots)),
                           dim3(sh.threads), 0, st, a, static_cast<const IO*>(dout), static_cast<const RES*>(dresidual_out),
                           static_cast<RES*>(dresidual), static_cast<IO*>(dh), part);
      });
      return launched();
    });
    if (rc != MM_OK) return rc;
  }
  NormParts np{};
  int k = 0;
  float* const outs[] = {dweight, post_weight != nullptr ? dpost_weight : nullptr, scale_vec != nullptr ? dscale_vec : nullptr};
  for (int i = 0; i < 3; ++i)
    if (outs[i] != nullptr) {
      np.part[k] = part + static_cast<int64_t>(i) * d;
      np.out[k++] = outs[i];
    }
  hipLaunchKernelGGL(k_norm_parts, dim3(static_cast<unsigned>(cdiv(d, 16)), static_cast<unsigned>(k)), dim3(256), 0, st, np,
                     static_cast<int>(nrows > 0 ? slots : 0), static_cast<int64_t>(3) * d, d);
  return launched();
}

}  // extern "C"
