// The causal depthwise convolution by itself: kernels, argument checks and entry points.
//   u[p] = bias + sum_k w_k X(p - W + 1 + k),  y = u sigmoid(u) or u;  X(q < 0): the state's inputs
//   dX(q) = sum_k w_k du(q + W - 1 - k) + what the final state asks for,  dw_k = sum_p du(p) X(p - W + 1 + k)
// Bound by memory.  A wave walks L tokens of 64 V channels (512 bytes of bfloat16 a row: narrower rows cost a fifth of the
// bandwidth), its window, weights and the weights' gradients in registers: an input is read once, but for the W - 1 tokens
// around a walk.  kStep tokens are loaded at a time, the next ones while these are used (8 at a time: backward 53 us for
// 48.7, and fewer walks fit; 2: 65.3 forward for 63.9).  16384 x 4352 of bfloat16: 286 MB in 61 us, 4.7 TB/s; backward
// 8 x 2048 x 1792: 177 MB in 48 us with the sum of the partial gradients (4 us), half of the time vector instructions.
// Longer: 65536 x 2048 5.1 TB/s forward, 4.9 backward.
#include <algorithm>
#include <type_traits>

#include "layer/common.h"

namespace mm {
namespace {

constexpr int kConvWaves = 4, kConvThreads = kConvWaves * 64, kStep = 4;
// A walk has at most kConvTokens tokens, fewer where there would be fewer than kConvWalks of them (one for each SIMD).
// More and shorter walks read more rows twice: 8192 x 2048 f32 4096 walks 28.9 us, 2048 27.4, 1024 25.9; backward 46.7 with
// 2048, 44.1 with 1024.  Longer ones leave fewer: backward 8 x 2048 x 1792 bf16 with 128 tokens 63 us, with 64 47.5.
constexpr int64_t kConvTokens = 64, kConvWalks = 1024;

struct ConvArgs {
  const void* x;
  const float *w, *bias;
  const int32_t* cu;
  const float* state_in;
  int64_t x_ts, T;
  int S, d, L, silu;
};

// ---------------------------------------------------------------- a thread's channel, one by one: states
template <typename IO>
__device__ __forceinline__ float conv_raw(const ConvArgs& a, int W, int s, int64_t g0, int64_t q, int c) {
  if (q >= 0) return ld_io(static_cast<const IO*>(a.x), (g0 + q) * a.x_ts + c);
  return a.state_in != nullptr ? a.state_in[(static_cast<int64_t>(s) * a.d + c) * (W - 1) + W - 1 + q] : 0.0f;
}
__device__ __forceinline__ float conv_slope(float u, float g, bool silu) {
  if (!silu) return g;
  const Sigmoids v = sigmoids(u);
  return g * v.s * __builtin_fmaf(u, v.s1, 1.0f);
}
__device__ __forceinline__ void conv_place(int64_t i, int d, int& s, int& c) {
  s = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(d));  // S d < 2^31
  c = static_cast<int>(i - static_cast<int64_t>(s) * d);
}
// the final state of (sequence, channel) i; state_out may be state_in
template <typename IO, int W>
__device__ __forceinline__ void conv_state(const ConvArgs& a, float* state_out, int64_t i) {
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  int s, c;
  conv_place(i, a.d, s, c);
  const int64_t g0 = a.cu[s], n = a.cu[s + 1] - g0;
  float v[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k) v[k] = conv_raw<IO>(a, W, s, g0, n - W + 1 + k, c);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) state_out[i * (W - 1) + k] = v[k];
}
// the gradient of the initial state of (sequence, channel) i, from its first W - 1 tokens
template <typename IO, int W>
__device__ __forceinline__ void conv_dstate(const ConvArgs& a, const IO* dy, const float* dstate_out, float* dstate_in, int64_t i) {
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  int s, c;
  conv_place(i, a.d, s, c);
  const int64_t g0 = a.cu[s], n = a.cu[s + 1] - g0;
  const float b = a.bias != nullptr ? a.bias[c] : 0.0f;
  float w[W], du[W - 1];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = a.w[static_cast<int64_t>(c) * W + k];
#pragma unroll
  for (int p = 0; p < W - 1; ++p) {
    du[p] = 0.0f;
    if (p < n) {
      float u = b;
#pragma unroll
      for (int k = 0; k < W; ++k) u = __builtin_fmaf(w[k], conv_raw<IO>(a, W, s, g0, p - W + 1 + k, c), u);
      du[p] = conv_slope(u, ld_io(dy, (g0 + p) * a.d + c), a.silu);
    }
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {  // X(q), q = j - W + 1; a sequence shorter than that leaves it in its final state
    const int64_t f = j - n;
    float v = dstate_out != nullptr && f >= 0 ? dstate_out[i * (W - 1) + f] : 0.0f;
#pragma unroll
    for (int p = 0; p <= j; ++p) v = __builtin_fmaf(w[j - p], du[p], v);
    dstate_in[i * (W - 1) + j] = v;
  }
}

// ---------------------------------------------------------------- walks
// what a wave's walk knows of its tokens and channels
template <typename IO, int V, int W>
struct ConvWalk {
  const ConvArgs& a;
  int64_t c0, c, t0, t1;
  uint32_t off;      // of this lane's channels in a row; lanes without channels do the first ones' work again
  int s;             // the sequence of the present token,
  int64_t lo, hi;    // its first token and the one behind its last
  float w[W][V], b[V], win[W - 1][V];
  Chans<IO, V> before[W - 1];

  // asks for what the walk begins with, begin() waits for it
  __device__ __forceinline__ ConvWalk(const ConvArgs& a, int64_t slice, int64_t walk) : a(a) {
    const int lane = threadIdx.x & 63;
    c0 = slice * 64 * V;
    c = c0 + lane * V < a.d ? c0 + lane * V : c0;
    off = static_cast<uint32_t>(c - c0) * static_cast<uint32_t>(sizeof(IO));
    t0 = walk * a.L;
    t1 = std::min(t0 + a.L, a.T);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) before[j] = row(std::max<int64_t>(t0 - W + 1 + j, 0));
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b[i] = a.bias != nullptr ? a.bias[c + i] : 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = a.w[(c + i) * W + k];
    }
    s = seq_of(a.cu, a.S, t0);
    lo = a.cu[s];
    hi = a.cu[s + 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) win[j][i] = before[j][i];
    }
    if (t0 - W + 1 < lo) from_state(t0);
  }
  // the base in scalar registers, and an offset that the compiler cannot make part of a 64-bit address ahead of its use
  __device__ __forceinline__ Chans<IO, V> row(int64_t t) {
    asm volatile("" : "+v"(off));
    return load_chans<IO, V>(sbase(static_cast<const IO*>(a.x) + t * a.x_ts + c0), off);
  }
  __device__ __forceinline__ Chans<IO, V> grads(const IO* dy, int64_t t) {
    asm volatile("" : "+v"(off));
    return load_chans<IO, V>(sbase(dy + t * a.d + c0), off);
  }
  __device__ __forceinline__ void store(IO* p, int64_t t, int64_t ts, const float (&v)[V]) {
    asm volatile("" : "+v"(off));
    store_chans<IO, V>(sbase(p + t * ts + c0), off, v);
  }
  // those of the inputs before token t that its sequence has from its state.  The wait stands here, so
  // that the way around it needs none.
  __device__ __forceinline__ void from_state(int64_t t) {
    const int64_t n = lo + W - 1 - t;  // of them (t - lo of the state's have left the window), if not all
    if (a.state_in != nullptr) {
      const float* p = a.state_in + (s * static_cast<int64_t>(a.d) + c) * (W - 1) + (t - lo);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (j < n) {
#pragma unroll
          for (int i = 0; i < V; ++i) win[j][i] = p[i * (W - 1) + j];
        }
    } else {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) win[j][i] = j < n ? 0.0f : win[j][i];
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) asm volatile("" : "+v"(win[j][i]));
  }
  // Token t = hi is the first of another sequence: the next one, or if that is empty one that halving finds (one after the
  // other, 400000 empty ones between two tokens took 30 ms).
  __device__ __forceinline__ void enter(int64_t t) {
    hi = a.cu[++s + 1];
    if (t >= hi) {
      s = seq_of(a.cu, a.S, t);
      hi = a.cu[s + 1];
    }
    lo = t;
    from_state(t);
  }
  __device__ __forceinline__ void pre(const Chans<IO, V>& r, float (&u)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      u[i] = b[i];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) u[i] = __builtin_fmaf(w[k][i], win[k][i], u[i]);
      u[i] = __builtin_fmaf(w[W - 1][i], r[i], u[i]);
    }
  }
  __device__ __forceinline__ void shift(const Chans<IO, V>& r) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
      win[W - 2][i] = r[i];
    }
  }
};
// The walk's steps of kStep tokens: load(rows, t) asks for a step's rows, use(t + k, rows, k) is called for each token in
// turn.  Two sets of rows take turns: while one is used the other is on its way.  The first step stands before the loop, so
// that each pass begins with the same accesses under way (a step's loads, then its stores) and waits for the loads alone.
template <typename Rows, typename Load, typename Use>
__device__ __forceinline__ int64_t conv_steps(int64_t t, int64_t t1, Rows& r0, Load load, Use use) {
  const int64_t te = t + (t1 - t) / kStep * kStep;
  const auto step = [&](const Rows& now, Rows& next) {
    load(next, t + kStep < te ? t + kStep : t);  // the last step asks for its own rows again, which nothing uses
#pragma unroll
    for (int k = 0; k < kStep; ++k) use(t + k, now, k);
    t += kStep;
  };
  Rows r1;
  if (t < te) {
    step(r0, r1);
    while (t < te) {
      step(r1, r0);
      if (t < te) step(r0, r1);
      else break;
    }
  }
  return t;
}

// blocks of `walks` (kConvWaves to a block, slice by slice), then those of the states where state_out is given
template <typename IO, int V, int W>
__global__ __launch_bounds__(kConvThreads) void k_conv(ConvArgs a, int64_t blocks, uint32_t slices, IO* __restrict__ y, float* state_out) {
  if (blockIdx.x >= blocks) {
    conv_state<IO, W>(a, state_out, (blockIdx.x - blocks) * kConvThreads + threadIdx.x);
    return;
  }
  const int64_t walk = static_cast<int64_t>(blockIdx.x / slices) * kConvWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  if (walk * a.L >= a.T) return;
  struct Rows {
    Chans<IO, V> x[kStep];
  };
  ConvWalk<IO, V, W> x(a, blockIdx.x % slices, walk);
  const auto load = [&](Rows& r, int64_t t) {
#pragma unroll
    for (int k = 0; k < kStep; ++k) r.x[k] = x.row(t + k);
  };
  const auto out = [&](int64_t t, const Chans<IO, V>& r) {
    if (t >= x.hi) x.enter(t);
    float u[V];
    x.pre(r, u);
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] *= a.silu ? sigmoid(u[i]) : 1.0f;
    x.store(y, t, a.d, u);
    x.shift(r);
  };
  Rows r0;
  if (x.t0 + kStep <= x.t1) load(r0, x.t0);
  x.begin();
  int64_t t = conv_steps(x.t0, x.t1, r0, load, [&](int64_t t, const Rows& r, int k) { out(t, r.x[k]); });
#pragma unroll 1
  for (; t < x.t1; ++t) out(t, x.row(t));
}

// One token a row, a thread for V channels of it.
template <typename IO, int V, int W>
__global__ __launch_bounds__(256) void k_conv_decode(ConvArgs a, float* state_out, IO* __restrict__ y) {
  const int64_t n = static_cast<int64_t>(a.S) * a.d, i0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  if (i0 >= n) return;
  const int64_t s = i0 / a.d, c = i0 - s * a.d;
  const Chans<IO, V> r = load_chans<IO, V>(global(static_cast<const IO*>(a.x) + s * a.x_ts + c), 0);
  float v[V][W - 1], w[V][W], u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    u[i] = a.bias != nullptr ? a.bias[c + i] : 0.0f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) v[i][k] = a.state_in != nullptr ? a.state_in[(i0 + i) * (W - 1) + k] : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[i][k] = a.w[(c + i) * W + k];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) u[i] = __builtin_fmaf(w[i][k], v[i][k], u[i]);
    u[i] = __builtin_fmaf(w[i][W - 1], r[i], u[i]);
    if (a.silu) u[i] *= sigmoid(u[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) state_out[(i0 + i) * (W - 1) + k] = k < W - 2 ? v[i][k + 1] : r[i];
  store_chans<IO, V>(global(y + i0), 0, u);
}

// A walk computes du for its own tokens and up to W - 1 behind them; pend holds the gradients of the last W tokens as they
// gather.
// part: [blocks / slices][W + 1][d], a block's sums of dw and dbias.  Registers allow three waves of a SIMD; asking for
// four spills (121 us).
template <typename IO, int V, int W>
__global__ __launch_bounds__(kConvThreads) void k_conv_bwd(ConvArgs a, int64_t blocks, uint32_t slices, const IO* __restrict__ dy,
                                                           const float* __restrict__ dstate_out, IO* __restrict__ dx, int64_t dx_ts,
                                                           float* __restrict__ part, float* __restrict__ dstate_in) {
  if (blockIdx.x >= blocks) {
    conv_dstate<IO, W>(a, dy, dstate_out, dstate_in, (blockIdx.x - blocks) * kConvThreads + threadIdx.x);
    return;
  }
  __shared__ float sums[kConvWaves][W + 1][64 * V];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int64_t slice = blockIdx.x % slices, group = blockIdx.x / slices, walk = group * kConvWaves + wave;
  float dw[W][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][i] = 0.0f;
  }
  if (walk * a.L < a.T) {
    struct Rows {
      Chans<IO, V> x[kStep], g[kStep];
    };
    ConvWalk<IO, V, W> x(a, slice, walk);
    const auto load = [&](Rows& r, int64_t t) {
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        r.x[k] = x.row(t + k);
        r.g[k] = x.grads(dy, t + k);
      }
    };
    Rows r0;
    if (x.t0 + kStep <= x.t1) load(r0, x.t0);
    x.begin();
    float pend[W][V];  // of tokens p - W + 1 .. p
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) pend[j][i] = 0.0f;
    int64_t first = std::max(x.t0, x.lo);  // of the tokens whose gradients this walk gathers now
    // the first token that asks for more than its taps: of the final state or of another sequence
    const auto more = [&] { return dstate_out != nullptr ? x.hi - W + 1 : x.hi; };
    int64_t event = more();
    // no token from p on adds to those before it
    const auto flush = [&](int64_t p) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int64_t q = p - W + 1 + j;
        if (q >= first && q < x.t1) x.store(dx, q, dx_ts, pend[j]);
      }
    };
    // du of token p, and what it adds to tokens p - W + 1 .. p
    const auto taps = [&](const Chans<IO, V>& r, const Chans<IO, V>& g, float(&du)[V]) {
      float u[V];
      x.pre(r, u);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float v = conv_slope(u[i], g[i], true);
        du[i] = a.silu ? v : g[i];
#pragma unroll
        for (int j = 0; j < W; ++j) pend[j][i] = __builtin_fmaf(x.w[j][i], du[i], pend[j][i]);
      }
    };
    // behind token p: token q is through.  What stands before `first` goes to its row, which gets its own value after it.
    const auto leave = [&](int64_t p, const Chans<IO, V>& r) {
      x.shift(r);
      x.store(dx, std::max(p - W + 1, first), dx_ts, pend[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) pend[j][i] = pend[j + 1][i];
        pend[W - 1][i] = 0.0f;
      }
    };
    const auto back = [&](int64_t p, const Chans<IO, V>& r, const Chans<IO, V>& g) {
      if (p >= event) {
        if (p >= x.hi) {
          flush(p);
          x.enter(p);
          first = p;
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) pend[j][i] = 0.0f;
          event = more();
        }
        if (p >= event) {
          const int64_t f = p - event;  // its place in the final state
#pragma unroll
          for (int i = 0; i < V; ++i)
            pend[W - 1][i] = dstate_out[(x.s * static_cast<int64_t>(a.d) + x.c + i) * (W - 1) + f];
#pragma unroll
          for (int i = 0; i < V; ++i) asm volatile("" : "+v"(pend[W - 1][i]));  // waited for here
        }
      }
      float du[V];
      taps(r, g, du);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        db[i] += du[i];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dw[k][i] = __builtin_fmaf(du[i], x.win[k][i], dw[k][i]);
        dw[W - 1][i] = __builtin_fmaf(du[i], r[i], dw[W - 1][i]);
      }
      leave(p, r);
    };
    int64_t t = conv_steps(x.t0, x.t1, r0, load, [&](int64_t p, const Rows& r, int k) { back(p, r.x[k], r.g[k]); });
#pragma unroll 1
    for (; t < x.t1; ++t) back(t, x.row(t), x.grads(dy, t));
#pragma unroll 1
    for (; t < x.t1 + W - 1 && t < x.hi; ++t) {
      const Chans<IO, V> r = x.row(t);
      float du[V];
      taps(r, x.grads(dy, t), du);
      leave(t, r);
    }
    flush(t);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) sums[wave][k][lane * V + i] = dw[k][i];
    sums[wave][W][lane * V + i] = db[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (W + 1) * 64 * V; i += kConvThreads) {
    const int k = i / (64 * V), j = i % (64 * V);
    const int64_t c = slice * 64 * V + j;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kConvWaves; ++q) v += sums[q][k][j];
    if (c < a.d) part[(group * (W + 1) + k) * a.d + c] = v;
  }
}

// the weights' gradients from `parts` rows of [W + 1, d] partial sums
__global__ __launch_bounds__(256) void k_conv_parts(const float* __restrict__ part, int64_t parts, int d, int W,
                                                    float* __restrict__ dw, float* __restrict__ db) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kPartColumns + threadIdx.x % kPartColumns, n = static_cast<int64_t>(W + 1) * d;
  const float v = sum_parts(part, parts, n, i);
  if (i >= n || threadIdx.x >= kPartColumns) return;
  const int64_t k = i / d, c = i % d;
  if (k < W) dw[c * W + k] = v;
  else if (db != nullptr) db[c] = v;
}

// ---------------------------------------------------------------- host
// Channels of a lane: all there or none.  Two in place of four: 16384 x 4352 68 us for 65.8, backward 8 x 2048 x 1792 67
// for 56.5.
int conv_channels(int32_t d) { return d % 4 == 0 ? 4 : d % 2 == 0 ? 2 : 1; }
int64_t conv_slices(int32_t d) { return cdiv(d, 64 * conv_channels(d)); }
// tokens of a walk, in steps of kStep
int64_t conv_tokens(int64_t T, int32_t d) {
  return std::min(kConvTokens, std::max<int64_t>(kStep, T * conv_slices(d) / kConvWalks / kStep * kStep));
}
int64_t conv_groups(int64_t T, int32_t d) { return cdiv(T, conv_tokens(T, d) * kConvWaves); }

int check_conv(int64_t S, int64_t T, int32_t d, int32_t W, int32_t io, int64_t x_ts) {
  const int rc = check_tokens(S, T, d, io);
  if (rc != MM_OK) return rc;
  if (W < 2 || W > MM_CONV_MAX_W) return MM_ERR_UNSUPPORTED;
  if (x_ts < d) return MM_ERR_DIM;
  if (d == 0) return MM_OK;
  const int64_t blocks = conv_groups(T, d) * conv_slices(d) + cdiv(S * d, kConvThreads);
  return blocks * kConvThreads > kMaxThreads || cdiv(int64_t{W + 1} * d, kPartColumns) * 256 > kMaxThreads ? MM_ERR_DIM : MM_OK;
}
// f(IO, channels of a lane, taps)
template <typename F>
int by_conv(int32_t io, int32_t d, int32_t W, F f) {
  return by_io(io, [&](auto t) {
    const auto taps = [&](auto v) {
      if (W == 2) return f(t, v, std::integral_constant<int, 2>{});
      if (W == 3) return f(t, v, std::integral_constant<int, 3>{});
      return f(t, v, std::integral_constant<int, 4>{});
    };
    switch (conv_channels(d)) {
      case 4: return taps(std::integral_constant<int, 4>{});
      case 2: return taps(std::integral_constant<int, 2>{});
      default: return taps(std::integral_constant<int, 1>{});
    }
  });
}
}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mamba_mixer_conv_prefill(const void* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                             const float* state_in, float* state_out, void* y, int32_t S, int64_t T, int32_t d,
                             int32_t W, int32_t silu, int32_t io_dtype, int64_t x_stride, void* stream) {
  int rc = check_conv(S, T, d, W, io_dtype, x_stride);
  if (rc != MM_OK) return rc;
  if (d == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  const int64_t ns = static_cast<int64_t>(S) * d * (W - 1);
  rc = check_args({strided(x, T, d, x_stride, es), flat(weight, static_cast<int64_t>(d) * W, 4), flat(bias, d, 4, true),
                   flat(cu_seqlens, S > 0 ? S + int64_t{1} : 0, 4), flat(state_in, ns, 4, true)},
                  {flat(state_out, ns, 4), flat(y, T * d, es)}, {{0, 4}});
  if (rc != MM_OK) return rc;
  if (S == 0) return MM_OK;
  const ConvArgs a{x, weight, bias, cu_seqlens, state_in, x_stride, T, S, d, static_cast<int>(conv_tokens(T, d)), silu != 0};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_conv(io_dtype, d, W, [&](auto io, auto v, auto taps) {
    using IO = decltype(io);
    constexpr int V = decltype(v)::value, K = decltype(taps)::value;
    const uint32_t slices = static_cast<uint32_t>(conv_slices(d));
    const int64_t blocks = T > 0 ? conv_groups(T, d) * slices : 0, states = cdiv(static_cast<int64_t>(S) * d, kConvThreads);
    const auto launch = [&](int64_t walks, int64_t rest) {
      hipLaunchKernelGGL((k_conv<IO, V, K>), dim3(static_cast<unsigned>(walks + rest)), dim3(kConvThreads), 0, st, a, walks, slices,
                         static_cast<IO*>(y), state_out);
    };
    if (state_out == state_in && blocks > 0) {  // in place: the initial states are read until the walks are through
      launch(blocks, 0);
      launch(0, states);
    } else {
      launch(blocks, states);
    }
    return launched();
  });
}

int mamba_mixer_conv_decode(const void* x, const float* weight, const float* bias, const float* state_in,
                            float* state_out, void* y, int32_t Bs, int32_t d, int32_t W, int32_t silu,
                            int32_t io_dtype, int64_t x_stride, void* stream) {
  int rc = check_conv(Bs, Bs, d, W, io_dtype, x_stride);
  if (rc != MM_OK) return rc;
  const int64_t n = static_cast<int64_t>(Bs) * d;
  if (n == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  rc = check_args({strided(x, Bs, d, x_stride, es), flat(weight, static_cast<int64_t>(d) * W, 4), flat(bias, d, 4, true),
                   flat(state_in, n * (W - 1), 4, true)},
                  {flat(state_out, n * (W - 1), 4), flat(y, n, es)}, {{0, 3}});
  if (rc != MM_OK) return rc;
  const ConvArgs a{x, weight, bias, nullptr, state_in, x_stride, Bs, Bs, d, 1, silu != 0};
  return by_conv(io_dtype, d, W, [&](auto io, auto v, auto taps) {
    using IO = decltype(io);
    constexpr int V = decltype(v)::value;
    hipLaunchKernelGGL((k_conv_decode<IO, V, decltype(taps)::value>), dim3(static_cast<unsigned>(cdiv(n, 256 * V))), dim3(256), 0,
                       static_cast<hipStream_t>(stream), a, state_out, static_cast<IO*>(y));
    return launched();
  });
}

size_t mamba_mixer_conv_backward_workspace_bytes(int64_t T, int32_t d, int32_t W) {
  if (check_conv(1, T, d, W, MM_IO_F32, d) != MM_OK || d == 0) return 0;
  return align256(static_cast<size_t>(conv_groups(T, d)) * d * (W + 1) * 4);
}

int mamba_mixer_conv_backward(const void* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                              const float* state_in, const void* dy, const float* dstate_out, void* dx,
                              float* dweight, float* dbias, float* dstate_in, int32_t S, int64_t T, int32_t d,
                              int32_t W, int32_t silu, int32_t io_dtype, int64_t x_stride, int64_t dx_stride,
                              void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_conv(S, T, d, W, io_dtype, x_stride);
  if (rc != MM_OK) return rc;
  if (dx_stride < d) return MM_ERR_DIM;
  if (d == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  const int64_t ns = static_cast<int64_t>(S) * d * (W - 1), nw = static_cast<int64_t>(d) * W;
  rc = check_args({strided(x, T, d, x_stride, es), flat(weight, nw, 4), flat(bias, d, 4, true),
                   flat(cu_seqlens, S > 0 ? S + int64_t{1} : 0, 4), flat(state_in, ns, 4, true), flat(dy, T * d, es),
                   flat(dstate_out, ns, 4, true)},
                  {strided(dx, T, d, dx_stride, es), flat(dweight, nw, 4), flat(dbias, bias != nullptr ? d : 0, 4),
                   flat(dstate_in, ns, 4, true)});
  if (rc != MM_OK) return rc;
  rc = check_workspace(workspace, workspace_bytes, mamba_mixer_conv_backward_workspace_bytes(T, d, W));
  if (rc != MM_OK) return rc;
  const ConvArgs a{x, weight, bias, cu_seqlens, state_in, x_stride, T, S, d, static_cast<int>(conv_tokens(T, d)), silu != 0};
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  return by_conv(io_dtype, d, W, [&](auto io, auto v, auto taps) {
    using IO = decltype(io);
    constexpr int V = decltype(v)::value, K = decltype(taps)::value;
    const uint32_t slices = static_cast<uint32_t>(conv_slices(d));
    const int64_t groups = T > 0 ? conv_groups(T, d) : 0, blocks = groups * slices;
    const int64_t states = dstate_in != nullptr ? cdiv(static_cast<int64_t>(S) * d, kConvThreads) : 0;
    if (blocks + states > 0)
      hipLaunchKernelGGL((k_conv_bwd<IO, V, K>), dim3(static_cast<unsigned>(blocks + states)), dim3(kConvThreads), 0, st, a, blocks,
                         slices, static_cast<const IO*>(dy), dstate_out, static_cast<IO*>(dx), dx_stride, part, dstate_in);
    hipLaunchKernelGGL(k_conv_parts, dim3(static_cast<unsigned>(cdiv(nw + d, kPartColumns))), dim3(256), 0, st, part, groups, d, W,
                       dweight, bias != nullptr ? dbias : nullptr);
    return launched();
  });
}

}  // extern "C"
