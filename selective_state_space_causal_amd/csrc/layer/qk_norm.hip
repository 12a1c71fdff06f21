// The norms of queries and keys with their rotation: kernels, argument checks and entry points.
//   u = weight v / sqrt(mean(v^2) + eps);  the pair (u_i, u_j) of number k turns by positions[t] inv_freq[k]
#include <algorithm>
#include <type_traits>

#include "layer/common.h"

namespace mm {
namespace {

struct QkArgs {
  const void *q, *k;
  const float *wq, *wk;
  const int32_t* pos;
  const float* freq;
  int64_t q_ts, k_ts, T;
  int Hq, Hk, D, R, inter;
  float eps;
};

// cos and sin of pos freq.  The turns are taken in 64 bits and their whole part dropped there.
__device__ __forceinline__ void qk_angle(int32_t pos, float freq, float& c, float& s) {
  const double turns = static_cast<double>(pos) * (static_cast<double>(freq) * 0.15915494309189535);
  sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
}
// ---------------------------------------------------------------- rows of 8 GP' columns
// A group of GP lanes takes a row (one token's head) at a time, a lane eight columns: two pieces of four that hold whole
// pairs.  The angles of a block of tokens are computed once for all of its heads and lie in LDS.  A group stays with its
// heads and walks over the block's tokens, kQkRows of them at a time so that loads are in flight.  Bound by memory: 16384 x
// (8 + 8) x 128 of bfloat16 are 134 MB in 27 us, 5 TB/s.  With 2 rows 29.6 for 28.8, backward 68 for 64.5; with 8 29.0 and
// 66; blocks of 8 or 32 tokens within 2%.
constexpr int kQkThreads = 256, kQkTokens = 16, kQkRows = 4;

struct QkAngles {
  float c[kQkTokens][MM_QK_MAX_D / 2], s[kQkTokens][MM_QK_MAX_D / 2];
};
__device__ __forceinline__ void qk_angles(const QkArgs& a, int64_t t0, int tokens, QkAngles& ang) {
  const int P = a.R / 2;
  for (int i = threadIdx.x; i < tokens * P; i += kQkThreads) {
    const int t = i / P, p = i - t * P;
    qk_angle(a.pos[t0 + t], a.freq[p], ang.c[t][p], ang.s[t][p]);
  }
}
// The places of a lane's columns: where its two pieces start, and its first pair.
struct QkPlace {
  int c0, c1, pair;
  bool on, turns;
};
template <bool INTER>
__device__ __forceinline__ QkPlace qk_place(const QkArgs& a, int lane) {
  QkPlace p;
  p.pair = 4 * lane;
  p.on = 8 * lane < a.D;
  p.turns = p.pair < a.R / 2;
  const int rest = (a.D - a.R) / 2;
  p.c0 = INTER ? 8 * lane : p.turns ? p.pair : a.R + p.pair - a.R / 2;
  p.c1 = INTER ? p.c0 + 4 : p.c0 + (p.turns ? a.R / 2 : rest);
  return p;
}
// v[0..3], v[4..7]: the lane's pieces; sign -1 turns back
template <bool INTER>
__device__ __forceinline__ void qk_turn(const QkPlace& p, const QkAngles& ang, int t, float sign, float (&v)[8]) {
  if (!p.turns) return;
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = ang.c[t][p.pair + i];
    s[i] = sign * ang.s[t][p.pair + i];
  }
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = __builtin_fmaf(x, c[i], -y * s[i]);
      v[2 * i + 1] = __builtin_fmaf(y, c[i], x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = v[i], y = v[i + 4];
      v[i] = __builtin_fmaf(x, c[i], -y * s[i]);
      v[i + 4] = __builtin_fmaf(y, c[i], x * s[i]);
    }
  }
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) { return v + __builtin_amdgcn_update_dpp(0.0f, v, CTRL, 0xF, 0xF, true); }
// the sum over a group's lanes, in all of them
template <int GP>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (GP >= 2) v = dpp_add<0xB1>(v);   // quad_perm 1 0 3 2
  if constexpr (GP >= 4) v = dpp_add<0x4E>(v);   // quad_perm 2 3 0 1
  if constexpr (GP >= 8) v = dpp_add<0x141>(v);  // row_half_mirror: the other four of eight
  if constexpr (GP >= 16) v = dpp_add<0x140>(v); // row_mirror: the other eight of sixteen
  if constexpr (GP >= 32) v += __shfl_xor(v, 16);
  return v;
}
// a lane's columns of a row: neighbours when interleaved, else two pieces
template <bool INTER, typename IO>
__device__ __forceinline__ void qk_load(const IO* row, const QkPlace& p, Chans<IO, 4>& lo, Chans<IO, 4>& hi) {
  if constexpr (INTER) {
    const Chans<IO, 8> v = load_chans<IO, 8>(global(row + p.c0), 0);
#pragma unroll
    for (int i = 0; i < Chans<IO, 4>::W; ++i) {
      lo.w[i] = v.w[i];
      hi.w[i] = v.w[Chans<IO, 4>::W + i];
    }
  } else {
    lo = load_chans<IO, 4>(global(row + p.c0), 0);
    hi = load_chans<IO, 4>(global(row + p.c1), 0);
  }
}
template <bool INTER, typename IO>
__device__ __forceinline__ void qk_store(IO* row, const QkPlace& p, const float (&v)[8]) {
  if constexpr (INTER) {
    store_chans<IO, 8>(global(row + p.c0), 0, v);
  } else {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    store_chans<IO, 4>(global(row + p.c0), 0, lo);
    store_chans<IO, 4>(global(row + p.c1), 0, hi);
  }
}

// Heads of one kind: how a workgroup's groups share them and the tokens.
struct QkShare {
  int head, heads, token, tokens;  // first head and token of this group, and their steps
};
template <int GP>
__device__ __forceinline__ QkShare qk_share(int H) {
  constexpr int groups = kQkThreads / GP;
  const int g = threadIdx.x / GP;
  int n = 1;
  while (n < H && n < groups) n *= 2;
  return {g % n, n, g / n, groups / n};
}

template <typename IO, int GP, bool INTER>
__global__ __launch_bounds__(kQkThreads) void k_qk_rows(QkArgs a, int block, IO* q_out, IO* k_out, int64_t qo_ts, int64_t ko_ts) {
  __shared__ QkAngles ang;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * block;
  const int tokens = static_cast<int>(a.T - t0 < block ? a.T - t0 : block);
  qk_angles(a, t0, tokens, ang);
  __syncthreads();
  const QkPlace p = qk_place<INTER>(a, threadIdx.x % GP);
  const float mean = 1.0f / a.D;
  const auto kind = [&](const IO* in, int64_t ts, IO* out, int64_t o_ts, const float* weight, int H) {
    const QkShare sh = qk_share<GP>(H);
    float w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = p.on ? weight[p.c0 + i] : 0.0f;
      w[i + 4] = p.on ? weight[p.c1 + i] : 0.0f;
    }
    for (int h = sh.head; h < H; h += sh.heads) {
      const IO* src = in + t0 * ts + static_cast<int64_t>(h) * a.D;
      IO* dst = out + t0 * o_ts + static_cast<int64_t>(h) * a.D;
      for (int t = sh.token; t < tokens; t += sh.tokens * kQkRows) {
        Chans<IO, 4> r0[kQkRows], r1[kQkRows];
#pragma unroll
        for (int j = 0; j < kQkRows; ++j) {
          const int tj = t + j * sh.tokens;
          r0[j] = r1[j] = Chans<IO, 4>{};
          if (p.on && tj < tokens) {
            qk_load<INTER>(src + tj * ts, p, r0[j], r1[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < kQkRows; ++j) {
          const int tj = t + j * sh.tokens;
          float v[8], s = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = r0[j][i];
            v[i + 4] = r1[j][i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) s = __builtin_fmaf(v[i], v[i], s);
          const float k = rsqrtf(__builtin_fmaf(group_sum<GP>(s), mean, a.eps));
          if (!p.on || tj >= tokens) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= k * w[i];
          qk_turn<INTER>(p, ang, tj, 1.0f, v);
          qk_store<INTER>(dst + tj * o_ts, p, v);
        }
      }
    }
  };
  kind(static_cast<const IO*>(a.q), a.q_ts, q_out, qo_ts, a.wq, a.Hq);
  kind(static_cast<const IO*>(a.k), a.k_ts, k_out, ko_ts, a.wk, a.Hk);
}

// With g the output's gradient turned back, n = v k and dn = g w:  dv = k (dn - n mean(dn n)),  dw = sum g n.  A workgroup
// takes blocks of tokens and leaves its sums of dw: part [2][parts][D], queries' and keys'.  8 x 2048 x (24 + 24) x 64 of
// bfloat16: 302 MB in 61 us, 4.9 TB/s; 256 workgroups 84 us for 64.5, 1024 67.
constexpr int kQkParts = 512;
template <typename IO, int GP, bool INTER>
__global__ __launch_bounds__(kQkThreads) void k_qk_rows_bwd(QkArgs a, int block, const IO* dqo, const IO* dko, IO* dq, IO* dk,
                                                            int64_t dq_ts, int64_t dk_ts, float* part) {
  __shared__ QkAngles ang;
  __shared__ float sums[kQkThreads / GP][8 * GP];
  const QkPlace p = qk_place<INTER>(a, threadIdx.x % GP);
  const float mean = 1.0f / a.D;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.0f;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * block; t0 < a.T; t0 += static_cast<int64_t>(gridDim.x) * block) {
    const int tokens = static_cast<int>(a.T - t0 < block ? a.T - t0 : block);
    __syncthreads();
    qk_angles(a, t0, tokens, ang);
    __syncthreads();
    const auto kind = [&](const IO* in, int64_t ts, const IO* dout, IO* out, int64_t o_ts, const float* weight, int H, float(&sum)[8]) {
      const QkShare sh = qk_share<GP>(H);
      float w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = p.on ? weight[p.c0 + i] : 0.0f;
        w[i + 4] = p.on ? weight[p.c1 + i] : 0.0f;
      }
      const int64_t g_ts = static_cast<int64_t>(H) * a.D;
      for (int h = sh.head; h < H; h += sh.heads) {
        const IO* src = in + t0 * ts + static_cast<int64_t>(h) * a.D;
        const IO* grad = dout + t0 * g_ts + static_cast<int64_t>(h) * a.D;
        IO* dst = out + t0 * o_ts + static_cast<int64_t>(h) * a.D;
        for (int t = sh.token; t < tokens; t += sh.tokens * kQkRows) {
          Chans<IO, 4> r0[kQkRows], r1[kQkRows], g0[kQkRows], g1[kQkRows];
#pragma unroll
          for (int j = 0; j < kQkRows; ++j) {
            const int tj = t + j * sh.tokens;
            r0[j] = r1[j] = g0[j] = g1[j] = Chans<IO, 4>{};
            if (p.on && tj < tokens) {
              qk_load<INTER>(src + tj * ts, p, r0[j], r1[j]);
              qk_load<INTER>(grad + tj * g_ts, p, g0[j], g1[j]);
            }
          }
#pragma unroll
          for (int j = 0; j < kQkRows; ++j) {
            const int tj = t + j * sh.tokens;
            float v[8], g[8], s = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = r0[j][i];
              v[i + 4] = r1[j][i];
              g[i] = g0[j][i];
              g[i + 4] = g1[j][i];
            }
            if (tj < tokens) qk_turn<INTER>(p, ang, tj, -1.0f, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              s = __builtin_fmaf(v[i], v[i], s);
              dot = __builtin_fmaf(g[i] * w[i], v[i], dot);
            }
            const float k = rsqrtf(__builtin_fmaf(group_sum<GP>(s), mean, a.eps)), m = group_sum<GP>(dot) * mean * k;
            if (!p.on || tj >= tokens) continue;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float n = v[i] * k;
              sum[i] = __builtin_fmaf(g[i], n, sum[i]);
              o[i] = k * __builtin_fmaf(g[i], w[i], -n * m);
            }
            qk_store<INTER>(dst + tj * o_ts, p, o);
          }
        }
      }
    };
    kind(static_cast<const IO*>(a.q), a.q_ts, dqo, dq, dq_ts, a.wq, a.Hq, dw[0]);
    kind(static_cast<const IO*>(a.k), a.k_ts, dko, dk, dk_ts, a.wk, a.Hk, dw[1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    __syncthreads();
    if (p.on) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sums[threadIdx.x / GP][p.c0 + i] = dw[n][i];
        sums[threadIdx.x / GP][p.c1 + i] = dw[n][i + 4];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kQkThreads) {
      float v = 0.0f;
#pragma unroll
      for (int g = 0; g < kQkThreads / GP; ++g) v += sums[g][i];
      part[(static_cast<int64_t>(n) * gridDim.x + blockIdx.x) * a.D + i] = v;
    }
  }
}

// ---------------------------------------------------------------- rows of any width
// A workgroup takes a token, its angles in LDS, a wave one head after another, its row in LDS: pairs may lie anywhere.  Bound
// by a row's chain of loads, sums and LDS; the backward's 512 workgroups take 591 us where 1024 take 341.
constexpr int kQkWaves = kQkThreads / 64, kQkCols = MM_QK_MAX_D / 64, kQkTokenParts = 1024;
struct QkToken {
  float c[MM_QK_MAX_D / 2], s[MM_QK_MAX_D / 2], row[kQkWaves][MM_QK_MAX_D];
};
__device__ __forceinline__ void qk_token_angles(const QkArgs& a, int64_t t, QkToken& tok) {
  __syncthreads();
  for (int p = threadIdx.x; p < a.R / 2; p += kQkThreads) qk_angle(a.pos[t], a.freq[p], tok.c[p], tok.s[p]);
  __syncthreads();
}
// Column i of the row u, turned: (first, second) by (cos, sin); sign -1 turns back.
__device__ __forceinline__ float qk_turned(const QkArgs& a, const QkToken& tok, const float* u, int i, float sign) {
  if (i >= a.R) return u[i];
  const bool first = a.inter ? i % 2 == 0 : i < a.R / 2;
  const int mate = a.inter ? i ^ 1 : first ? i + a.R / 2 : i - a.R / 2, pair = a.inter ? i / 2 : first ? i : mate;
  const float s = sign * tok.s[pair];
  return __builtin_fmaf(u[i], tok.c[pair], first ? -u[mate] * s : u[mate] * s);
}
// Between a row's stores to LDS and its loads by other lanes of the wave, and before the next row's stores: the fences keep the
// accesses in the program's order.  They cost no instruction, as a wave's accesses to LDS run in order.
__device__ __forceinline__ void qk_row_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}
__device__ __forceinline__ float wave_sum(float v) { return group_sum<32>(v) + __shfl_xor(group_sum<32>(v), 32); }

template <typename IO>
__global__ __launch_bounds__(kQkThreads) void k_qk(QkArgs a, IO* q_out, IO* k_out, int64_t qo_ts, int64_t ko_ts) {
  __shared__ QkToken tok;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  float* const u = tok.row[wave];
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    qk_token_angles(a, t, tok);
    for (int h = wave; h < a.Hq + a.Hk; h += kQkWaves) {
      const bool key = h >= a.Hq;
      const int64_t at = static_cast<int64_t>(key ? h - a.Hq : h) * a.D;
      const IO* v = static_cast<const IO*>(key ? a.k : a.q) + t * (key ? a.k_ts : a.q_ts) + at;
      IO* out = (key ? k_out : q_out) + t * (key ? ko_ts : qo_ts) + at;
      const float* w = key ? a.wk : a.wq;
      float x[kQkCols], s = 0.0f;
#pragma unroll
      for (int e = 0; e < kQkCols; ++e) {
        const int i = lane + 64 * e;
        x[e] = i < a.D ? ld_io(v, i) : 0.0f;
        s = __builtin_fmaf(x[e], x[e], s);
      }
      const float r = rsqrtf(wave_sum(s) / a.D + a.eps);
      qk_row_order();
#pragma unroll
      for (int e = 0; e < kQkCols; ++e) {
        const int i = lane + 64 * e;
        if (i < a.D) u[i] = x[e] * r * w[i];
      }
      qk_row_order();
#pragma unroll
      for (int e = 0; e < kQkCols; ++e) {
        const int i = lane + 64 * e;
        if (i < a.D) st_io(out, i, qk_turned(a, tok, u, i, 1.0f));
      }
    }
  }
}

template <typename IO>
__global__ __launch_bounds__(kQkThreads) void k_qk_bwd(QkArgs a, const IO* dqo, const IO* dko, IO* dq, IO* dk, int64_t dq_ts,
                                                       int64_t dk_ts, float* part) {
  __shared__ QkToken tok;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  float* const u = tok.row[wave];
  float dw[2][kQkCols] = {};
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    qk_token_angles(a, t, tok);
    const auto kind = [&](const IO* in, int64_t ts, const IO* dout, IO* out, int64_t o_ts, const float* w, int H, float(&sum)[kQkCols]) {
      for (int h = wave; h < H; h += kQkWaves) {
        const IO* v = in + t * ts + static_cast<int64_t>(h) * a.D;
        const IO* go = dout + (t * H + h) * a.D;
        qk_row_order();
#pragma unroll
        for (int e = 0; e < kQkCols; ++e) {
          const int i = lane + 64 * e;
          if (i < a.D) u[i] = ld_io(go, i);
        }
        qk_row_order();
        float s = 0.0f, dot = 0.0f, g[kQkCols], x[kQkCols];
#pragma unroll
        for (int e = 0; e < kQkCols; ++e) {
          const int i = lane + 64 * e;
          x[e] = g[e] = 0.0f;
          if (i < a.D) {
            x[e] = ld_io(v, i);
            g[e] = qk_turned(a, tok, u, i, -1.0f);
            s = __builtin_fmaf(x[e], x[e], s);
            dot = __builtin_fmaf(g[e] * w[i], x[e], dot);
          }
        }
        const float r = rsqrtf(wave_sum(s) / a.D + a.eps), m = wave_sum(dot) * r / a.D;
        IO* o = out + t * o_ts + static_cast<int64_t>(h) * a.D;
#pragma unroll
        for (int e = 0; e < kQkCols; ++e) {
          const int i = lane + 64 * e;
          if (i < a.D) {
            const float n = x[e] * r;
            sum[e] = __builtin_fmaf(g[e], n, sum[e]);
            st_io(o, i, r * (g[e] * w[i] - n * m));
          }
        }
      }
    };
    kind(static_cast<const IO*>(a.q), a.q_ts, dqo, dq, dq_ts, a.wq, a.Hq, dw[0]);
    kind(static_cast<const IO*>(a.k), a.k_ts, dko, dk, dk_ts, a.wk, a.Hk, dw[1]);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kQkCols; ++e) u[lane + 64 * e] = dw[n][e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kQkThreads) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kQkWaves; ++k) v += tok.row[k][i];
      part[(static_cast<int64_t>(n) * gridDim.x + blockIdx.x) * a.D + i] = v;
    }
  }
}
// dwq, dwk from `parts` rows each
__global__ __launch_bounds__(256) void k_qk_parts(const float* __restrict__ part, int64_t parts, int D, float* __restrict__ dwq,
                                                  float* __restrict__ dwk) {
  const int i = blockIdx.x * kPartColumns + threadIdx.x % kPartColumns;
  const float v = sum_parts(part + blockIdx.y * parts * D, parts, D, i);
  if (i < D && threadIdx.x < kPartColumns) (blockIdx.y == 0 ? dwq : dwk)[i] = v;
}

// Whole pairs lie in pieces of four columns where D and R are multiples of eight; the rest goes row by row through LDS
// (16384 x (8 + 8) x 128 102 us for 28.8, backward 8 x 2048 x (24 + 24) x 64 341 for 64.5).
bool qk_by_groups(int D, int R) { return D % 8 == 0 && R % 8 == 0; }
// tokens of a block: fewer where the blocks would not fill the GPU
int qk_block(int64_t T) { return static_cast<int>(std::min<int64_t>(kQkTokens, std::max<int64_t>(1, T / 1024))); }
int64_t qk_parts(int64_t T, int D, int R) {
  return qk_by_groups(D, R) ? std::min<int64_t>(kQkParts, cdiv(T, qk_block(T))) : std::min<int64_t>(kQkTokenParts, T);
}
// f(lanes of a group, interleaved)
template <typename F>
void by_group(int D, bool inter, F f) {
  const int n = D / 8;
  const auto go = [&](auto lanes) {
    if (inter) f(lanes, std::true_type{});
    else f(lanes, std::false_type{});
  };
  if (n <= 1) go(std::integral_constant<int, 1>{});
  else if (n <= 2) go(std::integral_constant<int, 2>{});
  else if (n <= 4) go(std::integral_constant<int, 4>{});
  else if (n <= 8) go(std::integral_constant<int, 8>{});
  else if (n <= 16) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
}

int check_qk(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, float eps, int32_t io) {
  if (T < 0 || Hq < 1 || Hk < 1 || R < 0 || R % 2 != 0 || !(eps >= 0.0f)) return MM_ERR_DIM;
  if ((io != MM_IO_F32 && io != MM_IO_BF16) || D < 1 || D > MM_QK_MAX_D) return MM_ERR_UNSUPPORTED;
  if (R > D || T > INT32_MAX / (static_cast<int64_t>(Hq) + Hk)) return MM_ERR_DIM;
  return MM_OK;
}
}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

int mamba_mixer_qk_norm(const void* q, const void* k, const float* q_weight, const float* k_weight,
                        const int32_t* positions, const float* inv_freq, void* q_out, void* k_out, int64_t T,
                        int32_t Hq, int32_t Hk, int32_t D, int32_t R, float eps, int32_t interleaved, int32_t io_dtype,
                        int64_t q_stride, int64_t k_stride, int64_t qo_stride, int64_t ko_stride, void* stream) {
  int rc = check_qk(T, Hq, Hk, D, R, eps, io_dtype);
  if (rc != MM_OK) return rc;
  const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
  if (q_stride < wq || qo_stride < wq || k_stride < wk || ko_stride < wk) return MM_ERR_DIM;
  if (T == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  rc = check_args({strided(q, T, wq, q_stride, es), strided(k, T, wk, k_stride, es), flat(q_weight, D, 4), flat(k_weight, D, 4),
                   flat(positions, R > 0 ? T : 0, 4), flat(inv_freq, R / 2, 4)},
                  {strided(q_out, T, wq, qo_stride, es), strided(k_out, T, wk, ko_stride, es)}, {{0, 0}, {1, 1}});
  if (rc != MM_OK) return rc;
  const QkArgs a{q, k, q_weight, k_weight, positions, inv_freq, q_stride, k_stride, T, Hq, Hk, D, R, interleaved != 0, eps};
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (qk_by_groups(D, R)) {
      const int block = qk_block(T);
      const int64_t most = (kMaxThreads / kQkThreads) * block;  // tokens of a launch
      by_group(D, interleaved != 0, [&](auto n, auto inter) {
        for (int64_t t0 = 0; t0 < T; t0 += most) {
          QkArgs b = a;
          b.q = static_cast<const IO*>(q) + t0 * q_stride;
          b.k = static_cast<const IO*>(k) + t0 * k_stride;
          b.pos = R > 0 ? positions + t0 : nullptr;
          b.T = std::min(most, T - t0);
          const dim3 grid(static_cast<unsigned>(cdiv(b.T, block)));
          hipLaunchKernelGGL((k_qk_rows<IO, decltype(n)::value, decltype(inter)::value>), grid, dim3(kQkThreads), 0, st, b, block,
                             static_cast<IO*>(q_out) + t0 * qo_stride, static_cast<IO*>(k_out) + t0 * ko_stride, qo_stride, ko_stride);
        }
      });
    } else {
      hipLaunchKernelGGL((k_qk<IO>), dim3(static_cast<unsigned>(std::min<int64_t>(T, 1 << 16))), dim3(kQkThreads), 0, st, a,
                         static_cast<IO*>(q_out), static_cast<IO*>(k_out), qo_stride, ko_stride);
    }
    return launched();
  });
}

size_t mamba_mixer_qk_norm_backward_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
  if (check_qk(T, Hq, Hk, D, 0, 0.0f, MM_IO_F32) != MM_OK) return 0;
  return align256(static_cast<size_t>(2) * std::max(kQkParts, kQkTokenParts) * D * 4);
}

int mamba_mixer_qk_norm_backward(const void* dq_out, const void* dk_out, const void* q, const void* k,
                                 const float* q_weight, const float* k_weight, const int32_t* positions,
                                 const float* inv_freq, void* dq, void* dk, float* dq_weight, float* dk_weight,
                                 int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, float eps,
                                 int32_t interleaved, int32_t io_dtype, int64_t q_stride, int64_t k_stride,
                                 int64_t dq_stride, int64_t dk_stride, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  int rc = check_qk(T, Hq, Hk, D, R, eps, io_dtype);
  if (rc != MM_OK) return rc;
  const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hk) * D;
  if (q_stride < wq || dq_stride < wq || k_stride < wk || dk_stride < wk) return MM_ERR_DIM;
  const size_t es = esize(io_dtype);
  rc = check_args({flat(dq_out, T * wq, es), flat(dk_out, T * wk, es), strided(q, T, wq, q_stride, es),
                   strided(k, T, wk, k_stride, es), flat(q_weight, D, 4), flat(k_weight, D, 4),
                   flat(positions, R > 0 ? T : 0, 4), flat(inv_freq, R / 2, 4)},
                  {strided(dq, T, wq, dq_stride, es), strided(dk, T, wk, dk_stride, es), flat(dq_weight, D, 4),
                   flat(dk_weight, D, 4)});
  if (rc != MM_OK) return rc;
  rc = check_workspace(workspace, workspace_bytes, mamba_mixer_qk_norm_backward_workspace_bytes(T, Hq, Hk, D));
  if (rc != MM_OK) return rc;
  const QkArgs a{q, k, q_weight, k_weight, positions, inv_freq, q_stride, k_stride, T, Hq, Hk, D, R, interleaved != 0, eps};
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    const int64_t parts = qk_parts(T, D, R);
    if (T > 0 && qk_by_groups(D, R)) {
      by_group(D, interleaved != 0, [&](auto n, auto inter) {
        const dim3 grid(static_cast<unsigned>(parts));
        hipLaunchKernelGGL((k_qk_rows_bwd<IO, decltype(n)::value, decltype(inter)::value>), grid, dim3(kQkThreads), 0, st, a, qk_block(T),
                           static_cast<const IO*>(dq_out), static_cast<const IO*>(dk_out), static_cast<IO*>(dq),
                           static_cast<IO*>(dk), dq_stride, dk_stride, part);
      });
    } else if (T > 0) {
      hipLaunchKernelGGL((k_qk_bwd<IO>), dim3(static_cast<unsigned>(parts)), dim3(kQkThreads), 0, st, a, static_cast<const IO*>(dq_out),
                         static_cast<const IO*>(dk_out), static_cast<IO*>(dq), static_cast<IO*>(dk), dq_stride, dk_stride, part);
    }
    hipLaunchKernelGGL(k_qk_parts, dim3(static_cast<unsigned>(cdiv(D, kPartColumns)), 2), dim3(256), 0, st, part, parts, D, dq_weight,
                       dk_weight);
    return launched();
  });
}

}  // extern "C"
