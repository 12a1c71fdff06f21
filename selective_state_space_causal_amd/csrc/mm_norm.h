// The norms around a mixer block, one pass over their rows:
//   gate_norm       s = z sigmoid(z);  gate first: out = w n(y s),  gate last: out = w n(y) s,
//                   n(u) = u rsqrt(mean(u^2) + eps) over each of `groups` equal column ranges
//   residual_norm   p = h or w_post n(h);  r' = r + scale scale_vec p;  out = w n(r')
// and their gradients.  All arithmetic is float32; the outputs are rounded once.
//
// Bound by memory.  A workgroup takes a (row, group) at a time, E neighbouring columns per thread and NV
// such pieces, in registers from the load to the store: every array is read and written once.
// The next row is loaded before this one's sums are taken.  In the backward a workgroup keeps to one
// column range over all its rows, so the weights' gradients gather in registers too and leave as one
// partial sum per workgroup, added in a fixed order by k_norm_parts.
// Rows may start anywhere: wide accesses need no alignment here, and a row's last piece is taken
// element by element.
// Measured, as the fraction of a plain copy's 6.2 TB/s: gate_norm 16384 x 4096 75 us (0.88), residual_norm
// 16384 x 2048 with a float32 residual 73 us (0.91); their backward 8192 x 5120 in 8 groups 88 us (0.78: VALU issue 70%,
// two exponential-class operations an element and 17% idle lanes) and 8191 x 2560 89 us (0.70: a row is one barrier and
// twelve loaded bytes a column, then its stores; 6 us of it add up the weights' partial sums).
#pragma once

#include "mm_device.h"

namespace mm {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormUnit = kNormMaxThreads * 8;  // columns that fit: 8 for each thread

// E (8 or 4) neighbouring elements as loaded
template <typename IO, int E>
struct Raw {
  static constexpr int W = E * sizeof(IO) / 4;
  typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(sizeof(IO))));
  vec v;
};
// n: how many exist (the others read as zeros)
template <int E, typename IO>
__device__ __forceinline__ Raw<IO, E> load_raw(const IO* p, int n) {
  typedef Raw<IO, E> R;
  R r;
  if (n >= E) {
    if constexpr (R::W > 4) {  // float32: two 16-byte loads
      typedef uint32_t half __attribute__((ext_vector_type(4), aligned(4)));
      const half a = *reinterpret_cast<const half*>(p), b = *reinterpret_cast<const half*>(p + E / 2);
      r.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      r.v = *reinterpret_cast<const typename R::vec*>(p);
    }
    return r;
  }
#pragma unroll
  for (int i = 0; i < R::W; ++i) r.v[i] = 0;
#pragma unroll
  for (int i = 0; i < E - 1; ++i)
    if (i < n) {
      if constexpr (sizeof(IO) == 2) r.v[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i % 2));
      else r.v[i] = __float_as_uint(p[i]);
    }
  return r;
}
template <int E>
__device__ __forceinline__ float get(const Raw<uint16_t, E>& r, int i) {
  return __uint_as_float(i % 2 ? r.v[i / 2] & 0xFFFF0000u : r.v[i / 2] << 16);
}
template <int E>
__device__ __forceinline__ float get(const Raw<float, E>& r, int i) { return __uint_as_float(r.v[i]); }
template <int E>
__device__ __forceinline__ void set(Raw<float, E>& r, int i, float v) { r.v[i] = __float_as_uint(v); }
template <int E>
__device__ __forceinline__ void store_raw(uint16_t* p, int n, const float (&v)[E]) {
  typedef __bf16 bE __attribute__((ext_vector_type(E)));
  typedef float fE __attribute__((ext_vector_type(E)));
  typedef typename Raw<uint16_t, E>::vec vec;
  fE f;
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = v[i];
  const vec u = __builtin_bit_cast(vec, __builtin_convertvector(f, bE));  // round to nearest even
  if (n >= E) {
    *reinterpret_cast<vec*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < E - 1; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i % 2)));
  }
}
template <int E>
__device__ __forceinline__ void store_raw(float* p, int n, const float (&v)[E]) {
  typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
  if (n >= E) {
#pragma unroll
    for (int i = 0; i < E; i += 4) *reinterpret_cast<f4*>(p + i) = f4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < E - 1; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Sums of K values over the workgroup, in every thread; LDS for two calls in turn, so that one barrier
// serves each.  Within a wave by DPP (a row of 16, then rows broadcast into the next ones: lane 63 has all);
// each lane then reads one wave's sum, not every lane all of them: with ten waves and six sums those reads
// alone took a third of the time.
struct NormRed {
  float s[2][6][kNormMaxThreads / kWave];
};
template <int K>
__device__ __forceinline__ void group_sums(float (&v)[K], NormRed& red, int& turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = row_sum16(v[k]);
    v[k] += __builtin_amdgcn_update_dpp(0.0f, v[k], 0x142, 0xA, 0xF, false);  // row_bcast:15, rows 1 and 3
    v[k] += __builtin_amdgcn_update_dpp(0.0f, v[k], 0x143, 0xC, 0xF, false);  // row_bcast:31, rows 2 and 3
  }
  const int waves = blockDim.x / kWave, lane = threadIdx.x & 63;
  if (waves == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      v[k] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v[k]), 63));
    return;
  }
  if (lane == 63)
#pragma unroll
    for (int k = 0; k < K; ++k) red.s[turn][k][threadIdx.x >> 6] = v[k];
  __syncthreads();
  const int w = lane & 15;
  static_assert(kNormMaxThreads / kWave <= 16, "one lane of a row for each wave");
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = row_sum16(w < waves ? red.s[turn][k][w] : 0.0f);
  turn ^= 1;
}
__device__ __forceinline__ float sigmoid(float z) { return rcp_hw(1.0f + exp2_hw(-z * kLog2e)); }

template <typename IO>
struct GateArgs {
  const IO *y, *z, *dout;
  int64_t y_ts, z_ts;
  const float* w;
  int64_t rows;
  int d, groups;
  float eps;
  int gate_first;
};

// Workgroups b, b + groups, ...: the rows b / groups, b / groups + slots, ... of group b % groups.
template <typename IO, int E, int NV, bool FIRST>
__global__ __launch_bounds__(kNormMaxThreads) void k_gate_norm(GateArgs<IO> a, IO* __restrict__ out) {
  __shared__ NormRed red;
  int turn = 0;
  const int n = a.d / a.groups, g = blockIdx.x % a.groups, T = blockDim.x;
  const int64_t slots = gridDim.x / a.groups;
  Raw<float, E> w[NV];
  Raw<IO, E> y[NV], z[NV];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      y[i] = load_raw<E>(a.y + row * a.y_ts + g * n + c, n - c);
      z[i] = load_raw<E>(a.z + row * a.z_ts + g * n + c, n - c);
    }
  };
  int64_t row = blockIdx.x / a.groups;
  load(row);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    w[i] = load_raw<E>(a.w + g * n + c, n - c);
  }
  for (; row < a.rows; row += slots) {
    float v[NV][E], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float yv = get(y[i], e), zv = get(z[i], e);
        v[i][e] = yv * (zv * sigmoid(zv));
        const float u = FIRST ? v[i][e] : yv;
        sum[0] = __builtin_fmaf(u, u, sum[0]);
      }
    if (row + slots < a.rows) load(row + slots);
    group_sums(sum, red, turn);
    const float k = rsqrtf(sum[0] / n + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] *= k * get(w[i], e);
      if (c < n) store_raw<E>(out + row * a.d + g * n + c, n - c, v[i]);
    }
  }
}

// With u = y s (gate first) or y, n = u k, k = rsqrt(mean(u^2) + eps) and dn = dout w (times s, gate last):
//   du = k (dn - n mean(dn n));  first: dy = du s, dz = du y s';  last: dy = du, dz = dout w n s'
// part: [slots, d] partial sums of dw.
template <typename IO, int E, int NV, bool FIRST>
__global__ __launch_bounds__(kNormMaxThreads) void k_gate_norm_bwd(GateArgs<IO> a, IO* __restrict__ dy, IO* __restrict__ dz,
                                                                   int64_t dy_ts, int64_t dz_ts,
                                                                   float* __restrict__ part) {
  __shared__ NormRed red;
  int turn = 0;
  const int n = a.d / a.groups, g = blockIdx.x % a.groups, T = blockDim.x;
  const int64_t slots = gridDim.x / a.groups;
  Raw<float, E> w[NV];
  Raw<IO, E> y[NV], z[NV], go[NV];
  float dw[NV][E];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      y[i] = load_raw<E>(a.y + row * a.y_ts + g * n + c, n - c);
      z[i] = load_raw<E>(a.z + row * a.z_ts + g * n + c, n - c);
      go[i] = load_raw<E>(a.dout + row * a.d + g * n + c, n - c);
    }
  };
  int64_t row = blockIdx.x / a.groups;
  load(row);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    w[i] = load_raw<E>(a.w + g * n + c, n - c);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[i][e] = 0.0f;
  }
  for (; row < a.rows; row += slots) {
    Raw<IO, E> yr[NV], zr[NV], gr[NV];
    float sg[NV][E];  // sigmoid(z): its exponential and reciprocal are the costly part, taken once
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      yr[i] = y[i];
      zr[i] = z[i];
      gr[i] = go[i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float zv = get(zr[i], e), yv = get(yr[i], e);
        sg[i][e] = sigmoid(zv);
        const float s = zv * sg[i][e];
        const float u = FIRST ? yv * s : yv, gw = get(gr[i], e) * get(w[i], e);
        sum[0] = __builtin_fmaf(u, u, sum[0]);
        sum[1] = __builtin_fmaf(gw * s, yv, sum[1]);  // dn u, either way
      }
    }
    if (row + slots < a.rows) load(row + slots);
    group_sums(sum, red, turn);
    const float k = rsqrtf(sum[0] / n + a.eps);
    const float km = k * k * (sum[1] / n);  // k mean(dn n): n mean(dn n) = u km
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      float oy[E], oz[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float zv = get(zr[i], e), g1 = sg[i][e], s = zv * g1, ds = g1 * (1.0f + zv * (1.0f - g1));
        const float yv = get(yr[i], e), gv = get(gr[i], e), gw = gv * get(w[i], e);
        if (FIRST) {
          const float du = k * (gw - yv * s * km);
          oy[e] = du * s;
          oz[e] = du * yv * ds;
        } else {
          oy[e] = k * (gw * s - yv * km);
          oz[e] = gw * yv * k * ds;
        }
        dw[i][e] = __builtin_fmaf(gv * k, yv * s, dw[i][e]);
      }
      if (c < n) {
        store_raw<E>(dy + row * dy_ts + g * n + c, n - c, oy);
        store_raw<E>(dz + row * dz_ts + g * n + c, n - c, oz);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    if (c < n) store_raw<E>(part + static_cast<int64_t>(blockIdx.x / a.groups) * a.d + g * n + c, n - c, dw[i]);
  }
}

// out[c] = the sum of part[i][c] over i: 16 columns per workgroup, 16 threads for each, in a fixed order
struct NormParts {
  const float* part[3];
  float* out[3];
};
__global__ __launch_bounds__(256) void k_norm_parts(NormParts p, int parts, int64_t stride, int d) {
  __shared__ float s[16][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
  const float* part = p.part[blockIdx.y];
  float v = 0.0f;
  if (c < d) {
    int i = r;
    for (; i + 112 < parts; i += 128) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = part[(i + 16 * k) * stride + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += t[k];
    }
    for (; i < parts; i += 16) v += part[i * stride + c];
  }
  s[r][threadIdx.x & 15] = v;
  __syncthreads();
  if (r == 0 && c < d) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += s[k][threadIdx.x & 15];
    p.out[blockIdx.y][c] = t;
  }
}

template <typename IO, typename RES>
struct ResArgs {
  const IO* h;
  const RES* res;  // the residual before (forward) or after (backward) the addition; forward: may be NULL
  const float *w, *wp, *vec;
  float scale, eps;
  int64_t rows;
  int d;
};
// E of a per-column parameter; ones where there is none
template <int E>
__device__ __forceinline__ Raw<float, E> load_or_one(const float* p, int c, int n) {
  if (p != nullptr) return load_raw<E>(p + c, n);
  Raw<float, E> r;
#pragma unroll
  for (int i = 0; i < E; ++i) set(r, i, 1.0f);
  return r;
}

template <typename IO, typename RES, int E, int NV>
__global__ __launch_bounds__(kNormMaxThreads) void k_residual_norm(ResArgs<IO, RES> a, RES* __restrict__ res_out,
                                                                   IO* __restrict__ out) {
  __shared__ NormRed red;
  int turn = 0;
  const int n = a.d, T = blockDim.x;
  Raw<float, E> w[NV], f[NV];  // f: everything that multiplies h's norm
  Raw<IO, E> h[NV];
  Raw<RES, E> res[NV];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      h[i] = load_raw<E>(a.h + row * n + c, n - c);
      res[i] = load_raw<E>(a.res + (a.res != nullptr ? row * n + c : 0), a.res != nullptr ? n - c : 0);
    }
  };
  int64_t row = blockIdx.x;
  load(row);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    w[i] = load_raw<E>(a.w + c, n - c);
    f[i] = load_or_one<E>(a.wp, c, n - c);
    const Raw<float, E> v = load_or_one<E>(a.vec, c, n - c);
#pragma unroll
    for (int e = 0; e < E; ++e) set(f[i], e, get(f[i], e) * (a.scale * get(v, e)));
  }
  for (; row < a.rows; row += gridDim.x) {
    float kp = 1.0f;
    if (a.wp != nullptr) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) sum[0] = __builtin_fmaf(get(h[i], e), get(h[i], e), sum[0]);
      group_sums(sum, red, turn);
      kp = rsqrtf(sum[0] / n + a.eps);
    }
    float r[NV][E], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[i][e] = __builtin_fmaf(get(h[i], e) * kp, get(f[i], e), get(res[i], e));
        sum[0] = __builtin_fmaf(r[i][e], r[i][e], sum[0]);
      }
    if (row + gridDim.x < a.rows) load(row + gridDim.x);
    group_sums(sum, red, turn);
    const float k = rsqrtf(sum[0] / n + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      if (c < n) store_raw<E>(res_out + row * n + c, n - c, r[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) r[i][e] *= k * get(w[i], e);
      if (c < n) store_raw<E>(out + row * n + c, n - c, r[i]);
    }
  }
}

// With r the new residual, k = rsqrt(mean(r^2) + eps), n = r k and dn = dout w:
//   dr = dr' + k (dn - n mean(dn n)),  dp = scale vec dr,  and through the norm of h, kp = rsqrt(mean(h^2) + eps):
//   dh = kp (dp wp - h kp^2 mean(dp wp h))          (without wp: dh = dp)
// part: per slot the partial sums of dw = dout n, dwp = dp h kp and dvec = scale dr p.
template <typename IO, typename RES, int E, int NV>
__global__ __launch_bounds__(kNormMaxThreads) void k_residual_norm_bwd(ResArgs<IO, RES> a, const IO* __restrict__ dout,
                                                                       const RES* dres_out, RES* dres,
                                                                       IO* __restrict__ dh, float* __restrict__ part) {
  __shared__ NormRed red;
  int turn = 0;
  const int n = a.d, T = blockDim.x;
  const bool post = a.wp != nullptr;
  Raw<float, E> w[NV], wp[NV], vec[NV];
  Raw<IO, E> h[NV], go[NV];
  Raw<RES, E> res[NV], up[NV];
  float acc[3][NV][E];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      h[i] = load_raw<E>(a.h + row * n + c, n - c);
      go[i] = load_raw<E>(dout + row * n + c, n - c);
      res[i] = load_raw<E>(a.res + row * n + c, n - c);
      up[i] = load_raw<E>(dres_out + (dres_out != nullptr ? row * n + c : 0), dres_out != nullptr ? n - c : 0);
    }
  };
  constexpr bool kAhead = NV == 1;  // the next row's loads wait in registers, where there are enough
  int64_t row = blockIdx.x;
  if (kAhead) load(row);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    w[i] = load_raw<E>(a.w + c, n - c);
    wp[i] = load_or_one<E>(a.wp, c, n - c);
    vec[i] = load_or_one<E>(a.vec, c, n - c);
#pragma unroll
    for (int e = 0; e < E; ++e) set(vec[i], e, get(vec[i], e) * a.scale);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[0][i][e] = acc[1][i][e] = acc[2][i][e] = 0.0f;
  }
  for (; row < a.rows; row += gridDim.x) {
    if (!kAhead) load(row);
    // r^2, w g r, h^2 and the three parts of dr f h (f = vec w_p), so that one reduction serves both norms
    float sum[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    Raw<IO, E> hr[NV], gr[NV];
    Raw<RES, E> rr[NV], ur[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      hr[i] = h[i];
      gr[i] = go[i];
      rr[i] = res[i];
      ur[i] = up[i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float rv = get(res[i], e), hv = get(h[i], e), gw = get(go[i], e) * get(w[i], e);
        sum[0] = __builtin_fmaf(rv, rv, sum[0]);
        sum[1] = __builtin_fmaf(gw, rv, sum[1]);
        if (post) {
          const float fh = get(vec[i], e) * get(wp[i], e) * hv;
          sum[2] = __builtin_fmaf(hv, hv, sum[2]);
          sum[3] = __builtin_fmaf(get(up[i], e), fh, sum[3]);
          sum[4] = __builtin_fmaf(gw, fh, sum[4]);
          sum[5] = __builtin_fmaf(rv, fh, sum[5]);
        }
      }
    }
    if (kAhead && row + gridDim.x < a.rows) load(row + gridDim.x);
    float kp = 1.0f, m = 0.0f;
    if (post) {
      group_sums(sum, red, turn);
    } else {
      float two[2] = {sum[0], sum[1]};
      group_sums(two, red, turn);
      sum[0] = two[0];
      sum[1] = two[1];
    }
    const float k = rsqrtf(sum[0] / n + a.eps), km = k * k * (sum[1] / n);
    if (post) {
      kp = rsqrtf(sum[2] / n + a.eps);
      m = kp * kp * ((sum[3] + k * (sum[4] - km * sum[5])) / n);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * T + threadIdx.x) * E;
      float dr[E], gh[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float rv = get(rr[i], e), gv = get(gr[i], e), hv = get(hr[i], e);
        dr[e] = get(ur[i], e) + k * (gv * get(w[i], e) - rv * km);
        const float dp = dr[e] * get(vec[i], e), hk = hv * kp;
        acc[0][i][e] = __builtin_fmaf(gv, rv * k, acc[0][i][e]);
        acc[1][i][e] = __builtin_fmaf(dp, hk, acc[1][i][e]);
        // scale dr p; the parameter may be zero, so not dp p / vec
        acc[2][i][e] = __builtin_fmaf(a.scale * dr[e], hk * get(wp[i], e), acc[2][i][e]);
        gh[e] = post ? kp * (dp * get(wp[i], e) - hv * m) : dp;
      }
      if (c < n) {
        store_raw<E>(dres + row * n + c, n - c, dr);
        store_raw<E>(dh + row * n + c, n - c, gh);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * T + threadIdx.x) * E;
    if (c < n)
#pragma unroll
      for (int k = 0; k < 3; ++k) store_raw<E>(part + (static_cast<int64_t>(blockIdx.x) * 3 + k) * n + c, n - c, acc[k][i]);
  }
}

// ------------------------------------------------------------------------------------ wide rows
// Units of more than 8192 columns do not fit the registers: 256 threads walk the row once for its sums and
// again for its outputs (from the caches), and the weights' gradients are sums down the columns, in a kernel
// of their own, from the rows' saved factors.
constexpr int kWideThreads = 256;
constexpr int kWideParts = 256;  // row ranges of the weight gradients' sums
struct WideRed {
  float s[4];
};
__device__ __forceinline__ float wide_sum(float v, WideRed& red) {
  v = row_sum16(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red.s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red.s[0] + red.s[1]) + (red.s[2] + red.s[3]);
}

template <typename IO>
__global__ __launch_bounds__(kWideThreads) void k_wide_gate_norm(GateArgs<IO> a, IO* __restrict__ out) {
  __shared__ WideRed red;
  const int n = a.d / a.groups, g = blockIdx.x % a.groups;
  const int64_t row = blockIdx.x / a.groups;
  const IO *y = a.y + row * a.y_ts + g * n, *z = a.z + row * a.z_ts + g * n;
  float ss = 0.0f;
  for (int i = threadIdx.x; i < n; i += kWideThreads) {
    const float zv = ld_io(z, i);
    const float u = a.gate_first ? ld_io(y, i) * (zv * sigmoid(zv)) : ld_io(y, i);
    ss = __builtin_fmaf(u, u, ss);
  }
  const float k = rsqrtf(wide_sum(ss, red) / n + a.eps);
  for (int i = threadIdx.x; i < n; i += kWideThreads) {
    const float zv = ld_io(z, i);
    st_io(out, row * a.d + g * n + i, ld_io(y, i) * (zv * sigmoid(zv)) * k * a.w[g * n + i]);
  }
}

template <typename IO>
__global__ __launch_bounds__(kWideThreads) void k_wide_gate_norm_bwd(GateArgs<IO> a, IO* __restrict__ dy, IO* __restrict__ dz,
                                                                int64_t dy_ts, int64_t dz_ts, float* __restrict__ stats) {
  __shared__ WideRed red;
  const int n = a.d / a.groups, g = blockIdx.x % a.groups;
  const int64_t row = blockIdx.x / a.groups;
  const IO *y = a.y + row * a.y_ts + g * n, *z = a.z + row * a.z_ts + g * n, *go = a.dout + row * a.d + g * n;
  const float* w = a.w + g * n;
  float ss = 0.0f, sd = 0.0f;
  for (int i = threadIdx.x; i < n; i += kWideThreads) {
    const float zv = ld_io(z, i), s = zv * sigmoid(zv), yv = ld_io(y, i);
    const float u = a.gate_first ? yv * s : yv;
    ss = __builtin_fmaf(u, u, ss);
    sd = __builtin_fmaf(ld_io(go, i) * w[i] * (a.gate_first ? 1.0f : s), u, sd);
  }
  ss = wide_sum(ss, red);
  sd = wide_sum(sd, red);
  const float k = rsqrtf(ss / n + a.eps);
  const float m = sd * k / n;  // mean(dn n)
  for (int i = threadIdx.x; i < n; i += kWideThreads) {
    const float zv = ld_io(z, i), sg = sigmoid(zv), s = zv * sg, ds = sg * (1.0f + zv * (1.0f - sg));
    const float yv = ld_io(y, i), go_w = ld_io(go, i) * w[i];
    const float u = a.gate_first ? yv * s : yv;
    const float dn = a.gate_first ? go_w : go_w * s;
    const float du = k * (dn - u * k * m);
    st_io(dy, row * dy_ts + g * n + i, a.gate_first ? du * s : du);
    st_io(dz, row * dz_ts + g * n + i, a.gate_first ? du * yv * ds : go_w * u * k * ds);
  }
  if (threadIdx.x == 0) stats[row * a.groups + g] = k;
}

template <typename IO>
__global__ __launch_bounds__(kWideThreads) void k_wide_gate_norm_dw(GateArgs<IO> a, const float* __restrict__ stats,
                                                               float* __restrict__ part, int64_t per) {
  const int c = blockIdx.x * kWideThreads + threadIdx.x;
  if (c >= a.d) return;
  const int g = c / (a.d / a.groups);
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
  float sum = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float zv = ld_io(a.z + r * a.z_ts, c);
    sum = __builtin_fmaf(ld_io(a.dout + r * a.d, c) * stats[r * a.groups + g],
                         ld_io(a.y + r * a.y_ts, c) * (zv * sigmoid(zv)), sum);
  }
  part[static_cast<int64_t>(blockIdx.y) * a.d + c] = sum;
}

template <typename IO, typename RES>
__global__ __launch_bounds__(kWideThreads) void k_wide_residual_norm(ResArgs<IO, RES> a, RES* __restrict__ res_out,
                                                                IO* __restrict__ out) {
  __shared__ WideRed red;
  extern __shared__ float r[];  // the row's new residual
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.d;
  float kp = 1.0f;
  if (a.wp != nullptr) {
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.d; i += kWideThreads) {
      const float v = ld_io(a.h, base + i);
      ss = __builtin_fmaf(v, v, ss);
    }
    kp = rsqrtf(wide_sum(ss, red) / a.d + a.eps);
  }
  float ss = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kWideThreads) {
    float p = ld_io(a.h, base + i);
    if (a.wp != nullptr) p *= kp * a.wp[i];
    const float v = __builtin_fmaf(a.vec != nullptr ? a.scale * a.vec[i] : a.scale, p,
                                   a.res != nullptr ? ld_io(a.res, base + i) : 0.0f);
    r[i] = v;
    ss = __builtin_fmaf(v, v, ss);
    st_io(res_out, base + i, v);
  }
  const float k = rsqrtf(wide_sum(ss, red) / a.d + a.eps);
  for (int i = threadIdx.x; i < a.d; i += kWideThreads) st_io(out, base + i, r[i] * k * a.w[i]);
}

template <typename IO, typename RES>
__global__ __launch_bounds__(kWideThreads) void k_wide_residual_norm_bwd(ResArgs<IO, RES> a, const IO* __restrict__ dout,
                                                                    const RES* dres_out,
                                                                    RES* dres, IO* __restrict__ dh,
                                                                    float* __restrict__ stats) {
  __shared__ WideRed red;
  extern __shared__ float dr[];  // the row's gradient of the residual
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.d;
  float ss = 0.0f, sd = 0.0f, sp = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kWideThreads) {
    const float v = ld_io(a.res, base + i), hv = ld_io(a.h, base + i);
    ss = __builtin_fmaf(v, v, ss);
    sd = __builtin_fmaf(ld_io(dout, base + i) * a.w[i], v, sd);
    sp = __builtin_fmaf(hv, hv, sp);
  }
  ss = wide_sum(ss, red);
  sd = wide_sum(sd, red);
  sp = wide_sum(sp, red);
  const float k = rsqrtf(ss / a.d + a.eps), m = sd * k / a.d;
  const float kp = a.wp != nullptr ? rsqrtf(sp / a.d + a.eps) : 1.0f;
  if (dres == nullptr) {  // the rows' factors alone
    if (threadIdx.x == 0) {
      stats[blockIdx.x * 3 + 0] = k;
      stats[blockIdx.x * 3 + 1] = m;
      stats[blockIdx.x * 3 + 2] = kp;
    }
    return;
  }
  float sh = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kWideThreads) {
    const float v = ld_io(a.res, base + i);
    const float g = (dres_out != nullptr ? ld_io(dres_out, base + i) : 0.0f) +
                    k * (ld_io(dout, base + i) * a.w[i] - v * k * m);
    dr[i] = g;
    st_io(dres, base + i, g);
    if (a.wp != nullptr)
      sh = __builtin_fmaf(g * (a.vec != nullptr ? a.scale * a.vec[i] : a.scale) * a.wp[i], ld_io(a.h, base + i), sh);
  }
  const float mp = a.wp != nullptr ? wide_sum(sh, red) * kp / a.d : 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kWideThreads) {
    const float dp = dr[i] * (a.vec != nullptr ? a.scale * a.vec[i] : a.scale);
    st_io(dh, base + i, a.wp != nullptr ? kp * (dp * a.wp[i] - ld_io(a.h, base + i) * kp * mp) : dp);
  }
}

template <typename IO, typename RES>
__global__ __launch_bounds__(kWideThreads) void k_wide_residual_norm_dw(ResArgs<IO, RES> a, const IO* __restrict__ dout,
                                                                   const RES* dres_out,
                                                                   const float* __restrict__ stats,
                                                                   float* __restrict__ part, int64_t per) {
  const int c = blockIdx.x * kWideThreads + threadIdx.x;
  if (c >= a.d) return;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < a.rows ? r0 + per : a.rows;
  const float w = a.w[c], wp = a.wp != nullptr ? a.wp[c] : 1.0f;
  const float sc = a.vec != nullptr ? a.scale * a.vec[c] : a.scale;
  float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float k = stats[r * 3], m = stats[r * 3 + 1], kp = stats[r * 3 + 2];
    const float v = ld_io(a.res, r * a.d + c), go = ld_io(dout, r * a.d + c), hv = ld_io(a.h, r * a.d + c);
    const float g = (dres_out != nullptr ? ld_io(dres_out, r * a.d + c) : 0.0f) + k * (go * w - v * k * m);
    s0 = __builtin_fmaf(go, v * k, s0);
    s1 = __builtin_fmaf(g * sc, hv * kp, s1);
    s2 = __builtin_fmaf(g * a.scale, hv * kp * wp, s2);
  }
  float* p = part + static_cast<int64_t>(blockIdx.y) * 3 * a.d;
  p[c] = s0;
  p[a.d + c] = s1;
  p[2 * a.d + c] = s2;
}

}  // namespace mm
