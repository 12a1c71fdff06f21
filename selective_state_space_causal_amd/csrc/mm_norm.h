// The norms around a mixer block, one pass each over their rows:
//   gate_norm       s = z sigmoid(z);  gate first: out = w n(y s),  gate last: out = w n(y) s,
//                   n(u) = u rsqrt(mean(u^2) + eps) over each of `groups` equal column ranges
//   residual_norm   p = h or w_post n(h);  r' = r + scale scale_vec p;  out = w n(r')
// and their gradients.  All arithmetic is float32; the outputs are rounded once.
#pragma once

#include "mm_device.h"

namespace mm {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 256;  // row ranges of the weight gradients' sums

__device__ __forceinline__ float wave_sum(float v) {
  for (int k = 32; k > 0; k /= 2) v += __shfl_xor(v, k);
  return v;
}
// sum over the workgroup, in every thread; `s` is 4 floats of LDS
__device__ __forceinline__ float group_sum(float v, float* s) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
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

template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_gate_norm(GateArgs<IO> a, IO* __restrict__ out) {
  __shared__ float red[4];
  const int n = a.d / a.groups, g = blockIdx.x % a.groups;
  const int64_t row = blockIdx.x / a.groups;
  const IO *y = a.y + row * a.y_ts + g * n, *z = a.z + row * a.z_ts + g * n;
  float ss = 0.0f;
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
    const float zv = ld_io(z, i);
    const float u = a.gate_first ? ld_io(y, i) * (zv * sigmoid(zv)) : ld_io(y, i);
    ss = __builtin_fmaf(u, u, ss);
  }
  const float k = rsqrtf(group_sum(ss, red) / n + a.eps);
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
    const float zv = ld_io(z, i);
    st_io(out, row * a.d + g * n + i, ld_io(y, i) * (zv * sigmoid(zv)) * k * a.w[g * n + i]);
  }
}

// dy, dz and, for the weight gradient's sums, each unit's factor k = rsqrt(mean + eps)
template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_gate_norm_bwd(GateArgs<IO> a, IO* __restrict__ dy, IO* __restrict__ dz,
                                                                int64_t dy_ts, int64_t dz_ts, float* __restrict__ stats) {
  __shared__ float red[4];
  const int n = a.d / a.groups, g = blockIdx.x % a.groups;
  const int64_t row = blockIdx.x / a.groups;
  const IO *y = a.y + row * a.y_ts + g * n, *z = a.z + row * a.z_ts + g * n, *go = a.dout + row * a.d + g * n;
  const float* w = a.w + g * n;
  float ss = 0.0f, sd = 0.0f;
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
    const float zv = ld_io(z, i), s = zv * sigmoid(zv), yv = ld_io(y, i);
    const float u = a.gate_first ? yv * s : yv;
    ss = __builtin_fmaf(u, u, ss);
    sd = __builtin_fmaf(ld_io(go, i) * w[i] * (a.gate_first ? 1.0f : s), u, sd);
  }
  ss = group_sum(ss, red);
  sd = group_sum(sd, red);
  const float k = rsqrtf(ss / n + a.eps);
  const float m = sd * k / n;  // mean(dn n)
  for (int i = threadIdx.x; i < n; i += kNormThreads) {
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

// partial sums of dw over the rows of one of kNormParts ranges
template <typename IO>
__global__ __launch_bounds__(kNormThreads) void k_gate_norm_dw(GateArgs<IO> a, const float* __restrict__ stats,
                                                               float* __restrict__ part, int64_t per) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
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

// out[c] = sum of the parts' c, in order
__global__ __launch_bounds__(kNormThreads) void k_norm_parts(const float* __restrict__ part, float* __restrict__ out,
                                                             int parts, int64_t stride, int d) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
  if (c >= d) return;
  float s = 0.0f;
  for (int i = 0; i < parts; ++i) s += part[i * stride + c];
  out[c] = s;
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

template <typename IO, typename RES>
__global__ __launch_bounds__(kNormThreads) void k_residual_norm(ResArgs<IO, RES> a, RES* __restrict__ res_out,
                                                                IO* __restrict__ out) {
  __shared__ float red[4];
  extern __shared__ float r[];  // the row's new residual
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.d;
  float kp = 1.0f;
  if (a.wp != nullptr) {
    float ss = 0.0f;
    for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
      const float v = ld_io(a.h, base + i);
      ss = __builtin_fmaf(v, v, ss);
    }
    kp = rsqrtf(group_sum(ss, red) / a.d + a.eps);
  }
  float ss = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
    float p = ld_io(a.h, base + i);
    if (a.wp != nullptr) p *= kp * a.wp[i];
    const float v = __builtin_fmaf(a.vec != nullptr ? a.scale * a.vec[i] : a.scale, p,
                                   a.res != nullptr ? ld_io(a.res, base + i) : 0.0f);
    r[i] = v;
    ss = __builtin_fmaf(v, v, ss);
    st_io(res_out, base + i, v);
  }
  const float k = rsqrtf(group_sum(ss, red) / a.d + a.eps);
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) st_io(out, base + i, r[i] * k * a.w[i]);
}

template <typename IO, typename RES>
__global__ __launch_bounds__(kNormThreads) void k_residual_norm_bwd(ResArgs<IO, RES> a, const IO* __restrict__ dout,
                                                                    const RES* __restrict__ dres_out,
                                                                    RES* __restrict__ dres, IO* __restrict__ dh,
                                                                    float* __restrict__ stats) {
  __shared__ float red[4];
  extern __shared__ float dr[];  // the row's gradient of the residual
  const int64_t base = static_cast<int64_t>(blockIdx.x) * a.d;
  float ss = 0.0f, sd = 0.0f, sp = 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
    const float v = ld_io(a.res, base + i), hv = ld_io(a.h, base + i);
    ss = __builtin_fmaf(v, v, ss);
    sd = __builtin_fmaf(ld_io(dout, base + i) * a.w[i], v, sd);
    sp = __builtin_fmaf(hv, hv, sp);
  }
  ss = group_sum(ss, red);
  sd = group_sum(sd, red);
  sp = group_sum(sp, red);
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
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
    const float v = ld_io(a.res, base + i);
    const float g = (dres_out != nullptr ? ld_io(dres_out, base + i) : 0.0f) +
                    k * (ld_io(dout, base + i) * a.w[i] - v * k * m);
    dr[i] = g;
    st_io(dres, base + i, g);
    if (a.wp != nullptr)
      sh = __builtin_fmaf(g * (a.vec != nullptr ? a.scale * a.vec[i] : a.scale) * a.wp[i], ld_io(a.h, base + i), sh);
  }
  const float mp = a.wp != nullptr ? group_sum(sh, red) * kp / a.d : 0.0f;
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
    const float dp = dr[i] * (a.vec != nullptr ? a.scale * a.vec[i] : a.scale);
    st_io(dh, base + i, a.wp != nullptr ? kp * (dp * a.wp[i] - ld_io(a.h, base + i) * kp * mp) : dp);
  }
}

// partial sums of dw, dw_post and dscale_vec over the rows of one range
template <typename IO, typename RES>
__global__ __launch_bounds__(kNormThreads) void k_residual_norm_dw(ResArgs<IO, RES> a, const IO* __restrict__ dout,
                                                                   const RES* __restrict__ dres_out,
                                                                   const float* __restrict__ stats,
                                                                   float* __restrict__ part, int64_t per) {
  const int c = blockIdx.x * kNormThreads + threadIdx.x;
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
