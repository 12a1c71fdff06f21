// The gated recurrence: kernels, argument checks and entry points.
#include <cmath>

#include "layer/common.h"

namespace mm {
namespace {

struct GatedArgs {
  const void *x, *r, *g, *z;
  const float* lam;
  const int32_t* cu;
  const float* state_in;
  int64_t x_ts, r_ts, g_ts, z_ts, T;
  int S, d;
  float c, c0, c1;  // the output gate: z sigmoid(z (c0 + c1 z^2))
};

// c softplus(lam) log2(e), so that a = exp2(-kap rho); NaN stays NaN
__device__ __forceinline__ float gated_kap(const GatedArgs& a, int c) {
  if (a.lam == nullptr) return 0.0f;
  const float v = a.lam[c];
  return (v != v ? v : softplus(v)) * a.c * kLog2e;
}

// The decay and the input's factor of one element, and what their gradients need.
//   1 - a^2 = -expm1(t), t = 2 log a: a series near 0 (six terms, 5e-8 of it at t = -1/4), 1 - a a beyond.
struct Decay {
  float a, m;      // decay, input factor
  float rho, rho1; // sigmoid(r), sigmoid(-r)
  float L, q;      // log a, log a / m (lam given)
};
__device__ __forceinline__ Decay gated_decay(float r, float kap, bool lam) {
  Decay v;
  const Sigmoids s0 = sigmoids(r);
  v.rho = s0.s;
  v.rho1 = s0.s1;
  if (!lam) {
    v.a = v.rho;
    v.m = v.rho1;
    v.L = v.q = 0.0f;
    return v;
  }
  const float la = -kap * v.rho;
  v.a = exp2_hw(la);
  v.L = la * kLn2;
  const float t = 2.0f * v.L;
  float s = __builtin_fmaf(t, 1.0f / 6, 1.0f);
  s = __builtin_fmaf(s * t, 1.0f / 5, 1.0f);
  s = __builtin_fmaf(s * t, 1.0f / 4, 1.0f);
  s = __builtin_fmaf(s * t, 1.0f / 3, 1.0f);
  s = __builtin_fmaf(s * t, 1.0f / 2, 1.0f);
  const float m2 = t > -0.25f ? -t * s : __builtin_fmaf(-v.a, v.a, 1.0f);
  // a decay of 1 has m = 0, and log a / m tends to 0 with it
  const float rm = __builtin_amdgcn_rsqf(__builtin_elementwise_maximum(m2, 1.2e-38f));
  v.m = m2 * rm;
  v.q = v.L * rm;
  return v;
}
__device__ __forceinline__ float gated_act(const GatedArgs& a, float z, float& slope) {
  const float z2 = fminf(z * z, 1e8f);  // far beyond where the sigmoid is 0 or 1; c1 may be 0
  const Sigmoids v = sigmoids(z * __builtin_fmaf(a.c1, z2, a.c0));
  slope = __builtin_fmaf(z * v.s * v.s1, __builtin_fmaf(3.0f * a.c1, z2, a.c0), v.s);
  return z * v.s;
}

template <typename IO>
__device__ float at(const void* p, int64_t ts, int64_t t, int c) { return ld_io(static_cast<const IO*>(p), t * ts + c); }

// a thread for each (sequence, channel); before: NULL or [T, d], the state before each token
template <typename IO>
__global__ __launch_bounds__(256) void k_gated(GatedArgs a, float* state_out, IO* __restrict__ y, float* __restrict__ ckpt,
                                               float* __restrict__ before) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  const int s = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
  const int64_t t0 = a.cu != nullptr ? a.cu[s] : s, t1 = a.cu != nullptr ? a.cu[s + 1] : s + 1;
  const float kap = gated_kap(a, c);
  float h = a.state_in != nullptr ? a.state_in[i] : 0.0f, slope;
  for (int64_t t = t0; t < t1; ++t) {
    if (ckpt != nullptr && t % MM_GATED_BLOCK == 0) ckpt[t / MM_GATED_BLOCK * a.d + c] = h;
    if (before != nullptr) before[t * a.d + c] = h;
    const Decay v = gated_decay(at<IO>(a.r, a.r_ts, t, c), kap, a.lam != nullptr);
    float u = at<IO>(a.x, a.x_ts, t, c);
    if (a.g != nullptr) u *= sigmoid(at<IO>(a.g, a.g_ts, t, c));
    h = __builtin_fmaf(v.a, h, v.m * u);
    if (y != nullptr) st_io(y, t * a.d + c, a.z != nullptr ? h * gated_act(a, at<IO>(a.z, a.z_ts, t, c), slope) : h);
  }
  if (state_out != nullptr) state_out[i] = h;
}

// With G the adjoint of h:  dx = G m iota,  dg = G m x iota (1 - iota),  dz = dy h act'(z), and
//   lam given: log a's gradient times log a is  e = G (a h' L - u a^2 L / m),  dr = e (1 - rho),
//              dlam = sum e sigmoid(lam) / softplus(lam)
//   else:      dr = G (h' - u) rho (1 - rho)                    (h' the state before, u = iota x)
struct GatedGrads {
  const void* dy;
  const float* dstate_out;
  float* before;  // the states before each token; then log a's gradients times log a
  void *dx, *dr, *dg, *dz;
  int64_t dx_ts, dr_ts, dg_ts, dz_ts;
  float* dstate_in;
};
template <typename IO>
__global__ __launch_bounds__(256) void k_gated_bwd(GatedArgs a, GatedGrads o) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  const int s = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
  const float kap = gated_kap(a, c);
  float G = o.dstate_out != nullptr ? o.dstate_out[i] : 0.0f;
  for (int64_t t = a.cu[s + 1] - int64_t{1}; t >= a.cu[s]; --t) {
    const Decay v = gated_decay(at<IO>(a.r, a.r_ts, t, c), kap, a.lam != nullptr);
    const float x = at<IO>(a.x, a.x_ts, t, c), h0 = o.before[t * a.d + c];
    float iota = 1.0f, iota1 = 0.0f;
    if (a.g != nullptr) {
      const Sigmoids v = sigmoids(at<IO>(a.g, a.g_ts, t, c));
      iota = v.s;
      iota1 = v.s1;
    }
    const float u = iota * x;
    float dh = ld_io(static_cast<const IO*>(o.dy), t * a.d + c);
    if (a.z != nullptr) {
      float slope;
      const float act = gated_act(a, at<IO>(a.z, a.z_ts, t, c), slope);
      st_io(static_cast<IO*>(o.dz), t * o.dz_ts + c, dh * __builtin_fmaf(v.a, h0, v.m * u) * slope);
      dh *= act;
    }
    G += dh;
    st_io(static_cast<IO*>(o.dx), t * o.dx_ts + c, G * v.m * iota);
    if (a.g != nullptr) st_io(static_cast<IO*>(o.dg), t * o.dg_ts + c, G * v.m * u * iota1);
    float dr;
    if (a.lam != nullptr) {
      const float e = G * v.a * (h0 * v.L - u * v.a * v.q);
      o.before[t * a.d + c] = e;
      dr = e * v.rho1;
    } else {
      dr = G * (h0 - u) * v.rho * v.rho1;
    }
    st_io(static_cast<IO*>(o.dr), t * o.dr_ts + c, dr);
    G *= v.a;
  }
  if (o.dstate_in != nullptr) o.dstate_in[i] = G;
}

// dlam from `parts` rows of partial sums, in their order.  sigmoid / softplus tends to 1 for lam -> -infinity.
__global__ __launch_bounds__(256) void k_gated_dlam(const float* __restrict__ part, int64_t parts, int d,
                                                    const float* __restrict__ lam, float* __restrict__ dlam) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float v = 0.0f;
  for (int64_t k = 0; k < parts; ++k) v += part[k * d + c];
  const float l = lam[c];
  dlam[c] = v * (l < -20.0f ? 1.0f : sigmoid(l) / (l != l ? l : softplus(l)));
}

int64_t gated_blocks(int64_t T) { return cdiv(T, MM_GATED_BLOCK); }

int check_gated(int64_t S, int64_t T, int32_t d, float c, int32_t gate, int32_t io) {
  const int rc = check_tokens(S, T, d, io);
  if (rc != MM_OK) return rc;
  if (gate != MM_GATE_SILU && gate != MM_GATE_GELU) return MM_ERR_UNSUPPORTED;
  if (!(c >= 0.0f) || std::isinf(c)) return MM_ERR_DIM;
  if (gated_blocks(T) * cdiv(d, 32) >= (int64_t{1} << 23)) return MM_ERR_DIM;
  return MM_OK;
}
bool strides(const GatedArgs& a) {
  return a.x_ts >= a.d && a.r_ts >= a.d && (a.g == nullptr || a.g_ts >= a.d) && (a.z == nullptr || a.z_ts >= a.d);
}
GatedArgs gated_args(const void* x, const void* r, const void* g, const void* z, const float* lam, const int32_t* cu,
                     const float* state_in, int64_t x_ts, int64_t r_ts, int64_t g_ts, int64_t z_ts, int64_t T, int S, int d,
                     float c, int gate) {
  // GELU's tanh form is z sigmoid(2 sqrt(2 / pi) (z + 0.044715 z^3))
  const float k = 1.5957691216057308f;
  return GatedArgs{x, r, g, z, lam, cu, state_in, x_ts, r_ts, g_ts, z_ts, T, S, d, c,
                   gate == MM_GATE_GELU ? k : 1.0f, gate == MM_GATE_GELU ? k * 0.044715f : 0.0f};
}
}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mamba_mixer_gated_prefill_workspace_bytes(int64_t T, int32_t d) { return 0; }

size_t mamba_mixer_gated_checkpoint_bytes(int64_t T, int32_t d) {
  if (check_gated(1, T, d, 0.0f, MM_GATE_SILU, MM_IO_F32) != MM_OK) return 0;
  return static_cast<size_t>(gated_blocks(T)) * d * 4;
}

int mamba_mixer_gated_prefill(const void* x, const void* r, const void* g, const void* z, const float* lam,
                              const int32_t* cu_seqlens, const float* state_in, float* state_out, void* y, float* ckpt,
                              int32_t S, int64_t T, int32_t d, float c, int32_t gate, int32_t io_dtype,
                              int64_t x_stride, int64_t r_stride, int64_t g_stride, int64_t z_stride, void* workspace,
                              size_t workspace_bytes, void* stream) {
  int rc = check_gated(S, T, d, c, gate, io_dtype);
  if (rc != MM_OK) return rc;
  const GatedArgs a = gated_args(x, r, g, z, lam, cu_seqlens, state_in, x_stride, r_stride, g_stride, z_stride, T, S, d, c, gate);
  if (!strides(a)) return MM_ERR_DIM;
  if (d == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  const int64_t ns = static_cast<int64_t>(S) * d;
  rc = check_args({strided(x, T, d, x_stride, es), strided(r, T, d, r_stride, es), strided(g, T, d, g_stride, es, true),
                   strided(z, T, d, z_stride, es, true), flat(lam, d, 4, true), flat(cu_seqlens, S > 0 ? S + int64_t{1} : 0, 4),
                   flat(state_in, ns, 4, true)},
                  {flat(state_out, ns, 4), flat(y, T * d, es), flat(ckpt, gated_blocks(T) * d, 4, true)}, {{0, 6}});
  if (rc != MM_OK) return rc;
  rc = check_workspace(workspace, workspace_bytes, mamba_mixer_gated_prefill_workspace_bytes(T, d));
  if (rc != MM_OK || S == 0) return rc;
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    hipLaunchKernelGGL((k_gated<IO>), dim3(static_cast<unsigned>(cdiv(ns, 256))), dim3(256), 0, static_cast<hipStream_t>(stream),
                       a, state_out, static_cast<IO*>(y), ckpt, static_cast<float*>(nullptr));
    return launched();
  });
}

int mamba_mixer_gated_decode(const void* x, const void* r, const void* g, const void* z, const float* lam,
                             const float* state_in, float* state_out, void* y, int32_t Bs, int32_t d, float c,
                             int32_t gate, int32_t io_dtype, int64_t x_stride, int64_t r_stride, int64_t g_stride,
                             int64_t z_stride, void* stream) {
  int rc = check_gated(Bs, Bs, d, c, gate, io_dtype);
  if (rc != MM_OK) return rc;
  const GatedArgs a = gated_args(x, r, g, z, lam, nullptr, state_in, x_stride, r_stride, g_stride, z_stride, Bs, Bs, d, c, gate);
  if (!strides(a)) return MM_ERR_DIM;
  const int64_t n = static_cast<int64_t>(Bs) * d;
  if (n == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  rc = check_args({strided(x, Bs, d, x_stride, es), strided(r, Bs, d, r_stride, es), strided(g, Bs, d, g_stride, es, true),
                   strided(z, Bs, d, z_stride, es, true), flat(lam, d, 4, true), flat(state_in, n, 4, true)},
                  {flat(state_out, n, 4), flat(y, n, es)}, {{0, 5}});
  if (rc != MM_OK) return rc;
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    hipLaunchKernelGGL((k_gated<IO>), dim3(static_cast<unsigned>(cdiv(n, 256))), dim3(256), 0, static_cast<hipStream_t>(stream),
                       a, state_out, static_cast<IO*>(y), static_cast<float*>(nullptr), static_cast<float*>(nullptr));
    return launched();
  });
}

size_t mamba_mixer_gated_backward_workspace_bytes(int64_t T, int32_t d, int32_t has_ckpt) {
  if (check_gated(1, T, d, 0.0f, MM_GATE_SILU, MM_IO_F32) != MM_OK) return 0;
  return align256(static_cast<size_t>(T) * d * 4);
}

int mamba_mixer_gated_backward(const void* x, const void* r, const void* g, const void* z, const float* lam,
                               const int32_t* cu_seqlens, const float* state_in, const void* dy,
                               const float* dstate_out, const float* ckpt, void* dx, void* dr, void* dg, void* dz,
                               float* dlam, float* dstate_in, int32_t S, int64_t T, int32_t d, float c, int32_t gate,
                               int32_t io_dtype, int64_t x_stride, int64_t r_stride, int64_t g_stride,
                               int64_t z_stride, int64_t dx_stride, int64_t dr_stride, int64_t dg_stride,
                               int64_t dz_stride, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_gated(S, T, d, c, gate, io_dtype);
  if (rc != MM_OK) return rc;
  const GatedArgs a = gated_args(x, r, g, z, lam, cu_seqlens, state_in, x_stride, r_stride, g_stride, z_stride, T, S, d, c, gate);
  if (!strides(a) || dx_stride < d || dr_stride < d || (g != nullptr && dg_stride < d) || (z != nullptr && dz_stride < d))
    return MM_ERR_DIM;
  if (d == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  const int64_t ns = static_cast<int64_t>(S) * d;
  rc = check_args({strided(x, T, d, x_stride, es), strided(r, T, d, r_stride, es), strided(g, T, d, g_stride, es, true),
                   strided(z, T, d, z_stride, es, true), flat(lam, d, 4, true), flat(cu_seqlens, S > 0 ? S + int64_t{1} : 0, 4),
                   flat(state_in, ns, 4, true), flat(dy, T * d, es), flat(dstate_out, ns, 4, true),
                   flat(ckpt, gated_blocks(T) * d, 4, true)},
                  {strided(dx, T, d, dx_stride, es), strided(dr, T, d, dr_stride, es), strided(dg, g != nullptr ? T : 0, d, dg_stride, es),
                   strided(dz, z != nullptr ? T : 0, d, dz_stride, es), flat(dlam, lam != nullptr ? d : 0, 4),
                   flat(dstate_in, ns, 4, true)});
  if (rc != MM_OK) return rc;
  rc = check_workspace(workspace, workspace_bytes, mamba_mixer_gated_backward_workspace_bytes(T, d, ckpt != nullptr));
  if (rc != MM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* before = static_cast<float*>(workspace);
  const GatedGrads o{dy, dstate_out, before, dx, dr, dg, dz, dx_stride, dr_stride, dg_stride, dz_stride, dstate_in};
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    const dim3 grid(static_cast<unsigned>(cdiv(ns, 256)));
    if (S > 0) {
      hipLaunchKernelGGL((k_gated<IO>), grid, dim3(256), 0, st, a, static_cast<float*>(nullptr), static_cast<IO*>(nullptr),
                         static_cast<float*>(nullptr), before);
      hipLaunchKernelGGL((k_gated_bwd<IO>), grid, dim3(256), 0, st, a, o);
    }
    if (lam != nullptr)
      hipLaunchKernelGGL(k_gated_dlam, dim3(static_cast<unsigned>(cdiv(d, 256))), dim3(256), 0, st, before, T, d, lam,
                         dlam);
    return launched();
  });
}

}  // extern "C"
