// The causal depthwise convolution by itself: kernels, argument checks and entry points.
#include "layer/common.h"

namespace mm {
namespace {

struct ConvArgs {
  const void* x;
  const float *w, *bias;
  const int32_t* cu;
  const float* state_in;
  int64_t x_ts, T;
  int S, d, W, silu;
};

// X(q) of sequence s (its first token g0, channel c): a token's raw input or the state's
template <typename IO>
__device__ float conv_raw(const ConvArgs& a, int s, int64_t g0, int64_t q, int c) {
  if (q >= 0) return ld_io(static_cast<const IO*>(a.x), (g0 + q) * a.x_ts + c);
  return a.state_in != nullptr ? a.state_in[(static_cast<int64_t>(s) * a.d + c) * (a.W - 1) + a.W - 1 + q] : 0.0f;
}
template <typename IO>
__device__ float conv_u(const ConvArgs& a, int s, int64_t g0, int64_t p, int c) {
  float u = a.bias != nullptr ? a.bias[c] : 0.0f;
  for (int k = 0; k < a.W; ++k) u = __builtin_fmaf(a.w[c * a.W + k], conv_raw<IO>(a, s, g0, p - a.W + 1 + k, c), u);
  return u;
}

template <typename IO>
__global__ __launch_bounds__(256) void k_conv(ConvArgs a, IO* __restrict__ y) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t0 = i / a.d * 16;
  const int c = static_cast<int>(i % a.d);
  for (int64_t t = t0; t < t0 + 16 && t < a.T; ++t) {
    const int s = seq_of(a.cu, a.S, t);
    const int64_t g0 = a.cu[s];
    const float u = conv_u<IO>(a, s, g0, t - g0, c);
    st_io(y, t * a.d + c, a.silu ? u * sigmoid(u) : u);
  }
}

// final states, a thread for each (sequence, channel); state_out may be state_in
template <typename IO>
__global__ __launch_bounds__(256) void k_conv_state(ConvArgs a, float* state_out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  const int s = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
  const int64_t g0 = a.cu[s], n = a.cu[s + 1] - g0;
  float v[MM_CONV_MAX_W - 1];
  for (int k = 0; k < a.W - 1; ++k) v[k] = conv_raw<IO>(a, s, g0, n - a.W + 1 + k, c);
  for (int k = 0; k < a.W - 1; ++k) state_out[i * (a.W - 1) + k] = v[k];
}

template <typename IO>
__global__ __launch_bounds__(256) void k_conv_decode(ConvArgs a, float* state_out, IO* __restrict__ y) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  const int64_t s = i / a.d;
  const int c = static_cast<int>(i % a.d);
  float u = a.bias != nullptr ? a.bias[c] : 0.0f, v[MM_CONV_MAX_W];
  for (int k = 0; k < a.W - 1; ++k) v[k] = a.state_in != nullptr ? a.state_in[i * (a.W - 1) + k] : 0.0f;
  v[a.W - 1] = ld_io(static_cast<const IO*>(a.x), s * a.x_ts + c);
  for (int k = 0; k < a.W; ++k) u = __builtin_fmaf(a.w[c * a.W + k], v[k], u);
  for (int k = 0; k < a.W - 1; ++k) state_out[i * (a.W - 1) + k] = v[k + 1];
  st_io(y, i, a.silu ? u * sigmoid(u) : u);
}

// dL/du at place p of sequence s
template <typename IO>
__device__ float conv_du(const ConvArgs& a, const IO* dy, int s, int64_t g0, int64_t p, int c) {
  const float g = ld_io(dy, (g0 + p) * a.d + c);
  if (!a.silu) return g;
  const float u = conv_u<IO>(a, s, g0, p, c);
  const Sigmoids v = sigmoids(u);
  return g * v.s * __builtin_fmaf(u, v.s1, 1.0f);
}

// dX(q) = sum_k w_k du(q + W - 1 - k), and what the final state asks for
template <typename IO>
__device__ float conv_dx(const ConvArgs& a, const IO* dy, const float* dstate_out, int s, int64_t g0, int64_t n, int64_t q, int c) {
  float v = 0.0f;
  for (int k = 0; k < a.W; ++k) {
    const int64_t p = q + a.W - 1 - k;
    if (p >= 0 && p < n) v = __builtin_fmaf(a.w[c * a.W + k], conv_du(a, dy, s, g0, p, c), v);
  }
  const int64_t j = q - (n - a.W + 1);
  if (dstate_out != nullptr && j >= 0) v += dstate_out[(static_cast<int64_t>(s) * a.d + c) * (a.W - 1) + j];
  return v;
}

template <typename IO>
__global__ __launch_bounds__(256) void k_conv_bwd(ConvArgs a, const IO* __restrict__ dy, const float* __restrict__ dstate_out,
                                                  IO* __restrict__ dx, int64_t dx_ts, float* __restrict__ part) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t0 = i / a.d * 16;
  const int c = static_cast<int>(i % a.d);
  if (t0 >= a.T) return;
  float dw[MM_CONV_MAX_W] = {}, db = 0.0f;
  for (int64_t t = t0; t < t0 + 16 && t < a.T; ++t) {
    const int s = seq_of(a.cu, a.S, t);
    const int64_t g0 = a.cu[s], n = a.cu[s + 1] - g0;
    st_io(dx, t * dx_ts + c, conv_dx(a, dy, dstate_out, s, g0, n, t - g0, c));
    const float g = conv_du(a, dy, s, g0, t - g0, c);
    db += g;
    for (int k = 0; k < a.W; ++k) dw[k] = __builtin_fmaf(g, conv_raw<IO>(a, s, g0, t - g0 - a.W + 1 + k, c), dw[k]);
  }
  float* p = part + t0 / 16 * a.d * (a.W + 1) + c;
  for (int k = 0; k < a.W; ++k) p[static_cast<int64_t>(k) * a.d] = dw[k];
  p[static_cast<int64_t>(a.W) * a.d] = db;
}

template <typename IO>
__global__ __launch_bounds__(256) void k_conv_dstate(ConvArgs a, const IO* __restrict__ dy, const float* __restrict__ dstate_out,
                                                     float* __restrict__ dstate_in) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.S) * a.d) return;
  const int s = static_cast<int>(i / a.d), c = static_cast<int>(i % a.d);
  const int64_t g0 = a.cu[s], n = a.cu[s + 1] - g0;
  for (int k = 0; k < a.W - 1; ++k)
    dstate_in[i * (a.W - 1) + k] = conv_dx(a, dy, dstate_out, s, g0, n, k - a.W + 1, c);
}

// the weights' gradients from `parts` rows of [W + 1, d] partial sums, in their order
__global__ __launch_bounds__(256) void k_conv_parts(const float* __restrict__ part, int64_t parts, int d, int W,
                                                    float* __restrict__ dw, float* __restrict__ db) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = static_cast<int64_t>(W + 1) * d;
  if (i >= n) return;
  float v = 0.0f;
  for (int64_t k = 0; k < parts; ++k) v += part[k * n + i];
  const int64_t k = i / d, c = i % d;
  if (k < W) dw[c * W + k] = v;
  else if (db != nullptr) db[c] = v;
}

int check_conv(int64_t S, int64_t T, int32_t d, int32_t W, int32_t io, int64_t x_ts) {
  const int rc = check_tokens(S, T, d, io);
  if (rc != MM_OK) return rc;
  if (W < 2 || W > MM_CONV_MAX_W) return MM_ERR_UNSUPPORTED;
  if (cdiv(T, 16) * d >= (int64_t{1} << 31)) return MM_ERR_DIM;
  return x_ts < d ? MM_ERR_DIM : MM_OK;
}
unsigned blocks(int64_t threads) { return static_cast<unsigned>(cdiv(threads, 256)); }
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
  const ConvArgs a{x, weight, bias, cu_seqlens, state_in, x_stride, T, S, d, W, silu};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    if (T > 0)
      hipLaunchKernelGGL((k_conv<IO>), dim3(blocks(cdiv(T, 16) * d)), dim3(256), 0, st, a, static_cast<IO*>(y));
    hipLaunchKernelGGL((k_conv_state<IO>), dim3(blocks(static_cast<int64_t>(S) * d)), dim3(256), 0, st, a, state_out);
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
  const ConvArgs a{x, weight, bias, nullptr, state_in, x_stride, Bs, Bs, d, W, silu};
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    hipLaunchKernelGGL((k_conv_decode<IO>), dim3(blocks(n)), dim3(256), 0, static_cast<hipStream_t>(stream), a, state_out,
                       static_cast<IO*>(y));
    return launched();
  });
}

size_t mamba_mixer_conv_backward_workspace_bytes(int64_t T, int32_t d, int32_t W) {
  if (check_conv(1, T, d, W, MM_IO_F32, d) != MM_OK || d == 0) return 0;
  return align256(static_cast<size_t>(cdiv(T, 16)) * d * (W + 1) * 4);
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
  const ConvArgs a{x, weight, bias, cu_seqlens, state_in, x_stride, T, S, d, W, silu};
  hipStream_t st = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  const int64_t parts = cdiv(T, 16);
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    const IO* g = static_cast<const IO*>(dy);
    if (T > 0)
      hipLaunchKernelGGL((k_conv_bwd<IO>), dim3(blocks(parts * d)), dim3(256), 0, st, a, g, dstate_out,
                         static_cast<IO*>(dx), dx_stride, part);
    if (dstate_in != nullptr && S > 0)
      hipLaunchKernelGGL((k_conv_dstate<IO>), dim3(blocks(static_cast<int64_t>(S) * d)), dim3(256), 0, st, a, g, dstate_out,
                         dstate_in);
    hipLaunchKernelGGL(k_conv_parts, dim3(blocks(nw + d)), dim3(256), 0, st, part, parts, d, W, dweight,
                       bias != nullptr ? dbias : nullptr);
    return launched();
  });
}

}  // extern "C"
