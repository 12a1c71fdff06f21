// The norms of queries and keys with their rotation: kernels, argument checks and entry points.
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
// the other column of column i's pair, and whether i is its first
__device__ __forceinline__ int qk_mate(const QkArgs& a, int i, bool& first) {
  first = a.inter ? i % 2 == 0 : i < a.R / 2;
  return a.inter ? i ^ 1 : first ? i + a.R / 2 : i - a.R / 2;
}
__device__ __forceinline__ int qk_pair(const QkArgs& a, int i) { return a.inter ? i / 2 : i % (a.R / 2); }
__device__ __forceinline__ float wave_sum(float v) {
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k);
  return v;
}

// a wave for each (token, head); with `dout` the gradients, else the outputs
template <typename IO>
__global__ __launch_bounds__(64) void k_qk(QkArgs a, IO* q_out, IO* k_out, int64_t qo_ts, int64_t ko_ts) {
  __shared__ float u[MM_QK_MAX_D];
  const int H = a.Hq + a.Hk;
  const int64_t t = blockIdx.x / H;
  int h = blockIdx.x % H;
  const bool key = h >= a.Hq;
  if (key) h -= a.Hq;
  const IO* v = static_cast<const IO*>(key ? a.k : a.q) + t * (key ? a.k_ts : a.q_ts) + h * a.D;
  const float* w = key ? a.wk : a.wq;
  float s = 0.0f;
  for (int i = threadIdx.x; i < a.D; i += 64) {
    u[i] = ld_io(v, i);
    s = __builtin_fmaf(u[i], u[i], s);
  }
  const float r = rsqrtf(wave_sum(s) / a.D + a.eps);
  __syncthreads();
  IO* out = (key ? k_out : q_out) + t * (key ? ko_ts : qo_ts) + h * a.D;
  for (int i = threadIdx.x; i < a.D; i += 64) {
    float o = u[i] * r * w[i];
    if (i < a.R) {
      bool first;
      const int j = qk_mate(a, i, first);
      float c, sn;
      qk_angle(a.pos[t], a.freq[qk_pair(a, i)], c, sn);
      const float m = u[j] * r * w[j];
      o = first ? o * c - m * sn : o * c + m * sn;
    }
    st_io(out, i, o);
  }
}

// With g the output's gradient turned back, n = v r and dn = g w:  dv = r (dn - n mean(dn n)),  dw = sum g n.
// A workgroup takes rows of one kind (queries or keys) and keeps the weight's gradient.
constexpr int kQkParts = 512;
template <typename IO>
__global__ __launch_bounds__(64) void k_qk_bwd(QkArgs a, const IO* dqo, const IO* dko, IO* dq, IO* dk, int64_t dq_ts, int64_t dk_ts,
                                               float* part) {
  __shared__ float u[MM_QK_MAX_D];
  const bool key = blockIdx.y != 0;
  const int H = key ? a.Hk : a.Hq;
  const float* w = key ? a.wk : a.wq;
  float dw[MM_QK_MAX_D / 64] = {};
  for (int64_t row = blockIdx.x; row < a.T * H; row += kQkParts) {
    const int64_t t = row / H;
    const int h = row % H;
    const IO* v = static_cast<const IO*>(key ? a.k : a.q) + t * (key ? a.k_ts : a.q_ts) + h * a.D;
    const IO* go = (key ? dko : dqo) + row * a.D;
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += 64) u[i] = ld_io(go, i);
    __syncthreads();
    float s = 0.0f, dot = 0.0f, g[MM_QK_MAX_D / 64], x[MM_QK_MAX_D / 64];
    for (int i = threadIdx.x, e = 0; i < a.D; i += 64, ++e) {
      x[e] = ld_io(v, i);
      g[e] = u[i];
      if (i < a.R) {
        bool first;
        const int j = qk_mate(a, i, first);
        float c, sn;
        qk_angle(a.pos[t], a.freq[qk_pair(a, i)], c, sn);
        g[e] = first ? u[i] * c + u[j] * sn : u[i] * c - u[j] * sn;
      }
      s = __builtin_fmaf(x[e], x[e], s);
      dot = __builtin_fmaf(g[e] * w[i], x[e], dot);
    }
    const float r = rsqrtf(wave_sum(s) / a.D + a.eps), m = wave_sum(dot) * r / a.D;
    IO* out = (key ? dk : dq) + t * (key ? dk_ts : dq_ts) + h * a.D;
    for (int i = threadIdx.x, e = 0; i < a.D; i += 64, ++e) {
      const float n = x[e] * r;
      dw[e] = __builtin_fmaf(g[e], n, dw[e]);
      st_io(out, i, r * (g[e] * w[i] - n * m));
    }
  }
  for (int i = threadIdx.x, e = 0; i < a.D; i += 64, ++e) part[(blockIdx.y * kQkParts + blockIdx.x) * a.D + i] = dw[e];
}
__global__ __launch_bounds__(256) void k_qk_parts(const float* part, int parts, int D, float* dwq, float* dwk) {
  const int i = threadIdx.x;
  if (i >= D) return;
  float v = 0.0f;
  for (int p = 0; p < parts; ++p) v += part[(blockIdx.x * kQkParts + p) * D + i];
  (blockIdx.x == 0 ? dwq : dwk)[i] = v;
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
    hipLaunchKernelGGL((k_qk<IO>), dim3(static_cast<unsigned>(T * (Hq + Hk))), dim3(64), 0, static_cast<hipStream_t>(stream), a,
                       static_cast<IO*>(q_out), static_cast<IO*>(k_out), qo_stride, ko_stride);
    return launched();
  });
}

size_t mamba_mixer_qk_norm_backward_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
  if (check_qk(T, Hq, Hk, D, 0, 0.0f, MM_IO_F32) != MM_OK) return 0;
  return align256(static_cast<size_t>(2) * kQkParts * D * 4);
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
    if (T > 0)
      hipLaunchKernelGGL((k_qk_bwd<IO>), dim3(kQkParts, 2), dim3(64), 0, st, a, static_cast<const IO*>(dq_out),
                         static_cast<const IO*>(dk_out), static_cast<IO*>(dq), static_cast<IO*>(dk), dq_stride, dk_stride, part);
    hipLaunchKernelGGL(k_qk_parts, dim3(2), dim3(256), 0, st, part, T > 0 ? kQkParts : 0, D, dq_weight, dk_weight);
    return launched();
  });
}

}  // extern "C"
