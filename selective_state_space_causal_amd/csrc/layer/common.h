// What the units of the convolution, the gated recurrence and the head norm share: argument checks, and on the device
// the sigmoid's pieces and the sums of partial results.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include <stddef.h>
#include <stdint.h>

#include "mambamix.h"
#include "mm_device.h"
#include "mm_host.h"

namespace mm {
namespace {

constexpr int64_t kMaxThreads = (int64_t{1} << 32) - 1;  // of one launch

int launched() { return hipGetLastError() == hipSuccess ? MM_OK : MM_ERR_HIP; }
size_t esize(int32_t io) { return io == MM_IO_BF16 ? 2 : 4; }

// An array of a call: rows of `width` elements `stride` apart.  Arrays of zero bytes, and optional ones, may be NULL.
struct Arg {
  Rows r;
  size_t es;
  bool optional;
};
Arg strided(const void* p, int64_t rows, int64_t width, int64_t stride, size_t es, bool optional = false) {
  return Arg{Rows{p, rows, static_cast<size_t>(width) * es, static_cast<size_t>(stride) * es}, es, optional};
}
Arg flat(const void* p, int64_t elements, size_t es, bool optional = false) {
  const size_t n = static_cast<size_t>(elements) * es;
  return Arg{Rows{p, 1, n, n}, es, optional};
}
struct Pair {
  int out, in;
};

// NULL where an array is needed, addresses that are not of whole elements, outputs on an input or on another output;
// `same`: the outputs that may be written over an input, at that very address.
int check_args(std::initializer_list<Arg> ins, std::initializer_list<Arg> outs, std::initializer_list<Pair> same = {}) {
  for (const auto& list : {ins, outs})
    for (const Arg& a : list)
      if (a.r.p == nullptr && !a.optional && a.r.extent() > 0) return MM_ERR_NULL;
  for (const auto& list : {ins, outs})
    for (const Arg& a : list)
      if (!aligned(a.r.p, a.es)) return MM_ERR_ALIGN;
  int o = 0;
  for (const Arg* out = outs.begin(); out != outs.end(); ++out, ++o) {
    if (out->r.p == nullptr) continue;
    int i = 0;
    for (const Arg* in = ins.begin(); in != ins.end(); ++in, ++i) {
      bool in_place = false;
      for (const Pair& s : same) in_place |= s.out == o && s.in == i && out->r.p == in->r.p && out->r.stride == in->r.stride;
      if (in->r.p != nullptr && !in_place && overlap(out->r, in->r)) return MM_ERR_ALIAS;
    }
    for (const Arg* next = out + 1; next != outs.end(); ++next)
      if (next->r.p != nullptr && overlap(out->r, next->r)) return MM_ERR_ALIAS;
  }
  return MM_OK;
}

// sizes of a call over T tokens in S sequences with d channels
int check_tokens(int64_t S, int64_t T, int32_t d, int32_t io) {
  if (S < 0 || T < 0 || d < 0 || T > INT32_MAX) return MM_ERR_DIM;
  if (io != MM_IO_F32 && io != MM_IO_BF16) return MM_ERR_UNSUPPORTED;
  if (S == 0 && T > 0) return MM_ERR_DIM;
  const uint64_t n = static_cast<uint64_t>(d);
  if (n > 0 && (static_cast<uint64_t>(T) > MM_MAX_ROWS_X_D / n || S * d >= (int64_t{1} << 31))) return MM_ERR_DIM;
  return MM_OK;
}
int check_workspace(const void* p, size_t bytes, size_t need) {
  if (need > 0 && (p == nullptr || bytes < need)) return MM_ERR_WORKSPACE;
  return aligned(p, 256) ? MM_OK : MM_ERR_ALIGN;
}

// f(IO{}) for the io type
template <typename F>
int by_io(int32_t io, F f) {
  return io == MM_IO_BF16 ? f(uint16_t{}) : f(float{});
}

}  // namespace

// sigmoid(v), and both it and sigmoid(-v), the latter without the cancellation of 1 - sigmoid(v): e s with e = exp(-v).  The
// hardware's reciprocal has no denormal results: past e = 2^126 (v < -87.34) s is 0, and sigmoid(-v) is 1 (it is from 2^24 on).
// An infinite or NaN v is taken as the formula has it.
__device__ __forceinline__ float sigmoid(float v) { return rcp_hw(1.0f + exp2_hw(-v * kLog2e)); }
struct Sigmoids {
  float s, s1;
};
__device__ __forceinline__ Sigmoids sigmoids(float v) {
  const float e = exp2_hw(-v * kLog2e), s = rcp_hw(1.0f + e);
  return {s, e >= 0x1p126f ? 1.0f : e * s};  // v = NaN in both
}

// V neighbouring channels of one token as loaded.  Rows may start at any element: accesses need no more alignment.
template <typename IO, int V>
struct Chans {
  static constexpr int W = (V * static_cast<int>(sizeof(IO)) + 3) / 4;
  uint32_t w[W];
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};
// `off` bytes behind a base that is the same in the whole wave
template <typename IO, int V>
__device__ __forceinline__ Chans<IO, V> load_chans(gmem<const IO>* p, uint32_t off) {
  constexpr int W = Chans<IO, V>::W;
  Chans<IO, V> r;
  gmem<const char>* q = reinterpret_cast<gmem<const char>*>(p) + off;
  if constexpr (V * sizeof(IO) == 2) {
    r.w[0] = __builtin_nontemporal_load(reinterpret_cast<gmem<const uint16_t>*>(q));
  } else if constexpr (W == 1) {
    typedef uint32_t word __attribute__((aligned(2)));
    r.w[0] = __builtin_nontemporal_load(reinterpret_cast<gmem<const word>*>(q));
  } else if constexpr (W > 4) {
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
#pragma unroll
    for (int j = 0; j < W; j += 4) {
      const vec v = __builtin_nontemporal_load(reinterpret_cast<gmem<const vec>*>(q + 4 * j));
#pragma unroll
      for (int i = 0; i < 4; ++i) r.w[j + i] = v[i];
    }
  } else {
    typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(sizeof(IO))));
    const vec v = __builtin_nontemporal_load(reinterpret_cast<gmem<const vec>*>(q));
#pragma unroll
    for (int i = 0; i < W; ++i) r.w[i] = v[i];
  }
  return r;
}
template <typename IO, int V>
__device__ __forceinline__ void store_chans(gmem<IO>* p, uint32_t off, const float (&f)[V]) {
  gmem<char>* q = reinterpret_cast<gmem<char>*>(p) + off;
  typedef float fv __attribute__((ext_vector_type(V), aligned(4)));
  fv t;
#pragma unroll
  for (int i = 0; i < V; ++i) t[i] = f[i];
  if constexpr (sizeof(IO) == 2) {
    typedef __bf16 bv __attribute__((ext_vector_type(V)));
    typedef uint16_t hv __attribute__((ext_vector_type(V), aligned(2)));
    __builtin_nontemporal_store(__builtin_bit_cast(hv, __builtin_convertvector(t, bv)), reinterpret_cast<gmem<hv>*>(q));  // round to nearest even
  } else {
    __builtin_nontemporal_store(t, reinterpret_cast<gmem<fv>*>(q));
  }
}
template <typename IO>
__device__ __forceinline__ gmem<IO>* global(IO* p) { return reinterpret_cast<gmem<IO>*>(reinterpret_cast<uint64_t>(p)); }

// The sum of `parts` rows' column c (d columns), in the first kPartColumns threads of a workgroup of 256: kPartColumns columns, eight
// threads each, in a fixed order.
constexpr int kPartColumns = 32;
__device__ __forceinline__ float sum_parts(const float* __restrict__ part, int64_t parts, int64_t d, int64_t c) {
  __shared__ float s[256 / kPartColumns][kPartColumns];
  const int row = threadIdx.x / kPartColumns, col = threadIdx.x % kPartColumns;
  constexpr int rows = 256 / kPartColumns;
  float v = 0.0f;
  if (c < d) {
    int64_t i = row;
    for (; i + 7 * rows < parts; i += 8 * rows) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = part[(i + k * rows) * d + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) v += t[k];
    }
    for (; i < parts; i += rows) v += part[i * d + c];
  }
  s[row][col] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < rows; ++k) t += s[k][col];
  return t;
}

}  // namespace mm
