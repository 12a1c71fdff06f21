// The gated recurrence: kernels, argument checks and entry points.
#include <algorithm>
#include <cmath>
#include <type_traits>

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
  float c;
  bool gelu;
};

// c softplus(lam) log2(e), so that a = exp2(-kap rho); NaN stays NaN
__device__ __forceinline__ float gated_kap(float lam, float c) { return (lam != lam ? lam : softplus(lam)) * c * kLog2e; }

// The decay a and the input's factor m of one element.  With l = log2 a = -kap rho, 1 - a^2 = -expm1(2 ln2 l): five terms
// of its series near 0 (4e-8 of it at a^2 = e^-1/8), 1 - a a beyond (there a's last unit is 5e-7 of m).
struct Decay {
  float a, m;
};
__device__ __forceinline__ float gated_m2(float l, float a) {
  constexpr float b = 2.0f * kLn2;
  float s = __builtin_fmaf(l, -b * b * b * b * b / 120, -b * b * b * b / 24);
  s = __builtin_fmaf(s, l, -b * b * b / 6);
  s = __builtin_fmaf(s, l, -b * b / 2);
  s = __builtin_fmaf(s, l, -b);
  return l > -0.125f / b ? s * l : __builtin_fmaf(-a, a, 1.0f);
}
template <bool LAM>
__device__ __forceinline__ Decay gated_decay(float r, float kap) {
  if constexpr (!LAM) {
    const Sigmoids s = sigmoids(r);
    return {s.s, s.s1};
  } else {
    const float l = -kap * sigmoid(r), a = exp2_hw(l);
    return {a, __builtin_amdgcn_sqrtf(gated_m2(l, a))};
  }
}
// The output gate z sigmoid(k): k = z, or for GELU's tanh form k = 2 sqrt(2 / pi) (z + 0.044715 z^3).
constexpr float kGelu0 = 1.5957691216057308f, kGelu1 = 1.5957691216057308f * 0.044715f;
__device__ __forceinline__ float gated_act(bool gelu, float z) {
  return gelu ? z * rcp_hw(1.0f + exp2_hw(z * __builtin_fmaf(-kGelu1 * kLog2e, z * z, -kGelu0 * kLog2e))) : z * sigmoid(z);
}

// One pass over the tokens.  A workgroup takes a tile: kGatedTile tokens of the packed stream by 256 bytes of channels.  A
// thread has V neighbouring channels and a run of K tokens: every (a, b = m iota x) of them is in registers from the load
// to the store, so each array is read and written once.  Runs compose as pairs (A, h): h_out = A h_in + h; the first
// threads put a tile's runs together, one for each channel, and the tiles of a channel are a chain in memory:
//   - a tile publishes its own pair as soon as it has it;
//   - the last of each group of tiles also publishes its final state;
//   - a tile's initial state is that of the last whole group of tiles before it, taken through the pairs of the tiles since.
// The order of these products does not depend on timing: results repeat bit for bit.  The links that wait for one another,
// a microsecond each, are one in a group.  Tiles are numbered by tickets, not by the workgroup's index, so a tile waits
// only for tiles whose workgroups run already or are done, and every wait ends.
// 16384 x 4096 of bfloat16 with all gates: 671 MB in 173 us, 3.9 TB/s (a copy of its size would take 109), vector
// instructions half of the time.  Two workgroups of a CU hold 128 registers a thread (four channels of bfloat16 spill four
// more, 20 bytes a thread), and a tile's loads, its arithmetic and its wait follow each other: what the other workgroup does
// meanwhile is all the overlap.  The wait itself is 5 us of it.  Rows of 128 bytes of channels: 193 us; tiles of 64 tokens:
// 180; workgroups that stay and load the next tile ahead: 214 and more, their registers left room for smaller tiles only.
// Where a sequence starts, A is set to -1: what comes before has no part in what follows, whatever it is (0 times an
// infinity would have).
constexpr int kGatedTile = 2 * MM_GATED_BLOCK, kGatedThreads = 512;
constexpr uint32_t kGatedQueues = 2, kGatedQueueStep = 64;  // tickets: counters, and elements between them
template <typename IO, int V, int TILE>
struct GatedShape {
  static constexpr int C = V == 1 ? 64 : 256 / sizeof(IO);  // channels of a tile
  static constexpr int lanes = C / V;                     // of a token
  static constexpr int runs = kGatedThreads / lanes;
  static constexpr int K = TILE / runs;                     // tokens of a run
};

// ---------------------------------------------------------------- the chain of a channel's tiles
typedef unsigned long long u64;
constexpr u64 kUnset = ~0ull;  // no pair: a NaN is published as 0x7FC00000 in its place

struct GatedChain {
  u64* pairs;         // [tiles, d]: A in the upper half, h in the lower
  u64* states;        // [tiles >> group, d]: h
  uint32_t* tickets;  // a counter for each queue, apart
  int group;          // log2 of a group's tiles
};
__device__ __forceinline__ u64 gated_pair(float A, float h) {
  return static_cast<u64>(A != A ? 0x7FC00000u : __float_as_uint(A)) << 32 | __float_as_uint(h);
}
// Written through to where all XCDs see it; the value itself says that it is there, so nothing else has to be ordered.
__device__ __forceinline__ void gated_publish(u64* p, u64 v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// What comes into tile `n` (in the chain's order) of a run that goes back to tile `first`: the last whole group's state,
// and the pairs of the tiles since, kGatedLook of them at a time.
constexpr int kGatedLook = 4;
struct Incoming {
  u64 state, pairs[kGatedLook];
  int64_t from;  // the first of the tiles since
  int count;
  bool older;    // a state comes in
};
__device__ __forceinline__ Incoming gated_from(const GatedChain& ch, int64_t n, int64_t first) {
  const int64_t group = n >> ch.group << ch.group;
  Incoming in;
  in.older = first < group;
  in.from = in.older ? group : first;
  in.count = static_cast<int>(n - in.from);
  in.state = in.older ? kUnset : 0;
#pragma unroll
  for (int i = 0; i < kGatedLook; ++i) in.pairs[i] = kUnset;
  return in;
}
// A look at channel c0 + c of d: the state, and the pairs from number `first` on.  It runs where every thread's tile is in
// registers: bases in scalar ones, and offsets that do not become 64-bit addresses ahead of their use.
__device__ __forceinline__ u64 gated_read(const u64* p, int64_t row, int64_t d, int64_t c0, uint32_t c) {
  uint32_t off = c * static_cast<uint32_t>(sizeof(u64));
  asm volatile("" : "+v"(off));
  gmem<const char>* base = reinterpret_cast<gmem<const char>*>(sbase(p + row * d + c0));
  return __hip_atomic_load(reinterpret_cast<gmem<const u64>*>(base + off), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void gated_look(Incoming& in, int first, const GatedChain& ch, int64_t d, int64_t c0, uint32_t c) {
  if (in.older) in.state = gated_read(ch.states, (in.from >> ch.group) - 1, d, c0, c);
#pragma unroll
  for (int i = 0; i < kGatedLook; ++i)
    if (first + i < in.count) in.pairs[i] = gated_read(ch.pairs, in.from + first + i, d, c0, c);
}
// Every wait ends: the tiles before have their tickets, and what waits for them never holds them up.  A workspace that
// another call overwrites meanwhile would break that: after so many looks (seconds) the tile goes on with what it has,
// kUnset being a NaN.
constexpr int kGatedLooks = 1 << 21;
// The state that comes in, from the first look on: the pairs put together, then the state taken through them.
__device__ __forceinline__ float gated_state(Incoming& in, const GatedChain& ch, int64_t d, int64_t c0, uint32_t c) {
  float A = 1.0f, h = 0.0f;
  int looks = 0;
  for (int at = 0; at < in.count;) {
    bool there = true;
#pragma unroll
    for (int i = 0; i < kGatedLook; ++i) there &= at + i >= in.count || in.pairs[i] != kUnset;
    if (__all(there) || looks >= kGatedLooks) {  // the wave goes on together: its bases stay scalar
#pragma unroll
      for (int i = 0; i < kGatedLook; ++i)
        if (at + i < in.count) {
          const float Ai = __uint_as_float(static_cast<uint32_t>(in.pairs[i] >> 32)), hi = __uint_as_float(static_cast<uint32_t>(in.pairs[i]));
          h = Ai < 0.0f ? hi : __builtin_fmaf(Ai, h, hi);
          A = Ai < 0.0f || A < 0.0f ? -1.0f : A * Ai;
        }
      at += kGatedLook;
    } else {
      __builtin_amdgcn_s_sleep(1);
    }
    ++looks;
    if (at < in.count) gated_look(in, at, ch, d, c0, c);
  }
  for (; !__all(in.state != kUnset) && looks < kGatedLooks; ++looks) {
    __builtin_amdgcn_s_sleep(1);
    gated_look(in, in.count, ch, d, c0, c);
  }
  return A < 0.0f ? h : __builtin_fmaf(A, __uint_as_float(static_cast<uint32_t>(in.state)), h);
}

// Final states of empty sequences, `in` (NULL: zeros) to `out`.  The tiles see to kTileSlots sequences each (gated_empty) where
// that is all of them, as it is where there are no more sequences than tokens.  Otherwise they are taken ahead of the tiles, in
// the kernel that clears the chain: a workgroup looks through 64 of them for kEmptyChannels channels, its waves take turns, a
// wave's loads are on their way together.  Taken by the tiles however many there are, 40000 empty ones beside 16 tokens x 256
// took 3.2 ms for 30 us, 5000 beside 16 x 2048 411 us for 31; taken ahead however few, 512 sequences of 16 tokens x 2048 take
// 54.5 us for 53.2, two of 4 tokens x 4096 18.4 for 16.0; in workgroups of the tiles' kernels, 8192 x 2048 58 us for 52.
constexpr int kEmptySlots = 64, kEmptyChannels = 128, kTileSlots = 128;
struct EmptySlots {
  const int32_t* cu;
  const float* in;
  float* out;
  int64_t d;
  int S;
};
__global__ __launch_bounds__(256) void k_gated_begin(u64* p, int64_t n, uint32_t* tickets, EmptySlots e) {
  const int64_t blocks = (n + 255) / 256;
  if (blockIdx.x < blocks) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) p[i] = kUnset;
    if (i < kGatedQueues) tickets[i * kGatedQueueStep] = 0;
    return;
  }
  constexpr int waves = 4, N = kEmptySlots / waves, W = kEmptyChannels / 64;
  const uint32_t block = static_cast<uint32_t>(blockIdx.x - blocks), slices = static_cast<uint32_t>((e.d + kEmptyChannels - 1) / kEmptyChannels);
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const int64_t s0 = static_cast<int64_t>(block / slices) * kEmptySlots, c = static_cast<int64_t>(block % slices) * kEmptyChannels + lane;
  const int64_t s = s0 + lane < e.S ? s0 + lane : e.S - 1;
  const u64 empty = __ballot(s0 + lane < e.S && e.cu[s] == e.cu[s + 1]);
  const auto here = [&](int j, int k) { return (empty >> (wave + j * waves) & 1) && c + 64 * k < e.d; };
  const auto at = [&](int j, int k) { return (s0 + wave + j * waves) * e.d + c + 64 * k; };
  float v[N][W];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int k = 0; k < W; ++k) v[j][k] = e.in != nullptr && here(j, k) ? e.in[at(j, k)] : 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int k = 0; k < W; ++k)
      if (here(j, k)) e.out[at(j, k)] = v[j][k];
}

// A tile's share of them, channels c0 .. c0 + width: its waves take turns.
__device__ __forceinline__ void gated_empty(const int32_t* __restrict__ cu, int S, uint32_t tile, uint32_t tiles, const float* in, float* out,
                                            int64_t d, int64_t c0, int width) {
  const int64_t first = static_cast<int64_t>(tile) * kTileSlots;
  if (first >= S || S > static_cast<int64_t>(tiles) * kTileSlots) return;
  const int lane = threadIdx.x & 63;
  for (int64_t s0 = first; s0 < first + kTileSlots && s0 < S; s0 += 64) {
    const int64_t s = s0 + lane < S ? s0 + lane : S - 1;
    u64 empty = __ballot(s0 + lane < S && cu[s] == cu[s + 1]) & (0x0101010101010101ull << threadIdx.x / 64);
    for (; empty != 0; empty &= empty - 1) {
      const int64_t e = (s0 + __builtin_ctzll(empty)) * d;
      for (int64_t c = c0 + lane; c < c0 + width && c < d; c += 64) out[e + c] = in != nullptr ? in[e + c] : 0.0f;
    }
  }
}

// A token's place: its sequence and whether it is the first or the last of it.  Behind the last token: neither.
struct Place {
  int v;
  __device__ bool starts() const { return v & 1; }
  __device__ bool ends() const { return v & 2; }
  __device__ int seq() const { return v >> 2; }
};
template <int TILE>
__device__ __forceinline__ void gated_places(const int32_t* __restrict__ cu, int S, int64_t T, int64_t t0, Place* place) {
  for (int i = threadIdx.x; i < TILE; i += kGatedThreads) {
    const int64_t t = t0 + i;
    int v = 0;
    if (t < T) {
      const int s = seq_of(cu, S, t);
      v = s << 2 | (cu[s] == t ? 1 : 0) | (cu[s + 1] == t + 1 ? 2 : 0);
    }
    place[i].v = v;
  }
}
// LDS is written, a wave's loads from memory may stay in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The ticket's tile: queue q has the slices q, q + kGatedQueues, ..., tile by tile (one counter gives a ticket in 10 ns:
// 4 x 2048 x 768 31.1 us with one, 29.5 with two; with four the slices drift apart, 262144 x 256 191 -> 219).  There are as
// many workgroups as tiles, and a queue that is through hands its workgroups on to the next one, so each has found its tile
// when it has asked every queue once; kGatedNone would mean that another call has the workspace too.
constexpr uint32_t kGatedNone = ~0u;
__device__ __forceinline__ uint32_t gated_take(uint32_t* tickets, uint32_t tiles, uint32_t slices) {
  for (uint32_t i = 0; i < kGatedQueues; ++i) {
    const uint32_t q = (blockIdx.x + i) % kGatedQueues, w = (slices + kGatedQueues - 1 - q) / kGatedQueues;
    const uint32_t t = atomicAdd(tickets + q * kGatedQueueStep, 1u);
    if (t < w * tiles) return t / w * slices + t % w * kGatedQueues + q;
  }
  return kGatedNone;
}

// OUT: y and the final states; else only the checkpoints (for a backward without the forward's)
template <typename IO, int V, bool LAM, bool OUT>
__global__ __launch_bounds__(kGatedThreads, 4) void k_gated(GatedArgs a, GatedChain ch, float* state_out, IO* y, float* ckpt) {
  typedef GatedShape<IO, V, kGatedTile> Shape;
  constexpr int K = Shape::K, C = Shape::C, NG = Shape::runs;
  __shared__ float sA[NG][C], sH[NG][C], sC[C];
  __shared__ Place place[kGatedTile];
  __shared__ uint32_t turn;
  const int64_t d = a.d;
  const uint32_t slices = static_cast<uint32_t>((d + C - 1) / C), tiles = gridDim.x / slices;
  uint32_t id = blockIdx.x;
  if (tiles > 1) {
    if (threadIdx.x == 0) turn = gated_take(ch.tickets, tiles, slices);
    lds_barrier();
    id = __builtin_amdgcn_readfirstlane(turn);
    if (id == kGatedNone) return;
  }
  const uint32_t tile = id / slices;
  const int64_t c0 = static_cast<int64_t>(id % slices) * C, t0 = static_cast<int64_t>(tile) * kGatedTile;
  const int lane = threadIdx.x % Shape::lanes, run = threadIdx.x / Shape::lanes;
  const int64_t c = c0 + lane * V;
  const bool on = c < d, whole = t0 + kGatedTile <= a.T;
  const int64_t left = a.T - t0 - run * K;  // tokens of this run, if under K

  Chans<IO, V> rx[K], rr[K], rg[K], rz[K];
  const auto load = [&](const void* p, int64_t ts, Chans<IO, V>(&v)[K]) {
    gmem<const IO>* base = sbase(static_cast<const IO*>(p) + t0 * ts + c0);
    const uint32_t step = static_cast<uint32_t>(ts * static_cast<int64_t>(sizeof(IO)));
    uint32_t off = run * K * step + lane * V * static_cast<uint32_t>(sizeof(IO));
    if (whole) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = load_chans<IO, V>(base, off);
        off += step;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = Chans<IO, V>{};
        if (k < left) v[k] = load_chans<IO, V>(base, off);
        off += step;
      }
    }
  };
  float kap[V];
  if (on) {
    load(a.r, a.r_ts, rr);
    load(a.x, a.x_ts, rx);
    if (a.g != nullptr) load(a.g, a.g_ts, rg);
#pragma unroll
    for (int i = 0; i < V; ++i) kap[i] = LAM ? gated_kap(a.lam[c + i], a.c) : 0.0f;
  }
  const int seq = seq_of(a.cu, a.S, t0);
  const int64_t lo = a.cu[seq], hi = a.cu[seq + 1];
  const bool cut = lo == t0 || hi <= t0 + kGatedTile;  // sequences start or end in the tile
  if (cut) {
    gated_places<kGatedTile>(a.cu, a.S, a.T, t0, place);
    lds_barrier();
  }

  float da[K][V], db[K][V], A[V], h[V];
  uint32_t starts = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    A[i] = 1.0f;
    h[i] = 0.0f;
  }
  if (on) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Decay v = gated_decay<LAM>(rr[k][i], kap[i]);
        da[k][i] = v.a;
        db[k][i] = v.m * rx[k][i];
      }
      if (a.g != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) db[k][i] *= sigmoid(rg[k][i]);
      }
      if (cut) {
        const Place p = place[run * K + k];
        if (p.starts()) {  // the run so far has no part in it; its initial state becomes part of its input
          starts |= 1u << k;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if (a.state_in != nullptr) db[k][i] = __builtin_fmaf(da[k][i], a.state_in[p.seq() * d + c + i], db[k][i]);
            h[i] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        A[i] *= da[k][i];
        h[i] = __builtin_fmaf(da[k][i], h[i], db[k][i]);
      }
      __builtin_amdgcn_sched_barrier(0);  // one token after the other: fewer registers
    }
    if (OUT && a.z != nullptr) load(a.z, a.z_ts, rz);  // on its way while the tile waits for the one before
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sA[run][lane * V + i] = starts != 0 ? -1.0f : A[i];
    sH[run][lane * V + i] = h[i];
  }
  const int64_t cc = c0 + threadIdx.x;
  const bool chain = threadIdx.x < C && cc < d, waits = lo != t0;
  Incoming in = gated_from(ch, tile, lo / kGatedTile);
  if (chain && waits) gated_look(in, 0, ch, d, c0, threadIdx.x);  // under way while the runs are put together
  lds_barrier();
  if (chain) {
    const int j = threadIdx.x;
    float At = 1.0f, ht = 0.0f, from = 0.0f, Am = 0.0f, hm = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float Ag = sA[g][j], hg = sH[g][j];
      if (g == NG / 2) {
        Am = At;
        hm = ht;
      }
      sA[g][j] = At;
      sH[g][j] = ht;
      ht = Ag < 0.0f ? hg : __builtin_fmaf(Ag, ht, hg);
      At = Ag < 0.0f || At < 0.0f ? -1.0f : At * Ag;
    }
    static_assert(kGatedTile == 2 * MM_GATED_BLOCK, "a checkpoint before the tile and one in its middle");
    float* const cp = ckpt + static_cast<int64_t>(2) * tile * d + cc;
    const bool halfway = t0 + MM_GATED_BLOCK < a.T, restarts = cut && halfway && place[MM_GATED_BLOCK].starts();
    if (ckpt != nullptr) {
      // Sequences that start at a checkpoint.  Their initial states are read before the pair is out: where state_out is
      // state_in, the tile in which such a sequence ends may then write over them.
      if (!waits) cp[0] = a.state_in != nullptr ? a.state_in[seq * d + cc] : 0.0f;
      if (restarts) cp[d] = a.state_in != nullptr ? a.state_in[place[MM_GATED_BLOCK].seq() * d + cc] : 0.0f;
      asm volatile("" : : : "memory");
    }
    if (tile + 1 < tiles) gated_publish(ch.pairs + tile * d + cc, gated_pair(At, ht));
    if (waits) from = gated_state(in, ch, d, c0, threadIdx.x);
    if (tile + 1 < tiles && (tile + 1) >> ch.group << ch.group == tile + 1)
      gated_publish(ch.states + (tile >> ch.group) * d + cc, __float_as_uint(At < 0.0f ? ht : __builtin_fmaf(At, from, ht)));
    if (ckpt != nullptr) {
      if (waits) cp[0] = from;
      if (halfway && !restarts) cp[d] = Am < 0.0f ? hm : __builtin_fmaf(Am, from, hm);
    }
    sC[j] = from;
  }
  if (!OUT) return;
  lds_barrier();
  if (state_out != a.state_in) gated_empty(a.cu, a.S, tile, tiles, a.state_in, state_out, d, c0, C);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float Ap = sA[run][lane * V + i], hp = sH[run][lane * V + i];
    h[i] = Ap < 0.0f ? hp : __builtin_fmaf(Ap, sC[lane * V + i], hp);
  }
  gmem<IO>* base = sbase(y + t0 * d + c0);
  const uint32_t step = static_cast<uint32_t>(d * static_cast<int64_t>(sizeof(IO)));
  uint32_t off = run * K * step + lane * V * static_cast<uint32_t>(sizeof(IO));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (cut && (starts >> k & 1)) {
#pragma unroll
      for (int i = 0; i < V; ++i) h[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) db[k][i] = h[i] = __builtin_fmaf(da[k][i], h[i], db[k][i]);
    if (cut) {
      const Place p = place[run * K + k];
      if (p.ends()) {
#pragma unroll
        for (int i = 0; i < V; ++i) state_out[p.seq() * d + c + i] = h[i];
      }
    }
    if (a.z != nullptr) {
      if (a.gelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) db[k][i] *= gated_act(true, rz[k][i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) db[k][i] *= gated_act(false, rz[k][i]);
      }
    }
    if (whole || k < left) store_chans<IO, V>(base, off, db[k]);
    off += step;
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One token a row: V channels a thread.  256 x 8192 of bfloat16 with all gates: 38 MB in 11 us, 3.4 TB/s.
template <typename IO, int V, bool LAM>
__global__ __launch_bounds__(256) void k_gated_decode(GatedArgs a, float* state_out, IO* y) {
  const int64_t n = static_cast<int64_t>(a.S) * a.d;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  if (i0 >= n) return;
  const int64_t row = i0 / a.d;
  const int c = static_cast<int>(i0 - row * a.d);
  const auto load = [&](const void* p, int64_t ts) {
    return load_chans<IO, V>(global(static_cast<const IO*>(p) + row * ts + c), 0);
  };
  const Chans<IO, V> r = load(a.r, a.r_ts), x = load(a.x, a.x_ts);
  Chans<IO, V> g{}, z{};
  if (a.g != nullptr) g = load(a.g, a.g_ts);
  if (a.z != nullptr) z = load(a.z, a.z_ts);
  float h[V], o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float h0 = a.state_in != nullptr ? a.state_in[i0 + i] : 0.0f;
    const Decay v = gated_decay<LAM>(r[i], LAM ? gated_kap(a.lam[c + i], a.c) : 0.0f);
    const float u = a.g != nullptr ? x[i] * sigmoid(g[i]) : x[i];
    h[i] = __builtin_fmaf(v.a, h0, v.m * u);
    o[i] = a.z != nullptr ? h[i] * gated_act(a.gelu, z[i]) : h[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) state_out[i0 + i] = h[i];
  store_chans<IO, V>(global(y + i0), 0, o);
}

// ---------------------------------------------------------------- backward
// With G the adjoint of h, h' the state before the token and u = iota x:
//   G_t = dy act(z) + a_{t+1} G_{t+1};   dx = G m iota,  dg = G m u (1 - iota),  dz = dy h act'(z)
//   lam given: log a's gradient times log a is  e = G (a h' L - u a^2 L / m),  L = log a:  dr = e (1 - rho),
//              dlam = sum e sigmoid(lam) / softplus(lam)
//   else:      dr = G (h' - u) rho (1 - rho)
// m tends to 0 with L, and L / m with it.
// One pass from the last tile to the first, in the forward's manner: R = a G is what a token hands to the one before it, so
// a run is a pair (A, R) and the tiles are a chain.  The states before each token come from the checkpoint before the tile.
// What a thread keeps of a token from the first look to the gradients are a, h' and dy act'(z) in registers, dy act(z) in
// shared memory, and the other inputs as they were loaded: the rest is computed twice, which costs less than the registers.
// 8 x 2048 x 1536 of bfloat16 with all gates: 453 MB in 140 us, 3.2 TB/s; vector instructions take 60% of the time (fifteen
// exponentials, reciprocals and roots an element), and as in the forward little of it overlaps the loads.
struct GatedGrads {
  const void* dy;
  const float *dstate_out, *ckpt;
  void *dx, *dr, *dg, *dz;
  int64_t dx_ts, dr_ts, dg_ts, dz_ts;
  float *dstate_in, *part;  // part: [tiles, d], sums of e over a tile's tokens
};
// the output gate and its slope
struct Act {
  float act, slope;
};
__device__ __forceinline__ Act gated_act_slope(bool gelu, float z) {
  const float z2 = z * z;
  const Sigmoids s = sigmoids(gelu ? z * __builtin_fmaf(kGelu1, z2, kGelu0) : z);
  const float act = z * s.s;
  // an infinite slope of the argument meets a sigmoid that is 0 or 1
  return {act, __builtin_fmaf(act * s.s1, gelu ? fminf(__builtin_fmaf(3.0f * kGelu1, z2, kGelu0), 1e30f) : 1.0f, s.s)};
}
template <typename IO, int V>
__device__ __forceinline__ void again(Chans<IO, V>& v) {  // a value that the compiler does not know to be the same
#pragma unroll
  for (int i = 0; i < Chans<IO, V>::W; ++i) asm volatile("" : "+v"(v.w[i]));
}

constexpr int kGatedBwdTile = MM_GATED_BLOCK;
template <typename IO, int V, bool LAM>
__global__ __launch_bounds__(kGatedThreads, 4) void k_gated_bwd(GatedArgs a, GatedChain ch, GatedGrads o) {
  typedef GatedShape<IO, V, kGatedBwdTile> Shape;
  constexpr int K = Shape::K, C = Shape::C, NG = Shape::runs;
  __shared__ float sA[NG][C], sH[NG][C], sR[NG][C];
  __shared__ __align__(16) float sD[K][kGatedThreads][V];  // each thread's own
  __shared__ Place place[kGatedBwdTile];
  __shared__ int cuts[NG];  // of a run: 1 a sequence starts in it, 2 one ends
  __shared__ uint32_t turn;
  const int64_t d = a.d;
  const uint32_t slices = static_cast<uint32_t>((d + C - 1) / C), tiles = gridDim.x / slices;
  uint32_t id = blockIdx.x;
  if (tiles > 1) {
    if (threadIdx.x == 0) turn = gated_take(ch.tickets, tiles, slices);
    lds_barrier();
    id = __builtin_amdgcn_readfirstlane(turn);
    if (id == kGatedNone) return;
  }
  const uint32_t n = id / slices, tile = tiles - 1 - n;
  const int64_t c0 = static_cast<int64_t>(id % slices) * C, t0 = static_cast<int64_t>(tile) * kGatedBwdTile;
  const int lane = threadIdx.x % Shape::lanes, run = threadIdx.x / Shape::lanes;
  const int64_t c = c0 + lane * V;
  const bool on = c < d, whole = t0 + kGatedBwdTile <= a.T;
  const int64_t left = a.T - t0 - run * K;  // tokens of this run, if under K

  const auto offset = [&](int64_t ts, uint32_t& step) {
    step = static_cast<uint32_t>(ts * static_cast<int64_t>(sizeof(IO)));
    return run * K * step + lane * V * static_cast<uint32_t>(sizeof(IO));
  };
  Chans<IO, V> rx[K], rr[K], rg[K], rz[K], ry[K];
  const auto load = [&](const void* p, int64_t ts, Chans<IO, V>(&v)[K]) {
    gmem<const IO>* base = sbase(static_cast<const IO*>(p) + t0 * ts + c0);
    uint32_t step, off = offset(ts, step);
    if (whole) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = load_chans<IO, V>(base, off);
        off += step;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = Chans<IO, V>{};
        if (k < left) v[k] = load_chans<IO, V>(base, off);
        off += step;
      }
    }
  };
  float kap[V];
  if (on) {
    load(a.r, a.r_ts, rr);
    load(a.x, a.x_ts, rx);
    if (a.g != nullptr) load(a.g, a.g_ts, rg);
    load(o.dy, d, ry);
    if (a.z != nullptr) load(a.z, a.z_ts, rz);
#pragma unroll
    for (int i = 0; i < V; ++i) kap[i] = LAM ? gated_kap(a.lam[c + i], a.c) : 0.0f;
  }
  const int seq = seq_of(a.cu, a.S, t0);
  const int64_t lo = a.cu[seq];
  int64_t hi = a.cu[seq + 1];
  const bool cut = lo == t0 || hi <= t0 + kGatedBwdTile;  // sequences start or end in the tile
  if (cut) {
    gated_places<kGatedBwdTile>(a.cu, a.S, a.T, t0, place);
    const int64_t last = whole ? t0 + kGatedBwdTile - 1 : a.T - 1;
    hi = a.cu[seq_of(a.cu, a.S, last) + 1];  // the end of the tile's last sequence
    lds_barrier();
  }

  // a, b and the runs; b makes room for the state before the token afterwards
  float da[K][V], db[K][V], dz[K][V], A[V], h[V], R[V];
  int marks = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    A[i] = 1.0f;
    h[i] = R[i] = 0.0f;
  }
  // what the final state of a sequence that ends at token k asks for
  const auto final_adjoint = [&](int k, float(&dh)[V]) {
    if (cut && o.dstate_out != nullptr) {
      const Place p = place[run * K + k];
      if (p.ends()) {
#pragma unroll
        for (int i = 0; i < V; ++i) dh[i] += o.dstate_out[p.seq() * d + c + i];
      }
    }
  };
  if (on) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Decay v = gated_decay<LAM>(rr[k][i], kap[i]);
        da[k][i] = v.a;
        db[k][i] = v.m * rx[k][i];
      }
      if (a.g != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) db[k][i] *= sigmoid(rg[k][i]);
      }
      if (cut) {
        const Place p = place[run * K + k];
        if (p.starts()) {
          marks |= 1;
#pragma unroll
          for (int i = 0; i < V; ++i) h[i] = a.state_in != nullptr ? a.state_in[p.seq() * d + c + i] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        A[i] *= da[k][i];
        h[i] = __builtin_fmaf(da[k][i], h[i], db[k][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      float dh[V];
      if (a.z != nullptr) {
        const auto gate = [&](bool gelu) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const Act v = gated_act_slope(gelu, rz[k][i]);
            dz[k][i] = v.slope * ry[k][i];
            dh[i] = ry[k][i] * v.act;
          }
        };
        if (a.gelu) gate(true);
        else gate(false);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) dh[i] = ry[k][i];
      }
      final_adjoint(k, dh);
#pragma unroll
      for (int i = 0; i < V; ++i) sD[k][threadIdx.x][i] = dh[i];
      if (cut && place[run * K + k].ends()) {
        marks |= 2;
#pragma unroll
        for (int i = 0; i < V; ++i) R[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) R[i] = da[k][i] * (dh[i] + R[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    sA[run][lane * V + i] = A[i];
    sH[run][lane * V + i] = h[i];
    sR[run][lane * V + i] = R[i];
  }
  if (lane == 0) cuts[run] = marks;  // the first channels of a slice are there
  const int64_t cc = c0 + threadIdx.x;
  const bool chain = threadIdx.x < C && cc < d, waits = hi > t0 + kGatedBwdTile;
  Incoming in = gated_from(ch, n, tiles - 1 - (hi - 1) / kGatedBwdTile);
  if (chain && waits) gated_look(in, 0, ch, d, c0, threadIdx.x);
  lds_barrier();
  if (chain) {
    const int j = threadIdx.x;
    float At = 1.0f, Rt = 0.0f, from = 0.0f, state = o.ckpt[tile * d + cc];
#pragma unroll
    for (int g = NG - 1; g >= 0; --g) {
      const float Ag = sA[g][j], Rg = sR[g][j];
      const bool ends = cuts[g] & 2;
      Rt = ends ? Rg : __builtin_fmaf(Ag, Rt, Rg);
      At = ends || At < 0.0f ? -1.0f : At * Ag;
    }
    if (n + 1 < tiles) gated_publish(ch.pairs + n * d + cc, gated_pair(At, Rt));
#pragma unroll
    for (int g = 0; g < NG; ++g) {  // the state that each run starts from
      const float hg = sH[g][j];
      sH[g][j] = state;
      state = cuts[g] & 1 ? hg : __builtin_fmaf(sA[g][j], state, hg);
    }
    if (waits) from = gated_state(in, ch, d, c0, threadIdx.x);
    if (n + 1 < tiles && (n + 1) >> ch.group << ch.group == n + 1)
      gated_publish(ch.states + (n >> ch.group) * d + cc, __float_as_uint(At < 0.0f ? Rt : __builtin_fmaf(At, from, Rt)));
#pragma unroll
    for (int g = NG - 1; g >= 0; --g) {  // what each run's last token is handed
      const float Rg = sR[g][j];
      sR[g][j] = from;
      from = cuts[g] & 2 ? Rg : __builtin_fmaf(sA[g][j], from, Rg);
    }
  }
  lds_barrier();
  if (o.dstate_in != nullptr) gated_empty(a.cu, a.S, tile, tiles, o.dstate_out, o.dstate_in, d, c0, C);
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    h[i] = sH[run][lane * V + i];
    R[i] = sR[run][lane * V + i];
    sum[i] = 0.0f;
  }
  if (on) {
    uint32_t step, off = offset(o.dz_ts, step);
    gmem<IO>* base = sbase(static_cast<IO*>(o.dz) + t0 * o.dz_ts + c0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      again(rr[k]);
      again(rg[k]);
      if (cut) {
        const Place p = place[run * K + k];
        if (p.starts()) {
#pragma unroll
          for (int i = 0; i < V; ++i) h[i] = a.state_in != nullptr ? a.state_in[p.seq() * d + c + i] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float before = h[i];
        h[i] = __builtin_fmaf(da[k][i], h[i], db[k][i]);
        db[k][i] = before;
      }
      if (a.z != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) dz[k][i] *= h[i];
        if (whole || k < left) store_chans<IO, V>(base, off, dz[k]);
        off += step;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    uint32_t sx, sr, sg;
    uint32_t ox = offset(o.dx_ts, sx) + K * sx, og = offset(o.dg_ts, sg) + K * sg, orr = offset(o.dr_ts, sr) + K * sr;
    gmem<IO>* const bx = sbase(static_cast<IO*>(o.dx) + t0 * o.dx_ts + c0);
    gmem<IO>* const br = sbase(static_cast<IO*>(o.dr) + t0 * o.dr_ts + c0);
    gmem<IO>* const bg = sbase(static_cast<IO*>(o.dg) + t0 * o.dg_ts + c0);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      const Place p = cut ? place[run * K + k] : Place{0};
      if (p.ends()) {
#pragma unroll
        for (int i = 0; i < V; ++i) R[i] = 0.0f;
      }
      ox -= sx;
      orr -= sr;
      og -= sg;
      const bool here = whole || k < left;
      float G[V], u[V], dr[V], dx[V], dg[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        G[i] = sD[k][threadIdx.x][i] + R[i];
        R[i] = da[k][i] * G[i];
        u[i] = rx[k][i];
        dx[i] = G[i];
      }
      if (a.g != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const Sigmoids s = sigmoids(rg[k][i]);
          u[i] *= s.s;
          dx[i] *= s.s;
          dg[i] = s.s1 * u[i] * G[i];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Sigmoids s = sigmoids(rr[k][i]);
        const float av = da[k][i], before = db[k][i];
        float m;
        if constexpr (LAM) {
          const float l = -kap[i] * s.s, m2 = gated_m2(l, av);
          const float rm = __builtin_amdgcn_rsqf(__builtin_elementwise_maximum(m2, 1.2e-38f)), L = l * kLn2;
          m = m2 * rm;
          const float e = R[i] * L * __builtin_fmaf(-u[i] * av, rm, before);
          sum[i] += e;
          dr[i] = e * s.s1;
        } else {
          m = s.s1;
          dr[i] = G[i] * (before - u[i]) * s.s * s.s1;
        }
        dx[i] *= m;
        dg[i] *= m;
      }
      if (here) {
        store_chans<IO, V>(br, orr, dr);
        store_chans<IO, V>(bx, ox, dx);
        if (a.g != nullptr) store_chans<IO, V>(bg, og, dg);
      }
      if (p.starts() && o.dstate_in != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) o.dstate_in[p.seq() * d + c + i] = R[i];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (LAM) {
#pragma unroll
    for (int i = 0; i < V; ++i) sA[run][lane * V + i] = sum[i];
    lds_barrier();
    if (chain) {
      float t = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) t += sA[g][threadIdx.x];
      o.part[tile * d + cc] = t;
    }
  }
}

// dlam from the tiles' sums.  sigmoid / softplus tends to 1 for lam -> -infinity.
__global__ __launch_bounds__(256) void k_gated_dlam(const float* __restrict__ part, int64_t parts, int d,
                                                    const float* __restrict__ lam, float* __restrict__ dlam) {
  const int c = blockIdx.x * kPartColumns + threadIdx.x % kPartColumns;
  const float v = sum_parts(part, parts, d, c);
  if (c >= d || threadIdx.x >= kPartColumns) return;
  const float l = lam[c];
  dlam[c] = v * (l < -20.0f ? 1.0f : sigmoid(l) / (l != l ? l : softplus(l)));
}

int64_t gated_blocks(int64_t T) { return cdiv(T, MM_GATED_BLOCK); }  // checkpoints
int64_t gated_tiles(int64_t T) { return cdiv(T, kGatedTile); }

int check_gated(int64_t S, int64_t T, int32_t d, float c, int32_t gate, int32_t io) {
  const int rc = check_tokens(S, T, d, io);
  if (rc != MM_OK) return rc;
  if (gate != MM_GATE_SILU && gate != MM_GATE_GELU) return MM_ERR_UNSUPPORTED;
  if (!(c >= 0.0f) || std::isinf(c)) return MM_ERR_DIM;
  if (S >= (int64_t{1} << 29)) return MM_ERR_DIM;  // a token's place holds its sequence and two bits
  if (gated_blocks(T) * cdiv(d, 64) >= (int64_t{1} << 23)) return MM_ERR_DIM;  // workgroups of 512 threads
  return MM_OK;
}
// the chain in the workspace: the ticket, the tiles' pairs, their groups' states
constexpr size_t kTicketBytes = kGatedQueues * kGatedQueueStep * 4;
// log2 of a group's tiles: 4, more (up to 32) where a chain would have more than 128 links.  A tile's looks grow with its
// group, a chain's links shrink: 65536 x 8192 with groups of 4 1147 us, of 8 1160; 262144 x 256 with groups of 4 406, of 16
// 191.
int gated_group(int64_t tiles) {
  int g = 2;
  while (g < 5 && tiles >> g > 128) ++g;
  return g;
}
struct ChainLayout {
  int64_t pairs, states;  // elements
  size_t total;
};
ChainLayout chain_layout(int64_t tiles, int32_t d) {
  if (tiles <= 1) return {0, 0, 0};
  const int64_t pairs = tiles * d, states = (tiles >> gated_group(tiles)) * d;
  return {pairs, states, align256(kTicketBytes + static_cast<size_t>(pairs + states) * 8)};
}
// Clears the chain of a call's tiles, and sees to its empty sequences where the tiles do not (e.out == NULL: nobody does).
GatedChain start_chain(int64_t tiles, int32_t d, void* ws, hipStream_t st, EmptySlots e) {
  const ChainLayout l = chain_layout(tiles, d);
  const bool chain = l.total > 0, slots = e.out != nullptr && e.S > tiles * kTileSlots;
  u64* p = chain ? reinterpret_cast<u64*>(static_cast<char*>(ws) + kTicketBytes) : nullptr;
  const int64_t n = l.pairs + l.states, rest = slots ? cdiv(e.S, kEmptySlots) * cdiv(d, kEmptyChannels) : 0;
  if (chain || slots)
    hipLaunchKernelGGL(k_gated_begin, dim3(static_cast<unsigned>(cdiv(n, 256) + rest)), dim3(256), 0, st, p, n, static_cast<uint32_t*>(ws), e);
  return chain ? GatedChain{p, p + l.pairs, static_cast<uint32_t*>(ws), gated_group(tiles)} : GatedChain{};
}
// the backward's workspace: a chain (the forward's first, where the states are made again), the tiles' sums, those states
struct BackwardLayout {
  size_t part, ckpt, total;
};
BackwardLayout backward_layout(int64_t T, int32_t d, bool has_ckpt) {
  const int64_t n = gated_blocks(T) * d;
  BackwardLayout l;
  l.part = std::max(chain_layout(gated_blocks(T), d).total, chain_layout(gated_tiles(T), d).total);
  l.ckpt = l.part + align256(static_cast<size_t>(n) * 4);
  l.total = l.ckpt + (has_ckpt ? 0 : align256(static_cast<size_t>(n) * 4));
  return l;
}
// f(V as a type) for d channels: as many of them, up to 4, as let every thread's be all there or all missing.  16384 x 4096
// of bfloat16 with 4: 173 us, with 2: 175 (both spill, see k_gated); single ones make rows of 128 bytes (193).
template <typename IO, typename F>
int by_channels(int32_t d, F f) {
  if (d % 4 == 0) return f(std::integral_constant<int, 4>{});
  if constexpr (sizeof(IO) == 2)
    if (d % 2 == 0) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}
// rows at least d apart, and near enough for the offsets within a tile to have 32 bits
int check_strides(int32_t d, std::initializer_list<int64_t> ts) {
  for (int64_t s : ts)
    if (s < d) return MM_ERR_DIM;
  for (int64_t s : ts)
    if (s > MM_LAYER_MAX_STRIDE) return MM_ERR_UNSUPPORTED;
  return MM_OK;
}
GatedArgs gated_args(const void* x, const void* r, const void* g, const void* z, const float* lam, const int32_t* cu,
                     const float* state_in, int64_t x_ts, int64_t r_ts, int64_t g_ts, int64_t z_ts, int64_t T, int S, int d,
                     float c, int gate) {
  return GatedArgs{x, r, g, z, lam, cu, state_in, x_ts, r_ts, g_ts, z_ts, T, S, d, c, gate == MM_GATE_GELU};
}
}  // namespace
}  // namespace mm

using namespace mm;

extern "C" {

size_t mamba_mixer_gated_prefill_workspace_bytes(int64_t T, int32_t d) {
  if (check_gated(1, T, d, 0.0f, MM_GATE_SILU, MM_IO_F32) != MM_OK) return 0;
  return chain_layout(gated_tiles(T), d).total;
}

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
  if ((rc = check_strides(d, {x_stride, r_stride, g != nullptr ? g_stride : d, z != nullptr ? z_stride : d})) != MM_OK) return rc;
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
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    return by_channels<IO>(d, [&](auto v) {
      constexpr int V = decltype(v)::value;
      const EmptySlots e{cu_seqlens, state_in, state_out != state_in ? state_out : nullptr, d, S};
      const GatedChain ch = start_chain(gated_tiles(T), d, workspace, st, e);
      if (T == 0) return launched();
      const dim3 grid(static_cast<unsigned>(gated_tiles(T) * cdiv(d, GatedShape<IO, V, kGatedTile>::C)));
      IO* const out = static_cast<IO*>(y);
      if (lam != nullptr) hipLaunchKernelGGL((k_gated<IO, V, true, true>), grid, dim3(kGatedThreads), 0, st, a, ch, state_out, out, ckpt);
      else hipLaunchKernelGGL((k_gated<IO, V, false, true>), grid, dim3(kGatedThreads), 0, st, a, ch, state_out, out, ckpt);
      return launched();
    });
  });
}

int mamba_mixer_gated_decode(const void* x, const void* r, const void* g, const void* z, const float* lam,
                             const float* state_in, float* state_out, void* y, int32_t Bs, int32_t d, float c,
                             int32_t gate, int32_t io_dtype, int64_t x_stride, int64_t r_stride, int64_t g_stride,
                             int64_t z_stride, void* stream) {
  int rc = check_gated(Bs, Bs, d, c, gate, io_dtype);
  if (rc != MM_OK) return rc;
  const GatedArgs a = gated_args(x, r, g, z, lam, nullptr, state_in, x_stride, r_stride, g_stride, z_stride, Bs, Bs, d, c, gate);
  if ((rc = check_strides(d, {x_stride, r_stride, g != nullptr ? g_stride : d, z != nullptr ? z_stride : d})) != MM_OK) return rc;
  const int64_t n = static_cast<int64_t>(Bs) * d;
  if (n == 0) return MM_OK;
  const size_t es = esize(io_dtype);
  rc = check_args({strided(x, Bs, d, x_stride, es), strided(r, Bs, d, r_stride, es), strided(g, Bs, d, g_stride, es, true),
                   strided(z, Bs, d, z_stride, es, true), flat(lam, d, 4, true), flat(state_in, n, 4, true)},
                  {flat(state_out, n, 4), flat(y, n, es)}, {{0, 5}});
  if (rc != MM_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    return by_channels<IO>(d, [&](auto v) {
      constexpr int V = decltype(v)::value;
      const dim3 grid(static_cast<unsigned>(cdiv(n, 256 * V)));
      if (lam != nullptr) hipLaunchKernelGGL((k_gated_decode<IO, V, true>), grid, dim3(256), 0, st, a, state_out, static_cast<IO*>(y));
      else hipLaunchKernelGGL((k_gated_decode<IO, V, false>), grid, dim3(256), 0, st, a, state_out, static_cast<IO*>(y));
      return launched();
    });
  });
}

size_t mamba_mixer_gated_backward_workspace_bytes(int64_t T, int32_t d, int32_t has_ckpt) {
  if (check_gated(1, T, d, 0.0f, MM_GATE_SILU, MM_IO_F32) != MM_OK) return 0;
  return backward_layout(T, d, has_ckpt != 0).total;
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
  rc = check_strides(d, {x_stride, r_stride, g != nullptr ? g_stride : d, z != nullptr ? z_stride : d, dx_stride, dr_stride,
                         g != nullptr ? dg_stride : d, z != nullptr ? dz_stride : d});
  if (rc != MM_OK) return rc;
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
  const BackwardLayout l = backward_layout(T, d, ckpt != nullptr);
  char* ws = static_cast<char*>(workspace);
  float* part = reinterpret_cast<float*>(ws + l.part);
  float* states = reinterpret_cast<float*>(ws + l.ckpt);
  const GatedGrads o{dy, dstate_out, ckpt != nullptr ? ckpt : states, dx, dr, dg, dz, dx_stride, dr_stride, dg_stride, dz_stride,
                     dstate_in, part};
  return by_io(io_dtype, [&](auto io) {
    using IO = decltype(io);
    return by_channels<IO>(d, [&](auto v) {
      constexpr int V = decltype(v)::value;
      const int64_t tiles = gated_blocks(T);
      if (ckpt == nullptr && T > 0) {
        const dim3 forward(static_cast<unsigned>(gated_tiles(T) * cdiv(d, GatedShape<IO, V, kGatedTile>::C)));
        const GatedChain ch = start_chain(gated_tiles(T), d, workspace, st, EmptySlots{});
        IO* const none = nullptr;
        if (lam != nullptr) hipLaunchKernelGGL((k_gated<IO, V, true, false>), forward, dim3(kGatedThreads), 0, st, a, ch, nullptr, none, states);
        else hipLaunchKernelGGL((k_gated<IO, V, false, false>), forward, dim3(kGatedThreads), 0, st, a, ch, nullptr, none, states);
      }
      const GatedChain ch = start_chain(tiles, d, workspace, st, EmptySlots{cu_seqlens, dstate_out, S > 0 ? dstate_in : nullptr, d, S});
      if (T > 0) {
        const dim3 grid(static_cast<unsigned>(tiles * cdiv(d, GatedShape<IO, V, kGatedBwdTile>::C)));
        if (lam != nullptr) hipLaunchKernelGGL((k_gated_bwd<IO, V, true>), grid, dim3(kGatedThreads), 0, st, a, ch, o);
        else hipLaunchKernelGGL((k_gated_bwd<IO, V, false>), grid, dim3(kGatedThreads), 0, st, a, ch, o);
      }
      if (lam != nullptr)
        hipLaunchKernelGGL(k_gated_dlam, dim3(static_cast<unsigned>(cdiv(d, kPartColumns))), dim3(256), 0, st, part, tiles, d, lam, dlam);
      return launched();
    });
  });
}

}  // extern "C"
