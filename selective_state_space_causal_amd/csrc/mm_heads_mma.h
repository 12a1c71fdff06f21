// The head scan on the matrix cores (bfloat16 io), 64 tokens at a time.  With c the inclusive sum of
// log a in a 64-token chunk and h0 the state at its start:
//   y_i = e^{c_i} h0 C_i + sum_{j<=i} M_ij x_j + D x_i,   M_ij = (C_i . B_j) e^{c_i - c_j} delta_j
//   h   = e^{c_63} h0 + sum_j e^{c_63 - c_j} delta_j x_j B_j^T
// Every exponent is <= 0.  A workgroup (4 waves) walks a segment with two blocks of 64 head channels
// of one group, which share B, C and the products C . B; a wave owns 32 of the 128 columns and keeps
// their states, transposed [N][32], in its accumulators for the whole walk, so a state touches
// memory only at the segment's ends.
//
// Operands of v_mfma_f32_16x16x32_bf16: lane l supplies row (or column) l % 16 and eight K indices
// of the group g = l / 16; the result leaves rows 4g .. 4g+3 of column l % 16.  The K order is free as
// long as both operands share it; with the order {4g .. 4g+3, 16+4g .. 16+4g+3} a result pair is an
// operand as it stands: the state's accumulators are the operand of h0 C, without a transposition.  x
// and B enter the products over tokens transposed, which LDS transpose reads (4 x 16 elements per
// 16 lanes) give from their natural layout.
//
// Precision: x, B and C are exact operands; M and h0 are rounded to bfloat16 for their products, whose
// sums are float32 and leave in bfloat16.  Where the walk makes the final states, float32 results, the
// products that update the state take e^{..} delta x in three bfloat16 parts (PARTS = 3: 24 bits).
// Where sequences are cut into segments, the states between them and at the ends come from
// k_heads_states with that precision, this walk's state serves y alone, and one part does.
//
// Two blocks of 64 channels a workgroup, because C . B and the staged B and C serve both; one block, with three
// workgroups to a CU, ran out of registers and took 590 us where two took 260.  A chunk is a chain of two barriers,
// the products C . B, their decay, and two more products, and two workgroups (2 waves per SIMD: 245 registers, 75 KB
// of LDS) overlap only in part: VALU issue 34%, MFMA 16% of the cycles, waves waiting 38%, LDS bank conflicts 15%.
// Traced means, inputs of successive calls in different memory: 16384 packed tokens of 64 heads 64 x 128, one group, 120 us
// (325 MB, 2.7 TB/s; the call 228); 32768 tokens of 80 heads, 8 groups, 281 us (3.5 TB/s; the call 450).
#pragma once

#include <type_traits>

#include "mm_heads.h"

namespace mm {

typedef __bf16 hb8 __attribute__((ext_vector_type(8)));
typedef __bf16 hb4 __attribute__((ext_vector_type(4)));
typedef __bf16 hb2 __attribute__((ext_vector_type(2)));
typedef short hs4 __attribute__((ext_vector_type(4)));
typedef float hf4 __attribute__((ext_vector_type(4)));
typedef float hf2 __attribute__((ext_vector_type(2)));
typedef uint32_t hu4 __attribute__((ext_vector_type(4)));
typedef uint32_t hu2 __attribute__((ext_vector_type(2)));

constexpr int kMmaTok = 64;      // tokens per chunk
constexpr int kMmaThreads = 256;
constexpr int kMmaCols = 128;    // head channels per workgroup: two blocks of 64
constexpr int kMmaMaxStride = MM_HEADS_MAX_STRIDE;  // elements between rows: a chunk's offsets stay far below 2^31
constexpr int kMmaPastEnd = 0x40000000;  // a buffer offset past every range

struct MmaArgs {
  Tok<uint16_t> x, B, C;
  int P, N;
  int npb;     // 64-channel blocks per head
  int vper;    // such blocks per group
  int ppg;     // pairs of them per group
  int pairs;   // in all
  int64_t Ls;
  const float* state_in;
  float* state_out;
  const float* carry;  // [rows] the states of the segments' starts, or NULL: whole sequences from state_in
  uint16_t* y;
  int64_t even;  // not 0: whole sequences (PARTS = 3) only if none is longer, stretches only if one is
};

// Tiles in LDS are rows of PC 16-byte pieces without padding.  Piece c of row r lies at c ^ swz(r): for any
// 16 rows one piece of each (operands in natural order), and for any 8 rows a pair of pieces of each (transpose
// reads of 32 lanes), fall on different banks.
template <int PC>
__device__ __forceinline__ int swz(int row) {
  constexpr int LP = PC == 16 ? 4 : PC == 8 ? 3 : 2;
  const int u = (row >> (4 - LP)) & (PC - 1);
  return ((u << 1) & (PC - 1)) | (u >> (LP - 1));
}
// byte offset of (row, column) of such a tile of bfloat16
template <int PC>
__device__ __forceinline__ int tile_at(int row, int col) {
  return row * (PC * 16) + (((col >> 3) ^ swz<PC>(row)) << 4) + ((col & 7) << 1);
}
constexpr int kMmaXP = kMmaCols / 8;  // pieces per row of the x tile
constexpr int kMmaMP = kMmaTok / 8;   // and of M

// per-token factors of a head block, in LDS
enum { kFci, kFcf, kFdel, kFe, kFw, kFw16, kFe16, kFn = kFe16 + 3 };
constexpr int kMmaFSet = 2 * kFn * kMmaTok + 4;  // the factors of two blocks, and their e^{c_63}
template <int NK>
struct MmaGeo {
  static constexpr int NP = NK * 32, PC = NP / 8;  // N padded; its pieces
  static constexpr int B = 0, C = B + kMmaTok * NP * 2, X = C + kMmaTok * NP * 2, M = X + kMmaTok * kMmaCols * 2,
                       F = M + 2 * kMmaTok * kMmaTok * 2, bytes = F + 2 * kMmaFSet * 4 + 16;
};

__device__ __forceinline__ hf4 mfma(hb8 a, hb8 b, hf4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ hb8 join(hb4 a, hb4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
// elements [row][16 t .. 16 t + 15] of 4 rows per 16 lanes, transposed: lane gets column l % 16 of rows 4g .. 4g+3
__device__ __forceinline__ hb4 tr_read(const char* p) {
  return __builtin_bit_cast(hb4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) hs4*)(p)));
}
__device__ __forceinline__ hb4 lds4(const char* p) { return *reinterpret_cast<const hb4*>(p); }
__device__ __forceinline__ hb8 lds8(const char* p) { return *reinterpret_cast<const hb8*>(p); }
__device__ __forceinline__ hb2 to_bf2(float a, float b) {
  const hf2 v = {a, b};
  return __builtin_convertvector(v, hb2);
}
__device__ __forceinline__ hb4 to_bf4(hf4 v) { return __builtin_convertvector(v, hb4); }
__device__ __forceinline__ hf4 to_f4(hb4 v) { return __builtin_convertvector(v, hf4); }

// Inclusive sum over the 64 lanes in double: the exponents' differences are taken in whole and
// fractional parts (below), which needs the sums beyond float32.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u), CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double lane_scan(double v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr:1
  v = dpp_add<0x112, 0xF>(v);  // row_shr:2
  v = dpp_add<0x114, 0xF>(v);  // row_shr:4
  v = dpp_add<0x118, 0xF>(v);  // row_shr:8
  v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(u), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(u >> 32), 63);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// A token's exponent (log2 of its decay) for the sums.  Below 2^-512 a decay is 0 in float32 whatever it multiplies,
// and the sums stay finite; a NaN stays one.
__device__ __forceinline__ double exponent(float del, float A2) {
  return static_cast<double>(__builtin_elementwise_maximum(del * A2, -512.0f));
}

// eight float32 as bfloat16 parts; the sum of three has all 24 bits (of a value that is not finite the first part
// says so and the others are NaN or zero)
template <int PARTS>
__device__ __forceinline__ void bf_parts(hf4 a, hf4 b, hb8 (&part)[PARTS]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float v[2] = {e < 4 ? a[e & 3] : b[e & 3], e < 4 ? a[(e + 1) & 3] : b[(e + 1) & 3]};
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
      const hb2 o = to_bf2(v[0], v[1]);
      part[k][e] = o[0];
      part[k][e + 1] = o[1];
      v[0] -= static_cast<float>(o[0]);
      v[1] -= static_cast<float>(o[1]);
    }
  }
}
// the same of w x, the weights of the operand's K indices in w0 and w1
template <int PARTS>
__device__ __forceinline__ void weighted_parts(hb8 x, hf4 w0, hf4 w1, hb8 (&part)[PARTS]) {
  hf4 a, b;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = w0[e] * static_cast<float>(x[e]);
    b[e] = w1[e] * static_cast<float>(x[4 + e]);
  }
  bf_parts(a, b, part);
}

// Rows of a token tensor from token tb on as a range-checked buffer: rows from `cnt` on read as zeros (and
// stores to them are dropped), so nothing branches on a sequence's end.
typedef __amdgpu_buffer_rsrc_t hbuf;
__device__ __forceinline__ hbuf token_rows(const uint16_t* p, int64_t tb, int64_t ts, int cnt, int row) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p + tb * ts), 0,
                                           static_cast<int>(((cnt - 1) * ts + row) * 2), 0x00020000);
}
// eight elements at byte offset `off`, of which `n` exist in the row
template <bool VEC>
__device__ __forceinline__ hu4 load8(hbuf b, int off, int n) {
  if (VEC) return __builtin_bit_cast(hu4, __builtin_amdgcn_raw_buffer_load_b128(b, n > 0 ? off : kMmaPastEnd, 0, 0));
  hu4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(b, 2 * i < n ? off + 4 * i : kMmaPastEnd, 0, 0);
    const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(b, 2 * i + 1 < n ? off + 4 * i + 2 : kMmaPastEnd, 0, 0);
    v[i] = (lo & 0xFFFFu) | (hi << 16);
  }
  return v;
}
template <bool VEC>
__device__ __forceinline__ void store8(hbuf b, int off, int n, hu4 v) {
  if (VEC) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), b, n > 0 ? off : kMmaPastEnd, 0, 0);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2))), b,
                                          i < n ? off + 2 * i : kMmaPastEnd, 0, 0);
}
// nonzero if one of the values is not finite: an exponent of ones carries into the sign's place
__device__ __forceinline__ uint32_t not_finite(hu4 v) {
  uint32_t f = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) f |= ((v[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  return f;
}

// Workgroups are dealt to the eight XCDs in turn, each with an L2 of its own.  Those of one unit (`size` neighbours,
// which read the same B and C) go to one XCD, so that its L2 serves all but the first; the units go in turn.  A number
// of units that eight does not divide leaves the last ones as they come.
__device__ __forceinline__ int xcd_unit(int b, int blocks, int size) {
  constexpr int kXcds = 8;
  const int even = blocks / size / kXcds * kXcds * size;
  if (b >= even) return b;
  const int i = b / kXcds;
  return (i / size * kXcds + b % kXcds) * size + i % size;
}

template <int NK, int PARTS, bool VEC>
__global__ __launch_bounds__(kMmaThreads, 2) void k_heads_mma(MmaArgs q, HeadPar hp) {
  typedef MmaGeo<NK> G;
  constexpr int NT = 2 * NK, PC = G::PC;
  extern __shared__ __align__(16) char lds[];
  char *const sB = lds + G::B, *const sC = lds + G::C, *const sX = lds + G::X;
  float* const sF = reinterpret_cast<float*>(lds + G::F);  // two sets: this chunk's and the next one's
  int* const sFlag = reinterpret_cast<int*>(sF + 2 * kMmaFSet);

  if (q.even > 0 && longer_than(hp.cu, hp.S, q.even) == (PARTS == 3)) return;
  const int tid = threadIdx.x;
  int lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wg = xcd_unit(blockIdx.x, gridDim.x, q.ppg);
  const int pair = wg % q.pairs;
  SegmentWalk walk(hp.cu, hp.S, wg / q.pairs, q.Ls, PARTS == 3);

  // the wave's block of head channels, and where its columns lie
  const int group = pair / q.ppg, blk = wave >> 1;
  const int in_group = 2 * (pair % q.ppg);
  const bool have = in_group + blk < q.vper;
  const int vh = group * q.vper + in_group + (have ? blk : 0);
  const int h = vh / q.npb, p0 = (vh % q.npb) * 64;
  const int pw = q.P - p0 < 64 ? q.P - p0 : 64;  // channels of the block
  const int col0 = (wave & 1) * 32;              // the wave's first column in it
  const int64_t PN = static_cast<int64_t>(q.P) * q.N, set = hp.H * PN;
  char* const sM = lds + G::M + blk * (kMmaTok * kMmaTok * 2);
  const float Dh = hp.D != nullptr ? hp.D[h] : 0.0f;

  Segment sg;
  int64_t rho;
  while (walk.next(sg, rho)) {
  hf4 st[NT][2];  // the state: [n = 16 nt + 4g + r][column 16 ct + li]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) st[nt][ct] = hf4{0, 0, 0, 0};
  {
    const float* from = q.carry != nullptr ? q.carry + rho * set : (q.state_in ? q.state_in + sg.s * set : nullptr);
    if (from != nullptr && have)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        const int p = col0 + 16 * ct + li;
        if (p < pw)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int n = 16 * nt + 4 * g;
            const float* a = from + h * PN + static_cast<int64_t>(p0 + p) * q.N + n;
            if (VEC) {
              if (n < q.N) st[nt][ct] = *reinterpret_cast<const hf4*>(a);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (n + r < q.N) st[nt][ct][r] = a[r];
            }
          }
      }
  }

  // staging: a thread's pieces of the B and C tiles are (row0 + i rows, col), of the x tile (xrow + 16 i, xcol)
  const int brow = tid / PC, bcol = (tid % PC) * 8;
  constexpr int bstep = kMmaThreads / PC;
  const int xrow = tid >> 4, xcol = (tid & 15) * 8, xv = group * q.vper + in_group + (xcol >> 6);
  const int xin = (xv % q.npb) * 64 + (xcol & 63);  // column in its head
  const int xn = in_group + (xcol >> 6) < q.vper ? q.P - xin : 0, bn = q.N - bcol;
  const int dH = hp.H * q.P, gn = (hp.H / q.B.div) * q.N;
  const int b_off = (brow * static_cast<int>(q.B.ts) + group * q.N + bcol) * 2;
  const int c_off = (brow * static_cast<int>(q.C.ts) + group * q.N + bcol) * 2;
  const int x_off = (xrow * static_cast<int>(q.x.ts) + (xv / q.npb) * q.P + xin) * 2;
  hu4 rB[NK], rC[NK], rX[4];
  const auto load = [&](int64_t tb) {
    const int cnt = static_cast<int>(sg.t1 - tb < kMmaTok ? sg.t1 - tb : kMmaTok);
    const hbuf bB = token_rows(q.B.p, tb, q.B.ts, cnt, gn), bX = token_rows(q.x.p, tb, q.x.ts, cnt, dH);
    const hbuf bC = token_rows(q.C.p, tb, q.C.ts, cnt, gn);
#pragma unroll
    for (int i = 0; i < NK; ++i) rB[i] = load8<VEC>(bB, b_off + i * bstep * static_cast<int>(q.B.ts) * 2, bn);
#pragma unroll
    for (int i = 0; i < NK; ++i) rC[i] = load8<VEC>(bC, c_off + i * bstep * static_cast<int>(q.C.ts) * 2, bn);
#pragma unroll
    for (int i = 0; i < 4; ++i) rX[i] = load8<VEC>(bX, x_off + i * 16 * static_cast<int>(q.x.ts) * 2, xn);
  };

  // LDS offsets of a lane's operands: one base for each kind, the tiles at constants from it (exclusive or within a
  // row, added between rows).  The bases are opaque in each chunk: kept as invariants, the sums of all of them
  // would take some 50 registers.
  const int w8 = 8 * blk + (col0 >> 3);  // the wave's first piece in a row of the x tile
  int aN = tile_at<PC>(li, 8 * g);                                   // row li, 8 columns
  int aK = tile_at<PC>(li, 4 * g);                                   // row li, 4 columns
  int aT = tile_at<PC>(4 * g + (li >> 2), 4 * (li & 3));             // transposed
  int xT = tile_at<kMmaXP>(4 * g + (li >> 2), 8 * w8 + 4 * (li & 3));
  int xK = tile_at<kMmaXP>(li, 8 * w8 + 4 * g);
  int xN = tile_at<kMmaXP>(li, 8 * w8 + 8 * g);
  int mK = tile_at<kMmaMP>(li, 4 * g);
  constexpr int R16 = 16 * PC * 16, X16 = 16 * kMmaXP * 16, M16 = 16 * kMmaMP * 16;  // bytes of 16 rows

  // The tokens' factors: wave 0 makes those of block 0, wave 1 those of block 1, a chunk ahead of their use.
  const bool dhave = in_group + wave < q.vper;
  const int dh = (group * q.vper + in_group + (dhave ? wave & 1 : 0)) / q.npb;
  const float A2 = head_A2(hp, dh), bias = hp.dt != nullptr ? hp.dt_bias[dh] : 0.0f;
  uint32_t rdt = 0;  // as loaded: its use waits for it
  const auto load_dt = [&](int64_t tb) {
    if (wave < 2 && hp.dt != nullptr && tb + lane < sg.t1)
      rdt = static_cast<const uint16_t*>(hp.dt)[(tb + lane) * hp.dt_ts + dh];
  };
  const auto factors = [&](int64_t tb, int set) {
    if (wave >= 2) return;
    float* f = sF + set * kMmaFSet + wave * (kFn * kMmaTok) + lane;
    const bool token = dhave && tb + lane < sg.t1;
    const float del = !token ? 0.0f : hp.dt == nullptr ? 1.0f : head_softplus(io_value<uint16_t>(rdt) + bias);
    const double c = lane_scan(exponent(del, A2));
    const double last = last_lane(c);
    const double whole = floor(c);
    const float ci = static_cast<float>(whole), cf = static_cast<float>(c - whole);
    f[kFe * kMmaTok] = exp2_hw(static_cast<float>(c));
    f[kFw * kMmaTok] = exp2_hw(static_cast<float>(last - c)) * del;
    {
      f[kFci * kMmaTok] = ci;
      f[kFcf * kMmaTok] = cf;
      f[kFdel * kMmaTok] = del;
      // from tile ends on: the ends' exponents from lanes 15, 31 and 47
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const float ti = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ci), 16 * t + 15));
        const float tf = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, cf), 16 * t + 15));
        const float d = (ci - ti) + (cf - tf);
        f[(kFe16 + t) * kMmaTok] = exp2_hw(d);                                    // tokens after the end
        if (lane >> 4 == t) f[kFw16 * kMmaTok] = exp2_hw(-d) * del;               // tokens up to it
      }
    }
    if (lane == 0) sF[set * kMmaFSet + 2 * kFn * kMmaTok + wave] = exp2_hw(static_cast<float>(last));
  };
  int par = 0;  // two flags in turn: one is cleared while the other may still be read
  if (tid == 0) sFlag[0] = 0;
  if (sg.t0 < sg.t1) {
    load_dt(sg.t0);
    if (VEC) load(sg.t0);
    factors(sg.t0, 0);
    load_dt(sg.t0 + kMmaTok);
  }
  for (int64_t tb = sg.t0; tb < sg.t1; tb += kMmaTok) {
    const int cnt = static_cast<int>(sg.t1 - tb < kMmaTok ? sg.t1 - tb : kMmaTok);
    if (!VEC) load(tb);  // element by element: too many registers to hold ahead
    asm volatile("" : "+v"(aN), "+v"(aK), "+v"(aT), "+v"(xT), "+v"(xK), "+v"(xN), "+v"(mK), "+v"(lane), "+v"(li), "+v"(g));
    __syncthreads();
    if (tid == 0) sFlag[par ^ 1] = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int a = tile_at<PC>(brow + i * bstep, bcol);
      *reinterpret_cast<hu4*>(sB + a) = rB[i];
      *reinterpret_cast<hu4*>(sC + a) = rC[i];
    }
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<hu4*>(sX + tile_at<kMmaXP>(xrow + 16 * i, xcol)) = rX[i];
      odd |= not_finite(rX[i]);
    }
    if (__any(odd != 0) && lane == 0) sFlag[par] = 1;
    __syncthreads();
    const bool flag = sFlag[par] != 0;
    const float* const fs = sF + par * kMmaFSet;
    const float* const f = fs + blk * (kFn * kMmaTok);
    const float el = fs[2 * kFn * kMmaTok + blk];
    par ^= 1;
    hf4 acc[4][2];  // y transposed: [p = 16 ct + 4g + r][token 16 it + li]
    {
      // C . B for 16 x 16 tiles (it, jt <= it), M of both blocks from it.  Below the diagonal's tiles the decay is
      // split at the end of tile jt, both parts <= 1: one exponential for each token instead of one for each pair.
      // All of a wave's products and factors come before its first write: a read from LDS is not moved over a write.
      const auto product = [&](auto it_, auto jt_) {  // rows j, columns i
        constexpr int it = decltype(it_)::value, jt = decltype(jt_)::value;
        hf4 raw = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < NK; ++k)
          raw = mfma(lds8(sB + jt * R16 + (aN ^ (k << 6))), lds8(sC + it * R16 + (aN ^ (k << 6))), raw);
        return raw;
      };
      struct Pair {
        hb4 b[2];
      };
      const auto decayed = [&](auto it_, auto jt_, hf4 raw) {
        constexpr int it = decltype(it_)::value, jt = decltype(jt_)::value;
        const int i = 16 * it + li, j = 16 * jt + 4 * g;
        Pair o;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float* d = fs + b * (kFn * kMmaTok);
          hf4 m;
          if (it != jt) {
            m = raw * d[(kFe16 + (jt < 3 ? jt : 0)) * kMmaTok + i] * *reinterpret_cast<const hf4*>(d + kFw16 * kMmaTok + j);
          } else {
            const float ci = d[kFci * kMmaTok + i], cf = d[kFcf * kMmaTok + i];
            const hf4 cj = *reinterpret_cast<const hf4*>(d + kFci * kMmaTok + j), fj = *reinterpret_cast<const hf4*>(d + kFcf * kMmaTok + j);
            const hf4 dj = *reinterpret_cast<const hf4*>(d + kFdel * kMmaTok + j);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float v = raw[r] * (exp2_hw((ci - cj[r]) + (cf - fj[r])) * dj[r]);
              m[r] = 4 * g + r <= li ? v : 0.0f;
            }
          }
          o.b[b] = to_bf4(m);
        }
        return o;
      };
      const auto keep = [&](auto it_, auto jt_, Pair m) {
        constexpr int it = decltype(it_)::value, jt = decltype(jt_)::value;
#pragma unroll
        for (int b = 0; b < 2; ++b)
          *reinterpret_cast<hb4*>(lds + G::M + b * (kMmaTok * kMmaTok * 2) + it * M16 + (mK ^ (jt << 5))) = m.b[b];
      };
      constexpr auto n0 = std::integral_constant<int, 0>{};
      constexpr auto n1 = std::integral_constant<int, 1>{};
      constexpr auto n2 = std::integral_constant<int, 2>{};
      constexpr auto n3 = std::integral_constant<int, 3>{};
      const auto two = [&](auto i0, auto j0, auto i1, auto j1) {
        const hf4 r0 = product(i0, j0), r1 = product(i1, j1);
        const Pair m0 = decayed(i0, j0, r0), m1 = decayed(i1, j1, r1);
        keep(i0, j0, m0), keep(i1, j1, m1);
      };
      const auto three = [&](auto i0, auto j0, auto i1, auto j1, auto i2, auto j2) {
        const hf4 r0 = product(i0, j0), r1 = product(i1, j1), r2 = product(i2, j2);
        const Pair m0 = decayed(i0, j0, r0), m1 = decayed(i1, j1, r1), m2 = decayed(i2, j2, r2);
        keep(i0, j0, m0), keep(i1, j1, m1), keep(i2, j2, m2);
      };
      if (wave == 0) {
        two(n3, n0, n3, n1);
      } else if (wave == 1) {
        two(n3, n2, n3, n3);
      } else if (wave == 2) {
        three(n2, n0, n2, n1, n2, n2);
      } else {
        three(n1, n0, n1, n1, n0, n0);
      }
      factors(tb + kMmaTok, par);
      load_dt(tb + 2 * kMmaTok);
      __builtin_amdgcn_sched_barrier(0);
      // h0 C
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) acc[it][ct] = hf4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const hb8 s0 = join(to_bf4(st[2 * k][0]), to_bf4(st[2 * k + 1][0]));
        const hb8 s1 = join(to_bf4(st[2 * k][1]), to_bf4(st[2 * k + 1][1]));
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const hb8 cc = join(lds4(sC + it * R16 + (aK ^ (k << 6))), lds4(sC + it * R16 + (aK ^ (k << 6) ^ 32)));
          acc[it][0] = mfma(s0, cc, acc[it][0]);
          acc[it][1] = mfma(s1, cc, acc[it][1]);
        }
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const float e = f[kFe * kMmaTok + 16 * it + li];
        acc[it][0] *= e;
        acc[it][1] *= e;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // x transposed: the operand of the products over tokens
    hb8 xt[2][2];  // [32 tokens ks][ct]
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        const char* a = sX + 2 * ks * X16 + (xT ^ (ct << 5));
        xt[ks][ct] = join(tr_read(a), tr_read(a + X16));
      }
    {
      __syncthreads();
      const hb4 none = to_bf4(hf4{0, 0, 0, 0});
      if (!flag) {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            if (ks == 1 && it < 2) continue;
            // the tiles above the diagonal's were not written: zeros
            const hb4 m0 = lds4(sM + it * M16 + (mK ^ (ks << 6)));
            const hb8 m = join(m0, (it & 1) == 0 && it / 2 == ks ? none : lds4(sM + it * M16 + (mK ^ (ks << 6) ^ 32)));
            acc[it][0] = mfma(xt[ks][0], m, acc[it][0]);
            acc[it][1] = mfma(xt[ks][1], m, acc[it][1]);
          }
      } else {  // a value that is not finite must not meet the zeros of earlier tokens: token by token
        for (int j = 0; j < cnt; ++j)
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) {
            const hf4 v = to_f4(lds4(sX + tile_at<kMmaXP>(j, 64 * blk + col0 + 16 * ct + 4 * g)));
#pragma unroll
            for (int it = 0; it < 4; ++it)
              if (j <= 16 * it + li)
                acc[it][ct] += v * io_value<uint16_t>(*reinterpret_cast<const uint16_t*>(sM + tile_at<kMmaMP>(16 * it + li, j)));
          }
      }
      // + D x, to bfloat16 in the x tile's place (the wave's own columns), and out in rows
      hb4 xv4[4][2];  // (read before the first write)
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) xv4[it][ct] = lds4(sX + it * X16 + (xK ^ (ct << 5)));
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
          *reinterpret_cast<hb4*>(sX + it * X16 + (xK ^ (ct << 5))) = to_bf4(to_f4(xv4[it][ct]) * Dh + acc[it][ct]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const hbuf bY = token_rows(q.y, tb, dH, cnt, dH);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * k + li, col = col0 + 8 * g;
        const hu4 v = *reinterpret_cast<const hu4*>(sX + k * X16 + xN);
        store8<VEC>(bY, (row * dH + h * q.P + p0 + col) * 2, have ? pw - col : 0, v);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (VEC && tb + kMmaTok < sg.t1) load(tb + kMmaTok);  // only now: the accumulators of y have left their registers
    // the state: e^{c_63} h0 + B^T (w x)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) st[nt][ct] *= el;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const hf4 w0 = *reinterpret_cast<const hf4*>(f + kFw * kMmaTok + 32 * ks + 4 * g);
      const hf4 w1 = *reinterpret_cast<const hf4*>(f + kFw * kMmaTok + 32 * ks + 16 + 4 * g);
      hb8 part[2][PARTS];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) weighted_parts(xt[ks][ct], w0, w1, part[ct]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const char* a = sB + 2 * ks * R16 + (aT ^ (nt << 5));
        const hb8 bt = join(tr_read(a), tr_read(a + R16));
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
          st[nt][0] = mfma(bt, part[0][k], st[nt][0]);
          st[nt][1] = mfma(bt, part[1][k], st[nt][1]);
        }
      }
    }
  }
  float* to = PARTS == 3 && sg.last() ? q.state_out + sg.s * set : nullptr;
  if (to != nullptr && have)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const int p = col0 + 16 * ct + li;
      if (p < pw)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int n = 16 * nt + 4 * g;
          float* a = to + h * PN + static_cast<int64_t>(p0 + p) * q.N + n;
          if (VEC) {
            if (n < q.N) *reinterpret_cast<hf4*>(a) = st[nt][ct];
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < q.N) a[r] = st[nt][ct][r];
          }
        }
    }
  if (PARTS != 3) __syncthreads();  // the last chunk's factors are read until here
  }
}

}  // namespace mm
