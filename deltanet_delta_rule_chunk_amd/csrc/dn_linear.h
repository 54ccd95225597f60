// dn_linear.h -- the gated linear recurrence on gfx950 matrix cores: the
// chunked product that its forward and every vector gradient of its backward
// are instances of.
//
// Per (b, h), with a log decay g_t <= 0 (0 = keep, -inf = wipe):
//     S_t = e^{g_t} S_{t-1} + k_t^T v_t,      o_t = q_t S_t.
// Over a chunk of C rows, with G_r the sum of g over the chunk's rows up to r,
//     O  = diag(e^G) Q S + (tril(Q K^T) o e^{G_r - G_i}) V
//     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V
// and every factor is a decay between two rows.  Write F(q, k, v) for this
// map and R(q, k, v) for the same map with time reversed (row t sees the rows
// at and after it).  With dS_t the gradient of the state after token t,
//     dS_t = q_t^T dO_t + e^{g_{t+1}} dS_{t+1},
//     dq_t = dO_t S_t^T,  dv_t = k_t dS_t,  dk_t = v_t dS_t^T,
// so dq = F(dO, v, k) on the transposed state, dv = R(k, q, dO) and
// dk = R(v, dO, q) on the transposed gradient: one kernel serves all four.
//
// Reversed time is only a row order: row u of a chunk is token 63 - u of it,
// and the decay in front of a row is that of the token after it.  The chunk
// boundaries stay those of forward time (a ragged last chunk then has its
// empty rows first; empty rows are zeros with no decay, an exact no-op), so
// the row sums that the decay's gradient needs line up between the passes.
//
// Parallelism over the sequence.  B H heads alone do not fill 256 CUs, so a
// head's chunks are cut into segments (split_of()).  A state kernel sums each segment from
// a zero state (it reads k and v only), a combine kernel turns the sums into
// the state entering every segment, and the output kernel walks each segment
// from there.  With one segment the output kernel runs alone.
//
// Output kernel: wave w owns 16 columns of the state, which stay
// in fp32 MFMA accumulators for the whole segment and never pass through LDS:
// the accumulator layout of two stacked 16 x 16 tiles is the operand layout
// of the next product (the "d4" slot order of dn_mfma.h), so Q S takes the
// state straight from the accumulators.  Outputs are formed as transposed
// tiles (S^T Q^T + V^T P^T): a lane then holds 4 consecutive columns of one
// row.  P is formed once per workgroup (10 tiles over its waves) and passed
// through LDS as operand fragments.
//
// Precision.  bf16 q, k, v (and dO) enter products as they are.  An fp32
// operand enters as a sum of bf16 pieces: 3 pieces (24 bits, all of fp32) wherever
// it reaches an fp32 result: the rows added to a state that is a result or enters
// a segment, the state and P read for an fp32 output, the state read for what
// the decay's gradient is summed from.  2 pieces (they leave 2^-17 of a term) only
// on the way to bf16 outputs, whose own rounding is 2^-8: the state that a walk
// reads and what it adds to it (with 3 pieces there the long forward's outputs
// take 553 us for 482), and P in the walks of dq and dk beyond 64 x 64, whose sums
// leave no LDS for a third piece beside a second workgroup.  P's third piece
// elsewhere costs 3% of the outputs' time (486 -> 501 us); without it an fp32 o is
// off by 2.3e-6 of its norm, with it by 0.8e-7.  fp32 inputs run the
// same kernels on the fp32 matrix instruction, with nothing split.  Log decays
// are summed in fp64: a difference of two sums keeps the accuracy of the short
// sum between them however long the chunk's own is.
//
// What bounds it.  32 heads of 128 x 128, bf16, L = 65536: segment sums 231 us (reads
// 1.0 GB, 4.4 TB/s), outputs 490 us (2.2 GB, 4.5 TB/s): near the rate of HBM (a
// copy reaches 5.2), with the matrix instructions busy for 45% of the time (770
// TFLOP/s as executed) and about as many cycles of vector work (pieces,
// decays) beside them, which they hardly overlap.  At few rows, the latency of a
// chunk: about 4 us, two barriers with P's way through LDS between them.
#pragma once

#include <hip/hip_runtime.h>

#include "dn_buffer.h"
#include "dn_common.h"
#include "dn_launch.h"
#include "dn_mfma.h"

namespace dn {
namespace lin {

constexpr int C = 64;  // rows of a chunk
// Waves of a workgroup: each owns 16 columns of the state.
__host__ __device__ constexpr int waves(int DV) { return DV / 16; }
constexpr double kLog2e = 1.4426950408889634074;
// Log decays (base 2) are floored here: 2^-220 is zero in fp32, so a wipe
// (-inf) is exact and differences of sums stay finite.
constexpr double kWipe2 = -220.0;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// One token's log decay in base 2.  (NaN stays NaN.)
__device__ __forceinline__ double log2_decay(float g) {
  const double x = (double)g * kLog2e;
  return x < kWipe2 ? kWipe2 : x;
}

// Whether a head's first token wipes the state it starts from, which may then be
// memory never written and is not read.  (Only there: a wipe behind it multiplies
// by 0, which leaves what is not finite so, however the sequence is cut.)
__device__ __forceinline__ bool starts_with_wipe(const float* g) { return g && exp2_hw((float)log2_decay(g[0])) == 0.f; }

// ---- operands ------------------------------------------------------------------
//
// A fragment holds, per lane (g = lane / 16, i = lane % 16), the 8 values of
// row (or column) i of a 16 x 32 operand in contraction slots e = 0 .. 7.  Two
// slot orders are in use:
//   over a row's elements:  8 g + e, so a fragment is 8 adjacent elements;
//   over rows (tokens):     4 g + e and 16 + 4 g + e - 4, what two stacked
//                           accumulator tiles hold ("d4" of dn_mfma.h).
// The state's accumulator tiles (2 kb, 2 kb + 1) then hold, in their rows
// 4 g + e, the state's rows 32 kb + 8 g + e and 32 kb + 8 g + 4 + e, so that
// they too are read in the first order: see state_row().

struct F32x8 {
  float v[8];
};

// Row of the state in accumulator tile kt, lane group g, element 0 (the
// elements are 4 adjacent rows).
__device__ __forceinline__ int state_row(int kt, int g) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1); }

// LDS tile of C rows x D, in 16-byte pieces XOR-swizzled by a function of the
// row so that row reads (16 rows, one piece) and column reads (4 or 16 rows,
// pieces 2 apart) spread over the banks.  Pieces arrive straight from HBM.
template <typename IT, int D>
struct Tile;

template <int D>
struct Tile<bf16, D> {
  typedef bf16x8 Frag;
  static constexpr int bytes = C * D * 2;
  static constexpr int PPR = D / 8;  // pieces per row
  unsigned char* p;
  // 16-byte reads are answered 16 lanes at a time, of two lane groups (lanes
  // 0-3, 12-15, 20-23, 24-27 and so on): all 16 rows once, rows 4 .. 11 of the
  // one group and the others of its neighbour.  With the low bits a Gray code of
  // row / 4 their pieces differ either way (480 bytes/ns per CU, against 287 with
  // the plain row / 4 there).
  static __device__ __forceinline__ int swizzle(int row) {
    const int hi = D == 128 ? (row & 3) << 2 : (row & 2) << 1, r = row >> 2;
    return hi | ((r ^ r >> 1) & 1) << 1 | (r & 1);
  }
  // Element offset in row r0 + row, r0 a multiple of 16 (which the swizzle does
  // not see) and row below 16.
  static __device__ __forceinline__ int off(int r0, int row, int piece) {
    return r0 * D + (row * D + ((piece ^ swizzle(row)) << 3));
  }
  __device__ __forceinline__ uint16_t* e(int off) const { return reinterpret_cast<uint16_t*>(p) + off; }
  // Row r0 + i, contraction over elements 32 kb ..
  __device__ __forceinline__ Frag row(int r0, int kb, int l) const {
    return as_bf16x8(*reinterpret_cast<const uint4*>(e(off(r0, l & 15, 4 * kb + (l >> 4)))));
  }
  __device__ __forceinline__ uint2 tr(int at) const {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(e(at))));
  }
  // Column c(i), contraction over rows 32 tb .. (transposing reads: lane
  // 4 m + a of a 16-lane group addresses row m, 4 columns; lane 4 a + b receives
  // its column b of every row).
  __device__ __forceinline__ Frag cols(int piece, int half, int tb, int l) const {
    const int r = 4 * (l >> 4) + ((l & 15) >> 2);
    return as_bf16x8(tr(off(32 * tb, r, piece) + 4 * half), tr(off(32 * tb + 16, r, piece) + 4 * half));
  }
  // ... of adjacent columns c0 + i.
  __device__ __forceinline__ Frag col(int c0, int tb, int l) const {
    return cols((c0 >> 3) + ((l & 3) >> 1), l & 1, tb, l);
  }
  // ... of the columns that are the state's rows in accumulator tile kt.
  __device__ __forceinline__ Frag state_col(int kt, int tb, int l) const {
    return cols(4 * (kt >> 1) + (l & 3), kt & 1, tb, l);
  }
};

template <int D>
struct Tile<float, D> {
  typedef F32x8 Frag;
  static constexpr int bytes = C * D * 4;
  static constexpr int PPR = D / 4;
  unsigned char* p;
  static __device__ __forceinline__ int swizzle(int row) {
    return ((row >> 2) & 1) | ((row & 3) << 1) | (row & 8);
  }
  __device__ __forceinline__ float* e(int off) const { return reinterpret_cast<float*>(p) + off; }
  __device__ __forceinline__ static int off(int row, int c) { return row * D + (((c >> 2) ^ swizzle(row)) << 2) + (c & 3); }
  __device__ __forceinline__ Frag row(int r0, int kb, int l) const {
    const int r = r0 + (l & 15), c = 32 * kb + 8 * (l >> 4);
    const f32x4 a = *reinterpret_cast<const f32x4*>(e(off(r, c)));
    const f32x4 b = *reinterpret_cast<const f32x4*>(e(off(r, c + 4)));
    return Frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  __device__ __forceinline__ Frag at_col(int c, int tb, int l) const {
    const int r = 32 * tb + 4 * (l >> 4);
    Frag f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f.v[x] = *e(off(r + x, c));
      f.v[4 + x] = *e(off(r + 16 + x, c));
    }
    return f;
  }
  __device__ __forceinline__ Frag col(int c0, int tb, int l) const { return at_col(c0 + (l & 15), tb, l); }
  __device__ __forceinline__ Frag state_col(int kt, int tb, int l) const {
    const int i = l & 15;
    return at_col(state_row(kt, i >> 2) + (i & 3), tb, l);
  }
};

// Two bf16 values packed from fp32.  (Opaque to the optimiser, which would
// otherwise convert the low value a second time for its use as fp32.)
__device__ __forceinline__ uint32_t pack_once(float a, float b) {
  uint32_t u = pack_bf16(a, b);
  asm("" : "+v"(u));
  return u;
}

// An operand made of fp32 values: NS bf16 pieces, or the values themselves.
template <typename IT, int NS>
struct Made;

template <int NS>
struct Made<bf16, NS> {
  bf16x8 p[NS];
  __device__ __forceinline__ Made() {}
  __device__ __forceinline__ explicit Made(const float (&x)[8]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = pack_once(r[2 * i], r[2 * i + 1]);
        if (s + 1 < NS) {
          r[2 * i] -= __uint_as_float(u[i] << 16);
          r[2 * i + 1] -= __uint_as_float(u[i] & 0xffff0000u);
        }
      }
      p[s] = as_bf16x8(make_uint4(u[0], u[1], u[2], u[3]));
    }
  }
};

template <int NS>
struct Made<float, NS> {
  F32x8 p;
  __device__ __forceinline__ Made() {}
  __device__ __forceinline__ explicit Made(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p.v[i] = x[i];
  }
};

// acc += A B.
__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, f32x4 c) { return mfma16(a, b, c); }
__device__ __forceinline__ f32x4 mma(const F32x8& a, const F32x8& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}
template <int NS>
__device__ __forceinline__ f32x4 mma(const Made<bf16, NS>& a, const bf16x8& b, f32x4 c) {
#pragma unroll
  for (int s = NS - 1; s >= 0; --s) c = mfma16(a.p[s], b, c);
  return c;
}
template <int NS>
__device__ __forceinline__ f32x4 mma(const bf16x8& a, const Made<bf16, NS>& b, f32x4 c) {
#pragma unroll
  for (int s = NS - 1; s >= 0; --s) c = mfma16(a, b.p[s], c);
  return c;
}
template <int NS>
__device__ __forceinline__ f32x4 mma(const Made<float, NS>& a, const F32x8& b, f32x4 c) { return mma(a.p, b, c); }
template <int NS>
__device__ __forceinline__ f32x4 mma(const F32x8& a, const Made<float, NS>& b, f32x4 c) { return mma(a, b.p, c); }

// The 8 values of a fragment as fp32.
__device__ __forceinline__ void to_floats(const bf16x8& f, float (&x)[8]) {
  const uint4 u = __builtin_bit_cast(uint4, f);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void to_floats(const F32x8& f, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = f.v[i];
}

// ---- what a chunk's rows are multiplied by ---------------------------------------

// The tables of a chunk and the next: `up` is read until the state's update, while
// the next chunk's is filled; G is not read as late as that.  A row's factor to
// the chunk's end is 1 for the last row, whose place holds the whole chunk's.
struct alignas(16) Decays {
  double G[C];      // log2 decay from the chunk's start through a row
  float up[2][C];   // by chunk's parity: 2^(G_last - G); [C - 1]: 2^G_last
};

// Row u of chunk c: token, and the log decay in front of it.
template <bool REV>
__device__ __forceinline__ int token_of(int c, int u) { return c * C + (REV ? C - 1 - u : u); }

template <bool REV>
__device__ __forceinline__ float load_decay(const float* g, int c, int L) {
  const int t = token_of<REV>(c, threadIdx.x & 63) + (REV ? 1 : 0);
  return g && t < L ? g[t] : 0.f;
}

// Lane moves within the vector ALUs (no LDS round trip).  CTRL: 0x100 + n moves
// by n lanes down and 0x110 + n up within each 16, 0x120 + n turns each 16 by n, 0x142 and
// 0x143 hand lane 15 of a 16 to the next and lane 31 to the upper 32.  Lanes
// that receive nothing get 0.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int dpp(int x) { return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false); }
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = dpp<CTRL, ROWS>((int)(uint32_t)u), hi = dpp<CTRL, ROWS>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) { return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, x))); }

// Inclusive sums over a wave's 64 lanes.
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp<0x111>(x);
  x += dpp<0x112>(x);
  x += dpp<0x114>(x);
  x += dpp<0x118>(x);
  x += dpp<0x142, 0xa>(x);
  x += dpp<0x143, 0xc>(x);
  return x;
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// One wave fills a chunk's table from its rows' log decays; returns the sum.
__device__ __forceinline__ double fill_decays(Decays* d, int chunk, float g) {
  const int l = threadIdx.x & 63;
  const double G = wave_scan(log2_decay(g)), last = lane_value(G, 63);
  d->G[l] = G;
  d->up[chunk & 1][l] = exp2_hw((float)(l == 63 ? G : last - G));
  return last;
}

// ---- staging ---------------------------------------------------------------------

typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from a buffer straight into LDS at lds + 16 lane; the
// range check of the descriptor `r` makes rows past the end zeros.  Written in
// assembly so that the compiler does not order LDS reads of other buffers
// behind it: the caller waits with wait_loads() and a barrier before reading.
// (m0 is named as changed, so that a value that the compiler keeps there is set
// again; it warns that it will not be preserved, which is what is meant.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(i32x4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(r) : "memory", "m0");
}
#pragma clang diagnostic pop
// Waits for all of this wave's vector memory operations.  (They end in order,
// and the compiler does not count those issued above, so any wait of its own for
// a load into registers waits for them too: such loads are made to arrive here,
// by passing them through keep().)
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
template <typename T>
__device__ __forceinline__ void keep(T& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ void keep(F32x8& x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) keep(x.v[i]);
}

// A workgroup's LDS: as a pointer, and as an address for load_to_lds().
struct Lds {
  unsigned char* p;
  uint32_t at;
};
__device__ __forceinline__ Lds dynamic_lds() {
  extern __shared__ __align__(16) unsigned char smem[];
  return Lds{smem, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem};
}

// Descriptor of chunk c's rows (D elements each) of a head.
template <typename IT, int D>
__device__ __forceinline__ i32x4 chunk_rsrc(const IT* base, int c, int L) {
  const uint64_t a = reinterpret_cast<uint64_t>(base + (size_t)c * C * D);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(a >> 32)) & 0xffff;
  r[2] = __builtin_amdgcn_readfirstlane(min(C, L - c * C) * D * (int)sizeof(IT));
  r[3] = 0x00020000;
  return r;
}

// A chunk's rows of one tensor on their way to an LDS tile: each of NW waves
// fills C / NW rows, its lanes 64 adjacent pieces of LDS at a time; each lane
// fetches the piece that the swizzle puts there.
template <typename IT, int D, int NW, bool REV>
struct Stage {
  typedef Tile<IT, D> T;
  static constexpr int N = C * T::PPR / (64 * NW);  // pieces per lane
  static constexpr int RPI = 64 / T::PPR;           // rows per 64 pieces
  static_assert(N * RPI * NW == C, "whole rows per wave");
  uint32_t voff[N];
  __device__ __forceinline__ Stage() {
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = (C / NW) * w + i * RPI + l / T::PPR, piece = (l % T::PPR) ^ T::swizzle(row);
      voff[i] = (uint32_t)((REV ? C - 1 - row : row) * D * (int)sizeof(IT) + piece * 16);
    }
  }
  // `base` is the head's first row, `tile` the tile's address in LDS.
  __device__ __forceinline__ void load(const IT* base, int c, int L, uint32_t tile) const {
    const i32x4 r = chunk_rsrc<IT, D>(base, c, L);
    const uint32_t lds = __builtin_amdgcn_readfirstlane((int)(tile + (threadIdx.x >> 6) * (T::bytes / NW)));
#pragma unroll
    for (int i = 0; i < N; ++i) load_to_lds(r, voff[i], lds + i * 1024);
  }
};

// ---- the state kernel --------------------------------------------------------------

// A tensor's head for state head bh: bh / div (heads shared by div state heads).
struct Src {
  const void* p;
  int div;
  template <typename IT>
  __device__ __forceinline__ const IT* head(int bh, int L, int D) const {
    return static_cast<const IT*>(p) + (size_t)(bh / div) * L * D;
  }
};

// Segments of a head: chunks per segment and their number.
struct Split {
  int nc, cps, nseg;
};

// How many segments.  More of them fill the 256 CUs and shorten the walks; each
// costs a state's write and two reads and a step of the combination, and more
// than one costs two launches.  An estimate in us decides, from times measured at
// few rows: a walk's start, its chunks (the segment sums' take about half),
// two bf16 workgroups on a CU taking up to 1.6 times as long as one (fp32: one per
// CU).  Against segments of 4 chunks at the least and 512 workgroups for every
// call, forward + backward: 4 bf16 heads of 128 x 128, L = 2000 100 -> 80 us of
// kernels, 32 heads, L = 600 105 -> 91; 4 fp32 heads of 64 x 64, L = 1000 108 -> 64;
// forward of 16 fp32 heads of 128 x 128, L = 2000 95 -> 69.  Long sequences of few
// heads come out at 512 workgroups (32 heads of 128 x 128, L = 65536, P in 2 pieces:
// 711 us of kernels; with 1024 798, 384 798, 256 818).
// None is longer than kMaxChunks, which bounds how far the decay's gradient is
// carried from an exact value.
constexpr int kMaxChunks = 256;
struct WalkTime {
  double pair, slots;  // of two workgroups on a CU against one; workgroups the card takes
  // n workgroups of cps chunks each: full rounds of the card, and a last one.
  double us(double n, int cps, double per_chunk) const {
    const double full = (double)(long long)(n / slots), rest = n - full * slots;
    return (2.5 + cps * per_chunk) * (full * pair + (rest > 256 ? pair : rest > 0 ? 1.0 : 0.0));
  }
};
inline Split split_of(int BH, int L, int d_k, int d_v, bool f32, bool bwd) {
  Split best{cdiv(L, C), 0, 0};
  const int nc = best.nc, d = d_k + d_v, fill = cdiv(512, BH);
  const double chunk = f32 ? d / 20.0 : 0.7 + d / 64.0;
  const WalkTime t{f32 ? 1.0 : 1.0 + 0.6 * d / 256, f32 ? 256.0 : 512.0};
  double least = 0.0;
  for (const int k : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64, fill}) {
    Split s{nc, cdiv(nc, k), 0};
    if (s.cps > kMaxChunks) s.cps = kMaxChunks;
    s.nseg = cdiv(nc, s.cps);
    const double n = (double)BH * s.nseg;
    double us = bwd ? t.us(3 * n, s.cps, 1.3 * chunk) : t.us(n, s.cps, chunk);
    if (s.nseg > 1)
      us += bwd ? t.us(2 * n, s.cps, 0.45 * chunk) + 9 + 0.5 * s.nseg : t.us(n, s.cps, 0.45 * chunk) + 6 + 0.45 * s.nseg;
    if (best.nseg == 0 || us < least) best = s, least = us;
  }
  return best;
}

// Work items (unit, member): the `grp` heads that share q and k rows run on
// one XCD (workgroups go to the 8 XCDs round-robin by flat id), whose L2 then
// serves the shared rows.  unit = (head group, segment).
__device__ __forceinline__ bool item_of(int flat, int BH, int grp, int nseg, int& bh, int& seg) {
  const int x = flat & 7, y = flat >> 3;
  const long long unit = (long long)(y / grp) * 8 + x;
  const long long units = (long long)(BH / grp) * nseg;
  if (unit >= units) return false;
  seg = (int)(unit % nseg);
  bh = (int)(unit / nseg) * grp + y % grp;
  return true;
}
inline long long items(int BH, int grp, int nseg) {
  const long long units = (long long)(BH / grp) * nseg;
  return (units + 7) / 8 * 8 * grp;
}

struct StateArgs {
  Src k, v;
  const float* g;     // [BH][L] or null
  float* states;      // [BH][slots][DK][DV]: slot s receives segment s's sum
  double* decays;     // [BH][nseg]: log2 decay over a segment
  int slots, L, BH, grp;
  int first, count;   // the segments to sum: first .. first + count - 1
  Split s;
};

// S = total S + K^T diag(up) V on this wave's columns, diag(up) V in NU pieces.
template <int NU, typename IT, int DK>
__device__ __forceinline__ void update_state(f32x4 (&st)[DK / 16], Tile<IT, DK> K,
                                             const typename Tile<IT, 64>::Frag (&vf)[C / 32], const float* up, int l) {
  // Column fragments are read AHEAD tiles before their products, so that LDS
  // answers meanwhile.
  // The waves that are here go first: theirs are the long runs of matrix
  // instructions that the others' vector work hides behind (3% of a walk).
  __builtin_amdgcn_s_setprio(1);
  constexpr int KT = DK / 16, N = KT * (C / 32), AHEAD = 4;
  const int g = l >> 4;
  typename Tile<IT, DK>::Frag a[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) a[i] = K.state_col(i % KT, i / KT, l);
  const float total = up[C - 1];
#pragma unroll
  for (int tb = 0; tb < C / 32; ++tb) {
    const f32x4 u0 = *reinterpret_cast<const f32x4*>(&up[32 * tb + 4 * g]);
    f32x4 u1 = *reinterpret_cast<const f32x4*>(&up[32 * tb + 16 + 4 * g]);
    if (tb == C / 32 - 1 && g == 3) u1[3] = 1.f;  // (row C - 1: see Decays)
    float x[8];
    to_floats(vf[tb], x);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= u0[e], x[4 + e] *= u1[e];
    const Made<IT, NU> y(x);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int i = tb * KT + kt;
      if (tb == 0) st[kt] *= total;
      st[kt] = mma(a[i % AHEAD], y, st[kt]);
      if (i + AHEAD < N) a[i % AHEAD] = K.state_col((i + AHEAD) % KT, (i + AHEAD) / KT, l);
    }
  }
  __builtin_amdgcn_s_setprio(0);
}

// fp32 state (row-major [DK][DV], or [DV][DK] when TRANS) <-> this wave's
// accumulators: rows state_row() + e, column j.
template <int DK, int DV, bool TRANS>
__device__ __forceinline__ void load_state(f32x4 (&st)[DK / 16], const float* S) {
  const int l = threadIdx.x & 63, g = l >> 4, j = (threadIdx.x >> 6) * 16 + (l & 15);
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt) st[kt] = zero4();
  if (!S) return;
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt) {
    const int k0 = state_row(kt, g);
    if (TRANS) {
      st[kt] = *reinterpret_cast<const f32x4*>(S + (size_t)j * DK + k0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) st[kt][e] = S[(size_t)(k0 + e) * DV + j];
    }
  }
}
template <int DK, int DV, bool TRANS>
__device__ __forceinline__ void store_state(const f32x4 (&st)[DK / 16], float* S, float scale) {
  const int l = threadIdx.x & 63, g = l >> 4, j = (threadIdx.x >> 6) * 16 + (l & 15);
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt) {
    const int k0 = state_row(kt, g);
    const f32x4 x = st[kt] * scale;
    if (TRANS) {
      *reinterpret_cast<f32x4*>(S + (size_t)j * DK + k0) = x;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[(size_t)(k0 + e) * DV + j] = x[e];
    }
  }
}

template <typename IT, int DV>
__device__ __forceinline__ void value_frags(typename Tile<IT, DV>::Frag (&vf)[C / 32], Tile<IT, DV> V, int w, int l) {
#pragma unroll
  for (int tb = 0; tb < C / 32; ++tb) vf[tb] = V.col(w * 16, tb, l);
}

// Waves per SIMD to compile for: two workgroups per CU with bf16 tiles, one
// with fp32 tiles.
template <typename IT>
__host__ __device__ constexpr int simd_waves(int DV) { return waves(DV) / 4 * (sizeof(IT) == 2 ? 2 : 1); }

// Two sets of tiles: a chunk's rows arrive while the one before is used.
template <typename IT, int DK, int DV>
constexpr int state_lds() { return 2 * (Tile<IT, DK>::bytes + Tile<IT, DV>::bytes) + (int)sizeof(Decays); }

template <typename IT, int DK, int DV, bool REV>
__device__ __forceinline__ void state_walk(const StateArgs& a, int flat, Lds m) {
  unsigned char* const smem = m.p;
  constexpr int NW = waves(DV);
  constexpr int TB = Tile<IT, DK>::bytes + Tile<IT, DV>::bytes;
  Decays* const table = reinterpret_cast<Decays*>(smem + 2 * TB);

  int bh, seg;
  if (!item_of(flat, a.BH, a.grp, a.count, bh, seg)) return;
  seg += a.first;
  const int L = a.L, c0 = seg * a.s.cps, c1 = min(c0 + a.s.cps, a.s.nc);
  const IT* k = a.k.head<IT>(bh, L, DK);
  const IT* v = a.v.head<IT>(bh, L, DV);
  const float* g = a.g ? a.g + (size_t)bh * L : nullptr;
  const int n = c1 - c0, lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto chunk = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };
  const bool tables_wave = w == NW - 1;

  f32x4 st[DK / 16];
  load_state<DK, DV, false>(st, nullptr);
  const Stage<IT, DK, NW, REV> sk;
  const Stage<IT, DV, NW, REV> sv;
  auto load = [&](int i) {
    const uint32_t at = m.at + (i & 1) * TB;
    sk.load(k, chunk(i), L, at);
    sv.load(v, chunk(i), L, at + Tile<IT, DK>::bytes);
  };
  double sum = 0.0;
  load(0);
  if (tables_wave) sum += fill_decays(table, 0, load_decay<REV>(g, chunk(0), L));
  wait_loads();
  __syncthreads();
  for (int i = 0; i < n; ++i) {
    const bool more = i + 1 < n;
    float gn = 0.f;
    if (more) {
      if (tables_wave) {
        gn = load_decay<REV>(g, chunk(i + 1), L);
        keep(gn);
      }
      load(i + 1);
    }
    unsigned char* const at = smem + (i & 1) * TB;
    typename Tile<IT, DV>::Frag vf[C / 32];
    value_frags<IT, DV>(vf, Tile<IT, DV>{at + Tile<IT, DK>::bytes}, w, lane);
    update_state<3, IT, DK>(st, Tile<IT, DK>{at}, vf, table->up[i & 1], lane);
    if (more && tables_wave) sum += fill_decays(table, i + 1, gn);
    wait_loads();
    __syncthreads();
  }
  store_state<DK, DV, false>(st, a.states + ((size_t)bh * a.slots + seg) * (DK * DV), 1.f);
  if (threadIdx.x == 64 * NW - 1) a.decays[(size_t)bh * a.s.nseg + seg] = sum;
}

template <typename IT, int DK, int DV>
__global__ __launch_bounds__(64 * waves(DV), simd_waves<IT>(DV)) void state_kernel(StateArgs a) {
  state_walk<IT, DK, DV, false>(a, blockIdx.x, dynamic_lds());
}

// ---- the combine kernel --------------------------------------------------------------

// Per head: segment sums -> the state entering each segment, in place.
// Forward: slot s receives the state that enters segment s; reversed: the
// reversed walk's state when it reaches the segment's last token (the gradient
// of the state after the token behind it).  (The sum of the walk's last segment
// is not needed.)
struct CombineArgs {
  float* states;
  const double* decays;
  const float* S0;  // [BH][N] or null: the first state of the walk
  const float* g;   // [BH][L] or null: log decays (forward)
  int slots, nseg, N, L;
};

template <bool REV>
__device__ __forceinline__ void combine(const CombineArgs& a) {
  const int bh = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= a.N) return;
  float* S = a.states + (size_t)bh * a.slots * a.N + e;
  const double* d = a.decays + (size_t)bh * a.nseg;
  const bool none = !a.S0 || (!REV && starts_with_wipe(a.g ? a.g + (size_t)bh * a.L : nullptr));
  f32x4 run = none ? zero4() : *reinterpret_cast<const f32x4*>(a.S0 + (size_t)bh * a.N + e);
  const int steps = a.nseg - 1;
  for (int i0 = 0; i0 < steps; i0 += 8) {
    f32x4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = min(i0 + j, steps - 1), s = REV ? a.nseg - 1 - i : i;
      x[j] = *reinterpret_cast<const f32x4*>(S + (size_t)s * a.N);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i0 + j < steps) {
        const int s = REV ? a.nseg - 1 - (i0 + j) : i0 + j;
        *reinterpret_cast<f32x4*>(S + (size_t)s * a.N) = run;
        run = run * exp2_hw((float)d[s]) + x[j];
      }
    }
  }
  const int s = REV ? 0 : a.nseg - 1;
  *reinterpret_cast<f32x4*>(S + (size_t)s * a.N) = run;
}

static __global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) { combine<false>(a); }

// ---- the output kernel ---------------------------------------------------------------

// Which extra sums a pass leaves for the decay's gradient.
enum Extra {
  kNone = 0,
  kDots = 1,   // per row: (row of w) . (the part of the output that comes from the entering state)
  kPairs = 2   // kDots, and per row t the sum of the chunk's pair terms that cross t (below)
};

struct OutArgs {
  Src q, k, v, w;      // w: [..][L][DV], with Extra only
  const float* g;      // [BH][L] or null
  const float* states; // [BH][slots][..] entering states (nseg > 1), else null
  const float* S0;     // [BH][..] entering state of the whole (nseg == 1) or null
  void* out;           // [BH][L][DV]
  float* last;         // [BH][..] state after the walk, or null
  long long last_stride;
  float* dots;         // [BH][nc C] (Extra)
  float* pairs;        // [BH][nc C] (kPairs)
  int slots, L, BH, grp;
  Split s;
};

// P's lower triangle as operand fragments (columns: output rows; contraction:
// key rows): fragment (rt, kb), kb <= rt / 2, holds key tiles 2 kb and 2 kb + 1;
// of fragments (0, 0) and (2, 1) the second is above the diagonal, and absent.
// at(): units of a half fragment before it.
__host__ __device__ constexpr int pat(int rt, int kb) {
  return rt == 0 ? 0 : rt == 1 ? 1 : rt == 2 ? (kb ? 5 : 3) : (kb ? 8 : 6);
}
__host__ __device__ constexpr bool pwhole(int rt, int kb) { return 2 * kb + 1 <= rt; }

template <typename IT, int NS>
struct PBuf;
template <int NS>
struct PBuf<bf16, NS> {
  static constexpr int plane = 10 * 512;
  static constexpr int bytes = NS * plane;
  unsigned char* p;
  __device__ __forceinline__ void put(int rt, int it, f32x4 x, int l) const {
    const int kb = it >> 1;
    unsigned char* const at = p + pat(rt, kb) * 512 + (pwhole(rt, kb) ? l * 16 + (it & 1) * 8 : l * 8);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint2 u = make_uint2(pack_once(x[0], x[1]), pack_once(x[2], x[3]));
      *reinterpret_cast<uint2*>(at + s * plane) = u;
      if (s + 1 < NS) {
        x[0] -= __uint_as_float(u.x << 16);
        x[1] -= __uint_as_float(u.x & 0xffff0000u);
        x[2] -= __uint_as_float(u.y << 16);
        x[3] -= __uint_as_float(u.y & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ Made<bf16, NS> get(int rt, int kb, int l) const {
    const unsigned char* const at = p + pat(rt, kb) * 512;
    Made<bf16, NS> m;
#pragma unroll
    for (int s = 0; s < NS; ++s)
      m.p[s] = pwhole(rt, kb) ? as_bf16x8(*reinterpret_cast<const uint4*>(at + s * plane + l * 16))
                              : as_bf16x8(*reinterpret_cast<const uint2*>(at + s * plane + l * 8), make_uint2(0, 0));
    return m;
  }
};
template <int NS>
struct PBuf<float, NS> {
  static constexpr int bytes = 10 * 1024;
  unsigned char* p;
  __device__ __forceinline__ f32x4* at(int rt, int kb, int half, int l) const {
    return reinterpret_cast<f32x4*>(p + (pat(rt, kb) + half) * 1024) + l;
  }
  __device__ __forceinline__ void put(int rt, int it, f32x4 x, int l) const { *at(rt, it >> 1, it & 1, l) = x; }
  __device__ __forceinline__ Made<float, NS> get(int rt, int kb, int l) const {
    const f32x4 a = *at(rt, kb, 0, l), b = pwhole(rt, kb) ? *at(rt, kb, 1, l) : zero4();
    Made<float, NS> m;
    m.p = F32x8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    return m;
  }
};

// Sums for the decay's gradient, gathered per chunk without atomics: every
// writer has a slot of its own.
template <int NW>
struct Sums {
  float dots[NW][C];  // by wave
  float out[10][16];  // pair terms of an output tile's rows, by tile of P (none on the diagonal)
  float key[10][16];  // ... of a key tile's rows; on the diagonal the tile's terms that cross each row
};
__device__ __forceinline__ int tri(int rt, int it) { return rt * (rt + 1) / 2 + it; }

__device__ __forceinline__ float sum_groups(float x) {  // over the 4 lane groups (same i)
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}
__device__ __forceinline__ float sum_lanes16(float x) {  // over the 16 lanes of a group
  x += dpp<0x128>(x);
  x += dpp<0x124>(x);
  x += dpp<0x122>(x);
  x += dpp<0x121>(x);
  return x;
}

template <typename OT>
__device__ __forceinline__ void store4(OT* p, f32x4 x);
template <>
__device__ __forceinline__ void store4<float>(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
template <>
__device__ __forceinline__ void store4<bf16>(bf16* p, f32x4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// Bytes of LDS: four tile buffers, P, the decay tables, and the sums.
template <typename IT, typename OT, int DK, int DV, int EXTRA>
struct OutLds {
  // Pieces of an fp32 operand (see "Precision" above): of P, of the state.
  static constexpr int NSP = EXTRA == kNone || (DK == 64 && DV == 64) ? 3 : 2;
  static constexpr int NSS = sizeof(OT) == 2 && EXTRA == kNone ? 2 : 3;
  static constexpr int tile = Tile<IT, (DK > DV ? DK : DV)>::bytes;
  static constexpr int P = 4 * tile;
  static constexpr int D = P + PBuf<IT, NSP>::bytes;
  static constexpr int S = D + (int)sizeof(Decays);
  static constexpr int bytes = S + (EXTRA != kNone ? (int)sizeof(Sums<waves(DV)>) : 0);
};

// Four adjacent elements of a row of w straight from HBM.  Rows past the end read
// as zeros: the whole offset goes through the vector operand, which the
// descriptor's range check sees (a scalar offset on top of it need not be seen).
template <typename IT>
struct Four;
template <>
struct Four<float> {
  f32x4 x;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t at) { x = __builtin_bit_cast(f32x4, bload16(r, at, 0)); }
  __device__ __forceinline__ f32x4 get() const { return x; }
};
template <>
struct Four<bf16> {
  uint2 x;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t at) { x = bload8(r, at, 0); }
  __device__ __forceinline__ f32x4 get() const {
    return f32x4{__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                 __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u)};
  }
};
template <typename IT, int D>
__device__ __forceinline__ typename Tile<IT, D>::Frag row_frag(rsrc_t r, int row, int kb, int lane) {
  const uint32_t at = (uint32_t)(row * D + 32 * kb + 8 * (lane >> 4)) * sizeof(IT);
  if constexpr (sizeof(IT) == 2) {
    return as_bf16x8(bload16(r, at, 0));
  } else {
    Four<float> a, b;
    a.load(r, at);
    b.load(r, at + 16);
    return F32x8{{a.x[0], a.x[1], a.x[2], a.x[3], b.x[0], b.x[1], b.x[2], b.x[3]}};
  }
}

// A chunk takes two phases with a barrier behind each:
//   1  P (from Q, K) and Q S;                       V arrives
//   2  P V, the output, the state's update (K, V);  the next Q and K arrive
// Four tile buffers suffice: the next Q goes where V was a chunk ago, the next
// K where Q is no longer read, the next V where K is no longer read.
template <typename IT, typename OT, int DK, int DV, bool REV, int EXTRA, int NU>
__device__ __forceinline__ void walk_segment(const OutArgs& a, int bh, int seg, Lds m) {
  unsigned char* const smem = m.p;
  using LD = OutLds<IT, OT, DK, DV, EXTRA>;
  constexpr int NW = waves(DV), NRT = C / 16, NSP = LD::NSP, NSS = LD::NSS;
  constexpr bool TRANS = EXTRA != kNone;  // dq and dk walk the transposed state
  typedef Tile<IT, DK> TK;
  typedef Tile<IT, DV> TV;
  const PBuf<IT, NSP> P{smem + LD::P};
  Sums<NW>* const sums = reinterpret_cast<Sums<NW>*>(smem + LD::S);

  const int L = a.L, c0 = seg * a.s.cps, c1 = min(c0 + a.s.cps, a.s.nc), n = c1 - c0;
  const IT* q = a.q.head<IT>(bh, L, DK);
  const IT* k = a.k.head<IT>(bh, L, DK);
  const IT* v = a.v.head<IT>(bh, L, DV);
  const IT* wp = EXTRA != kNone ? a.w.head<IT>(bh, L, DV) : nullptr;
  const float* g = a.g ? a.g + (size_t)bh * L : nullptr;
  OT* out = static_cast<OT*>(a.out) + (size_t)bh * L * DV;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto chunk = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };

  // This wave's tiles of P (output tile rt, key tile it <= rt), 10 over the
  // waves: NA adjacent ones of one rt, and on two waves one more; the decay
  // table's wave is not one of those.
  //   8 waves: (3,0) (3,1) (3,2) (3,3) (2,0) (0,0) (2,1)+(2,2) (1,0)+(1,1)
  //   4 waves: (3,0)(3,1)  (3,2)(3,3)  (2,0)(2,1)+(2,2)  (1,0)(1,1)+(0,0)
  constexpr int NA = NW == 8 ? 1 : 2, kTableWave = 1;
  const int prt = NW == 8 ? (w < 4 ? 3 : w == 5 ? 0 : w == 7 ? 1 : 2) : (w < 2 ? 3 : w == 2 ? 2 : 1);
  const int pit = NW == 8 ? (w < 4 ? w : w == 6 ? 1 : 0) : (w == 1 ? 2 : 0);
  const bool more_p = w >= NW - 2, other = NW == 4 && w == 3;  // other: of another rt
  const int prt2 = other ? 0 : prt, pit2 = other ? 0 : pit + NA;

  const Stage<IT, DK, NW, REV> sk;
  const Stage<IT, DV, NW, REV> sv;
  int bq = 0, bk = LD::tile, bv = 2 * LD::tile, bf = 3 * LD::tile;
  sk.load(q, chunk(0), L, m.at + bq);
  sk.load(k, chunk(0), L, m.at + bk);
  if (w == kTableWave) fill_decays(reinterpret_cast<Decays*>(smem + LD::D), 0, load_decay<REV>(g, chunk(0), L));
  f32x4 st[DK / 16];
  const float* S = a.s.nseg > 1 ? a.states + ((size_t)bh * a.slots + seg) * (DK * DV)
                                : (a.S0 ? a.S0 + (size_t)bh * (DK * DV) : nullptr);
  if (!REV && c0 == 0 && starts_with_wipe(g)) S = nullptr;
  load_state<DK, DV, TRANS>(st, S);
  wait_loads();
  __syncthreads();

  // A chunk's pair sums, once every wave has left its own: for row t the terms of
  // pairs (i, r), i < t <= r, and of no other.  By tiles, t in tile lg: both of
  // the pair in it; r in it and i before; i in it and r behind; the two of them
  // around it.
  auto store_pairs = [&](int c) {
    const int lane = threadIdx.x & 63, lg = lane >> 4, li = lane & 15;
    float before = 0.f, behind = 0.f, around = 0.f;
    for (int x = 0; x < NRT; ++x) {
      if (x < lg) before += sums->out[tri(lg, x)][li];
      if (x > lg) behind += sums->key[tri(x, lg)][li];
    }
    if (lg == 1 || lg == 2) around = sums->out[tri(3, 0)][li] + sums->out[lg == 1 ? tri(2, 0) : tri(3, 1)][li];
    // (Rows r from t on; rows i up to the one before t.)
    before += dpp<0x101>(before);
    before += dpp<0x102>(before);
    before += dpp<0x104>(before);
    before += dpp<0x108>(before);
    behind = dpp<0x111>(behind);
    behind += dpp<0x111>(behind);
    behind += dpp<0x112>(behind);
    behind += dpp<0x114>(behind);
    behind += dpp<0x118>(behind);
    a.pairs[(size_t)bh * a.s.nc * C + token_of<REV>(c, lane)] =
        (sums->key[tri(lg, lg)][li] + before) + (behind + sum_lanes16(around));
  };

  for (int ci = 0; ci < n; ++ci) {
    const int c = chunk(ci);
    const bool more = ci + 1 < n;
    // (dq and dk: addresses are formed anew in each chunk.  Kept over the loop they
    // do not fit beside the state, and a reload from scratch memory waits for
    // every row on its way.  Of the bf16 walks the 64 x 128 ones keep one value there,
    // 8 bytes per lane; the others none.)
    int lane = threadIdx.x & 63;
    if (EXTRA != kNone) asm volatile("" : "+v"(lane));
    const int lg = lane >> 4, li = lane & 15;
    // (Where the table lies is formed anew in each chunk as well: known for the whole
    // loop, every address into it would stay in a register.)
    int table = LD::D;
    asm volatile("" : "+s"(table));
    Decays* const dec = reinterpret_cast<Decays*>(smem + table);
    const TK Q{smem + bq}, K{smem + bk};
    const TV V{smem + bv};
    rsrc_t wr;
    Four<IT> wd[NRT];
    auto w_row = [&](int r) { return REV ? C - 1 - r : r; };
    if constexpr (EXTRA != kNone) {
      wr = make_rsrc(wp + (size_t)c * C * DV, (uint32_t)(min(C, L - c * C) * DV * (int)sizeof(IT)));
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt)
        wd[rt].load(wr, (uint32_t)(w_row(16 * rt + li) * DV + w * 16 + 4 * lg) * sizeof(IT));
    }
    sv.load(v, c, L, m.at + bv);
    float gn = 0.f;
    if (w == kTableWave && more) gn = load_decay<REV>(g, chunk(ci + 1), L);
    if (EXTRA == kPairs && w == 0 && ci > 0) store_pairs(chunk(ci - 1));

    // P^T tiles: rows are key rows 16 it + 4 lg + e, the column is output row
    // 16 rt + li.
    // (First, so that their way through LDS is hidden behind Q S; with the pair
    // terms' fragments they come second, which leaves registers for both.)
    f32x4 p[NA + 1];
    auto make_p = [&] {
#pragma unroll
      for (int x = 0; x <= NA; ++x) p[x] = zero4();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) {
        const auto b = Q.row(16 * prt, kb, lane);
#pragma unroll
        for (int x = 0; x < NA; ++x) p[x] = mma(K.row(16 * (pit + x), kb, lane), b, p[x]);
      }
      if (more_p) {
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) p[NA] = mma(K.row(16 * pit2, kb, lane), Q.row(16 * prt2, kb, lane), p[NA]);
      }
      auto decay_tile = [&](f32x4& x, int rt, int it) {
        const double Gr = dec->G[16 * rt + li];
        double Gi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) Gi[e] = dec->G[16 * it + 4 * lg + e];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (Above the diagonal the factor may be infinite: it is not used.)
          const float f = exp2_hw((float)(Gr - Gi[e])) * x[e];
          x[e] = it < rt || 4 * lg + e <= li ? f : 0.f;
        }
        P.put(rt, it, x, lane);
      };
#pragma unroll
      for (int x = 0; x < NA; ++x) decay_tile(p[x], prt, pit + x);
      if (more_p) decay_tile(p[NA], prt2, pit2);
    };
    if (EXTRA != kPairs) make_p();

    // Output tiles (rows: this wave's columns, column: row 16 rt + li), first
    // what comes from the entering state.
    f32x4 acc[NRT];
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) acc[rt] = zero4();
    typename TK::Frag b[NRT];
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) b[rt] = Q.row(16 * rt, 0, lane);
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) {
      const f32x4 x = st[2 * kb], y = st[2 * kb + 1];
      const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      const Made<IT, NSS> s(z);
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        acc[rt] = mma(s, b[rt], acc[rt]);
        if (kb + 1 < DK / 32) b[rt] = Q.row(16 * rt, kb + 1, lane);
      }
    }
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      acc[rt] *= exp2_hw((float)dec->G[16 * rt + li]);
      if constexpr (EXTRA != kNone) {
        const f32x4 y = wd[rt].get();
        float dot = (acc[rt][0] * y[0] + acc[rt][1] * y[1]) + (acc[rt][2] * y[2] + acc[rt][3] * y[3]);
        dot = sum_groups(dot);
        if (lg == 0) sums->dots[w][16 * rt + li] = dot;
      }
    }
    constexpr int WF = EXTRA == kPairs ? DV / 32 : 0;
    typename TV::Frag wf[WF + 1], wf2[NW == 4 ? WF + 1 : 1];
#pragma unroll
    for (int kb = 0; kb < WF; ++kb) {
      wf[kb] = row_frag<IT, DV>(wr, w_row(16 * prt + li), kb, lane);
    }
    if (EXTRA == kPairs) make_p();
    // (Behind P, whose fragments leave no registers for it.)
#pragma unroll
    for (int kb = 0; kb < WF; ++kb) {
      if constexpr (NW == 4) wf2[kb] = row_frag<IT, DV>(wr, w_row(16 * prt2 + li), kb, lane);
    }
    keep(gn);
#pragma unroll
    for (int kb = 0; kb < WF; ++kb) {
      keep(wf[kb]);
      if constexpr (NW == 4) keep(wf2[kb]);
    }
    wait_loads();
    __syncthreads();

    // ... then what comes from the chunk's own rows.
    if (more) {
      sk.load(q, chunk(ci + 1), L, m.at + bf);
      sk.load(k, chunk(ci + 1), L, m.at + bq);
    }
    if (EXTRA != kNone && w == 0) {
      float y = 0.f;
#pragma unroll
      for (int x = 0; x < NW; ++x) y += sums->dots[x][lane];
      a.dots[(size_t)bh * a.s.nc * C + token_of<REV>(c, lane)] = y;
    }
    if constexpr (EXTRA == kPairs) {
      // Pair terms: P_ri (w_r . v_i), i < r.
      auto pair_sums = [&](const f32x4& x, const f32x4& y, int rt, int it) {
        const int i = li, g4 = 4 * lg, t = tri(rt, it);
        f32x4 m, row;
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = it < rt || g4 + e < i ? x[e] * y[e] : 0.f;
        const float sum = (m[0] + m[1]) + (m[2] + m[3]);
        if (it < rt) {
          const float col = sum_groups(sum);
          if (g4 == 0) sums->out[t][i] = col;
        } else {
          // Of output row i: the sum over the key rows in front of g4 + e.
          const float up1 = __shfl_up(sum, 16, 64), u = g4 > 0 ? up1 : 0.f;
          const float up2 = __shfl_up(u, 16, 64), up3 = __shfl_up(u, 32, 64);
          float run = u + (g4 > 4 ? up2 : 0.f) + (g4 > 8 ? up3 : 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float next = run + m[e];
            m[e] = i >= g4 + e ? run : 0.f;
            run = next;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) row[e] = sum_lanes16(m[e]);
        if (i == 0) *reinterpret_cast<f32x4*>(&sums->key[t][g4]) = row;
      };
#pragma unroll
      for (int x = 0; x <= NA; ++x) {
        if (x == NA && !more_p) break;
        const bool second = NW == 4 && x == NA;
        const int rt = x < NA ? prt : prt2, it = x < NA ? pit + x : pit2;
        f32x4 y = zero4();
#pragma unroll
        for (int kb = 0; kb < DV / 32; ++kb) {
          if constexpr (NW == 4) y = mma(V.row(16 * it, kb, lane), second ? wf2[kb] : wf[kb], y);
          else y = mma(V.row(16 * it, kb, lane), wf[kb], y);
        }
        pair_sums(p[x], y, rt, it);
      }
    }
    typename TV::Frag vf[C / 32];
    value_frags<IT, DV>(vf, V, w, lane);
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb) acc[rt] = mma(vf[kb], P.get(rt, kb, lane), acc[rt]);
    update_state<NU, IT, DK>(st, K, vf, dec->up[ci & 1], lane);
    if (w == kTableWave && more) fill_decays(dec, ci + 1, gn);
    wait_loads();
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const int t = token_of<REV>(c, 16 * rt + li);
      if (t < L) store4(out + (size_t)t * DV + w * 16 + 4 * lg, acc[rt]);
    }
    __syncthreads();
    const int free = bv;
    bv = bk;
    bk = bq;
    bq = bf;
    bf = free;
  }
  if (EXTRA == kPairs && w == 0) store_pairs(chunk(n - 1));

  if (a.last && seg == (REV ? 0 : a.s.nseg - 1)) {
    // Reversed, the walk ends with the gradient of the state after token 0;
    // the state before it is one decay further.
    const float f = REV && g ? exp2_hw((float)log2_decay(g[0])) : 1.f;
    store_state<DK, DV, TRANS>(st, a.last + (size_t)bh * a.last_stride, f);
  }
}

template <typename IT, typename OT, int DK, int DV, bool REV, int EXTRA>
__device__ __forceinline__ void out_walk(const OutArgs& a, int flat, Lds m) {
  int bh, seg;
  if (!item_of(flat, a.BH, a.grp, a.s.nseg, bh, seg)) return;
  // A segment whose last state goes nowhere and whose outputs are stored in
  // bf16 keeps 16 bits of what it adds to its state.
  constexpr bool rough = sizeof(IT) == 2 && sizeof(OT) == 2 && EXTRA == kNone;
  if (rough && !(a.last && seg == (REV ? 0 : a.s.nseg - 1)))
    walk_segment<IT, OT, DK, DV, REV, EXTRA, rough ? 2 : 3>(a, bh, seg, m);
  else
    walk_segment<IT, OT, DK, DV, REV, EXTRA, 3>(a, bh, seg, m);
}

template <typename IT, typename OT, int DK, int DV>
__global__ __launch_bounds__(64 * waves(DV), simd_waves<IT>(DV)) void out_kernel(OutArgs a) {
  out_walk<IT, OT, DK, DV, false, kNone>(a, blockIdx.x, dynamic_lds());
}

// ---- launches --------------------------------------------------------------------------

template <typename K>
hipError_t allow_lds(K* kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// One launch of `kernel`, bracketed for the profiling hook.  (The sizes that the
// entry points accept stay below a launch's limit wherever their tensors fit the card.)
template <typename K, typename... A>
hipError_t launch(K* kernel, int slot, long long blocks, int threads, int lds, hipStream_t stream, const A&... args) {
  if (blocks > max_blocks(threads)) return hipErrorInvalidConfiguration;
  hipError_t e = lds > 65536 ? allow_lds(kernel, lds) : hipSuccess;
  if (e != hipSuccess) return e;
  prof_mark(slot, false, stream);
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), lds, stream, args...);
  e = hipGetLastError();
  prof_mark(slot, true, stream);
  return e;
}

// The state of a call without tokens: dst = src, or zeros.
hipError_t launch_copy_state(float* dst, const float* src, size_t n, hipStream_t stream);

}  // namespace lin
}  // namespace dn
