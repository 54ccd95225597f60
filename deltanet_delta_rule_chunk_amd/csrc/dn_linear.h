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
// head's chunks are cut into segments.  A state kernel sums each segment from
// a zero state (it reads k and v only), a combine kernel turns the sums into
// the state entering every segment, and the output kernel walks each segment
// from there.  With one segment the output kernel runs alone.
//
// Output kernel: 4 waves; wave w owns DV / 4 columns of the state, which stay
// in fp32 MFMA accumulators for the whole segment and never pass through LDS:
// the accumulator layout of two stacked 16 x 16 tiles is the operand layout
// of the next product (the "d4" slot order of dn_mfma.h), so Q S takes the
// state straight from the accumulators.  Outputs are formed as transposed
// tiles (S^T Q^T + V^T P^T): a lane then holds 4 consecutive columns of one
// row.  P is formed once per workgroup (10 tiles over the 4 waves) and passed
// through LDS as operand fragments.
//
// Precision.  bf16 q, k, v (and dO) enter products as they are.  An fp32
// operand enters as a sum of bf16 pieces: 2 pieces (16 bits) where the result
// is stored in bf16, whose own rounding is 256 times coarser, and 3 pieces
// (24 bits, all of fp32) where it reaches an fp32 result: the state, and what
// the gradients of the decay are summed from.  fp32 inputs run the same
// kernels on the fp32 matrix instruction, with nothing split.  Log decays are
// summed in fp64: a difference of two sums keeps the accuracy of the short
// sum between them however long the chunk's own is.
#pragma once

#include <hip/hip_runtime.h>

#include "dn_buffer.h"
#include "dn_common.h"
#include "dn_ktile.h"
#include "dn_launch.h"
#include "dn_mfma.h"

namespace dn {
namespace lin {

constexpr int C = 64;       // rows of a chunk
constexpr int NTHR = 256;   // 4 waves
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

// ---- operands ------------------------------------------------------------------
//
// A fragment holds, per lane (g = lane / 16, i = lane % 16), 8 values of row
// (or column) i of a 16 x 32 operand: contraction slots 4 g + e and
// 16 + 4 g + e, e = 0 .. 3.

struct F32x8 {
  float v[8];
};

// LDS tile of C rows x D and its fragments.
template <typename IT, int D>
struct Tile;

template <int D>
struct Tile<bf16, D> {
  typedef bf16x8 Frag;
  static constexpr int bytes = C * D * 2;
  static constexpr int PPR = D / 8;  // 16-byte pieces per row
  unsigned char* p;
  __device__ __forceinline__ uint16_t* e(int off) const { return reinterpret_cast<uint16_t*>(p) + off; }
  __device__ __forceinline__ void put(int row, int piece, uint4 x) const {
    *reinterpret_cast<uint4*>(e(koff<D>(row, piece))) = x;
  }
  // Row r0 + i, contraction over columns 32 kb ..
  __device__ __forceinline__ Frag row(int r0, int kb) const {
    const int l = threadIdx.x & 63, g = l >> 4, r = r0 + (l & 15);
    const int ch = 4 * kb + (g >> 1), h = 4 * (g & 1);
    const uint2 a = *reinterpret_cast<const uint2*>(e(koff<D>(r, ch) + h));
    const uint2 b = *reinterpret_cast<const uint2*>(e(koff<D>(r, ch + 2) + h));
    return as_bf16x8(a, b);
  }
  __device__ __forceinline__ uint2 tr(int off) const {
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(e(off))));
  }
  // Column c0 + i, contraction over rows 32 tb ..  (transposing reads: lane
  // 4 m + a of a 16-lane group addresses row m, columns 4 a .. + 3).
  __device__ __forceinline__ Frag col(int c0, int tb) const {
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15, m = i >> 2, a = i & 3;
    const int r = 32 * tb + 4 * g + m, ch = (c0 >> 3) + (a >> 1), h = 4 * (a & 1);
    return as_bf16x8(tr(koff<D>(r, ch) + h), tr(koff<D>(r + 16, ch) + h));
  }
  // Columns c .. c + 3 (c % 4 == 0) of a row, as fp32.
  __device__ __forceinline__ f32x4 four(int row, int c) const {
    const uint2 a = *reinterpret_cast<const uint2*>(e(koff<D>(row, c >> 3) + (c & 4)));
    return f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u),
                 __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u)};
  }
};

template <int D>
struct Tile<float, D> {
  typedef F32x8 Frag;
  static constexpr int P = D + 4;  // row pitch: column reads of 4 row groups miss each other's banks
  static constexpr int bytes = C * P * 4;
  static constexpr int PPR = D / 4;
  unsigned char* p;
  __device__ __forceinline__ float* e(int off) const { return reinterpret_cast<float*>(p) + off; }
  __device__ __forceinline__ void put(int row, int piece, uint4 x) const {
    *reinterpret_cast<uint4*>(e(row * P + 4 * piece)) = x;
  }
  __device__ __forceinline__ Frag row(int r0, int kb) const {
    const int l = threadIdx.x & 63, g = l >> 4, off = (r0 + (l & 15)) * P + 32 * kb + 4 * g;
    const f32x4 a = *reinterpret_cast<const f32x4*>(e(off));
    const f32x4 b = *reinterpret_cast<const f32x4*>(e(off + 16));
    return Frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  __device__ __forceinline__ Frag col(int c0, int tb) const {
    const int l = threadIdx.x & 63, g = l >> 4, off = (32 * tb + 4 * g) * P + c0 + (l & 15);
    Frag f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f.v[x] = *e(off + x * P);
      f.v[4 + x] = *e(off + (16 + x) * P);
    }
    return f;
  }
  __device__ __forceinline__ f32x4 four(int row, int c) const {
    return *reinterpret_cast<const f32x4*>(e(row * P + c));
  }
};

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
        u[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
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

struct alignas(16) Decays {
  double G[C];    // log2 decay from the chunk's start through a row
  float up[C];    // 2^(G_last - G): from a row to the chunk's end
  float total;    // 2^G_last
};

// Row u of chunk c: token, and the log decay in front of it.
template <bool REV>
__device__ __forceinline__ int token_of(int c, int u) { return c * C + (REV ? C - 1 - u : u); }

template <bool REV>
__device__ __forceinline__ float load_decay(const float* g, int c, int L) {
  const int t = token_of<REV>(c, threadIdx.x & 63) + (REV ? 1 : 0);
  return g && t < L ? g[t] : 0.f;
}

// Inclusive sums over a wave's 64 lanes.
__device__ __forceinline__ double wave_scan(double x) {
  const int l = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double y = __shfl_up(x, off, 64);
    if (l >= off) x += y;
  }
  return x;
}

// One wave fills a chunk's table from its rows' log decays; returns the sum.
__device__ __forceinline__ double fill_decays(Decays* d, float g) {
  const int l = threadIdx.x & 63;
  const double G = wave_scan(log2_decay(g)), last = __shfl(G, 63, 64);
  d->G[l] = G;
  d->up[l] = exp2_hw((float)(last - G));
  if (l == 63) d->total = exp2_hw((float)G);
  return last;
}

// ---- staging ---------------------------------------------------------------------

// The next chunk's rows of one tensor on their way to LDS.
template <typename IT, int D, bool REV>
struct Stage {
  typedef Tile<IT, D> T;
  static constexpr int N = C * T::PPR / NTHR;  // 16-byte pieces per thread
  uint4 x[N];
  // `base` is the head's first row.
  __device__ __forceinline__ void load(const IT* base, int c, int L) {
    const int rows = min(C, L - c * C);
    const rsrc_t r = make_rsrc(base + (size_t)c * C * D, (uint32_t)(rows * D * sizeof(IT)));
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = bload16(r, (i * NTHR + threadIdx.x) * 16, 0);
  }
  __device__ __forceinline__ void store(T t) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * NTHR + threadIdx.x, row = e / T::PPR;
      t.put(REV ? C - 1 - row : row, e % T::PPR, x[i]);
    }
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

// Enough segments for two workgroups on each of the 256 CUs, none of them
// shorter than kMinChunks chunks (a segment costs a state's write and two
// reads, 4 d_k d_v bytes each, against the rows it spares a walk).
constexpr int kWorkgroups = 512, kMinChunks = 4;
inline Split split_of(int BH, int L) {
  Split s;
  s.nc = cdiv(L, C);
  s.cps = cdiv(s.nc, cdiv(kWorkgroups, BH));
  if (s.cps < kMinChunks) s.cps = kMinChunks;
  s.nseg = cdiv(s.nc, s.cps);
  return s;
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

// S += K^T diag(up) V after S *= total, on this wave's columns.
template <typename IT, int DK, int DV>
__device__ __forceinline__ void update_state(f32x4 (&st)[DK / 16][DV / 64], Tile<IT, DK> K,
                                             const typename Tile<IT, DV>::Frag (&vf)[C / 32][DV / 64],
                                             const Decays* d) {
  constexpr int CT = DV / 64;
  const int g = (threadIdx.x & 63) >> 4;
  const float total = d->total;
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) st[kt][ct] *= total;
#pragma unroll
  for (int tb = 0; tb < C / 32; ++tb) {
    const f32x4 u0 = *reinterpret_cast<const f32x4*>(&d->up[32 * tb + 4 * g]);
    const f32x4 u1 = *reinterpret_cast<const f32x4*>(&d->up[32 * tb + 16 + 4 * g]);
    Made<IT, 3> y[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float x[8];
      to_floats(vf[tb][ct], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= u0[e], x[4 + e] *= u1[e];
      y[ct] = Made<IT, 3>(x);
    }
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
      const auto a = K.col(16 * kt, tb);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) st[kt][ct] = mma(a, y[ct], st[kt][ct]);
    }
  }
}

// fp32 state (row-major [DK][DV], or [DV][DK] when TRANS) <-> this wave's
// accumulators: rows 16 kt + 4 g + e, column j.
template <int DK, int DV, bool TRANS>
__device__ __forceinline__ void load_state(f32x4 (&st)[DK / 16][DV / 64], const float* S) {
  const int l = threadIdx.x & 63, g = l >> 4, w = threadIdx.x >> 6;
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < DV / 64; ++ct) {
      const int j = w * (DV / 4) + 16 * ct + (l & 15), k0 = 16 * kt + 4 * g;
      if (!S) {
        st[kt][ct] = zero4();
      } else if (TRANS) {
        st[kt][ct] = *reinterpret_cast<const f32x4*>(S + (size_t)j * DK + k0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) st[kt][ct][e] = S[(size_t)(k0 + e) * DV + j];
      }
    }
}
template <int DK, int DV, bool TRANS>
__device__ __forceinline__ void store_state(const f32x4 (&st)[DK / 16][DV / 64], float* S, float scale) {
  const int l = threadIdx.x & 63, g = l >> 4, w = threadIdx.x >> 6;
#pragma unroll
  for (int kt = 0; kt < DK / 16; ++kt)
#pragma unroll
    for (int ct = 0; ct < DV / 64; ++ct) {
      const int j = w * (DV / 4) + 16 * ct + (l & 15), k0 = 16 * kt + 4 * g;
      const f32x4 x = st[kt][ct] * scale;
      if (TRANS) {
        *reinterpret_cast<f32x4*>(S + (size_t)j * DK + k0) = x;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[(size_t)(k0 + e) * DV + j] = x[e];
      }
    }
}

template <typename IT, int DV>
__device__ __forceinline__ void value_frags(typename Tile<IT, DV>::Frag (&vf)[C / 32][DV / 64], Tile<IT, DV> V) {
  const int w = threadIdx.x >> 6;
#pragma unroll
  for (int tb = 0; tb < C / 32; ++tb)
#pragma unroll
    for (int ct = 0; ct < DV / 64; ++ct) vf[tb][ct] = V.col(w * (DV / 4) + 16 * ct, tb);
}

template <typename IT, int DK, int DV>
constexpr int state_lds() { return Tile<IT, DK>::bytes + Tile<IT, DV>::bytes + (int)sizeof(Decays); }

template <typename IT, int DK, int DV, bool REV>
__global__ __launch_bounds__(NTHR, sizeof(IT) == 2 ? 2 : 1) void state_kernel(StateArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const Tile<IT, DK> K{smem};
  const Tile<IT, DV> V{smem + Tile<IT, DK>::bytes};
  Decays* const dec = reinterpret_cast<Decays*>(smem + Tile<IT, DK>::bytes + Tile<IT, DV>::bytes);

  int bh, seg;
  if (!item_of(blockIdx.x, a.BH, a.grp, a.count, bh, seg)) return;
  seg += a.first;
  const int L = a.L, c0 = seg * a.s.cps, c1 = min(c0 + a.s.cps, a.s.nc);
  const IT* k = a.k.head<IT>(bh, L, DK);
  const IT* v = a.v.head<IT>(bh, L, DV);
  const float* g = a.g ? a.g + (size_t)bh * L : nullptr;
  const int n = c1 - c0;
  auto chunk = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };
  const bool last_wave = threadIdx.x >= NTHR - 64;

  f32x4 st[DK / 16][DV / 64];
  load_state<DK, DV, false>(st, nullptr);
  Stage<IT, DK, REV> sk;
  Stage<IT, DV, REV> sv;
  sk.load(k, chunk(0), L);
  sv.load(v, chunk(0), L);
  float gn = load_decay<REV>(g, chunk(0), L);
  double sum = 0.0;
  for (int i = 0; i < n; ++i) {
    sk.store(K);
    sv.store(V);
    if (last_wave) sum += fill_decays(dec, gn);
    __syncthreads();
    const int cn = chunk(min(i + 1, n - 1));
    sk.load(k, cn, L);
    sv.load(v, cn, L);
    gn = load_decay<REV>(g, cn, L);
    typename Tile<IT, DV>::Frag vf[C / 32][DV / 64];
    value_frags<IT, DV>(vf, V);
    update_state<IT, DK, DV>(st, K, vf, dec);
    __syncthreads();
  }
  store_state<DK, DV, false>(st, a.states + ((size_t)bh * a.slots + seg) * (DK * DV), 1.f);
  if (threadIdx.x == NTHR - 1) a.decays[(size_t)bh * a.s.nseg + seg] = sum;
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
  int slots, nseg, N;
};

template <bool REV>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int bh = blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (e >= a.N) return;
  float* S = a.states + (size_t)bh * a.slots * a.N + e;
  const double* d = a.decays + (size_t)bh * a.nseg;
  f32x4 run = a.S0 ? *reinterpret_cast<const f32x4*>(a.S0 + (size_t)bh * a.N + e) : zero4();
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

// ---- the output kernel ---------------------------------------------------------------

// Which extra sums a pass leaves for the decay's gradient.
enum Extra {
  kNone = 0,
  kDots = 1,   // per row: (row of w) . (the part of the output that comes from the entering state)
  kPairs = 2   // kDots, and per row the sums of the chunk's pair terms (below)
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
// key rows): fragment (rt, kb), kb <= rt / 2, holds key tiles 2 kb, 2 kb + 1.
__host__ __device__ constexpr int pfrag(int rt, int kb) { return (rt >> 1) * ((rt >> 1) + 1) + (rt & 1) * ((rt >> 1) + 1) + kb; }
constexpr int kPFrags = 6;
static_assert(pfrag(0, 0) == 0 && pfrag(1, 0) == 1 && pfrag(2, 0) == 2 && pfrag(2, 1) == 3 &&
              pfrag(3, 0) == 4 && pfrag(3, 1) == 5, "six fragments");

template <typename IT, int NS>
struct PBuf;
template <int NS>
struct PBuf<bf16, NS> {
  static constexpr int bytes = kPFrags * NS * 64 * 16;
  unsigned char* p;
  __device__ __forceinline__ uint2* at(int f, int s, int half) const {
    return reinterpret_cast<uint2*>(p + ((f * NS + s) * 64 + (threadIdx.x & 63)) * 16) + half;
  }
  __device__ __forceinline__ void put(int f, int half, f32x4 x) const {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint2 u = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
      *at(f, s, half) = u;
      x[0] -= __uint_as_float(u.x << 16);
      x[1] -= __uint_as_float(u.x & 0xffff0000u);
      x[2] -= __uint_as_float(u.y << 16);
      x[3] -= __uint_as_float(u.y & 0xffff0000u);
    }
  }
  __device__ __forceinline__ Made<bf16, NS> get(int f) const {
    Made<bf16, NS> m;
#pragma unroll
    for (int s = 0; s < NS; ++s) m.p[s] = as_bf16x8(*reinterpret_cast<const uint4*>(at(f, s, 0)));
    return m;
  }
};
template <int NS>
struct PBuf<float, NS> {
  static constexpr int bytes = kPFrags * 64 * 32;
  unsigned char* p;
  __device__ __forceinline__ f32x4* at(int f, int half) const {
    return reinterpret_cast<f32x4*>(p + (f * 2 + half) * 1024) + (threadIdx.x & 63);
  }
  __device__ __forceinline__ void put(int f, int half, f32x4 x) const { *at(f, half) = x; }
  __device__ __forceinline__ Made<float, NS> get(int f) const {
    const f32x4 a = *at(f, 0), b = *at(f, 1);
    Made<float, NS> m;
    m.p = F32x8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    return m;
  }
};

// Sums for the decay's gradient, gathered per chunk without atomics: every
// writer has a slot of its own.
struct Sums {
  float dots[4][C];   // by wave
  float out[10][16];  // pair terms of an output tile's rows, by tile of P
  float key[10][16];  // ... of a key tile's rows
};
__device__ __forceinline__ int tri(int rt, int it) { return rt * (rt + 1) / 2 + it; }

__device__ __forceinline__ float sum_groups(float x) {  // over the 4 lane groups (same i)
  x += __shfl_xor(x, 16, 64);
  x += __shfl_xor(x, 32, 64);
  return x;
}
__device__ __forceinline__ float sum_lanes16(float x) {  // over the 16 lanes of a group
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) x += __shfl_xor(x, off, 64);
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

// Bytes of LDS: the tiles, P, the decay tables of this chunk and the next,
// and the sums.
template <typename IT, typename OT, int DK, int DV, int EXTRA>
struct OutLds {
  // Pieces of an fp32 operand (see "Precision" above): P and the state where
  // they only reach the output; the state where it reaches the row sums.
  static constexpr int NSP = sizeof(OT) == 2 || EXTRA != kNone ? 2 : 3;
  static constexpr int NSS = sizeof(OT) == 2 && EXTRA == kNone ? 2 : 3;
  static constexpr int K = Tile<IT, DK>::bytes;
  static constexpr int V = K + Tile<IT, DK>::bytes;
  static constexpr int W = V + Tile<IT, DV>::bytes;
  static constexpr int P = W + (EXTRA != kNone ? Tile<IT, DV>::bytes : 0);
  static constexpr int D = P + PBuf<IT, NSP>::bytes;
  static constexpr int S = D + 2 * (int)sizeof(Decays);
  static constexpr int bytes = S + (EXTRA != kNone ? (int)sizeof(Sums) : 0);
};

template <typename IT, typename OT, int DK, int DV, bool REV, int EXTRA>
__global__ __launch_bounds__(NTHR, sizeof(IT) == 2 ? 2 : 1) void out_kernel(OutArgs a) {
  using LD = OutLds<IT, OT, DK, DV, EXTRA>;
  constexpr int NRT = C / 16, CT = DV / 64, NSP = LD::NSP, NSS = LD::NSS;
  constexpr bool TRANS = EXTRA != kNone;  // dq and dk walk the transposed state
  extern __shared__ __align__(16) unsigned char smem[];
  const Tile<IT, DK> Q{smem}, K{smem + LD::K};
  const Tile<IT, DV> V{smem + LD::V}, W{smem + LD::W};
  const PBuf<IT, NSP> P{smem + LD::P};
  Decays* const tables = reinterpret_cast<Decays*>(smem + LD::D);
  Sums* const sums = reinterpret_cast<Sums*>(smem + LD::S);

  int bh, seg;
  if (!item_of(blockIdx.x, a.BH, a.grp, a.s.nseg, bh, seg)) return;
  const int L = a.L, c0 = seg * a.s.cps, c1 = min(c0 + a.s.cps, a.s.nc), n = c1 - c0;
  const IT* q = a.q.head<IT>(bh, L, DK);
  const IT* k = a.k.head<IT>(bh, L, DK);
  const IT* v = a.v.head<IT>(bh, L, DV);
  const IT* wp = EXTRA != kNone ? a.w.head<IT>(bh, L, DV) : nullptr;
  const float* g = a.g ? a.g + (size_t)bh * L : nullptr;
  OT* out = static_cast<OT*>(a.out) + (size_t)bh * L * DV;
  const int lane = threadIdx.x & 63, lg = lane >> 4, li = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto chunk = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };

  // This wave's tiles of P (output tile rt, key tile it <= rt): 10 over 4 waves.
  constexpr int kRt[4][3] = {{3, 3, 0}, {3, 3, 2}, {2, 2, -1}, {1, 1, -1}};
  constexpr int kIt[4][3] = {{0, 1, 0}, {2, 3, 0}, {1, 2, -1}, {0, 1, -1}};
  int prt[3], pit[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    prt[x] = w == 0 ? kRt[0][x] : w == 1 ? kRt[1][x] : w == 2 ? kRt[2][x] : kRt[3][x];
    pit[x] = w == 0 ? kIt[0][x] : w == 1 ? kIt[1][x] : w == 2 ? kIt[2][x] : kIt[3][x];
  }
  // The tiles above the diagonal that share a fragment with one below.
  if (w == 0) P.put(pfrag(0, 0), 1, zero4());
  if (w == 1) P.put(pfrag(2, 1), 1, zero4());

  f32x4 st[DK / 16][CT];
  const float* S = a.s.nseg > 1 ? a.states + ((size_t)bh * a.slots + seg) * (DK * DV)
                                : (a.S0 ? a.S0 + (size_t)bh * (DK * DV) : nullptr);
  load_state<DK, DV, TRANS>(st, S);

  Stage<IT, DK, REV> sq, sk;
  Stage<IT, DV, REV> sv, sw;
  auto load = [&](int c) {
    sq.load(q, c, L);
    sk.load(k, c, L);
    sv.load(v, c, L);
    if (EXTRA != kNone) sw.load(wp, c, L);
  };
  load(chunk(0));
  float gn = load_decay<REV>(g, chunk(0), L);
  if (w == 3) fill_decays(&tables[0], gn);

  for (int ci = 0; ci < n; ++ci) {
    const int c = chunk(ci);
    const Decays* dec = &tables[ci & 1];
    sq.store(Q);
    sk.store(K);
    sv.store(V);
    if (EXTRA != kNone) sw.store(W);
    __syncthreads();
    const int cn = chunk(min(ci + 1, n - 1));
    load(cn);
    gn = load_decay<REV>(g, cn, L);

    // P^T tiles: rows are key rows 16 it + 4 lg + e, the column is output row
    // 16 rt + li.
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const int rt = prt[x], it = pit[x];
      if (rt < 0) continue;
      f32x4 p = zero4();
#pragma unroll
      for (int kb = 0; kb < DK / 32; ++kb) p = mma(K.row(16 * it, kb), Q.row(16 * rt, kb), p);
      const int r = 16 * rt + li;
      const double Gr = dec->G[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * it + 4 * lg + e;
        p[e] = i <= r ? p[e] * exp2_hw((float)(Gr - dec->G[i])) : 0.f;
      }
      P.put(pfrag(rt, it >> 1), it & 1, p);
      if (EXTRA == kPairs) {
        // Pair terms: P_ri (w_r . v_i), i < r.
        f32x4 y = zero4();
#pragma unroll
        for (int kb = 0; kb < DV / 32; ++kb) y = mma(V.row(16 * it, kb), W.row(16 * rt, kb), y);
        float col = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 16 * it + 4 * lg + e;
          const float m = i < r ? p[e] * y[e] : 0.f;
          col += m;
          const float row = sum_lanes16(m);
          if (li == 0) sums->key[tri(rt, it)][4 * lg + e] = row;
        }
        col = sum_groups(col);
        if (lg == 0) sums->out[tri(rt, it)][li] = col;
      }
    }

    // Output tiles (rows: this wave's columns, column: row 16 rt + li), first
    // what comes from the entering state.
    f32x4 acc[NRT][CT];
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = zero4();
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) {
      Made<IT, NSS> s[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const f32x4 x = st[2 * kb][ct], y = st[2 * kb + 1][ct];
        const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        s[ct] = Made<IT, NSS>(z);
      }
#pragma unroll
      for (int rt = 0; rt < NRT; ++rt) {
        const auto b = Q.row(16 * rt, kb);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = mma(s[ct], b, acc[rt][ct]);
      }
    }
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
      const float f = exp2_hw((float)dec->G[16 * rt + li]);
      float dot = 0.f;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        acc[rt][ct] *= f;
        if (EXTRA != kNone) {
          const f32x4 y = W.four(16 * rt + li, w * (DV / 4) + 16 * ct + 4 * lg);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot += acc[rt][ct][e] * y[e];
        }
      }
      if (EXTRA != kNone) {
        dot = sum_groups(dot);
        if (lg == 0) sums->dots[w][16 * rt + li] = dot;
      }
    }
    __syncthreads();

    // ... then what comes from the chunk's own rows.
    typename Tile<IT, DV>::Frag vf[C / 32][CT];
    value_frags<IT, DV>(vf, V);
#pragma unroll
    for (int rt = 0; rt < NRT; ++rt) {
#pragma unroll
      for (int kb = 0; kb <= rt / 2; ++kb) {
        const auto b = P.get(pfrag(rt, kb));
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[rt][ct] = mma(vf[kb][ct], b, acc[rt][ct]);
      }
      const int t = token_of<REV>(c, 16 * rt + li);
      if (t < L) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          store4(out + (size_t)t * DV + w * (DV / 4) + 16 * ct + 4 * lg, acc[rt][ct]);
      }
    }
    if (EXTRA != kNone && w == 0) {
      const size_t at = (size_t)bh * a.s.nc * C + token_of<REV>(c, lane);
      a.dots[at] = (sums->dots[0][lane] + sums->dots[1][lane]) + (sums->dots[2][lane] + sums->dots[3][lane]);
      if (EXTRA == kPairs) {
        const int tile = lane >> 4;
        float y = 0.f;
        for (int x = 0; x < NRT; ++x) {
          if (x <= tile) y += sums->out[tri(tile, x)][li];
          if (x >= tile) y -= sums->key[tri(x, tile)][li];
        }
        a.pairs[at] = y;
      }
    }
    update_state<IT, DK, DV>(st, K, vf, dec);
    if (w == 3) fill_decays(&tables[(ci + 1) & 1], gn);
    __syncthreads();
  }

  if (a.last && seg == (REV ? 0 : a.s.nseg - 1)) {
    // Reversed, the walk ends with the gradient of the state after token 0;
    // the state before it is one decay further.
    const float f = REV && g ? exp2_hw((float)log2_decay(g[0])) : 1.f;
    store_state<DK, DV, TRANS>(st, a.last + (size_t)bh * a.last_stride, f);
  }
}

// ---- launches --------------------------------------------------------------------------

template <typename K>
hipError_t allow_lds(K* kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename IT, int DK, int DV, bool REV>
hipError_t launch_state(const StateArgs& a, hipStream_t stream) {
  constexpr int lds = state_lds<IT, DK, DV>();
  static_assert(lds <= 160 * 1024, "LDS budget");
  auto* kernel = &state_kernel<IT, DK, DV, REV>;
  hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  prof_mark(kSlotLinearState, false, stream);
  hipLaunchKernelGGL(kernel, dim3((unsigned)items(a.BH, a.grp, a.count)), dim3(NTHR), lds, stream, a);
  e = hipGetLastError();
  prof_mark(kSlotLinearState, true, stream);
  return e;
}

template <bool REV>
hipError_t launch_combine(const CombineArgs& a, int BH, hipStream_t stream) {
  prof_mark(kSlotLinearState, false, stream);
  hipLaunchKernelGGL(combine_kernel<REV>, dim3((unsigned)cdiv(a.N, 1024), (unsigned)BH), dim3(256), 0, stream, a);
  hipError_t e = hipGetLastError();
  prof_mark(kSlotLinearState, true, stream);
  return e;
}

template <typename IT, typename OT, int DK, int DV, bool REV, int EXTRA>
hipError_t launch_out(const OutArgs& a, int slot, hipStream_t stream) {
  constexpr int lds = OutLds<IT, OT, DK, DV, EXTRA>::bytes;
  static_assert(lds <= (sizeof(IT) == 2 ? 80 : 160) * 1024, "two bf16 workgroups share a CU's LDS");
  auto* kernel = &out_kernel<IT, OT, DK, DV, REV, EXTRA>;
  hipError_t e = allow_lds(kernel, lds);
  if (e != hipSuccess) return e;
  prof_mark(slot, false, stream);
  hipLaunchKernelGGL(kernel, dim3((unsigned)items(a.BH, a.grp, a.s.nseg)), dim3(NTHR), lds, stream, a);
  e = hipGetLastError();
  prof_mark(slot, true, stream);
  return e;
}

// The state of a call without tokens: dst = src, or zeros.
hipError_t launch_copy_state(float* dst, const float* src, size_t n, hipStream_t stream);

}  // namespace lin
}  // namespace dn
