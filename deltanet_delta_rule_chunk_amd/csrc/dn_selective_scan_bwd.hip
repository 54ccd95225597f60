// dn_selective_scan_bwd.hip -- gradient of the selective state space scan on
// gfx950 (the recurrence, segments and a workgroup's tile: dn_selective_scan.h).
//
// With g_t = dy_t silu(z_t) and G_t the gradient of h_t,
//     G_t = C_t g_t + e^{dt_{t+1} A} G_{t+1}
//     dC_t = sum_d h_t g_t           dB_t = sum_d G_t dt_t u_t
//     d(dt u)_t = sum_n G_t B_t      thr_t = G_t e^{dt_t A} h_{t-1}
//     ddt_t = u_t d(dt u)_t + sum_n thr_t A,   dA = sum_t thr_t dt_t
//     du_t = dt_t d(dt u)_t + D g_t,           dz_t = dy_t (C_t h_t + D u_t) silu'(z_t).
//
// A walk forward leaves the state in front of every 8 tokens; the walk back takes
// them from the last to the first: 8 steps forward from the state, decays and
// states kept in registers, then 8 back (16 at a time need more registers than
// there are: 2040 us against 1878 for 2 x 8192 tokens of 4096 channels).  Where sequences are
// cut into segments, the first launch walks every segment from zero in both
// directions, combine() joins them, and a state in front of 8 tokens is what the
// segment makes of it plus the segment's entering state times e^{A sum dt}.
//
// Sums over channels (dB, dC) are sums over lanes: 4 values of a token become one
// register per lane by two exchanges of half a wave, 8 tokens' registers become
// one by four more steps within rows of 16 lanes: 2.2 vector operations per value.
// Every block of 64 channels leaves its part, added up in fixed order at the end,
// as are the segments' parts of dA, dD and the bias's gradient.
//
// Bound by the vector units: busy for 92% of the walk back and 98% of the sums
// before it (890 and 410 us at those sizes).  The walk back keeps 64 to 193 scalar registers in
// vector lanes (rows' addresses and strides: 110 to 130 reads of them among its 1578 vector
// instructions per 16 tokens), and with 8 states and the gate, in three of four forms, 5 to 20 vector
// registers in scratch memory (2 x 4096 tokens of 2048 channels 235 us; 16 states 377).

#include "dn_selective_scan.h"

namespace dn {
namespace ssm {

constexpr int kHalf = kTile / 2;

struct BwdSpace {
  float* tiles;   // [half tile][D][N] state in front of a half (cut sequences: from the segment's zero)
  float* before;  // cut sequences: [half tile][D] sum of dt from the segment's first token to the half
  float* ahead;   // cut sequences: [seg][D][N] states in front of segments
  float* back;    // cut sequences: [seg][D][N] gradients of the states behind segments
  float* logs;    // cut sequences: [seg][D] sum of dt
  float* dBC;     // [2][block of channels][B L][N]
  float* dA;      // [seg][D][N]
  float* dvec;    // [seg][2][D]: D's and the bias's gradients
};

// ---- states in front of tiles; what segments make from zero in both directions ----------------

// blockIdx.y = 0: forward.  1 (cut sequences only): backward.
template <int NW, typename T, bool GATE, bool SPLIT, bool BACK>
__device__ __forceinline__ void sums(const ScanArgs& a, const Plan& pl, int blocks_d, const BwdSpace& ws,
                                     float2 (&sx)[2][kTile][kCh]) {
  constexpr int N = 4 * NW, R = group_rows<T>();
  using At = Spot<NW>;
  const int id = blockIdx.x / blocks_d, ch0 = (blockIdx.x - id * blocks_d) * kCh;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), ch = ch0 + lane;
  Segment g;
  if (!segment_of(pl, id, g) || g.seq < 0) return;
  if (BACK && g.first) return;  // nothing asks for what arrives at its front
  const At at;
  const bool on = ch < a.D;
  const int c = ch0 + at.c < a.D ? ch0 + at.c : a.D - 4;
  const int tiles = (g.n + kTile - 1) / kTile;
  const int begin = BACK ? (tiles - 1) * kTile : 0;  // first row of the first tile
  const long long row = g.row + begin;
  Feed<NW, T> x(BACK ? a.dy : a.u.p, BACK ? ((long long)g.batch * a.L + row) * a.D : g.batch * a.u.sb + row * a.u.sl,
                BACK ? a.D : a.u.sl, at, c);
  Feed<NW, T> dt(a.dt.p, g.batch * a.dt.sb + row * a.dt.sl, a.dt.sl, at, c);
  Feed<NW, T> z(a.z.p, g.batch * a.z.sb + row * a.z.sl, a.z.sl, at, c);
  const TokenRows& m = BACK ? a.Cm : a.Bm;
  const T* M = static_cast<const T*>(m.p) + g.batch * m.sb + row * m.sl + 4 * w;  // of the tile
  const f32x4 bias = a.dt_bias ? get4(a.dt_bias + c) : zero4();
  f32x4 A2 = zero4(), h = zero4();
  const size_t place = (size_t)ch * N + 4 * w, state = (size_t)a.D * N;
  if (on) {
    A2 = get4(a.A + place) * kLog2e;
    if (BACK ? g.last && a.dhT : g.first && a.h0) h = get4((BACK ? a.dhT : a.h0) + (size_t)g.seq * state + place);
  }
  const long long tile0 = first_tile(pl, g, id);
  float sum = 0.f;
  Ahead<NW, T> next(m.p, g.batch * m.sb + row * m.sl, m.sl);
  const auto fetch = [&](int n) {
    x.fetch(at, c, n);
    dt.fetch(at, c, n);
    if (GATE && BACK) z.fetch(at, c, n);
    next.fetch(n);
  };
  constexpr int kStep = BACK ? -1 : 1;
  int tile = BACK ? tiles - 1 : 0, buf = 0;
  if (tiles > 0) fetch(g.n - begin);
  for (int i = 0; i < tiles; ++i, tile += kStep, buf ^= 1) {
    if (at.in_tile()) {
#pragma unroll
      for (int p = 0; p < At::kPasses; ++p) {
        const f32x4 d = softplus4(wide(dt.raw[p]) + bias, a.softplus);
        f32x4 v = wide(x.raw[p]);
        if (!BACK) v *= d;
        if (GATE && BACK) {
          const f32x4 zz = wide(z.raw[p]);
          v *= zz * sigmoid4(zz);
        }
        f32x4* const out = reinterpret_cast<f32x4*>(&sx[buf][at.row(p)][at.c]);
        out[0] = f32x4{d[0], v[0], d[1], v[1]};
        out[1] = f32x4{d[2], v[2], d[3], v[3]};
      }
    }
    next.arrived();
    x.move(kStep);
    dt.move(kStep);
    if (GATE && BACK) z.move(kStep);
    next.move(kStep);
    if (i + 1 < tiles) fetch(g.n - (tile + kStep) * kTile);
    const int n = min(kTile, g.n - tile * kTile);
    float part = 0.f;
    const auto step = [&](f32x4 b, float2 v) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (BACK) h[s] = exp2_fast(v.x * A2[s]) * fmaf(b[s], v.y, h[s]);
        else h[s] = fmaf(exp2_fast(v.x * A2[s]), h[s], v.y * b[s]);
      }
      if (!BACK) part += v.x;
    };
    const auto keep = [&](int half) {
      if (BACK || !on) return;
      const size_t at_ = (size_t)(tile0 + tile) * 2 + half;
      *reinterpret_cast<f32x4*>(ws.tiles + at_ * state + place) = h;
      if (SPLIT && w == 0) ws.before[at_ * a.D + ch] = sum + part;
    };
    keep(0);
    if (n == kTile) {
      // Groups of rows in the walk's direction.
      constexpr int Q = kTile / R;
      Group<T> gm[2];
      float2 v[2][R];
      const int q0 = BACK ? Q - 1 : 0;
      gm[0].load(M + q0 * R * m.sl, m.sl);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j) v[0][j] = sx[buf][q0 * R + j][lane];
      wait_reads();
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const int now = k & 1, next = now ^ 1, q = BACK ? Q - 2 - k : k + 1;
        if (k + 1 < Q) {
          gm[next].load(M + q * R * m.sl, m.sl);
#pragma unroll
          for (int j = 0; j < R; ++j) v[next][j] = sx[buf][q * R + j][lane];
        }
        __builtin_amdgcn_sched_barrier(0);
        if (k == Q / 2) keep(1);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int r = BACK ? R - 1 - j : j;
          step(wide(gm[now].r[r]), v[now][r]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      __syncthreads();
      for (int j = 0; j < n; ++j) {
        const int t = BACK ? n - 1 - j : j;
        if (t == kHalf) keep(1);
        step(wide(uniform4(M + t * m.sl)), sx[buf][t][lane]);
      }
    }
    M += kStep * kTile * m.sl;
    sum += part;
  }
  if (SPLIT && on) {
    *reinterpret_cast<f32x4*>((BACK ? ws.back : ws.ahead) + (size_t)id * state + place) = h;
    if (!BACK && w == 0) ws.logs[(size_t)id * a.D + ch] = sum;
  }
}
template <int NW, typename T, bool GATE, bool SPLIT>
__global__ __launch_bounds__(64 * NW) void sums_kernel(ScanArgs a, Plan pl, int blocks_d, BwdSpace ws) {
  __shared__ float2 sx[2][kTile][kCh];  // dt, and dt u or g
  if (SPLIT && blockIdx.y) sums<NW, T, GATE, SPLIT, true>(a, pl, blocks_d, ws, sx);
  else sums<NW, T, GATE, SPLIT, false>(a, pl, blocks_d, ws, sx);
}

// ---- sums over lanes ---------------------------------------------------------------------------

__device__ __forceinline__ float swap32_add(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_add(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Four values per lane: row r of 16 lanes gets sums over the four rows of v[r].
__device__ __forceinline__ float rows_sum(f32x4 v) { return swap16_add(swap32_add(v[0], v[2]), swap32_add(v[1], v[3])); }
// Lanes whose `bit` is set get a sum of b over themselves and a partner, the others of a.
template <int CTRL>
__device__ __forceinline__ float fold(float a, float b, bool bit) {
  const float keep = bit ? b : a, send = bit ? a : b;
  return keep + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(send), CTRL, 0xf, 0xf, true));
}
// 8 values per lane: lanes i and i + 8 of 16 get the sum of v[i] over the 16.
__device__ __forceinline__ float lanes_sum(float (&v)[8], int lane) {
  constexpr int kMirror8 = 0x141, kMirror4 = 0x1b, kMirror2 = 0xb1, kTurn8 = 0x128;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fold<kMirror8>(v[i], v[i + 4], lane & 4);
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = fold<kMirror4>(v[i], v[i + 2], lane & 2);
  const float x = fold<kMirror2>(v[0], v[1], lane & 1);
  return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), kTurn8, 0xf, 0xf, true));
}

// ---- the walk back -------------------------------------------------------------------------------

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

template <int NW, typename T, bool GATE, bool SPLIT>
__global__ __launch_bounds__(64 * NW, 2) void back_kernel(ScanArgs a, Plan pl, int blocks_d, BwdSpace ws) {
  constexpr int N = 4 * NW, R = 2 * group_rows<T>(), Q = kHalf / R;
  using At = Spot<NW>;
  __shared__ float2 sx[kTile][kCh];                    // dt, dt u
  __shared__ float sg[kTile][kCh];                     // g
  __shared__ float sdx[NW][kTile][kCh];                // the waves' parts of d(dt u),
  __shared__ float sda[NW][kTile][kCh];                // of sum_n thr A (times log2 e),
  __shared__ float sy[GATE ? NW : 1][GATE ? kTile : 1][kCh];  // of C h
  const int id = blockIdx.x / blocks_d, block = blockIdx.x - id * blocks_d, ch0 = block * kCh;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), ch = ch0 + lane;
  Segment g;
  if (!segment_of(pl, id, g)) return;
  const At at;
  const bool has = ch0 + at.c < a.D, on = ch < a.D;
  const int c = has ? ch0 + at.c : a.D - 4;
  const size_t token = (size_t)g.batch * a.L + g.row;  // of the segment's first row
  const size_t tokens = (size_t)a.B * a.L;
  const size_t place = (size_t)ch * N + 4 * w, state = (size_t)a.D * N;
  float* const dA_to = ws.dA + (size_t)id * state + place;
  float* const dvec = ws.dvec + (size_t)id * 2 * a.D;
  const int tiles = (g.n + kTile - 1) / kTile, begin = max(tiles - 1, 0) * kTile;
  // Of the tile, from the segment's last on.
  T* du = static_cast<T*>(a.du) + (token + begin) * a.D;
  T* ddt = static_cast<T*>(a.ddt) + (token + begin) * a.D;
  T* dz = static_cast<T*>(a.dz) + (GATE ? (token + begin) * a.D : 0);
  float* dB = ws.dBC + ((size_t)block * tokens + token + begin) * N;
  float* dC = dB + (size_t)blocks_d * tokens * N;
  if (g.seq < 0) {
    const size_t back = (size_t)begin * a.D;
    for (int r = at.r; r < g.n && has; r += At::kRows) {
      const size_t o = (size_t)r * a.D + c;
      put4(du - back + o, zero4());
      put4(ddt - back + o, zero4());
      if (GATE) put4(dz - back + o, zero4());
    }
    const size_t first = (size_t)begin * N;
    for (size_t i = threadIdx.x; i < (size_t)g.n * N; i += 64 * NW) (dB - first)[i] = (dC - first)[i] = 0.f;
    if (on) *reinterpret_cast<f32x4*>(dA_to) = zero4();
    if (on && w == 0) dvec[ch] = dvec[a.D + ch] = 0.f;
    return;
  }
  const long long row = g.row + begin;
  Feed<NW, T> u(a.u.p, g.batch * a.u.sb + row * a.u.sl, a.u.sl, at, c);
  Feed<NW, T> dt(a.dt.p, g.batch * a.dt.sb + row * a.dt.sl, a.dt.sl, at, c);
  Feed<NW, T> z(a.z.p, g.batch * a.z.sb + row * a.z.sl, a.z.sl, at, c);
  Feed<NW, T> dy(a.dy, (long long)(token + begin) * a.D, a.D, at, c);
  const T* Bt = static_cast<const T*>(a.Bm.p) + g.batch * a.Bm.sb + row * a.Bm.sl + 4 * w;  // of the tile
  const T* Ct = static_cast<const T*>(a.Cm.p) + g.batch * a.Cm.sb + row * a.Cm.sl + 4 * w;
  const f32x4 bias = a.dt_bias ? get4(a.dt_bias + c) : zero4();
  const f32x4 skip = a.skip ? get4(a.skip + c) : zero4();
  f32x4 A2 = zero4(), G = zero4(), enter = zero4();
  if (on) {
    A2 = get4(a.A + place) * kLog2e;
    if (SPLIT && !g.first) enter = get4(ws.ahead + (size_t)id * state + place);
    if (SPLIT && !g.last) G = get4(ws.back + (size_t)id * state + place);
    if (g.last && a.dhT) G = get4(a.dhT + (size_t)g.seq * state + place);
  }
  const long long tile0 = first_tile(pl, g, id);
  f32x4 dA = zero4(), dskip = zero4(), dbias = zero4();
  f32x4 held[2] = {zero4(), zero4()};  // the next tile's states
  float since[2] = {0.f, 0.f};
  Ahead<NW, T> nB(a.Bm.p, g.batch * a.Bm.sb + row * a.Bm.sl, a.Bm.sl), nC(a.Cm.p, g.batch * a.Cm.sb + row * a.Cm.sl, a.Cm.sl);
  // (8 states leave no registers for it: two passes of rows per thread.  2 x 4096 tokens of 2048
  // channels, forward + backward, 347 us with it, 328 without; 16 states, 2 x 8192 of 4096, 1715 and 1743.)
  constexpr bool kAhead = NW > 2;
  const auto fetch = [&](int tile) {
    const int n = g.n - tile * kTile;
    if (kAhead) {
      nB.fetch(n);
      nC.fetch(n);
    }
    u.fetch(at, c, n);
    dt.fetch(at, c, n);
    dy.fetch(at, c, n);
    if (GATE) z.fetch(at, c, n);
    if (on) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i * kHalf >= n) break;
        const size_t at_ = (size_t)(tile0 + tile) * 2 + i;
        held[i] = get4(ws.tiles + at_ * state + place);
        if (SPLIT && !g.first) since[i] = ws.before[at_ * a.D + ch];
      }
    }
  };
  if (tiles > 0) fetch(tiles - 1);
  // One tile; only the segment's last may be short.
  const auto one = [&](int tile, auto full) {
    constexpr bool kFull = decltype(full)::value;
    const int n = kFull ? kTile : g.n - tile * kTile;
    Raw4<T> ru[At::kPasses], rd[At::kPasses], rz[At::kPasses], ry[At::kPasses];
    if (at.in_tile()) {
#pragma unroll
      for (int p = 0; p < At::kPasses; ++p) {
        const int r = at.row(p);
        ru[p] = u.raw[p];
        rd[p] = dt.raw[p];
        ry[p] = dy.raw[p];
        if (GATE) rz[p] = z.raw[p];
        f32x4 d = softplus4(wide(rd[p]) + bias, a.softplus), x = d * wide(ru[p]), gy = wide(ry[p]);
        if (GATE) {
          const f32x4 zz = wide(rz[p]);
          gy *= zz * sigmoid4(zz);
        }
        // Channels behind D add nothing to the sums over channels, rows behind the segment
        // change nothing.
        if (!has || (!kFull && r >= n)) d = x = gy = zero4();
        f32x4* const out = reinterpret_cast<f32x4*>(&sx[r][at.c]);
        out[0] = f32x4{d[0], x[0], d[1], x[1]};
        out[1] = f32x4{d[2], x[2], d[3], x[3]};
        *reinterpret_cast<f32x4*>(&sg[r][at.c]) = gy;
      }
    }
    f32x4 start[2];  // states in front of the halves
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        start[i][s] = SPLIT && !g.first ? fmaf(exp2_fast(since[i] * A2[s]), enter[s], held[i][s]) : held[i][s];
    if (kAhead) {
      nB.arrived();
      nC.arrived();
    }
    u.move(-1);
    dt.move(-1);
    dy.move(-1);
    if (GATE) z.move(-1);
    nB.move(-1);
    nC.move(-1);
    if (tile > 0) fetch(tile - 1);
    __syncthreads();
    f32x4 dAt = zero4();
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      const int t0 = half * kHalf;
      if (!kFull && t0 >= n) continue;
      // Rows behind the segment are read at its last row and count as 0.
      const auto load = [&](Group<T, R>& to, const T* rows, long long stride, int q) {
        if (kFull) {
          to.load(rows + (t0 + q * R) * stride, stride);
        } else {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int t = t0 + q * R + i;
            to.r[i] = uniform4(rows + min(t, n - 1) * stride);
            if (t >= n) to.r[i] = Uniform4<T>{};
          }
        }
      };
      float h[kHalf + 1][4], decay[kHalf][4];  // states in front of the tokens and behind the last
      float lB[kHalf], lC[kHalf];
#pragma unroll
      for (int s = 0; s < 4; ++s) h[0][s] = start[half][s];
      const auto ahead = [&](int t, f32x4 b, float2 x) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          decay[t][s] = exp2_fast(x.x * A2[s]);
          h[t + 1][s] = fmaf(decay[t][s], h[t][s], x.y * b[s]);
        }
      };
      const auto back = [&](int t, f32x4 b, f32x4 cc, float2 x, float gy) {
        f32x4 vB, vC;
        float px = 0.f, pa = 0.f, py = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          G[s] = fmaf(cc[s], gy, G[s]);
          vC[s] = h[t + 1][s] * gy;
          vB[s] = G[s] * x.y;
          px = fmaf(G[s], b[s], px);
          if (GATE) py = fmaf(h[t + 1][s], cc[s], py);
          G[s] *= decay[t][s];
          const float thr = G[s] * h[t][s];
          pa = fmaf(thr, A2[s], pa);
          dAt[s] = fmaf(thr, x.x, dAt[s]);
        }
        lB[t] = rows_sum(vB);
        lC[t] = rows_sum(vC);
        sdx[w][t0 + t][lane] = px;
        sda[w][t0 + t][lane] = pa;
        if (GATE) sy[w][t0 + t][lane] = py;
      };
      Group<T, R> gb[2], gc[2];
      float2 x[2][R];
      float gy[2][R];
      load(gb[0], Bt, a.Bm.sl, 0);
#pragma unroll
      for (int i = 0; i < R; ++i) x[0][i] = sx[t0 + i][lane];
      wait_reads();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int now = q & 1, next = now ^ 1;
        if (q + 1 < Q) {
          load(gb[next], Bt, a.Bm.sl, q + 1);
#pragma unroll
          for (int i = 0; i < R; ++i) x[next][i] = sx[t0 + (q + 1) * R + i][lane];
        } else {
          // The last group is the first of the way back.
          load(gc[now], Ct, a.Cm.sl, q);
#pragma unroll
          for (int i = 0; i < R; ++i) gy[now][i] = sg[t0 + q * R + i][lane];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < R; ++i) ahead(q * R + i, wide(gb[now].r[i]), x[now][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = Q - 1; q >= 0; --q) {
        const int now = q & 1, next = now ^ 1;
        if (q > 0) {
          load(gb[next], Bt, a.Bm.sl, q - 1);
          load(gc[next], Ct, a.Cm.sl, q - 1);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            x[next][i] = sx[t0 + (q - 1) * R + i][lane];
            gy[next][i] = sg[t0 + (q - 1) * R + i][lane];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) back(q * R + i, wide(gb[now].r[i]), wide(gc[now].r[i]), x[now][i], gy[now][i]);
        // (Formed here, or their terms are kept in registers to the end of the tile.)
#pragma unroll
        for (int s = 0; s < 4; ++s) asm volatile("" : "+v"(dAt[s]));
        __builtin_amdgcn_sched_barrier(0);
      }
      const float tB = lanes_sum(lB, lane), tC = lanes_sum(lC, lane);
      const int t = t0 + (lane & 7);
      if ((lane & 8) == 0 && (kFull || t < n)) {
        const int o = t * N + 4 * w + (lane >> 4);
        dB[o] = tB;
        dC[o] = tC;
      }
    }
    dA += dAt;
    __syncthreads();
    if (at.in_tile()) {
#pragma unroll
      for (int p = 0; p < At::kPasses; ++p) {
        const int r = at.row(p);
        const f32x4 uu = wide(ru[p]);
        f32x4 dx = zero4(), da = zero4(), yv = skip * uu;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          dx += get4(&sdx[i][r][at.c]);
          da += get4(&sda[i][r][at.c]);
          if (GATE) yv += get4(&sy[i][r][at.c]);
        }
        if (!has || (!kFull && r >= n)) continue;
        const f32x4 p0 = get4(&sx[r][at.c].x), p1 = get4(&sx[r][at.c + 2].x), gg = get4(&sg[r][at.c]);
        const f32x4 d{p0[0], p0[2], p1[0], p1[2]};
        f32x4 draw = da * kLn2 + dx * uu;
        if (a.softplus) draw *= sigmoid4(wide(rd[p]) + bias);
        const uint32_t o = offset_of<T>(r, a.D, c);
        put4(const_cast<T*>(at_bytes(du, o)), dx * d + skip * gg);
        put4(const_cast<T*>(at_bytes(ddt, o)), draw);
        dskip += gg * uu;
        dbias += draw;
        if (GATE) {
          const f32x4 zz = wide(rz[p]), sig = sigmoid4(zz);
          put4(const_cast<T*>(at_bytes(dz, o)), wide(ry[p]) * yv * (sig + zz * sig * (1.f - sig)));
        }
      }
    }
    Bt -= kTile * a.Bm.sl;
    Ct -= kTile * a.Cm.sl;
    du -= kTile * (size_t)a.D;
    ddt -= kTile * (size_t)a.D;
    if (GATE) dz -= kTile * (size_t)a.D;
    dB -= kTile * N;
    dC -= kTile * N;
    // (What a thread reads of sx and sg here it wrote itself, so the next tile's may follow.)
  };
  int tile = tiles - 1;
  if (g.n % kTile) one(tile--, Flag<false>{});
  for (; tile >= 0; --tile) one(tile, Flag<true>{});
  if (on) {
    *reinterpret_cast<f32x4*>(dA_to) = dA;
    if (g.first && a.dh0) *reinterpret_cast<f32x4*>(a.dh0 + (size_t)g.seq * state + place) = G;
  }
  // The rows' parts of D's and the bias's gradients.
  constexpr int kSum = At::kRows < kTile ? At::kRows : kTile;
  __syncthreads();
  if (at.r < kSum) {
    *reinterpret_cast<f32x4*>(&sg[at.r][at.c]) = dskip;
    *reinterpret_cast<f32x4*>(&sdx[0][at.r][at.c]) = dbias;
  }
  __syncthreads();
  if (on && w == 0) {
    float s0 = 0.f, s1 = 0.f;
    for (int r = 0; r < kSum; ++r) s0 += sg[r][lane], s1 += sdx[0][r][lane];
    dvec[ch] = s0;
    dvec[a.D + ch] = s1;
  }
}

// ---- adding up parts -------------------------------------------------------------------------------

// blockIdx.y = 0, 1: dB, dC over the blocks of channels, 4 values per thread.
template <typename T>
__global__ __launch_bounds__(256) void channels_kernel(const float* parts, long long values, int blocks_d, T* dB, T* dC) {
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= values) return;
  const float* p = parts + (blockIdx.y ? values * blocks_d : 0) + i;
  f32x4 s = zero4();
#pragma unroll 8
  for (int k = 0; k < blocks_d; ++k) s += get4(p + (size_t)k * values);
  put4((blockIdx.y ? dC : dB) + i, s);
}

// dA, then D's and the bias's gradients, over the segments: 16 columns of
// `dA` [seg][state] and `dvec` [seg][2 D] per workgroup.
static __global__ __launch_bounds__(256) void segments_kernel(const int* used, int segments, int state, int D, const float* dA,
                                                              const float* dvec, float* out_A, float* out_skip, float* out_bias) {
  __shared__ double red[16][17];
  const int n = used ? *used : segments;
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  int e = blockIdx.x * 16 + c;
  const bool vec = e >= state;  // (both are multiples of 16)
  const float* p = vec ? dvec : dA;
  const size_t stride = vec ? 2 * (size_t)D : state;
  if (vec) e -= state;
  double s = 0.0;
#pragma unroll 8
  for (int i = r; i < n; i += 16) s += (double)p[(size_t)i * stride + e];
  red[r][c] = s;
  __syncthreads();
  if (r) return;
  for (int i = 1; i < 16; ++i) s += red[i][c];
  float* const to = !vec ? out_A + e : e < D ? (out_skip ? out_skip + e : nullptr) : (out_bias ? out_bias + e - D : nullptr);
  if (to) *to = (float)s;
}

// ---- launches --------------------------------------------------------------------------------------

// 512 workgroups need no cut here either (forward + backward of 16 x 2048 tokens of 2048
// channels, 512 of them: 840 us uncut, 906 cut; 16 x 64 of 1024, 256 of them: 41 uncut and 43).
// With one, 4096: 2 x 8192 tokens of 4096 channels take 1873 us with 1024, 1790 with 2048, 1771 with
// 4096, 1811 with 8192.  Pieces: 512 tokens of 768 channels, 46 us in pieces of 64, 40 of 48, 35
// of 32, 37 of 16; 128 of them 43, 37, 31 and 26 (62 uncut).
Sizes backward_sizes(int B, int L, int D, bool packed, int n_seq) {
  return sizes_of(packed, B, L, n_seq, D, {512, 4096, 512, 32, 4});
}
static size_t up(size_t n) { return (n + 3) / 4 * 4; }  // floats, to 16 bytes

// Places the parts in a workspace; returns its size in bytes (ws may be null).
static size_t place(int B, int L, int D, int N, bool packed, int n_seq, const Sizes& s, void* ws, BwdSpace* out) {
  const size_t table = table_bytes(packed, n_seq, s), state = (size_t)D * N, tokens = (size_t)B * L;
  const size_t tiles = 2 * (tokens / kTile + s.segments + 1), seg = s.segments;
  float* p = reinterpret_cast<float*>(static_cast<char*>(ws) + table);
  size_t at = 0;
  const auto take = [&](size_t n) {
    float* r = p + at;
    at += up(n);
    return r;
  };
  out->tiles = take(tiles * state);
  out->before = take(s.split ? tiles * D : 0);
  out->ahead = take(s.split ? seg * state : 0);
  out->back = take(s.split ? seg * state : 0);
  out->logs = take(s.split ? seg * D : 0);
  out->dBC = take(2 * (size_t)channel_blocks(D) * tokens * N);
  out->dA = take(seg * state);
  out->dvec = take(seg * 2 * D);
  return table + at * sizeof(float);
}

template <int NW, typename T, bool GATE>
static hipError_t backward(const ScanArgs& a) {
  const Sizes s = backward_sizes(a.B, a.L, a.D, a.cu, a.n_seq);
  const int blocks_d = (int)channel_blocks(a.D);
  BwdSpace ws;
  place(a.B, a.L, a.D, a.N, a.cu, a.n_seq, s, a.workspace, &ws);
  Plan p;
  prof_mark(kSlotSelectiveScanBwd, false, a.stream);
  hipError_t e = make_plan(a.cu, a.n_seq, a.L, s, a.workspace, a.stream, &p);
  const dim3 grid((unsigned)(s.segments * blocks_d)), block(64 * NW);
  if (e == hipSuccess) {
    if (s.split) {
      hipLaunchKernelGGL((sums_kernel<NW, T, GATE, true>), dim3(grid.x, 2), block, 0, a.stream, a, p, blocks_d, ws);
      e = hipGetLastError();
      if (e == hipSuccess) e = combine(p, a.n_seq, a.D, a.N, a.A, ws.logs, a.h0, ws.ahead, ws.back, a.stream);
      if (e == hipSuccess) {
        hipLaunchKernelGGL((back_kernel<NW, T, GATE, true>), grid, block, 0, a.stream, a, p, blocks_d, ws);
        e = hipGetLastError();
      }
    } else {
      hipLaunchKernelGGL((sums_kernel<NW, T, GATE, false>), grid, block, 0, a.stream, a, p, blocks_d, ws);
      e = hipGetLastError();
      if (e == hipSuccess) {
        hipLaunchKernelGGL((back_kernel<NW, T, GATE, false>), grid, block, 0, a.stream, a, p, blocks_d, ws);
        e = hipGetLastError();
      }
    }
  }
  const long long values = (long long)a.B * a.L * a.N;
  if (e == hipSuccess && values > 0) {
    hipLaunchKernelGGL(channels_kernel<T>, dim3((unsigned)((values / 4 + 255) / 256), 2), dim3(256), 0, a.stream, ws.dBC,
                       values, blocks_d, static_cast<T*>(a.dB), static_cast<T*>(a.dC));
    e = hipGetLastError();
  }
  if (e == hipSuccess) {
    hipLaunchKernelGGL(segments_kernel, dim3((unsigned)((a.D * a.N + 2 * a.D) / 16)), dim3(256), 0, a.stream, p.used,
                       (int)s.segments, a.D * a.N, a.D, ws.dA, ws.dvec, a.dA, a.dskip, a.dbias);
    e = hipGetLastError();
  }
  prof_mark(kSlotSelectiveScanBwd, true, a.stream);
  return e;
}

template <int NW>
static hipError_t backward_t(const ScanArgs& a) {
  if (a.dtype == 1) return a.z.p ? backward<NW, bf16, true>(a) : backward<NW, bf16, false>(a);
  return a.z.p ? backward<NW, float, true>(a) : backward<NW, float, false>(a);
}

}  // namespace ssm

size_t selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, bool packed, int n_seq) {
  ssm::BwdSpace ws;
  return ssm::place(B, L, D, N, packed, n_seq, ssm::backward_sizes(B, L, D, packed, n_seq), nullptr, &ws);
}

hipError_t launch_selective_scan_bwd(const ScanArgs& a) {
  return a.N == 8 ? ssm::backward_t<2>(a) : a.N == 16 ? ssm::backward_t<4>(a) : ssm::backward_t<8>(a);
}

}  // namespace dn
