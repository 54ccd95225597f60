// dn_qk_norm_rope.hip -- per-head norm of q and k and rotation by position in
// one pass, and its gradient.
//
// For every row x of d (one head of one token):
//     n = x / sqrt(mean(x^2) + eps) o w        (norm = 0: n = x o w)
//     (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = p inv_freq[j],
// for the pairs j of the first d_rot elements, (j, j + d_rot / 2) or, when
// interleaved, (2 j, 2 j + 1); p is the token's position on the axis whose
// section holds j.  With dy the gradient of the result, rotated back by -t to
// dn, and r = 1 / sqrt(mean(x^2) + eps):
//     dw = sum over rows of dn o x r,
//     dx = r (u - (x r) mean(u o x r)),   u = dn o w.
//
// Bound by HBM (2 rows moved per row forward, 3 backward).
//
// Lanes.  A row is d / 8 adjacent lanes, 8 elements each in two pieces of 4:
// for the first d_rot / 8 lanes the pieces are the two halves of 4 pairs, so
// a pair never leaves its lane whatever the pairing and d_rot; the others
// hold elements behind d_rot.  A group of lanes keeps its token and walks
// over heads, so a token's 4 angles per lane are formed once for all of them.
//
// Heads.  A workgroup takes 4 of them at most, and the workgroups that follow
// it the next ones of the same tokens: together they read adjacent parts of a
// fused projection's rows at one time.  32 + 32 heads of 128 bf16 elements, 65536
// tokens out of rows of 3 x 4096: 392 us (5.5 TB/s); with 2 heads 475, with 6
// 402, 8 429, 16 448, all 64 471 (few workgroups, each far from the others'
// rows).  The gradient at 16384 tokens: 179 us (4.5 TB/s) against 186 with all
// heads, at 2048 tokens of 12 + 12 heads of 64 fp32 elements 15 against 31 (few
// tokens alone do not fill the card).
//
// Angles.  p inv_freq reaches millions of turns; it is taken in turns in
// fp64, its whole turns dropped there, and only the rest (below half a turn)
// goes to fp32 sine and cosine.

#include "dn_common.h"
#include "dn_launch.h"
#include "dn_mfma.h"

namespace dn {
namespace qkr {

constexpr int NT = 256;

// Everything a lane needs to know about its place in a row.
struct Place {
  int o0, o1;   // first elements of its two pieces
  int pair;     // first of its 4 pairs
  bool turns;   // whether its elements rotate
};
__device__ __forceinline__ Place place_of(int lane, int d_rot, bool interleaved) {
  Place p;
  p.turns = lane < d_rot / 8;
  p.pair = 4 * lane;
  const bool halves = p.turns && !interleaved;
  p.o0 = halves ? 4 * lane : 8 * lane;
  p.o1 = p.o0 + (halves ? d_rot / 2 : 4);
  return p;
}

template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p);
template <>
__device__ __forceinline__ f32x4 load4<float>(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
template <>
__device__ __forceinline__ f32x4 load4<bf16>(const bf16* p) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  return f32x4{__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u),
               __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u)};
}
template <typename T>
__device__ __forceinline__ void store4(T* p, f32x4 x);
template <>
__device__ __forceinline__ void store4<float>(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
template <>
__device__ __forceinline__ void store4<bf16>(bf16* p, f32x4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// cos and sin of the lane's 4 angles.
__device__ __forceinline__ void angles(const QkNormRopeArgs& a, const Place& p, int b, int l, f32x4& c, f32x4& s) {
  c = f32x4{1.f, 1.f, 1.f, 1.f};
  s = zero4();
  if (!p.turns) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = p.pair + i;
    int axis = 0;
#pragma unroll
    for (int x = 0; x + 1 < kMaxAxes; ++x) axis += j >= a.ends[x];
    const int pos = a.positions[((size_t)axis * a.B + b) * a.L + l];
    const double turns = (double)pos * ((double)a.inv_freq[j] * 0.15915494309189533577);
    const float x = 2.f * (float)(turns - rint(turns));
    float sn, cs;
    sincospif(x, &sn, &cs);
    s[i] = sn;
    c[i] = cs;
  }
}

// Rotates the lane's 4 pairs by (c, s): halves hold (x0[i], x1[i]), interleaved
// pieces hold the pairs themselves.
__device__ __forceinline__ void rotate(f32x4& x0, f32x4& x1, f32x4 c, f32x4 s, bool interleaved) {
  if (interleaved) {
    const f32x4 a = x0, b = x1;
    x0 = f32x4{a[0] * c[0] - a[1] * s[0], a[0] * s[0] + a[1] * c[0], a[2] * c[1] - a[3] * s[1], a[2] * s[1] + a[3] * c[1]};
    x1 = f32x4{b[0] * c[2] - b[1] * s[2], b[0] * s[2] + b[1] * c[2], b[2] * c[3] - b[3] * s[3], b[2] * s[3] + b[3] * c[3]};
  } else {
    const f32x4 a = x0, b = x1;
    x0 = a * c - b * s;
    x1 = a * s + b * c;
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]); }

// A workgroup takes NT / LPR tokens and `hpb` heads, counted over q's heads
// and then k's.
template <int D, typename T>
__global__ __launch_bounds__(NT) void forward_kernel(QkNormRopeArgs a, long long tokens, int hpb, int blocks_h) {
  constexpr int LPR = D / 8, TPB = NT / LPR;
  const int lane = threadIdx.x % LPR;
  const int hb = blockIdx.x % blocks_h;
  const long long tok = (long long)(blockIdx.x / blocks_h) * TPB + threadIdx.x / LPR;
  const bool on = tok < tokens;
  const int b = on ? (int)(tok / a.L) : 0, l = on ? (int)(tok % a.L) : 0;
  const Place p = place_of(lane, a.d_rot, a.interleaved);
  f32x4 c, s;
  angles(a, p, b, l, c, s);
  const int h0 = hb * hpb, h1 = min(h0 + hpb, a.H[0] + a.H[1]);
  for (int part = 0; part < 2; ++part) {
    const int first = part ? max(h0 - a.H[0], 0) : h0, end = part ? h1 - a.H[0] : min(h1, a.H[0]);
    if (first >= end) continue;
    f32x4 w0{1.f, 1.f, 1.f, 1.f}, w1 = w0;
    if (a.weight[part]) w0 = load4(a.weight[part] + p.o0), w1 = load4(a.weight[part] + p.o1);
    const T* x = static_cast<const T*>(a.x[part].p) + (long long)b * a.x[part].sb + (long long)l * a.x[part].sl;
    T* y = static_cast<T*>(a.y[part]) + ((size_t)b * a.H[part] * a.L + l) * D;
    for (int h = first; h < end; ++h) {
      const T* xr = x + (long long)h * a.x[part].sh;
      f32x4 x0 = load4(xr + p.o0), x1 = load4(xr + p.o1);
      if (a.norm) {
        const float ss = row_sum<LPR>(dot4(x0, x0) + dot4(x1, x1));
        const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
        x0 *= r;
        x1 *= r;
      }
      x0 *= w0;
      x1 *= w1;
      rotate(x0, x1, c, s, a.interleaved);
      if (on) {
        T* yr = y + (size_t)h * a.L * D;
        store4(yr + p.o0, x0);
        store4(yr + p.o1, x1);
      }
    }
  }
}

// The gradient.  Workgroups take a block of heads and walk over blocks of
// tokens; each leaves one partial row of dw for q and one for k.
template <int D, typename T>
__global__ __launch_bounds__(NT) void backward_kernel(QkNormRopeArgs a, long long tokens, int hpb, int blocks_h, float* partial) {
  constexpr int LPR = D / 8, TPB = NT / LPR;
  __shared__ float red[TPB][D];
  const int lane = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const Place p = place_of(lane, a.d_rot, a.interleaved);
  f32x4 acc[2][2] = {{zero4(), zero4()}, {zero4(), zero4()}};
  const int h0 = blockIdx.x % blocks_h * hpb, h1 = min(h0 + hpb, a.H[0] + a.H[1]);
  const long long step = gridDim.x / blocks_h;  // a whole number
  for (long long t0 = blockIdx.x / blocks_h * TPB; t0 < tokens; t0 += step * TPB) {
    const long long tok = t0 + row;
    const bool on = tok < tokens;
    const int b = on ? (int)(tok / a.L) : 0, l = on ? (int)(tok % a.L) : 0;
    f32x4 c, s;
    angles(a, p, b, l, c, s);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int first = part ? max(h0 - a.H[0], 0) : h0, end = part ? h1 - a.H[0] : min(h1, a.H[0]);
      if (first >= end) continue;
      f32x4 w0{1.f, 1.f, 1.f, 1.f}, w1 = w0;
      if (a.weight[part]) w0 = load4(a.weight[part] + p.o0), w1 = load4(a.weight[part] + p.o1);
      const T* x = static_cast<const T*>(a.x[part].p) + (long long)b * a.x[part].sb + (long long)l * a.x[part].sl;
      T* dx = static_cast<T*>(const_cast<void*>(a.dx[part].p)) + (long long)b * a.dx[part].sb + (long long)l * a.dx[part].sl;
      const T* dy = static_cast<const T*>(a.y[part]) + ((size_t)b * a.H[part] * a.L + l) * D;
      for (int h = first; h < end; ++h) {
        const T* xr = x + (long long)h * a.x[part].sh;
        const T* dr = dy + (size_t)h * a.L * D;
        f32x4 x0 = load4(xr + p.o0), x1 = load4(xr + p.o1);
        f32x4 d0 = load4(dr + p.o0), d1 = load4(dr + p.o1);
        rotate(d0, d1, c, -s, a.interleaved);
        float r = 1.f;
        if (a.norm) {
          const float ss = row_sum<LPR>(dot4(x0, x0) + dot4(x1, x1));
          r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
          x0 *= r;
          x1 *= r;
        }
        if (on) {
          acc[part][0] += d0 * x0;
          acc[part][1] += d1 * x1;
        }
        d0 *= w0;
        d1 *= w1;
        if (a.norm) {
          const float m = row_sum<LPR>(dot4(x0, d0) + dot4(x1, d1)) * (1.f / D);
          d0 = (d0 - x0 * m) * r;
          d1 = (d1 - x1 * m) * r;
        }
        if (on) {
          T* out = dx + (long long)h * a.dx[part].sh;
          store4(out + p.o0, d0);
          store4(out + p.o1, d1);
        }
      }
    }
  }
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    __syncthreads();
    *reinterpret_cast<f32x4*>(&red[row][p.o0]) = acc[part][0];
    *reinterpret_cast<f32x4*>(&red[row][p.o1]) = acc[part][1];
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += NT) {
      float sum = 0.f;
      for (int i = 0; i < TPB; ++i) sum += red[i][e];
      partial[((size_t)blockIdx.x * 2 + part) * D + e] = sum;
    }
  }
}

// dw of q (y = 0) and k (y = 1): the workgroups' partial rows added in order,
// 16 columns per workgroup.
static __global__ __launch_bounds__(NT) void weight_kernel(const float* partial, int n, int d, float* dq, float* dk) {
  __shared__ double red[16][17];
  float* out = blockIdx.y ? dk : dq;
  if (!out) return;
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  double sum = 0.0;
#pragma unroll 8
  for (int i = r; i < n; i += 16) sum += (double)partial[((size_t)i * 2 + blockIdx.y) * d + e];
  red[r][c] = sum;
  __syncthreads();
  if (r == 0) {
    for (int i = 1; i < 16; ++i) sum += red[i][c];
    out[e] = (float)sum;
  }
}

static long long token_blocks(long long tokens, int d) {
  const int tpb = NT / (d / 8);
  return (tokens + tpb - 1) / tpb;
}
// Heads per workgroup and blocks of heads, with `n` blocks of heads wanted at
// the least.
struct HeadSplit {
  int hpb, blocks;
};
static HeadSplit split_heads(int H, long long n) {
  if (n < (H + 3) / 4) n = (H + 3) / 4;
  if (n > H) n = H;
  const int hpb = (int)((H + n - 1) / n);
  return HeadSplit{hpb, (H + hpb - 1) / hpb};
}
// Workgroups of the backward: each leaves partial rows to add up, so about
// 1024 of them at most.
static int backward_blocks(long long tokens, int H, int d) {
  const int bh = split_heads(H, 1).blocks;
  const long long tb = token_blocks(tokens, d), most = bh < 1024 ? 1024 / bh : 1;
  return (int)(tb < most ? tb : most) * bh;
}

template <int D, typename T>
static hipError_t forward(const QkNormRopeArgs& a) {
  const long long tokens = (long long)a.B * a.L, tb = token_blocks(tokens, D);
  const int H = a.H[0] + a.H[1];
  // Fewer heads per workgroup, down to one, spread few tokens.
  const HeadSplit h = split_heads(H, (2048 + tb - 1) / tb);
  prof_mark(kSlotQkNormRope, false, a.stream);
  hipLaunchKernelGGL((forward_kernel<D, T>), dim3((unsigned)(tb * h.blocks)), dim3(NT), 0, a.stream, a, tokens, h.hpb, h.blocks);
  hipError_t e = hipGetLastError();
  prof_mark(kSlotQkNormRope, true, a.stream);
  return e;
}

template <int D, typename T>
static hipError_t backward(const QkNormRopeArgs& a) {
  const long long tokens = (long long)a.B * a.L;
  const int H = a.H[0] + a.H[1], n = backward_blocks(tokens, H, D);
  const HeadSplit h = split_heads(H, 1);
  float* partial = static_cast<float*>(a.workspace);
  prof_mark(kSlotQkNormRopeBwd, false, a.stream);
  hipError_t e = hipSuccess;
  if (n > 0) {
    hipLaunchKernelGGL((backward_kernel<D, T>), dim3((unsigned)n), dim3(NT), 0, a.stream, a, tokens, h.hpb, h.blocks, partial);
    e = hipGetLastError();
  }
  if (e == hipSuccess && (a.dw[0] || a.dw[1])) {
    hipLaunchKernelGGL(weight_kernel, dim3(D / 16, 2), dim3(NT), 0, a.stream, partial, n, D, a.dw[0], a.dw[1]);
    e = hipGetLastError();
  }
  prof_mark(kSlotQkNormRopeBwd, true, a.stream);
  return e;
}

}  // namespace qkr

// Most tokens one launch takes.  (Few tokens, over which more blocks of heads are
// spread, stay far below the launch's limit.)
long long qk_norm_rope_max_tokens(int heads, int d) {
  return max_blocks(qkr::NT) / qkr::split_heads(heads, 1).blocks * (qkr::NT / (d / 8));
}

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a) {
  if (a.dtype == 1) return a.d == 64 ? qkr::forward<64, bf16>(a) : qkr::forward<128, bf16>(a);
  return a.d == 64 ? qkr::forward<64, float>(a) : qkr::forward<128, float>(a);
}

size_t qk_norm_rope_bwd_workspace_bytes(int B, int heads, int L, int d) {
  return (size_t)qkr::backward_blocks((long long)B * L, heads, d) * 2 * d * sizeof(float);
}

hipError_t launch_qk_norm_rope_bwd(const QkNormRopeArgs& a) {
  if (a.dtype == 1) return a.d == 64 ? qkr::backward<64, bf16>(a) : qkr::backward<128, bf16>(a);
  return a.d == 64 ? qkr::backward<64, float>(a) : qkr::backward<128, float>(a);
}

}  // namespace dn
