// dn_add_norm.hip -- root-mean-square norm of every row with the residual's
// addition on gfx950, y in the inputs' type or in 8 bits, and the gradient.
//
//     total = x + residual (rounded to the residual's type, what the next layer adds to)
//     y = total r o w,   r = 1 / sqrt(mean(total^2) + eps)
//     8 bits: scale = max |y| / 448 of the row, e4m3(y / scale)
// and, with dt the gradient of total from elsewhere and v = dy o w,
//     d = dt + r (v - n mean(n o v)),  n = total r     (the gradient of x and of the residual)
//     dw = sum over rows of dy o n.
// The norm is taken of the rounded total: it is what the backward has in hand.
//
// Bound by HBM.  A row's elements stay in the registers of a group of LPR lanes
// (pieces of 8) between the sum of squares and the result, so each is read once: 65536 rows
// of 4096 bf16 elements into 8 bits 330 us (5.7 TB/s), 16385 of 2072 with an fp32 stream
// 74 us (5.5 TB/s) and their gradient 113 (4.8); fp32, 65536 x 4096, 764 and 807 us (5.6 and
// 5.3).  The gradient is far from that at both ends of the widths: above 16384 elements its rows
// do not fit 128 registers a lane (2048 x 20480 bf16 260 us, 1.3 TB/s, 16384 70), and narrow rows
// leave a part of dw per group of lanes (65536 x 16: 59 us, 48 of them the parts' sum).

#include "dn_launch.h"
#include "dn_vec.h"

namespace dn {
namespace norm {

constexpr float kE4m3Max = 448.f;

struct Eight { f32x4 a, b; };
template <typename T>
__device__ __forceinline__ Eight load8(const T* p) {
  struct alignas(8 * sizeof(T)) Two { Raw4<T> a, b; };
  const Two t = *reinterpret_cast<const Two*>(p);
  return {wide(t.a), wide(t.b)};
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Eight& x) {
  struct alignas(8 * sizeof(T)) Two { Raw4<T> a, b; };
  *reinterpret_cast<Two*>(p) = Two{narrow<T>(x.a), narrow<T>(x.b)};
}
template <typename T>
__device__ __forceinline__ Eight rounded(const Eight& x) { return {wide(narrow<T>(x.a)), wide(narrow<T>(x.b))}; }
__device__ __forceinline__ float dot8(const Eight& x, const Eight& y) {
  const f32x4 s = x.a * y.a + x.b * y.b;
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ float at(const Eight& x, int k) { return k < 4 ? x.a[k] : x.b[k - 4]; }

struct Sum { static __device__ __forceinline__ float of(float a, float b) { return a + b; } };
// (A NaN stays one: the other side of a comparison with it is never taken.)
struct Max { static __device__ __forceinline__ double of(double a, double b) { return a > b || a != a ? a : b; } };

// A value as a sum of two; a product of two fp32 is one exactly.
struct Pair { float hi, lo; };
__device__ __forceinline__ Pair product(float a, float b) {
  const float p = a * b;
  return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ Pair larger(Pair a, Pair b) {
  const bool second = b.hi > a.hi || (b.hi == a.hi && b.lo > a.lo);
  return {second ? b.hi : a.hi, second ? b.lo : a.lo};
}

// Over the LPR lanes of a row, the same for all of them.  `red` has a place for
// every wave; rows of more than a wave use it and every thread of the workgroup calls this.
template <int LPR, typename Op, typename F>
__device__ __forceinline__ F row_all(F x, F* red) {
#pragma unroll
  for (int off = (LPR < 64 ? LPR : 64) / 2; off > 0; off >>= 1) x = Op::of(x, __shfl_xor(x, off, 64));
  if (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x = Op::of(x, red[i]);
    __syncthreads();
  }
  return x;
}

template <int LPR> constexpr int threads() { return LPR > 256 ? LPR : 256; }

template <int LPR, int P, typename T, typename R, bool E4M3>
__global__ __launch_bounds__(threads<LPR>()) void forward_kernel(AddNormArgs a) {
  constexpr int NT = threads<LPR>(), RPB = NT / LPR;
  __shared__ float red[NT / 64];
  __shared__ double red8[E4M3 ? NT / 64 : 1];
  const int lane = threadIdx.x % LPR;
  const long long row = (long long)blockIdx.x * RPB + threadIdx.x / LPR;
  const bool on = row < a.rows;
  const size_t base = (size_t)(on ? row : 0) * a.D;
  const T* const x = static_cast<const T*>(a.x) + base;
  const R* const res = a.residual ? static_cast<const R*>(a.residual) + base : nullptr;
  R* const total = a.residual ? static_cast<R*>(a.total) + base : nullptr;
  const int pieces = a.D / 8;
  Eight v[P], w[P];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = lane + i * LPR;
    v[i] = {zero4(), zero4()};
    w[i] = {f32x4{1.f, 1.f, 1.f, 1.f}, f32x4{1.f, 1.f, 1.f, 1.f}};
    if (p >= pieces) continue;
    v[i] = load8(x + p * 8);
    if (a.weight) w[i] = load8(a.weight + p * 8);
    if (res) {
      const Eight r = load8(res + p * 8);
      v[i].a += r.a;
      v[i].b += r.b;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = lane + i * LPR;
    if (res) {
      v[i] = rounded<R>(v[i]);
      if (on && p < pieces) store8(total + p * 8, v[i]);
    }
    ss += dot8(v[i], v[i]);
  }
  ss = row_all<LPR, Sum>(ss, red);
  const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
  if (!E4M3) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = lane + i * LPR;
      if (p >= pieces || !on) continue;
      v[i].a = v[i].a * r * w[i].a;
      v[i].b = v[i].b * r * w[i].b;
      store8(static_cast<T*>(a.y) + base + p * 8, v[i]);
    }
    return;
  }
  // r is in every y of the row and in the scale, so the 8-bit values do not depend on it:
  // y / scale = (total w) (448 / max |total w|).  With products and quotient held as two fp32
  // each, the quotient is rounded once to fp32 (2^-24) and then to e4m3, as one formed in 64 bits
  // and converted is; in single fp32 a few values in a million are a step off, for the same
  // time (330 us for 65536 rows of 4096; fp64 359).  Of r the power of
  // two is taken out first, which is exact and keeps the products in range.
  const float r2 = __uint_as_float(__float_as_uint(r) & 0x7f800000u);
  Pair top{0.f, 0.f};
  float odd = 0.f;  // NaN once a product is not finite
#pragma unroll
  for (int i = 0; i < P; ++i) {
    v[i].a *= r2;
    v[i].b *= r2;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Pair x = product(at(v[i], k), at(w[i], k));
      odd = fmaf(x.hi, 0.f, odd);
      top = larger(top, x.hi < 0.f ? Pair{-x.hi, -x.lo} : x);
    }
  }
  const double most = row_all<LPR, Max>(odd == 0.f ? (double)top.hi + top.lo : (double)odd, red8);
  float scale = (float)(most * (r / r2) * (1.0 / kE4m3Max));
  double by = kE4m3Max / most;
  if (most == 0.0) {
    scale = 1.f;
    by = 0.0;
  } else if (scale < 1.17549435e-38f) {  // (not below the smallest normal number)
    scale = 1.17549435e-38f;
    by = (double)(r / r2) / scale;
  }
  if (on && lane == 0) a.scale[row] = scale;
  // (A row whose y are all below 2^-90 keeps the quotient in fp64: it is past fp32's range.)
  const bool small = by > 0x1p99;
  const float by_hi = (float)by, by_lo = (float)(by - by_hi);
  unsigned char* const y = static_cast<unsigned char*>(a.y) + base;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = lane + i * LPR;
    if (p >= pieces || !on) continue;
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Pair x = product(at(v[i], k), at(w[i], k));
      const float t = small ? (float)(((double)x.hi + x.lo) * by) : fmaf(x.hi, by_hi, fmaf(x.hi, by_lo, x.lo * by_hi));
      // The largest may come out a little above 448; a NaN stays one.
      q[k] = t > kE4m3Max ? kE4m3Max : t < -kE4m3Max ? -kE4m3Max : t;
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    *reinterpret_cast<int2*>(y + p * 8) = make_int2(lo, hi);
  }
}

// Workgroups walk over rows; each group of LPR lanes leaves a partial row of dw.  (1024 lanes of 4
// pieces: 97 to 110 of w, dw, n and g in scratch memory, 264 to 280 bytes a lane.)
template <int LPR, int P, typename T, typename R>
__global__ __launch_bounds__(threads<LPR>()) void backward_kernel(AddNormArgs a, float* parts) {
  constexpr int NT = threads<LPR>(), RPB = NT / LPR;
  __shared__ float red[NT / 64];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int pieces = a.D / 8;
  Eight w[P], dw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = lane + i * LPR;
    w[i] = {f32x4{1.f, 1.f, 1.f, 1.f}, f32x4{1.f, 1.f, 1.f, 1.f}};
    if (a.weight && p < pieces) w[i] = load8(a.weight + p * 8);
    dw[i] = {zero4(), zero4()};
  }
  for (long long first = (long long)blockIdx.x * RPB; first < a.rows; first += (long long)gridDim.x * RPB) {
    const long long row = first + sub;
    const bool on = row < a.rows;
    const size_t base = (size_t)(on ? row : 0) * a.D;
    Eight n[P], g[P];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = lane + i * LPR;
      n[i] = g[i] = {zero4(), zero4()};
      if (p >= pieces || !on) continue;
      n[i] = load8(static_cast<const R*>(a.total) + base + p * 8);
      g[i] = load8(static_cast<const T*>(a.dy) + base + p * 8);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) ss += dot8(n[i], n[i]);
    ss = row_all<LPR, Sum>(ss, red);
    const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!on) continue;
      n[i].a *= r;
      n[i].b *= r;
      dw[i].a += g[i].a * n[i].a;
      dw[i].b += g[i].b * n[i].b;
      g[i].a *= w[i].a;
      g[i].b *= w[i].b;
      m += dot8(n[i], g[i]);
    }
    m = row_all<LPR, Sum>(m, red) / (float)a.D;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = lane + i * LPR;
      if (p >= pieces || !on) continue;
      Eight d{(g[i].a - n[i].a * m) * r, (g[i].b - n[i].b * m) * r};
      if (a.dtotal) {
        const Eight t = load8(static_cast<const R*>(a.dtotal) + base + p * 8);
        d.a += t.a;
        d.b += t.b;
      }
      store8(static_cast<T*>(a.dx) + base + p * 8, d);
      if (a.dresidual) store8(static_cast<R*>(a.dresidual) + base + p * 8, d);
    }
  }
  if (!a.dweight) return;
  // One partial row per group of lanes.
  float* const to = parts + ((size_t)blockIdx.x * RPB + sub) * a.D;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = lane + i * LPR;
    if (p < pieces) store8(to + p * 8, dw[i]);
  }
}

// Partial rows added in order, 16 columns per workgroup.
static __global__ __launch_bounds__(256) void weight_kernel(const float* parts, int n, int D, float* out) {
  __shared__ double red[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  double s = 0.0;
  if (e < D) {
#pragma unroll 8
    for (int i = r; i < n; i += 16) s += (double)parts[(size_t)i * D + e];
  }
  red[r][c] = s;
  __syncthreads();
  if (r || e >= D) return;
  for (int i = 1; i < 16; ++i) s += red[i][c];
  out[e] = (float)s;
}

// Lanes per row and pieces per lane for rows of D.
struct Shape {
  int lpr, p;
};
static Shape shape_of(int D) {
  const int pieces = D / 8;
  if (pieces <= 16) return {16, 1};
  if (pieces <= 64) return {64, 1};
  if (pieces <= 128) return {64, 2};
  if (pieces <= 256) return {64, 4};
  if (pieces <= 512) return {256, 2};
  if (pieces <= 1024) return {256, 4};
  if (pieces <= 2048) return {1024, 2};
  return {1024, 4};
}
constexpr int kMostD = 1024 * 4 * 8;
static int rows_per_block(const Shape& s) { return (s.lpr > 256 ? s.lpr : 256) / s.lpr; }
static int backward_blocks(int rows, int D) {
  const Shape s = shape_of(D);
  const int rpb = rows_per_block(s), blocks = (int)(((long long)rows + rpb - 1) / rpb);
  const int most = s.lpr > 256 ? 512 : 1024;
  return blocks < most ? blocks : most;
}

template <int LPR, int P, typename T, typename R>
static hipError_t forward(const AddNormArgs& a) {
  constexpr int NT = threads<LPR>(), RPB = NT / LPR;
  const unsigned n = (unsigned)(((long long)a.rows + RPB - 1) / RPB);
  prof_mark(kSlotAddNorm, false, a.stream);
  if (a.scale)
    hipLaunchKernelGGL((forward_kernel<LPR, P, T, R, true>), dim3(n), dim3(NT), 0, a.stream, a);
  else
    hipLaunchKernelGGL((forward_kernel<LPR, P, T, R, false>), dim3(n), dim3(NT), 0, a.stream, a);
  const hipError_t e = hipGetLastError();
  prof_mark(kSlotAddNorm, true, a.stream);
  return e;
}

template <int LPR, int P, typename T, typename R>
static hipError_t backward(const AddNormArgs& a) {
  constexpr int NT = threads<LPR>(), RPB = NT / LPR;
  const int n = backward_blocks(a.rows, a.D);
  float* const parts = static_cast<float*>(a.workspace);
  prof_mark(kSlotAddNormBwd, false, a.stream);
  hipError_t e = hipSuccess;
  if (n > 0) {
    hipLaunchKernelGGL((backward_kernel<LPR, P, T, R>), dim3(n), dim3(NT), 0, a.stream, a, parts);
    e = hipGetLastError();
  }
  if (e == hipSuccess && a.dweight) {
    hipLaunchKernelGGL(weight_kernel, dim3((unsigned)((a.D + 15) / 16)), dim3(256), 0, a.stream, parts, n * RPB, a.D, a.dweight);
    e = hipGetLastError();
  }
  prof_mark(kSlotAddNormBwd, true, a.stream);
  return e;
}

template <typename T, typename R, bool BACK>
static hipError_t by_shape(const AddNormArgs& a) {
  const Shape s = shape_of(a.D);
#define DN_NORM(L, P) \
  if (s.lpr == L && s.p == P) return BACK ? backward<L, P, T, R>(a) : forward<L, P, T, R>(a)
  DN_NORM(16, 1);
  DN_NORM(64, 1);
  DN_NORM(64, 2);
  DN_NORM(64, 4);
  DN_NORM(256, 2);
  DN_NORM(256, 4);
  DN_NORM(1024, 2);
#undef DN_NORM
  return BACK ? backward<1024, 4, T, R>(a) : forward<1024, 4, T, R>(a);
}
template <bool BACK>
static hipError_t by_type(const AddNormArgs& a) {
  if (a.dtype == 1) return a.residual_dtype == 1 ? by_shape<bf16, bf16, BACK>(a) : by_shape<bf16, float, BACK>(a);
  return by_shape<float, float, BACK>(a);
}

}  // namespace norm

bool add_norm_fits(int rows, int D) {
  const norm::Shape s = norm::shape_of(D);
  const long long rpb = norm::rows_per_block(s);
  return D <= norm::kMostD && (rows + rpb - 1) / rpb <= max_blocks(s.lpr > 256 ? s.lpr : 256);
}

hipError_t launch_add_norm(const AddNormArgs& a) { return norm::by_type<false>(a); }

size_t add_norm_bwd_workspace_bytes(int rows, int D) {
  return (size_t)norm::backward_blocks(rows, D) * norm::rows_per_block(norm::shape_of(D)) * D * sizeof(float);
}

hipError_t launch_add_norm_bwd(const AddNormArgs& a) { return norm::by_type<true>(a); }

}  // namespace dn
