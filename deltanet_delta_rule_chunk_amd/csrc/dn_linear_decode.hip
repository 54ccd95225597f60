// dn_linear_decode.hip -- one token of the gated linear recurrence on gfx950:
//     S <- e^g S + k^T v,   o = q S.
//
// Bound by HBM: per head it reads and writes the 4 d_k d_v byte state and
// does 4 d_k d_v flops on it.  Nothing in the step waits for a sum over the
// state: each element is read, updated, multiplied by its q and written.
//
// A workgroup takes a head; thread (rg, cg) of its 256 holds 4 adjacent columns
// of rows rg, rg + ROWG, ....  The partial sums of o meet in LDS.  All of a
// thread's loads are under way at once, and the new state is stored past the
// caches: 8192 heads of 128 x 128 (256 sequences of 32) take 160 us, 6.7 TB/s.
// Cutting a head's columns over 4 workgroups, for calls of few heads, made 32
// heads no faster (6.4 us against 6.3 between two events) and 4096 slower (102
// against 87).

#include "dn_common.h"
#include "dn_launch.h"

namespace dn {
namespace lin {

constexpr int kThreads = 256;

typedef float vf4 __attribute__((ext_vector_type(4)));

template <int DK, int DV, typename IT, typename OT>
__global__ __launch_bounds__(kThreads) void decode_kernel(const IT* __restrict__ q, const IT* __restrict__ k,
                                                     const IT* __restrict__ v, const float* __restrict__ g,
                                                     float* __restrict__ S, OT* __restrict__ o, int grp) {
  constexpr int COLG = DV / 4, ROWG = kThreads / COLG, RPT = DK / ROWG;
  static_assert(COLG * 4 == DV && RPT * ROWG == DK, "tile shape");
  __shared__ float ks[DK], qs[DK];
  __shared__ vf4 red[ROWG][COLG];
  const int tid = threadIdx.x, cg = tid % COLG, rg = tid / COLG;
  const int bh = blockIdx.x;
  float* const Sh = S + (size_t)bh * (DK * DV) + cg * 4;
  vf4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = *reinterpret_cast<const vf4*>(Sh + (size_t)(rg + i * ROWG) * DV);
  const size_t row = (size_t)(bh / grp) * DK;
  for (int i = tid; i < DK; i += kThreads) {
    ks[i] = to_f32(k[row + i]);
    qs[i] = to_f32(q[row + i]);
  }
  vf4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = to_f32(v[(size_t)bh * DV + cg * 4 + e]);
  const float a = g ? expf(g[bh]) : 1.f;
  // A wipe drops the state whatever it holds (memory never written, say).
  if (a == 0.f) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) s[i] = 0.f;
  }
  __syncthreads();
  vf4 acc = 0.f;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + i * ROWG;
    s[i] = a * s[i] + ks[r] * x;
    acc += qs[r] * s[i];
    __builtin_nontemporal_store(s[i], reinterpret_cast<vf4*>(Sh + (size_t)r * DV));
  }
  red[rg][cg] = acc;
  __syncthreads();
  if (tid < DV) {
    float y = 0.f;
#pragma unroll
    for (int r = 0; r < ROWG; ++r) y += red[r][tid / 4][tid % 4];
    o[(size_t)bh * DV + tid] = from_f32<OT>(y);
  }
}

template <int DK, int DV, typename IT, typename OT>
static hipError_t launch(const LinearDecodeArgs& a) {
  const int BH = a.B * a.H;
  prof_mark(kSlotLinearDecode, false, a.stream);
  hipLaunchKernelGGL((decode_kernel<DK, DV, IT, OT>), dim3((unsigned)BH), dim3(kThreads), 0, a.stream,
                     static_cast<const IT*>(a.q), static_cast<const IT*>(a.k), static_cast<const IT*>(a.v),
                     a.log_decay, a.S, static_cast<OT*>(a.o), a.H / a.H_qk);
  hipError_t e = hipGetLastError();
  prof_mark(kSlotLinearDecode, true, a.stream);
  return e;
}

template <int DK, int DV>
static hipError_t launch_d(const LinearDecodeArgs& a) {
  if (a.in_dtype == 1)
    return a.out_dtype == 1 ? launch<DK, DV, bf16, bf16>(a) : launch<DK, DV, bf16, float>(a);
  return a.out_dtype == 1 ? launch<DK, DV, float, bf16>(a) : launch<DK, DV, float, float>(a);
}

}  // namespace lin

long long linear_decode_max_heads() { return max_blocks(lin::kThreads); }

hipError_t launch_linear_decode(const LinearDecodeArgs& a) {
  if (a.d_k == 64 && a.d_v == 64) return lin::launch_d<64, 64>(a);
  if (a.d_k == 64 && a.d_v == 128) return lin::launch_d<64, 128>(a);
  if (a.d_k == 128 && a.d_v == 64) return lin::launch_d<128, 64>(a);
  return lin::launch_d<128, 128>(a);
}

}  // namespace dn
