// dn_linear.hip -- launches of the gated linear recurrence's forward (the
// kernels and what they compute: dn_linear.h).

#include "dn_linear.h"

namespace dn {
namespace lin {

static __global__ __launch_bounds__(256) void copy_state_kernel(float* dst, const float* src, size_t n) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i < n)
    *reinterpret_cast<f32x4*>(dst + i) = src ? *reinterpret_cast<const f32x4*>(src + i) : zero4();
}

hipError_t launch_copy_state(float* dst, const float* src, size_t n, hipStream_t stream) {
  hipLaunchKernelGGL(copy_state_kernel, dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, dst, src, n);
  return hipGetLastError();
}

template <typename IT, typename OT, int DK, int DV>
static hipError_t forward(const LinearArgs& a) {
  const int BH = a.B * a.H, grp = a.H / a.H_qk;
  const Split s = split_of(BH, a.L, DK, DV, sizeof(IT) == 4, false);
  const size_t N = (size_t)DK * DV;
  float* states = static_cast<float*>(a.workspace);
  hipError_t e;
  if (s.nseg > 1) {
    double* decays = reinterpret_cast<double*>(states + (size_t)BH * s.nseg * N);
    StateArgs st{{a.k, grp}, {a.v, 1}, a.log_decay, states, decays, s.nseg, a.L, BH, grp, 0, s.nseg - 1, s};
    e = launch(&state_kernel<IT, DK, DV>, kSlotLinearState, items(BH, grp, st.count), 64 * waves(DV),
               state_lds<IT, DK, DV>(), a.stream, st);
    if (e != hipSuccess) return e;
    CombineArgs cb{states, decays, a.S0, a.log_decay, s.nseg, s.nseg, (int)N, a.L};
    prof_mark(kSlotLinearState, false, a.stream);
    hipLaunchKernelGGL(combine_kernel, dim3(cdiv((int)N, 1024), (unsigned)BH), dim3(256), 0, a.stream, cb);
    e = hipGetLastError();
    prof_mark(kSlotLinearState, true, a.stream);
    if (e != hipSuccess) return e;
  }
  OutArgs o{{a.q, grp}, {a.k, grp}, {a.v, 1}, {nullptr, 1}, a.log_decay, states, a.S0, a.o,
            a.S_final, (long long)N, nullptr, nullptr, s.nseg, a.L, BH, grp, s};
  constexpr int lds = OutLds<IT, OT, DK, DV, kNone>::bytes;
  static_assert(lds <= (sizeof(IT) == 2 ? 80 : 160) * 1024, "two bf16 workgroups share a CU's LDS");
  return launch(&out_kernel<IT, OT, DK, DV>, kSlotLinearOut, items(BH, grp, s.nseg), 64 * waves(DV), lds, a.stream, o);
}

template <int DK, int DV>
static hipError_t forward_d(const LinearArgs& a) {
  if (a.in_dtype == 1)
    return a.out_dtype == 1 ? forward<bf16, bf16, DK, DV>(a) : forward<bf16, float, DK, DV>(a);
  return a.out_dtype == 1 ? forward<float, bf16, DK, DV>(a) : forward<float, float, DK, DV>(a);
}

}  // namespace lin

size_t linear_workspace_bytes(int B, int H, int L, int d_k, int d_v, int in_dtype) {
  if (L == 0) return 0;
  const size_t BH = (size_t)B * H;
  const lin::Split s = lin::split_of((int)BH, L, d_k, d_v, in_dtype == 0, false);
  return s.nseg > 1 ? BH * s.nseg * ((size_t)d_k * d_v * 4 + 8) : 0;
}

hipError_t launch_linear_fwd(const LinearArgs& a) {
  if (a.L == 0)
    return a.S_final && a.S_final != a.S0
               ? lin::launch_copy_state(a.S_final, a.S0, (size_t)a.B * a.H * a.d_k * a.d_v, a.stream)
               : hipSuccess;
  if (a.d_k == 64 && a.d_v == 64) return lin::forward_d<64, 64>(a);
  if (a.d_k == 64 && a.d_v == 128) return lin::forward_d<64, 128>(a);
  if (a.d_k == 128 && a.d_v == 64) return lin::forward_d<128, 64>(a);
  return lin::forward_d<128, 128>(a);
}

}  // namespace dn
