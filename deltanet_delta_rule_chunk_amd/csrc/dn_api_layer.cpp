// dn_api_layer.cpp -- the C ABI's entry points of a state space layer: the short
// convolution, the selective scan, the norm with the residual's addition.  As in
// dn_api.cpp, every check is made on the host before any HIP call.

#include "dn_api_util.h"
#include "dn_launch.h"

using namespace dn::api;

namespace {

// Rows of `d` elements of [B, L, *] at strides (null: dense) and their extent.
struct Tokens {
  dn::TokenRows r;
  size_t bytes;
};
int check_tokens(const void* p, const long long* strides, int B, int L, int d, size_t size, Tokens* out) {
  const long long s[2] = {strides ? strides[0] : (long long)L * d, strides ? strides[1] : d};
  const long long n[2] = {B, L};
  out->r = dn::TokenRows{p, s[0], s[1]};
  out->bytes = 0;
  if (!p || L == 0) return DN_OK;
  if (!aligned16(p)) return DN_ERR_MISALIGNED;
  long long last = 0;
  for (int i = 0; i < 2; ++i) {
    if (n[i] == 1) continue;  // this stride is not used
    if (s[i] < 0) return DN_ERR_BAD_SHAPE;
    if (s[i] > (1LL << 58) / n[i] || (i == 1 && s[i] > dn::kMostTokenStride)) return DN_ERR_UNSUPPORTED;
    if (s[i] * (long long)size % 16) return DN_ERR_MISALIGNED;
    last += (n[i] - 1) * s[i];
  }
  out->bytes = (size_t)(last + d) * size;
  return DN_OK;
}

int check_sequences(const int* cu, int B, int n_seq) {
  if (!cu) return DN_OK;
  if (B != 1 || n_seq < 1) return DN_ERR_BAD_SHAPE;
  return reinterpret_cast<uintptr_t>(cu) % 4 ? DN_ERR_MISALIGNED : DN_OK;
}
size_t cu_bytes(const int* cu, int n_seq) { return cu ? ((size_t)n_seq + 1) * sizeof(int) : 0; }

int check_conv(const void* x, const long long* strides, const float* weight, const float* bias, const void* state0,
               const int* cu, int B, int L, int D, int K, int n_seq, int silu, int dtype, hipStream_t stream,
               dn::ShortConvArgs* a, Tokens* rows) {
  if (B < 1 || L < 0 || D < 1 || K < 1) return DN_ERR_BAD_SHAPE;
  if (!dtype_ok(dtype) || D % 8 || K < 2 || K > 4) return DN_ERR_UNSUPPORTED;
  int st = check_sequences(cu, B, n_seq);
  if (st != DN_OK) return st;
  if (!cu) n_seq = B;
  if (L > 0x7fffffff - 1024 || D > dn::kMostTokenStride || !dn::short_conv_fits(B, L, D, n_seq, dtype)) return DN_ERR_UNSUPPORTED;
  if (!weight || (L > 0 && !x)) return DN_ERR_NULL_ARG;
  st = check_tokens(x, strides, B, L, D, dtype_size(dtype), rows);
  if (st != DN_OK) return st;
  if (any_misaligned({weight, bias, state0})) return DN_ERR_MISALIGNED;
  *a = dn::ShortConvArgs{};
  a->x = rows->r;
  a->weight = weight;
  a->bias = bias;
  a->state0 = state0;
  a->cu = cu;
  a->B = B;
  a->L = L;
  a->D = D;
  a->K = K;
  a->n_seq = n_seq;
  a->silu = silu != 0;
  a->dtype = dtype;
  a->stream = stream;
  return DN_OK;
}

struct ScanIn {
  const void *u, *dt, *Bm, *Cm, *z;
  const long long* strides;  // batch, token of each of these in turn; or null (dense)
  const float *A, *skip, *dt_bias, *h0;
  const int* cu;
  int B, L, D, N, n_seq, softplus, dtype;
  hipStream_t stream;
};
int check_scan_sizes(const int* cu, int B, int L, int D, int N, int* n_seq, int dtype, bool backward) {
  if (B < 1 || L < 0 || D < 1 || N < 1) return DN_ERR_BAD_SHAPE;
  if (!dtype_ok(dtype) || D % 8 || (N != 8 && N != 16 && N != 32)) return DN_ERR_UNSUPPORTED;
  const int st = check_sequences(cu, B, *n_seq);
  if (st != DN_OK) return st;
  if (!cu) *n_seq = B;
  return D <= dn::kMostTokenStride && dn::selective_scan_fits(B, L, D, N, cu, *n_seq, backward) ? DN_OK : DN_ERR_UNSUPPORTED;
}
int check_scan(const ScanIn& x, bool backward, dn::ScanArgs* a, Tokens (&rows)[5]) {
  int n_seq = x.n_seq;
  int st = check_scan_sizes(x.cu, x.B, x.L, x.D, x.N, &n_seq, x.dtype, backward);
  if (st != DN_OK) return st;
  if (!x.A || (x.L > 0 && (!x.u || !x.dt || !x.Bm || !x.Cm))) return DN_ERR_NULL_ARG;
  const void* p[5] = {x.u, x.dt, x.Bm, x.Cm, x.z};
  for (int i = 0; i < 5; ++i) {
    st = check_tokens(p[i], x.strides ? x.strides + 2 * i : nullptr, x.B, x.L, i == 2 || i == 3 ? x.N : x.D,
                      dtype_size(x.dtype), &rows[i]);
    if (st != DN_OK) return st;
  }
  if (any_misaligned({x.A, x.skip, x.dt_bias, x.h0})) return DN_ERR_MISALIGNED;
  *a = dn::ScanArgs{};
  a->u = rows[0].r;
  a->dt = rows[1].r;
  a->Bm = rows[2].r;
  a->Cm = rows[3].r;
  a->z = rows[4].r;
  a->A = x.A;
  a->skip = x.skip;
  a->dt_bias = x.dt_bias;
  a->h0 = x.h0;
  a->cu = x.cu;
  a->B = x.B;
  a->L = x.L;
  a->D = x.D;
  a->N = x.N;
  a->n_seq = n_seq;
  a->softplus = x.softplus != 0;
  a->dtype = x.dtype;
  a->stream = x.stream;
  return DN_OK;
}

int check_norm(int rows, int D, float eps, int dtype, int residual_dtype) {
  if (rows < 0 || D < 1) return DN_ERR_BAD_SHAPE;
  if (!dtype_ok(dtype) || !dtype_ok(residual_dtype) || D % 8) return DN_ERR_UNSUPPORTED;
  if (dtype == DN_F32 && residual_dtype != DN_F32) return DN_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || eps > 3.0e38f) return DN_ERR_UNSUPPORTED;
  return dn::add_norm_fits(rows, D) ? DN_OK : DN_ERR_UNSUPPORTED;
}

int done(hipError_t e) { return e == hipSuccess ? DN_OK : hip_fail(e); }

}  // namespace

extern "C" {

int deltanet_short_conv_fwd(const void* x, const long long* x_strides, const float* weight, const float* bias,
                            const void* state0, const int* cu_seqlens, void* y, void* state, int B, int L, int D, int K,
                            int n_seq, int silu, dn_dtype dtype, hipStream_t stream) {
  dn::ShortConvArgs a;
  Tokens rows;
  const int st = check_conv(x, x_strides, weight, bias, state0, cu_seqlens, B, L, D, K, n_seq, silu, dtype, stream, &a, &rows);
  if (st != DN_OK) return st;
  if (L > 0 && !y) return DN_ERR_NULL_ARG;
  if (any_misaligned({y, state})) return DN_ERR_MISALIGNED;
  const size_t e = dtype_size(dtype), kept = (size_t)a.n_seq * (K - 1) * D * e;
  const Span in[] = {{x, rows.bytes}, {weight, (size_t)D * K * 4}, {bias, (size_t)D * 4}, {state0, kept}, {cu_seqlens, cu_bytes(cu_seqlens, a.n_seq)}};
  const Span out[] = {{y, (size_t)B * L * D * e}, {state, kept}};
  if (any_overlap(in, out, Span{nullptr, 0})) return DN_ERR_ALIASING;
  a.y = y;
  a.state = state;
  return done(dn::launch_short_conv(a));
}

size_t deltanet_short_conv_bwd_workspace_bytes(int B, int L, int D, int K) {
  if (B < 1 || L < 0 || D < 1 || D % 8 || K < 2 || K > 4) return 0;
  if (L > 0x7fffffff - 1024 || D > dn::kMostTokenStride || !dn::short_conv_fits(B, L, D, 1, DN_F32)) return 0;
  return dn::short_conv_bwd_workspace_bytes(B, L, D, K);
}

int deltanet_short_conv_bwd(const void* x, const long long* x_strides, const float* weight, const float* bias,
                            const void* state0, const int* cu_seqlens, const void* dy, const void* dstate, void* dx,
                            float* dweight, float* dbias, void* dstate0, int B, int L, int D, int K, int n_seq, int silu,
                            dn_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  dn::ShortConvArgs a;
  Tokens rows;
  const int st = check_conv(x, x_strides, weight, bias, state0, cu_seqlens, B, L, D, K, n_seq, silu, dtype, stream, &a, &rows);
  if (st != DN_OK) return st;
  if (!dweight || (L > 0 && (!dy || !dx))) return DN_ERR_NULL_ARG;
  if (any_misaligned({dy, dstate, dx, dweight, dbias, dstate0, workspace})) return DN_ERR_MISALIGNED;
  const size_t e = dtype_size(dtype), kept = (size_t)a.n_seq * (K - 1) * D * e, tokens = (size_t)B * L * D * e;
  const size_t wb = (size_t)D * K * 4, need = dn::short_conv_bwd_workspace_bytes(B, L, D, K);
  const Span in[] = {{x, rows.bytes}, {weight, wb}, {bias, (size_t)D * 4}, {state0, kept}, {cu_seqlens, cu_bytes(cu_seqlens, a.n_seq)},
                     {dy, tokens}, {dstate, kept}};
  const Span out[] = {{dx, tokens}, {dweight, wb}, {dbias, (size_t)D * 4}, {dstate0, kept}};
  if (workspace && workspace_bytes < need) return DN_ERR_WORKSPACE;
  if (any_overlap(in, out, Span{workspace, workspace ? need : 0})) return DN_ERR_ALIASING;
  Workspace w(workspace, need, stream);
  if (w.error() != hipSuccess) return hip_fail(w.error());
  a.dy = dy;
  a.dstate = dstate;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dstate0 = dstate0;
  a.workspace = w.get();
  return done(w.done(dn::launch_short_conv_bwd(a)));
}

int deltanet_short_conv_step(const void* x, const long long* x_stride, const float* weight, const float* bias, void* state,
                             void* y, int B, int D, int K, int silu, dn_dtype dtype, hipStream_t stream) {
  const long long strides[2] = {x_stride ? *x_stride : D, D};
  dn::ShortConvArgs a;
  Tokens rows;
  const int st = check_conv(x, strides, weight, bias, state, nullptr, B, 1, D, K, 0, silu, dtype, stream, &a, &rows);
  if (st != DN_OK) return st;
  if (!state || !y) return DN_ERR_NULL_ARG;
  if (any_misaligned({y})) return DN_ERR_MISALIGNED;
  const size_t e = dtype_size(dtype);
  const Span in[] = {{x, rows.bytes}, {weight, (size_t)D * K * 4}, {bias, (size_t)D * 4}};
  const Span out[] = {{y, (size_t)B * D * e}, {state, (size_t)B * (K - 1) * D * e}};
  if (any_overlap(in, out, Span{nullptr, 0})) return DN_ERR_ALIASING;
  a.y = y;
  a.state = state;
  return done(dn::launch_short_conv_step(a));
}

size_t deltanet_selective_scan_fwd_workspace_bytes(int B, int L, int D, int N, int packed, int n_seq) {
  const int any = 0;
  if (check_scan_sizes(packed ? &any : nullptr, B, L, D, N, &n_seq, DN_F32, false) != DN_OK) return 0;
  return dn::selective_scan_workspace_bytes(B, L, D, N, packed, n_seq);
}

int deltanet_selective_scan_fwd(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                const long long* strides, const float* A, const float* D_skip, const float* dt_bias,
                                const float* h0, const int* cu_seqlens, void* y, float* hT, int B, int L, int D, int N,
                                int n_seq, int softplus, dn_dtype dtype, void* workspace, size_t workspace_bytes,
                                hipStream_t stream) {
  dn::ScanArgs a;
  Tokens rows[5];
  const int st = check_scan({u, dt, Bm, Cm, z, strides, A, D_skip, dt_bias, h0, cu_seqlens, B, L, D, N, n_seq, softplus, dtype, stream},
                            false, &a, rows);
  if (st != DN_OK) return st;
  if (L > 0 && !y) return DN_ERR_NULL_ARG;
  if (any_misaligned({y, hT, workspace})) return DN_ERR_MISALIGNED;
  const size_t vec = (size_t)D * 4, state = vec * N, states = (size_t)a.n_seq * state;
  const size_t need = dn::selective_scan_workspace_bytes(B, L, D, N, cu_seqlens, a.n_seq);
  const Span in[] = {{u, rows[0].bytes}, {dt, rows[1].bytes}, {Bm, rows[2].bytes}, {Cm, rows[3].bytes}, {z, rows[4].bytes}, {A, state},
                     {D_skip, vec}, {dt_bias, vec}, {hT == h0 ? nullptr : h0, states}, {cu_seqlens, cu_bytes(cu_seqlens, a.n_seq)}};
  const Span out[] = {{y, (size_t)B * L * D * dtype_size(dtype)}, {hT, states}};
  if (workspace && workspace_bytes < need) return DN_ERR_WORKSPACE;
  if (any_overlap(in, out, Span{workspace, workspace ? need : 0})) return DN_ERR_ALIASING;
  Workspace w(workspace, need, stream);
  if (w.error() != hipSuccess) return hip_fail(w.error());
  a.y = y;
  a.hT = hT;
  a.workspace = w.get();
  return done(w.done(dn::launch_selective_scan(a)));
}

size_t deltanet_selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, int packed, int n_seq) {
  const int any = 0;
  if (check_scan_sizes(packed ? &any : nullptr, B, L, D, N, &n_seq, DN_F32, true) != DN_OK) return 0;
  return dn::selective_scan_bwd_workspace_bytes(B, L, D, N, packed, n_seq);
}

int deltanet_selective_scan_bwd(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                const long long* strides, const float* A, const float* D_skip, const float* dt_bias,
                                const float* h0, const int* cu_seqlens, const void* dy, const float* dhT, void* du, void* ddt,
                                void* dB, void* dC, void* dz, float* dA, float* dD_skip, float* ddt_bias, float* dh0, int B,
                                int L, int D, int N, int n_seq, int softplus, dn_dtype dtype, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  dn::ScanArgs a;
  Tokens rows[5];
  const int st = check_scan({u, dt, Bm, Cm, z, strides, A, D_skip, dt_bias, h0, cu_seqlens, B, L, D, N, n_seq, softplus, dtype, stream},
                            true, &a, rows);
  if (st != DN_OK) return st;
  if (!dA || (L > 0 && (!dy || !du || !ddt || !dB || !dC || (z && !dz)))) return DN_ERR_NULL_ARG;
  if (any_misaligned({dy, dhT, du, ddt, dB, dC, dz, dA, dD_skip, ddt_bias, dh0, workspace})) return DN_ERR_MISALIGNED;
  const size_t vec = (size_t)D * 4, state = vec * N, states = (size_t)a.n_seq * state;
  const size_t e = dtype_size(dtype), tokens = (size_t)B * L * D * e, bc = (size_t)B * L * N * e;
  const size_t need = dn::selective_scan_bwd_workspace_bytes(B, L, D, N, cu_seqlens, a.n_seq);
  const Span in[] = {{u, rows[0].bytes}, {dt, rows[1].bytes}, {Bm, rows[2].bytes}, {Cm, rows[3].bytes}, {z, rows[4].bytes}, {A, state},
                     {D_skip, vec}, {dt_bias, vec}, {h0, states}, {cu_seqlens, cu_bytes(cu_seqlens, a.n_seq)}, {dy, tokens}, {dhT, states}};
  const Span out[] = {{du, tokens}, {ddt, tokens}, {dB, bc}, {dC, bc}, {z ? dz : nullptr, tokens}, {dA, state},
                      {dD_skip, vec}, {ddt_bias, vec}, {dh0, states}};
  if (workspace && workspace_bytes < need) return DN_ERR_WORKSPACE;
  if (any_overlap(in, out, Span{workspace, workspace ? need : 0})) return DN_ERR_ALIASING;
  Workspace w(workspace, need, stream);
  if (w.error() != hipSuccess) return hip_fail(w.error());
  a.dy = dy;
  a.dhT = dhT;
  a.du = du;
  a.ddt = ddt;
  a.dB = dB;
  a.dC = dC;
  a.dz = dz;
  a.dA = dA;
  a.dskip = dD_skip;
  a.dbias = ddt_bias;
  a.dh0 = dh0;
  a.workspace = w.get();
  return done(w.done(dn::launch_selective_scan_bwd(a)));
}

int deltanet_selective_scan_step(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                 const long long* strides, const float* A, const float* D_skip, const float* dt_bias, float* h,
                                 void* y, int B, int D, int N, int softplus, dn_dtype dtype, hipStream_t stream) {
  long long s[10];
  for (int i = 0; i < 5; ++i) {
    const int d = i == 2 || i == 3 ? N : D;
    s[2 * i] = strides ? strides[i] : d;
    s[2 * i + 1] = d;
  }
  dn::ScanArgs a;
  Tokens rows[5];
  const int st = check_scan({u, dt, Bm, Cm, z, s, A, D_skip, dt_bias, h, nullptr, B, 1, D, N, 0, softplus, dtype, stream}, false, &a, rows);
  if (st != DN_OK) return st;
  if (!h || !y) return DN_ERR_NULL_ARG;
  if (any_misaligned({y})) return DN_ERR_MISALIGNED;
  const size_t vec = (size_t)D * 4;
  const Span in[] = {{u, rows[0].bytes}, {dt, rows[1].bytes}, {Bm, rows[2].bytes}, {Cm, rows[3].bytes}, {z, rows[4].bytes}, {A, vec * N},
                     {D_skip, vec}, {dt_bias, vec}};
  const Span out[] = {{y, (size_t)B * D * dtype_size(dtype)}, {h, (size_t)B * vec * N}};
  if (any_overlap(in, out, Span{nullptr, 0})) return DN_ERR_ALIASING;
  a.y = y;
  a.hT = h;
  return done(dn::launch_selective_scan_step(a));
}

int deltanet_add_rms_norm(const void* x, const void* residual, const float* weight, void* total, void* y, float* scale, int rows,
                          int D, float eps, dn_dtype dtype, dn_dtype residual_dtype, hipStream_t stream) {
  const int st = check_norm(rows, D, eps, dtype, residual_dtype);
  if (st != DN_OK) return st;
  if (!residual != !total) return DN_ERR_NULL_ARG;
  if (rows == 0) return DN_OK;
  if (!x || !y) return DN_ERR_NULL_ARG;
  if (any_misaligned({x, residual, weight, total, y, scale})) return DN_ERR_MISALIGNED;
  const size_t n = (size_t)rows * D, e = dtype_size(dtype), r = dtype_size(residual_dtype);
  // total may take the place of the residual, or of x where their types agree.
  const Span in[] = {{total == x && e == r ? nullptr : x, n * e}, {total == residual ? nullptr : residual, n * r}, {weight, (size_t)D * 4}};
  const Span out[] = {{total, n * r}, {y, scale ? n : n * e}, {scale, (size_t)rows * 4}};
  if (any_overlap(in, out, Span{nullptr, 0})) return DN_ERR_ALIASING;
  dn::AddNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.total = total;
  a.y = y;
  a.scale = scale;
  a.rows = rows;
  a.D = D;
  a.dtype = dtype;
  a.residual_dtype = residual ? (int)residual_dtype : (int)dtype;
  a.eps = eps;
  a.stream = stream;
  return done(dn::launch_add_norm(a));
}

size_t deltanet_add_rms_norm_bwd_workspace_bytes(int rows, int D) {
  return check_norm(rows, D, 0.f, DN_F32, DN_F32) == DN_OK ? dn::add_norm_bwd_workspace_bytes(rows, D) : 0;
}

int deltanet_add_rms_norm_bwd(const void* total, const float* weight, const void* dy, const void* dtotal, void* dx,
                              void* dresidual, float* dweight, int rows, int D, float eps, dn_dtype dtype,
                              dn_dtype residual_dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_norm(rows, D, eps, dtype, residual_dtype);
  if (st != DN_OK) return st;
  if (rows > 0 && (!total || !dy || !dx)) return DN_ERR_NULL_ARG;
  if (any_misaligned({total, weight, dy, dtotal, dx, dresidual, dweight, workspace})) return DN_ERR_MISALIGNED;
  const size_t n = (size_t)rows * D, e = dtype_size(dtype), r = dtype_size(residual_dtype), wb = (size_t)D * 4;
  const size_t need = dweight ? dn::add_norm_bwd_workspace_bytes(rows, D) : 0;
  const Span in[] = {{total, n * r}, {weight, wb}, {dy, n * e}, {dtotal, n * r}};
  const Span out[] = {{dx, n * e}, {dresidual, n * r}, {dweight, wb}};
  if (workspace && workspace_bytes < need) return DN_ERR_WORKSPACE;
  if (any_overlap(in, out, Span{workspace, workspace ? need : 0})) return DN_ERR_ALIASING;
  Workspace w(workspace, need, stream);
  if (w.error() != hipSuccess) return hip_fail(w.error());
  dn::AddNormArgs a{};
  a.total = const_cast<void*>(total);
  a.weight = weight;
  a.dy = dy;
  a.dtotal = dtotal;
  a.dx = dx;
  a.dresidual = dresidual;
  a.dweight = dweight;
  a.rows = rows;
  a.D = D;
  a.dtype = dtype;
  a.residual_dtype = residual_dtype;
  a.eps = eps;
  a.workspace = w.get();
  a.stream = stream;
  return done(w.done(dn::launch_add_norm_bwd(a)));
}

}  // extern "C"
