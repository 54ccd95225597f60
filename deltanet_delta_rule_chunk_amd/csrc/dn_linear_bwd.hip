// dn_linear_bwd.hip -- the gated linear recurrence's backward.
//
// The vector gradients are three walks of the forward's output kernel
// (dn_linear.h):
//     dq = F(dO, v, k) on S^T,  dv = R(k, q, dO) on dS,  dk = R(v, dO, q) on dS^T.
//
// The decay's gradient.  With c_t the product <S_{t-1}, dS_t> e^{g_t} of the
// state before token t with the gradient it receives through token t,
//     d g_t = sum over pairs (write i < t, read r >= t) of the pair's term
//           + what reads r >= t take from before the pairs' reach
//           + what the state that leaves keeps of it,
// which splits by 64-row chunks into sums over pairs that cross t alone:
//     d g_t =  sum_{r >= t} x_r  +  sum_{i < t} y_i  +  m_t  +  D_c
//   x_r = q_r . (dq_r's part from the entering state)        (walk of dq)
//   y_i = k_i . (dk_i's part from the exit gradient)         (walk of dk)
//   m_t = sum_{i < t <= r} P_ri (dO_r . v_i), the chunk's own pairs (walk of dq)
//   D_c = e^{G_C} <S_c, dS_c'>: entering state against exit gradient.
// D follows from chunk to chunk: <S_{c+1}, dS_c'> = D_{c+1} + sum x (chunk
// c+1) = D_c + sum y (chunk c), anchored at both ends of each segment, where
// both states are at hand, and at every chunk that leaves less than 2^-64 of what
// enters it (a wipe in it, say): D is 0 there, which gives both its neighbours.
// Nothing is carried past such a chunk, so documents in one row stay apart bit
// for bit.  Walked from one anchor the roundings of the sums would reach the next
// as an offset; D is taken from both, each weighted with the squares of the sums
// passed on the way from the other, which is the best estimate if those are what
// the roundings go by.  Between two anchors D is off by about 2^-24 of the largest
// <state, gradient> there, and so is the gradient of each of the chunk's tokens:
// far below its neighbours', but not small against a single token's whose decay
// leaves less than that of the state.  (The state and its gradient at every chunk
// would show more; they are 4 times a chunk's rows.)  A token's own
// pair (r = i) and the pairs on one side of t never enter x, y and m, so a strong
// decay, whose gradient is small beside q . dq, keeps its accuracy.  The sums
// over rows and chunks are taken in fp64; they are a few bytes per token.
//
// 32 heads of 128 x 128, bf16, L = 65536: sums of both directions 455 us, walks 1.84
// ms (7.7 GB, 4.2 TB/s; matrix instructions busy for 42%, 745 TFLOP/s as
// executed), the decay's gradient 28 us.  dk's and dv's walks of a segment side by
// side on one XCD, for the rows that both read, took 1.84 ms for 1.75.
//
// Heads that share q and k: each state head's dq and dk go to the workspace
// in fp32, and a last kernel adds the group's in head order and rounds once.

#include "dn_linear.h"

namespace dn {
namespace lin {

constexpr int max_of(int a, int b) { return a > b ? a : b; }
constexpr int walk_threads(int DK, int DV) { return 64 * max_of(waves(DK), waves(DV)); }

// Segment sums of the state (k, v) and of its gradient (q, dO) side by side.
template <typename IT, int DK, int DV>
__global__ __launch_bounds__(64 * waves(DV), simd_waves<IT>(DV)) void bwd_state_kernel(StateArgs s, StateArgs x, int ns) {
  const Lds m = dynamic_lds();
  if ((int)blockIdx.x < ns) state_walk<IT, DK, DV, false>(s, blockIdx.x, m);
  else state_walk<IT, DK, DV, true>(x, blockIdx.x - ns, m);
}
static __global__ __launch_bounds__(256) void bwd_combine_kernel(CombineArgs s, CombineArgs x) {
  if (blockIdx.z == 0) combine<false>(s);
  else combine<true>(x);
}

// The three walks side by side, the longest first.  A walk with fewer waves
// than the launch lets the others end at once.
template <typename IT, typename OT, int DK, int DV>
constexpr int walks_lds() {
  return max_of(OutLds<IT, OT, DV, DK, kPairs>::bytes,
                max_of(OutLds<IT, IT, DK, DV, kNone>::bytes, OutLds<IT, OT, DV, DK, kDots>::bytes));
}
// Behind them in the grid, one workgroup per inner border of the segments: the
// state there against its gradient, which the decay's gradient starts from.
struct BorderArgs {
  const float *S, *X;  // [BH][nseg + 1][N], [BH][nseg][N]
  const float* g;
  double* border;      // [BH][nseg]: entry s for the start of segment s >= 1
  int L, N;
  Split s;
};

// <u, v> over T threads, every thread's answer.  (Where v is 0, u may be
// anything: the state of a call that wipes it first has no gradient.)
template <int T>
__device__ __forceinline__ double dot_states(const float* u, const float* v, int n, double* part) {
  double acc = 0.0;
  for (int i = threadIdx.x * 4; i < n; i += T * 4) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(u + i), b = *reinterpret_cast<const f32x4*>(v + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc += b[e] == 0.f ? 0.0 : (double)a[e] * (double)b[e];
  }
  acc = lane_value(wave_scan(acc), 63);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = acc;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < T / 64; ++i) sum += part[i];
  return sum;
}

template <int T>
__device__ __forceinline__ void border_dot(const BorderArgs& a, int i, double* part) {
  const int bh = i / (a.s.nseg - 1), s = i % (a.s.nseg - 1) + 1;
  const double d = dot_states<T>(a.S + ((size_t)bh * (a.s.nseg + 1) + s) * a.N, a.X + ((size_t)bh * a.s.nseg + s - 1) * a.N,
                                 a.N, part);
  // The reversed walk's states are gradients of the state after the token
  // behind them; that token's decay stands between.
  const float f = exp2_hw((float)log2_decay(a.g[(size_t)bh * a.L + (size_t)s * a.s.cps * C]));
  if (threadIdx.x == 0) a.border[(size_t)bh * a.s.nseg + s] = f == 0.f ? 0.0 : d * (double)f;
}

template <typename IT, typename OT, int DK, int DV>
__global__ __launch_bounds__(walk_threads(DK, DV), simd_waves<IT>(max_of(DK, DV))) void walks_kernel(
    OutArgs q, OutArgs k, OutArgs v, int n, BorderArgs b) {
  const Lds m = dynamic_lds();
  const int walk = blockIdx.x / n, flat = blockIdx.x % n;
  if ((int)blockIdx.x >= 3 * n) {
    border_dot<walk_threads(DK, DV)>(b, blockIdx.x - 3 * n, reinterpret_cast<double*>(m.p));
    return;
  }
  if ((int)threadIdx.x >= 64 * waves(walk < 2 ? DK : DV)) return;
  if (walk == 0) out_walk<IT, OT, DV, DK, false, kPairs>(q, flat, m);
  else if (walk == 1) out_walk<IT, OT, DV, DK, true, kDots>(k, flat, m);
  else out_walk<IT, IT, DK, DV, true, kNone>(v, flat, m);
}

struct DecayGradArgs {
  const float *g, *x, *y, *m;
  const float* S;      // [BH][nseg + 1][N]: slot nseg = the last state
  const double* border;
  const float *S0, *dS0;  // [BH][N]: the first state and its gradient; S0 null: zero; dS0 null: not known
  const float* dS;     // [BH][N] or null: gradient of the last state
  float* dg;
  int L, BH, N;
  Split s;
};

constexpr int kGradThreads = 1024;
// log2 of what a chunk has to leave of its entering state for D to be more than
// 0: 2^40 under the roundings of the sums that it would be a difference of.
constexpr double kThrough2 = -64.0;

// One step of a wave's inclusive sums that start anew behind every lane whose
// `cut` is set (its own value is the first).
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ void cut_scan_step(double& v, double& q, int& cut) {
  const double pv = dpp<CTRL, ROWS>(v), pq = dpp<CTRL, ROWS>(q);
  const int pc = dpp<CTRL, ROWS>(cut);
  if (!cut) v += pv, q += pq;
  cut |= pc;
}

// <state, gradient> in front of each of n chunks in the walk's order, from `first`
// in front of them all on: behind a chunk it is in[i] where the chunk lets nothing
// through, else in[i] - out[i] more than in front.  v[i] receives it and q[i] the
// squares of the sums that it is made of, of which `first` has q0.  One wave.
__device__ __forceinline__ void carry_walk(const double* in, const double* out, const unsigned char* shut, int n,
                                           bool reversed, double first, double q0, double* v, double* q) {
  const int l = threadIdx.x & 63;
  for (int base = 0; base < n; base += 64) {
    const int j = base + l, i = reversed ? n - 1 - j : j;
    const bool on = j < n;
    int cut = on && shut[i];
    const double a = on ? in[i] : 0.0, b = on && !cut ? out[i] : 0.0;
    double x = a - b, y = a * a + b * b;
    cut_scan_step<0x111>(x, y, cut);
    cut_scan_step<0x112>(x, y, cut);
    cut_scan_step<0x114>(x, y, cut);
    cut_scan_step<0x118>(x, y, cut);
    cut_scan_step<0x142, 0xa>(x, y, cut);
    cut_scan_step<0x143, 0xc>(x, y, cut);
    if (!cut) x += first, y += q0;
    const double px = __shfl_up(x, 1, 64), py = __shfl_up(y, 1, 64);
    if (on) v[i] = l == 0 ? first : px, q[i] = l == 0 ? q0 : py;
    first = lane_value(x, 63);
    q0 = lane_value(y, 63);
  }
}

// One workgroup per (head, segment).
__device__ __forceinline__ void decay_grad(const DecayGradArgs& a, int block) {
  __shared__ double part[kGradThreads / 64], tx[kMaxChunks], ty[kMaxChunks];
  __shared__ double left[kMaxChunks], left_q[kMaxChunks], right[kMaxChunks], right_q[kMaxChunks];
  __shared__ unsigned char shut[kMaxChunks];
  const int bh = block / a.s.nseg, seg = block % a.s.nseg;
  const int w = threadIdx.x >> 6, l = threadIdx.x & 63;
  const int c0 = seg * a.s.cps, c1 = min(c0 + a.s.cps, a.s.nc), n = c1 - c0;
  const bool end = seg == a.s.nseg - 1;
  const size_t row0 = ((size_t)bh * a.s.nc + c0) * C, tok0 = (size_t)bh * a.L;
  // <state that leaves the segment, its gradient>, and the same at its start
  // (nothing is known there only if S0 is given and dS0 not asked for).
  double held = 0.0, enter = 0.0;
  bool known = true;
  if (!end) {
    held = a.border[(size_t)bh * a.s.nseg + seg + 1];
  } else if (a.dS) {
    held = dot_states<kGradThreads>(a.S + ((size_t)bh * (a.s.nseg + 1) + a.s.nseg) * a.N, a.dS + (size_t)bh * a.N, a.N, part);
  }
  if (seg > 0) {
    enter = a.border[(size_t)bh * a.s.nseg + seg];
  } else if (a.S0) {
    known = a.dS0 != nullptr;
    if (known) enter = dot_states<kGradThreads>(a.S0 + (size_t)bh * a.N, a.dS0 + (size_t)bh * a.N, a.N, part);
  }

  for (int i = w; i < n; i += kGradThreads / 64) {
    const size_t at = row0 + (size_t)i * C + l;
    const int t = (c0 + i) * C + l;
    const double x = wave_scan(a.x[at]), y = wave_scan(a.y[at]), g = wave_scan(log2_decay(t < a.L ? a.g[tok0 + t] : 0.f));
    // (Nothing enters a zero state's first chunk or leaves the last towards no gradient.)
    if (l == 63) {
      tx[i] = x, ty[i] = y;
      shut[i] = g < kThrough2 || (seg == 0 && i == 0 && !a.S0) || (end && i == n - 1 && !a.dS);
    }
  }
  __syncthreads();
  // <state, its gradient> in front of each chunk from the left, behind it from the right.
  if (w == 0) carry_walk(ty, tx, shut, n, false, enter, known ? 0.0 : HUGE_VAL, left, left_q);
  else if (w == 1) carry_walk(tx, ty, shut, n, true, held, 0.0, right, right_q);
  __syncthreads();
  for (int i = w; i < n; i += kGradThreads / 64) {
    // What the chunk lets through: from the left, from the right, both.
    const double lo = left[i] - tx[i], hi = right[i] - ty[i];
    const double lq = left_q[i] + tx[i] * tx[i], hq = right_q[i] + ty[i] * ty[i];
    double through = hi;
    if (lq < HUGE_VAL && lq + hq > 0.0) through += (lo - hi) * (hq / (lq + hq));
    if (shut[i]) through = 0.0;
    const size_t at = row0 + (size_t)i * C;
    const int t = (c0 + i) * C + l;
    // Sums over the rows from t on (lane l: from row 63 - l on, then handed to
    // its lane) and over those in front of t.
    const double from = __shfl(wave_scan(a.x[at + C - 1 - l]), C - 1 - l, 64);
    const double before = wave_scan(l > 0 ? a.y[at + l - 1] : 0.f);
    const double v = from + before + (double)a.m[at + l] + through;
    if (t < a.L) a.dg[tok0 + t] = log2_decay(a.g[tok0 + t]) <= kWipe2 ? 0.f : (float)v;
  }
}

// out[u] = sum over the group's members of in[u grp + m], rounded once.
struct GroupSumArgs {
  const float *dq, *dk;
  void *out_q, *out_k;
  size_t per_head, n;  // elements of a head, of an output
  int grp;
};
template <typename OT>
__device__ __forceinline__ void group_sum(const GroupSumArgs& a, size_t i4) {
  const bool first = i4 * 4 < a.n;
  const size_t i = first ? i4 * 4 : i4 * 4 - a.n;
  const size_t u = i / a.per_head;
  const float* p = (first ? a.dq : a.dk) + u * a.grp * a.per_head + (i - u * a.per_head);
  f32x4 x = *reinterpret_cast<const f32x4*>(p);
  for (int m = 1; m < a.grp; ++m) x += *reinterpret_cast<const f32x4*>(p + (size_t)m * a.per_head);
  store4(static_cast<OT*>(first ? a.out_q : a.out_k) + i, x);
}

// What is left after the walks: the decay's gradient (the first `ng`
// workgroups) and the sums over shared heads.
template <typename OT>
__global__ __launch_bounds__(kGradThreads) void finish_kernel(DecayGradArgs g, int ng, GroupSumArgs s) {
  if ((int)blockIdx.x < ng) decay_grad(g, blockIdx.x);
  else
    for (size_t i = (size_t)(blockIdx.x - ng) * kGradThreads + threadIdx.x; i < s.n / 2; i += (size_t)(gridDim.x - ng) * kGradThreads)
      group_sum<OT>(s, i);
}

struct BwdWs {
  size_t S, X, dS, dX, border, x, y, m, dq, dk, total;  // byte offsets
};
static BwdWs bwd_ws(int B, int H, int H_qk, int L, int d_k, int d_v, bool f32) {
  const size_t BH = (size_t)B * H, N = (size_t)d_k * d_v * 4;
  const Split s = split_of((int)BH, L, d_k, d_v, f32, true);
  const size_t rows = BH * s.nc * C * 4, vec = H == H_qk ? 0 : BH * L * d_k * 4;
  BwdWs w{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at += (n + 255) & ~(size_t)255;
    return p;
  };
  w.S = take(BH * (s.nseg + 1) * N);
  w.X = take(s.nseg > 1 ? BH * s.nseg * N : 0);
  w.dS = take(BH * s.nseg * 8);
  w.dX = take(BH * s.nseg * 8);
  w.border = take(BH * s.nseg * 8);
  w.x = take(rows);
  w.y = take(rows);
  w.m = take(rows);
  w.dq = take(vec);
  w.dk = take(vec);
  w.total = at;
  return w;
}

// Workgroups of the sums over shared heads at most: 32 rounds of the card.
constexpr size_t kSumBlocks = 16384;

template <typename IT, typename OT, int DK, int DV>
static hipError_t backward(const LinearBwdArgs& a) {
  const int BH = a.B * a.H, grp = a.H / a.H_qk;
  const Split s = split_of(BH, a.L, DK, DV, sizeof(IT) == 4, true);
  const BwdWs o = bwd_ws(a.B, a.H, a.H_qk, a.L, DK, DV, sizeof(IT) == 4);
  const int N = DK * DV;
  char* const base = static_cast<char*>(a.workspace);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  auto d = [&](size_t off) { return reinterpret_cast<double*>(base + off); };
  hipError_t e;
  if (s.nseg > 1) {
    StateArgs st{{a.k, grp}, {a.v, 1}, a.log_decay, f(o.S), d(o.dS), s.nseg + 1, a.L, BH, grp, 0, s.nseg - 1, s};
    StateArgs sx{{a.q, grp}, {a.dO, 1}, a.log_decay, f(o.X), d(o.dX), s.nseg, a.L, BH, grp, 1, s.nseg - 1, s};
    const int ns = (int)items(BH, grp, s.nseg - 1);
    e = launch(&bwd_state_kernel<IT, DK, DV>, kSlotLinearState, 2LL * ns, 64 * waves(DV), state_lds<IT, DK, DV>(),
               a.stream, st, sx, ns);
    if (e != hipSuccess) return e;
    CombineArgs cs{f(o.S), d(o.dS), a.S0, a.log_decay, s.nseg + 1, s.nseg, N, a.L};
    CombineArgs cx{f(o.X), d(o.dX), a.dS_final, nullptr, s.nseg, s.nseg, N, a.L};
    prof_mark(kSlotLinearState, false, a.stream);
    hipLaunchKernelGGL(bwd_combine_kernel, dim3(cdiv(N, 1024), (unsigned)BH, 2), dim3(256), 0, a.stream, cs, cx);
    e = hipGetLastError();
    prof_mark(kSlotLinearState, true, a.stream);
    if (e != hipSuccess) return e;
  }
  // The last state is wanted only against its own gradient.
  float* last = a.dS_final ? f(o.S) + (size_t)s.nseg * N : nullptr;
  const bool shared = grp > 1;
  OutArgs q{{a.dO, 1}, {a.v, 1}, {a.k, grp}, {a.q, grp}, a.log_decay, f(o.S), a.S0,
            shared ? (void*)f(o.dq) : a.dq, last, (long long)(s.nseg + 1) * N, f(o.x), f(o.m), s.nseg + 1,
            a.L, BH, grp, s};
  OutArgs v{{a.k, grp}, {a.q, grp}, {a.dO, 1}, {nullptr, 1}, a.log_decay, f(o.X), a.dS_final,
            a.dv, a.dS0, N, nullptr, nullptr, s.nseg, a.L, BH, grp, s};
  OutArgs k{{a.v, 1}, {a.dO, 1}, {a.q, grp}, {a.k, grp}, a.log_decay, f(o.X), a.dS_final,
            shared ? (void*)f(o.dk) : a.dk, nullptr, 0, f(o.y), nullptr, s.nseg, a.L, BH, grp, s};
  constexpr int lds = walks_lds<IT, OT, DK, DV>();
  static_assert(lds <= (sizeof(IT) == 2 ? 80 : 160) * 1024, "two bf16 workgroups share a CU's LDS");
  const int n = (int)items(BH, grp, s.nseg);
  BorderArgs b{f(o.S), f(o.X), a.log_decay, d(o.border), a.L, N, s};
  const long long borders = a.dlog_decay ? (long long)BH * (s.nseg - 1) : 0;
  e = launch(&walks_kernel<IT, OT, DK, DV>, kSlotLinearBwd, 3LL * n + borders, walk_threads(DK, DV), lds, a.stream, q,
             k, v, n, b);
  if (e != hipSuccess) return e;
  if (!a.dlog_decay && !shared) return hipSuccess;
  DecayGradArgs g{a.log_decay, f(o.x), f(o.y), f(o.m), f(o.S), d(o.border), a.S0, a.dS0, a.dS_final, a.dlog_decay,
                  a.L, BH, N, s};
  const size_t per = (size_t)a.L * DK, total = shared ? (size_t)a.B * a.H_qk * per : 0;
  GroupSumArgs sum{f(o.dq), f(o.dk), a.dq, a.dk, per, total, grp};
  const int ng = a.dlog_decay ? BH * s.nseg : 0;
  const size_t sums = (2 * total / 4 + kGradThreads - 1) / kGradThreads;
  const long long blocks = ng + (long long)(sums < kSumBlocks ? sums : kSumBlocks);
  return launch(&finish_kernel<IT>, kSlotLinearBwd, blocks, kGradThreads, 0, a.stream, g, ng, sum);
}

template <int DK, int DV>
static hipError_t backward_d(const LinearBwdArgs& a) {
  if (a.in_dtype == 0) return backward<float, float, DK, DV>(a);
  return a.H == a.H_qk ? backward<bf16, bf16, DK, DV>(a) : backward<bf16, float, DK, DV>(a);
}

}  // namespace lin

size_t linear_bwd_workspace_bytes(int B, int H, int H_qk, int L, int d_k, int d_v, int in_dtype) {
  return L == 0 ? 0 : lin::bwd_ws(B, H, H_qk, L, d_k, d_v, in_dtype == 0).total;
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a) {
  if (a.L == 0)
    return a.dS0 && a.dS0 != a.dS_final
               ? lin::launch_copy_state(a.dS0, a.dS_final, (size_t)a.B * a.H * a.d_k * a.d_v, a.stream)
               : hipSuccess;
  if (a.d_k == 64 && a.d_v == 64) return lin::backward_d<64, 64>(a);
  if (a.d_k == 64 && a.d_v == 128) return lin::backward_d<64, 128>(a);
  if (a.d_k == 128 && a.d_v == 64) return lin::backward_d<128, 64>(a);
  return lin::backward_d<128, 128>(a);
}

}  // namespace dn
