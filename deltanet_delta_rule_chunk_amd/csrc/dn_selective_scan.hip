// dn_selective_scan.hip -- the selective state space scan's forward on gfx950,
// over sequences and for single tokens (the recurrence and a workgroup's tile: see
// dn_selective_scan.h).
//
// Few sequences of few channels do not fill the card: their sequences are cut
// into segments.  A first walk makes every segment's last state from zero and
// the sum of its dt (the decay over a segment is e^{A sum dt}), combine() turns
// them into the states in front of the segments, and the second walk makes the
// outputs.  Enough of them take one walk.

#include "dn_selective_scan.h"

namespace dn {
namespace ssm {

// ---- segments of packed sequences -----------------------------------------------------

// One workgroup.  Sequence i holds the rows from cu[i] to cu[i + 1]; whatever
// cu holds, begins and ends are brought into 0 .. L and never fall, so the rows
// of all segments lie in the tensors and their number is at most L / len + n_seq + 2.
__device__ __forceinline__ int pieces_of(int n, int len) { return n > 0 ? (n - 1) / len + 1 : 0; }
static __global__ __launch_bounds__(256) void segment_table_kernel(const int* cu, int n_seq, int L, int len, int* used,
                                                                   int* first_of, int4* table) {
  __shared__ int ends[256], counts[256];
  const int tid = threadIdx.x;
  int end = min(max(cu[0], 0), L);  // of the sequence before
  int at = pieces_of(end, len);     // segments so far: the rows in front of the first sequence
  for (int i = tid; i < at; i += 256) table[i] = make_int4(i * len, min(len, end - i * len), -1, 3);
  for (int base = 0; base < n_seq; base += 256) {
    const int i = base + tid;
    ends[tid] = i < n_seq ? min(max(cu[i + 1], 0), L) : 0;
    __syncthreads();
    for (int off = 1; off < 256; off <<= 1) {
      const int o = tid >= off ? ends[tid - off] : 0;
      __syncthreads();
      ends[tid] = max(ends[tid], o);
      __syncthreads();
    }
    const int my_end = max(ends[tid], end), begin = tid ? max(ends[tid - 1], end) : end;
    const int next_end = max(ends[255], end);
    const int n = my_end - begin, pieces = i < n_seq ? max(1, pieces_of(n, len)) : 0;
    counts[tid] = pieces;
    __syncthreads();
    for (int off = 1; off < 256; off <<= 1) {
      const int o = tid >= off ? counts[tid - off] : 0;
      __syncthreads();
      counts[tid] += o;
      __syncthreads();
    }
    const int first = at + counts[tid] - pieces;
    if (i < n_seq) first_of[i] = first;
    for (int p = 0; p < pieces; ++p)
      table[first + p] = make_int4(begin + p * len, min(len, n - p * len), i, (p == 0 ? 1 : 0) | (p == pieces - 1 ? 2 : 0));
    at += counts[255];
    end = next_end;
    __syncthreads();
  }
  const int behind = pieces_of(L - end, len);
  for (int i = tid; i < behind; i += 256) table[at + i] = make_int4(end + i * len, min(len, L - end - i * len), -1, 3);
  if (tid == 0) {
    first_of[n_seq] = at;
    *used = at + behind;
  }
}

hipError_t make_plan(const int* cu, int n_seq, int L, const Sizes& s, void* ws, hipStream_t stream, Plan* p) {
  *p = Plan{nullptr, nullptr, nullptr, s.len, s.per_row, L, (int)s.segments};
  if (!cu) return hipSuccess;
  int* ints = static_cast<int*>(ws);
  int4* table = reinterpret_cast<int4*>(ints + (n_seq + 2 + 3) / 4 * 4);
  hipLaunchKernelGGL(segment_table_kernel, dim3(1), dim3(256), 0, stream, cu, n_seq, L, s.len, ints, ints + 1, table);
  p->used = ints;
  p->first_of = ints + 1;
  p->table = table;
  return hipGetLastError();
}

// ---- states between segments -----------------------------------------------------------

// A thread takes one (sequence, channel, state) in one direction; loads of 8 segments
// are under way at a time.  Serial over a sequence's segments: 8 us for 32, 14 for 64, but 64 for 512
// (64 channels x 32768 tokens, whose walks take 11 and 16) and about 490 for 4096 (262144 tokens, walks
// of 51 and 67).
static __global__ __launch_bounds__(256) void combine_kernel(Plan pl, long long items, int DN, int N, const float* A,
                                                             const float* logs, const float* h0, float* ahead, float* back) {
  const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
  if (item >= items) return;
  const int seq = (int)(item / DN), e = (int)(item - (long long)seq * DN), d = e / N;
  const int D = DN / N;
  float* const x = blockIdx.y ? back : ahead;
  int s0, s1;
  segments_of(pl, seq, s0, s1);
  const int step = blockIdx.y ? -1 : 1;
  const int from = blockIdx.y ? s1 : s0, n = s1 - s0;
  const float a2 = A[e] * kLog2e;
  float carry = x[(size_t)from * DN + e];
  if (!blockIdx.y) x[(size_t)from * DN + e] = h0 ? h0[item] : 0.f;
  for (int i = 1; i <= n; i += 8) {
    float v[8], g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = from + step * min(i + j, n);
      const bool need = i + j < n;  // the last one's own part goes nowhere
      v[j] = need ? x[(size_t)s * DN + e] : 0.f;
      g[j] = need ? logs[(size_t)s * D + d] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j > n) break;
      x[(size_t)(from + step * (i + j)) * DN + e] = carry;
      carry = fmaf(exp2_fast(a2 * g[j]), carry, v[j]);
    }
  }
}

hipError_t combine(const Plan& p, int n_seq, int D, int N, const float* A, const float* logs, const float* h0, float* ahead,
                   float* back, hipStream_t stream) {
  const long long items = (long long)n_seq * D * N;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((items + 255) / 256), back ? 2 : 1), dim3(256), 0, stream, p, items,
                     D * N, N, A, logs, h0, ahead, back);
  return hipGetLastError();
}

// ---- the walk ----------------------------------------------------------------------------

// OUT: outputs from the states in front of the segments (`states`, or h0 where no
// sequence is cut).  Otherwise: each segment's last state and sum of dt.
template <int NW, typename T, bool GATE, bool OUT>
__global__ __launch_bounds__(64 * NW) void walk_kernel(ScanArgs a, Plan pl, int blocks_d, float* states, float* logs) {
  constexpr int N = 4 * NW, R = group_rows<T>();
  using At = Spot<NW>;
  __shared__ float2 sx[OUT ? 1 : 2][kTile][kCh];  // dt, dt u
  __shared__ float sy[OUT ? NW : 1][OUT ? kTile : 1][kCh];
  const int id = blockIdx.x / blocks_d, ch0 = (blockIdx.x - id * blocks_d) * kCh;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), ch = ch0 + lane;
  Segment g;
  if (!segment_of(pl, id, g)) return;
  const At at;
  const bool has = ch0 + at.c < a.D, on = ch < a.D;
  const int c = has ? ch0 + at.c : a.D - 4;
  T* y = static_cast<T*>(a.y) + ((size_t)g.batch * a.L + g.row) * a.D;  // of the tile
  if (g.seq < 0) {
    if (OUT && has)
      for (int r = at.r; r < g.n; r += At::kRows) put4(y + (size_t)r * a.D + c, zero4());
    return;
  }
  if (!OUT && g.last) return;  // nothing asks for its last state
  Feed<NW, T> u(a.u.p, g.batch * a.u.sb + g.row * a.u.sl, a.u.sl, at, c);
  Feed<NW, T> dt(a.dt.p, g.batch * a.dt.sb + g.row * a.dt.sl, a.dt.sl, at, c);
  Feed<NW, T> z(a.z.p, g.batch * a.z.sb + g.row * a.z.sl, a.z.sl, at, c);
  const T* Bt = static_cast<const T*>(a.Bm.p) + g.batch * a.Bm.sb + g.row * a.Bm.sl + 4 * w;  // of the tile
  const T* Ct = static_cast<const T*>(a.Cm.p) + g.batch * a.Cm.sb + g.row * a.Cm.sl + 4 * w;
  const f32x4 bias = a.dt_bias ? get4(a.dt_bias + c) : zero4();
  const f32x4 skip = OUT && a.skip ? get4(a.skip + c) : zero4();
  f32x4 A2 = zero4(), h = zero4();
  if (on) {
    A2 = get4(a.A + (size_t)ch * N + 4 * w) * kLog2e;
    // (With cut sequences h0 is not read here: it may be where hT goes.)
    const float* from = OUT && logs ? states + (size_t)id * a.D * N : g.first && a.h0 ? a.h0 + (size_t)g.seq * a.D * N : nullptr;
    if (from) h = get4(from + (size_t)ch * N + 4 * w);
  }
  float sum = 0.f;
  Ahead<NW, T> nB(a.Bm.p, g.batch * a.Bm.sb + g.row * a.Bm.sl, a.Bm.sl), nC(a.Cm.p, g.batch * a.Cm.sb + g.row * a.Cm.sl, a.Cm.sl);
  const auto fetch = [&](int n) {
    if (n <= 0) return;
    u.fetch(at, c, n);
    dt.fetch(at, c, n);
    if (OUT && GATE) z.fetch(at, c, n);
    nB.fetch(n);
    if (OUT) nC.fetch(n);
  };
  fetch(g.n);
  int buf = 0;
  for (int left = g.n; left > 0; left -= kTile) {
    Raw4<T> uu[At::kPasses], zz[At::kPasses];
    if (at.in_tile()) {
#pragma unroll
      for (int p = 0; p < At::kPasses; ++p) {
        uu[p] = u.raw[p];
        if (OUT && GATE) zz[p] = z.raw[p];
        const f32x4 d = softplus4(wide(dt.raw[p]) + bias, a.softplus), x = d * wide(uu[p]);
        f32x4* const out = reinterpret_cast<f32x4*>(&sx[buf][at.row(p)][at.c]);
        out[0] = f32x4{d[0], x[0], d[1], x[1]};
        out[1] = f32x4{d[2], x[2], d[3], x[3]};
      }
    }
    nB.arrived();
    if (OUT) nC.arrived();
    u.move(1);
    dt.move(1);
    if (OUT && GATE) z.move(1);
    nB.move(1);
    if (OUT) nC.move(1);
    fetch(left - kTile);
    float part = 0.f;
    const auto step = [&](int t, f32x4 b, f32x4 cc, float2 x) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(exp2_fast(x.x * A2[i]), h[i], x.y * b[i]);
        if (OUT) s = fmaf(h[i], cc[i], s);
      }
      if (OUT) sy[w][t][lane] = s;
      else part += x.x;
    };
    if (left >= kTile) {
      Group<T> gb[2], gc[2];
      float2 x[2][R];
      gb[0].load(Bt, a.Bm.sl);
      if (OUT) gc[0].load(Ct, a.Cm.sl);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < R; ++i) x[0][i] = sx[buf][i][lane];
      wait_reads();
#pragma unroll
      for (int q = 0; q < kTile / R; ++q) {
        const int now = q & 1, next = now ^ 1;
        if (q + 1 < kTile / R) {
          gb[next].load(Bt + (q + 1) * R * a.Bm.sl, a.Bm.sl);
          if (OUT) gc[next].load(Ct + (q + 1) * R * a.Cm.sl, a.Cm.sl);
#pragma unroll
          for (int i = 0; i < R; ++i) x[next][i] = sx[buf][(q + 1) * R + i][lane];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < R; ++i) step(q * R + i, wide(gb[now].r[i]), OUT ? wide(gc[now].r[i]) : zero4(), x[now][i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      __syncthreads();
      for (int t = 0; t < left; ++t)
        step(t, wide(uniform4(Bt + t * a.Bm.sl)), OUT ? wide(uniform4(Ct + t * a.Cm.sl)) : zero4(), sx[buf][t][lane]);
    }
    Bt += kTile * a.Bm.sl;
    Ct += kTile * a.Cm.sl;
    sum += part;
    if (OUT) {
      __syncthreads();
      if (at.in_tile()) {
#pragma unroll
        for (int p = 0; p < At::kPasses; ++p) {
          const int r = at.row(p);
          f32x4 s = skip * wide(uu[p]);
#pragma unroll
          for (int i = 0; i < NW; ++i) s += get4(&sy[i][r][at.c]);
          if (GATE) {
            const f32x4 v = wide(zz[p]);
            s *= v * sigmoid4(v);
          }
          if (has && r < left) put4(const_cast<T*>(at_bytes(y, offset_of<T>(r, a.D, c))), s);
        }
      }
      y += (size_t)kTile * a.D;
    } else {
      buf ^= 1;
    }
  }
  if (!on) return;
  float* to = nullptr;
  if (OUT) {
    if (g.last && a.hT) to = a.hT + (size_t)g.seq * a.D * N;
  } else {
    to = states + (size_t)id * a.D * N;
    if (w == 0) logs[(size_t)id * a.D + ch] = sum;
  }
  if (to) *reinterpret_cast<f32x4*>(to + (size_t)ch * N + 4 * w) = h;
}

// 512 workgroups need no cut (bf16, 32 x 2048 tokens of 1024 channels, 512 of them: 354 us uncut,
// 402 cut; 384 of them 349 and 323; 256, 1024 tokens: 145 and 121), and short sequences
// need it later the more there are (256 tokens of 1024 channels: 16 of them, 256 workgroups, 41 us
// uncut, 42 cut; 8 of them 41 and 31; one 40 and 18).  With a cut, 4096: 65536 tokens of 4096
// channels take 1974 us with 1024, 1765 with 1536, 1710 with 2048, 1630 with 4096, 1604 with 8192,
// which costs shorter sequences as much.  Pieces: 512 tokens of 1024 channels, 26 us in pieces
// of 64, 23 of 48, 21 of 32, 22 of 16; 128 of them 26, 22, 20 and 17; 8192 of 768, 69, 74 and 83
// of 64, 48, 32.  All of these are of batches of equal sequences, with 16 states.  With 8 states a workgroup
// has half the waves and the cut ends too early: 16 x 1024 tokens of 2048 channels, 512 workgroups, 193 us, 8 of
// them, cut, 87 (16 states: 177 and 112; 32: 254 and 200).  Packed sequences are cut as one long one: 32 of
// 1024 tokens, 1024 channels, 230 us, as a batch, uncut, 178; 24 of 4096, 2048 channels, 1171 and 883.
static Sizes forward_sizes(int B, int L, int D, bool packed, int n_seq) {
  return sizes_of(packed, B, L, n_seq, D, {512, 4096, 640, 80, 1});
}

template <int NW, typename T, bool GATE>
static hipError_t forward(const ScanArgs& a) {
  const Sizes s = forward_sizes(a.B, a.L, a.D, a.cu, a.n_seq);
  const int blocks_d = (int)channel_blocks(a.D);
  char* ws = static_cast<char*>(a.workspace);
  Plan p;
  prof_mark(kSlotSelectiveScan, false, a.stream);
  hipError_t e = make_plan(a.cu, a.n_seq, a.L, s, ws, a.stream, &p);
  ws += table_bytes(a.cu, a.n_seq, s);
  float* states = reinterpret_cast<float*>(ws);
  float* logs = s.split ? states + (size_t)s.segments * a.D * a.N : nullptr;
  const dim3 grid((unsigned)(s.segments * blocks_d));
  if (e == hipSuccess && s.split) {
    hipLaunchKernelGGL((walk_kernel<NW, T, GATE, false>), grid, dim3(64 * NW), 0, a.stream, a, p, blocks_d, states, logs);
    e = hipGetLastError();
    if (e == hipSuccess) e = combine(p, a.n_seq, a.D, a.N, a.A, logs, a.h0, states, nullptr, a.stream);
  }
  if (e == hipSuccess) {
    hipLaunchKernelGGL((walk_kernel<NW, T, GATE, true>), grid, dim3(64 * NW), 0, a.stream, a, p, blocks_d, states, logs);
    e = hipGetLastError();
  }
  prof_mark(kSlotSelectiveScan, true, a.stream);
  return e;
}

template <int NW>
static hipError_t forward_t(const ScanArgs& a) {
  if (a.dtype == 1) return a.z.p ? forward<NW, bf16, true>(a) : forward<NW, bf16, false>(a);
  return a.z.p ? forward<NW, float, true>(a) : forward<NW, float, false>(a);
}

// ---- one token ---------------------------------------------------------------------------

// Bound by HBM: the state is read and written once (256 x 4096 x 16 in 26 us, 5.4 TB/s).  A
// lane takes 4 states of a
// channel; N / 4 adjacent lanes add up their channel's y.
template <int N, typename T>
__global__ __launch_bounds__(256) void step_kernel(ScanArgs a, long long items) {
  constexpr int Q = N / 4;
  const long long item = (long long)blockIdx.x * 256 + threadIdx.x;
  if (item >= items) return;  // (whole channels: D is a multiple of 8)
  const int q = (int)(item % Q);
  const long long bd = item / Q;
  const int b = (int)(bd / a.D), d = (int)(bd - (long long)b * a.D);
  float* const hp = a.hT + item * 4;
  f32x4 h = get4(hp);
  const f32x4 A2 = get4(a.A + (size_t)d * N + 4 * q) * kLog2e;
  const f32x4 Bq = wide(raw4(static_cast<const T*>(a.Bm.p) + b * a.Bm.sb + 4 * q));
  const f32x4 Cq = wide(raw4(static_cast<const T*>(a.Cm.p) + b * a.Cm.sb + 4 * q));
  const float u = to_f32(static_cast<const T*>(a.u.p)[b * a.u.sb + d]);
  float dt = to_f32(static_cast<const T*>(a.dt.p)[b * a.dt.sb + d]) + (a.dt_bias ? a.dt_bias[d] : 0.f);
  if (a.softplus) dt = softplus(dt);
  const float x = dt * u;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], x * Bq[i]);
    y = fmaf(h[i], Cq[i], y);
  }
  __builtin_nontemporal_store(h, reinterpret_cast<f32x4*>(hp));
#pragma unroll
  for (int off = Q / 2; off > 0; off >>= 1) y += __shfl_xor(y, off, 64);
  if (q == 0) {
    if (a.skip) y = fmaf(a.skip[d], u, y);
    if (a.z.p) {
      const float z = to_f32(static_cast<const T*>(a.z.p)[b * a.z.sb + d]);
      y *= z * sigmoid(z);
    }
    static_cast<T*>(a.y)[bd] = from_f32<T>(y);
  }
}

template <int N, typename T>
static hipError_t step(const ScanArgs& a) {
  const long long items = (long long)a.B * a.D * (N / 4);
  prof_mark(kSlotSelectiveStep, false, a.stream);
  hipLaunchKernelGGL((step_kernel<N, T>), dim3((unsigned)((items + 255) / 256)), dim3(256), 0, a.stream, a, items);
  const hipError_t e = hipGetLastError();
  prof_mark(kSlotSelectiveStep, true, a.stream);
  return e;
}

}  // namespace ssm

// Whether the launches hold these sizes.
bool selective_scan_fits(int B, int L, int D, int N, bool packed, int n_seq, bool backward) {
  const long long D64 = ssm::channel_blocks(D), states = (long long)D * N;
  if (L > 0x7fffffff - 64 || states > 0x7fffffff || (packed && n_seq > (1 << 24))) return false;
  const ssm::Sizes s = backward ? ssm::backward_sizes(B, L, D, packed, n_seq) : ssm::forward_sizes(B, L, D, packed, n_seq);
  if (s.segments > max_blocks(16 * N) / D64 || (long long)n_seq > max_blocks(256) * 256 / states) return false;
  // (The gradient's last two launches: 1024 values of dB and dC, 16 columns of dA, dD and the bias's gradient per workgroup.)
  return !backward || ((long long)B * L <= max_blocks(256) * 1024 / N && states + 2LL * D <= max_blocks(256) * 16);
}

size_t selective_scan_workspace_bytes(int B, int L, int D, int N, bool packed, int n_seq) {
  const ssm::Sizes s = ssm::forward_sizes(B, L, D, packed, n_seq);
  const size_t table = ssm::table_bytes(packed, n_seq, s);
  return s.split ? table + (size_t)s.segments * D * (N + 1) * sizeof(float) : table;
}

hipError_t launch_selective_scan(const ScanArgs& a) {
  return a.N == 8 ? ssm::forward_t<2>(a) : a.N == 16 ? ssm::forward_t<4>(a) : ssm::forward_t<8>(a);
}

hipError_t launch_selective_scan_step(const ScanArgs& a) {
  if (a.dtype == 1) return a.N == 8 ? ssm::step<8, bf16>(a) : a.N == 16 ? ssm::step<16, bf16>(a) : ssm::step<32, bf16>(a);
  return a.N == 8 ? ssm::step<8, float>(a) : a.N == 16 ? ssm::step<16, float>(a) : ssm::step<32, float>(a);
}

}  // namespace dn
