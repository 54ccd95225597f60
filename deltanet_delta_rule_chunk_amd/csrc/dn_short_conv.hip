// dn_short_conv.hip -- short causal convolution of every channel on gfx950, its
// gradient, and one token with the kept rows updated in place.
//
// With x_e the K - 1 rows kept from before a sequence followed by its rows,
//     p_t = b + sum_j w[j] x_e[t + j],  y_t = silu(p_t) (or p_t),  j = 0 .. K - 1,
// and the rows kept behind it are x_e's last K - 1.  With q_t = dy_t silu'(p_t),
//     dx_e[i] = sum_j w[j] q_{i - j} (+ the kept rows' gradient),
//     dw[j] = sum_t q_t x_e[t + j],   db = sum_t q_t.
//
// Bound by HBM: x is read and y written once (65536 tokens of 4096 bf16 channels: 195 to 213
// us, 5.0 to 5.5 TB/s; the gradient reads x and dy and writes dx in 364 to 450, 3.6 to 4.4 TB/s; fp32
// 376 and 670 us, 5.7 and 4.8 TB/s).  A thread walks down a run of
// rows of its channels with the last K - 1 of them in registers; neighbouring
// threads hold neighbouring channels, so every load is a whole piece of a row.
// Where packed sequences meet inside a run, the registers take the new sequence's
// kept rows.  Rows that no sequence holds give zeros.

#include "dn_launch.h"
#include "dn_vec.h"

namespace dn {
namespace conv {

constexpr int NT = 256;

// A sequence, or rows that are in none (seq < 0 or >= n), from begin to end.
struct Place {
  int n, batch;
  int seq, begin, end;
  bool packed;
  __device__ __forceinline__ bool inside() const { return !packed || (seq >= 0 && seq < n); }
};
// The whole of sequence `seq`.
__device__ __forceinline__ Place sequence(const ShortConvArgs& a, int seq) {
  Place s{a.n_seq, a.cu ? 0 : seq, seq, 0, a.L, a.cu != nullptr};
  if (a.cu) {
    s.begin = min(max(a.cu[seq], 0), a.L);
    s.end = min(max(a.cu[seq + 1], s.begin), a.L);
  }
  return s;
}

// The sequences' cuts, in LDS where they fit: a search in memory is a chain of loads
// (7 prompts in 6001 rows of 2304 channels: 21.9 us in memory, 19.0 in LDS).  The two are
// never one pointer: a generic address into LDS may not start below it, which `cut + 1`
// as an offset would have it do.
constexpr int kCuts = 512;
struct Cuts {
  const int* cu;
  int n, L;
  bool at_hand;
  // Every thread of the workgroup calls this.
  __device__ __forceinline__ Cuts(const ShortConvArgs& a, int (&lds)[kCuts]) : cu(a.cu), n(a.n_seq), L(a.L) {
    at_hand = cu && n < kCuts;
    if (at_hand) {
      for (int i = threadIdx.x; i <= n; i += NT) lds[i] = cu[i];
      __syncthreads();
    }
  }
  __device__ __forceinline__ int cut(const int (&lds)[kCuts], int i) const {
    typedef const __attribute__((address_space(3))) int* local_ptr;
    typedef const __attribute__((address_space(1))) int* global_ptr;
    return at_hand ? ((local_ptr)lds)[i] : ((global_ptr)(uintptr_t)cu)[i];
  }
  __device__ __forceinline__ Place find(const int (&lds)[kCuts], int batch, int row) const {
    if (!cu) return Place{n, batch, batch, 0, L, false};
    int lo = 0, hi = n + 1;  // as many cuts, at least and at most, are not behind the row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (cut(lds, mid) <= row) lo = mid + 1;
      else hi = mid;
    }
    const int begin = lo > 0 ? cut(lds, lo - 1) : 0, end = lo <= n ? cut(lds, lo) : L;
    // Whatever the cuts are, the row is between the two.
    return Place{n, batch, lo - 1, min(max(begin, 0), row), min(max(end, row + 1), L), true};
  }
};

template <int V> struct Vals { f32x4 v[V / 4]; };
template <int V>
__device__ __forceinline__ Vals<V> zeros() {
  Vals<V> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) r.v[i] = zero4();
  return r;
}
template <int V, typename T>
struct Raws { Raw4<T> v[V / 4]; };
template <int V, typename T>
__device__ __forceinline__ Raws<V, T> load(const T* p) {
  Raws<V, T> r;
  __builtin_memcpy(&r, __builtin_assume_aligned(p, V * sizeof(T)), sizeof(r));
  return r;
}
template <int V, typename T>
__device__ __forceinline__ Raws<V, T> none() {
  Raws<V, T> r;
  __builtin_memset(&r, 0, sizeof(r));
  return r;
}
template <int V, typename T>
__device__ __forceinline__ void store(T* p, const Raws<V, T>& r) {
  __builtin_memcpy(__builtin_assume_aligned(p, V * sizeof(T)), &r, sizeof(r));
}
template <int V, typename T>
__device__ __forceinline__ Vals<V> widen(const Raws<V, T>& r) {
  Vals<V> x;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) x.v[i] = wide(r.v[i]);
  return x;
}
template <int V, typename T>
__device__ __forceinline__ Raws<V, T> narrowed(const Vals<V>& x) {
  Raws<V, T> r;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) r.v[i] = narrow<T>(x.v[i]);
  return r;
}

// Weights of V channels, tap by tap.
template <int V, int K>
struct Taps {
  Vals<V> w[K], b;
  __device__ __forceinline__ Taps(const float* weight, const float* bias, int c) {
    float t[V * K];
    __builtin_memcpy(t, __builtin_assume_aligned(weight + (size_t)c * K, 16), sizeof(t));
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) w[j].v[i / 4][i % 4] = t[i * K + j];
    b = zeros<V>();
    if (bias)
#pragma unroll
      for (int i = 0; i < V / 4; ++i) b.v[i] = *reinterpret_cast<const f32x4*>(bias + c + 4 * i);
  }
};
template <int V>
__device__ __forceinline__ void add_product(Vals<V>& a, const Vals<V>& x, const Vals<V>& y) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) a.v[i] += x.v[i] * y.v[i];
}
// The tap sums in front of the activation; past[K - 2] is the row before.
template <int V, int K>
__device__ __forceinline__ Vals<V> pre(const Taps<V, K>& t, const Vals<V> (&past)[K - 1], const Vals<V>& x) {
  Vals<V> p = t.b;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) add_product(p, t.w[j], past[j]);
  add_product(p, t.w[K - 1], x);
  return p;
}
template <int V, int K>
__device__ __forceinline__ void push(Vals<V> (&past)[K], const Vals<V>& x) {
#pragma unroll
  for (int j = 0; j + 1 < K; ++j) past[j] = past[j + 1];
  past[K - 1] = x;
}

// Row `t` of the sequence's extended rows (t may lie up to K - 1 before its begin).
template <int V, typename T>
__device__ __forceinline__ Raws<V, T> row_of(const ShortConvArgs& a, const Place& s, int t, int c) {
  if (!s.inside()) return none<V, T>();
  if (t >= s.begin) return load<V>(static_cast<const T*>(a.x.p) + s.batch * a.x.sb + t * a.x.sl + c);
  const int kept = a.K - 1 + t - s.begin;
  if (!a.state0 || kept < 0) return none<V, T>();
  return load<V>(static_cast<const T*>(a.state0) + ((size_t)s.seq * (a.K - 1) + kept) * a.D + c);
}
template <int V, int K, typename T>
__device__ __forceinline__ void enter(const ShortConvArgs& a, const Place& s, int t, int c, Vals<V> (&past)[K - 1]) {
#pragma unroll
  for (int j = 0; j < K - 1; ++j) past[j] = widen<V>(row_of<V, T>(a, s, t - (K - 1) + j, c));
}

// A run of R rows of V channels per thread.  The workgroups behind `runs` copy the
// kept rows.
template <int K, int V, int R, typename T>
__global__ __launch_bounds__(NT) void forward_kernel(ShortConvArgs a, int per_row, long long run_items, unsigned run_blocks) {
  __shared__ int cuts[kCuts];
  const int groups = a.D / V;
  if (blockIdx.x >= run_blocks) {
    // One (sequence, kept row, channels) per thread.
    const long long item = (long long)(blockIdx.x - run_blocks) * NT + threadIdx.x;
    if (item >= (long long)a.n_seq * (K - 1) * groups) return;
    const long long row = item / groups;
    const int c = (int)(item - row * groups) * V, seq = (int)(row / (K - 1)), j = (int)(row - (long long)seq * (K - 1));
    const Place s = sequence(a, seq);
    store<V>(static_cast<T*>(a.state) + row * a.D + c, row_of<V, T>(a, s, s.end - (K - 1) + j, c));
    return;
  }
  const long long item = (long long)blockIdx.x * NT + threadIdx.x;
  const bool on = item < run_items;
  const long long run = on ? item / groups : 0;
  const int c = on ? (int)(item - run * groups) * V : 0;
  const int b = (int)(run / per_row), t0 = (int)(run - (long long)b * per_row) * R, t1 = min(t0 + R, a.L);
  const T* const x = static_cast<const T*>(a.x.p) + b * a.x.sb + c;
  T* const y = static_cast<T*>(a.y) + (size_t)b * a.L * a.D + c;
  Raws<V, T> rows[R];
#pragma unroll
  for (int i = 0; i < R; ++i) rows[i] = load<V>(x + min(t0 + i, t1 - 1) * a.x.sl);
  const Taps<V, K> taps(a.weight, a.bias, c);
  const Cuts cu(a, cuts);
  Place s = cu.find(cuts, b, t0);
  if (!on) return;
  Vals<V> past[K - 1];
  enter<V, K, T>(a, s, t0, c, past);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = t0 + i;
    if (t >= t1) break;
    if (a.cu && t >= s.end) {
      s = cu.find(cuts, b, t);
      enter<V, K, T>(a, s, t, c, past);
    }
    const Vals<V> xt = widen<V>(rows[i]);
    Vals<V> p = pre<V, K>(taps, past, xt);
    push(past, xt);
    if (a.silu)
#pragma unroll
      for (int k = 0; k < V; ++k) p.v[k / 4][k % 4] *= sigmoid(p.v[k / 4][k % 4]);
    if (!s.inside()) p = zeros<V>();
    store<V>(y + (size_t)t * a.D, narrowed<V, T>(p));
  }
}

// ---- gradient ------------------------------------------------------------------------

constexpr int BV = 4;  // channels per thread

// dy silu'(p)
__device__ __forceinline__ Vals<BV> through(const Vals<BV>& p, const Vals<BV>& dy, int silu) {
  if (!silu) return dy;
  Vals<BV> q;
#pragma unroll
  for (int k = 0; k < BV; ++k) {
    const float v = p.v[0][k], s = sigmoid(v);
    q.v[0][k] = dy.v[0][k] * (s * (1.f + v * (1.f - s)));
  }
  return q;
}

constexpr int WAVES = NT / 64;

// A wave takes 64 groups of channels and a run of `len` rows, walked K - 1 rows
// further for the q that reach back into it; the workgroup's waves take runs that
// follow each other and add up dw and db, which go to `parts` [workgroup's runs][K + 1][D].
// The workgroups behind `run_blocks` form the gradients of the kept rows in front of
// sequences.
template <int K, typename T>
__global__ __launch_bounds__(NT) void backward_kernel(ShortConvArgs a, int len, int per_row, long long runs, int blocks_d,
                                                      unsigned run_blocks, float* parts) {
  __shared__ f32x4 sums[WAVES][K + 1][64];
  __shared__ int cuts[kCuts];
  const int groups = a.D / BV;
  if (blockIdx.x >= run_blocks) {
    const long long item = (long long)(blockIdx.x - run_blocks) * NT + threadIdx.x;
    if (item >= (long long)a.n_seq * groups) return;
    const int seq = (int)(item / groups), c = (int)(item - (long long)seq * groups) * BV;
    const Place s = sequence(a, seq);
    const int n = s.end - s.begin;
    const Taps<BV, K> taps(a.weight, a.bias, c);
    Vals<BV> past[K - 1], d[K - 1];
    enter<BV, K, T>(a, s, s.begin, c, past);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      d[j] = zeros<BV>();
      // A kept row that is still kept behind a short sequence.
      if (a.dstate && j >= n) d[j] = widen<BV>(load<BV>(static_cast<const T*>(a.dstate) + ((size_t)seq * (K - 1) + j - n) * a.D + c));
    }
    const T* const dy = static_cast<const T*>(a.dy) + (size_t)s.batch * a.L * a.D + c;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      if (i >= n) break;
      const Vals<BV> x = widen<BV>(row_of<BV, T>(a, s, s.begin + i, c));
      const Vals<BV> q = through(pre<BV, K>(taps, past, x), widen<BV>(load<BV>(dy + (size_t)(s.begin + i) * a.D)), a.silu);
      push(past, x);
      // q_i reads kept rows i .. K - 2 with taps 0 .. K - 2 - i.
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        if (i + j < K - 1) add_product(d[i + j], taps.w[j], q);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      store<BV>(static_cast<T*>(a.dstate0) + ((size_t)seq * (K - 1) + j) * a.D + c, narrowed<BV, T>(d[j]));
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const long long set = blockIdx.x / blocks_d, run = set * WAVES + wave;
  const int group = (int)(blockIdx.x - set * blocks_d) * 64 + lane;
  const bool on = group < groups && run < runs;
  const int c = (group < groups ? group : groups - 1) * BV;
  const long long r0 = run < runs ? run : 0;
  const int b = (int)(r0 / per_row), t0 = (int)(r0 - (long long)b * per_row) * len, t1 = on ? min(t0 + len, a.L) : t0;
  const int stop = min(t0 + len + K - 1, a.L);  // (not below t0 + 1)
  const T* const x = static_cast<const T*>(a.x.p) + b * a.x.sb + c;
  const T* const dy = static_cast<const T*>(a.dy) + (size_t)b * a.L * a.D + c;
  T* const dx = static_cast<T*>(a.dx) + (size_t)b * a.L * a.D + c;
  const Taps<BV, K> taps(a.weight, a.bias, c);
  const Cuts cu(a, cuts);
  Place s = cu.find(cuts, b, t0);  // of the row whose q is formed
  Place o = s;                         // of the row whose dx is finished
  Vals<BV> past[K - 1], q[K], dw[K], db = zeros<BV>();
  enter<BV, K, T>(a, s, t0, c, past);
#pragma unroll
  for (int j = 0; j < K; ++j) q[j] = dw[j] = zeros<BV>();
  constexpr int U = 4;  // rows whose loads are under way
  Raws<BV, T> rx[U], ry[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int t = min(t0 + i, stop - 1);
    rx[i] = load<BV>(x + t * a.x.sl);
    ry[i] = load<BV>(dy + (size_t)t * a.D);
  }
  // Row t forms q_t and finishes dx of row t - K + 1.
  for (int base = t0; base < t1 + K - 1 && t1 > t0; base += U) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int t = base + i;
      const Vals<BV> xt = widen<BV>(rx[i]), dyt = widen<BV>(ry[i]);
      const int ahead = min(t + U, stop - 1);
      rx[i] = load<BV>(x + ahead * a.x.sl);
      ry[i] = load<BV>(dy + (size_t)ahead * a.D);
      Vals<BV> qt = zeros<BV>();
      if (t < stop) {
        if (a.cu && t >= s.end) {
          s = cu.find(cuts, b, t);
          enter<BV, K, T>(a, s, t, c, past);
        }
        if (s.inside()) {
          qt = through(pre<BV, K>(taps, past, xt), dyt, a.silu);
          if (t < t1) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) add_product(dw[j], past[j], qt);
            add_product(dw[K - 1], xt, qt);
            db.v[0] += qt.v[0];
          }
        }
        push(past, xt);
      }
      push(q, qt);
      const int r = t - (K - 1);
      if (r >= t0 && r < t1) {
        if (a.cu && r >= o.end) o = cu.find(cuts, b, r);
        Vals<BV> d = zeros<BV>();
        if (o.inside()) {
          // q[j] is of row r + j, which reads row r with tap K - 1 - j.
#pragma unroll
          for (int j = 0; j < K; ++j)
            if (r + j < o.end) add_product(d, taps.w[K - 1 - j], q[j]);
          const int kept = r - (o.end - (K - 1));
          if (a.dstate && kept >= 0) {
            const Vals<BV> e = widen<BV>(load<BV>(static_cast<const T*>(a.dstate) + ((size_t)o.seq * (K - 1) + kept) * a.D + c));
            d.v[0] += e.v[0];
          }
        }
        store<BV>(dx + (size_t)r * a.D, narrowed<BV, T>(d));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) sums[wave][j][lane] = dw[j].v[0];
  sums[wave][K][lane] = db.v[0];
  __syncthreads();
  if (group >= groups) return;
  for (int j = wave; j < K + 1; j += WAVES) {
    f32x4 s = sums[0][j][lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) s += sums[i][j][lane];
    *reinterpret_cast<f32x4*>(parts + ((size_t)set * (K + 1) + j) * a.D + c) = s;
  }
}

// The parts [runs][K + 1][D] added in order, 16 columns per workgroup.
static __global__ __launch_bounds__(NT) void weight_kernel(const float* parts, int runs, int D, int K, float* dweight, float* dbias) {
  __shared__ double red[16][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + c, columns = (K + 1) * D;
  double s = 0.0;
  if (e < columns) {
#pragma unroll 8
    for (int i = r; i < runs; i += 16) s += (double)parts[(size_t)i * columns + e];
  }
  red[r][c] = s;
  __syncthreads();
  if (r || e >= columns) return;
  for (int i = 1; i < 16; ++i) s += red[i][c];
  const int j = e / D, d = e - j * D;
  if (j < K) dweight[(size_t)d * K + j] = (float)s;
  else if (dbias) dbias[d] = (float)s;
}

// ---- one token ------------------------------------------------------------------------

template <int K, int V, typename T>
__global__ __launch_bounds__(NT) void step_kernel(ShortConvArgs a, long long items) {
  const long long item = (long long)blockIdx.x * NT + threadIdx.x;
  if (item >= items) return;
  const int groups = a.D / V, b = (int)(item / groups), c = (int)(item - (long long)b * groups) * V;
  T* const kept = static_cast<T*>(a.state) + (size_t)b * (K - 1) * a.D + c;
  const Raws<V, T> x = load<V>(static_cast<const T*>(a.x.p) + b * a.x.sb + c);
  Raws<V, T> rows[K - 1];
  Vals<V> past[K - 1];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) rows[j] = load<V>(kept + (size_t)j * a.D);
  const Taps<V, K> taps(a.weight, a.bias, c);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) past[j] = widen<V>(rows[j]);
  Vals<V> p = pre<V, K>(taps, past, widen<V>(x));
  if (a.silu)
#pragma unroll
    for (int k = 0; k < V; ++k) p.v[k / 4][k % 4] *= sigmoid(p.v[k / 4][k % 4]);
#pragma unroll
  for (int j = 0; j + 1 < K - 1; ++j) store<V>(kept + (size_t)j * a.D, rows[j + 1]);
  store<V>(kept + (size_t)(K - 2) * a.D, x);
  store<V>(static_cast<T*>(a.y) + (size_t)b * a.D + c, narrowed<V, T>(p));
}

// ---- launches -------------------------------------------------------------------------

// Rows per run of the forward, of which each re-reads K - 1: 16, or 8 where runs of 16
// would be fewer than 4 workgroups per CU (between two events, 500 x 2048 channels: 8.4 us
// against 10.4, 4 x 512: 9.1 against 12.1, 4 x 2048: 19.0 and 18.9; runs of 4: no less).
constexpr int kRun = 16, kShortRun = 8, kFewBlocks = 1024;

static unsigned blocks_for(long long items) { return (unsigned)((items + NT - 1) / NT); }

template <int K, int R, typename T>
static hipError_t forward_run(const ShortConvArgs& a) {
  constexpr int V = 16 / sizeof(T);
  const int per_row = (int)(((long long)a.L + R - 1) / R);
  const long long items = (long long)a.B * per_row * (a.D / V), kept = a.state ? (long long)a.n_seq * (K - 1) * (a.D / V) : 0;
  const unsigned n = blocks_for(items), m = blocks_for(kept);
  if (n + m == 0) return hipSuccess;
  prof_mark(kSlotShortConv, false, a.stream);
  hipLaunchKernelGGL((forward_kernel<K, V, R, T>), dim3(n + m), dim3(NT), 0, a.stream, a, per_row, items, n);
  const hipError_t e = hipGetLastError();
  prof_mark(kSlotShortConv, true, a.stream);
  return e;
}
template <int K, typename T>
static hipError_t forward(const ShortConvArgs& a) {
  const bool few = (long long)a.B * a.L * a.D * (int)sizeof(T) < kFewBlocks * kRun * 16LL * NT;
  return few ? forward_run<K, kShortRun, T>(a) : forward_run<K, kRun, T>(a);
}

// Rows per run of the backward: 8192 waves, runs of 16 to 64 rows.
struct Runs {
  int len, per_row, blocks_d;
  long long n, sets;  // runs, and sets of them that a workgroup adds up
};
static Runs backward_runs(int B, int L, int D) {
  Runs r;
  r.blocks_d = (D / BV + 63) / 64;
  long long len = (long long)B * L * r.blocks_d / 8192;
  len = len < 16 ? 16 : len > 64 ? 64 : len;
  r.len = (int)len;
  r.per_row = (int)((L + len - 1) / len);
  r.n = (long long)B * r.per_row;
  r.sets = (r.n + WAVES - 1) / WAVES;
  return r;
}

template <int K, typename T>
static hipError_t backward(const ShortConvArgs& a) {
  const Runs r = backward_runs(a.B, a.L, a.D);
  const unsigned n = (unsigned)(r.sets * r.blocks_d), m = a.dstate0 ? blocks_for((long long)a.n_seq * (a.D / BV)) : 0;
  float* const parts = static_cast<float*>(a.workspace);
  prof_mark(kSlotShortConvBwd, false, a.stream);
  hipError_t e = hipSuccess;
  if (n + m > 0) {
    hipLaunchKernelGGL((backward_kernel<K, T>), dim3(n + m), dim3(NT), 0, a.stream, a, r.len, r.per_row, r.n, r.blocks_d, n, parts);
    e = hipGetLastError();
  }
  if (e == hipSuccess) {
    hipLaunchKernelGGL(weight_kernel, dim3((unsigned)(((K + 1) * a.D + 15) / 16)), dim3(NT), 0, a.stream, parts, (int)r.sets, a.D,
                       K, a.dweight, a.dbias);
    e = hipGetLastError();
  }
  prof_mark(kSlotShortConvBwd, true, a.stream);
  return e;
}

template <int K, typename T>
static hipError_t step(const ShortConvArgs& a) {
  constexpr int V = 16 / sizeof(T);
  const long long items = (long long)a.B * (a.D / V);
  prof_mark(kSlotShortConv, false, a.stream);
  hipLaunchKernelGGL((step_kernel<K, V, T>), dim3(blocks_for(items)), dim3(NT), 0, a.stream, a, items);
  const hipError_t e = hipGetLastError();
  prof_mark(kSlotShortConv, true, a.stream);
  return e;
}

}  // namespace conv

// Whether the forward's and backward's launches hold these sizes.
bool short_conv_fits(int B, int L, int D, int n_seq, int dtype) {
  const long long v = dtype == 1 ? 8 : 4, most = max_blocks(conv::NT) - 1;
  const long long runs = (long long)B * (((long long)L + conv::kRun - 1) / conv::kRun);
  // (Either product may be beyond 64 bits only where its first factor is already too much.)
  if (runs > (most << 8) || n_seq > (1 << 24)) return false;
  const long long items = runs * (D / v), kept = (long long)n_seq * 3 * (D / v), edge = (long long)n_seq * (D / 4);
  // (A workgroup of the backward takes 64 rows or more of 64 groups of channels.)
  const long long sets = (runs + conv::WAVES - 1) / conv::WAVES * ((D / 4 + 63) / 64);
  return (items >> 8) + (kept >> 8) + 2 <= most && sets + (edge >> 8) + 2 <= most;
}

hipError_t launch_short_conv(const ShortConvArgs& a) {
  if (a.dtype == 1) return a.K == 2 ? conv::forward<2, bf16>(a) : a.K == 3 ? conv::forward<3, bf16>(a) : conv::forward<4, bf16>(a);
  return a.K == 2 ? conv::forward<2, float>(a) : a.K == 3 ? conv::forward<3, float>(a) : conv::forward<4, float>(a);
}

size_t short_conv_bwd_workspace_bytes(int B, int L, int D, int K) {
  return (size_t)conv::backward_runs(B, L, D).sets * (K + 1) * D * sizeof(float);
}

hipError_t launch_short_conv_bwd(const ShortConvArgs& a) {
  if (a.dtype == 1) return a.K == 2 ? conv::backward<2, bf16>(a) : a.K == 3 ? conv::backward<3, bf16>(a) : conv::backward<4, bf16>(a);
  return a.K == 2 ? conv::backward<2, float>(a) : a.K == 3 ? conv::backward<3, float>(a) : conv::backward<4, float>(a);
}

hipError_t launch_short_conv_step(const ShortConvArgs& a) {
  if (a.dtype == 1) return a.K == 2 ? conv::step<2, bf16>(a) : a.K == 3 ? conv::step<3, bf16>(a) : conv::step<4, bf16>(a);
  return a.K == 2 ? conv::step<2, float>(a) : a.K == 3 ? conv::step<3, float>(a) : conv::step<4, float>(a);
}

}  // namespace dn
