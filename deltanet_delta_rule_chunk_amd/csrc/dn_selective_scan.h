// dn_selective_scan.h -- what the selective scan's forward and backward share:
// the segments that sequences are cut into, and a workgroup's tile of tokens.
//
// Per channel d and state n, token t in order:
//     h = e^{dt_t A} h + dt_t u_t B_t,   y_t = sum_n C_t h + D u_t
// with dt_t = softplus(raw_t + bias).  Each (d, n) is a recurrence of its own
// with a decay of its own, so there is no matrix product in it: the work is a
// multiplication, an exponential and three more operations on every
// (token, channel, state) and the vector units bound it: 65536 tokens of 4096 channels
// with 16 states take 1560 us (two walks, the vector units busy throughout), 458 at the
// rate of a copy.
//
// A workgroup takes 64 channels, one per lane, and a wave 4 of their states, so
// that B_t and C_t are the same for all lanes of a wave (scalar loads) and a
// token's sum over states is 4 steps in registers and one sum over the waves.
// Tokens go in tiles of 16: the threads first form dt and dt u of the tile
// (4 channels of one token each) and leave them in LDS, then every wave walks
// the 16 tokens, then the threads add up the waves' parts and finish y.
#pragma once

#include "dn_launch.h"
#include "dn_vec.h"

namespace dn {
namespace ssm {

constexpr int kTile = 16;  // tokens
constexpr int kCh = 64;    // channels per workgroup

// A piece of one sequence.  Rows that no sequence holds form segments too (seq
// < 0), whose outputs are zeros.
struct Segment {
  int row, n;     // first token within the batch row, tokens
  int seq, batch;
  bool first, last;  // of its sequence
};

// Where the segments lie: counted out for a batch of equal sequences, from a
// table in the workspace (segment_table_kernel) for packed ones.
struct Plan {
  const int* used;      // packed: segments in the table, or null
  const int* first_of;  // packed: first segment of each sequence [n_seq + 1]
  const int4* table;    // packed: {row, n, seq, first | last << 1}
  int len;              // tokens per segment, a multiple of kTile
  int per_row;          // equal sequences: segments of each
  int L;
  int count;            // segments launched (packed: the most there can be)
};

__device__ __forceinline__ bool segment_of(const Plan& p, int id, Segment& s) {
  if (!p.table) {
    s.batch = s.seq = id / p.per_row;
    const int i = id - s.seq * p.per_row;
    s.row = i * p.len;
    s.n = min(p.len, p.L - s.row);
    s.first = i == 0;
    s.last = i == p.per_row - 1;
    return true;
  }
  if (id >= *p.used) return false;
  const int4 e = p.table[id];
  s.row = e.x;
  s.n = e.y;
  s.seq = e.z;
  s.batch = 0;
  s.first = e.w & 1;
  s.last = e.w & 2;
  return true;
}
// First and last segment of a sequence.
__device__ __forceinline__ void segments_of(const Plan& p, int seq, int& first, int& last) {
  first = p.table ? p.first_of[seq] : seq * p.per_row;
  last = p.table ? p.first_of[seq + 1] - 1 : first + p.per_row - 1;
}
// Number of a segment's first tile, when tiles are kept: segments follow each other
// by rows, so each may take one tile more than its rows fill.
__device__ __forceinline__ long long first_tile(const Plan& p, const Segment& s, int id) {
  return ((long long)s.batch * p.L + s.row) / kTile + id;
}

// Host side.
struct Sizes {
  int len, per_row;
  long long segments;  // the most there can be
  bool split;          // whether a sequence may have more than one
};
inline long long channel_blocks(int D) { return (D + kCh - 1) / kCh; }
// How sequences are cut: not if there are `enough` workgroups without a cut, or no more than
// `whole` tokens (where workgroups are many, 1 token per `each` of them); else into `want`
// workgroups, but pieces of no less than 64 tokens, or 48 or 32 where those give no more than `few`
// workgroups, or 16 where they give one per CU (then a call waits for a walk's length, not for the
// units).  Workgroups are counted whatever their waves (N / 4), packed sequences as if they were one, and
// combine()'s time is not weighed: what that costs is at forward_sizes() and combine_kernel().
struct Cutting {
  long long enough, want, few;
  int whole, each;
};
inline Sizes sizes_of(bool packed, int B, int L, int n_seq, int D, const Cutting& k) {
  const long long groups = B * channel_blocks(D);
  Sizes s;
  const long long whole = ((long long)L + kTile - 1) / kTile * kTile;
  s.len = (int)(whole < kTile ? kTile : whole > 0x7fffffe0LL ? 0x7fffffe0LL : whole);
  if (groups < k.enough && L > k.whole && L > groups / k.each) {
    int least = kTile;
    while (least < 64 && groups * ((L - 1) / least + 1) > (least == kTile ? 256 : k.few)) least += kTile;
    const long long pieces = (k.want + groups - 1) / groups;
    long long len = ((long long)L + pieces - 1) / pieces;
    len = (len + kTile - 1) / kTile * kTile;
    s.len = (int)(len < least ? least : len);
  }
  s.per_row = L > 0 ? (int)(((long long)L + s.len - 1) / s.len) : 1;
  s.segments = packed ? (long long)L / s.len + n_seq + 2 : (long long)B * s.per_row;
  s.split = s.per_row > 1;
  return s;
}
inline size_t table_bytes(bool packed, int n_seq, const Sizes& s) {
  if (!packed) return 0;
  return (size_t)((n_seq + 2 + 3) / 4 * 4) * sizeof(int) + (size_t)s.segments * sizeof(int4);
}
Sizes backward_sizes(int B, int L, int D, bool packed, int n_seq);  // (dn_selective_scan_bwd.hip)
// Places the table in `ws` and launches the kernel that fills it.
hipError_t make_plan(const int* cu, int n_seq, int L, const Sizes& s, void* ws, hipStream_t stream, Plan* p);

// Four values that are the same for a whole wave, through the scalar cache, as
// they lie in memory.
typedef const __attribute__((address_space(4))) uint32_t* scalar_ptr;
template <typename T>
struct Uniform4 {
  uint32_t v[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Uniform4<T> uniform4(const T* p) {
  const scalar_ptr q = (scalar_ptr)(uintptr_t)p;
  Uniform4<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r.v[i] = q[i];
  return r;
}
__device__ __forceinline__ f32x4 wide(const Uniform4<bf16>& u) {
  return f32x4{__uint_as_float(u.v[0] << 16), __uint_as_float(u.v[0] & 0xffff0000u), __uint_as_float(u.v[1] << 16),
               __uint_as_float(u.v[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 wide(const Uniform4<float>& u) {
  return f32x4{__uint_as_float(u.v[0]), __uint_as_float(u.v[1]), __uint_as_float(u.v[2]), __uint_as_float(u.v[3])};
}
// Rows whose loads are under way together while the group before is worked on.  (Left
// to the compiler, every row's load is waited for where it is used: 3.4 ms instead of
// 2.1 for 65536 tokens of 4096 channels; with groups of 8 rows 2.09.)
template <typename T> constexpr int group_rows() { return 8 / (int)sizeof(T); }
template <typename T, int R = group_rows<T>()>
struct Group {
  Uniform4<T> r[R];
  __device__ __forceinline__ void load(const T* p, long long stride) {
#pragma unroll
    for (int i = 0; i < R; ++i, p += stride) r[i] = uniform4(p);
  }
};
// Scalar loads and LDS reads share a counter and come back in any order, so what is
// needed first is waited for before the next ones start.
__device__ __forceinline__ void wait_reads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}

// A thread's place in the phases before and after the walk: a token of the tile and
// 4 channels.  Rows are read at a base that is the same for the workgroup and a
// 32-bit offset of the thread that is the same for every tile, so a tile's loads cost
// no vector operation.  Channels behind D read the last ones' place, tokens behind
// the segment its last token's: nothing that is kept depends on them.
template <int NW>
struct Spot {
  static constexpr int kRows = 4 * NW;                            // tokens per pass
  static constexpr int kPasses = kRows >= kTile ? 1 : kTile / kRows;
  int r, c;  // first token, first channel of the workgroup's
  __device__ __forceinline__ Spot() : r((int)threadIdx.x >> 4), c(((int)threadIdx.x & 15) * 4) {}
  __device__ __forceinline__ int row(int pass) const { return r + pass * kRows; }
  __device__ __forceinline__ bool in_tile() const { return kRows <= kTile || r < kTile; }
};
template <typename T>
__device__ __forceinline__ uint32_t offset_of(int row, long long stride, int c) {
  return ((uint32_t)row * (uint32_t)stride + (uint32_t)c) * (uint32_t)sizeof(T);
}
template <typename T>
__device__ __forceinline__ const T* at_bytes(const T* base, uint32_t off) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + off);
}
// Rows of one tensor, tile by tile.
template <int NW, typename T>
struct Feed {
  const T* tile;     // first row of the tile, first channel of the tensor
  long long stride;  // of a token
  uint32_t off[Spot<NW>::kPasses];
  Raw4<T> raw[Spot<NW>::kPasses];  // the next tile's
  __device__ __forceinline__ Feed(const void* p, long long first, long long stride, const Spot<NW>& at, int c)
      : tile(static_cast<const T*>(p) + first), stride(stride) {
#pragma unroll
    for (int i = 0; i < Spot<NW>::kPasses; ++i) off[i] = offset_of<T>(at.row(i), stride, c);
  }
  // n: tokens left from the tile's first on (at least 1).
  __device__ __forceinline__ void fetch(const Spot<NW>& at, int c, int n) {
    if (!at.in_tile()) return;
#pragma unroll
    for (int i = 0; i < Spot<NW>::kPasses; ++i)
      raw[i] = raw4(at_bytes(tile, n >= kTile ? off[i] : offset_of<T>(min(at.row(i), n - 1), stride, c)));
  }
  __device__ __forceinline__ void move(int tiles) { tile += tiles * kTile * stride; }
};

// The rows of B or C of the next tile, one element per thread, brought into L2 ahead of
// the scalar loads that use them, which otherwise wait for HBM (2 x 8192 tokens of 2048 fp32
// channels: 236 us with it, 254 without).
template <int NW, typename T>
struct Ahead {
  static constexpr int N = 4 * NW;
  const T* tile;
  long long stride;
  uint32_t off;
  T value;
  __device__ __forceinline__ Ahead(const void* p, long long first, long long stride)
      : tile(static_cast<const T*>(p) + first), stride(stride), off(offset_of<T>((int)threadIdx.x / N, stride, (int)threadIdx.x % N)),
        value{} {}
  __device__ __forceinline__ void fetch(int n) {
    value = *at_bytes(tile, n >= kTile ? off : offset_of<T>(min((int)threadIdx.x / N, n - 1), stride, (int)threadIdx.x % N));
  }
  __device__ __forceinline__ void arrived() { asm volatile("" ::"v"(to_f32(value))); }
  __device__ __forceinline__ void move(int tiles) { tile += tiles * kTile * stride; }
};

__device__ __forceinline__ f32x4 softplus4(f32x4 x, bool on) {
  if (!on) return x;
  return f32x4{softplus(x[0]), softplus(x[1]), softplus(x[2]), softplus(x[3])};
}
__device__ __forceinline__ f32x4 sigmoid4(f32x4 x) {
  return f32x4{sigmoid(x[0]), sigmoid(x[1]), sigmoid(x[2]), sigmoid(x[3])};
}
__device__ __forceinline__ f32x4 get4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// States of a sequence in front of each of its segments, in place of what each
// segment makes from zero (the first: from h0) -- and, where `back` is given, gradients
// of the states behind each segment in place of what each passes to its front (the
// last: from the last state's).  Both [seg][D][N]; logs [seg][D]: sums of dt.
// (dn_selective_scan.hip)
hipError_t combine(const Plan& p, int n_seq, int D, int N, const float* A, const float* logs, const float* h0,
                   float* ahead, float* back, hipStream_t stream);

}  // namespace ssm
}  // namespace dn
