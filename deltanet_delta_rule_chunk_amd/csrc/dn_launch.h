// dn_launch.h -- host-side launch descriptors between the C ABI layer and the
// kernel translation units.  Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

namespace dn {

struct DecodeArgs {
  const void *q, *k, *v;
  const float* alpha;  // decay of the gated step, or null (plain delta rule)
  const float* beta;   // write strength, or its logit when `features` is set
  float* S;
  void* o;
  int B, H, d_k, d_v, in_dtype, out_dtype;
  hipStream_t stream;
  // Apply the layer's feature maps in-kernel: q, k are the raw projections
  // (normalise(silu(.)) is taken, the result held in in_dtype) and beta is
  // the logit (sigmoid is taken).
  bool features;
  // alpha holds d_k decays per (b, h), one per key dimension (KDA), instead
  // of one.
  bool per_dim_alpha;
};

struct FeatureArgs;

// Outputs of the chunked forward when it runs as the forward pass of the
// backward (bf16 matrix-core path, C = 128, plain form): for every 64-token
// block of the backward's workspace, X = (I + A)^{-1} of the block (the
// block's own diagonal block of the 128-token inverse), the state entering
// the block, R = V - K S from that state and Delta, row-major fp32.  o and
// S_final are then not written.
struct BwdFwdOut {
  float* ws;
  size_t block;       // floats per (head, 64-token block)
  size_t x, s, r, d;  // offsets of X [64][64], S [d_k][d_v], R [64][d_v], Delta [64][d_v]
  int nb;             // 64-token blocks per head
};

struct ChunkArgs {
  const void *q, *k, *v;
  const float* alpha;  // per-token decay of the gated form, or null (plain delta rule);
                       // [B,H,L,d_k] when per_dim_alpha
  const float* beta;
  const float* S0;  // may be null (zero state)
  void* o;
  float* S_final;   // may be null
  int B, H, L, d_k, d_v, C, in_dtype, out_dtype;
  void* workspace;  // at least chunk_workspace_bytes(...) bytes (kda_workspace_bytes)
  hipStream_t stream;
  bool per_dim_alpha;  // one decay per key dimension (KDA, dn_kda.hip)
  // bf16 matrix-core path only: apply the layer's feature maps inside the
  // WY-prep kernel, from feat's raw inputs into its outputs, which q, k and
  // beta above must then point at (the scan reads them).
  const FeatureArgs* feat = nullptr;
  // The backward's forward pass (see BwdFwdOut), or null.
  const BwdFwdOut* bwd_out = nullptr;
};

hipError_t launch_decode(const DecodeArgs& a);

// The layer's feature maps over `rows` rows of d_k (dn_features.hip).
struct FeatureArgs {
  const void *q_raw, *k_raw;
  const float* beta_logit;
  void *q_hat, *k_hat;
  float* beta;
  long long rows;
  int d_k, dtype;
  hipStream_t stream;
};
hipError_t launch_features(const FeatureArgs& a);
// Most rows one launch takes (the grid's x extent times rows per workgroup).
long long feature_max_rows(int d_k, int dtype);

// Kernel slots of the profiling hook (see deltanet_profile_start).
enum ProfSlot {
  kSlotChunkPrep = 0,
  kSlotChunkScan = 1,
  kSlotDecode = 2,
  kSlotFeatures = 3,
  kSlotBwdPrep = 4,
  kSlotBwdFwdScan = 5,
  kSlotBwdScan = 6,
  kSlotBwdCc = 7,
  kSlotBwdQk = 8,
  kSlotLinearState = 9,
  kSlotLinearOut = 10,
  kSlotLinearBwd = 11,
  kSlotLinearDecode = 12,
  kSlotQkNormRope = 13,
  kSlotQkNormRopeBwd = 14,
  kSlotShortConv = 15,
  kSlotShortConvBwd = 16,
  kSlotSelectiveScan = 17,
  kSlotSelectiveScanBwd = 18,
  kSlotSelectiveStep = 19,
  kSlotAddNorm = 20,
  kSlotAddNormBwd = 21,
  kNumSlots = 22
};

// Records a HIP event on `s` before (end = false) or after (end = true) the
// kernel of `slot`, when profiling is on for the calling thread; a no-op
// otherwise.
void prof_mark(int slot, bool end, hipStream_t s);

// Chunked forward: bytes of scratch it needs, and the launch sequence.
size_t chunk_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C, int in_dtype,
                             bool gated);
hipError_t launch_chunk_fwd(const ChunkArgs& a);
// Gradient of the chunked forward (dn_backward.hip).
struct BwdArgs {
  const void *q, *k, *v;    // in_dtype
  const float* beta;
  const float* S0;          // may be null (zero state)
  const float* dO;          // [B,H,L,d_v] fp32
  const float* dS_final;    // may be null (zero)
  float *dq, *dk, *dv, *dbeta;
  float* dS0;               // may be null (not written)
  int B, H, L, d_k, d_v, in_dtype;
  void* workspace;          // at least chunk_bwd_workspace_bytes(...) bytes
  hipStream_t stream;
};
size_t chunk_bwd_workspace_bytes(int B, int H, int L, int d_k, int d_v);
hipError_t launch_chunk_bwd(const BwdArgs& a);

// The per-dimension-decay (KDA) chunked forward: its workspace and launches.
size_t kda_workspace_bytes(int B, int H, int L, int d_k);
hipError_t launch_kda_chunk_fwd(const ChunkArgs& a);
// Bytes of the gated form's per-chunk log-decay table; it sits at the end of
// the workspace, after the kernels' other scratch.
size_t gated_log_decay_bytes(int B, int H, int L, int C);

// Workgroups of `threads` that one launch takes: a dispatch counts its work-items
// per dimension in 32 bits.
constexpr long long max_blocks(int threads) { return 0xffffffffLL / threads; }

// The gated linear recurrence (dn_linear.hip, dn_linear_bwd.hip,
// dn_linear_decode.hip).  Head h reads q and k of head h / (H / H_qk).
struct LinearArgs {
  const void *q, *k, *v;
  const float* log_decay;  // [B,H,L] or null (no decay)
  const float* S0;         // may be null (zero state)
  void* o;
  float* S_final;          // may be null
  int B, H, H_qk, L, d_k, d_v, in_dtype, out_dtype;
  void* workspace;         // at least linear_workspace_bytes(...) bytes
  hipStream_t stream;
};
size_t linear_workspace_bytes(int B, int H, int L, int d_k, int d_v, int in_dtype);
hipError_t launch_linear_fwd(const LinearArgs& a);

struct LinearBwdArgs {
  const void *q, *k, *v;
  const float* log_decay;  // or null
  const float* S0;         // or null
  const void* dO;          // [B,H,L,d_v] in_dtype
  const float* dS_final;   // or null (zero)
  void *dq, *dk, *dv;      // in_dtype
  float* dlog_decay;       // or null (not written)
  float* dS0;              // or null (not written)
  int B, H, H_qk, L, d_k, d_v, in_dtype;
  void* workspace;         // at least linear_bwd_workspace_bytes(...) bytes
  hipStream_t stream;
};
size_t linear_bwd_workspace_bytes(int B, int H, int H_qk, int L, int d_k, int d_v, int in_dtype);
hipError_t launch_linear_bwd(const LinearBwdArgs& a);

struct LinearDecodeArgs {
  const void *q, *k, *v;
  const float* log_decay;  // [B,H] or null
  float* S;
  void* o;
  int B, H, H_qk, d_k, d_v, in_dtype, out_dtype;
  hipStream_t stream;
};
long long linear_decode_max_heads();
hipError_t launch_linear_decode(const LinearDecodeArgs& a);

// Per-head norm of q and k and rotation by position (dn_qk_norm_rope.hip).
constexpr int kMaxAxes = 4;
struct Rows {
  const void* p;
  long long sb, sh, sl;  // strides in elements
};
struct QkNormRopeArgs {
  Rows x[2];               // raw q, k
  const float* weight[2];  // [d] or null (ones)
  const int* positions;    // [axes][B][L]
  const float* inv_freq;   // [d_rot / 2]
  int ends[kMaxAxes];      // axis a rotates pairs up to ends[a] (exclusive)
  void* y[2];              // forward: [B][H][L][d]; backward: the gradients given there (read)
  Rows dx[2];              // backward: gradients of x (written)
  float* dw[2];            // backward: [d] or null
  int H[2];
  int B, L, d, d_rot, norm, interleaved, dtype;
  float eps;
  void* workspace;         // backward: at least qk_norm_rope_bwd_workspace_bytes(...) bytes
  hipStream_t stream;
};
hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a);
long long qk_norm_rope_max_tokens(int heads, int d);
size_t qk_norm_rope_bwd_workspace_bytes(int B, int heads, int L, int d);
hipError_t launch_qk_norm_rope_bwd(const QkNormRopeArgs& a);

// Rows of [B, L, D] at strides in elements.  32 rows at the largest token stride lie
// within 32 bits of bytes, where kernels keep a thread's offsets in a tile.
constexpr long long kMostTokenStride = 1LL << 24;
struct TokenRows {
  const void* p;
  long long sb, sl;
};

// Short causal convolution of every channel (dn_short_conv.hip).
struct ShortConvArgs {
  TokenRows x;
  const float* weight;  // [D][K]
  const float* bias;    // [D] or null
  const void* state0;   // [n_seq][K-1][D] or null (zeros)
  const int* cu;        // [n_seq + 1] or null: B sequences of L
  int B, L, D, K, n_seq, silu, dtype;
  void* y;              // forward
  void* state;          // forward: or null; step: updated in place
  const void *dy, *dstate;  // backward; dstate or null
  void *dx, *dstate0;       // backward; dstate0 or null
  float *dweight, *dbias;   // backward; dbias or null
  void* workspace;          // backward: at least short_conv_bwd_workspace_bytes(...) bytes
  hipStream_t stream;
};
bool short_conv_fits(int B, int L, int D, int n_seq, int dtype);
hipError_t launch_short_conv(const ShortConvArgs& a);
size_t short_conv_bwd_workspace_bytes(int B, int L, int D, int K);
hipError_t launch_short_conv_bwd(const ShortConvArgs& a);
hipError_t launch_short_conv_step(const ShortConvArgs& a);

// Selective state space scan (dn_selective_scan.hip, dn_selective_scan_bwd.hip).
struct ScanArgs {
  TokenRows u, dt, Bm, Cm, z;  // z.p null: no gate
  const float* A;              // [D][N]
  const float *skip, *dt_bias; // [D] or null
  const float* h0;             // [n_seq][D][N] or null (zeros)
  const int* cu;               // [n_seq + 1] or null: B sequences of L
  int B, L, D, N, n_seq, softplus, dtype;
  void* y;                     // forward, step
  float* hT;                   // forward: or null; step: updated in place
  const void* dy;              // backward
  const float* dhT;            // or null (zeros)
  void *du, *ddt, *dB, *dC, *dz;
  float *dA, *dskip, *dbias, *dh0;  // dskip, dbias, dh0 or null
  void* workspace;
  hipStream_t stream;
};
bool selective_scan_fits(int B, int L, int D, int N, bool packed, int n_seq, bool backward);
size_t selective_scan_workspace_bytes(int B, int L, int D, int N, bool packed, int n_seq);
hipError_t launch_selective_scan(const ScanArgs& a);
size_t selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, bool packed, int n_seq);
hipError_t launch_selective_scan_bwd(const ScanArgs& a);
hipError_t launch_selective_scan_step(const ScanArgs& a);

// Root-mean-square norm with the residual's addition (dn_add_norm.hip).
struct AddNormArgs {
  const void* x;
  const void* residual;  // or null
  const float* weight;   // or null (ones)
  void* total;           // x + residual; null without a residual
  void* y;
  float* scale;          // [rows]: y is e4m3; or null
  int rows, D, dtype, residual_dtype;
  float eps;
  const void *dy, *dtotal;  // backward (total is read); dtotal or null
  void *dx, *dresidual;     // backward; dresidual null where it is dx
  float* dweight;           // backward; or null
  void* workspace;
  hipStream_t stream;
};
bool add_norm_fits(int rows, int D);
hipError_t launch_add_norm(const AddNormArgs& a);
size_t add_norm_bwd_workspace_bytes(int rows, int D);
hipError_t launch_add_norm_bwd(const AddNormArgs& a);

// The fixed per-GPU scratch area of the allocation-free forward
// (dn_noalloc.hip): its size, and its address on the device `stream` belongs
// to (looked up on the first call for that device, then cached).
constexpr size_t kNoallocScratchBytes = (size_t)64 << 20;
hipError_t noalloc_scratch(hipStream_t stream, void** out);

}  // namespace dn
