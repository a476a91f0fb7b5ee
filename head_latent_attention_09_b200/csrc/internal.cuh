// Internal declarations shared by the host runtime and the kernels of the MLA
// decode library.  Nothing here is part of the public ABI (see include/mla.h).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "mla.h"

namespace mla {

// Devices a process may drive (per-device launch set-up is kept per index).
constexpr int kMaxDevices = 64;

// KV tokens per page of the paged fast paths (page_size == kTile), the
// granularity of a token range's first token, and the smallest tile of the
// split plan.
constexpr int kTile = 64;

// FP8 latent cache: channels per scale group (over c^KV, then over k^R).
constexpr int kFp8Group = 128;
__host__ __device__ inline int fp8_num_groups(int d_c, int d_r) {
  return (d_c + kFp8Group - 1) / kFp8Group + (d_r + kFp8Group - 1) / kFp8Group;
}

// Bits of the device status word.
constexpr unsigned kStatusTimeout = 1u;
constexpr unsigned kStatusBounds = 2u;

// Attention kernel chosen for a configuration at mla_create time.
enum AttnKind : int {
  kAttnSimt = 0,      // generic CUDA-core kernel (any shape, fp32 or bf16)
  kAttnTcPair = 1,    // bf16, n_h == 128, d_c == 512, d_r == 64: tcgen05, CTA pair
  kAttnTcSmallH = 2,  // bf16, n_h <= 32 (multiple of 16), d_c == 512, d_r == 64
};

enum GemmKind : int { kGemmSimt = 0, kGemmTc = 1 };

}  // namespace mla

namespace mla {

// cos and sin of the rotary angle pos * theta in single precision, accurate
// at positions up to 2^24.  theta is given as an unevaluated float sum
// hi + lo (its double value split in two); the product pos * hi is kept with
// its exact rounding error (fma), so the angle carries ~2^-48 relative error
// (a plain float product would err by ~1e-2 rad near position 131072), and it
// is reduced to [-pi, pi] with a three-part split of 2 pi (Cody and Waite).
// Error of the reduced angle: a few 1e-7 rad; the hardware sine and cosine on
// [-pi, pi] add at most ~4e-7 (far below the bf16 rounding of the results).
__device__ __forceinline__ void rope_sincos(int pos, float2 theta, float *s, float *c) {
  const float p = (float)pos;                                   // exact below 2^24
  const float a_hi = p * theta.x;
  const float a_lo = fmaf(p, theta.x, -a_hi) + p * theta.y;
  const float k = rintf(a_hi * 0.15915494309189535f);          // whole turns
  float r = fmaf(-k, 6.28125f, a_hi);                           // 2 pi = 6.28125 + 1.93548e-3 - 1.74846e-7
  r = fmaf(-k, 1.9354820251464844e-3f, r);
  r = fmaf(-k, -1.7484555314695172e-7f, r);
  __sincosf(r + a_lo, s, c);
}

// The handle's frequency table: theta_k in double [d_r / 2], then the same
// values split into float pairs (hi, lo) [d_r / 2], in one allocation.
__host__ __device__ inline const float2 *theta_pairs(const double *theta, int d_r) {
  return reinterpret_cast<const float2 *>(theta + d_r / 2);
}

// Programmatic dependent launch.  Kernels of this library are launched so
// that the next kernel in the stream may begin while the current one
// finishes (its set-up overlapping the tail); each kernel signals that its
// dependents may launch, and waits for the kernels before it to complete
// before it touches memory they write or read.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches kern(args...) with programmatic stream serialization (and a
// cluster shape when cluster_x > 1).  Only kernels that call pdl_wait()
// before their first dependent memory access may be launched this way.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster_x,
                       Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args &&>(args)...);
}

}  // namespace mla

struct mla_handle {
  mla_config cfg;
  int device;
  int num_sms;
  unsigned *d_status;  // device status word (kStatus* bits)
  double *d_theta;     // device RoPE frequencies theta_k: [d_r/2] double, then [d_r/2] float (hi, lo) pairs
  double score_mult;   // YaRN temperature t multiplying every score (1 without scaling)
  int attn_kind;       // mla::AttnKind
  int gemm_kind;       // mla::GemmKind
  int strict;          // 1: no CUDA-core substitute for a tensor-core kernel (mla_set_strict)
  void *noalloc_scratch;  // device address of the allocation-free entry point's array
};

namespace mla {

// ---------------------------------------------------------------------------
// Split plan.  Sequence b contributes T_b = ceil((end_b - begin_b) / tile)
// tiles of `tile` tokens (the MMA tile of the attention kernel that runs:
// 256 for 128 heads, 128 for 16/32 heads, 64 on the CUDA cores, so that a
// share never pays for a partial tile in the middle of a sequence); the
// batch's Ttot tiles, in sequence order, are cut into P equal shares
// [begin(w), begin(w+1)).  A (share, sequence) intersection is a piece: it
// yields one partial ctx_lat and log-sum-exp.  P is clamped to Ttot so that no
// share is empty, which makes the pieces of one sequence a run of consecutive
// shares.
// ---------------------------------------------------------------------------
// a / b of non-negative values, in 32 bits where both fit (a 64-bit division
// costs some hundred cycles, and every role of every kernel walks the plan).
__host__ __device__ inline long long plan_div(long long a, long long b) {
  if (((unsigned long long)(a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}
__host__ __device__ inline long long plan_begin(long long w, long long P, long long Ttot) {
  return plan_div(w * Ttot, P);
}
// Largest share index whose range starts at or before tile t (0 <= t < Ttot).
__host__ __device__ inline long long plan_share_of_tile(long long t, long long P, long long Ttot) {
  return plan_div((t + 1) * P - 1, Ttot);
}
__host__ __device__ inline long long ceil_div_ll(long long a, long long b) { return (a + b - 1) / b; }

// What the plan cuts into tiles.  A plan sequence is one of `runs` passes over a
// batch sequence (1 except for a tree of drafted tokens, whose query rows are
// taken in runs of groups; plan sequence v belongs to batch sequence v / runs).
struct PlanSource {
  const int *ctx_len;              // [B] cached tokens
  const int *ctx_begin = nullptr;  // [B] first attended token, or NULL (0)
  int runs = 1;
  int drafted = 0;                 // tree: drafted tokens behind the ctx_len cached ones
  const int *sel = nullptr;        // selected blocks [B, sel_k], or NULL (every block)
  const int *n_sel = nullptr;      // [B] how many of them
  int sel_k = 0;
};

// Workspace header written by the plan kernel; the per-sequence arrays follow.
struct WsHeader {
  long long B;
  long long P;           // effective number of shares (<= requested, <= Ttot)
  long long Ttot;        // total tiles
  long long n_pieces;    // total pieces
};

struct WsLayout {
  size_t tile_prefix_off;  // int64 [B+1]
  size_t piece_base_off;   // int64 [B+1]
  size_t ctx_off;          // int32 [2][B]: each sequence's end as attended (clamped by the plan), and its first token
                           // (selected blocks and trees: its cached tokens instead; they start at token 0)
  size_t share_first_off;  // int32 [P]: the first sequence whose tiles reach into each share
  size_t opart_off;        // float [n_h, max_pieces, d_c]: a head's pieces are consecutive rows
  size_t lse_off;          // float [n_h, max_pieces]
  size_t total;
  long long max_pieces;
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Plan sequences up to which the tensor-core attention kernels plan in line.
constexpr int kInlineSeqs = 256;

// Row of (piece, head) in the partials (units of d_c floats) and index of its
// log-sum-exp.
__host__ __device__ inline long long part_row(const WsLayout &L, long long piece, int head) {
  return (long long)head * L.max_pieces + piece;
}

// Layout for B plan sequences of `rows` query rows each, P shares and room for
// `pieces` pieces.
inline WsLayout ws_layout_rows(int rows, int d_c, int B, int P, long long pieces) {
  WsLayout L;
  L.max_pieces = pieces;
  size_t off = align_up(sizeof(WsHeader), 256);
  L.tile_prefix_off = off;
  off = align_up(off + sizeof(long long) * (size_t)(B + 1), 256);
  L.piece_base_off = off;
  off = align_up(off + sizeof(long long) * (size_t)(B + 1), 256);
  L.ctx_off = off;
  off = align_up(off + 2 * sizeof(int) * (size_t)(B > 0 ? B : 1), 256);
  L.share_first_off = off;
  off = align_up(off + sizeof(int) * (size_t)(P > 0 ? P : 1), 256);
  L.opart_off = off;
  off = align_up(off + sizeof(float) * (size_t)L.max_pieces * rows * d_c, 256);
  L.lse_off = off;
  off = align_up(off + sizeof(float) * (size_t)L.max_pieces * rows, 256);
  L.total = off;
  return L;
}

inline WsLayout ws_layout(const mla_config &cfg, int B, int P) {
  return ws_layout_rows(cfg.n_h, cfg.d_c, B, P, (long long)P + B);
}

// Tree attention: the query rows (drafted token, head) of a sequence are cut
// into groups of `rows`.  Only a group that is split between shares leaves
// partials, and each of a share's `gang` workers holds at most two such pieces
// (its first and its last): 2 P gang slots.
inline WsLayout tree_ws_layout(int rows, int d_c, int plan_seqs, int P, int gang) {
  return ws_layout_rows(rows, d_c, plan_seqs, P, 2ll * P * gang);
}

// The tensor-core kernel reads the blocks that hold drafted tokens, the last
// partial block of the cached ones with them, from a copy of at most two
// blocks per sequence behind the partials: bf16 [batch, kTreeCopyRows, 576],
// zeros past the drafted tokens, non-finite values of drafted tokens zero.
constexpr int kTreeCopyRows = 2 * kTile;
constexpr int kTreeMaxDrafted = 64;   // a tree's masks are 64-bit words
constexpr int kMaxPlanSeqs = 1 << 24; // row groups of one call (the plan's arrays and prefix sums)
constexpr int kMaxSelected = 1 << 20; // selected blocks per sequence
inline size_t tree_copy_bytes(int batch) { return (size_t)batch * kTreeCopyRows * 576 * 2; }

// Tree of drafted tokens: the query rows of sequence b are (t, head), t
// outermost, T * n_h of them in `groups` groups of `group_rows`; drafted token
// t sits in cache slot cached + t and attends every cached token and the
// drafted ones whose bit is set in mask[b, t].  Groups of a sequence are taken
// `gang` at a time: a plan sequence is a run of `gang` groups, and a share is
// worked on by `gang` workers that walk the same tokens at the same time, each
// for its own group, so that a row comes from HBM once for all of them.
struct TreeArgs {
  int T = 0;                                // 0: no tree
  int groups = 1, group_rows = 0, seq_rows = 0;
  int gang = 1, runs = 1;                   // runs = ceil(groups / gang): plan sequences per batch sequence
  const unsigned long long *mask = nullptr; // [batch, T]
  void *out = nullptr;                      // [batch, T, n_h, d_c], the cache's dtype
  float *lse = nullptr;                     // [batch, T, n_h] or NULL
  size_t copy_off = 0;                      // tensor-core kernel: offset of the copied blocks in the workspace
};

// Arguments shared by the attention kernels.
struct AttnArgs {
  const void *q_abs;
  const void *cache;
  long long cache_len;
  const int *block_table;
  int max_blocks;
  int page_size;
  int B;
  int n_h, d_c, d_r;
  float scale_log2;  // log2(e) / sqrt(d_h + d_r)
  // FP8 cache: the rows are E4M3 codes and kv_scale [rows, n_groups] holds
  // each row's group scales; NULL for a cache in cfg.dtype
  const float *kv_scale;
  int n_groups;
  char *ws;
  WsLayout L;
  int plan_tile;     // tokens per tile of the split plan
  unsigned *status;
  // Selected blocks [B, sel_k] of 64 tokens (NULL: every block): token t of a
  // sequence is then token t % 64 of its block sel[b, t / 64].
  const int *sel = nullptr;
  int sel_k = 0;
  TreeArgs tree;     // B is then the number of plan sequences (runs x batch)
  // Tensor-core kernels without a tree, B <= kInlineSeqs: every CTA makes the
  // plan itself in shared memory (plan.cuh) instead of reading a plan kernel's.
  int inline_plan = 0;
  PlanSource src{nullptr};
  long long cap = 0;
};

// ---------------------------------------------------------------------------
// Launchers (return cudaGetLastError() of the launch).
// ---------------------------------------------------------------------------
// The plan attends tokens [begin_b, end_b) of sequence b: end_b = ctx_len[b]
// clamped to [0, cap] (cap: the tokens the cache can address for one
// sequence), begin_b = ctx_begin[b] (0 when ctx_begin is NULL) rounded down to
// a multiple of kTile and clamped to [0, end_b].  Any value it has to change
// is flagged in the status word.  It stores both in the workspace; every
// attention kernel reads those instead of the caller's arrays, so that the
// plan's tiles and the kernels' token ranges agree.  `tile` (a multiple of
// kTile) is the plan's tile in tokens.
// With a tree the plan attends the cached tokens and the drafted ones behind
// them (clamped to cap); with selected blocks the tokens of those blocks, the
// last of which may be the sequence's partial one.
cudaError_t launch_plan(const PlanSource &src, int B, int P, long long cap, int tile, char *ws, const WsLayout &L,
                        unsigned *status, cudaStream_t s);

// Tree, for the tensor-core kernel: the plan, and in the same launch the copy
// of the blocks that hold drafted tokens.
cudaError_t launch_tree_plan_copy(const PlanSource &src, const AttnArgs &a, int P, long long cap, cudaStream_t s);

// Running maximum of a row that nothing has reached yet: the lowest finite value
// instead of -inf, so that scores of -inf (masked, or overflowed) subtract it
// without a NaN (-inf - -inf) and come out as 2^-inf = 0.
constexpr float kNoMax = -3.402823466e38f;

// The plan stores two values per plan sequence: the end of its attended tokens
// (clamped), and its first token (a multiple of kTile), or for selected blocks
// and trees, which start at token 0, the number of its cached tokens.
__device__ __forceinline__ const int *plan_ends(const AttnArgs &a) {
  return reinterpret_cast<const int *>(a.ws + a.L.ctx_off);
}
__device__ __forceinline__ const int *plan_seconds(const AttnArgs &a) { return plan_ends(a) + a.B; }

// Cache row of token t of batch sequence b (t below what the cache can
// address), or -1 when its page is unmapped or outside the pool.
__device__ __forceinline__ long long token_row(const AttnArgs &a, int b, long long t) {
  if (a.page_size == 0) return t < a.cache_len ? (long long)b * a.cache_len + t : -1;
  const unsigned bi = (unsigned)t / (unsigned)a.page_size;   // t is a position: 31 bits
  if (bi >= (unsigned)a.max_blocks) return -1;
  const int blk = a.block_table[(long long)b * a.max_blocks + bi];
  if (blk < 0 || blk >= a.cache_len) return -1;
  return (long long)blk * a.page_size + ((unsigned)t - bi * (unsigned)a.page_size);
}

// The same for token t of a sequence's selected blocks, of `cached` tokens in
// all.  -1 also for a block that the sequence does not have, and for its
// partial last block anywhere but at the end of the selection (end: the
// selected tokens).
__device__ __forceinline__ long long selected_row(const AttnArgs &a, int b, long long t, int end, int cached) {
  const int blk = a.sel[(long long)b * a.sel_k + t / kTile];
  if (blk < 0 || (long long)blk * kTile >= cached) return -1;
  if (((long long)blk + 1) * kTile > cached && t / kTile != (end - 1) / kTile) return -1;
  return token_row(a, b, (long long)blk * kTile + t % kTile);
}

// How a piece of tree attention ends.  A group whose tiles all lie in one
// share is written out at once; a part of a split group leaves a partial in
// one of its worker's two slots.
struct TreePiece {
  bool whole;
  long long slot;
};
__device__ __forceinline__ TreePiece tree_piece(const AttnArgs &a, const long long *tile_prefix, int v, long long w,
                                                int member, long long P, long long Ttot) {
  const long long s0 = tile_prefix[v], s1 = tile_prefix[v + 1];
  const long long t0 = plan_begin(w, P, Ttot), t1 = plan_begin(w + 1, P, Ttot);
  return {s0 >= t0 && s1 <= t1, 2 * (w * a.tree.gang + member) + (s0 > t0 ? 1 : 0)};
}

cudaError_t launch_attn_simt(const AttnArgs &a, int P, bool fp32, cudaStream_t s);
cudaError_t launch_tree_attn_simt(const AttnArgs &a, int P, bool fp32, cudaStream_t s);
// With out_f32, ctx_lat is written in float32 whatever cfg.dtype.
cudaError_t launch_combine(const mla_config &cfg, const char *ws, const WsLayout &L, int B,
                           void *ctx_lat, float *lse, cudaStream_t s, bool out_f32 = false);
// Tree attention: merge of the groups that are split between shares, straight
// into the outputs (the others are there already).
cudaError_t launch_tree_combine(const AttnArgs &a, int P, bool fp32, cudaStream_t s);
// Accepted path of a drafted tree: row ctx_len[b] + path[b, i] of the cache
// moves to ctx_len[b] + i, i < n_path[b]; new_len[b] = ctx_len[b] + n_path[b].
cudaError_t launch_tree_accept(const mla_config &cfg, void *cache, long long cache_len, const int *block_table,
                               int max_blocks, const int *ctx_len, const int *path, const int *n_path, int B, int T,
                               int *new_len, unsigned *status, cudaStream_t s);

// Selection of cached blocks (blocks.cu).
cudaError_t launch_block_keys(const mla_config &cfg, const void *cache, long long cache_len, const int *block_table,
                              int max_blocks, const int *ctx_begin, const int *ctx_len, int B, int max_new, void *keys,
                              int key_blocks, unsigned *status, cudaStream_t s);
struct ScoreLayout {   // workspace of the CUDA-core kernels
  size_t logit_off;    // float [B, blocks rounded up to 128, head_rows]
  size_t stat_off;     // float2 [B, block tiles, head_rows]: a tile's maximum and sum of exponentials
  size_t total;
  int head_rows;       // heads rounded up to 32
  int tiles;           // 128-block tiles
};
ScoreLayout score_layout(const mla_config &cfg, int B, int key_blocks);
cudaError_t launch_block_scores_tc(const mla_config &cfg, float scale_log2, const void *q_abs, const void *keys,
                                   int key_blocks, const int *ctx_len, int B, float *scores, unsigned *status,
                                   cudaStream_t s);
cudaError_t launch_block_scores_simt(const mla_config &cfg, float scale_log2, const void *q_abs, const void *keys,
                                     int key_blocks, const int *ctx_len, int B, float *scores, char *ws,
                                     const ScoreLayout &L, unsigned *status, cudaStream_t s);
cudaError_t launch_block_select(const float *scores, int n_blocks, const int *ctx_len, int B, int k, int n_first,
                                int n_last, int *sel, int *n_sel, unsigned *status, cudaStream_t s);

// Merge of R float32 token-range results [R, B, n_h, d_c] with their
// log-sum-exps [R, B, n_h] into ctx_lat [B, n_h, d_c] (cfg.dtype) and lse.
cudaError_t launch_merge_ranges(const mla_config &cfg, const float *parts, const float *lse_parts, int R, int B,
                                void *ctx_lat, float *lse, cudaStream_t s);

cudaError_t launch_append_simt(const mla_config &cfg, const void *h, int B, int T,
                               const int *start_pos, const void *w_dkv, const void *w_kr,
                               void *cache, long long cache_len, const int *block_table,
                               int max_blocks, const double *theta, unsigned *status,
                               cudaStream_t s, float *rows_out = nullptr, const int *depth = nullptr);
// FP8 E4M3 quantisation of n_rows rows [n_rows, d_c + d_r] (cfg.dtype, or
// float32 when src_f32): per row and 128-channel group, sigma = amax / 448 and
// codes E4M3(x / sigma).  With start_pos, row r is token r % T of sequence
// r / T and goes to its cache row (bounds flagged); without, to row r.
cudaError_t launch_quantize_fp8(const mla_config &cfg, const void *src, bool src_f32, long long n_rows,
                                int T, const int *start_pos, uint8_t *codes, float *scales,
                                long long cache_len, const int *block_table, int max_blocks,
                                unsigned *status, cudaStream_t s);
cudaError_t launch_absorb_simt(const mla_config &cfg, const void *q_nope, const void *q_rope,
                               const int *pos, const void *w_uk, void *q_abs, int B,
                               const double *theta, cudaStream_t s);
cudaError_t launch_outproj_simt(const mla_config &cfg, const void *ctx_lat, const void *w_uv,
                                void *o, int B, cudaStream_t s);
// CUDA-core form of the fused combine and output projection (any dtype/shape).
cudaError_t launch_combine_outproj_simt(const mla_config &cfg, const char *ws, const WsLayout &L, int B,
                                        const void *w_uv, void *o, void *ctx_lat, float *lse, cudaStream_t s);
cudaError_t launch_wo_simt(const mla_config &cfg, const void *o, const void *w_o, void *u, int B,
                           cudaStream_t s);
// y[N, M] = x[N, K] w[M, K]^T (row-major, the config's dtype).
cudaError_t launch_linear_simt(const void *x, const void *w, void *y, int M, int K, int N, bool fp32,
                               cudaStream_t s);

// tcgen05 paths (bf16 only); return cudaErrorNotSupported for shapes they lack.
// With depth [B, T] set, token t of sequence b is rotated by position
// start_pos[b] + depth[b, t] (its slot stays start_pos[b] + t).
// With rows_out set, the rotated rows go to rows_out [B*T, d_c + d_r] in
// float32 instead of to the cache (the cache arguments are then unused).
cudaError_t launch_append_tc(const mla_config &cfg, const void *h, int B, int T,
                             const int *start_pos, const void *w_dkv, const void *w_kr,
                             void *cache, long long cache_len, const int *block_table,
                             int max_blocks, const double *theta, unsigned *status,
                             cudaStream_t s, float *rows_out = nullptr, const int *depth = nullptr);
cudaError_t launch_absorb_tc(const mla_config &cfg, const void *q_nope, const void *q_rope,
                             const int *pos, const void *w_uk, void *q_abs, int B,
                             const double *theta, unsigned *status, cudaStream_t s);
cudaError_t launch_outproj_tc(const mla_config &cfg, const void *ctx_lat, const void *w_uv,
                              void *o, int B, unsigned *status, cudaStream_t s);
cudaError_t launch_wo_tc(const mla_config &cfg, const void *o, const void *w_o, void *u, int B,
                         unsigned *status, cudaStream_t s);
cudaError_t launch_linear_tc(const void *x, const void *w, void *y, int M, int K, int N, unsigned *status,
                             cudaStream_t s);
// Split combine fused with the output projection: o[b, i] = W^UV_i ctx_lat[b, i]
// with ctx_lat merged from the workspace's partials inside the kernel
// (written out too when ctx_lat is set; lse likewise).
cudaError_t launch_combine_outproj_tc(const mla_config &cfg, const char *ws, const WsLayout &L, int B,
                                      const void *w_uv, void *o, void *ctx_lat, float *lse, unsigned *status,
                                      cudaStream_t s);
// `before` launches what goes before the kernel (a plan, a copy), once the
// arguments are known to be ones it can take.
class Before {   // refers to a callable that outlives it (or to none); owns nothing and never throws
 public:
  Before() = default;
  template <typename Fn>
  explicit Before(const Fn &fn)
      : what_(&fn), call_([](const void *w) { return (*static_cast<const Fn *>(w))(); }) {}
  explicit operator bool() const { return call_ != nullptr; }
  cudaError_t operator()() const { return call_(what_); }

 private:
  const void *what_ = nullptr;
  cudaError_t (*call_)(const void *) = nullptr;
};
cudaError_t launch_attn_tc_pair(const AttnArgs &a, int P, cudaStream_t s, const Before &before);
// The same kernel over a tree of drafted tokens, 128 query rows at a time.
cudaError_t launch_tree_attn_tc_pair(const AttnArgs &a, int P, cudaStream_t s, const Before &before);
cudaError_t launch_attn_tc_smallh(const AttnArgs &a, int P, cudaStream_t s, const Before &before);

// One bounded wait on a barrier that nothing completes, giving up after
// limit_ns: sets the status word's time-out bit (self-test of that path).
cudaError_t launch_wait_timeout_selftest(unsigned *status, unsigned long long limit_ns, cudaStream_t s);

// Resolve the driver entry point for tensor-map encoding (no libcuda link).
bool tma_available();

// Device address, on the current device, of the fixed scratch array of the
// allocation-free entry point (noalloc.cu).  MLA_OK or MLA_ERR_CUDA.
int noalloc_scratch_lookup(void **out);

// Once-per-device launch set-up (the dynamic shared-memory opt-in, which
// applies per device): runs `fn` the first time it is called for the current
// device and caches its result; concurrent callers wait for the first.
template <typename Fn>
cudaError_t once_per_device(std::atomic<int> (&state)[kMaxDevices], Fn fn) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorNotSupported;
  if (state[dev].load(std::memory_order_acquire) == 2) return cudaSuccess;
  static std::mutex mu;
  std::lock_guard<std::mutex> g(mu);
  if (state[dev].load(std::memory_order_relaxed) == 2) return cudaSuccess;
  e = fn();
  if (e == cudaSuccess) state[dev].store(2, std::memory_order_release);
  return e;
}

}  // namespace mla
