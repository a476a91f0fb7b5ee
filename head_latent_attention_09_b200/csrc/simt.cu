// CUDA-core kernels: the split plan, the log-sum-exp combine, and generic
// (any shape, fp32 or bf16) versions of append / absorb / attention /
// output projection.  The fp32 configuration runs entirely here; bf16 shapes
// with a tensor-core kernel use those instead (see api.cu).
#include <cuda_fp8.h>
#include <math_constants.h>

#include "plan.cuh"

namespace mla {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Row index (in units of D-element rows) of token p of sequence b, or -1 when
// the position is outside the cache / unmapped (the caller flags it).
__device__ __forceinline__ long long cache_row(int b, long long p, long long cache_len,
                                               const int *block_table, int max_blocks,
                                               int page_size) {
  if (p < 0) return -1;
  if (page_size == 0) {
    if (p >= cache_len) return -1;
    return (long long)b * cache_len + p;
  }
  long long bi = p / page_size;
  if (bi >= max_blocks) return -1;
  int blk = block_table[(long long)b * max_blocks + bi];
  if (blk < 0 || blk >= cache_len) return -1;
  return (long long)blk * page_size + (p % page_size);
}

// ---------------------------------------------------------------------------
// plan: one block of up to 1024 threads (a multiple of 32)
// ---------------------------------------------------------------------------
// Exclusive prefix sum over the block (thread order), and the total: a
// shuffle scan within each warp, then one warp scans the warp totals.
// `smem` holds 32 values.
__device__ long long block_exclusive_scan(long long v, long long *smem, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long t = lane < nw ? smem[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    if (lane < nw) smem[lane] = t;   // inclusive prefix of the warp totals
  }
  __syncthreads();
  const long long before = warp > 0 ? smem[warp - 1] : 0;
  *total = smem[nw - 1];
  __syncthreads();   // smem is reused by the next scan
  return before + x - v;
}

__device__ void make_plan(const PlanSource &src, int B, int P_req, long long cap, int tile, char *ws,
                          const WsLayout &L, unsigned *status) {
  __shared__ long long scan[32];
  // the tile counts and their prefix for up to 1024 plan sequences (a thread each)
  __shared__ long long prefix[1025];
  __shared__ int ntiles[1024];
  long long *tile_prefix = reinterpret_cast<long long *>(ws + L.tile_prefix_off);
  long long *piece_base = reinterpret_cast<long long *>(ws + L.piece_base_off);
  int *ctx_eff = reinterpret_cast<int *>(ws + L.ctx_off);   // [B] ends, then [B] first tokens
  int *beg_eff = ctx_eff + B;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int per = (B + nt - 1) / nt;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);

  long long local = 0;
  for (int b = b0; b < b1; ++b) {
    int end, second;
    plan_entry<true>(src, b, cap, status, &end, &second);
    ctx_eff[b] = end;
    beg_eff[b] = second;
    const long long t = ceil_div_ll(end - (plan_from0(src) ? 0 : second), tile);
    if (B <= 1024) ntiles[b] = (int)t;
    local += t;
  }
  const bool from0 = plan_from0(src);
  auto tiles_of = [&](int b) -> long long {
    return B <= 1024 ? ntiles[b] : ceil_div_ll(ctx_eff[b] - (from0 ? 0 : beg_eff[b]), tile);
  };
  long long Ttot;
  long long run = block_exclusive_scan(local, scan, &Ttot);
  for (int b = b0; b < b1; ++b) {
    tile_prefix[b] = run;
    if (B <= 1024) prefix[b] = run;
    run += tiles_of(b);
  }
  if (tid == 0) {
    tile_prefix[B] = Ttot;
    if (B <= 1024) prefix[B] = Ttot;
  }
  const long long *tpre = B <= 1024 ? prefix : tile_prefix;
  const long long P = Ttot < (long long)P_req ? Ttot : (long long)P_req;

  long long local_pieces = 0;
  for (int b = b0; b < b1; ++b) {
    long long s = tpre[b];
    long long t = tiles_of(b);
    if (t > 0) local_pieces += plan_share_of_tile(s + t - 1, P, Ttot) - plan_share_of_tile(s, P, Ttot) + 1;
  }
  long long n_pieces;
  long long prun = block_exclusive_scan(local_pieces, scan, &n_pieces);
  for (int b = b0; b < b1; ++b) {
    piece_base[b] = prun;
    long long s = tpre[b];
    long long t = tiles_of(b);
    if (t > 0) prun += plan_share_of_tile(s + t - 1, P, Ttot) - plan_share_of_tile(s, P, Ttot) + 1;
  }
  // Each share's first sequence (the first whose tiles reach past the share's
  // first tile), so that the attention kernels need no search; tile_prefix is
  // complete here (the scan above synchronised the block).
  int *share_first = reinterpret_cast<int *>(ws + L.share_first_off);
  for (long long w = tid; w < P; w += nt) {
    share_first[w] = plan_first(tpre, B, w, P, Ttot);
  }
  if (tid == 0) {
    piece_base[B] = n_pieces;
    WsHeader *hd = reinterpret_cast<WsHeader *>(ws);
    hd->B = B;
    hd->P = P;
    hd->Ttot = Ttot;
    hd->n_pieces = n_pieces;
    if (src.drafted == 0 && n_pieces > L.max_pieces) atomicOr(status, kStatusBounds);  // cannot happen by construction
  }
}

__global__ void __launch_bounds__(1024) plan_kernel(PlanSource src, int B, int P_req, long long cap, int tile,
                                                    char *ws, WsLayout L, unsigned *status) {
  pdl_trigger();
  pdl_wait();   // the workspace may still be read by the previous step's combine
  make_plan(src, B, P_req, cap, tile, ws, L, status);
}

// Eight bf16 values with the non-finite ones replaced by zero.
__device__ __forceinline__ uint4 finite_or_zero(uint4 v) {
  auto one = [](uint32_t x) {
    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0x0000ffffu;
    return x;
  };
  return make_uint4(one(v.x), one(v.y), one(v.z), one(v.w));
}

// Tree: block 0 makes the plan while the others copy the blocks that hold
// drafted tokens, kCopyBlocks blocks of kCopyRows rows per sequence (rows of
// 72 16-byte units).  At most 147 KB a sequence, so the time is that of the
// launch and of two dependent reads.  (The plan made in line, with the attention
// kernel waiting for the copy only where it reads it, saved 0.7 us of 25 on one
// short sequence and cost 2 % on long ones, whose kernel then spilled registers.)
constexpr int kCopyRows = 8, kCopyBlocks = kTreeCopyRows / kCopyRows;
__global__ void __launch_bounds__(1024) tree_plan_copy_kernel(PlanSource src, AttnArgs a, int P_req, long long cap) {
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0) {
    make_plan(src, a.B, P_req, cap, a.plan_tile, a.ws, a.L, a.status);
    return;
  }
  const int b = (blockIdx.x - 1) / kCopyBlocks, r0 = (blockIdx.x - 1) % kCopyBlocks * kCopyRows;
  const long long cached = min(max((long long)src.ctx_len[b], 0ll), cap);
  const long long end = min(cached + src.drafted, cap);
  const long long first = cached / kTile * kTile;
  if (first + r0 >= ceil_div_ll(end, kTile) * kTile) return;   // a block that is not there
  uint4 *dst = reinterpret_cast<uint4 *>(a.ws + a.tree.copy_off) + ((long long)b * kTreeCopyRows + r0) * 72;
  for (int u = threadIdx.x; u < kCopyRows * 72; u += blockDim.x) {
    const long long t = first + r0 + u / 72;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t < end) {
      const long long row = token_row(a, b, t);
      if (row >= 0) v = reinterpret_cast<const uint4 *>(a.cache)[row * 72 + u % 72];
      else atomicOr(a.status, kStatusBounds);
      if (t >= cached) v = finite_or_zero(v);
    }
    dst[u] = v;
  }
}

// ---------------------------------------------------------------------------
// generic attention: one warp per head, lanes split the row's features; kBatch
// tokens at a time, their loads in flight together, their products summed by one
// transposing reduction and each exponential taken by one lane.  Bound by that
// chain of loads, shuffles and sums: a token at a time waited for its own loads
// (float32, 4 heads x 144 columns, 16 blocks of each of four sequences: 47 us a
// call, in batches of 16 15 us).
// ---------------------------------------------------------------------------
constexpr int kSimtMaxD = 576;      // d_c + d_r
constexpr int kSimtMaxC = 512;      // d_c
constexpr int kQPerLane = kSimtMaxD / 32;
constexpr int kOPerLane = kSimtMaxC / 32;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// Group of channel f of a cached row (see fp8_group_range).
__device__ __forceinline__ int fp8_group_of(int f, int d_c) {
  return f < d_c ? f / kFp8Group : (d_c + kFp8Group - 1) / kFp8Group + (f - d_c) / kFp8Group;
}

// T: element type of the query; F8: the cache holds E4M3 codes with group
// scales (else elements of type T).  Tree: plan sequence b holds the heads of
// one drafted token (b / T its batch sequence, b % T the token); a drafted
// token that is masked is skipped, so whatever its row holds reaches nothing.
template <typename T, bool F8, bool kTree, int kQ>
__global__ void __launch_bounds__(256) attn_simt_kernel(AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int kO = kQ < kOPerLane ? kQ : kOPerLane;
  // long rows: two at a time keep twice the blocks resident of four (64 heads, 16
  // x 2048 tokens 650 and 850 us; few tokens would rather have four: 42 and 35)
  constexpr int kBatch = kQ <= 6 ? 16 : 2;
  const WsHeader *hd = reinterpret_cast<const WsHeader *>(a.ws);
  const long long P = hd->P, Ttot = hd->Ttot;
  const int w = blockIdx.x;
  if (w >= P) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * (blockDim.x >> 5) + warp;
  if (h >= a.n_h) return;
  const int D = a.d_c + a.d_r;
  const long long *tp = reinterpret_cast<const long long *>(a.ws + a.L.tile_prefix_off);
  const long long *pb = reinterpret_cast<const long long *>(a.ws + a.L.piece_base_off);
  float *opart = reinterpret_cast<float *>(a.ws + a.L.opart_off);
  float *lse = reinterpret_cast<float *>(a.ws + a.L.lse_off);
  const T *cache = reinterpret_cast<const T *>(a.cache);
  const uint8_t *cache8 = reinterpret_cast<const uint8_t *>(a.cache);
  const T *qg = reinterpret_cast<const T *>(a.q_abs);

  const long long t0 = plan_begin(w, P, Ttot), t1 = plan_begin(w + 1, P, Ttot);
  // first sequence whose tiles reach past t0 (found by the plan)
  const int lo = reinterpret_cast<const int *>(a.ws + a.L.share_first_off)[w];
  for (int b = lo; b < a.B && tp[b] < t1; ++b) {
    const long long s0 = t0 > tp[b] ? t0 : tp[b];
    const long long s1 = t1 < tp[b + 1] ? t1 : tp[b + 1];
    if (s0 >= s1) continue;
    const long long piece = pb[b] + (w - plan_share_of_tile(tp[b], P, Ttot));
    const int ctx = plan_ends(a)[b];
    const long long beg = kTree || a.sel ? 0 : plan_seconds(a)[b];
    const long long p_begin = beg + (s0 - tp[b]) * a.plan_tile;
    const long long p_end = min((long long)ctx, beg + (s1 - tp[b]) * a.plan_tile);
    const int seq = kTree ? b / a.tree.T : b;
    const int cached = kTree || a.sel ? plan_seconds(a)[b] : 0;
    const unsigned long long bits = kTree ? a.tree.mask[b] : 0ull;

    float q[kQ];
#pragma unroll
    for (int j = 0; j < kQ; ++j) {
      const int f = lane + 32 * j;
      q[j] = f < D ? to_f(qg[((long long)b * a.n_h + h) * D + f]) : 0.f;
    }
    float o[kO];
#pragma unroll
    for (int j = 0; j < kO; ++j) o[j] = 0.f;
    float m = -CUDART_INF_F, l = 0.f;

    for (long long p0 = p_begin; p0 < p_end; p0 += kBatch) {
      // lane t looks up token t of the batch; -1: masked, past the piece or not there
      long long mine = -1;
      const long long p = p0 + lane;
      if (lane < kBatch && p < p_end && !(kTree && p >= cached && !((bits >> (p - cached)) & 1ull))) {
        mine = a.sel ? selected_row(a, b, p, ctx, cached) : token_row(a, seq, p);
        if (mine < 0) atomicOr(a.status, kStatusBounds);
      }
      // every load of the batch before any conversion, which would wait for it
      T raw[kBatch][F8 ? 1 : kQ];
      uint8_t code[kBatch][F8 ? kQ : 1];
      float sigma[kBatch][F8 ? kQ : 1];
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const long long row = __shfl_sync(0xffffffffu, mine, t);
        const bool there = row >= 0;
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
          const int f = lane + 32 * j;
          const bool ld = there && f < D;
          if (F8) {
            code[t][j] = ld ? cache8[row * D + f] : (uint8_t)0;
            sigma[t][j] = ld ? a.kv_scale[row * a.n_groups + fp8_group_of(f, a.d_c)] : 0.f;
          } else {
            raw[t][j] = ld ? cache[row * D + f] : from_f<T>(0.f);
          }
        }
      }
      float val[kBatch][kQ], x[kBatch];
#pragma unroll
      for (int t = 0; t < kBatch; ++t)
#pragma unroll
        for (int j = 0; j < kQ; ++j) val[t][j] = F8 ? e4m3_value(code[t][F8 ? j : 0]) * sigma[t][F8 ? j : 0] : to_f(raw[t][F8 ? 0 : j]);
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        x[t] = 0.f;
#pragma unroll
        for (int j = 0; j < kQ; ++j) x[t] += q[j] * val[t][j];
      }
      // Sums over the lanes, each exchange halving the tokens a lane is in charge
      // of: lane t ends with the product of token t (mod kBatch).
#pragma unroll
      for (int d = kBatch / 2; d > 0; d >>= 1) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int j = 0; j < d; ++j) {
          const float give = up ? x[j] : x[j + d], keep = up ? x[j + d] : x[j];
          x[j] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
      }
#pragma unroll
      for (int d = kBatch; d < 32; d <<= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
      const bool here = __shfl_sync(0xffffffffu, mine >= 0 ? 1 : 0, lane & (kBatch - 1)) != 0;
      const float s = here ? x[0] * a.scale_log2 : -CUDART_INF_F;   // score in log2 units
      float top = fmaxf(m, s);
#pragma unroll
      for (int d = kBatch / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      // scores of -inf alone so far: -inf - -inf is NaN
      const float m_use = top == -CUDART_INF_F ? 0.f : top;
      const float corr = exp2f(m - m_use), pr = exp2f(s - m_use);
      l = l * corr + (lane < kBatch ? pr : 0.f);
#pragma unroll
      for (int j = 0; j < kO; ++j) o[j] *= corr;
      // An infinity of a drafted row counts as zero behind its score of -inf (any
      // other score of such a row makes its weight NaN).
      if (kTree && __any_sync(0xffffffffu, s == -CUDART_INF_F && here && p0 + (lane & (kBatch - 1)) >= cached)) {
#pragma unroll
        for (int t = 0; t < kBatch; ++t)
#pragma unroll
          for (int j = 0; j < kO; ++j)
            if (p0 + t >= cached && isinf(val[t][j])) val[t][j] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < kBatch; ++t) {
        const float wt = __shfl_sync(0xffffffffu, pr, t);
#pragma unroll
        for (int j = 0; j < kO; ++j)
          if (lane + 32 * j < a.d_c) o[j] += wt * val[t][j];
      }
      m = top;
    }
    l = warp_sum(l);   // a lane's tokens so far
    // a row that attends nothing is zero; a NaN sum stays NaN
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float z = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
    if (kTree) {
      const TreePiece tpc = tree_piece(a, tp, b, w, 0, P, Ttot);
      const long long orow = (long long)b * a.n_h + h, prow = part_row(a.L, tpc.slot, h);
      T *out = reinterpret_cast<T *>(a.tree.out) + orow * a.d_c;
#pragma unroll
      for (int j = 0; j < kO; ++j) {
        const int f = lane + 32 * j;
        if (f >= a.d_c) continue;
        if (tpc.whole) out[f] = from_f<T>(o[j] * inv);
        else opart[prow * a.d_c + f] = o[j] * inv;
      }
      if (lane == 0) {
        if (!tpc.whole) lse[prow] = z;
        else if (a.tree.lse) a.tree.lse[orow] = z;
      }
      continue;
    }
    float *dst = opart + part_row(a.L, piece, h) * (long long)a.d_c;
#pragma unroll
    for (int j = 0; j < kO; ++j) {
      const int f = lane + 32 * j;
      if (f < a.d_c) dst[f] = o[j] * inv;
    }
    if (lane == 0) lse[part_row(a.L, piece, h)] = z;
  }
}

// What a merge subtracts from its pieces' log-sum-exps: their maximum, or 0
// where that is -inf (-inf - -inf is NaN).  A maximum does not show a NaN, so the
// merges take a row for empty by its sum being 0, not by its maximum.
__device__ __forceinline__ float merge_max(float m) { return m == -CUDART_INF_F ? 0.f : m; }

// ---------------------------------------------------------------------------
// log-sum-exp combine, generic form: one block per (sequence, head)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(128) combine_kernel(const char *ws, WsLayout L, int n_h, int d_c,
                                                      T *ctx_lat, float *lse_out) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, h = blockIdx.y;
  const long long *pb = reinterpret_cast<const long long *>(ws + L.piece_base_off);
  const float *lse = reinterpret_cast<const float *>(ws + L.lse_off);
  const float *op = reinterpret_cast<const float *>(ws + L.opart_off);
  const long long p0 = pb[b], p1 = pb[b + 1];
  float m = -CUDART_INF_F;
  for (long long p = p0; p < p1; ++p) m = fmaxf(m, lse[part_row(L, p, h)]);
  T *dst = ctx_lat + ((long long)b * n_h + h) * d_c;
  m = merge_max(m);
  float tot = 0.f;
  for (long long p = p0; p < p1; ++p) tot += expf(lse[part_row(L, p, h)] - m);
  if (tot == 0.f) {
    for (int f = threadIdx.x; f < d_c; f += blockDim.x) dst[f] = from_f<T>(0.f);
    if (lse_out && threadIdx.x == 0) lse_out[(long long)b * n_h + h] = -CUDART_INF_F;
    return;
  }
  const float inv = 1.f / tot;
  for (int f = threadIdx.x; f < d_c; f += blockDim.x) {
    float acc = 0.f;
    for (long long p = p0; p < p1; ++p)
      acc += expf(lse[part_row(L, p, h)] - m) * op[part_row(L, p, h) * (long long)d_c + f];
    dst[f] = from_f<T>(acc * inv);
  }
  if (lse_out && threadIdx.x == 0) lse_out[(long long)b * n_h + h] = m + logf(tot);
}

// ---------------------------------------------------------------------------
// cache append: one block per token; each warp computes a pair of features (of
// the latent part, whose last pair is half one where d_c is odd, or rotary)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) append_simt_kernel(
    const T *h, int T_new, int d, int d_c, int d_r, const int *start_pos, const T *w_dkv,
    const T *w_kr, T *cache, long long cache_len, const int *block_table, int max_blocks,
    int page_size, const double *theta, unsigned *status, float *rows_out, const int *depth) {
  extern __shared__ float sh[];
  const long long tok = blockIdx.x;
  const int b = (int)(tok / T_new), t = (int)(tok % T_new);
  for (int k = threadIdx.x; k < d; k += blockDim.x) sh[k] = to_f(h[tok * d + k]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = d_c + d_r;
  const int unit = blockIdx.y * (blockDim.x >> 5) + warp, latent = (d_c + 1) / 2;
  const int f0 = unit < latent ? 2 * unit : d_c + 2 * (unit - latent);
  if (f0 >= D) return;
  const bool two = f0 + 1 != d_c;   // a second feature
  const T *w0 = f0 < d_c ? w_dkv + (long long)f0 * d : w_kr + (long long)(f0 - d_c) * d;
  const T *w1 = two ? w0 + d : w0;
  float a0 = 0.f, a1 = 0.f;
  for (int k = lane; k < d; k += 32) {
    a0 += to_f(w0[k]) * sh[k];
    a1 += to_f(w1[k]) * sh[k];
  }
  a0 = warp_sum(a0);
  a1 = warp_sum(a1);
  if (lane != 0) return;
  const long long p = (long long)start_pos[b] + t;
  if (f0 >= d_c) {
    const long long rp = depth ? (long long)start_pos[b] + depth[tok] : p;   // the position it is rotated by
    double sn, cs;
    sincos((double)rp * theta[(f0 - d_c) >> 1], &sn, &cs);
    const float c = (float)cs, s = (float)sn;
    const float r0 = a0 * c - a1 * s, r1 = a0 * s + a1 * c;
    a0 = r0;
    a1 = r1;
  }
  if (rows_out) {
    rows_out[tok * D + f0] = a0;
    if (two) rows_out[tok * D + f0 + 1] = a1;
    return;
  }
  const long long row = cache_row(b, p, cache_len, block_table, max_blocks, page_size);
  if (row < 0) {
    atomicOr(status, kStatusBounds);
    return;
  }
  cache[row * D + f0] = from_f<T>(a0);
  if (two) cache[row * D + f0 + 1] = from_f<T>(a1);
}

// ---------------------------------------------------------------------------
// FP8 E4M3 quantisation of cached rows: one warp per row; per 128-channel
// group (over c^KV, then over k^R) sigma = amax / 448 and the codes of
// x / sigma, both divisions rounded to nearest in float32, the conversion
// rounding to nearest even and saturating at 448.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ void fp8_group_range(int g, int d_c, int d_r, int &a, int &e) {
  const int gc = (d_c + kFp8Group - 1) / kFp8Group;
  if (g < gc) {
    a = g * kFp8Group;
    e = min(a + kFp8Group, d_c);
  } else {
    a = d_c + (g - gc) * kFp8Group;
    e = min(a + kFp8Group, d_c + d_r);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) quantize_fp8_kernel(
    const T *src, long long n_rows, int d_c, int d_r, int T_new, const int *start_pos,
    uint8_t *codes, float *scales, long long cache_len, const int *block_table, int max_blocks,
    int page_size, unsigned *status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  if (r >= n_rows) return;
  long long dst = r;
  if (start_pos) {
    const int b = (int)(r / T_new), t = (int)(r % T_new);
    dst = cache_row(b, (long long)start_pos[b] + t, cache_len, block_table, max_blocks, page_size);
    if (dst < 0) {
      if (lane == 0) atomicOr(status, kStatusBounds);
      return;
    }
  }
  const int D = d_c + d_r, G = fp8_num_groups(d_c, d_r);
  const T *x = src + r * D;
  uint8_t *out = codes + dst * D;
  for (int g = 0; g < G; ++g) {
    int a, e;
    fp8_group_range(g, d_c, d_r, a, e);
    float amax = 0.f;
    for (int f = a + lane; f < e; f += 32) amax = fmaxf(amax, fabsf(to_f(x[f])));
    amax = warp_max(amax);
    const float sigma = __fdiv_rn(amax, 448.f);
    for (int f = a + lane; f < e; f += 32)
      out[f] = sigma > 0.f ? (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(to_f(x[f]), sigma), __NV_SATFINITE, __NV_E4M3)
                           : (uint8_t)0;
    if (lane == 0) scales[dst * G + g] = sigma;
  }
}

// ---------------------------------------------------------------------------
// query absorption: one block per (sequence, head)
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) absorb_simt_kernel(const T *q_nope, const T *q_rope,
                                                          const int *pos, const T *w_uk, T *q_abs,
                                                          int n_h, int d_h, int d_c, int d_r,
                                                          const double *theta) {
  extern __shared__ float sq[];
  const int b = blockIdx.x, i = blockIdx.y;
  const long long bi = (long long)b * n_h + i;
  for (int r = threadIdx.x; r < d_h; r += blockDim.x) sq[r] = to_f(q_nope[bi * d_h + r]);
  __syncthreads();
  const int D = d_c + d_r;
  for (int m = threadIdx.x; m < d_c; m += blockDim.x) {
    float acc = 0.f;
    for (int r = 0; r < d_h; ++r) acc += to_f(w_uk[((long long)i * d_h + r) * d_c + m]) * sq[r];
    q_abs[bi * D + m] = from_f<T>(acc);
  }
  const double p = (double)pos[b];
  for (int k = threadIdx.x; k < d_r / 2; k += blockDim.x) {
    const float x0 = to_f(q_rope[bi * d_r + 2 * k]), x1 = to_f(q_rope[bi * d_r + 2 * k + 1]);
    double sn, cs;
    sincos(p * theta[k], &sn, &cs);
    const float c = (float)cs, s = (float)sn;
    q_abs[bi * D + d_c + 2 * k] = from_f<T>(x0 * c - x1 * s);
    q_abs[bi * D + d_c + 2 * k + 1] = from_f<T>(x0 * s + x1 * c);
  }
}

// ---------------------------------------------------------------------------
// output projection: one block per (sequence, head), one warp per output
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) outproj_simt_kernel(const T *ctx, const T *w_uv, T *o,
                                                           int n_h, int d_h, int d_c) {
  const int b = blockIdx.x, i = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const T *c = ctx + ((long long)b * n_h + i) * d_c;
  for (int r = warp; r < d_h; r += nw) {
    const T *wr = w_uv + ((long long)i * d_h + r) * d_c;
    float acc = 0.f;
    for (int k = lane; k < d_c; k += 32) acc += to_f(wr[k]) * to_f(c[k]);
    acc = warp_sum(acc);
    if (lane == 0) o[((long long)b * n_h + i) * d_h + r] = from_f<T>(acc);
  }
}

// Split combine fused with the output projection, CUDA-core form: one block
// per (sequence, head).  The merge is the vectorised combine's arithmetic per
// element (weights exp(lse_p - max) / sum, accumulated in piece order), the
// merged row is rounded to the dtype as ctx_lat would be, and the projection
// is the output-projection kernel's, reading the row from shared memory.
template <typename T>
__global__ void __launch_bounds__(256) combine_outproj_simt_kernel(const char *ws, WsLayout L, int n_h, int d_h,
                                                                   int d_c, const T *w_uv, T *o, T *ctx_lat,
                                                                   float *lse_out) {
  extern __shared__ float sctx[];   // [d_c]
  __shared__ float s_m, s_inv;
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const long long row = (long long)b * n_h + h;
  const long long *pb = reinterpret_cast<const long long *>(ws + L.piece_base_off);
  const float *lse = reinterpret_cast<const float *>(ws + L.lse_off);
  const float *op = reinterpret_cast<const float *>(ws + L.opart_off);
  const long long p0 = pb[b], p1 = pb[b + 1];
  if (warp == 0) {
    float m = -CUDART_INF_F;
    for (long long p = p0 + lane; p < p1; p += 32) m = fmaxf(m, lse[part_row(L, p, h)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    m = merge_max(m);
    float tot = 0.f;
    for (long long p = p0 + lane; p < p1; p += 32) tot += expf(lse[part_row(L, p, h)] - m);
    tot = warp_sum(tot);
    if (lane == 0) {
      s_m = m;
      s_inv = tot == 0.f ? 0.f : 1.f / tot;
      if (lse_out) lse_out[row] = tot == 0.f ? -CUDART_INF_F : m + logf(tot);
    }
  }
  __syncthreads();
  const float m = s_m, inv = s_inv;
  for (int c = threadIdx.x; c < d_c; c += blockDim.x) {
    float acc = 0.f;
    if (inv != 0.f)   // the row attends something
      for (long long p = p0; p < p1; ++p) {
        const float w = expf(lse[part_row(L, p, h)] - m) * inv;
        acc += w * op[part_row(L, p, h) * (long long)d_c + c];
      }
    const T v = from_f<T>(acc);
    if (ctx_lat) ctx_lat[row * d_c + c] = v;
    sctx[c] = to_f(v);
  }
  __syncthreads();
  for (int r = warp; r < d_h; r += nw) {
    const T *wr = w_uv + ((long long)h * d_h + r) * d_c;
    float acc = 0.f;
    for (int k = lane; k < d_c; k += 32) acc += to_f(wr[k]) * sctx[k];
    acc = warp_sum(acc);
    if (lane == 0) o[row * d_h + r] = from_f<T>(acc);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) linear_simt_kernel(const T *o, const T *w_o, T *u, int K, int d) {
  const int b = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.y * (blockDim.x >> 5) + warp;
  if (j >= d) return;
  const T *wr = w_o + (long long)j * K;
  const T *x = o + (long long)b * K;
  float acc = 0.f;
  for (int k = lane; k < K; k += 32) acc += to_f(wr[k]) * to_f(x[k]);
  acc = warp_sum(acc);
  if (lane == 0) u[(long long)b * d + j] = from_f<T>(acc);
}

}  // namespace

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
cudaError_t launch_plan(const PlanSource &src, int B, int P, long long cap, int tile, char *ws, const WsLayout &L,
                        unsigned *status, cudaStream_t s) {
  if (tile < kTile || tile % kTile != 0) return cudaErrorInvalidValue;
  // one thread per sequence up to 1024 (each thread takes a run of sequences beyond)
  const int threads = B >= 1024 ? 1024 : (B <= 32 ? 32 : (B + 31) / 32 * 32);
  return launch_pdl(plan_kernel, dim3(1), dim3(threads), 0, s, 1, src, B, P, cap, tile, ws, L, status);
}

cudaError_t launch_tree_plan_copy(const PlanSource &src, const AttnArgs &a, int P, long long cap, cudaStream_t s) {
  const long long blocks = 1 + (long long)(a.B / src.runs) * kCopyBlocks;
  if (a.d_c + a.d_r != 576 || src.drafted > kTreeMaxDrafted || blocks > 0x7fffffffLL) return cudaErrorNotSupported;
  const int threads = a.B >= 1024 ? 1024 : (a.B <= 288 ? 288 : (a.B + 31) / 32 * 32);
  return launch_pdl(tree_plan_copy_kernel, dim3((unsigned)blocks), dim3(threads), 0, s, 1, src, a, P, cap);
}

namespace {
template <typename T, bool F8, bool kTree>
cudaError_t launch_simt(const AttnArgs &a, int P, cudaStream_t s) {
  if (a.d_c + a.d_r > kSimtMaxD || a.d_c > kSimtMaxC) return cudaErrorNotSupported;
  const int warps = a.n_h < 8 ? a.n_h : 8;
  const dim3 grid(P, (a.n_h + warps - 1) / warps);
  // rows of up to 192 columns: six a lane, which leaves registers for longer batches
  if (a.d_c + a.d_r <= 192) return launch_pdl(attn_simt_kernel<T, F8, kTree, 6>, grid, dim3(warps * 32), 0, s, 1, a);
  return launch_pdl(attn_simt_kernel<T, F8, kTree, kQPerLane>, grid, dim3(warps * 32), 0, s, 1, a);
}
}  // namespace

cudaError_t launch_attn_simt(const AttnArgs &a, int P, bool fp32, cudaStream_t s) {
  if (a.kv_scale) return fp32 ? launch_simt<float, true, false>(a, P, s) : launch_simt<__nv_bfloat16, true, false>(a, P, s);
  return fp32 ? launch_simt<float, false, false>(a, P, s) : launch_simt<__nv_bfloat16, false, false>(a, P, s);
}

cudaError_t launch_tree_attn_simt(const AttnArgs &a, int P, bool fp32, cudaStream_t s) {
  return fp32 ? launch_simt<float, false, true>(a, P, s) : launch_simt<__nv_bfloat16, false, true>(a, P, s);
}

// Vectorised combine for d_c a multiple of 4 and at most 512: `segs` warps per
// (sequence, head), each for 128 / segs of every 128 float4 columns, 8 warps
// per block.  A warp reduces the pieces' log-sum-exps across its lanes; then
// the lanes compute the weights of 32 pieces at a time, one each, and pass them
// round by shuffles while the loads of kAhead pieces are in flight.  With
// many rows one warp each fills the GPU; with few (long contexts split many
// times) four warps a row and the loads in flight take the place of the missing
// rows (256 rows of 37 pieces: 10.0 and 5.3 us; sixteen loads in flight instead
// of eight took most of 3 us off a sparse attention of 20.6).
template <typename T>
__device__ __forceinline__ void store4(T *dst, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float *dst, float4 v) {
  *reinterpret_cast<float4 *>(dst) = v;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *dst, float4 v) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t *>(&lo);
  u.y = *reinterpret_cast<uint32_t *>(&hi);
  *reinterpret_cast<uint2 *>(dst) = u;
}

template <typename T, int kPer>   // float4 columns of a lane: 4 (one warp a row) or 1 (four warps a row)
__global__ void __launch_bounds__(256, kPer == 1 ? 2 : 4) combine_vec_kernel(const char *ws, WsLayout L, int B, int n_h, int d_c,
                                                             T *ctx_lat, float *lse_out) {
  pdl_trigger();
  pdl_wait();
  constexpr int kSegs = 4 / kPer;
  constexpr int kAhead = kPer == 1 ? 16 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * 8 + warp;
  const long long row = unit / kSegs;   // = b * n_h + h
  const int f0 = (int)(unit % kSegs) * 32 * kPer + lane;
  if (row >= (long long)B * n_h) return;
  const int b = (int)plan_div(row, n_h), h = (int)(row - (long long)b * n_h);
  const long long *pb = reinterpret_cast<const long long *>(ws + L.piece_base_off);
  const float *lse = reinterpret_cast<const float *>(ws + L.lse_off) + part_row(L, pb[b], h);
  const int n = (int)(pb[b + 1] - pb[b]);   // the row's pieces are consecutive
  const int n4 = d_c / 4;
  const float4 *src = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(ws + L.opart_off) +
                                                       part_row(L, pb[b], h) * (long long)d_c) + f0;
  // Partials j0 .. of the row; the first batch is requested before the weights
  // are known.
  float4 v[kAhead][kPer];
  auto request = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        v[j][i] = j0 + j < n && f0 + 32 * i < n4 ? __ldg(src + (long long)(j0 + j) * n4 + 32 * i)
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  request(0);
  const float l0 = lane < n ? lse[lane] : -CUDART_INF_F;
  float m = l0;
  for (int p = 32 + lane; p < n; p += 32) m = fmaxf(m, lse[p]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  T *dst = ctx_lat + row * d_c;
  m = merge_max(m);
  float tot = lane < n ? expf(l0 - m) : 0.f;
  for (int p = 32 + lane; p < n; p += 32) tot += expf(lse[p] - m);
  tot = warp_sum(tot);
  if (tot == 0.f) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (f0 + 32 * i < n4) store4<T>(dst + 4 * (f0 + 32 * i), make_float4(0.f, 0.f, 0.f, 0.f));
    if (lse_out && f0 == 0) lse_out[row] = -CUDART_INF_F;
    return;
  }
  const float inv = 1.f / tot;
  float4 acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float wl = lane < n ? expf(l0 - m) * inv : 0.f;
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    if (j0 > 0) {
      request(j0);
      if ((j0 & 31) == 0) wl = j0 + lane < n ? expf(lse[j0 + lane] - m) * inv : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float w = __shfl_sync(0xffffffffu, wl, (j0 + j) & 31);
      if (j0 + j >= n) continue;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        acc[i].x += w * v[j][i].x;
        acc[i].y += w * v[j][i].y;
        acc[i].z += w * v[j][i].z;
        acc[i].w += w * v[j][i].w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (f0 + 32 * i < n4) store4<T>(dst + 4 * (f0 + 32 * i), acc[i]);
  if (lse_out && f0 == 0) lse_out[row] = m + logf(tot);
}

cudaError_t launch_combine(const mla_config &cfg, const char *ws, const WsLayout &L, int B,
                           void *ctx_lat, float *lse, cudaStream_t s, bool out_f32) {
  const bool f32 = out_f32 || cfg.dtype == MLA_FP32;
  const size_t esz = f32 ? 4 : 2;
  if (cfg.d_c % 4 == 0 && cfg.d_c <= 512 && ((uintptr_t)ctx_lat % (4 * esz)) == 0 &&
      ((uintptr_t)ws % 16) == 0) {
    const long long rows = (long long)B * cfg.n_h;
    // Four warps a row while their blocks are resident at once (two an SM: 592
    // rows), or for rows of sixteen pieces, as long contexts have them; other rows
    // do better with one warp each (one / four, us: 512 rows of 5 pieces 3.1 / 2.6,
    // 1024 of 3 3.2 / 4.1, 2048 of 3 3.9 / 7.0, 1024 of 16 7.1 / 5.0, 2048 of 16
    // 9.8 / 8.0).
    const bool split = rows <= 592 || L.max_pieces - B >= 16ll * B;
    const unsigned blocks = (unsigned)((rows * (split ? 4 : 1) + 7) / 8);
    auto go = [&](auto kern, auto *out) {
      return launch_pdl(kern, dim3(blocks), dim3(256), 0, s, 1, ws, L, B, cfg.n_h, cfg.d_c, out, lse);
    };
    if (f32)
      return split ? go(combine_vec_kernel<float, 1>, (float *)ctx_lat) : go(combine_vec_kernel<float, 4>, (float *)ctx_lat);
    return split ? go(combine_vec_kernel<__nv_bfloat16, 1>, (__nv_bfloat16 *)ctx_lat)
                 : go(combine_vec_kernel<__nv_bfloat16, 4>, (__nv_bfloat16 *)ctx_lat);
  }
  dim3 grid(B, cfg.n_h);
  if (f32)
    return launch_pdl(combine_kernel<float>, grid, dim3(128), 0, s, 1, ws, L, cfg.n_h, cfg.d_c, (float *)ctx_lat, lse);
  else
    return launch_pdl(combine_kernel<__nv_bfloat16>, grid, dim3(128), 0, s, 1, ws, L, cfg.n_h, cfg.d_c,
                      (__nv_bfloat16 *)ctx_lat, lse);
}

// ---------------------------------------------------------------------------
// merge of R token-range results (split-KV across devices): one warp per
// (sequence, head) row; the same log-sum-exp algebra as the combine, over the
// R float32 results [R, B, n_h, d_c] and their log-sum-exps [R, B, n_h], in
// range order.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) merge_ranges_kernel(const float *parts, const float *lse_parts, int R,
                                                           int B, int n_h, int d_c, T *ctx_lat, float *lse_out) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + warp;   // = b * n_h + h
  const long long rows = (long long)B * n_h;
  if (row >= rows) return;
  float m = -CUDART_INF_F;
  for (int r = lane; r < R; r += 32) m = fmaxf(m, lse_parts[r * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  T *dst = ctx_lat + row * d_c;
  m = merge_max(m);
  float tot = 0.f;
  for (int r = lane; r < R; r += 32) tot += expf(lse_parts[r * rows + row] - m);
  tot = warp_sum(tot);
  if (tot == 0.f) {
    for (int f = lane; f < d_c; f += 32) dst[f] = from_f<T>(0.f);
    if (lse_out && lane == 0) lse_out[row] = -CUDART_INF_F;
    return;
  }
  const float inv = 1.f / tot;
  for (int f = lane; f < d_c; f += 32) {
    float acc = 0.f;
    for (int r = 0; r < R; ++r) acc += expf(lse_parts[r * rows + row] - m) * inv * parts[(r * rows + row) * d_c + f];
    dst[f] = from_f<T>(acc);
  }
  if (lse_out && lane == 0) lse_out[row] = m + logf(tot);
}

cudaError_t launch_merge_ranges(const mla_config &cfg, const float *parts, const float *lse_parts, int R, int B,
                                void *ctx_lat, float *lse, cudaStream_t s) {
  const long long rows = (long long)B * cfg.n_h;
  const unsigned blocks = (unsigned)((rows + 7) / 8);
  if (cfg.dtype == MLA_FP32)
    return launch_pdl(merge_ranges_kernel<float>, dim3(blocks), dim3(256), 0, s, 1, parts, lse_parts, R, B,
                      cfg.n_h, cfg.d_c, (float *)ctx_lat, lse);
  return launch_pdl(merge_ranges_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, s, 1, parts, lse_parts, R, B,
                    cfg.n_h, cfg.d_c, (__nv_bfloat16 *)ctx_lat, lse);
}

cudaError_t launch_append_simt(const mla_config &cfg, const void *h, int B, int T,
                               const int *start_pos, const void *w_dkv, const void *w_kr,
                               void *cache, long long cache_len, const int *block_table,
                               int max_blocks, const double *theta, unsigned *status,
                               cudaStream_t s, float *rows_out, const int *depth) {
  const int units = (cfg.d_c + 1) / 2 + cfg.d_r / 2;
  dim3 grid((unsigned)((long long)B * T), (units + 7) / 8);
  const size_t smem = sizeof(float) * cfg.d_model;
  if (smem > 48 * 1024) return cudaErrorNotSupported;
  if (cfg.dtype == MLA_FP32)
    append_simt_kernel<float><<<grid, 256, smem, s>>>(
        (const float *)h, T, cfg.d_model, cfg.d_c, cfg.d_r, start_pos, (const float *)w_dkv,
        (const float *)w_kr, (float *)cache, cache_len, block_table, max_blocks, cfg.page_size,
        theta, status, rows_out, depth);
  else
    append_simt_kernel<__nv_bfloat16><<<grid, 256, smem, s>>>(
        (const __nv_bfloat16 *)h, T, cfg.d_model, cfg.d_c, cfg.d_r, start_pos,
        (const __nv_bfloat16 *)w_dkv, (const __nv_bfloat16 *)w_kr, (__nv_bfloat16 *)cache,
        cache_len, block_table, max_blocks, cfg.page_size, theta, status, rows_out, depth);
  return cudaGetLastError();
}

cudaError_t launch_quantize_fp8(const mla_config &cfg, const void *src, bool src_f32, long long n_rows,
                                int T, const int *start_pos, uint8_t *codes, float *scales,
                                long long cache_len, const int *block_table, int max_blocks,
                                unsigned *status, cudaStream_t s) {
  if (n_rows <= 0) return cudaSuccess;
  const long long blocks = (n_rows + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
  if (src_f32 || cfg.dtype == MLA_FP32)
    quantize_fp8_kernel<float><<<(unsigned)blocks, 256, 0, s>>>(
        (const float *)src, n_rows, cfg.d_c, cfg.d_r, T, start_pos, codes, scales, cache_len,
        block_table, max_blocks, cfg.page_size, status);
  else
    quantize_fp8_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, s>>>(
        (const __nv_bfloat16 *)src, n_rows, cfg.d_c, cfg.d_r, T, start_pos, codes, scales, cache_len,
        block_table, max_blocks, cfg.page_size, status);
  return cudaGetLastError();
}

cudaError_t launch_absorb_simt(const mla_config &cfg, const void *q_nope, const void *q_rope,
                               const int *pos, const void *w_uk, void *q_abs, int B,
                               const double *theta, cudaStream_t s) {
  dim3 grid(B, cfg.n_h);
  const size_t smem = sizeof(float) * cfg.d_h;
  if (cfg.dtype == MLA_FP32)
    absorb_simt_kernel<float><<<grid, 256, smem, s>>>(
        (const float *)q_nope, (const float *)q_rope, pos, (const float *)w_uk, (float *)q_abs,
        cfg.n_h, cfg.d_h, cfg.d_c, cfg.d_r, theta);
  else
    absorb_simt_kernel<__nv_bfloat16><<<grid, 256, smem, s>>>(
        (const __nv_bfloat16 *)q_nope, (const __nv_bfloat16 *)q_rope, pos,
        (const __nv_bfloat16 *)w_uk, (__nv_bfloat16 *)q_abs, cfg.n_h, cfg.d_h, cfg.d_c, cfg.d_r,
        theta);
  return cudaGetLastError();
}

cudaError_t launch_outproj_simt(const mla_config &cfg, const void *ctx_lat, const void *w_uv,
                                void *o, int B, cudaStream_t s) {
  dim3 grid(B, cfg.n_h);
  if (cfg.dtype == MLA_FP32)
    outproj_simt_kernel<float><<<grid, 256, 0, s>>>((const float *)ctx_lat, (const float *)w_uv,
                                                    (float *)o, cfg.n_h, cfg.d_h, cfg.d_c);
  else
    outproj_simt_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        (const __nv_bfloat16 *)ctx_lat, (const __nv_bfloat16 *)w_uv, (__nv_bfloat16 *)o, cfg.n_h,
        cfg.d_h, cfg.d_c);
  return cudaGetLastError();
}

cudaError_t launch_combine_outproj_simt(const mla_config &cfg, const char *ws, const WsLayout &L, int B,
                                        const void *w_uv, void *o, void *ctx_lat, float *lse, cudaStream_t s) {
  if (B > 0x7fffffff || cfg.n_h > 65535) return cudaErrorNotSupported;
  const dim3 grid(B, cfg.n_h);
  const size_t smem = sizeof(float) * cfg.d_c;
  if (cfg.dtype == MLA_FP32)
    return launch_pdl(combine_outproj_simt_kernel<float>, grid, dim3(256), smem, s, 1, ws, L, cfg.n_h, cfg.d_h,
                      cfg.d_c, (const float *)w_uv, (float *)o, (float *)ctx_lat, lse);
  return launch_pdl(combine_outproj_simt_kernel<__nv_bfloat16>, grid, dim3(256), smem, s, 1, ws, L, cfg.n_h,
                    cfg.d_h, cfg.d_c, (const __nv_bfloat16 *)w_uv, (__nv_bfloat16 *)o, (__nv_bfloat16 *)ctx_lat,
                    lse);
}

cudaError_t launch_linear_simt(const void *x, const void *w, void *y, int M, int K, int N, bool fp32,
                               cudaStream_t s) {
  // y[N, M] = x[N, K] w[M, K]^T: one warp per output element.
  if (M <= 0 || N <= 0 || K <= 0 || (M + 7) / 8 > 65535) return cudaErrorNotSupported;
  dim3 grid(N, (M + 7) / 8);
  if (fp32)
    linear_simt_kernel<float><<<grid, 256, 0, s>>>((const float *)x, (const float *)w, (float *)y, K, M);
  else
    linear_simt_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>((const __nv_bfloat16 *)x, (const __nv_bfloat16 *)w,
                                                       (__nv_bfloat16 *)y, K, M);
  return cudaGetLastError();
}

cudaError_t launch_wo_simt(const mla_config &cfg, const void *o, const void *w_o, void *u, int B,
                           cudaStream_t s) {
  return launch_linear_simt(o, w_o, u, cfg.d_model, cfg.n_h * cfg.d_h, B, cfg.dtype == MLA_FP32, s);
}

}  // namespace mla
