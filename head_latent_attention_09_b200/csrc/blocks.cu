// Selection of cached blocks for sparse decode attention: the blocks' mean
// rows, their scores against a sequence's query heads, and the best k.
//
// A block is 64 consecutive tokens of a sequence (the last one may be partial).
//   mean:   key_j = (sum over the block's n_j tokens of [c ; k^R]) / n_j
//   score:  x_ij = q_abs_i . key_j / sqrt(d_h + d_r) + log n_j,
//           score_j = sum over heads i of softmax_j(x_i)_j
// i.e. the attention every head would pay block j if each of the block's
// tokens had the block's mean row, added over the heads (all heads of absorbed
// attention read the same rows, so one selection serves them all).
#include <math_constants.h>

#include "ptx.cuh"

namespace mla {
namespace {

template <typename T> __device__ __forceinline__ float widen(T x);
template <> __device__ __forceinline__ float widen<float>(float x) { return x; }
template <> __device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// ---------------------------------------------------------------------------
// block means.  One block of threads per cached block: thread (g, u) adds
// column unit u (V elements, 16 bytes where the alignment allows) of the rows
// g, g + G, ..., all loads of a batch in flight, and the G partial sums meet
// in shared memory.  It reads every row once and writes 1/64 of that: bound
// by HBM for a whole prompt, by the launch for a decode step.
// ---------------------------------------------------------------------------
constexpr int kKeyThreads = 288;     // bf16 rows of 576: 72 units x 4 row groups
constexpr int kKeyBatch = 8;         // rows a thread has in flight (x 3 resident blocks: 110 KB an SM)

template <typename T, int V>
struct alignas(sizeof(T) * V) Unit {
  T e[V];
};

template <typename T, int V>
__global__ void __launch_bounds__(kKeyThreads, 3) block_keys_kernel(AttnArgs a, const int *ctx_begin, const int *ctx_len,
                                                                 T *keys, int key_blocks, int D) {
  __shared__ float part[kKeyThreads * V];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const long long cap = a.page_size ? (long long)a.max_blocks * a.page_size : a.cache_len;
  long long end = ctx_len[b], beg = ctx_begin ? ctx_begin[b] : 0;
  if (end < 0 || end > cap || beg < 0) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
    end = min(max(end, 0ll), cap);
    beg = max(beg, 0ll);
  }
  if (beg >= end) return;
  const int units = D / V;
  const int upb = min(units, kKeyThreads);        // units at a time
  const int G = kKeyThreads / upb;                // row groups
  const int g = threadIdx.x / upb, ul = threadIdx.x % upb;
  const Unit<T, V> *cache = reinterpret_cast<const Unit<T, V> *>(a.cache);
  for (long long j = beg / kTile + blockIdx.x; j * kTile < end; j += gridDim.x) {
    if (j >= key_blocks) {
      if (threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
      return;
    }
    const int n = (int)min((long long)kTile, end - j * kTile);
    // a page of a multiple of 64 tokens holds the block's rows one after another
    const bool run = a.page_size % kTile == 0;
    const long long first = token_row(a, b, j * kTile);
    if (run && first < 0) {
      if (threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
      continue;
    }
    for (int u0 = 0; u0 < units; u0 += upb) {
      const int u = u0 + ul;
      float acc[V];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = 0.f;
      if (g < G && u < units) {
        if (run && n == kTile && kTile % (G * kKeyBatch) == 0) {
          const Unit<T, V> *p = cache + (first + g) * units + u;
          const long long step = (long long)G * units;
#pragma unroll 1
          for (int r0 = 0; r0 < kTile; r0 += G * kKeyBatch, p += kKeyBatch * step) {
            Unit<T, V> x[kKeyBatch];
#pragma unroll
            for (int k = 0; k < kKeyBatch; ++k) x[k] = p[k * step];
#pragma unroll
            for (int k = 0; k < kKeyBatch; ++k)
#pragma unroll
              for (int e = 0; e < V; ++e) acc[e] += widen<T>(x[k].e[e]);
          }
        } else {
#pragma unroll 1
          for (int r = g; r < n; r += G) {
            const long long row = run ? first + r : token_row(a, b, j * kTile + r);
            if (row < 0) {
              atomicOr(a.status, kStatusBounds);
              continue;
            }
            const Unit<T, V> x = cache[row * units + u];
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += widen<T>(x.e[e]);
          }
        }
        if (g > 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) part[(g * upb + ul) * V + e] = acc[e];
        }
      }
      __syncthreads();
      if (g == 0 && u < units) {
        for (int gg = 1; gg < G; ++gg)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += part[(gg * upb + ul) * V + e];
        Unit<T, V> o;   // the one rounding: to the type the keys are kept in, that of the cache's rows
#pragma unroll
        for (int e = 0; e < V; ++e) o.e[e] = narrow<T>(acc[e] / (float)n);
        reinterpret_cast<Unit<T, V> *>(keys)[((long long)b * key_blocks + j) * units + u] = o;
      }
      __syncthreads();
    }
  }
}

template <typename T, int V>
cudaError_t launch_keys(const AttnArgs &a, const int *ctx_begin, const int *ctx_len, int B, int max_new, void *keys,
                        int key_blocks, int D, cudaStream_t s) {
  const long long most = std::min<long long>(((long long)max_new + kTile - 2) / kTile + 1, key_blocks);
  const dim3 grid((unsigned)std::max<long long>(most, 1), B);
  return launch_pdl(block_keys_kernel<T, V>, grid, dim3(kKeyThreads), 0, s, 1, a, ctx_begin, ctx_len, (T *)keys,
                    key_blocks, D);
}

// ---------------------------------------------------------------------------
// scores, first half: x (in log2 units) of a tile of 128 blocks against the
// heads, and per head the tile's maximum and sum of 2^(x - maximum).
// ---------------------------------------------------------------------------
constexpr int kScoreTile = 128;

__device__ __forceinline__ int blocks_of(int ctx) { return ctx <= 0 ? 0 : (ctx + kTile - 1) / kTile; }
// log2 of the tokens in block j of a sequence of ctx tokens
__device__ __forceinline__ float log2_tokens(int j, int ctx) {
  const int n = ctx - j * kTile;
  return n >= kTile ? 6.f : log2f((float)n);
}

// CUDA cores: one warp per head, the query row in registers.
template <typename T>
__global__ void __launch_bounds__(256) score_logits_simt_kernel(const T *q_abs, const T *keys, int key_blocks,
                                                                const int *ctx_len, int n_h, int D, float scale_log2,
                                                                float *logits, float2 *stats, ScoreLayout L) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x, b = blockIdx.z, h = blockIdx.y * 8 + warp;
  if (h >= n_h) return;
  const int ctx = ctx_len[b], nb = min(blocks_of(ctx), key_blocks);
  const int j1 = min(nb, (tile + 1) * kScoreTile);
  float q[18];
#pragma unroll
  for (int i = 0; i < 18; ++i) {
    const int f = lane + 32 * i;
    q[i] = f < D ? widen<T>(q_abs[((long long)b * n_h + h) * D + f]) : 0.f;
  }
  float m = -CUDART_INF_F, sum = 0.f;
  for (int j = tile * kScoreTile; j < j1; ++j) {
    const T *key = keys + ((long long)b * key_blocks + j) * D;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 18; ++i) {
      const int f = lane + 32 * i;
      if (f < D) x += q[i] * widen<T>(key[f]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x = x * scale_log2 + log2_tokens(j, ctx);
    const float m2 = fmaxf(m, x);
    sum = sum * exp2f(m - m2) + exp2f(x - m2);
    m = m2;
    if (lane == 0) logits[((long long)b * L.tiles * kScoreTile + j) * L.head_rows + h] = x;
  }
  if (lane == 0) stats[((long long)b * L.tiles + tile) * L.head_rows + h] = make_float2(m, sum);
}

// Tensor cores (rows of 576 bf16): S = Q K^T with the heads as M (128, zero
// filled) and the tile's 128 blocks as N, so that a thread owns one head's row
// of the accumulator and its statistics need no exchange.  Nine 64-column
// chunks of both operands stream through a ring of six 32 KB stages.  At one
// to a few tiles per sequence the time is that of one load-multiply-store
// chain; the means are 1/64 of the cache's bytes.
constexpr int kSThreads = 192;
constexpr int kSStages = 6;
constexpr int kSStage = 32768;
constexpr int kSSmem = kSStages * kSStage + 1024;

__global__ void __launch_bounds__(kSThreads, 1)
    score_logits_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                           int key_blocks, const int *ctx_len, int n_h, float scale_log2, float *logits, float2 *stats,
                           ScoreLayout L, unsigned *status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kSStages], empty[kSStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x, h0 = blockIdx.y * 128, b = blockIdx.z;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(&done, 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_slot, 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  const int ctx = ctx_len[b], nb = min(blocks_of(ctx), key_blocks);
  const bool work = tile * kScoreTile < nb;
  if (warp == 0) {
    if (work && ptx::elect_one()) {
      ptx::tma_prefetch_desc(&mapQ);
      ptx::tma_prefetch_desc(&mapK);
      for (int c = 0; c < 9; ++c) {
        const int s = c % kSStages;
        if (c >= kSStages && !ptx::mbar_wait(&empty[s], 0, status, &abort_flag)) break;
        ptx::mbar_arrive_expect_tx(&full[s], kSStage);
        ptx::tma_load_3d(sm + s * kSStage, &mapQ, &full[s], 64 * c, h0, b);
        ptx::tma_load_3d(sm + s * kSStage + 16384, &mapK, &full[s], 64 * c, tile * kScoreTile, b);
      }
    }
  } else if (warp == 1) {
    if (work && ptx::elect_one()) {
      constexpr uint32_t id = idesc_bf16(128, kScoreTile, false, false);
      bool ok = true;
      for (int c = 0; c < 9 && ok; ++c) {
        const int s = c % kSStages;
        ok = ptx::mbar_wait(&full[s], c / kSStages, status, &abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t at = ptx::smem_u32(sm + s * kSStage);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::mma_bf16_ss(tmem, ptx::sdesc(at + 32 * k, 16, 1024, 2), ptx::sdesc(at + 16384 + 32 * k, 16, 1024, 2),
                           id, (c | k) != 0 ? 1u : 0u);
        ptx::mma_commit(&empty[s]);
      }
      if (ok) ptx::mma_commit(&done);
    }
  } else if (work) {
    const int q = warp & 3, h = h0 + 32 * q + lane;
    bool ok = true;
    if (lane == 0) ok = ptx::mbar_wait(&done, 0, status, &abort_flag);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (ok && lane != 0) ptx::mbar_test_wait(&done, 0);
    __syncwarp();
    if (ok && h0 + 32 * q < n_h) {
      ptx::tc_fence_after();
      float v[kScoreTile];
      const uint32_t at = tmem + ((uint32_t)(q * 32) << 16);
      ptx::tmem_ld64_sync(at, reinterpret_cast<uint32_t *>(v));
      ptx::tmem_ld64_sync(at + 64, reinterpret_cast<uint32_t *>(v) + 64);
      const int j0 = tile * kScoreTile;
      float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
      const float last = log2_tokens(nb - 1, ctx);
#pragma unroll
      for (int j = 0; j < kScoreTile; ++j) {
        const int jj = j0 + j;
        v[j] = jj < nb ? fmaf(v[j], scale_log2, jj == nb - 1 ? last : 6.f) : -CUDART_INF_F;
        mx[j & 3] = fmaxf(mx[j & 3], v[j]);
      }
      const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      float *out = logits + ((long long)b * L.tiles * kScoreTile + j0) * L.head_rows + h;
      float sm4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kScoreTile; ++j) {
        sm4[j & 3] += ptx::exp2_approx(v[j] - m);
        if (j0 + j < nb) out[(long long)j * L.head_rows] = v[j];
      }
      stats[((long long)b * L.tiles + tile) * L.head_rows + h] = make_float2(m, (sm4[0] + sm4[1]) + (sm4[2] + sm4[3]));
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 128);
  }
}

// Second half: score_j = sum over heads of 2^(x - lse of the head), one warp
// per block, the heads across the lanes; blocks the sequence lacks score 0.
constexpr int kSumBlocks = 64;
__global__ void __launch_bounds__(256) score_sum_kernel(const float *logits, const float2 *stats, ScoreLayout L,
                                                        int key_blocks, const int *ctx_len, int n_h, float *scores,
                                                        unsigned *status) {
  extern __shared__ float lse[];   // [n_h], log2 units
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y, j0 = blockIdx.x * kSumBlocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int all = blocks_of(ctx_len[b]);
  const int nb = min(all, key_blocks);
  if ((all > key_blocks || ctx_len[b] < 0) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, kStatusBounds);
  const int tiles = (nb + kScoreTile - 1) / kScoreTile;
  if (j0 < nb) {
    for (int h = threadIdx.x; h < n_h; h += blockDim.x) {
      const float2 *st = stats + (long long)b * L.tiles * L.head_rows + h;
      float m = -CUDART_INF_F, sum = 0.f;
      for (int t = 0; t < tiles; ++t) m = fmaxf(m, st[(long long)t * L.head_rows].x);
      for (int t = 0; t < tiles; ++t) {
        const float2 v = st[(long long)t * L.head_rows];
        sum += v.y * exp2f(v.x - m);
      }
      lse[h] = m + log2f(sum);
    }
  }
  __syncthreads();
  for (int j = j0 + warp; j < min(j0 + kSumBlocks, key_blocks); j += 8) {
    float s = 0.f;
    if (j < nb) {
      const float *x = logits + ((long long)b * L.tiles * kScoreTile + j) * L.head_rows;
      for (int h = lane; h < n_h; h += 32) s += exp2f(x[h] - lse[h]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (lane == 0) scores[(long long)b * key_blocks + j] = s;
  }
}

// ---------------------------------------------------------------------------
// selection: the k best blocks of a sequence in rising order.  One block of
// threads per sequence, the scores in shared memory as unsigned integers of
// the same order.  The k-th largest is found two bits at a time (16 rounds of
// three counts, no atomics on shared bins, whose order would not matter but
// whose collisions would: softmax masses share their leading bits), then one
// scan over the threads' runs of blocks places the winners.  The order is
// total (value, then the lower index), so the result is the same however the
// threads run.
// ---------------------------------------------------------------------------
constexpr int kSelMaxBlocks = 49152;   // 192 KB of keys

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;                     // NaN ranks below everything
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(1024) block_select_kernel(const float *scores, int n_blocks, const int *ctx_len,
                                                            int k, int n_first, int n_last, int *sel, int *n_sel,
                                                            unsigned *status) {
  extern __shared__ uint32_t key[];
  __shared__ int cnt[16][3];
  __shared__ int wsum[32][2];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int all = blocks_of(ctx_len[b]);
  const int n = min(all, n_blocks);
  if (tid == 0 && (all > n_blocks || ctx_len[b] < 0)) atomicOr(status, kStatusBounds);
  if (tid < 48) cnt[tid / 3][tid % 3] = 0;
  if (nt < 48 && tid < 16) cnt[(tid + 32) / 3][(tid + 32) % 3] = 0;
  int *out = sel + (long long)b * k;
  const int take = min(n, k);
  for (int i = take + tid; i < k; i += nt) out[i] = -1;
  if (tid == 0) n_sel[b] = take;
  if (take == n) {
    for (int i = tid; i < n; i += nt) out[i] = i;
    return;
  }
  const float *x = scores + (long long)b * n_blocks;
  for (int i = tid; i < n; i += nt) key[i] = i < n_first || i >= n - n_last ? 0xffffffffu : order_key(x[i]);
  __syncthreads();
  uint32_t v = 0;   // largest value with at least `take` keys >= it
#pragma unroll 1
  for (int r = 0; r < 16; ++r) {
    const uint32_t bit = 1u << (30 - 2 * r);
    int c1 = 0, c2 = 0, c3 = 0;
    for (int i = tid; i < n; i += nt) {
      const uint32_t kk = key[i];
      c1 += kk >= v + bit;
      c2 += kk >= v + 2 * bit;
      c3 += kk >= v + 3 * bit;
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if (lane < 3) atomicAdd(&cnt[r][lane], lane == 0 ? c1 : (lane == 1 ? c2 : c3));
    __syncthreads();
    v += cnt[r][2] >= take ? 3 * bit : (cnt[r][1] >= take ? 2 * bit : (cnt[r][0] >= take ? bit : 0u));
  }
  // Thread t places its run of consecutive blocks: those above v, and the
  // first of those equal to it.
  const int per = (n + nt - 1) / nt, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    gt += key[i] > v;
    eq += key[i] == v;
  }
  int g = gt, e = eq;   // inclusive prefix over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int g2 = __shfl_up_sync(0xffffffffu, g, o), e2 = __shfl_up_sync(0xffffffffu, e, o);
    if (lane >= o) {
      g += g2;
      e += e2;
    }
  }
  if (lane == 31) {
    wsum[warp][0] = g;
    wsum[warp][1] = e;
  }
  __syncthreads();
  int gb = 0, eb = 0, gall = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    if (w < warp) {
      gb += wsum[w][0];
      eb += wsum[w][1];
    }
    gall += wsum[w][0];
  }
  const int want = take - gall;   // how many of the equal ones
  int gi = gb + g - gt, ei = eb + e - eq;
  for (int i = i0; i < i1; ++i) {
    const uint32_t kk = key[i];
    if (kk > v) {
      out[gi + min(ei, want)] = i;
      ++gi;
    } else if (kk == v) {
      if (ei < want) out[gi + ei] = i;
      ++ei;
    }
  }
}

}  // namespace

cudaError_t launch_block_keys(const mla_config &cfg, const void *cache, long long cache_len, const int *block_table,
                              int max_blocks, const int *ctx_begin, const int *ctx_len, int B, int max_new, void *keys,
                              int key_blocks, unsigned *status, cudaStream_t s) {
  if (B > 65535) return cudaErrorNotSupported;
  AttnArgs a = {};
  a.cache = cache;
  a.cache_len = cache_len;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.page_size = cfg.page_size;
  a.status = status;
  const int D = cfg.d_c + cfg.d_r;
  const uintptr_t mix = (uintptr_t)cache | (uintptr_t)keys | (uintptr_t)(D * (cfg.dtype == MLA_FP32 ? 4 : 2));
  const bool wide = mix % 16 == 0;
  if (cfg.dtype == MLA_FP32)
    return wide ? launch_keys<float, 4>(a, ctx_begin, ctx_len, B, max_new, keys, key_blocks, D, s)
                : launch_keys<float, 1>(a, ctx_begin, ctx_len, B, max_new, keys, key_blocks, D, s);
  return wide ? launch_keys<__nv_bfloat16, 8>(a, ctx_begin, ctx_len, B, max_new, keys, key_blocks, D, s)
              : launch_keys<__nv_bfloat16, 1>(a, ctx_begin, ctx_len, B, max_new, keys, key_blocks, D, s);
}

ScoreLayout score_layout(const mla_config &cfg, int B, int key_blocks) {
  ScoreLayout L;
  L.head_rows = (cfg.n_h + 127) / 128 * 128;
  L.tiles = (key_blocks + kScoreTile - 1) / kScoreTile;
  L.logit_off = 0;
  size_t off = align_up(sizeof(float) * (size_t)B * L.tiles * kScoreTile * L.head_rows, 256);
  L.stat_off = off;
  off = align_up(off + sizeof(float2) * (size_t)B * L.tiles * L.head_rows, 256);
  L.total = off > 256 ? off : 256;
  return L;
}

cudaError_t launch_block_scores(const mla_config &cfg, bool tc, float scale_log2, const void *q_abs, const void *keys,
                                int key_blocks, const int *ctx_len, int B, float *scores, char *ws,
                                const ScoreLayout &L, unsigned *status, cudaStream_t s) {
  if (B > 65535 || cfg.n_h > 8 * 65535 || L.tiles == 0) return cudaErrorNotSupported;
  float *logits = reinterpret_cast<float *>(ws + L.logit_off);
  float2 *stats = reinterpret_cast<float2 *>(ws + L.stat_off);
  const int D = cfg.d_c + cfg.d_r;
  cudaError_t e;
  if (tc) {
    if (D != 576 || cfg.dtype != MLA_BF16 || ((uintptr_t)q_abs | (uintptr_t)keys) % 16 != 0) return cudaErrorNotSupported;
    CUtensorMap mq, mk;
    const uint64_t dq[3] = {576, (uint64_t)cfg.n_h, (uint64_t)B}, dk[3] = {576, (uint64_t)key_blocks, (uint64_t)B};
    const uint64_t sq[2] = {1152, 1152ull * cfg.n_h}, sk[2] = {1152, 1152ull * key_blocks};
    const uint32_t box[3] = {64, 128, 1};
    if (!encode_map_bf16(&mq, q_abs, 3, dq, sq, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map_bf16(&mk, keys, 3, dk, sk, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorNotSupported;
    static std::atomic<int> configured[kMaxDevices];
    e = once_per_device(configured, [] {
      return cudaFuncSetAttribute(score_logits_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSSmem);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(score_logits_tc_kernel, dim3(L.tiles, L.head_rows / 128, B), dim3(kSThreads), kSSmem, s, 1, mq, mk,
                   key_blocks, ctx_len, cfg.n_h, scale_log2, logits, stats, L, status);
  } else {
    const dim3 grid(L.tiles, (cfg.n_h + 7) / 8, B);
    e = cfg.dtype == MLA_FP32
            ? launch_pdl(score_logits_simt_kernel<float>, grid, dim3(256), 0, s, 1, (const float *)q_abs,
                         (const float *)keys, key_blocks, ctx_len, cfg.n_h, D, scale_log2, logits, stats, L)
            : launch_pdl(score_logits_simt_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1,
                         (const __nv_bfloat16 *)q_abs, (const __nv_bfloat16 *)keys, key_blocks, ctx_len, cfg.n_h, D,
                         scale_log2, logits, stats, L);
  }
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(float) * cfg.n_h;
  if (smem > 48 * 1024) return cudaErrorNotSupported;
  return launch_pdl(score_sum_kernel, dim3((key_blocks + kSumBlocks - 1) / kSumBlocks, B), dim3(256), smem, s, 1,
                    (const float *)logits, (const float2 *)stats, L, key_blocks, ctx_len, cfg.n_h, scores, status);
}

cudaError_t launch_block_select(const float *scores, int n_blocks, const int *ctx_len, int B, int k, int n_first,
                                int n_last, int *sel, int *n_sel, unsigned *status, cudaStream_t s) {
  if (n_blocks > kSelMaxBlocks) return cudaErrorNotSupported;
  static std::atomic<int> configured[kMaxDevices];
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(block_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxBlocks * 4);
  });
  if (e != cudaSuccess) return e;
  // about four blocks to a thread: fewer warps to meet at each round's barrier
  const int threads = std::min(1024, std::max(32, (n_blocks + 127) / 128 * 32));
  return launch_pdl(block_select_kernel, dim3(B), dim3(threads), sizeof(uint32_t) * (size_t)n_blocks, s, 1, scores,
                    n_blocks, ctx_len, k, n_first, n_last, sel, n_sel, status);
}

}  // namespace mla
