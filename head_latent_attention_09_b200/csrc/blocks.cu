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
// by HBM for a whole prompt (four of 131072 tokens: 91 us, 6.66 TB/s of rows),
// by the launch and three dependent reads for a decode step (one block of each
// of 64 sequences: 6.3 us).
// ---------------------------------------------------------------------------
constexpr int kKeyThreads = 288;     // bf16 rows of 576: 72 units x 4 row groups
constexpr int kKeyBatch = 8;         // rows a thread has in flight (x 3 resident blocks: 110 KB an SM)

template <typename T, int V>
struct alignas(sizeof(T) * V) Unit {
  T e[V];
};

template <typename T, int V, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kKeyThreads ? 3 : 1) block_keys_kernel(AttnArgs a, const int *ctx_begin, const int *ctx_len,
                                                                 T *keys, int key_blocks, int D) {
  constexpr bool kSpread = kThreads > kKeyThreads;
  __shared__ float part[kThreads * V];
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
  const int upb = min(units, kThreads);           // units at a time
  const int G = kThreads / upb;                   // row groups
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
          for (int r0 = g; r0 < n; r0 += G * kKeyBatch) {
            Unit<T, V> x[kKeyBatch];
#pragma unroll
            for (int k = 0; k < kKeyBatch; ++k) {
              const int r = r0 + G * k;
              const long long row = r >= n ? -1 : (run ? first + r : token_row(a, b, j * kTile + r));
              if (row >= 0) {
                x[k] = cache[row * units + u];
              } else {
                if (r < n) atomicOr(a.status, kStatusBounds);
#pragma unroll
                for (int e = 0; e < V; ++e) x[k].e[e] = narrow<T>(0.f);
              }
            }
#pragma unroll
            for (int k = 0; k < kKeyBatch; ++k)
#pragma unroll
              for (int e = 0; e < V; ++e) acc[e] += widen<T>(x[k].e[e]);
          }
        }
        if (kSpread || g > 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) part[(g * upb + ul) * V + e] = acc[e];
        }
      }
      __syncthreads();
      if (kSpread) {   // many groups: a thread to a column
        for (int c = threadIdx.x; c < min(upb, units - u0) * V; c += kThreads) {
          float sum = part[c];
          for (int gg = 1; gg < G; ++gg) sum += part[gg * upb * V + c];
          keys[(((long long)b * key_blocks + j) * units + u0) * V + c] = narrow<T>(sum / (float)n);
        }
      } else if (g == 0 && u < units) {
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
  // Where the blocks leave SMs idle (a decode step), more row groups take each
  // in one batch of loads instead of two (64 sequences: 6.8 -> 6.3 us).
  if ((long long)grid.x * B <= 148)
    return launch_pdl(block_keys_kernel<T, V, 1024>, grid, dim3(1024), 0, s, 1, a, ctx_begin, ctx_len, (T *)keys,
                      key_blocks, D);
  return launch_pdl(block_keys_kernel<T, V, kKeyThreads>, grid, dim3(kKeyThreads), 0, s, 1, a, ctx_begin, ctx_len,
                    (T *)keys, key_blocks, D);
}

// ---------------------------------------------------------------------------
// scores: x (in log2 units) of a tile of 128 blocks against the heads, per head
// the tile's maximum and sum of 2^(x - maximum), and from these the shares.
// ---------------------------------------------------------------------------
constexpr int kScoreTile = 128;

// Blocks of a sequence of ctx tokens, any int: ctx + kTile - 1 would overflow near
// 2^31 and come out negative.
__device__ __forceinline__ int blocks_of(int ctx) { return ctx <= 0 ? 0 : (ctx - 1) / kTile + 1; }
// log2 of the tokens in block j of a sequence of ctx tokens
__device__ __forceinline__ float log2_tokens(int j, int ctx) {
  const int n = ctx - j * kTile;
  return n >= kTile ? 6.f : log2f((float)n);
}

// Maxima are subtracted through this: scores of -inf alone (overflows) then add
// nothing (-inf - -inf is NaN), while a NaN, which no maximum shows, still
// reaches the sum and with it every share of the head.
__device__ __forceinline__ float minus_inf_to_0(float m) { return m == -CUDART_INF_F ? 0.f : m; }
// The log-sum-exp that a head's shares are taken through; finite also for a head
// with nothing but scores of -inf, whose shares then are 2^(-inf - 0) = 0.
__device__ __forceinline__ float share_lse(float m, float sum) { return sum == 0.f ? 0.f : m + log2f(sum); }

// CUDA cores, two launches: first x and the statistics, one warp per head, the
// query row in registers (also bf16 beyond the tensor-core kernel's 4096 blocks).
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
    const float m2 = fmaxf(m, x), m_use = minus_inf_to_0(m2);
    sum = sum * exp2f(m - m_use) + exp2f(x - m_use);
    m = m2;
    if (lane == 0) logits[((long long)b * L.tiles * kScoreTile + j) * L.head_rows + h] = x;
  }
  if (lane == 0) stats[((long long)b * L.tiles + tile) * L.head_rows + h] = make_float2(m, sum);
}

// Tensor cores (rows of 576 bf16), both halves in one launch: a cluster of up
// to eight CTAs per sequence, each with up to four tiles of 128 blocks.
//   S = Q K^T  M = 128 heads (zero filled), N = 128 blocks a tile; nine
//              64-column chunks of Q and of the tiles' rows stream through a
//              ring of stages.
// A thread owns one head's row of the accumulator, so its maximum and sum need
// no exchange within the CTA; the cluster's CTAs exchange them through
// distributed shared memory, and the shares are then added over the heads by a
// transposing reduction (31 shuffles for 32 columns).  The logits never leave
// tensor memory.  The rows are 1/64 of the cache's bytes: the time is one chain
// of load, multiply and two passes over tensor memory (64 sequences of 128
// blocks at 128 heads: 9.8 us, 18.9 MB of means; four of 2048 blocks at 16 heads:
// 15.3 us, eight CTAs a sequence with two tiles each).
constexpr int kSThreads = 192;
constexpr int kSMaxTiles = 4, kSMaxCluster = 8;
constexpr int kSRing = 6 * 32768;      // bytes of stages: 6, 4, 3 or 2 of (1 + tiles) 16 KB chunks
constexpr int kSSmem = kSRing + 1024;

__global__ void __launch_bounds__(kSThreads, 1)
    score_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK, int key_blocks,
                    const int *ctx_len, int n_h, float scale_log2, float *scores, int tiles_per_cta, int stages,
                    uint32_t tmem_cols, unsigned *status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[6], empty[6], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ float2 stat[2][128];                         // per head: maximum and sum over this CTA's blocks
  __shared__ float part[4][kSMaxTiles * kScoreTile];      // per epilogue warp: shares summed over its 32 heads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, b = blockIdx.y;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 6; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(&done, 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_slot, tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  const int ctx = ctx_len[b], all = blocks_of(ctx), nb = min(all, key_blocks);
  if ((all > key_blocks || ctx < 0) && rank == 0 && threadIdx.x == 0) atomicOr(status, kStatusBounds);
  const int j0 = rank * tiles_per_cta * kScoreTile;       // first block of this CTA
  const int own = min(max((nb - j0 + kScoreTile - 1) / kScoreTile, 0), tiles_per_cta);   // its tiles that hold blocks
  const int stage = (1 + tiles_per_cta) * 16384;
  const int head_tiles = (n_h + 127) / 128;
  const int q = warp & 3;
  const bool epi = warp >= 2;
  float acc[kSMaxTiles] = {0.f, 0.f, 0.f, 0.f};           // thread t of the epilogue: block t of each tile
  // Columns [32 g, 32 g + 32) of this thread's row over the CTA's tiles, in log2
  // units.  (32 at a time: the passes run a few times each, so their code is
  // fetched about as often as it runs, and its length counts.)
  auto row32 = [&](int g, float (&v)[32]) {
    ptx::tmem_ld32_sync(tmem + ((uint32_t)(q * 32) << 16) + 32 * g, reinterpret_cast<uint32_t *>(v));
    const int jb = j0 + 32 * g;
    const float last = log2_tokens(nb - 1, ctx);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = jb + j < nb ? fmaf(v[j], scale_log2, jb + j == nb - 1 ? last : 6.f) : -CUDART_INF_F;
  };
  const int groups = min((nb - j0 + 31) / 32, own * 4);   // 32-column groups that hold blocks
  for (int ht = 0; ht < head_tiles; ++ht) {
    if (warp == 0) {
      if (own > 0 && ptx::elect_one()) {
        for (int c = 0; c < 9; ++c) {
          const int it = ht * 9 + c, s = it % stages;
          if (it >= stages && !ptx::mbar_wait(&empty[s], (it / stages - 1) & 1, status, &abort_flag)) break;
          uint8_t *at = sm + s * stage;
          ptx::mbar_arrive_expect_tx(&full[s], (1 + own) * 16384);
          ptx::tma_load_3d(at, &mapQ, &full[s], 64 * c, ht * 128, b);
          for (int t = 0; t < own; ++t)
            ptx::tma_load_3d(at + (1 + t) * 16384, &mapK, &full[s], 64 * c, j0 + t * kScoreTile, b);
        }
      }
    } else if (warp == 1) {
      if (own > 0 && ptx::elect_one()) {
        constexpr uint32_t id = idesc_bf16(128, kScoreTile, false, false);
        bool ok = true;
        for (int c = 0; c < 9 && ok; ++c) {
          const int it = ht * 9 + c, s = it % stages;
          ok = ptx::mbar_wait(&full[s], (it / stages) & 1, status, &abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t at = ptx::smem_u32(sm + s * stage);
          for (int t = 0; t < own; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_bf16_ss(tmem + t * kScoreTile, ptx::sdesc(at + 32 * k, 16, 1024, 2),
                               ptx::sdesc(at + (1 + t) * 16384 + 32 * k, 16, 1024, 2), id, (c | k) != 0 ? 1u : 0u);
          ptx::mma_commit(&empty[s]);
        }
        if (ok) ptx::mma_commit(&done);
      }
    } else {
      const int h = ht * 128 + 32 * q + lane;
      float m = -CUDART_INF_F, sum = 0.f;
      bool ok = own > 0;
      if (ok && lane == 0) ok = ptx::mbar_wait(&done, ht & 1, status, &abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (ok && lane != 0) ptx::mbar_test_wait(&done, ht & 1);
      __syncwarp();
      if (ok && ht * 128 + 32 * q < n_h) {
        ptx::tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
          float v[32];
          row32(g, v);
          float mx[4] = {m, m, m, m};
#pragma unroll
          for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
          const float m2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const float m_use = minus_inf_to_0(m2);
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) s4[j & 3] += ptx::exp2_approx(v[j] - m_use);
          sum = sum * exp2f(m - m_use) + ((s4[0] + s4[1]) + (s4[2] + s4[3]));
          m = m2;
        }
      }
      stat[ht & 1][32 * q + lane] = h < n_h ? make_float2(m, sum) : make_float2(-CUDART_INF_F, 0.f);
    }
    __syncwarp();
    ptx::cluster_sync_all();
    if (epi) {
      if (own > 0 && ht * 128 + 32 * q < n_h) {
        // the head's log-sum-exp over the sequence's blocks
        const int h = 32 * q + lane;
        const uint32_t mine = ptx::smem_u32(&stat[ht & 1][h]);
        float m = -CUDART_INF_F, sum = 0.f;
        const int nc = (int)ptx::cluster_nctarank();
        for (int p = 0; p < nc; ++p) {
          const float2 s = ptx::ld_shared_cluster_v2f(ptx::mapa_peer(mine, (uint32_t)p));
          const float m2 = fmaxf(m, s.x), m_use = minus_inf_to_0(m2);
          sum = sum * exp2f(m - m_use) + s.y * exp2f(s.x - m_use);
          m = m2;
        }
        const bool real = ht * 128 + h < n_h;
        const float lse = real ? share_lse(m, sum) : 0.f;
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
          float v[32];
          row32(g, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = real ? ptx::exp2_approx(v[j] - lse) : 0.f;
          // Sums over the 32 lanes: halving the columns a lane is in charge of
          // with every exchange leaves lane l column l.
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int j = 0; j < o; ++j) {
              const float give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
              v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          }
          part[q][32 * g + lane] = v[0];
        }
      }
      ptx::named_bar_sync(1, 128);
      const int warps = min(4, (n_h - ht * 128 + 31) / 32);    // epilogue warps that hold heads
      for (int t = 0; t < own; ++t)
        for (int w = 0; w < warps; ++w) acc[t] += part[w][t * kScoreTile + 32 * q + lane];
    }
    ptx::tc_fence_before();
    __syncthreads();   // the next heads' MMAs overwrite the accumulator, their sums `part`
    ptx::tc_fence_after();
  }
  if (epi)
    for (int t = 0; t < tiles_per_cta; ++t) {
      const int j = j0 + t * kScoreTile + 32 * q + lane;
      if (j < key_blocks) scores[(long long)b * key_blocks + j] = j < nb ? acc[t] : 0.f;
    }
  __syncwarp();
  if (warp == 1) ptx::tmem_dealloc(tmem, tmem_cols);
  ptx::cluster_sync_all();   // no CTA leaves while others still read its statistics
}

// Second launch: score_j = sum over heads of 2^(x - lse of the head), one warp
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
        sum += v.y * exp2f(v.x - minus_inf_to_0(m));
      }
      lse[h] = share_lse(m, sum);
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
// threads per sequence; the scores become unsigned integers of the same order,
// thread t holding a run of consecutive ones (in registers up to 4096 blocks,
// in shared memory beyond).  The k-th largest is found two bits a round: three
// counts per thread, summed within the warps by redux and across them through
// one shared-memory line, so a round is one barrier and no atomics (softmax
// masses share their leading bits: bins would collide).  The rounds end once
// a bound leaves exactly k.  One scan over the threads then places the
// winners.  The order is total (value, then the lower index), so the result
// is the same however the threads run.  The work is a few KB a sequence: the
// time is the launch, two dependent reads and the rounds' barriers (64 of 2047
// blocks: 4.5 us; 128 sequences of up to 512 blocks: 5.9 us).
// ---------------------------------------------------------------------------
constexpr int kSelMaxBlocks = 49152;   // 192 KB of keys
constexpr int kSelRegs = 4;            // keys a thread holds in registers

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;                     // NaN ranks below everything
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 counts as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <bool kReg>
__global__ void __launch_bounds__(1024) block_select_kernel(const float *scores, int n_blocks, const int *ctx_len,
                                                            int k, int n_first, int n_last, int *sel, int *n_sel,
                                                            unsigned *status) {
  extern __shared__ uint32_t skey[];
  __shared__ uint32_t cnt[2][32][2];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const float *x = scores + (long long)b * n_blocks;
  const int per = kReg ? kSelRegs : (n_blocks + nt - 1) / nt;
  const int i0 = tid * per;                                // this thread's run of blocks
  float xr[kSelRegs];
  if (kReg) {
#pragma unroll
    for (int e = 0; e < kSelRegs; ++e) xr[e] = i0 + e < n_blocks ? x[i0 + e] : 0.f;
  }
  const int all = blocks_of(ctx_len[b]);
  const int n = min(all, n_blocks);
  if (tid == 0 && (all > n_blocks || ctx_len[b] < 0)) atomicOr(status, kStatusBounds);
  int *out = sel + (long long)b * k;
  const int take = min(n, k);
  for (int i = take + tid; i < k; i += nt) out[i] = -1;
  if (tid == 0) n_sel[b] = take;
  if (take == n) {
    for (int i = tid; i < n; i += nt) out[i] = i;
    return;
  }
  auto key_of = [&](int i, float v) { return i < n_first || i >= n - n_last ? 0xffffffffu : order_key(v); };
  uint32_t key[kSelRegs];
  const int i1 = min(n, i0 + per);
  if (kReg) {
#pragma unroll
    for (int e = 0; e < kSelRegs; ++e) key[e] = key_of(i0 + e, xr[e]);
  } else {
    for (int i = tid; i < n; i += nt) skey[i] = key_of(i, x[i]);
    __syncthreads();
  }
  // f(key) for each block of this thread's run, in order
  auto each = [&](auto f) {
    if (kReg) {
#pragma unroll
      for (int e = 0; e < kSelRegs; ++e)
        if (i0 + e < n) f(i0 + e, key[e]);
    } else {
      for (int i = i0; i < i1; ++i) f(i, skey[i]);
    }
  };
  // Sum over the block of two counts below 2^16 in one word, and of another.
  auto total = [&](int buf, uint32_t a, uint32_t c, uint32_t &sa, uint32_t &sc) {
    a = __reduce_add_sync(0xffffffffu, a);
    c = __reduce_add_sync(0xffffffffu, c);
    if (nw > 1) {
      if (lane == 0) {
        cnt[buf][warp][0] = a;
        cnt[buf][warp][1] = c;
      }
      __syncthreads();
      a = __reduce_add_sync(0xffffffffu, lane < nw ? cnt[buf][lane][0] : 0u);
      c = __reduce_add_sync(0xffffffffu, lane < nw ? cnt[buf][lane][1] : 0u);
    }
    sa = a;
    sc = c;
  };
  uint32_t v = 0;   // largest value found so far with at least `take` keys >= it
#pragma unroll 1
  for (int r = 0; r < 16; ++r) {
    const uint32_t bit = 1u << (30 - 2 * r);
    uint32_t c12 = 0, c3 = 0, s12, s3;
    each([&](int, uint32_t kk) {
      c12 += (kk >= v + bit ? 1u : 0u) + (kk >= v + 2 * bit ? 0x10000u : 0u);
      c3 += kk >= v + 3 * bit ? 1u : 0u;
    });
    total(r & 1, c12, c3, s12, s3);
    const int t1 = s12 & 0xffffu, t2 = s12 >> 16, t3 = s3;
    const int step = t3 >= take ? 3 : (t2 >= take ? 2 : (t1 >= take ? 1 : 0));
    v += step * bit;
    if ((step == 3 ? t3 : (step == 2 ? t2 : t1)) == take && step > 0) break;   // exactly the winners are >= v
  }
  // Thread t places those of its run above v, and the first of those equal to
  // it as far as the k-th place reaches.
  int gt = 0, eq = 0;
  each([&](int, uint32_t kk) {
    gt += kk > v;
    eq += kk == v;
  });
  int ge = gt | eq << 16;   // inclusive prefix over the lanes (both below 2^16)
  uint32_t s = (uint32_t)ge;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  uint32_t before = 0, gall;
  if (nw > 1) {
    __syncthreads();   // the rounds' last counts have been read
    if (lane == 31) cnt[0][warp][0] = s;
    __syncthreads();
    const uint32_t c = lane < nw ? cnt[0][lane][0] : 0u;
    before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0u);
    gall = __reduce_add_sync(0xffffffffu, c) & 0xffffu;
  } else {
    gall = __shfl_sync(0xffffffffu, s, 31) & 0xffffu;
  }
  s += before - (uint32_t)ge;   // exclusive
  const int want = take - (int)gall;   // how many of the equal ones
  int gi = s & 0xffffu, ei = s >> 16;
  each([&](int i, uint32_t kk) {
    if (kk > v) {
      out[gi + min(ei, want)] = i;
      ++gi;
    } else if (kk == v) {
      if (ei < want) out[gi + ei] = i;
      ++ei;
    }
  });
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
  L.head_rows = (cfg.n_h + 31) / 32 * 32;
  L.tiles = (key_blocks + kScoreTile - 1) / kScoreTile;
  L.logit_off = 0;
  size_t off = align_up(sizeof(float) * (size_t)B * L.tiles * kScoreTile * L.head_rows, 256);
  L.stat_off = off;
  off = align_up(off + sizeof(float2) * (size_t)B * L.tiles * L.head_rows, 256);
  L.total = off > 256 ? off : 256;
  return L;
}

cudaError_t launch_block_scores_tc(const mla_config &cfg, float scale_log2, const void *q_abs, const void *keys,
                                   int key_blocks, const int *ctx_len, int B, float *scores, unsigned *status,
                                   cudaStream_t s) {
  const int tiles = (key_blocks + kScoreTile - 1) / kScoreTile;
  if (B > 65535 || cfg.d_c + cfg.d_r != 576 || cfg.dtype != MLA_BF16 || tiles > kSMaxTiles * kSMaxCluster ||
      ((uintptr_t)q_abs | (uintptr_t)keys) % 16 != 0)
    return cudaErrorNotSupported;
  CUtensorMap mq, mk;
  const uint64_t dq[3] = {576, (uint64_t)cfg.n_h, (uint64_t)B}, dk[3] = {576, (uint64_t)key_blocks, (uint64_t)B};
  const uint64_t sq[2] = {1152, 1152ull * cfg.n_h}, sk[2] = {1152, 1152ull * key_blocks};
  const uint32_t box[3] = {64, 128, 1};
  if (!encode_map_bf16(&mq, q_abs, 3, dq, sq, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_bf16(&mk, keys, 3, dk, sk, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  static std::atomic<int> configured[kMaxDevices];
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(score_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSSmem);
  });
  if (e != cudaSuccess) return e;
  const int cluster = tiles > 4 ? 8 : (tiles > 2 ? 4 : tiles);
  const int per = (tiles + cluster - 1) / cluster;
  const int stages = kSRing / ((1 + per) * 16384);
  const uint32_t cols = per == 1 ? 128 : (per == 2 ? 256 : 512);
  return launch_pdl(score_tc_kernel, dim3(cluster, B), dim3(kSThreads), kSSmem, s, cluster, mq, mk, key_blocks, ctx_len,
                    cfg.n_h, scale_log2, scores, per, stages, cols, status);
}

cudaError_t launch_block_scores_simt(const mla_config &cfg, float scale_log2, const void *q_abs, const void *keys,
                                     int key_blocks, const int *ctx_len, int B, float *scores, char *ws,
                                     const ScoreLayout &L, unsigned *status, cudaStream_t s) {
  const size_t smem = sizeof(float) * cfg.n_h;
  if (B > 65535 || smem > 48 * 1024 || L.tiles == 0) return cudaErrorNotSupported;
  float *logits = reinterpret_cast<float *>(ws + L.logit_off);
  float2 *stats = reinterpret_cast<float2 *>(ws + L.stat_off);
  const int D = cfg.d_c + cfg.d_r;
  const dim3 grid(L.tiles, (cfg.n_h + 7) / 8, B);
  const cudaError_t e =
      cfg.dtype == MLA_FP32
          ? launch_pdl(score_logits_simt_kernel<float>, grid, dim3(256), 0, s, 1, (const float *)q_abs,
                       (const float *)keys, key_blocks, ctx_len, cfg.n_h, D, scale_log2, logits, stats, L)
          : launch_pdl(score_logits_simt_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1, (const __nv_bfloat16 *)q_abs,
                       (const __nv_bfloat16 *)keys, key_blocks, ctx_len, cfg.n_h, D, scale_log2, logits, stats, L);
  if (e != cudaSuccess) return e;
  return launch_pdl(score_sum_kernel, dim3((key_blocks + kSumBlocks - 1) / kSumBlocks, B), dim3(256), smem, s, 1,
                    (const float *)logits, (const float2 *)stats, L, key_blocks, ctx_len, cfg.n_h, scores, status);
}

cudaError_t launch_block_select(const float *scores, int n_blocks, const int *ctx_len, int B, int k, int n_first,
                                int n_last, int *sel, int *n_sel, unsigned *status, cudaStream_t s) {
  if (n_blocks > kSelMaxBlocks) return cudaErrorNotSupported;
  if (n_blocks <= 1024 * kSelRegs) {
    const int threads = std::max(32, (n_blocks + 32 * kSelRegs - 1) / (32 * kSelRegs) * 32);
    return launch_pdl(block_select_kernel<true>, dim3(B), dim3(threads), 0, s, 1, scores, n_blocks, ctx_len, k, n_first,
                      n_last, sel, n_sel, status);
  }
  static std::atomic<int> configured[kMaxDevices];
  const cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(block_select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSelMaxBlocks * 4);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(block_select_kernel<false>, dim3(B), dim3(1024), sizeof(uint32_t) * (size_t)n_blocks, s, 1, scores,
                    n_blocks, ctx_len, k, n_first, n_last, sel, n_sel, status);
}

}  // namespace mla
