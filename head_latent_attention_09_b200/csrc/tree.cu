// Tree of drafted tokens (speculative decoding): the merge of tree attention's
// split groups, and the cache's side of accepting a path.
#include <math_constants.h>

#include "internal.cuh"

namespace mla {
namespace {

template <typename T> __device__ __forceinline__ T cast(float x);
template <> __device__ __forceinline__ float cast<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 cast<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <int V>
struct alignas(4 * V) Vec {
  float e[V];
};
template <typename T, int V>
struct alignas(sizeof(T) * V) Out {
  T e[V];
};

// Log-sum-exp merge of the groups that are split between shares.  A share
// boundary cuts at most one plan sequence (gang groups).  Block x takes one
// member of a run: by_seq, member x % gang of plan sequence x / gang; otherwise
// (more sequences than shares) of the one that begins in share x / gang and runs
// on into the next, if there is one.  A warp takes a row, all its columns or,
// where there are few rows, a quarter of them (kSplit).  Groups that lie in one
// share were written by the attention kernel, so the traffic is that of at most
// 2 P gang pieces however many groups there are, and it mostly comes from L2:
// bound by latency, a chain of three reads (the plan, the sequence's shares, the
// partials).  A row's first partials are requested beside their log-sum-exps,
// kAhead at a time.  3 us behind the attention kernel for one sequence (16 pieces
// of 128 rows), 8 us for 34 MB of partials.
template <typename T, int V, bool kSplit>   // V columns to a lane and step: 4, or 1 where widths or pointers forbid it
__global__ void __launch_bounds__(256) tree_combine_kernel(AttnArgs a, int by_seq) {
  constexpr int kSteps = 16 / V / (kSplit ? 4 : 1);   // d_c <= 512
  constexpr int kAhead = kSteps >= 8 ? 1 : 8 / kSteps;
  pdl_trigger();
  pdl_wait();
  const int x = blockIdx.x / a.tree.gang, member = blockIdx.x % a.tree.gang;
  const WsHeader *hd = reinterpret_cast<const WsHeader *>(a.ws);
  const int *share_first = reinterpret_cast<const int *>(a.ws + a.L.share_first_off);
  const long long P = hd->P, Ttot = hd->Ttot;
  // by share: the plan sequence that holds the first tile of the next share
  const int v = by_seq ? x : (x + 1 < (int)(gridDim.x / a.tree.gang) ? share_first[x + 1] : 0);
  const long long *tp = reinterpret_cast<const long long *>(a.ws + a.L.tile_prefix_off);
  const float *lse = reinterpret_cast<const float *>(a.ws + a.L.lse_off);
  const float *op = reinterpret_cast<const float *>(a.ws + a.L.opart_off);
  T *out = reinterpret_cast<T *>(a.tree.out);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (Ttot == 0) {   // a cache without room for a single token: no row attends anything
    const long long rows = (long long)(a.B / a.tree.runs) * a.tree.seq_rows;
    const long long n = (long long)gridDim.x * gridDim.y * 8;
    for (long long r = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * 8 + warp; r < rows; r += n) {
      for (int f = lane; f < a.d_c; f += 32) out[r * a.d_c + f] = cast<T>(0.f);
      if (a.tree.lse && lane == 0) a.tree.lse[r] = -CUDART_INF_F;
    }
    return;
  }
  if (!by_seq && x + 1 >= P) return;
  const long long s0 = tp[v], s1 = tp[v + 1];
  if (s1 <= s0) return;
  const long long w0 = plan_share_of_tile(s0, P, Ttot), w1 = plan_share_of_tile(s1 - 1, P, Ttot);
  if (w0 == w1 || (!by_seq && w0 != x)) return;   // in one share, or begins in another
  const int b = v / a.tree.runs, g = (v - b * a.tree.runs) * a.tree.gang + member;
  const int n = (int)(w1 - w0) + 1;
  // partials: the last piece of share w0 (or its only one), the first of the others
  const long long part0 = 2 * (w0 * a.tree.gang + member) + (s0 > plan_begin(w0, P, Ttot) ? 1 : 0);
  auto slot = [&](int i) { return i == 0 ? part0 : 2 * ((w0 + i) * a.tree.gang + member); };
  const int f0 = (kSplit ? (warp & 3) * (32 * V * kSteps) : 0) + lane * V;
  const int r = blockIdx.y * (kSplit ? 2 : 8) + (kSplit ? warp >> 2 : warp);
  const int row = g * a.tree.group_rows + r;    // past the sequence's rows where there is no group g
  if (r >= a.tree.group_rows || row >= a.tree.seq_rows) return;
  const long long first = part_row(a.L, 0, r);
  Vec<V> p[kAhead][kSteps];
  auto request = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= n) break;
      const float *src = op + (first + slot(i0 + j)) * a.d_c + f0;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (f0 + 32 * V * i < a.d_c) p[j][i] = *reinterpret_cast<const Vec<V> *>(src + 32 * V * i);
    }
  };
  request(0);
  // each lane holds the log-sum-exp of one piece of 32
  float z = lane < n ? lse[first + slot(lane)] : -CUDART_INF_F;
  const float z0 = z;
  float m = z;
  for (int i = 32 + lane; i < n; i += 32) m = fmaxf(m, lse[first + slot(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // A row that attends nothing has -inf everywhere (weights of 0 and no sum);
  // a NaN keeps its way into the sum.
  const float m_use = m == -CUDART_INF_F ? 0.f : m;
  float tot = expf(z0 - m_use);
  for (int i = 32 + lane; i < n; i += 32) tot += expf(lse[first + slot(i)] - m_use);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  Vec<V> acc[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i].e[e] = 0.f;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    if (i0 > 0) {
      if ((i0 & 31) == 0) z = i0 + lane < n ? lse[first + slot(i0 + lane)] : -CUDART_INF_F;
      request(i0);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= n) break;
      const float wt = expf(__shfl_sync(0xffffffffu, z, (i0 + j) & 31) - m_use) * inv;
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[i].e[e] += wt * p[j][i].e[e];
    }
  }
  const long long orow = (long long)b * a.tree.seq_rows + row;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (f0 + 32 * V * i >= a.d_c) continue;
    Out<T, V> o;
#pragma unroll
    for (int e = 0; e < V; ++e) o.e[e] = cast<T>(acc[i].e[e]);
    *reinterpret_cast<Out<T, V> *>(out + orow * a.d_c + f0 + 32 * V * i) = o;
  }
  if (a.tree.lse && lane == 0 && f0 < V) a.tree.lse[orow] = tot == 0.f ? -CUDART_INF_F : m_use + logf(tot);
}

// Accepted path: row cached + path[i] -> cached + i, one block per sequence.
// A path rises, so path[i] >= i and no store covers a row that is still to be
// read when each column of the rows goes in path order: a thread carries
// columns (units of up to 16 bytes), and issues the loads of kAhead rows
// before their stores (a store to slot i lies below every source after i).
// The traffic is at most 2 x 64 rows, so the time is that of the launch and
// of two dependent reads (64 sequences, paths of up to 16: 2.4 us).
constexpr int kAhead = 8;
template <typename U>
__global__ void __launch_bounds__(1024) tree_accept_kernel(U *cache, int units, AttnArgs a, const int *ctx_len,
                                                           const int *path, const int *n_path, int T, int *new_len) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x;
  const long long cached = ctx_len[b];
  const long long cap = a.page_size ? (long long)a.max_blocks * a.page_size : a.cache_len;
  int n = n_path[b];
  // (a length past 2^31 - 1 could not be stored, however many tokens a table addresses)
  bool bad = n < 0 || n > T || cached < 0 || cached > cap || cached + n > 0x7fffffffLL;
  if (bad) n = 0;
  __shared__ long long src[kTreeMaxDrafted], dst[kTreeMaxDrafted];
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int p = path[(long long)b * T + i], q = i > 0 ? path[(long long)b * T + i - 1] : -1;
    src[i] = p > q && p < T ? token_row(a, b, cached + p) : -1;
    dst[i] = token_row(a, b, cached + i);
    if (src[i] < 0 || dst[i] < 0) bad = true;
  }
  // With one wrong entry the whole sequence stays as it is.
  bad = __syncthreads_or(bad);
  if (bad) n = 0;
  if (threadIdx.x == 0) {
    if (bad) atomicOr(a.status, kStatusBounds);
    if (new_len) new_len[b] = (int)cached + n;   // may be ctx_len itself: every thread has read it
  }
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      U v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k < n) v[k] = cache[src[i0 + k] * units + u];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k < n && src[i0 + k] != dst[i0 + k]) cache[dst[i0 + k] * units + u] = v[k];
    }
  }
}

template <typename U>
cudaError_t accept_units(int row_bytes, void *cache, const AttnArgs &a, const int *ctx_len, const int *path,
                         const int *n_path, int B, int T, int *new_len, cudaStream_t s) {
  const int units = row_bytes / (int)sizeof(U);
  const int threads = units >= 1024 ? 1024 : (units + 31) / 32 * 32;   // bf16 rows of 576: 72 units of 16 bytes
  return launch_pdl(tree_accept_kernel<U>, dim3(B), dim3(threads), 0, s, 1, (U *)cache, units, a, ctx_len, path,
                    n_path, T, new_len);
}

}  // namespace

cudaError_t launch_tree_combine(const AttnArgs &a, int P, bool fp32, cudaStream_t s) {
  if (a.d_c > 512) return cudaErrorNotSupported;
  const bool wide = a.d_c % 4 == 0 && (uintptr_t)a.tree.out % 16 == 0;
  // at most min(P - 1, plan sequences) runs are split
  const int by_seq = a.B <= 2 * P;
  const long long rows = (long long)std::min(a.B, P) * a.tree.gang * a.tree.group_rows;
  const bool split = wide && rows <= 1024;   // up to 1024 rows: four warps each
  const int block_rows = split ? 2 : 8;
  const dim3 grid((by_seq ? a.B : P) * a.tree.gang, (a.tree.group_rows + block_rows - 1) / block_rows);
  if (grid.y > 65535) return cudaErrorNotSupported;
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(256), 0, s, 1, a, by_seq); };
  if (fp32)
    return split ? go(tree_combine_kernel<float, 4, true>)
                 : (wide ? go(tree_combine_kernel<float, 4, false>) : go(tree_combine_kernel<float, 1, false>));
  return split ? go(tree_combine_kernel<__nv_bfloat16, 4, true>)
               : (wide ? go(tree_combine_kernel<__nv_bfloat16, 4, false>)
                       : go(tree_combine_kernel<__nv_bfloat16, 1, false>));
}

cudaError_t launch_tree_accept(const mla_config &cfg, void *cache, long long cache_len, const int *block_table,
                               int max_blocks, const int *ctx_len, const int *path, const int *n_path, int B, int T,
                               int *new_len, unsigned *status, cudaStream_t s) {
  AttnArgs a = {};
  a.cache_len = cache_len;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.page_size = cfg.page_size;
  a.status = status;
  const int row_bytes = (cfg.d_c + cfg.d_r) * (cfg.dtype == MLA_FP32 ? 4 : 2);
  const uintptr_t mix = (uintptr_t)cache | (uintptr_t)row_bytes;
  auto go = [&](auto unit) {
    return accept_units<decltype(unit)>(row_bytes, cache, a, ctx_len, path, n_path, B, T, new_len, s);
  };
  if (mix % 16 == 0) return go(uint4{});
  if (mix % 4 == 0) return go(uint32_t{});
  return go(uint16_t{});
}

}  // namespace mla
