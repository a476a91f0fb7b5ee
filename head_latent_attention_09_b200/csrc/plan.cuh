// The split plan's arithmetic per sequence, and the plan as the tensor-core
// attention kernels make it for themselves: every CTA computes the whole plan
// of up to kInlineSeqs plan sequences in its own shared memory.  That takes a
// launch and its gap off every call, and the roles read the plan at shared
// memory's latency (a few dependent reads each); one CTA stores it in the
// workspace for the merge that follows.
#pragma once

#include "internal.cuh"

namespace mla {

__device__ __forceinline__ bool plan_from0(const PlanSource &src) { return src.drafted > 0 || src.sel; }

// End and second value of plan sequence b (see plan_ends).  A length outside
// [0, cap], a first token that is negative, past the end or not a multiple of
// kTile, drafted tokens past the cap, a count of selected blocks that the
// sequence does not have: each is flagged and clamped, and the tiles and every
// attention kernel use the clamped values.
template <bool kTree>   // kTree: `runs` and `drafted` may be set
__device__ __forceinline__ void plan_entry(const PlanSource &src, int b, long long cap, unsigned *status, int *end_out,
                                           int *second_out) {
  const int seq = kTree && src.runs > 1 ? b / src.runs : b;
  long long n = src.sel ? src.n_sel[seq] : 0;
  long long c = src.ctx_len[seq];
  bool bad = c < 0 || c > cap;
  if (bad) c = c < 0 ? 0 : cap;
  long long end = c, second = c;
  if (src.sel) {
    const long long most = min((long long)src.sel_k, ceil_div_ll(c, kTile));
    if (n < 0 || n > most) {
      bad = true;
      n = n < 0 ? 0 : most;
    }
    end = n * kTile;
    if (n > 0) {
      const long long last = src.sel[(long long)seq * src.sel_k + n - 1];
      if (last >= 0 && last * kTile < c) end -= max(0ll, (last + 1) * kTile - c);   // the partial block
    }
  } else if (kTree && src.drafted > 0) {
    end = c + src.drafted;
    if (end > cap) {
      bad = true;
      end = cap;
    }
  } else {
    long long g = src.ctx_begin ? src.ctx_begin[b] : 0;
    if (g < 0 || g > c || g % kTile != 0) {
      bad = true;
      g = g < 0 ? 0 : (g > c ? c : g);
      g -= g % kTile;
    }
    second = g;
  }
  if (bad) atomicOr(status, kStatusBounds);
  *end_out = (int)end;
  *second_out = (int)second;
}

struct PlanSmem {
  long long tp[kInlineSeqs + 1], pb[kInlineSeqs + 1];
  int ends[kInlineSeqs], seconds[kInlineSeqs];
  long long P, Ttot;
  unsigned t0, t1;   // tiles of this CTA's share
  int first;         // its first plan sequence
};

// First plan sequence whose tiles reach past the first tile of share w.
__device__ __forceinline__ int plan_first(const long long *tp, int B, long long w, long long P, long long Ttot) {
  const long long t0 = plan_begin(w, P, Ttot);
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid + 1] <= t0) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Exclusive prefix over a warp's lanes, and the total.
__device__ __forceinline__ unsigned lanes_before(unsigned x, unsigned *total) {
  unsigned s = x;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, s, d);
    if ((int)(threadIdx.x & 31) >= d) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  return s - x;
}

// Makes the plan for P_req shares in `o` (every thread of the CTA, which works
// on share `share`); block 0 stores it in the workspace.  The caller has made
// sure that tiles x shares fits 32 bits (plan_fits): this code runs once per CTA
// and its instructions are fetched as it runs, so it is kept short (in 64 bits
// and unrolled the scans took 10100 cycles, so 2700 for 64 sequences, 2300 for
// four; the two dependent reads of the lengths before them 1600 to 2700).
__device__ __forceinline__ void plan_in_line(const AttnArgs &a, int share, int P_req, PlanSmem &o) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
#pragma unroll 1
  for (int b = tid; b < a.B; b += nt) {
    int end, second;
    plan_entry<false>(a.src, b, a.cap, a.status, &end, &second);
    o.ends[b] = end;
    o.seconds[b] = second;
    o.pb[b] = ((unsigned)(end - (a.src.sel ? 0 : second)) + (unsigned)a.plan_tile - 1u) / (unsigned)a.plan_tile;   // tiles
  }
  __syncthreads();
  if (tid < 32) {
    const int per = (a.B + 31) / 32, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
    unsigned sum = 0, Ttot, pieces;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) sum += (unsigned)o.pb[b];
    unsigned run = lanes_before(sum, &Ttot);
    const unsigned P = min(Ttot, (unsigned)P_req);
    const unsigned mine = (unsigned)share < P ? (unsigned)share * Ttot / P : 0xffffffffu;   // this share's first tile
    sum = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const unsigned t = (unsigned)o.pb[b];
      o.tp[b] = run;
      const unsigned n = t > 0 ? ((run + t) * P - 1u) / Ttot - ((run + 1u) * P - 1u) / Ttot + 1u : 0u;
      if (mine - run < t) o.first = b;
      o.pb[b] = n;
      run += t;
      sum += n;
    }
    run = lanes_before(sum, &pieces);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const unsigned n = (unsigned)o.pb[b];
      o.pb[b] = run;
      run += n;
    }
    if (lane == 0) {
      o.tp[a.B] = Ttot;
      o.pb[a.B] = pieces;
      o.P = P;
      o.Ttot = Ttot;
      o.t0 = mine;
      o.t1 = (unsigned)share < P ? ((unsigned)share + 1u) * Ttot / P : 0u;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {   // for the merge (which needs no share_first)
    long long *tp = reinterpret_cast<long long *>(a.ws + a.L.tile_prefix_off);
    long long *pb = reinterpret_cast<long long *>(a.ws + a.L.piece_base_off);
    int *ends = reinterpret_cast<int *>(a.ws + a.L.ctx_off);
#pragma unroll 1
    for (int b = tid; b <= a.B; b += nt) {
      tp[b] = o.tp[b];
      pb[b] = o.pb[b];
      if (b < a.B) {
        ends[b] = o.ends[b];
        ends[a.B + b] = o.seconds[b];
      }
    }
    if (tid == 0) {
      WsHeader *hd = reinterpret_cast<WsHeader *>(a.ws);
      hd->B = a.B;
      hd->P = o.P;
      hd->Ttot = o.Ttot;
      hd->n_pieces = o.pb[a.B];
    }
  }
}

// Whether plan_in_line can make the plan: at most kInlineSeqs sequences, and
// tiles x shares in 32 bits whatever the lengths.
inline bool plan_fits(const PlanSource &src, int B, int P_req, long long cap, int tile) {
  const long long most = src.sel ? std::min(cap, (long long)src.sel_k * kTile) : cap;
  return B <= kInlineSeqs && (double)B * (double)ceil_div_ll(most, tile) * ((double)P_req + 1.0) < 4e9;
}

}  // namespace mla
