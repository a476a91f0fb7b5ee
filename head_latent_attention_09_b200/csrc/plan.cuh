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
__device__ __forceinline__ void plan_entry(const PlanSource &src, int b, long long cap, unsigned *status, int *end_out,
                                           int *second_out) {
  const int seq = src.runs > 1 ? b / src.runs : b;
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
  } else if (src.drafted > 0) {
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
  int first;   // first plan sequence of this CTA's share
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

// Makes the plan for P_req shares in `o` (every thread of the CTA, which works
// on share `share`); block 0 stores it in the workspace.
__device__ __forceinline__ void plan_in_line(const AttnArgs &a, int share, int P_req, PlanSmem &o) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  const bool from0 = plan_from0(a.src);
  for (int b = tid; b < a.B; b += nt) {
    int end, second;
    plan_entry(a.src, b, a.cap, a.status, &end, &second);
    o.ends[b] = end;
    o.seconds[b] = second;
    o.pb[b] = ((unsigned)(end - (from0 ? 0 : second)) + (unsigned)a.plan_tile - 1u) / (unsigned)a.plan_tile;   // tiles
  }
  __syncthreads();
  if (tid < 32) {
    const int per = (a.B + 31) / 32, b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
    auto before = [&](long long x, long long *total) {   // exclusive prefix over the lanes
      long long s = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
      }
      *total = __shfl_sync(0xffffffffu, s, 31);
      return s - x;
    };
    long long sum = 0, Ttot, pieces;
    for (int b = b0; b < b1; ++b) sum += o.pb[b];
    long long run = before(sum, &Ttot);
    for (int b = b0; b < b1; ++b) {
      o.tp[b] = run;
      run += o.pb[b];
    }
    const long long P = Ttot < (long long)P_req ? Ttot : (long long)P_req;
    long long np = 0;
    for (int b = b0; b < b1; ++b) {
      const long long t = o.pb[b];
      const long long n =
          t > 0 ? plan_share_of_tile(o.tp[b] + t - 1, P, Ttot) - plan_share_of_tile(o.tp[b], P, Ttot) + 1 : 0;
      o.pb[b] = n;
      np += n;
    }
    long long prun = before(np, &pieces);
    for (int b = b0; b < b1; ++b) {
      const long long n = o.pb[b];
      o.pb[b] = prun;
      prun += n;
    }
    if (lane == 0) {
      o.tp[a.B] = Ttot;
      o.pb[a.B] = pieces;
      o.P = P;
      o.Ttot = Ttot;
    }
    __syncwarp();
    if (lane == 0 && share < P) o.first = plan_first(o.tp, a.B, share, P, Ttot);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    long long *tp = reinterpret_cast<long long *>(a.ws + a.L.tile_prefix_off);
    long long *pb = reinterpret_cast<long long *>(a.ws + a.L.piece_base_off);
    int *ends = reinterpret_cast<int *>(a.ws + a.L.ctx_off), *first = reinterpret_cast<int *>(a.ws + a.L.share_first_off);
    for (int b = tid; b <= a.B; b += nt) {
      tp[b] = o.tp[b];
      pb[b] = o.pb[b];
      if (b < a.B) {
        ends[b] = o.ends[b];
        ends[a.B + b] = o.seconds[b];
      }
    }
    for (int w = tid; w < o.P; w += nt) first[w] = plan_first(o.tp, a.B, w, o.P, o.Ttot);
    if (tid == 0) {
      WsHeader *hd = reinterpret_cast<WsHeader *>(a.ws);
      hd->B = a.B;
      hd->P = o.P;
      hd->Ttot = o.Ttot;
      hd->n_pieces = o.pb[a.B];
    }
  }
}

}  // namespace mla
