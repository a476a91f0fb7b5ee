// Split-KV decode attention over the latent cache for 128 heads (DeepSeek-V2
// shapes: d_c = 512, d_h^R = 64, bf16), on pairs of SMs.
//
// What it computes (absorbed MLA, "DeepSeek-V2", Appendix C; softmax of the
// "DeepSeek-V3" note's o_{t,i}): for every (sequence, share) piece,
//   s_j   = q_abs_i . [c_j ; k^R_j] / sqrt(d_h + d_h^R)
//   ctx_i = sum_j softmax_j(s) c_j      and   lse_i = log sum_j e^{s_j}
// over the piece's tokens, written as fp32 partials for the log-sum-exp merge.
//
// Why a pair: the output accumulator of 128 heads x 512 latent columns in fp32
// is 256 KB -- all of one SM's tensor memory -- so it is split across the two
// SMs of a cluster, 64 heads each, and the MMAs are pair MMAs
// (tcgen05.mma.cta_group::2, M = 128).  A pair MMA takes half of A's rows and
// half of B's columns from each CTA's shared memory.  Per 256-token tile:
//   S = Q K^T  (N = 256 tokens): CTA r holds Q rows 64r.. and tokens 128r..
//               of the tile; each CTA receives S for its 64 heads x 256 tokens,
//               folded into 128 lanes x 128 columns (lanes 64.. = tokens 128..).
//   O += P V   (N = 256 latent columns per MMA, two MMAs): CTA r holds P for
//               its heads and columns 128r.. of each 256-column group; each CTA
//               accumulates O for its 64 heads x 512 columns in 256 columns.
// The cache is therefore staged twice per CTA -- once token-split for S, once
// column-split for O -- which raises L2->SM traffic but reads HBM once and
// needs no exchange of partial scores between the SMs.
//
// Why 256-token tiles: one thread issues the MMAs, and a tcgen05.mma takes at
// least 45 cycles however little work it carries (measured); a pair MMA of
// M = 128 has the tensor pipe's full rate at N = 256 (64 cycles), not at
// N = 128 (45 for half the work).  A 256-token tile does not fit in shared
// memory beside the resident query (72 KB), so it is streamed: S = Q K^T in nine
// chunks of 64 columns (this CTA's 128 tokens, 16 KB each), O += P V in eight
// sub-stages of 64 tokens x 128 columns (16 KB each), all through one ring of
// 16 KB slots filled in the order the MMAs consume them.
//
// The roles that issue (TMA, MMA) run in a thread that elect.sync picks: with
// the thread picked by its lane number a wait, four MMAs and a commit took 493
// cycles instead of 257, which is the MMAs' own time.
//
// What bounds it: one call of a tree runs at 1.17 to 1.28 PFLOP/s (16 sequences
// of 8192 tokens x 1024 query rows 248 us; two of 12 to 16 thousand x 8192 rows
// 396 us), where the MMAs wait for ring slots (16 KB from L2 per 256 cycles and
// SM, seven in flight); back to back the board's power limit takes the clock to
// 1450-1700 MHz and the rate to 1.0-1.1 PFLOP/s.  Decode attention (128 rows a
// sequence, 64 x 8192 tokens: 146 us, 4.1 TB/s) adds the latency of HBM in every
// K slot, the pieces' boundaries and a start of some 8 us; 2048 selected tokens of
// each of 64 sequences take 56 us, 2.7 TB/s, nearly half of it boundaries and start.
//
// Warp roles per CTA (352 threads): warp 0 TMA producer, warp 1
// tensor-memory allocation and (leader CTA only) MMA issue, warps 2-9 softmax,
// O rescale and epilogue (two threads per tensor-memory lane), warp 10 the
// zeroes behind a sequence's last partial block.
//
// Tree of drafted tokens (kTree): the query rows of a sequence are (drafted
// token, head), any number of them, cut into groups of 128; a group takes the
// place of the 128 heads of one sequence and walks the cached tokens and the
// drafted ones behind them.  Only tiles that reach past the cached tokens look
// at the mask: the validity of a thread's 64 columns is two 32-bit words built
// from the row's 64-bit mask by shifts.  P.V takes the one or two blocks that hold
// drafted tokens (and the zeros behind them) from a copy that the plan's
// launch made, with non-finite values replaced by zero: a masked token has
// probability 0, but 0 * NaN would reach every row of the tile (a row that
// does attend such a token has a NaN score and so a NaN result).  That copy
// also spares every group the copy by hand.  A group whose tiles lie in one
// share is written out in bf16 at once, without a partial.
//
// Every wait is bounded; a wait that runs out flags MLA_ERR_TIMEOUT and the
// kernel winds down without further waits.
#include <math_constants.h>

#include <type_traits>

#include "plan.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 352;
constexpr int kSoftmaxWarps = 8;        // warps 2-9
constexpr int kHelperWarp = 10;
constexpr int kTileTok = 256;           // tokens per pair tile (MMA N of S = Q K^T)
constexpr int kHalfTok = 128;           // tokens of a tile each CTA stages for S
constexpr int kSubTok = 64;             // tokens per O += P V sub-stage
constexpr int kSlot = 16384;            // ring slot: a K chunk (128 rows x 128 B) or a V sub-stage
constexpr int kSlots = 7;               // 112 KB of ring: what is left beside Q (72 KB) and P (32 KB)
constexpr int kQBytes = 9 * 8192;       // 64 heads x 576 bf16, nine 64-column chunks
constexpr int kPBytes = 4 * 8192;       // 64 heads x 256 tokens bf16, four 64-token chunks
constexpr float kRescale = 8.0f;        // rescale O only when the running max grows by > 2^8

constexpr int kOffQ = 0;
constexpr int kOffRing = kOffQ + kQBytes;
constexpr int kOffP = kOffRing + kSlots * kSlot;
constexpr int kOffRed = kOffP + kPBytes;                // float red_m[2][4][64], red_l[4][64]
constexpr int kOffBar = kOffRed + 12 * 64 * 4;
// barriers
constexpr int kBarFull = 0;                     // [7] leader: an arrival from each CTA + tx bytes of both
constexpr int kBarEmpty = kBarFull + kSlots;    // [7] both: pair commit
constexpr int kBarQFull = kBarEmpty + kSlots;   // leader: 1 arrival + tx
constexpr int kBarQEmpty = kBarQFull + 1;       // both: pair commit
constexpr int kBarSFull = kBarQEmpty + 1;       // [2] both: pair commit
constexpr int kBarPFull = kBarSFull + 2;        // leader: 16 warp arrivals per tile
constexpr int kBarPFree = kBarPFull + 1;        // both: pair commit after each tile's P.V
constexpr int kBarODone = kBarPFree + 1;        // [2] both: pair commit after P.V of even / odd tiles
constexpr int kBarOFree = kBarODone + 2;        // leader: 16 warp arrivals
constexpr int kBarXchg = kBarOFree + 1;         // [2] local: 8 softmax-warp arrivals (row-max exchange)
constexpr int kBarLsum = kBarXchg + 2;          // local: 8 softmax-warp arrivals (row-sum exchange)
constexpr int kBarEnd = kBarLsum + 1;           // [2][2] local: the two loads of a sequence's last partial block
constexpr int kNumBars = kBarEnd + 4;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffPlan = kOffMisc + 32;
constexpr int kSmemBytes = kOffPlan + (int)sizeof(PlanSmem);
static_assert(kOffPlan % 8 == 0, "the plan holds 64-bit values");
constexpr int kSmemAlloc = kSmemBytes + 1024;
static_assert(kSmemAlloc <= 232448, "shared memory budget");
static_assert(kOffRing % 1024 == 0 && kOffP % 1024 == 0 && kSlot % 1024 == 0,
              "128-byte-swizzled buffers must be 1024-byte aligned");

constexpr uint32_t kTmemCols = 512;         // S: 2 x 128 columns, O: columns 256..511
constexpr uint32_t kColS = 128;
constexpr uint32_t kColO = 256;

constexpr uint32_t kIdescQK = idesc_bf16(128, kTileTok, false, false);
constexpr uint32_t kIdescPV = idesc_bf16(128, 256, false, true);

struct Piece {
  int b;               // batch sequence
  int v;               // plan sequence (b, or a run of row groups of b for a tree)
  int g;               // tree: the worker's row group of the run
  long long piece;     // global piece index
  int tok_begin;       // first token of the piece in sequence b
  int tok_end;         // one past the last token attended by this piece
  int ctx;             // the sequence's context length (clamped to the cache)
  int cached;          // tokens before a tree's drafted ones; of the sequence, where blocks of it are selected
  int ntiles;          // 256-token MMA tiles
};

// A role's position in its share.  The plan lies in shared memory (kInl) or in
// the workspace; either way its arrays are found again at every use, so that
// they take no registers through the loops.
template <bool kInl>
struct Walk {
  const PlanSmem *o;
  long long t0, t1;
  int b;
  int member;   // tree: which of the share's workers this is
};
template <bool kInl>
__device__ __forceinline__ const long long *plan_tp(const AttnArgs &a, const Walk<kInl> &w) {
  return kInl ? w.o->tp : reinterpret_cast<const long long *>(a.ws + a.L.tile_prefix_off);
}
template <bool kInl>
__device__ __forceinline__ const long long *plan_pb(const AttnArgs &a, const Walk<kInl> &w) {
  return kInl ? w.o->pb : reinterpret_cast<const long long *>(a.ws + a.L.piece_base_off);
}
template <bool kInl>
__device__ __forceinline__ long long plan_P(const AttnArgs &a, const Walk<kInl> &w) {
  return kInl ? w.o->P : reinterpret_cast<const WsHeader *>(a.ws)->P;
}
template <bool kInl>
__device__ __forceinline__ long long plan_Ttot(const AttnArgs &a, const Walk<kInl> &w) {
  return kInl ? w.o->Ttot : reinterpret_cast<const WsHeader *>(a.ws)->Ttot;
}

template <bool kInl>
__device__ __forceinline__ void walk_init(Walk<kInl> &w, const AttnArgs &a, const PlanSmem &o, int share) {
  w.o = &o;
  w.member = (blockIdx.x >> 1) % a.tree.gang;
  const long long P = plan_P(a, w), Ttot = plan_Ttot(a, w);
  w.b = a.B;
  if (share >= P) return;
  w.b = kInl ? o.first : reinterpret_cast<const int *>(a.ws + a.L.share_first_off)[share];
  w.t0 = kInl ? o.t0 : plan_begin(share, P, Ttot);
  w.t1 = kInl ? o.t1 : plan_begin(share + 1, P, Ttot);
}

// Next piece of this share; false when done.
template <bool kTree, bool kInl>
__device__ __forceinline__ bool walk_next(Walk<kInl> &w, const AttnArgs &a, int share, Piece &pc) {
  const long long *tp = plan_tp(a, w);
  const int *ends = kInl ? w.o->ends : plan_ends(a), *seconds = kInl ? w.o->seconds : plan_seconds(a);
  while (w.b < a.B && tp[w.b] < w.t1) {
    const int b = w.b++;
    const long long s0 = w.t0 > tp[b] ? w.t0 : tp[b];
    const long long s1 = w.t1 < tp[b + 1] ? w.t1 : tp[b + 1];
    if (s0 >= s1) continue;
    pc.b = kTree ? b / a.tree.runs : b;
    pc.v = b;
    pc.g = kTree ? (b - pc.b * a.tree.runs) * a.tree.gang + w.member : 0;
    if (kTree && pc.g >= a.tree.groups) continue;
    const int ctx = ends[b];
    const int beg = kTree || a.sel ? 0 : seconds[b];
    pc.cached = kTree || a.sel ? seconds[b] : ctx;
    pc.piece = kTree ? 0 : plan_pb(a, w)[b] + (share - plan_share_of_tile(tp[b], plan_P(a, w), plan_Ttot(a, w)));
    pc.tok_begin = beg + (int)((s0 - tp[b]) * a.plan_tile);
    const long long e = beg + (s1 - tp[b]) * a.plan_tile;
    pc.tok_end = (int)(e < ctx ? e : ctx);
    pc.ctx = ctx;
    pc.ntiles = (pc.tok_end - pc.tok_begin + kTileTok - 1) / kTileTok;
    return true;
  }
  return false;
}

// The k lowest bits (none for k <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int k) { return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u); }

// Bits of word w (columns 32w .. 32w + 31) of a row's validity: column c holds
// token base + c, valid below `cached` and, past it, where `bits` has the
// drafted token's bit; `n` columns lie inside the piece.
__device__ __forceinline__ uint32_t tree_valid(int w, int base, int n, int cached, unsigned long long bits) {
  const int sh = cached - base - 32 * w;     // column of the first drafted token within the word
  uint32_t d = 0;
  if (sh >= 0 && sh < 32) d = (uint32_t)(bits << sh);
  else if (sh < 0 && sh > -64) d = (uint32_t)(bits >> -sh);
  return (low_bits(sh) | d) & low_bits(n - 32 * w);
}

struct Bars {
  uint64_t *b;
  __device__ uint64_t *full(int s) { return b + kBarFull + s; }
  __device__ uint64_t *empty(int s) { return b + kBarEmpty + s; }
  __device__ uint64_t *qfull() { return b + kBarQFull; }
  __device__ uint64_t *qempty() { return b + kBarQEmpty; }
  __device__ uint64_t *sfull(int i) { return b + kBarSFull + i; }
  __device__ uint64_t *pfull() { return b + kBarPFull; }
  __device__ uint64_t *pfree() { return b + kBarPFree; }
  __device__ uint64_t *odone(int i) { return b + kBarODone + i; }
  __device__ uint64_t *ofree() { return b + kBarOFree; }
  __device__ uint64_t *xchg(int i) { return b + kBarXchg + i; }
  __device__ uint64_t *lsum() { return b + kBarLsum; }
  __device__ uint64_t *end(int n, int g) { return b + kBarEnd + 2 * (n & 1) + g; }
};

// Warp-uniform bounded wait: lane 0 waits, the result is broadcast, the other
// lanes then observe the completed phase themselves (acquire).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, unsigned *status,
                                          volatile int *abort) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = ptx::mbar_wait(bar, parity, status, abort);
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  if (ok && (threadIdx.x & 31) != 0) ptx::mbar_test_wait(bar, parity);
  __syncwarp();
  return ok;
}

// Row coordinates of the four 64-token blocks of the tile at token t0 of a
// piece: an out-of-range row (TMA then fills zeros) for a block past the piece
// and, marked in `bad`, for one that is unmapped, outside the cache or not a
// block of the sequence (see selected_row).  The table and selection entries
// of all four are requested before any is used, and nothing branches on them.
struct Rows {
  int r[4];
  unsigned bad;
};
template <bool kTree>
__device__ __forceinline__ Rows look_up(const AttnArgs &a, const Piece &p, int t0, int kv_rows) {
  Rows x;
  x.bad = 0;
  const bool chosen = !kTree && a.sel != nullptr;
  int blk[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    blk[t] = t0 / kTile + t;
    if (chosen && t0 + kTile * t < p.tok_end) blk[t] = a.sel[(long long)p.b * a.sel_k + blk[t]];
  }
  bool ok[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    ok[t] = true;
    if (chosen) {
      const long long e = (long long)blk[t] * kTile;
      ok[t] = blk[t] >= 0 && e < p.cached && (e + kTile <= p.cached || t0 / kTile + t == (p.ctx - 1) / kTile);
    }
    if (a.page_size) {
      ok[t] = ok[t] && blk[t] < a.max_blocks;
      if (ok[t] && t0 + kTile * t < p.tok_end) blk[t] = a.block_table[(long long)p.b * a.max_blocks + blk[t]];
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (a.page_size) ok[t] = ok[t] && blk[t] >= 0 && blk[t] < a.cache_len;
    const bool here = t0 + kTile * t < p.tok_end;
    const long long row = (a.page_size ? 0 : (long long)p.b * a.cache_len) + (long long)blk[t] * kTile;
    x.r[t] = here && ok[t] ? (int)row : kv_rows;
    x.bad |= here && !ok[t] ? 1u << t : 0u;
  }
  return x;
}

// O += P V sub-stages of a tile that starts at token t0 of the piece (the
// sub-stages past the piece's end are skipped by the producer and the MMAs).
__device__ __forceinline__ int tile_subs(const Piece &p, int t0) {
  const int n = min(p.tok_end - t0, kTileTok);
  return (n + kSubTok - 1) / kSubTok;
}

template <bool kTree, bool kInl>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attn_pair_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                     const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapV2,
                     const __grid_constant__ CUtensorMap mapT, const AttnArgs a, const long long kv_rows) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = sm + kOffQ;
  uint8_t *sRing = sm + kOffRing;
  uint8_t *sP = sm + kOffP;
  float *red_m = reinterpret_cast<float *>(sm + kOffRed);   // [2][4][64]
  float *red_l = red_m + 512;                                // [4][64]
  Bars bars{reinterpret_cast<uint64_t *>(sm + kOffBar)};
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffMisc + 4);
  int *end_slot = reinterpret_cast<int *>(sm + kOffMisc + 8);   // [2][2] ring slots of a last partial block

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int share = kTree ? (blockIdx.x >> 1) / a.tree.gang : blockIdx.x >> 1;
  pdl_trigger();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      ptx::mbar_init(bars.full(s), 2);
      ptx::mbar_init(bars.empty(s), 1);
    }
    ptx::mbar_init(bars.qfull(), 1);
    ptx::mbar_init(bars.qempty(), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars.sfull(i), 1);
      ptx::mbar_init(bars.odone(i), 1);
      ptx::mbar_init(bars.xchg(i), kSoftmaxWarps);
    }
    for (int i = 0; i < 4; ++i) ptx::mbar_init(bars.end(i >> 1, i & 1), 1);
    ptx::mbar_init(bars.pfull(), 2 * kSoftmaxWarps);
    ptx::mbar_init(bars.pfree(), 1);
    ptx::mbar_init(bars.ofree(), 2 * kSoftmaxWarps);
    ptx::mbar_init(bars.lsum(), kSoftmaxWarps);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync_all();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The set-up above overlaps the previous kernel; from here on the lengths,
  // the query and the cache it wrote are read.
  pdl_wait();
  PlanSmem &plan_smem = *reinterpret_cast<PlanSmem *>(sm + kOffPlan);
  if (kInl) plan_in_line(a, share, gridDim.x / 2, plan_smem);

  if (warp == 0) {
    // --------------------------------------------------------------- producer
    // Fills the ring in the order the MMAs consume it: the nine K chunks of
    // tile i, then the V sub-stages of tile i-1; at the end of a piece its last
    // tile's V comes before the next piece's K, which waits for another Q.  A
    // slot's full barrier (the leader's) takes an arrival from each CTA; the
    // leader's also arms it with the bytes both CTAs' loads bring (the peer's
    // loads count on the leader's barrier directly).  One elected thread does it
    // all, in few instructions a slot (the MMAs want one every 256 cycles): a
    // tile's four cache rows are looked up once, for the tile after the one being
    // loaded, so that a paged cache's table reads are not waited for.
    if (ptx::elect_one()) {
      const bool boxes64 = a.page_size != 0 || (!kTree && a.sel != nullptr);
      const uint32_t lq = ptx::leader_addr(bars.qfull());
      const uint32_t lf0 = ptx::leader_addr(bars.full(0));
      ptx::tma_prefetch_desc(&mapQ);
      ptx::tma_prefetch_desc(&mapK);
      ptx::tma_prefetch_desc(&mapV);
      ptx::tma_prefetch_desc(&mapV2);
      if (kTree) ptx::tma_prefetch_desc(&mapT);
      Walk<kInl> w;
      walk_init(w, a, plan_smem, share);
      const uint64_t last_read = ptx::l2_policy_evict_first();
      int slot = 0;              // ring slot of the next job
      uint32_t phase = 1;        // parity of its empty barrier to wait for (the first round passes at once)
      // Waits for the next slot and arms its full barrier.
      auto take = [&]() -> bool {
        if (!ptx::mbar_wait(bars.empty(slot), phase, a.status, abort_flag)) return false;
        if (leader) ptx::mbar_arrive_expect_tx(bars.full(slot), 2 * kSlot);
        else ptx::mbar_arrive_remote_addr(lf0 + 8 * slot);
        return true;
      };
      auto step = [&]() {
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      };
      // V sub-stages of the tile at token t0 of piece p: tokens t0 + 64t..,
      // latent columns 256g + 128 * rank .. +128, one 3D box: 64 rows x both
      // 64-column chunks.
      int nend = 0;              // partial blocks so far
      auto issue_v = [&](const Piece &p, int t0, const Rows &x) -> bool {
        const int nsub = tile_subs(p, t0);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (t >= nsub) break;
          const int tok0 = t0 + kSubTok * t;
          const bool copied = kTree && tok0 + kSubTok > p.cached;
          const CUtensorMap *map = copied ? &mapT : &mapV2;
          const int y = copied ? p.b * kTreeCopyRows + tok0 - p.cached / kTile * kTile : x.r[t];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int chunk0 = 4 * g + 2 * (int)rank;
            uint8_t *dst = sRing + slot * kSlot;
            if (!kTree && tok0 + kSubTok > p.ctx) {
              // The block runs past the sequence: its load completes on a
              // barrier of its own, where the helper warp waits, which zeroes
              // the rows past the end and then arrives for this CTA.  Between
              // two such blocks lie nine K chunks, more than a ring; with two
              // sets of barriers and slot numbers nothing rests on that count.
              if (!ptx::mbar_wait(bars.empty(slot), phase, a.status, abort_flag)) return false;
              end_slot[2 * (nend & 1) + g] = slot;
              ptx::mbar_arrive_expect_tx(bars.end(nend, g), kSlot);
              ptx::tma_load_3d(dst, map, bars.end(nend, g), 0, y, chunk0);
              if (g == 1) ++nend;
            } else {
              if (!take()) return false;
              ptx::tma_load_3d_pair_hint(dst, map, lf0 + 8 * slot, 0, y, chunk0, last_read);
            }
            step();
          }
        }
        return true;
      };
      Piece pc, vpc;             // vpc, vt0, vx: the tile whose V sub-stages are pending
      Rows x, vx;
      int vt0 = 0, npc = 0;
      bool vpending = false, ok = true;
      while (ok && walk_next<kTree, kInl>(w, a, share, pc)) {
        if (vpending && !issue_v(vpc, vt0, vx)) break;
        vpending = false;
        if (npc > 0 && !ptx::mbar_wait(bars.qempty(), (npc - 1) & 1, a.status, abort_flag)) break;
        if (leader) ptx::mbar_arrive_expect_tx(bars.qfull(), 2 * kQBytes);
#pragma unroll 1
        for (int c = 0; c < 9; ++c) {
          if (kTree)   // rows past the sequence's are zero-filled
            ptx::tma_load_3d_pair(sQ + c * 8192, &mapQ, lq, 64 * c, 128 * pc.g + 64 * (int)rank, pc.b);
          else
            ptx::tma_load_2d_pair(sQ + c * 8192, &mapQ, lq, 64 * c, pc.b * 128 + 64 * (int)rank);
        }
        Rows next = look_up<kTree>(a, pc, pc.tok_begin, (int)kv_rows);
        for (int k = 0; k < pc.ntiles && ok; ++k) {
          const int t0 = pc.tok_begin + kTileTok * k;
          x = next;
          if (x.bad) atomicOr(a.status, kStatusBounds);
          // K chunks of this tile: this CTA's 128 tokens x 64 columns each.
          const int y0 = rank ? x.r[2] : x.r[0], y1 = rank ? x.r[3] : x.r[1];
#pragma unroll 1
          for (int c = 0; c < 9; ++c) {
            if (!take()) { ok = false; break; }
            uint8_t *dst = sRing + slot * kSlot;
            if (!boxes64) {
              ptx::tma_load_2d_pair(dst, &mapK, lf0 + 8 * slot, 64 * c, y0);
            } else {
              // 64-token pages or selected blocks: two 64-row boxes.
              ptx::tma_load_2d_pair(dst, &mapV, lf0 + 8 * slot, 64 * c, y0);
              ptx::tma_load_2d_pair(dst + 8192, &mapV, lf0 + 8 * slot, 64 * c, y1);
            }
            step();
          }
          if (!ok) break;
          if (k + 1 < pc.ntiles) next = look_up<kTree>(a, pc, t0 + kTileTok, (int)kv_rows);
          if (vpending && !issue_v(vpc, vt0, vx)) { ok = false; break; }
          vpc = pc;
          vt0 = t0;
          vx = x;
          vpending = true;
        }
        ++npc;
      }
      if (ok && vpending) issue_v(vpc, vt0, vx);
    }
  } else if (warp == kHelperWarp) {
    // ----------------------------------------- rows behind a sequence's end
    // Zeroes what the last partial block's load brought from behind the
    // sequence, so that no unwritten cache row (possibly NaN) reaches P.V.
    if (!kTree) {
      const uint32_t lf0 = ptx::leader_addr(bars.full(0));
      Walk<kInl> w;
      walk_init(w, a, plan_smem, share);
      Piece pc;
      int n = 0;
      bool ok = true;
      while (ok && walk_next<kTree, kInl>(w, a, share, pc)) {
        const int row0 = pc.ctx % kSubTok;
        if (pc.tok_end != pc.ctx || row0 == 0) continue;
        for (int g = 0; g < 2; ++g) {
          if (!warp_wait(bars.end(n, g), (n >> 1) & 1, a.status, abort_flag)) { ok = false; break; }
          const int s = end_slot[2 * (n & 1) + g];
          uint8_t *dst = sRing + s * kSlot;
          for (int u = lane; u < (kSubTok - row0) * 16; u += 32)
            *reinterpret_cast<uint4 *>(dst + (u & 8) * 1024 + (row0 + (u >> 4)) * 128 + (u & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote_addr(lf0 + 8 * s);
        }
        ++n;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    const bool issuer = ptx::elect_one();
    if (leader && issuer) {
      Walk<kInl> w;
      walk_init(w, a, plan_smem, share);
      Piece pc;
      int npc = 0, i = 0;
      int rs = 0;                 // ring slot of the next job
      uint32_t rph = 0;           // its full-barrier phase parity
      bool ok = true;
      struct PrevTile { int i, first, npc, nsub; } prev{0, 0, 0, 0};
      bool have_prev = false;
      // Descriptors are built once; the start address (bits 0-13, 16-byte
      // units) is advanced by adding offsets.  The issue loop is kept lean:
      // one thread issues every MMA, and its own instruction latency, not the
      // tensor pipe, bounds the rate when the loop does more than it must.
      const uint64_t dQ = ptx::sdesc(ptx::smem_u32(sQ), 16, 1024, 2);
      const uint64_t dK = ptx::sdesc(ptx::smem_u32(sRing), 16, 1024, 2);
      const uint64_t dV = ptx::sdesc(ptx::smem_u32(sRing), 8192, 1024, 2);
      const uint64_t dP = ptx::sdesc(ptx::smem_u32(sP), 16, 1024, 2);
      // Waits for the next ring job; returns its slot or -1.
      auto slot_wait = [&]() -> int {
        const int s = rs;
        if (!ptx::mbar_wait(bars.full(s), rph, a.status, abort_flag)) return -1;
        ptx::tc_fence_after();
        if (++rs == kSlots) {
          rs = 0;
          rph ^= 1u;
        }
        return s;
      };
      auto pv = [&](const PrevTile &t) -> bool {
        if (t.first && t.npc > 0 && !ptx::mbar_wait(bars.ofree(), (t.npc - 1) & 1, a.status, abort_flag))
          return false;
        if (!ptx::mbar_wait(bars.pfull(), t.i & 1, a.status, abort_flag)) return false;
        ptx::tc_fence_after();
        for (int tt = 0; tt < t.nsub; ++tt) {
          const uint64_t ad = dP + (uint64_t)((tt * 8192) >> 4);
          const uint32_t acc0 = (t.first && tt == 0) ? 0u : 1u;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int s = slot_wait();
            if (s < 0) return false;
            // A = P rows (heads) x tokens 64tt + 16j.. (K-major); B = V rows
            // (tokens 16j.. of the sub-stage) x 128 columns in two 64-column
            // chunks 8 KB apart.
            const uint64_t bd = dV + (uint64_t)((s * kSlot) >> 4);
            const uint32_t d = tmem + kColO + 128 * g;
            ptx::mma_bf16_ss_pair(d, ad, bd, kIdescPV, acc0);
            ptx::mma_bf16_ss_pair(d, ad + 2, bd + 128, kIdescPV, 1u);
            ptx::mma_bf16_ss_pair(d, ad + 4, bd + 256, kIdescPV, 1u);
            ptx::mma_bf16_ss_pair(d, ad + 6, bd + 384, kIdescPV, 1u);
            ptx::mma_commit_pair_both(bars.empty(s));
          }
        }
        ptx::mma_commit_pair_both(bars.pfree());
        ptx::mma_commit_pair_both(bars.odone(t.i & 1));
        return true;
      };
      while (ok && walk_next<kTree, kInl>(w, a, share, pc)) {
        // The previous piece's last P.V goes first: this piece's S waits for its
        // Q, which is loaded once the previous piece's last S is done (a
        // piece's output is ready 2 to 3 us earlier than behind that S).
        if (have_prev && !pv(prev)) { ok = false; break; }
        have_prev = false;
        if (!ptx::mbar_wait(bars.qfull(), npc & 1, a.status, abort_flag)) { ok = false; break; }
        for (int k = 0; k < pc.ntiles && ok; ++k) {
          const uint32_t dS = tmem + (i & 1) * kColS;
#pragma unroll
          for (int c = 0; c < 9; ++c) {
            const int s = slot_wait();
            if (s < 0) { ok = false; break; }
            // A = Q chunk c (64-column chunks 8 KB apart), B = this slot's
            // 128 tokens x 64 columns; k steps of 16 columns are 32 B apart.
            const uint64_t ad = dQ + (uint64_t)((c * 8192) >> 4);
            const uint64_t bd = dK + (uint64_t)((s * kSlot) >> 4);
            ptx::mma_bf16_ss_pair(dS, ad, bd, kIdescQK, c != 0 ? 1u : 0u);
            ptx::mma_bf16_ss_pair(dS, ad + 2, bd + 2, kIdescQK, 1u);
            ptx::mma_bf16_ss_pair(dS, ad + 4, bd + 4, kIdescQK, 1u);
            ptx::mma_bf16_ss_pair(dS, ad + 6, bd + 6, kIdescQK, 1u);
            ptx::mma_commit_pair_both(bars.empty(s));
          }
          if (!ok) break;
          ptx::mma_commit_pair_both(bars.sfull(i & 1));
          if (k == pc.ntiles - 1) ptx::mma_commit_pair_both(bars.qempty());
          if (have_prev && !pv(prev)) { ok = false; break; }
          prev = {i, k == 0 ? 1 : 0, npc, tile_subs(pc, pc.tok_begin + kTileTok * k)};
          have_prev = true;
          ++i;
        }
        ++npc;
      }
      if (ok && have_prev) pv(prev);
    }
  } else {
    // ------------------------------------------- softmax, rescale, epilogue
    // Two warps to a tensor-memory quadrant: thread (l, hf) owns lane l, i.e.
    // local head h and token half th, and columns 64 hf .. of that half's 128
    // scores: token chunk part = 2 th + hf of the tile.  A head's row is held
    // by four threads, which exchange their maxima and sums through shared
    // memory.
    const int q = warp & 3, hf = (warp - 2) >> 2;
    const int l = q * 32 + lane;
    const int h = l & 63, th = l >> 6, part = 2 * th + hf;
    const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t o_addr = lane_addr + kColO + 128 * hf;   // latent columns 256 hf + 128 th ..
    const uint32_t leader_pfull = ptx::leader_addr(bars.pfull());
    const uint32_t leader_ofree = ptx::leader_addr(bars.ofree());
    float *opart = reinterpret_cast<float *>(a.ws + a.L.opart_off);
    float *lse_out = reinterpret_cast<float *>(a.ws + a.L.lse_off);
    uint8_t *prow = sP + part * 8192 + h * 128;   // this row of the thread's 64-token P chunk
    Walk<kInl> w;
    walk_init(w, a, plan_smem, share);
    Piece pc;
    int i = 0, npc_s = 0;
    bool ok = true;
    while (ok && walk_next<kTree, kInl>(w, a, share, pc)) {
      float m_run = kNoMax, l_part = 0.f;
      // tree: this thread's query row of the sequence, and its drafted tokens
      const int row = 128 * pc.g + 64 * (int)rank + h;
      unsigned long long bits = 0ull;
      if (kTree && row < a.tree.seq_rows) {
        bits = a.tree.mask[(long long)pc.b * a.tree.T + row / a.n_h];
        if (a.tree.T < 64) bits &= (1ull << a.tree.T) - 1ull;
      }
      for (int k = 0; k < pc.ntiles; ++k, ++i) {
        const int base = pc.tok_begin + kTileTok * k + 64 * part;
        const int nvalid = min(max(pc.tok_end - base, 0), 64);
        if (!warp_wait(bars.sfull(i & 1), (i >> 1) & 1, a.status, abort_flag)) { ok = false; break; }
        ptx::tc_fence_after();
        // This thread's 64 products, invalid tokens at -inf.  The scale to log2
        // units is positive, so the maximum is taken first and the scale
        // joins the subtraction in one (two-wide) multiply-add: the kernel
        // runs into the board's power limit, and every instruction a score
        // costs counts.
        float v[64];
        ptx::tmem_ld64_sync(lane_addr + (i & 1) * kColS + 64 * hf, reinterpret_cast<uint32_t *>(v));
        float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
        if (base + 64 <= (kTree ? min(pc.cached, pc.tok_end) : pc.tok_end)) {
#pragma unroll
          for (int j = 0; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
        } else {
          uint32_t valid[2];
#pragma unroll
          for (int w2 = 0; w2 < 2; ++w2)
            valid[w2] = kTree ? tree_valid(w2, base, nvalid, pc.cached, bits) : low_bits(nvalid - 32 * w2);
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            v[j] = (valid[j >> 5] >> (j & 31)) & 1u ? v[j] : -CUDART_INF_F;
            mx[j & 3] = fmaxf(mx[j & 3], v[j]);
          }
        }
        const float mloc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        float *rm = red_m + (i & 1) * 256;
        rm[part * 64 + h] = mloc;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.xchg(i & 1));
        if (!warp_wait(bars.xchg(i & 1), (i >> 1) & 1, a.status, abort_flag)) { ok = false; break; }
        const float m_tile = fmaxf(fmaxf(rm[h], rm[64 + h]), fmaxf(rm[128 + h], rm[192 + h])) * a.scale_log2;
        bool rescale = false;
        float alpha = 1.f;
        if (m_tile > m_run + kRescale) {
          alpha = exp2f(m_run - m_tile);       // 0 when m_run = kNoMax
          m_run = m_tile;
          l_part *= alpha;
          rescale = k > 0;
        }
        // Probabilities (bf16 pairs) and their sum, before waiting for the
        // previous tile's P.V, so that only the store below waits for it.
        // P is rounded to bf16 because the MMA takes both operands in one
        // 16-bit type and V is bf16; the sum is of the unrounded values.
        uint32_t pk[32];
        float2 ps[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        const float2 scale2 = {a.scale_log2, a.scale_log2}, m2 = {-m_run, -m_run};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float2 p = ptx::fma2({v[2 * j], v[2 * j + 1]}, scale2, m2);
          p.x = ptx::exp2_approx(p.x);
          p.y = ptx::exp2_approx(p.y);
          ps[j & 3] = ptx::add2(ps[j & 3], p);
          __nv_bfloat162 b2 = __float22bfloat162_rn(p);
          pk[j] = *reinterpret_cast<uint32_t *>(&b2);
        }
        const float2 sum2 = ptx::add2(ptx::add2(ps[0], ps[1]), ptx::add2(ps[2], ps[3]));
        l_part += sum2.x + sum2.y;
        // P of the previous tile must have been read by its P.V.
        if (i >= 1 && !warp_wait(bars.pfree(), (i - 1) & 1, a.status, abort_flag)) { ok = false; break; }
        // Tokens 8u .. of the chunk are 16-byte unit u of row h (128-byte swizzle by row).
#pragma unroll
        for (int u = 0; u < 8; ++u)
          *reinterpret_cast<uint4 *>(prow + ((u ^ (h & 7)) << 4)) =
              make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        // The rescale (tensor-memory loads and stores, .sync.aligned) is done by
        // the whole warp when any of its rows needs it; other rows use alpha = 1.
        if (__any_sync(0xffffffffu, rescale)) {
          // P.V of the previous tile must be complete before O is rescaled.
          // o_done[b] completes for the P.V of tiles b, b+2, ...; since S of
          // this tile is complete, every P.V up to tile i-2 is too (MMAs of
          // one thread complete in order), so the wait below is never more
          // than one phase away from the barrier's state.
          if (!warp_wait(bars.odone((i - 1) & 1), ((i - 1) >> 1) & 1, a.status, abort_flag)) { ok = false; break; }
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t r[16];
            ptx::tmem_ld16(o_addr + 16 * c, r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha);
            ptx::tmem_st16(o_addr + 16 * c, r);
          }
          ptx::tmem_st_wait();
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_addr(leader_pfull);
      }
      if (!ok) break;
      // ---- epilogue of the piece: O / l and the log-sum-exp
      red_l[part * 64 + h] = l_part;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars.lsum());
      if (!warp_wait(bars.lsum(), npc_s & 1, a.status, abort_flag)) { ok = false; break; }
      ++npc_s;
      const float lsum = (red_l[h] + red_l[64 + h]) + (red_l[128 + h] + red_l[192 + h]);
      if (!warp_wait(bars.odone((i - 1) & 1), ((i - 1) >> 1) & 1, a.status, abort_flag)) { ok = false; break; }
      ptx::tc_fence_after();
      const int head = 64 * (int)rank + h;
      // a row that attends nothing is zero, a NaN sum stays NaN
      const bool some = lsum != 0.f;
      const float inv = some ? 1.f / lsum : 0.f;
      const float z = some ? (m_run + log2f(lsum)) * 0.69314718055994531f : -CUDART_INF_F;
      long long slot = pc.piece;
      bool whole = false;
      if (kTree) {
        const TreePiece t = tree_piece(a, plan_tp(a, w), pc.v, share, w.member, plan_P(a, w), plan_Ttot(a, w));
        whole = t.whole;
        slot = t.slot;
      }
      if (hf == 0 && th == 0 && !(kTree && row >= a.tree.seq_rows)) {
        if (!whole) lse_out[part_row(a.L, slot, head)] = z;
        else if (a.tree.lse) a.tree.lse[(long long)pc.b * a.tree.seq_rows + row] = z;
      }
      // The warp's 32 rows x 128 columns pass through shared memory 128 bytes
      // of every row at a time (its 4 KB of the P buffer, which no P.V reads
      // any more; the next P is stored only after all eight warps have met at
      // a row-maximum exchange), so that a store instruction writes whole
      // 128-byte lines of four rows, not 16 bytes of 32 rows (a piece's
      // epilogue 7 -> 2.5 us).  16-byte units are swizzled by row.
      uint8_t *stage = sP + (warp - 2) * 4096;
      const int col0 = 256 * hf + 128 * th;
      const int r0 = 64 * (int)rank + (q & 1) * 32;   // first head / row of the warp within the 128
      if (kTree && whole) {
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.tree.out);
        const int g0 = 128 * pc.g + r0;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          float v[64];
          ptx::tmem_ld64_sync(o_addr + 64 * c, reinterpret_cast<uint32_t *>(v));
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * u + 2 * j] * inv, v[8 * u + 2 * j + 1] * inv);
              o[j] = *reinterpret_cast<const uint32_t *>(&b2);
            }
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int r = 4 * it + (lane >> 3), u = lane & 7;
            const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((u ^ (r & 7)) << 4));
            if (g0 + r < a.tree.seq_rows)
              *reinterpret_cast<uint4 *>(out + ((long long)pc.b * a.tree.seq_rows + g0 + r) * a.d_c + col0 + 64 * c +
                                         8 * u) = x;
          }
          __syncwarp();
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          ptx::tmem_ld16(o_addr + 32 * c, *reinterpret_cast<uint32_t(*)[16]>(v));
          ptx::tmem_ld16(o_addr + 32 * c + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
          ptx::tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<float4 *>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) =
                make_float4(__uint_as_float(v[4 * u]) * inv, __uint_as_float(v[4 * u + 1]) * inv,
                            __uint_as_float(v[4 * u + 2]) * inv, __uint_as_float(v[4 * u + 3]) * inv);
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int r = 4 * it + (lane >> 3), u = lane & 7;
            *reinterpret_cast<float4 *>(opart + part_row(a.L, slot, r0 + r) * (long long)a.d_c + col0 + 32 * c + 4 * u) =
                *reinterpret_cast<const float4 *>(stage + r * 128 + ((u ^ (r & 7)) << 4));
          }
          __syncwarp();
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote_addr(leader_ofree);
      // red_l is rewritten only after the next piece's per-tile exchanges
    }
  }

  // ---------------------------------------------------------------- teardown
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync_all();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

namespace {
template <bool kTree>
cudaError_t launch_pair(const AttnArgs &a, int P, cudaStream_t s, const Before &before) {
  if (a.d_c != 512 || a.d_r != 64) return cudaErrorNotSupported;
  if (a.page_size != 0 && a.page_size != kTile) return cudaErrorNotSupported;
  const int batch = kTree ? a.B / a.tree.runs : a.B;
  const long long rows = a.page_size ? a.cache_len * kTile : (long long)batch * a.cache_len;
  if (rows <= 0 || rows >= (1ll << 31) - 256) return cudaErrorNotSupported;
  CUtensorMap mq, mk, mv, mv2, mt;
  // queries: [B * 128 rows], or [B][seq_rows] for a tree, 64 rows to a box
  const uint64_t dq[3] = {576, kTree ? (uint64_t)a.tree.seq_rows : (uint64_t)a.B * 128, (uint64_t)batch};
  const uint64_t sq[2] = {576 * 2, 576 * 2 * dq[1]};
  const uint64_t dkv[2] = {576, (uint64_t)rows};
  const uint64_t st[1] = {576 * 2};
  const uint32_t boxq[3] = {64, 64, 1};
  const uint32_t boxk[2] = {64, kHalfTok};
  const uint32_t boxv[2] = {64, kSubTok};
  // The cache viewed as [9 chunks][rows][64 columns]: one box of 64 rows x 2
  // chunks lands as two 8 KB row-major chunks, the V sub-stage layout.
  const uint64_t dkv3[3] = {64, (uint64_t)rows, 9};
  const uint64_t st3[2] = {576 * 2, 64 * 2};
  const uint32_t boxv3[3] = {64, kSubTok, 2};
  if (!encode_map_bf16(&mq, a.q_abs, kTree ? 3 : 2, dq, sq, boxq, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_bf16(&mk, a.cache, 2, dkv, st, boxk, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_bf16(&mv, a.cache, 2, dkv, st, boxv, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_bf16(&mv2, a.cache, 3, dkv3, st3, boxv3, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  mt = mv2;
  const uint64_t dt3[3] = {64, (uint64_t)batch * kTreeCopyRows, 9};
  if (kTree && !encode_map_bf16(&mt, a.ws + a.tree.copy_off, 3, dt3, st3, boxv3, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorNotSupported;
  auto go = [&](auto inl) {
    constexpr bool kInl = decltype(inl)::value;
    static std::atomic<int> configured[kMaxDevices];
    cudaError_t e = once_per_device(configured, [] {
      return cudaFuncSetAttribute(attn_pair_kernel<kTree, kInl>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
    });
    if (e == cudaSuccess && before) e = before();
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_pair_kernel<kTree, kInl>, dim3(2 * P * a.tree.gang), dim3(kThreads), kSmemAlloc, s, 1, mq, mk,
                      mv, mv2, mt, a, rows);
  };
  if constexpr (!kTree)
    if (a.inline_plan) return go(std::true_type());
  return go(std::false_type());
}
}  // namespace

cudaError_t launch_attn_tc_pair(const AttnArgs &a, int P, cudaStream_t s, const Before &before) {
  if (a.n_h != 128) return cudaErrorNotSupported;
  return launch_pair<false>(a, P, s, before);
}

cudaError_t launch_tree_attn_tc_pair(const AttnArgs &a, int P, cudaStream_t s, const Before &before) {
  return launch_pair<true>(a, P, s, before);
}

}  // namespace mla
