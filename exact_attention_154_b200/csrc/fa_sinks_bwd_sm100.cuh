// fa_sinks_bwd_sm100.cuh -- gradient of causal attention with a sliding window
// and sinks (key / value heads shared by groups of query heads), for sm_100a.
//
// The formulas are those of fa_bwd_sm100.cuh (P from the saved logsumexp, D_i =
// dO_i . O_i by bwd_dsum_kernel), over the pairs the mask leaves visible:
//
//   dV_j = sum_i P_ij dO_i,  dS = P (dO V^T - D),  dK_j = scale sum_i dS_ij Q_i,
//   dQ_i = scale sum_j dS_ij K_j
//
// with dK and dV summed over the query heads of a group in one accumulator.
//
// dK/dV kernel: a unit is a 128-key block of a key head with the query blocks
// that see it, of each query head in turn: S^T = K Q^T and dP^T = V dO^T into
// TMEM, P^T and dS^T packed back to 16 bits there, dV += P^T dO and dK += dS^T
// Q from TMEM.  A block that holds sinks is seen by every later query, so its
// query blocks are dealt out as several units ("pieces") whose fp32 sums
// sinks_sum_kernel adds; where units are few, all are split by their steps in the
// same manner.  dQ kernel: a unit is a 128-query block of a query head
// with the key blocks it sees; dQ += dS K.
//
// What bounds a step (128 x 128 pairs) is a chain: exponentials (the
// exponential unit alone needs 1024 of a step's cycles), dS, the products that
// read them, the next scores.  So P's chain and dS's are kept apart:
//
//   warps   | load S, exp, P ->|<- load dP, dS ->| (next) load S, exp, P ->| ..
//   tensor  |    dP(it)        | dV(it), S(it+1) | dK(it), dP(it+1)        | ..
//
// P^T is packed over the S columns it came from and dS^T over the dP columns,
// each by the warp that read them; S(it+1) follows dV(it), and dP(it+1) dK(it),
// in the MMA thread's order, which also is all the hand-back those columns
// need.  The dQ kernel has no P to keep, so its S(it+1) only waits for S(it) to
// be read, and two dP regions let dP(it+1) precede dS(it).
//
// Measured (bf16, d = 128; inputs not in L2): window 256, 4 x 4096 rows, 16 query
// heads on 2, 281 us (alone dK/dV 158, dQ 131, beside it and after; row statistic
// 23, sums 7); window 2048, 8205 rows, 16 heads on 4, 465 us.  A dK/dV step takes about 3400 cycles, of
// which its four products need 2048.  Masks found from the warp's bounds and one
// vote a step gained 2% over votes on the bits and at each wait.
//
// Roles, rings and the accumulators' hand-over are as in fa_bwd_sm100.cuh: 16
// compute warps (thread = TMEM lane = tile row, warpgroup g the columns 32 g ..
// 32 g + 31), a TMA warp with three slots for the A stream (Q; K) and two for
// the B stream (dO; V), one MMA thread; every wait is bounded.
#pragma once

#include "fa_bwd_sm100.cuh"
#include "fa_sinks_fwd_sm100.cuh"

namespace fa_sm100 {

struct SinksBwdParams {
  CUtensorMap tmap_q;  // 4-D (d, N, heads, B) views, box 64 elements x 128 rows
  CUtensorMap tmap_k;
  CUtensorMap tmap_v;
  CUtensorMap tmap_do;
  const void* o;       // [B, H, N, d]
  const void* dout;    // [B, H, N, d]
  const float* lse;    // [B, H, N]
  float* dsum;         // workspace [B, H, N]: D_i
  void* dq;            // [B, H, N, d]
  void* dk;            // [B, Hk, N, d]
  void* dv;
  int B, H, Hk, group, N;  // group = H / Hk
  // key j is visible from query i iff j <= i and (window < 0 or i - j <= window
  // or j < sinks)
  int window, sinks;
  float scale;
  float scale_log2;    // scale * log2(e)
  int nblk;            // 128-row blocks of a sequence
  int units;
  int out_vec32;       // dq, dk, dv 32-byte aligned
  int sink_blocks;     // key blocks holding sinks (0 when window < 0)
  int pieces, piece_blocks;  // of a sink block: pieces of that many query blocks
  int splits;          // of the steps of each dK/dV unit, when there are few units
  // pieces or splits > 1: fp32 [part, {dV, dK}, 128, d], parts numbered (B, Hk, sink
  // block, piece, split), then, with splits > 1, (B, Hk, other key block, split)
  float* parts;
  unsigned long long wait_limit_ns;
  FastDiv div_kv, div_q, div_hk, div_h, div_group, div_pieces, div_splits;
};

template <int HD, bool KV>
struct SinksBwdCfg {
  static_assert(HD == 64 || HD == 128, "backward head dim");
  static constexpr int CHUNKS = HD / 64;
  static constexpr int CHUNK_BYTES = 128 * 128;
  static constexpr int TILE_BYTES = CHUNKS * CHUNK_BYTES;  // one [128 x HD] 16-bit tile
  static constexpr int COMPUTE_WARPS = 16;
  static constexpr int THREADS = 32 * (COMPUTE_WARPS + 2);
  static constexpr int PRODUCER_WARP = COMPUTE_WARPS, MMA_WARP = COMPUTE_WARPS + 1;
  static constexpr int A_SLOTS = 3, B_SLOTS = 2;
  // Barriers.  S_READ (dQ), P_FULL (dK/dV) and DS_FULL take one arrival per
  // compute warp.  In the dK/dV kernel the next S follows every warp's P of
  // this step and the next dP every warp's dS, so no warp is ever a step ahead
  // of another at any of them.  In the dQ kernel the next S and dP only need
  // this S read, so the next dP can be complete before a warp has waited for
  // this one, and a warp's next dS written before another's: one step, never
  // two, hence a barrier for each step parity.
  static constexpr int B_RES_FULL = 0, B_A_FULL = 1 /* [A slot] */, B_A_EMPTY = 4,
                       B_B_FULL = 7 /* [B slot] */, B_B_EMPTY = 9, B_S_FULL = 11,
                       B_DP_FULL = 12 /* [2] */, B_DONE = 14, B_DRAIN = 15, B_RES_EMPTY = 16,
                       B_S_READ = 17, B_P_FULL = 18, B_DS_FULL = 19 /* [2] */, NUM_BARS = 21;
  static constexpr int SA_OFF = 0;                              // K (dK/dV) / Q (dQ)
  static constexpr int SB_OFF = TILE_BYTES;                     // V / dO
  static constexpr int RA_OFF = 2 * TILE_BYTES;                 // A ring: Q / K
  static constexpr int RB_OFF = RA_OFF + A_SLOTS * TILE_BYTES;  // B ring: dO / V
  static constexpr int BAR_OFF = RB_OFF + B_SLOTS * TILE_BYTES;
  static constexpr int MISC_OFF = BAR_OFF + (NUM_BARS + 1) / 2 * 16;
  // dK/dV: the statistics of a step's 128 columns, -(LSE log2 e)[32] and -D[32]
  // for each compute group, by step parity
  static constexpr int STAT_OFF = MISC_OFF + 16;
  static constexpr int END_OFF = STAT_OFF + (KV ? 2 * 4 * 64 * 4 : 0);
  // what is left up to the limit pads the base to 1024 bytes (checked)
  static constexpr int SLACK = 232448 - END_OFF < 1008 ? 232448 - END_OFF : 1008;
  static constexpr int SMEM_BYTES = END_OFF + SLACK;
  static_assert(SLACK >= 0, "shared memory budget");
  // TMEM columns: S (S^T), dP (dP^T), the accumulators, and for dQ a second dP.
  // Compute group g packs P^T over [32 g, 32 g + 16) of the S region and dS over
  // the same columns of the dP region, two values a column.
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_COL = 0, DP_COL = 128, ACC0_COL = 256, ACC1_COL = 256 + HD;
  static constexpr uint32_t DP2_COL = 256 + HD;
  static_assert(KV ? 256 + 2 * HD <= 512 : DP2_COL + 128 <= 512, "TMEM budget");
  // DP_FULL / DS_FULL barrier of step gs and the parity of its phase
  __device__ static constexpr int step_bar(int bar, int gs) { return KV ? bar : bar + (gs & 1); }
  __device__ static constexpr uint32_t step_parity(int gs) { return KV ? gs & 1 : (gs >> 1) & 1; }
  __host__ __device__ static constexpr uint32_t dp_col(int it) {
    return !KV && (it & 1) ? DP2_COL : DP_COL;
  }
  // offset of the packed operand of MMA K-step kk (16 columns of the tile)
  __host__ __device__ static constexpr uint32_t packed(int kk) {
    return 32u * static_cast<uint32_t>(kk / 2) + 8u * static_cast<uint32_t>(kk % 2);
  }
};

// One unit of work.
struct SinksUnit {
  int bh, blk, b, h;  // dK/dV: (b, key head h) and key block; dQ: (b, query head h), query block
  int first, per_head;  // dK/dV: query blocks first .. first + per_head - 1 of each head
  int ns, gap_end;    // dQ: key blocks 0 .. ns - 1, then gap_end on
  int count;          // streamed steps
  int start;          // dK/dV: the first of them among its query blocks of all heads
  int h0;             // first streamed head
  int part;           // dK/dV: this piece's partial sums, or -1
};

// Query blocks [first, end) that see key block blk; of a sink block, those of
// one piece.
__device__ __forceinline__ void key_block_queries(const SinksBwdParams& p, int blk, int piece,
                                                  int* first, int* end) {
  if (blk < p.sink_blocks) {
    *first = min(p.nblk, blk + piece * p.piece_blocks);
    *end = min(p.nblk, *first + p.piece_blocks);
  } else {
    // those with a row at most `window` past the block's last key
    *first = blk;
    *end = p.window < 0 ? p.nblk
                        : static_cast<int>(min(static_cast<long long>(p.nblk),
                                               (blk * 128ll + 127 + p.window) / 128 + 1));
  }
}

// First of the steps of split i (the steps dealt out as evenly as they go).
__device__ __forceinline__ int split_start(const SinksBwdParams& p, int steps, int i) {
  return p.div_splits.div(steps * i);
}

// Where the partial sums of (b, key head) bh's key block blk begin.
__device__ __forceinline__ int first_part(const SinksBwdParams& p, int bh, int blk) {
  if (blk < p.sink_blocks) return (bh * p.sink_blocks + blk) * p.pieces * p.splits;
  return (p.B * p.Hk * p.sink_blocks * p.pieces + bh * (p.nblk - p.sink_blocks) + blk -
          p.sink_blocks) * p.splits;
}

// Units with the most blocks first: the sink blocks' pieces, then the other key
// blocks from the front; for dQ the query blocks from the back.
template <bool KV>
__device__ __forceinline__ SinksUnit sinks_unit(const SinksBwdParams& p, int u) {
  SinksUnit w;
  const int nh = KV ? p.Hk : p.H, heads = p.B * nh;
  int rank = (KV ? p.div_kv : p.div_q).div(u);
  w.bh = u - rank * heads;
  w.b = (KV ? p.div_hk : p.div_h).div(w.bh);
  w.h = w.bh - w.b * nh;
  w.part = -1;
  w.start = 0;
  if (KV) {
    w.h0 = w.h * p.group;
    w.ns = w.gap_end = 0;
    const int sub = p.splits > 1 ? rank - p.div_splits.div(rank) * p.splits : 0;
    if (p.splits > 1) rank = p.div_splits.div(rank);
    const int sink_units = p.sink_blocks * p.pieces;
    w.blk = rank < sink_units ? p.div_pieces.div(rank) : p.sink_blocks + rank - sink_units;
    const int piece = rank < sink_units ? rank - w.blk * p.pieces : 0;
    int end;
    key_block_queries(p, w.blk, piece, &w.first, &end);
    w.per_head = end - w.first;
    w.count = w.per_head * p.group;
    if (p.splits > 1 || (rank < sink_units && p.pieces > 1))
      w.part = first_part(p, w.bh, w.blk) + piece * p.splits + sub;
    if (p.splits > 1) {
      w.start = split_start(p, w.count, sub);
      w.count = split_start(p, w.count, sub + 1) - w.start;
    }
  } else {
    w.blk = p.nblk - 1 - rank;
    w.h0 = p.div_group.div(w.h);
    const int lo = p.window < 0 ? 0 : max(0, w.blk * 128 - p.window) / 128;
    w.ns = min(p.sink_blocks, w.blk + 1);
    w.gap_end = max(w.ns, lo);
    w.first = w.per_head = 0;
    w.count = w.blk + 1 - (w.gap_end - w.ns);
  }
  return w;
}

// Head and block of a unit's streamed steps, from the first on.
template <bool KV>
struct SinksStep {
  int h, blk;
  __device__ __forceinline__ explicit SinksStep(const SinksUnit& w) {
    h = w.h0;
    blk = KV ? w.first : w.ns == 0 ? w.gap_end : 0;
    if (KV && w.start > 0) h += w.start / w.per_head, blk += w.start % w.per_head;
  }
  __device__ __forceinline__ void next(const SinksUnit& w) {
    ++blk;
    if (KV && blk == w.first + w.per_head) blk = w.first, ++h;
    if (!KV && blk == w.ns) blk = w.gap_end;
  }
};

// Writes NC fp32 columns of row r of dV (a0) and dK (a1) of one piece or split
// of a key block to its partial sums.
template <int NC>
__device__ __forceinline__ void store_part(float* parts, int part, int hd, int r, int c,
                                           const uint32_t* a0, const uint32_t* a1) {
  float* at = parts + (static_cast<long long>(part) * 2 * 128 + r) * hd + c;
#pragma unroll
  for (int i = 0; i < NC / 8; ++i) {
    st_global_v8(at + 8 * i, a0 + 8 * i);
    st_global_v8(at + 128ll * hd + 8 * i, a1 + 8 * i);
  }
}

template <int HD, bool BF16, bool KV>
__global__ void __launch_bounds__(SinksBwdCfg<HD, KV>::THREADS, 1)
    sinks_bwd_kernel(const __grid_constant__ SinksBwdParams p) {
  using C = SinksBwdCfg<HD, KV>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw > static_cast<uint32_t>(C::SLACK)) {
    // the aligned layout would not fit the allocation: refuse
    if (threadIdx.x == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleTest << 8) | kSiteAlign);
    return;
  }
  // the dQ kernel needs nothing of the dK/dV kernel and may start as this
  // grid's CTAs leave their SMs
  if constexpr (KV) asm volatile("griddepcontrol.launch_dependents;");
  uint8_t* smem = smem_raw + (base - raw);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  const uint32_t bars = base + C::BAR_OFF;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned long long lim = p.wait_limit_ns;
  const int G = gridDim.x, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NUM_BARS; ++i)
      mbar_init(bars + 8 * i, i >= C::B_S_READ ? C::COMPUTE_WARPS : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::PRODUCER_WARP && lane == 0) {
    tma_prefetch_desc(&p.tmap_q);
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
    tma_prefetch_desc(&p.tmap_do);
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp == C::PRODUCER_WARP) {
    if (lane == 0) {
      bool ok = true;
      int g = 0, k = 0;                // streamed steps and units so far
      int issued_a = 0, issued_b = 0;  // ring loads issued (= g after each unit)
      for (int round = 0; ok && round * G < p.units; ++round) {
        const int u = bwd_unit_of(round, cta, G);
        if (u >= p.units) continue;
        const SinksUnit w = sinks_unit<KV>(p, u);
        if (w.count <= 0) continue;  // a piece past the sequence's end
        // resident pair: K_j, V_j (dK/dV) or Q_i, dO_i (dQ), once the previous
        // unit's S and dP products have ended
        if (k > 0 && !(ok = wait_phase(bars + 8 * C::B_RES_EMPTY, (k - 1) & 1, abort_flag, lim,
                                       (kRoleProducer << 8) | kSiteQEmpty)))
          break;
        mbar_arrive_expect_tx(bars + 8 * C::B_RES_FULL, 2 * C::TILE_BYTES);
        load_tile<HD>(base + C::SA_OFF, KV ? &p.tmap_k : &p.tmap_q, bars + 8 * C::B_RES_FULL,
                      w.blk * 128, w.h, w.b);
        load_tile<HD>(base + C::SB_OFF, KV ? &p.tmap_v : &p.tmap_do, bars + 8 * C::B_RES_FULL,
                      w.blk * 128, w.h, w.b);
        ++k;
        SinksStep<KV> st(w);
        for (int it = 0; ok && it < w.count; ++it, st.next(w)) {
          const int gs = g + it;
#pragma unroll 1
          for (int ring = 0; ring < 2; ++ring) {
            const int slots = ring ? C::B_SLOTS : C::A_SLOTS;
            const int slot = gs % slots, use = gs / slots;
            const int b_empty = ring ? C::B_B_EMPTY : C::B_A_EMPTY;
            if (use > 0 && !(ok = wait_phase(bars + 8 * (b_empty + slot), (use - 1) & 1, abort_flag,
                                             lim, (kRoleProducer << 8) | kSiteKvEmpty)))
              break;
            const uint32_t full = bars + 8 * ((ring ? C::B_B_FULL : C::B_A_FULL) + slot);
            mbar_arrive_expect_tx(full, C::TILE_BYTES);
            load_tile<HD>(base + (ring ? C::RB_OFF : C::RA_OFF) + slot * C::TILE_BYTES,
                          ring ? (KV ? &p.tmap_do : &p.tmap_v) : (KV ? &p.tmap_q : &p.tmap_k),
                          full, st.blk * 128, st.h, w.b);
            ++(ring ? issued_b : issued_a);
          }
        }
        g += w.count;
      }
      if (!ok) {
        // let the loads in flight land before the shared memory goes away
        volatile int no_abort = 0;
        if (k > 0)
          wait_phase(bars + 8 * C::B_RES_FULL, (k - 1) & 1, &no_abort, 10000000ull,
                     (kRoleProducer << 8) | kSiteDrain);
        for (int i = issued_a > C::A_SLOTS ? issued_a - C::A_SLOTS : 0; i < issued_a; ++i)
          wait_phase(bars + 8 * (C::B_A_FULL + i % C::A_SLOTS), (i / C::A_SLOTS) & 1, &no_abort,
                     10000000ull, (kRoleProducer << 8) | kSiteDrain);
        for (int i = issued_b > C::B_SLOTS ? issued_b - C::B_SLOTS : 0; i < issued_b; ++i)
          wait_phase(bars + 8 * (C::B_B_FULL + i % C::B_SLOTS), (i / C::B_SLOTS) & 1, &no_abort,
                     10000000ull, (kRoleProducer << 8) | kSiteDrain);
      }
    }
  } else if (warp == C::MMA_WARP) {
    if (lane == 0) {
      const uint32_t idesc_sq = f16_idesc(BF16, 128, 128, false);
      const uint32_t idesc_acc = f16_idesc(BF16, 128, HD, true);
      bool ok = true;
      const uint32_t a0 = sw128_desc_lo(base + C::SA_OFF, 16), a1 = sw128_desc_lo(base + C::SB_OFF, 16);
      auto ra = [&](int gs) { return base + C::RA_OFF + (gs % C::A_SLOTS) * C::TILE_BYTES; };
      auto rb = [&](int gs) { return base + C::RB_OFF + (gs % C::B_SLOTS) * C::TILE_BYTES; };
      auto wait_ring = [&](int gs, int ring) -> bool {
        const int slots = ring ? C::B_SLOTS : C::A_SLOTS;
        const bool r = wait_phase(bars + 8 * ((ring ? C::B_B_FULL : C::B_A_FULL) + gs % slots),
                                  (gs / slots) & 1, abort_flag, lim, (kRoleMma << 8) | kSiteKvFull);
        tc_fence_after_sync();
        return r;
      };
      auto wait_warps = [&](int bar, uint32_t parity, unsigned site) -> bool {
        const bool r = wait_phase(bars + 8 * bar, parity, abort_flag, lim, (kRoleMma << 8) | site);
        tc_fence_after_sync();
        return r;
      };
      auto issue_sq = [&](uint32_t d_col, uint32_t a, uint32_t bt) {
        const uint32_t bd = sw128_desc_lo(bt, 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = ((kk / 4) * C::CHUNK_BYTES + (kk % 4) * 32) >> 4;
          mma_ss(tmem + d_col, desc_from_lo(a + off), desc_from_lo(bd + off), idesc_sq,
                 kk > 0 ? 1u : 0u);
        }
      };
      auto issue_s = [&](int gs) {
        issue_sq(C::S_COL, a0, ra(gs));
        tc_commit(bars + 8 * C::B_S_FULL);
      };
      // dP of step gs; in the dQ kernel the B-ring tile (V) has no other use
      auto issue_dp = [&](int gs) {
        issue_sq(C::dp_col(gs), a1, rb(gs));
        tc_commit(bars + 8 * C::step_bar(C::B_DP_FULL, gs));
        if (!KV) tc_commit(bars + 8 * (C::B_B_EMPTY + gs % C::B_SLOTS));
      };
      int g = 0, k = 0;  // streamed steps and units so far
      for (int round = 0; ok && round * G < p.units; ++round) {
        const int u = bwd_unit_of(round, cta, G);
        if (u >= p.units) continue;
        const int count = sinks_unit<KV>(p, u).count;
        if (count <= 0) continue;
        // The unit's resident pair.  (Every warp has read the previous unit's
        // last S and dP: its last accumulating product waited for their dS.
        // The accumulators are read out by each warp's epilogue before that
        // warp's P / dS of this unit's first step.)
        if (!(ok = wait_phase(bars + 8 * C::B_RES_FULL, k & 1, abort_flag, lim,
                              (kRoleMma << 8) | kSiteQFull)))
          break;
        tc_fence_after_sync();
        ++k;
        if (!(ok = wait_ring(g, 0))) break;
        issue_s(g);
        if (!(ok = wait_ring(g, 1))) break;
        issue_dp(g);
        if (count == 1) tc_commit(bars + 8 * C::B_RES_EMPTY);
        for (int it = 0; ok && it < count; ++it) {
          const int gs = g + it;
          const uint32_t mq = sw128_desc_lo(ra(gs), C::CHUNK_BYTES);
          const uint32_t md = sw128_desc_lo(rb(gs), C::CHUNK_BYTES);
          const bool more = it + 1 < count;
          if (KV) {
            // dV += P^T dO; then dO's slot and the S columns are free
            if (!(ok = wait_warps(C::B_P_FULL, gs & 1, kSitePFull))) break;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + C::ACC0_COL, tmem + C::S_COL + C::packed(kk),
                     desc_from_lo(md + ((kk * 16 * 128) >> 4)), idesc_acc, (it > 0 || kk > 0) ? 1u : 0u);
            tc_commit(bars + 8 * (C::B_B_EMPTY + gs % C::B_SLOTS));
          } else if (more) {
            if (!(ok = wait_warps(C::B_S_READ, gs & 1, kSiteSFree))) break;
          }
          if (more) {
            if (!(ok = wait_ring(gs + 1, 0))) break;
            issue_s(gs + 1);
            if (!KV) {
              // (the region's last dS was read by a product issued before)
              if (!(ok = wait_ring(gs + 1, 1))) break;
              issue_dp(gs + 1);
              if (it + 2 == count) tc_commit(bars + 8 * C::B_RES_EMPTY);
            }
          }
          // dK += dS^T Q or dQ += dS K; then the A slot and the dP columns are free
          if (!(ok = wait_warps(C::step_bar(C::B_DS_FULL, gs), C::step_parity(gs), kSitePFull))) break;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + (KV ? C::ACC1_COL : C::ACC0_COL), tmem + C::dp_col(gs) + C::packed(kk),
                   desc_from_lo(mq + ((kk * 16 * 128) >> 4)), idesc_acc, (it > 0 || kk > 0) ? 1u : 0u);
          tc_commit(bars + 8 * (C::B_A_EMPTY + gs % C::A_SLOTS));
          if (KV && more) {
            if (!(ok = wait_ring(gs + 1, 1))) break;
            issue_dp(gs + 1);
            if (it + 2 == count) tc_commit(bars + 8 * C::B_RES_EMPTY);
          }
        }
        if (!ok) break;
        // the unit's accumulators are complete once these products end
        tc_commit(bars + 8 * C::B_DONE);
        g += count;
      }
      if (!ok) {
        // wait for every MMA this thread issued before TMEM is released
        volatile int no_abort = 0;
        tc_commit(bars + 8 * C::B_DRAIN);
        wait_phase(bars + 8 * C::B_DRAIN, 0, &no_abort, 10000000ull, (kRoleMma << 8) | kSiteDrain);
      }
    }
  } else {
    // compute warps: thread = tile row = TMEM lane; this warpgroup's columns
    const int uw = __shfl_sync(0xffffffffu, warp, 0);  // (uniform for the compiler too)
    const int quad = uw % 4, grp = uw / 4, cb = 32 * grp;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + ((static_cast<uint32_t>(quad) * 32u) << 16);
    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
    constexpr float kLog2e = 1.4426950408889634f;
    bool ok = true;
    int g = 0, k = 0;  // streamed steps and units so far
    for (int round = 0; ok && round * G < p.units; ++round) {
      const int u = bwd_unit_of(round, cta, G);
      if (u >= p.units) continue;
      const SinksUnit w = sinks_unit<KV>(p, u);
      if (w.count <= 0) continue;
      const int row0 = w.blk * 128 + 32 * quad;
      const int my_row = row0 + lane;  // key row (dK/dV) or query row (dQ)
      // Statistics are kept as loaded: scaling them here would wait for the load.
      float my_lse = INFINITY, my_d = 0.f;  // dQ: LSE and D of the row
      if (!KV && my_row < p.N) {
        const long long at = static_cast<long long>(w.bh) * p.N + my_row;
        my_lse = __ldg(p.lse + at);
        my_d = p.dsum[at];
      }
      SinksStep<KV> st(w);
      // dK/dV: the statistics of the streamed query block's columns, lane l
      // holding column cb + l (+inf: a row past N, weight 0)
      float col_lse = INFINITY, col_d = 0.f;
      auto load_stats = [&]() {
        const int qi = st.blk * 128 + cb + lane;
        col_lse = INFINITY, col_d = 0.f;
        if (qi < p.N) {
          const long long at = (static_cast<long long>(w.b) * p.H + st.h) * p.N + qi;
          col_lse = __ldg(p.lse + at);
          col_d = p.dsum[at];
        }
      };
      if (KV) load_stats();
      for (int it = 0; it < w.count; ++it) {
        const int gs = g + it;
        // This row's visible columns among the group's 32, as bits.  dK/dV:
        // queries from the key's own position to the window's end (a sink
        // key's: to the end); dQ: the window's keys and the sinks.  Most warps
        // see all of their columns or none, so the bits are only applied where
        // they differ, and not even looked for in a block that is wholly visible
        // (below the diagonal, inside the window).
        const int q_lo = KV ? st.blk * 128 + cb : row0, k_lo = KV ? row0 : st.blk * 128 + cb;
        const bool all = k_lo + 31 <= q_lo &&
                         (p.window < 0 || q_lo + 31 - k_lo <= p.window || k_lo + 32 <= p.sinks);
        const bool none = k_lo > q_lo + 31 ||
                          (p.window >= 0 && q_lo - k_lo - 31 > p.window && k_lo >= p.sinks);
        ok = wait_phase(bars + 8 * C::B_S_FULL, gs & 1, abort_flag, lim,
                        (kRoleSoftmax << 8) | kSiteSFull);
        __syncwarp();  // (a wait given up is acted on below, with the next one's)
        tc_fence_after_sync();
        // P, kept in fp32
        float2 pv[16];
        uint32_t sv[32];
        tmem_ld32_sync(lane_base + C::S_COL + cb, sv);
        if (!KV) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + 8 * C::B_S_READ);
        }
        // the columns' statistics to shared memory (the group's four warps write
        // the same values), read back four columns at a time.  Step gs + 2
        // reuses the buffer: its S follows every warp's P of step gs + 1.
        const float4* stat = nullptr;
        if constexpr (KV) {
          float* to = reinterpret_cast<float*>(smem + C::STAT_OFF) + ((gs & 1) * 4 + grp) * 64;
          to[lane] = -col_lse * kLog2e;
          to[32 + lane] = -col_d;
          stat = reinterpret_cast<const float4*>(to);
          __syncwarp();
        }
        const float my_nlse2 = -my_lse * kLog2e;
        if (none) {
#pragma unroll
          for (int q = 0; q < 16; ++q) pv[q] = make_float2(0.f, 0.f);
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float2 nl = make_float2(my_nlse2, my_nlse2);
            if constexpr (KV) {
              const float4 l4 = stat[q / 2];
              nl = q % 2 ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
            }
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1])), sl2, nl);
            pv[q] = make_float2(ex2(x.x), ex2(x.y));
          }
          if (!all) {
            const int rel = my_row - st.blk * 128 - cb;
            uint32_t bits;
            if (KV) {
              bits = ~low_bits(rel);
              if (p.window >= 0 && my_row >= p.sinks) bits &= low_bits(rel + p.window + 1);
            } else {
              bits = low_bits(rel + 1);
              if (p.window >= 0)
                bits &= ~low_bits(rel - p.window) | low_bits(p.sinks - st.blk * 128 - cb);
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              pv[q].x = (bits >> (2 * q)) & 1u ? pv[q].x : 0.f;
              pv[q].y = (bits >> (2 * q + 1)) & 1u ? pv[q].y : 0.f;
            }
          }
        }
        uint32_t pk[16];
        if constexpr (KV) {
#pragma unroll
          for (int q = 0; q < 16; ++q) pk[q] = pack2<BF16>(pv[q].x, pv[q].y);
          // P^T over the first 16 of the group's S^T columns (read above)
          tmem_st16(lane_base + C::S_COL + cb, pk);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + 8 * C::B_P_FULL);
        }
        // the next step's statistics, on their way during this step's rest
        st.next(w);
        if (KV && it + 1 < w.count) load_stats();
        // dS = P (dP - D)
        ok &= wait_phase(bars + 8 * C::step_bar(C::B_DP_FULL, gs), C::step_parity(gs), abort_flag,
                         lim, (kRoleSoftmax << 8) | kSiteSFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t dpc = C::dp_col(gs);
        tmem_ld32_sync(lane_base + dpc + cb, sv);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float2 nd = make_float2(-my_d, -my_d);
          if constexpr (KV) {
            const float4 d4 = stat[8 + q / 2];
            nd = q % 2 ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
          }
          const float2 ds = __fmul2_rn(
              pv[q],
              __fadd2_rn(make_float2(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1])), nd));
          pk[q] = pack2<BF16>(ds.x, ds.y);
        }
        // over the first 16 of the group's dP columns (read above)
        tmem_st16(lane_base + dpc + cb, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * C::step_bar(C::B_DS_FULL, gs));
      }
      if (ok) {
        ok = wait_phase(bars + 8 * C::B_DONE, k & 1, abort_flag, lim, (kRoleSoftmax << 8) | kSiteODone);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc_fence_after_sync();
          using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
          const long long row_off = (static_cast<long long>(w.bh) * p.N + my_row) * HD;
          // this group's quarter of the accumulator columns
          constexpr int EC = HD / 4;
          const bool vec32 = p.out_vec32 != 0;
          const int c = grp * EC;
          uint32_t a0[EC], a1[EC];
          if constexpr (EC == 32) {
            tmem_ld32_sync(lane_base + C::ACC0_COL + c, a0);
            if (KV) tmem_ld32_sync(lane_base + C::ACC1_COL + c, a1);
          } else {
            tmem_ld16_sync(lane_base + C::ACC0_COL + c, a0);
            if (KV) tmem_ld16_sync(lane_base + C::ACC1_COL + c, a1);
          }
          if (KV && w.part >= 0) {
            store_part<EC>(p.parts, w.part, HD, r, c, a0, a1);
          } else if (my_row < p.N) {
            if (KV) {
              store_acc<BF16, EC>(static_cast<T*>(p.dv) + row_off + c, a0, 1.f, vec32);
              store_acc<BF16, EC>(static_cast<T*>(p.dk) + row_off + c, a1, p.scale, vec32);
            } else {
              store_acc<BF16, EC>(static_cast<T*>(p.dq) + row_off + c, a0, p.scale, vec32);
            }
          }
          tc_fence_before_sync();
        }
      }
      g += w.count;
      ++k;
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // the dQ grid ends only once the dK/dV grid, beside which it may have run,
  // has; the last CTA sees to it
  if constexpr (!KV) {
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// dV and dK of the key blocks that were dealt out (the sink blocks', or all with
// splits > 1): the partial sums added in order, dK times the scale, rounded
// once.  A thread takes 4 columns of one row.
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) sinks_sum_kernel(const __grid_constant__ SinksBwdParams p) {
  constexpr int C4 = HD / 4;
  const int blocks = p.splits > 1 ? p.nblk : p.sink_blocks;  // of a head
  const long long n = static_cast<long long>(p.B) * p.Hk * blocks * 2 * 128 * C4;
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const int c = static_cast<int>(i % C4) * 4;
  const int r = static_cast<int>(i / C4 % 128);
  const int which = static_cast<int>(i / (C4 * 128) % 2);  // 0: dV, 1: dK
  const int block = static_cast<int>(i / (C4 * 128 * 2));
  const int bh = block / blocks, blk = block - bh * blocks;
  const int row = blk * 128 + r;
  if (row >= p.N) return;
  const int pieces = blk < p.sink_blocks ? p.pieces : 1;
  const float* at = p.parts + ((first_part(p, bh, blk) * 2ll + which) * 128 + r) * HD + c;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int piece = 0; piece < pieces; ++piece) {
    int first, end;
    key_block_queries(p, blk, piece, &first, &end);
    const int steps = (end - first) * p.group;
#pragma unroll 4
    for (int sub = 0; sub < p.splits; ++sub, at += 2 * 128 * HD) {
      // (a piece past the sequence's end or a split without a step has no sums)
      if (p.splits == 1 ? steps <= 0 : split_start(p, steps, sub) == split_start(p, steps, sub + 1))
        continue;
      const float4 v = __ldg(reinterpret_cast<const float4*>(at));
      t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    }
  }
  const float mul = which ? p.scale : 1.f;
  uint2 w = make_uint2(pack2<BF16>(t.x * mul, t.y * mul), pack2<BF16>(t.z * mul, t.w * mul));
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  T* out = static_cast<T*>(which ? p.dk : p.dv);
  *reinterpret_cast<uint2*>(out + (static_cast<long long>(bh) * p.N + row) * HD + c) = w;
}

}  // namespace fa_sm100
