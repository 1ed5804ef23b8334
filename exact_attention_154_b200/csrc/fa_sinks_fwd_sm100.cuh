// fa_sinks_fwd_sm100.cuh -- causal attention with a sliding window and sinks
// (key / value heads shared by groups of query heads), for sm_100a.
//
//   O_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  s_ij = scale q_i . k_j,  over the
//   keys j <= i with i - j <= window or j < sinks; LSE_i = ln sum_j exp(s_ij)
//
// by the online recurrence of fa_fwd_sm100.cuh (running reference, lazily moved;
// row sum and O in fp32).  The weights are rounded to 16 bits before P V, since one
// matrix instruction takes P and V in one type; the row sum adds them unrounded.
//
// What bounds it under a window: latency.  A 128-row query tile meets only
// window / 64 + 3 blocks of 64 keys, so the chain of a block (scores,
// exponentials, weights back to TMEM) and what a tile starts and ends with
// are not hidden behind other blocks of the same tile.  So tiles are kept
// small and independent, and two CTAs share an SM (d <= 128): one computes
// while the other starts, ends or waits.  One warpgroup owns a tile's rows
// whole (thread = row = TMEM lane, 64 columns a block), so row maxima and sums
// need no exchange.  P is packed over the scores it came from, in TMEM: the
// shared-memory port, which feeds the products and takes the loads, would have
// 32 of its 128 KB a block more to move with P there (window 256 83 -> 77 us, 4096
// 560 -> 518, short 10.2 -> 8.6).  S has two buffers, so the next block's scores
// are there when its turn comes: S(j+1) only waits for P(j-1) V.
//
//   warps 0-3  softmax: S from TMEM, mask, exponentials, P back over S, O
//              rescaled in TMEM when the reference moves, O / l written out
//   warp 4     TMA: Q once a tile, K and V blocks through a ring
//   warp 5, 6  one thread each issues S = Q K^T and O += P V (a thread that
//              issues MMAs runs only about one instruction ahead of the pipe)
//
// Blocks outside every row's view are neither loaded nor multiplied: a tile's
// blocks are those holding sinks, then the window's.  Every wait is bounded.
//
// Measured (bf16, d = 128, 16 query heads on 2; inputs not in L2): window 256, 4 x
// 4096 rows, 77 us; window 4096, 16384 rows, 525 us (917 TFLOP/s of visible pairs);
// 2 x 12 heads of 333 rows at d = 64, 8.3 us.  The plain forward's shape given the
// same masks (128-key blocks, two tiles and four softmax warpgroups a CTA, one CTA
// an SM, P in shared memory) took 111, 519 and 12.2 us.  By clocks read in a copy, window
// 256 takes 15,900 cycles a tile of 6.7 blocks: a block 1140 of work on its scores, 400
// of bounds and loop before them, 200 of waiting; the tile's first scores 1040, its last
// P V 1530, its output 1800.  Under the wide window the
// two CTAs of an SM take 1880 cycles a block each; the tensor pipe is busy 72% of
// them (54% of its rate: a product with 64 keys on its wide side reads its 128
// query rows for half as many columns), the exponential unit 53%.  A part of the
// exponentials as a polynomial on the FMA pipe, and P handed over in halves, were no
// faster under window 256 and 3% slower under the wide one.
#pragma once

#include "fa_fwd_sm100.cuh"

namespace fa_sm100 {

// Division of a 31-bit number by a constant of the launch as a multiplication
// (the round-up method of Granlund and Montgomery).
struct FastDiv {
  uint32_t mul, shift;
  __host__ static FastDiv make(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint64_t m = ((1ull << 32) * ((1ull << l) - d)) / d + 1;
    return {static_cast<uint32_t>(m), l};
  }
  __device__ __forceinline__ int div(int n) const {
    const uint32_t u = static_cast<uint32_t>(n), t = __umulhi(mul, u);
    return static_cast<int>((t + ((u - t) >> (shift > 0))) >> (shift > 0 ? shift - 1 : 0));
  }
};

// The low n of 32 bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

__device__ __forceinline__ float row_max32(const float* sv) {
  float t[11];
#pragma unroll
  for (int i = 0; i < 10; ++i) t[i] = max3(sv[3 * i], sv[3 * i + 1], sv[3 * i + 2]);
  t[10] = fmaxf(sv[30], sv[31]);
  return max3(max3(t[0], t[1], t[2]), max3(t[3], t[4], t[5]),
              max3(max3(t[6], t[7], t[8]), t[9], t[10]));
}

struct SinksFwdParams {
  CUtensorMap tmap_q;  // 4-D (d, N, heads, B) views, box 64 elements x 128 rows
  CUtensorMap tmap_k;  // box 64 elements x 64 rows
  CUtensorMap tmap_v;
  CUtensorMap tmap_o;  // [B, H, N, d], box 64 elements x 32 rows
  float* lse;          // [B, H, N] or nullptr
  int B, H, N, window, sinks;
  float scale_log2;    // scale * log2(e)
  int sink_blocks;     // 64-key blocks holding sinks (0 when window < 0)
  int qblocks, tiles;  // query tiles of a head, and in all
  FastDiv div_bh, div_h, div_group;  // by B * H, H, H / Hk
  unsigned long long wait_limit_ns;
};

template <int HD>
struct SinksFwdCfg {
  static_assert(HD == 64 || HD == 128 || HD == 256, "head dim");
  static constexpr int KEYS = 64;                    // keys of a block
  static constexpr int CHUNKS = HD / 64;             // 128-byte columns of a row
  static constexpr int Q_CHUNK = 128 * 128, KV_CHUNK = KEYS * 128;
  static constexpr int Q_BYTES = CHUNKS * Q_CHUNK, KV_BYTES = CHUNKS * KV_CHUNK;
  static constexpr int O_BYTES = 128 * 64 * 2;       // 64 columns of O on their way out
  static constexpr int RING = HD == 64 ? 8 : 4;      // K or V blocks
  static constexpr int CTAS = HD == 256 ? 1 : 2;     // of an SM
  static constexpr int WARPS = 7, THREADS = 32 * WARPS;
  static constexpr int PRODUCER_WARP = 4, S_WARP = 5, PV_WARP = 6;
  static constexpr int Q_OFF = 0, O_OFF = Q_BYTES, RING_OFF = O_OFF + O_BYTES;
  static constexpr int BAR_OFF = RING_OFF + RING * KV_BYTES;
  // A ring slot holds K or V blocks in turn, each completing on a barrier of
  // its own consumer, so that every barrier's phases are waited in order.
  static constexpr int B_Q_FULL = 0, B_Q_EMPTY = 1, B_K_FULL = 2, B_V_FULL = B_K_FULL + RING,
                       B_EMPTY = B_V_FULL + RING, B_S_FULL = B_EMPTY + RING /* [2] */,
                       B_P_FULL = B_S_FULL + 2 /* [2] */, B_S_FREE = B_P_FULL + 2 /* [2] */,
                       B_O_FINAL = B_S_FREE + 2, B_DRAIN = B_O_FINAL + 1, NUM_BARS = B_DRAIN + 2;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
  static constexpr int END_OFF = MISC_OFF + 16;
  // shared memory of a CTA (228 KB an SM, 1 KB of each CTA's reserved); what is
  // left pads the base to 1024 bytes (checked)
  static constexpr int LIMIT = CTAS == 2 ? 233472 / 2 - 1024 : 232448;
  static constexpr int SLACK = LIMIT - END_OFF < 1008 ? LIMIT - END_OFF : 1008;
  static constexpr int SMEM_BYTES = END_OFF + SLACK;
  static_assert(SLACK >= 0, "shared memory budget");
  // TMEM columns: two S buffers (P over the first half of its S), O
  static constexpr uint32_t O_COL = 2 * KEYS;
  static constexpr uint32_t TMEM_COLS = HD == 256 ? 512 : 256;
  static_assert(O_COL + HD <= TMEM_COLS, "TMEM budget");
};

// One work tile: 128 query rows of one head, from row q0; its n key blocks are
// 0 .. ns - 1 (those below it), then gap_end on.
struct SinksTile {
  int b, h, hk, q0, n, ns, gap_end;
};

// Longest first over the whole grid: all heads' last query block, then the one
// before, ...
__device__ __forceinline__ SinksTile sinks_tile(const SinksFwdParams& p, int t) {
  SinksTile w;
  const int rank = p.div_bh.div(t);
  const int bh = t - rank * p.B * p.H;
  w.b = p.div_h.div(bh);
  w.h = bh - w.b * p.H;
  w.hk = p.div_group.div(w.h);
  w.q0 = (p.qblocks - 1 - rank) * 128;
  const int hi = min(w.q0 + 127, p.N - 1) / 64 + 1;
  const int lo = p.window < 0 ? 0 : max(0, w.q0 - p.window) / 64;
  w.ns = p.sink_blocks;
  w.gap_end = max(w.ns, lo);
  w.n = hi - (w.gap_end - w.ns);
  return w;
}
__device__ __forceinline__ int sinks_block(const SinksTile& w, int jj) {
  return jj < w.ns ? jj : jj - w.ns + w.gap_end;
}

template <int HD, bool BF16>
__device__ void sinks_softmax(const SinksFwdParams& p, uint32_t base, uint32_t tmem,
                              volatile int* abort_flag) {
  using C = SinksFwdCfg<HD>;
  const uint32_t bars = base + C::BAR_OFF;
  const int lane = threadIdx.x % 32;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);  // (uniform for the compiler too)
  const int r = warp * 32 + lane;  // query row within the tile == TMEM lane
  const uint32_t lane_base = tmem + ((static_cast<uint32_t>(warp) * 32u) << 16);
  const unsigned long long lim = p.wait_limit_ns;
  const float sl2 = p.scale_log2;
  const int G = gridDim.x, cta = blockIdx.x;
  int blocks = 0;  // blocks so far, over all tiles: S buffer, phases
  uint32_t fin_par = 0u;
  for (int round = 0; round * G < p.tiles; ++round) {
    const int t = tile_of(round, cta, G);
    if (t >= p.tiles) continue;
    const SinksTile w = sinks_tile(p, t);
    const int row0 = w.q0 + 32 * warp, row = row0 + lane;
    float m_ref = -INFINITY, l = 0.f;
    for (int jj = 0; jj < w.n; ++jj, ++blocks) {
      const int k0 = sinks_block(w, jj) * C::KEYS;
      // Which keys the warp's 32 rows see, of each half of the block: bounds that
      // are the same for the whole warp (keys past the sequence's end lie past
      // every row's own position).  Only a half that some row sees in part is
      // masked, by bits; one that no row sees is not looked at (by halves rather
      // than whole blocks: window 256 2.5% faster).
      bool all[2], none[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ka = k0 + 32 * c;
        all[c] = ka + 31 <= row0 &&
                 (p.window < 0 || ka >= row0 + 31 - p.window || ka + 32 <= p.sinks);
        none[c] = ka > row0 + 31 || (p.window >= 0 && ka + 31 < row0 - p.window && ka >= p.sinks);
      }
      const int buf = blocks & 1;
      bool ok = wait_phase(bars + 8 * (C::B_S_FULL + buf), (blocks >> 1) & 1, abort_flag, lim,
                           (kRoleSoftmax << 8) | kSiteSFull);
      __syncwarp();  // (a wait given up is acted on below, with the next one's)
      tc_fence_after_sync();
      uint32_t sr[64];
      tmem_ld64_nowait(lane_base + C::KEYS * buf, sr);
      tmem_ld64_wait(sr);
      float sv[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) sv[c] = __uint_as_float(sr[c]);
      float m_blk = -INFINITY;
      if (all[0] && all[1]) {
        m_blk = row_max64(sv);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (none[c]) continue;
          if (!all[c]) {
            const int rel = row - k0 - 32 * c;
            uint32_t bits = low_bits(rel + 1);
            if (p.window >= 0) bits &= ~low_bits(rel - p.window) | low_bits(p.sinks - k0 - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sv[32 * c + i] = (bits >> i) & 1u ? sv[32 * c + i] : -INFINITY;
          }
          m_blk = fmaxf(m_blk, row_max32(sv + 32 * c));
        }
      }
      m_blk *= sl2;
      // Lazy reference, as in the plain forward: moved only when the block's
      // maximum exceeds it by more than 2^8, and by the first block.  A row
      // that has seen no key yet has m_ref = -inf, l = 0 and O = 0.
      const bool rescale = jj > 0 && m_blk > m_ref + kLazyRescaleLog2;
      const float m_new = jj == 0 || rescale ? m_blk : m_ref;
      const float alpha = jj == 0 || m_ref == -INFINITY ? 0.f : ex2(m_ref - m_new);
      m_ref = m_new;
      const float neg_ref = m_ref == -INFINITY ? 0.f : -m_ref;
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                       make_float2(0.f, 0.f)};
      uint32_t pk[32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (none[c]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[16 * c + i] = 0u;
        } else {
          softmax_chunk<BF16 ? kBF16 : kF16, 0>(sv + 32 * c, sl2, neg_ref, pk + 16 * c, acc);
        }
      }
      const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
      l = l * alpha + ((a01.x + a23.x) + (a01.y + a23.y));
      // O is only touched where the reference moved, once the last P V has run
      // (which hands back the other buffer)
      const bool move = __any_sync(0xffffffffu, rescale);
      if (move)
        ok &= wait_phase(bars + 8 * (C::B_S_FREE + (buf ^ 1)), ((blocks - 1) >> 1) & 1, abort_flag,
                         lim, (kRoleSoftmax << 8) | kSitePFree);
      if (!__all_sync(0xffffffffu, ok)) return;
      if (move) {
        tc_fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          uint32_t ov[16];
          tmem_ld16_sync(lane_base + C::O_COL + c, ov);
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st16(lane_base + C::O_COL + c, ov);
        }
      }
      // P, two keys a column, over the scores just read
      tmem_st32(lane_base + C::KEYS * buf, pk);
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (C::B_P_FULL + buf));
    }

    // O / l and the logsumexp, once the tile's last P V has run.  The next
    // tile's first P V overwrites O only after this warp's next P arrival.
    const bool ok = wait_phase(bars + 8 * C::B_O_FINAL, fin_par, abort_flag, lim,
                               (kRoleSoftmax << 8) | kSiteODone);
    fin_par ^= 1u;
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after_sync();
    const float inv_l = 1.f / l;
    if (p.lse != nullptr && row < p.N)
      p.lse[(static_cast<long long>(w.b) * p.H + w.h) * p.N + row] =
          (m_ref + log2f(l)) * 0.69314718055994530942f;
    // 64 columns at a time through the warp's own rows of the staging buffer, in
    // the tensor map's layout; rows past the sequence's end are not written
#pragma unroll 1
    for (int c = 0; c < HD; c += 64) {
      uint32_t ov[64];
      tmem_ld64_nowait(lane_base + C::O_COL + c, ov);
      tmem_ld64_wait(ov);
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        pk[i] = pack2<BF16>(__uint_as_float(ov[2 * i]) * inv_l, __uint_as_float(ov[2 * i + 1]) * inv_l);
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
      store_p_chunk(base + C::O_OFF, r, pk);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && row0 < p.N) {
        tma_store_4d(&p.tmap_o, base + C::O_OFF + warp * 4096, c, row0, w.h, w.b);
        bulk_commit_group();
      }
    }
    tc_fence_before_sync();
  }
}

template <int HD, bool BF16>
__global__ void __launch_bounds__(SinksFwdCfg<HD>::THREADS, SinksFwdCfg<HD>::CTAS)
    sinks_fwd_kernel(const __grid_constant__ SinksFwdParams p) {
  using C = SinksFwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  if (base - raw > static_cast<uint32_t>(C::SLACK)) {
    // the aligned layout would not fit the allocation: refuse
    if (threadIdx.x == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleTest << 8) | kSiteAlign);
    return;
  }
  uint8_t* smem = smem_raw + (base - raw);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  const uint32_t bars = base + C::BAR_OFF;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const unsigned long long lim = p.wait_limit_ns;
  const int G = gridDim.x, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NUM_BARS; ++i)
      mbar_init(bars + 8 * i, (i >= C::B_P_FULL && i < C::B_S_FREE) ? 4 : 1);  // a softmax warp each
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::PRODUCER_WARP && lane == 0) {
    tma_prefetch_desc(&p.tmap_q);
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
    tma_prefetch_desc(&p.tmap_o);
  }
  if (warp == C::S_WARP) {
    tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp < 4) {
    sinks_softmax<HD, BF16>(p, base, tmem, abort_flag);
    // the stores of O have read shared memory, and are complete
    if (lane == 0) bulk_wait_all();
  } else if (warp == C::PRODUCER_WARP && lane == 0) {
    int used = 0, q_count = 0;
    bool ok = true;
    // the last load into each slot (its barrier and phase), for the drain
    uint32_t k_par = 0u, v_par = 0u;  // bit i: parity of slot i's next K / V load
    uint32_t last_bar[C::RING], last_par[C::RING];
#pragma unroll
    for (int i = 0; i < C::RING; ++i) last_bar[i] = last_par[i] = 0u;
    auto load = [&](const CUtensorMap* map, int block, const SinksTile& w, bool is_k) -> bool {
      const int slot = used % C::RING, use = used / C::RING;
      if (use > 0 && !wait_phase(bars + 8 * (C::B_EMPTY + slot), (use - 1) & 1, abort_flag, lim,
                                 (kRoleProducer << 8) | kSiteKvEmpty))
        return false;
      const uint32_t full = bars + 8 * ((is_k ? C::B_K_FULL : C::B_V_FULL) + slot);
      uint32_t& par = is_k ? k_par : v_par;
#pragma unroll
      for (int i = 0; i < C::RING; ++i)
        if (i == slot) last_bar[i] = full, last_par[i] = (par >> slot) & 1u;
      par ^= 1u << slot;
      mbar_arrive_expect_tx(full, C::KV_BYTES);
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c)
        tma_load_4d(base + C::RING_OFF + slot * C::KV_BYTES + c * C::KV_CHUNK, map, full, c * 64,
                    block * C::KEYS, w.hk, w.b);
      ++used;
      return true;
    };
    for (int round = 0; ok && round * G < p.tiles; ++round) {
      const int t = tile_of(round, cta, G);
      if (t >= p.tiles) continue;
      const SinksTile w = sinks_tile(p, t);
      // the first K block needs only a ring slot: before the wait for the Q buffer
      if (!(ok = load(&p.tmap_k, sinks_block(w, 0), w, true))) break;
      if (q_count > 0 && !(ok = wait_phase(bars + 8 * C::B_Q_EMPTY, (q_count - 1) & 1, abort_flag,
                                           lim, (kRoleProducer << 8) | kSiteQEmpty)))
        break;
      mbar_arrive_expect_tx(bars + 8 * C::B_Q_FULL, C::Q_BYTES);
#pragma unroll
      for (int c = 0; c < C::CHUNKS; ++c)
        tma_load_4d(base + C::Q_OFF + c * C::Q_CHUNK, &p.tmap_q, bars + 8 * C::B_Q_FULL, c * 64, w.q0,
                    w.h, w.b);
      ++q_count;
      // each K one block ahead of V
      for (int jj = 0; ok && jj < w.n; ++jj) {
        if (jj + 1 < w.n && !(ok = load(&p.tmap_k, sinks_block(w, jj + 1), w, true))) break;
        ok = load(&p.tmap_v, sinks_block(w, jj), w, false);
      }
    }
    if (!ok) {
      // let the loads in flight land before the shared memory goes away
      volatile int no_abort = 0;
      if (q_count > 0)
        wait_phase(bars + 8 * C::B_Q_FULL, (q_count - 1) & 1, &no_abort, 10000000ull,
                   (kRoleProducer << 8) | kSiteDrain);
#pragma unroll 1
      for (int i = 0; i < C::RING; ++i)
        if (last_bar[i] != 0u)
          wait_phase(last_bar[i], last_par[i], &no_abort, 10000000ull,
                     (kRoleProducer << 8) | kSiteDrain);
    }
  } else if (warp == C::S_WARP && lane == 0) {
    const uint32_t idesc = f16_idesc(BF16, 128, C::KEYS, false);
    const uint32_t qa = sw128_desc_lo(base + C::Q_OFF, 16);
    int used = 0, q_count = 0, blocks = 0;
    uint32_t k_par = 0u;
    bool ok = true;
    for (int round = 0; ok && round * G < p.tiles; ++round) {
      const int t = tile_of(round, cta, G);
      if (t >= p.tiles) continue;
      const int n = sinks_tile(p, t).n;
      if (!(ok = wait_phase(bars + 8 * C::B_Q_FULL, q_count & 1, abort_flag, lim,
                            (kRoleMma << 8) | kSiteQFull)))
        break;
      tc_fence_after_sync();
      ++q_count;
      for (int jj = 0; ok && jj < n; ++jj, ++blocks) {
        const int slot = (used + ring_k(jj)) % C::RING, buf = blocks & 1;
        if (!(ok = wait_phase(bars + 8 * (C::B_K_FULL + slot), (k_par >> slot) & 1u, abort_flag, lim,
                              (kRoleMma << 8) | kSiteKvFull)))
          break;
        k_par ^= 1u << slot;
        if (blocks > 1 && !(ok = wait_phase(bars + 8 * (C::B_S_FREE + buf), ((blocks >> 1) - 1) & 1,
                                            abort_flag, lim, (kRoleMma << 8) | kSiteSFree)))
          break;
        tc_fence_after_sync();
        const uint32_t kb = sw128_desc_lo(base + C::RING_OFF + slot * C::KV_BYTES, 16);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          mma_ss(tmem + C::KEYS * buf, desc_from_lo(qa + (((kk / 4) * C::Q_CHUNK + (kk % 4) * 32) >> 4)),
                 desc_from_lo(kb + (((kk / 4) * C::KV_CHUNK + (kk % 4) * 32) >> 4)), idesc,
                 kk > 0 ? 1u : 0u);
        tc_commit(bars + 8 * (C::B_S_FULL + buf));
        tc_commit(bars + 8 * (C::B_EMPTY + slot));
        if (jj + 1 == n) tc_commit(bars + 8 * C::B_Q_EMPTY);
      }
      used += 2 * n;
    }
    if (!ok) {
      // wait for every MMA this thread issued before TMEM is released
      volatile int no_abort = 0;
      tc_commit(bars + 8 * C::B_DRAIN);
      wait_phase(bars + 8 * C::B_DRAIN, 0, &no_abort, 10000000ull, (kRoleMma << 8) | kSiteDrain);
    }
  } else if (warp == C::PV_WARP && lane == 0) {
    const uint32_t idesc = f16_idesc(BF16, 128, HD, true);
    int used = 0, blocks = 0;
    uint32_t v_par = 0u;
    bool ok = true;
    for (int round = 0; ok && round * G < p.tiles; ++round) {
      const int t = tile_of(round, cta, G);
      if (t >= p.tiles) continue;
      const int n = sinks_tile(p, t).n;
      for (int jj = 0; ok && jj < n; ++jj, ++blocks) {
        const int slot = (used + ring_v(jj, n)) % C::RING, buf = blocks & 1;
        if (!(ok = wait_phase(bars + 8 * (C::B_V_FULL + slot), (v_par >> slot) & 1u, abort_flag, lim,
                              (kRoleMma << 8) | kSiteKvFull)))
          break;
        v_par ^= 1u << slot;
        if (!(ok = wait_phase(bars + 8 * (C::B_P_FULL + buf), (blocks >> 1) & 1, abort_flag, lim,
                              (kRoleMma << 8) | kSitePFull)))
          break;
        tc_fence_after_sync();
        const uint32_t vb = sw128_desc_lo(base + C::RING_OFF + slot * C::KV_BYTES, C::KV_CHUNK);
#pragma unroll
        for (int kk = 0; kk < C::KEYS / 16; ++kk)
          mma_ts(tmem + C::O_COL, tmem + C::KEYS * buf + 8 * kk, desc_from_lo(vb + ((kk * 16 * 128) >> 4)),
                 idesc, (jj > 0 || kk > 0) ? 1u : 0u);
        tc_commit(bars + 8 * (C::B_S_FREE + buf));
        tc_commit(bars + 8 * (C::B_EMPTY + slot));
        if (jj + 1 == n) tc_commit(bars + 8 * C::B_O_FINAL);
      }
      used += 2 * n;
    }
    if (!ok) {
      volatile int no_abort = 0;
      tc_commit(bars + 8 * (C::B_DRAIN + 1));
      wait_phase(bars + 8 * (C::B_DRAIN + 1), 0, &no_abort, 10000000ull, (kRoleMma << 8) | kSiteDrain);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::S_WARP) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace fa_sm100
