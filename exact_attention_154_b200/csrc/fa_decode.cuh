// fa_decode.cuh -- attention of one query per sequence over a key / value
// cache, with a window and sinks, for sm_100a.
//
// Sequence b holds n = seqlens[b] tokens, the last being the query's own.
// Visible are the keys of the last window + 1 tokens and the first `sinks`;
// O = sum_j exp(s_j) v_j / sum_j exp(s_j), s_j = scale q . k_j, by the online
// recurrence (reference m, row sum l and O in fp32, lazily rescaled as in the
// forward), over keys spread on many warps and joined at the end.
//
// What bounds it: the bytes of the visible keys and values, each of which
// meets only the G = H / Hk query heads that share it.  So the work is split
// over keys: a cluster of CTAs takes one key head of one sequence (up to 8 NT of
// its query heads), each warp every (4 x cluster)-th step of 32 keys, and the
// CTAs' partial results are joined through distributed shared memory, in one
// launch and without scratch.
//
// Loads run ahead in a ring of shared memory that each warp keeps for itself,
// the keys and the values of a step being one slot each, filled by TMA from one
// lane (any strides; 128-byte swizzle).  A step lies wholly among the sinks or
// wholly in the window, so it is rows on end; rows a step holds beyond the
// visible ones get score -infinity, and their values are zeroed before use.
//
// The products are transposed so that keys, not the few queries, fill the
// 16-row side of the matrix instruction (mma.sync m16n8k16; the instruction's
// rate is far from binding here):
//   S^T [16 keys x 8 queries] = K Q^T      K is the row-major A operand
//   O^T [d x 8 queries]      += V^T P^T    V^T is the A operand
// The d axis of the first product may be summed in any order and the d axis
// of the second is a row index, so each lane loads 16-byte pieces of a row and
// hands them out over the instructions' columns (rows): no transposition
// through shared memory, and every load covers whole 32-byte sectors.
#pragma once

#include "fa_fwd_sm100.cuh"

namespace fa_sm100 {

constexpr unsigned kRoleDecode = 7;
constexpr unsigned kSiteCacheLens = 18;  // with kRoleArgs: a cache length out of range

struct DecodeParams {
  CUtensorMap tmap_k;  // 4-D (d, S, Hk, B) views, box 64 elements x a step's rows
  CUtensorMap tmap_v;
  const void* q;  // [B, H, d]
  void* o;        // [B, H, d]
  float* lse;     // [B, H] or nullptr
  const int* seqlens;
  int H, Hk, S, window, sinks;
  int group, row_tiles;  // query heads of a key head; tiles of 8 NT of them
  float scale_log2;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
// D += A B, m16n8k16, 16-bit A (row-major) and B (column-major), fp32 D.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values spread over the warp (lane i:
// row i / 4, columns 2 (i % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Shared-memory address `addr` of this CTA, in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}

// Weight of a partial result with reference m against the joint reference:
// 0 where it saw no key.
__device__ __forceinline__ float join_weight(float m, float top) {
  return m == -INFINITY ? 0.f : ex2(m - top);
}

// The order in which the operands' rows take a step's first eight keys (and
// the next eight): 0 5 2 7 4 1 6 3.  In the 128-byte swizzle (16-byte unit u of
// row r at u ^ r % 8) every eight lanes' reads then fall on distinct banks: K
// reads take units t of two rows 5 apart, V reads units g, g + 1 of the four
// even rows or the four odd ones.
__device__ __forceinline__ int key_order(int i) { return (0x36147250u >> (4 * i)) & 7; }

constexpr int kDecodeWarps = 4;
constexpr int kDecodeMaxCluster = 16;
// Bytes of ring a warp has.  16 KB leave three CTAs on an SM; 24 KB (two) measured
// 2 to 8% slower on full batches and 5% faster for one long sequence.
constexpr int kDecodeRing = 16384;

template <int HD, int NT>
struct DecodeCfg {
  static constexpr int Q = 8 * NT;         // queries of a tile
  static constexpr int ROW = HD + 4;       // floats of a partial O row (padded)
  // per warp the ring, over which its partial O [Q][ROW] is written at the end
  // keys of a step: two 16-row tiles whose products interleave (one of their
  // chains alone would leave the warp waiting), one at d = 256 for the registers
  static constexpr int TILES = HD == 256 ? 1 : 2;
  static constexpr int KEYS = 16 * TILES;
  static constexpr int CHUNK_BYTES = KEYS * 128;            // 64 columns of a step
  static constexpr int SLOT_BYTES = HD / 64 * CHUNK_BYTES;  // keys or values of a step
  static constexpr int SLOTS = kDecodeRing / SLOT_BYTES;
  static constexpr int WARP_FLOATS = SLOTS * SLOT_BYTES / 4;
  static_assert(Q * ROW <= WARP_FLOATS, "partial result over the ring");
  // then the warps' references [warp][Q] and row sums [warp][Q], the CTA's
  // [Q] and [Q], and the cluster's weights [rank][Q]
  static constexpr int M_OFF = kDecodeWarps * WARP_FLOATS;
  static constexpr int L_OFF = M_OFF + kDecodeWarps * Q;
  static constexpr int CM_OFF = L_OFF + kDecodeWarps * Q;
  static constexpr int CL_OFF = CM_OFF + Q;
  static constexpr int W_OFF = CL_OFF + Q;
  static constexpr int BAR_OFF = W_OFF + kDecodeMaxCluster * Q;  // mbarriers [warp][slot]
  static constexpr int SMEM_FLOATS = BAR_OFF + 2 * kDecodeWarps * SLOTS + 2;  // abort word
  static_assert(WARP_FLOATS % 256 == 0, "1024-byte aligned rings");
  static_assert(BAR_OFF % 2 == 0, "8-byte aligned barriers");
  static constexpr int SMEM_BYTES = 4 * SMEM_FLOATS + 1008;  // and the base's alignment
};

template <int HD, int NT, bool BF16>
__global__ void __launch_bounds__(32 * kDecodeWarps) decode_kernel(const __grid_constant__ DecodeParams p) {
  using C = DecodeCfg<HD, NT>;
  constexpr int KS = HD / 32;  // 16-byte pieces of a key row in a lane
  constexpr int VS = HD / 64;  // of a value row
  extern __shared__ uint8_t dsm_raw[];
  // 1024-byte aligned (the same offset in every CTA)
  float* dsm = reinterpret_cast<float*>(dsm_raw + ((0u - smem_u32(dsm_raw)) & 1023u));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int rank = static_cast<int>(cluster_rank()), CL = static_cast<int>(cluster_size());
  const int tile = blockIdx.x / CL;
  const int rt = tile % p.row_tiles;
  const int bh = tile / p.row_tiles;
  const int b = bh / p.Hk, hk = bh - b * p.Hk;
  const int h0 = hk * p.group + rt * C::Q;            // first query head of the tile
  const int nq = min(C::Q, p.group - rt * C::Q);      // query heads of the tile
  const int len = __ldg(p.seqlens + b);
  if (len < 0 || len > p.S) {
    // out of range: the sequence's rows are left unwritten, and reported (the
    // whole cluster takes this way)
    if (threadIdx.x == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleArgs << 8) | kSiteCacheLens);
    return;
  }
  // visible keys: `ns` sinks, then from `lo` on; in steps of KEYS rows,
  // the sinks' first
  const int lo = p.window < 0 ? 0 : max(0, len - 1 - p.window);
  const int ns = min(p.sinks, lo);
  const int sink_steps = (ns + C::KEYS - 1) / C::KEYS;
  const int steps = sink_steps + (len - lo + C::KEYS - 1) / C::KEYS;

  // Q^T operand: query g of each tile of 8, the d axis in the order of the
  // key pieces
  uint4 qf[NT][KS];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qf[n][s] = make_uint4(0u, 0u, 0u, 0u);
      if (8 * n + g < nq)
        qf[n][s] = *reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) +
            (static_cast<long long>(b) * p.H + h0 + 8 * n + g) * HD + 32 * s + 8 * t);
    }

  float acc[NT][VS][4][4];  // [query tile][64 columns][row pair][operand D register]
  float m[NT][2], l[NT][2];  // of queries 2t, 2t + 1
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int c = 0; c < VS; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][c][r][i] = 0.f;
  }

  // The keys of a step in the order the operands' rows take them
  const int my_key = key_order(g), key_a = key_order(2 * t), key_b = key_order(2 * t + 1);

  // The ring: slot by slot the keys of this warp's first step, its values, the
  // keys of the next, ...
  const uint32_t ring = smem_u32(dsm + warp * C::WARP_FLOATS);
  const uint32_t bars = smem_u32(dsm + C::BAR_OFF) + 8 * warp * C::SLOTS;
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(dsm + C::BAR_OFF + 2 * kDecodeWarps * C::SLOTS);
  if (lane == 0) {
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  __syncthreads();
  const int stride = kDecodeWarps * CL;
  int step = rank * kDecodeWarps + warp;
  // half-steps still to be copied: the next one's step and which half
  int next_step = step, filled = 0;
  bool next_is_v = false;
  auto copy_next = [&](uint32_t slot) {
    if (next_step >= steps) return;
    __syncwarp();  // every lane has used the slot's last contents
    if (lane == 0) {
      const uint32_t bar = bars + 8 * slot;
      const int row = next_step < sink_steps ? C::KEYS * next_step
                                              : lo + C::KEYS * (next_step - sink_steps);
      mbar_arrive_expect_tx(bar, C::SLOT_BYTES);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c)
        tma_load_4d(ring + slot * C::SLOT_BYTES + c * C::CHUNK_BYTES,
                    next_is_v ? &p.tmap_v : &p.tmap_k, bar, 64 * c, row, hk, b);
    }
    if (next_is_v) next_step += stride;
    next_is_v = !next_is_v;
    ++filled;
  };
#pragma unroll 1
  for (int i = 0; i < C::SLOTS; ++i) copy_next(i);
  uint32_t slot = 0, parity = 0;
  int used = 0;
  bool ok = true;
  // the next slot's contents, to every lane
  auto wait_slot = [&]() -> bool {
    ok = wait_phase(bars + 8 * slot, parity, abort_flag, p.wait_limit_ns,
                    (kRoleDecode << 8) | kSiteKvFull);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  // the products have the slot's contents: refill it
  auto next_slot = [&]() {
    copy_next(slot);
    ++used;
    if (++slot == C::SLOTS) slot = 0, parity ^= 1u;
  };
  for (; step < steps; step += stride) {
    // visible rows of this step
    const int rows = step < sink_steps
                         ? min(C::KEYS, ns - C::KEYS * step)
                         : min(C::KEYS, len - lo - C::KEYS * (step - sink_steps));
    if (!wait_slot()) break;
    float s[C::TILES][NT][4];
#pragma unroll
    for (int j = 0; j < C::TILES; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) s[j][n][0] = s[j][n][1] = s[j][n][2] = s[j][n][3] = 0.f;
#pragma unroll
    for (int x0 = 0; x0 < KS; x0 += 4) {  // 128 columns at a time
      constexpr int XS = KS < 4 ? KS : 4;
      uint4 kf[C::TILES][2][XS];
#pragma unroll
      for (int x = 0; x < XS; ++x)
#pragma unroll
        for (int j = 0; j < C::TILES; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            kf[j][i][x] = ld_shared_v4(ring + slot * C::SLOT_BYTES + ((x0 + x) / 2) * C::CHUNK_BYTES +
                                       (my_key + 8 * i + 16 * j) * 128 +
                                       (((4 * (x % 2) + t) ^ my_key) << 4));
#pragma unroll
      for (int x = 0; x < XS; ++x) {
#pragma unroll
        for (int j = 0; j < C::TILES; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<BF16>(s[j][n], kf[j][0][x].x, kf[j][1][x].x, kf[j][0][x].y, kf[j][1][x].y,
                           qf[n][x0 + x].x, qf[n][x0 + x].y);
#pragma unroll
        for (int j = 0; j < C::TILES; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<BF16>(s[j][n], kf[j][0][x].z, kf[j][1][x].z, kf[j][0][x].w, kf[j][1][x].w,
                           qf[n][x0 + x].z, qf[n][x0 + x].w);
      }
    }
    next_slot();
    uint32_t pt[C::TILES][NT][2];  // P^T operand: keys 0-7 and 8-15 of a tile, query g
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // log2-domain scores: [0], [1] this lane's key of the tile, [2], [3] the
      // one eight further, of queries 2t, 2t + 1
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < C::TILES; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[j][n][i] = my_key + 8 * (i >> 1) + 16 * j < rows ? s[j][n][i] * p.scale_log2 : -INFINITY;
          top[i & 1] = fmaxf(top[i & 1], s[j][n][i]);
        }
      // the reference moves only when a score exceeds it by 2^8 (the first
      // step always moves it): weights stay below 2^8
      const bool over = top[0] > m[n][0] + kLazyRescaleLog2 || top[1] > m[n][1] + kLazyRescaleLog2;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1)
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], sh));
          const float to = fmaxf(m[n][i], top[i]);
          const float alpha = to == -INFINITY ? 1.f : ex2(m[n][i] - to);
          m[n][i] = to;
          l[n][i] *= alpha;
#pragma unroll
          for (int c = 0; c < VS; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              acc[n][c][r][i] *= alpha;
              acc[n][c][r][i + 2] *= alpha;
            }
        }
      }
      // (a warp that has met only scores of -infinity has no reference yet, and its
      // weights are 0: finite queries and keys reach that where fp32 overflows)
      const float ref[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
      for (int j = 0; j < C::TILES; ++j) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = ex2(s[j][n][i] - ref[i & 1]);
        l[n][0] += e[0] + e[2];
        l[n][1] += e[1] + e[3];
        // weights in 16 bits, as the matrix instruction takes them beside V
        pt[j][n][0] = transpose8x8(pack2<BF16>(e[0], e[1]));
        pt[j][n][1] = transpose8x8(pack2<BF16>(e[2], e[3]));
      }
    }
    if (!wait_slot()) break;
    if (rows < C::KEYS) {
      // values of rows that are not visible: weight 0, but 0 times whatever the
      // cache holds there need not be 0
      if (lane >= rows && lane < C::KEYS) {
#pragma unroll
        for (int x = 0; x < HD / 8; ++x)
          st_shared_v4(ring + slot * C::SLOT_BYTES + (x / 8) * C::CHUNK_BYTES + lane * 128 + (x % 8) * 16,
                       0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // before the TMA that refills the slot
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < C::TILES; ++j)
#pragma unroll
      for (int c = 0; c < VS; ++c) {
        // keys 2t, 2t + 1 of the operand's order, and the two eight further
        uint4 vf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = i & 1 ? key_b : key_a;
          vf[i] = ld_shared_v4(ring + slot * C::SLOT_BYTES + c * C::CHUNK_BYTES +
                               (key + 8 * (i >> 1) + 16 * j) * 128 + ((g ^ key) << 4));
        }
        const uint32_t va[4] = {vf[0].x, vf[0].y, vf[0].z, vf[0].w};
        const uint32_t vb[4] = {vf[1].x, vf[1].y, vf[1].z, vf[1].w};
        const uint32_t vc[4] = {vf[2].x, vf[2].y, vf[2].z, vf[2].w};
        const uint32_t vd[4] = {vf[3].x, vf[3].y, vf[3].z, vf[3].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // rows g and g + 8 of V^T: columns 64 c + 8 g + 2 r and the next
          const uint32_t a0 = __byte_perm(va[r], vb[r], 0x5410);
          const uint32_t a1 = __byte_perm(va[r], vb[r], 0x7632);
          const uint32_t a2 = __byte_perm(vc[r], vd[r], 0x5410);
          const uint32_t a3 = __byte_perm(vc[r], vd[r], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816<BF16>(acc[n][c][r], a0, a1, a2, a3, pt[j][n][0], pt[j][n][1]);
        }
      }
    next_slot();
  }
  if (!ok) {
    // gave up: let the copies in flight land; the results are undefined
    volatile int no_abort = 0;
    for (int i = used; i < filled; ++i)
      wait_phase(bars + 8 * (i % C::SLOTS), (i / C::SLOTS) & 1, &no_abort, 10000000ull,
                 (kRoleDecode << 8) | kSiteDrain);
  }
  __syncwarp();  // the warp's ring is idle: partial results go over it

  // Join the CTA's warps: each scales its O to the largest reference, then
  // the warps' rows are added.
  constexpr int kThreads = 32 * kDecodeWarps;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[n][i];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
      if (g == 0) {
        dsm[C::M_OFF + warp * C::Q + 8 * n + 2 * t + i] = m[n][i];
        dsm[C::L_OFF + warp * C::Q + 8 * n + 2 * t + i] = sum;
      }
    }
  __syncthreads();
  float* mine = dsm + warp * C::WARP_FLOATS;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = 8 * n + 2 * t + i;
      float top = dsm[C::M_OFF + q];
#pragma unroll
      for (int x = 1; x < kDecodeWarps; ++x) top = fmaxf(top, dsm[C::M_OFF + x * C::Q + q]);
      const float w = join_weight(m[n][i], top);
#pragma unroll
      for (int c = 0; c < VS; ++c) {
        float4* at = reinterpret_cast<float4*>(mine + q * C::ROW + 64 * c + 8 * g);
        at[0] = make_float4(acc[n][c][0][i] * w, acc[n][c][0][i + 2] * w, acc[n][c][1][i] * w,
                            acc[n][c][1][i + 2] * w);
        at[1] = make_float4(acc[n][c][2][i] * w, acc[n][c][2][i + 2] * w, acc[n][c][3][i] * w,
                            acc[n][c][3][i + 2] * w);
      }
    }
  if (threadIdx.x < C::Q) {
    const int q = threadIdx.x;
    float top = -INFINITY, sum = 0.f;
    for (int x = 0; x < kDecodeWarps; ++x) top = fmaxf(top, dsm[C::M_OFF + x * C::Q + q]);
    for (int x = 0; x < kDecodeWarps; ++x)
      sum = fmaf(join_weight(dsm[C::M_OFF + x * C::Q + q], top), dsm[C::L_OFF + x * C::Q + q], sum);
    dsm[C::CM_OFF + q] = top;
    dsm[C::CL_OFF + q] = sum;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nq * (HD / 4); e += kThreads) {
    float4* at = reinterpret_cast<float4*>(dsm + e / (HD / 4) * C::ROW + e % (HD / 4) * 4);
    float4 o = *at;
#pragma unroll
    for (int x = 1; x < kDecodeWarps; ++x) {
      const float4 v = at[x * (C::WARP_FLOATS / 4)];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
    }
    *at = o;
  }
  cluster_sync();

  // Join the CTAs: a half-warp per query, a lane per CTA, weighs them; then
  // the rows' columns are dealt out, four to a thread.
  const uint32_t base = smem_u32(dsm);
  for (int q = 2 * warp + lane / 16; q < C::Q; q += 2 * kDecodeWarps) {
    const int x = lane % 16;
    float mx = -INFINITY, lx = 0.f;
    if (x < CL) {
      mx = ld_cluster(cluster_map(base + 4 * (C::CM_OFF + q), x));
      lx = ld_cluster(cluster_map(base + 4 * (C::CL_OFF + q), x));
    }
    float top = mx;
#pragma unroll
    for (int sh = 8; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
    const float w = join_weight(mx, top);
    float sum = x < CL ? w * lx : 0.f;
#pragma unroll
    for (int sh = 8; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
    // no visible key: O = 0 (a NaN among them stays one)
    dsm[C::W_OFF + x * C::Q + q] = sum == 0.f ? 0.f : w / sum;
    if (rank == 0 && x == 0 && q < nq && p.lse != nullptr)
      p.lse[static_cast<long long>(b) * p.H + h0 + q] = (top + log2f(sum)) * 0.69314718055994530942f;
  }
  __syncthreads();
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  for (int e = rank * kThreads + threadIdx.x; e < nq * (HD / 4); e += CL * kThreads) {
    const int q = e / (HD / 4), c = e % (HD / 4) * 4;
    const uint32_t at = base + 4 * (q * C::ROW + c);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < CL; ++x) {
      const float w = dsm[C::W_OFF + x * C::Q + q];
      const float4 v = ld_cluster4(cluster_map(at, x));
      o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    }
    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) +
                              (static_cast<long long>(b) * p.H + h0 + q) * HD + c) =
        make_uint2(pack2<BF16>(o.x, o.y), pack2<BF16>(o.z, o.w));
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace fa_sm100
