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
// its query heads), each warp every (4 x cluster)-th step of 16 keys, straight
// from global memory into registers, and the CTAs' partial results are joined
// through distributed shared memory, in one launch and without scratch.
// Only visible rows are read: whatever the cache holds elsewhere is not.
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

constexpr unsigned kSiteCacheLens = 18;  // with kRoleArgs: a cache length out of range

struct DecodeParams {
  const void* q;  // [B, H, d]
  const void* k;  // [B, Hk, S, d], strides below in elements
  const void* v;
  void* o;        // [B, H, d]
  float* lse;     // [B, H] or nullptr
  const int* seqlens;
  long long kb, kh, kn, vb, vh, vn;
  int H, Hk, S, window, sinks;
  int group, row_tiles;  // query heads of a key head; tiles of 8 NT of them
  float scale_log2;
};

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
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

constexpr int kDecodeWarps = 4;
constexpr int kDecodeMaxCluster = 16;

template <int HD, int NT>
struct DecodeCfg {
  static constexpr int Q = 8 * NT;         // queries of a tile
  static constexpr int ROW = HD + 4;       // floats of a partial O row (padded)
  // per warp: O [Q][ROW], then m [Q] and l [Q]
  static constexpr int WARP_FLOATS = Q * ROW + 2 * Q;
  // the cluster's weights: [rank * warps + warp][Q], then the row sums [Q] and
  // references [Q]
  static constexpr int W_OFF = kDecodeWarps * WARP_FLOATS;
  static constexpr int SMEM_FLOATS = W_OFF + (kDecodeMaxCluster * kDecodeWarps + 2) * Q;
  static constexpr int SMEM_BYTES = 4 * SMEM_FLOATS;
};

template <int HD, int NT, bool BF16>
__global__ void __launch_bounds__(32 * kDecodeWarps) decode_kernel(const DecodeParams p) {
  using C = DecodeCfg<HD, NT>;
  constexpr int KS = HD / 32;  // 16-byte pieces of a key row in a lane
  constexpr int VS = HD / 64;  // of a value row
  extern __shared__ __align__(16) float dsm[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int rank = static_cast<int>(cluster_rank()), CL = static_cast<int>(cluster_size());
  const int tile = blockIdx.y;
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
  // visible keys: `ns` sinks, then from `lo` on; numbered 0 .. L - 1
  const int lo = p.window < 0 ? 0 : max(0, len - 1 - p.window);
  const int ns = min(p.sinks, lo);
  const int L = ns + len - lo, skip = lo - ns;
  const uint16_t* kbase = static_cast<const uint16_t*>(p.k) + b * p.kb + hk * p.kh + 8 * t;
  const uint16_t* vbase = static_cast<const uint16_t*>(p.v) + b * p.vb + hk * p.vh + 8 * g;

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

  uint4 kf[2][KS], vf[4][VS];
  // keys g and g + 8 of the step from visible key v0 on; rows past L are zero
  auto load_k = [&](int v0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = v0 + g + 8 * i;
      const uint16_t* row = kbase + static_cast<long long>(x < ns ? x : x + skip) * p.kn;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        kf[i][s] = x < L ? ld_stream(row + 32 * s) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // values of keys 2t, 2t + 1, 2t + 8, 2t + 9
  auto load_v = [&](int v0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = v0 + 2 * t + (i & 1) + 8 * (i >> 1);
      const uint16_t* row = vbase + static_cast<long long>(x < ns ? x : x + skip) * p.vn;
#pragma unroll
      for (int c = 0; c < VS; ++c)
        vf[i][c] = x < L ? ld_stream(row + 64 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  const int stride = 16 * kDecodeWarps * CL;
  int v0 = 16 * (rank * kDecodeWarps + warp);
  if (v0 < L) {
    load_k(v0);
    load_v(v0);
  }
  for (; v0 < L; v0 += stride) {
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        mma16816<BF16>(s[n], kf[0][x].x, kf[1][x].x, kf[0][x].y, kf[1][x].y, qf[n][x].x, qf[n][x].y);
        mma16816<BF16>(s[n], kf[0][x].z, kf[1][x].z, kf[0][x].w, kf[1][x].w, qf[n][x].z, qf[n][x].w);
      }
    }
    const bool more = v0 + stride < L;
    if (more) load_k(v0 + stride);  // in flight while this step is finished
    uint32_t pt[NT][2];  // P^T operand: keys 0-7 and 8-15 of query g
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // log2-domain scores: [0], [1] key g, [2], [3] key g + 8 of queries 2t, 2t + 1
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[n][i] = v0 + g + 8 * (i >> 1) < L ? s[n][i] * p.scale_log2 : -INFINITY;
      // the reference moves only when a score exceeds it by 2^8 (the first
      // step always moves it): weights stay below 2^8
      const float top0 = fmaxf(s[n][0], s[n][2]), top1 = fmaxf(s[n][1], s[n][3]);
      const bool over = top0 > m[n][0] + kLazyRescaleLog2 || top1 > m[n][1] + kLazyRescaleLog2;
      if (__any_sync(0xffffffffu, over)) {
        float top[2] = {top0, top1};
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
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = ex2(s[n][i] - m[n][i & 1]);
      l[n][0] += e[0] + e[2];
      l[n][1] += e[1] + e[3];
      // weights in 16 bits, as the matrix instruction takes them beside V
      pt[n][0] = transpose8x8(pack2<BF16>(e[0], e[1]));
      pt[n][1] = transpose8x8(pack2<BF16>(e[2], e[3]));
    }
#pragma unroll
    for (int c = 0; c < VS; ++c) {
      const uint32_t va[4] = {vf[0][c].x, vf[0][c].y, vf[0][c].z, vf[0][c].w};
      const uint32_t vb[4] = {vf[1][c].x, vf[1][c].y, vf[1][c].z, vf[1][c].w};
      const uint32_t vc[4] = {vf[2][c].x, vf[2][c].y, vf[2][c].z, vf[2][c].w};
      const uint32_t vd[4] = {vf[3][c].x, vf[3][c].y, vf[3][c].z, vf[3][c].w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // rows g and g + 8 of V^T: columns 64 c + 8 g + 2 r and the next
        const uint32_t a0 = __byte_perm(va[r], vb[r], 0x5410);
        const uint32_t a1 = __byte_perm(va[r], vb[r], 0x7632);
        const uint32_t a2 = __byte_perm(vc[r], vd[r], 0x5410);
        const uint32_t a3 = __byte_perm(vc[r], vd[r], 0x7632);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<BF16>(acc[n][c][r], a0, a1, a2, a3, pt[n][0], pt[n][1]);
      }
    }
    if (more) load_v(v0 + stride);
  }

  // this warp's partial result
  float* mine = dsm + warp * C::WARP_FLOATS;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int q = 8 * n + 2 * t + i;
      float sum = l[n][i];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
      if (g == 0) {
        mine[C::Q * C::ROW + q] = m[n][i];
        mine[C::Q * C::ROW + C::Q + q] = sum;
      }
#pragma unroll
      for (int c = 0; c < VS; ++c) {
        float4* at = reinterpret_cast<float4*>(mine + q * C::ROW + 64 * c + 8 * g);
        at[0] = make_float4(acc[n][c][0][i], acc[n][c][0][i + 2], acc[n][c][1][i], acc[n][c][1][i + 2]);
        at[1] = make_float4(acc[n][c][2][i], acc[n][c][2][i + 2], acc[n][c][3][i], acc[n][c][3][i + 2]);
      }
    }
  cluster_sync();

  // join: the weight of every warp's partial result, in every CTA
  const uint32_t base = smem_u32(dsm);
  float* weight = dsm + C::W_OFF;
  const int parts = CL * kDecodeWarps;
  for (int q = threadIdx.x; q < nq; q += 32 * kDecodeWarps) {
    float top = -INFINITY;
    for (int x = 0; x < parts; ++x) {
      const float mx = ld_cluster(cluster_map(
          base + 4 * ((x % kDecodeWarps) * C::WARP_FLOATS + C::Q * C::ROW + q), x / kDecodeWarps));
      weight[x * C::Q + q] = mx;
      top = fmaxf(top, mx);
    }
    float sum = 0.f;
    for (int x = 0; x < parts; ++x) {
      const float lx = ld_cluster(cluster_map(
          base + 4 * ((x % kDecodeWarps) * C::WARP_FLOATS + C::Q * C::ROW + C::Q + q),
          x / kDecodeWarps));
      const float w = weight[x * C::Q + q] == -INFINITY ? 0.f : ex2(weight[x * C::Q + q] - top);
      weight[x * C::Q + q] = w;
      sum = fmaf(w, lx, sum);
    }
    weight[kDecodeMaxCluster * kDecodeWarps * C::Q + q] = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    if (rank == 0 && p.lse != nullptr)
      p.lse[static_cast<long long>(b) * p.H + h0 + q] = (top + log2f(sum)) * 0.69314718055994530942f;
  }
  __syncthreads();
  // O: four columns a thread, the rows' columns dealt out over the CTAs
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  for (int e = rank * 32 * kDecodeWarps + threadIdx.x; e < nq * (HD / 4);
       e += CL * 32 * kDecodeWarps) {
    const int q = e / (HD / 4), c = e % (HD / 4) * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
      const float w = weight[x * C::Q + q];
      const float4 v = ld_cluster4(cluster_map(
          base + 4 * ((x % kDecodeWarps) * C::WARP_FLOATS + q * C::ROW + c), x / kDecodeWarps));
      o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    }
    const float inv = weight[kDecodeMaxCluster * kDecodeWarps * C::Q + q];
    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) +
                              (static_cast<long long>(b) * p.H + h0 + q) * HD + c) =
        make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace fa_sm100
