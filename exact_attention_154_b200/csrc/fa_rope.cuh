// fa_rope.cuh -- RMS norm of every head's query and key and the rotation by
// position, in one pass, its gradient, and the cos / sin table it reads.
//
// For one row x (a head of a token, d values), weight w and position p:
//
//   n = x * rsqrt(mean(x^2) + eps),  y = n * w          (no norm: y = x)
//   out[a] = y[a] cos - y[b] sin,  out[b] = y[a] sin + y[b] cos
//
// over the pairs (a, b) of the first `rot` columns -- (i, i + rot/2), or
// (2i, 2i + 1) when interleaved -- with cos, sin of pair i at row p of the
// table; columns past rot pass through.  For an arriving gradient g_out:
//
//   g  = the same pairs turned back,  dw = sum over rows g * n
//   dn = g * w,  dx = rsqrt(..) * (dn - n * mean(dn * n))
//
// The statistics and both sums are fp32; each result is rounded once.
//
// What bounds it: memory.  Every row is read once and written once (the
// gradient reads two), there is no reuse to tile for.  d / 8 lanes hold a row
// in 16-byte pieces, so a warp's access covers whole rows; the two halves of
// a pair sit in different lanes when the pairs are (i, i + rot/2) and are
// exchanged by shuffles.  A warp keeps its tokens' cos / sin in registers and
// walks over heads, several rows in flight.
#pragma once

#include "fa_fwd_sm100.cuh"

namespace fa_sm100 {

constexpr unsigned kSitePositions = 17;  // with kRoleArgs: a position outside the table

// One of q and k: rows [b, h, n, :] of the input x, the output y and, in the
// gradient, the arriving gradient g (strides in elements, rows contiguous).
struct RopeOperand {
  const void* x;
  const void* g;
  void* y;
  const void* w;  // [d] or nullptr (no norm)
  void* dw;       // [d] gradient of w, of its type
  long long xb, xh, xn, gb, gh, gn, yb, yh, yn;
  int heads;
};

struct RopeParams {
  RopeOperand op[2];  // q, k
  const float* cos;   // [max_pos, rot / 2]
  const float* sin;
  const int* positions;  // [B, N], or nullptr: the row index
  float* parts;          // gradient: [gridDim.x][2][d] sums of g * n
  int B, N, max_pos, rot, w_fp32;
  float eps;
  int heads_per_warp, chunks;  // head chunks of the q and k heads together
  long long items;             // token groups x chunks
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 p;
    if constexpr (BF16)
      p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    else
      p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                    pack2<BF16>(f[6], f[7]));
}

// Eight consecutive weights as fp32, from the operands' type or from fp32.
template <bool BF16>
__device__ __forceinline__ void load_weight8(const void* w, int w_fp32, int e0, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w_fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + e0);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + e0)), f);
  }
}

// cos / sin of a lane's eight columns e0 .. e0 + 7 of the rotated part.  Half
// layout: one value a column (the columns lie in one half, rot / 2 being a
// multiple of 8), sin negated in the first half, so that
// out = y * cos + partner * sin.  Interleaved: the four pairs' values twice.
template <bool INTER>
__device__ __forceinline__ void load_angles(const float* cos, const float* sin, long long row,
                                            int half, int e0, float (&c)[8], float (&s)[8]) {
  if constexpr (INTER) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(cos + row * half + e0 / 2));
    const float4 b = __ldg(reinterpret_cast<const float4*>(sin + row * half + e0 / 2));
    const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[2 * i] = c[2 * i + 1] = ca[i];
      s[2 * i] = -sa[i];
      s[2 * i + 1] = sa[i];
    }
  } else {
    const bool second = e0 >= half;
    const long long at = row * half + (second ? e0 - half : e0);
    const float4* pc = reinterpret_cast<const float4*>(cos + at);
    const float4* ps = reinterpret_cast<const float4*>(sin + at);
    const float4 a = __ldg(pc), b = __ldg(pc + 1), u = __ldg(ps), v = __ldg(ps + 1);
    const float sg = second ? 1.f : -1.f;
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, c[4] = b.x, c[5] = b.y, c[6] = b.z, c[7] = b.w;
    s[0] = sg * u.x, s[1] = sg * u.y, s[2] = sg * u.z, s[3] = sg * u.w;
    s[4] = sg * v.x, s[5] = sg * v.y, s[6] = sg * v.z, s[7] = sg * v.w;
  }
}

// Turns a lane's eight columns; `partner` is the lane holding the other
// halves of its pairs (half layout).  Every lane of the warp takes part.
template <bool INTER>
__device__ __forceinline__ void rotate8(float (&y)[8], const float (&c)[8], const float (&s)[8],
                                        bool turned, int partner) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = INTER ? y[i ^ 1] : __shfl_sync(0xffffffffu, y[i], partner);
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(y[i], c[i], o[i] * s[i]);
  }
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int sh = LANES / 2; sh > 0; sh >>= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
  return v;
}

constexpr int kRopeThreads = 256;

// One warp item: 32 / (HD / 8) tokens x up to heads_per_warp of the q and k
// heads.  BWD: turns the arriving gradient back and takes it through the
// norm; each CTA sums its rows' g * n and leaves the sums in `parts`.
template <int HD, bool BF16, bool INTER, bool BWD>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int LANES = HD / 8;         // lanes of a row
  constexpr int TOKENS = 32 / LANES;    // tokens of a warp item
  constexpr int WARPS = kRopeThreads / 32;
  constexpr int U = BWD ? 2 : 4;        // rows in flight
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = lane % LANES, e0 = sub * 8;
  const int half = p.rot / 2;
  const bool turned = e0 < p.rot;
  // half layout: column e pairs with e + rot/2, rot / 16 lanes further
  const int partner = turned ? (e0 < half ? lane + p.rot / 16 : lane - p.rot / 16) : lane;
  const int HT = p.op[0].heads + p.op[1].heads;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weight8<BF16>(p.op[0].w, p.w_fp32, e0, wq);
  load_weight8<BF16>(p.op[1].w, p.w_fp32, e0, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) dwq[i] = dwk[i] = 0.f;

  for (long long item = static_cast<long long>(blockIdx.x) * WARPS + warp; item < p.items;
       item += static_cast<long long>(gridDim.x) * WARPS) {
    const long long group = item / p.chunks;
    const int chunk = static_cast<int>(item - group * p.chunks);
    const long long token = group * TOKENS + lane / LANES;
    bool live = token < tokens;
    const int b = live ? static_cast<int>(token / p.N) : 0;
    const int n = live ? static_cast<int>(token - static_cast<long long>(b) * p.N) : 0;
    int pos = n;
    if (p.positions != nullptr && live) pos = __ldg(p.positions + token);
    if (live && (pos < 0 || pos >= p.max_pos)) {
      // outside the table: the token's rows are left unwritten, and reported
      if (sub == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleArgs << 8) | kSitePositions);
      live = false;
    }
    float c[8], s[8];
    if (turned) {
      load_angles<INTER>(p.cos, p.sin, live ? pos : 0, half, e0, c, s);
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
      }
    }
    const int h_end = min(HT, (chunk + 1) * p.heads_per_warp);
    for (int h0 = chunk * p.heads_per_warp; h0 < h_end; h0 += U) {
      uint4 xv[U], gv[U];
      const bool normed0 = p.op[0].w != nullptr, normed1 = p.op[1].w != nullptr;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xv[u] = gv[u] = make_uint4(0u, 0u, 0u, 0u);
        const int hh = h0 + u;
        if (live && hh < h_end) {
          const bool is_k = hh >= p.op[0].heads;
          const RopeOperand& o = p.op[is_k];
          const int h = is_k ? hh - p.op[0].heads : hh;
          if (!BWD || (is_k ? normed1 : normed0))
            xv[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o.x) + b * o.xb +
                                                    h * o.xh + n * o.xn + e0);
          if constexpr (BWD)
            gv[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o.g) + b * o.gb +
                                                    h * o.gh + n * o.gn + e0);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h0 + u;
        if (hh >= h_end) break;
        const bool is_k = hh >= p.op[0].heads;
        const bool normed = is_k ? normed1 : normed0;
        float x[8], y[8];
        unpack8<BF16>(xv[u], x);
        float r = 1.f;
        if (normed) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
          r = rsqrtf(row_sum<LANES>(ss) * (1.f / HD) + p.eps);
          if (!live) r = 0.f;  // no row here: 0 * inf must not reach the sums
        }
        if constexpr (!BWD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i] * r * (is_k ? wk[i] : wq[i]);
          rotate8<INTER>(y, c, s, turned, partner);
        } else {
          unpack8<BF16>(gv[u], y);
          rotate8<INTER>(y, c, s, turned, partner);
          if (normed) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] *= r;  // n
              if (is_k)
                dwk[i] = fmaf(y[i], x[i], dwk[i]);
              else
                dwq[i] = fmaf(y[i], x[i], dwq[i]);
              y[i] *= is_k ? wk[i] : wq[i];
              dot = fmaf(y[i], x[i], dot);
            }
            dot = row_sum<LANES>(dot) * (1.f / HD);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = r * fmaf(-x[i], dot, y[i]);
          }
        }
        if (live) {
          const RopeOperand& o = p.op[is_k];
          const int h = is_k ? hh - p.op[0].heads : hh;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.y) + b * o.yb + h * o.yh + n * o.yn +
                                    e0) = pack8<BF16>(y);
        }
      }
    }
  }
  if constexpr (BWD) {
    // the CTA's sums: lanes of different tokens, then the warps in order
    __shared__ float sums[WARPS][2][HD];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int sh = LANES; sh < 32; sh <<= 1) {
        dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], sh);
        dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], sh);
      }
      if (lane < LANES) {
        sums[warp][0][e0 + i] = dwq[i];
        sums[warp][1][e0 + i] = dwk[i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * HD; i += kRopeThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) t += (&sums[w][0][0])[i];
      p.parts[static_cast<long long>(blockIdx.x) * 2 * HD + i] = t;
    }
  }
}

// dw of q and k: the CTAs' sums added in a fixed order (32 columns a block,
// eight warps over the parts, then the warps in order), rounded to the
// weight's type.
template <bool BF16>
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const float* __restrict__ parts,
                                                              int nparts, int d, void* dq, void* dk,
                                                              int w_fp32) {
  __shared__ float sums[8][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int col = blockIdx.x * 32 + lane;  // of the 2 d columns (q, then k)
  float t = 0.f;
#pragma unroll 8
  for (int i = warp; i < nparts; i += 8) t += parts[static_cast<long long>(i) * 2 * d + col];
  sums[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
    t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += sums[w][lane];
    void* out = col < d ? dq : dk;
    if (out != nullptr) {
      const int e = col < d ? col : col - d;
      if (w_fp32)
        static_cast<float*>(out)[e] = t;
      else if (BF16)
        static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(t);
      else
        static_cast<__half*>(out)[e] = __float2half_rn(t);
    }
  }
}

// cos and sin of position x inverse frequency.  The product and the functions
// are fp64: in fp32 a far position's angle keeps few digits of its fraction
// of a turn.
struct RopeTableParams {
  double inv_freq[128];
  double factor;  // on cos and sin
  float* cos;
  float* sin;
  int max_pos, half;
};
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
  const long long n = static_cast<long long>(p.max_pos) * p.half;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long pos = i / p.half;
    double s, c;
    sincos(static_cast<double>(pos) * p.inv_freq[i - pos * p.half], &s, &c);
    p.cos[i] = static_cast<float>(c * p.factor);
    p.sin[i] = static_cast<float>(s * p.factor);
  }
}

}  // namespace fa_sm100
