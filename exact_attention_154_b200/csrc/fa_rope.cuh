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
// gradient reads two), there is no reuse to tile for.  d / 8 lanes hold a row,
// each two pieces of four columns chosen so that it holds whole pairs (columns
// 4 l and rot/2 + 4 l on, or 8 l on when interleaved): no exchange between
// lanes but the row's sum, and a warp's accesses still cover whole rows.  A
// warp keeps its tokens' four cos / sin values in registers and walks over
// heads of one operand, several rows in flight.
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
  float* parts;          // gradient: [gridDim.x][d] sums of g * n
  int B, N, max_pos, rot, w_fp32;
  float eps;
  int heads_per_warp;
  int chunks[2];       // head chunks of q and of k
  int ctas_q;          // CTAs that take q's items; the rest take k's
  long long groups;    // token groups
};

template <bool BF16>
__device__ __forceinline__ void unpack4(const uint2& v, float* f) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
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
__device__ __forceinline__ uint2 pack4(const float* f) {
  return make_uint2(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]));
}

// Four consecutive weights as fp32, from the operands' type or from fp32.
template <bool BF16>
__device__ __forceinline__ void load_weight4(const void* w, int w_fp32, int e, float* f) {
  if (w == nullptr) {
    f[0] = f[1] = f[2] = f[3] = 1.f;
  } else if (w_fp32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + e));
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  } else {
    unpack4<BF16>(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + e)), f);
  }
}

// Turns a lane's four pairs: (x[i], x[4 + i]), or (x[2i], x[2i + 1]).
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& a = x[INTER ? 2 * i : i];
    float& b = x[INTER ? 2 * i + 1 : 4 + i];
    const float u = a * c[i] - b * s[i];
    b = fmaf(a, s[i], b * c[i]);
    a = u;
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

// One warp item: 32 / (HD / 8) tokens x up to heads_per_warp heads of q or k.
// BWD: turns the arriving gradient back and takes it through the norm; each
// CTA sums its rows' g * n and leaves the sums in `parts`.
template <int HD, bool BF16, bool INTER, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? 2 : 3)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = HD / 8;         // lanes of a row
  constexpr int TOKENS = 32 / LANES;    // tokens of a warp item
  constexpr int WARPS = kRopeThreads / 32;
  constexpr int U = 4;                  // rows in flight
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = lane % LANES;
  const int half = p.rot / 2;
  // this lane's columns: ea .. ea + 3 and eb .. eb + 3
  const bool turned = 8 * sub < p.rot;
  const int ea = !INTER && turned ? 4 * sub : 8 * sub;
  const int eb = !INTER && turned ? half + 4 * sub : 8 * sub + 4;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.ctas_q;
  const RopeOperand& op = p.op[is_k];
  const int cta = is_k ? blockIdx.x - p.ctas_q : blockIdx.x;
  const int ctas = is_k ? gridDim.x - p.ctas_q : p.ctas_q;
  const int chunks = p.chunks[is_k];
  const bool normed = op.w != nullptr;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const long long items = p.groups * chunks;
  float w[8], dw[8];
  load_weight4<BF16>(op.w, p.w_fp32, ea, w);
  load_weight4<BF16>(op.w, p.w_fp32, eb, w + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;

  for (long long item = static_cast<long long>(cta) * WARPS + warp; item < items;
       item += static_cast<long long>(ctas) * WARPS) {
    const long long group = item / chunks;
    const int h_begin = static_cast<int>(item - group * chunks) * p.heads_per_warp;
    const int h_end = min(op.heads, h_begin + p.heads_per_warp);
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
    const uint16_t* x_row = static_cast<const uint16_t*>(op.x) + b * op.xb + n * op.xn;
    const uint16_t* g_row = static_cast<const uint16_t*>(op.g) + b * op.gb + n * op.gn;
    uint16_t* y_row = static_cast<uint16_t*>(op.y) + b * op.yb + n * op.yn;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (turned && live) {
      const long long at = static_cast<long long>(pos) * half + 4 * sub;
      const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + at));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + at));
      const float sg = BWD ? -1.f : 1.f;  // the gradient turns back
      c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
      s[0] = sg * sv.x, s[1] = sg * sv.y, s[2] = sg * sv.z, s[3] = sg * sv.w;
    }
#pragma unroll 1
    for (int h0 = h_begin; h0 < h_end; h0 += U) {
      uint2 xv[U][2], gv[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xv[u][0] = xv[u][1] = gv[u][0] = gv[u][1] = make_uint2(0u, 0u);
        if (live && h0 + u < h_end) {
          if (!BWD || normed) {
            const uint16_t* x = x_row + (h0 + u) * op.xh;
            xv[u][0] = *reinterpret_cast<const uint2*>(x + ea);
            xv[u][1] = *reinterpret_cast<const uint2*>(x + eb);
          }
          if constexpr (BWD) {
            const uint16_t* g = g_row + (h0 + u) * op.gh;
            gv[u][0] = *reinterpret_cast<const uint2*>(g + ea);
            gv[u][1] = *reinterpret_cast<const uint2*>(g + eb);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u >= h_end) break;
        float x[8], y[8];
        unpack4<BF16>(xv[u][0], x);
        unpack4<BF16>(xv[u][1], x + 4);
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
          for (int i = 0; i < 8; ++i) y[i] = x[i] * r * w[i];
          rotate<INTER>(y, c, s);
        } else {
          unpack4<BF16>(gv[u][0], y);
          unpack4<BF16>(gv[u][1], y + 4);
          rotate<INTER>(y, c, s);
          if (normed) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] *= r;  // n
              dw[i] = fmaf(y[i], x[i], dw[i]);
              y[i] *= w[i];
              dot = fmaf(y[i], x[i], dot);
            }
            dot = row_sum<LANES>(dot) * (1.f / HD);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = r * fmaf(-x[i], dot, y[i]);
          }
        }
        if (live) {
          uint16_t* out = y_row + (h0 + u) * op.yh;
          *reinterpret_cast<uint2*>(out + ea) = pack4<BF16>(y);
          *reinterpret_cast<uint2*>(out + eb) = pack4<BF16>(y + 4);
        }
      }
    }
  }
  if constexpr (BWD) {
    if (!normed) return;
    // the CTA's sums: lanes of different tokens, then the warps in order
    __shared__ float sums[WARPS][HD];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int sh = LANES; sh < 32; sh <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], sh);
      if (lane < LANES) sums[warp][(i < 4 ? ea : eb - 4) + i] = dw[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < HD; i += kRopeThreads) {
      float t = 0.f;
#pragma unroll
      for (int v = 0; v < WARPS; ++v) t += sums[v][i];
      p.parts[static_cast<long long>(blockIdx.x) * HD + i] = t;
    }
  }
}

// dw of q (blockIdx.y 0) and k (1): the sums of the operand's CTAs added in a
// fixed order (32 columns a block, 32 warps over the parts, then the warps in
// order), rounded to the weight's type.
template <bool BF16>
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* __restrict__ parts,
                                                               int ctas_q, int ctas, int d, void* dq,
                                                               void* dk, int w_fp32) {
  __shared__ float sums[32][33];
  void* out = blockIdx.y == 0 ? dq : dk;
  if (out == nullptr) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int col = blockIdx.x * 32 + lane;
  const int first = blockIdx.y == 0 ? 0 : ctas_q, end = blockIdx.y == 0 ? ctas_q : ctas;
  float t = 0.f;
#pragma unroll 8
  for (int i = first + warp; i < end; i += 32) t += parts[static_cast<long long>(i) * d + col];
  sums[warp][lane] = t;
  __syncthreads();
  // warp w sums column w's 32 partial sums, lane by lane in tree order
  t = sums[lane][warp];
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) t += __shfl_xor_sync(0xffffffffu, t, sh);
  if (lane == 0) {
    const int e = blockIdx.x * 32 + warp;
    if (w_fp32)
      static_cast<float*>(out)[e] = t;
    else if (BF16)
      static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(t);
    else
      static_cast<__half*>(out)[e] = __float2half_rn(t);
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
