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
  int chunks[2];  // head chunks of q and of k
  int ctas_q;     // CTAs that take q's items; the rest take k's
  int blocks;     // blocks of a CTA's tokens (one token group a warp)
};

// Four 16-bit values as two pairs of fp32, and back.
template <bool BF16>
__device__ __forceinline__ void unpack4(const uint2& v, float2* f) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (BF16)
      f[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    else
      f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
}
template <bool BF16>
__device__ __forceinline__ uint2 pack4(const float2* f) {
  return make_uint2(pack2<BF16>(f[0].x, f[0].y), pack2<BF16>(f[1].x, f[1].y));
}

// Four consecutive weights as fp32, from the operands' type or from fp32.
template <bool BF16>
__device__ __forceinline__ void load_weight4(const void* w, int w_fp32, int e, float2* f) {
  if (w == nullptr) {
    f[0] = f[1] = make_float2(1.f, 1.f);
  } else if (w_fp32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + e));
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
  } else {
    unpack4<BF16>(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + e)), f);
  }
}

// The other halves of the pairs that register pair k of a lane's eight columns
// belongs to: the same places of the other piece, or its own two swapped.
template <bool INTER>
__device__ __forceinline__ float2 partner(const float2 (&x)[4], int k) {
  if constexpr (INTER) return make_float2(x[k].y, x[k].x);
  return x[k ^ 2];
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int sh = LANES / 2; sh > 0; sh >>= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
  return v;
}
template <int LANES>
__device__ __forceinline__ float row_dot(const float2 (&x)[4], const float2 (&y)[4]) {
  float2 t = __fmul2_rn(x[0], y[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) t = __ffma2_rn(x[k], y[k], t);
  return row_sum<LANES>(t.x + t.y);
}

constexpr int kRopeThreads = 256;

// A CTA's item: up to heads_per_warp heads of q or k x one group of 32 / (HD / 8)
// tokens for each warp.  Lanes without a token compute its last one again and
// write nothing.
// BWD: turns the arriving gradient back and takes it through the norm; each
// CTA sums its rows' g * n and leaves the sums in `parts`.
template <int HD, bool BF16, bool INTER, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, 4)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = HD / 8;         // lanes of a row
  constexpr int TOKENS = 32 / LANES;    // tokens of a warp item
  constexpr int WARPS = kRopeThreads / 32;
  constexpr int U = BWD ? 1 : 2;        // rows in work; as many more are on their way
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
  const int tokens = p.B * p.N;
  const int items = p.blocks * chunks;
  float2 w[4], dw[4];
  load_weight4<BF16>(op.w, p.w_fp32, ea, w);
  load_weight4<BF16>(op.w, p.w_fp32, eb, w + 2);
#pragma unroll
  for (int k = 0; k < 4; ++k) dw[k] = make_float2(0.f, 0.f);

#pragma unroll 1
  for (int item = cta; item < items; item += ctas) {
    const int block = item / chunks;
    const int h_begin = (item - block * chunks) * p.heads_per_warp;
    const int heads = min(op.heads - h_begin, p.heads_per_warp);
    const long long at_token = static_cast<long long>(block) * (WARPS * TOKENS) + warp * TOKENS + lane / LANES;
    bool live = at_token < tokens;
    const int token = live ? static_cast<int>(at_token) : tokens - 1;
    const int b = token / p.N, n = token - b * p.N;
    const uint16_t* x_at = static_cast<const uint16_t*>(op.x) + b * op.xb + h_begin * op.xh + n * op.xn;
    const uint16_t* g_at = static_cast<const uint16_t*>(op.g) + b * op.gb + h_begin * op.gh + n * op.gn;
    uint16_t* y_at = static_cast<uint16_t*>(op.y) + b * op.yb + h_begin * op.yh + n * op.yn;
    // the rows of heads h .. h + U - 1 of the chunk
    auto load = [&](int h, uint2 (&x)[U][2], uint2 (&g)[U][2]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= heads) break;
        if (!BWD || normed) {
          x[u][0] = *reinterpret_cast<const uint2*>(x_at + ea);
          x[u][1] = *reinterpret_cast<const uint2*>(x_at + eb);
          x_at += op.xh;
        }
        if constexpr (BWD) {
          g[u][0] = *reinterpret_cast<const uint2*>(g_at + ea);
          g[u][1] = *reinterpret_cast<const uint2*>(g_at + eb);
          g_at += op.gh;
        }
      }
    };
    uint2 xv[U][2], gv[U][2];
    load(0, xv, gv);  // before the position, which the cos / sin loads wait for
    int pos = n;
    if (p.positions != nullptr) pos = __ldg(p.positions + token);
    if (pos < 0 || pos >= p.max_pos) {
      // outside the table: the token's rows are left unwritten, and reported
      if (sub == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleArgs << 8) | kSitePositions);
      live = false;
      pos = 0;
    }
    float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turned) {
      const long long at = static_cast<long long>(pos) * half + 4 * sub;
      const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + at));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + at));
      c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
      sn[0] = sv.x, sn[1] = sv.y, sn[2] = sv.z, sn[3] = sv.w;
    }
    // Forward: out = own * own_c + partner * other_c, the weights included
    // (first of a pair: a cos - b sin; second: b cos + a sin).  The gradient
    // turns back with c and sn as they are.
    float2 own_c[4], other_c[4];
    if constexpr (!BWD) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (INTER) {
          own_c[k] = make_float2(c[k], c[k]);
          other_c[k] = make_float2(-sn[k], sn[k]);
        } else {
          const float sg = k < 2 ? -1.f : 1.f;
          own_c[k] = make_float2(c[2 * (k % 2)], c[2 * (k % 2) + 1]);
          other_c[k] = make_float2(sg * sn[2 * (k % 2)], sg * sn[2 * (k % 2) + 1]);
        }
        own_c[k] = __fmul2_rn(own_c[k], w[k]);
        other_c[k] = __fmul2_rn(other_c[k], partner<INTER>(w, k));
      }
    }
#pragma unroll 1
    for (int h0 = 0; h0 < heads; h0 += U) {
      uint2 xn[U][2], gn[U][2];
      load(h0 + U, xn, gn);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h0 + u >= heads) break;
        float2 x[4], y[4], o[4];
        unpack4<BF16>(xv[u][0], x);
        unpack4<BF16>(xv[u][1], x + 2);
        if constexpr (BWD) {
          unpack4<BF16>(gv[u][0], y);
          unpack4<BF16>(gv[u][1], y + 2);
        }
        if constexpr (!BWD) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = __ffma2_rn(x[k], own_c[k], __fmul2_rn(partner<INTER>(x, k), other_c[k]));
        } else if constexpr (INTER) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = make_float2(y[k].x * c[k] + y[k].y * sn[k], y[k].y * c[k] - y[k].x * sn[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            o[k] = make_float2(y[k].x * c[2 * k] + y[k + 2].x * sn[2 * k],
                               y[k].y * c[2 * k + 1] + y[k + 2].y * sn[2 * k + 1]);
            o[k + 2] = make_float2(y[k + 2].x * c[2 * k] - y[k].x * sn[2 * k],
                                   y[k + 2].y * c[2 * k + 1] - y[k].y * sn[2 * k + 1]);
          }
        }
        if (normed) {
          const float r = rsqrtf(row_dot<LANES>(x, x) * (1.f / HD) + p.eps);
          const float2 rr = make_float2(r, r);
          if constexpr (BWD) {
            // o = g; n = x r; dn = g w; dx = r (dn - n mean(dn n))
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = __fmul2_rn(x[k], rr);
              if (live) dw[k] = __ffma2_rn(o[k], x[k], dw[k]);
              o[k] = __fmul2_rn(o[k], w[k]);
            }
            const float dot = row_dot<LANES>(o, x) * (-1.f / HD);
            const float2 dd = make_float2(dot, dot);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __ffma2_rn(x[k], dd, o[k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = __fmul2_rn(o[k], rr);
        }
        if (live) {
          *reinterpret_cast<uint2*>(y_at + ea) = pack4<BF16>(o);
          *reinterpret_cast<uint2*>(y_at + eb) = pack4<BF16>(o + 2);
          y_at += op.yh;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) xv[u][i] = xn[u][i], gv[u][i] = gn[u][i];
    }
  }
  if constexpr (BWD) {
    if (!normed) return;
    // the CTA's sums: lanes of different tokens, then the warps in order
    __shared__ float sums[WARPS][HD];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t = i & 1 ? dw[i / 2].y : dw[i / 2].x;
#pragma unroll
      for (int sh = LANES; sh < 32; sh <<= 1) t += __shfl_xor_sync(0xffffffffu, t, sh);
      if (lane < LANES) sums[warp][(i < 4 ? ea : eb - 4) + i] = t;
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
