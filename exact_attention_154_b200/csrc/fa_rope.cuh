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
// What bounds it: memory, if the instructions a row takes stay few.  Every row
// is read once and written once (the gradient reads two), there is no reuse to
// tile for.  d / 16 lanes hold a row, each two 16-byte pieces chosen so that it
// holds whole pairs (columns 8 l and rot/2 + 8 l on, or 16 l on when
// interleaved): no exchange between lanes but the row's sum.  A warp keeps its
// tokens' eight cos / sin values a lane in registers and walks over heads of one
// operand, the next row on its way.  Measured, 16384 tokens x 18 heads of 128, inputs
// not in L2: forward 28.8 us (23.4 at the measured copy rate), issue slots 58% used;
// gradient 53.4 us (34.9), where registers leave 16 warps an SM, issue slots are 43%
// used and the wait for loads is the largest part of a warp's time.
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

// Eight 16-bit values as four pairs of fp32, and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float2* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)
      f[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    else
      f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float2* f) {
  return make_uint4(pack2<BF16>(f[0].x, f[0].y), pack2<BF16>(f[1].x, f[1].y),
                    pack2<BF16>(f[2].x, f[2].y), pack2<BF16>(f[3].x, f[3].y));
}
__device__ __forceinline__ void load_float8(const float* at, float2* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(at));
  const float4 b = __ldg(reinterpret_cast<const float4*>(at) + 1);
  f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
}

// Eight consecutive weights as fp32, from the operands' type or from fp32.
template <bool BF16>
__device__ __forceinline__ void load_weight8(const void* w, int w_fp32, int e, float2* f) {
  if (w == nullptr) {
    f[0] = f[1] = f[2] = f[3] = make_float2(1.f, 1.f);
  } else if (w_fp32) {
    load_float8(static_cast<const float*>(w) + e, f);
  } else {
    unpack8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + e)), f);
  }
}

// The other halves of the pairs that register pair k of a lane's sixteen
// columns belongs to: the same places of the other piece, or its own two swapped.
template <bool INTER>
__device__ __forceinline__ float2 partner(const float2 (&x)[8], int k) {
  if constexpr (INTER) return make_float2(x[k].y, x[k].x);
  return x[k ^ 4];
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_dot(const float2 (&x)[8], const float2 (&y)[8]) {
  float2 t = __fmul2_rn(x[0], y[0]), u = __fmul2_rn(x[1], y[1]);
#pragma unroll
  for (int k = 2; k < 8; k += 2) {
    t = __ffma2_rn(x[k], y[k], t);
    u = __ffma2_rn(x[k + 1], y[k + 1], u);
  }
  t = __fadd2_rn(t, u);
  float v = t.x + t.y;
#pragma unroll
  for (int sh = LANES / 2; sh > 0; sh >>= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
  return v;
}

// Threads, and CTAs of an SM that the registers are limited for (80 and 128).
// Measured on 16384 tokens x 18 heads of 128, forward / gradient, before rows were
// requested ahead (with it, inputs not in L2: 28.8 / 53.7): 32.4 / 53 us;
// 64 registers (spilled) 41 / 83, 128 in the forward 37; d / 8 lanes a row with
// 8-byte pieces 35 / 70 (its per-row instructions weigh twice as much), and the
// same with rows through a ring of asynchronous copies 42 / 59.
constexpr int kRopeThreads = 128;
constexpr int kRopeFwdCtas = 6, kRopeBwdCtas = 4;

// PART: rot < HD, and some lanes' columns stay as they are: selects keep them apart from
// their neighbours.  With rot == HD there are none, and the selects fall away (16384
// tokens x 18 heads, forward / gradient: 64 of 128 columns 27.8 / 53.7 us, 128 of 128
// 26.6 / 52.2; a branch on the lane, in every call, 28.7 / 54.8 for 128 of 128).
//
// A CTA's item: up to heads_per_warp heads of q or k x one group of 32 / (HD / 16)
// tokens for each warp.  Lanes without a token compute its last one again and
// write nothing.  BWD: turns the arriving gradient back and takes it through
// the norm; each CTA sums its rows' g * n and leaves the sums in `parts`.
template <int HD, bool BF16, bool INTER, bool PART, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? kRopeBwdCtas : kRopeFwdCtas)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LANES = HD / 16;        // lanes of a row
  constexpr int TOKENS = 32 / LANES;    // tokens of a warp item
  constexpr int WARPS = kRopeThreads / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sub = lane % LANES;
  const int half = p.rot / 2;
  // this lane's columns: ea .. ea + 7 and eb .. eb + 7
  const bool turned = !PART || 16 * sub < p.rot;
  const int ea = !INTER && turned ? 8 * sub : 16 * sub;
  const int eb = !INTER && turned ? half + 8 * sub : 16 * sub + 8;
  const bool is_k = static_cast<int>(blockIdx.x) >= p.ctas_q;
  const RopeOperand& op = p.op[is_k];
  const int cta = is_k ? blockIdx.x - p.ctas_q : blockIdx.x;
  const int ctas = is_k ? gridDim.x - p.ctas_q : p.ctas_q;
  const int chunks = p.chunks[is_k];
  const bool normed = op.w != nullptr;
  const int tokens = p.B * p.N;
  const int items = p.blocks * chunks;
  const long long xh = op.xh, gh = op.gh, yh = op.yh;
  float2 w[8], dw[8];
  if constexpr (BWD) {
    // norm_weight_sum_kernel may take its place, and waits there for this grid's end
    // (gradient 55.3 -> 53.7 us, a small one 19.1 -> 18.4)
    asm volatile("griddepcontrol.launch_dependents;");
    load_weight8<BF16>(op.w, p.w_fp32, ea, w);
    load_weight8<BF16>(op.w, p.w_fp32, eb, w + 4);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) dw[k] = make_float2(0.f, 0.f);

#pragma unroll 1
  for (int item = cta; item < items; item += ctas) {
    const int block = item / chunks;
    const int h_begin = (item - block * chunks) * p.heads_per_warp;
    const int heads = min(op.heads - h_begin, p.heads_per_warp);
    const long long at_token = static_cast<long long>(block) * (WARPS * TOKENS) + warp * TOKENS + lane / LANES;
    bool live = at_token < tokens;
    const int token = live ? static_cast<int>(at_token) : tokens - 1;
    const int b = token / p.N, n = token - b * p.N;
    const uint16_t* x_at = static_cast<const uint16_t*>(op.x) + b * op.xb + h_begin * xh + n * op.xn;
    const uint16_t* g_at = static_cast<const uint16_t*>(op.g) + b * op.gb + h_begin * gh + n * op.gn;
    uint16_t* y_at = static_cast<uint16_t*>(op.y) + b * op.yb + h_begin * yh + n * op.yn;
    // the row at x_at and g_at; moves on to the next head's
    auto load = [&](uint4 (&x)[2], uint4 (&g)[2]) {
      if (!BWD || normed) {
        x[0] = *reinterpret_cast<const uint4*>(x_at + ea);
        x[1] = *reinterpret_cast<const uint4*>(x_at + eb);
        x_at += xh;
      }
      if constexpr (BWD) {
        g[0] = *reinterpret_cast<const uint4*>(g_at + ea);
        g[1] = *reinterpret_cast<const uint4*>(g_at + eb);
        g_at += gh;
      }
    };
    // the row `by` heads after x_at's to L2: the registers hold one row on its way,
    // too little to cover the latency of memory (forward 33.0 -> 28.8 us; the
    // gradient, with two operands' rows, lost 4%)
    auto ahead = [&](int by) {
      if (!BWD) asm volatile("prefetch.global.L2 [%0];" ::"l"(x_at + by * xh + 16 * sub));
    };
    uint4 xv[2], gv[2];
    load(xv, gv);  // before the position, which the cos / sin loads wait for
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (i < heads) ahead(i - 1);
    int pos = n;
    if (p.positions != nullptr) pos = __ldg(p.positions + token);
    if (pos < 0 || pos >= p.max_pos) {
      // outside the table: the token's rows are left unwritten, and reported
      if (sub == 0) atomicCAS(&g_fa_watchdog, 0u, (kRoleArgs << 8) | kSitePositions);
      live = false;
      pos = 0;
    }
    // Of the lane's eight pairs.  Columns past rot are their own times 1 plus a zero in
    // place of their neighbour times -0: the neighbour may be infinite, and adding
    // -0 changes nothing, not even the sign of a zero.
    float2 c[4], sn[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = make_float2(1.f, 1.f), sn[k] = make_float2(-0.f, -0.f);
    if (turned) {
      const long long at = static_cast<long long>(pos) * half + 8 * sub;
      load_float8(p.cos + at, c);
      load_float8(p.sin + at, sn);
    }
    // Forward: out = own * own_c + partner * other_c, the weights included
    // (first of a pair: a cos - b sin; second: b cos + a sin).  The gradient
    // turns back with c and sn as they are.
    float2 own_c[8], other_c[8];
    if constexpr (!BWD) {
      load_weight8<BF16>(op.w, p.w_fp32, ea, w);
      load_weight8<BF16>(op.w, p.w_fp32, eb, w + 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (INTER) {
          const float ck = k & 1 ? c[k / 2].y : c[k / 2].x, sk = k & 1 ? sn[k / 2].y : sn[k / 2].x;
          own_c[k] = make_float2(ck, ck);
          other_c[k] = make_float2(-sk, sk);
        } else {
          const float sg = k < 4 ? -1.f : 1.f;
          own_c[k] = c[k % 4];
          other_c[k] = make_float2(sg * sn[k % 4].x, sg * sn[k % 4].y);
        }
        own_c[k] = __fmul2_rn(own_c[k], w[k]);
        other_c[k] = __fmul2_rn(other_c[k], partner<INTER>(w, k));
        if (!turned) other_c[k] = make_float2(-0.f, -0.f);
      }
    }
#pragma unroll 1
    for (int h = 0; h < heads; ++h) {
      float2 x[8], o[8];
      if (!BWD || normed) {
        unpack8<BF16>(xv[0], x);
        unpack8<BF16>(xv[1], x + 4);
      }
      if constexpr (!BWD) {
        if (h + 1 < heads) load(xv, gv);
        if (h + 4 < heads) ahead(2);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 z = partner<INTER>(x, k);
          o[k] = __ffma2_rn(x[k], own_c[k], __fmul2_rn(turned ? z : make_float2(0.f, 0.f), other_c[k]));
        }
        if (normed) {
          const float r = rsqrtf(row_dot<LANES>(x, x) * (1.f / HD) + p.eps);
          const float2 rr = make_float2(r, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = __fmul2_rn(o[k], rr);
        }
      } else {
        // o = g, the gradient turned back
        {
          float2 y[8];
          unpack8<BF16>(gv[0], y);
          unpack8<BF16>(gv[1], y + 4);
          if (h + 1 < heads) load(xv, gv);
          if constexpr (INTER) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float ck = k & 1 ? c[k / 2].y : c[k / 2].x, sk = k & 1 ? sn[k / 2].y : sn[k / 2].x;
              const float a = turned ? y[k].x : -0.f, b = turned ? y[k].y : 0.f;
              o[k] = make_float2(y[k].x * ck + b * sk, y[k].y * ck - a * sk);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 a = turned ? y[k] : make_float2(-0.f, -0.f);
              const float2 b = turned ? y[k + 4] : make_float2(0.f, 0.f);
              o[k] = __ffma2_rn(y[k], c[k], __fmul2_rn(b, sn[k]));
              o[k + 4] = make_float2(y[k + 4].x * c[k].x - a.x * sn[k].x,
                                     y[k + 4].y * c[k].y - a.y * sn[k].y);
            }
          }
        }
        if (normed) {
          // n = x r; dn = g w; dx = r (dn - n mean(dn n))
          const float r = rsqrtf(row_dot<LANES>(x, x) * (1.f / HD) + p.eps);
          const float2 rr = make_float2(r, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[k] = __fmul2_rn(x[k], rr);
            if (live) dw[k] = __ffma2_rn(o[k], x[k], dw[k]);
            o[k] = __fmul2_rn(o[k], w[k]);
          }
          const float dot = row_dot<LANES>(o, x) * (-1.f / HD);
          const float2 dd = make_float2(dot, dot);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = __fmul2_rn(__ffma2_rn(x[k], dd, o[k]), rr);
        }
      }
      if (live) {
        *reinterpret_cast<uint4*>(y_at + ea) = pack8<BF16>(o);
        *reinterpret_cast<uint4*>(y_at + eb) = pack8<BF16>(o + 4);
      }
      y_at += yh;
    }
  }
  if constexpr (BWD) {
    if (!normed) return;
    // the CTA's sums: lanes of different tokens, then the warps in order
    __shared__ float sums[WARPS][HD];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float t = i & 1 ? dw[i / 2].y : dw[i / 2].x;
#pragma unroll
      for (int sh = LANES; sh < 32; sh <<= 1) t += __shfl_xor_sync(0xffffffffu, t, sh);
      if (lane < LANES) sums[warp][(i < 8 ? ea : eb - 8) + i] = t;
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
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const float* parts, int ctas_q,
                                                               int ctas, int d, void* dq,
                                                               void* dk, int w_fp32) {
  __shared__ float sums[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // `parts` is written now
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
