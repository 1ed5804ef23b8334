// fa_layer_api.cuh -- host side of the entry points around the attention
// itself (norm and rotation of queries and keys) and of the attention with a
// causal window and sinks; part of fa_api.cu, whose device state and checks it
// uses.
#pragma once

#include "fa_decode.cuh"
#include "fa_rope.cuh"
#include "fa_sinks_bwd_sm100.cuh"
#include "fa_sinks_fwd_sm100.cuh"

namespace {

constexpr long long kMaxElems = 1ll << 46;  // largest element offset of an operand

// Strides {batch, head, row} in elements of a [B, H, N, d] operand; nullptr:
// contiguous.  They must keep every row 16-byte aligned; the stride of a
// dimension of size 1 is not used.
struct Strides {
  long long b, h, n;
};
int read_strides(const long long* s, int B, int H, int N, int d, Strides* out) {
  *out = {(long long)H * N * d, (long long)N * d, d};
  if ((double)B * H * N * d > (double)kMaxElems) return FA_ERR_ARG;
  if (s == nullptr) return FA_OK;
  const int sizes[3] = {B, H, N};
  long long* to[3] = {&out->b, &out->h, &out->n};
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] == 1) {
      *to[i] = d;  // any valid value
      continue;
    }
    if (s[i] < d || s[i] >= 1ll << 39) return FA_ERR_ARG;  // a tensor map's limit is 2^40 bytes
    if (s[i] % 8 != 0) return FA_ERR_ALIGN;
    *to[i] = s[i];
  }
  // every element's offset must fit the index type used on the device
  long long last = d;
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] > 1 && *to[i] > kMaxElems / (sizes[i] - 1)) return FA_ERR_ARG;
    last += (sizes[i] - 1) * *to[i];
  }
  return last > kMaxElems ? FA_ERR_ARG : FA_OK;
}

struct RopeArgs {
  const void *x[2], *g[2], *w[2];
  void *y[2], *dw[2];
  const long long *xs[2], *gs[2], *ys[2];
  const float *cos, *sin;
  const int* positions;
  float* parts;
  int max_pos, weight_dtype, B, H, Hk, N, d, rot, interleaved, dtype;
  float eps;
};

template <int HD, bool BF16, bool INTER, bool PART, bool BWD>
int launch_rope(RopeParams& p, DeviceState& st, int d, cudaStream_t stream) {
  constexpr int kTokens = 32 / (HD / 16), kWarps = kRopeThreads / 32;
  const int HT = p.op[0].heads + p.op[1].heads;
  const long long groups = ((long long)p.B * p.N + kTokens - 1) / kTokens;
  p.blocks = (int)((groups + kWarps - 1) / kWarps);
  // heads a warp walks over: more of them share the loaded cos / sin, fewer
  // give a small call more warps (measured at 16384 tokens x 18 heads: 8 heads
  // 32.4 us, 4: 32.7, 16: 37)
  int hpw = 1;
  while (hpw < 8 && hpw < HT && groups * ((HT + 2 * hpw - 1) / (2 * hpw)) >= 32ll * st.sm_count)
    hpw *= 2;
  p.heads_per_warp = hpw;
  // CTAs in proportion to q's and k's items; the gradient's leave a row of
  // partial sums each
  long long ctas[2];
  for (int i = 0; i < 2; ++i) {
    p.chunks[i] = (p.op[i].heads + hpw - 1) / hpw;
    ctas[i] = (long long)p.blocks * p.chunks[i];
    if (ctas[i] > 1 << 30) return FA_ERR_ARG;
  }
  const long long wave = (long long)kRopeBwdCtas * st.sm_count;
  const long long most = !BWD ? 1 << 20 : wave < FA_NORM_ROPE_PARTS ? wave : FA_NORM_ROPE_PARTS;
  if (ctas[0] + ctas[1] > most) {
    const long long k = most * p.op[1].heads / HT;
    ctas[1] = k < 1 ? 1 : k > most - 1 ? most - 1 : k;
    ctas[0] = most - ctas[1];
  }
  p.ctas_q = (int)ctas[0];
  const int grid = (int)(ctas[0] + ctas[1]);
  qk_norm_rope_kernel<HD, BF16, INTER, PART, BWD><<<grid, kRopeThreads, 0, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  if (BWD && (p.op[0].w != nullptr || p.op[1].w != nullptr)) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(d / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, norm_weight_sum_kernel<BF16>, static_cast<const float*>(p.parts),
                           p.ctas_q, grid, d, p.op[0].dw, p.op[1].dw, p.w_fp32) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_CUDA;
    }
  }
  return FA_OK;
}

template <int HD, bool BF16, bool BWD>
int launch_rope_form(RopeParams& p, DeviceState& st, const RopeArgs& a, cudaStream_t stream) {
  if (a.rot == HD)
    return a.interleaved ? launch_rope<HD, BF16, true, false, BWD>(p, st, a.d, stream)
                         : launch_rope<HD, BF16, false, false, BWD>(p, st, a.d, stream);
  return a.interleaved ? launch_rope<HD, BF16, true, true, BWD>(p, st, a.d, stream)
                       : launch_rope<HD, BF16, false, true, BWD>(p, st, a.d, stream);
}

template <int HD, bool BWD>
int launch_rope_types(RopeParams& p, DeviceState& st, const RopeArgs& a, cudaStream_t stream) {
  return a.dtype == FA_BF16 ? launch_rope_form<HD, true, BWD>(p, st, a, stream)
                            : launch_rope_form<HD, false, BWD>(p, st, a, stream);
}

template <bool BWD>
int run_rope(const RopeArgs& a, cudaStream_t stream) {
  if (a.dtype != FA_FP16 && a.dtype != FA_BF16) return FA_ERR_DTYPE;
  if (a.d != 64 && a.d != 128 && a.d != 256) return FA_ERR_HEADDIM;
  if (a.B < 1 || a.H < 1 || a.Hk < 1 || a.N < 1 || a.max_pos < 1) return FA_ERR_ARG;
  if (a.H > 65535 || a.Hk > 65535 || (long long)a.B * a.N > 0x7fffffffLL) return FA_ERR_ARG;
  if (a.rot < 16 || a.rot > a.d || a.rot % 16 != 0) return FA_ERR_ARG;
  if (a.interleaved != 0 && a.interleaved != 1) return FA_ERR_ARG;
  if (!std::isfinite(a.eps) || a.eps < 0.f) return FA_ERR_ARG;
  if (!a.cos || !a.sin) return FA_ERR_ARG;
  if (a.positions == nullptr && a.N > a.max_pos) return FA_ERR_ARG;
  const bool normed = a.w[0] != nullptr || a.w[1] != nullptr;
  if (normed && a.weight_dtype != a.dtype && a.weight_dtype != FA_FP32) return FA_ERR_DTYPE;
  if (!aligned16(a.cos) || !aligned16(a.sin) || !aligned4(a.positions)) return FA_ERR_ALIGN;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  for (int i = 0; i < 2; ++i) {
    // without a norm the gradient does not need the input itself
    const bool needs_x = !BWD || a.w[i] != nullptr;
    if ((needs_x && !a.x[i]) || !a.y[i]) return FA_ERR_ARG;
    if (BWD && (!a.g[i] || (a.w[i] && !a.dw[i]))) return FA_ERR_ARG;
    for (const void* t : {a.x[i], a.g[i], static_cast<const void*>(a.y[i]), a.w[i]})
      if (!aligned16(t)) return FA_ERR_ALIGN;
    if (!aligned4(a.dw[i])) return FA_ERR_ALIGN;
    RopeOperand& o = p.op[i];
    o.heads = i == 0 ? a.H : a.Hk;
    Strides s;
    int rc = read_strides(a.xs[i], a.B, o.heads, a.N, a.d, &s);
    if (rc != FA_OK) return rc;
    o.xb = s.b, o.xh = s.h, o.xn = s.n;
    if ((rc = read_strides(a.ys[i], a.B, o.heads, a.N, a.d, &s)) != FA_OK) return rc;
    o.yb = s.b, o.yh = s.h, o.yn = s.n;
    if ((rc = read_strides(a.gs[i], a.B, o.heads, a.N, a.d, &s)) != FA_OK) return rc;
    o.gb = s.b, o.gh = s.h, o.gn = s.n;
    o.x = a.x[i], o.g = a.g[i], o.y = a.y[i], o.w = a.w[i], o.dw = a.w[i] ? a.dw[i] : nullptr;
  }
  if (BWD && (!a.parts || !aligned4(a.parts))) return a.parts ? FA_ERR_ALIGN : FA_ERR_ARG;
  p.cos = a.cos, p.sin = a.sin, p.positions = a.positions, p.parts = a.parts;
  p.B = a.B, p.N = a.N, p.max_pos = a.max_pos, p.rot = a.rot, p.eps = a.eps;
  p.w_fp32 = a.weight_dtype == FA_FP32;
  DeviceState* st = nullptr;
  int dev = 0;
  const int rc = device_state(&st, &dev);
  if (rc != FA_OK) return rc;
  switch (a.d) {
    case 64: return launch_rope_types<64, BWD>(p, *st, a, stream);
    case 128: return launch_rope_types<128, BWD>(p, *st, a, stream);
    default: return launch_rope_types<256, BWD>(p, *st, a, stream);
  }
}

// ------------------------------------------------ causal window and sinks

struct SinksState {
  std::atomic<bool> fwd_attr[6] = {};
  std::atomic<bool> bwd_attr[8] = {};
};
SinksState g_sinks[kMaxDevices];

// Checks of a window-and-sinks problem; brings window and sinks into the range
// the kernels use (-1: every earlier key is visible).
int check_sinks(int B, int H, int Hk, int N, int d, float* scale, int* window, int* sinks,
                int dtype) {
  if (dtype == FA_E4M3) return FA_ERR_DTYPE;
  const int rc = check_common(B, H, N, d, scale, 1, dtype);
  if (rc != FA_OK) return rc;
  if (Hk < 1 || H % Hk != 0 || N > 1 << 30) return FA_ERR_ARG;
  if (*window < -1 || *sinks < 0) return FA_ERR_ARG;
  if (*window >= N - 1) *window = -1;
  if (*window < 0) *sinks = 0;
  if (*sinks > N) *sinks = N;
  return FA_OK;
}

int check_strides(const long long* q, const long long* k, const long long* v, int B, int H, int Hk,
                  int N, int d) {
  Strides s;
  int rc = read_strides(q, B, H, N, d, &s);
  if (rc == FA_OK) rc = read_strides(k, B, Hk, N, d, &s);
  return rc == FA_OK ? read_strides(v, B, Hk, N, d, &s) : rc;
}

int encode_rows(CUtensorMap* map, const void* ptr, const long long* strides, int dtype, int d,
                int N, int H, int B, int rows) {
  Strides s;
  const int rc = read_strides(strides, B, H, N, d, &s);
  if (rc != FA_OK) return rc;
  return encode_operand(map, ptr, dtype, d, N, H, B, s.n, s.h, s.b, rows);
}

template <int HD, bool BF16>
int launch_sinks_fwd(const SinksFwdParams& p, DeviceState& st, int dev, cudaStream_t stream) {
  using C = SinksFwdCfg<HD>;
  auto kernel = sinks_fwd_kernel<HD, BF16>;
  const int slot = (HD == 64 ? 0 : HD == 128 ? 1 : 2) * 2 + (BF16 ? 1 : 0);
  const int rc = ensure_smem_attr(g_sinks[dev].fwd_attr[slot], kernel, C::SMEM_BYTES);
  if (rc != FA_OK) return rc;
  // persistent: as many CTAs as the SMs hold at once
  const int most = C::CTAS * st.sm_count;
  kernel<<<p.tiles < most ? p.tiles : most, C::THREADS, C::SMEM_BYTES, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// How the dK/dV kernel splits a sink block's query blocks: into pieces about
// as long as the other key blocks' share of a head (window + 2 blocks), at
// most 32 steps over the group's heads (measured: 68-step pieces cost a long
// sequence 7%, 16-step ones a short window 2%), and at most so many that the pieces
// of all sink blocks hold no more sums than the head has key blocks.
void sink_pieces(int N, int window, int sinks, int group, int* sink_blocks, int* pieces,
                 int* piece_blocks) {
  const int nblk = (N + 127) / 128;
  *sink_blocks = window < 0 ? 0 : (sinks + 127) / 128;
  *pieces = 1;
  *piece_blocks = nblk;
  if (*sink_blocks == 0) return;
  int share = (window + 127) / 128 + 2;
  if (share > (32 + group - 1) / group) share = (32 + group - 1) / group;
  int want = (nblk + share - 1) / share;
  if (want > nblk / *sink_blocks) want = nblk / *sink_blocks;
  if (want <= 1) return;
  *piece_blocks = (nblk + want - 1) / want;
  *pieces = (nblk + *piece_blocks - 1) / *piece_blocks;
}

// How many ways the dK/dV kernel's units (key blocks and pieces, `units` in
// all) are each split when there are few: up to one for every SM, of at least 4
// steps, or, for the balance of long ones, up to two for every SM of at least 32.
// Measured (us, d = 128, no split / one / two an SM): 4 heads on 1, causal, 2000
// rows 120 / 40 / 48, 8000 rows 460 / 248 / 206; 16 heads on 2, window 256, 600
// rows 56 / 36; at least 2 steps instead of 4: 45, 6: 34, but 2 x 8 heads on 2,
// 500 rows, d = 64: none 34, 2: 20, 4: 19, 6: 25.
int bwd_splits(int N, int window, int group, long long units, int piece_blocks, int sink_blocks) {
  constexpr int kSms = 148;
  const int nblk = (N + 127) / 128;
  int longest = window < 0 ? nblk : (window + 127) / 128 + 2;
  if (longest > nblk) longest = nblk;
  if (sink_blocks > 0 && piece_blocks > longest) longest = piece_blocks;
  const long long steps = (long long)longest * group;
  const long long one = std::min<long long>(kSms / units, steps / 4);
  const long long two = std::min<long long>(2 * kSms / units, steps / 32);
  // (the kernel counts steps times splits in 31 bits)
  const long long n = std::min(std::max(one, two), 0x7fffffffLL / steps);
  return n > 1 ? (int)n : 1;
}

// How the work of a gradient is dealt out, and its partial sums.
struct BwdShape {
  int sink_blocks, pieces, piece_blocks, splits;
  long long units, part_floats;
  BwdShape(int B, int Hk, int group, int N, int d, int window, int sinks) {
    sink_pieces(N, window, sinks, group, &sink_blocks, &pieces, &piece_blocks);
    const long long heads = (long long)B * Hk, nblk = (N + 127) / 128;
    units = heads * (sink_blocks * (long long)pieces + nblk - sink_blocks);
    splits = bwd_splits(N, window, group, units, piece_blocks, sink_blocks);
    const long long parts = splits > 1   ? units * splits
                            : pieces > 1 ? heads * sink_blocks * pieces
                                         : 0;
    part_floats = parts * 2 * 128 * d;
  }
};

// The dK/dV kernel is persistent, a CTA an SM.  The dQ kernel may start beside
// it (programmatic dependent launch), filling the SMs that the dK/dV kernel's
// few long units leave one by one; so its CTAs are short, 16 steps or one unit.
template <int HD, bool BF16, bool KV>
int launch_sinks_bwd_kernel(const SinksBwdParams& p, DeviceState& st, int dev, cudaStream_t stream) {
  using C = SinksBwdCfg<HD, KV>;
  auto kernel = sinks_bwd_kernel<HD, BF16, KV>;
  const int slot = (HD == 64 ? 0 : 4) + (BF16 ? 2 : 0) + (KV ? 1 : 0);
  const int rc = ensure_smem_attr(g_sinks[dev].bwd_attr[slot], kernel, C::SMEM_BYTES);
  if (rc != FA_OK) return rc;
  int grid = p.units < st.sm_count ? p.units : st.sm_count;
  if (!KV) {
    const int steps = p.window < 0 ? p.nblk : (p.window + 127) / 128 + 1 + p.sink_blocks;
    const int each = steps < p.nblk && steps < 16 ? 16 / steps : 1;
    grid = (p.units + each - 1) / each;
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = KV ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <int HD, bool BF16>
int launch_sinks_bwd(SinksBwdParams& p, DeviceState& st, int dev, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.H * p.N;
  constexpr long long kRowsPerBlock = 256 / (HD / 8);  // bwd_dsum_kernel: HD / 8 threads a row
  bwd_dsum_kernel<HD, BF16><<<(unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock), 256, 0,
                              stream>>>(p.o, p.dout, p.dsum, rows);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  p.units = p.B * p.Hk * (p.sink_blocks * p.pieces + p.nblk - p.sink_blocks) * p.splits;
  int rc = launch_sinks_bwd_kernel<HD, BF16, true>(p, st, dev, stream);
  if (rc != FA_OK) return rc;
  p.units = p.B * p.H * p.nblk;
  if ((rc = launch_sinks_bwd_kernel<HD, BF16, false>(p, st, dev, stream)) != FA_OK) return rc;
  if (p.pieces > 1 || p.splits > 1) {
    const long long n =
        (long long)p.B * p.Hk * (p.splits > 1 ? p.nblk : p.sink_blocks) * 2 * 128 * (HD / 4);
    sinks_sum_kernel<HD, BF16><<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

// ------------------------------------------------------ one token at a time

struct DecodeState {
  std::atomic<bool> attr[10] = {};
};
DecodeState g_decode[kMaxDevices];

template <int HD, int NT, bool BF16>
int launch_decode(DecodeParams& p, int B, DeviceState& st, int dev, cudaStream_t stream) {
  using C = DecodeCfg<HD, NT>;
  auto kernel = decode_kernel<HD, NT, BF16>;
  constexpr int slot = (HD == 64 ? 0 : HD == 128 ? 4 : 8) + (NT - 1) * 2 + (BF16 ? 1 : 0);
  std::atomic<bool>& flag = g_decode[dev].attr[slot];
  if (!flag.load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
        cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_CUDA;
    }
    const int rc = ensure_smem_attr(flag, kernel, C::SMEM_BYTES);
    if (rc != FA_OK) return rc;
  }
  p.row_tiles = (p.group + C::Q - 1) / C::Q;
  const long long tiles = (long long)B * p.Hk * p.row_tiles;
  if (tiles > 0x7fffffffLL / kDecodeMaxCluster) return FA_ERR_ARG;
  // Cluster size: two CTAs for every SM and no more (measured at 128 tiles of
  // 8192 keys: 2 CTAs a tile 78 us, 1: 84, 4: 86, 8: 85; at 32 tiles 8: 26 us,
  // 4: 28, 16: 44), and at least one step for every second warp (one tile pair
  // of 17 steps: 8 CTAs 6.0 us, 16: 6.6, 4: 6.7).
  const long long most = p.window < 0 ? p.S : (long long)p.window + 1 + p.sinks;
  const long long steps = ((most < p.S ? most : p.S) + C::KEYS - 1) / C::KEYS;
  int cl = 1;
  while (cl < kDecodeMaxCluster && tiles * 2 * cl <= 2ll * st.sm_count &&
         2 * cl * kDecodeWarps <= 2 * steps)
    cl *= 2;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(cl * tiles));
  cfg.blockDim = dim3(32 * kDecodeWarps);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  std::memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Query heads a tile holds: 8, or 16 where a key head has more than 8 (its
// keys are then read once for 16; at d = 256 the registers hold 8).
template <bool BF16>
int launch_decode_dims(DecodeParams& p, int B, int d, DeviceState& st, int dev, cudaStream_t s) {
  if (d == 256) return launch_decode<256, 1, BF16>(p, B, st, dev, s);
  if (d == 128)
    return p.group > 8 ? launch_decode<128, 2, BF16>(p, B, st, dev, s)
                       : launch_decode<128, 1, BF16>(p, B, st, dev, s);
  return p.group > 8 ? launch_decode<64, 2, BF16>(p, B, st, dev, s)
                     : launch_decode<64, 1, BF16>(p, B, st, dev, s);
}

}  // namespace

extern "C" {

int fa_decode_sinks(const void* q, const void* k, const void* v, void* o, float* lse,
                    const int* seqlens, const long long* k_strides, const long long* v_strides,
                    int B, int H, int Hk, int S, int d, int window, int sinks, float scale,
                    int dtype, struct CUstream_st* stream) {
  if (!q || !k || !v || !o || !seqlens) return FA_ERR_ARG;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_DTYPE;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_HEADDIM;
  if (B < 1 || H < 1 || Hk < 1 || S < 1 || H % Hk != 0 || S > 1 << 30) return FA_ERR_ARG;
  if (window < -1 || sinks < 0) return FA_ERR_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_ARG;
  if (scale == 0.f) scale = 1.0f / std::sqrt(static_cast<float>(d));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse) ||
      !aligned4(seqlens))
    return FA_ERR_ALIGN;
  if ((long long)B * H > 0x7fffffffLL) return FA_ERR_ARG;
  Strides ks, vs;
  int rc = read_strides(k_strides, B, Hk, S, d, &ks);
  if (rc == FA_OK) rc = read_strides(v_strides, B, Hk, S, d, &vs);
  if (rc != FA_OK) return rc;
  if ((rc = get_encode_fn()) != FA_OK) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  if ((rc = device_state(&st, &dev)) != FA_OK) return rc;
  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q, p.o = o, p.lse = lse, p.seqlens = seqlens;
  const int keys = d == 256 ? DecodeCfg<256, 1>::KEYS : DecodeCfg<128, 1>::KEYS;  // of a step
  if ((rc = encode_operand(&p.tmap_k, k, dtype, d, S, Hk, B, ks.n, ks.h, ks.b, keys)) != FA_OK ||
      (rc = encode_operand(&p.tmap_v, v, dtype, d, S, Hk, B, vs.n, vs.h, vs.b, keys)) != FA_OK)
    return rc;
  p.H = H, p.Hk = Hk, p.S = S, p.window = window, p.sinks = sinks, p.group = H / Hk;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = g_wait_limit_ns.load();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == FA_BF16 ? launch_decode_dims<true>(p, B, d, *st, dev, s)
                          : launch_decode_dims<false>(p, B, d, *st, dev, s);
}

int fa_fwd_sinks(const void* q, const void* k, const void* v, void* o, float* lse,
                 const long long* q_strides, const long long* k_strides,
                 const long long* v_strides, int B, int H, int Hk, int N, int d, int window,
                 int sinks, float scale, int dtype, struct CUstream_st* stream) {
  if (!q || !k || !v || !o) return FA_ERR_ARG;
  int rc = check_sinks(B, H, Hk, N, d, &scale, &window, &sinks, dtype);
  if (rc != FA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse))
    return FA_ERR_ALIGN;
  if ((rc = check_strides(q_strides, k_strides, v_strides, B, H, Hk, N, d)) != FA_OK) return rc;
  if ((rc = get_encode_fn()) != FA_OK) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  if ((rc = device_state(&st, &dev)) != FA_OK) return rc;
  SinksFwdParams p;
  std::memset(&p, 0, sizeof(p));
  constexpr int kKeys = SinksFwdCfg<128>::KEYS;
  if ((rc = encode_rows(&p.tmap_q, q, q_strides, dtype, d, N, H, B, 128)) != FA_OK ||
      (rc = encode_rows(&p.tmap_k, k, k_strides, dtype, d, N, Hk, B, kKeys)) != FA_OK ||
      (rc = encode_rows(&p.tmap_v, v, v_strides, dtype, d, N, Hk, B, kKeys)) != FA_OK ||
      (rc = encode_rows(&p.tmap_o, o, nullptr, dtype, d, N, H, B, 32)) != FA_OK)
    return rc;
  p.lse = lse;
  p.B = B, p.H = H, p.N = N, p.window = window, p.sinks = sinks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sink_blocks = window < 0 ? 0 : (sinks + kKeys - 1) / kKeys;
  p.qblocks = (N + 127) / 128;
  if ((long long)B * H * p.qblocks > 0x7fffffffLL) return FA_ERR_ARG;
  p.tiles = B * H * p.qblocks;
  p.div_bh = FastDiv::make((uint32_t)B * H);
  p.div_h = FastDiv::make(H);
  p.div_group = FastDiv::make(H / Hk);
  p.wait_limit_ns = g_wait_limit_ns.load();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == FA_BF16;
  switch (d) {
    case 64: return bf16 ? launch_sinks_fwd<64, true>(p, *st, dev, s) : launch_sinks_fwd<64, false>(p, *st, dev, s);
    case 128: return bf16 ? launch_sinks_fwd<128, true>(p, *st, dev, s) : launch_sinks_fwd<128, false>(p, *st, dev, s);
    default: return bf16 ? launch_sinks_fwd<256, true>(p, *st, dev, s) : launch_sinks_fwd<256, false>(p, *st, dev, s);
  }
}

long long fa_bwd_sinks_workspace(int B, int H, int Hk, int N, int d, int window, int sinks) {
  float scale = 0.f;
  int rc = check_sinks(B, H, Hk, N, d, &scale, &window, &sinks, FA_BF16);
  if (rc == FA_OK && d > 128) rc = FA_ERR_HEADDIM;
  if (rc != FA_OK) return rc;
  return BwdShape(B, Hk, H / Hk, N, d, window, sinks).part_floats + (long long)B * H * N;
}

int fa_bwd_sinks(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dout, void* dq, void* dk, void* dv, const long long* q_strides,
                 const long long* k_strides, const long long* v_strides, float* workspace, int B,
                 int H, int Hk, int N, int d, int window, int sinks, float scale, int dtype,
                 struct CUstream_st* stream) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace) return FA_ERR_ARG;
  int rc = check_sinks(B, H, Hk, N, d, &scale, &window, &sinks, dtype);
  if (rc != FA_OK) return rc;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  for (const void* t : {q, k, v, o, dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!aligned16(t)) return FA_ERR_ALIGN;
  if (!aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 31u) != 0) return FA_ERR_ALIGN;
  if ((rc = check_strides(q_strides, k_strides, v_strides, B, H, Hk, N, d)) != FA_OK) return rc;
  SinksBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.nblk = (N + 127) / 128;
  const BwdShape shape(B, Hk, H / Hk, N, d, window, sinks);
  if ((long long)B * H * p.nblk > 0x7fffffffLL || shape.units > 0x7fffffffLL) return FA_ERR_ARG;
  p.sink_blocks = shape.sink_blocks, p.pieces = shape.pieces, p.piece_blocks = shape.piece_blocks;
  p.splits = shape.splits;
  if ((rc = get_encode_fn()) != FA_OK) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  if ((rc = device_state(&st, &dev)) != FA_OK) return rc;
  if ((rc = encode_rows(&p.tmap_q, q, q_strides, dtype, d, N, H, B, 128)) != FA_OK ||
      (rc = encode_rows(&p.tmap_k, k, k_strides, dtype, d, N, Hk, B, 128)) != FA_OK ||
      (rc = encode_rows(&p.tmap_v, v, v_strides, dtype, d, N, Hk, B, 128)) != FA_OK ||
      (rc = encode_rows(&p.tmap_do, dout, nullptr, dtype, d, N, H, B, 128)) != FA_OK)
    return rc;
  p.o = o;
  p.dout = dout;
  p.lse = lse;
  p.parts = workspace;
  p.dsum = workspace + shape.part_floats;
  p.dq = dq, p.dk = dk, p.dv = dv;
  p.out_vec32 = ((reinterpret_cast<uintptr_t>(dq) | reinterpret_cast<uintptr_t>(dk) |
                  reinterpret_cast<uintptr_t>(dv)) & 31u) == 0;
  p.B = B, p.H = H, p.Hk = Hk, p.group = H / Hk, p.N = N;
  p.window = window, p.sinks = sinks;
  p.div_kv = FastDiv::make((uint32_t)B * Hk), p.div_q = FastDiv::make((uint32_t)B * H);
  p.div_hk = FastDiv::make(Hk), p.div_h = FastDiv::make(H);
  p.div_group = FastDiv::make(p.group), p.div_pieces = FastDiv::make(p.pieces);
  p.div_splits = FastDiv::make(p.splits);
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = g_wait_limit_ns.load();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == FA_BF16;
  if (d == 64)
    return bf16 ? launch_sinks_bwd<64, true>(p, *st, dev, s) : launch_sinks_bwd<64, false>(p, *st, dev, s);
  return bf16 ? launch_sinks_bwd<128, true>(p, *st, dev, s) : launch_sinks_bwd<128, false>(p, *st, dev, s);
}

int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                    const long long* q_strides, const long long* k_strides,
                    const long long* qo_strides, const long long* ko_strides, const float* cos,
                    const float* sin, const int* positions, int max_pos, const void* q_weight,
                    const void* k_weight, int weight_dtype, float eps, int B, int H, int Hk, int N,
                    int d, int rot, int interleaved, int dtype, struct CUstream_st* stream) {
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x[0] = q, a.x[1] = k, a.y[0] = q_out, a.y[1] = k_out;
  a.xs[0] = q_strides, a.xs[1] = k_strides, a.ys[0] = qo_strides, a.ys[1] = ko_strides;
  a.cos = cos, a.sin = sin, a.positions = positions, a.max_pos = max_pos;
  a.w[0] = q_weight, a.w[1] = k_weight, a.weight_dtype = weight_dtype, a.eps = eps;
  a.B = B, a.H = H, a.Hk = Hk, a.N = N, a.d = d, a.rot = rot;
  a.interleaved = interleaved, a.dtype = dtype;
  return run_rope<false>(a, reinterpret_cast<cudaStream_t>(stream));
}

int fa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                        void* dq, void* dk, void* dq_weight, void* dk_weight,
                        const long long* dqo_strides, const long long* dko_strides,
                        const long long* q_strides, const long long* k_strides, const float* cos,
                        const float* sin, const int* positions, int max_pos, const void* q_weight,
                        const void* k_weight, int weight_dtype, float eps, float* workspace, int B,
                        int H, int Hk, int N, int d, int rot, int interleaved, int dtype,
                        struct CUstream_st* stream) {
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.g[0] = dq_out, a.g[1] = dk_out, a.x[0] = q, a.x[1] = k, a.y[0] = dq, a.y[1] = dk;
  a.dw[0] = dq_weight, a.dw[1] = dk_weight, a.parts = workspace;
  a.gs[0] = dqo_strides, a.gs[1] = dko_strides, a.xs[0] = q_strides, a.xs[1] = k_strides;
  a.cos = cos, a.sin = sin, a.positions = positions, a.max_pos = max_pos;
  a.w[0] = q_weight, a.w[1] = k_weight, a.weight_dtype = weight_dtype, a.eps = eps;
  a.B = B, a.H = H, a.Hk = Hk, a.N = N, a.d = d, a.rot = rot;
  a.interleaved = interleaved, a.dtype = dtype;
  return run_rope<true>(a, reinterpret_cast<cudaStream_t>(stream));
}

int fa_rope_table(float* cos, float* sin, int max_pos, int rot, double base, int scaling,
                  double factor, int original_max_pos, struct CUstream_st* stream) {
  if (!cos || !sin || max_pos < 1) return FA_ERR_ARG;
  if (rot < 16 || rot > 256 || rot % 16 != 0) return FA_ERR_ARG;
  if (!std::isfinite(base) || !(base > 1.0)) return FA_ERR_ARG;
  if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_YARN) return FA_ERR_ARG;
  if (scaling != FA_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return FA_ERR_ARG;
  if (scaling == FA_ROPE_YARN && original_max_pos < 1) return FA_ERR_ARG;
  if (!aligned16(cos) || !aligned16(sin)) return FA_ERR_ALIGN;
  DeviceState* st = nullptr;
  int dev = 0;
  const int rc = device_state(&st, &dev);
  if (rc != FA_OK) return rc;
  RopeTableParams p;
  std::memset(&p, 0, sizeof(p));
  p.cos = cos, p.sin = sin, p.max_pos = max_pos, p.half = rot / 2, p.factor = 1.0;
  if (scaling == FA_ROPE_NTK) base *= std::pow(factor, rot / (rot - 2.0));
  // yarn: the pair whose wavelength fits original_max_pos `turns` times
  const double two_pi = 6.283185307179586;
  double low = 0.0, high = 1.0;
  if (scaling == FA_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return rot * std::log(original_max_pos / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_of(32.0)), 0.0);
    high = std::fmin(std::ceil(pair_of(1.0)), rot - 1.0);
    if (high <= low) high = low + 0.001;
    p.factor = 0.1 * std::log(factor) + 1.0;
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == FA_ROPE_LINEAR) f /= factor;
    if (scaling == FA_ROPE_YARN) {
      // fast pairs keep their frequency, slow ones are interpolated
      const double slow = std::fmin(std::fmax((i - low) / (high - low), 0.0), 1.0);
      f = f / factor * slow + f * (1.0 - slow);
    }
    p.inv_freq[i] = f;
  }
  const long long blocks = ((long long)max_pos * p.half + 255) / 256;
  const int grid = (int)(blocks < 16ll * st->sm_count ? blocks : 16ll * st->sm_count);
  rope_table_kernel<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
