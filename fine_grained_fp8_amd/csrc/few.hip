// Products for a few tokens on gfx950: the whole mixture-of-experts layer for
// up to 64 tokens, and the projection with low-rank adapters in its form for
// up to 64 tokens (plus the adapters' two small products for any number).
//
// With so few rows every weight byte is used for a handful of products: the
// kernels are bound by reading the weights once from HBM, so they are laid
// out for that.  A workgroup owns 16 output rows (one operand tile row) and
// all its columns' tokens; its eight waves split the K blocks, each wave
// loading whole 2 KB operand tiles (16 bytes a lane) straight into MFMA
// operand registers; the partial sums meet in LDS.  The weight rows are the
// MFMA's "A" rows, the tokens its 16 columns: a lane ends with 4 consecutive
// outputs of one token.
#include "device.hpp"
#include "layers.hpp"

namespace fp8bs {

namespace {

typedef int fv4i __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kB = 512;         // threads of the streaming kernels
constexpr int kW = kB / 64;     // and their waves
constexpr int kPB = 1024;       // threads of the kernels that prepare and combine
constexpr int kPW = kPB / 64;
// 16-row tiles from which on a workgroup takes two of them
constexpr int64_t kWideTiles = 1024;

__device__ __forceinline__ v8bf as_bf16x8(const fv4i& v) { return __builtin_bit_cast(v8bf, v); }

// 8 E4M3 codes (two dwords) as BF16, exactly
__device__ __forceinline__ v8bf codes_to_bf16(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One 128-wide K block of a 16-row operand: a lane's 32 codes (bytes 16 g.. and
// 64 + 16 g.. of the block for lane group g), as the framework's tiles and
// its FP8 MFMA order them.
struct Block {
  fv4i lo, hi;
};
__device__ __forceinline__ Block load_tile(const uint8_t* tile, int lane) {
  return Block{*reinterpret_cast<const fv4i*>(tile + lane * 16), *reinterpret_cast<const fv4i*>(tile + 1024 + lane * 16)};
}
// the same of a token's row-major codes
__device__ __forceinline__ Block load_row(const uint8_t* row, int lgrp) {
  return Block{*reinterpret_cast<const fv4i*>(row + lgrp * 16), *reinterpret_cast<const fv4i*>(row + 64 + lgrp * 16)};
}
__device__ __forceinline__ v8i as_operand(const Block& b) {
  return v8i{b.lo[0], b.lo[1], b.lo[2], b.lo[3], b.hi[0], b.hi[1], b.hi[2], b.hi[3]};
}
struct Bf16Block {
  v8bf f[4];
};
__device__ __forceinline__ Bf16Block to_bf16(const Block& b) {
  return Bf16Block{{codes_to_bf16(b.lo[0], b.lo[1]), codes_to_bf16(b.lo[2], b.lo[3]),
                    codes_to_bf16(b.hi[0], b.hi[1]), codes_to_bf16(b.hi[2], b.hi[3])}};
}
// partial sums of one K block with exact products and FP32 additions
__device__ __forceinline__ v4f block_product(const Bf16Block& a, const Bf16Block& b) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(a.f[i], b.f[i], c);
  return c;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Selection order of routing values: larger first, NaN last, equal values by
// index.  Keys are never 0 for an index below 2^32 - 1.
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 counts as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(float v, int index) {
  return ((uint64_t)order_bits(v) << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)index);
}

// Dot products of 16 BF16 rows (row l & 15 of the lane at `a`, 16-byte
// aligned) with 16 BF16 token rows (at `b`), K % 128 == 0, the K blocks
// dealt to the workgroup's kPW waves in turn; this wave's partial sums.  Two
// blocks' loads are in flight at a time: one round trip to memory takes longer
// than all the arithmetic.
__device__ __forceinline__ v4f dot_rows_bf16(const uint16_t* a, const uint16_t* b, int K, int wave, int lgrp) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
  const int kb_n = K / 128;
  for (int kb = wave; kb < kb_n; kb += 2 * kPW) {
    const bool two = kb + kPW < kb_n;
    fv4i va[2][4], vb[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !two) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        va[h][i] = *reinterpret_cast<const fv4i*>(a + (kb + h * kPW) * 128 + i * 32 + lgrp * 8);
        vb[h][i] = *reinterpret_cast<const fv4i*>(b + (kb + h * kPW) * 128 + i * 32 + lgrp * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(as_bf16x8(va[0][i]), as_bf16x8(vb[0][i]), c);
    if (two) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(as_bf16x8(va[1][i]), as_bf16x8(vb[1][i]), c);
    }
  }
  return c;
}

// 1x128 quantization of token rows: 64 tiles a workgroup, 16 lanes each.
__device__ __forceinline__ void quant_tokens(const uint16_t* x, int64_t ldx, int T, int K, int block, uint8_t* xq,
                                             float* xs) {
  const int kb_n = K / 128;
  const int tile = block * (kPB / 16) + (threadIdx.x >> 4);
  if (tile >= T * kb_n) return;   // whole 16-lane groups
  const int t = tile / kb_n, kb = tile - t * kb_n, l16 = threadIdx.x & 15;
  const fv4i d = *reinterpret_cast<const fv4i*>(x + t * ldx + kb * 128 + l16 * 8);
  float s;
  const uint2 q = quant8_bf16(make_uint4((uint32_t)d[0], (uint32_t)d[1], (uint32_t)d[2], (uint32_t)d[3]), s);
  *reinterpret_cast<uint2*>(xq + (int64_t)t * K + kb * 128 + l16 * 8) = q;
  if (l16 == 0) xs[t * kb_n + kb] = s;
}
int quant_blocks(int64_t T, int64_t K) { return (int)((T * (K / 128) + kPB / 16 - 1) / (kPB / 16)); }

__device__ __forceinline__ void store_out(void* y, int64_t at, int fp32, float v) {
  if (fp32) static_cast<float*>(y)[at] = v;
  else static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ===========================================================================
// Mixture of experts for up to 64 tokens, four launches.
// ===========================================================================

// 1. Router logits and the values experts are chosen by (16 experts x 16 tokens
//    a workgroup), and the 1x128 quantization of x.
__global__ __launch_bounds__(kPB) void moe_prepare_kernel(MoeProblem p, int router_blocks) {
  if ((int)blockIdx.x >= router_blocks) {
    quant_tokens(p.x, p.ldx, p.T, p.H, blockIdx.x - router_blocks, p.xq, p.xs);
    return;
  }
  __shared__ v4f part[kPW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const int e_tiles = (p.E + 15) / 16;
  const int e0 = (blockIdx.x % e_tiles) * 16, t0 = (blockIdx.x / e_tiles) * 16;
  const int e = e0 + lrow < p.E ? e0 + lrow : p.E - 1;
  const int t = t0 + lrow < p.T ? t0 + lrow : p.T - 1;
  part[wave][lane] = dot_rows_bf16(p.router + e * p.ld_r, p.x + t * p.ldx, p.H, wave, lgrp);
  __syncthreads();
  if (wave == 0) {
    v4f c = part[0][lane];
#pragma unroll
    for (int w = 1; w < kPW; ++w) c += part[w][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int ee = e0 + lgrp * 4 + v;
      if (ee < p.E && t0 + lrow < p.T) {
        const int at = (t0 + lrow) * p.E + ee;
        p.logits[at] = c[v];
        if (p.bias) p.value[at] = sigmoid(c[v]) + p.bias[ee];   // otherwise value is logits
      }
    }
  }
}

// One wave: the chosen experts of token t, best first, with their gates.
// Lane l holds experts l, l + 64, ...
__device__ __forceinline__ void route_token(const MoeProblem& p, int t, int lane) {
  constexpr int kMost = kMoeMaxExperts / 64;
  float l[kMost];
  uint64_t key[kMost];
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    const int e = c * 64 + lane;
    const bool in = c * 64 < p.E && e < p.E;
    l[c] = in ? p.logits[t * p.E + e] : -INFINITY;
    key[c] = in ? order_key(p.value[t * p.E + e], e) : 0;
  }
  float m = -INFINITY, sum = 1.0f;
  if (!p.sigmoid) {
#pragma unroll
    for (int c = 0; c < kMost; ++c) m = fmaxf(m, l[c]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < kMost; ++c)
      if (c * 64 < p.E) sum += c * 64 + lane < p.E ? expf(l[c] - m) : 0.f;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  }
  uint64_t below = ~0ull;         // keys at or above it are taken
  float my_score = 0.f, total = 0.f;
  int my_expert = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
    float lb = 0.f;
#pragma unroll
    for (int c = 0; c < kMost; ++c)
      if (c * 64 < p.E && key[c] < below && key[c] > best) {
        best = key[c];
        lb = l[c];
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t o = __shfl_xor(best, d);
      const float ol = __shfl_xor(lb, d);
      if (o > best) {
        best = o;
        lb = ol;
      }
    }
    below = best;
    const float score = p.sigmoid ? sigmoid(lb) : expf(lb - m) / sum;
    total += score;
    if (lane == j) {
      my_score = score;
      my_expert = (int)(0xFFFFFFFFu - (uint32_t)best);
    }
  }
  if (lane < p.top_k) {
    p.slot_expert[t * p.top_k + lane] = my_expert;
    p.slot_gate[t * p.top_k + lane] = (p.normalize ? my_score / total : my_score) * p.gate_scale;
  }
}

// One K block of the up kernel as loaded: the gate tile, the up tile, 16
// tokens' codes and their scales.
struct UpLoads {
  Block g, u, x;
  float sx, fg, fu;
};

// The sums of one 16-channel tile for n <= 16 NT listed tokens, this wave's
// share of the K blocks.  The next block's loads are issued before the
// present one's products (the weights alone for more than 16 tokens: a second
// set of token operands would spill).
template <int NT>
__device__ __forceinline__ void up_sums(const MoeProblem& p, int el, int tile, const int* list_t, int n, int wave,
                                        int lane, v4f (&ag)[NT], v4f (&au)[NT]) {
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int kb_n = p.H / 128;
  const uint8_t* wg = p.w13 + (int64_t)el * 2 * p.I * p.H + (int64_t)tile * kb_n * 2048;
  const uint8_t* wu = wg + (int64_t)p.I * p.H;
  const float* sg = p.s13 + ((int64_t)el * 2 * (p.I / 128) + tile / 8) * kb_n;
  const float* su = sg + (int64_t)(p.I / 128) * kb_n;
  int tok[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int c = j * 16 + lrow;
    tok[j] = list_t[c < n ? c : 0];
    ag[j] = au[j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  auto fetch = [&](int kb, UpLoads& f) {
    f.g = load_tile(wg + (int64_t)kb * 2048, lane);
    f.u = load_tile(wu + (int64_t)kb * 2048, lane);
    if constexpr (NT == 1) {
      f.x = load_row(p.xq + (int64_t)tok[0] * p.H + kb * 128, lgrp);
      f.sx = p.xs[tok[0] * kb_n + kb];
    }
    f.fg = sg[kb];
    f.fu = su[kb];
  };
  auto products = [&](int kb, const UpLoads& f) {
    const Bf16Block g16 = to_bf16(f.g), u16 = to_bf16(f.u);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 16 < n) {
        Block xb = f.x;
        float sx = f.sx;
        if constexpr (NT > 1) {
          xb = load_row(p.xq + (int64_t)tok[j] * p.H + kb * 128, lgrp);
          sx = p.xs[tok[j] * kb_n + kb];
        }
        const Bf16Block b = to_bf16(xb);
        const v4f pg = block_product(g16, b), pu = block_product(u16, b);
        const float cg = sx * f.fg, cu = sx * f.fu;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          ag[j][v] = __builtin_fmaf(pg[v], cg, ag[j][v]);
          au[j][v] = __builtin_fmaf(pu[v], cu, au[j][v]);
        }
      }
    }
  };
  int kb = wave;
  if (kb >= kb_n) return;
  UpLoads f0{}, f1{};
  fetch(kb, f0);
  for (;;) {
    const bool two = kb + kW < kb_n, three = kb + 2 * kW < kb_n;
    if (two) fetch(kb + kW, f1);
    products(kb, f0);
    if (!two) break;
    if (three) fetch(kb + 2 * kW, f0);
    products(kb + kW, f1);
    if (!three) break;
    kb += 2 * kW;
  }
}

// 2. Routing (the first blocks, a wave per token), and h = silu(W1 x) (W3 x)
//    for the tokens that chose a held expert: workgroup (expert, 16 channels)
//    with the gate rows and the up rows of the same channels.  A workgroup
//    finds its expert's tokens itself: a token chose expert e if fewer than
//    top_k experts come before e, and that count is e's slot (one round trip
//    for all tokens, with no launch between routing and products).  The
//    products convert the codes to BF16: exact, with FP32 sums, because h is
//    quantized again and the FP8 instruction's truncation would move codes.
__global__ __launch_bounds__(kB, 4) void moe_up_kernel(MoeProblem p, int route_blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  if ((int)blockIdx.x < route_blocks) {
    const int t = blockIdx.x * kW + wave;
    if (t < p.T) route_token(p, t, lane);
    return;
  }
  __shared__ v4f part[kW][2][64];
  __shared__ int slot_of[kMoeMaxTokens];     // the expert's slot of each token, or -1
  __shared__ int list_t[kMoeMaxTokens], list_slot[kMoeMaxTokens], count;
  const int tiles = p.I / 16;
  const int el = (blockIdx.x - route_blocks) / tiles, tile = (blockIdx.x - route_blocks) % tiles;
  const int e = p.first + el;
  {
    constexpr int kPer = kMoeMaxTokens / kW;   // tokens of a wave
    uint64_t mine[kPer];
    int before[kPer];
    float own[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = wave + i * kW;
      own[i] = t < p.T ? p.value[t * p.E + e] : 0.f;
      before[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine[i] = order_key(own[i], e);
    for (int c = 0; c < p.E; c += 64) {
      float v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = wave + i * kW;
        v[i] = t < p.T && c + lane < p.E ? p.value[t * p.E + c + lane] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        before[i] += __popcll(__ballot(c + lane < p.E && order_key(v[i], c + lane) > mine[i]));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int t = wave + i * kW;
      if (lane == 0) slot_of[t] = t < p.T && before[i] < p.top_k ? before[i] : -1;
    }
  }
  __syncthreads();
  if (wave == 0) {
    const int s = slot_of[lane];
    const uint64_t mask = __ballot(s >= 0);
    const int at = __popcll(mask & ((1ull << lane) - 1));
    if (s >= 0) {
      list_t[at] = lane;
      list_slot[at] = lane * p.top_k + s;
    }
    if (lane == 0) count = __popcll(mask);
    if (tile == 0) {   // for the down kernel
      if (lane == 0) p.counts[el] = __popcll(mask);
      if (s >= 0) p.lists[el * kMoeMaxTokens + at] = lane * p.top_k + s;
    }
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;

  // column group j of the sums: a lane has 4 channels of one token
  auto finish = [&](int j, const v4f& ag, const v4f& au) {
    if (j > 0) __syncthreads();
    part[wave][0][lane] = ag;
    part[wave][1][lane] = au;
    __syncthreads();
    if (wave != 0) return;
    v4f a = part[0][0][lane], u = part[0][1][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) {
      a += part[w][0][lane];
      u += part[w][1][lane];
    }
    if (j * 16 + lrow < n) {
      float4 h;
      h.x = a[0] * sigmoid(a[0]) * u[0];
      h.y = a[1] * sigmoid(a[1]) * u[1];
      h.z = a[2] * sigmoid(a[2]) * u[2];
      h.w = a[3] * sigmoid(a[3]) * u[3];
      *reinterpret_cast<float4*>(p.h + (int64_t)list_slot[j * 16 + lrow] * p.I + tile * 16 + lgrp * 4) = h;
    }
  };
  if (n <= 16) {
    v4f ag[1], au[1];
    up_sums<1>(p, el, tile, list_t, n, wave, lane, ag, au);
    finish(0, ag[0], au[0]);
  } else if (n <= 32) {
    v4f ag[2], au[2];
    up_sums<2>(p, el, tile, list_t, n, wave, lane, ag, au);
#pragma unroll
    for (int j = 0; j < 2; ++j) finish(j, ag[j], au[j]);
  } else {
    v4f ag[4], au[4];
    up_sums<4>(p, el, tile, list_t, n, wave, lane, ag, au);
#pragma unroll
    for (int j = 0; j < 4; ++j) finish(j, ag[j], au[j]);
  }
}

// 3. The 1x128 quantization of h (FP32 in): a tile spans eight workgroups of
//    the up kernel, so it waits for the next launch.
__global__ __launch_bounds__(kPB) void moe_quant_kernel(MoeProblem p) {
  const int kb_n = p.I / 128;
  const int tile = blockIdx.x * (kPB / 16) + (threadIdx.x >> 4), l16 = threadIdx.x & 15;
  if (tile >= p.T * p.top_k * kb_n) return;
  const int slot = tile / kb_n, kb = tile - slot * kb_n;
  const int el = p.slot_expert[slot] - p.first;
  if (el < 0 || el >= p.local) return;   // h of that slot was not computed
  const float* src = p.h + (int64_t)slot * p.I + kb * 128 + l16 * 8;
  const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
  const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(y[k]) & 0x7FFFFFFFu);
  float s;
  const uint2 q = quant8_f32(y, row16_max_u32(m), s);
  *reinterpret_cast<uint2*>(p.hq + (int64_t)slot * p.I + kb * 128 + l16 * 8) = q;
  if (l16 == 0) p.hs[slot * kb_n + kb] = s;
}

// 4. y: a workgroup has 16 output channels of every token.  The (expert, K
//    block) units are dealt to the waves in equal runs; a wave adds gate x its
//    sums into its own copy of the outputs in LDS when its expert ends, and
//    the copies are summed in wave order at the end, so that the result does
//    not depend on timing.  The next unit's weights are loaded before the
//    present one's products, across experts too.
template <int NT>
__global__ __launch_bounds__(kPB) void moe_down_kernel(MoeProblem p) {
  __shared__ float out[kPW][NT * 16][16 + 4];
  __shared__ int slots[kMoeMaxTokens * kMoeMaxTopK];    // the chosen slots, expert by expert
  __shared__ int16_t active[kMoeMaxExperts];            // chosen held experts
  __shared__ int16_t start[kMoeMaxExperts + 1];         // the first of each one's slots
  __shared__ int n_active;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  for (int i = threadIdx.x; i < kPW * NT * 16 * 20; i += kPB) (&out[0][0][0])[i] = 0.f;
  if (wave == 0) {
    int na = 0, ns = 0;
    for (int c = 0; c < p.local; c += 64) {
      const int cnt = c + lane < p.local ? p.counts[c + lane] : 0;
      int incl = cnt;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
      }
      const uint64_t mask = __ballot(cnt > 0);
      const int at = na + __popcll(mask & ((1ull << lane) - 1));
      if (cnt > 0) {
        active[at] = (int16_t)(c + lane);
        start[at] = (int16_t)(ns + incl - cnt);
      }
      na += __popcll(mask);
      ns += __shfl(incl, 63);
    }
    if (lane == 0) {
      n_active = na;
      start[na] = (int16_t)ns;
    }
  }
  __syncthreads();
  const int na = n_active;
  for (int a = wave; a < na; a += kPW) {
    const int n = start[a + 1] - start[a];
    if (lane < n) slots[start[a] + lane] = p.lists[active[a] * kMoeMaxTokens + lane];
  }
  __syncthreads();

  const int tile = blockIdx.x, kb_n = p.I / 128;
  const int units = na * kb_n;
  const int u0 = (int)((int64_t)units * wave / kPW), u1 = (int)((int64_t)units * (wave + 1) / kPW);
  if (u0 < u1) {
    int a = u0 / kb_n, kb = u0 - a * kb_n;      // the unit at hand
    int na_ = a, nkb = kb;                      // the unit being fetched
    auto advance = [&](int& ea, int& ek) {
      if (++ek == kb_n) {
        ek = 0;
        ++ea;
      }
    };
    Block w0, w1;
    float f0, f1;
    auto fetch = [&](Block& w, float& f) {
      const int el = active[na_];
      w = load_tile(p.w2 + ((int64_t)el * (p.H / 16) + tile) * kb_n * 2048 + (int64_t)nkb * 2048, lane);
      f = p.s2[((int64_t)el * (p.H / 128) + tile / 8) * kb_n + nkb];
    };
    int n = 0, slot[NT];
    v4f acc[NT];
    auto begin = [&]() {
      const int s0 = start[a];
      n = start[a + 1] - s0;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = j * 16 + lrow;
        slot[j] = slots[s0 + (c < n ? c : 0)];
        acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    };
    auto flush = [&]() {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j * 16 + lrow < n) {
          const float g = p.slot_gate[slot[j]];
          float4* o = reinterpret_cast<float4*>(&out[wave][slot[j] / p.top_k][lgrp * 4]);
          float4 v = *o;
          v.x = __builtin_fmaf(acc[j][0], g, v.x);
          v.y = __builtin_fmaf(acc[j][1], g, v.y);
          v.z = __builtin_fmaf(acc[j][2], g, v.z);
          v.w = __builtin_fmaf(acc[j][3], g, v.w);
          *o = v;
        }
      }
    };
    auto unit = [&](const Block& w, float f) {
      const v8i wa = as_operand(w);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j * 16 < n) {
          const v8i b = as_operand(load_row(p.hq + (int64_t)slot[j] * p.I + kb * 128, lgrp));
          const float c = p.hs[slot[j] * kb_n + kb] * f;
          const v4f zero = {0.f, 0.f, 0.f, 0.f};
          const v4f q = mfma_e4m3_16x16x128(wa, b, zero);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(q[v], c, acc[j][v]);
        }
      }
    };
    auto step = [&](const Block& w, float f, bool last) {
      unit(w, f);
      advance(a, kb);
      if (last || kb == 0) {
        flush();
        if (!last) begin();
      }
    };
    begin();
    fetch(w0, f0);
    for (int u = u0; u < u1; u += 2) {
      const bool more = u + 1 < u1;
      if (more) {
        advance(na_, nkb);
        fetch(w1, f1);
      }
      step(w0, f0, !more);
      if (!more) break;
      if (u + 2 < u1) {
        advance(na_, nkb);
        fetch(w0, f0);
      }
      step(w1, f1, u + 2 >= u1);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * 16; i += kPB) {
    const int t = i >> 4, c = i & 15;
    float v = out[0][t][c];
#pragma unroll
    for (int w = 1; w < kPW; ++w) v += out[w][t][c];
    store_out(p.y, t * p.ldy + tile * 16 + c, p.y_fp32, v);
  }
}

// ===========================================================================
// Low-rank adapters beside a shared projection.
// ===========================================================================

// z[t] = scale_a (A_a x_t) goes to memory as the expand's products take it:
// for every 8 ranks the 8 BF16 terms hi, then the 8 BF16 terms lo of z = hi +
// lo (to 2^-17 of z), so it is split once here and not by every reader.
__device__ __forceinline__ void store_z(uint16_t* zrow, int r0, const v4f& c, float s) {
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  v4bf hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float z = c[i] * s;
    hi[i] = (__bf16)z;
    const float d = z - (float)hi[i];
    lo[i] = (__bf16)(d == d ? d : 0.f);   // Inf and NaN sit in hi
  }
  uint16_t* at = zrow + (r0 >> 3) * 16 + (r0 & 7);
  *reinterpret_cast<v4bf*>(at) = hi;
  *reinterpret_cast<v4bf*>(at + 8) = lo;
}

// The ids of a chunk of 16 tokens (in every 16-lane group; -1 past the last
// token) and which of them have an adapter.
__device__ __forceinline__ uint32_t chunk_ids(const AdapterProblem& p, int64_t t0, int lrow, int& id) {
  id = t0 + lrow < p.T ? p.ids[t0 + lrow] : -1;
  return (uint32_t)(__ballot(id >= 0) & 0xFFFFull);
}

// z of the chunk's tokens with adapter a, 16 rows of A: every wave's partial
// sums meet in LDS.  An id past the last adapter gives NaN.
__device__ __forceinline__ void shrink_rows(const AdapterProblem& p, int64_t t0, int rt, int a, int id,
                                            v4f (*part)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const int row = rt * 16 + lrow < p.r ? rt * 16 + lrow : p.r - 1;
  const uint16_t* xr = p.x + (t0 + lrow < p.T ? t0 + lrow : t0) * p.ldx;
  v4f c = {NAN, NAN, NAN, NAN};
  if (a < p.n) c = dot_rows_bf16(p.A + ((int64_t)a * p.r + row) * p.K, xr, (int)p.K, wave, lgrp);
  __syncthreads();
  part[wave][lane] = c;
  __syncthreads();
  const int r0 = rt * 16 + lgrp * 4;
  if (wave == 0 && id == a && r0 < p.r) {
    c = part[0][lane];
#pragma unroll
    for (int w = 1; w < kPW; ++w) c += part[w][lane];
    store_z(p.z + (t0 + lrow) * 2 * p.r, r0, c, p.scales != nullptr && a < p.n ? p.scales[a] : 1.0f);
  }
}

// 1. Few tokens: the quantization of x, and the shrink: workgroup (chunk of 16
//    tokens, 16 rows of A, one of `step` shares of the chunk's adapters, which
//    are taken in the order of their first token).
__global__ __launch_bounds__(kPB) void adapter_prepare_kernel(AdapterProblem p, int shrink_blocks, int step) {
  __shared__ v4f part[kPW][64];
  const int b = blockIdx.x;
  if (b >= shrink_blocks) {
    quant_tokens(p.x, p.ldx, (int)p.T, (int)p.K, b - shrink_blocks, p.xq, p.xs);
    return;
  }
  const int rts = (p.r + 15) / 16;
  const int first = b % step, rt = (b / step) % rts;
  const int64_t t0 = (int64_t)(b / (step * rts)) * 16;
  int id;
  uint32_t left = chunk_ids(p, t0, threadIdx.x & 15, id);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __shfl(id, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(id == a);
    if (turn % step == first) shrink_rows(p, t0, rt, a, id, part);
  }
}

// Prompts: the quantization of x (codes and MN-major scales as the row
// quantizer writes them) and the shrink in one pass over x: a workgroup has 16
// tokens, its waves deal the K blocks.  A lane holds 32 values of one token's
// 1x128 tile, which are both the quantizer's input and the products' operand.
// The tokens of the chunk's first adapter get their products in that pass;
// further adapters in the chunk take another over x (from L2).
template <int RT>
__global__ __launch_bounds__(kPB) void adapter_prompt_kernel(AdapterProblem p, int64_t ld_s) {
  __shared__ v4f part[RT][kPW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16, t = t0 + lrow;
  const bool in = t < p.T;
  int id;
  uint32_t left = chunk_ids(p, t0, lrow, id);
  const int lead = left != 0 ? __shfl(id, __builtin_ctz(left)) : -1;
  const bool dot = lead >= 0 && lead < p.n;
  const uint16_t* xr = p.x + (in ? t : t0) * p.ldx + lgrp * 8;
  const uint16_t* ar[RT];
  v4f acc[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = rt * 16 + lrow < p.r ? rt * 16 + lrow : p.r - 1;
    ar[rt] = p.A + ((int64_t)(dot ? lead : 0) * p.r + row) * p.K + lgrp * 8;
    acc[rt] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  const int kb_n = (int)(p.K / 128);
  for (int kb = wave; kb < kb_n; kb += kPW) {
    fv4i x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const fv4i*>(xr + kb * 128 + i * 32);
    if (dot) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        fv4i a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const fv4i*>(ar[rt] + kb * 128 + i * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[rt] = mfma_bf16_16x16x32(as_bf16x8(a[i]), as_bf16x8(x[i]), acc[rt]);
      }
    }
    uint32_t m = 0;
    uint4 d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d[i] = make_uint4((uint32_t)x[i][0], (uint32_t)x[i][1], (uint32_t)x[i][2], (uint32_t)x[i][3]);
      m = max(m, absmax_bits8(d[i]));
    }
    const auto h = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(h[0], h[1]);
    const auto f = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max(f[0], f[1]);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 q = quant8_bf16_tile(d[i], m, s);
      if (in) *reinterpret_cast<uint2*>(p.xq + t * p.K + kb * 128 + i * 32 + lgrp * 8) = q;
    }
    if (in && lgrp == 0) p.xs[kb * ld_s + t] = s;
  }
  if (left == 0) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) part[rt][wave][lane] = acc[rt];
  __syncthreads();
  for (int rt = wave; rt < RT; rt += kPW) {
    const int r0 = rt * 16 + lgrp * 4;
    if (id == lead && r0 < p.r) {
      v4f c = part[rt][0][lane];
#pragma unroll
      for (int w = 1; w < kPW; ++w) c += part[rt][w][lane];
      if (!dot) c = v4f{NAN, NAN, NAN, NAN};
      store_z(p.z + t * 2 * p.r, r0, c, p.scales != nullptr && dot ? p.scales[lead] : 1.0f);
    }
  }
  left &= ~(uint32_t)__ballot(id == lead);
  while (left != 0) {
    const int a = __shfl(id, __builtin_ctz(left));
    left &= ~(uint32_t)__ballot(id == a);
    for (int rt = 0; rt < (p.r + 15) / 16; ++rt) shrink_rows(p, t0, rt, a, id, part[0]);
  }
}

// 2. Few tokens: projection and expand, 16 RT output columns a workgroup; the
//    next K block's weights are loaded before the present one's products.
template <int NT, int RT>
__global__ __launch_bounds__(kB, (NT > 2 && RT > 1) ? 2 : 4) void adapter_project_kernel(AdapterProblem p) {
  __shared__ v4f part[kW][RT][NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const int tile = blockIdx.x * RT, kb_n = (int)(p.K / 128), T = (int)p.T;
  const uint8_t* w = p.W + (int64_t)tile * kb_n * 2048;
  const float* sw = p.sW + (tile / 8) * p.ld_sw;      // RT divides 8: one block row
  int tok[NT];
  v4f acc[RT][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    tok[j] = j * 16 + lrow < T ? j * 16 + lrow : T - 1;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  auto fetch = [&](int kb, Block (&a)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) a[i] = load_tile(w + ((int64_t)i * kb_n + kb) * 2048, lane);
  };
  auto products = [&](int kb, const Block (&a)[RT]) {
    const float f = sw[kb];
    Block b[NT];
    float c[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      b[j] = load_row(p.xq + tok[j] * p.K + kb * 128, lgrp);
      c[j] = p.xs[tok[j] * kb_n + kb] * f;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const v8i bj = as_operand(b[j]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const v4f zero = {0.f, 0.f, 0.f, 0.f};
        const v4f q = mfma_e4m3_16x16x128(as_operand(a[i]), bj, zero);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(q[v], c[j], acc[i][j][v]);
      }
    }
  };
  Block a0[RT], a1[RT];
  if (wave < kb_n) fetch(wave, a0);
  // the adapters of the batch, dealt to the waves in the order of their first
  // token; the rows of other adapters enter as zero columns
  const int id = lane < T ? p.ids[lane] : -1;
  uint64_t left = __ballot(id >= 0);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __shfl(id, __builtin_ctzll(left));
    const uint64_t members = __ballot(id == a);
    left &= ~members;
    if (turn % kW != wave) continue;
    const uint16_t* brow = p.B + ((int64_t)(a < p.n ? a : 0) * p.N + tile * 16 + lrow) * p.r;
    for (int r0 = 0; r0 < p.r; r0 += 32) {
      const int r = r0 + lgrp * 8;
      const fv4i none = {0, 0, 0, 0};
      fv4i bw[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i)
        bw[i] = r < p.r ? *reinterpret_cast<const fv4i*>(brow + (int64_t)i * 16 * p.r + r) : none;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t m = (uint32_t)(members >> (16 * j)) & 0xFFFFu;
        if (m == 0) continue;
        const bool on = ((m >> lrow) & 1) && r < p.r;
        const uint16_t* z = p.z + (int64_t)tok[j] * 2 * p.r + 2 * r;
        const fv4i hi = on ? *reinterpret_cast<const fv4i*>(z) : none;
        const fv4i lo = on ? *reinterpret_cast<const fv4i*>(z + 8) : none;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          acc[i][j] = mfma_bf16_16x16x32(as_bf16x8(bw[i]), as_bf16x8(hi), acc[i][j]);
          acc[i][j] = mfma_bf16_16x16x32(as_bf16x8(bw[i]), as_bf16x8(lo), acc[i][j]);
        }
      }
    }
  }
  for (int kb = wave; kb < kb_n; kb += 2 * kW) {
    const bool two = kb + kW < kb_n;
    if (two) fetch(kb + kW, a1);
    products(kb, a0);
    if (!two) break;
    if (kb + 2 * kW < kb_n) fetch(kb + 2 * kW, a0);
    products(kb + kW, a1);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  for (int ij = wave; ij < RT * NT; ij += kW) {
    const int i = ij / NT, j = ij % NT;
    v4f c = part[0][i][j][lane];
#pragma unroll
    for (int q = 1; q < kW; ++q) c += part[q][i][j][lane];
    if (j * 16 + lrow < T) {
      const int64_t at = (j * 16 + lrow) * p.ldc + (tile + i) * 16 + lgrp * 4;
      if (p.out_fp32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.C) + at) = make_float4(c[0], c[1], c[2], c[3]);
      } else {
        typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
        *reinterpret_cast<v4bf*>(static_cast<uint16_t*>(p.C) + at) = __builtin_convertvector(c, v4bf);
      }
    }
  }
}

template <int RT>
void project(const AdapterProblem& p, hipStream_t stream) {
  const dim3 grid((unsigned)(p.N / 16 / RT));
  switch ((p.T + 15) / 16) {
    case 1: hipLaunchKernelGGL((adapter_project_kernel<1, RT>), grid, dim3(kB), 0, stream, p); break;
    case 2: hipLaunchKernelGGL((adapter_project_kernel<2, RT>), grid, dim3(kB), 0, stream, p); break;
    case 3: hipLaunchKernelGGL((adapter_project_kernel<3, RT>), grid, dim3(kB), 0, stream, p); break;
    default: hipLaunchKernelGGL((adapter_project_kernel<4, RT>), grid, dim3(kB), 0, stream, p); break;
  }
}

}  // namespace

hipError_t launch_moe_few_tokens(const MoeProblem& p, hipStream_t stream) {
  const int t_tiles = (p.T + 15) / 16;
  const int router_blocks = (p.E + 15) / 16 * t_tiles;
  hipLaunchKernelGGL(moe_prepare_kernel, dim3(router_blocks + quant_blocks(p.T, p.H)), dim3(kPB), 0, stream, p,
                     router_blocks);
  const int route_blocks = (p.T + kW - 1) / kW;
  hipLaunchKernelGGL(moe_up_kernel, dim3(route_blocks + p.local * (p.I / 16)), dim3(kB), 0, stream, p, route_blocks);
  hipLaunchKernelGGL(moe_quant_kernel, dim3(quant_blocks((int64_t)p.T * p.top_k, p.I)), dim3(kPB), 0, stream, p);
  const dim3 down(p.H / 16);
  if (t_tiles == 1) hipLaunchKernelGGL(moe_down_kernel<1>, down, dim3(kPB), 0, stream, p);
  else if (t_tiles == 2) hipLaunchKernelGGL(moe_down_kernel<2>, down, dim3(kPB), 0, stream, p);
  else hipLaunchKernelGGL(moe_down_kernel<4>, down, dim3(kPB), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_adapter_few(const AdapterProblem& p, hipStream_t stream) {
  const int chunks = (int)((p.T + 15) / 16), rts = (p.r + 15) / 16;
  const int step = p.T < 16 ? (int)p.T : 16;
  const int shrink_blocks = chunks * rts * step;
  hipLaunchKernelGGL(adapter_prepare_kernel, dim3(shrink_blocks + quant_blocks(p.T, p.K)), dim3(kPB), 0, stream, p,
                     shrink_blocks, step);
  if (p.N / 16 >= kWideTiles) project<2>(p, stream);
  else project<1>(p, stream);
  return hipGetLastError();
}

hipError_t launch_adapter_prompt(const AdapterProblem& p, int64_t ld_s, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16));
  if (p.r <= 16) hipLaunchKernelGGL(adapter_prompt_kernel<1>, grid, dim3(kPB), 0, stream, p, ld_s);
  else if (p.r <= 32) hipLaunchKernelGGL(adapter_prompt_kernel<2>, grid, dim3(kPB), 0, stream, p, ld_s);
  else if (p.r <= 64) hipLaunchKernelGGL(adapter_prompt_kernel<4>, grid, dim3(kPB), 0, stream, p, ld_s);
  else hipLaunchKernelGGL(adapter_prompt_kernel<8>, grid, dim3(kPB), 0, stream, p, ld_s);
  return hipGetLastError();
}

}  // namespace fp8bs
