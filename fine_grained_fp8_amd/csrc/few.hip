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

constexpr int kB = 512;        // threads of every workgroup here
constexpr int kW = kB / 64;    // waves

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
// dealt to the waves in turn; this wave's partial sums.
__device__ __forceinline__ v4f dot_rows_bf16(const uint16_t* a, const uint16_t* b, int K, int wave, int lgrp) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < K / 128; kb += kW) {
    fv4i va[4], vb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      va[i] = *reinterpret_cast<const fv4i*>(a + kb * 128 + i * 32 + lgrp * 8);
      vb[i] = *reinterpret_cast<const fv4i*>(b + kb * 128 + i * 32 + lgrp * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mfma_bf16_16x16x32(as_bf16x8(va[i]), as_bf16x8(vb[i]), c);
  }
  return c;
}

// 1x128 quantization of token rows: 32 tiles a workgroup, 16 lanes each.
__device__ __forceinline__ void quant_tokens(const uint16_t* x, int64_t ldx, int T, int K, int block, uint8_t* xq,
                                             float* xs) {
  const int kb_n = K / 128;
  const int tile = block * (kB / 16) + (threadIdx.x >> 4);
  if (tile >= T * kb_n) return;   // whole 16-lane groups
  const int t = tile / kb_n, kb = tile - t * kb_n, l16 = threadIdx.x & 15;
  const fv4i d = *reinterpret_cast<const fv4i*>(x + t * ldx + kb * 128 + l16 * 8);
  float s;
  const uint2 q = quant8_bf16(make_uint4((uint32_t)d[0], (uint32_t)d[1], (uint32_t)d[2], (uint32_t)d[3]), s);
  *reinterpret_cast<uint2*>(xq + (int64_t)t * K + kb * 128 + l16 * 8) = q;
  if (l16 == 0) xs[t * kb_n + kb] = s;
}
int quant_blocks(int64_t T, int64_t K) { return (int)((T * (K / 128) + kB / 16 - 1) / (kB / 16)); }

template <typename P>
__device__ __forceinline__ void store_out(const P* /*tag*/, void* y, int64_t at, int fp32, float v) {
  if (fp32) static_cast<float*>(y)[at] = v;
  else static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ===========================================================================
// Mixture of experts for up to 64 tokens, four launches.
// ===========================================================================

// 1. Router logits (16 experts x 16 tokens a workgroup) and the 1x128
//    quantization of x.
__global__ __launch_bounds__(kB) void moe_prepare_kernel(MoeProblem p, int router_blocks) {
  if ((int)blockIdx.x >= router_blocks) {
    quant_tokens(p.x, p.ldx, p.T, p.H, blockIdx.x - router_blocks, p.xq, p.xs);
    return;
  }
  __shared__ v4f part[kW][64];
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
    for (int w = 1; w < kW; ++w) c += part[w][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int ee = e0 + lgrp * 4 + v;
      if (ee < p.E && t0 + lrow < p.T) p.logits[(t0 + lrow) * p.E + ee] = c[v];
    }
  }
}

// the value experts are chosen by
__device__ __forceinline__ float choice_value(const MoeProblem& p, int t, int e) {
  const float l = p.logits[t * p.E + e];
  return p.bias ? sigmoid(l) + p.bias[e] : l;
}

// One wave: the chosen experts of token t, best first, with their gates.
__device__ __forceinline__ void route_token(const MoeProblem& p, int t, int lane) {
  float m = -INFINITY, sum = 1.0f;
  if (!p.sigmoid) {
    for (int e = lane; e < p.E; e += 64) m = fmaxf(m, p.logits[t * p.E + e]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    sum = 0.f;
    for (int e = lane; e < p.E; e += 64) sum += expf(p.logits[t * p.E + e] - m);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  }
  uint64_t below = ~0ull;         // keys at or above it are taken
  float my_score = 0.f, total = 0.f;
  int my_expert = 0;
  for (int j = 0; j < p.top_k; ++j) {
    uint64_t best = 0;
    for (int e = lane; e < p.E; e += 64) {
      const uint64_t k = order_key(choice_value(p, t, e), e);
      if (k < below && k > best) best = k;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t o = __shfl_xor(best, d);
      if (o > best) best = o;
    }
    below = best;
    const int e = (int)(0xFFFFFFFFu - (uint32_t)best);
    const float l = p.logits[t * p.E + e];
    const float score = p.sigmoid ? sigmoid(l) : expf(l - m) / sum;
    total += score;
    if (lane == j) {
      my_score = score;
      my_expert = e;
    }
  }
  if (lane < p.top_k) {
    p.slot_expert[t * p.top_k + lane] = my_expert;
    p.slot_gate[t * p.top_k + lane] = (p.normalize ? my_score / total : my_score) * p.gate_scale;
  }
}

// 2. Routing (the first blocks, a wave per token), and h = silu(W1 x) (W3 x)
//    for the tokens that chose a held expert: workgroup (expert, 16 rows)
//    with the gate rows and the up rows of the same 16 channels.  A workgroup
//    finds its expert's tokens itself: a token chose expert e if fewer than
//    top_k experts come before e, and that count is e's slot.
template <int NT>
__global__ __launch_bounds__(kB) void moe_up_kernel(MoeProblem p, int route_blocks) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  if ((int)blockIdx.x < route_blocks) {
    const int t = blockIdx.x * kW + wave;
    if (t < p.T) route_token(p, t, lane);
    return;
  }
  __shared__ v4f part[kW][2][NT][64];
  __shared__ int slot_of[kMoeMaxTokens];     // the expert's slot of each token, or -1
  __shared__ int list_t[kMoeMaxTokens], list_slot[kMoeMaxTokens], count;
  const int tiles = p.I / 16;
  const int el = (blockIdx.x - route_blocks) / tiles, tile = (blockIdx.x - route_blocks) % tiles;
  const int e = p.first + el;
  for (int t = wave; t < p.T; t += kW) {
    const uint64_t mine = order_key(choice_value(p, t, e), e);
    int before = 0;
    for (int c = 0; c < p.E; c += 64) {
      const bool ahead = c + lane < p.E && order_key(choice_value(p, t, c + lane), c + lane) > mine;
      before += __popcll(__ballot(ahead));
    }
    if (lane == 0) slot_of[t] = before < p.top_k ? before : -1;
  }
  __syncthreads();
  if (wave == 0) {
    const int s = lane < p.T ? slot_of[lane] : -1;
    const uint64_t mask = __ballot(s >= 0);
    if (s >= 0) {
      const int at = __popcll(mask & ((1ull << lane) - 1));
      list_t[at] = lane;
      list_slot[at] = lane * p.top_k + s;
    }
    if (lane == 0) count = __popcll(mask);
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;

  const int kb_n = p.H / 128;
  const uint8_t* wg = p.w13 + (int64_t)el * 2 * p.I * p.H + (int64_t)tile * kb_n * 2048;
  const uint8_t* wu = wg + (int64_t)p.I * p.H;
  const float* sg = p.s13 + ((int64_t)el * 2 * (p.I / 128) + tile / 8) * kb_n;
  const float* su = sg + (int64_t)(p.I / 128) * kb_n;
  const uint8_t* xrow[NT];
  const float* xscale[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int c = j * 16 + lrow;
    const int t = list_t[c < n ? c : 0];
    xrow[j] = p.xq + (int64_t)t * p.H;
    xscale[j] = p.xs + t * kb_n;
  }
  v4f ag[NT], au[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) ag[j] = au[j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < kb_n; kb += kW) {
    const Block g = load_tile(wg + (int64_t)kb * 2048, lane), u = load_tile(wu + (int64_t)kb * 2048, lane);
    const float fg = sg[kb], fu = su[kb];
    const Bf16Block g16 = to_bf16(g), u16 = to_bf16(u);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 16 < n) {
        const Bf16Block b = to_bf16(load_row(xrow[j] + kb * 128, lgrp));
        const float sx = xscale[j][kb];
        const v4f pg = block_product(g16, b), pu = block_product(u16, b);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          ag[j][v] = __builtin_fmaf(pg[v], sx * fg, ag[j][v]);
          au[j][v] = __builtin_fmaf(pu[v], sx * fu, au[j][v]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    part[wave][0][j][lane] = ag[j];
    part[wave][1][j][lane] = au[j];
  }
  __syncthreads();
  // wave j finishes column group j: a lane has 4 channels of one token
  for (int j = wave; j * 16 < n; j += kW) {
    v4f a = part[0][0][j][lane], u = part[0][1][j][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) {
      a += part[w][0][j][lane];
      u += part[w][1][j][lane];
    }
    if (j * 16 + lrow < n) {
      float4 h;
      h.x = a[0] * sigmoid(a[0]) * u[0];
      h.y = a[1] * sigmoid(a[1]) * u[1];
      h.z = a[2] * sigmoid(a[2]) * u[2];
      h.w = a[3] * sigmoid(a[3]) * u[3];
      *reinterpret_cast<float4*>(p.h + (int64_t)list_slot[j * 16 + lrow] * p.I + tile * 16 + lgrp * 4) = h;
    }
  }
}

// 3. The 1x128 quantization of h (FP32 in), and, in block 0, the list of the
//    held experts that were chosen: lists[0] = their number n, lists[2..2+n)
//    the local indexes, lists[2+local..2+local+n] the first slot entry of
//    each, lists[3+2 local..] the slots, expert by expert in token order.
__global__ __launch_bounds__(kB) void moe_mid_kernel(MoeProblem p) {
  const int slots = p.T * p.top_k;
  if (blockIdx.x == 0) {
    __shared__ int expert[kMoeMaxTokens * kMoeMaxTopK];
    __shared__ int cnt[kMoeMaxExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < slots; i += kB) expert[i] = p.slot_expert[i] - p.first;
    __syncthreads();
    for (int e = wave; e < p.local; e += kW) {
      int c = 0;
      for (int i = 0; i < slots; i += 64) c += __popcll(__ballot(i + lane < slots && expert[i + lane] == e));
      if (lane == 0) cnt[e] = c;
    }
    __syncthreads();
    int32_t* active = p.lists + 2;
    int32_t* start = active + p.local;
    int32_t* order = start + p.local + 1;
    if (threadIdx.x == 0) {
      int n = 0, at = 0;
      for (int e = 0; e < p.local; ++e) {
        const int c = cnt[e];
        cnt[e] = at;             // now the expert's first entry
        if (c) {
          active[n] = e;
          start[n] = at;
          ++n;
        }
        at += c;
      }
      start[n] = at;
      p.lists[0] = n;
    }
    __syncthreads();
    for (int e = wave; e < p.local; e += kW) {
      int at = cnt[e];
      for (int i = 0; i < slots; i += 64) {
        const bool hit = i + lane < slots && expert[i + lane] == e;
        const uint64_t mask = __ballot(hit);
        if (hit) order[at + __popcll(mask & ((1ull << lane) - 1))] = i + lane;
        at += __popcll(mask);
      }
    }
    return;
  }
  const int kb_n = p.I / 128;
  const int tile = (blockIdx.x - 1) * (kB / 16) + (threadIdx.x >> 4), l16 = threadIdx.x & 15;
  if (tile >= slots * kb_n) return;
  const int slot = tile / kb_n, kb = tile - slot * kb_n;
  const int el = p.slot_expert[slot] - p.first;
  if (el < 0 || el >= p.local) return;
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
//    the copies are summed in wave order at the end.
template <int NT>
__global__ __launch_bounds__(kB) void moe_down_kernel(MoeProblem p) {
  __shared__ float out[kW][NT * 16][16 + 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  for (int i = threadIdx.x; i < kW * NT * 16 * 20; i += kB) (&out[0][0][0])[i] = 0.f;
  __syncthreads();
  const int tile = blockIdx.x, kb_n = p.I / 128;
  const int na = p.lists[0];
  const int32_t* active = p.lists + 2;
  const int32_t* start = active + p.local;
  const int32_t* order = start + p.local + 1;
  const int units = na * kb_n;
  int u = (int)((int64_t)units * wave / kW);
  const int u_end = (int)((int64_t)units * (wave + 1) / kW);
  while (u < u_end) {
    const int a = u / kb_n, kb0 = u - a * kb_n;
    const int kb1 = min(kb_n, kb0 + (u_end - u));
    u += kb1 - kb0;
    const int el = active[a], s0 = start[a], n = start[a + 1] - s0;
    const uint8_t* w = p.w2 + (int64_t)el * p.H * p.I + (int64_t)tile * kb_n * 2048;
    const float* sw = p.s2 + ((int64_t)el * (p.H / 128) + tile / 8) * kb_n;
    int slot[NT];
    v4f acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int c = j * 16 + lrow;
      slot[j] = order[s0 + (c < n ? c : 0)];
      acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    for (int kb = kb0; kb < kb1; ++kb) {
      const v8i wa = as_operand(load_tile(w + (int64_t)kb * 2048, lane));
      const float f = sw[kb];
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
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 16 + lrow < n) {
        const float g = p.slot_gate[slot[j]];
        float* o = &out[wave][slot[j] / p.top_k][lgrp * 4];
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = __builtin_fmaf(acc[j][v], g, o[v]);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * 16; i += kB) {
    const int t = i >> 4, c = i & 15;
    float v = out[0][t][c];
#pragma unroll
    for (int w = 1; w < kW; ++w) v += out[w][t][c];
    store_out((const int*)nullptr, p.y, t * p.ldy + tile * 16 + c, p.y_fp32, v);
  }
}

// ===========================================================================
// Low-rank adapters beside a shared projection.
// ===========================================================================

// z[t] = scale_a (A_a x_t) for 16 tokens and 16 rows of A: workgroup (chunk of
// tokens, rows of A, share of the chunk's adapters).  The adapters of a chunk
// are taken in the order of their first token.  A negative id has no adapter
// (its z is not read); an id past the last adapter gives NaN.
__device__ __forceinline__ void shrink_chunk(const AdapterProblem& p, int64_t t0, int rt, int first, int step,
                                             v4f (*part)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const bool in = t0 + lrow < p.T;
  const int id = in ? p.ids[t0 + lrow] : -1;
  const uint16_t* xr = p.x + (in ? t0 + lrow : t0) * p.ldx;
  const int row = rt * 16 + lrow < p.r ? rt * 16 + lrow : p.r - 1;
  uint32_t left = (uint32_t)(__ballot(id >= 0) & 0xFFFFull);
  for (int turn = 0; left != 0; ++turn) {
    const int lead = __builtin_ctz(left);
    const int a = __shfl(id, lead);
    left &= ~(uint32_t)__ballot(id == a);
    if (turn % step != first) continue;
    v4f c;
    if (a < p.n) {
      c = dot_rows_bf16(p.A + ((int64_t)a * p.r + row) * p.K, xr, (int)p.K, wave, lgrp);
    } else {
      c = v4f{NAN, NAN, NAN, NAN};
    }
    part[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && id == a) {
#pragma unroll
      for (int w = 1; w < kW; ++w) c += part[w][lane];
      const float s = p.scales != nullptr && a < p.n ? p.scales[a] : 1.0f;
      const int r0 = rt * 16 + lgrp * 4;
      if (r0 < p.r)
        *reinterpret_cast<float4*>(p.z + (t0 + lrow) * p.r + r0) = make_float4(c[0] * s, c[1] * s, c[2] * s, c[3] * s);
    }
    __syncthreads();
  }
}

// 1. Few tokens: the quantization of x and the shrink.
__global__ __launch_bounds__(kB) void adapter_prepare_kernel(AdapterProblem p, int shrink_blocks, int step) {
  __shared__ v4f part[kW][64];
  const int b = blockIdx.x;
  if (b >= shrink_blocks) {
    quant_tokens(p.x, p.ldx, (int)p.T, (int)p.K, b - shrink_blocks, p.xq, p.xs);
    return;
  }
  const int rts = (p.r + 15) / 16;
  const int first = b % step, rt = (b / step) % rts;
  shrink_chunk(p, (int64_t)(b / (step * rts)) * 16, rt, first, step, part);
}

__global__ __launch_bounds__(kB) void adapter_shrink_kernel(AdapterProblem p) {
  __shared__ v4f part[kW][64];
  shrink_chunk(p, (int64_t)blockIdx.x * 16, blockIdx.y, 0, 1, part);
}

// acc += B_a z for 16 output rows (row n0 + l & 15 of adapter a) and 16 tokens
// (this lane's column: z row `zt`, `on` if its id is a)
__device__ __forceinline__ v4f expand_add(const AdapterProblem& p, int a, int64_t n0, const float* zt, bool on,
                                          int lane, v4f acc) {
  const int lrow = lane & 15, lgrp = lane >> 4;
  const uint16_t* brow = p.B + ((int64_t)(a < p.n ? a : 0) * p.N + n0 + lrow) * p.r;
  for (int r0 = 0; r0 < p.r; r0 += 32) {
    const int r = r0 + lgrp * 8;
    fv4i bw = {0, 0, 0, 0};
    float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < p.r) {
      bw = *reinterpret_cast<const fv4i*>(brow + r);
      if (on) {
        const float4 u = *reinterpret_cast<const float4*>(zt + r), w = *reinterpret_cast<const float4*>(zt + r + 4);
        z[0] = u.x; z[1] = u.y; z[2] = u.z; z[3] = u.w;
        z[4] = w.x; z[5] = w.y; z[6] = w.z; z[7] = w.w;
      }
    }
    v8bf hi, lo;
    split_bf16(z, hi, lo);
    acc = mfma_bf16_16x16x32(as_bf16x8(bw), hi, acc);
    acc = mfma_bf16_16x16x32(as_bf16x8(bw), lo, acc);
  }
  return acc;
}

// 2. Few tokens: projection and expand, 16 output columns a workgroup.
template <int NT>
__global__ __launch_bounds__(kB) void adapter_project_kernel(AdapterProblem p) {
  __shared__ v4f part[kW][NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, lrow = lane & 15, lgrp = lane >> 4;
  const int tile = blockIdx.x, kb_n = (int)(p.K / 128), T = (int)p.T;
  const uint8_t* w = p.W + (int64_t)tile * kb_n * 2048;
  const float* sw = p.sW + (tile / 8) * p.ld_sw;
  int tok[NT];
  v4f acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    tok[j] = j * 16 + lrow < T ? j * 16 + lrow : T - 1;
    acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  for (int kb = wave; kb < kb_n; kb += kW) {
    const v8i wa = as_operand(load_tile(w + (int64_t)kb * 2048, lane));
    const float f = sw[kb];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const v8i b = as_operand(load_row(p.xq + tok[j] * p.K + kb * 128, lgrp));
      const float c = p.xs[tok[j] * kb_n + kb] * f;
      const v4f zero = {0.f, 0.f, 0.f, 0.f};
      const v4f q = mfma_e4m3_16x16x128(wa, b, zero);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(q[v], c, acc[j][v]);
    }
  }
  // the adapters of the batch, dealt to the waves in the order of their first token
  const int id = lane < T ? p.ids[lane] : -1;
  uint64_t left = __ballot(id >= 0);
  for (int turn = 0; left != 0; ++turn) {
    const int a = __shfl(id, __builtin_ctzll(left));
    const uint64_t members = __ballot(id == a);
    left &= ~members;
    if (turn % kW != wave) continue;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t m = (uint32_t)(members >> (16 * j)) & 0xFFFFu;
      if (m) acc[j] = expand_add(p, a, tile * 16, p.z + (int64_t)tok[j] * p.r, (m >> lrow) & 1, lane, acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave < NT) {
    const int j = wave;
    v4f c = part[0][j][lane];
#pragma unroll
    for (int q = 1; q < kW; ++q) c += part[q][j][lane];
    if (j * 16 + lrow < T) {
      const int64_t at = (j * 16 + lrow) * p.ldc + tile * 16 + lgrp * 4;
#pragma unroll
      for (int v = 0; v < 4; ++v) store_out((const int*)nullptr, p.C, at + v, p.out_fp32, c[v]);
    }
  }
}

}  // namespace

hipError_t launch_moe_few_tokens(const MoeProblem& p, hipStream_t stream) {
  const int t_tiles = (p.T + 15) / 16;
  const int router_blocks = (p.E + 15) / 16 * t_tiles;
  hipLaunchKernelGGL(moe_prepare_kernel, dim3(router_blocks + quant_blocks(p.T, p.H)), dim3(kB), 0, stream, p,
                     router_blocks);
  const int route_blocks = (p.T + kW - 1) / kW;
  const dim3 up(route_blocks + p.local * (p.I / 16));
  if (t_tiles == 1) hipLaunchKernelGGL(moe_up_kernel<1>, up, dim3(kB), 0, stream, p, route_blocks);
  else if (t_tiles == 2) hipLaunchKernelGGL(moe_up_kernel<2>, up, dim3(kB), 0, stream, p, route_blocks);
  else hipLaunchKernelGGL(moe_up_kernel<4>, up, dim3(kB), 0, stream, p, route_blocks);
  hipLaunchKernelGGL(moe_mid_kernel, dim3(1 + quant_blocks((int64_t)p.T * p.top_k, p.I)), dim3(kB), 0, stream, p);
  const dim3 down(p.H / 16);
  if (t_tiles == 1) hipLaunchKernelGGL(moe_down_kernel<1>, down, dim3(kB), 0, stream, p);
  else if (t_tiles == 2) hipLaunchKernelGGL(moe_down_kernel<2>, down, dim3(kB), 0, stream, p);
  else hipLaunchKernelGGL(moe_down_kernel<4>, down, dim3(kB), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_adapter_few(const AdapterProblem& p, hipStream_t stream) {
  const int chunks = (int)((p.T + 15) / 16), rts = (p.r + 15) / 16;
  const int step = p.T < 16 ? (int)p.T : 16;
  const int shrink_blocks = chunks * rts * step;
  hipLaunchKernelGGL(adapter_prepare_kernel, dim3(shrink_blocks + quant_blocks(p.T, p.K)), dim3(kB), 0, stream, p,
                     shrink_blocks, step);
  const dim3 grid((unsigned)(p.N / 16));
  if (chunks == 1) hipLaunchKernelGGL(adapter_project_kernel<1>, grid, dim3(kB), 0, stream, p);
  else if (chunks == 2) hipLaunchKernelGGL(adapter_project_kernel<2>, grid, dim3(kB), 0, stream, p);
  else hipLaunchKernelGGL(adapter_project_kernel<4>, grid, dim3(kB), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_adapter_shrink(const AdapterProblem& p, hipStream_t stream) {
  hipLaunchKernelGGL(adapter_shrink_kernel, dim3((unsigned)((p.T + 15) / 16), (unsigned)((p.r + 15) / 16)), dim3(kB),
                     0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bs
