// Products for a few tokens on gfx950: the whole mixture-of-experts layer for
// up to 64 tokens, and the projection with low-rank adapters in its form for
// up to 64 tokens (plus the adapters' two small products for any number).
//
// With so few rows every weight byte is used for a handful of products: the
// kernels are bound by reading the weights once, so they are laid out for
// that.  A workgroup owns 16 output rows (one operand tile row), or two or four
// such; its waves split the K blocks, each loading whole 2 KB operand tiles (16
// bytes a lane) straight into MFMA operand registers, one block ahead of the
// products; the partial sums meet in LDS.  The weight rows are the MFMA's "A"
// rows, the tokens its 16 columns: a lane ends with 4 consecutive outputs of
// one token.
//
// What bounds them, measured: a CU takes in about 25 GB/s here, weights and
// token operands alike, and all of them 5.2 - 6.4 TB/s; so work goes to all 256
// CUs, and operands that are read again from L2 cost like weights.  A small
// dependent launch costs 4 - 5 us.
#include "device.hpp"
#include "layers.hpp"
#include "operands.hpp"

namespace fp8bs {

namespace {

typedef int fv4i __attribute__((ext_vector_type(4)));

constexpr int kB = 512;         // threads of a workgroup
constexpr int kW = kB / 64;     // and its waves

__device__ __forceinline__ v8bf as_bf16x8(const fv4i& v) { return __builtin_bit_cast(v8bf, v); }

// a lane's part of an operand tile
__device__ __forceinline__ Block load_tile(const uint8_t* tile, int lane) {
  return Block{*reinterpret_cast<const fv4i*>(tile + lane * 16), *reinterpret_cast<const fv4i*>(tile + 1024 + lane * 16)};
}
// the same of a token's row-major codes: `block` (one for the wave) + the lane's
// 32-bit offset, row start + 16 g (the code arrays here stay below 2^31 bytes)
__device__ __forceinline__ Block load_row(const uint8_t* block, uint32_t lane_off) {
  return Block{*reinterpret_cast<const fv4i*>(block + lane_off), *reinterpret_cast<const fv4i*>(block + 64 + lane_off)};
}
__device__ __forceinline__ v8i as_operand(const Block& b) {
  return v8i{b.lo[0], b.lo[1], b.lo[2], b.lo[3], b.hi[0], b.hi[1], b.hi[2], b.hi[3]};
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Selection order of routing values as unsigned numbers: larger first, NaN
// last (1; 0 is left for "none").
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (v != v) return 1u;
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 counts as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);   // -infinity: 0x007FFFFF
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = row16_max_u32(v);
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// max (NaN left out) and sum over the wave, in every lane
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 16));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v += __shfl_xor(v, d, 16);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Dot products of 16 BF16 rows (row l & 15 of the lane at `a`, 16-byte
// aligned) with 16 BF16 token rows (at `b`) over K blocks [kb0, kb1), dealt to
// the workgroup's kW waves in turn; this wave's partial sums.
__device__ __forceinline__ v4f dot_rows_bf16(const uint16_t* a, const uint16_t* b, int kb0, int kb1, int wave,
                                             int lgrp) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
  for (int kb = kb0 + wave; kb < kb1; kb += kW) {
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

// Share s of S of kb_n K blocks.  The small dot products (router, shrink) are
// cut along K over S workgroups, whose partial sums the reader adds in order:
// one compute unit alone would take 8 - 17 us to read 16 rows of 7168 and
// their tokens.
__device__ __forceinline__ int share(int kb_n, int s, int S) { return (int)((int64_t)kb_n * s / S); }

// 1x128 quantization of token rows: 32 tiles a workgroup, 16 lanes each.  The
// codes row-major [T][K], or (kTiled) as operand tiles of 16 tokens x 128, whose
// loads are whole lines (16 rows of 64 bytes a load cost twice as much).
template <bool kTiled>
__device__ __forceinline__ void quant_tokens(const uint16_t* x, int64_t ldx, int T, int K, int block, uint8_t* xq,
                                             float* xs) {
  const int kb_n = K / 128;
  const int tile = block * (kB / 16) + (threadIdx.x >> 4);
  if (tile >= T * kb_n) return;   // whole 16-lane groups
  const int t = tile / kb_n, kb = tile - t * kb_n, l16 = threadIdx.x & 15;
  const fv4i d = *reinterpret_cast<const fv4i*>(x + t * ldx + kb * 128 + l16 * 8);
  float s;
  const uint2 q = quant8_bf16(make_uint4((uint32_t)d[0], (uint32_t)d[1], (uint32_t)d[2], (uint32_t)d[3]), s);
  const int64_t at = kTiled ? ((int64_t)(t >> 4) * kb_n + kb) * 2048 + (l16 >> 3) * 1024 +
                                  ((l16 & 7) >> 1) * 256 + (t & 15) * 16 + (l16 & 1) * 8
                            : (int64_t)t * K + kb * 128 + l16 * 8;
  *reinterpret_cast<uint2*>(xq + at) = q;
  if (l16 == 0) xs[t * kb_n + kb] = s;
}
int quant_blocks(int64_t T, int64_t K) { return (int)((T * (K / 128) + kB / 16 - 1) / (kB / 16)); }

__device__ __forceinline__ void store_out(void* y, int64_t at, int fp32, float v) {
  if (fp32) static_cast<float*>(y)[at] = v;
  else static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// ===========================================================================
// Mixture of experts for up to 64 tokens, four to six launches.
// ===========================================================================

// 1. Router logits (16 experts x 16 tokens x a share of K a workgroup), and the
//    1x128 quantization of x.
__global__ __launch_bounds__(kB) void moe_prepare_kernel(MoeProblem p, int router_blocks) {
  if ((int)blockIdx.x >= router_blocks) {
    quant_tokens<false>(p.x, p.ldx, p.T, p.H, blockIdx.x - router_blocks, p.xq, p.xs);
    return;
  }
  __shared__ v4f part[kW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int e_tiles = (p.E + 15) / 16, s = blockIdx.x % p.splits, et = blockIdx.x / p.splits;
  const int e0 = (et % e_tiles) * 16, t0 = (et / e_tiles) * 16;
  const int e = e0 + lrow < p.E ? e0 + lrow : p.E - 1;
  const int t = t0 + lrow < p.T ? t0 + lrow : p.T - 1;
  const int kb_n = p.H / 128;
  part[wave][lane] = dot_rows_bf16(p.router + e * p.ld_r, p.x + t * p.ldx, share(kb_n, s, p.splits),
                                   share(kb_n, s + 1, p.splits), wave, lgrp);
  __syncthreads();
  if (wave == 0) {
    v4f c = part[0][lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) c += part[w][lane];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int ee = e0 + lgrp * 4 + v;
      if (ee < p.E && t0 + lrow < p.T) p.logits[((int64_t)s * p.T + t0 + lrow) * p.E + ee] = c[v];
    }
  }
}

// The logit of expert e for token t; out of range (on: false): -infinity.
__device__ __forceinline__ float logit(const MoeProblem& p, int t, int e, bool on) {
  if (!on) return -INFINITY;
  float v[kMoeSplits];
#pragma unroll
  for (int s = 0; s < kMoeSplits; ++s) v[s] = s < p.splits ? p.logits[((int64_t)s * p.T + t) * p.E + e] : 0.f;
#pragma unroll
  for (int s = 1; s < kMoeSplits; ++s) v[0] += v[s];
  return v[0];
}
// what experts are chosen by
__device__ __forceinline__ float choice_value(const MoeProblem& p, float l, int e) {
  return p.bias ? sigmoid(l) + p.bias[e] : l;
}

// One wave: the chosen experts of token t, best first, with their gates.
// Lane l holds experts l, l + 64, ..., at most kMost of them.
template <int kMost>
__device__ __forceinline__ void route_token(const MoeProblem& p, int t, int lane) {
  float l[kMost];
  uint32_t key[kMost];   // order_bits; 0: no such expert, or taken
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    const int e = c * 64 + lane;
    l[c] = -INFINITY;
    key[c] = 0;
    if (c * 64 < p.E) {
      l[c] = logit(p, t, e, e < p.E);
      if (e < p.E) key[c] = order_bits(choice_value(p, l[c], e));
    }
  }
  float m = -INFINITY, sum = 1.0f;
  if (!p.sigmoid) {
#pragma unroll
    for (int c = 0; c < kMost; ++c) m = fmaxf(m, l[c]);
    m = wave_max(m);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < kMost; ++c)
      if (c * 64 < p.E) sum += c * 64 + lane < p.E ? expf(l[c] - m) : 0.f;
    sum = wave_sum(sum);
  }
  float my_score = 0.f, total = 0.f;
  int my_expert = 0;
  for (int j = 0; j < p.top_k; ++j) {
    // the lane's best that is left (bits 0: taken or absent), the lowest index first
    uint32_t best = 0;
    int at = 0;
    float lb = 0.f;
#pragma unroll
    for (int c = 0; c < kMost; ++c)
      if (c * 64 < p.E && key[c] > best) {
        best = key[c];
        at = c;
        lb = l[c];
      }
    const uint32_t top = wave_max_u32(best);
    const uint32_t index = best == top ? (uint32_t)(at * 64 + lane) : 0xFFFFFFFFu;
    const uint32_t e = ~wave_max_u32(~index);      // the smallest index among equals
    const float le = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lb), (int)(e & 63)));
#pragma unroll
    for (int c = 0; c < kMost; ++c)
      if (e == (uint32_t)(c * 64 + lane)) key[c] = 0;
    const float score = p.sigmoid ? sigmoid(le) : expf(le - m) / sum;
    total += score;
    if (lane == j) {
      my_score = score;
      my_expert = (int)e;
    }
  }
  if (lane < p.top_k) {
    p.slot_expert[t * p.top_k + lane] = my_expert;
    p.slot_gate[t * p.top_k + lane] = (p.normalize ? my_score / total : my_score) * p.gate_scale;
  }
}

// 2. Routing, a wave per token.
template <int kMost>
__global__ __launch_bounds__(256) void moe_route_kernel(MoeProblem p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < p.T) route_token<kMost>(p, t, threadIdx.x & 63);
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
  uint32_t xoff[NT], soff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int c = j * 16 + lrow;
    const uint32_t t = (uint32_t)list_t[c < n ? c : 0];
    xoff[j] = t * (uint32_t)p.H + lgrp * 16;
    soff[j] = t * (uint32_t)kb_n;
    ag[j] = au[j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  auto fetch = [&](int kb, UpLoads& f) {
    f.g = load_tile(wg + (int64_t)kb * 2048, lane);
    f.u = load_tile(wu + (int64_t)kb * 2048, lane);
    if constexpr (NT == 1) {
      f.x = load_row(p.xq + kb * 128, xoff[0]);
      f.sx = (p.xs + kb)[soff[0]];
    }
    f.fg = sg[kb];
    f.fu = su[kb];
  };
  // Loads return in the order of their issue: the token operands of the
  // present block are asked for before the next block's weights.
  Block x[NT];
  float sx[NT];
  auto tokens = [&](int kb, const UpLoads& f) {
    if constexpr (NT == 1) {
      x[0] = f.x;
      sx[0] = f.sx;
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        x[j] = load_row(p.xq + kb * 128, xoff[j]);
        sx[j] = (p.xs + kb)[soff[j]];
      }
      __asm__ volatile("" ::: "memory");
    }
  };
  auto products = [&](const UpLoads& f) {
    const Bf16Block g16 = to_bf16(f.g), u16 = to_bf16(f.u);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (j * 16 < n) {
        const Bf16Block b = to_bf16(x[j]);
        const v4f pg = block_product(g16, b), pu = block_product(u16, b);
        const float cg = sx[j] * f.fg, cu = sx[j] * f.fu;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          ag[j][v] = __builtin_fmaf(pg[v], cg, ag[j][v]);
          au[j][v] = __builtin_fmaf(pu[v], cu, au[j][v]);
        }
      }
    }
  };
  if (wave >= kb_n) return;
  const int last = kb_n - 1;
  UpLoads f0, f1;
  fetch(wave, f0);
  for (int kb = wave;; kb += 2 * kW) {
    tokens(kb, f0);
    fetch(min(kb + kW, last), f1);     // past the wave's last block: one that is not used
    products(f0);
    if (kb + kW >= kb_n) break;
    tokens(kb + kW, f1);
    fetch(min(kb + 2 * kW, last), f0);
    products(f1);
    if (kb + 2 * kW >= kb_n) break;
  }
}

// 3. h = silu(W1 x) (W3 x) for the tokens that chose a held expert: workgroup
//    (expert, 16 channels) with the gate rows and the up rows of the same
//    channels.  The products convert the codes to BF16: exact, with FP32 sums,
//    because h is quantized again and the FP8 instruction's truncation would
//    move codes.
//    A workgroup lists its expert's tokens itself.  kRouted: from the chosen
//    slots (at most 1024 numbers).  Otherwise (a token per wave at most) it
//    finds them from the logits, while the first blocks of the same launch do
//    the routing for the kernels that follow: a token chose expert e if fewer
//    than top_k experts come before e, and that count is e's slot.  That saves
//    a launch (about 4 us); with more tokens every workgroup would repeat too
//    many sums over the shares.
//    64 tokens on 64 experts of 2048 x 1408: 63 us for 369 MB (5.8 TB/s); 8 of 64
//    experts of 7168 x 2048, 32 tokens: 41 us for 208 MB (5.0 TB/s); one token on
//    two experts: 13 - 16 us for 59 MB.  Without the block loaded ahead 97 us in
//    the first case, with three blocks a wave in flight (spilled) 400.
template <int NT, bool kRouted>
__global__ __launch_bounds__(kB, NT > 2 ? 2 : 4) void moe_up_kernel(MoeProblem p, int route_blocks) {
  __shared__ v4f part[kW][2][64];
  __shared__ int slot_of[kMoeMaxTokens];     // the expert's slot of each token, or -1
  __shared__ int list_t[kMoeMaxTokens], list_slot[kMoeMaxTokens], count;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  if (!kRouted && (int)blockIdx.x < route_blocks) {
    if (wave < p.T) route_token<1>(p, wave, lane);
    return;
  }
  const int tiles = p.I / 16, block = kRouted ? blockIdx.x : blockIdx.x - route_blocks;
  const int el = block / tiles, tile = block % tiles;
  if (threadIdx.x < kMoeMaxTokens) slot_of[threadIdx.x] = -1;
  __syncthreads();
  if constexpr (kRouted) {
    for (int i = threadIdx.x; i < p.T * p.top_k; i += kB)
      if (p.slot_expert[i] == p.first + el) slot_of[i / p.top_k] = i;
  } else if (wave < p.T) {
    const int e = p.first + el;
    const uint32_t mine = order_bits(choice_value(p, logit(p, wave, e, true), e));
    int before = 0;
    for (int c = 0; c < p.E; c += 64) {
      const int ce = c + lane;
      const uint32_t k = ce < p.E ? order_bits(choice_value(p, logit(p, wave, ce, true), ce)) : 0u;
      before += __popcll(__ballot(k > mine || (k == mine && ce < e)));
    }
    if (lane == 0 && before < p.top_k) slot_of[wave] = wave * p.top_k + before;
  }
  __syncthreads();
  if (wave == 0) {
    const int s = slot_of[lane];
    const uint64_t mask = __ballot(s >= 0);
    const int at = __popcll(mask & ((1ull << lane) - 1));
    if (s >= 0) {
      list_t[at] = lane;
      list_slot[at] = s;
    }
    if (lane == 0) count = __popcll(mask);
    if (tile == 0) {   // for the down kernel
      if (lane == 0) p.counts[el] = __popcll(mask);
      if (s >= 0) p.lists[el * kMoeMaxTokens + at] = s;
    }
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;

  // column group j of the sums: a lane has 4 channels of one token
  auto finish = [&](int j, const v4f& ag, const v4f& au) {
    __syncthreads();
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
  // an expert with more than 16 NT tokens reads its weights again, from the
  // last-level cache
  for (int j0 = 0; j0 * 16 < n; j0 += NT) {
    v4f ag[NT], au[NT];
    up_sums<NT>(p, el, tile, list_t + j0 * 16, n - j0 * 16, wave, lane, ag, au);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if ((j0 + j) * 16 < n) finish(j0 + j, ag[j], au[j]);
  }
}

// The plan of the down kernel: the chosen held experts' tokens in parts of at
// most `span`.  plan[0] = parts, then [most] each part's expert, [most + 1] the
// first of its slots, [T top_k] the slots and [T top_k] their gates (FP32).
__host__ __device__ inline int plan_parts(const MoeProblem& p) {
  const int slots = p.T * p.top_k;
  return (p.local < slots ? p.local : slots) + slots / 16;
}
__device__ __forceinline__ void make_plan(const MoeProblem& p, int span) {
  constexpr int kSlots = kMoeMaxTokens * kMoeMaxTopK, kParts = kSlots + kSlots / 16;
  __shared__ int from[kParts];          // a part's first entry in p.lists
  __shared__ int16_t first[kParts + 1];
  __shared__ int entry[kSlots];         // where in p.lists the plan's slots come from
  __shared__ int n_parts;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, most = plan_parts(p);
  int32_t* plan_expert = p.plan + 1;
  int32_t* plan_start = plan_expert + most;
  int32_t* plan_slot = plan_start + most + 1;
  float* plan_gate = reinterpret_cast<float*>(plan_slot + p.T * p.top_k);
  if (wave == 0) {
    int np = 0, ns = 0;
    for (int c = 0; c < p.local; c += 64) {
      const int cnt = c + lane < p.local ? p.counts[c + lane] : 0;
      const int parts = (cnt + span - 1) / span;
      int ic = cnt, ip = parts;     // inclusive sums over the lanes
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int oc = __shfl_up(ic, d), op = __shfl_up(ip, d);
        if (lane >= d) {
          ic += oc;
          ip += op;
        }
      }
      for (int q = 0; q < parts; ++q) {
        const int at = np + ip - parts + q, s0 = ns + ic - cnt + q * span;
        from[at] = (c + lane) * kMoeMaxTokens + q * span;
        first[at] = (int16_t)s0;
        plan_expert[at] = c + lane;
        plan_start[at] = s0;
      }
      np += __shfl(ip, 63);
      ns += __shfl(ic, 63);
    }
    if (lane == 0) {
      n_parts = np;
      first[np] = (int16_t)ns;
      plan_start[np] = ns;
      p.plan[0] = np;
    }
  }
  __syncthreads();
  for (int a = wave; a < n_parts; a += kW)
    if (lane < first[a + 1] - first[a]) entry[first[a] + lane] = from[a] + lane;
  __syncthreads();
  // all slots at once: two round trips to memory
  for (int i = threadIdx.x; i < first[n_parts]; i += kB) {
    const int s = p.lists[entry[i]];
    plan_slot[i] = s;
    plan_gate[i] = p.slot_gate[s];
  }
}

// 4. The 1x128 quantization of h (FP32 in): a tile spans eight workgroups of
//    the up kernel, so it waits for the next launch.  The first block makes the
//    down kernel's plan meanwhile.
__global__ __launch_bounds__(kB) void moe_quant_kernel(MoeProblem p, int span) {
  if (blockIdx.x == 0) {
    make_plan(p, span);
    return;
  }
  const int kb_n = p.I / 128;
  const int tile = (blockIdx.x - 1) * (kB / 16) + (threadIdx.x >> 4), l16 = threadIdx.x & 15;
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

// A unit of the down kernel as loaded: the weights, and the codes and scales
// of the expert's first 16 tokens.
struct DownLoads {
  Block w, x;
  float sh, f;
};

// 5. y: a workgroup has 16 output channels of every token.  The plan's (part,
//    K block) units are dealt to the waves in equal runs.  A wave adds gate x its
//    sums into its own copy of the outputs in LDS when a part ends, and the
//    copies are summed in wave order at the end, so that the result does not
//    depend on timing.  The next unit is loaded before the present one's
//    products, across parts too.
//    Where the channels give fewer workgroups than the card has compute units,
//    `cuts` workgroups share a tile's units: one compute unit loads about 25
//    GB/s here, so that 128 of them would take twice as long as 256.  Each
//    leaves its FP32 sums in the workspace for one more small launch, about 4
//    us; a count of arrivals in this one cost 40 us: its release makes every
//    workgroup write back its XCD's L2 (sums written through to memory ahead of a
//    relaxed count have not been tried).
//    64 tokens on 64 experts of 2048 x 1408: 39 us for 185 MB, uncut 61; 8 experts
//    of 7168 x 2048, 32 tokens: 24 us for 117 MB (4.9 TB/s).
template <int NT, int DW>
__global__ __launch_bounds__(DW * 64) void moe_down_kernel(MoeProblem p, int cuts) {
  extern __shared__ float out[];      // [DW][T][20], 16 of 20 used, then the plan
  constexpr int kDB = DW * 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int most = plan_parts(p), n_plan = 2 + 2 * most + 2 * p.T * p.top_k;
  int32_t* plan = reinterpret_cast<int32_t*>(out + DW * p.T * 20);
  for (int i = threadIdx.x; i < n_plan; i += kDB) plan[i] = p.plan[i];
  for (int i = threadIdx.x; i < DW * p.T * 20; i += kDB) out[i] = 0.f;
  const int32_t* active = plan + 1;
  const int32_t* start = active + most;
  const int32_t* slots = start + most + 1;
  const float* gates = reinterpret_cast<const float*>(slots + p.T * p.top_k);
  __syncthreads();

  const int tile = blockIdx.x / cuts, cut = blockIdx.x % cuts, kb_n = p.I / 128;
  const int units = plan[0] * kb_n, run = cut * DW + wave;
  const int u0 = __builtin_amdgcn_readfirstlane((int)((int64_t)units * run / (DW * cuts)));
  const int u1 = __builtin_amdgcn_readfirstlane((int)((int64_t)units * (run + 1) / (DW * cuts)));
  if (u0 < u1) {
    int a = __builtin_amdgcn_readfirstlane(u0 / kb_n), kb = u0 - a * kb_n;   // the unit at hand
    int fa = a, fk = kb, left = u1 - u0;        // the unit to fetch next, and how many are left
    // addresses of the unit to fetch: a part's are set when it begins
    const uint8_t* fw = nullptr;
    const float* fs = nullptr;
    uint32_t fx = 0, fh = 0;
    auto aim = [&]() {
      const int el = __builtin_amdgcn_readfirstlane(active[fa]), s0 = start[fa];
      const uint32_t s = (uint32_t)slots[s0 + (lrow < start[fa + 1] - s0 ? lrow : 0)];
      fw = p.w2 + ((int64_t)el * (p.H / 16) + tile) * kb_n * 2048;
      fs = p.s2 + ((int64_t)el * (p.H / 128) + tile / 8) * kb_n;
      fx = s * (uint32_t)p.I + lgrp * 16;
      fh = s * (uint32_t)kb_n;
    };
    auto fetch = [&](DownLoads& f) {
      f.w = load_tile(fw + fk * 2048, lane);
      f.x = load_row(p.hq + fk * 128, fx);
      f.sh = (p.hs + fk)[fh];
      f.f = fs[fk];
      if (--left > 0 && ++fk == kb_n) {         // past the wave's last unit: that unit again, not used
        fk = 0;
        ++fa;
        aim();
      }
    };
    int n = 0;
    uint32_t slot[NT];
    v4f acc[NT];
    auto begin = [&]() {
      const int s0 = start[a];
      n = __builtin_amdgcn_readfirstlane(start[a + 1] - s0);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = j * 16 + lrow;
        slot[j] = (uint32_t)slots[s0 + (c < n ? c : 0)];
        acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
      }
    };
    auto flush = [&](int part) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j * 16 + lrow < n) {
          const float g = gates[start[part] + j * 16 + lrow];
          float4* o = reinterpret_cast<float4*>(&out[(wave * p.T + (int)slot[j] / p.top_k) * 20 + lgrp * 4]);
          float4 v = *o;
          v.x = __builtin_fmaf(acc[j][0], g, v.x);
          v.y = __builtin_fmaf(acc[j][1], g, v.y);
          v.z = __builtin_fmaf(acc[j][2], g, v.z);
          v.w = __builtin_fmaf(acc[j][3], g, v.w);
          *o = v;
        }
      }
    };
    int u = u0;
    // the unit's products; false after the wave's last one
    auto step = [&](const DownLoads& l) {
      const v8i wa = as_operand(l.w);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j * 16 < n) {
          const v8i b = as_operand(j == 0 ? l.x : load_row(p.hq + kb * 128, slot[j] * (uint32_t)p.I + lgrp * 16));
          const float c = (j == 0 ? l.sh : (p.hs + kb)[slot[j] * (uint32_t)kb_n]) * l.f;
          const v4f zero = {0.f, 0.f, 0.f, 0.f};
          const v4f q = mfma_e4m3_16x16x128(wa, b, zero);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][v] = __builtin_fmaf(q[v], c, acc[j][v]);
        }
      }
      const int part = a;
      if (++kb == kb_n) {
        kb = 0;
        ++a;
      }
      const bool more = ++u < u1;
      if (!more || kb == 0) {
        flush(part);
        if (more) begin();
      }
      return more;
    };
    DownLoads l0, l1;
    begin();
    aim();
    fetch(l0);
    for (;;) {
      fetch(l1);
      if (!step(l0)) break;
      fetch(l0);
      if (!step(l1)) break;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * 16; i += kDB) {
    const int t = i >> 4, c = i & 15;
    float v = out[t * 20 + c];
#pragma unroll
    for (int w = 1; w < DW; ++w) v += out[(w * p.T + t) * 20 + c];
    if (cuts == 1) store_out(p.y, t * p.ldy + tile * 16 + c, p.y_fp32, v);
    else p.parts[((int64_t)blockIdx.x * p.T + t) * 16 + c] = v;
  }
}

// 6. Where tiles were cut: the sums of a tile's workgroups, in order.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeProblem p, int cuts) {
  const int i = blockIdx.x * 256 + threadIdx.x;     // (tile, token, channel)
  if (i >= p.T * p.H) return;
  const int per = p.T * 16, tile = i / per, t = i % per >> 4, c = i & 15;
  const float* src = p.parts + (int64_t)tile * cuts * per + t * 16 + c;
  float v = src[0];
  for (int q = 1; q < cuts; ++q) v += src[q * per];
  store_out(p.y, t * p.ldy + tile * 16 + c, p.y_fp32, v);
}

// ===========================================================================
// Low-rank adapters beside a shared projection.
// ===========================================================================

// The shrink z[t] = scale_a (A_a x_t) leaves FP32 partial sums zp[s][t][rank],
// one per share of K; z8 adds 8 of them in order, scales them and gives the
// expand's operands: z = hi + lo in BF16.  Both terms have z's sign and only 0
// has a zero term (hi is the BF16 value next below |z|, lo the rest), so that
// an infinite weight times them is the infinity that it is times z; hi rounded
// to nearest would leave a lo of 0 or of the other sign, and NaN (and itself
// be infinite for z past BF16's largest value).  The price is a bit: z is kept
// to 2^-16, to nearest 2^-17; B z alone, in FP32 out, is within 4.9e-6 of the
// 64-bit product by 2-norm (to nearest 2.4e-6), where the projection beside it
// is within 2e-5.  Looking for such weights in the GEMM's epilogue instead costs
// 1% of a call at 4096 x 18432 x 7168 and 4 - 10% with an adapter for every few
// rows.
// A token without an adapter has no sums (zeros here); an id past the last one
// gives NaN.
__device__ __forceinline__ void z8(const AdapterProblem& p, int64_t t, int r, v8bf& hi, v8bf& lo) {
  float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int id = p.ids[t];
  if (id >= 0) {
    float4 u[kAdapterSplits][2];
#pragma unroll
    for (int s = 0; s < kAdapterSplits; ++s) {
      const float4* src = reinterpret_cast<const float4*>(p.zp + ((int64_t)s * p.T + t) * p.r + r);
      u[s][0] = u[s][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < p.splits && id < p.n) {
        u[s][0] = src[0];
        u[s][1] = src[1];
      }
    }
    const float scale = id >= p.n ? NAN : p.scales != nullptr ? p.scales[id] : 1.0f;
#pragma unroll
    for (int s = 0; s < kAdapterSplits; ++s) {
      z[0] += u[s][0].x; z[1] += u[s][0].y; z[2] += u[s][0].z; z[3] += u[s][0].w;
      z[4] += u[s][1].x; z[5] += u[s][1].y; z[6] += u[s][1].z; z[7] += u[s][1].w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(z[i]), mag = u & 0x7FFFFFFFu, sign = u >> 31 << 15;
    if (mag - 1u < 0x7F7FFFFFu) {          // finite and not 0
      const uint32_t h = (mag - 1u) >> 16;
      const __bf16 rest = (__bf16)(__uint_as_float(mag) - __uint_as_float(h << 16));   // exact, then rounded
      hi[i] = __builtin_bit_cast(__bf16, (uint16_t)(sign | h));
      lo[i] = __builtin_bit_cast(__bf16, (uint16_t)(sign | max((uint32_t)__builtin_bit_cast(uint16_t, rest), 1u)));
    } else {
      hi[i] = lo[i] = (__bf16)z[i];
    }
  }
}

// The ids of a chunk of 16 tokens (in every 16-lane group; -1 past the last
// token) and which of them have an adapter that exists.
__device__ __forceinline__ uint32_t chunk_ids(const AdapterProblem& p, int64_t t0, int lrow, int& id) {
  id = t0 + lrow < p.T ? p.ids[t0 + lrow] : -1;
  if (id >= p.n) id = -1;
  return (uint32_t)(__ballot(id >= 0) & 0xFFFFull);
}

// 1. Few tokens: the quantization of x, and the shrink: workgroup (chunk of 16
//    tokens, 16 rows of A, share of K, one of `step` shares of the chunk's
//    adapters, which are taken in the order of their first token).
__global__ __launch_bounds__(kB) void adapter_prepare_kernel(AdapterProblem p, int shrink_blocks, int step) {
  __shared__ v4f part[kW][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  int b = blockIdx.x;
  if (b >= shrink_blocks) {
    quant_tokens<true>(p.x, p.ldx, (int)p.T, (int)p.K, b - shrink_blocks, p.xq, p.xs);
    return;
  }
  const int rts = (p.r + 15) / 16, kb_n = (int)(p.K / 128);
  const int first = b % step;
  b /= step;
  const int s = b % p.splits;
  b /= p.splits;
  const int rt = b % rts;
  const int64_t t0 = (int64_t)(b / rts) * 16;
  const int row = rt * 16 + lrow < p.r ? rt * 16 + lrow : p.r - 1, r0 = rt * 16 + lgrp * 4;
  int id;
  uint32_t left = chunk_ids(p, t0, lrow, id);
  for (int turn = 0; left != 0; ++turn) {
    const int one = __builtin_ctz(left), a = __shfl(id, one);
    left &= ~(uint32_t)__ballot(id == a);
    if (turn % step != first) continue;
    // other adapters' tokens: the column is not used, and reads a line that is
    const uint16_t* xr = p.x + (t0 + (id == a ? lrow : one)) * p.ldx;
    __syncthreads();
    part[wave][lane] = dot_rows_bf16(p.A + ((int64_t)a * p.r + row) * p.K, xr, share(kb_n, s, p.splits),
                                     share(kb_n, s + 1, p.splits), wave, lgrp);
    __syncthreads();
    if (wave == 0 && id == a && r0 < p.r) {
      v4f c = part[0][lane];
#pragma unroll
      for (int w = 1; w < kW; ++w) c += part[w][lane];
      *reinterpret_cast<v4f*>(p.zp + ((int64_t)s * p.T + t0 + lrow) * p.r + r0) = c;
    }
  }
}

// Prompts: the quantization of x (codes and MN-major scales as the row
// quantizer writes them) and the shrink in one pass over x: workgroup (chunk
// of 16 tokens, share of K), its waves dealing the K blocks.  A lane holds 32
// values of one token's 1x128 tile, which are both the quantizer's input and
// the products' operand.  The adapters of the chunk take turns on the same
// accumulators: a column belongs to one token, and its sums are kept only in
// its own adapter's turn (a select, not a product with zero, so that an
// adapter with infinite weights stays among its own tokens).
template <int RT>
__global__ __launch_bounds__(kB) void adapter_prompt_kernel(AdapterProblem p, int64_t ld_s) {
  __shared__ v4f part[kW][RT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int s = blockIdx.x % p.splits, kb_n = (int)(p.K / 128);
  const int64_t t0 = (int64_t)(blockIdx.x / p.splits) * 16, t = t0 + lrow;
  const bool in = t < p.T;
  int id;
  const uint32_t any = chunk_ids(p, t0, lrow, id);
  const uint16_t* xr = p.x + (in ? t : t0) * p.ldx + lgrp * 8;
  v4f acc[RT];
  int64_t arow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    arow[rt] = (rt * 16 + lrow < p.r ? rt * 16 + lrow : p.r - 1) * p.K + lgrp * 8;
    acc[rt] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  for (int kb = share(kb_n, s, p.splits) + wave; kb < share(kb_n, s + 1, p.splits); kb += kW) {
    fv4i x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const fv4i*>(xr + kb * 128 + i * 32);
    for (uint32_t left = any; left != 0;) {
      const int a = __shfl(id, __builtin_ctz(left));
      left &= ~(uint32_t)__ballot(id == a);
      const uint16_t* A = p.A + (int64_t)a * p.r * p.K + kb * 128;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        v4f c = acc[rt];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c = mfma_bf16_16x16x32(as_bf16x8(*reinterpret_cast<const fv4i*>(A + arow[rt] + i * 32)), as_bf16x8(x[i]), c);
        if (id == a) acc[rt] = c;
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
    float sc = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 q = quant8_bf16_tile(d[i], m, sc);
      if (in) *reinterpret_cast<uint2*>(p.xq + t * p.K + kb * 128 + i * 32 + lgrp * 8) = q;
    }
    if (in && lgrp == 0) p.xs[kb * ld_s + t] = sc;
  }
  if (any == 0) return;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) part[wave][rt][lane] = acc[rt];
  __syncthreads();
  for (int rt = wave; rt < RT; rt += kW) {
    const int r0 = rt * 16 + lgrp * 4;
    if (id >= 0 && r0 < p.r) {
      v4f c = part[0][rt][lane];
#pragma unroll
      for (int w = 1; w < kW; ++w) c += part[w][rt][lane];
      *reinterpret_cast<v4f*>(p.zp + ((int64_t)s * p.T + t) * p.r + r0) = c;
    }
  }
}

// Prompts: the sums over the shares of K, as the GEMM's epilogue reads them
// (for every 8 ranks the 8 terms hi, then the 8 terms lo).
__global__ __launch_bounds__(256) void adapter_z_kernel(AdapterProblem p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int r8 = p.r / 8;
  if (i >= p.T * r8) return;
  v8bf hi, lo;
  z8(p, i / r8, (int)(i % r8) * 8, hi, lo);
  reinterpret_cast<v8bf*>(p.z)[2 * i] = hi;
  reinterpret_cast<v8bf*>(p.z)[2 * i + 1] = lo;
}

// 2. Few tokens: projection and expand, RT tiles of 16 output columns a
//    workgroup (every token operand is read once for them); the next K block's
//    weights are loaded before the present one's products.
template <int NT, int RT, int PW>
__global__ __launch_bounds__(PW * 64, 2) void adapter_project_kernel(AdapterProblem p) {
  __shared__ v4f part[PW][RT][64];
  extern __shared__ v8bf zs[];            // [T][r / 8][hi, lo]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int kb_n = (int)(p.K / 128), T = (int)p.T, r8 = p.r / 8;
  int tile[RT];                           // past the last one: the last one again, not stored
#pragma unroll
  for (int i = 0; i < RT; ++i) tile[i] = min((int)blockIdx.x * RT + i, (int)(p.N / 16) - 1);
  int tok[NT];
  uint32_t soff[NT];
  v4f acc[RT][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    tok[j] = j * 16 + lrow < T ? j * 16 + lrow : T - 1;
    soff[j] = (uint32_t)tok[j] * (uint32_t)kb_n;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  auto fetch = [&](int kb, Block (&a)[RT]) {
#pragma unroll
    for (int i = 0; i < RT; ++i) a[i] = load_tile(p.W + ((int64_t)tile[i] * kb_n + kb) * 2048, lane);
  };
  // the batch's adapters, in the order of their first token, and the tokens of each
  __shared__ int adapter[kAdapterFewTokens];
  __shared__ uint64_t member[kAdapterFewTokens];
  __shared__ int n_adapters;
  const int last = kb_n - 1;
  Block a0[RT], a1[RT];
  fetch(min(wave, last), a0);
  if (wave == PW - 1) {
    const int id = lane < T ? p.ids[lane] : -1;
    uint64_t left = __ballot(id >= 0);
    int n = 0;
    while (left != 0) {
      const int a = __shfl(id, __builtin_ctzll(left));
      const uint64_t m = __ballot(id == a);
      left &= ~m;
      if (lane == 0) {
        adapter[n] = a < p.n ? a : 0;      // its tokens' z is NaN
        member[n] = m;
      }
      ++n;
    }
    if (lane == 0) n_adapters = n;
  }
  for (int i = threadIdx.x; i < T * r8; i += PW * 64) z8(p, i / r8, (i % r8) * 8, zs[2 * i], zs[2 * i + 1]);
  __syncthreads();

  const v8bf none = __builtin_bit_cast(v8bf, fv4i{0, 0, 0, 0});
  const int n_ad = n_adapters;
  auto fetch_b = [&](int turn, int r0, v8bf (&bw)[RT]) {
    const uint16_t* brow = p.B + ((int64_t)adapter[turn] * p.N + lrow) * p.r;
    const int r = r0 + lgrp * 8;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      bw[i] = r < p.r ? *reinterpret_cast<const v8bf*>(brow + (int64_t)tile[i] * 16 * p.r + r) : none;
  };
  // a column's sums are kept in its own adapter's turn
  auto expand = [&](int turn, int r0, const v8bf (&bw)[RT]) {
    const uint64_t members = member[turn];
    const int r = r0 + lgrp * 8;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint32_t m = (uint32_t)(members >> (16 * j)) & 0xFFFFu;
      if (m == 0) continue;
      const int at = 2 * (tok[j] * r8 + r / 8);
      const v8bf hi = r < p.r ? zs[at] : none, lo = r < p.r ? zs[at + 1] : none;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const v4f c = mfma_bf16_16x16x32(bw[i], lo, mfma_bf16_16x16x32(bw[i], hi, acc[i][j]));
        if ((m >> lrow) & 1) acc[i][j] = c;
      }
    }
  };
  // One K block and one of the wave's adapters a step.  Loads return in the
  // order of their issue: the token operands of the present block are asked
  // for first, then the next block's weights and the adapter's.
  auto step = [&](int kb, int turn, const Block (&a)[RT], Block (&next)[RT]) {
    const int kc = min(kb, last);        // past the wave's last block: one that is not used
    Block b[NT];
    float c[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      b[j] = load_tile(p.xq + ((int64_t)j * kb_n + kc) * 2048, lane);
      c[j] = (p.xs + kc)[soff[j]];
    }
    __asm__ volatile("" ::: "memory");
    v8bf bw[RT];
    const bool ad = turn < n_ad;
    fetch(min(kb + PW, last), next);
    if (ad) fetch_b(turn, 0, bw);
    if (kb < kb_n) {
      float f[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) f[i] = p.sW[(tile[i] / 8) * p.ld_sw + kb];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v8i bj = as_operand(b[j]);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const v4f zero = {0.f, 0.f, 0.f, 0.f};
          const float cj = c[j] * f[i];
          const v4f q = mfma_e4m3_16x16x128(as_operand(a[i]), bj, zero);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(q[v], cj, acc[i][j][v]);
        }
      }
    }
    if (ad) {
      expand(turn, 0, bw);
      for (int r0 = 32; r0 < p.r; r0 += 32) {
        fetch_b(turn, r0, bw);
        expand(turn, r0, bw);
      }
    }
  };
  for (int kb = wave, turn = wave; kb < kb_n || turn < n_ad; kb += 2 * PW, turn += 2 * PW) {
    step(kb, turn, a0, a1);
    step(kb + PW, turn + PW, a1, a0);
  }
  for (int j = 0; j < NT; ++j) {
    if (j != 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      v4f v = acc[i][0];
#pragma unroll
      for (int q = 1; q < NT; ++q) v = j == q ? acc[i][q] : v;
      part[wave][i][lane] = v;
    }
    __syncthreads();
    for (int i = wave; i < RT; i += PW) {
      v4f c = part[0][i][lane];
#pragma unroll
      for (int q = 1; q < PW; ++q) c += part[q][i][lane];
      const int n = (blockIdx.x * RT + i) * 16;
      if (j * 16 + lrow < T && n < p.N) {
        const int64_t at = (j * 16 + lrow) * p.ldc + n + lgrp * 4;
        if (p.out_fp32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.C) + at) = make_float4(c[0], c[1], c[2], c[3]);
        } else {
          typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
          *reinterpret_cast<v4bf*>(static_cast<uint16_t*>(p.C) + at) = __builtin_convertvector(c, v4bf);
        }
      }
    }
  }
}

template <int NT, int RT, int PW>
void project(const AdapterProblem& p, hipStream_t stream) {
  const size_t lds = (size_t)p.T * p.r * 4;
  hipLaunchKernelGGL((adapter_project_kernel<NT, RT, PW>), dim3((unsigned)((p.N / 16 + RT - 1) / RT)),
                     dim3(PW * 64), lds, stream, p);
}

// Tiles of a workgroup: one workgroup of eight waves for each of the 256 CUs
// where up to 5 tiles suffice for that (more would not fit the registers), as
// a workgroup reads all token operands, which count like weights against its
// CU's load rate; wider outputs take several smaller workgroups a CU.
// Measured at K x N with rank 32, every token its own adapter, us:
//   7168 x 18432 (1152 tiles), 48 tokens: 1 tile 84, 2 70, 3 69, 4 79, 5 57;
//     2, 3 and 4 tiles with 4 waves 67, 62 and 68; 64 tokens: 5 tiles 66, 3 x 4 waves 76;
//   7168 x 16384 (1024 tiles), 48 tokens: 72, 55, 68, 51, 54; 4 x 4 waves 52;
//   7168 x 12288 (768 tiles), 48 tokens: 60, 53, 45, 47, 51; 3 x 4 waves 45;
//   7168 x 8320 (520 tiles), 48 tokens: 54, 50, 40, 44, 48; 3 x 4 waves 43;
//   18432 x 7168 (448 tiles), 48 tokens: 81, 63, 68, 75, 81;
//   4096 x 4096 (256 tiles), 64 tokens: 31, 32, 35, 38, 43;
//   1536 x 24576 (1536 tiles), 64 tokens: 80, 67, 54, 58, 67; 3 x 4 waves 46.
// With one token the same order, within a tenth (1024 tiles: 34, 31, 35, 31, 31).
template <int NT>
void project_few(const AdapterProblem& p, hipStream_t stream) {
  switch ((p.N / 16 + 255) / 256) {
    case 1: return project<NT, 1, 8>(p, stream);
    case 2: return project<NT, 2, 8>(p, stream);
    case 3: return project<NT, 3, 8>(p, stream);
    case 4: return project<NT, 4, 8>(p, stream);
    case 5: return project<NT, 5, 8>(p, stream);
    default: return project<NT, 3, 4>(p, stream);
  }
}

}  // namespace

template <int NT>
static void down(const MoeProblem& p, hipStream_t stream) {
  const int tiles = p.H / 16, cuts = moe_cuts(p.H);
  const size_t lds = ((size_t)8 * p.T * 20 + 2 + 2 * plan_parts(p) + 2 * p.T * p.top_k) * 4;
  hipLaunchKernelGGL((moe_down_kernel<NT, 8>), dim3(tiles * cuts), dim3(512), lds, stream, p, cuts);
  if (cuts > 1)
    hipLaunchKernelGGL(moe_combine_kernel, dim3((p.T * p.H + 255) / 256), dim3(256), 0, stream, p, cuts);
}

hipError_t launch_moe_few_tokens(const MoeProblem& p, hipStream_t stream) {
  const int t_tiles = (p.T + 15) / 16;
  const int router_blocks = (p.E + 15) / 16 * t_tiles * p.splits;
  hipLaunchKernelGGL(moe_prepare_kernel, dim3(router_blocks + quant_blocks(p.T, p.H)), dim3(kB), 0, stream, p,
                     router_blocks);
  const int up = p.local * (p.I / 16);
  // Tokens that an expert gets on average: how many groups of 16 a workgroup
  // takes in a pass over an expert's weights.  Measured with 1 / 2 / 4 groups, us a
  // call, all experts held, 64 tokens: on average 8 of them at 2048 x 1408 46 / 50 / 61,
  // 24 67 / 64 / 78; at 7168 x 2048 8 87 / 87 / 100, 10 91 / 93 / 105, 16 112 / 106 / 119,
  // 25 101 / 88 / 95, 32 88 / 79 / 81, 64 76 / 68 / 65; 32 tokens, 16 64 / 60 / 67.
  const int per = p.T * p.top_k / p.E;
  if (p.T <= kW && p.E <= 64) {
    hipLaunchKernelGGL((moe_up_kernel<1, false>), dim3(1 + up), dim3(kB), 0, stream, p, 1);
  } else {
    const dim3 route((p.T + 3) / 4);
    if (p.E <= 64) hipLaunchKernelGGL(moe_route_kernel<1>, route, dim3(256), 0, stream, p);
    else if (p.E <= 256) hipLaunchKernelGGL(moe_route_kernel<4>, route, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(moe_route_kernel<kMoeMaxExperts / 64>, route, dim3(256), 0, stream, p);
    if (per <= 8) hipLaunchKernelGGL((moe_up_kernel<1, true>), dim3(up), dim3(kB), 0, stream, p, 0);
    else if (per <= 32) hipLaunchKernelGGL((moe_up_kernel<2, true>), dim3(up), dim3(kB), 0, stream, p, 0);
    else hipLaunchKernelGGL((moe_up_kernel<4, true>), dim3(up), dim3(kB), 0, stream, p, 0);
  }
  const int span = per <= 8 ? 16 : per <= 32 ? 32 : 64;
  hipLaunchKernelGGL(moe_quant_kernel, dim3(1 + quant_blocks((int64_t)p.T * p.top_k, p.I)), dim3(kB), 0, stream, p,
                     span);
  if (span == 16) down<1>(p, stream);
  else if (span == 32) down<2>(p, stream);
  else down<4>(p, stream);
  return hipGetLastError();
}

hipError_t launch_adapter_few(const AdapterProblem& p, hipStream_t stream) {
  const int chunks = (int)((p.T + 15) / 16), rts = (p.r + 15) / 16;
  const int step = p.T < 16 ? (int)p.T : 16;
  const int shrink_blocks = chunks * rts * step * p.splits;
  hipLaunchKernelGGL(adapter_prepare_kernel, dim3(shrink_blocks + quant_blocks(p.T, p.K)), dim3(kB), 0, stream, p,
                     shrink_blocks, step);
  switch (chunks) {
    case 1: project_few<1>(p, stream); break;
    case 2: project_few<2>(p, stream); break;
    case 3: project_few<3>(p, stream); break;
    default: project_few<4>(p, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_adapter_prompt(const AdapterProblem& p, int64_t ld_s, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 15) / 16 * p.splits));
  if (p.r <= 16) hipLaunchKernelGGL(adapter_prompt_kernel<1>, grid, dim3(kB), 0, stream, p, ld_s);
  else if (p.r <= 32) hipLaunchKernelGGL(adapter_prompt_kernel<2>, grid, dim3(kB), 0, stream, p, ld_s);
  else if (p.r <= 64) hipLaunchKernelGGL(adapter_prompt_kernel<4>, grid, dim3(kB), 0, stream, p, ld_s);
  else hipLaunchKernelGGL(adapter_prompt_kernel<8>, grid, dim3(kB), 0, stream, p, ld_s);
  hipLaunchKernelGGL(adapter_z_kernel, dim3((unsigned)((p.T * (p.r / 8) + 255) / 256)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bs
