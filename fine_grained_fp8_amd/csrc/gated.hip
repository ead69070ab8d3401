// The gated feed-forward block's own kernels for gfx950: the product for few tokens,
// and the backward pass up to the operands of Dgrad and Wgrad.  (More tokens: the
// block GEMM with its gated epilogue, gemm.hip.)
//
//   a = X W1^T, u = X W3^T,  h = act(a) u,  act(a) = a logistic(v(a))
//   da = dh u act'(a),  du = dh act(a)
//   act'(a) = z + a z (1 - z) v'(a),  z = logistic(v(a))
#include <atomic>

#include "block_rules.hpp"
#include "blocks.hpp"
#include "device.hpp"
#include "gate.hpp"
#include "operands.hpp"
#include "rows.hpp"

namespace fp8bs {

namespace {

typedef int gv4i __attribute__((ext_vector_type(4)));
typedef int gv2i __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

// ===========================================================================
// Few tokens, or few tiles
// ===========================================================================

constexpr int kRowWaves = 8;                     // waves of a workgroup of the kernel for up to 16 tokens

__device__ __forceinline__ float gated(float a, float u, int gelu) {
  return a * logistic(gelu ? gelu_argument(a) : a) * u;
}

// wait until at most n vector-memory operations of this wave are outstanding and
// all LDS and scalar ones are done
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | (0 << 8) | ((n >> 4) << 14));
}

// 4 channels of a token, from n: the sums for the finishing launch, or what the call
// asked for
__device__ __forceinline__ void leave(const GatedFewProblem& p, int cut, int t, int64_t n, const v4f& a, const v4f& u) {
  if (p.cuts > 1) {
    float* at = p.parts + ((int64_t)cut * p.M + t) * 2 * p.N + n;
    *reinterpret_cast<v4f*>(at) = a;
    *reinterpret_cast<v4f*>(at + p.N) = u;
    return;
  }
  if (p.gated.gate_up != nullptr) {
    uint16_t* at = p.gated.gate_up + t * p.gated.ld_gu + n;
    *reinterpret_cast<v4bf*>(at) = __builtin_convertvector(a, v4bf);
    *reinterpret_cast<v4bf*>(at + p.N) = __builtin_convertvector(u, v4bf);
  }
  v4f h;
#pragma unroll
  for (int v = 0; v < 4; ++v) h[v] = gated(a[v], u[v], p.gated.gelu);
  if (p.gated.q != nullptr) *reinterpret_cast<v4f*>(p.parts + t * p.N + n) = h;
  else if (p.out_fp32) *reinterpret_cast<v4f*>(static_cast<float*>(p.C) + t * p.ldc + n) = h;
  else *reinterpret_cast<v4bf*>(static_cast<uint16_t*>(p.C) + t * p.ldc + n) = __builtin_convertvector(h, v4bf);
}

// Up to 16 tokens and 8192 channels.  A workgroup has RT tiles of 16 channels, the gate rows and
// the up rows of each; its eight waves deal the K blocks of its share (all of
// K, unless its codes would not fit LDS).  The weights go from memory straight
// into MFMA operand registers, D blocks of a wave in flight.  The token codes are
// copied into LDS first (DMA, in operand order: 1 KB for 16 tokens and 64 bytes of
// K), so that the loop's only loads from memory are weights: loads return in the
// order of their issue, and a token operand asked for in the loop would wait for
// all weights asked for before it.
// What bounds it: reading the weights (one token, 7168 x 8192: 117 MB in 24 us, 4.9
// TB/s), and for small ones the latency of a launch and of the first load (7168 x 2048,
// 29 MB: 10.4 us; 2048 x 1408: 5.1).
template <int RT, int D>
__global__ __launch_bounds__(kRowWaves * 64) void gated_row_kernel(GatedFewProblem p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];   // codes [share][2048], scales [share][16]; then sums
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int kb_n = (int)(p.K / 128), M = p.M;
  const int cut = blockIdx.x % p.cuts, group = blockIdx.x / p.cuts;
  const int kb0 = (int)((int64_t)kb_n * cut / p.cuts), kb1 = (int)((int64_t)kb_n * (cut + 1) / p.cuts), share = kb1 - kb0;
  const int tiles = (int)(p.N / 16);
  // the token codes; tokens past the last one lie outside of the buffer and read as zero
  using lds_u8 = __attribute__((address_space(3))) uint8_t;
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)p.A, (short)0, (int)((M - 1) * p.lda + p.K), 0x00020000);
  for (int o = wave; o < share * 2; o += kRowWaves) {
    const uint32_t at = lrow < M ? (uint32_t)(lrow * (int)p.lda + (kb0 + o / 2) * 128 + (o & 1) * 64 + lgrp * 16) : 0xFFFFFF00u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)((lds_u8*)lds + o * 1024), 16, at, 0, 0, 0);
  }
  float* scales = reinterpret_cast<float*>(lds + share * 2048);
  for (int i = threadIdx.x; i < share * 16; i += kRowWaves * 64)
    scales[i] = (i & 15) < M ? p.sA[(int64_t)(kb0 + i / 16) * p.ld_sa + (i & 15)] : 0.f;
  const uint8_t* w[RT][2];
  const float* s[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int t = min(group * RT + i, tiles - 1);      // past the last one: the last one again, not stored
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      w[i][g] = p.W + ((int64_t)g * tiles + t) * kb_n * 2048 + lane * 16;
      s[i][g] = p.sW + ((int64_t)g * (tiles / 8) + t / 8) * p.ld_sw;
    }
  }
  v4f acc[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = v4f{0.f, 0.f, 0.f, 0.f};
  auto fetch = [&](int kb, Block (&b)[RT][2]) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint8_t* at = w[i][g] + (int64_t)kb * 2048;
        b[i][g] = Block{*reinterpret_cast<const gv4i*>(at), *reinterpret_cast<const gv4i*>(at + 1024)};
      }
  };
  __asm__ volatile("" ::: "memory");
  Block b[D][RT][2];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (kb0 + wave + d * kRowWaves < kb1) fetch(kb0 + wave + d * kRowWaves, b[d]);
  // the wave's copies into LDS have landed when only the D blocks asked for after
  // them are outstanding; a bare barrier, which leaves those in flight
  __asm__ volatile("" ::: "memory");
  if (kb0 + wave + (D - 1) * kRowWaves < kb1) wait_loads<D * RT * 4>();
  else wait_loads<0>();
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
  auto products = [&](int kb, const Block (&b)[RT][2]) {
    const uint8_t* at = lds + (kb - kb0) * 2048 + lane * 16;
    const float sc = scales[(kb - kb0) * 16 + lrow];
    const Bf16Block x = to_bf16(Block{*reinterpret_cast<const gv4i*>(at), *reinterpret_cast<const gv4i*>(at + 1024)});
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float c = sc * s[i][g][kb];
        const v4f q = block_product(to_bf16(b[i][g]), x);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][g][v] = __builtin_fmaf(q[v], c, acc[i][g][v]);
      }
  };
  for (int k0 = kb0 + wave; k0 < kb1; k0 += D * kRowWaves) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int kb = k0 + d * kRowWaves;
      if (kb >= kb1) break;
      products(kb, b[d]);
      if (kb + D * kRowWaves < kb1) fetch(kb + D * kRowWaves, b[d]);
    }
  }
  v4f (*part)[RT][2][64] = reinterpret_cast<v4f (*)[RT][2][64]>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    part[wave][i][0][lane] = acc[i][0];
    part[wave][i][1][lane] = acc[i][1];
  }
  __syncthreads();
  for (int i = wave; i < RT; i += kRowWaves) {
    v4f a = part[0][i][0][lane], u = part[0][i][1][lane];
#pragma unroll
    for (int q = 1; q < kRowWaves; ++q) {
      a += part[q][i][0][lane];
      u += part[q][i][1][lane];
    }
    const int tile = group * RT + i;
    if (lrow < M && tile < tiles) leave(p, cut, lrow, tile * 16 + lgrp * 4, a, u);
  }
}

// More tokens or channels, in blocks of 16 NT tokens, to where the block GEMM takes over.  A wave has RT
// tiles of 16 channels, the gate rows and the up rows of each, for every token of its
// block; a workgroup's W waves have neighbouring tiles, and `cuts` workgroups share
// the K blocks.  Weights go from memory straight into MFMA operand
// registers; the token codes, which the waves share, through LDS by DMA.  Both are
// asked for D blocks ahead, in the order they are needed (loads return in the
// order of their issue); one barrier a block.  Measured against the waves dealing the
// K blocks, each with its own token operands (as for up to 16 tokens), us: 64
// tokens, 7168 x 18432 58 for 99 (a workgroup's tokens are read once for its four
// waves; with five, few_waves(), 48 to 58 from run to run), 48 tokens, 7168 x 2048 14.3 for 15.6, 64 tokens, 2048 x 1408 10.4 for 10.0; one
// token, 7168 x 2048 11.8 for 9.8, 7168 x 18432 47.7 for 50 (264 MB: 5.5 TB/s).  kExact: products of the codes as BF16, exact with FP32
// sums, so that FP32 values, scales and codes do not move with the FP8 instruction's
// truncation (exact_products(); 64 tokens, 7168 x 18432: 61 us for 49).
// What bounds it: a CU's loads, 25 - 30 bytes a clock of weights and token codes alike,
// and one wave a SIMD whose products and folds take as long (1333 tokens, 2048 x 1408: loads
// alone 12 us, products alone 14, both 14.7; 700, 7168 x 2048: 32, 32 and 38).
template <int NT, int RT, int D, bool kExact, int W>
__global__ __launch_bounds__(64 * W) void gated_few_kernel(GatedFewProblem p) {
  static_assert(RT == 1 || W == 4);
  constexpr int kTokens = NT * 2048, kStage = kTokens + 256 + W * 256;   // codes, token scales, each wave's two weight scales
  constexpr int kXOps = (NT * 2 + W - 1) / W, kOps = kXOps + 2 + 4 * RT;     // loads of a wave for one block
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];        // [D + 1][kStage]
  using lds_u8 = __attribute__((address_space(3))) uint8_t;
  using lds_ptr = __attribute__((address_space(3))) void*;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int kb_n = (int)(p.K / 128), tiles = (int)(p.N / 16);
  // workgroups of the same tiles follow each other: the token blocks, and for each the cuts
  const int blocks = (p.M + NT * 16 - 1) / (NT * 16);
  // on one XCD (workgroup i starts on XCD i % 8), whose L2 then has their weights once (700
  // tokens, 2048 x 1408: 13.1 to 10.8 us; 1333: 17.5 to 16.4; 512, 7168 x 2048: 39 to 33)
  const int xcd = blockIdx.x & 7, each = gridDim.x >> 3;
  const int id = blocks == 1 ? blockIdx.x : xcd * each + min(xcd, (int)(gridDim.x & 7)) + (blockIdx.x >> 3);
  const int cut = id % p.cuts, block = id / p.cuts % blocks;
  const int first = (id / p.cuts / blocks * W + wave) * RT;                          // the wave's first tile
  const int t0 = W == 4 ? first : min(first, tiles - 1);                             // past the last one: that one again, not stored
  const int m0 = block * NT * 16, M = min(p.M - m0, NT * 16);
  const int kb0 = (int)((int64_t)kb_n * cut / p.cuts), n = (int)((int64_t)kb_n * (cut + 1) / p.cuts) - kb0;
  // buffers end behind the last token and the last scale: what lies past them reads as zero
  const __amdgpu_buffer_rsrc_t rsrc_x = __builtin_amdgcn_make_buffer_rsrc((void*)(p.A + m0 * p.lda), (short)0, (int)((M - 1) * p.lda + p.K), 0x00020000);
  const __amdgpu_buffer_rsrc_t rsrc_s =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.sW, (short)0, (int)(2 * (p.N / 128) * p.ld_sw * 4), 0x00020000);
  // DMA instruction o of a block: rows 8 o .. + 7, 128 bytes each, 16-byte chunks XOR-swizzled by row & 7
  const uint32_t x_off = (uint32_t)((lane >> 3) * (int)p.lda + (((lane & 7) ^ (lane >> 3)) << 4));
  const uint32_t s_off = (uint32_t)((t0 / 8 + (lane >= 32 ? tiles / 8 : 0)) * (int)p.ld_sw) * 4u;
  const uint8_t* w[RT][2];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int g = 0; g < 2; ++g) w[i][g] = p.W + ((int64_t)g * tiles + t0 + i) * kb_n * 2048 + lane * 16;
  v8i b[D][RT][2];
  // Step k's block.  Workgroups of the same weights ask for them at the same time, and
  // neighbouring token blocks take four blocks in another order each, so that they
  // meet at different channels of the L2 (700 tokens, 7168 x 2048: 42.5 to 38 us; 2560 x
  // 2048 18.5 to 17.3; not for 16 blocks: 1333 tokens, 2048 x 1408 14.6 to 15.0).
  const int turn = n >= 20 ? block & 3 : 0;
  auto block_of = [&](int k) {
    const int t = k ^ turn;
    return kb0 + (t < n ? t : k);
  };
  auto issue_shared = [&](int k, int stage) {
    lds_u8* st = (lds_u8*)lds + stage * kStage;
    const int kb = block_of(k);
#pragma unroll
    for (int q = 0; q < kXOps; ++q) {
      int o = wave * kXOps + q;
      if constexpr (kXOps * W != NT * 2) o = o < NT * 2 ? o : NT * 2 - 1;       // again: every wave counts the same loads
      const uint32_t at = x_off + (uint32_t)(kb * 128 + o * 8 * (int)p.lda);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_x, (lds_ptr)(st + o * 1024), 16, at, 0, 0, 0);
    }
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)(p.sA + (int64_t)kb * p.ld_sa + m0), (short)0, M * 4, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr)(st + kTokens), 4, (uint32_t)lane * 4u, 0, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_s, (lds_ptr)(st + kTokens + 256 + wave * 256), 4, s_off + (uint32_t)kb * 4u, 0, 0, 0);
    __asm__ volatile("" ::: "memory");
  };
  auto issue_weight = [&](int k, int i, int g) {
    const uint8_t* at = w[i][g] + (int64_t)block_of(k) * 2048;
    const gv4i lo = *reinterpret_cast<const gv4i*>(at), hi = *reinterpret_cast<const gv4i*>(at + 1024);
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  v4f acc[RT][2][NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i][0][j] = acc[i][1][j] = v4f{0.f, 0.f, 0.f, 0.f};
  auto operand = [&](const v8i& v) {
    if constexpr (kExact)
      return Bf16Block{{codes_to_bf16(v[0], v[1]), codes_to_bf16(v[2], v[3]), codes_to_bf16(v[4], v[5]), codes_to_bf16(v[6], v[7])}};
    else
      return v;
  };
  // the products of a step, and the weights of block `ahead` into the registers that they leave
  auto products = [&](int stage, v8i (&f)[RT][2], int ahead) {
    const uint8_t* st = lds + stage * kStage;
    const float* sx = reinterpret_cast<const float*>(st + kTokens) + lrow;
    const float* sw = reinterpret_cast<const float*>(st + kTokens + 256 + wave * 256);
    const float cg = sw[0], cu = sw[32];
    const uint8_t* at = st + lrow * 128;
    decltype(operand(v8i{})) x[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const gv4i lo = *reinterpret_cast<const gv4i*>(at + j * 2048 + ((lgrp ^ (lrow & 7)) << 4));
      const gv4i hi = *reinterpret_cast<const gv4i*>(at + j * 2048 + (((4 + lgrp) ^ (lrow & 7)) << 4));
      x[j] = operand(v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
    float c[2][NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float t = sx[j * 16];
      c[0][j] = t * cg;
      c[1][j] = t * cu;
    }
    v4f q[2][NT];
    auto fold = [&](int n) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[n >> 1][n & 1][j][v] = __builtin_fmaf(q[n & 1][j][v], c[n & 1][j], acc[n >> 1][n & 1][j][v]);
    };
    // product n on the matrix unit while n - 1 is folded and n's registers are asked for again:
    // the loads in one burst after the products, their issue and the folds were as long as
    // the products (1333 tokens, 2048 x 1408: 17.1 to 14.7 us; 700, 7168 x 2048: 48.6 to 42.5)
#pragma unroll
    for (int n = 0; n < 2 * RT; ++n) {
      const int i = n >> 1, g = n & 1;
      const auto wf = operand(f[i][g]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (kExact) q[g][j] = block_product(wf, x[j]);
        else q[g][j] = mfma_e4m3_16x16x128(wf, x[j], v4f{0.f, 0.f, 0.f, 0.f});
      }
      f[i][g] = issue_weight(ahead, i, g);
      if (n > 0) fold(n - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    fold(2 * RT - 1);
  };
  // Past the share's last block its loads are asked for again (not used), so that
  // every step counts the same loads.
#pragma unroll
  for (int d = 0; d < D; ++d) {
    issue_shared(d < n ? d : n - 1, d);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int g = 0; g < 2; ++g) b[d][i][g] = issue_weight(d < n ? d : n - 1, i, g);
    __asm__ volatile("" ::: "memory");
  }
  int stage = 0;
  auto step = [&](int k, v8i (&f)[RT][2]) {
    wait_loads<(D - 1) * kOps>();
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    const int ahead = k + D < n ? k + D : n - 1;
    issue_shared(ahead, stage == 0 ? D : stage - 1);     // the stage of the step before: every wave is past its reads
    products(stage, f, ahead);
    __asm__ volatile("" ::: "memory");
    stage = stage == D ? 0 : stage + 1;
  };
  int k = 0;
  for (; k + D <= n; k += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) step(k + d, b[d]);
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (k + d < n) step(k + d, b[d]);
  wait_loads<0>();     // the loads asked for again land before the workgroup's LDS goes
  if constexpr (RT == 2) {
    if (p.gated.q != nullptr && p.cuts == 1) {
      // the workgroup has whole 1x128 tiles: their maxima over the waves, the codes
      // through LDS into whole rows
      __syncthreads();
      uint32_t* most = reinterpret_cast<uint32_t*>(lds + NT * 2048);      // [wave][16 NT]
      float h[NT][8];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          h[j][v] = gated(acc[v >> 2][0][j][v & 3], acc[v >> 2][1][j][v & 3], p.gated.gelu);
          m = max(m, __float_as_uint(h[j][v]) & 0x7FFFFFFFu);
        }
        const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
        m = max(a[0], a[1]);
        const auto c = __builtin_amdgcn_permlane32_swap(m, m, false, false);
        m = max(c[0], c[1]);
        if (lgrp == 0) most[wave * NT * 16 + j * 16 + lrow] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = j * 16 + lrow;
        const uint32_t m = max(max(most[t], most[NT * 16 + t]), max(most[2 * NT * 16 + t], most[3 * NT * 16 + t]));
        float sc;
        const uint2 q = quant8_f32(h[j], m, sc);
        uint8_t* row = lds + t * 128 + lgrp * 4;
        *reinterpret_cast<uint32_t*>(row + (((wave * 2) ^ (t & 7)) << 4)) = q.x;
        *reinterpret_cast<uint32_t*>(row + (((wave * 2 + 1) ^ (t & 7)) << 4)) = q.y;
        if (wave == 0 && lgrp == 0 && t < M) p.gated.s[(t0 / 8) * p.gated.ld_s + m0 + t] = sc;
        if (p.gated.gate_up != nullptr && t < M) {
          uint16_t* at = p.gated.gate_up + (m0 + t) * p.gated.ld_gu + t0 * 16 + lgrp * 4;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<v4bf*>(at + i * 16) = __builtin_convertvector(acc[i][0][j], v4bf);
            *reinterpret_cast<v4bf*>(at + p.N + i * 16) = __builtin_convertvector(acc[i][1][j], v4bf);
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < M * 8; i += 256) {
        const int t = i >> 3, ch = i & 7;
        *reinterpret_cast<gv4i*>(p.gated.q + (m0 + t) * p.gated.ldq + (t0 / 8) * 128 + ch * 16) =
            *reinterpret_cast<const gv4i*>(lds + t * 128 + ((ch ^ (t & 7)) << 4));
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = j * 16 + lrow;
    if (t >= M || (W != 4 && first >= tiles)) continue;
#pragma unroll
    for (int i = 0; i < RT; ++i) leave(p, cut, m0 + t, (int64_t)(t0 + i) * 16 + lgrp * 4, acc[i][0][j], acc[i][1][j]);
  }
}

// What the product's workgroups left: the sums of a cut tile, and the codes
// of h (a 1x128 tile spans eight 16-channel tiles).  16 lanes a tile.
__global__ __launch_bounds__(256) void gated_finish_kernel(GatedFewProblem p) {
  const int kb_n = (int)(p.N / 128), tile = blockIdx.x * 16 + (threadIdx.x >> 4), l16 = threadIdx.x & 15;
  if (tile >= p.M * kb_n) return;                 // whole 16-lane groups
  const int t = tile / kb_n, kb = tile - t * kb_n;
  const int64_t n = kb * 128 + l16 * 8;
  float h[8];
  if (p.cuts > 1) {
    const float* src = p.parts + (int64_t)t * 2 * p.N + n;
    const int64_t step = (int64_t)p.M * 2 * p.N;
    v4f a[2], u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = *reinterpret_cast<const v4f*>(src + 4 * k);
      u[k] = *reinterpret_cast<const v4f*>(src + p.N + 4 * k);
    }
    for (int c = 1; c < p.cuts; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        a[k] += *reinterpret_cast<const v4f*>(src + c * step + 4 * k);
        u[k] += *reinterpret_cast<const v4f*>(src + c * step + p.N + 4 * k);
      }
    if (p.gated.gate_up != nullptr) {
      uint16_t* at = p.gated.gate_up + t * p.gated.ld_gu + n;
      *reinterpret_cast<gv4i*>(at) = gv4i{bf16_pair(a[0][0], a[0][1]), bf16_pair(a[0][2], a[0][3]),
                                          bf16_pair(a[1][0], a[1][1]), bf16_pair(a[1][2], a[1][3])};
      *reinterpret_cast<gv4i*>(at + p.N) = gv4i{bf16_pair(u[0][0], u[0][1]), bf16_pair(u[0][2], u[0][3]),
                                                bf16_pair(u[1][0], u[1][1]), bf16_pair(u[1][2], u[1][3])};
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = gated(a[k >> 2][k & 3], u[k >> 2][k & 3], p.gated.gelu);
  } else {
    const float* src = p.parts + t * p.N + n;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = src[k];
  }
  if (p.gated.q != nullptr) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(h[k]) & 0x7FFFFFFFu);
    float sc;
    const uint2 q = quant8_f32(h, row16_max_u32(m), sc);
    *reinterpret_cast<gv2i*>(p.gated.q + t * p.gated.ldq + n) = gv2i{(int)q.x, (int)q.y};
    if (l16 == 0) p.gated.s[kb * p.gated.ld_s + t] = sc;
  } else if (p.out_fp32) {
    float* at = static_cast<float*>(p.C) + t * p.ldc + n;
    *reinterpret_cast<float4*>(at) = make_float4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<float4*>(at + 4) = make_float4(h[4], h[5], h[6], h[7]);
  } else {
    *reinterpret_cast<gv4i*>(static_cast<uint16_t*>(p.C) + t * p.ldc + n) =
        gv4i{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3]), bf16_pair(h[4], h[5]), bf16_pair(h[6], h[7])};
  }
}

// A launch with its dynamic LDS.  More than 64 KB has to be announced, once for
// each kernel and device.
template <auto kKernel>
hipError_t start(int64_t grid, int block, int64_t lds, const GatedFewProblem& p, hipStream_t stream) {
  static std::atomic<uint64_t> announced{0};       // a bit for each device
  if (lds > 65536) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    if ((announced.load(std::memory_order_relaxed) & bit) == 0) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel), hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
      if (e != hipSuccess) return e;
      announced.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(kKernel, dim3((unsigned)grid), dim3(block), lds, stream, p);
  return hipGetLastError();
}

template <int RT, int D>
hipError_t row(const GatedFewProblem& p, hipStream_t stream) {
  const int64_t share = (p.K / 128 + p.cuts - 1) / p.cuts, sums = (int64_t)kRowWaves * RT * 2048;
  const int64_t codes = share * kRowBlockLds;
  return start<gated_row_kernel<RT, D>>((p.N / 16 + RT - 1) / RT * p.cuts, kRowWaves * 64, codes > sums ? codes : sums, p, stream);
}

template <int NT, int RT, int D, bool kExact, int W>
hipError_t few(const GatedFewProblem& p, hipStream_t stream) {
  const int64_t blocks = (p.M + NT * 16 - 1) / (NT * 16), groups = (p.N / 16 + W * RT - 1) / (W * RT);
  return start<gated_few_kernel<NT, RT, D, kExact, W>>(groups * blocks * p.cuts, 64 * W, (D + 1) * (NT * 2048 + 256 + W * 256), p,
                                                       stream);
}
// FP32 values leave: an FP32 result, or codes of one
bool fp32_values(const GatedFewProblem& p) { return p.gated.q != nullptr || p.out_fp32; }
bool has_whole_tiles(const GatedFewProblem& p) { return whole_tiles(p.M, p.N, fp32_values(p)); }
template <int NT, bool kExact>
hipError_t few_tokens(const GatedFewProblem& p, hipStream_t stream) {
  const int w = few_waves(p.M, p.N);
  if constexpr (!kExact) {
    // of more than 64 tokens, codes need whole tiles or a launch more
    if (has_whole_tiles(p) && (w == 4 || p.gated.q != nullptr)) return few<NT, 2, 2, false, 4>(p, stream);
  }
  return w == 5 ? few<NT, 1, 3, kExact, 5>(p, stream) : w == 6 ? few<NT, 1, 3, kExact, 6>(p, stream) : few<NT, 1, 3, kExact, 4>(p, stream);
}
template <int NT>
hipError_t few_tokens(const GatedFewProblem& p, hipStream_t stream) {
  return exact_products(p.M, fp32_values(p)) ? few_tokens<NT, true>(p, stream) : few_tokens<NT, false>(p, stream);
}

// ===========================================================================
// Backward
// ===========================================================================

// quotient y / s of the online rule, as in quant8_f32: r + l = 1 / s
struct ScaleInverse {
  float r, l;
};
// scale of a tile from its |y| maximum's bits; infinite or NaN: r = l = 0 or NaN
__device__ __forceinline__ float tile_scale_f32(uint32_t amax_bits, ScaleInverse& inv) {
  if (amax_bits >= 0x7F800000u) {
    inv.r = inv.l = amax_bits == 0x7F800000u ? 0.0f : NAN;
    return __uint_as_float(amax_bits == 0x7F800000u ? amax_bits : kCanonicalNaN);
  }
  const float s = fmaxf(div448_bf16(__uint_as_float(amax_bits)), scale_floor());
  inv.r = __uint_as_float(__float_as_uint(__builtin_amdgcn_rcpf(s)) - 2u);
  const float e = __builtin_fmaf(-s, inv.r, 1.0f);
  inv.l = inv.r * __builtin_fmaf(e, e, e);
  return s;
}
__device__ __forceinline__ float quotient(float y, const ScaleInverse& i) { return __builtin_fmaf(y, i.r, y * i.l); }

// One 128 x 128 block of tokens x channels: dh, gate and up are read once, da
// and du (and h) stay in registers as FP32 for both orientations' codes.  Lane
// (sub, l16) of wave w has kGR consecutive rows and channels 8 l16 .. + 7, so that a row
// tile is one 16-lane DPP row and a column's codes are packed in the lane; the
// columns' maxima and the transposed codes meet in LDS.  Tokens past the last one are
// zeros, which the transposed codes are padded with.
// Bound by memory with the vector unit close behind: 4096 x 18432, 755 MB, 170 us (4.4
// TB/s; BF16 gradients alone 140).  The registers decide: at most 128 let two workgroups
// of 512 lanes share a CU (left to the compiler, 131: one, 222 us); with h three
// sets of values need 1024 lanes of two rows (242 us; four rows: 342 with spills; four
// rows with gate and up asked for again, for h alone, after da and du: 243).
// kOne: one of the sets, which blockIdx.y names.
template <bool kH, int kGR, int kWavesPerSimd, bool kOne = false>
__global__ __launch_bounds__(2048 / kGR, kWavesPerSimd) void gated_backward_kernel(GatedGradProblem p) {
  constexpr int kGW = 32 / kGR, kGB = kGW * 64;              // waves and threads: kGR rows a lane
  constexpr int kSets = kOne ? 1 : kH ? 3 : 2;               // da, du, h
  __shared__ uint32_t most[kSets][kGW][128];
  __shared__ __attribute__((aligned(16))) float inv[kSets][2][128];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kSets][128 * 128];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane >> 4, l16 = lane & 15;
  const int64_t ncb = p.I / 128, nrb = (p.T + 127) / 128;
  const int64_t rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int first = kOne ? blockIdx.y : 0;                   // the workgroup's first set
  const int64_t r0 = rb * 128 + wave * 4 * kGR + sub * kGR, c0 = cb * 128 + l16 * 8;

  float y[kSets][kGR][8];
  {
    gv4i dh[kGR], g[kGR], u[kGR];
#pragma unroll
    for (int i = 0; i < kGR; ++i) {
      dh[i] = g[i] = u[i] = gv4i{0, 0, 0, 0};
      if (r0 + i < p.T) {
        const uint16_t* gu = p.gate_up + (r0 + i) * p.ld_gu + c0;
        dh[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(p.dh + (r0 + i) * p.ld_dh + c0));
        g[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(gu));
        u[i] = __builtin_nontemporal_load(reinterpret_cast<const gv4i*>(gu + p.I));
      }
    }
#pragma unroll
    for (int i = 0; i < kGR; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t gw = (uint32_t)g[i][k >> 1], uw = (uint32_t)u[i][k >> 1], dw = (uint32_t)dh[i][k >> 1];
        const float a = (k & 1) ? bf16_hi(gw) : bf16_lo(gw), b = (k & 1) ? bf16_hi(uw) : bf16_lo(uw);
        const float d = (k & 1) ? bf16_hi(dw) : bf16_lo(dw);
        const float z = logistic(p.gelu ? gelu_argument(a) : a);
        const float f = a * z;                               // act(a)
        const float slope = p.gelu ? gelu_argument_slope(a) : 1.0f;
        const float da = d * b * __builtin_fmaf(f * (1.0f - z), slope, z), du = d * f, h = f * b;
        if constexpr (kOne) {
          y[0][i][k] = first == 0 ? da : first == 1 ? du : h;
        } else {
          y[0][i][k] = da;
          y[1][i][k] = du;
          if constexpr (kH) y[2][i][k] = h;
        }
      }
  }

  // row tiles, from registers
#pragma unroll
  for (int n = 0; n < kSets; ++n) {
    const int m = first + n;
    if (m == 2) break;                                       // h has none
    const int64_t col = m * p.I + c0;
    if (p.d != nullptr) {
#pragma unroll
      for (int i = 0; i < kGR; ++i)
        if (r0 + i < p.T) {
          const float* v = y[n][i];
          __builtin_nontemporal_store(gv4i{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                                      reinterpret_cast<gv4i*>(p.d + (r0 + i) * p.ld_d + col));
        }
    }
    if (p.q != nullptr) {
#pragma unroll
      for (int i = 0; i < kGR; ++i) {
        uint32_t t = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(y[n][i][k]) & 0x7FFFFFFFu);
        float s;
        const uint2 q = quant8_f32(y[n][i], row16_max_u32(t), s);
        if (r0 + i < p.T) {
          __builtin_nontemporal_store(gv2i{(int)q.x, (int)q.y}, reinterpret_cast<gv2i*>(p.q + (r0 + i) * p.ldq + col));
          if (l16 == 0) p.s[(m * ncb + cb) * p.ld_s + r0 + i] = s;
        }
      }
    }
  }
  if (p.qt == nullptr && (!kH || (kOne && first < 2))) return;

  // column tiles: their maxima over the waves
#pragma unroll
  for (int m = 0; m < kSets; ++m) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < kGR; ++i) t = max(t, __float_as_uint(y[m][i][k]) & 0x7FFFFFFFu);
      const auto a = __builtin_amdgcn_permlane16_swap(t, t, false, false);
      t = max(a[0], a[1]);
      const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
      t = max(b[0], b[1]);
      if (sub == 0) most[m][wave][l16 * 8 + k] = t;
    }
  }
  __syncthreads();
  if (threadIdx.x < kSets * 128) {
    const int n = threadIdx.x >> 7, m = first + n, c = threadIdx.x & 127;
    uint32_t t = most[n][0][c];
#pragma unroll
    for (int w = 1; w < kGW; ++w) t = max(t, most[n][w][c]);
    ScaleInverse v;
    const float s = tile_scale_f32(t, v);
    inv[n][0][c] = v.r;
    inv[n][1][c] = v.l;
    if (m == 2) p.hst[rb * p.ld_hst + cb * 128 + c] = s;
    else if (p.qt != nullptr) p.st[rb * p.ld_st + m * p.I + cb * 128 + c] = s;
  }
  __syncthreads();
  // codes: column c's 128 bytes (tokens) at c * 128, 16-byte chunks XOR-swizzled by c / 8
#pragma unroll
  for (int m = 0; m < kSets; ++m) {
    float r[8], l[8];
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const v4f a = *reinterpret_cast<const v4f*>(&inv[m][0][l16 * 8 + k]);
      const v4f b = *reinterpret_cast<const v4f*>(&inv[m][1][l16 * 8 + k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[k + e] = a[e];
        l[k + e] = b[e];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const ScaleInverse v{r[k], l[k]};
      float q[kGR];
#pragma unroll
      for (int i = 0; i < kGR; ++i) q[i] = quotient(y[m][i][k], v);
      // row 4 kGR wave + kGR sub of the column's 128: 16-byte chunk, place in it
      const int row = wave * 4 * kGR + sub * kGR;
      uint8_t* at = &codes[m][(l16 * 8 + k) * 128 + (((row >> 4) ^ (l16 & 7)) << 4) + (row & 15)];
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      if constexpr (kGR == 4) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
        if (!(r[k] > 0.0f)) w = (int)pack4_sat_nan(q[0], q[1], q[2], q[3]);   // an infinite or NaN scale
        *reinterpret_cast<uint32_t*>(at) = (uint32_t)w;
      } else {
        if (!(r[k] > 0.0f)) w = (int)pack4_sat_nan(q[0], q[1], 0.f, 0.f);
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < kSets; ++n) {
    const int m = first + n;
    if (p.qt == nullptr || m == 2) break;
#pragma unroll
    for (int i = 0; i < 1024 / kGB; ++i) {
      const int at = i * kGB + threadIdx.x, c = at >> 3, ch = at & 7;
      const gv4i v = *reinterpret_cast<const gv4i*>(&codes[n][c * 128 + ((ch ^ ((c >> 3) & 7)) << 4)]);
      __builtin_nontemporal_store(v, reinterpret_cast<gv4i*>(p.qt + (m * p.I + cb * 128 + c) * p.ldqt + rb * 128 + ch * 16));
    }
  }
  if (kH && (!kOne || first == 2)) {
    // operand tiles: 16 columns x 128 tokens are 2 KB, lane 16 g + c of half h: tokens 64 h + 16 g ..
#pragma unroll
    for (int i = 0; i < 1024 / kGB; ++i) {
      const int at = i * kGB + threadIdx.x, c = (at >> 7) * 16 + (at & 15), ch = (at >> 4) & 7;
      const gv4i v = *reinterpret_cast<const gv4i*>(&codes[kSets - 1][c * 128 + ((ch ^ ((c >> 3) & 7)) << 4)]);
      uint8_t* tile = p.ht + ((cb * 8 + (at >> 7)) * nrb + rb) * 2048;
      __builtin_nontemporal_store(v, reinterpret_cast<gv4i*>(tile + (at & 127) * 16));
    }
  }
}

}  // namespace

int gated_few_cuts(int64_t M, int64_t N, int64_t K, bool fp32) { return gated_cuts(M, N, K, fp32); }
int64_t gated_few_parts(int64_t M, int64_t N, int64_t K, bool fp32, bool codes) { return gated_parts(M, N, K, fp32, codes); }

hipError_t launch_gated_few(const GatedFewProblem& p, hipStream_t stream) {
  hipError_t e;
  if (by_rows(p.M, p.N)) {
    e = p.N <= 4096 ? row<1, 2>(p, stream) : row<2, 1>(p, stream);     // one workgroup for each of the 256 CUs
  } else if (p.M <= 16) {
    e = few_tokens<1, true>(p, stream);
  } else {
    e = p.M <= 32 ? few_tokens<2>(p, stream) : p.M <= 48 ? few_tokens<3>(p, stream) : few_tokens<4>(p, stream);
  }
  if (e != hipSuccess) return e;
  // sums of cut tiles; codes of tiles that no workgroup has whole
  if (p.cuts > 1 || (p.gated.q != nullptr && !has_whole_tiles(p))) {
    const int64_t groups = (int64_t)p.M * (p.N / 128);
    hipLaunchKernelGGL(gated_finish_kernel, dim3((unsigned)((groups + 15) / 16)), dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_gated_backward(const GatedGradProblem& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.T + 127) / 128 * (p.I / 128)));
  // few blocks: a workgroup for each of da, du and h, which reads what it needs by itself
  // (1333 x 1408, 121 blocks: 12.0 to 10.2 us, with h 13.0 to 12.5; 100 x 512, 4: 9.8 to 7.3;
  // 2048 x 1408, 176: 12.7 to 13.1, with h 13.4 to 16.4)
  if (grid.x <= 128) hipLaunchKernelGGL((gated_backward_kernel<true, 2, 4, true>), dim3(grid.x, p.ht != nullptr ? 3 : 2), dim3(1024), 0, stream, p);
  else if (p.ht != nullptr) hipLaunchKernelGGL((gated_backward_kernel<true, 2, 4>), grid, dim3(1024), 0, stream, p);
  else hipLaunchKernelGGL((gated_backward_kernel<false, 4, 4>), grid, dim3(512), 0, stream, p);
  return hipGetLastError();
}

}  // namespace fp8bs
